"""The grouped-query layer's calls on a machine without a GPU: sizes, defaults,
the rotation's table, and the refusals that come before any launch."""
import ctypes
import math

import pytest

FAKE, ODD = 0x10000, 0x10002  # never dereferenced: every call below is refused or has nothing to do


@pytest.fixture(scope="module")
def csa():
    import __graft_entry__
    __graft_entry__._load_builder().build()
    import compressed_sparse_attention_02_gb300 as m
    return m


def cache(csa, **kw):
    f = dict(n_kv_heads=2, head_dim=128, page_size=64, n_pages=10, k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE,
             table=FAKE, table_stride=4)
    f.update(kw)
    return csa.CsaPagedCache(**f)


def test_structs_and_defaults(csa):
    assert ctypes.sizeof(csa.CsaRopeParams) == 40 and ctypes.sizeof(csa.CsaPagedCache) == 72
    r = csa.rope_params()
    assert (r.rope_dim, r.offset, r.layout, r.scaling, r.theta, r.mscale) == (128, 0, 1, 0, 1e4, 1.0)
    with pytest.raises(csa.CsaError):
        csa.rope_params(dim=64)


def test_rope_table(csa):
    buf = (ctypes.c_uint64 * 64)()
    f = csa._lib.csa_rope_table
    assert f(ctypes.byref(csa.rope_params()), ctypes.addressof(buf)) == 0
    for j in (0, 1, 31, 63):
        assert abs(buf[j] / 2.0 ** 64 - 1e4 ** (-j / 64) / (2 * math.pi)) < 1e-15
    for kw, want in ((dict(rope_dim=8), 2), (dict(rope_dim=40), 2), (dict(rope_dim=528), 2), (dict(offset=8), 2),
                     (dict(offset=-16), 2), (dict(layout=2), 1), (dict(scaling=3), 1), (dict(theta=0.5), 1),
                     (dict(theta=math.nan), 1), (dict(mscale=math.inf), 1), (dict(scaling=1, factor=0.5), 1),
                     (dict(scaling=1, factor=math.nan), 1), (dict(scaling=2, factor=2.0, orig_len=0), 1),
                     (dict(scaling=2, factor=2.0, theta=1.0), 1), (dict(scaling=2, beta_fast=1.0, beta_slow=1.0), 1),
                     (dict(scaling=2, beta_slow=0.0), 1)):
        assert f(ctypes.byref(csa.rope_params(**kw)), ctypes.addressof(buf)) == want, kw
    assert f(None, ctypes.addressof(buf)) == 1 and f(ctypes.byref(csa.rope_params()), None) == 1


def test_rope_refusals(csa):
    def call(r=None, turns=FAKE, rows=4, heads=2, dim=128, pos=FAKE, x=FAKE, xs=256, xh=128, y=FAKE + 4096, ys=256,
             yh=128, inverse=0):
        return csa._lib.csa_rope(ctypes.byref(r or csa.rope_params()), turns, rows, heads, dim, pos, x, xs, xh, y, ys,
                                 yh, inverse, None)
    for kw in (dict(turns=None), dict(turns=FAKE + 4), dict(pos=None), dict(pos=ODD), dict(x=None), dict(x=FAKE + 8),
               dict(y=None), dict(y=FAKE + 8), dict(rows=-1), dict(rows=1 << 31), dict(heads=-1), dict(heads=2000),
               dict(xs=100), dict(xh=64), dict(xs=260), dict(yh=132), dict(ys=0), dict(inverse=2),
               dict(y=FAKE, ys=512), dict(dim=64), dict(r=csa.rope_params(offset=16))):
        assert call(**kw) == 1, kw
    assert call(dim=136, xh=136, yh=136, xs=272, ys=272) == 2
    assert call(dim=528) == 2
    assert call(rows=0, x=None, y=None) == 0 and call(heads=0) == 0


def test_append_refusals(csa):
    def call(c=None, r=None, turns=FAKE, B=2, rows=2, cu=None, pos=FAKE, k=FAKE, ks=256, kh=128, v=FAKE, vs=256,
             vh=128):
        return csa._lib.csa_kv_append(ctypes.byref(c or cache(csa)), None if r is None else ctypes.byref(r), turns, B,
                                      rows, cu, pos, k, ks, kh, v, vs, vh, None)
    for kw in (dict(n_kv_heads=0), dict(n_pages=0), dict(n_pages=1 << 31), dict(k=None), dict(v=ODD),
               dict(k_scale=None), dict(v_scale=ODD), dict(table=None), dict(table_stride=0),
               dict(table_stride=(1 << 24) + 1)):
        assert call(cache(csa, **kw)) == 1, kw
    for kw in (dict(head_dim=96), dict(head_dim=256), dict(page_size=8), dict(page_size=48), dict(page_size=256)):
        assert call(cache(csa, **kw)) == 2, kw
    for kw in (dict(B=-1), dict(rows=3), dict(rows=-1), dict(cu=ODD), dict(pos=None), dict(k=None), dict(k=FAKE + 8),
               dict(v=None), dict(ks=64), dict(kh=130), dict(vh=0), dict(r=csa.rope_params(), turns=None),
               dict(r=csa.rope_params(rope_dim=128, offset=16))):
        assert call(**kw) == 1, kw
    assert call(B=0, rows=0, pos=None, k=None, v=None) == 0
    assert call(cu=FAKE, rows=0) == 0


def test_paged_attention_refusals(csa):
    def call(c=None, B=2, heads=4, lens=FAKE, q=FAKE, qs=512, qh=128, sm=0.1, window=0, sink=None, out=FAKE, lse=None,
             ws=FAKE, size=1 << 40):
        return csa._lib.csa_paged_attn(ctypes.byref(c or cache(csa)), B, heads, lens, q, qs, qh, sm, window, sink, out,
                                       lse, ws, size, None)
    for kw in (dict(B=-1), dict(heads=0), dict(heads=3), dict(heads=2048), dict(lens=None), dict(lens=ODD),
               dict(q=None), dict(q=FAKE + 4), dict(qs=64), dict(qh=129), dict(sm=0.0), dict(sm=-1.0),
               dict(sm=math.inf), dict(sm=math.nan), dict(window=-1), dict(sink=ODD), dict(out=None),
               dict(out=FAKE + 8), dict(lse=ODD), dict(c=cache(csa, table=None))):
        assert call(**kw) == 1, kw
    assert call(c=cache(csa, head_dim=32)) == 2
    assert call(B=0, lens=None, q=None, out=None, ws=None, size=0) == 0
    size = csa._lib.csa_paged_attn_workspace_size
    assert size(ctypes.byref(cache(csa, head_dim=80)), 1, 4) == 0
    assert size(ctypes.byref(cache(csa)), 1, 5) == 0 and size(None, 1, 4) == 0
    assert size(ctypes.byref(cache(csa)), -1, 4) == 0


def test_prompt_attention_refusals(csa):
    def call(B=1, heads=4, kv=2, dim=128, nq=8, nk=8, cu_q=FAKE, cu_k=FAKE, q=FAKE, qs=512, qh=128, k=FAKE, ks=256,
             kh=128, v=FAKE, vs=256, vh=128, sm=0.1, causal=1, window=0, sink=None, out=FAKE, lse=None):
        return csa._lib.csa_prompt_attn(B, heads, kv, dim, nq, nk, cu_q, cu_k, q, qs, qh, k, ks, kh, v, vs, vh, sm,
                                        causal, window, sink, out, lse, None)
    for kw in (dict(B=-1), dict(heads=3), dict(heads=0), dict(kv=0), dict(heads=2048), dict(nq=-1), dict(nk=-1),
               dict(nq=(1 << 27) + 1), dict(nk=(1 << 27) + 1), dict(cu_q=None), dict(cu_k=ODD), dict(q=None), dict(k=None), dict(v=FAKE + 8),
               dict(qs=64), dict(kh=100), dict(vs=257), dict(sm=0.0), dict(sm=math.nan), dict(causal=2),
               dict(window=-1), dict(window=5, causal=0), dict(sink=ODD), dict(out=FAKE + 2), dict(out=None),
               dict(lse=ODD), dict(ks=1 << 39)):
        assert call(**kw) == 1, kw
    for d in (32, 96, 256):
        assert call(dim=d) == 2
    assert call(heads=1024, kv=1, nq=1 << 27) == 2
    assert call(nq=0, q=None, out=None) == 0 and call(B=0) == 0


def test_tensors_of_another_kind_are_refused(csa):
    """The binding's own checks, with host tensors (no call may take one)."""
    import torch
    r = csa.rope_params()
    x = torch.zeros(2, 3, 128, dtype=torch.bfloat16)
    for f in (lambda: csa.csa_rope(r, torch.zeros(64, dtype=torch.int64), torch.zeros(2, dtype=torch.int32), x, x),
              lambda: csa.paged_cache(x, x, x, x, x),
              lambda: csa.csa_prompt_attn(x, x, x, x, x, 0.1, True, 0, None, x)):
        with pytest.raises(csa.CsaError) as e:
            f()
        assert e.value.status == 1


def test_more_sequences_than_a_call_takes(csa):
    many, one, c = (1 << 20) + 1, ctypes.c_void_p(None), cache(csa)
    assert csa._lib.csa_kv_append(ctypes.byref(c), None, None, many, many, None, FAKE, FAKE, 256, 128, FAKE, 256, 128,
                                  one) == 1
    assert csa._lib.csa_paged_attn(ctypes.byref(c), many, 4, FAKE, FAKE, 512, 128, 0.1, 0, None, FAKE, None, FAKE,
                                   1 << 40, one) == 1
    assert csa._lib.csa_prompt_attn(many, 4, 2, 128, 8, 8, FAKE, FAKE, FAKE, 512, 128, FAKE, 256, 128, FAKE, 256, 128,
                                    0.1, 1, 0, None, FAKE, None, one) == 1
