"""The paged cache's further calls on a machine without a GPU: structs, sizes
and the refusals that come before any launch."""
import ctypes

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


def book(csa, **kw):
    f = dict(n_seqs=3, page_size=64, n_pages=10, table=FAKE, table_stride=4, lens=FAKE, refs=FAKE)
    f.update(kw)
    return csa.CsaPageBook(**f)


def test_chunk_attention_refusals(csa):
    def call(c=None, B=2, heads=4, nq=8, cu=FAKE, lens=FAKE, q=FAKE, qs=512, qh=128, sm=0.1, window=0, sink=None,
             out=FAKE, lse=None, ws=FAKE, size=1 << 40):
        return csa._lib.csa_chunk_attn(ctypes.byref(c or cache(csa)), B, heads, nq, cu, lens, q, qs, qh, sm, window,
                                       sink, out, lse, ws, size, None)
    for kw in (dict(B=-1), dict(B=(1 << 20) + 1), dict(heads=0), dict(heads=3), dict(heads=2048), dict(nq=-1),
               dict(nq=(1 << 27) + 1), dict(cu=None), dict(cu=ODD), dict(lens=None), dict(lens=ODD), dict(q=None),
               dict(q=FAKE + 4), dict(qs=64), dict(qh=129), dict(qs=1 << 39), dict(sm=0.0), dict(sm=-1.0),
               dict(sm=float("inf")), dict(sm=float("nan")), dict(window=-1), dict(sink=ODD), dict(out=None),
               dict(out=FAKE + 8), dict(lse=ODD), dict(c=cache(csa, table=None)), dict(c=cache(csa, n_pages=0)),
               dict(c=cache(csa, k=ODD)), dict(c=cache(csa, v_scale=None))):
        assert call(**kw) == 1, kw
    assert call(c=cache(csa, head_dim=32)) == 2 and call(c=cache(csa, page_size=256)) == 2
    assert call(c=cache(csa, n_kv_heads=1), heads=64, nq=1 << 25) == 2
    assert call(B=0, cu=None, lens=None, q=None, out=None, ws=None, size=0) == 0
    assert call(nq=0, q=None, out=None, ws=None, size=0) == 0
    assert csa._lib.csa_chunk_attn(None, 1, 4, 1, FAKE, FAKE, FAKE, 512, 128, 0.1, 0, None, FAKE, None, FAKE, 1 << 40,
                                   None) == 1
    size = csa._lib.csa_chunk_attn_workspace_size
    assert size(ctypes.byref(cache(csa, head_dim=80)), 4) == 0 and size(None, 4) == 0
    assert size(ctypes.byref(cache(csa)), 5) == 0 and size(ctypes.byref(cache(csa)), 0) == 0


def test_page_books(csa):
    assert ctypes.sizeof(csa.CsaPageBook) == 48
    size = csa._lib.csa_pages_workspace_size
    assert size(ctypes.byref(book(csa))) > 0 and size(None) == 0
    # a bit and a number a page, and some words a sequence: it may not depend on the arrays
    assert size(ctypes.byref(book(csa, table=None, lens=None, refs=None))) == size(ctypes.byref(book(csa)))
    big = book(csa, n_seqs=1 << 20, n_pages=0x7fffffff)
    assert size(ctypes.byref(big)) >= 0x7fffffff * 4 + 0x7fffffff // 8 + (1 << 20) * 12
    for kw in (dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(n_seqs=-1), dict(n_seqs=(1 << 20) + 1),
               dict(n_pages=0), dict(n_pages=1 << 31)):
        assert size(ctypes.byref(book(csa, **kw))) == 0, kw


def test_pages_refusals(csa):
    L, big = csa._lib, 1 << 40

    def resize(k=None, target=FAKE, pos0=None, src=None, dst=None, ws=FAKE, size=big):
        return L.csa_pages_resize(ctypes.byref(k or book(csa)), target, pos0, src, dst, ws, size, None)

    def fork(k=None, parent=FAKE, src=FAKE, dst=FAKE, ws=FAKE, size=big):
        return L.csa_pages_fork(ctypes.byref(k or book(csa)), parent, src, dst, ws, size, None)

    def compact(k=None, src=FAKE, dst=FAKE, used=FAKE, table=FAKE, refs=FAKE, ws=FAKE, size=big):
        return L.csa_pages_compact(ctypes.byref(k or book(csa)), src, dst, used, table, refs, ws, size, None)

    for f in (resize, fork, compact):
        for kw in (dict(n_seqs=-1), dict(n_pages=0), dict(n_pages=1 << 31), dict(table=None), dict(table=ODD),
                   dict(table_stride=0), dict(table_stride=(1 << 24) + 1), dict(lens=None), dict(lens=ODD),
                   dict(refs=None), dict(refs=ODD)):
            assert f(book(csa, **kw)) == 1, (f, kw)
        assert f(book(csa, page_size=96)) == 2
        assert f(ws=None) == 6 and f(ws=FAKE + 8) == 6 and f(size=100) == 6
    for kw in (dict(target=None), dict(target=ODD), dict(pos0=ODD), dict(src=FAKE), dict(dst=FAKE),
               dict(src=ODD, dst=FAKE), dict(src=FAKE, dst=ODD)):
        assert resize(**kw) == 1, kw
    for kw in (dict(parent=None), dict(parent=ODD), dict(src=None), dict(dst=None), dict(src=ODD), dict(dst=ODD)):
        assert fork(**kw) == 1, kw
    for kw in (dict(src=None), dict(dst=ODD), dict(used=None), dict(used=ODD), dict(table=None), dict(table=ODD),
               dict(refs=None), dict(refs=ODD)):
        assert compact(**kw) == 1, kw
    none = book(csa, n_seqs=0, table=None, lens=None)
    assert resize(none, ws=None) == 0 and fork(none, ws=None) == 0
    for f in (L.csa_pages_resize, L.csa_pages_fork, L.csa_pages_compact):
        assert f(None, *[FAKE] * (len(f.argtypes) - 3), big, None) == 1


def test_copy_refusals(csa):
    def call(c=None, n=2, src=FAKE, dst=FAKE):
        return csa._lib.csa_pages_copy(ctypes.byref(c or cache(csa)), n, src, dst, None)
    for kw in (dict(n=-1), dict(n=1 << 31), dict(src=None), dict(src=ODD), dict(dst=None), dict(dst=ODD),
               dict(c=cache(csa, k=None)), dict(c=cache(csa, v=ODD)), dict(c=cache(csa, k_scale=None)),
               dict(c=cache(csa, n_pages=0)), dict(c=cache(csa, n_kv_heads=0))):
        assert call(**kw) == 1, kw
    assert call(c=cache(csa, head_dim=256)) == 2 and call(c=cache(csa, page_size=4)) == 2
    assert call(n=0, src=None, dst=None) == 0
    assert call(c=cache(csa, table=None, table_stride=0), n=0) == 0
    assert csa._lib.csa_pages_copy(None, 1, FAKE, FAKE, None) == 1


def test_tensors_of_another_kind_are_refused(csa):
    """The binding's own checks, with host tensors and with none."""
    import torch
    x = torch.zeros(3, dtype=torch.int32)
    c = csa.CsaPagedCache(2, 128, 64, 10)
    c.n_seqs, c.device = 3, 0
    k = csa.CsaPageBook(3, 64, 10)
    k.device = 0
    q = torch.zeros(4, 4, 128, dtype=torch.bfloat16)
    for f in (lambda: csa.page_book(torch.zeros(3, 4, dtype=torch.int32), x, x, 64),
              lambda: csa.page_book(x, x, x, 64), lambda: csa.page_book(None, None, None, 64),
              lambda: csa.csa_chunk_attn(c, x, x, q, 0.1, 0, None, q, None, None),
              lambda: csa.csa_chunk_attn(c, None, None, None, 0.1, 0, None, None, None, None)):
        with pytest.raises(csa.CsaError) as e:
            f()
        assert e.value.status == 1
