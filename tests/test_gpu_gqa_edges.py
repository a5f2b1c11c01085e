"""The grouped-query calls at the edges of what they document: values that lie
far apart, what a row does not see, offsets that are wrong."""
import numpy as np
import pytest
import torch

import _gqa as ref
import test_gpu_kv_append as append
import test_gpu_paged_attn as paged
import test_gpu_prompt_attn as prompt

pytestmark = pytest.mark.gpu
DEV = "cuda"
LN2 = 0.6931471805599453


@pytest.fixture(scope="module")
def csa():
    import compressed_sparse_attention_02_gb300 as m
    return m


# ---- csa_paged_attn: logits and value scales far apart ---------------------------------

def far_apart(L, B, Hq, Hkv, D, P, place):
    """Sequences of L tokens with logits of about a binary order around 0, but for one page of each, whose logits
    will be the queries' channel 0 (in binary orders)."""
    x = paged.make([L] * B, Hq, Hkv, D, P, seed=D + P, scales=(0, 1))
    page = x["table"][:, {"first": 0, "middle": L // P // 2, "last": (L - 1) // P}[place]].long()
    x["q"][..., 1:] *= 2.0 ** -6
    k = x["k"].float()
    written = ~k.isnan()
    k[..., 0] = 0.0
    k[page, :, :, 0] = 1.0
    k[~written] = float("nan")
    x["k"] = k.to(torch.float8_e4m3fn)
    x["ks"][page] = 1.0
    return x, page


def sample(x, csa, sm, sequences, **kw):
    """The call on all sequences, checked on some."""
    out, lse = paged.run(csa, x, sm=sm, **kw)
    kw.pop("ws", None)
    y = dict(x, q=x["q"][sequences], lens=x["lens"][sequences], table=x["table"][sequences])
    ref.check_attention(out[sequences], lse[sequences], *paged.want(y, sm=sm, **kw), paged.STEP, "far apart")


@pytest.mark.parametrize("place", ["first", "middle", "last"])
@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("B,Hq,Hkv,D,L", [
    (1, 2, 1, 128, 3000), (1, 3, 1, 64, 3000),      # one pair: sixteen warps join its parts
    (50, 1, 1, 128, 250), (70, 1, 1, 64, 250),      # some pairs: eight do
    (60, 4, 4, 128, 250), (60, 4, 4, 64, 250),      # many pairs, each of several parts
    (300, 16, 8, 128, 120), (300, 16, 8, 64, 120),  # ... and many of one part
    (40, 16, 1, 128, 250),                          # groups of more than eight heads
])
def test_paged_attn_of_logits_and_scales_far_apart(csa, B, Hq, Hkv, D, L, P, place):
    """A page whose logits stand 50 to 150 binary orders above all others: with values of zero (the append gives
    such a page the scale 2^-126) or ordinary ones, beside values of ordinary size and of 2^119."""
    x, page = far_apart(L, B, Hq, Hkv, D, P, place)
    codes, scales = x["v"].view(torch.uint8).clone(), x["vs"].clone()
    some = torch.tensor(sorted({0, B // 2, B - 1}), device=DEV)
    for orders in (50, 100, 116, 120, 127, 150):
        x["q"][..., 0] = orders
        for others in (-6, 119):
            for top in (None, 0, -126):
                x["v"].view(torch.uint8).copy_(codes)
                x["vs"].copy_(scales * 2.0 ** others)
                x["vs"][page] = 2.0 ** (-126 if top is None else top)
                if top is None:  # (what lies behind the sequence's end stays NaN)
                    at = x["v"].view(torch.uint8)[page]
                    x["v"].view(torch.uint8)[page] = torch.where(at == 0x7F, at, 0)
                sample(x, csa, LN2, some, sink=others == 119 and orders == 100)
    # one query head after the other far from the page's keys, and a window's border inside its tile
    x["q"][..., 0] = torch.tensor([0, 150, 60, 120], device=DEV).repeat(Hq)[:Hq].bfloat16()
    sample(x, csa, LN2, some, window=L - 5)
    assert csa.csa_check_status() == 0


def test_paged_attn_of_what_the_append_stored(csa):
    """Tokens appended one page after the other, one page's values all zero and its keys far above the others'."""
    H, D, P, T = 2, 128, 16, 80
    k, v = (torch.zeros(8, H, P, D, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(8, H, device=DEV) for _ in range(2))
    table = torch.arange(8, dtype=torch.int32, device=DEV)[None]
    cache = csa.paged_cache(k, v, ks, vs, table)
    g = torch.Generator(DEV).manual_seed(0)
    a, c = (torch.randn(T, H, D, device=DEV, generator=g).bfloat16() for _ in range(2))
    a[:, :, 0] = 0
    a[32:48, :, 0], c[32:48] = 8.0, 0.0
    csa.csa_kv_append(cache, None, None, torch.tensor([0, T], dtype=torch.int32, device=DEV),
                      torch.zeros(1, dtype=torch.int32, device=DEV), a, c)
    assert (vs[2] == 2.0 ** -126).all()
    q = (torch.randn(1, 8, D, device=DEV, generator=g) * 2.0 ** -6).bfloat16()
    q[..., 0] = 16.0
    x = dict(k=k.view(torch.float8_e4m3fn), v=v.view(torch.float8_e4m3fn), ks=ks, vs=vs, table=table, q=q,
             lens=torch.tensor([T], dtype=torch.int32, device=DEV), sink=None)
    out, lse = paged.run(csa, x, sm=1.0)  # 128 nats, 185 binary orders
    ref.check_attention(out, lse, *paged.want(x, sm=1.0), paged.STEP, "appended")
    assert csa.csa_check_status() == 0


# ---- csa_prompt_attn: what a row does not see ------------------------------------------

@pytest.mark.parametrize("heads", [3, 48])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,window", [([(300, 300), (170, 170)], 0), ([(300, 300), (170, 170)], 150),
                                         ([(40, 700), (30, 900)], 0), ([(2000, 2000), (257, 1900)], 700),
                                         ([(2000, 2000), (257, 2300)], 1500)])
def test_prompt_attn_rows_are_those_of_what_they_see(csa, heads, D, lens, window):
    """Large and infinite keys where a row does not see them, and a neighbour's queries in the rows that its last
    tile leaves empty, change no bit of it."""
    x = prompt.make(lens, heads, 1, D, seed=D + window)
    clean, clean_lse = prompt.run(csa, x, window=window)
    first = 0
    for b, (nq, nk) in enumerate(lens):
        k0 = sum(m for _, m in lens[:b])
        pos = torch.arange(nq) + nk - nq
        for j in (nk - 2, nk - nq // 2, nk - nq + 3, nk - nq - (window or nk) + 1 + nq // 3, 5):
            if not 0 <= j < nk:
                continue
            for value in (3e4, -3e4, float("inf"), float("nan")):
                y = dict(x, k=x["k"].clone())
                y["k"][k0 + j] = torch.where(x["k"][k0 + j] < 0, -value, value).bfloat16()
                out, lse = prompt.run(csa, y, window=window)
                blind = torch.ones(x["q"].shape[0], dtype=torch.bool)
                blind[first:first + nq] = (pos < j) | (pos >= j + (window or nk))
                blind = blind.to(DEV)
                assert torch.equal(out[blind], clean[blind]), (b, j, value)
                assert torch.equal(lse[blind], clean_lse[blind]), (b, j, value)
        for value in (0.0, 1e4, float("inf")):
            y = dict(x, q=x["q"].clone())
            y["q"][first:first + nq] *= value
            out, lse = prompt.run(csa, y, window=window)
            others = torch.ones(x["q"].shape[0], dtype=torch.bool, device=DEV)
            others[first:first + nq] = False
            assert torch.equal(out[others], clean[others]) and torch.equal(lse[others], clean_lse[others])
        first += nq
    assert csa.csa_check_status() == 0

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [2, 48])
def test_prompt_attn_of_a_large_scale(csa, D, heads):
    """sm_scale of 2^28 and 2^60 over rows so small that their logits are ordinary ones: the same bits as with the
    power of two in the queries, rows that see nothing at first or at all among them."""
    lens = [(200, 90), (130, 130), (33, 500), (257, 1900), (40, 0)]
    x = prompt.make(lens, heads, 1, D, seed=D)
    x["sink"][0] = -float("inf")
    for window, sink in ((0, False), (0, True), (129, True)):
        want, want_lse = prompt.run(csa, x, window=window, sink=sink, sm=2.0 ** -3)
        for e in (28, 60):
            y = dict(x, q=x["q"] * 2.0 ** (-3 - e))
            out, lse = prompt.run(csa, y, window=window, sink=sink, sm=2.0 ** e)
            assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert csa.csa_check_status() == 0


# ---- csa_kv_append: pages that another program began -----------------------------------

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows_a_sequence", [1, 14])
def test_append_to_a_scale_that_is_no_power_of_two(csa, D, rows_a_sequence):
    """Codes are those of the quotient in binary32, also where the reciprocal's product is another number."""
    H, P = 2, 16
    n = 896 // D  # rows that hold every bf16 magnitude of seven binary orders, up to 16
    bf = np.float32([m * 2.0 ** e for e in range(-10, -3) for m in range(128, 256)])
    differ = 0
    for scale in map(float.fromhex, ("0x1.cp-4", "0x1.eb851ep-4", "0x1.fca1bp-4", "0x1.fa6f4ep-4", "0x1.f9e79ep-4")):
        s = np.float32(scale)
        quotient, product = (torch.from_numpy(y.astype(np.float64)) for y in (bf / s, bf * (np.float32(1) / s)))
        differ += int((ref.e4m3(quotient) != ref.e4m3(product)).sum())
        want = ref.e4m3(quotient).view(n, 1, D).expand(n, H, D)
        rows = torch.from_numpy(bf).view(n, 1, D).expand(n, H, D).contiguous().to(DEV).bfloat16()
        rows[:, 1] *= -1
        want = torch.stack([want[:, 0], -want[:, 1]], 1)
        B = n if rows_a_sequence == 1 else 1
        k, v, ks, vs, table = append.pool(B, 1, H, D, P)
        ks.fill_(scale), vs.fill_(scale)
        k[:, :, 0], v[:, :, 0] = 0x38, 0x38  # the token that was there: ones
        cu = None if B == n else torch.tensor([0, n], dtype=torch.int32, device=DEV)
        csa.csa_kv_append(csa.paged_cache(k, v, ks, vs, table), None, None, cu,
                          torch.ones(B, dtype=torch.int32, device=DEV), rows, rows)
        for codes, sc in ((k, ks), (v, vs)):
            assert (sc == float(s)).all()
            at = codes[table[:, 0].long()]
            got = at[:, :, 1].contiguous() if B == n else at[0, :, 1:1 + n].transpose(0, 1).contiguous()
            assert torch.equal(append.values(got), want)
            assert (at[:, :, 0] == 0x38).all()
    assert differ > 10
    assert csa.csa_check_status() == 0


@pytest.mark.parametrize("many", [False, True])
def test_append_under_wrong_offsets_and_positions(csa, many):
    """Negative positions store nothing at all; offsets that fall or pass the rows, and tokens past the table, store
    nothing but the other sequences' tokens (a warp a head, and a block a page)."""
    H, D, P, B = 2, 64, 16, 6
    scale = 20 if many else 1
    n = 6 * scale
    a, c = append.rows(n, H, D, 3)
    cu = [0, 3 * scale, 2 * scale, 4 * scale, 9999, 9999, n]  # good: sequences 0 and 2
    k, v, ks, vs, table = append.pool(B, 2, H, D, P)
    g = torch.Generator(DEV).manual_seed(1)
    for x in (k, v):  # every page holds something
        x.copy_(torch.randint(0, 0x7F, x.shape, device=DEV, generator=g, dtype=torch.uint8))
    ks.fill_(2.0 ** -9), vs.fill_(2.0 ** -9)
    cache = csa.paged_cache(k, v, ks, vs, table)
    before = [t.clone() for t in (k, v, ks, vs)]
    cu_t = torch.tensor(cu, dtype=torch.int32, device=DEV)
    csa.csa_kv_append(cache, None, None, cu_t, torch.full((B,), -1, dtype=torch.int32, device=DEV), a, c)
    assert csa.csa_check_status() == 5
    for t, was in zip((k, v, ks, vs), before):
        assert torch.equal(t, was)
    m = append.Model(k, v, ks, vs, table)
    csa.csa_kv_append(cache, None, None, cu_t, torch.full((B,), 2 * P - 1, dtype=torch.int32, device=DEV), a, c)
    assert csa.csa_check_status() == 5
    for b in (0, 2):  # token 31 is the table's last
        r = slice(cu[b], cu[b] + 1)
        m.append(b, 2 * P - 1, {"k": a[r].double().cpu(), "v": c[r].double().cpu()})
    m.check(k, v, ks, vs)
    # pages outside the pool and negative ones, under offsets that are right
    table[0, 0], table[3, 1] = -5, k.shape[0]
    m = append.Model(k, v, ks, vs, table)
    cu = [b * scale for b in range(B + 1)]
    csa.csa_kv_append(cache, None, None, torch.tensor(cu, dtype=torch.int32, device=DEV),
                      torch.full((B,), P - 1, dtype=torch.int32, device=DEV), a, c)
    assert csa.csa_check_status() == 5
    for b in range(B):
        for t in range(scale):
            p, r = P - 1 + t, slice(cu[b] + t, cu[b] + t + 1)
            if p >= 2 * P or not 0 <= int(table[b, p // P]) < k.shape[0]:
                continue
            take = min(scale - t, P - p % P)
            if t and p % P:
                continue  # (stored with its page's first)
            r = slice(cu[b] + t, cu[b] + t + take)
            m.append(b, p, {"k": a[r].double().cpu(), "v": c[r].double().cpu()})
    m.check(k, v, ks, vs)


# ---- offsets that fall far behind, and that overlap ------------------------------------

def test_a_fall_behind_the_last_row_is_reported(csa):
    """Sequences of one row each take as many places as a launch can have; offsets that fall after them (in another
    block of the search) are reported all the same."""
    n, H, D, P = 300, 1, 64, 16
    k, v, ks, vs, table = append.pool(2 * n, 1, H, D, P)
    cache = csa.paged_cache(k, v, ks, vs, table)
    a, c = append.rows(n, H, D, 0)
    for last in ([n] * n, list(range(1, n + 1))):  # no more rows; the same rows again
        for fall in (False, True):
            cu = list(range(n + 1)) + last
            if fall:
                cu[-2] = 7
            elif last[0] != n:
                continue
            csa.csa_kv_append(cache, None, None, torch.tensor(cu, dtype=torch.int32, device=DEV),
                              torch.zeros(2 * n, dtype=torch.int32, device=DEV), a, c)
            assert csa.csa_check_status() == (5 if fall else 0)
    for n, heads, D in ((36, 1, 64), (36, 4, 128), (70, 2, 128), (70, 16, 64)):
        x = prompt.make([(1, 1)] * n, heads, 1, D, seed=n)
        good = prompt.run(csa, x)[0]
        assert csa.csa_check_status() == 0
        more = torch.full((41,), n, dtype=torch.int32, device=DEV)
        for fall in (False, True):
            cu = torch.cat([x["cu_q"], more])
            if fall:
                cu[-2] = 7
            y = dict(x, cu_q=cu, cu_k=torch.cat([x["cu_k"], more]))
            assert torch.equal(prompt.run(csa, y)[0][:7], good[:7])  # (the rows behind may be the overlapping ones' too)
            assert csa.csa_check_status() == (5 if fall else 0)


def test_prompt_attn_of_offsets_that_overlap_a_million_times(csa):
    """Sequences that all begin at row 0 again: the call does no more work than one of as many rows could ask for
    (the items of all of them would pass 32 bits), stays inside its rows and reports the falls."""
    B, n = 1 << 20, 1 << 20
    cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    cu[1::2] = n
    for D, heads in ((64, 1), (128, 1)):
        wide = torch.full((n + 512, heads, D), 3.0, dtype=torch.bfloat16, device=DEV)
        q = wide[256:-256]
        k = torch.zeros(256, 1, D, dtype=torch.bfloat16, device=DEV)
        for keys in (0, 256):
            cu_k = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
            cu_k[1::2] = keys
            out = torch.full_like(wide, 3.0)
            csa.csa_prompt_attn(cu, cu_k, q, k, k, 0.1, keys == 0, 0, None, out[256:-256])
            assert csa.csa_check_status() == 5
            assert (out[:256] == 3).all() and (out[-256:] == 3).all()
            assert (out[256:-256] == 0).all()


# ---- csa_rope on the compressed layer's rows --------------------------------------------

def test_rope_turns_the_compressed_layers_queries(csa):
    """The rotation that the layer calls expect their queries to have (the last 64 of 512 channels, interleaved
    pairs), and the one that inverse_rope takes back: csa_rope gives both, over the library's own oracle.

    The tolerance: an angle is right to 8e-8 rad and the polynomials to 2e-9, their steps' roundings stay below 2^-23,
    and a channel is two products and a sum of 2^-24 each: below 2^-21 of its pair, and one rounding to bf16."""
    import oracle
    T, H, D, R = 24, 64, 512, 64
    r = csa.rope_params(rope_dim=R, offset=D - R, layout=csa.CSA_ROPE_INTERLEAVED, theta=1e4)
    turns = csa.rope_table(r)
    g = torch.Generator(DEV).manual_seed(0)
    x = torch.randn(T, H, D, device=DEV, generator=g).bfloat16()
    pos = torch.randint(0, 1 << 18, (T,), device=DEV, generator=g, dtype=torch.int32)
    for inverse in (False, True):
        got = csa.csa_rope(r, turns, pos, x, inverse=inverse).double().cpu()
        rows = x.double().cpu().numpy()
        want = np.stack([oracle.inverse_rope(rows[t], int(pos[t]), rope_dim=R) if inverse else
                         np.stack([oracle.rope(h, R, 1e4, int(pos[t])) for h in rows[t]]) for t in range(T)])
        want = torch.from_numpy(want)
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -21 * ref.pair_size(r, x)
        assert ((got - want).abs() <= tol).all()
        assert torch.equal(got[..., :D - R], x[..., :D - R].double().cpu())
    assert csa.csa_check_status() == 0


# ---- arguments that are no tensors ------------------------------------------------------

def test_what_is_no_tensor_is_refused(csa):
    """Every tensor argument as None or a list: CSA_ERR_INVALID_ARG, as for one of another type."""
    x = paged.make([40, 9], 4, 2, 64, 16)
    cache = csa.paged_cache(x["k"], x["v"], x["ks"], x["vs"], x["table"])
    r = csa.rope_params(rope_dim=64)
    turns, pos = csa.rope_table(r), torch.zeros(2, dtype=torch.int32, device=DEV)
    kv, out = x["q"][:, :2].contiguous(), torch.empty_like(x["q"])
    y = prompt.make([(5, 5)], 4, 2, 64)
    calls = (
        (csa.paged_cache, dict(k=x["k"], v=x["v"], k_scale=x["ks"], v_scale=x["vs"], table=x["table"]), ()),
        (csa.csa_rope, dict(r=r, turns=turns, pos=pos, x=x["q"], out=out), ("r", "out")),
        (csa.csa_kv_append, dict(cache=cache, r=r, turns=turns, cu_rows=None, pos0=pos, k=kv, v=kv),
         ("cache", "r", "cu_rows")),
        (csa.csa_paged_attn, dict(cache=cache, lens=x["lens"], q=x["q"], sm_scale=0.1, window=0, sink=None, out=out,
                                  lse=None, ws=csa.paged_attn_workspace(cache, 2, 4)),
         ("cache", "sm_scale", "window", "sink", "lse", "ws")),
        (csa.csa_prompt_attn, dict(cu_q=y["cu_q"], cu_k=y["cu_k"], q=y["q"], k=y["k"], v=y["v"], sm_scale=0.1,
                                   causal=True, window=0, sink=None, out=torch.empty_like(y["q"])),
         ("sm_scale", "causal", "window", "sink")))
    for call, args, free in calls:
        call(**args)
        for name in args:
            for bad in ([1.0, 2.0],) if name in ("sink", "lse", "ws", "cu_rows") else (None, [1.0, 2.0]):
                if name in free and name not in ("sink", "lse", "ws", "cu_rows"):
                    continue
                with pytest.raises(csa.CsaError) as e:
                    call(**dict(args, **{name: bad}))
                assert e.value.status == 1, (call, name)
