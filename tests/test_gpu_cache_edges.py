"""The grouped-query attention calls and the cache's pages at the edges of what
they take: logits far past what fp32 resolves to one, next to value scales of
any size; logits near -1e30; arrays beside which nothing else may be written."""
import numpy as np
import pytest
import torch

import _gqa as ref
import test_gpu_chunk_attn as chunk
import test_gpu_paged_attn as paged
import test_gpu_pages as pages
import test_gpu_prompt_attn as prompt

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def csa():
    import compressed_sparse_attention_02_gb300 as m
    return m


# ---- large logits ----------------------------------------------------------------------

# Heads' logits are 2^(a - 3) times 1 or 2, or times -1 or -1/2.  From the second head on a
# row's largest logit stands 2^9 and more above its other ones, whose weights are then 0 in
# 64 bits as in 32, and keys of equal logits have equal ones in fp32 too: their products are
# the same.  So no error of a logit has a part in the result, and the tolerance has none for
# it.
POWERS = (3, 13, 20, 25, 29, 31, 63, 99)


def large(seqs, Hkv, D, P, scales, seed, sign):
    """Sequences whose keys have 1 or (one in 37) 2 or 1/2 in the channel that the queries have; pages of value scale 2^e for
    the e of `scales`, or (None) of zeros with the scale 2^-126 that the append gives them."""
    x = chunk.make(seqs, Hkv * len(POWERS), Hkv, D, P, seed=seed)
    g = torch.Generator().manual_seed(seed)
    n = x["k"].shape[0]
    codes = (torch.rand(n, Hkv, P, D, generator=g) * 7 + 1) * (torch.randint(0, 2, (n, Hkv, P, D), generator=g) * 2 - 1)
    written = ~x["v"].float().isnan().cpu()
    e = torch.randint(0, len(scales), (n,), generator=g)
    for i, s in enumerate(scales):
        x["vs"][e == i] = 2.0 ** (-126 if s is None else s)
        if s is None:
            codes[e == i] = 0.0
    x["v"] = codes.where(written, float("nan")).to(torch.float8_e4m3fn).to(DEV)
    k = x["k"].float().cpu()
    k[..., 0] = 1.0
    for b, L in enumerate(x["lens"].tolist()):
        t = torch.arange(5, L, 37)
        k[x["table"][b].cpu().long()[t // P], :, t % P, 0] = 2.0 if sign > 0 else 0.5
    x["k"] = k.where(written, float("nan")).to(torch.float8_e4m3fn).to(DEV)
    x["ks"].fill_(1.0)
    x["q"].zero_()
    x["q"][..., 0] = sign * torch.exp2(torch.tensor(POWERS * Hkv, device=DEV).float())
    return x


def exact(want, x, **kw):
    """`want` without an allowance for logits' errors.  Past 2^53 a logit of 64 bits does not hold its sum's logarithm
    either: such heads' weights are those of 2^29, their lse the largest logit."""
    powers = torch.tensor(POWERS * (x["q"].shape[1] // len(POWERS)))
    less = (powers - 29).clamp(min=0)
    q = (x["q"].double() * torch.exp2(-less.double()).to(DEV)[:, None]).bfloat16()
    out, lse, A, Q = want(dict(x, q=q), sm=0.125, **kw)
    return out, lse * torch.exp2(less.double()), A, Q * (powers == POWERS[0])


SCALES = [(0,), (20,), (-30,), (0, None), (0, 40), (-100, 30), (0, -60, 9), (100, None)]


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("scales", SCALES)
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
def test_chunk_attn_of_large_logits(csa, D, P, scales, sign):
    """In tiles that a share holds whole, some of one block, and in tiles that many shares divide."""
    for seqs, Hkv in (([(2, 300), (40, 130)] * 40 + [(1, 50)] * 60, 2), ([(3, 100), (4, 2500), (40, 2000)], 1)):
        x = large(seqs, Hkv, D, P, scales, 17 + D, sign)
        out, lse = chunk.run(csa, x, sm=0.125)
        n = int(x["cu"][-1])
        rows = list(range(0, n, 1 + n // 30))
        w = exact(chunk.want, x, rows=rows)
        ref.check_attention(out[rows], lse[rows], *w, chunk.STEP, "large logits")
    assert csa.csa_check_status() == 0


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("scales", SCALES)
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
def test_paged_attn_of_large_logits(csa, D, P, scales, sign):
    """The same for single tokens: pairs of a sequence and a key head that one warp has whole, and divided ones, whose
    parts a warp or several join."""
    for lens, Hkv in (([300, 40, 7] * 100, 2), ([250] * 50, 1), ([3000], 1)):
        x = large([(1, L) for L in lens], Hkv, D, P, scales, 29 + D, sign)
        out, lse = paged.run(csa, x, sm=0.125)
        some = list(range(0, len(lens), 1 + len(lens) // 40))
        y = dict(x, q=x["q"][some], lens=x["lens"][some], table=x["table"][some])
        w = exact(paged.want, y)
        ref.check_attention(out[some], lse[some], *w, paged.STEP, "large logits")
    assert csa.csa_check_status() == 0


# ---- logits near the least that the calls take -----------------------------------------

LEAST = -1.5 * 2.0 ** 99               # -9.5e29


def lowest(make, seqs, Hq, D, c):
    """make's book or prompts, every logit LEAST under a scale of 1/8 (from two factors that bf16 and the codes hold)."""
    x = make(seqs, Hq, 1, D, *(() if c == "prompt" else (32,)), seed=D)
    x["q"].zero_()
    if c == "prompt":
        x["q"][..., 0], x["k"][..., 0] = -1.5 * 2.0 ** 51, 2.0 ** 51
    else:
        x["q"][..., 0] = -1.5 * 2.0 ** 102
        k = x["k"].float()
        k[..., 0] = torch.where(k[..., 0].isnan(), k[..., 0], 1.0)
        x["k"] = k.to(torch.float8_e4m3fn)
        x["ks"].fill_(1.0)
    x["sink"] = torch.tensor([LEAST / 2, LEAST * 0.75, LEAST, -3e38], device=DEV)
    return x


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("call", ["chunk", "paged", "prompt"])
def test_lowest_logits(csa, call, D):
    """Rows all of whose logits are -9.5e29 have the mean of what they see, rows that see nothing their sink, however low
    (a sink of -3e38 has no weight beside anything)."""
    seqs = {"chunk": [(3, 100), (140, 400), (2, 0), (3, 1), (2, 5000)], "paged": [100, 0, 1, 5000],
            "prompt": [(3, 100), (140, 400), (2, 0), (3, 1), (300, 300)]}[call]
    of = {"chunk": chunk, "paged": paged, "prompt": prompt}[call]
    x = lowest(of.make, seqs, 4, D, call)
    same = dict(x, q=torch.zeros_like(x["q"]))      # (logits of 0: the same weights)
    want, lse, A, Q = of.want(same, sm=0.125)
    seen = ~torch.isinf(lse)
    lse[seen] = LEAST
    got = of.run(csa, x, sm=0.125)
    ref.check_attention(*got, want, lse, A, Q, of.STEP, "lowest")
    # beside a sink: all of the weight is the higher one's (LEAST itself: whose share is what follows from fp32 products)
    sink = x["sink"].double().cpu()
    got, got_lse = (y.double().cpu() for y in of.run(csa, x, sm=0.125, sink=True))
    for h in range(4):
        s = seen[:, h]
        assert (got[~s, h] == 0).all() and ((got_lse[~s, h] - sink[h]).abs() <= 2.0 ** -20 * sink[h].abs()).all()
        if h < 2:
            assert (got[s, h] == 0).all() and ((got_lse[s, h] - sink[h]).abs() <= 2.0 ** -20 * sink[h].abs()).all()
    s = seen[:, 3]
    ref.check_attention(got[s][:, 3:], got_lse[s][:, 3:], want[s][:, 3:], lse[s][:, 3:], A[s][:, 3:], Q[s][:, 3:], of.STEP,
                        "a sink without weight")
    assert csa.csa_check_status() == 0


# ---- nothing is written outside what a call is given -----------------------------------

GUARD, MARGIN = 0x5A5A5A5A, 256


class Margins:
    """Arrays with filled memory directly before and behind them."""

    def __init__(self):
        self.whole = []

    def take(self, shape, dtype=torch.int32):
        n = -(-torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size() // 16) * 4
        w = torch.full((n + 2 * MARGIN,), GUARD, dtype=torch.int32, device=DEV)
        self.whole.append((w, MARGIN + n))
        x = w[MARGIN:MARGIN + n].view(dtype)
        return x[:torch.Size(shape).numel()].view(shape)

    def like(self, x):
        x = torch.as_tensor(x, dtype=None if torch.is_tensor(x) else torch.int32, device=DEV)
        y = self.take(x.shape, x.dtype)
        y.copy_(x)
        return y

    def check(self):
        for w, end in self.whole:
            assert (w[:MARGIN] == GUARD).all() and (w[end:] == GUARD).all()


def guarded_book(csa, monkeypatch, m, table, lens, refs, page):
    """A book of test_gpu_pages, every array of which, and the workspace, is in margins."""
    monkeypatch.setattr(pages, "i32", lambda x: m.like(torch.tensor(np.asarray(x), dtype=torch.int32)))
    monkeypatch.setattr(pages.Both, "outs", lambda self, n, k: [m.take((k,)).fill_(77) for _ in range(n)])
    x = pages.Both(csa, table, lens, refs, page)
    x.ws = m.take((x.ws.numel(),), torch.uint8).fill_(0xA5)
    return x


def compacted(csa, m, x):
    """Out of place and then in place."""
    src, dst = x.outs(2, len(x.host.refs) // 2)
    used, = x.outs(1, 1)
    csa.csa_pages_compact(x.book, src, dst, used, m.take(x.table.shape), m.take(x.refs.shape), x.ws)
    csa.csa_check_status()
    x.compact(in_place=True)


def test_page_calls_write_in_their_arrays_alone(csa, monkeypatch):
    """Lengths past the table and below 0, entries outside the pool, counts that do not fit, targets past the table,
    parents that are none, pools that run out, tables of one entry."""
    table = np.array([[0, 1, 2], [3, -7, 99], [5, 6, 2 ** 31 - 1], [-1, -1, -1]], np.int32)
    refs = np.array([1, 1, 1, 1, 0, 1, 0, -4], np.int32)
    m = Margins()
    for lens, call in (([100, 40, 48, -3], lambda x: x.resize([48, 41, 2 ** 31 - 1, 17])),
                       ([100, 40, 48, -3], lambda x: x.resize([0, 0, 1, 0])),
                       ([48, 48, 48, 48], lambda x: x.resize([0, 0, 0, 0])),
                       ([2 ** 31 - 1, -2 ** 31, 48, 0], lambda x: x.resize([-2 ** 31, 2 ** 31 - 1, 49, 48])),
                       ([48, 40, 48, -3], lambda x: x.fork([-1, -1, -1, 1])),
                       ([48, 0, 40, 0], lambda x: x.fork([4, 2 ** 31 - 1, -2 ** 31, 2])),
                       ([2 ** 31 - 1, 0, 0, 0], lambda x: x.fork([-1, 0, 0, 3])),
                       ([100, 40, 48, -3], lambda x: compacted(csa, m, x))):
        x = guarded_book(csa, monkeypatch, m, table, lens, refs, 16)
        x.host.refused = max(lens) > 48      # (reported, as the header has it; the host's steps only cut such lengths)
        call(x)
        m.check()
    for pool in (1, 31, 33, 4097):
        x = guarded_book(csa, monkeypatch, m, np.full((5, 1), -1, np.int32), [0] * 5, np.zeros(pool, np.int32), 128)
        x.resize([1, 128, 129, 0, 2 ** 31 - 1])
        x.fork([-1, -1, -1, 0, 0])
        x.resize([0, -1, -1, -1, -1])
        compacted(csa, m, x)
        x.resize([128] * 5)
        compacted(csa, m, x)
        m.check()


def test_page_copies_write_in_their_pages_alone(csa):
    H, P, D, n = 3, 32, 64, 9
    m = Margins()
    g = torch.Generator(DEV).manual_seed(1)
    k, v = (m.like(torch.randint(0, 256, (n, H, P, D), device=DEV, generator=g, dtype=torch.uint8)) for _ in range(2))
    ks, vs = (m.like(torch.rand(n, H, device=DEV, generator=g)) for _ in range(2))
    cache = csa.paged_cache(k, v, ks, vs, m.take((1, 1)))
    before = [x.clone() for x in (k, v, ks, vs)]
    src = m.like([0, 3, -1, 8, 9, 2, 2 ** 31 - 1, -2 ** 31, 5])
    dst = m.like([1, 9, 4, 8, 7, 2 ** 31 - 1, 6, 3, -1])
    csa.csa_pages_copy(cache, src, dst)
    assert csa.csa_check_status() == 5
    for x, y in zip((k, v, ks, vs), before):
        y[1] = y[0]
        assert torch.equal(x, y)
    m.check()


def test_chunk_attn_writes_in_its_outputs_alone(csa):
    """Whole tiles, divided ones and their records, offsets and tables that are wrong among them."""
    for D, seqs in ((64, [(5, 300), (260, 700), (0, 9), (40, 90)]), (128, [(70, 3000), (1, 2000), (3, 5)])):
        x = chunk.make(seqs, 8, 2, D, 32, seed=D)
        n = x["q"].shape[0]
        cache = csa.paged_cache(x["k"], x["v"], x["ks"], x["vs"], x["table"])
        for cu, page, length in (([], None, None), ([(1, 2 ** 31 - 1)], 5, None), ([(2, -2 ** 31), (3, n + 1)], -1, 2 ** 31 - 1),
                                 ([(0, 3), (2, 1)], 2 ** 31 - 1, -2 ** 31)):
            y = dict(x, cu=x["cu"].clone(), table=x["table"].clone(), lens=x["lens"].clone())
            for i, value in cu:
                y["cu"][i] = value
            if page is not None:
                y["table"][0, 1] = page
            if length is not None:
                y["lens"][1] = length
            m = Margins()
            out, lse = m.take((n, 8, D), torch.bfloat16), m.take((n, 8), torch.float32)
            ws = m.take((csa.chunk_attn_workspace(cache, 8).numel(),), torch.uint8)
            bad = csa.paged_cache(x["k"], x["v"], x["ks"], x["vs"], y["table"])
            csa.csa_chunk_attn(bad, y["cu"], y["lens"], x["q"], D ** -0.5, 0, x["sink"], out, lse, ws)
            assert csa.csa_check_status() == (5 if cu else 0)
            m.check()


# ---- a chunk far into a sequence -------------------------------------------------------

def test_chunk_far_into_a_long_sequence(csa):
    """2048 tokens behind 60000 of 32 query heads on 4: rows at the tiles' and the chunk's ends against 64 bits."""
    D, P, n, L, heads = 128, 128, 2048, 62048, (0, 13, 31)
    x = chunk.make([(n, L)], 32, 4, D, P, seed=62)
    rows = [0, 31, 32, 33, 1000, 2015, 2016, 2047]
    out, lse = chunk.run(csa, x)
    assert csa.csa_check_status() == 0
    pages_of = x["table"][0].long()
    for h in heads:
        k, v = ((x[c][pages_of, h // 8].double() * x[c + "s"][pages_of, h // 8].double()[:, None, None])
                .reshape(-1, D)[:L].cpu() for c in "kv")
        q = x["q"][rows, h].double().cpu()
        seen = torch.arange(L) <= torch.tensor(rows)[:, None] + L - n
        want, want_lse, A, Q = ref.attend(q, k, v, D ** -0.5, seen)
        # (what a query's two parts leave out, as test_gpu_chunk_attn.want has it)
        Q += 0.5 * q.abs().amax(1) * k.abs().sum(1).max() * D ** -0.5
        ref.check_attention(out[rows, h], lse[rows, h], want, want_lse, A, Q, chunk.STEP, "far into a sequence")
