"""csa_chunk_attn against attention in 64 bits over the values its codes stand
for.  Weights are rounded to f16 (half a step 2^-11); a query row is held as two
E4M3 parts, which leaves out less than 2^-17 of its largest value."""
import math

import pytest
import torch

import _gqa as ref
import test_gpu_paged_attn as paged

pytestmark = pytest.mark.gpu
DEV = "cuda"
STEP = 2.0 ** -11


@pytest.fixture(scope="module")
def csa():
    import compressed_sparse_attention_02_gb300 as m
    return m


def make(seqs, Hq, Hkv, D, P, seed=0, **kw):
    """seqs: (new tokens, cached tokens with them).  A pool whose unwritten tokens are NaN codes, shuffled pages."""
    x = paged.make([L for _, L in seqs], Hq, Hkv, D, P, seed, **kw)
    g = torch.Generator(DEV).manual_seed(seed + 1)
    n = [q for q, _ in seqs]
    x["q"] = torch.randn(sum(n), Hq, D, device=DEV, generator=g).bfloat16()
    x["cu"] = torch.tensor([0] + n, device=DEV).cumsum(0).int()
    return x


def run(csa, x, window=0, sink=False, lse=True, ws=None, sm=None, q=None, stream=None):
    cache = csa.paged_cache(x["k"], x["v"], x["ks"], x["vs"], x["table"])
    q = x["q"] if q is None else q
    n, Hq, D = q.shape
    out = torch.full((n, Hq, D), 9.0, dtype=torch.bfloat16, device=DEV)
    l = torch.full((n, Hq), 9.0, device=DEV) if lse else None
    csa.csa_chunk_attn(cache, x["cu"], x["lens"], q, D ** -0.5 if sm is None else sm, window,
                       x["sink"] if sink else None, out, l, csa.chunk_attn_workspace(cache, Hq) if ws is None else ws,
                       stream)
    return out, l


def want(x, window=0, sink=False, sm=None, skip=(), rows=None):
    """Oracle results of all rows (or of those listed), [rows][Hq] of each; skip: (sequence, page of its table) left
    out.  What the two parts of a query leave out, 2^-17 of its largest value times the keys' magnitudes, is half of
    what DOT = 2^-16 makes of that product."""
    k, v = (x[c].to(torch.float32).double().cpu() * x[c + "s"].double().cpu()[..., None, None] for c in "kv")
    q, table, cu = x["q"].double().cpu(), x["table"].cpu(), x["cu"].cpu().tolist()
    n, Hq, D = q.shape
    Hkv, P = k.shape[1], k.shape[2]
    sm = D ** -0.5 if sm is None else sm
    rows = list(range(cu[-1])) if rows is None else rows
    res = [torch.zeros(len(rows), Hq, *s, dtype=torch.float64) for s in ((D,), (), (D,), ())]
    for b in range(len(cu) - 1):
        at = [i for i, r in enumerate(rows) if cu[b] <= r < cu[b + 1]]
        if not at:
            continue
        L = min(max(int(x["lens"][b]), 0), table.shape[1] * P)
        pos = torch.tensor([L - (cu[b + 1] - cu[b]) + rows[i] - cu[b] for i in at])[:, None]
        t = torch.arange(L)
        seen = t <= pos
        if window:
            seen &= t > pos - window
        for p in range(-(-L // P)):
            if (b, p) in skip:
                seen[:, p * P:(p + 1) * P] = False
        pages = table[b, :-(-L // P)].long().clamp(0, k.shape[0] - 1)
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            kk, vv = k[pages, hk].reshape(-1, D)[:L], v[pages, hk].reshape(-1, D)[:L]
            qq = q[[rows[i] for i in at], h]
            o, lse, A, Q = ref.attend(qq, kk, vv, sm, seen, float(x["sink"][h]) if sink else None)
            for i in range(len(at)):
                if seen[i].any():
                    Q[i] += 0.5 * qq[i].abs().max() * kk[seen[i]].abs().sum(1).max() * sm
            for r, y in zip(res, (o, lse, A, Q)):
                r[at, h] = y
    return res


def check(csa, x, what, **kw):
    skip, rows = kw.pop("skip", ()), kw.pop("rows", None)
    out, lse = run(csa, x, **kw)
    w = want(x, kw.get("window", 0), kw.get("sink", False), kw.get("sm"), skip, rows)
    if rows is None:
        ref.check_attention(out, lse, *w, STEP, what)
    else:
        ref.check_attention(out[rows], lse[rows], *w, STEP, what)
    return out


LENGTHS = [(1, 1), (0, 40), (1, 0), (5, 3), (2, 2), (16, 16), (17, 17), (1, 128), (1, 129), (31, 33), (33, 127),
           (3, 257), (64, 64), (65, 130), (0, 0), (100, 300), (7, 700)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_lengths_and_pages(csa, D, P):
    x = make(LENGTHS, 8, 2, D, P, seed=D + P)
    check(csa, x, "plain")
    assert csa.csa_check_status() == 0
    check(csa, x, "sink", sink=True)
    assert csa.csa_check_status() == 0


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (6, 2), (14, 2), (12, 1), (16, 1), (40, 1), (32, 8), (5, 5), (200, 1)])
def test_groups(csa, Hq, Hkv):
    """Rows of a tile that are all heads of few queries, and one head of many; tiles that end inside a query."""
    for D in (64, 128):
        check(csa, make([(5, 9), (30, 300), (1, 129), (12, 12)], Hq, Hkv, D, 32, seed=Hq), "group", sink=True)
    assert csa.csa_check_status() == 0


@pytest.mark.parametrize("window", [1, 2, 16, 100, 128, 129, 1000])
def test_windows(csa, window):
    for D, P in ((64, 16), (128, 64)):
        x = make([(1, 1), (40, 100), (5, 128), (130, 130), (3, 257), (150, 1001), (9, 4)], 4, 2, D, P, seed=window)
        check(csa, x, "window", window=window, sink=window % 2 == 0)
        # what the windows of all of a sequence's queries leave out has no effect, whatever it holds
        before = run(csa, x, window=window)
        n = (x["cu"][1:] - x["cu"][:-1]).tolist()
        for b, L in enumerate(x["lens"].tolist()):
            for t in range(max(0, L - n[b] - window + 1)):
                page = int(x["table"][b, t // P])
                for c in "kv":
                    x[c].view(torch.uint8)[page, :, t % P] = 0x7F
        after = run(csa, x, window=window)
        assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    assert csa.csa_check_status() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_keys_of_one_tile_in_many_shares(csa, D):
    """One sequence whose few tiles are cut into a share a CTA, whole and in part under a window; two tiles of 256 rows,
    one of fewer."""
    x = make([(70, 9000)], 8, 1, D, 64, seed=D)
    rows = [0, 1, 15, 16, 31, 32, 47, 68, 69]
    check(csa, x, "shares", rows=rows)
    check(csa, x, "shares under a window", rows=rows, window=3000, sink=True)
    check(csa, make([(3, 20000)], 2, 1, D, 128, seed=D + 1), "few rows")
    assert csa.csa_check_status() == 0


def test_many_sequences_of_mixed_lengths(csa):
    """700 sequences (several passes of the search), shares that cut some and hold several others."""
    g = torch.Generator().manual_seed(2)
    n = torch.randint(0, 4, (700,), generator=g).tolist()
    old = torch.randint(0, 60, (700,), generator=g).tolist()
    seqs = [(a, a + b) for a, b in zip(n, old)]
    seqs[7], seqs[200], seqs[650] = (90, 2000), (1, 1700), (200, 200)
    check(csa, make(seqs, 4, 2, 64, 16, seed=5), "mixed")
    x = make([(0, 5)] * 600 + [(140, 150)] + [(0, 0)] * 600 + [(1, 700)], 3, 1, 128, 32, seed=6)
    check(csa, x, "mostly without queries")
    assert csa.csa_check_status() == 0


def test_prompts_of_several_tiles(csa):
    """Tiles at the start, middle and end of prompts, more than a warp's worth of tiles a sequence."""
    x = make([(1500, 1500), (1100, 2300), (257, 257)], 8, 1, 64, 64, seed=12)
    rows = [0, 1, 31, 32, 33, 700, 1023, 1024, 1498, 1499, 1500, 1531, 1532, 2000, 2599, 2600, 2601, 2700, 2856]
    check(csa, x, "tiles", rows=rows, sink=True)
    check(csa, x, "tiles under a window", rows=rows, window=200)
    assert csa.csa_check_status() == 0


def test_scales_of_any_size(csa):
    """Pages whose scales differ by 2^40, pages of zeros with the smallest scale, a value scale of zero."""
    x = make([(20, 500), (4, 130), (3, 64)], 8, 2, 128, 16, seed=8)
    t = x["table"]
    x["vs"][t[0, 3].long()] *= 2.0 ** 40
    x["vs"][t[0, 9].long()] *= 2.0 ** -30
    for b, p in ((1, 2), (1, 0), (2, 1)):
        page = int(t[b, p])
        for c in "kv":
            x[c].view(torch.uint8)[page] = 0
            x[c + "s"][page] = 2.0 ** -126
    x["vs"][t[2, 2].long()] = 0.0
    check(csa, x, "scales")
    assert csa.csa_check_status() == 0


@pytest.mark.parametrize("place", ["first", "middle", "last"])
@pytest.mark.parametrize("logit,vexp", [(40, 0), (-40, 0), (0, 80), (0, -80), (90, -100), (-90, 100), (120, -126)])
def test_logits_and_value_scales_far_apart(csa, place, logit, vexp):
    """One page's logits are about `logit` binary orders from the others', and its values 2^vexp of theirs: the result is
    finite and right wherever the formula is."""
    D, P, L = 64, 32, 700
    x = make([(6, L), (2, 300)], 2, 1, D, P, seed=31, scales=(0, 1))
    pages = [int(x["table"][b, {"first": 0, "middle": n // P // 2, "last": n // P - 1}[place]])
             for b, n in enumerate((L - 6, 298))]
    x["q"][..., 0] = 1.0
    x["q"][..., 1:] *= 2.0 ** -6
    k = x["k"].float()
    written = ~k.isnan()
    k[..., 0] = 0.0
    for p in pages:
        k[p, :, :, 0] = 1.0 if logit > 0 else -1.0
        x["ks"][p] = max(abs(logit), 1) * math.log(2) / (D ** -0.5)
        k[p, :, :, 1:] = 0.0
        x["vs"][p] = 2.0 ** vexp
    k[~written] = float("nan")
    x["k"] = k.to(torch.float8_e4m3fn)
    check(csa, x, "far apart")
    check(csa, x, "far apart", sink=True)


def test_queries_of_any_size(csa):
    x = make([(3, 200)], 6, 1, 64, 32, seed=9, scales=(-12, -11))
    x["q"][:, 0] = 0
    x["q"][:, 1] *= 2.0 ** 60
    x["q"][:, 1, 1:] *= 2.0 ** -60
    x["q"][:, 2] *= 2.0 ** -100
    x["q"][:, 3] *= 30
    x["q"][:, 4, ::2] *= 2.0 ** -12       # (below what the two parts hold whole)
    x["sink"][1] = -math.inf
    # (row 1: one channel decides, its logits are of 2^60: differences below them do not matter)
    out, lse = run(csa, x, sink=True)
    w = want(x, 0, True)
    rows = [0, 2, 3, 4, 5]
    ref.check_attention(out[:, rows], lse[:, rows], *[y[:, rows] for y in w], STEP, "queries")
    assert torch.isfinite(out).all()


def test_values_that_are_not_finite(csa):
    """NaN codes among keys and values: rows that see them have the formula's NaN, in its channels only, the others
    nothing of them; a query row that is not finite gives NaN, the others of its tile nothing of it."""
    for D, Hq, Hkv, window in ((64, 4, 2, 0), (128, 8, 1, 0), (128, 2, 2, 70), (64, 16, 1, 130)):
        x = make([(40, 300), (140, 141), (2, 150)], Hq, Hkv, D, 32, seed=D)
        for b, t, ch in ((0, 299, 3), (0, 270, 5), (0, 1, 7), (1, 100, D - 1), (1, 0, 0), (2, 149, 20)):
            page = int(x["table"][b, t // 32])
            x["v"].view(torch.uint8)[page, 0, t % 32, ch] = 0xFF if ch % 2 else 0x7F
        page = int(x["table"][1, 120 // 32])
        x["k"].view(torch.uint8)[page, Hkv - 1, 120 % 32, 11] = 0x7F
        check(csa, x, "NaN", window=window)
    x = make([(40, 300)], 4, 2, 64, 32)
    clean, _ = run(csa, x)
    x["q"][7, 1, 3], x["q"][9, 0, 60], x["q"][39, 2, 0] = float("nan"), float("inf"), -float("inf")
    out, lse = run(csa, x)
    for i, h in ((7, 1), (9, 0), (39, 2)):
        assert torch.isnan(out[i, h].float()).all() and torch.isnan(lse[i, h])
        out[i, h] = clean[i, h]
    assert torch.equal(out, clean)


def test_bad_tables_and_lengths(csa):
    x = make([(5, 300), (40, 200), (3, 64), (4, 90)], 4, 2, 64, 32, seed=3)
    x["table"][0, 2] = -1
    x["table"][1, 0] = x["k"].shape[0]
    x["table"][1, 4] = -2 ** 31
    x["lens"][2] = 10 ** 6          # clamped to the table: the NaN codes behind token 64 are then seen
    x["lens"][3] = -5
    out, lse = run(csa, x)
    assert csa.csa_check_status() == 5
    x["lens"][2] = 0
    w = want(x, skip={(0, 2), (1, 0), (1, 4)})
    rows = list(range(45)) + [48, 49, 50, 51]
    ref.check_attention(out[rows], lse[rows], *[y[rows] for y in w], STEP, "bad pages")
    assert torch.isnan(out[45:48].float()).all()
    # a sequence all of whose pages are bad sees nothing
    x["table"][1] = -1
    out, lse = run(csa, x)
    assert csa.csa_check_status() == 5
    assert (out[5:45] == 0).all() and torch.isinf(lse[5:45]).all()
    assert csa.csa_check_status() == 0


def test_wrong_offsets(csa):
    """Entries that fall, are negative or pass the rows: such sequences are left out, others are served, and sequences
    that overlap add no work."""
    x = make([(10, 50), (20, 60), (5, 30), (7, 90)], 4, 2, 64, 16, seed=21)
    good, good_lse = run(csa, x)
    for at, value, gone in ((2, 5, (10, 30)), (2, -4, (10, 35)), (2, 1000, (10, 35)), (0, -1, (0, 10))):
        y = dict(x, cu=x["cu"].clone())
        y["cu"][at] = value
        out, lse = run(csa, y)
        assert csa.csa_check_status() == 5
        served = [r for r in range(42) if not gone[0] <= r < gone[1]]
        if at == 2 and value == 5:  # (the sequence behind then begins inside the first one: any part may be left out)
            served = [r for r in served if r < 10 or r >= 35]
        assert torch.equal(out[served], good[served]) and torch.equal(lse[served], good_lse[served])
    n = 3000
    y = dict(x, cu=torch.tensor([0, 42] * n + [0], dtype=torch.int32, device=DEV),
             lens=torch.full((2 * n,), 60, dtype=torch.int32, device=DEV), table=x["table"][:1].expand(2 * n, -1).contiguous())
    run(csa, y)
    assert csa.csa_check_status() == 5


def test_rows_behind_the_last_sequence(csa):
    x = make([(3, 40), (130, 200), (0, 3)], 4, 1, 128, 16, seed=22)
    want_out, want_lse = run(csa, x)
    wide = torch.full((150, 4, 128), float("nan"), device=DEV).bfloat16()
    wide[:133] = x["q"]
    out, lse = run(csa, x, q=wide)
    assert torch.equal(out[:133], want_out) and torch.equal(lse[:133], want_lse)
    assert (out[133:] == 9).all() and (lse[133:] == 9).all()
    empty = dict(x, cu=torch.zeros(4, dtype=torch.int32, device=DEV))
    out, lse = run(csa, empty, q=wide)
    assert (out == 9).all() and (lse == 9).all()
    assert csa.csa_check_status() == 0


def test_single_tokens_as_the_single_token_call_has_them(csa):
    x = make([(1, 1000), (1, 77), (1, 0), (1, 2500)], 16, 4, 128, 64, seed=4)
    for window, sink in ((0, False), (300, True)):
        out, lse = run(csa, x, window=window, sink=sink)
        other, other_lse = paged.run(csa, x, window=window, sink=sink)
        w = want(x, window, sink)
        ref.check_attention(out, lse, *w, STEP, "chunk")
        ref.check_attention(other, other_lse, *w, STEP, "single")


def test_strided_queries_streams_graphs_and_repeats(csa):
    x = make([(30, 1000), (1, 77), (300, 2500)], 16, 4, 128, 64, seed=4)
    out, lse = run(csa, x)
    for _ in range(3):
        again = run(csa, x)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    wide = torch.randn(331, 24, 128, device=DEV).bfloat16()
    wide[:, 4:20] = x["q"]
    assert torch.equal(out, run(csa, x, q=wide[:, 4:20])[0])
    assert torch.equal(out, run(csa, x, lse=False)[0])
    cache = csa.paged_cache(x["k"], x["v"], x["ks"], x["vs"], x["table"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out2, lse2 = run(csa, x)
    side.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    # two captured calls with a workspace each (kept as long as its graph), replayed on two streams at once
    graphs, kept = [], []
    for _ in range(2):
        ws = csa.chunk_attn_workspace(cache, 16)
        o, l = torch.zeros_like(out), torch.zeros_like(lse)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            csa.csa_chunk_attn(cache, x["cu"], x["lens"], x["q"], 128 ** -0.5, 0, None, o, l, ws)
        graphs.append((gr, o, l))
        kept.append(ws)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for (gr, _, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for _, o, l in graphs:
        assert torch.equal(o, out) and torch.equal(l, lse)
    # other lengths in the same memory: the graph reads them when it runs
    x["lens"].copy_(torch.tensor([10, 0, 2499], dtype=torch.int32))
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], run(csa, x)[0])
    assert csa.csa_check_status() == 0


def test_pool_past_four_gigabytes(csa):
    H, D, P = 4, 128, 32
    n = 300000                      # 4.9 GB of codes each for k and v
    x = make([(9, 150), (40, 33)], 8, H, D, P, seed=11, cap=5)
    small = run(csa, x)[0]
    far = (n - 1 - torch.arange(x["table"].numel(), device=DEV)).int().view(x["table"].shape)
    for c in "kv":
        big = torch.empty(n, H, P, D, dtype=torch.uint8, device=DEV)
        s = torch.ones(n, H, device=DEV)
        big[far.flatten().long()] = x[c].view(torch.uint8)[x["table"].flatten().long()]
        s[far.flatten().long()] = x[c + "s"][x["table"].flatten().long()]
        x[c], x[c + "s"] = big, s
    x["table"] = far
    assert torch.equal(small, run(csa, x)[0])
    assert csa.csa_check_status() == 0


def test_waits_give_up(csa):
    """With the scores' signal withheld every wait runs out, the call ends and reports it, and the next one is right."""
    for n, L in ((3, 300), (400, 900)):  # blocks shared out to the halves, and two full halves
        x = make([(n, L), (2, 100)], 4, 1, 128, 64, seed=n)
        good, _ = run(csa, x)
        assert csa.csa_check_status() == 0
        csa.csa_test_set_wait_fault(200, csa.CSA_TEST_FAULT_ATTN)
        try:
            run(csa, x)
            status = csa.csa_check_status()
        finally:
            csa.csa_test_set_wait_fault(0, 0)
        assert status == 4
        assert torch.equal(run(csa, x)[0], good)
        assert csa.csa_check_status() == 0


def test_tiles_of_one_block_again_and_again(csa):
    """Tiles of one block between longer ones, 300 calls on end of two books: no wait gives up, the bits stay."""
    seqs = [[(1 + i % 3, 5 + i % 120 if i % 5 else 500 + 10 * i) for i in range(n)] for n in (20, 90)]
    xs = [make(s, 16, 4, 64, 16, seed=i) for i, s in enumerate(seqs)]
    good = [run(csa, x)[0] for x in xs]
    cache = [csa.paged_cache(x["k"], x["v"], x["ks"], x["vs"], x["table"]) for x in xs]
    ws = [csa.chunk_attn_workspace(c, 16) for c in cache]
    outs = [torch.empty_like(g) for g in good]
    for _ in range(300):
        for x, c, w, o in zip(xs, cache, ws, outs):
            csa.csa_chunk_attn(c, x["cu"], x["lens"], x["q"], 0.125, 0, None, o, None, w)
    assert csa.csa_check_status() == 0
    for o, g in zip(outs, good):
        assert torch.equal(o, g)


def test_tiles_that_take_longer_than_a_wait(csa):
    """Shares of six tiles, each longer than the limit of a wait: the warp that is tiles ahead waits for their ends."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n, L = sms * 32, 32768                   # of two key heads that four query heads share: sms tiles
    x = make([(n, L)] * 6, 8, 2, 64, 128, seed=3)
    good, _ = run(csa, x)
    csa.csa_test_set_wait_fault(150, 0)      # (a tile takes some 400 us)
    try:
        out, _ = run(csa, x)
        status = csa.csa_check_status()
    finally:
        csa.csa_test_set_wait_fault(0, 0)
    assert status == 0 and torch.equal(out, good)


def test_refusals(csa):
    x = make([(5, 9), (2, 3)], 4, 2, 64, 16)
    cache = csa.paged_cache(x["k"], x["v"], x["ks"], x["vs"], x["table"])
    ws = csa.chunk_attn_workspace(cache, 4)
    out, lse = torch.empty_like(x["q"]), torch.empty(7, 4, device=DEV)

    def call(status, **kw):
        a = dict(cache=cache, cu_q=x["cu"], lens=x["lens"], q=x["q"], sm_scale=0.1, window=0, sink=None, out=out,
                 lse=lse, ws=ws)
        a.update(kw)
        with pytest.raises(csa.CsaError) as e:
            csa.csa_chunk_attn(**a)
        assert e.value.status == status, kw

    call(1, lens=x["lens"].long())
    call(1, lens=x["lens"][:1])
    call(1, cu_q=x["cu"][:2])
    call(1, lens=torch.zeros(3, dtype=torch.int32, device=DEV), cu_q=torch.zeros(4, dtype=torch.int32, device=DEV))
    call(1, q=x["q"].float())
    call(1, q=x["q"][:, :3], out=out[:, :3].contiguous(), lse=lse[:, :3].contiguous())
    call(1, out=out.transpose(0, 1).contiguous().transpose(0, 1))
    call(1, sm_scale=0.0)
    call(1, sm_scale=float("nan"))
    call(1, window=-1)
    call(1, sink=torch.zeros(3, device=DEV))
    call(1, lse=lse.double())
    call(6, ws=None)
    call(6, ws=ws[:-16])
    with pytest.raises(csa.CsaError):
        csa.chunk_attn_workspace(cache, 3)
