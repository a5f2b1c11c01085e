"""csa_prompt_attn against attention in 64 bits.  Weights are rounded to bf16
(half a step 2^-8)."""
import pytest
import torch

import _gqa as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
STEP = 2.0 ** -8


@pytest.fixture(scope="module")
def csa():
    import compressed_sparse_attention_02_gb300 as m
    return m


def make(lens, Hq, Hkv, D, seed=0, pad=0):
    """lens: (queries, keys) of each sequence."""
    g = torch.Generator(DEV).manual_seed(seed)
    nq, nk = sum(a for a, _ in lens) + pad, sum(b for _, b in lens) + pad
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g).bfloat16()  # noqa: E731
    cu = lambda i: torch.tensor([0] + [x[i] for x in lens]).cumsum(0).int().to(DEV)  # noqa: E731
    return dict(q=rnd(nq, Hq, D), k=rnd(nk, Hkv, D), v=rnd(nk, Hkv, D), cu_q=cu(0), cu_k=cu(1),
                sink=torch.randn(Hq, device=DEV, generator=g) * 2)


def run(csa, x, causal=True, window=0, sink=False, lse=True, sm=None, **kw):
    q = x["q"]
    out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device=DEV)
    l = torch.full(q.shape[:2], 9.0, device=DEV) if lse else None
    csa.csa_prompt_attn(x["cu_q"], x["cu_k"], q, x["k"], x["v"], q.shape[2] ** -0.5 if sm is None else sm, causal,
                        window, x["sink"] if sink else None, out, l, **kw)
    return out, l


def want(x, causal=True, window=0, sink=False, sm=None, heads=None):
    """Oracle results of the heads (all by default), [rows][heads]."""
    q, k, v = (x[n].double().cpu() for n in "qkv")
    n, Hq, D = q.shape
    heads = range(Hq) if heads is None else heads
    res = [torch.zeros(n, len(heads), *s, dtype=torch.float64) for s in ((D,), (), (D,), ())]
    cq, ck = x["cu_q"].tolist(), x["cu_k"].tolist()
    for b in range(len(cq) - 1):
        nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        i, j = torch.arange(nq)[:, None] + (nk - nq), torch.arange(nk)
        seen = (j <= i) if causal else torch.ones(nq, nk, dtype=torch.bool)
        if window:
            seen = seen & (j > i - window)
        for c, h in enumerate(heads):
            hk = h // (Hq // k.shape[1])
            got = ref.attend(q[cq[b]:cq[b + 1], h], k[ck[b]:ck[b + 1], hk], v[ck[b]:ck[b + 1], hk],
                             D ** -0.5 if sm is None else sm, seen, float(x["sink"][h]) if sink else None)
            for r, y in zip(res, got):
                r[cq[b]:cq[b + 1], c] = y
    return res


def check(csa, x, what, heads=None, **kw):
    out, lse = run(csa, x, **kw)
    n = int(x["cu_q"][-1])
    kw.pop("lse", None)
    w = [y[:n] for y in want(x, heads=heads, **kw)]
    at = list(range(x["q"].shape[1])) if heads is None else list(heads)
    ref.check_attention(out[:n, at], None if lse is None else lse[:n, at], *w, STEP, what)
    assert (out[n:] == 9).all() and (lse is None or (lse[n:] == 9).all())  # rows behind the last sequence
    return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 255, 256, 257, 400, 600])
def test_one_prompt(csa, D, n):
    check(csa, make([(n, n)], 2, 1, D, seed=n), "prompt")
    assert csa.csa_check_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 1, 100, 128, 129, 300])
@pytest.mark.parametrize("sink", [False, True])
def test_packed(csa, D, window, sink):
    """Prompts, one with a prefix, one without queries, one without keys, one with fewer keys than queries."""
    lens = [(130, 130), (0, 5), (33, 500), (3, 0), (200, 90), (1, 1), (300, 300), (1, 700)]
    check(csa, make(lens, 4, 2, D, seed=window, pad=7), "packed", window=window, sink=sink)
    assert csa.csa_check_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 1, 129, 300, 600])
@pytest.mark.parametrize("lens", [
    [(700, 700), (300, 900), (129, 40), (1, 300)],                        # more tiles than SMs, long sequences
    [(130, 130), (0, 5), (33, 500), (3, 0), (200, 90), (1, 1), (100, 100), (1, 700)],  # ... short ones
])
def test_many_tiles(csa, D, window, lens):
    """With 48 heads the tiles outnumber the SMs: two CTAs of one tile an SM."""
    many_tiles(csa, D, window, lens)


@pytest.mark.parametrize("window", [0, 700, 1025, 1100, 1281, 1700])
def test_many_tiles_that_see_many_keys(csa, window):
    """... and two tiles a CTA where they see more than 1024 keys."""
    many_tiles(csa, 128, window, [(2000, 2000), (300, 2300), (129, 40), (257, 1900)])


def many_tiles(csa, D, window, lens):
    x = make(lens, 48, 2, D, seed=window, pad=9)
    check(csa, x, "many tiles", heads=[0, 29, 47], window=window, sink=window % 2 == 0)
    if window in (0, 300, 700, 1100):  # a value that is not finite: seen or not as the formula has it
        clean = run(csa, x, window=window)[0]
        y = {k: v.clone() for k, v in x.items()}
        key = lens[0][1] - 60
        y["v"][key, 1, 7] = float("nan")
        y["v"][sum(b for _, b in lens):] = float("nan")
        out = run(csa, y, window=window)[0]
        n = lens[0][0]
        pos = torch.arange(n) + lens[0][1] - n
        rows = ((pos >= key) & (pos < key + (window or 10 ** 6))).nonzero()[:, 0].to(DEV)
        clean[rows, 24:, 7] = float("nan")
        assert torch.equal(out.isnan(), clean.isnan())
        assert torch.equal(out[~out.isnan()], clean[~clean.isnan()])
    assert csa.csa_check_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sink", [(0, True), (0, False), (700, True)])
@pytest.mark.parametrize("lens", [[(1, 2300)], [(130, 2300)], [(200, 1100)], [(128, 600)], [(64, 3100), (70, 2900)],
                                  [(3, 4000), (2, 9)]])
def test_few_queries_over_many_keys(csa, D, window, sink, lens):
    """Few tiles: a cluster of two, four or eight CTAs shares out a tile's keys."""
    x = make(lens, 3, 1, D, seed=len(lens) + window)
    check(csa, x, "cluster", window=window, sink=sink)
    clean = run(csa, x, window=window)[0]
    y = {k: v.clone() for k, v in x.items()}
    key = lens[0][1] - lens[0][0] // 2 - 1
    y["v"][key, 0, 3] = float("inf")
    out = run(csa, y, window=window)[0]
    pos = torch.arange(lens[0][0]) + lens[0][1] - lens[0][0]
    clean[((pos >= key) & (pos < key + (window or 10 ** 6))).nonzero()[:, 0].to(DEV), :, 3] = float("inf")
    assert torch.equal(out, clean)
    assert csa.csa_check_status() == 0


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (6, 1), (8, 2), (28, 4)])
def test_groups(csa, Hq, Hkv):
    x = make([(140, 140), (60, 300)], Hq, Hkv, 128, seed=Hq)
    check(csa, x, "groups", heads=sorted({0, Hq // 2, Hq - 1}))


def test_not_causal(csa):
    x = make([(130, 300), (5, 1), (70, 128), (9, 0)], 2, 1, 64, seed=3, pad=2)
    check(csa, x, "all keys", causal=False)
    check(csa, x, "all keys, sink", causal=False, sink=True)


def test_many_short_sequences(csa):
    g = torch.Generator().manual_seed(1)
    lens = [(int(n), int(n)) for n in torch.randint(0, 9, (900,), generator=g)]
    for D in (64, 128):
        check(csa, make(lens, 1, 1, D, seed=4), "short")
    assert csa.csa_check_status() == 0


def test_many_tiles_without_keys(csa):
    """Most tiles see no key (more queries than keys, or none): their softmax has nothing to wait for but the queries."""
    for D, lens in ((64, [(700, 0), (900, 1), (300, 0), (500, 130)] * 2), (128, [(700, 0), (900, 1), (300, 0)] * 3),
                    (128, [(700, 0), (2000, 9000), (900, 1), (1300, 300)])):
        x = make(lens, 48, 2, D, seed=D)
        check(csa, x, "no keys", heads=[0, 31], sink=D == 64)
        first = run(csa, x)[0]
        for _ in range(5):
            assert torch.equal(first, run(csa, x)[0])
    assert csa.csa_check_status() == 0


def test_long_rows_sampled(csa):
    """4100 keys: the last rows of the oracle only, over every tile's border."""
    x = make([(4100, 4100)], 2, 1, 128, seed=5)
    out, lse = run(csa, x)
    rows = torch.tensor([0, 127, 128, 2047, 2048, 3999, 4095, 4096, 4099])
    q, k, v = (x[n].double().cpu() for n in "qkv")
    for h in range(2):
        seen = torch.arange(4100) <= rows[:, None]
        w = ref.attend(q[rows, h], k[:, 0], v[:, 0], 128 ** -0.5, seen)
        ref.check_attention(out[rows.to(DEV), h], lse[rows.to(DEV), h], *w, STEP, "long")


@pytest.mark.parametrize("window", [520, 1024, 1500])
def test_windows_of_several_tiles(csa, window):
    """Rows whose keys begin and end in masked tiles with whole tiles between them, values that are not finite at
    both ends (a row has infinities only where its window holds them)."""
    T = 2200
    for D in (64, 128):
        x = make([(T, T), (300, T)], 2, 1, D, seed=window)
        clean = run(csa, x, window=window)[0]
        y = {k: v.clone() for k, v in x.items()}
        want_ = clean.clone()
        for first, shift, n in ((0, 0, T), (T, T - 300, 300)):
            for key in (700, 1100, 1101, 2100):
                y["v"][(0 if first == 0 else T) + key, 0, 9] = float("inf")
                pos = torch.arange(n) + shift
                want_[first + ((pos >= key) & (pos < key + window)).nonzero()[:, 0].to(DEV), :, 9] = float("inf")
        out = run(csa, y, window=window)[0]
        assert torch.equal(out, want_)
        rows = torch.tensor([0, window - 1, window, 1300, T - 1])
        for h in range(2):
            pos = torch.arange(T)
            seen = (pos <= rows[:, None]) & (pos > rows[:, None] - window)
            w = ref.attend(x["q"][rows.to(DEV), h].cpu(), x["k"][:T, 0].cpu(), x["v"][:T, 0].cpu(), D ** -0.5, seen)
            ref.check_attention(clean[rows.to(DEV), h], None, *w, STEP, "window")
    assert csa.csa_check_status() == 0


@pytest.mark.parametrize("window", [0, 50])
def test_values_that_are_not_finite(csa, window):
    """NaN and infinities in keys and values: rows that do not see them are as without them, bit for bit; rows that
    do have them where the formula does."""
    for D in (64, 128):
        x = make([(300, 300), (200, 260)], 2, 1, D, seed=6, pad=40)
        clean = run(csa, x, window=window)[0]
        y = {k: v.clone() for k, v in x.items()}
        y["v"][250, 0, 3] = float("nan")     # sequence 0, key 250
        y["v"][270, 0, 5] = float("inf")     # key 270
        y["v"][271, 0, 5] = float("inf")
        y["v"][299, 0, 7] = -float("inf")    # the last key
        y["v"][300 + 130, 0, 1] = float("nan")  # sequence 1, key 130: row 70
        y["v"][560:], y["k"][560:] = float("nan"), float("nan")  # behind the last sequence
        y["k"][300 + 200, 0, 0] = float("nan")  # sequence 1, key 200: row 140
        out, lse = run(csa, y, window=window)
        want_ = clean.clone()
        W = window or 10 ** 6
        i0, i1 = torch.arange(300), torch.arange(200) + 60
        def put(first, i, key, ch, val):  # noqa: E306
            at = ((i >= key) & (i < key + W)).nonzero()[:, 0] + first
            for h in range(2):
                for r in at.tolist():
                    want_[r, h, ch] = val
        put(0, i0, 250, 3, float("nan"))
        put(0, i0, 270, 5, float("inf"))
        put(0, i0, 271, 5, float("inf"))
        put(0, i0, 299, 7, -float("inf"))
        put(300, i1, 130, 1, float("nan"))
        for ch in range(D):
            put(300, i1, 200, ch, float("nan"))
        assert torch.equal(out.isnan(), want_.isnan())
        assert torch.equal(out[~out.isnan()], want_[~want_.isnan()])
    assert csa.csa_check_status() == 0


def test_large_logits_and_equal_rows(csa):
    """Logits that grow along the keys (the accumulators are rescaled again and again) and keys that are all alike."""
    x = make([(384, 384)], 2, 1, 64, seed=7)
    x["q"].fill_(1.0)
    x["k"].copy_((torch.arange(384, device=DEV)[:, None, None] * 0.25).expand(384, 1, 64).bfloat16())
    check(csa, x, "growing", sm=0.05)
    x["k"].copy_(x["k"].flip(0))
    check(csa, x, "falling", sm=0.05)
    x["k"].fill_(0.5)
    check(csa, x, "equal")


def test_logits_beyond_what_fp32_resolves(csa):
    """Logits of 2^50 and more: the weights are those of the row's largest key alone, whose values the row returns."""
    T = 300
    x = make([(T, T)], 2, 1, 64, seed=12)
    x["q"][:, 0] *= 2.0 ** 50
    out, lse = run(csa, x)
    q, k, v = (x[n].double().cpu() for n in "qkv")
    logits = (q[:, 0] @ k[:, 0].T).masked_fill_(torch.ones(T, T).triu(1).bool(), float("-inf"))
    best, second = logits.topk(2, dim=1).values[1:].T
    assert ((best - second) > 2.0 ** 30).all()  # (a tie would be shared)
    assert torch.equal(out[:, 0].cpu(), x["v"][:, 0].cpu()[logits.argmax(1)])
    assert ((lse[:, 0].cpu().double() - logits.max(1).values / 8).abs() <= 2.0 ** -16 * logits.max(1).values.abs()).all()
    w = want(x, heads=[1])
    ref.check_attention(out[:, 1:], lse[:, 1:], *w, STEP, "the other head")


def test_layouts_streams_and_graphs(csa):
    """A fused projection's views, heads outermost, another stream, a replayed graph: the same bits."""
    T, Hq, Hkv, D = 333, 8, 2, 128
    x = make([(200, 200), (133, 133)], Hq, Hkv, D, seed=8)
    out, lse = run(csa, x)
    fused = torch.cat([x["q"], x["k"], x["v"]], 1)
    y = dict(x, q=fused[:, :Hq], k=fused[:, Hq:Hq + Hkv], v=fused[:, Hq + Hkv:])
    assert torch.equal(out, run(csa, y)[0])
    z = dict(x, **{n: x[n].transpose(0, 1).contiguous().transpose(0, 1) for n in "qkv"})
    assert torch.equal(out, run(csa, z)[0])
    assert torch.equal(out, run(csa, x, lse=False)[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, l2 = run(csa, x)
    side.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    o3, l3 = torch.zeros_like(out), torch.zeros_like(lse)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        csa.csa_prompt_attn(x["cu_q"], x["cu_k"], x["q"], x["k"], x["v"], D ** -0.5, True, 0, None, o3, l3)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o3) and torch.equal(lse, l3)
    assert csa.csa_check_status() == 0


def test_bad_offsets(csa):
    x = make([(50, 50), (40, 40), (30, 30)], 2, 1, 64, seed=9)
    good = run(csa, x)[0]
    for n in ("cu_q", "cu_k"):
        for bad, lo, hi in (([0, 50, 20, 10], 0, 50), ([0, 50, 999, 120], 0, 50), ([0, 50, 90, 121], 0, 90),
                            ([-3, 50, 90, 120], 50, 120)):
            y = dict(x, **{n: torch.tensor(bad, dtype=torch.int32, device=DEV)})
            out, _ = run(csa, y)
            assert csa.csa_check_status() == 5
            assert torch.equal(out[lo:hi], good[lo:hi])
            assert (out[:lo] == 9).all() and (out[hi:] == 9).all()


def test_a_wait_that_runs_out(csa):
    """The products never announce the first scores: the call ends, reports the timeout, and the next one is right."""
    for D, Hq, lens in ((128, 4, [(500, 500)]), (128, 48, [(700, 700)]), (64, 48, [(700, 700)]), (64, 2, [(20, 3000)]),
                        (128, 48, [(100, 100)] * 8), (128, 48, [(1100, 1100)])):
        x = make(lens, Hq, 2, D, seed=10)
        good = run(csa, x)[0]
        csa.csa_test_set_wait_fault(200, csa.CSA_TEST_FAULT_ATTN)
        try:
            run(csa, x)
            assert csa.csa_check_status() == 4
        finally:
            csa.csa_test_set_wait_fault(0, 0)
        assert torch.equal(run(csa, x)[0], good)
        assert csa.csa_check_status() == 0


def test_refusals(csa):
    x = make([(5, 5), (9, 9)], 4, 2, 64)
    out, lse = torch.empty_like(x["q"]), torch.empty(14, 4, device=DEV)

    def call(status=1, **kw):
        a = dict(cu_q=x["cu_q"], cu_k=x["cu_k"], q=x["q"], k=x["k"], v=x["v"], sm_scale=0.1, causal=True, window=0,
                 sink=None, out=out, lse=lse)
        a.update(kw)
        with pytest.raises(csa.CsaError) as e:
            csa.csa_prompt_attn(**a)
        assert e.value.status == status, kw

    call(cu_q=x["cu_q"].long())
    call(cu_k=x["cu_k"][:2])
    call(cu_q=x["cu_q"][:0])
    call(q=x["q"].half())
    call(k=x["k"][:13])
    call(k=x["k"][..., :32])
    call(q=x["q"][:, :3], out=out[:, :3].contiguous(), lse=None)
    call(out=out[:-1])
    call(window=4, causal=False)
    call(window=-1)
    call(sm_scale=-0.1)
    call(sm_scale=float("inf"))
    call(sink=torch.zeros(4, device=DEV).half())
    big = torch.zeros(14, 4, 96, device=DEV).bfloat16()
    call(2, q=big, k=big[:, :2], v=big[:, :2], out=torch.empty_like(big), lse=None)
    csa.csa_prompt_attn(x["cu_q"], x["cu_k"], x["q"][:0], x["k"], x["v"], 0.1, True, 0, None, out[:0])
