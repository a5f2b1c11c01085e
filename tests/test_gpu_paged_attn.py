"""csa_paged_attn against attention in 64 bits over the values its codes stand
for.  Weights are rounded to f16 (half a step 2^-11)."""
import math

import pytest
import torch

import _gqa as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
STEP = 2.0 ** -11


@pytest.fixture(scope="module")
def csa():
    import compressed_sparse_attention_02_gb300 as m
    return m


def make(lens, Hq, Hkv, D, P, seed=0, cap=None, scales=(-7, -4)):
    """A pool whose unwritten tokens are NaN codes, shuffled pages, queries and sinks."""
    g = torch.Generator(DEV).manual_seed(seed)
    B = len(lens)
    cap = cap or max(1, -(-max(lens) // P))
    n = B * cap + 2
    x = {}
    for c in "kv":
        e = torch.randint(*scales, (n, Hkv), device=DEV, generator=g).float()
        x[c + "s"] = torch.exp2(e) * (1 + torch.rand(n, Hkv, device=DEV, generator=g))
        y = torch.randn(n, Hkv, P, D, device=DEV, generator=g) * 1.5
        x[c] = (y / x[c + "s"][..., None, None] * torch.exp2(e - e.mean())[..., None, None]).clamp(-448, 448)
        x[c] = x[c].to(torch.float8_e4m3fn)
    table = torch.randperm(n, device=DEV, generator=g)[:B * cap].int().view(B, cap)
    for b, L in enumerate(lens):
        for p in range(cap):
            from_ = max(0, min(P, L - p * P))
            for c in "kv":
                x[c].view(torch.uint8)[int(table[b, p]), :, from_:] = 0x7F
    x.update(table=table, q=torch.randn(B, Hq, D, device=DEV, generator=g).bfloat16(),
             lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
             sink=torch.randn(Hq, device=DEV, generator=g) * 2)
    return x


def run(csa, x, window=0, sink=False, lse=True, ws=None, sm=None, q=None, stream=None):
    cache = csa.paged_cache(x["k"], x["v"], x["ks"], x["vs"], x["table"])
    q = x["q"] if q is None else q
    B, Hq, D = q.shape
    out = torch.full((B, Hq, D), 9.0, dtype=torch.bfloat16, device=DEV)
    l = torch.full((B, Hq), 9.0, device=DEV) if lse else None
    csa.csa_paged_attn(cache, x["lens"], q, D ** -0.5 if sm is None else sm, window, x["sink"] if sink else None, out,
                       l, csa.paged_attn_workspace(cache, B, Hq) if ws is None else ws, stream)
    return out, l


def want(x, window=0, sink=False, sm=None, skip=()):
    """Oracle results, [B][Hq] of each; skip: (sequence, page of its table) left out."""
    k, v = (x[c].to(torch.float32).double().cpu() * x[c + "s"].double().cpu()[..., None, None] for c in "kv")
    q, table = x["q"].double().cpu(), x["table"].cpu()
    B, Hq, D = q.shape
    Hkv, P = k.shape[1], k.shape[2]
    res = [[], [], [], []]
    for b in range(B):
        L = min(max(int(x["lens"][b]), 0), table.shape[1] * P)
        lo = max(0, L - window) if window else 0
        seen = torch.arange(L) >= lo
        for p in range(-(-L // P)):
            if (b, p) in skip:
                seen[p * P:(p + 1) * P] = False
        pages = table[b, :-(-L // P)].long().clamp(0, k.shape[0] - 1)
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            got = ref.attend(q[b, h][None], k[pages, hk].reshape(-1, D)[:L], v[pages, hk].reshape(-1, D)[:L],
                             D ** -0.5 if sm is None else sm, seen[None],
                             float(x["sink"][h]) if sink else None)
            for r, y in zip(res, got):
                r.append(y[0])
    return [torch.stack(r).view(B, Hq, *r[0].shape) for r in res]


def check(csa, x, what, **kw):
    skip = kw.pop("skip", ())
    out, lse = run(csa, x, **kw)
    w = want(x, kw.get("window", 0), kw.get("sink", False), kw.get("sm"), skip)
    ref.check_attention(out, lse, *w, STEP, what)
    return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_lengths_and_pages(csa, D, P):
    x = make([1, 0, 15, 16, 17, 31, 33, 127, 128, 129, 255, 257, 700, 0], 8, 2, D, P, seed=D + P)
    check(csa, x, "plain")
    check(csa, x, "sink", sink=True)
    assert csa.csa_check_status() == 0


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (6, 2), (14, 2), (16, 1), (17, 1), (40, 1), (32, 8), (5, 5)])
def test_groups(csa, Hq, Hkv):
    for D in (64, 128):
        check(csa, make([5, 300, 129], Hq, Hkv, D, 32, seed=Hq), "group", sink=True)
    assert csa.csa_check_status() == 0


@pytest.mark.parametrize("window", [1, 2, 16, 100, 128, 129, 1000])
def test_windows(csa, window):
    for D, P in ((64, 16), (128, 64)):
        x = make([1, 100, 128, 130, 257, 1001], 4, 2, D, P, seed=window)
        check(csa, x, "window", window=window, sink=window % 2 == 0)
        # what the window leaves out has no effect, whatever it holds
        lens = x["lens"].tolist()
        before = run(csa, x, window=window)[0]
        for b, L in enumerate(lens):
            for t in range(max(0, L - window)):
                page = int(x["table"][b, t // P])
                for c in "kv":
                    x[c].view(torch.uint8)[page, :, t % P] = 0x7F
        assert torch.equal(before, run(csa, x, window=window)[0])
    assert csa.csa_check_status() == 0


def test_many_sequences_of_mixed_lengths(csa):
    """300 sequences (several passes of the search), shares that cut some and hold several others."""
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(0, 60, (300,), generator=g).tolist()
    lens[7], lens[200] = 3000, 1700
    check(csa, make(lens, 4, 2, 64, 16, seed=5), "mixed")
    check(csa, make([20000, 3], 8, 1, 128, 128, seed=6), "long")
    assert csa.csa_check_status() == 0


@pytest.mark.parametrize("seqs,Hq,Hkv", [(1, 2, 1), (6, 16, 8), (12, 10, 10), (24, 8, 8)])
def test_number_of_pairs(csa, seqs, Hq, Hkv):
    """One pair of a sequence and a KV head to some hundred, empty sequences among them: a pair's parts are joined in
    other ways where the pairs are few."""
    g = torch.Generator().manual_seed(seqs)
    lens = torch.randint(1, 900, (seqs,), generator=g).tolist()
    lens[0] = 5000
    if seqs > 2:
        lens[2] = 0
    for D in (64, 128):
        check(csa, make(lens, Hq, Hkv, D, 64, seed=seqs), "pairs", sink=D == 64)
    assert csa.csa_check_status() == 0


def test_scales_of_any_size(csa):
    """Pages whose scales differ by 2^40, pages of zeros with the smallest scale, a value scale of zero."""
    x = make([500, 130, 64], 8, 2, 128, 16, seed=8)
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


def test_queries_of_any_size(csa):
    x = make([200], 6, 1, 64, 32, seed=9, scales=(-12, -11))
    x["q"][0, 0] = 0
    x["q"][0, 1] *= 2.0 ** 60
    x["q"][0, 1, 1:] *= 2.0 ** -60
    x["q"][0, 2] *= 2.0 ** -100
    x["q"][0, 3] *= 30
    x["sink"][1] = -math.inf
    # (row 1: one channel decides, its logits are of 2^60: differences below them do not matter, so the weights are
    # those of the largest logits alone)
    out, lse = run(csa, x, sink=True)
    w = want(x, 0, True)
    rows = [0, 2, 3, 4, 5]
    ref.check_attention(out[:, rows], lse[:, rows], *[y[:, rows] for y in w], STEP, "queries")
    assert torch.isfinite(out).all()


def test_bad_tables_and_lengths(csa):
    x = make([300, 200, 64, 90], 4, 2, 64, 32, seed=3)
    x["table"][0, 2] = -1
    x["table"][1, 0] = x["k"].shape[0]
    x["lens"][2] = 10 ** 6          # clamped to the table: the NaN codes behind token 64 are then seen
    x["lens"][3] = -5
    out, lse = run(csa, x)
    assert csa.csa_check_status() == 5
    x["lens"][2] = 0
    w = want(x, skip={(0, 2), (1, 0)})
    rows = [0, 1, 3]
    ref.check_attention(out[rows], lse[rows], *[y[rows] for y in w], STEP, "bad pages")
    assert torch.isnan(out[2].float()).all()
    # a sequence all of whose pages are bad sees nothing
    x["table"][1] = -1
    out, lse = run(csa, x)
    assert csa.csa_check_status() == 5
    assert (out[1] == 0).all() and torch.isinf(lse[1]).all()


def test_strided_queries_streams_graphs_and_repeats(csa):
    x = make([1000, 77, 2500], 16, 4, 128, 64, seed=4)
    out, lse = run(csa, x)
    wide = torch.randn(3, 24, 128, device=DEV).bfloat16()
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
        ws = csa.paged_attn_workspace(cache, 3, 16)
        o, l = torch.zeros_like(out), torch.zeros_like(lse)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            csa.csa_paged_attn(cache, x["lens"], x["q"], 128 ** -0.5, 0, None, o, l, ws)
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


def test_pool_past_four_gigabytes(csa):
    H, D, P = 4, 128, 32
    n = 300000                      # 4.9 GB of codes each for k and v
    x = make([150, 33], 8, H, D, P, seed=11, cap=5)
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


def test_refusals(csa):
    x = make([5, 9], 4, 2, 64, 16)
    cache = csa.paged_cache(x["k"], x["v"], x["ks"], x["vs"], x["table"])
    ws = csa.paged_attn_workspace(cache, 2, 4)
    out, lse = torch.empty_like(x["q"]), torch.empty(2, 4, device=DEV)

    def call(status, **kw):
        a = dict(cache=cache, lens=x["lens"], q=x["q"], sm_scale=0.1, window=0, sink=None, out=out, lse=lse, ws=ws)
        a.update(kw)
        with pytest.raises(csa.CsaError) as e:
            csa.csa_paged_attn(**a)
        assert e.value.status == status, kw

    call(1, lens=x["lens"].long())
    call(1, lens=x["lens"][:1])
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
        csa.paged_attn_workspace(cache, 2, 3)
