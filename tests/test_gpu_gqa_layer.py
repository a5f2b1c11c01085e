"""The grouped-query calls together, as a layer uses them: prompts of different
lengths are rotated, attended to and appended to the paged cache; then tokens
are decoded, rotated, appended and attended to from the cache, eagerly and as
a replayed graph."""
import pytest
import torch

import _gqa as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64


@pytest.fixture(scope="module")
def csa():
    import compressed_sparse_attention_02_gb300 as m
    return m


class Layer:
    """What a program keeps for one layer and a batch of sequences; `project` stands for the fused projection."""

    def __init__(self, csa, B, Hq, Hkv, D, page, pages, window, sink, rope, seed):
        self.csa, self.B, self.Hq, self.Hkv, self.D, self.window = csa, B, Hq, Hkv, D, window
        g = torch.Generator(DEV).manual_seed(seed)
        n = B * pages
        self.k, self.v = (torch.zeros(n, Hkv, page, D, dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2))
        self.ks, self.vs = (torch.zeros(n, Hkv, device=DEV) for _ in range(2))
        self.table = torch.randperm(n, device=DEV, generator=g).int().view(B, pages)
        self.cache = csa.paged_cache(self.k, self.v, self.ks, self.vs, self.table)
        self.rope, self.turns = rope, csa.rope_table(rope)
        self.sink = torch.randn(Hq, device=DEV, generator=g) if sink else None
        self.ws = csa.paged_attn_workspace(self.cache, B, Hq)
        self.scale = D ** -0.5

    def project(self, n, seed):
        g = torch.Generator(DEV).manual_seed(seed)
        return torch.randn(n, self.Hq + 2 * self.Hkv, self.D, device=DEV, generator=g).bfloat16()

    def split(self, qkv):
        return qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.Hkv], qkv[:, self.Hq + self.Hkv:]

    def prompt(self, qkv, cu, pos0, pos):
        """Attention of whole prompts; their keys and values into the cache."""
        csa = self.csa
        _, k, v = self.split(qkv)
        turned = csa.csa_rope(self.rope, self.turns, pos, qkv[:, :self.Hq + self.Hkv])
        out = torch.zeros(qkv.shape[0], self.Hq, self.D, dtype=torch.bfloat16, device=DEV)
        lse = torch.zeros(qkv.shape[0], self.Hq, device=DEV)
        csa.csa_prompt_attn(cu, cu, turned[:, :self.Hq], turned[:, self.Hq:], v, self.scale, True, self.window, self.sink,
                            out, lse)
        csa.csa_kv_append(self.cache, self.rope, self.turns, cu, pos0, k, v)
        return turned, out, lse

    def decode(self, qkv, pos, lens, q, out, lse):
        """One token a sequence at `pos` (lens = pos + 1), into the given buffers."""
        csa = self.csa
        q0, k, v = self.split(qkv)
        csa.csa_rope(self.rope, self.turns, pos, q0, out=q)
        csa.csa_kv_append(self.cache, self.rope, self.turns, None, pos, k, v)
        csa.csa_paged_attn(self.cache, lens, q, self.scale, self.window, self.sink, out, lse, self.ws)


@pytest.mark.parametrize("Hq,Hkv,D,page,window,sink", [(8, 2, 128, 64, 0, False), (12, 2, 64, 16, 100, True),
                                                       (4, 4, 128, 32, 0, True)])
def test_prompts_then_decoding(csa, Hq, Hkv, D, page, window, sink):
    lens = [1, 130, 0, 67, 300]
    B, steps = len(lens), 5
    rope = csa.rope_params(rope_dim=64, offset=D - 64, layout=0 if D == 64 else 1, scaling=2, factor=4.0, orig_len=256,
                           mscale=1.1)

    def fresh():
        return Layer(csa, B, Hq, Hkv, D, page, -(-(max(lens) + steps) // page), window, sink, rope, 3)

    layer = fresh()
    cu = torch.tensor([0] + lens).cumsum(0).int().to(DEV)
    pos0 = torch.zeros(B, dtype=torch.int32, device=DEV)
    pos = torch.cat([torch.arange(n) for n in lens]).int().to(DEV)
    qkv = layer.project(sum(lens), 1)
    turned, out, lse = layer.prompt(qkv, cu, pos0, pos)
    assert csa.csa_check_status() == 0

    # the rotation, then the attention over the rotated rows the kernel was given
    both = Hq + Hkv
    want = ref.rope(rope, qkv[:, :both], pos)
    assert ((turned.double().cpu() - want).abs() <=
            2.0 ** -8 * want.abs() + ref.ROPE_ABS * ref.pair_size(rope, qkv[:, :both])).all()
    v = qkv[:, both:]
    for b, n in enumerate(lens):
        s = slice(int(cu[b]), int(cu[b]) + n)
        i = torch.arange(n)
        seen = (i[None] <= i[:, None]) & ((i[None] > i[:, None] - window) if window else True)
        for h in (0, Hq - 1):
            hk = h // (Hq // Hkv)
            w = ref.attend(turned[s, h].cpu(), turned[s, Hq + hk].cpu(), v[s, hk].cpu(), layer.scale, seen,
                           float(layer.sink[h]) if sink else None)
            ref.check_attention(out[s, h], lse[s, h], *w, 2.0 ** -8, "prompt")

    # every cached row within its rounding (half a step: 2^-4, or 2^-10 of the scale) of the row itself
    def cached(x, sc, b, n):
        pages = layer.table[b].long()
        y = x[pages].float().double().cpu() * sc[pages].double().cpu()[..., None, None]
        return y.transpose(1, 2).reshape(-1, Hkv, D)[:n], sc[pages].double().cpu().repeat_interleave(page, 0)[:n]

    rows = {b: (want[int(cu[b]):int(cu[b + 1]), Hq:], v[int(cu[b]):int(cu[b + 1])].double().cpu()) for b in range(B)}

    def check_cache(steps_done):
        for b in range(B):
            for x, sc, r in ((layer.k, layer.ks, rows[b][0]), (layer.v, layer.vs, rows[b][1])):
                got, s = cached(x, sc, b, len(r))
                # (a page whose scale grew after a row came rounds it again)
                tol = 2.0 ** -4 * r.abs() + s[..., None] * 2.0 ** -10 + 2.0 ** -20 * 8
                assert ((got - r).abs() <= tol * (1 if steps_done == 0 else 2)).all()

    check_cache(0)

    # decode: the attention over what the cache holds
    at = torch.tensor(lens, dtype=torch.int32, device=DEV)
    n1 = torch.empty_like(at)
    q = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=DEV)
    o, l = torch.empty_like(q), torch.empty(B, Hq, device=DEV)
    eager = []
    for t in range(steps):
        x = layer.project(B, 10 + t)
        p = at + t
        n1.copy_(p + 1)
        layer.decode(x, p, n1, q, o, l)
        eager.append((o.clone(), l.clone()))
        turned = ref.rope(rope, x[:, :both], p)
        for b in range(B):
            k1 = torch.cat([rows[b][0], turned[b:b + 1, Hq:]])
            v1 = torch.cat([rows[b][1], x[b:b + 1, both:].double().cpu()])
            rows[b] = (k1, v1)
            n = len(k1)
            kk, vv = cached(layer.k, layer.ks, b, n)[0], cached(layer.v, layer.vs, b, n)[0]
            seen = torch.arange(n)[None] >= (n - window if window else 0)
            for h in range(Hq):
                hk = h // (Hq // Hkv)
                w = ref.attend(q[b, h][None].cpu(), kk[:, hk], vv[:, hk], layer.scale, seen,
                               float(layer.sink[h]) if sink else None)
                ref.check_attention(o[b, h][None], l[b, h][None], *w, 2.0 ** -11, "decode")
        check_cache(t + 1)
    assert csa.csa_check_status() == 0

    # the same steps from a captured graph over a second cache: the same bits
    twin = fresh()
    twin.prompt(qkv, cu, pos0, pos)
    x, p = torch.empty(B, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV), at.clone()
    n1.copy_(p + 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        twin.decode(x, p, n1, q, o, l)
        p.add_(1)
        n1.add_(1)
    torch.cuda.current_stream().wait_stream(side)
    for t in range(steps):
        x.copy_(layer.project(B, 10 + t))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, eager[t][0]) and torch.equal(l, eager[t][1])
    assert torch.equal(twin.k.view(torch.uint8), layer.k.view(torch.uint8))
    assert torch.equal(twin.vs, layer.vs)
    assert csa.csa_check_status() == 0


def test_calls_on_several_streams(csa):
    """Prompts in every form of the kernel, decode attention and appends replayed on five streams at once: the bits of
    the same calls one after the other."""
    g = torch.Generator(DEV).manual_seed(9)
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g).bfloat16()  # noqa: E731
    work = []

    def prompts(lens, Hq, D):
        cu = torch.tensor([0] + lens).cumsum(0).int().to(DEV)
        q, k, v = rnd(sum(lens), Hq, D), rnd(sum(lens), 2, D), rnd(sum(lens), 2, D)
        out, lse = torch.empty_like(q), torch.empty(sum(lens), Hq, device=DEV)
        work.append(((lambda: csa.csa_prompt_attn(cu, cu, q, k, v, D ** -0.5, True, 0, None, out, lse)), (out, lse)))

    prompts([1700, 1300], 32, 128)      # two tiles of queries a CTA
    prompts([300] * 9, 32, 64)          # two CTAs an SM
    prompts([200], 8, 128)              # a cluster a tile
    for D in (64, 128):
        layer = Layer(csa, 12, 16, 2, D, 32, 40, 0, False, csa.rope_params(rope_dim=64), 5)
        lens = torch.randint(1, 1000, (12,), device=DEV, generator=g).int()
        x, pos = rnd(12, 20, D), lens - 1
        cu = torch.cat([torch.zeros(1, device=DEV), lens.cumsum(0)]).int()
        n = int(lens.sum())
        csa.csa_kv_append(layer.cache, layer.rope, layer.turns, cu, torch.zeros_like(lens), rnd(n, 2, D), rnd(n, 2, D))
        q, o = (torch.empty(12, 16, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        l = torch.empty(12, 16, device=DEV)
        work.append(((lambda y=layer, x=x, p=pos, n=lens, q=q, o=o, l=l: y.decode(x, p, n, q, o, l)),
                     (q, o, l, layer.k.view(torch.uint8), layer.vs)))
    want = []
    for call, outs in work:
        call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    graphs = []
    for call, _ in work:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                call()
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in work]
    for _, outs in work:
        outs[0].zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for (_, outs), w in zip(work, want):
        for a, b in zip(outs, w):
            assert torch.equal(a, b)
    assert csa.csa_check_status() == 0
