"""The paged cache's calls together, as a serving program uses them: prompts
come in chunks that take pages, are appended and attended to; sequences are
forked, go on apart, are cut back and end; the pool is compacted under them;
then tokens are decoded.  Every attention is checked against 64-bit arithmetic
over what the cache holds, and a captured step against eager ones."""
import pytest
import torch

import _gqa as ref
import test_gpu_chunk_attn as chunk

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def csa():
    import compressed_sparse_attention_02_gb300 as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Server:
    """One table for the caches of `layers` layers, and the call buffers."""

    def __init__(self, csa, slots, Hq, Hkv, D, page, pool, cap, layers=2, seed=0):
        self.csa, self.slots, self.Hq, self.Hkv, self.D, self.page = csa, slots, Hq, Hkv, D, page
        g = torch.Generator(DEV).manual_seed(seed)
        self.table = torch.full((slots, cap), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(slots, dtype=torch.int32, device=DEV)
        self.refs = torch.zeros(pool, dtype=torch.int32, device=DEV)
        self.book = csa.page_book(self.table, self.lens, self.refs, page)
        self.pages_ws = csa.pages_workspace(self.book)
        self.layers = []
        for _ in range(layers):
            k, v = (torch.full((pool, Hkv, page, D), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2))
            ks, vs = (torch.ones(pool, Hkv, device=DEV) for _ in range(2))
            self.layers.append(csa.paged_cache(k, v, ks, vs, self.table))
        self.rope = csa.rope_params(rope_dim=D)
        self.turns = csa.rope_table(self.rope)
        self.ws = csa.chunk_attn_workspace(self.layers[0], Hq)
        self.decode_ws = csa.paged_attn_workspace(self.layers[0], slots, Hq)
        self.pos0, self.src, self.dst = (torch.zeros(slots, dtype=torch.int32, device=DEV) for _ in range(3))
        self.g = g

    def project(self, rows):
        return [torch.randn(rows, self.Hq + 2 * self.Hkv, self.D, device=DEV, generator=self.g).bfloat16()
                for _ in self.layers]

    def copy(self):
        for c in self.layers:
            self.csa.csa_pages_copy(c, self.src, self.dst)

    def step(self, new, qkv, target, cu, out):
        """`new` tokens a slot: room, contents of pages taken apart, append, attention of the chunk (all layers)."""
        csa = self.csa
        csa.csa_pages_resize(self.book, target, self.pos0, self.src, self.dst, self.pages_ws)
        self.copy()
        for c, x, o in zip(self.layers, qkv, out):
            q, k, v = x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]
            csa.csa_kv_append(c, self.rope, self.turns, cu, self.pos0, k, v)
            csa.csa_chunk_attn(c, cu, self.lens, q, self.D ** -0.5, 0, None, o[0], o[1], self.ws)

    def run(self, new):
        target = torch.where(i32(new) > 0, self.lens + i32(new), -1)
        cu = i32([0] + new).cumsum(0).int()
        n = sum(new)
        qkv = self.project(n)
        out = [(torch.full((n, self.Hq, self.D), 9.0, device=DEV).bfloat16(), torch.full((n, self.Hq), 9.0, device=DEV))
               for _ in self.layers]
        self.step(new, qkv, target, cu, out)
        assert self.csa.csa_check_status() == 0
        for c, x, (o, lse) in zip(self.layers, qkv, out):
            y = self.view(c, x[:, :self.Hq].contiguous(), cu)
            ref.check_attention(o, lse, *chunk.want(y), chunk.STEP, "chunk")
        return qkv, cu

    def view(self, c, q, cu):
        k, v, ks, vs, table = c.tensors
        return dict(k=k.view(torch.float8_e4m3fn), v=v.view(torch.float8_e4m3fn), ks=ks, vs=vs, table=table, q=q, cu=cu,
                    lens=self.lens)

    def tokens(self, c, b):
        """The values that a layer's cache holds for a slot."""
        k, v, ks, vs, table = c.tensors
        L = int(self.lens[b])
        pages = table[b, :-(-L // self.page)].long()
        return [(x[pages].view(torch.float8_e4m3fn).float() * s[pages][..., None, None]).transpose(1, 2).flatten(0, 1)[:L]
                for x, s in ((k, ks), (v, vs))]

    def counts(self):
        n = torch.zeros_like(self.refs)
        for b, L in enumerate(self.lens.tolist()):
            n.index_add_(0, self.table[b, :-(-L // self.page)].long(),
                         torch.ones(-(-L // self.page), dtype=torch.int32, device=DEV))
        assert torch.equal(n, self.refs)


@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 128, 64), (12, 2, 64, 16), (4, 4, 64, 32)])
def test_a_cache_through_its_life(csa, Hq, Hkv, D, page):
    s = Server(csa, 8, Hq, Hkv, D, page, pool=120, cap=20)
    s.run([37, 0, 130, 1, 0, 0, 0, 0])            # prompts begin
    s.run([100, 0, 70, 1, 3, 0, 0, 0])            # go on, decode, begin
    s.counts()
    # slots 5 and 6 become copies of 2, slot 7 of 0; the copies hold the same values
    csa.csa_pages_fork(s.book, i32([-1, -1, -1, -1, -1, 2, 2, 0]), s.src, s.dst, s.pages_ws)
    s.copy()
    assert csa.csa_check_status() == 0
    for c in s.layers:
        for a, b in ((2, 5), (2, 6), (0, 7)):
            for x, y in zip(s.tokens(c, a), s.tokens(c, b)):
                assert torch.equal(x, y)
    kept = [s.tokens(c, 2) for c in s.layers]
    s.run([0, 0, 0, 1, 1, 5, 1, 40])              # the copies go on apart
    for c, was in zip(s.layers, kept):
        for x, y in zip(s.tokens(c, 2), was):
            assert torch.equal(x, y)
    s.counts()
    # slot 6 is cut back into a page that it shares, slot 0 ends; then both 6 and 2 go on
    csa.csa_pages_resize(s.book, i32([0, -1, -1, -1, -1, -1, page + 3, -1]), None, None, None, s.pages_ws)
    s.counts()
    s.run([0, 9, 2, 0, 0, 0, 4, 0])
    for c, was in zip(s.layers, kept):
        for x, y in zip(s.tokens(c, 2), was):
            assert torch.equal(x[:len(y)], y)
    s.counts()
    # the pool compacted: the same values, and the same attention to the bit
    before = [[s.tokens(c, b) for b in range(8)] for c in s.layers]
    q = [x[:, :Hq].contiguous() for x in s.project(8)]
    def decode():
        out = []
        for c, x in zip(s.layers, q):
            o, lse = torch.empty(8, Hq, D, device=DEV).bfloat16(), torch.empty(8, Hq, device=DEV)
            csa.csa_paged_attn(c, s.lens, x, D ** -0.5, 0, None, o, lse, s.decode_ws)
            o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
            csa.csa_chunk_attn(c, i32(list(range(9))), s.lens, x, D ** -0.5, 0, None, o2, lse2, s.ws)
            out += [o, lse, o2, lse2]
        return out
    results = decode()
    src, dst = (torch.empty(60, dtype=torch.int32, device=DEV) for _ in range(2))
    used = torch.empty(1, dtype=torch.int32, device=DEV)
    csa.csa_pages_compact(s.book, src, dst, used, s.table, s.refs, s.pages_ws)
    for c in s.layers:
        csa.csa_pages_copy(c, src, dst)
    assert csa.csa_check_status() == 0
    assert int((s.refs > 0).sum()) == int(used) and (s.refs[:int(used)] > 0).all()
    s.counts()
    for c, was in zip(s.layers, before):
        for b in range(8):
            for x, y in zip(s.tokens(c, b), was[b]):
                assert torch.equal(x, y)
    for x, y in zip(results, decode()):
        assert torch.equal(x, y)
    s.run([0, 1, 30, 0, 2, 1, 0, 1])
    csa.csa_pages_resize(s.book, i32([0] * 8), None, None, None, s.pages_ws)
    assert csa.csa_check_status() == 0 and (s.refs == 0).all()


def test_a_captured_step_replays(csa):
    """Growth by one token a slot, its append and its attention as one graph: replays equal eager steps bit for bit."""
    def fresh():
        s = Server(csa, 3, 8, 2, 128, 16, pool=40, cap=12, layers=1, seed=5)
        s.run([30, 47, 0])
        return s
    a, b = fresh(), fresh()
    cu, target = i32([0, 1, 2, 2]), i32([31, 48, -1])
    qkv = [torch.zeros(2, 12, 128, device=DEV).bfloat16()]
    out = [(torch.zeros(2, 8, 128, device=DEV).bfloat16(), torch.zeros(2, 8, device=DEV))]
    inputs = [torch.randn(2, 12, 128, device=DEV).bfloat16() for _ in range(6)]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        b.step(None, qkv, target, cu, out)
    for i, x in enumerate(inputs):
        t = i32([31 + i, 48 + i, -1])
        o = [(torch.zeros_like(out[0][0]), torch.zeros_like(out[0][1]))]
        a.step(None, [x], t, cu, o)
        qkv[0].copy_(x)
        target.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o[0][0], out[0][0]) and torch.equal(o[0][1], out[0][1])
        for u, v in ((a.table, b.table), (a.lens, b.lens), (a.refs, b.refs)):
            assert torch.equal(u, v)
    assert csa.csa_check_status() == 0
