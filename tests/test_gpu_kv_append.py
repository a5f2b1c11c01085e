"""csa_kv_append against the rotation, scale rule and E4M3 rounding in 64 bits."""
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


def pool(B, caps, H, D, P, seed=0, n_extra=3):
    """An empty pool (codes of NaN, scales of -1, which nothing may read) and tables of shuffled pages."""
    g = torch.Generator().manual_seed(seed)
    n = B * caps + n_extra
    k, v = (torch.full((n, H, P, D), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((n, H), -1.0, device=DEV) for _ in range(2))
    table = torch.randperm(n, generator=g)[:B * caps].int().view(B, caps)
    return k, v, ks, vs, table.to(DEV)


def values(codes):
    return codes.view(torch.float8_e4m3fn).to(torch.float32).double().cpu()


def step(y):
    """At least the distance of neighbouring codes around y."""
    return (y.abs() / 8).clamp(min=2.0 ** -9)


class Model:
    """The cache in 64 bits: the codes' values and scales of each page and head, updated as the header says."""

    def __init__(self, k, v, ks, vs, table):
        self.codes = {"k": values(k), "v": values(v)}
        self.scale = {"k": ks.double().cpu().clone(), "v": vs.double().cpu().clone()}
        self.slack = {x: torch.zeros_like(self.codes[x]) for x in "kv"}  # what a code may be off by: a step at a tie
        self.table = table.cpu()
        self.P = k.shape[2]

    def append(self, b, pos0, rows):
        """rows: {"k": [n][H][D] float64 rotated, "v": ..., "err": how far the kernel's rotated keys may be off}."""
        n = rows["k"].shape[0]
        t = 0
        while t < n:
            p = pos0 + t
            page, first = int(self.table[b, p // self.P]), p % self.P
            take = min(self.P - first, n - t)
            for x in "kv":
                new = rows[x][t:t + take].transpose(0, 1)  # [H][take][D]
                for h in range(new.shape[0]):
                    e = ref.scale_exp(float(new[h].abs().max()))
                    s = 2.0 ** e
                    if first:
                        was = float(self.scale[x][page, h])
                        s = max(s, was)
                        old = self.codes[x][page, h, :first] * (was / s)
                        self.codes[x][page, h, :first] = ref.e4m3(old)
                        if s != was:  # a code that fell on the other side may do so again
                            d = self.slack[x][page, h, :first]
                            self.slack[x][page, h, :first] = (d > 0) * (d * (was / s) + step(old))
                    y = new[h] / s
                    self.codes[x][page, h, first:first + take] = ref.e4m3(y)
                    err = rows["err"][t:t + take, h] / s if x == "k" and rows.get("err") is not None else 0.0
                    tie = ref.e4m3(y + err) != ref.e4m3(y - err)
                    self.slack[x][page, h, first:first + take] = tie * step(y)
                    self.scale[x][page, h] = s
            t += take

    def check(self, k, v, ks, vs):
        for x, codes, scale in (("k", k, ks), ("v", v, vs)):
            assert torch.equal(scale.double().cpu(), self.scale[x]), x
            got, want = values(codes), self.codes[x]
            both = torch.isnan(got) & torch.isnan(want)
            bad = ~both & ~((got - want).abs() <= self.slack[x])
            assert not bad.any(), "%s: %d codes differ, first at %s: %r, expected %r" % (
                x, bad.sum(), bad.nonzero()[0].tolist(), got[bad][0], want[bad][0])


def rows(n, H, D, seed, big=1.0, wide=True):
    g = torch.Generator(DEV).manual_seed(seed)
    kv = torch.randn(n, 2 * H + (1 if wide else 0), D, device=DEV, generator=g) * big
    kv = kv.bfloat16()
    return kv[:, :H], kv[:, H:2 * H]


def both(r, k, v, pos):
    """The rows as Model.append takes them."""
    if r is None:
        return {"k": k.double().cpu(), "v": v.double().cpu()}
    return {"k": ref.rope(r, k, pos), "v": v.double().cpu(), "err": ref.ROPE_ABS * ref.pair_size(r, k)}


@pytest.mark.parametrize("H,D,P,layout", [(1, 64, 16, 1), (2, 128, 16, 0), (3, 64, 32, 1), (8, 128, 32, 1),
                                          (2, 64, 64, 0), (2, 128, 64, 1), (1, 64, 128, None), (2, 128, 128, 1)])
def test_prompts_then_single_tokens(csa, H, D, P, layout):
    """Ragged prompts (one empty, one of a page, one that ends inside a page) at odd positions, a second stretch onto
    them with larger rows (the scales grow), then single tokens."""
    r = turns = None
    if layout is not None:
        r = csa.rope_params(rope_dim=D if D == 64 else 64, offset=0 if D == 64 else 32, layout=layout)
        turns = csa.rope_table(r)
    lens, pos0 = [5, 0, P, 2 * P + 3, 1], [0, 3, P, P - 1, 2 * P + 2]
    B = len(lens)
    k, v, ks, vs, table = pool(B, 8, H, D, P)
    m = Model(k, v, ks, vs, table)
    cache = csa.paged_cache(k, v, ks, vs, table)
    at = list(pos0)
    # a first token in front of those that start inside a page, so that what they read is written
    for b in range(B):
        if at[b] % P:
            n = at[b] % P
            a, c = rows(n, H, D, 100 + b, 0.5)
            p = torch.arange(at[b] - n, at[b])
            csa.csa_kv_append(csa.paged_cache(k, v, ks, vs, table[b:b + 1]), r, turns,
                              torch.tensor([0, n], dtype=torch.int32, device=DEV),
                              torch.tensor([at[b] - n], dtype=torch.int32, device=DEV), a, c)
            m.append(b, at[b] - n, both(r, a, c, p))
    m.check(k, v, ks, vs)
    for step, big in enumerate((1.0, 40.0)):
        n = sum(lens)
        a, c = rows(n + 2, H, D, step, big)  # two rows of padding behind the last sequence
        a[-2:], c[-2:] = float("nan"), float("nan")
        cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).int().to(DEV)
        csa.csa_kv_append(cache, r, turns, cu, torch.tensor(at, dtype=torch.int32, device=DEV), a, c)
        for b in range(B):
            s = slice(sum(lens[:b]), sum(lens[:b + 1]))
            p = torch.arange(at[b], at[b] + lens[b])
            if lens[b]:
                m.append(b, at[b], both(r, a[s], c[s], p))
            at[b] += lens[b]
        assert csa.csa_check_status() == 0
        m.check(k, v, ks, vs)
    for step in range(4):
        a, c = rows(B, H, D, 50 + step, 10.0 ** (step - 1))
        csa.csa_kv_append(cache, r, turns, None, torch.tensor(at, dtype=torch.int32, device=DEV), a, c)
        for b in range(B):
            p = torch.tensor([at[b]])
            m.append(b, at[b], both(r, a[b:b + 1], c[b:b + 1], p))
            at[b] += 1
        assert csa.csa_check_status() == 0
        m.check(k, v, ks, vs)


def test_scale_borders_and_special_values(csa):
    """Largest values next to 448 * 2^e, rows of zeros, subnormals, the largest bf16, NaN and infinities."""
    H, D, P = 1, 64, 16
    tops = [448.0, 450.0, 446.0, 0.0, 1e-40, 3.3895e38, 7.0, 0.875]
    B = len(tops)
    k, v, ks, vs, table = pool(B, 1, H, D, P)
    a = torch.zeros(B, H, D, device=DEV).bfloat16()
    a[:, 0, 5] = torch.tensor(tops, device=DEV).bfloat16()
    a[:, 0, 6] = -a[:, 0, 5] / 3
    c = a.clone()
    c[6, 0, 0], c[6, 0, 1], c[6, 0, 2] = float("nan"), float("inf"), -float("inf")
    m = Model(k, v, ks, vs, table)
    csa.csa_kv_append(csa.paged_cache(k, v, ks, vs, table), None, None, None,
                      torch.zeros(B, dtype=torch.int32, device=DEV), a, c)
    fin = c.double().cpu()
    fin[~torch.isfinite(fin)] = 0
    for b in range(B):
        m.append(b, 0, {"k": a[b:b + 1].double().cpu(), "v": fin[b:b + 1]})
    page = int(table[6, 0])
    m.codes["v"][page, 0, 0, :3] = torch.tensor([float("nan"), 448.0, -448.0])
    m.check(k, v, ks, vs)
    assert ks[int(table[3, 0]), 0] == 2.0 ** -126


def test_what_is_not_stored(csa):
    """Negative positions, tables that end, pages outside the pool, falling offsets: nothing but the good sequences'
    tokens is written."""
    H, D, P = 2, 64, 16
    B = 6
    k, v, ks, vs, table = pool(B, 2, H, D, P)
    table[2, 0] = -1
    table[3, 0] = k.shape[0]
    m = Model(k, v, ks, vs, table)
    a, c = rows(B, H, D, 3)
    pos = torch.tensor([0, -1, 4, 5, 2 * P, 17], dtype=torch.int32, device=DEV)
    cache = csa.paged_cache(k, v, ks, vs, table)
    ks[int(table[5, 1])] = 2.0 ** -6  # token 16 of sequence 5 stands for a row that was there
    vs[int(table[5, 1])] = 2.0 ** -6
    k[int(table[5, 1])] = 0
    v[int(table[5, 1])] = 0
    m = Model(k, v, ks, vs, table)
    csa.csa_kv_append(cache, None, None, None, pos, a, c)
    assert csa.csa_check_status() == 5
    for b in (0, 5):
        m.append(b, int(pos[b]), {"k": a[b:b + 1].double().cpu(), "v": c[b:b + 1].double().cpu()})
    m.check(k, v, ks, vs)
    # offsets that fall or pass the rows
    cu = torch.tensor([0, 3, 2, 4, 99, 99, 6], dtype=torch.int32, device=DEV)
    before = k.clone()
    csa.csa_kv_append(cache, None, None, cu, torch.full((B,), -1, dtype=torch.int32, device=DEV), a, c)
    csa.csa_kv_append(cache, None, None, cu, torch.full((B,), 2 * P - 1, dtype=torch.int32, device=DEV), a, c)
    assert csa.csa_check_status() == 5
    assert before.shape == k.shape


def test_many_sequences_and_a_pool_past_four_gigabytes(csa):
    """700 sequences of mixed lengths (several passes of the sequence search), into the last pages of a pool whose
    offsets pass 32 bits."""
    H, D, P, B = 4, 128, 32, 700
    n = 300000                      # 16 KiB a page: 4.9 GB for k, as much for v
    k, v = (torch.empty(n, H, P, D, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.ones(n, H, device=DEV) for _ in range(2))
    g = torch.Generator().manual_seed(9)
    table = (n - 1 - torch.randperm(2 * B, generator=g)).int().view(B, 2).to(DEV)
    lens = torch.randint(0, 40, (B,), generator=g)
    cu = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)]).int().to(DEV)
    a, c = rows(int(lens.sum()), H, D, 4)
    csa.csa_kv_append(csa.paged_cache(k, v, ks, vs, table), None, None, cu,
                      torch.zeros(B, dtype=torch.int32, device=DEV), a, c)
    assert csa.csa_check_status() == 0
    for b in range(0, B, 29):
        for p in range(0, int(lens[b]), P):
            page = int(table[b, p // P])
            take = min(P, int(lens[b]) - p)
            x = c[int(cu[b]) + p:int(cu[b]) + p + take].double().cpu().transpose(0, 1)
            s = vs[page].double().cpu()
            assert torch.equal(s, torch.tensor([2.0 ** ref.scale_exp(float(y.abs().max())) for y in x], dtype=F64))
            assert torch.equal(values(v[page, :, :take].contiguous()), ref.e4m3(x / s[:, None, None]))


def test_refusals(csa):
    H, D, P = 2, 64, 16
    k, v, ks, vs, table = pool(2, 2, H, D, P)
    cache = csa.paged_cache(k, v, ks, vs, table)
    a, c = rows(2, H, D, 1)
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    r = csa.rope_params(rope_dim=128)  # wider than the head
    for call in (lambda: csa.csa_kv_append(cache, r, csa.rope_table(r), None, pos, a, c),
                 lambda: csa.csa_kv_append(cache, None, None, None, pos[:1], a, c),
                 lambda: csa.csa_kv_append(cache, None, None, None, pos, a.float(), c),
                 lambda: csa.csa_kv_append(cache, None, None, pos, pos, a, c),
                 lambda: csa.csa_kv_append(cache, None, None, None, torch.zeros(3, dtype=torch.int32, device=DEV),
                                           torch.cat([a, a[:1]]), torch.cat([c, c[:1]])),
                 lambda: csa.paged_cache(k, v, ks[:1], vs, table),
                 lambda: csa.paged_cache(k, v, ks, vs, table.long())):
        with pytest.raises(csa.CsaError) as e:
            call()
        assert e.value.status == 1
    odd = csa.paged_cache(*(torch.zeros(3, H, 24, D, dtype=torch.uint8, device=DEV) for _ in range(2)), ks[:3].clone(),
                          vs[:3].clone(), table)
    with pytest.raises(csa.CsaError) as e:
        csa.csa_kv_append(odd, None, None, None, pos, a, c)
    assert e.value.status == 2
