"""csa_rope against the rotation in 64 bits."""
import pytest
import torch

import _gqa as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def csa():
    import compressed_sparse_attention_02_gb300 as m
    return m


def make(T, H, D, far, seed=0, extra=0):
    g = torch.Generator(DEV).manual_seed(seed)
    x = torch.randn(T, H + extra, D, device=DEV, generator=g).bfloat16()[:, :H]
    pos = torch.randint(0, far, (T,), device=DEV, generator=g, dtype=torch.int32)
    return x, pos


def check(r, got, x, pos, inverse=False):
    want = ref.rope(r, x, pos, inverse)
    tol = 2.0 ** -8 * want.abs() + ref.ROPE_ABS * ref.pair_size(r, x)
    off = (got.double().cpu() - want).abs()
    assert (off <= tol).all(), "off by %.3g of the tolerance" % (off / tol.clamp(min=1e-30)).max()


@pytest.mark.parametrize("T,H,D,rope_dim,offset,layout,scaling,inverse,extra", [
    (1, 1, 16, 16, 0, 1, 0, False, 0),
    (1, 32, 128, 128, 0, 1, 0, False, 0),
    (2, 7, 128, 64, 64, 0, 1, False, 3),
    (37, 5, 192, 64, 128, 0, 2, True, 2),
    (37, 5, 192, 96, 16, 1, 2, False, 0),
    (1000, 3, 64, 32, 0, 1, 2, True, 1),
    (601, 40, 128, 128, 0, 0, 0, False, 0),
    (3, 1024, 512, 512, 0, 1, 0, False, 0),
    (5, 33, 80, 48, 32, 1, 0, False, 0),
])
def test_rotation(csa, T, H, D, rope_dim, offset, layout, scaling, inverse, extra):
    r = csa.rope_params(rope_dim=rope_dim, offset=offset, layout=layout, scaling=scaling, factor=8.0, orig_len=2048,
                        theta=5e5 if scaling == 2 else 1e4, mscale=1.0 if scaling < 2 else 1.2)
    x, pos = make(T, H, D, 1 << 20, extra=extra)
    check(r, csa.csa_rope(r, csa.rope_table(r), pos, x, inverse=inverse), x, pos, inverse)
    assert csa.csa_check_status() == 0


def test_table_is_the_formula(csa):
    for kw in (dict(), dict(scaling=1, factor=4.0), dict(scaling=2, factor=16.0, orig_len=65536, theta=1e4),
               dict(rope_dim=64, scaling=2, factor=40.0, orig_len=4096)):
        r = csa.rope_params(**kw)
        turns = [t % (1 << 64) for t in csa.rope_table(r).tolist()]
        want = ref.freqs(r) / (2 * torch.pi)
        got = torch.tensor([t / 2.0 ** 64 for t in turns], dtype=torch.float64)
        assert ((got - want).abs() <= 1e-13 * want + 2.0 ** -63).all()


def test_far_positions_keep_their_angle(csa):
    r = csa.rope_params(rope_dim=64)
    x, _ = make(6, 2, 64, 2)
    pos = torch.tensor([0, 1, 2 ** 24 + 1, 2 ** 30 - 1, 2 ** 31 - 2, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    got = csa.csa_rope(r, csa.rope_table(r), pos, x).double().cpu()
    # the 64-bit oracle's own angle is good to 2^31 * 2^-53 rad; the table's to 2^31 * 2^-52
    want = ref.rope(r, x, pos)
    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + (ref.ROPE_ABS + 2e-6) * ref.pair_size(r, x)).all()


def test_in_place_and_views(csa):
    r = csa.rope_params(rope_dim=64, offset=32)
    turns = csa.rope_table(r)
    T, H, D = 77, 6, 128
    x, pos = make(T, H, D, 5000)
    want = csa.csa_rope(r, turns, pos, x)
    y = x.clone()
    assert csa.csa_rope(r, turns, pos, y, out=y) is y
    assert torch.equal(y, want)
    # heads outermost in memory, and the result into a slice of a wider buffer
    heads_first = x.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((T, H + 2, D), 7.0, device=DEV, dtype=torch.bfloat16)
    csa.csa_rope(r, turns, pos, heads_first, out=wide[:, 1:1 + H])
    assert torch.equal(wide[:, 1:1 + H], want)
    assert (wide[:, 0] == 7).all() and (wide[:, -1] == 7).all()


def test_negative_positions_leave_their_rows(csa):
    r = csa.rope_params()
    x, pos = make(9, 4, 128, 100)
    pos[3] = -1
    pos[8] = -2 ** 31
    out = torch.full_like(x, 3.0)
    csa.csa_rope(r, csa.rope_table(r), pos, x, out=out)
    keep = pos >= 0
    check(r, out[keep], x[keep], pos[keep])
    assert (out[~keep] == 3).all()


@pytest.mark.parametrize("layout", [0, 1])
def test_inverse_is_the_gradient(csa, layout):
    """<w, R x> = <R^T w, x> for the rotation R, and R^T's column sums are the differences of <w, R x> along a
    channel (R is linear: a difference of any size is exact but for the roundings)."""
    r = csa.rope_params(rope_dim=64, offset=16, layout=layout, mscale=1.5)
    turns = csa.rope_table(r)
    x, pos = make(40, 3, 96, 3000, seed=1)
    w, _ = make(40, 3, 96, 2, seed=2)
    y = csa.csa_rope(r, turns, pos, x).double().cpu()
    gx = csa.csa_rope(r, turns, pos, w, inverse=True).double().cpu()
    xd, wd = x.double().cpu(), w.double().cpu()
    # each side's terms carry one bf16 rounding
    slack = 2.0 ** -8 * ((wd * y).abs().sum() + (gx * xd).abs().sum())
    assert abs((wd * y).sum() - (gx * xd).sum()) <= slack
    for ch in (0, 16, 17, 48, 79, 80):
        x2 = x.clone()
        x2[..., ch] += 4.0
        h = (x2 - x).double().cpu()[..., ch]
        y2 = csa.csa_rope(r, turns, pos, x2).double().cpu()
        diff = (wd * (y2 - y)).sum(-1)
        slack = 2.0 ** -8 * ((wd * y).abs() + (wd * y2).abs()).sum(-1) + 2.0 ** -8 * (gx[..., ch] * h).abs()
        assert ((diff - gx[..., ch] * h).abs() <= slack + 1e-6).all()


def test_no_rows_and_refusals(csa):
    r = csa.rope_params(rope_dim=64)
    turns = csa.rope_table(r)
    x, pos = make(4, 2, 64, 10)
    csa.csa_rope(r, turns, pos[:0], x[:0])
    for bad in (dict(x=x.float()), dict(pos=pos.long()), dict(pos=pos[:3]), dict(turns=turns[:5]), dict(x=x.cpu()),
                dict(out=torch.empty(4, 2, 32, device=DEV, dtype=torch.bfloat16)),
                dict(x=x.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(x=torch.empty(4, 2, 68, device=DEV, dtype=torch.bfloat16)[..., :64])):
        kw = dict(r=r, turns=turns, pos=pos, x=x, out=None)
        kw.update(bad)
        with pytest.raises(csa.CsaError) as e:
            csa.csa_rope(kw["r"], kw["turns"], kw["pos"], kw["x"], kw["out"])
        assert e.value.status == 1
