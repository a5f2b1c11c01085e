"""The grouped-query layer's operators in 64 bits on the host, written from
their formulas (include/csa.h), and the tolerances the kernels' roundings
allow.  Half a step of a rounding, relative to the value: bf16 2^-8, f16 2^-11,
fp32 2^-24, E4M3 2^-4 (2^-10 of the scale below its normal numbers)."""
import math

import torch

F64 = torch.float64


def freqs(r):
    """Radians a position of each pair (r: CsaRopeParams)."""
    R = r.rope_dim
    out = []
    for j in range(R // 2):
        f = r.theta ** (-2.0 * j / R)
        if r.scaling == 1:
            f /= r.factor
        elif r.scaling == 2:
            c = [R * math.log(r.orig_len / (2 * math.pi * b)) / (2 * math.log(r.theta)) for b in
                 (r.beta_fast, r.beta_slow)]
            low, high = max(math.floor(c[0]), 0), min(math.ceil(c[1]), R - 1)
            g = min(max((j - low) / max(high - low, 1e-3), 0.0), 1.0)
            f = f * (1 - g) + f / r.factor * g
        out.append(f)
    return torch.tensor(out, dtype=F64)


def rope(r, x, pos, inverse=False):
    """x [rows][heads][channels] -> rotated, float64."""
    x = x.to(F64).cpu().clone()
    a = pos.to(F64).cpu()[:, None, None] * freqs(r) * (-1 if inverse else 1)
    c, s = a.cos() * r.mscale, a.sin() * r.mscale
    R, o = r.rope_dim, r.offset
    if r.layout == 1:
        i, j = slice(o, o + R // 2), slice(o + R // 2, o + R)
    else:
        i, j = slice(o, o + R, 2), slice(o + 1, o + R, 2)
    u, v = x[..., i].clone(), x[..., j].clone()
    x[..., i], x[..., j] = u * c - v * s, u * s + v * c
    return x


def pair_size(r, x):
    """|first| + |second| of every channel's pair (0 outside the rotated part): what an error of the sine or cosine
    is multiplied by."""
    x = x.to(F64).cpu().abs()
    R, o = r.rope_dim, r.offset
    y = torch.zeros_like(x)
    if r.layout == 1:
        i, j = slice(o, o + R // 2), slice(o + R // 2, o + R)
    else:
        i, j = slice(o, o + R, 2), slice(o + 1, o + R, 2)
    y[..., i] = y[..., j] = (x[..., i] + x[..., j]) * abs(r.mscale)
    return y


# sincospif is good to 2 units in the last place (2^-23 at 1), the angle to
# 2.4e-8 rad; two products and a sum of three binary32 roundings: below 2^-21.
ROPE_ABS = 2.0 ** -21


def scale_exp(amax):
    """The least e >= -126 with amax <= 448 * 2^e."""
    e = -126
    if amax > 0:
        e = max(e, math.frexp(amax / 448.0)[1] - 1)
        while amax > 448.0 * 2.0 ** e:
            e += 1
    return e


def e4m3(x):
    """The nearest E4M3 value (float64 in and out, |x| <= 448), ties to even."""
    e = torch.frexp(x.abs())[1].to(F64) - 1
    step = torch.exp2(e.clamp(min=-6) - 3)
    return torch.round(x / step) * step


def attend(q, k, v, sm_scale, seen, sink=None):
    """One head: q [n][D], k and v [m][D], seen [n][m] bool -> (out, lse, A, Q): out and lse in float64, A the weighted
    mean of |v| (what a relative error of a weight is multiplied by), Q the largest sum of |q||k| sm_scale that is seen
    (what a relative error of a product is multiplied by).  What is not seen has no part in any sum."""
    n, D = q.shape
    out, lse = torch.zeros(n, D, dtype=F64), torch.full((n,), -math.inf, dtype=F64)
    A, Q = torch.zeros(n, D, dtype=F64), torch.zeros(n, dtype=F64)
    q, k, v = q.to(F64), k.to(F64), v.to(F64)
    for i in range(n):
        at = seen[i].nonzero()[:, 0]
        logits = (k[at] @ q[i]) * sm_scale
        every = logits if sink is None else torch.cat([logits, torch.tensor([float(sink)], dtype=F64)])
        if not len(every):
            continue
        lse[i] = torch.logsumexp(every, 0)
        if not len(at):
            continue
        p = torch.exp(logits - lse[i])
        out[i], A[i] = p @ v[at], p @ v[at].abs()
        Q[i] = (k[at].abs() @ q[i].abs()).max() * sm_scale
    return out, lse, A, Q


# An fp32 sum of up to 128 products, in whatever order and with truncation, is
# within 2^-16 of the sum of their magnitudes.
DOT = 2.0 ** -16


def check_attention(got, got_lse, want, lse, A, Q, weight_step, what):
    """got within the output's rounding, the weights' rounding (weight_step) and the logits' error (Q * DOT, once in
    the weight and once in the sum) of want; exps and sums of binary32 are inside 2^-16."""
    d = Q[..., None] * DOT
    tol = 2.0 ** -8 * want.abs() + A * (weight_step + 2 * d + 2.0 ** -16) * (1 + 2.0 ** -7) + 1e-30
    fine = torch.isfinite(want)
    got = got.to(F64).cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "%s: NaN in other places" % what
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), "%s: infinities" % what
    bad = ((got - want).abs() > tol) & fine
    assert not bad.any(), "%s: %d of %d outside, worst by %.3g" % (
        what, bad.sum(), bad.numel(), ((got - want).abs() / tol)[fine].max())
    if got_lse is not None:
        got_lse = got_lse.to(F64).cpu()
        empty = torch.isinf(lse)
        assert torch.equal(got_lse[empty], lse[empty]), "%s: lse of rows that see nothing" % what
        ok = torch.isfinite(lse)
        far = (got_lse - lse).abs()[ok] - (Q[ok] * DOT + 2.0 ** -18 * (1 + lse[ok].abs()))
        assert not ok.any() or far.max() <= 0, "%s: lse off by %.3g too much" % (what, far.max())
