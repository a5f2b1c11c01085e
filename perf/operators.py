"""What is measured of the grouped-query layer's operators: rotary positions,
the append into the paged 8-bit cache, single-token attention over that cache,
and causal attention over packed prompts.

Every operator has its plain form here (elementary torch operations in 32 bits,
64 where angles or borders need it), its definition in 64 bits (`exact`), and
the framework's own calls (`own`).
"""
import math
import random

import numpy as np
import torch

own = False

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


# ---- cases ---------------------------------------------------------------------

def rope(name, tokens, heads, dim, rope_dim, offset, layout, scaling, inverse, far):
    c = dict(op="rope", tokens=tokens, heads=heads, dim=dim, rope_dim=rope_dim, offset=offset, layout=layout,
             scaling=scaling, inverse=inverse, far=far)
    return dict(c, name=name) if name else c


def append(name, seqs, longest, mix, kv_heads, dim, page, far):
    c = dict(op="append", seqs=seqs, longest=longest, mix=mix, kv_heads=kv_heads, dim=dim, page=page, far=far)
    return dict(c, name=name) if name else c


def paged(name, seqs, longest, mix, heads, kv_heads, dim, page, window, sink):
    c = dict(op="paged", seqs=seqs, longest=longest, mix=mix, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
             window=window, sink=sink)
    return dict(c, name=name) if name else c


def prompt(name, seqs, longest, mix, prefix, heads, kv_heads, dim, window, sink):
    c = dict(op="prompt", seqs=seqs, longest=longest, mix=mix, prefix=prefix, heads=heads, kv_heads=kv_heads,
             dim=dim, window=window, sink=sink)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decoded token's queries: the smallest call
        rope("rope-1-token", 1, 32, 128, 128, 0, "half", "none", False, 8192),
        # a packed batch's gradient through a partial rotation (the last 64 of 192 channels), stretched to a
        # million positions
        rope("rope-1003-partial-inverse", 1003, 24, 192, 64, 128, "interleaved", "parts", True, 1 << 20),
        # queries and keys of a long prompt out of one fused projection
        rope("rope-16k-prompt", 16384, 72, 128, 128, 0, "half", "none", False, 131072),
        # one decoded token of one sequence
        append("append-1-token", 1, 1, 0, 8, 128, 64, 5000),
        # a decode step of 128 sequences, short pages
        append("append-128-tokens", 128, 1, 0, 8, 64, 16, 2000),
        # the prompts of a serving batch
        append("append-5-prompts", 5, 6144, 1, 8, 128, 64, 4096),
        # one user's chat
        paged("paged-1x900", 1, 900, 0, 32, 8, 128, 64, 0, False),
        # a batch of mixed lengths with a sliding window's layer beside it: short pages, attention sinks
        paged("paged-96-window", 96, 16384, 2, 64, 8, 64, 16, 4096, True),
        # a full serving batch of mixed lengths
        paged("paged-64-mixed", 64, 32768, 3, 64, 8, 128, 64, 0, False),
        # a chunk of a prompt after what is already there
        prompt("prompt-chunk-200", 1, 200, 0, 900, 32, 8, 128, 0, False),
        # packed prompts of different lengths under a window, with sinks
        prompt("prompt-16-packed", 16, 2500, 4, 0, 32, 8, 64, 1024, True),
        # one long prompt
        prompt("prompt-1x16k", 1, 16384, 0, 0, 32, 4, 128, 0, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["rope", "append", "paged", "prompt"])
    mix = rng.randrange(1 << 20)
    if op == "rope":
        dim = rng.choice([64, 96, 128, 192, 256])
        rope_dim = rng.choice([r for r in (32, 64, 96, 128, 192, 256) if r <= dim])
        heads = rng.randint(1, 72)
        tokens = min(_log(rng, 1, 16384), 16384 * 72 * 128 // (heads * dim))
        return rope(None, tokens, heads, dim, rope_dim, rng.choice([0, dim - rope_dim]),
                    rng.choice(["half", "interleaved"]), rng.choice(["none", "linear", "parts"]),
                    rng.random() < 0.3, _log(rng, 4096, 1 << 21))
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "append":
        seqs = _log(rng, 1, 256)
        longest = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, 16384 // seqs))
        return append(None, seqs, longest, mix, kv_heads, dim, rng.choice([16, 32, 64, 128]),
                      _log(rng, 64, 262144 // seqs))
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8, 12, 16])
    window, sink = rng.choice([0, 0, 128, 1000, 4096]), rng.random() < 0.4
    if op == "paged":
        seqs = _log(rng, 1, 64)
        longest = min(_log(rng, 1, 32768), 1200000000 // (seqs * kv_heads * dim))
        return paged(None, seqs, longest, mix, heads, kv_heads, dim,
                     rng.choice([16, 32, 64, 128]), window, sink)
    longest = _log(rng, 1, 8192)
    prefix = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    while heads * dim * longest * (longest + 2 * prefix) > 16384 * 16384 * 32 * 128:
        longest, prefix = longest * 3 // 4, prefix * 3 // 4
    most = 32 * 16384 * 16384 // 4 // (heads * longest * (longest + prefix))
    return prompt(None, max(1, min(_log(rng, 1, 24), most)), longest, mix, prefix, heads, kv_heads, dim, window, sink)


def lengths(case):
    """The case's sequence lengths: the longest once, the others spread below it."""
    if case["mix"] == 0:
        return [case["longest"]] * case["seqs"]
    r = random.Random(case["mix"])
    return [case["longest"]] + [r.randint(max(1, case["longest"] // 16), case["longest"])
                                for _ in range(case["seqs"] - 1)]


def starts(case):
    """Positions of an append's first new rows."""
    r = random.Random(case["mix"] + 7)
    return [r.randint(0, case["far"]) for _ in range(case["seqs"])]


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 4 * n * case["dim"] + 4 * case["tokens"], "flops": 3 * n * case["rope_dim"]}
    D = case["dim"]
    L = lengths(case)
    if op == "append":  # rows in as bf16, codes out, a scale for each page and head touched
        n, P = sum(L), case["page"]
        pages = sum((s + x - 1) // P - s // P + 1 for s, x in zip(starts(case), L))
        return {"bytes": case["kv_heads"] * (n * D * 2 * 3 + pages * 2 * 4), "flops": 6 * n * case["kv_heads"] * D}
    W = case["window"]
    if op == "paged":
        n = sum(min(x, W) if W else x for x in L)
        rows = case["seqs"] * case["heads"]
        return {"bytes": n * case["kv_heads"] * 2 * D + rows * (4 * D + 4), "flops": 4 * D * case["heads"] * n}
    pairs = 0
    for x in L:
        i = np.arange(x, dtype=np.int64) + case["prefix"] + 1
        pairs += int((np.minimum(i, W) if W else i).sum())
    nq, nk = sum(L), sum(L) + case["prefix"] * case["seqs"]
    return {"bytes": nq * case["heads"] * (4 * D + 4) + nk * case["kv_heads"] * 4 * D,
            "flops": 4 * D * case["heads"] * pairs}


# ---- inputs ----------------------------------------------------------------------

def rope_kwargs(case):
    """The rotation of a case: base 1e4 as trained, stretched 16 times from 65536 positions where it is scaled."""
    kinds = {"none": 0, "linear": 1, "parts": 2}
    return dict(rope_dim=case.get("rope_dim", case["dim"]), offset=case.get("offset", 0),
                layout=1 if case.get("layout", "half") == "half" else 0, scaling=kinds[case.get("scaling", "none")],
                theta=1e4, factor=16.0, orig_len=65536, beta_fast=32.0, beta_slow=1.0,
                mscale=1.25 if case.get("scaling") == "parts" else 1.0)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(case, g, cap):
    """A pool of pages in shuffled order, filled with rows of about unit size: codes, a scale for each page and
    head, and each sequence's table."""
    B, H, D, P = case["seqs"], case["kv_heads"], case["dim"], case["page"]
    per = -(-cap // P)
    n = B * per + 3
    s = {}
    for x in ("k", "v"):
        e = torch.randint(-7, -4, (n, H), device="cuda", generator=g)
        s[x + "_scale"] = torch.exp2(e.float())
        s[x] = torch.empty(n, H, P, D, dtype=F8, device="cuda")
        for i in range(0, n, 8192):
            r = torch.randn(min(8192, n - i), H, P, D, device="cuda", generator=g)
            s[x][i:i + 8192] = (r / s[x + "_scale"][i:i + 8192, :, None, None]).clamp_(-448, 448).to(F8)
    s["table"] = torch.randperm(n, device="cuda", generator=g)[:B * per].int().view(B, per).contiguous()
    return s


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, device="cuda", generator=g).to(BF16)  # noqa: E731
    op = case["op"]
    s = {"case": case}
    if op == "rope":
        T, H, D = case["tokens"], case["heads"], case["dim"]
        s["x"] = randn(T, H + 2, D)[:, :H]  # the heads of a wider projection's rows
        s["pos"] = torch.randint(0, case["far"], (T,), device="cuda", generator=g, dtype=torch.int32)
        s["out"] = torch.empty(T, H, D, dtype=BF16, device="cuda")
    elif op == "append":
        L, S = lengths(case), starts(case)
        H, D = case["kv_heads"], case["dim"]
        s.update(_cache(case, g, max(a + b for a, b in zip(L, S))))
        kv = randn(sum(L), 2 * H, D)
        s["new_k"], s["new_v"] = kv[:, :H], kv[:, H:]
        s["new_k"][:, :, 1] *= 6  # a few channels of keys are far larger than the rest
        s["cu"] = _i32(np.concatenate([[0], np.cumsum(L)]))
        s["pos0"] = _i32(S)
    elif op == "paged":
        L = lengths(case)
        s.update(_cache(case, g, max(L)))
        s["q"] = randn(case["seqs"], case["heads"], case["dim"])
        s["lens"] = _i32(L)
    else:
        L = lengths(case)
        n, m, D = sum(L), sum(L) + case["prefix"] * case["seqs"], case["dim"]
        s["q"], s["k"], s["v"] = randn(n, case["heads"], D), randn(m, case["kv_heads"], D), randn(m, case["kv_heads"], D)
        s["cu_q"] = _i32(np.concatenate([[0], np.cumsum(L)]))
        s["cu_k"] = _i32(np.concatenate([[0], np.cumsum([x + case["prefix"] for x in L])]))
        s["longest"] = max(L)
    if op in ("paged", "prompt"):
        s["sm_scale"] = case["dim"] ** -0.5
        s["sink"] = torch.randn(case["heads"], device="cuda", generator=g) if case["sink"] else None
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], device="cuda")
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program keeps beside its tensors: the rotation's table, the cache's description, the workspace."""
    import compressed_sparse_attention_02_gb300 as csa
    c = s["case"]
    s["csa"] = csa
    if c["op"] in ("rope", "append"):
        s["rope"] = csa.rope_params(**rope_kwargs(c))
        s["turns"] = csa.rope_table(s["rope"])
    if c["op"] in ("append", "paged"):
        s["cache"] = csa.paged_cache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"])
    if c["op"] == "paged":
        s["ws"] = csa.paged_attn_workspace(s["cache"], c["seqs"], c["heads"])


# ---- one pass ----------------------------------------------------------------------

def run(s):
    c, op = s["case"], s["case"]["op"]
    if own:
        csa = s["csa"]
        if op == "rope":
            csa.csa_rope(s["rope"], s["turns"], s["pos"], s["x"], s["out"], inverse=c["inverse"])
            return s["out"]
        if op == "append":
            csa.csa_kv_append(s["cache"], s["rope"], s["turns"], s["cu"], s["pos0"], s["new_k"], s["new_v"])
            return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
        if op == "paged":
            csa.csa_paged_attn(s["cache"], s["lens"], s["q"], s["sm_scale"], c["window"], s["sink"], s["out"],
                               s["lse"], s["ws"])
            return s["out"], s["lse"]
        csa.csa_prompt_attn(s["cu_q"], s["cu_k"], s["q"], s["k"], s["v"], s["sm_scale"], True, c["window"],
                            s["sink"], s["out"], s["lse"])
        return s["out"], s["lse"]
    if op == "rope":
        return _rope(s["x"], s["pos"], rope_kwargs(c), c["inverse"])
    return {"append": _append, "paged": _paged, "prompt": _prompt}[op](s, c)


def _freqs(r, device):
    """Radians a position of each pair, in 64 bits."""
    R = r["rope_dim"]
    j = torch.arange(R // 2, dtype=torch.float64, device=device)
    f = r["theta"] ** (-2 * j / R)
    if r["scaling"] == 1:
        return f / r["factor"]
    if r["scaling"] == 2:
        at = lambda b: R * math.log(r["orig_len"] / (b * 2 * math.pi)) / (2 * math.log(r["theta"]))  # noqa: E731
        low, high = max(math.floor(at(r["beta_fast"])), 0), min(math.ceil(at(r["beta_slow"])), R - 1)
        g = ((j - low) / max(high - low, 1e-3)).clamp(0, 1)
        return f * (1 - g) + f / r["factor"] * g
    return f


def _rotated(x, pos, r, inverse=False):
    a = pos.double()[:, None, None] * _freqs(r, x.device)
    if inverse:
        a = -a
    cos, sin = (a.cos() * r["mscale"]).float(), (a.sin() * r["mscale"]).float()
    R, o = r["rope_dim"], r["offset"]
    y = x.float()
    part = y[..., o:o + R]
    if r["layout"]:
        u, v = part[..., :R // 2].clone(), part[..., R // 2:].clone()
    else:
        u, v = part[..., 0::2].clone(), part[..., 1::2].clone()
    u, v = u * cos - v * sin, u * sin + v * cos
    part = torch.cat([u, v], -1) if r["layout"] else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([y[..., :o], part, y[..., o + R:]], -1)


def _rope(x, pos, r, inverse):
    return _rotated(x, pos, r, inverse).to(BF16)


def _append(s, c):
    P, cu, pos0 = c["page"], s["cu"].long(), s["pos0"].long()
    T = s["new_k"].shape[0]
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(cu[1:], t, right=True)
    pos = pos0[seq] + t - cu[seq]
    slot, at = s["table"][seq, pos // P].long(), pos % P
    new = {"k": _rotated(s["new_k"], pos, rope_kwargs(c)), "v": s["new_v"].float()}
    touched, row_of = torch.unique(slot, return_inverse=True)
    # rows of a sequence's first page that were there before
    kept = torch.zeros(len(touched), dtype=torch.long, device="cuda")
    some = cu[1:] > cu[:-1]
    first = cu[:-1].clamp(max=T - 1)
    kept.scatter_reduce_(0, row_of[first], torch.where(some, pos0 % P, 0), "amax")
    for x in ("k", "v"):
        amax = torch.zeros(len(touched), c["kv_heads"], device="cuda")
        amax.index_reduce_(0, row_of, new[x].abs().amax(-1), "amax")
        f, e = torch.frexp(amax)  # the least power of two that holds 448 times as much: 448 = 0.875 * 2^9
        e = torch.where(amax > 0, e - 8 - (f <= 0.875).int(), -126).clamp(min=-126)
        was = s[x + "_scale"][touched]
        scale = torch.maximum(torch.exp2(e.float()), torch.where(kept[:, None] > 0, was, 0))
        codes = s[x][touched].float()
        old = torch.arange(P, device="cuda") < kept[:, None]
        codes = torch.where(old[:, None, :, None], codes * (was / scale)[:, :, None, None], codes).to(F8)
        codes.view(torch.uint8)[row_of, :, at] = (new[x] / scale[row_of][..., None]).to(F8).view(torch.uint8)
        s[x].view(torch.uint8)[touched] = codes.view(torch.uint8)
        s[x + "_scale"][touched] = scale
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _softmax(x, seen, sink, values):
    """(weights . values, log of the sum) of logits x [..., n] where `seen`, with a sink logit in the sum; rows that
    see nothing give 0."""
    x.masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    if sink is not None:
        m = torch.maximum(m, sink)
    m = m.clamp(min=-3e38)
    x.sub_(m).exp_()
    n = x.sum(-1, keepdim=True)
    if sink is not None:
        n = n + (sink - m).exp()
    o = torch.where(n > 0, torch.matmul(x, values) / n, 0)
    return o, (m + n.log())[..., 0]


def _paged(s, c):
    B, H, D, G = c["seqs"], c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    k, v = ((s[x].view(torch.uint8)[s["table"].long()].view(F8).float() *
             s[x + "_scale"][s["table"].long()][..., None, None]).transpose(1, 2).reshape(B, H, -1, D)
            for x in ("k", "v"))
    q = s["q"].float().view(B, H, G, D) * s["sm_scale"]
    j, n = torch.arange(k.shape[2], device="cuda"), s["lens"][:, None, None, None]
    seen = (j < n) & (j >= (n - c["window"] if c["window"] else 0))
    sink = s["sink"].view(H, G, 1) if c["sink"] else None
    o, lse = _softmax(q @ k.transpose(-1, -2), seen, sink, v)
    return o.reshape(B, -1, D).to(BF16), lse.reshape(B, -1)


def _prompt(s, c):
    B, H, D, G = c["seqs"], c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    Lq, Lk = s["longest"], s["longest"] + c["prefix"]
    i, j = torch.arange(Lq, device="cuda"), torch.arange(Lk, device="cuda")
    nq, nk = (cu_q[1:] - cu_q[:-1])[:, None], (cu_k[1:] - cu_k[:-1])[:, None]
    at_q, at_k = (cu_q[:-1, None] + i).clamp(max=s["q"].shape[0] - 1), (cu_k[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
    q = (s["q"].float() * s["sm_scale"])[at_q].view(B, Lq, H, G, D).permute(0, 2, 3, 1, 4)
    k, v = (s[x].float()[at_k].transpose(1, 2)[:, :, None] for x in ("k", "v"))
    last = (i + nk - nq)[:, None, None, :, None]
    seen = (j <= last) & (j < nk[:, None, None, :, None])
    if c["window"]:
        seen &= j > last - c["window"]
    sink = s["sink"].view(H, G, 1, 1) if c["sink"] else None
    o, lse = _softmax(q @ k.transpose(-1, -2), seen, sink, v)
    there = i < nq
    o, lse = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[there], lse.permute(0, 3, 1, 2).flatten(2, 3)[there]
    return o.to(BF16), lse


# ---- the definitions in 64 bits -----------------------------------------------------

def _turned(x, pos, r, inverse):
    """Rows x (numpy, 64 bits) with each pair as a complex number times c e^(i p f)."""
    R, o = r["rope_dim"], r["offset"]
    f = []
    for j in range(R // 2):
        w = r["theta"] ** (-2.0 * j / R)
        if r["scaling"] == 1:
            w /= r["factor"]
        elif r["scaling"] == 2:
            lo, hi = (R * math.log(r["orig_len"] / (2 * math.pi * b)) / (2 * math.log(r["theta"]))
                      for b in (r["beta_fast"], r["beta_slow"]))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), R - 1)
            share = min(max((j - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            w = (1 - share) * w + share * w / r["factor"]
        f.append(-w if inverse else w)
    z = np.exp(1j * pos.astype(np.float64)[:, None] * np.array(f))[:, None, :] * r["mscale"]
    at = [(o + j, o + j + R // 2) if r["layout"] else (o + 2 * j, o + 2 * j + 1) for j in range(R // 2)]
    a, b = np.array(at).T
    w = (x[..., a] + 1j * x[..., b]) * z
    y = x.copy()
    y[..., a], y[..., b] = w.real, w.imag
    return y


def exact(case, seed):
    op = case["op"]
    if op in ("rope", "append") and work(case)["bytes"] > 1.5e8:
        return None
    s = prepare(case, seed)
    if op == "rope":
        return torch.from_numpy(_turned(s["x"].double().cpu().numpy(), s["pos"].cpu().numpy(), rope_kwargs(case),
                                        case["inverse"]))
    if op == "append":
        return _exact_append(s, case)
    return _exact_paged(s, case) if op == "paged" else _exact_prompt(s, case)


def _exact_append(s, case):
    """Sequence by sequence and page by page, on the host."""
    P, table = case["page"], s["table"].cpu().numpy()
    L, S = lengths(case), starts(case)
    pos = np.concatenate([np.arange(a, a + n) for a, n in zip(S, L)])
    rows = {"k": _turned(s["new_k"].double().cpu().numpy(), pos, rope_kwargs(case), False),
            "v": s["new_v"].double().cpu().numpy()}
    out = {}
    for x in ("k", "v"):
        codes, scale = s[x].cpu().double().numpy(), s[x + "_scale"].cpu().double().numpy()
        end = 0
        for b, (a, n) in enumerate(zip(S, L)):
            at, end = end, end + n
            p = a
            while p < a + n:
                page, first = table[b, p // P], p % P
                take = min(P - first, a + n - p)
                new = rows[x][at:at + take].transpose(1, 0, 2)
                big = np.abs(new).max(axis=(1, 2))
                e = np.maximum(np.ceil(np.log2(np.maximum(big, 1e-300) / 448)), -126)
                sc = 2.0 ** e
                if first:
                    sc = np.maximum(sc, scale[page])
                    codes[page, :, :first] = _e4m3(codes[page, :, :first] * (scale[page] / sc)[:, None, None])
                codes[page, :, first:first + take] = _e4m3(new / sc[:, None, None])
                scale[page] = sc
                p, at = p + take, at + take
        out[x], out[x + "_scale"] = torch.from_numpy(codes), torch.from_numpy(scale)
    return out


def _e4m3(x):
    """The nearest E4M3 value, ties to the even one (steps of 2^(e-3), 2^-9 below 2^-6)."""
    e = np.maximum(np.frexp(np.abs(x))[1] - 1, -6)
    step = 2.0 ** (e - 3)
    return np.rint(x / step) * step


def _weighted(x, sink, v):
    """softmax(x).v with a sink logit [rows], rows x keys in 64 bits; log of the sum."""
    both = x if sink is None else torch.cat([x, sink[:, None]], 1)
    lse = torch.logsumexp(both, 1)
    return torch.exp(x - lse[:, None]) @ v, lse


def _exact_paged(s, case):
    H, G, P = case["kv_heads"], case["heads"] // case["kv_heads"], case["page"]
    out, lses = [], []
    for b, n in enumerate(lengths(case)):
        lo = max(0, n - case["window"]) if case["window"] else 0
        pages = s["table"][b, lo // P:(n - 1) // P + 1].long()
        for h in range(H):
            k, v = ((s[x].view(torch.uint8)[pages, h].view(F8).double() *
                     s[x + "_scale"][pages, h].double()[:, None, None]).flatten(0, 1)[lo % P:lo % P + n - lo]
                    for x in ("k", "v"))
            rows = slice(h * G, h * G + G)
            o, lse = _weighted(s["q"][b, rows].double() @ k.T * s["sm_scale"],
                               s["sink"][rows].double() if case["sink"] else None, v)
            out.append(o)
            lses.append(lse)
    return torch.cat(out).view(s["q"].shape), torch.cat(lses).view(s["lse"].shape)


def _exact_prompt(s, case):
    if work(case)["flops"] > 3e12:  # 64-bit products of this size take too long
        return None
    G, W = case["heads"] // case["kv_heads"], case["window"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lses = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for n in lengths(case):
        m = n + case["prefix"]
        for a in range(0, n, 1024):  # a stretch of queries and the keys that any of them sees
            z = min(a + 1024, n)
            lo, hi = max(0, a + m - n - W + 1) if W else 0, z + m - n
            i, j = torch.arange(a, z, device="cuda")[:, None] + m - n, torch.arange(lo, hi, device="cuda")
            gone = (j > i) | (j <= i - W if W else False)
            for h in range(case["heads"]):
                k, v = s["k"][k0 + lo:k0 + hi, h // G].double(), s["v"][k0 + lo:k0 + hi, h // G].double()
                x = (s["q"][q0 + a:q0 + z, h].double() @ k.T * s["sm_scale"]).masked_fill_(gone, -math.inf)
                sink = s["sink"][h].double().expand(z - a) if case["sink"] else None
                out[q0 + a:q0 + z, h], lses[q0 + a:q0 + z, h] = _weighted(x, sink, v)
        q0, k0 = q0 + n, k0 + m
    return out, lses
