"""What is measured of the paged cache's further operators: attention of a chunk
of new tokens over the cache, and the pages' bookkeeping: sequences that grow,
shrink and end, forks that share pages, the compaction of a pool, and the copy
of pages' contents that the last two leave to each layer's pool.

Every operator has its plain form here (elementary torch operations in 32
bits), its definition in 64 bits or in whole numbers on the host (`exact`), and
the framework's own calls (`own`).
"""
import math
import random

import numpy as np
import torch

own = False

BF16, F8, I32 = torch.bfloat16, torch.float8_e4m3fn, torch.int32


# ---- cases ---------------------------------------------------------------------

def chunk(name, seqs, new, cached, mix, singles, heads, kv_heads, dim, page, window, sink):
    c = dict(op="chunk", seqs=seqs, new=new, cached=cached, mix=mix, singles=singles, heads=heads, kv_heads=kv_heads,
             dim=dim, page=page, window=window, sink=sink)
    return dict(c, name=name) if name else c


def resize(name, seqs, longest, grow, mix, page, pool):
    c = dict(op="resize", seqs=seqs, longest=longest, grow=grow, mix=mix, page=page, pool=pool)
    return dict(c, name=name) if name else c


def fork(name, parents, children, longest, mix, page, pool):
    c = dict(op="fork", parents=parents, children=children, longest=longest, mix=mix, page=page, pool=pool)
    return dict(c, name=name) if name else c


def compact(name, seqs, longest, mix, page, pool):
    c = dict(op="compact", seqs=seqs, longest=longest, mix=mix, page=page, pool=pool)
    return dict(c, name=name) if name else c


def copy(name, pairs, listed_pairs, kv_heads, dim, page):
    c = dict(op="copy", pairs=pairs, listed_pairs=listed_pairs, kv_heads=kv_heads, dim=dim, page=page)
    return dict(c, name=name) if name else c


def listed():
    return [
        # five drafted tokens of one user's chat, looked at in one pass: the smallest call
        chunk("chunk-1x5", 1, 5, 900, 0, 0.0, 32, 8, 128, 64, 0, False),
        # a serving step: most sequences decode one token, some are in the middle of their prompts; a sliding window's
        # layer with attention sinks, short pages
        chunk("chunk-48-window", 48, 300, 16384, 5, 0.75, 64, 8, 64, 16, 4096, True),
        # a batch of prompts that share nothing, each some way in
        chunk("chunk-12-prompts", 12, 1000, 6000, 6, 0.0, 32, 8, 128, 64, 0, False),
        # one long document, a piece at a time
        chunk("chunk-1x2048-at-62k", 1, 2048, 63488, 0, 0.0, 32, 4, 128, 128, 0, False),
        # a decode step with drafts: 64 sequences give back what was rejected and take room for the next tokens
        resize("resize-64", 64, 4096, 8, 1, 64, 8192),
        # many sequences with short pages, some ending and some starting: the largest pool
        resize("resize-1024", 1024, 16384, 500, 2, 16, 1 << 20),
        # four beams of one prompt
        fork("fork-4-beams", 1, 4, 3000, 3, 64, 4096),
        # samples of a batch of prompts
        fork("fork-64-by-8", 64, 512, 8192, 4, 16, 1 << 17),
        # a pool of which some pages are free between others
        compact("compact-4k-pages", 48, 4096, 7, 64, 4096),
        compact("compact-512k-pages", 1024, 8192, 8, 16, 1 << 19),
        # the beams' last pages
        copy("copy-4-pages", 4, 8, 8, 128, 64),
        # what a compaction moves
        copy("copy-5000-pages", 5000, 8192, 8, 128, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["chunk", "chunk", "resize", "fork", "compact", "copy"])
    mix = rng.randrange(1, 1 << 20)
    page = rng.choice([16, 32, 64, 128])
    if op == "chunk":
        dim, kv_heads = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8, 12, 16])
        seqs, new, cached = _log(rng, 1, 64), _log(rng, 1, 2048), _log(rng, 1, 65536) - 1
        while seqs * new * (new + cached) * heads * dim > 2048 * 64512 * 32 * 128:
            seqs, new, cached = max(1, seqs * 3 // 4), max(1, new * 3 // 4), cached * 7 // 8
        cached = min(cached, 600000000 // (seqs * kv_heads * dim))
        return chunk(None, seqs, new, cached, mix, rng.choice([0.0, 0.0, 0.8]), heads, kv_heads, dim, page,
                     rng.choice([0, 0, 128, 1000, 4096]), rng.random() < 0.4)
    if op == "copy":
        kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        pairs = min(_log(rng, 1, 5000), 5000 * 8 * 64 * 128 // (kv_heads * dim * page))
        return copy(None, pairs, pairs * rng.choice([1, 1, 2, 3]) + rng.randint(0, 9), kv_heads, dim, page)
    pool = _log(rng, 500, 1 << 19)
    longest = max(1, min(_log(rng, 100, 32768), pool * page // 3))
    seqs = max(1, min(_log(rng, 1, 1024), pool * page // (longest + page) // 3))
    if op == "resize":
        return resize(None, seqs, longest, _log(rng, 1, 1000), mix, page, pool + 70 * seqs)
    if op == "compact":
        return compact(None, seqs, longest, mix, page, pool)
    per = rng.choice([1, 2, 4, 8])
    return fork(None, max(1, seqs // 2), max(1, seqs // 2) * per, longest, mix, page, pool + 4 * seqs)


def pages(tokens, page):
    return -(-tokens // page)


def chunk_lengths(case):
    """(new tokens, all tokens) of each sequence: the largest once, the others spread below it, a share of them with
    one new token."""
    r = random.Random(case["mix"])
    out = [(case["new"], case["new"] + case["cached"])]
    for _ in range(case["seqs"] - 1):
        n = 1 if r.random() < case["singles"] else r.randint(max(1, case["new"] // 8), case["new"])
        out.append((n, n + r.randint(case["cached"] // 16, case["cached"])))
    return out


def resize_lengths(case):
    """Lengths of the sequences before and after they grow: most by a few tokens, some from nothing."""
    r = random.Random(case["mix"])
    n, most = case["seqs"], case["longest"]
    before = [r.randint(1, most) for _ in range(n)]
    room = case["pool"] - sum(pages(x, case["page"]) for x in before) - 8 * n
    after = []
    for i in range(n):
        if r.random() < 0.15:
            room += pages(before[i], case["page"])
            before[i] = 0
        want = r.randint(1, most) if before[i] == 0 else before[i] + r.randint(0, case["grow"])
        extra = pages(want, case["page"]) - pages(before[i], case["page"])
        after.append(want if extra <= room else before[i])
        room -= extra if extra <= room else 0
    return before, after


def parent_lengths(case):
    r = random.Random(case["mix"])
    return [r.randint(1, case["longest"]) for _ in range(case["parents"])]


def compact_lengths(case):
    r = random.Random(case["mix"])
    left, out = case["pool"] - 1, []
    for _ in range(case["seqs"]):
        x = min(r.randint(0, case["longest"]), left * case["page"])
        left -= pages(x, case["page"])
        out.append(x)
    return out


def work(case):
    op, P = case["op"], case.get("page")
    if op == "chunk":
        D, W, flops, rows, keys = case["dim"], case["window"], 0, 0, 0
        for n, L in chunk_lengths(case):
            i = np.arange(L - n, L, dtype=np.int64) + 1
            flops += 4 * D * case["heads"] * int((np.minimum(i, W) if W else i).sum())
            rows += n * case["heads"]
            keys += (min(L, W + n - 1) if W else L) * case["kv_heads"]
        return {"bytes": rows * (4 * D + 4) + 2 * D * keys, "flops": flops}
    if op == "copy":  # codes and scales, once each way
        return {"bytes": case["pairs"] * case["kv_heads"] * (2 * P * case["dim"] + 8) * 2 + 8 * case["listed_pairs"],
                "flops": 0}
    if op == "resize":  # every page's count and two targets a sequence; entries and counts that change, both ways
        before, after = resize_lengths(case)
        moved = sum(pages(y, P) - pages(x, P) for x, y in zip(before, after))
        return {"bytes": 4 * case["pool"] + 24 * case["seqs"] + 2 * 12 * moved, "flops": 0}
    if op == "fork":  # every page's count, a row read and written for each child, the counts and the copies' list
        L = parent_lengths(case)
        own_pages = sum(pages(L[b % case["parents"]], P) for b in range(case["children"]))
        n = case["parents"] + case["children"]
        return {"bytes": 4 * case["pool"] + 12 * n + 12 * own_pages, "flops": 0}
    used = sum(pages(x, P) for x in compact_lengths(case))  # counts and tables, both ways
    return {"bytes": 8 * case["pool"] + 8 * used + 4 * case["pool"], "flops": 0}


# ---- inputs ----------------------------------------------------------------------

def _i32(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def _pool(n, H, P, D, g):
    """Pages filled with rows of about unit size: codes, a scale for each page and head."""
    s = {}
    for x in ("k", "v"):
        e = torch.randint(-7, -4, (n, H), device="cuda", generator=g)
        s[x + "_scale"] = torch.exp2(e.float())
        s[x] = torch.empty(n, H, P, D, dtype=F8, device="cuda")
        step = max(1, (1 << 28) // (H * P * D))
        for i in range(0, n, step):
            r = torch.randn(min(step, n - i), H, P, D, device="cuda", generator=g)
            s[x][i:i + step] = (r / s[x + "_scale"][i:i + step, :, None, None]).clamp_(-448, 448).to(F8)
    return s


def _book(lens, cap, page, pool, seed):
    """A table of shuffled pages, the sequences' lengths and the pages' counts."""
    r = np.random.default_rng(seed)
    n = [pages(x, page) for x in lens]
    order = r.permutation(pool)
    table, refs, at = np.full((len(lens), cap), -1, np.int32), np.zeros(pool, np.int32), 0
    for b, x in enumerate(n):
        table[b, :x] = order[at:at + x]
        at += x
    refs[order[:at]] = 1
    return dict(table=torch.from_numpy(table).cuda(), lens=_i32(lens), refs=torch.from_numpy(refs).cuda())


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    op, P = case["op"], case.get("page")
    s = {"case": case}
    if op == "chunk":
        L = chunk_lengths(case)
        B, D, H = case["seqs"], case["dim"], case["kv_heads"]
        per = [pages(t, P) for _, t in L]
        n = sum(per) + 3
        s.update(_pool(n, H, P, D, g))
        free = torch.randperm(n, device="cuda", generator=g).int()
        s["table"] = torch.full((B, max(per)), -1, dtype=I32, device="cuda")
        for b, at in enumerate(np.cumsum([0] + per[:-1])):
            s["table"][b, :per[b]] = free[at:at + per[b]]
        s["q"] = torch.randn(sum(x for x, _ in L), case["heads"], D, device="cuda", generator=g).to(BF16)
        s["cu"] = _i32(np.cumsum([0] + [x for x, _ in L]))
        s["lens"] = _i32([t for _, t in L])
        s["sm_scale"] = D ** -0.5
        s["sink"] = torch.randn(case["heads"], device="cuda", generator=g) if case["sink"] else None
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], device="cuda")
    elif op == "resize":
        before, after = resize_lengths(case)
        cap = max(pages(x, P) for x in before + after + [1])
        s.update(_book(before, cap, P, case["pool"], seed))
        s["before"], s["after"] = _i32(before), _i32(after)
        s["pos0"], s["src"], s["dst"] = (torch.empty(case["seqs"], dtype=I32, device="cuda") for _ in range(3))
    elif op == "fork":
        L = parent_lengths(case) + [0] * case["children"]
        s.update(_book(L, max(pages(x, P) for x in L), P, case["pool"], seed))
        n, m = case["parents"], case["children"]
        s["parent"] = _i32([-1] * n + [i % n for i in range(m)])
        s["none"] = _i32([-1] * n + [0] * m)
        s["src"], s["dst"] = (torch.empty(n + m, dtype=I32, device="cuda") for _ in range(2))
    elif op == "compact":
        L = compact_lengths(case)
        s.update(_book(L, max(pages(x, P) for x in L + [1]), P, case["pool"], seed))
        s["src"], s["dst"] = (torch.empty(case["pool"] // 2, dtype=I32, device="cuda") for _ in range(2))
        s["used"] = torch.empty(1, dtype=I32, device="cuda")
        s["new_table"], s["new_refs"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
    else:
        n, m = case["pairs"], case["listed_pairs"]
        s.update(_pool(2 * n + 1, case["kv_heads"], P, case["dim"], g))
        order = torch.randperm(2 * n + 1, device="cuda", generator=g).int()
        s["src"], s["dst"] = (torch.full((m,), -1, dtype=I32, device="cuda") for _ in range(2))
        s["src"][:n], s["dst"][:n] = order[:n], order[n:2 * n]
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program keeps beside its tensors: the cache's and the pages' description, workspaces."""
    import compressed_sparse_attention_02_gb300 as csa
    c = s["case"]
    s["csa"] = csa
    if c["op"] == "chunk":
        s["cache"] = csa.paged_cache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"])
        s["ws"] = csa.chunk_attn_workspace(s["cache"], c["heads"])
    elif c["op"] == "copy":
        table = torch.zeros(1, 1, dtype=I32, device="cuda")
        s["cache"] = csa.paged_cache(s["k"], s["v"], s["k_scale"], s["v_scale"], table)
    else:
        s["book"] = csa.page_book(s["table"], s["lens"], s["refs"], c["page"])
        s["ws"] = csa.pages_workspace(s["book"])


# ---- one pass ----------------------------------------------------------------------

def run(s):
    c, op = s["case"], s["case"]["op"]
    if op == "chunk":
        if not own:
            return _chunk(s, c)
        s["csa"].csa_chunk_attn(s["cache"], s["cu"], s["lens"], s["q"], s["sm_scale"], c["window"], s["sink"],
                                s["out"], s["lse"], s["ws"])
        return s["out"], s["lse"]
    if op == "copy":
        if own:
            s["csa"].csa_pages_copy(s["cache"], s["src"], s["dst"])
        else:
            _copy(s)
        return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if op == "resize":  # back to where they were, and on again: every pass leaves the same
        if own:
            s["csa"].csa_pages_resize(s["book"], s["before"], None, None, None, s["ws"])
            s["csa"].csa_pages_resize(s["book"], s["after"], s["pos0"], s["src"], s["dst"], s["ws"])
        else:
            _resize(s, s["before"], c["page"])
            s["pos0"], s["src"], s["dst"] = _resize(s, s["after"], c["page"])
        return {x: s[x] for x in ("table", "lens", "refs", "pos0", "src", "dst")}
    if op == "fork":  # the last step's children end, new ones start
        if own:
            s["csa"].csa_pages_resize(s["book"], s["none"], None, None, None, s["ws"])
            s["csa"].csa_pages_fork(s["book"], s["parent"], s["src"], s["dst"], s["ws"])
        else:
            _resize(s, s["none"], c["page"])
            s["src"], s["dst"] = _fork(s, c["page"])
        return {x: s[x] for x in ("table", "lens", "refs", "src", "dst")}
    if own:
        s["csa"].csa_pages_compact(s["book"], s["src"], s["dst"], s["used"], s["new_table"], s["new_refs"], s["ws"])
        return {x: s[x] for x in ("src", "dst", "used", "new_table", "new_refs")}
    return _compact(s, c["page"])


def _chunk(s, c):
    """Sequence by sequence, every head at once."""
    H, D, G, P, W = c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"], c["page"], c["window"]
    outs, lses, at = [], [], 0
    for b, (n, L) in enumerate(chunk_lengths(c)):
        first = max(0, L - n - W + 1) // P * P if W else 0  # (pages before every query's window)
        own_pages = s["table"][b, first // P:pages(L, P)].long()
        k, v = ((s[x].view(torch.uint8)[own_pages].view(F8).float() * s[x + "_scale"][own_pages][..., None, None])
                .transpose(0, 1).reshape(H, 1, -1, D)[:, :, :L - first] for x in ("k", "v"))
        q = (s["q"][at:at + n].float() * s["sm_scale"]).view(n, H, G, D).permute(1, 2, 0, 3)
        x = q @ k.transpose(-1, -2)
        i, j = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(first, L, device="cuda")
        x.masked_fill_((j > i) | (j <= i - W) if W else j > i, -math.inf)
        m = x.amax(-1, keepdim=True)
        sink = s["sink"].view(H, G, 1, 1) if c["sink"] else None
        if c["sink"]:
            m = torch.maximum(m, sink)
        x.sub_(m).exp_()
        total = x.sum(-1, keepdim=True)
        if c["sink"]:
            total = total + (sink - m).exp()
        outs.append(((x @ v) / total).permute(2, 0, 1, 3).reshape(n, -1, D))
        lses.append((m + total.log())[..., 0].permute(2, 0, 1).reshape(n, -1))
        at += n
    return torch.cat(outs).to(BF16), torch.cat(lses)


def _copy(s):
    there = (s["src"] >= 0).nonzero()[:, 0]
    src, dst = s["src"][there].long(), s["dst"][there].long()
    for x in ("k", "v"):
        codes = s[x].view(torch.uint8)
        codes[dst] = codes[src]
        s[x + "_scale"][dst] = s[x + "_scale"][src]


def _free_pages(refs):
    """Numbers of the free pages in order (and past them anything), how many there are."""
    free = refs <= 0
    rank = free.cumsum(0) - 1
    out = torch.zeros(len(refs) + 1, dtype=I32, device="cuda")
    out[torch.where(free, rank, len(refs))] = torch.arange(len(refs), dtype=I32, device="cuda")
    return out, free.sum()


def _resize(s, target, P):
    table, lens, refs = s["table"], s["lens"], s["refs"]
    n0 = (lens + P - 1) // P
    n1 = torch.where(target >= 0, (target + P - 1) // P, n0)
    free, count = _free_pages(refs)
    # a last page that is partly filled and has other holders is left to them
    last = table.gather(1, (lens // P).clamp(max=table.shape[1] - 1).long()[:, None])[:, 0]
    apart = (target > lens) & (lens % P > 0) & (refs[last.clamp(min=0).long()] > 1)
    from_ = n0 - apart.int()
    need = (n1 - from_).clamp(min=0).long()
    upto = need.cumsum(0)
    served = (upto <= count) | (need == 0)
    apart = apart & served
    j = torch.arange(table.shape[1], device="cuda")
    gone = (j >= n1[:, None]) & (j < n0[:, None]) | apart[:, None] & (j == from_[:, None])
    taken = (j >= from_[:, None]) & (j < n1[:, None]) & served[:, None]
    page = free[torch.where(taken, (upto - need)[:, None] + j - from_[:, None], 0)]
    refs.index_add_(0, torch.where(gone, table, 0).flatten().long(), -gone.flatten().int())
    refs.index_add_(0, torch.where(taken, page, 0).flatten().long(), taken.flatten().int())
    table.copy_(torch.where(taken, page, torch.where(gone, -1, table)))
    grown = (target > lens) & served
    pos0 = torch.where(grown, lens, -1)
    lens.copy_(torch.where((target >= 0) & served, target, lens))
    return pos0, torch.where(apart, last, -1), torch.where(apart, free[torch.where(apart, upto - need, 0)], -1)


def _fork(s, P):
    table, lens, refs, parent = s["table"], s["lens"], s["refs"], s["parent"]
    child = parent >= 0
    from_ = parent.clamp(min=0).long()
    L = torch.where(child, lens[from_], 0)
    whole = L // P
    part = child & (L % P > 0)
    free, count = _free_pages(refs)
    upto = part.long().cumsum(0)
    ok = child & ((upto <= count) | ~part)
    part = part & ok
    page = free[torch.where(part, upto - 1, 0)]
    j = torch.arange(table.shape[1], device="cuda")
    shared = (j < whole[:, None]) & ok[:, None]
    theirs = table[from_]
    last = (j == whole[:, None]) & part[:, None]
    src = torch.where(part, theirs.gather(1, whole.clamp(max=table.shape[1] - 1).long()[:, None])[:, 0], -1)
    refs.index_add_(0, torch.where(shared, theirs, 0).flatten().long(), shared.flatten().int())
    refs.index_add_(0, torch.where(part, page, 0).long(), part.int())
    table.copy_(torch.where(shared, theirs, torch.where(last, page[:, None], table)))
    lens.copy_(torch.where(ok, L, lens))
    return src, torch.where(part, page, -1)


def _compact(s, P):
    table, lens, refs = s["table"], s["lens"], s["refs"]
    n = len(refs)
    used = refs > 0
    U = used.sum()
    at = torch.arange(n, dtype=I32, device="cuda")
    late, hole = used & (at >= U), ~used & (at < U)
    lists = []
    for which in (late, hole):
        x = torch.full((n + 1,), -1, dtype=I32, device="cuda")
        x[torch.where(which, which.cumsum(0) - 1, n)] = at
        x[n] = -1
        lists.append(x[:n // 2])
    src, dst = lists
    to = at.clone()
    to_all = torch.cat([to, to[:1]])
    to_all[torch.where(src >= 0, src, n).long()] = dst
    j = torch.arange(table.shape[1], device="cuda")
    mine = j < ((lens + P - 1) // P)[:, None]
    new_table = torch.where(mine, to_all[torch.where(mine, table, 0).long()], table)
    new_refs = torch.zeros(n + 1, dtype=I32, device="cuda")
    new_refs[torch.where(used, to_all[:n], n).long()] = refs
    return {"src": src, "dst": dst, "used": U.int().view(1), "new_table": new_table, "new_refs": new_refs[:n]}


# ---- the definitions in 64 bits, and on the host ---------------------------------------

def exact(case, seed):
    op = case["op"]
    if op == "chunk":
        return None if work(case)["flops"] > 1e12 else _exact_chunk(prepare(case, seed), case)
    if op == "copy":
        if work(case)["bytes"] > 3e8:
            return None
        s = prepare(case, seed)
        out = {x: s[x].cpu().double() for x in ("k", "v", "k_scale", "v_scale")}
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            if a >= 0:
                for x in out.values():
                    x[b] = x[a]
        return out
    s = {x: (y.cpu().numpy() if torch.is_tensor(y) else y) for x, y in prepare(case, seed).items()}
    P = case["page"]
    if op == "resize":
        _walk_resize(s, s["before"], P)
        pos0 = _walk_resize(s, s["after"], P)
        none = torch.full((len(pos0),), -1, dtype=I32)  # (no two sequences share a page)
        return dict({x: torch.from_numpy(s[x]) for x in ("table", "lens", "refs")}, pos0=torch.tensor(pos0, dtype=I32),
                    src=none, dst=none)
    if op == "fork":
        _walk_resize(s, s["none"], P)
        free = [int(p) for p in np.flatnonzero(s["refs"] == 0)][::-1]
        src, dst = [-1] * len(s["lens"]), [-1] * len(s["lens"])
        for b, a in enumerate(s["parent"]):
            if a < 0:
                continue
            L = int(s["lens"][a])
            for j in range(L // P):
                s["table"][b, j] = s["table"][a, j]
                s["refs"][s["table"][a, j]] += 1
            if L % P:
                src[b], dst[b] = int(s["table"][a, L // P]), free.pop()
                s["table"][b, L // P] = dst[b]
                s["refs"][dst[b]] = 1
            s["lens"][b] = L
        return dict({x: torch.from_numpy(s[x]) for x in ("table", "lens", "refs")}, src=torch.tensor(src, dtype=I32),
                    dst=torch.tensor(dst, dtype=I32))
    refs = s["refs"]
    U = int((refs > 0).sum())
    holes = [p for p in range(U) if refs[p] == 0]
    moves = dict(zip((int(p) for p in range(U, len(refs)) if refs[p] > 0), holes))
    new_refs, table = refs.copy(), s["table"].copy()
    for a, b in moves.items():
        new_refs[a], new_refs[b] = 0, refs[a]
    for b, L in enumerate(s["lens"]):
        for j in range(pages(int(L), P)):
            table[b, j] = moves.get(int(table[b, j]), table[b, j])
    pad = [-1] * (len(refs) // 2 - len(moves))
    return {"src": torch.tensor(list(moves) + pad, dtype=I32), "dst": torch.tensor(list(moves.values()) + pad, dtype=I32),
            "used": torch.tensor([U], dtype=I32), "new_table": torch.from_numpy(table),
            "new_refs": torch.from_numpy(new_refs)}


def _walk_resize(s, target, P):
    """Page by page; there is room for all, and no page is shared but for whole ones."""
    free = [int(p) for p in np.flatnonzero(s["refs"] == 0)][::-1]
    pos0 = []
    for b, t in enumerate(int(t) for t in target):
        L = int(s["lens"][b])
        pos0.append(L if t > L else -1)
        if t < 0:
            continue
        for j in range(pages(t, P), pages(L, P)):
            s["refs"][s["table"][b, j]] -= 1
            s["table"][b, j] = -1
        for j in range(pages(L, P), pages(t, P)):
            s["table"][b, j] = free.pop()
            s["refs"][s["table"][b, j]] = 1
        s["lens"][b] = t
    return pos0


def _exact_chunk(s, case):
    G, W, P = case["heads"] // case["kv_heads"], case["window"], case["page"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lses = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    q0 = 0
    for b, (n, L) in enumerate(chunk_lengths(case)):
        for a in range(0, n, 1024):  # a stretch of queries and the pages that any of them sees
            z = min(a + 1024, n)
            lo, hi = max(0, L - n + a - W + 1) // P * P if W else 0, L - n + z
            there = s["table"][b, lo // P:pages(hi, P)].long()
            i, j = torch.arange(a, z, device="cuda")[:, None] + L - n, torch.arange(lo, hi, device="cuda")
            gone = (j > i) | (j <= i - W if W else False)
            for h in range(case["kv_heads"]):
                k, v = ((s[x].view(torch.uint8)[there, h].view(F8).double() *
                         s[x + "_scale"][there, h].double()[:, None, None]).flatten(0, 1)[:hi - lo] for x in ("k", "v"))
                for r in range(h * G, h * G + G):
                    x = (s["q"][q0 + a:q0 + z, r].double() @ k.T * s["sm_scale"]).masked_fill_(gone, -math.inf)
                    if case["sink"]:
                        x = torch.cat([x, s["sink"][r].double().expand(z - a, 1)], 1)
                    lse = torch.logsumexp(x, 1)
                    out[q0 + a:q0 + z, r] = torch.exp(x[:, :hi - lo] - lse[:, None]) @ v
                    lses[q0 + a:q0 + z, r] = lse
        q0 += n
    return out, lses
