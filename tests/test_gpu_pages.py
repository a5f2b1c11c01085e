"""csa_pages_resize, csa_pages_fork, csa_pages_compact and csa_pages_copy
against the same steps on the host, one page at a time: everything is whole
numbers or copies, so everything has to be equal."""
import numpy as np
import pytest
import torch

from _pages import Pages

pytestmark = pytest.mark.gpu
DEV = "cuda"
RANGE = 5  # CSA_ERR_INDEX_RANGE


@pytest.fixture(scope="module")
def csa():
    import compressed_sparse_attention_02_gb300 as m
    return m


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Both:
    """The same book on the host and on the GPU."""

    def __init__(self, csa, table, lens, refs, page):
        self.csa, self.host = csa, Pages(table, lens, refs, page)
        self.table, self.lens, self.refs = i32(table), i32(lens), i32(refs)
        self.book = csa.page_book(self.table, self.lens, self.refs, page)
        self.ws = csa.pages_workspace(self.book)
        self.ws.fill_(0xA5)  # (nothing in it needs to be clear)

    def same(self, **more):
        for name in ("table", "lens", "refs"):
            more[name] = (getattr(self, name), getattr(self.host, name))
        for name, (got, want) in more.items():
            got = got.cpu().numpy()
            assert np.array_equal(got, want), "%s: %d entries differ" % (name, (got != want).sum())
        want = RANGE if self.host.refused else 0
        assert self.csa.csa_check_status() == want
        self.host.refused = False

    def outs(self, n, m):
        return [torch.full((m,), 77, dtype=torch.int32, device=DEV) for _ in range(n)]

    def resize(self, target, copies=True):
        pos0, src, dst = self.outs(3, len(self.host.lens))
        self.csa.csa_pages_resize(self.book, i32(target), pos0, src if copies else None, dst if copies else None, self.ws)
        want = self.host.resize(target, copies)
        if copies:
            self.same(pos0=(pos0, want[0]), src=(src, want[1]), dst=(dst, want[2]))
        else:
            self.same(pos0=(pos0, want[0]))
        return want

    def fork(self, parent):
        src, dst = self.outs(2, len(self.host.lens))
        self.csa.csa_pages_fork(self.book, i32(parent), src, dst, self.ws)
        want = self.host.fork(parent)
        self.same(src=(src, want[0]), dst=(dst, want[1]))
        return want

    def compact(self, in_place):
        src, dst = self.outs(2, len(self.host.refs) // 2)
        used, = self.outs(1, 1)
        table, refs = (self.table, self.refs) if in_place else (torch.empty_like(self.table), torch.empty_like(self.refs))
        self.csa.csa_pages_compact(self.book, src, dst, used, table, refs, self.ws)
        if not in_place:
            assert np.array_equal(self.table.cpu().numpy(), self.host.table)
            assert np.array_equal(self.refs.cpu().numpy(), self.host.refs)
            self.table.copy_(table)
            self.refs.copy_(refs)
        want = self.host.compact()
        self.same(src=(src, want[0]), dst=(dst, want[1]), used=(used, np.array([want[2]])))
        return want


def make(csa, lens, cap, pool, page, seed=0):
    """Sequences on shuffled pages."""
    r = np.random.default_rng(seed)
    n = [-(-x // page) for x in lens]
    order, at = r.permutation(pool), 0
    table, refs = np.full((len(lens), cap), -1, np.int32), np.zeros(pool, np.int32)
    for b, x in enumerate(n):
        table[b, :x] = order[at:at + x]
        at += x
    refs[order[:at]] = 1
    return Both(csa, table, lens, refs, page)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_growing_and_shrinking(csa, page):
    lens = [0, 1, page - 1, page, page + 1, 3 * page, 7 * page - 2, 5]
    x = make(csa, lens, 9, 100, page, seed=page)
    x.resize([1, 1, page, page + 1, page + 1, 4 * page + 1, 0, -1])
    x.host.check()
    x.resize([9 * page, 0, page - 1, 2, 9 * page - 1, 0, 3 * page, 5])
    x.resize([-1] * 8)
    x.resize([0] * 8)
    assert (x.host.refs == 0).all() and (x.host.table == -1).all()


@pytest.mark.parametrize("pool", [1, 31, 32, 33, 4095, 4096, 4097, 20000, 130001])
def test_pools_of_any_size(csa, pool):
    """Stretches of the pool that are full, empty and mixed; a sequence that takes nearly all of it."""
    x = make(csa, [0, 0, 0], pool, pool, 16, seed=pool)
    most = 16 * pool
    x.resize([most // 3, most // 4, 0])
    x.resize([0, -1, most // 2])
    x.resize([most // 5, 0, most // 4])
    x.host.check()
    x.compact(in_place=False)
    x.resize([-1, -1, 0])
    x.compact(in_place=True)
    x.resize([-1, most // 2, most])          # the last one finds no pages
    x.host.check()


def test_more_is_wanted_than_is_free(csa):
    x = make(csa, [10, 100, 16, 0, 30], 20, 40, 16, seed=3)
    # 1 + 7 + 1 + 2 pages are held, 29 are free: 17, then 20 (37 > 29: refused), then one that needs none, then one that
    # would fit but comes behind
    x.resize([280, 320, 16, 32, 31])
    assert x.host.lens.tolist() == [280, 100, 16, 0, 31]
    x.resize([281, 16 * 20 + 1, -5, 0, 0])   # past the table
    x.resize([0, 320, 16, 32, 31])           # what is given back is not free in the same call
    x.resize([0, 320, 16, 32, 31])
    x.host.check()


def test_no_page_is_free(csa):
    x = make(csa, [64, 48], 4, 7, 16)
    x.resize([64, 49])
    x.fork([-1, -1])
    x.compact(in_place=True)
    y = make(csa, [0, 0], 4, 7, 16)
    y.compact(in_place=True)
    y.fork([-1, 0])


@pytest.mark.parametrize("page,children", [(16, 1), (16, 9), (64, 4), (128, 300)])
def test_forks(csa, page, children):
    lens = [5 * page, 3 * page + 1, page - 1, 0, 1] + [0] * children
    x = make(csa, lens, 8, 40 + 2 * children, page, seed=children)
    x.fork([-1] * 5 + [b % 5 for b in range(children)])
    x.host.check()
    # the children grow apart, and end
    x.resize([-1] * 5 + [int(x.host.lens[5 + b]) + b % 3 for b in range(children)])
    x.resize([0, 0, -1, -1, -1] + [0 if b % 2 else -1 for b in range(children)])
    x.host.check()
    x.compact(in_place=True)
    x.host.check()
    x.resize([0] * len(lens))
    assert (x.host.refs == 0).all()


def test_a_shared_page_that_is_cut_is_left_to_the_others(csa):
    """A fork cut back into a page that its parent has too, then both grow: whoever grows while it is shared takes a page
    of its own, and the pair is listed."""
    P = 16
    x = make(csa, [4 * P, 0, 0], 10, 40, P, seed=1)
    x.fork([-1, 0, 0])
    x.resize([-1, 2 * P + 3, 2 * P + 3])
    assert x.host.refs.max() == 3
    x.resize([-1, 2 * P + 4, -1])
    assert (x.resize([3 * P - 1, -1, -1])[1] < 0).all()
    src, dst = x.resize([3 * P, -1, 3 * P + 1])[1:]
    assert src[0] == src[2] >= 0 and dst[0] != dst[2]  # two holders, and both grow
    assert x.host.refs[src[0]] == 0
    x.host.check()
    # without the lists such a sequence stays as it is
    x.fork([-1, -1, -1])
    x.resize([0, 0, -1])
    x.fork([2, -1, -1])
    x.resize([P + 1, -1, -1])
    x.resize([P + 2, 5, -1], copies=False)
    assert x.host.lens[0] == P + 1 and x.host.lens[1] == 5


def test_forks_that_cannot_be(csa):
    x = make(csa, [33, 5, 0, 0, 0, 0], 4, 8, 16, seed=2)
    # a child with tokens, no such parent, itself, an empty parent that is forked too, one page left after
    x.fork([-1, 0, 6, 3, 2, -1])
    x.fork([-1, -1, 0, 0, 0, 0])             # four pages are free and three children need one each, the fourth too
    x.fork([-1, -1, -1, -1, -1, -1])
    y = make(csa, [33, 0, 0], 4, 4, 16)
    y.fork([-1, 0, 0])                       # one page for two
    assert y.host.lens.tolist() == [33, 33, 0]
    y.host.check()


@pytest.mark.parametrize("n,pool", [(2500, 60000), (6000, 150000), (40, 1100000)])
def test_many_sequences_and_large_pools(csa, n, pool):
    """More than one block of the sums, every kind of change at once, over several steps; as many sequences and pages as
    take the call's other way."""
    r, P = np.random.default_rng(7), 16
    x = make(csa, r.integers(0, 200, n).tolist(), 30, pool, P, seed=7)
    for step in range(3):
        target = np.where(r.random(n) < 0.3, -1, np.where(r.random(n) < 0.3, 0, r.integers(0, 480, n)))
        x.resize(target)
        empty = x.host.lens == 0
        parent = np.where(empty & (r.random(n) < 0.5), r.integers(0, n, n), -1)
        x.fork(parent)
        x.host.check()
    x.compact(in_place=False)
    x.host.check()


def test_wrong_numbers(csa):
    """Lengths past the table, entries outside the pool, counts that do not fit: reported, nothing outside is touched."""
    P = 16
    table = np.array([[0, 1, 2], [3, -7, 99], [5, 6, 2 ** 31 - 1], [-1, -1, -1]], np.int32)
    refs = np.array([1, 1, 1, 1, 0, 1, 0, -4], np.int32)
    guard = torch.full((64,), 5, dtype=torch.int32, device=DEV)
    x = Both(csa, table, [100, 40, 48, -3], refs, P)
    x.compact(in_place=True)
    x = Both(csa, table, [100, 40, 48, -3], refs, P)
    x.resize([48, 41, 2 ** 31 - 1, 17])      # cut to the table; grows in a page that is none; past the table; takes two
    x = Both(csa, table, [100, 40, 48, -3], refs, P)
    x.resize([0, 0, 1, 0])                   # (page 6 has no holder to take off)
    x = Both(csa, table, [48, 40, 48, -3], refs, P)
    x.fork([-1, -1, -1, 1])
    assert (guard == 5).all()


@pytest.mark.parametrize("last", [-1, -9, 8, 2 ** 31 - 1])
def test_fork_of_a_last_page_that_is_none(csa, last):
    """A parent whose partly filled page is outside the pool: reported; the child has a page and no pair to copy."""
    table = np.array([[0, last, -1], [-1, -1, -1], [2, 3, -1], [-1, -1, -1]], np.int32)
    x = Both(csa, table, [20, 0, 20, 0], [1, 0, 1, 1, 0, 0, 0, 0], 16)
    src, dst = x.fork([-1, 0, -1, 2])
    assert src.tolist() == [-1, -1, -1, 3] and dst.tolist() == [-1, -1, -1, 4]
    assert x.host.table[1].tolist() == [0, 1, -1] and x.host.table[3].tolist() == [2, 4, -1]


def test_streams_graphs_and_overlapping_calls(csa):
    """A captured growth replays on what is there then; two books' calls run at once with a workspace each."""
    P = 16
    x = make(csa, [5, 0, 40], 20, 200, P, seed=4)
    target = i32([0, 0, 0])
    pos0, src, dst = x.outs(3, 3)
    x.csa.csa_pages_resize(x.book, x.lens.clone(), pos0, src, dst, x.ws)  # (nothing changes)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        csa.csa_pages_resize(x.book, target, pos0, src, dst, x.ws)
    for want in ([20, 16, 41], [0, 100, 300], [33, 99, 0], [1, 1, 1]):
        target.copy_(i32(want))
        g.replay()
        torch.cuda.synchronize()
        p, a, b = x.host.resize(want)
        x.same(pos0=(pos0, p), src=(src, a), dst=(dst, b))
    ys = [make(csa, [100 * s, 0], 2000, 30000, P, seed=s) for s in range(4)]
    streams = [torch.cuda.Stream() for _ in ys]
    wants, out = [[17000, 5000], [0, 30000], [31000, 1], [2, 20000]], []
    targets = [i32(w) for w in wants]
    torch.cuda.synchronize()
    for rep in range(3):
        for y, s, t in zip(ys, streams, targets):
            with torch.cuda.stream(s):
                csa.csa_pages_resize(y.book, t, None, None, None, y.ws)
    torch.cuda.synchronize()
    for y, w in zip(ys, wants):
        y.host.resize(w)
        y.same()


@pytest.mark.parametrize("H,D,P", [(1, 64, 16), (3, 64, 32), (8, 128, 64), (5, 128, 128), (64, 128, 128)])
def test_copies(csa, H, D, P):
    g = torch.Generator(DEV).manual_seed(H)
    n = 60
    k, v = (torch.randint(0, 256, (n, H, P, D), device=DEV, generator=g, dtype=torch.uint8) for _ in range(2))
    ks, vs = (torch.rand(n, H, device=DEV, generator=g) for _ in range(2))
    cache = csa.paged_cache(k, v, ks, vs, torch.zeros(1, 1, dtype=torch.int32, device=DEV))
    src = [5, -1, 7, 7, 0, 59, -3, 12, 11, 60, 5, 2 ** 31 - 1, 13]
    dst = [9, 3, 1, 2, 58, 4, 6, 12, -1, 8, 60, 14, 20]
    want = [x.clone() for x in (k, v, ks, vs)]
    for a, b in zip(src, dst):
        if 0 <= a < n and 0 <= b < n:
            for x, y in zip(want, (k, v, ks, vs)):
                x[b] = y[a]
    csa.csa_pages_copy(cache, i32(src), i32(dst))
    assert csa.csa_check_status() == RANGE
    for x, y in zip((k, v, ks, vs), want):
        assert torch.equal(x, y)
    csa.csa_pages_copy(cache, i32([-1] * 5), i32([-1] * 5))
    csa.csa_pages_copy(cache, i32([]), i32([]))
    assert csa.csa_check_status() == 0
    for x, y in zip((k, v, ks, vs), want):
        assert torch.equal(x, y)


def test_copy_of_a_long_list(csa):
    """A list of which most is empty, longer than one look at it, in a pool past four gigabytes."""
    n, H, P, D = 140000, 4, 64, 128
    k, v = (torch.zeros(n, H, P, D, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(n, H, device=DEV) for _ in range(2))
    cache = csa.paged_cache(k, v, ks, vs, torch.zeros(1, 1, dtype=torch.int32, device=DEV))
    g = torch.Generator(DEV).manual_seed(1)
    pages = torch.randperm(n, device=DEV, generator=g)[:2000].int()
    for x in (k, v):
        x[pages[:1000].long()] = torch.randint(0, 256, (1000, H, P, D), device=DEV, generator=g, dtype=torch.uint8)
    for x in (ks, vs):
        x[pages[:1000].long()] = torch.rand(1000, H, device=DEV, generator=g) + 1
    src, dst = (torch.full((700001,), -1, dtype=torch.int32, device=DEV) for _ in range(2))
    at = torch.randperm(700001, device=DEV, generator=g)[:1000]
    src[at], dst[at] = pages[:1000], pages[1000:]
    csa.csa_pages_copy(cache, src, dst)
    assert csa.csa_check_status() == 0
    for x in (k, v, ks, vs):
        assert torch.equal(x[pages[:1000].long()], x[pages[1000:].long()])
        assert int((x.flatten(1) != 0).any(1).sum()) == 2000


def test_refusals(csa):
    x = make(csa, [5, 0], 4, 9, 16)
    a = i32([1, 1])
    for f in (lambda: csa.csa_pages_resize(x.book, a.long(), None, None, None, x.ws),
              lambda: csa.csa_pages_resize(x.book, i32([1]), None, None, None, x.ws),
              lambda: csa.csa_pages_resize(x.book, a, None, a, None, x.ws),
              lambda: csa.csa_pages_fork(x.book, a, a[:1], a, x.ws),
              lambda: csa.csa_pages_fork(x.book, a, None, a, x.ws),
              lambda: csa.csa_pages_compact(x.book, a, a, a[:1], x.table, x.refs, x.ws),
              lambda: csa.page_book(x.table.T, x.lens, x.refs, 16),
              lambda: csa.page_book(x.table, x.lens[:1], x.refs, 16)):
        with pytest.raises(csa.CsaError) as e:
            f()
        assert e.value.status == 1
    with pytest.raises(csa.CsaError) as e:
        csa.csa_pages_resize(x.book, a, None, None, None, x.ws[:-16])
    assert e.value.status == 6
    with pytest.raises(csa.CsaError):
        csa.pages_workspace(csa.page_book(x.table, x.lens, x.refs, 24))
    assert x.lens.tolist() == [5, 0]
