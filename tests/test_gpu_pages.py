"""Forking, growing, trimming and compacting against a plain sequential pool, and the copies inside a cache."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from oracle.pages import Pool
from persistent_megakernel_streaming_gb300 import cp

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Both:
    """The same calls on the GPU and on the plain pool, everything compared after each."""

    def __init__(self, refs, table, length, page, stride=0):
        table = np.asarray(table)
        wide = torch.full((table.shape[0], max(stride, table.shape[1])), -7, dtype=torch.int32, device="cuda")
        self.table = wide[:, : table.shape[1]]
        self.table.copy_(dev(table))
        self.wide = wide
        self.refs, self.length = dev(refs), dev(length)
        self.plain = Pool(refs, table, length, page)
        self.pool = cp.Pages(self.refs, self.table, self.length, page)
        n = max(len(length), len(refs) // 2, 1)
        self.moves = torch.full((n, 2), -9, dtype=torch.int32, device="cuda")
        self.count = torch.full((1,), -9, dtype=torch.int32, device="cuda")

    def same(self):
        np.testing.assert_array_equal(self.refs.cpu().numpy(), self.plain.refs)
        np.testing.assert_array_equal(self.table.cpu().numpy(), self.plain.table)
        np.testing.assert_array_equal(self.length.cpu().numpy(), self.plain.length)
        assert (self.wide[:, self.table.shape[1]:] == -7).all()
        assert self.pool.status() == (6 if self.plain.bad else 0)

    def moved(self, got):
        moves, count = got
        assert int(self.count) == count
        assert self.moves[: max(count, 0)].cpu().numpy().tolist() == [list(m) for m in moves]
        self.same()
        return moves

    def fork(self, src, dst):
        self.pool.fork(dev(src), dev(dst))
        self.plain.fork(src, dst)
        self.same()

    def trim(self, keep):
        self.pool.trim(dev(keep))
        self.plain.trim(keep)
        self.same()

    def grow(self, add):
        self.pool.grow(dev(add), self.moves, self.count)
        return self.moved(self.plain.grow(add))

    def compact(self):
        self.pool.compact(self.moves, self.count)
        return self.moved(self.plain.compact())


def empty(pages, sequences, width, page=16, stride=0):
    return Both(np.zeros(pages), np.full((sequences, width), -1), np.zeros(sequences), page, stride)


def test_a_page_shared_by_all_that_grow():
    b = empty(40, 6, 8)
    b.grow([37, 0, 0, 0, 0, 0])
    b.fork([0, 0, 0], [3, 1, 5])
    assert b.grow([1, 1, 0, 1, 0, 1]) == [(2, 3), (2, 4), (2, 5)]      # the last of the four keeps it
    b.fork([0, 0], [2, 4])
    b.grow([0, 0, 1, 0, 20, 0])                                        # sequence 0 still holds the shared page
    b.trim([36, 0, 5, 48, 16, 33])
    b.grow([11, 100, 0, 1, 1, 2])


def test_lengths_that_end_on_a_page_share_without_copies():
    b = empty(20, 3, 8)
    b.grow([32, 0, 0])
    b.fork([0, 0], [1, 2])
    assert b.grow([5, 5, 5]) == []
    b.trim([32, 32, 31])
    assert len(b.grow([0, 0, 1])) == 1


def test_a_pool_without_enough_pages_changes_nothing():
    b = empty(5, 3, 8)
    b.grow([40, 16, 0])
    b.fork([0], [2])
    before = b.refs.clone()
    b.grow([9, 20, 3])
    assert int(b.count) < 0 and torch.equal(before, b.refs)
    b.grow([8, 0, 0])                                                  # a shared page's copy alone fits
    assert int(b.count) == 1
    b.grow([0, 2000, 0])                                               # past its table


@pytest.mark.parametrize("seed", range(12))
def test_random_lives(seed):
    g = np.random.default_rng(seed)
    page = int(g.choice([16, 32, 64, 128]))
    n, width, pages = int(g.integers(1, 70)), int(g.integers(1, 40)), int(g.integers(1, 900))
    b = empty(pages, n, width, page, stride=width + int(g.integers(0, 5)))
    for _ in range(25):
        kind = g.integers(0, 5)
        if kind <= 1:
            b.grow([int(x) for x in g.integers(0, width * page // 2 + 2, n) * (g.random(n) < 0.4)])
        elif kind == 2:
            b.trim([int(x) for x in np.where(g.random(n) < 0.5, g.integers(0, width * page + 1, n), 2 ** 31 - 1)])
        elif kind == 3:
            m = int(g.integers(1, n + 1))
            b.fork([int(x) for x in g.integers(0, n, m)], [int(x) for x in g.permutation(n)[:m]])
            b.pool.clear_status()
            b.plain.bad = False
        else:
            b.compact()
        if b.plain.bad:
            b.pool.clear_status()
            b.plain.bad = False


@pytest.mark.parametrize("pages,sequences", [(4097, 3), (40000, 1500), (33000, 1025), (9000, 9000)])
def test_many_pages_and_sequences(pages, sequences):
    """Sizes that take one block, two, four and eight."""
    g = np.random.default_rng(pages)
    width = 12
    table, refs, length = np.full((sequences, width), -1), np.zeros(pages, np.int64), np.zeros(sequences, np.int64)
    order, at = g.permutation(pages), 0
    for i in range(sequences):
        k = int(g.integers(0, width + 1))
        if at + k > pages * 3 // 4:
            break
        table[i, :k], length[i] = order[at:at + k], max(0, k * 16 - int(g.integers(0, 16)))
        refs[order[at:at + k]] = 1
        at += k
    b = Both(refs, table, length, 16)
    b.compact()
    b.trim(np.where(g.random(sequences) < 0.3, 0, 10 ** 6).tolist())
    none = np.flatnonzero(b.plain.length == 0)
    some = np.flatnonzero(b.plain.length > 0)
    b.fork(g.choice(some, len(none)).tolist(), none.tolist())
    b.grow([min(int(x), width * 16 - int(l)) for x, l in zip(g.integers(0, 3, sequences), b.plain.length)])
    b.compact()


@pytest.mark.parametrize("sequences,pages,width", [(1, 64, 60), (33, 4096, 130), (80, 4097, 60), (129, 20000, 200), (1030, 33000, 40),
                                                   (8300, 70000, 9), (300, 40000, 130)])
def test_many_pages_at_once(sequences, pages, width):
    """Sequences that take up to `width` pages in one call, some none, some one or two, over shared pages too; half of them
    end, and the others move."""
    g = np.random.default_rng(sequences)
    b = empty(pages, sequences, width, stride=width + 3)
    some = g.random(sequences)
    add = np.where(some < 0.3, 0, np.where(some < 0.5, g.integers(1, 33, sequences), g.integers(1, 16 * width - 60, sequences)))
    add = np.where(g.random(sequences) < 0.05, 16 * (width - 4), add)
    while (-(-add // 16)).sum() > pages * 3 // 4:
        add = add // 2
    b.grow(add)
    empty_ones = np.flatnonzero(add == 0)
    n = len(empty_ones) // 2
    if n:
        b.fork(g.choice(np.flatnonzero(add > 0), n), empty_ones[:n])
    b.grow(np.where(b.plain.length > 0, g.integers(0, 58, sequences), 0))
    b.trim(np.where(g.random(sequences) < 0.5, 0, b.plain.length))
    b.compact()
    b.grow(np.where(b.plain.length == 0, np.minimum(g.integers(0, 200, sequences), 16 * width - 40), 3))
    b.trim(np.zeros(sequences))
    b.compact()


def test_what_the_arrays_hold_is_checked():
    """Bad lengths, pages, counts and sequences: nothing is touched but the status."""
    def fresh():
        table = np.array([[0, 1, 2], [3, 99, -5], [4, 5, 6], [-1, -1, -1], [0, 1, -1]])
        return Both([2, 2, 1, 1, 1, 0, 1, 0], table, [40, 40, -3, 0, 20], 16)
    for call in (lambda b: b.grow([1, 1, 1, 1, 1]), lambda b: b.trim([5, 0, 0, 0, 3]), lambda b: b.trim([-1, 1, 1, 1, 2 ** 31 - 1]),
                 lambda b: b.compact(), lambda b: b.grow([0, -1, 0, 9, 0]), lambda b: b.grow([2 ** 31 - 1] * 5),
                 lambda b: b.fork([0, 1, 2], [3, 3, 0]), lambda b: b.fork([1], [3]), lambda b: b.fork([5, -1, 0], [3, 3, -9]),
                 lambda b: b.fork([0], [4]), lambda b: b.fork([3], [3])):
        b = fresh()
        call(b)
        assert b.plain.bad
    # a count below the entries that name a page
    b = Both([0, 1], [[0, 1]], [20], 16)
    b.trim([0])
    b = Both([0, 1, 0], [[1, 0]], [20], 16)
    b.grow([1])
    # a length past what the table holds
    b = Both([1, 1, 0], [[0, 1]], [33], 16)
    b.grow([1])


def cache_of(dtype, pages, heads, page, d, seed, interleaved=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if dtype == "bf16":
        shape = (pages, heads, page, 2, d) if interleaved else (2, pages, heads, page, d)
        kv = torch.randint(-30000, 30000, shape, generator=g, device="cuda", dtype=torch.int16)
        k, v = (kv[..., 0, :], kv[..., 1, :]) if interleaved else (kv[0], kv[1])
        return cp.Cache(k, v), [k, v]
    k, v = (torch.randint(0, 255, (pages, heads, page, d), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
    if interleaved:
        sc = torch.randint(0, 255, (pages, page, heads, 2), generator=g, device="cuda", dtype=torch.uint8)
        ks, vs = (sc[..., x].permute(0, 2, 1) for x in range(2))
    else:
        ks, vs = (torch.randint(0, 255, (pages, heads, page), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
    return cp.Cache(k, v, ks, vs), [k, v, ks, vs]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,page,d", [(1, 16, 64), (2, 16, 64), (8, 64, 128), (3, 128, 64), (5, 32, 128), (16, 16, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_copies(dtype, heads, page, d, interleaved):
    cache, parts = cache_of(dtype, 60, heads, page, d, 1, interleaved)
    g = np.random.default_rng(heads)
    order = g.permutation(60)
    moves = np.stack([order[:23], order[30:53]], 1)
    moves[4] = 7, 7                                                    # onto itself
    moves[4, 0] = moves[4, 1] = order[55]
    want = [x.clone() for x in parts]
    for a, b in moves:
        for x, y in zip(want, parts):
            x[b] = y[a]
    cache.copy(dev(np.concatenate([moves, [[-1, 5], [1 << 30, 3]]])), dev([23]))
    for x, y in zip(want, parts):
        assert torch.equal(x, y)
    assert cache.status() == 0
    for n in (0, -4):
        cache.copy(dev([[0, 1]]), dev([n]))
    for x, y in zip(want, parts):
        assert torch.equal(x, y)
    assert cache.status() == 0


def test_bad_copies_are_left_out():
    cache, parts = cache_of("e4m3", 9, 2, 16, 64, 2)
    want = [x.clone() for x in parts]
    for x in want:
        x[2] = x[1]
    for moves, count in (([[9, 0], [1, 2], [0, -1], [-2 ** 31, 3], [3, 2 ** 31 - 1]], 5), ([[1, 2]], 2), ([[1, 2]], 2 ** 31 - 1)):
        cache.clear_status()
        cache.copy(dev(moves), dev([count]))
        assert cache.status() == 6
        for x, y in zip(want, parts):
            assert torch.equal(x, y)


def test_copies_past_32_bits():
    """Pages more than 4 GB apart."""
    pages, stride = 5, (1 << 30) // 2 + 64                             # elements: 1 GB a page and a little
    flat = torch.zeros(pages * stride, dtype=torch.int16, device="cuda")
    k = flat.as_strided((pages, 1, 16, 64), (stride, 1024, 64, 1))
    v = flat.as_strided((pages, 1, 16, 64), (stride, 1024, 64, 1), 2048)
    k[0], v[4] = 5, 9
    cache = cp.Cache(k, v)
    cache.copy(dev([[0, 4]]), dev([1]))
    assert (k[4] == 5).all() and (v[4] == 0).all() and cache.status() == 0
    cache.copy(dev([[4, 1]]), dev([1]))
    assert (k[1] == 5).all()


def test_captured_calls_follow_the_arrays():
    """Two graphs of the same calls, replayed in turn on one pool."""
    b = empty(64, 4, 10)
    b.grow([30, 20, 0, 0])
    add, keep, src, dst = dev([1, 1, 1, 1]), dev([99] * 4), dev([0]), dev([2])
    cache, parts = cache_of("bf16", 64, 2, 16, 64, 3)
    graphs = []
    torch.cuda.synchronize()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.pool.trim(keep)
            b.pool.fork(src, dst)
            b.pool.grow(add, b.moves, b.count)
            cache.copy(b.moves, b.count)
        graphs.append(graph)
    content = [p.clone() for p in parts]
    for k in range(6):
        keep.copy_(dev([99, 99, 0, 99]))
        src.fill_(k % 2)
        add.copy_(dev([k, 1, 2, 0]))
        graphs[k % 2].replay()
        b.plain.trim([99, 99, 0, 99])
        b.plain.fork([k % 2], [2])
        moves, count = b.plain.grow([k, 1, 2, 0])
        for p in content:
            for x, y in moves:
                p[y] = p[x]
        b.moved((moves, count))
        for p, q in zip(content, parts):
            assert torch.equal(p, q)


def test_refusals():
    b = empty(8, 2, 4)
    with pytest.raises(ValueError):
        b.pool.trim(torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        b.pool.trim(torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        b.pool.trim(torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        b.pool.fork(dev([0]), dev([0, 1]))
    with pytest.raises(cp.CPError):
        b.pool.fork(dev([0, 0, 0]), dev([1, 1, 1]))                    # more pairs than sequences
    with pytest.raises(cp.CPError):
        b.pool.grow(dev([0, 0]), b.moves[:1].contiguous(), b.count)
    with pytest.raises(cp.CPError):
        b.pool.compact(b.moves[:3].contiguous(), b.count)
    with pytest.raises(ValueError):
        cp.Pages(b.refs, b.table.cpu(), b.length, 16)
    with pytest.raises(cp.CPError):
        cp.Pages(b.refs, b.table, b.length, 24)
    cache, _ = cache_of("bf16", 4, 1, 16, 64, 0)
    with pytest.raises(ValueError):
        cache.copy(b.moves.cpu(), b.count)
    with pytest.raises(ValueError):
        cache.copy(b.moves[:, :1], b.count)
    with pytest.raises(ValueError):
        cache.copy(b.moves, dev([1, 2]))
