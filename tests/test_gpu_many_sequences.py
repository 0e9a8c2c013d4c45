"""Calls over as many sequences as there may be: what gets in whose way is found, and the work grows with their number, not
with its square."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from persistent_megakernel_streaming_gb300 import cp
from test_gpu_pages import Both

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.from_numpy(np.asarray(a, np.int32)).cuda()


def fastest(f, repeats=7):
    """Microseconds of the fastest of some calls."""
    f()
    best = np.inf
    for _ in range(repeats):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best


@pytest.mark.parametrize("pairs", [1535, 1536, 1537, 2500])
def test_forks_that_get_in_each_others_way(pairs):
    """Destinations named twice, copied from, out of range, held, and sources out of range, among many good pairs; then the
    same again: nothing is left behind of the first call."""
    g = np.random.default_rng(pairs)
    n = 2 * pairs + 40
    table, length, refs = np.full((n, 2), -1), np.zeros(n, np.int64), np.zeros(n, np.int64)
    held = g.permutation(n)[: pairs // 2]
    table[held, 0], length[held], refs[held] = held, g.integers(1, 17, len(held)), 1
    free = np.setdiff1d(np.arange(n), held)
    b = Both(refs, table, length, 16)
    for _ in range(2):
        src, dst = g.choice(held, pairs), g.permutation(free)[:pairs]
        at = g.permutation(pairs)
        dst[at[:40]] = dst[at[40:80]]                       # twice
        dst[at[80:100]] = src[at[100:120]]                  # copied from by another, and held
        src[at[120:140]] = dst[at[140:160]]                 # copied to by another
        src[at[160]] = dst[at[160]]
        src[at[161:165]], dst[at[165:169]] = [-1, n, 2 ** 31 - 1, -2 ** 31], [-1, n, 2 ** 31 - 1, -2 ** 31]
        b.fork(src, dst)
        assert b.plain.bad
        b.pool.clear_status()
        b.plain.bad = False
        b.trim(np.where(np.isin(np.arange(n), held), 99, 0))
    src, dst = g.choice(held, pairs), g.permutation(free)[:pairs]
    b.fork(src, dst)
    assert not b.plain.bad


def test_a_captured_fork_of_many_pairs():
    """Replayed with other pairs each time, some of them in each other's way."""
    n = 2000
    g = np.random.default_rng(0)
    refs, table, length = np.zeros(2 * n), np.full((2 * n, 2), -1), np.zeros(2 * n)
    refs[:n], table[:n, 0], length[:n] = 1, np.arange(n), g.integers(1, 17, n)
    b = Both(refs, table, length, 16)
    src, dst = i32(np.arange(n)), i32(np.arange(n) + n)
    b.pool.fork(src, dst)
    b.plain.fork(np.arange(n), np.arange(n) + n)
    keep = np.where(np.arange(2 * n) < n, 99, 0)
    b.trim(keep)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.pool.fork(src, dst)
    for k in range(4):
        s, d = g.integers(0, n, n), g.permutation(n) + n
        if k % 2:
            d[: n // 10] = d[n // 2: n // 2 + n // 10]
        src.copy_(i32(s))
        dst.copy_(i32(d))
        graph.replay()
        b.plain.fork(s, d)
        b.same()
        assert b.plain.bad == bool(k % 2)
        b.pool.clear_status()
        b.plain.bad = False
        b.trim(keep)


def test_the_time_of_a_fork_is_linear():
    times = []
    for n in (4000, 32000):
        refs, table, length = np.zeros(2 * n), np.full((2 * n, 2), -1), np.zeros(2 * n)
        refs[:n], table[:n, 0], length[:n] = 1, np.arange(n), 5
        pool = cp.Pages(*(i32(a) for a in (refs, table, length)), 16)
        src, dst, keep = i32(np.arange(n)), i32(np.arange(n) + n), i32(length)

        def call():
            pool.fork(src, dst)
            pool.trim(keep)

        times.append(fastest(call))
        assert pool.status() == 0
    assert times[1] < 16 * times[0], times                  # 8 times the pairs; 26 times as long with the square of them


def draws(n, vocab, dtype=torch.float32, **kw):
    """A batch of plain draws, and what a call on it leaves."""
    x = torch.zeros(n, vocab, dtype=dtype, device="cuda")
    x[:, 1] = 60.0                                          # the token
    z, f = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.full((n,), 0.5, device="cuda")
    accepted, token, prob = torch.full_like(z, -7), torch.full_like(z, -7), torch.full_like(f, -7.0)

    def call(start):
        cp.verify(x, z, start, f, f, f, accepted, token, prob=prob, **kw)
        return accepted, token, prob

    return call


@pytest.mark.parametrize("n", [1, 127, 128, 129, 2047, 2048, 2049, 4097, 65535])
@pytest.mark.parametrize("vocab", [3, 4100])
def test_one_start_out_of_order(n, vocab):
    """Wherever it is; the next call, in order again, finds nothing of it."""
    n = min(n, 5000) if vocab > 3 else n
    call, good = draws(n, vocab), np.arange(n + 1)
    for i in sorted({0, 1, n // 3, n - 128, n - 2, n - 1, n} & set(range(n + 1))):
        for wrong in (-1, good[i] - 2, n + 1, 2 ** 31 - 1, -2 ** 31):
            start = good.copy()
            start[i] = wrong
            if (np.diff(start) >= 0).all() and start[0] >= 0 and start[-1] <= n:
                continue
            accepted, token, prob = call(i32(start))
            assert (accepted == -1).all() and (token == -1).all() and (prob == -7).all(), (i, wrong)
        accepted, token, prob = call(i32(good))
        assert (accepted == 0).all() and (token == 1).all() and (prob == -7).all()


@pytest.mark.parametrize("vocab", [4, 4100])
def test_the_time_of_a_verification_is_linear(vocab):
    times = []
    for n in (8000, 64000):
        call, start = draws(n, vocab, torch.bfloat16), i32(np.arange(n + 1))
        times.append(fastest(lambda: call(start)))
    assert times[1] < 12 * times[0], times                  # 8 times the sequences; 16 to 20 times as long with the square of them


def test_captured_calls_over_many_sequences():
    """Two graphs with workspaces of their own, in turn, and one replayed behind a start out of order."""
    n = 3000
    good, bad = i32(np.arange(n + 1)), i32(np.arange(n + 1)[::-1])
    start = good.clone()
    graphs = []
    for _ in range(2):
        call = draws(n, 50, workspace=torch.full((cp.verify_workspace_bytes(n, n, 50),), 255, dtype=torch.uint8, device="cuda"))
        out = call(start)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(start)
        graphs.append((graph, out, call))                   # the graph reads what the call holds
    for k, which in enumerate((good, bad, good, good, bad, bad, good)):
        start.copy_(which)
        graph, (accepted, token, _), _ = graphs[k % 2]
        graph.replay()
        torch.cuda.synchronize()
        assert (token == (1 if which is good else -1)).all() and (accepted == (0 if which is good else -1)).all()
