"""The paged cache's kernels on the GPU against the float64 reference (oracle/cache.py).

Tolerances are derived, not fitted. bf16 rounds by at most 2^-8 of the value,
fp16 by 2^-11, e4m3 by 2^-4 (or half its least step, 2^-10 of the scale).

append: x is bf16, the norm and the rotation are some 20 fp32 operations each
off by 2^-24 of the pair's size, the sum of D squares by at most D * 2^-24
relative, half of that in the root: (D/2 + 40) * 2^-24 of the pair's size,
then one rounding.

attend: a score's error is at most (D + 8) * 2^-24 * reach (reach = scale *
sum |q_i k_i|, as an fp32 sum in any order has it), and a weight's relative
error that times 2 (numerator and sum; the running maximum cancels), plus
2^-21 for the exponential and its rescaling, plus the weight's rounding for
the product (2^-8 in bf16, 2^-11 in fp16) and L * 2^-24 for a sum of L terms
in fp32. All of it is relative to sum w |v|; the result is rounded once, 2^-8.
An fp16 weight below 2^-14 is rounded by at most 2^-25, next to a largest of at
least 1 in each part, and a part's scales differ from its largest by the power
of two that multiplies the weight: at most 2^-25 * L * max |v| is added.
"""
import numpy as np
import pytest
import torch

from oracle import cache as ref
from persistent_megakernel_streaming_gb300 import build, cp

pytestmark = pytest.mark.gpu

BOUNDS = 6      # CP_ERR_DEVICE_BOUNDS


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


class World:
    """A ragged batch over a pool whose every byte that no test wrote is NaN."""

    def __init__(self, lengths, new, hkv=2, d=64, page=16, e4m3=False, seed=0, pad=0, spread=0.5, interleaved=False,
                 device="cuda"):
        g = self.g = np.random.default_rng(seed)
        self.lengths, self.new, self.hkv, self.d, self.page, self.e4m3 = lengths, new, hkv, d, page, e4m3
        n = len(lengths)
        need = [max(0, -(-L // page)) for L in lengths]
        self.pages = sum(need) + 2
        order = g.permutation(self.pages)
        width = max(need + [1]) + 1
        self.table = np.full((n, width), -7, np.int32)
        at = 0
        for i, k in enumerate(need):
            self.table[i, :k] = order[at:at + k]
            at += k
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.rows = int(self.start[-1]) + pad
        dt = torch.uint8 if e4m3 else torch.int16
        # e4m3 0xff and bf16 0xffff are NaN; scales of unwritten places are 0 (2^-127)
        if interleaved:     # one tensor [page][token][head][k|v][D]
            base = torch.full((self.pages, page, hkv, 2, d), -1 if not e4m3 else 255, dtype=dt, device=device)
            self.k, self.v = (base[:, :, :, i].permute(0, 2, 1, 3) for i in range(2))
        else:
            self.k, self.v = (torch.full((self.pages, hkv, page, d), -1 if not e4m3 else 255, dtype=dt, device=device)
                              for _ in range(2))
        self.ks = self.vs = None
        if e4m3:
            self.ks, self.vs = (torch.zeros((self.pages, hkv, page), dtype=torch.uint8, device=device) for _ in range(2))
            if interleaved:
                base = torch.zeros((self.pages, page, hkv, 2), dtype=torch.uint8, device=device)
                self.ks, self.vs = (base[..., i].permute(0, 2, 1) for i in range(2))
        self.cache = cp.Cache(self.k, self.v, self.ks, self.vs)
        self.spread = spread
        self.batch_of = lambda **kw: cp.Batch(
            torch.from_numpy(self.start).to(device), torch.tensor(lengths, dtype=torch.int32, device=device),
            torch.from_numpy(self.table).to(device), self.rows,
            **{"max_new": max(new), "max_len": max(max(lengths), 1), **kw})
        self.batch = self.batch_of()

    def fill(self):
        """Random keys and values in every cached position; self.kv[i] = (k, v) float64 [L][hkv][d] as cached."""
        self.kv = []
        pool = [x.cpu().clone() for x in (self.k, self.v)]
        scales = [None if x is None else x.cpu().clone() for x in (self.ks, self.vs)]
        for i, L in enumerate(self.lengths):
            both = []
            t = np.arange(max(L, 0))
            pg, pl = self.table[i, t // self.page], t % self.page
            for j in range(2):
                x = self.g.standard_normal((len(t), self.hkv, self.d)) * np.exp(
                    self.spread * self.g.standard_normal((len(t), self.hkv, 1)))
                if self.e4m3:
                    byte, e = ref.quantise(x)
                    pool[j][pg, :, pl] = torch.from_numpy(byte)
                    scales[j][pg, :, pl] = torch.from_numpy((e + 127).astype(np.uint8))
                    both.append(ref.dequantise(byte, e))
                else:
                    b = bf16(x)
                    pool[j][pg, :, pl] = b.view(torch.int16)
                    both.append(b.double().numpy())
            self.kv.append(tuple(both))
        self.put(pool, scales)
        return self

    def put(self, pool, scales):
        self.k.copy_(pool[0])
        self.v.copy_(pool[1])
        if self.e4m3:
            self.ks.copy_(scales[0])
            self.vs.copy_(scales[1])

    def attend(self, hq, scale=0.0, causal=True, window=0, q=None, batch=None, **kw):
        q = bf16(self.g.standard_normal((self.rows, hq, self.d)) * 1.5) if q is None else q
        out = torch.full((self.rows, hq, self.d), 7.0, dtype=torch.bfloat16, device=self.k.device)
        self.cache.attend(batch or self.batch, q.to(self.k.device), out, scale=scale, causal=causal, window=window, **kw)
        return q, out

    def check(self, q, out, scale=0.0, causal=True, window=0):
        scale = scale or self.d ** -0.5
        got = out.double().cpu().numpy()
        q = q.double().cpu().numpy()
        for i, L in enumerate(self.lengths):
            r0, r1 = self.start[i], self.start[i + 1]
            if r0 == r1:
                continue
            k, v = self.kv[i]
            y, size, reach = ref.attend(q[r0:r1], k, v, L - (r1 - r0), scale, causal, window)
            weight = 2.0 ** -11 if self.e4m3 else 2.0 ** -8
            rel = 2 * (self.d + 8) * 2.0 ** -24 * reach[..., None] + 2.0 ** -21 + weight + max(L, 1) * 2.0 ** -24
            tol = np.abs(y) * 2.0 ** -8 + size * rel * 1.01 + 1e-30
            if self.e4m3:
                tol += 2.0 ** -25 * L * np.abs(v).max(initial=0)
            bad = np.abs(got[r0:r1] - y) > tol
            assert not bad.any(), (i, np.argwhere(bad)[:4], got[r0:r1][bad][:4], y[bad][:4], tol[bad][:4])
        assert (got[self.start[-1]:] == 7.0).all()      # rows behind the last sequence
        assert self.cache.status() == 0


FORMATS = [(False, 64), (False, 128), (True, 64), (True, 128)]


# ------------------------------------------------------------ append and read
def appended(w, hq, qkv, q_norm=None, k_norm=None, base=0.0, eps=1e-6):
    q_out = torch.full((w.rows, hq, w.d), 7.0, dtype=torch.bfloat16, device="cuda") if hq else None
    w.cache.append(w.batch, qkv.cuda(), q_out, q_norm=None if q_norm is None else q_norm.cuda(),
                   k_norm=None if k_norm is None else k_norm.cuda(), rms_eps=eps, rope_base=base)
    k, v = (torch.full((w.rows, w.hkv, w.d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w.cache.read(w.batch, k, v)
    assert w.cache.status() == 0
    return [None if x is None else x.double().cpu().numpy() for x in (q_out, k, v)]


@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("lengths,new,pad", [([1], [1], 0), ([37, 5, 300], [1, 1, 1], 0), ([40, 0, 131, 17], [33, 0, 131, 2], 3),
                                             ([1000003, 70], [3, 70], 1)])
def test_append(e4m3, d, page, lengths, new, pad):
    hkv, hq, base, eps = 3, 6, 1e4, 1e-5
    # a far position needs its own page only: its table is wide, its pool is not
    far = max(lengths) > 1000
    w = World([min(L, 300) for L in lengths], new, hkv, d, page, e4m3, seed=d + page, pad=pad)
    if far:
        w.lengths = lengths
        wide = np.full((len(lengths), -(-max(lengths) // page) + 1), -7, np.int32)
        for i, (L, n) in enumerate(zip(lengths, new)):
            for j, pg in enumerate(sorted({t // page for t in range(L - n, L)})):
                wide[i, pg] = w.table[i, j]
        w.table = wide
        w.batch = cp.Batch(torch.from_numpy(w.start).cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                           torch.from_numpy(wide).cuda(), w.rows)
    qkv = bf16(w.g.standard_normal((w.rows, (hq + 2 * hkv) * d)) * 3)
    gq, gk = (bf16(1 + 0.2 * w.g.standard_normal(d)) for _ in range(2))
    got = appended(w, hq, qkv, gq, gk, base, eps)
    x = qkv.double().numpy().reshape(w.rows, hq + 2 * hkv, d)
    pos = np.concatenate([np.arange(L - n, L) for L, n in zip(lengths, new)] + [np.zeros(0)])
    r = w.start[-1]
    q = ref.norm_rope(x[:r, :hq], pos, gq.double().numpy(), eps, base)
    k = ref.norm_rope(x[:r, hq:hq + hkv], pos, gk.double().numpy(), eps, base)
    v = x[:r, hq + hkv:]

    def pair(y):        # the size of each element's rotation pair
        m = np.hypot(y[..., :d // 2], y[..., d // 2:])
        return np.concatenate([m, m], -1)

    off = (d / 2 + 40) * 2.0 ** -24
    assert (np.abs(got[0][:r] - q) <= np.abs(q) * 2.0 ** -8 * 1.001 + pair(q) * off).all()
    if e4m3:
        s = np.exp2(ref.scale_exp(k).astype(np.float64))[..., None] * 2      # the next scale, at a border
        assert (np.abs(got[1][:r] - k) <= np.abs(k) * 2.0 ** -4 * 1.001 + s * 2.0 ** -10 + pair(k) * off).all()
        byte, e = ref.quantise(v)
        np.testing.assert_array_equal(got[2][:r], ref.dequantise(byte, e))
    else:
        assert (np.abs(got[1][:r] - k) <= np.abs(k) * 2.0 ** -8 * 1.001 + pair(k) * off).all()
        np.testing.assert_array_equal(got[2][:r], v)
    for y in got:       # rows behind the last sequence stay as they were
        assert (y[r:] == 7.0).all()


@pytest.mark.parametrize("e4m3,d", FORMATS)
def test_append_without_norm_or_rope_keeps_the_bits(e4m3, d):
    w = World([20, 9], [20, 4], 2, d, 16, e4m3, interleaved=True)
    x = w.g.standard_normal((w.rows, 4 * d)) * np.exp2(w.g.integers(-60, 60, (w.rows, 1)))
    x[3] = 0
    x[5, 7], x[6, 2 * d + 1] = np.nan, np.inf
    x[7] = np.linspace(-448, 448, 4 * d)
    qkv = bf16(x)
    _, k, v = appended(w, 0, qkv)
    want = qkv.double().numpy().reshape(w.rows, 4, d)
    if e4m3:
        want = ref.dequantise(*ref.quantise(want))
    np.testing.assert_array_equal(k, want[:, :2])
    np.testing.assert_array_equal(v, want[:, 2:])


def test_append_of_strided_rows_and_only_what_belongs():
    w = World([5, 40], [5, 2], 2, 64, 16, False, pad=2)
    before = [w.k.cpu().clone(), w.v.cpu().clone()]
    wide = bf16(w.g.standard_normal((w.rows, 8 * 64 + 16))).cuda()
    qkv = wide[:, 8:8 + 6 * 64]
    q = torch.zeros((w.rows, 4, 64), dtype=torch.bfloat16, device="cuda")[:, :2]
    w.cache.append(w.batch, qkv, q, rope_base=0.0)
    torch.testing.assert_close(q[:7].reshape(7, -1), qkv[:7, :128], rtol=0, atol=0)
    assert not q[7:].any()
    touched = torch.zeros_like(before[0], dtype=torch.bool)
    for i, (L, n) in enumerate(zip(w.lengths, w.new)):
        for t in range(L - n, L):
            touched[w.table[i, t // 16], :, t % 16] = True
    for now, was in zip((w.k, w.v), before):
        assert torch.equal(now.cpu()[~touched], was[~touched])
        assert (now.cpu() != was)[touched].any()


@pytest.mark.parametrize("e4m3,d", FORMATS)
def test_read_whole_sequences(e4m3, d):
    w = World([300, 0, 1, 77], [300, 0, 1, 70], 3, d, 32, e4m3, pad=2).fill()
    k, v = (torch.full((w.rows, 3, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w.cache.read(w.batch, k, v)
    only = torch.full_like(k, 7.0)
    w.cache.read(w.batch, None, only)
    for i, (L, n) in enumerate(zip(w.lengths, w.new)):
        for got, want in zip((k, v), w.kv[i]):
            np.testing.assert_array_equal(got[w.start[i]:w.start[i + 1]].double().cpu().numpy(), want[L - n:])
    assert (k[-2:] == 7).all() and torch.equal(only, v) and w.cache.status() == 0


# ------------------------------------------------------------ attention
SHAPES = [
    # lengths, new, query heads a kv head, pad
    ([1], [1], 1, 0),
    ([777], [1], 2, 0),
    ([63, 64, 65, 129, 1, 0, 2000], [1, 1, 1, 1, 1, 0, 1], 2, 3),
    ([300, 7, 5], [5, 3, 4], 4, 0),                       # a few rows each
    ([130, 40], [17, 40], 2, 1),
    ([500, 9, 1200], [129, 1, 1], 4, 2),                  # a chunk between steps
    ([256, 255], [256, 255], 2, 0),                       # prompts
    ([700], [333], 1, 0),
    ([90, 33], [40, 33], 8, 0),
    ([70], [9], 16, 0),
    ([20], [3], 64, 0),
    ([150], [77], 3, 0),                                  # a group that divides no tile
    ([3, 0, 10], [8, 5, 12], 2, 0),                       # more rows than positions: rows that see nothing
]


@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 33), (False, 100), (True, 1)])
def test_attend(e4m3, d, shape, causal, window):
    lengths, new, group, pad = SHAPES[shape]
    w = World(lengths, new, 2, d, (16, 32, 64, 128)[shape % 4], e4m3, seed=shape, pad=pad, interleaved=shape % 2 == 1).fill()
    q, out = w.attend(2 * group, causal=causal, window=window)
    w.check(q, out, causal=causal, window=window)


@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("new", [[1], [40]])
def test_attend_long(e4m3, d, new):
    """Long enough to be cut into parts and joined again."""
    w = World([20011], new, 1, d, 64, e4m3, seed=5).fill()
    q, out = w.attend(2)
    w.check(q, out)
    q, out = w.attend(2, window=9000)
    w.check(q, out, window=9000)


@pytest.mark.parametrize("e4m3,d", [(False, 64), (True, 128)])
@pytest.mark.parametrize("lengths,new", [([6000, 1500], [17, 17]), ([6000, 5900], [17, 17]), ([6000, 700, 40], [18, 17, 1]),
                                         ([6000, 300, 6000], [0, 20, 0])])
def test_attend_chunks_of_uneven_lengths(e4m3, d, lengths, new):
    """80 items or so in the plan's parts, and in fewer and longer ones where the lengths leave few blocks."""
    w = World(lengths, new, 40, d, 32, e4m3, seed=11, pad=1).fill()
    q, out = w.attend(40)
    w.check(q, out)


@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("window", [0, 90])
def test_attend_many_ragged_steps(e4m3, d, window):
    """More items than are resident at once, cut into parts of which some sequences have many and some one."""
    lengths = [1 + (i * 379) % 1500 for i in range(40)]
    w = World(lengths, [1 + i % 3 for i in range(40)], 2, d, 32, e4m3, seed=8, pad=1).fill()
    q, out = w.attend(4, window=window)
    w.check(q, out, window=window)


@pytest.mark.parametrize("e4m3,d", FORMATS)
def test_attend_many_steps_ignore_what_is_masked(e4m3, d):
    """As test_attend_ignores_what_is_masked, where the parts go through the workspace."""
    lengths = [300 + i for i in range(40)]
    w = World(lengths, [2] * 40, 1, d, 16, e4m3, seed=8).fill()
    pool = [w.k.cpu().clone(), w.v.cpu().clone()]
    for i, L in enumerate(lengths):         # the last position: the first of the two rows does not see it
        for x in pool:
            x[w.table[i, (L - 1) // 16], 0, (L - 1) % 16, 1] = 255 if e4m3 else -1
    w.put(pool, [None if s is None else s.cpu() for s in (w.ks, w.vs)])
    q, out = w.attend(2)
    assert torch.isnan(out[1::2, :, 1]).all()
    w.lengths, w.start, w.rows = [L - 1 for L in lengths], np.arange(41, dtype=np.int32), 40
    w.kv = [(k[:-1], v[:-1]) for k, v in w.kv]
    w.check(q[::2], out[::2])


@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("new", [[1, 2], [70, 9]])
def test_attend_sharp_and_scaled(e4m3, d, new):
    """Scores that grow along the sequence (the running maximum rises at every tile) and fall along it, sizes of
    values that differ by powers of two from token to token, and a scale of the caller's."""
    w = World([900, 401], new, 2, d, 32, e4m3, seed=9, spread=2.0)
    grow = np.ones((w.rows, 4, d)) / np.sqrt(d)
    inner = w.g.standard_normal

    class Growing:
        def __init__(self):
            self.calls = 0

        def standard_normal(self, shp):
            self.calls += 1
            x = inner(shp)
            if self.calls == 1:                 # sequence 0's keys: rising; the sizes (every second call) stay
                x = x * 0.1 + np.linspace(0, 60, shp[0])[:, None, None]
            if self.calls == 5:                 # sequence 1's keys: falling
                x = x * 0.1 + np.linspace(60, 0, shp[0])[:, None, None]
            if self.calls in (2, 6):
                x = x * 0
            return x

    w.g = Growing()
    w.fill()
    q = bf16(grow * 1.0)
    q, out = w.attend(4, scale=0.7, q=q)
    w.check(q, out, scale=0.7)


@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("new", [[2], [50]])
@pytest.mark.parametrize("window", [0, 20])
def test_attend_ignores_what_is_masked(e4m3, d, new, window):
    """NaN in K and V of positions that some rows do not see: those rows are as if it were not there, the rows that
    see it are NaN."""
    L = 200
    w = World([L], new, 1, d, 16, e4m3, seed=3).fill()
    bad = L - 1 if not window else L - new[0] - 10     # seen by the last row only; or by the first rows only
    pool = [w.k.cpu().clone(), w.v.cpu().clone()]
    for x in pool:
        x[w.table[0, bad // 16], 0, bad % 16, 3] = 255 if e4m3 else 0x7f80
        x[w.table[0, bad // 16], 0, bad % 16, 5] = 255 if e4m3 else -1
    w.put(pool, [None if s is None else s.cpu() for s in (w.ks, w.vs)])
    q, out = w.attend(2, window=window)
    k, v = w.kv[0]
    first = L - new[0]
    sees = np.array([t >= bad and (not window or bad > t - window) for t in range(first, L)])
    assert sees.any() and not sees.all() or new == [2] and window == 20
    y, size, reach = ref.attend(q.double().numpy(), k, v, first, d ** -0.5, True, window)
    got = out.double().cpu().numpy()
    assert np.isnan(got[sees]).all(-1).all() or np.isnan(got[sees][..., 5]).all()
    rel = 2 * (d + 8) * 2.0 ** -24 * reach[..., None] + 2.0 ** -21 + (2.0 ** -11 if e4m3 else 2.0 ** -8) + L * 2.0 ** -24
    tol = np.abs(y) * 2.0 ** -8 + size * rel * 1.01 + (2.0 ** -25 * L * np.abs(v).max() if e4m3 else 0)
    assert (np.abs(got[~sees] - y[~sees]) <= tol[~sees]).all()


@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("L,window", [(1500, 0), (1500, 700), (30011, 0)])
def test_attend_chunk_parts_ignore_what_is_masked(e4m3, d, L, window):
    """NaN in V at positions that some of a chunk's rows see, in a chunk whose positions are cut into parts (a few, that
    a cluster joins, and many)."""
    n = 50
    w = World([L], [n], 1, d, 64, e4m3, seed=3).fill()
    bad = [L - n + 20] + ([L - n - window + 30] if window else [])      # rows from 20 on; and rows up to 29
    pool = [w.k.cpu().clone(), w.v.cpu().clone()]
    for t in bad:
        pool[1][w.table[0, t // 64], 0, t % 64, 3] = 255 if e4m3 else -1
    w.put(pool, [None if s is None else s.cpu() for s in (w.ks, w.vs)])
    q, out = w.attend(2, window=window)
    got = out.double().cpu().numpy()
    k, v = w.kv[0]
    y, size, reach = ref.attend(q.double().numpy(), k, v, L - n, d ** -0.5, True, window)
    rel = 2 * (d + 8) * 2.0 ** -24 * reach[..., None] + 2.0 ** -21 + (2.0 ** -11 if e4m3 else 2.0 ** -8) + L * 2.0 ** -24
    tol = np.abs(y) * 2.0 ** -8 + size * rel * 1.01 + (2.0 ** -25 * L * np.abs(v).max() if e4m3 else 0)
    rows = np.arange(n)
    sees = rows >= 20
    if window:
        sees |= rows < 30
    assert np.isnan(got[sees][..., 3]).all() and not np.isnan(got[~sees]).any()
    other = np.arange(d) != 3
    assert (np.abs(got - y) <= tol)[..., other].all() and (np.abs(got - y) <= tol)[~sees].all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [[2], [50]])
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("which", ["k", "v", "kv"])
@pytest.mark.parametrize("gap,shift", [(10, 0), (20, 0), (40, 0), (100, 0), (115, -90)])
def test_attend_rows_that_do_not_see_a_far_scale(d, new, window, which, gap, shift):
    """One position's key or value 2^gap times the others (e4m3): rows that do not see it are as exact as if it were
    not there. `shift` lowers all scales, so that a rise of the gap stays in range.

    Beside the usual bound: weights are fp16 times the value's scale relative to the largest that the kernel keeps in
    one reference, which is at most 2^12 above those of a row's own, so that one below 2^-14 is off by 2^-25 next to a
    largest of 2^-12 at least (they start at 2^8): 2^-13 * L * max |v| over the positions the row sees, of which a
    smaller gap keeps its part, 2^(gap - 25)."""
    L = 200
    w = World([L], new, 1, d, 16, True, seed=3).fill()
    far = L - 1 if not window else L - new[0] - 10     # seen by the last row only; or by the first rows only
    scales = [w.ks.cpu().int(), w.vs.cpu().int()]
    kv = [x * 2.0 ** shift for x in w.kv[0]]
    for i in range(2):
        t = np.arange(L)
        scales[i][w.table[0, t // 16], :, t % 16] += shift
        if "kv"[i] in which:
            scales[i][w.table[0, far // 16], :, far % 16] += gap
    w.put([w.k.cpu(), w.v.cpu()], scales)
    first = L - new[0]
    q, out = w.attend(2, window=window)
    got, rows = out.double().cpu().numpy(), 0
    for r in range(new[0]):
        lo, hi = max(0, first + r - window + 1) if window else 0, first + r + 1
        if lo <= far < hi:
            continue
        rows += 1
        k, v = (x[lo:hi] for x in kv)
        y, size, reach = ref.attend(q.double().numpy()[r:r + 1], k, v, hi - lo - 1, d ** -0.5, True, 0)
        rel = 2 * (d + 8) * 2.0 ** -24 * reach[..., None] + 2.0 ** -21 + 2.0 ** -11 + L * 2.0 ** -24
        tol = np.abs(y) * 2.0 ** -8 + size * rel * 1.01 + 2.0 ** (min(gap, 12) - 25) * (hi - lo) * np.abs(v).max()
        assert (np.abs(got[r:r + 1] - y) <= tol).all(), (r, np.abs(got[r:r + 1] - y).max(), tol.max())
    assert rows == (new[0] - 1 if not window else max(0, new[0] - 10)) and w.cache.status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [[2], [50]])
def test_attend_zeros_between_values(d, new):
    """Keys and values of zeros have the least scale (e4m3), 2^-110, whatever the others'."""
    L = 400
    w = World([L], new, 1, d, 16, True, seed=6).fill()
    t = np.arange(0, L, 3)
    scales, pool = [w.ks.cpu().clone(), w.vs.cpu().clone()], [w.k.cpu().clone(), w.v.cpu().clone()]
    for i in range(2):
        scales[i][w.table[0, t // 16], :, t % 16] = 17
        pool[i][w.table[0, t // 16], :, t % 16] = 0
        w.kv[0][i][t] = 0
    w.put(pool, scales)
    q, out = w.attend(2)
    w.check(q, out)


@pytest.mark.parametrize("e4m3,d", FORMATS)
def test_a_window_as_large_as_its_type(e4m3, d):
    """...is none, also for rows in front of the first position."""
    for new in ([1, 12], [40, 40]):
        w = World([100, 10], new, 1, d, 16, e4m3, seed=6).fill()
        for causal in (True, False):
            q, out = w.attend(2, causal=causal, window=2 ** 31 - 1)
            w.check(q, out, causal=causal)


@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("lengths,new", [([777], [1]), ([5000], [3]), ([900, 70, 3000], [300, 1, 40])])
def test_in_place(e4m3, d, lengths, new):
    """out in q's place, and q_out in qkv's."""
    w = World(lengths, new, 2, d, 32, e4m3, seed=7).fill()
    q, out = w.attend(4)
    same = q.cuda()
    w.cache.attend(w.batch, same, same)
    assert torch.equal(same, out)
    qkv = bf16(w.g.standard_normal((w.rows, 8 * d)))
    gain = bf16(w.g.standard_normal(d)).cuda()
    apart = torch.empty((w.rows, 4, d), dtype=torch.bfloat16, device="cuda")
    w.cache.append(w.batch, qkv.cuda(), apart, gain, gain, rope_base=1e4)
    same = qkv.cuda()
    w.cache.append(w.batch, same, same[:, :4 * d].view(w.rows, 4, d), gain, gain, rope_base=1e4)
    assert torch.equal(same[:, :4 * d].reshape(w.rows, 4, d), apart) and torch.equal(same[:, 4 * d:].cpu(), qkv[:, 4 * d:])
    assert w.cache.status() == 0


@pytest.mark.parametrize("new", [[1], [40]])
def test_attend_infinite_scores(new):
    """Keys of the type's lowest value: their scores are minus infinity or far below the others, never NaN."""
    w = World([100], new, 1, 64, 16, False, seed=4).fill()
    pool = [w.k.cpu().clone(), w.v.cpu().clone()]
    for t in range(0, 60, 3):
        pool[0][w.table[0, t // 16], 0, t % 16] = -129       # 0xff7f: the lowest finite bf16
        w.kv[0][0][t] = -3.3895313892515355e38
    w.put(pool, (None, None))
    q = bf16(np.abs(w.g.standard_normal((w.rows, 2, 64))) + 0.1)
    q, out = w.attend(2, q=q)
    keep = [t for t in range(100) if t >= 60 or t % 3]
    got = out.double().cpu().numpy()
    for i in range(new[0]):
        see = [t for t in keep if t <= 100 - new[0] + i]
        y, size, reach = ref.attend(q.double().numpy()[i:i + 1], w.kv[0][0][see], w.kv[0][1][see], len(see) - 1, 64 ** -0.5,
                                    True, 0)
        rel = 2 * 72 * 2.0 ** -24 * reach[..., None] + 2.0 ** -21 + 2.0 ** -8 + 100 * 2.0 ** -24
        assert (np.abs(got[i] - y[0]) <= np.abs(y[0]) * 2.0 ** -8 + (size * rel)[0] * 1.01).all()


@pytest.mark.parametrize("e4m3,d", FORMATS)
def test_attend_strided_rows_and_repeatable(e4m3, d):
    w = World([150, 3000, 77], [60, 1, 77], 2, d, 32, e4m3, pad=1).fill()
    q0 = bf16(w.g.standard_normal((w.rows, 4, d)))
    q1, out = w.attend(4, q=q0)
    w.check(q1, out)
    wide = torch.zeros((w.rows, 5, 2 * d), dtype=torch.bfloat16, device="cuda")
    wide[:, :4, :d] = q0.cuda()
    dst = torch.full((4, w.rows, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    w.cache.attend(w.batch, wide[:, :4, :d], dst.permute(1, 0, 2)[..., :d])
    assert torch.equal(dst.permute(1, 0, 2)[..., :d], out) and (dst[..., d:] == 7).all()
    for _ in range(3):
        assert torch.equal(w.attend(4, q=q0)[1], out)


@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("new", [[1, 1], [30, 2]])
def test_attend_offsets_past_32_bits(e4m3, d, new):
    """The same rows out of a pool whose pages lie a gigabyte apart."""
    w = World([100, 50], new, 2, d, 16, e4m3, seed=1).fill()
    q, out = w.attend(4)
    step = (1 << 32) // (1 if e4m3 else 2) // 4 + 16 * 2 * d
    n = w.pages
    big = [torch.zeros((n - 1) * step + 2 * 16 * d, dtype=w.k.dtype, device="cuda") for _ in range(2)]
    far = [b.as_strided((n, 2, 16, d), (step, 16 * d, d, 1)) for b in big]
    for f, x in zip(far, (w.k, w.v)):
        f.copy_(x)
    c = cp.Cache(far[0], far[1], w.ks, w.vs)
    got = torch.full_like(out, 7.0)
    c.attend(w.batch, q.cuda(), got)
    assert torch.equal(got, out) and c.status() == 0
    k = torch.zeros((w.rows, 2, d), dtype=torch.bfloat16, device="cuda")
    c.read(w.batch, k, None)
    np.testing.assert_array_equal(k[0].double().cpu().numpy(), w.kv[0][0][100 - new[0]])


# ------------------------------------------------------------ what the device checks
@pytest.mark.parametrize("new", [[1, 1], [30, 2]])
def test_bad_pages_are_reported_and_skipped(new):
    w = World([100, 50], new, 1, 64, 16, False, seed=1).fill()
    q, good = w.attend(2)
    table = w.table.copy()
    table[0, 2], table[1, 3] = w.pages, -1          # position 48 of sequence 1, its last, is on page entry 3
    w.table, batch = table, None
    batch = w.batch_of()
    out = torch.full_like(good, 7.0)
    w.cache.attend(batch, q.cuda(), out)
    assert w.cache.status() == BOUNDS and torch.isfinite(out.float()).all()
    w.cache.clear_status()
    before = [w.k.clone(), w.v.clone()]
    qkv = bf16(w.g.standard_normal((w.rows, 3 * 64))).cuda()
    k = torch.full((w.rows, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    w.cache.read(batch, k, None)
    assert w.cache.status() == BOUNDS and (k[-1] == 7).all()
    w.cache.clear_status()
    w.cache.append(batch, qkv, torch.zeros((w.rows, 1, 64), dtype=torch.bfloat16, device="cuda"))
    assert w.cache.status() == BOUNDS
    page = int(w.table[0, 99 // 16])
    same = [i for i in range(w.pages) if i not in (page, int(w.table[0, 5]), int(w.table[0, 4]), int(w.table[0, 6]))]
    for now, was in zip((w.k, w.v), before):
        assert torch.equal(now[same], was[same])
    w.cache.clear_status()
    assert w.cache.status() == 0


@pytest.mark.parametrize("start,length", [([0, 3, 2], [50, 40]), ([0, 1, 99], [50, 40]), ([-5, 1, 2], [50, 40]),
                                          ([0, 1, 2], [-3, 40]), ([0, 1, 2], [50, 2 ** 31 - 1]), ([0, 40, 41], [50, 40])])
def test_bad_starts_and_lengths_are_clamped(start, length):
    w = World([50, 40], [1, 30], 1, 64, 16, False, seed=1).fill()
    batch = cp.Batch(torch.tensor(start, dtype=torch.int32, device="cuda"),
                     torch.tensor(length, dtype=torch.int32, device="cuda"), torch.from_numpy(w.table).cuda(), w.rows,
                     max_new=30, max_len=50)
    q = bf16(w.g.standard_normal((w.rows, 2, 64))).cuda()
    guard = torch.full((w.rows + 2, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    w.cache.attend(batch, q, guard[1:-1])
    assert w.cache.status() == BOUNDS
    assert (guard[0] == 7).all() and (guard[-1] == 7).all()


# ------------------------------------------------------------ streams, graphs, two calls at once
def test_another_stream_and_a_raw_handle():
    w = World([3000, 70], [1, 20], 2, 128, 64, True).fill()
    q, out = w.attend(4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other, raw = torch.full_like(out, 7.0), torch.full_like(out, 7.0)
    s.wait_stream(torch.cuda.current_stream())
    qd = q.cuda()
    s.wait_stream(torch.cuda.current_stream())
    w.cache.attend(w.batch, qd, other, stream=s)
    w.cache.attend(w.batch, qd, raw, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(other, out) and torch.equal(raw, out)


def test_captured_step_follows_lengths_tables_and_rows():
    """append + attend + read captured once, replayed while the sequences grow past pages and one ends."""
    w = World([30, 200, 15], [1, 1, 1], 2, 64, 16, True, seed=2).fill()
    lens = [30, 200, 15]
    need = [-(-(L + 40) // 16) for L in lens]
    pool = torch.zeros((sum(need) + 1, 2, 16, 64), dtype=torch.uint8, device="cuda")
    k, v, ks, vs = pool, pool.clone(), torch.zeros((sum(need) + 1, 2, 16), dtype=torch.uint8, device="cuda"), None
    vs = ks.clone()
    cache = cp.Cache(k, v, ks, vs)
    table = np.zeros((3, max(need)), np.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = np.arange(at, at + m)
        at += m
    start, length = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
    batch = cp.Batch(start, length, torch.from_numpy(table).cuda(), 3, max_new=1, max_len=max(need) * 16)
    qkv = torch.zeros((3, 8 * 64), dtype=torch.bfloat16, device="cuda")
    q, out = (torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gain = torch.ones(64, dtype=torch.bfloat16, device="cuda")

    def step():
        cache.append(batch, qkv, q, q_norm=gain, k_norm=gain, rope_base=1e4)
        cache.attend(batch, q, out)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(25):
        length += 1
        if i == 10:
            start.copy_(torch.tensor([0, 1, 1, 2], dtype=torch.int32))      # the second sequence has no row now
        if i > 10:
            length[1] -= 1
        qkv.copy_(torch.randn(3, 8 * 64))
        out.fill_(7.0)
        graph.replay()
        got, gq = out.clone(), q.clone()
        out.fill_(7.0)
        step()
        assert torch.equal(got, out) and torch.equal(gq, q), i
        assert i < 10 or (out[2] == 7).all()
    assert cache.status() == 0


@pytest.mark.parametrize("e4m3,d", [(False, 64), (True, 128)])
def test_captured_chunks_and_steps_follow_the_lengths(e4m3, d):
    """A call of every kernel, read by the next one in the graph, replayed at lengths that are cut up differently."""
    w = World([6000, 5900, 700], [17, 17, 1], 40, d, 32, e4m3, seed=12).fill()
    q = bf16(w.g.standard_normal((w.rows, 40, d))).cuda()
    outs = [torch.zeros((w.rows, 40, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    w.cache.attend(w.batch, q, outs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.cache.attend(w.batch, q, outs[0])
        outs[1].copy_(outs[0])
    for lengths in ([6000, 1500, 700], [6000, 5900, 1], [40, 30, 700], [900, 5900, 20], [6000, 5900, 700]):
        w.batch.length.copy_(torch.tensor(lengths, dtype=torch.int32))
        for x in outs:
            x.zero_()
        graph.replay()
        got = outs[1].clone()
        w.lengths, kv = lengths, w.kv
        w.kv = [(k[:L], v[:L]) for (k, v), L in zip(kv, lengths)]
        w.check(q, got)
        w.kv = kv
        outs[0].zero_()
        w.cache.attend(w.batch, q, outs[0])
        assert torch.equal(outs[0], got)


def test_two_captured_graphs_and_eager_calls_at_once():
    """Each call's workspace is its own: two graphs replayed together on two streams, with eager calls between."""
    w = World([6000, 4000], [1, 40], 2, 64, 32, False, seed=2).fill()
    qs = [bf16(w.g.standard_normal((w.rows, 4, 64))).cuda() for _ in range(3)]
    want = [w.attend(4, q=q)[1] for q in qs]
    outs, graphs = [torch.zeros_like(want[0]) for _ in range(3)], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            w.cache.attend(w.batch, qs[i], outs[i])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        w.cache.attend(w.batch, qs[2], outs[2])
        torch.cuda.synchronize()
        for o, y in zip(outs, want):
            assert torch.equal(o, y)


def test_a_workspace_of_the_callers():
    w = World([9000], [1], 1, 64, 64, False).fill()
    q, out = w.attend(2)
    need = w.cache.workspace_bytes(w.batch, 2)
    assert need > 0
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    got = torch.zeros_like(out)
    w.cache.attend(w.batch, q.cuda(), got, workspace=ws[:need])
    assert torch.equal(got, out) and (ws[need:] == 255).all()
    with pytest.raises(cp.CPError):
        w.cache.attend(w.batch, q.cuda(), got, workspace=ws[:need - 16])
    with pytest.raises(cp.CPError):
        w.cache.attend(w.batch, q.cuda(), got, workspace=ws[8:need + 8])


def test_loose_bounds_change_nothing_but_rounding():
    w = World([700, 33], [1, 20], 2, 64, 16, False).fill()
    q, out = w.attend(4)
    q, loose = w.attend(4, q=q, batch=w.batch_of(max_new=0, max_len=0))
    w.check(q, loose)


def test_binding_refuses_wrong_rows_and_devices():
    w = World([40], [4], 2, 64, 16, False).fill()
    q = torch.zeros((4, 4, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (q[:3], q[..., :32], q.cpu(), q.float(), q[:, :3]):
        with pytest.raises((ValueError, cp.CPError)):
            w.cache.attend(w.batch, bad, torch.zeros_like(bad))
    with pytest.raises(ValueError):
        w.cache.attend(w.batch, q[:, :1].expand(4, 4, 64), torch.zeros_like(q))
    with pytest.raises(cp.CPError):
        w.cache.read(w.batch, None, None)
    with pytest.raises(ValueError):
        w.cache.append(w.batch, torch.zeros((4, 5 * 64), dtype=torch.bfloat16, device="cuda"), q[:, :2])


def test_binding_refuses_other_types_of_the_same_size():
    w = World([20], [3], 1, 64).fill()
    q = torch.zeros((3, 2, 64), dtype=torch.float16, device="cuda")
    out, qkv = torch.zeros_like(q, dtype=torch.bfloat16), torch.zeros((3, 4 * 64), dtype=torch.bfloat16, device="cuda")
    for call in (lambda: w.cache.attend(w.batch, q, out), lambda: w.cache.attend(w.batch, out, q),
                 lambda: w.cache.append(w.batch, qkv.half(), out), lambda: w.cache.append(w.batch, qkv, q),
                 lambda: w.cache.append(w.batch, qkv, out, q_norm=q[0, 0]), lambda: w.cache.read(w.batch, q[:, :1]),
                 lambda: cp.Cache(w.k.view(torch.float16), w.v.view(torch.float16)),
                 lambda: cp.Cache(w.k.view(torch.uint8), w.v.view(torch.uint8).view(torch.float8_e5m2),
                                  torch.zeros(w.k.shape[:3], dtype=torch.uint8, device="cuda"),
                                  torch.zeros(w.k.shape[:3], dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    w.cache.attend(w.batch, out.view(torch.int16), out)
    assert w.cache.status() == 0


@pytest.mark.parametrize("e4m3,d", FORMATS)
def test_a_wait_that_runs_out_is_reported(e4m3, d):
    """The first load of every block is left out: the waits for it end, the call returns, the status says so, and the
    device goes on."""
    w = World([400, 300], [200, 9], 2, d, 32, e4m3).fill()
    q, good = w.attend(4)
    stalled = cp.Cache(w.k, w.v, w.ks, w.vs, timeout_ns=20_000_000, debug_stall=True)
    out = torch.full_like(good, 7.0)
    stalled.attend(w.batch, q.cuda(), out)
    assert stalled.status() == cp.CP_ERR_TIMEOUT
    stalled.clear_status()
    assert stalled.status() == 0        # (what a call that timed out leaves in out is not specified)
    assert torch.equal(w.attend(4, q=q)[1], good)


def test_batches_of_many_sequences():
    """More sequences than a warp looks at at once, most without rows."""
    n = 700
    new = [(3 if i % 50 == 7 else 40 if i % 300 == 11 else 0) for i in range(n)]
    w = World([50 + i % 30 if new[i] else 0 for i in range(n)], new, 1, 64, 16, False, seed=6, pad=1).fill()
    q, out = w.attend(2)
    w.check(q, out)
    k = torch.full((w.rows, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    w.cache.read(w.batch, k, None)
    for i in range(n):
        if new[i]:
            np.testing.assert_array_equal(k[w.start[i]:w.start[i + 1]].double().cpu().numpy(),
                                          w.kv[i][0][w.lengths[i] - new[i]:])


# ------------------------------------------------------------ together, in front of a frame
def test_talker_layer_in_front_of_a_frame():
    """Two prompt pieces and three steps through append and attend, each compared with attention over what the cache
    reads back; the last step's rows (16 heads of 128: the frame's 2048-wide input) then run one frame."""
    import synth
    from helpers import handle, run_gpu
    g = np.random.default_rng(0)
    hq, hkv, d, page = 16, 8, 128, 32
    pools = [torch.zeros((40, hkv, page, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((40, hkv, page), dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = cp.Cache(*pools, *scales)
    table = torch.from_numpy(g.permutation(40)[:20].reshape(2, 10).astype(np.int32)).cuda()
    gain = bf16(1 + 0.1 * g.standard_normal(d)).cuda()
    length = [0, 0]
    for new in ([100, 37], [60, 1], [1, 1], [1, 1], [1, 1]):
        length = [a + b for a, b in zip(length, new)]
        rows = sum(new)
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        batch = cp.Batch(torch.from_numpy(start).cuda(), torch.tensor(length, dtype=torch.int32, device="cuda"), table, rows,
                         max_new=max(new), max_len=max(length))
        qkv = bf16(g.standard_normal((rows, (hq + 2 * hkv) * d))).cuda()
        q, out = (torch.empty((rows, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        cache.append(batch, qkv, q, q_norm=gain, k_norm=gain, rope_base=1e6)
        cache.attend(batch, q, out)
        whole = np.concatenate([[0], np.cumsum(length)]).astype(np.int32)
        k, v = (torch.empty((sum(length), hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        cache.read(cp.Batch(torch.from_numpy(whole).cuda(), batch.length, table, sum(length)), k, v)
        assert cache.status() == 0
        for i in range(2):
            r, t = slice(start[i], start[i + 1]), slice(whole[i], whole[i + 1])
            y, size, reach = ref.attend(q[r].double().cpu().numpy(), k[t].double().cpu().numpy(), v[t].double().cpu().numpy(),
                                        length[i] - new[i], d ** -0.5, True, 0)
            rel = 2 * (d + 8) * 2.0 ** -24 * reach[..., None] + 2.0 ** -21 + 2.0 ** -11 + length[i] * 2.0 ** -24
            tol = np.abs(y) * 2.0 ** -8 + size * rel * 1.01 + 2.0 ** -25 * length[i] * float(v.abs().max())
            assert (np.abs(out[r].double().cpu().numpy() - y) <= tol).all()
    s = synth.shape("full")
    assert s["talker_hidden"] == hq * d
    fr = handle("full")
    h = out.float().reshape(2, hq * d).cpu().numpy()
    got = run_gpu(fr, s, h, synth.first_codes(s, 2), synth.sampler("greedy", 2))
    assert got["status"] == 0 and got["codes"].min() >= 0 and got["codes"].max() < s["vocab"]
