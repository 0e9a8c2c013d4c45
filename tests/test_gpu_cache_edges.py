"""The paged cache at the ends of its ranges: few tiles, zeros, rows and scales of wide range, bounds far above what a call
holds. The world, the reference and the derivation of the tolerances are test_gpu_cache's; the comparison here takes
NaN for wrong."""
import time

import numpy as np
import pytest
import torch

import test_gpu_cache as base
from oracle import cache as ref
from persistent_megakernel_streaming_gb300 import build, cp
from test_gpu_cache import FORMATS, bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


class World(base.World):
    def check(self, q, out, scale=0.0, causal=True, window=0):
        assert torch.isfinite(out).all()
        super().check(q, out, scale, causal, window)


@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("L,n", [(128, 40), (128, 128), (100, 9), (256, 256)])
def test_streams_of_one_tile(e4m3, d, L, n):
    """The two threads of a row exchange their maxima and then their sums through the same words: the same result every
    time, with one tile (or none, as the second of two tiles of rows has) between the two."""
    w = World([L] * 16, [n] * 16, 2, d, 32, e4m3, seed=21).fill()
    q, out = w.attend(4)
    w.check(q, out)
    q = q.cuda()
    for _ in range(30):
        again = torch.full_like(out, 7.0)
        w.cache.attend(w.batch, q, again)
        assert torch.equal(again, out)


@pytest.mark.parametrize("e4m3,d", FORMATS)
def test_a_timeout_that_any_wait_may_meet(e4m3, d):
    """Whichever wait gives up first, a block only waits for what it has asked for and the call ends."""
    w = World([4000, 900, 300], [300, 200, 9], 2, d, 32, e4m3, seed=24).fill()
    q, good = w.attend(4)
    torch.cuda.synchronize()
    hasty = cp.Cache(w.k, w.v, w.ks, w.vs, timeout_ns=1)
    out, q = torch.full_like(good, 7.0), q.cuda()
    for _ in range(20):
        t0 = time.monotonic()
        hasty.attend(w.batch, q, out)
        status = hasty.status()
        assert status in (cp.CP_OK, cp.CP_ERR_TIMEOUT) and time.monotonic() - t0 < 1.0
        if status == cp.CP_OK:
            assert torch.equal(out, good)
        hasty.clear_status()
    again = torch.full_like(good, 7.0)
    w.cache.attend(w.batch, q, again)
    assert torch.equal(again, good) and w.cache.status() == cp.CP_OK


@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 33), (False, 100)])
@pytest.mark.parametrize("lengths,new", [([40, 300], [40, 300]), ([1000, 77], [40, 9]), ([130, 3], [1, 2]),
                                         ([10, 600], [60, 300]), ([9000], [40])])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -40])
def test_zero_queries_over_zero_keys(e4m3, d, causal, window, lengths, new, size):
    """...give the mean of the visible values: a tile whose last positions are masked, rows that see nothing, one part
    and several."""
    w = World(lengths, new, 2, d, 32, e4m3, seed=22, pad=1).fill()
    w.kv = [(k * 0, v) for k, v in w.kv]
    pool, scale = w.k.cpu().clone(), None if w.ks is None else w.ks.cpu().clone()
    for i, L in enumerate(lengths):
        t = np.arange(L)
        pool[w.table[i, t // 32], :, t % 32] = 0
        if e4m3:
            scale[w.table[i, t // 32], :, t % 32] = 17          # 2^-110, as rows of zeros are appended
    w.put([pool, w.v.cpu()], [scale, None if w.vs is None else w.vs.cpu()])
    q, out = w.attend(4, causal=causal, window=window, q=bf16(np.full((w.rows, 4, d), size)))
    w.check(q, out, causal=causal, window=window)


@pytest.mark.parametrize("e4m3,d", FORMATS)
def test_a_batch_of_zeros_through_append_and_attend(e4m3, d):
    """What a warm-up does: zeros through the norm, the rotation and the cache."""
    w = World([60, 200], [60, 33], 2, d, 16, e4m3, seed=25).fill()
    gain, zeros = torch.ones(d, dtype=torch.bfloat16, device="cuda"), torch.zeros((w.rows, 8 * d), dtype=torch.bfloat16, device="cuda")
    q = torch.full((w.rows, 4, d), 7.0, dtype=torch.bfloat16, device="cuda")
    w.cache.append(w.batch, zeros, q, gain, gain, rope_base=1e4)
    for i, (L, n) in enumerate(zip(w.lengths, w.new)):
        for x in w.kv[i]:
            x[L - n:] = 0
    q, out = w.attend(4, q=q)
    w.check(q, out)


# test_gpu_cache's own cases, whose comparison lets NaN pass, with this one
@pytest.fixture
def strict(monkeypatch):
    monkeypatch.setattr(base, "World", World)


@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("shape", range(len(base.SHAPES)))
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 33), (False, 100), (True, 1)])
def test_attend_is_finite(strict, e4m3, d, shape, causal, window):
    base.test_attend(e4m3, d, shape, causal, window)


@pytest.mark.parametrize("e4m3,d", FORMATS)
def test_long_ragged_and_sharp_are_finite(strict, e4m3, d):
    for new in ([1], [40]):
        base.test_attend_long(e4m3, d, new)
    for window in (0, 90):
        base.test_attend_many_ragged_steps(e4m3, d, window)
    for new in ([1, 2], [70, 9]):
        base.test_attend_sharp_and_scaled(e4m3, d, new)
    base.test_attend_many_steps_ignore_what_is_masked(e4m3, d)
    base.test_a_window_as_large_as_its_type(e4m3, d)
    base.test_attend_strided_rows_and_repeatable(e4m3, d)


@pytest.mark.parametrize("e4m3,d", [(False, 64), (True, 128)])
def test_uneven_captured_and_loose_are_finite(strict, e4m3, d):
    for lengths, new in (([6000, 700, 40], [18, 17, 1]), ([6000, 300, 6000], [0, 20, 0])):
        base.test_attend_chunks_of_uneven_lengths(e4m3, d, lengths, new)
    if e4m3:
        for n in ([2], [50]):
            base.test_attend_zeros_between_values(d, n)
    else:
        base.test_attend_chunks_of_uneven_lengths(e4m3, d, [6000, 5900], [17, 17])
        base.test_captured_chunks_and_steps_follow_the_lengths(e4m3, d)
        base.test_loose_bounds_change_nothing_but_rounding()
        base.test_batches_of_many_sequences()


# ------------------------------------------------------------ the lower end of a window, rows apart
@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("L,n,window", [(200, 2, 20), (200, 5, 20), (900, 3, 300), (200, 50, 20), (40, 2, 16), (1500, 2, 1)])
def test_rows_ignore_what_left_their_window(e4m3, d, L, n, window):
    """NaN and infinity in K and V of the first position that the first row sees: the others are as if it were not there."""
    w = World([L], [n], 1, d, 16, e4m3, seed=3).fill()
    bad = L - n - window + 1
    pool = [w.k.cpu().clone(), w.v.cpu().clone()]
    for x in pool:
        x[w.table[0, bad // 16], 0, bad % 16, 3] = 255 if e4m3 else 0x7f80
        x[w.table[0, bad // 16], 0, bad % 16, 5] = 255 if e4m3 else -1
    w.put(pool, [None if s is None else s.cpu() for s in (w.ks, w.vs)])
    q, out = w.attend(2, window=window)
    assert torch.isnan(out[0, :, 5]).all()
    k, v = w.kv[0]
    got = out.double().cpu().numpy()[1:]
    y, size, reach = ref.attend(q.double().numpy()[1:], k, v, L - n + 1, d ** -0.5, True, window)
    rel = 2 * (d + 8) * 2.0 ** -24 * reach[..., None] + 2.0 ** -21 + (2.0 ** -11 if e4m3 else 2.0 ** -8) + L * 2.0 ** -24
    tol = np.abs(y) * 2.0 ** -8 + size * rel * 1.01 + (2.0 ** -25 * L * np.abs(v).max() if e4m3 else 0)
    assert len(got) == n - 1 and (np.abs(got - y) <= tol).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [2, 4])
@pytest.mark.parametrize("which", ["k", "v", "kv"])
@pytest.mark.parametrize("gap,shift", [(10, 0), (20, 0), (40, 0), (100, 0), (115, -90)])
def test_a_far_scale_that_left_the_window(d, n, which, gap, shift):
    """As test_gpu_cache's test_attend_rows_that_do_not_see_a_far_scale, with its bound, for the first position that the
    first of a few rows sees."""
    L, window = 200, 20
    w = World([L], [n], 1, d, 16, True, seed=3).fill()
    far = L - n - window + 1
    scales = [w.ks.cpu().int(), w.vs.cpu().int()]
    k, v = (x * 2.0 ** shift for x in w.kv[0])
    t = np.arange(L)
    for i in range(2):
        scales[i][w.table[0, t // 16], :, t % 16] += shift
        if "kv"[i] in which:
            scales[i][w.table[0, far // 16], :, far % 16] += gap
    w.put([w.k.cpu(), w.v.cpu()], scales)
    q, out = w.attend(2, window=window)
    got = out.double().cpu().numpy()[1:]
    y, size, reach = ref.attend(q.double().numpy()[1:], k, v, L - n + 1, d ** -0.5, True, window)
    rel = 2 * (d + 8) * 2.0 ** -24 * reach[..., None] + 2.0 ** -21 + 2.0 ** -11 + window * 2.0 ** -24
    tol = np.abs(y) * 2.0 ** -8 + size * rel * 1.01 + 2.0 ** (min(gap, 12) - 25) * window * np.abs(v[far + 1:]).max()
    assert len(got) == n - 1 and (np.abs(got - y) <= tol).all() and w.cache.status() == 0


# ------------------------------------------------------------ queries of wide range
def channels(w, up):
    """World of one sequence, whose keys' channel c is 2^up[c] times what it would be (as the cache holds it)."""
    inner, calls = w.g.standard_normal, []

    class Wide:
        def standard_normal(self, shp):
            calls.append(1)
            x = inner(shp)
            return x * np.exp2(up) if len(calls) == 1 else x * 0 if len(calls) == 2 else x

    w.g = Wide()
    return w.fill()


def compare(w, q, out, window=0):
    """test_gpu_cache's bound, and the 2^-12 that a score over e4m3 may be off for its q in fp16: twice (the weight and
    the sum) ln 2 times that, below 2^-11."""
    (k, v), (L,), (n,) = w.kv[0], w.lengths, w.new
    y, size, reach = ref.attend(q.double().cpu().numpy(), k, v, L - n, w.d ** -0.5, True, window)
    rel = 2 * (w.d + 8) * 2.0 ** -24 * reach[..., None] + 2.0 ** -21 + (2.0 ** -10 if w.e4m3 else 2.0 ** -8) + L * 2.0 ** -24
    tol = np.abs(y) * 2.0 ** -8 + size * rel * 1.01 + (2.0 ** -25 * L * np.abs(v).max() if w.e4m3 else 0)
    bad = ~(np.abs(out.double().cpu().numpy() - y) <= tol)
    assert not bad.any() and w.cache.status() == 0, np.argwhere(bad)[:4]


@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("L,n", [(300, 2), (300, 40), (6000, 1), (6000, 50), (700, 700)])
@pytest.mark.parametrize("width", [8, 12, 16, 18, 24, 40])
def test_queries_of_wide_range(e4m3, d, L, n, width):
    """Channels whose keys are up to 2^width larger and whose queries are as much smaller: each counts alike in a score."""
    up = np.linspace(0, width, d)
    w = channels(World([L], [n], 2, d, 32, e4m3, seed=26), up)
    q, out = w.attend(4, q=bf16(w.g.standard_normal((n, 4, d)) * np.exp2(-up)))
    compare(w, q, out)


@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("n", [2, 40])
@pytest.mark.parametrize("shift", [-110, -99, -60, 60, 100])
def test_queries_of_any_size(e4m3, d, n, shift):
    """All of q 2^shift times as large, and the keys as much smaller (but for what the least scale leaves of them)."""
    w = channels(World([300], [n], 2, d, 32, e4m3, seed=27), np.full(d, -float(shift)))
    q, out = w.attend(4, q=bf16(w.g.standard_normal((n, 4, d)) * 2.0 ** shift))
    compare(w, q, out)


@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("n", [1, 2, 40])
@pytest.mark.parametrize("top", [0, 19, 120])
def test_a_channel_of_q_that_no_key_has(e4m3, d, n, top):
    """One element of q far above the others meets keys of zero there: the score is the others'."""
    up = np.full(d, 20.0 if top < 100 else 0.0)
    w = channels(World([300], [n], 2, d, 32, e4m3, seed=28), up)
    w.kv[0][0][..., 5] = 0
    t, pool = np.arange(300), w.k.cpu().clone()
    pool[w.table[0, t // 32], :, t % 32, 5] = 0
    w.put([pool, w.v.cpu()], [None if s is None else s.cpu() for s in (w.ks, w.vs)])
    q = w.g.standard_normal((n, 4, d)) * np.exp2(-up)
    q[..., 5] = 2.0 ** top
    q, out = w.attend(4, q=bf16(q))
    compare(w, q, out)


# ------------------------------------------------------------ bounds far above what a call holds
@pytest.mark.parametrize("e4m3,d", [(False, 64), (True, 128)])
@pytest.mark.parametrize("lengths,new,group,hkv", [([777], [1], 2, 1), ([1000, 40], [2, 1], 1, 1), ([500], [300], 2, 2),
                                                   ([2432], [2432], 2, 8)])
def test_a_table_that_holds_as_many_positions_as_there_are(e4m3, d, lengths, new, group, hkv):
    """max_len as large as it may be: what a call cuts up is the bound, what it computes the lengths."""
    w = World(lengths, new, hkv, d, 128, e4m3, seed=29).fill()
    wide = torch.full((len(lengths), 1 << 24), -7, dtype=torch.int32, device="cuda")
    wide[:, :w.table.shape[1]] = torch.from_numpy(w.table).cuda()
    loose = cp.Batch(w.batch.start, w.batch.length, wide, w.rows, max_new=max(new))
    q, out = w.attend(group * hkv, batch=loose)
    w.check(q, out)
    q, out = w.attend(group * hkv, batch=loose, window=200)
    w.check(q, out, window=200)


# ------------------------------------------------------------ the largest elements
LOWEST = -3.3895313892515355e38         # of bf16


@pytest.mark.parametrize("d", [64, 128])
def test_the_largest_elements_stay_finite_in_e4m3(d):
    w = World([40], [40], 2, d, 16, True, seed=30)
    x = w.g.standard_normal((40, 4 * d))
    x[0], x[1, 3], x[2, d + 5] = LOWEST, -LOWEST, LOWEST
    x[3, ::2], x[4, ::7], x[5, 2] = 2.0 ** 127 * 1.9375, -(2.0 ** 127) * 1.9296875, 2.0 ** 127 * 1.875
    x[6, 1], x[6, 2], x[6, 3] = LOWEST, np.inf, np.nan
    qkv = bf16(x)
    w.cache.append(w.batch, qkv.cuda())
    k, v = (torch.empty((40, 2, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w.cache.read(w.batch, k, v)
    want = qkv.double().numpy().reshape(40, 4, d)
    most = 2.0 ** 127 * 1.875                                   # the largest step below 2^128
    byte, e = ref.quantise(np.where(np.isfinite(want), np.clip(want, -most, most), want))
    want = ref.dequantise(byte, e)
    np.testing.assert_array_equal(k.double().cpu().numpy(), want[:, :2])
    np.testing.assert_array_equal(v.double().cpu().numpy(), want[:, 2:])
    assert not torch.isinf(k).any() and not torch.isinf(v).any() and w.cache.status() == 0


@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("n", [1, 40])
def test_keys_of_the_lowest_value_weigh_nothing(e4m3, d, n):
    """...to queries above zero: scores below all others, or minus infinity, through append and attend."""
    L = 100
    w = World([L], [L], 1, d, 16, e4m3, seed=31)
    x = w.g.standard_normal((L, 2 * d))
    low = np.arange(0, 60, 3)
    x[low, :d] = LOWEST
    w.cache.append(w.batch, bf16(x).cuda())
    k, v = (torch.empty((L, 1, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w.cache.read(w.batch, k, v)
    keep = np.setdiff1d(np.arange(L), low)
    w.start, w.new, w.rows = np.array([0, n], np.int32), [n], n
    w.batch = w.batch_of(max_new=n)
    q, out = w.attend(2, q=bf16(np.abs(w.g.standard_normal((n, 2, d))) + 0.1))
    k, v = k.double().cpu().numpy()[keep], v.double().cpu().numpy()[keep]
    w.lengths, w.kv = [len(keep)], [(k, v)]             # the rows are the last positions, none of them low
    compare(w, q, out)


# ------------------------------------------------------------ what the binding refuses
def test_binding_refuses_what_its_types_would_change():
    """A window past 32 bits would lose its upper bits, a scale or a base below fp32 would be "none given"."""
    w = World([40], [2], 1, 64).fill()
    q, out = w.attend(2)
    q = q.cuda()
    qkv = torch.zeros((2, 4 * 64), dtype=torch.bfloat16, device="cuda")
    for call in (lambda: w.cache.attend(w.batch, q, out, window=2 ** 32 + 7), lambda: w.cache.attend(w.batch, q, out, window=2 ** 31),
                 lambda: w.cache.workspace_bytes(w.batch, 2, window=2 ** 32), lambda: w.cache.attend(w.batch, q, out, scale=1e-50),
                 lambda: w.cache.append(w.batch, qkv, out, rope_base=1e-50)):
        with pytest.raises(ValueError):
            call()
    w.check(q, out)


@pytest.mark.parametrize("e4m3,d", FORMATS)
@pytest.mark.parametrize("scale", [1e-44, 1e-30])
def test_scales_next_to_zero(e4m3, d, scale):
    """...make every visible position count alike; masked ones stay out."""
    w = World([300, 70], [40, 2], 2, d, 32, e4m3, seed=33).fill()
    for window in (0, 33):
        q, out = w.attend(4, scale=scale, window=window)
        w.check(q, out, scale=scale, window=window)
