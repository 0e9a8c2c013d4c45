"""The paged cache at the ends of its ranges: few tiles, zeros, rows and scales of wide range, bounds far above what a call
holds. The world, the reference and the derivation of the tolerances are test_gpu_cache's; the comparison here takes
NaN for wrong."""
import time

import numpy as np
import pytest
import torch

import test_gpu_cache as base
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
