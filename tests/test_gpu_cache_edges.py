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
