"""The paged cache at the ends of its ranges: few tiles, zeros, rows and scales of wide range, bounds far above what a call
holds. The world, the reference and the derivation of the tolerances are test_gpu_cache's; the comparison here takes
NaN for wrong."""
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
