"""The paged cache's host side at the ends of its ranges, on the CPU (no device memory is touched)."""
import ctypes as C

import pytest
import torch

from persistent_megakernel_streaming_gb300 import build, cp
from test_cache import P, attend, batch, desc


@pytest.fixture(scope="module", autouse=True)
def L():
    build.build()
    return cp.lib()


def workspace(d, b, a):
    need = C.c_size_t()
    assert cp.lib().cp_cache_check(C.byref(d), C.byref(b), None, C.byref(a), C.byref(need)) == 0
    return need.value


@pytest.mark.parametrize("head_dim", [64, 128])
def test_the_plan_of_long_bounds(head_dim):
    """How 512 rows are cut up depends on the shares of 152 SMs, not on the bound, once blocks are long."""
    d = desc(head_dim=head_dim, page_size=128)
    sizes = [workspace(d, batch(sequences=1, rows=512, max_new=512, max_length=n, table_width=1 << 24), attend())
             for n in (100_000_000, 200_000_000, 500_000_000, 1 << 30, 2_000_000_000, (1 << 31) - 1025)]
    assert sizes[0] > 0 and len(set(sizes)) == 1, sizes


@pytest.mark.parametrize("kw", [dict(rows=2 ** 32 + 5), dict(rows=5, max_new=2 ** 32 + 2), dict(rows=5, max_len=2 ** 31),
                                dict(rows=5, max_len=2 ** 33 + 7), dict(rows=-2 ** 32 + 5)])
def test_binding_refuses_numbers_past_32_bits(kw):
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        cp.Batch(i, i[:2], torch.zeros(2, 4, dtype=torch.int32), **kw)
    assert cp.Batch(i, i[:2], torch.zeros(2, 4, dtype=torch.int32), 5, 2, 64).desc.max_length == 64
