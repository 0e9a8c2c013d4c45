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


@pytest.mark.parametrize("kw", [dict(token_stride=64), dict(token_stride=120), dict(head_stride=128), dict(head_stride=63 * 128),
                                dict(page_stride=7 * 64 * 128), dict(page_stride=8 * 64 * 128 - 8), dict(token_stride=8 * 128),
                                dict(token_stride=8 * 128, head_stride=120), dict(page_stride=8),
                                dict(dtype=1, k_scale=P, v_scale=P, scale_token_stride=8),
                                dict(dtype=1, k_scale=P, v_scale=P, scale_page_stride=64)])
def test_pages_that_overlap_are_refused(kw):
    assert cp.lib().cp_cache_check(C.byref(desc(**kw)), None, None, None, None) == 1


@pytest.mark.parametrize("kw", [dict(token_stride=8 * 128, head_stride=128), dict(token_stride=200, head_stride=63 * 200 + 128, page_stride=8 * 12728),
                                dict(page_stride=128, head_stride=100 * 128, token_stride=8 * 100 * 128),     # pages innermost
                                dict(pages=1, page_stride=8), dict(kv_heads=1, head_stride=8),
                                dict(pages=(1 << 31) - 1, page_stride=1 << 38),
                                dict(pages=1 << 20, page_stride=128, head_stride=1 << 38, kv_heads=2, token_stride=1 << 30),
                                dict(dtype=1, k_scale=P, v_scale=P, scale_token_stride=16, scale_head_stride=2, scale_page_stride=1024)])
def test_pages_of_any_order_are_accepted(kw):
    assert cp.lib().cp_cache_check(C.byref(desc(**kw)), None, None, None, None) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(out_stride=2040), 1), (dict(out_head_stride=120), 1), (dict(out_head_stride=64), 1), (dict(out_stride=128), 1),
    (dict(out_stride=64, out_head_stride=7 * 128), 1), (dict(out_stride=128, out_head_stride=7 * 128), 0),
    (dict(out_stride=4096, out_head_stride=256), 0), (dict(q_stride=8, q_head_stride=8), 0)])
def test_outputs_that_overlap_are_refused(kw, want):
    """7 rows of 16 heads of 128; what is only read may overlap."""
    assert cp.lib().cp_cache_check(C.byref(desc()), C.byref(batch()), None, C.byref(attend(**kw)), None) == want
    assert cp.lib().cp_cache_check(C.byref(desc()), C.byref(batch(rows=1, max_new=1)), None,
                                   C.byref(attend(out_stride=8)), None) == 0


def test_a_batch_stays_what_it_was_made_of():
    """The C side has the tensors' addresses: one that took another's place would not be read, and the old one freed."""
    i, table = torch.zeros(3, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    b = cp.Batch(i, i[:2], table, 5, 2, 64)
    for name, value in (("start", i.clone()), ("length", i[:2].clone()), ("pages", table.clone()), ("rows", 3), ("desc", None)):
        with pytest.raises(AttributeError):
            setattr(b, name, value)
    assert b.rows == 5 and b.start is i and b.pages is table
    b.length += 1               # in place, and what stood there again
    assert i.tolist() == [1, 1, 0]


@pytest.mark.parametrize("scale,want", [(2.3e38, 0), (2.4e38, 1), (3.4e38, 1), (1e-45, 0)])
def test_scales_next_to_the_ends_of_fp32(scale, want):
    """The kernels multiply by scale * log2(e): as an infinity it would make NaN of a score of zero."""
    assert cp.lib().cp_cache_check(C.byref(desc()), C.byref(batch()), None, C.byref(attend(scale=scale)), None) == want
