"""The paged cache's checks of arguments and its look-up of positions, on the CPU (no device memory is touched),
and pins of the float64 reference the GPU tests compare with."""
import ctypes as C

import numpy as np
import pytest

from oracle import cache as ref
from persistent_megakernel_streaming_gb300 import build, cp

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 0x10000   # a stand-in for device memory: the checks look at addresses only


@pytest.fixture(scope="module", autouse=True)
def L():
    build.build()
    return cp.lib()


def desc(**kw):
    d = dict(dtype=0, kv_heads=8, head_dim=128, page_size=64, pages=100, k=P, v=2 * P)
    d.update(kw)
    return cp.CacheDesc(**d)


def batch(**kw):
    b = dict(sequences=3, rows=7, max_new=5, max_length=900, table_width=20, start=P, length=P, page_table=P)
    b.update(kw)
    return cp.BatchDesc(**b)


def append(**kw):
    a = dict(qkv=P, q_out=2 * P, q_heads=16, q_norm=P, k_norm=P, rms_eps=1e-6, rope_base=1e4)
    a.update(kw)
    return cp.AppendArgs(**a)


def attend(**kw):
    a = dict(q=P, out=2 * P, q_heads=16, causal=1)
    a.update(kw)
    return cp.AttendArgs(**a)


def check(d=None, b=None, ap=None, at=None):
    def ref_(x):
        return None if x is None else C.byref(x)
    return cp.lib().cp_cache_check(ref_(d), ref_(b), ref_(ap), ref_(at), None)


def test_plain_arguments_are_accepted():
    assert check(desc(), batch(), append(), attend()) == OK
    e = desc(dtype=1, k_scale=P, v_scale=P)
    assert check(e, batch(max_new=0, max_length=0), append(q_heads=0, q_out=None), attend(window=5, scale=0.5)) == OK
    assert check(desc()) == OK
    # a strided view, e.g. keys and values interleaved in one tensor
    assert check(desc(token_stride=256, head_stride=64 * 256, page_stride=8 * 64 * 256)) == OK


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID),
    (dict(kv_heads=0), INVALID), (dict(kv_heads=129), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED),
    (dict(pages=0), INVALID), (dict(dtype=1), INVALID), (dict(k_scale=P, v_scale=P), INVALID),
    (dict(dtype=1, k_scale=P), INVALID), (dict(k=P + 2), UNSUPPORTED), (dict(token_stride=132), UNSUPPORTED),
    (dict(timeout_ns=-1), INVALID), (dict(page_stride=-8), INVALID), (dict(page_stride=1 << 39), UNSUPPORTED), (dict(head_stride=1 << 40), UNSUPPORTED), (dict(dtype=1, k_scale=P, v_scale=P, token_stride=136), UNSUPPORTED)])
def test_bad_layouts_are_refused(kw, want):
    assert check(desc(**kw)) == want
    h = C.c_void_p()
    assert cp.lib().cp_cache_create(C.byref(desc(**kw)), 0, C.byref(h)) == want and not h.value


@pytest.mark.parametrize("kw,want", [
    (dict(sequences=0), INVALID), (dict(sequences=65536), INVALID), (dict(rows=0), INVALID), (dict(start=None), INVALID),
    (dict(length=None), INVALID), (dict(page_table=None), INVALID), (dict(max_new=-1), INVALID),
    (dict(max_length=-1), INVALID), (dict(max_length=20 * 64 + 1), INVALID), (dict(table_width=0), INVALID),
    (dict(table_stride=19), INVALID)])
def test_bad_batches_are_refused(kw, want):
    assert check(desc(), batch(**kw)) == want


def test_a_table_that_holds_more_than_32_bit_positions():
    assert check(desc(), batch(table_width=1 << 25, max_length=1 << 30)) == OK
    assert check(desc(), batch(table_width=1 << 25, max_length=0)) == OK       # bounded to what positions reach
    assert check(desc(), batch(table_width=1 << 25, max_length=(1 << 31) - 1)) == UNSUPPORTED


@pytest.mark.parametrize("kw,want", [
    (dict(qkv=None), INVALID), (dict(q_out=None), INVALID), (dict(q_heads=0), INVALID), (dict(q_heads=-1), INVALID),
    (dict(q_heads=1025), UNSUPPORTED), (dict(rms_eps=-1.0), INVALID), (dict(rms_eps=float("nan")), INVALID),
    (dict(rope_base=-1.0), INVALID), (dict(rope_base=float("inf")), INVALID), (dict(qkv_stride=4095), INVALID),
    (dict(qkv_stride=4100), UNSUPPORTED), (dict(q_stride=2047), INVALID), (dict(q_stride=2052), UNSUPPORTED),
    (dict(qkv=P + 8), UNSUPPORTED), (dict(q_norm=P + 2), UNSUPPORTED)])
def test_bad_appends_are_refused(kw, want):
    assert check(desc(), batch(), append(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(q_heads=0), INVALID), (dict(q_heads=12), INVALID),
    (dict(q_heads=8 * 65), UNSUPPORTED), (dict(window=-1), INVALID), (dict(scale=-0.5), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(q_stride=-8), INVALID),
    (dict(q_stride=2052), UNSUPPORTED), (dict(out_head_stride=130), UNSUPPORTED), (dict(out=P + 4), UNSUPPORTED)])
def test_bad_attends_are_refused(kw, want):
    assert check(desc(), batch(), None, attend(**kw)) == want


def test_more_rows_than_tiles_can_count_are_refused():
    assert check(desc(kv_heads=1), batch(rows=1 << 26), None, attend(q_heads=16)) == UNSUPPORTED
    assert check(desc(kv_heads=1), batch(rows=1 << 26), None, attend(q_heads=15)) == OK


def test_append_and_attend_need_a_batch_and_a_cache(L):
    assert check(desc(), None, append()) == INVALID
    assert check(desc(), None, None, attend()) == INVALID
    assert L.cp_cache_append(None, C.byref(batch()), C.byref(append()), None) == INVALID
    assert L.cp_cache_read(None, C.byref(batch()), P, P, None) == INVALID
    assert L.cp_cache_attend(None, C.byref(batch()), C.byref(attend()), None, 0, None) == INVALID
    assert L.cp_cache_status(None) == INVALID and L.cp_cache_clear_status(None) == INVALID
    L.cp_cache_destroy(None)


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    import torch
    with pytest.raises(ValueError):
        cp.Cache(torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        cp.Batch(torch.zeros(3, dtype=torch.int64), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32), 5)
    with pytest.raises(ValueError):
        cp.Batch(torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32), 5)
    with pytest.raises(ValueError):   # an expanded page table
        cp.Batch(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                 torch.zeros(1, 4, dtype=torch.int32).expand(2, 4), 5)


# ------------------------------------------------------------ positions
def slot(d, table, pos, head=0):
    arr = (C.c_int32 * len(table))(*table)
    return cp.lib().cp_test_slot(C.byref(d), arr, len(table), pos, head)


@pytest.mark.parametrize("page_size", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [0, 1])
def test_slots(page_size, dtype):
    d = desc(page_size=page_size, dtype=dtype, k_scale=P if dtype else None, v_scale=P if dtype else None)
    table = [3, 99, 0]
    for pos in (0, 1, page_size - 1, page_size, 2 * page_size - 1, 3 * page_size - 1):
        page, place = table[pos // page_size], pos % page_size
        assert slot(d, table, pos, 5) == ((page * 8 + 5) * page_size + place) * 128


def test_bad_pages_and_positions_have_no_slot():
    table = [3, -1, 100, 2 ** 31 - 1, -2 ** 31, 99]
    d = desc()
    assert slot(d, table, 63) >= 0 and slot(d, table, 5 * 64) >= 0
    for pos in (64, 2 * 64, 3 * 64, 4 * 64 + 63, 6 * 64, 2 ** 31 - 1, -1, -2 ** 31):
        assert slot(d, table, pos) == -1


def test_offsets_pass_32_bits():
    d = desc(pages=1 << 20, page_size=128)
    assert slot(d, [(1 << 20) - 1], 127, 7) == (((1 << 20) - 1) * 8 + 7) * 128 * 128 + 127 * 128
    s = desc(pages=1 << 20, page_stride=1 << 33)
    assert slot(s, [1000], 3) == 1000 * (1 << 33) + 3 * 128


# ------------------------------------------------------------ the reference itself
def test_reference_quantiser():
    x = np.array([[448.0, 1.0, -0.5, 0.0], [449.0, 1.0, 2.0 ** -9, -3.0], [0, 0, 0, 0], [np.inf, 1.0, np.nan, -2.0]])
    byte, e = ref.quantise(x)
    assert e.tolist() == [0, 1, -110, -7]
    v = ref.dequantise(byte, e)
    assert v[0].tolist() == [448.0, 1.0, -0.5, 0.0]
    assert v[1, 0] == 448.0 and v[1, 3] == -3.0 and v[1, 2] == 0.0   # 2^-10 of the scale: half the least step, to even
    assert v[2].tolist() == [0.0] * 4
    assert np.isnan(v[3, 0]) and np.isnan(v[3, 2]) and v[3, 1] == 1.0 and v[3, 3] == -2.0
    # ties go to the even byte: 17 lies between 16 and 18
    b, _ = ref.quantise(np.array([[17.0, 19.0, 448.0]]))
    assert ref.e4m3_table()[b[0]].tolist()[:2] == [16.0, 20.0]


def test_reference_against_torch_quantiser():
    import torch
    x = np.random.default_rng(0).standard_normal((50, 64)) * np.exp2(np.arange(50) - 25.0)[:, None]
    byte, e = ref.quantise(x)
    t = torch.from_numpy(x / np.exp2(e.astype(np.float64))[:, None]).to(torch.float8_e4m3fn)
    np.testing.assert_array_equal(byte, t.view(torch.uint8).numpy())


def test_reference_attention_of_equal_keys_is_the_mean():
    g = np.random.default_rng(1)
    q, v = g.standard_normal((3, 4, 8)), g.standard_normal((10, 2, 8))
    k = np.broadcast_to(g.standard_normal((1, 2, 8)), (10, 2, 8))
    out, _, _ = ref.attend(q, k, v, 7, 0.3, True, 0)
    for i in range(3):
        for h in range(4):
            np.testing.assert_allclose(out[i, h], v[:8 + i, h // 2].mean(0), rtol=1e-12)
    out, _, _ = ref.attend(q, k, v, 7, 0.3, False, 2)
    np.testing.assert_allclose(out[0, 0], v[6:, 0].mean(0), rtol=1e-12)
    out, _, _ = ref.attend(q, k, v, -2, 0.3, True, 0)
    assert not out[0].any() and not out[1].any()


def test_reference_rope_keeps_scores_relative():
    g = np.random.default_rng(2)
    q, k = g.standard_normal((1, 1, 64)), g.standard_normal((1, 1, 64))
    def dot(a, b):
        return float((ref.norm_rope(q, np.array([a]), None, 0, 1e4) * ref.norm_rope(k, np.array([b]), None, 0, 1e4)).sum())
    assert abs(dot(5, 3) - dot(1005, 1003)) < 1e-10 and abs(dot(5, 3) - dot(5, 4)) > 1e-3
