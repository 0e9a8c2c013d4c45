"""Checks of arguments of the projections, of verification and of the pages' management, on the CPU (no device memory is
touched), and pins of the plain references that the GPU tests compare with."""
import ctypes as C

import numpy as np
import pytest

from oracle import linear, verify
from oracle.pages import Pool
from persistent_megakernel_streaming_gb300 import build, cp

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 0x10000   # a stand-in for device memory: the checks look at addresses only


@pytest.fixture(scope="module", autouse=True)
def L():
    build.build()
    return cp.lib()


def of(cls, base, kw):
    return cls(**{**base, **kw})


LINEAR = dict(features=100, width=256, group=64, q=P, scale=P)
ARGS = dict(x=P, rows=3, out=2 * P)


def linear_check(d=None, a=None):
    args = None if a is None else C.byref(of(cp.LinearArgs, ARGS, a))
    return cp.lib().cp_linear_check(C.byref(of(cp.LinearDesc, LINEAR, d or {})), args)


@pytest.mark.parametrize("d,want", [
    ({}, OK), (dict(zero=P), OK), (dict(gated=1), OK), (dict(width=32, group=32), OK), (dict(features=1), OK),
    (dict(q=None), INVALID), (dict(scale=None), INVALID), (dict(features=0), INVALID), (dict(width=0), INVALID),
    (dict(width=250), INVALID), (dict(group=0), INVALID), (dict(group=16), UNSUPPORTED), (dict(group=256), UNSUPPORTED),
    (dict(features=101, gated=1), INVALID), (dict(features=(1 << 24) + 1), UNSUPPORTED), (dict(width=(1 << 20) + 64), UNSUPPORTED),
    (dict(width=-64), INVALID), (dict(timeout_ns=-1), INVALID), (dict(timeout_ns=5), OK)])
def test_weights(d, want, L):
    assert linear_check(d) == want
    h = C.c_void_p()
    if want:
        assert L.cp_linear_create(C.byref(of(cp.LinearDesc, LINEAR, d)), 0, C.byref(h)) == want and not h.value


@pytest.mark.parametrize("a,want", [
    ({}, OK), (dict(add=2 * P), OK), (dict(out_dtype=1, x_stride=264, out_stride=101, add=P + 4, add_stride=100), OK),
    (dict(rows=65535), OK), (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(rows=0), INVALID), (dict(rows=65536), UNSUPPORTED),
    (dict(out_dtype=2), INVALID), (dict(out_dtype=-1), INVALID), (dict(x=P + 8), UNSUPPORTED), (dict(x_stride=260), UNSUPPORTED),
    (dict(x_stride=-256), INVALID), (dict(x_stride=248), INVALID), (dict(x_stride=8, rows=1), OK), (dict(out_stride=99), INVALID), (dict(out=P + 1), UNSUPPORTED),
    (dict(out_dtype=1, out=P + 2), UNSUPPORTED), (dict(add=P + 1), UNSUPPORTED), (dict(add=P, add_stride=-1), INVALID),
    (dict(x_stride=1 << 39), UNSUPPORTED), (dict(x_stride=(1 << 39) - 8), OK), (dict(out_stride=1 << 41), UNSUPPORTED)])
def test_applications(a, want):
    assert linear_check({}, a) == want


def test_null_objects_are_refused(L):
    assert L.cp_linear_check(None, None) == INVALID
    assert L.cp_linear_apply(None, C.byref(of(cp.LinearArgs, ARGS, {})), None) == INVALID
    assert L.cp_linear_unpack(None, P, None) == INVALID
    assert L.cp_linear_status(None) == INVALID and L.cp_linear_clear_status(None) == INVALID
    assert L.cp_pages_check(None) == INVALID
    assert L.cp_pages_fork(None, P, P, 1, None) == INVALID and L.cp_pages_grow(None, P, P, 9, P, None) == INVALID
    assert L.cp_pages_trim(None, P, None) == INVALID and L.cp_pages_compact(None, P, 9, P, None) == INVALID
    assert L.cp_pages_status(None) == INVALID and L.cp_pages_clear_status(None) == INVALID
    assert L.cp_cache_copy(None, P, 1, P, None) == INVALID
    assert L.cp_verify(None, 0, P, 100, None) == INVALID and L.cp_verify_check(None, None) == INVALID
    assert L.cp_linear_create(None, 0, None) == INVALID and L.cp_pages_create(None, 0, None) == INVALID
    L.cp_linear_destroy(None)
    L.cp_pages_destroy(None)


PAGES = dict(pages=100, page_size=64, sequences=7, table_width=20, refs=P, page_table=P, length=P)


@pytest.mark.parametrize("d,want", [
    ({}, OK), (dict(page_size=16, table_stride=21), OK), (dict(sequences=1, table_stride=3), OK), (dict(refs=None), INVALID),
    (dict(page_table=None), INVALID), (dict(length=None), INVALID), (dict(pages=0), INVALID), (dict(pages=(1 << 30) + 1), UNSUPPORTED),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(page_size=0), INVALID), (dict(sequences=0), INVALID),
    (dict(sequences=65536), UNSUPPORTED), (dict(table_width=0), INVALID), (dict(table_stride=19), INVALID), (dict(table_stride=-1), INVALID)])
def test_pools(d, want, L):
    desc = of(cp.PagesDesc, PAGES, d)
    assert L.cp_pages_check(C.byref(desc)) == want
    h = C.c_void_p()
    if want:
        assert L.cp_pages_create(C.byref(desc), 0, C.byref(h)) == want and not h.value


VERIFY = dict(sequences=3, rows=9, vocab=10000, start=P, logits=P, draft=P, temperature=P, u_accept=P, u_token=P, accepted=P, token=P)


@pytest.mark.parametrize("a,want", [
    ({}, OK), (dict(dtype=1, draft_logits=P, prob=P, logits_stride=10001, draft_stride=1), OK), (dict(start=None), INVALID),
    (dict(logits=None), INVALID), (dict(draft=None), INVALID), (dict(temperature=None), INVALID), (dict(u_accept=None), INVALID),
    (dict(u_token=None), INVALID), (dict(accepted=None), INVALID), (dict(token=None), INVALID), (dict(sequences=0), INVALID),
    (dict(sequences=65536), UNSUPPORTED), (dict(rows=0), INVALID), (dict(rows=(1 << 20) + 1), UNSUPPORTED), (dict(vocab=0), INVALID),
    (dict(vocab=(1 << 24) + 1), UNSUPPORTED), (dict(dtype=2), INVALID), (dict(logits_stride=-1), INVALID), (dict(draft_stride=-1), INVALID),
    (dict(logits=P + 2), UNSUPPORTED), (dict(dtype=1, logits=P + 2), OK), (dict(dtype=1, draft_logits=P + 1), UNSUPPORTED),
    (dict(rows=1 << 20, vocab=1 << 24), UNSUPPORTED)])
def test_verifications(a, want, L):
    need = C.c_size_t(7)
    args = of(cp.VerifyArgs, VERIFY, a)
    assert L.cp_verify_check(C.byref(args), C.byref(need)) == want
    assert (need.value > 0) == (want == OK)
    if want:
        assert L.cp_verify(C.byref(args), 0, P, 1 << 30, None) == want
    else:
        assert L.cp_verify(C.byref(args), 0, None, 1 << 30, None) == INVALID
        assert L.cp_verify(C.byref(args), 0, P, need.value - 1, None) == INVALID
        assert L.cp_verify(C.byref(args), 0, P + 8, 1 << 30, None) == UNSUPPORTED


def test_a_small_vocabulary_needs_no_workspace(L):
    need = C.c_size_t(7)
    assert L.cp_verify_check(C.byref(of(cp.VerifyArgs, VERIFY, dict(vocab=2048))), C.byref(need)) == OK and need.value == 0


@pytest.mark.parametrize("vocab", [4097, 4603, 4604, 4605, 4606, 5113, 5114, 8184, 8185, 8186, 8187, 8188, 8189, 8190, 16380, 16381, 32000, 1 << 24])
def test_the_workspace_is_the_same_for_both_types(L, vocab):
    a = of(cp.VerifyArgs, VERIFY, dict(vocab=vocab))
    sizes = []
    for a.dtype in (0, 1):
        n = C.c_size_t()
        assert L.cp_verify_check(C.byref(a), C.byref(n)) == OK
        sizes.append(n.value)
    assert sizes == [cp.verify_workspace_bytes(a.sequences, a.rows, vocab)] * 2


def test_the_workspace_depends_on_sizes_alone():
    assert cp.verify_workspace_bytes(3, 9, 1000) == cp.verify_workspace_bytes(3, 9, 1000)
    assert cp.verify_workspace_bytes(3, 18, 100000) > cp.verify_workspace_bytes(3, 9, 100000) > 0


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    import torch
    with pytest.raises(ValueError):
        cp.Linear(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        cp.Pages(torch.zeros(4, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 16)
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        cp.verify(torch.zeros(2, 5), z, z, z, z, z, z, z)


# ------------------------------------------------------------ the references themselves
def test_reference_weights():
    q = np.array([[0x21, 0xf8]], np.uint8)
    np.testing.assert_array_equal(linear.nibbles(q), [[1, 2, 8, 15]])
    np.testing.assert_array_equal(linear.weights(q, np.array([[0.5, 2.0]])), [[-3.5, -3.0, 0.0, 14.0]])
    np.testing.assert_array_equal(linear.weights(q, np.array([[1.0, 1.0]]), np.array([[1, 15]])), [[0, 1, -7, 0]])
    # 3 * (1 + 2^-7) has nine bits: a tie, to even
    assert linear.bf16(np.array([3 * (1 + 2.0 ** -7)]))[0] == 3.03125


def test_reference_projection():
    w = np.array([[1.0, 0], [0, 2.0]])
    y, off = linear.apply(np.array([[3.0, 5.0]]), w, False, np.array([[1.0, 1.0]]))
    assert y.tolist() == [[4.0, 11.0]] and (off > 0).all() and (off < 1e-5).all()
    y, _ = linear.apply(np.array([[3.0, 5.0]]), w, True)
    assert abs(y[0, 0] - 3 / (1 + np.exp(-3.0)) * 10) < 1e-12


def test_reference_verification_keeps_the_targets_distribution():
    """Over a grid of uniforms, what comes out first has the target's probabilities."""
    x, y = np.log([[0.5, 0.2, 0.3]] * 2), np.log([[0.2, 0.7, 0.1]] * 2)
    seen = np.zeros(3)
    n = 40
    for d, q in enumerate([0.2, 0.7, 0.1]):
        for ua in (np.arange(n) + 0.5) / n:
            for ut in (np.arange(n) + 0.5) / n:
                (one,), _ = verify.verify([0, 2], x, np.array([d, 0]), [ua, 0], [ut], [1.0], y)
                seen[d if one["accepted"] else one["token"]] += q / n / n
    np.testing.assert_allclose(seen, [0.5, 0.2, 0.3], atol=0.02)


def test_reference_pool():
    p = Pool([0] * 6, [[-1] * 4] * 3, [0] * 3, 16)
    assert p.grow([20, 0, 0]) == ([], 0) and p.table[0].tolist() == [0, 1, -1, -1]
    p.fork([0], [2])
    assert p.refs.tolist() == [2, 2, 0, 0, 0, 0]
    assert p.grow([1, 0, 1]) == ([(1, 2)], 1) and p.refs.tolist() == [2, 1, 1, 0, 0, 0]
    assert p.table[0].tolist() == [0, 2, -1, -1] and p.table[2].tolist() == [0, 1, -1, -1]
    p.trim([0, 0, 99])
    assert p.refs.tolist() == [1, 1, 0, 0, 0, 0] and p.table[0].tolist() == [-1] * 4
    p.grow([40, 0, 0])
    p.trim([40, 0, 16])
    assert p.compact() == ([(4, 1)], 1) and p.table[0].tolist() == [2, 3, 1, -1] and not p.bad
