"""Limits of the operators' sizes that include/cp.h states, at their ends, on the CPU."""
import ctypes as C

import pytest

from persistent_megakernel_streaming_gb300 import build, cp

OK, UNSUPPORTED = 0, 2
P = 0x10000   # a stand-in for device memory: the checks look at addresses only


@pytest.fixture(scope="module", autouse=True)
def L():
    build.build()
    return cp.lib()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rows,vocab,want", [
    (1 << 20, 1 << 22, OK), (1 << 20, (1 << 22) - 4095, OK), (700000, 4096 * 1533, OK), (1 << 18, 1 << 24, OK), (1, 1 << 24, OK),
    (65, 16519105, OK), ((1 << 20) - 1, 1 << 22, OK), (1 << 20, 1, OK), (1 << 20, 1 << 23, UNSUPPORTED), (1 << 20, 1 << 24, UNSUPPORTED),
    (1 << 19, 1 << 24, UNSUPPORTED)])
def test_rows_and_vocabulary_of_a_verification(L, dtype, rows, vocab, want):
    inside = rows * -(-vocab // 4096) <= 1 << 30
    assert inside == (want == OK)
    a = cp.VerifyArgs(3, rows, vocab, dtype, P, P, 0, None, 0, P, P, P, P, P, P, None)
    need = C.c_size_t()
    assert L.cp_verify_check(C.byref(a), C.byref(need)) == want
    assert (need.value > 0) == (want == OK and vocab > 4096)


@pytest.mark.parametrize("sequences,vocab,some", [(1, 1, False), (2048, 4096, False), (2049, 4096, True), (65535, 1, True), (1, 4097, True)])
def test_the_workspace_of_small_vocabularies(L, sequences, vocab, some):
    assert (cp.verify_workspace_bytes(sequences, 65535, vocab) > 0) == some


def test_rows_of_a_projection(L):
    d = cp.LinearDesc(100, 256, 64, 0, P, P)
    for rows, want in ((65535, OK), (65536, UNSUPPORTED)):
        a = cp.LinearArgs(P, 0, rows, 0, 2 * P, 0)
        assert L.cp_linear_check(C.byref(d), C.byref(a)) == want
