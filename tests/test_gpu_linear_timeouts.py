"""The time after which a projection's wait gives up is its own, not the kernel's in front of it."""
import pytest

torch = pytest.importorskip("torch")
from persistent_megakernel_streaming_gb300 import cp

pytestmark = pytest.mark.gpu


def test_a_long_kernel_in_front():
    """Eight rows of 2^20 inputs to 40 features keep a few SMs for longer than the next projection, which starts beside it and
    reads what it writes, would wait for its own loads."""
    q = torch.zeros(40, 1 << 19, dtype=torch.uint8, device="cuda")
    q[:, 0] = 9                                             # 1 at the first input, -8 at the others
    long = cp.Linear(q, torch.ones(40, 1 << 13, dtype=torch.bfloat16, device="cuda"))
    x = torch.zeros(8, 1 << 20, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 3.0
    y = torch.zeros(40, 32, dtype=torch.bfloat16, device="cuda")
    w = torch.full((48, 16), 0x88, dtype=torch.uint8, device="cuda")
    w[:, 0] = 0x89
    short = cp.Linear(w, torch.ones(48, 1, dtype=torch.bfloat16, device="cuda"), timeout_ns=100_000)
    out = torch.zeros(40, 48, device="cuda")
    first = torch.zeros(8, 40, dtype=torch.bfloat16, device="cuda")
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    long.apply(x, first)
    a.record()
    long.apply(x, first)
    b.record()
    b.synchronize()
    assert a.elapsed_time(b) > 0.3                          # milliseconds: longer than three times the wait
    y[:, 0] = 5.0
    for _ in range(5):
        long.apply(x, first)
        short.apply(y, out)
        assert short.status() == 0 and (out == 5).all() and (first == 3).all()
        out.zero_()
