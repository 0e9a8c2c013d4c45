"""Numbers that the C side's types would change are refused."""
import pytest

torch = pytest.importorskip("torch")
from persistent_megakernel_streaming_gb300 import cp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("timeout", [2 ** 63, 2 ** 64, 2 ** 64 + 5, -2 ** 63 - 1])
def test_timeouts_past_64_bits(timeout):
    q, scale = torch.zeros(4, 16, dtype=torch.uint8, device="cuda"), torch.ones(4, 1, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        cp.Linear(q, scale, timeout_ns=timeout)
    kv = [torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    with pytest.raises(ValueError):
        cp.Cache(*kv, timeout_ns=timeout)
    cp.Linear(q, scale, timeout_ns=2 ** 63 - 1)
    cp.Cache(*kv, timeout_ns=2 ** 63 - 1)
