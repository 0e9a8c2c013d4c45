"""Gates far below zero, whose exponentials leave fp32's range before the results do."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from persistent_megakernel_streaming_gb300 import cp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 5, 12, 40, 200])
@pytest.mark.parametrize("up", [0, 40, -20])
def test_gates_of_every_size(rows, up):
    """Each sum is one product, exactly: gates of 2^-10 to 240 below zero and above. The gate's function and the two products 16
    half steps, and its own rounding where it is below the normal numbers, times up."""
    size = np.concatenate([np.exp2(np.arange(-10, 8)), np.linspace(1, 255, 255), np.linspace(80.25, 107.75, 111)])
    size = torch.tensor(size).to(torch.bfloat16)            # all are bf16 numbers but those from 128 on
    half = len(size)
    q = np.full((2 * half, 16), 0x88, np.uint8)
    q[:half, 0], q[half:, 0] = 0x89, 0x98                   # 1 at the first input of gates, at the second of up
    scale = torch.cat([size, torch.full((half,), 2.0 ** up, dtype=torch.bfloat16)])[:, None]
    lin = cp.Linear(torch.from_numpy(q).cuda(), scale.cuda(), gated=True)
    x = torch.zeros(rows, 32, dtype=torch.bfloat16)
    x[:, 0] = torch.where(torch.arange(rows) % 4 == 3, 1.0, -1.0)
    x[:, 1] = torch.where(torch.arange(rows) % 2 == 0, 1.0, -1.0)
    out = torch.zeros(rows, half, device="cuda")
    lin.apply(x.cuda(), out)
    g = x[:, :1].double().numpy() * size.double().numpy()[None]
    u = x[:, 1:2].double().numpy() * 2.0 ** up
    with np.errstate(over="ignore"):
        y = g / (1 + np.exp(-g)) * u
    got = out.cpu().double().numpy()
    off = 16 * 2.0 ** -24 * np.abs(y) + 2.0 ** -149 * (np.abs(u) + 1)
    worst = np.abs(got - y) / off
    assert worst.max() <= 1, (g.flat[worst.argmax()], got.flat[worst.argmax()], y.flat[worst.argmax()])


def test_gates_at_the_ends():
    """Infinite gates: below, what the formula gives in fp32, NaN; above, the gate itself."""
    for rows in (2, 40):
        q = np.full((2, 16), 0x99, np.uint8)
        lin = cp.Linear(torch.from_numpy(q).cuda(), torch.ones(2, 1, dtype=torch.bfloat16, device="cuda"), gated=True)
        x = torch.zeros(rows, 32, dtype=torch.bfloat16, device="cuda")
        x[0, 0], x[1, 0] = float("inf"), -float("inf")
        out = torch.zeros(rows, 1, device="cuda")
        lin.apply(x, out)
        assert out[0, 0] == float("inf") and out[1, 0].isnan() and (out[2:] == 0).all()
