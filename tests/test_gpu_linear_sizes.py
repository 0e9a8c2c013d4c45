"""Projections of as many rows as a call takes, and rows that lie further apart than 32 bits count: whole numbers, exactly."""
import pytest

torch = pytest.importorskip("torch")
from persistent_megakernel_streaming_gb300 import cp

pytestmark = pytest.mark.gpu


def whole(n, k, rows, gated=False, zero=False):
    g = torch.Generator(device="cuda").manual_seed(rows)
    q = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.exp2(torch.randint(-2, 2, (n, k // 64), generator=g, device="cuda").float()).to(torch.bfloat16)
    z = torch.randint(0, 16, (n, k // 64), generator=g, device="cuda", dtype=torch.uint8) if zero else None
    lin = cp.Linear(q, scale, z, gated=gated)
    w = torch.empty(n, k, dtype=torch.bfloat16, device="cuda")
    lin.unpack(w)
    x = torch.randint(-8, 9, (rows, k), generator=g, device="cuda").to(torch.bfloat16)
    return lin, x, x.double() @ w.double().T


@pytest.mark.parametrize("rows,n,k", [(1025, 272, 320), (4096, 500, 1024), (8191, 272, 192), (65535, 130, 64)])
@pytest.mark.parametrize("zero", [False, True])
def test_many_rows(rows, n, k, zero):
    lin, x, want = whole(n, k, rows, zero=zero)
    out = torch.full((rows, n), 7.0, device="cuda")
    lin.apply(x, out)
    assert torch.equal(out.double(), want)
    lin.apply(x, out, add=out)
    assert torch.equal(out.double(), 2 * want)


@pytest.mark.parametrize("rows", [8, 14, 40])
def test_rows_far_apart(rows):
    lin, x, want = whole(272, 192, rows)
    row = (1 << 32) // (rows - 1) // 8 * 8 + 8                      # elements: the last row starts past 2^32 of them
    pool = torch.zeros(row * (rows - 1) + 272, dtype=torch.bfloat16, device="cuda")
    far = pool.as_strided((rows, 192), (row, 1))
    far.copy_(x)
    out = torch.zeros(rows, 272, device="cuda")
    lin.apply(far, out)
    assert torch.equal(out.double(), want)
    far = pool.as_strided((rows, 272), (row, 1))
    lin.apply(x, far)
    assert torch.equal(far, want.to(torch.bfloat16))
    lin.apply(x, far, add=far)
    assert torch.equal(far, (want + want.to(torch.bfloat16).double()).to(torch.bfloat16))
