"""Calls as a thread's first use of CUDA: what a server's worker threads make."""
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from persistent_megakernel_streaming_gb300 import cp

pytestmark = pytest.mark.gpu


def in_thread(f):
    out = []

    def go():
        try:
            out.append((f(), None))
        except BaseException as e:
            out.append((None, e))

    t = threading.Thread(target=go)
    t.start()
    t.join()
    torch.cuda.synchronize()
    result, error = out[0]
    if error:
        raise error
    return result


def weights(n=272, k=256):
    g = torch.Generator(device="cuda").manual_seed(0)
    return (torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8),
            torch.rand((n, k // 64), generator=g, device="cuda").to(torch.bfloat16))


@pytest.mark.parametrize("rows", [1, 12, 40, 200])
def test_projections(rows):
    q, scale = weights()
    lin = cp.Linear(q, scale)
    x = torch.randn(rows, 256, device="cuda").to(torch.bfloat16)
    out, want = (torch.zeros(rows, 272, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    in_thread(lambda: lin.apply(x, out))
    lin.apply(x, want)
    assert torch.equal(out, want) and (want != 0).any()


def test_weights_laid_out():
    q, scale = weights()
    torch.cuda.synchronize()
    lin = in_thread(lambda: cp.Linear(q, scale))
    a, b = (torch.zeros(272, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lin.unpack(a)
    cp.Linear(q, scale).unpack(b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("vocab", [100, 9000])
def test_verifications(vocab):
    x = torch.zeros(3, vocab, device="cuda")
    x[:, 5] = 90
    z, f = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.full((3,), 0.5, device="cuda")
    start, accepted, token = torch.arange(4, dtype=torch.int32, device="cuda"), z.clone(), z.clone()
    workspace = torch.zeros(max(16, cp.verify_workspace_bytes(3, 3, vocab)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    in_thread(lambda: cp.verify(x, z, start, f, f, f, accepted, token, workspace=workspace))
    assert token.tolist() == [5] * 3


def test_pages_and_copies():
    refs, table, length = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in ((9,), (2, 4), (2,)))
    add, moves, count = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in ((2,), (9, 2), (1,)))
    kv = [torch.randn(9, 2, 16, 64, device="cuda").to(torch.bfloat16) for _ in range(2)]
    add[:] = 20
    torch.cuda.synchronize()
    pool = in_thread(lambda: cp.Pages(refs, table, length, 16))
    in_thread(lambda: pool.grow(add, moves, count))
    assert table.tolist() == [[0, 1, 0, 0], [2, 3, 0, 0]]
    in_thread(lambda: pool.trim(torch.zeros_like(add)))
    in_thread(lambda: pool.compact(moves, count))
    cache = in_thread(lambda: cp.Cache(*kv))
    moves[0, 1], count[0] = 7, 1
    torch.cuda.synchronize()
    in_thread(lambda: cache.copy(moves, count))
    assert torch.equal(kv[0][0], kv[0][7]) and pool.status() == 0 and cache.status() == 0


def test_attention():
    """A cache made, written and attended to, each by a thread of its own."""
    kv = [torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    rows, heads = 40, 4
    batch = cp.Batch(i32([0, rows]), i32([rows]), i32([[0, 1, 2, 3]]), rows)
    qkv = torch.randn(rows, (heads + 4) * 64, device="cuda").to(torch.bfloat16)
    q, out, want = (torch.zeros(rows, heads, 64, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    torch.cuda.synchronize()
    cache = in_thread(lambda: cp.Cache(*kv))
    in_thread(lambda: cache.append(batch, qkv, q))
    need = cache.workspace_bytes(batch, heads)
    workspace = torch.zeros(max(16, need), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    in_thread(lambda: cache.attend(batch, q, out, workspace=workspace))
    cache.attend(batch, q, want, workspace=workspace)
    assert torch.equal(out, want) and (want != 0).any() and cache.status() == 0
