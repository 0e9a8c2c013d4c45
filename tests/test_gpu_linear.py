"""Projections with 4-bit weights against float64: sizes, groups, zero points, gates, residuals, types and strides."""
import ctypes as C

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from oracle import linear as ref
from persistent_megakernel_streaming_gb300 import cp

pytestmark = pytest.mark.gpu
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def make(n, k, group, zero, seed, x_rows=1, spread=1.0):
    g = np.random.default_rng(seed)
    q = g.integers(0, 256, (n, k // 2)).astype(np.uint8)
    scale = torch.from_numpy((np.exp(spread * g.standard_normal((n, k // group))) * 0.05).astype(np.float32)).to(torch.bfloat16)
    z = g.integers(0, 16, (n, k // group)).astype(np.uint8) if zero else None
    x = torch.from_numpy(g.standard_normal((x_rows, k)).astype(np.float32)).to(torch.bfloat16)
    return q, scale, z, x


def linear(q, scale, z, gated=False):
    return cp.Linear(torch.from_numpy(q).cuda(), scale.cuda(), None if z is None else torch.from_numpy(z).cuda(), gated=gated)


def wide(t):
    return t.float().double().cpu().numpy()


def check(got, y, off, dtype):
    """Within the sums' bound and the result's own rounding."""
    most = off + HALF_STEP[dtype] * (np.abs(y) + off) + 1e-38
    worst = (np.abs(wide(got) - y) / most).max()
    assert worst <= 1, worst


def compare(rows, n, k, group, zero, gated, add, dtype, seed=0):
    q, scale, z, x = make(n, k, group, zero, seed, rows)
    outs = n // 2 if gated else n
    res = torch.from_numpy(np.random.default_rng(seed + 1).standard_normal((rows, outs)).astype(np.float32)).to(dtype) if add else None
    out = torch.full((rows, outs), 7.0, dtype=dtype, device="cuda")
    lin = linear(q, scale, z, gated)
    lin.apply(x.cuda(), out, add=None if res is None else res.cuda())
    y, off = ref.apply(wide(x), ref.weights(q, wide(scale), z), gated, None if res is None else wide(res))
    check(out, y, off, dtype)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_kinds(group, zero, gated):
    compare(5, 96, 384, group, zero, gated, True, torch.bfloat16)
    compare(3, 96, 384, group, zero, gated, False, torch.float32, seed=4)


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 15, 16, 17, 24, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 160, 161, 255, 256, 257, 320,
                                  321, 400, 700])
def test_rows(rows):
    compare(rows, 272, 448, 64, True, False, True, torch.float32, seed=rows)
    compare(rows, 320, 640, 128, False, True, False, torch.bfloat16, seed=rows)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 255, 2049])
@pytest.mark.parametrize("rows", [1, 20, 130])
def test_features(n, rows):
    compare(rows, n, 256, 32, False, False, True, torch.float32, seed=n)
    compare(rows, 2 * n, 256, 128, True, True, True, torch.bfloat16, seed=n)


@pytest.mark.parametrize("k,group", [(32, 32), (64, 32), (64, 64), (96, 32), (128, 128), (160, 32), (192, 64), (544, 32), (1024, 128),
                                     (2048, 64), (5120, 128), (8224, 32), (16384, 128)])
@pytest.mark.parametrize("rows", [1, 12, 40])
def test_widths(k, group, rows):
    compare(rows, 80, k, group, True, False, False, torch.float32, seed=k)


@pytest.mark.parametrize("n,k", [(2400, 384), (4870, 384), (9700, 640), (9800, 1000 - 40), (14500, 1152), (14500, 640), (14700, 640),
                                 (19450, 384), (19500, 384), (30000, 256)])
@pytest.mark.parametrize("group,zero,gated", [(128, False, False), (32, True, True), (64, True, False), (64, False, True)])
def test_numbers_of_blocks(n, k, group, zero, gated):
    """Few rows, over as many features as make each number of warps, tiles and records a block."""
    k = k // group * group
    compare(5, n, k, group, zero, gated, True, torch.bfloat16, seed=n)
    compare(8, n, k, group, zero, gated, False, torch.float32, seed=n + 1)


@pytest.mark.parametrize("rows,n,k", [(17, 20000, 256), (40, 33000, 128), (64, 66000, 128), (30, 130, 4096), (100, 12000, 256),
                                      (190, 20000, 128), (192, 300, 2048), (350, 9000, 384), (64, 8200, 512), (200, 2049, 1024)])
@pytest.mark.parametrize("gated", [False, True])
def test_plans(rows, n, k, gated):
    """Many rows, over what makes one, two and four pieces a block, clusters of one to four, and each number of rows a block."""
    compare(rows, n // 2 * 2, k, 128, False, gated, True, torch.bfloat16, seed=n)
    compare(rows, n // 2 * 2, k, 32, True, gated, False, torch.float32, seed=n + 1)


def test_larger_layers():
    compare(1, 4096, 2048, 128, False, False, False, torch.bfloat16)
    compare(64, 4098, 2048, 64, True, True, True, torch.bfloat16)
    compare(33, 1000, 6144, 32, True, False, True, torch.float32)


def test_the_plain_sum_exactly():
    """Whole numbers whose sums fp32 holds: no error at all, for every weight's place."""
    g = np.random.default_rng(5)
    for rows in (1, 9, 30, 150):
        q = g.integers(0, 256, (200, 160)).astype(np.uint8)
        scale = torch.from_numpy(np.exp2(g.integers(-2, 3, (200, 5))).astype(np.float32)).to(torch.bfloat16)
        x = torch.from_numpy(g.integers(-8, 9, (rows, 320)).astype(np.float32)).to(torch.bfloat16)
        out = torch.empty((rows, 200), dtype=torch.float32, device="cuda")
        linear(q, scale, None).apply(x.cuda(), out)
        np.testing.assert_array_equal(wide(out), wide(x) @ ref.weights(q, wide(scale)).T)


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_unpack(zero, gated):
    for n, k, group in ((2, 32, 32), (250, 448, 64), (130, 128, 128)):
        q, scale, z, _ = make(n, k, group, zero, n, spread=4.0)
        scale[-1] = -scale[-1]
        scale[0] = 2.0 ** -126 * 1.5                  # the least exponent of a normal number
        out = torch.zeros((n, k), dtype=torch.bfloat16, device="cuda")
        linear(q, scale, z, gated).unpack(out)
        np.testing.assert_array_equal(wide(out), ref.weights(q, wide(scale), z))


def test_strides_and_in_place_residual():
    for rows in (3, 40):
        q, scale, z, x = make(100, 256, 64, True, 1, rows)
        y, off = ref.apply(wide(x), ref.weights(q, wide(scale), z), False)
        pool = torch.zeros((rows, 3, 256), dtype=torch.bfloat16, device="cuda")
        pool[:, 1] = x.cuda()
        out = torch.full((rows, 133), -5.0, dtype=torch.bfloat16, device="cuda")
        lin = linear(q, scale, z)
        lin.apply(pool[:, 1], out[:, 7:107])
        check(out[:, 7:107], y, off, torch.bfloat16)
        assert (out[:, :7] == -5).all() and (out[:, 107:] == -5).all()
        res = torch.from_numpy(np.random.default_rng(2).standard_normal((rows, 101)).astype(np.float32)).cuda()
        before = wide(res)
        lin.apply(x.cuda(), res[:, 1:], add=res[:, 1:])
        check(res[:, 1:], *ref.apply(wide(x), ref.weights(q, wide(scale), z), False, before[:, 1:]), torch.float32)
        assert (wide(res)[:, 0] == before[:, 0]).all()


def test_rows_do_not_touch_one_another():
    """NaN and infinities stay in their rows, and what lies behind the last row in memory is not looked at."""
    for rows in (5, 16, 50, 200):
        q, scale, z, x = make(96, 320, 64, False, 3, rows)
        lin = linear(q, scale, z)
        clean = torch.empty((rows, 96), dtype=torch.float32, device="cuda")
        lin.apply(x.cuda(), clean)
        bad = torch.full((rows + 9, 320), float("nan"), dtype=torch.bfloat16, device="cuda")
        bad[:rows] = x.cuda()
        bad[2] = float("nan")
        bad[4, 7] = float("inf")
        out = torch.zeros((rows + 9, 96), dtype=torch.float32, device="cuda")
        lin.apply(bad[:rows], out[:rows])
        keep = torch.tensor([r for r in range(rows) if r not in (2, 4)], device="cuda")
        assert torch.equal(out[keep], clean[keep])
        assert out[2].isnan().all() and not out[4].isfinite().any() and (out[rows:] == 0).all()


def test_extreme_scales():
    """Results from 2^-100 to 2^100; scales of zero, infinity, NaN, the largest taken and the least refused."""
    for rows in (2, 70):
        q, _, _, x = make(64, 128, 128, False, 9, rows)
        s = np.zeros((64, 1), np.float32)
        s[:, 0] = np.exp2(np.linspace(-100, 100, 64).round())
        s[5] = 0
        scale = torch.from_numpy(s).to(torch.bfloat16)
        out = torch.empty((rows, 64), dtype=torch.float32, device="cuda")
        lin = linear(q, scale, None)
        lin.apply(x.cuda(), out)
        y, off = ref.apply(wide(x), ref.weights(q, wide(scale)), False)
        check(out, y, off, torch.float32)
        assert (out[:, 5] == 0).all()
    # an infinite weight and no other: the result is infinite, whatever the block's share of the inputs
    one = np.full((512, 64), 0x88, np.uint8)
    one[3, 5] = 0x98
    big = np.full((512, 1), 1.0, np.float32)
    big[3] = np.inf
    zeros = torch.full((512, 1), 8, dtype=torch.uint8)
    for n in (64, 512):
        y = torch.empty((2, n), dtype=torch.float32, device="cuda")
        lin = cp.Linear(torch.from_numpy(one[:n]).cuda(), torch.from_numpy(big[:n]).to(torch.bfloat16).cuda(), zeros[:n].cuda())
        lin.apply(torch.ones((2, 128), dtype=torch.bfloat16, device="cuda"), y)
        assert y[:, 3].isnan().all() and (y[:, :3] == 0).all() and (y[:, 4:] == 0).all()      # 0 times infinity is in there
    s[7], s[9] = np.inf, np.nan
    s[11] = -2.0 ** 121                            # the largest exponent that is taken
    lin = linear(q, torch.from_numpy(s).to(torch.bfloat16), None)
    lin.apply(x.cuda(), out)
    assert not out[:, [7, 9]].isfinite().any() and out[:, [8, 10]].isfinite().all()
    w = torch.zeros((64, 128), dtype=torch.bfloat16, device="cuda")
    lin.unpack(w)
    np.testing.assert_array_equal(wide(w)[11], (ref.nibbles(q)[11] - 8) * -2.0 ** 121)
    s[7] = 2.0 ** 122
    with pytest.raises(cp.CPError) as e:
        linear(q, torch.from_numpy(s).to(torch.bfloat16), None)
    assert e.value.code == 2


def test_streams_graphs_and_repeats():
    for rows in (2, 48):
        q, scale, z, x = make(512, 1024, 128, True, 11, rows)
        lin, xd = linear(q, scale, z), x.cuda()
        want, out = (torch.zeros((rows, 512), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        lin.apply(xd, want)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        lin.apply(xd, out, stream=side)
        side.synchronize()
        assert torch.equal(out, want)
        graph = torch.cuda.CUDAGraph()
        out.zero_()
        with torch.cuda.graph(graph):
            lin.apply(xd, out)
        xd.copy_(xd * 2)                          # a power of two: the results double exactly
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.float(), 2 * want.float())


def test_captured_behind_two_streams_and_a_copy():
    """A captured call behind a copy, and behind kernels of two streams that met."""
    for rows in (2, 60):
        q, scale, z, x = make(256, 512, 64, True, 13, rows)
        lin = linear(q, scale, z)
        a, b, out = (torch.zeros((rows, 512), dtype=torch.bfloat16, device="cuda") for _ in range(3))
        out = torch.zeros((rows, 256), dtype=torch.float32, device="cuda")
        want = torch.zeros_like(out)
        src = x.cuda()
        lin.apply(src, want)
        main, side = torch.cuda.Stream(), torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=main):
            a.copy_(src)
            lin.apply(a, out)
            out.zero_()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                b.copy_(src)
                b.add_(0)
            a.zero_()
            main.wait_stream(side)
            lin.apply(b, out)
            lin.apply(b, out, add=out)
        for _ in range(3):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want + want)


def test_a_wait_that_runs_out_is_reported():
    q, scale, z, x = make(256, 512, 64, False, 12, 40)
    lin = cp.Linear(torch.from_numpy(q).cuda(), scale.cuda(), timeout_ns=50_000_000, debug_stall=True)
    out = torch.zeros((40, 256), dtype=torch.float32, device="cuda")
    lin.apply(x.cuda(), out)
    assert lin.status() == cp.CP_ERR_TIMEOUT
    lin.clear_status()
    assert lin.status() == 0
    lin.apply(x.cuda()[:9], out[:9])               # few rows come through no ring
    assert lin.status() == 0
    check(out[:9], *ref.apply(wide(x[:9]), ref.weights(q, wide(scale)), False), torch.float32)


def test_refusals_on_the_gpu():
    q, scale, z, x = make(64, 128, 64, True, 0)
    lin = linear(q, scale, z)
    xd, out = x.cuda(), torch.zeros((1, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        lin.apply(xd[:, :64], out)
    with pytest.raises(ValueError):
        lin.apply(xd.float(), out)
    with pytest.raises(ValueError):
        lin.apply(xd, out.half())
    with pytest.raises(ValueError):
        lin.apply(xd, out[:, :63])
    with pytest.raises(ValueError):
        lin.apply(xd, out, add=out.float())
    with pytest.raises(ValueError):
        lin.apply(xd.cpu(), out)
    with pytest.raises(ValueError):
        lin.apply(torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda"), out.expand(2, 64))
    with pytest.raises(cp.CPError):
        lin.apply(torch.zeros((1, 129), dtype=torch.bfloat16, device="cuda")[:, 1:], out)      # x not on 16 bytes
    with pytest.raises(cp.CPError):
        z[3, 1] = 16
        linear(q, scale, z)
    with pytest.raises(ValueError):
        cp.Linear(torch.from_numpy(q), scale)
    h = C.c_void_p()
    assert cp.lib().cp_linear_create(C.byref(lin.desc), 99, C.byref(h)) == 2 and not h.value
    host = torch.zeros(64, 64, dtype=torch.uint8)
    d = cp.LinearDesc(64, 128, 64, 0, host.data_ptr(), scale.cuda().data_ptr(), None)
    assert cp.lib().cp_linear_create(C.byref(d), 0, C.byref(h)) == 1
