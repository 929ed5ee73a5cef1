"""GPU: MXFP4 quantization and back, and products, against plain 64-bit forms."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import expert_helpers as H
import mxfp4_helpers as M
import nvfp4_block_scaled_05_amd as nv
from fp8_helpers import plan_of
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


def rand(shape, dtype, seed, spread=2.0):
    g = torch.Generator(DEV).manual_seed(seed)
    x = torch.randn(shape, device=DEV, generator=g) * torch.exp(spread * torch.randn(shape[-1], device=DEV, generator=g))
    return x.to(dtype)


def check_orientation(q, x, block_2d, what):
    """q against the definition for the rows of x (binary64), bit for bit; the padding is zero."""
    r, c = x.shape
    want, scales = M.quantize(x, block_2d)
    assert (q.n, q.k) == (r, c)
    assert np.array_equal(q.scales.cpu().numpy(), scales), what + " scales"
    got = M.codes(q.data)
    assert got.shape == want.shape and np.array_equal(got, want) and np.array_equal(np.signbit(got[:, :c]), np.signbit(want[:, :c])), what + " data"
    assert not np.any(q.data.cpu().numpy()[:, (c + 1) // 2:])


def same(a, b):
    return (a.n, a.k) == (b.n, b.k) and torch.equal(a.data, b.data) and torch.equal(a.scales, b.scales)


SHAPES = [(1, 1), (1, 128), (16, 5120), (127, 129), (128, 128), (129, 127), (200, 333), (1000, 264), (3, 2047), (515, 8), (33, 31)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_2d", [False, True])
def test_quantize(rows, cols, dtype, block_2d):
    x = rand((rows, cols), dtype, rows * 7 + cols)
    x[rows // 2] = 0
    row, col = nv.mxfp4_quantize(x, rowwise=True, columnwise=True, block_2d=block_2d)
    check_orientation(row, H.f64(x), block_2d, "row")
    check_orientation(col, H.f64(x).T, block_2d, "col")
    only, none = nv.mxfp4_quantize(x, block_2d=block_2d)
    assert none is None and same(only, row)
    none, only = nv.mxfp4_quantize(x, rowwise=False, columnwise=True, block_2d=block_2d)
    assert none is None and same(only, col)
    for q in (row, col):
        want = M.values(q)[:, :q.k]
        for out in (torch.bfloat16, torch.float32):
            assert torch.equal(nv.mxfp4_dequantize(q, out_dtype=out).double(), want)
    if block_2d:
        assert torch.equal(nv.mxfp4_dequantize(row), nv.mxfp4_dequantize(col).t())


@pytest.mark.parametrize("shape", [(3, 100, 200), (16, 8, 352), (2, 256, 128), (5, 1, 1), (0, 4, 4), (2, 0, 7), (2, 7, 0)])
@pytest.mark.parametrize("block_2d", [False, True])
def test_quantize_batch(shape, block_2d):
    x = rand(shape, torch.bfloat16, 3)
    row, col = nv.mxfp4_quantize(x, columnwise=True, block_2d=block_2d)
    back = [nv.mxfp4_dequantize(q) for q in (row, col)]
    assert back[0].shape == shape and back[1].shape == (shape[0], shape[2], shape[1])
    for b in range(shape[0] if x.numel() else 0):
        for q, y, v, what in ((row, back[0], H.f64(x[b]), "row"), (col, back[1], H.f64(x[b]).T, "col")):
            one = nv.Mxfp4Tensor(q.data[b], q.scales[b], q.n, q.k)
            check_orientation(one, v, block_2d, f"{what} {b}")
            assert torch.equal(y[b], nv.mxfp4_dequantize(one))


def test_quantize_every_bf16_value_and_the_steps_around_every_code():
    # all finite BF16 values, each row of one binade so that small ones are not all zero
    bits = np.arange(0x7F80, dtype=np.uint16).reshape(255, 128)
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).to(DEV)
    row, col = nv.mxfp4_quantize(torch.cat([x, -x]), columnwise=True)
    check_orientation(row, H.f64(torch.cat([x, -x])), False, "row")
    check_orientation(col, H.f64(torch.cat([x, -x])).T, False, "col")
    # binary32 values next to the middles between neighbouring codes, in blocks whose scale is 1, and in others
    mids = ((M.E2M1[1:] + M.E2M1[:-1]) / 2).astype(np.float32)
    v = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(9)), np.float32([6.5, 7, 7.9999995, 0, 4])])
    v = np.concatenate([v, -v])
    v = np.concatenate([v, np.zeros(-v.size % 31, np.float32)]).reshape(-1, 31)
    v = np.concatenate([v, np.full((v.shape[0], 1), 4, np.float32)], 1)
    v = np.concatenate([v * np.float32(2.0 ** p) for p in (0, 1, -1, 60, -60, 120, -120)])
    row, _ = nv.mxfp4_quantize(torch.from_numpy(v).to(DEV))
    check_orientation(row, v.astype(np.float64), False, "row")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_extremes(dtype):
    tiny, most = float(np.finfo(np.float32).tiny), 3.3895313892515355e38  # the largest BF16 number
    rows = [[0.0] * 32, [most] + [1.0] * 31, [-most] * 32, [tiny] * 32, [tiny * 4] * 32, [tiny * 8] * 32, [tiny / 2] * 32, [tiny / 128] * 32,
            [tiny / 64] + [0.0] * 31, [-0.0] * 31 + [1.0], [1e30, -1e30] + [1e-30] * 30, [2.0 ** -125] * 31 + [2.0 ** -127]]
    if dtype == torch.float32:
        rows += [[1.4e-45] * 32, [1e-40] * 32]
    x = torch.tensor(rows, dtype=torch.float32, device=DEV).to(dtype)
    row, col = nv.mxfp4_quantize(x, columnwise=True)
    check_orientation(row, H.f64(x), False, "row")
    check_orientation(col, H.f64(x).T, False, "col")
    for q in (row, col):
        want = M.values(q)[:, :q.k]
        for out in (torch.bfloat16, torch.float32):
            assert torch.equal(nv.mxfp4_dequantize(q, out_dtype=out).double(), want)


def test_dequantize_every_scale():
    # every code under every scale; past the type's largest number an infinity
    data = torch.arange(16, dtype=torch.uint8, device=DEV).repeat(4)
    data = (data | data.flip(0) << 4).repeat(64, 1)  # [64][64]: 128 values a row
    scales = torch.arange(256, dtype=torch.int32, device=DEV).to(torch.uint8).reshape(1, 64, 4)
    q = nv.Mxfp4Tensor(data, scales, 64, 128)
    want = M.values(q)
    for out in (torch.bfloat16, torch.float32):
        got = nv.mxfp4_dequantize(q, out_dtype=out)
        expected = want.float().to(out)
        assert torch.equal(torch.isnan(got), torch.isnan(expected)) and torch.equal(got.nan_to_num(1.0), expected.nan_to_num(1.0))
        assert bool(torch.isnan(got[63, 96:]).all()) and not bool(torch.isnan(got[:63]).any())


@pytest.mark.parametrize("block_2d", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_non_finite_blocks_decode_to_nan(block_2d, dtype):
    x = torch.ones((256, 256), device=DEV, dtype=dtype)
    x[3, 5], x[200, 130], x[70, 255] = float("nan"), float("inf"), float("-inf")
    row, col = nv.mxfp4_quantize(x, columnwise=True, block_2d=block_2d)
    check_orientation(row, H.f64(x), block_2d, "row")
    check_orientation(col, H.f64(x).T, block_2d, "col")
    want = torch.zeros((256, 256), dtype=torch.bool, device=DEV)
    for i, j in ((3, 5), (200, 130), (70, 255)):
        want[i // 32 * 32 if block_2d else i:i // 32 * 32 + 32 if block_2d else i + 1, j // 32 * 32:j // 32 * 32 + 32] = True
    assert torch.equal(torch.isnan(nv.mxfp4_dequantize(row)), want)


@pytest.mark.parametrize("tokens,topk,experts,cols,align", [(1, 1, 3, 128, 128), (40, 3, 5, 200, 16), (300, 4, 8, 517, 128)])
def test_quantize_by_plan_is_gather_then_quantize(tokens, topk, experts, cols, align):
    g = torch.Generator(DEV).manual_seed(tokens)
    ids = torch.randint(-1, experts, (tokens, topk), dtype=torch.int32, device=DEV, generator=g)
    plan = nv.expert_sort(ids, experts, align=align)
    for dtype in (torch.bfloat16, torch.float32):
        x = rand((tokens, cols), dtype, cols)
        for block_2d in (False, True):
            got = nv.mxfp4_quantize(x, columnwise=True, block_2d=block_2d, plan=plan)
            want = nv.mxfp4_quantize(nv.expert_gather(x, plan), columnwise=True, block_2d=block_2d)
            assert all(same(a, b) for a, b in zip(got, want))


# ---- products ----------------------------------------------------------------

PRODUCTS = [(1, 1, 1), (1, 8192, 128), (3, 17, 129), (16, 64, 640), (17, 33, 5120), (32, 2048, 2048), (32, 31, 100), (33, 100, 300),
            (64, 64, 128), (100, 200, 257), (128, 128, 4096), (257, 129, 1999), (300, 1000, 385), (777, 1361, 640), (1024, 2048, 896),
            (2048, 4096, 256), (2300, 4100, 384), (4096, 4096, 640), (5, 7, 0), (600, 600, 0), (4000, 4352, 128)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_product(m, n, k, out):
    a, b = M.operand(m, k, m + k, exponents=(-3, 3)), M.operand(n, k, n + 2 * k + 1, exponents=(-3, 3))
    M.check_product(nv.mxfp4_matmul(a, b, out_dtype=out), M.values(a), M.values(b))


@pytest.mark.parametrize("m,n,k", [(16, 64, 1024), (100, 200, 640), (1024, 2048, 896), (4096, 4096, 512)])
@pytest.mark.parametrize("exponents", [(-40, 40), (-125, -70), (-20, 0)])
def test_product_of_scales_far_apart(m, n, k, exponents):
    a, b = M.operand(m, k, 1, exponents=exponents), M.operand(n, k, 2, exponents=(-10, 10) if exponents[0] > -100 else (-60, 0))
    M.check_product(nv.mxfp4_matmul(a, b, out_dtype=torch.float32), M.values(a), M.values(b))


@pytest.mark.parametrize("m,n,k", [(16, 64, 1024), (100, 200, 640), (1024, 2048, 256), (4096, 4096, 128)])
def test_product_of_equal_scales_is_exact(m, n, k):
    # sums of multiples of 1/4 below 2^22: binary32 holds each on the way
    a, b = M.operand(m, k, 3), M.operand(n, k, 4)
    a.scales.fill_(130), b.scales.fill_(121)
    got = nv.mxfp4_matmul(a, b, out_dtype=torch.float32)
    assert torch.equal(got.double(), M.values(a) @ M.values(b).t())


@pytest.mark.parametrize("m,n,k", [(16, 64, 1024), (100, 200, 640), (1024, 2048, 256), (4096, 4096, 128)])
def test_product_with_nan_blocks(m, n, k):
    a, b = M.operand(m, k, 5), M.operand(n, k, 6)
    a.scales[0, m // 2, 1] = 255
    b.scales[-1, n // 3, 0] = 255
    d = nv.mxfp4_matmul(a, b, out_dtype=torch.float32)
    want = torch.zeros((m, n), dtype=torch.bool, device=DEV)
    want[m // 2] = want[:, n // 3] = True
    assert torch.equal(torch.isnan(d), want)


def test_zero_blocks_under_any_scale_do_not_count():
    a, b = M.operand(200, 512, 7), M.operand(300, 512, 8)
    a.data[:, 64:96] = 0
    a.data[5, :] = 0x88  # zeros of the other sign
    a.scales[1, :, :2] = torch.randint(0, 255, (200, 2), device=DEV).to(torch.uint8)
    b.scales[1, :, :2] = torch.randint(100, 255, (300, 2), device=DEV).to(torch.uint8)
    va, vb = M.values(a), M.values(b)
    va[:, 128:192] = 0
    vb[:, 128:192] = 0
    M.check_product(nv.mxfp4_matmul(a, b, out_dtype=torch.float32), va, vb)


GROUPS = [([5], 1, 64, 256), ([0, 3, 0, 40, 1], 16, 100, 300), ([30, 0, 64, 65, 17], 16, 520, 1152), ([1] * 64, 16, 96, 640),
          ([200, 0, 129, 128, 300], 128, 384, 640), ([700, 900, 0, 500], 128, 1024, 384), ([2000, 100, 3000, 1], 128, 2048, 256), ([0, 0], 16, 64, 128)]


@pytest.mark.parametrize("counts,align,n,k", GROUPS)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_grouped(counts, align, n, k, out):
    plan = plan_of(counts, align)
    a, b = M.operand(plan.rows, k, 9, exponents=(-2, 2)), M.operand(n, k, 10, lead=(len(counts),), exponents=(-2, 2))
    d = nv.mxfp4_matmul_grouped(a, b, plan, out_dtype=out)
    va, off = M.values(a), plan.offsets.tolist()
    for e in range(len(counts)):
        if off[e] < off[e + 1]:
            M.check_product(d[off[e]:off[e + 1]], va[off[e]:off[e + 1]], M.values(b, e), f"group {e}")
    assert not bool(d[off[-1]:].any())


def test_rows_past_the_last_group_are_zero_whatever_they_held():
    ids = torch.randint(0, 4, (50, 1), dtype=torch.int32, device=DEV)
    plan = nv.expert_sort(ids, 4, align=16, rows=1000)
    a, b = M.operand(1000, 256, 11), M.operand(200, 256, 12, lead=(4,))
    a.scales[:, plan.offsets.tolist()[-1]:] = 255
    for rows in (1000,):
        assert not bool(nv.mxfp4_matmul_grouped(a, b, plan)[plan.offsets.tolist()[-1]:].any())


@pytest.mark.parametrize("counts", [[5], [0, 3, 0, 400, 1], [200, 0, 129, 128, 300], [700, 900, 0, 500], [0, 0]])
@pytest.mark.parametrize("m,n", [(64, 96), (257, 300), (1024, 2048)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_grouped_k(counts, m, n, out):
    plan = plan_of(counts, 128)
    a, b = M.operand(m, plan.rows, 13, exponents=(-2, 2)), M.operand(n, plan.rows, 14, exponents=(-2, 2))
    d = nv.mxfp4_matmul_grouped_k(a, b, plan, out_dtype=out)
    va, vb, off = M.values(a), M.values(b), plan.offsets.tolist()
    for e in range(len(counts)):
        M.check_product(d[e], va[:, off[e]:off[e + 1]], vb[:, off[e]:off[e + 1]], f"group {e}")


def test_the_same_bits_every_time():
    a, b = M.operand(777, 1999, 15, exponents=(-9, 9)), M.operand(1361, 1999, 16, exponents=(-9, 9))
    first = nv.mxfp4_matmul(a, b, out_dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(nv.mxfp4_matmul(a, b, out_dtype=torch.float32), first)


def test_captured_and_replayed():
    g = torch.Generator(DEV).manual_seed(17)
    x, w = torch.randn((300, 520), device=DEV, generator=g), torch.randn((640, 520), device=DEV, generator=g)

    def run():
        q, c = nv.mxfp4_quantize(x, columnwise=True)
        d = nv.mxfp4_matmul(q, nv.mxfp4_quantize(w)[0], out_dtype=torch.float32)
        return d, nv.mxfp4_dequantize(c)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for i in range(4):
        x.copy_(torch.randn(x.shape, device=DEV, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), i


@pytest.mark.parametrize("name", ["quantize", "dequantize", "matmul", "grouped", "grouped_k"])
def test_on_another_stream(name):
    plan = plan_of([100, 28], 128)
    x = rand((plan.rows, 256), torch.float32, 18)
    a, at = nv.mxfp4_quantize(x, columnwise=True)
    b = M.operand(64, 256, 19, lead=(2,))
    one = nv.Mxfp4Tensor(b.data[0], b.scales[0], 64, 256)
    call = {"quantize": lambda s: nv.mxfp4_quantize(x, stream=s)[0].data, "dequantize": lambda s: nv.mxfp4_dequantize(a, stream=s),
            "matmul": lambda s: nv.mxfp4_matmul(a, one, stream=s), "grouped": lambda s: nv.mxfp4_matmul_grouped(a, b, plan, stream=s),
            "grouped_k": lambda s: nv.mxfp4_matmul_grouped_k(at, at, plan, stream=s)}[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream, 0):
        got = call(s)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
