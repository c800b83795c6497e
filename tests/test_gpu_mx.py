"""MXFP4 quantisation, decoding and product on the GPU against plain numpy in 64
bits (mx_oracle.py).

Quantisation and decoding are exact: bytes and values are compared for equality.
Tolerance of the product: products of elements and scales are exact, so an
output's error is that of at most K additions in FP32 (each off by at most
2^-23 relative, whichever way the matrix unit rounds), K 2^-23 sum |a b|, then the
update's two roundings (2^-24 each) and the rounding into C's type, half a step
of the result (2^-8 BF16, 2^-11 FP16).
"""
import numpy as np
import pytest
import torch

import dense_gemm_16_amd as mg
import mx_oracle as mx
from gpu_helpers import say

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def _source(rows, cols, dtype, seed):
    """Values of every size the type holds in one matrix: ordinary rows, rows of
    midpoints between codes, tiny and huge rows, zeros."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)))
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.9, -0.25, -1.75, -5.0, 0.0])
    for r in range(rows):
        if r % 5 == 1:
            x[r] = rng.choice(mid, cols) * 2.0 ** int(rng.integers(-6, 7))
        if r % 7 == 3:
            x[r] *= 2.0 ** (-120 if dtype != "f16" else -20)
        if r % 7 == 5:
            x[r] *= 2.0 ** (100 if dtype != "f16" else 9)
        if r % 11 == 9:
            x[r] = 0.0
    return torch.from_numpy(x).to(TORCH[dtype])


def _quantize_and_check(x, view):
    q = mg.quantize_mx(view)
    torch.cuda.synchronize()
    rows, cols = x.shape
    codes, byte = mx.quantize(x.double().numpy())
    blocks = byte.shape[1]
    data, scales = q.data.cpu().numpy(), q.scales.cpu().numpy()
    assert np.array_equal(scales[:, :blocks], byte)
    got = mx.unpack(data[:, :16 * blocks])
    finite = np.repeat(byte != 255, 32, axis=1)
    # the sign of a zero is the source's; a NaN block's codes are 0
    assert np.array_equal(np.where(finite, got, 0), np.where(finite, codes, 0))
    assert not got[~finite].any()
    return q


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 31), (5, 33), (16, 160), (37, 257),
                                       (2, 2100), (130, 64), (65, 1000)])
@pytest.mark.parametrize("trans", [False, True])
def test_quantize_matches_the_rule(dtype, rows, cols, trans):
    say(f"quantize {dtype} {rows}x{cols} trans={trans}")
    x = _source(rows, cols, dtype, 7 * rows + cols)
    dx = (x.t().contiguous() if trans else x).cuda()
    q = _quantize_and_check(x, dx.t() if trans else dx)
    back = mg.dequantize_mx(q, torch.float32).cpu().numpy()
    want = mx.decode(q.data.cpu().numpy(), q.scales.cpu().numpy(), cols)
    # an element times its scale is an FP32 value unless it falls below 2^-149
    assert np.array_equal(back, want.astype(np.float32))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("trans", [False, True])
def test_quantize_strided_and_misaligned_source(dtype, trans):
    rows, cols = 33, 95
    x = _source(rows, cols, dtype, 5)
    stored = x.t().contiguous() if trans else x
    r, c = stored.shape
    buf = torch.full((1 + r * (c + 3) + 8,), float("nan"), dtype=x.dtype, device="cuda")
    view = buf[1:1 + r * (c + 3)].view(r, c + 3)[:, :c]
    view.copy_(stored.cuda())
    say(f"quantize {dtype} strided trans={trans}")
    _quantize_and_check(x, view.t() if trans else view)


def test_quantize_special_blocks():
    x = torch.zeros(6, 96)
    x[0, 5] = float("inf")
    x[1, 40] = float("nan")
    x[2, 64:] = torch.finfo(torch.float32).max
    x[3, :] = -torch.finfo(torch.float32).tiny / 4   # subnormal
    x[4, 33] = -float("inf")
    x[5, :32] = 1.0
    say("quantize special blocks")
    q = _quantize_and_check(x, x.cuda())
    back = mg.dequantize_mx(q, torch.float32).cpu()
    assert back[0, :32].isnan().all() and not back[0, 32:].any()
    assert back[1, 32:64].isnan().all() and not back[1, :32].any()
    assert torch.equal(back[5, :32], torch.ones(32))


def test_quantize_leaves_row_padding_alone():
    rows, cols, blocks = 9, 70, 3
    data = torch.full((rows, 80), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, 32), 0xCD, dtype=torch.uint8, device="cuda")
    x = _source(rows, cols, "bf16", 3).cuda()
    say("quantize into wide rows")
    for view in (x, x.t().contiguous().t()):
        mg.quantize_mx(view, out=mg.MxMatrix(data, scales, cols))
        torch.cuda.synchronize()
        assert (data[:, 16 * blocks:] == 0xAB).all() and (scales[:, blocks:] == 0xCD).all()


# results past 32 MiB take wide rows four pieces a lane; a padded `out` with rows off
# 16-byte boundaries is written by plain stores
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad", [0, 3])
def test_dequantize_large(dtype, pad):
    rows, cols = 4099, 5001
    rng = np.random.default_rng(5)
    data = rng.integers(0, 256, (rows, 157 * 16), dtype=np.uint8)
    scales = np.zeros((rows, 160), np.uint8)
    scales[:, :157] = rng.integers(118, 136, (rows, 157))
    want = torch.from_numpy(mx.decode(data, scales, cols)).to(TORCH[dtype])
    out = torch.full((rows, cols + 7 + pad), 7.0, dtype=TORCH[dtype], device="cuda")
    say(f"dequantize {dtype} {rows}x{cols} ld={out.stride(0)}")
    q = mg.MxMatrix(torch.from_numpy(data).cuda(), torch.from_numpy(scales).cuda(), cols)
    mg.dequantize_mx(q, TORCH[dtype], out[:, :cols])
    assert torch.equal(out[:, :cols].cpu(), want)
    assert (out[:, cols:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_dequantize_rounds_and_handles_every_code(dtype):
    rows, blocks = 16, 16
    data = torch.arange(rows * blocks * 16, dtype=torch.int64).mul_(37).remainder_(256)
    data = data.to(torch.uint8).view(rows, blocks * 16)
    scales = torch.arange(rows * blocks, dtype=torch.int64).to(torch.uint8).view(rows, blocks)
    for cols in (512, 509):
        say(f"dequantize {dtype} {cols}")
        got = mg.dequantize_mx(mg.MxMatrix(data.cuda(), scales.cuda(), cols), TORCH[dtype]).cpu()
        want = torch.from_numpy(mx.decode(data.numpy(), scales.numpy(), cols))
        want = want.float().to(TORCH[dtype])  # at most 3 significant bits: one rounding
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got[~got.isnan()], want[~want.isnan()])


def _operand(rows, k, rng, low=118, high=124):
    data = rng.integers(0, 256, (rows, k // 2), dtype=np.uint8)
    scales = np.full((rows, max(16, -(-(k // 32) // 16) * 16)), 255, np.uint8)  # padding: NaN bytes
    scales[:, :k // 32] = rng.integers(low, high, (rows, k // 32))
    return data, scales


def _device(op, k):
    return mg.MxMatrix(torch.from_numpy(op[0]).cuda(), torch.from_numpy(op[1]).cuda(), k)


def _check_product(M, N, K, c_type, alpha, beta, seed, ldc_extra=0, low=118, high=124,
                   config=-1):
    rng = np.random.default_rng(seed)
    a, b = _operand(M, K, rng, low, high), _operand(N, K, rng, low, high)
    prev = torch.from_numpy(rng.standard_normal((M, N))).to(TORCH[c_type])
    buf = torch.full((M, N + ldc_extra), float("nan"), dtype=TORCH[c_type], device="cuda")
    out = buf[:, :N]
    if beta != 0.0:
        out.copy_(prev)
    say(f"gemm_mx {M}x{N}x{K} {c_type} alpha={alpha} beta={beta}")
    mg.gemm_mx(_device(a, K), _device(b, K), out, alpha=alpha, beta=beta, config=config)
    torch.cuda.synchronize()
    if ldc_extra:
        assert buf[:, N:].isnan().all()
    A, B = mx.decode(*a, K), mx.decode(*b, K)
    s = A @ B.T
    S = np.abs(A) @ np.abs(B).T
    old = prev.double().numpy() if beta != 0.0 else 0.0
    want = alpha * s + beta * old
    tol = abs(alpha) * S * K * 2.0 ** -23
    tol = tol + 2.0 ** -23 * (np.abs(alpha * s) + np.abs(beta * old))
    tol = tol + HALF_STEP[c_type] * (np.abs(want) + tol) + 2.0 ** -24  # FP16 subnormals
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.isfinite(err).all() and (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 32), (1, 17, 64), (1, 4096, 4096), (3, 100, 96), (16, 512, 8192), (17, 33, 160),
    (32, 1000, 2080), (40, 64, 256), (63, 65, 288), (64, 64, 512), (100, 300, 1056),
    (129, 257, 1024), (256, 256, 2048), (300, 520, 2080), (512, 768, 1536), (700, 1100, 320),
    (1024, 1024, 992), (2048, 2304, 1280), (2, 70000, 64)])
@pytest.mark.parametrize("c_type", ["f32", "bf16"])
def test_product(M, N, K, c_type):
    _check_product(M, N, K, c_type, 1.0, 0.0, M + N + K)


@pytest.mark.parametrize("config", range(6))
@pytest.mark.parametrize("M,N,K,c_type,beta", [
    (1, 1, 32, "f32", 0.0), (5, 300, 1568, "bf16", 1.0), (70, 129, 256, "f16", 0.0),
    (256, 512, 768, "bf16", 0.0), (257, 255, 544, "f32", -1.0), (300, 700, 2304, "f16", 0.5),
    (520, 260, 4128, "bf16", 0.0), (128, 64, 480, "f32", 0.0)])
def test_every_configuration(M, N, K, c_type, beta, config):
    _check_product(M, N, K, c_type, 1.0, beta, M + N, 4, config=config)


@pytest.mark.parametrize("M,N,K,c_type,alpha,beta,extra", [
    (5, 48, 320, "f16", 0.5, 0.0, 0), (5, 48, 320, "f32", 1.0, 1.0, 3),
    (130, 200, 416, "f16", 0.25, -1.5, 1), (300, 300, 512, "bf16", 1.0, 1.0, 4),
    (512, 512, 512, "f32", -2.0, 0.5, 0), (1100, 1300, 736, "f16", 0.125, 2.0, 0),
    (260, 2000, 1024, "bf16", 1.0, 0.0, 8)])
def test_product_output_step(M, N, K, c_type, alpha, beta, extra):
    _check_product(M, N, K, c_type, alpha, beta, 3 * M + N, extra)


@pytest.mark.parametrize("M,N,K", [(7, 96, 640), (200, 256, 640)])
@pytest.mark.parametrize("low,high", [(66, 72), (180, 184)])
def test_product_of_small_and_large_scales(M, N, K, low, high):
    # scales down to 2^-61 (products down to 2^-124) and up to 2^56: 640 terms of
    # at most 36 x 2^112 stay below 2^127
    if low > 127:
        _check_product(M, N, K, "f32", 1.0, 0.0, M + low, low=low, high=high)
    else:
        _check_product(M, N, K, "f32", 2.0 ** 100, 0.0, M + low, low=low, high=high)


@pytest.mark.parametrize("M,N,K", [(7, 96, 640), (200, 256, 640)])
def test_product_past_the_range_of_fp32(M, N, K):
    # scales up to 2^62: single terms reach 36 x 2^124 > 2^128, past FP32
    rng = np.random.default_rng(M + 186)
    a, b = _operand(M, K, rng, 186, 190), _operand(N, K, rng, 186, 190)
    say(f"gemm_mx {M}x{N}x{K} out of range")
    got = mg.gemm_mx(_device(a, K), _device(b, K)).cpu().numpy()
    want = mx.decode(*a, K) @ mx.decode(*b, K).T
    assert not np.isfinite(got[np.abs(want) >= 2.0 ** 128]).any()


def test_product_of_no_columns_and_nan_scales():
    rng = np.random.default_rng(1)
    a, b = _operand(20, 64, rng), _operand(50, 64, rng)
    b[1][7, 1] = 255
    say("gemm_mx with a NaN block")
    out = mg.gemm_mx(_device(a, 64), _device(b, 64)).cpu()
    assert out[:, 7].isnan().all() and not out[:, :7].isnan().any()
    assert not out[:, 8:].isnan().any()
    # an empty sum: C = beta C
    c = torch.ones(20, 50, device="cuda")
    p = 1 << 20
    assert mg.migemm_gemm_mx(-1, 20, 50, 0, p, 16, p, 16, p, 16, p, 16, 1.0, 0.5, mg.F32,
                             c.data_ptr(), 50, torch.cuda.current_stream().cuda_stream) == mg.OK
    assert (c == 0.5).all()


def test_rows_of_k_need_not_be_whole_blocks():
    x, w = torch.randn(10, 75).bfloat16(), torch.randn(75, 40).bfloat16()
    say("gemm_mx of 75 columns")
    qx, qw = mg.quantize_mx(x.cuda()), mg.quantize_mx(w.cuda().t())
    assert qw.shape == (40, 75)
    out = mg.gemm_mx(qx, qw).double().cpu()
    dx, dw = (mg.dequantize_mx(q, torch.float32).double().cpu() for q in (qx, qw))
    tol = 96 * 2.0 ** -23 * (dx.abs() @ dw.abs().t()) + 2.0 ** -24
    assert ((out - dx @ dw.t()).abs() <= tol).all()


def test_product_on_another_stream_and_replayed_in_a_graph():
    rng = np.random.default_rng(3)
    cases = []
    for M, N, K in ((4, 512, 1024), (300, 512, 1056), (1024, 1024, 1024)):
        a, b = _device(_operand(M, K, rng), K), _device(_operand(N, K, rng), K)
        cases.append((a, b, mg.gemm_mx(a, b, out_dtype=torch.bfloat16)))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    say("gemm_mx on a side stream by handle")
    for a, b, want in cases:
        side.wait_stream(torch.cuda.current_stream())
        got = mg.gemm_mx(a, b, out_dtype=torch.bfloat16, stream=side.cuda_stream)
        side.synchronize()
        assert torch.equal(got, want)
    x = torch.randn(64, 1024, device="cuda")
    outs = [torch.empty_like(w) for _, _, w in cases]
    say("quantize_mx and gemm_mx in a graph")
    warm = mg.gemm_mx(mg.quantize_mx(x), cases[0][1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chained = mg.gemm_mx(mg.quantize_mx(x), cases[0][1])
        for (a, b, _), o in zip(cases, outs):
            mg.gemm_mx(a, b, o)
    for i in range(3):
        x.normal_()
        for o in outs:
            o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(chained, mg.gemm_mx(mg.quantize_mx(x), cases[0][1]))
        assert all(torch.equal(o, w) for o, (_, _, w) in zip(outs, cases))
    assert warm.shape == chained.shape


# ------------------------------------------- past 2^32 threads, one launch's limit

def _spots(n, *borders):
    """Ranges of 300 at both ends and around the borders that lie inside n."""
    starts = [0, n - 300] + [b - 150 for b in borders if 150 < b < n - 150]
    return [slice(s, s + 300) for s in starts]


@pytest.mark.parametrize("dtype,trans", [("bf16", False), ("f32", True)])
def test_quantize_and_decode_more_rows_than_one_launch_takes(dtype, trans):
    # rows of one element, four threads each: 2^32 at 2^30 rows
    rows = (1 << 30) + 333
    say(f"quantize {dtype} {rows}x1 trans={trans}")
    values = torch.tensor([0.0, 1.0, -1.5, 3.0, -0.25, 96.0, 0.375], device="cuda")
    pick = torch.randint(0, 7, (rows,), device="cuda", dtype=torch.uint8)
    x = torch.empty(rows, dtype=TORCH[dtype], device="cuda")
    for s in range(0, rows, 1 << 27):
        x[s:s + (1 << 27)] = values[pick[s:s + (1 << 27)].int()].to(x.dtype)
    del pick
    if trans:   # stored 1 x rows (the wrapper takes a single column for row-major)
        q = mg.MxMatrix(torch.empty(rows, 16, dtype=torch.uint8, device="cuda"),
                        torch.empty(rows, 16, dtype=torch.uint8, device="cuda"), 1)
        assert mg.migemm_quantize_mx(mg.F32, mg.OP_T, rows, 1, x.data_ptr(), rows,
                                     q.data.data_ptr(), 16, q.scales.data_ptr(), 16,
                                     torch.cuda.current_stream().cuda_stream) == mg.OK
    else:
        q = mg.quantize_mx(x[:, None])
    # a block of one element of at most two significant bits holds it exactly
    back = mg.dequantize_mx(q, x.dtype)
    assert torch.equal(back[:, 0], x)
    for s in _spots(rows, 1 << 30):
        part = mg.quantize_mx(x[s, None])
        assert torch.equal(q.data[s], part.data) and torch.equal(q.scales[s, 0], part.scales[:, 0])


def test_quantize_more_columns_than_one_launch_takes():
    # k as the source's row index, 512 threads for 256 of k: 2^32 at nearly 2^31
    cols = ((1 << 23) - 1) * 256 + 33
    blocks = (cols + 31) // 32
    say(f"quantize bf16 1x{cols} k as the row index")
    x = torch.empty(cols, dtype=torch.bfloat16, device="cuda")
    for s in range(0, cols, 1 << 28):
        x[s:s + (1 << 28)].normal_()
    ldd, ldsc = 16 * blocks, (blocks + 15) // 16 * 16
    data = torch.zeros(1, ldd, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(1, ldsc, dtype=torch.uint8, device="cuda")
    assert mg.migemm_quantize_mx(mg.BF16, mg.OP_T, 1, cols, x.data_ptr(), 1, data.data_ptr(), ldd,
                                 scales.data_ptr(), ldsc,
                                 torch.cuda.current_stream().cuda_stream) == mg.OK
    want = mg.quantize_mx(x[None])
    assert torch.equal(data, want.data) and torch.equal(scales[:, :blocks], want.scales[:, :blocks])


# 16 columns of C to a workgroup of 512 in the rows kernel (32 from 8161 on), 64 to one of
# 64x64 tiles
@pytest.mark.parametrize("M,config,N", [(2, 0, (1 << 28) + 333), (3, 1, (1 << 29) + 333)])
def test_product_of_more_columns_than_one_launch_takes(M, config, N):
    say(f"gemm_mx {M}x{N}x32 config {config}")
    rng = np.random.default_rng(M)
    a = _device(_operand(M, 32, rng), 32)
    data = torch.randint(0, 256, (N, 16), dtype=torch.uint8, device="cuda")
    scales = torch.zeros(N, 16, dtype=torch.uint8, device="cuda")
    scales[:, 0] = torch.randint(118, 124, (N,), dtype=torch.uint8, device="cuda")
    got = mg.gemm_mx(a, mg.MxMatrix(data, scales, 32), out_dtype=torch.bfloat16, config=config)
    for s in _spots(N, ((1 << 23) - 1) * 16, 1 << 28, ((1 << 23) - 1) * 64):
        part = mg.MxMatrix(data[s].contiguous(), scales[s].contiguous(), 32)
        assert torch.equal(got[:, s], mg.gemm_mx(a, part, out_dtype=torch.bfloat16, config=config))
    step = 1 << 24
    for s in range(0, N, step):   # nothing is left out in between
        part = mg.MxMatrix(data[s:s + step], scales[s:s + step], 32)
        assert torch.equal(got[:, s:s + step],
                           mg.gemm_mx(a, part, out_dtype=torch.bfloat16, config=config))


# Sources past 192 MiB on 8-byte boundaries are read with non-temporal loads: rows that end
# inside a lane's group, k that ends inside a block, and (one element off) the plain form
@pytest.mark.parametrize("dtype,rows,cols,ld", [("f32", 7003, 7337, 7004), ("f32", 7004, 7330, 7005),
                                                ("bf16", 10007, 10273, 10008),
                                                ("f16", 10006, 10300, 10012)])
def test_quantize_large_sources_with_k_as_the_row_index(dtype, rows, cols, ld):
    say(f"quantize {dtype} {rows}x{cols} ld={ld} k as the row index")
    g = torch.Generator(device="cuda").manual_seed(rows)
    stored = torch.full((cols, ld), float("nan"), dtype=TORCH[dtype], device="cuda")
    x = stored[:, :rows].t()
    x.copy_(torch.randn(rows, cols, generator=g, device="cuda") *
            torch.exp(torch.randn(rows, 1, generator=g, device="cuda")))
    assert cols * ld * x.element_size() > 192 << 20
    q = mg.quantize_mx(x)
    # rows along k go through the other kernel, and the last rows through the oracle
    want = mg.quantize_mx(x.contiguous())
    blocks = (cols + 31) // 32
    assert torch.equal(q.data[:, :16 * blocks], want.data[:, :16 * blocks])
    assert torch.equal(q.scales[:, :blocks], want.scales[:, :blocks])
    codes, byte = mx.quantize(x[-70:].double().cpu().numpy())
    assert np.array_equal(q.scales[-70:, :blocks].cpu().numpy(), byte)
    assert np.array_equal(mx.unpack(q.data[-70:, :16 * blocks].cpu().numpy()), codes)


@pytest.mark.parametrize("M,N,K", [(7, 96, 640), (64, 70, 512), (200, 256, 640)])
def test_product_below_the_normal_range_of_fp32(M, N, K):
    """Scales of 2^-64 to 2^-62: terms are multiples of 0.25 2^-128 = 2^-130, sums of 640
    of them below 2^-109, so every partial sum below 2^-106 is a multiple of 2^-130 that
    FP32 holds exactly, subnormal or not.  With scales of A down to 2^-127 every term lies
    below 36 2^-187: the sums round to 0, or to the smallest FP32 number."""
    rng = np.random.default_rng(M + 5)
    a, b = _operand(M, K, rng, 63, 66), _operand(N, K, rng, 63, 66)
    say(f"gemm_mx {M}x{N}x{K} below the normal range")
    want = mx.decode(*a, K) @ mx.decode(*b, K).T
    got = mg.gemm_mx(_device(a, K), _device(b, K)).double().cpu().numpy()
    assert np.abs(want).max() < 2.0 ** -106 and (np.abs(want) < 2.0 ** -126).any()
    assert np.array_equal(got, want)
    a, b = _operand(M, K, rng, 0, 3), _operand(N, K, rng, 60, 66)
    got = mg.gemm_mx(_device(a, K), _device(b, K)).double().cpu().numpy()
    assert (np.abs(got) <= 2.0 ** -149).all()
