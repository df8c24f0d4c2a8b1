"""The INT8 payload by rows byte for byte against its definition, its products and the
linear layer against float64, and the refusals."""
import os

import numpy as np
import pytest
import torch

import quantized_collective_payloads_amd as qcp
from tests import int8_reference as R

GPU = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NAME = {v: k for k, v in DT.items()}


@pytest.fixture()
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    qcp.library()


def wide(t):
    return t.detach().to(torch.float64).cpu().numpy()


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def values(rows, cols, dt, seed):
    """Rows of very different sizes, with outliers, zeros, signed zeros, and rows whose scale is
    a power of two and whose quotients are half-integers."""
    g = generator(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x[torch.rand(rows, cols, generator=g, device="cuda") < 0.01] *= 30
    k = torch.randint(-6 if dt == "f16" else -30, 7, (rows, 1), generator=g, device="cuda").float()
    x = x * torch.exp2(k)
    ties = torch.randint(-254, 255, (rows, cols), generator=g, device="cuda").float() / 2
    ties[:, 0] = 127.0
    x = torch.where(torch.rand(rows, 1, generator=g, device="cuda") < 0.3, ties * torch.exp2(k), x)
    if rows > 2:
        x[1] = 0
        x[2] = -0.0
    return x.to(DT[dt])


def host(codes, scales):
    return codes.view(torch.int8).cpu().numpy(), scales.cpu().numpy()


def check_payload(x, what, got=None):
    codes, scales = got or qcp.int8_quantize(x)
    (gc, gs), (wc, ws) = host(codes, scales), R.payload(wide(x))
    assert gs.shape == ws.shape and np.array_equal(gs, ws, equal_nan=True), (what, np.argwhere(gs != ws)[:4])
    assert gc.shape == wc.shape and np.array_equal(gc, wc), (what, np.argwhere(gc != wc)[:4])
    return codes, scales


# every way a row is dealt to lanes, at its edges: by 16-bit rows of up to 1024, 4096,
# 16384, 65536 values and longer (fp32: half), few rows and many
SHAPES = [(1, 1), (1, 127), (3, 128), (2, 129), (5, 255), (37, 1003), (128, 64), (1, 1024), (9, 1025), (1, 4096), (6, 4097),
          (1023, 2500), (1024, 2500), (1030, 513), (1, 16384), (255, 5000), (256, 5000), (257, 8193), (2, 16500), (1, 40001),
          (3, 65536), (2, 65537), (2, 140003), (5000, 1)]


@GPU
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_and_back(gpu, rows, cols, dt):
    x = values(rows, cols, dt, rows * 7 + cols)
    codes, scales = check_payload(x, (rows, cols, dt))
    gc, gs = host(codes, scales)
    for yt in DT:
        y = qcp.int8_dequantize(codes, scales, cols, DT[yt])
        assert np.array_equal(wide(y), R.read(gc[:, :cols], gs, yt)), (rows, cols, dt, yt)


@GPU
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_every_16_bit_value(gpu, dt):
    """All 65,536 patterns, each the largest of its row, and all beside larger ones; an
    infinity or a NaN makes its row's scale NaN and its codes 0."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(DT[dt]).cuda()
    alone = torch.zeros(65536, 5, dtype=DT[dt], device="cuda")
    alone[:, 1] = bits
    alone[:, 3] = bits / 3
    codes, scales = check_payload(alone, "alone")
    bad = ~torch.isfinite(alone).all(1)
    assert torch.equal(torch.isnan(scales), bad) and not codes[bad].any()
    assert torch.isnan(qcp.int8_dequantize(codes, scales, 5)[bad]).all()
    for top in (127.0, 1.0, 448.0, 2.0 ** -13):
        beside = torch.full((1024, 130), top, dtype=DT[dt], device="cuda")
        beside[:, 1:65] = bits.view(1024, 64)
        check_payload(beside, ("beside", top))


@GPU
@pytest.mark.parametrize("cols", [40, 3000, 20000, 70000])
def test_fp32_extremes(gpu, cols):
    """Scales that are subnormal, underflow or are the largest, and values that are not finite
    in one place only."""
    tops = [0.0, -0.0, 1e-45, -1e-45, 63 * 2.0 ** -149, 64 * 2.0 ** -149, 2.0 ** -140, 2.0 ** -127, 2.0 ** -126, 127 * 2.0 ** -126,
            2.0 ** -64, 2.0 ** -57, 2.0 ** 70, 2.0 ** 71, 3.4e38, -3.4028e38, float("inf"), float("-inf"), float("nan"), 1.0]
    a = torch.zeros(len(tops), cols, device="cuda")
    t = torch.tensor(tops, device="cuda")
    a[:, cols - 1], a[:, 7], a[:, 9] = t, t / 5, -t / 2
    check_payload(a, "extremes")


@GPU
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_strides(gpu, dt):
    """Row strides, unaligned starts, transposed, overlapping and stepped inputs: all as their
    contiguous copy; results to the caller's buffers, and nothing beside them."""
    big = values(140, 1300, dt, 5)
    for v in (big[1:, 3:1004], big[::2, :777], big.t()[5:900], big[:, ::3], big[:1].expand(6, 1300), big[:, 1:2], big[3:4, 5:900]):
        a, b = qcp.int8_quantize(v), qcp.int8_quantize(v.contiguous())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), (tuple(v.shape), v.stride())
    rows, cols = 70, 1001
    x = big[:rows, :cols]
    codes = torch.full((rows + 2, 1024), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows + 8,), 5.0, device="cuda")
    got = qcp.int8_quantize(x, codes=codes[1:rows + 1], scales=scales[4:rows + 4])
    check_payload(x, "buffers", got)
    assert (codes[0] == 77).all() and (codes[-1] == 77).all() and (scales[:4] == 5).all() and (scales[-4:] == 5).all()
    y = torch.full((rows + 2, cols), 3.0, dtype=DT[dt], device="cuda")
    qcp.int8_dequantize(*got, cols, out=y[1:rows + 1])
    assert torch.equal(y[1:rows + 1], qcp.int8_dequantize(*got, cols, DT[dt])) and (y[0] == 3).all() and (y[-1] == 3).all()


@GPU
def test_empty(gpu):
    none = torch.empty(0, 300, device="cuda")
    codes, scales = qcp.int8_quantize(none)
    assert codes.shape == (0, 384) and scales.shape == (0,) and qcp.int8_dequantize(codes, scales, 300).shape == (0, 300)
    codes, scales = qcp.int8_quantize(torch.empty(7, 0, device="cuda", dtype=torch.bfloat16), scales=torch.ones(7, device="cuda"))
    assert codes.shape == (7, 0) and not scales.any()
    full = qcp.int8_quantize(torch.ones(5, 300, device="cuda"))
    assert qcp.int8_dequantize(codes, scales, 0).shape == (7, 0)
    assert qcp.int8_matmul(codes, scales, codes, scales).eq(0).all()
    assert qcp.int8_matmul(*qcp.int8_quantize(none), *full).shape == (0, 5)
    assert qcp.int8_matmul(*full, *qcp.int8_quantize(none)).shape == (5, 0)
    a = torch.ones(4, 0, device="cuda", dtype=torch.bfloat16)
    nothing = qcp.int8_quantize(none)
    assert qcp.int8_matmul_mixed(a, *nothing, 300).eq(0).all()
    assert qcp.int8_matmul_mixed(a.t(), *nothing, 300, transpose=True).shape == (4, 300)
    assert qcp.int8_matmul_mixed(torch.ones(0, 5, device="cuda", dtype=torch.bfloat16), *full, 300).shape == (0, 300)
    assert qcp.int8_matmul_mixed(torch.ones(4, 7, device="cuda", dtype=torch.bfloat16), codes, scales, 0).shape == (4, 0)


@GPU
def test_offsets_past_32_bits(gpu):
    """A matrix of more than 2^31 elements: its first, last and middle rows as by themselves."""
    rows, cols = 66001, 33001
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.view(-1)[: 1 << 20].normal_()
    x.view(-1)[1 << 20:].fill_(0.25)
    x[-3:].normal_()
    x[65080:65090].normal_()                       # element 2^31 lies in row 65074, byte 2^31 of the codes in 64527
    x[64520:64530].normal_()
    codes, scales = qcp.int8_quantize(x)
    for r in (0, 64520, 65070, 65080, rows - 3):
        part = qcp.int8_quantize(x[r:r + 3].clone())
        assert torch.equal(codes[r:r + 3], part[0]) and torch.equal(scales[r:r + 3], part[1]), r
    y = qcp.int8_dequantize(codes, scales, cols)
    for r in (0, 64520, 65070, 65080, rows - 3):
        assert torch.equal(y[r:r + 3], qcp.int8_dequantize(codes[r:r + 3].clone(), scales[r:r + 3].clone(), cols)), r


# ------------------------------------------------------------------ the product

# every kernel and its edges: one token, few rows, tiles of 64, 128 and 256, slices of K
MATMULS = [(1, 1, 1), (1, 16, 128), (1, 1001, 4096), (1, 257, 16384), (3, 130, 100), (16, 100, 640), (17, 300, 5000), (31, 64, 8300),
           (33, 65, 129), (77, 1001, 1111), (200, 520, 8192), (129, 127, 384), (300, 260, 257), (513, 1030, 900),
           (64, 512, 9000), (40, 200, 20000), (256, 256, 6000), (2000, 17, 700), (700, 900, 1)]


def random_payload(rows, cols, seed):
    """Any bytes, -128 too, and scales of several sizes; what pads a row is 0."""
    g = generator(seed)
    codes = torch.randint(0, 256, (rows, R.padded(cols)), generator=g, device="cuda").to(torch.uint8)
    codes[:, cols:] = 0
    return codes, torch.exp2(torch.rand(rows, generator=g, device="cuda") * 8 - 12)


def check_product(a, b, dt, what):
    c = qcp.int8_matmul(*a, *b, dtype=DT[dt])
    want = R.product(host(*a), host(*b))
    assert c.dtype == DT[dt] and c.shape == want.shape
    off = np.abs(wide(c) - want) - R.product_bound(want, dt)
    assert (off <= 0).all(), (what, np.argwhere(~(off <= 0))[:4], off.max())
    return c


@GPU
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", MATMULS)
def test_product(gpu, M, N, K, dt):
    a, b = random_payload(M, K, M + N), random_payload(N, K, K)
    if dt == "f16":                                # within its range
        a = a[0], a[1] * 2.0 ** -10
    c = check_product(a, b, dt, (M, N, K, dt))
    out = torch.full((M + 2, N), 3.0, dtype=DT[dt], device="cuda")
    qcp.int8_matmul(*a, *b, out=out[1:M + 1])
    assert torch.equal(out[1:M + 1], c) and (out[0] == 3).all() and (out[-1] == 3).all()


@GPU
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(4100, 4130, 4200), (3000, 3010, 1111), (700, 3030, 520), (65, 8200, 900), (5121, 2050, 640),
                                   (2100, 8230, 130)])
def test_product_over_several_rounds_of_tiles(gpu, M, N, K, dt):
    check_product(random_payload(M, K, M + N), random_payload(N, K, K), dt, (M, N, K, dt))


@GPU
@pytest.mark.parametrize("M,N", [(1, 40), (20, 40), (70, 300)])
def test_the_longest_k_with_the_largest_sums(gpu, M, N):
    """130944 times (-128)^2 is the largest sum there is."""
    K = 130944
    a = torch.full((M, K), 128, dtype=torch.uint8, device="cuda"), torch.ones(M, device="cuda")
    b = torch.full((N, K), 128, dtype=torch.uint8, device="cuda"), torch.ones(N, device="cuda")
    b[0][N // 2:] = 127
    c = qcp.int8_matmul(*a, *b, dtype=torch.float32)
    assert (c[:, :N // 2] == float(K * 16384)).all()
    assert (c[:, N // 2:] == float(np.float32(-K * 128 * 127))).all()
    with pytest.raises(qcp.QcpError, match="EINVAL"):
        big = torch.zeros(2, K + 128, dtype=torch.uint8, device="cuda"), torch.ones(2, device="cuda")
        qcp.int8_matmul(*big, *big)


@GPU
@pytest.mark.parametrize("M,N", [(1, 50), (40, 70), (300, 600), (2100, 2200)])
def test_product_extreme_scales(gpu, M, N):
    """Scales whose products leave fp32 on the way to a result that does not, subnormal ones,
    zeros, and NaN, which stays in its row or column."""
    a, b = random_payload(M, 200, 1), random_payload(N, 200, 2)
    sa, sb = a[1].clone(), b[1].clone()
    sa[0], sb[0], sb[1], sb[2], sb[3] = 2.0 ** 120, 2.0 ** -140, 2.0 ** -126, float("nan"), 0.0
    if M > 5:
        sa[1], sa[2], sa[3], sa[4] = 2.0 ** -149, 2.0 ** -100, float("nan"), 0.0
        sa[M - 1] = 2.0 ** 119
    sb[N - 1], sb[N - 2], sb[N - 3] = 2.0 ** 100, 2.0 ** -100, 2.0 ** -149
    want = R.product(host(a[0], sa), host(b[0], sb))
    got = wide(qcp.int8_matmul(a[0], sa, b[0], sb, dtype=torch.float32))
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan) and nan[:, 2].all() and not nan.all()
    over = np.abs(want) > float(np.finfo(np.float32).max)
    assert np.array_equal(np.isinf(got), over)
    live = ~nan & ~over
    assert (np.abs(got - want)[live] <= R.product_bound(want, "f32")[live]).all()


@GPU
def test_product_with_more_than_2_31_results(gpu):
    M, N, K = 50001, 44003, 128
    a, b = random_payload(M, K, 1), random_payload(N, K, 2)
    c = qcp.int8_matmul(*a, *b)
    for r in (0, 24400, 48800, 48806, M - 2):      # result 2^31 lies in row 48803
        part = qcp.int8_matmul(a[0][r:r + 2].clone(), a[1][r:r + 2].clone(), *b)
        assert torch.equal(c[r:r + 2], part), r


# ------------------------------------------------------------------ the mixed product

# tiles of 64, 128 and 256, slices of K; each size at and beside the edges of a tile
MIXED = [(1, 1, 1), (1, 130, 9), (5, 64, 128), (64, 64, 64), (65, 129, 63), (77, 520, 1033), (130, 300, 257), (7, 40, 5000),
         (300, 1000, 100), (1500, 2100, 65), (1100, 3100, 200), (3000, 4000, 70), (4097, 3590, 130), (16, 4100, 2000)]


# copied to LDS as they lie, in tiles of 128 and 256, over one round and several, with K of whole stages
# and not, in slices and not, with rows that are first copied to aligned ones
LARGER = [(260, 4000, 3000), (2050, 2060, 1000), (1024, 1500, 8), (1024, 4096, 64), (2048, 2048, 1088), (4104, 4104, 136), (4096, 4096, 8),
          (8192, 4104, 520), (5000, 9000, 192), (2048, 4096, 4104), (1027, 4100, 4099), (4099, 1500, 2051), (520, 4099, 8200), (9001, 4111, 1029)]


def mixed_case(M, N, K, dt, transpose, seed):
    g = generator(seed)
    a = torch.randn(*((K, M) if transpose else (M, K)), generator=g, device="cuda").to(DT[dt])
    codes, scales = random_payload(K, N, seed + 1)
    return a, codes, scales


def check_mixed(a, codes, scales, N, transpose, out, what, c=None):
    if c is None:
        c = qcp.int8_matmul_mixed(a, codes, scales, N, transpose=transpose, dtype=DT[out])
    A = wide(a.t() if transpose else a)
    gc, gs = host(codes, scales)
    X = R.read(gc[:, :N], gs, NAME[a.dtype])
    want, size = A @ X, np.abs(A) @ np.abs(X)
    # K products, exact in fp32, and as many sums, each off by a unit of the last place of at most the sum of sizes
    bound = A.shape[1] * 2.0 ** -23 * size + R.UNIT[out] * np.abs(want) * 1.01 + R.LEAST[out]
    assert c.dtype == DT[out] and c.shape == want.shape
    off = np.abs(wide(c) - want) - bound
    assert (off <= 0).all(), (what, np.argwhere(~(off <= 0))[:4], off.max())
    return c


@GPU
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", MIXED)
def test_mixed_product(gpu, M, N, K, dt, transpose):
    a, codes, scales = mixed_case(M, N, K, dt, transpose, M + N + K)
    for out in ("f32", dt):
        c = check_mixed(a, codes, scales, N, transpose, out, (M, N, K, dt, transpose, out))
        to = torch.full((M + 2, N), 3.0, dtype=DT[out], device="cuda")
        qcp.int8_matmul_mixed(a, codes, scales, N, transpose=transpose, out=to[1:M + 1])
        assert torch.equal(to[1:M + 1], c) and (to[0] == 3).all() and (to[-1] == 3).all()


@GPU
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", MIXED + LARGER)
def test_mixed_product_of_integers_is_exact(gpu, M, N, K, dt, transpose):
    """Small integers times powers of two: all sums are exact, so every value is, whatever the
    order.  K takes each row of a stage, its last one too."""
    g = generator(K)
    a = torch.randint(-3, 4, (K, M) if transpose else (M, K), generator=g, device="cuda").to(DT[dt])
    codes = torch.randint(-9, 10, (K, R.padded(N)), generator=g, device="cuda").to(torch.int8).view(torch.uint8)
    scales = torch.exp2(torch.randint(-3, 1, (K,), generator=g, device="cuda").float())
    c = qcp.int8_matmul_mixed(a, codes, scales, N, transpose=transpose, dtype=torch.float32)
    x = codes.view(torch.int8)[:, :N].double() * scales.double()[:, None]
    assert torch.equal(c.double(), (a.double().t() if transpose else a.double()) @ x)


@GPU
@pytest.mark.parametrize("transpose", [False, True])
def test_mixed_product_strides(gpu, transpose):
    """Rows apart, starts that are not aligned, transposed views and other strides: all as their
    contiguous copy, bit for bit."""
    g = generator(3)
    big = torch.randn(400, 701, generator=g, device="cuda").to(torch.bfloat16)
    for v in (big[:300, :600], big[1:301, 3:604], big.t()[1:601, 5:306], big[::2, 1:500], big[:200, ::3], big[:1].expand(90, 701),
              big[:, 5:6], big[7:8, 1:333]):
        K = v.shape[0 if transpose else 1]
        codes, scales = random_payload(K, 333, 5)
        got = qcp.int8_matmul_mixed(v, codes, scales, 333, transpose=transpose)
        want = qcp.int8_matmul_mixed(v.contiguous(), codes, scales, 333, transpose=transpose)
        assert torch.equal(got, want), (tuple(v.shape), v.stride())
        flipped = qcp.int8_matmul_mixed(v.contiguous().t(), codes, scales, 333, transpose=not transpose)
        assert torch.equal(got, flipped)


@GPU
@pytest.mark.parametrize("transpose", [False, True])
def test_mixed_product_beside_rows_that_are_not_finite(gpu, transpose):
    """What lies beside a view of the gradient, before, behind and between its rows, is not read into the sums."""
    M, N, K = 300, 200, 333
    shape = (K, M) if transpose else (M, K)
    g = generator(1)
    a = torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)
    codes, scales = random_payload(K, N, 4)
    around = torch.full((shape[0] + 2, shape[1] + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    around[1:-1, 7:7 + shape[1]] = a
    got = qcp.int8_matmul_mixed(around[1:-1, 7:7 + shape[1]], codes, scales, N, transpose=transpose)
    assert torch.equal(got, qcp.int8_matmul_mixed(a, codes, scales, N, transpose=transpose))
    # and NaN or infinity within them reaches its own results alone
    b = a.clone()
    b[5, 9], b[11, 20] = float("nan"), float("inf")
    got = qcp.int8_matmul_mixed(b, codes, scales, N, transpose=transpose)
    rows = (9, 20) if transpose else (5, 11)
    kept = torch.ones(M, dtype=torch.bool, device="cuda")
    kept[list(rows)] = False
    want = qcp.int8_matmul_mixed(a, codes, scales, N, transpose=transpose)
    assert torch.equal(got[kept], want[kept]) and torch.isnan(got[rows[0]]).all() and not torch.isfinite(got[rows[1]]).any()


@GPU
def test_mixed_product_of_small_fp16_values(gpu):
    """fp16's subnormal numbers count, in the gradient and in what the payload stands for."""
    a = torch.full((70, 96), 3 * 2.0 ** -24, device="cuda").to(torch.float16)
    codes = torch.full((96, 128), 1, dtype=torch.uint8, device="cuda")
    for scale in (2.0, 2.0 ** -20):
        c = qcp.int8_matmul_mixed(a, codes, torch.full((96,), scale, device="cuda"), 100, dtype=torch.float32)
        assert (c == 96 * 3 * 2.0 ** -24 * scale).all(), scale


@GPU
@pytest.mark.parametrize("transpose", [False, True])
def test_mixed_product_past_32_bits(gpu, transpose):
    """Gradients and results of more than 2^31 elements."""
    rows, cols = 70001, 31013
    a = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    for r in (0, 35000, 69244, 69260, rows - 5):   # element 2^31 lies in row 69244
        a[r:r + 5].normal_()
    if transpose:                                  # summed over the 70001 rows: those that are not zero
        live = [r + i for r in (0, 35000, 69244, 69260, rows - 5) for i in range(5)]
        codes, scales = random_payload(rows, 130, 3)
        c = qcp.int8_matmul_mixed(a, codes, scales, 130, transpose=True, dtype=torch.float32)
        check_mixed(a[live][:, -700:].contiguous(), codes[live].contiguous(), scales[live].contiguous(), 130, True, "f32", "rows", c[-700:])
    else:
        codes, scales = random_payload(cols, 20, 3)
        c = qcp.int8_matmul_mixed(a, codes, scales, 20, dtype=torch.float32)
        for r in (0, 35000, 69244, 69260, rows - 5):
            check_mixed(a[r:r + 5].contiguous(), codes, scales, 20, False, "f32", r, c[r:r + 5])
        del c
        b, (codes, scales) = a[:, :40].clone(), random_payload(40, cols, 4)
        c = qcp.int8_matmul_mixed(b, codes, scales, cols)
        for r in (0, 35000, 69244, 69260, rows - 5):
            check_mixed(b[r:r + 5].contiguous(), codes, scales, cols, False, "bf16", r, c[r:r + 5])


# ------------------------------------------------------------------ streams, graphs, repeats

@GPU
def test_streams_and_graph(gpu):
    """On a side stream, and captured: replays with eager work between them give the same bytes,
    with scratch memory (a long K) and without."""
    x, w = values(300, 1000, "bf16", 1), values(520, 1000, "bf16", 2)
    long = values(64, 9000, "bf16", 3)
    dy = values(300, 520, "bf16", 4)
    tall = torch.randn(6000, 64, device="cuda").to(torch.bfloat16)

    def chain():
        a, b, c = qcp.int8_quantize(x), qcp.int8_quantize(w), qcp.int8_quantize(long)
        t = qcp.int8_quantize(tall)
        return [*a, *b, qcp.int8_matmul(*a, *b, dtype=torch.float32), qcp.int8_matmul(a[0][:1], a[1][:1], *b),
                qcp.int8_matmul(*c, *c), qcp.int8_dequantize(*a, 1000), qcp.int8_matmul_mixed(dy, *b, 1000),
                qcp.int8_matmul_mixed(dy, *a, 1000, transpose=True, dtype=torch.float32),
                qcp.int8_matmul_mixed(tall, *t, 64, transpose=True), qcp.int8_linear(x, w), qcp.int8_linear(x, b)]
    same = lambda p, q: torch.equal(p.view(torch.uint8), q.view(torch.uint8))  # noqa: E731
    lib = qcp.library()
    assert lib.qcp_int8_matmul_work(64, 64, 9000) > 0 and lib.qcp_int8_mixed_work(64, 64, 6000, 1, 1) > 0
    want = [t.clone() for t in chain()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = chain()
    torch.cuda.synchronize()
    assert all(map(same, got, want))
    graphs = []
    for _ in range(2):                             # two graphs, replayed in turn
        graphs.append(torch.cuda.CUDAGraph())
        with torch.no_grad(), torch.cuda.graph(graphs[-1]):
            graphs[-1].got = chain()
    for k in range(4):
        for graph in graphs:
            for t in graph.got:
                t.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for graph in graphs:
            assert all(map(same, graph.got, want)), k
        chain()


@GPU
def test_two_calls_at_once(gpu):
    """On two streams, each with its own scratch memory."""
    a, b = random_payload(64, 9000, 1), random_payload(128, 9000, 2)
    dy, t = torch.randn(6000, 64, device="cuda").to(torch.bfloat16), random_payload(6000, 128, 3)
    want = qcp.int8_matmul(*a, *b), qcp.int8_matmul_mixed(dy, *t, 128, transpose=True)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for k in range(20):
        with torch.cuda.stream(streams[k % 2]):
            got.append((qcp.int8_matmul(*a, *b), qcp.int8_matmul_mixed(dy, *t, 128, transpose=True)))
    torch.cuda.synchronize()
    assert all(torch.equal(p, want[0]) and torch.equal(q, want[1]) for p, q in got)


# ------------------------------------------------------------------ the layer

def layer_formula(x, w, dy):
    """(y, dx, dw) in 64 bits, and for each the sum of sizes its rounding goes by."""
    dt = NAME[dy.dtype]
    qx, qw = R.payload(wide(x)), R.payload(wide(w))
    X, W, D = R.read(qx[0][:, :x.shape[1]], qx[1], dt), R.read(qw[0][:, :w.shape[1]], qw[1], dt), wide(dy)
    return R.product(qx, qw), (D @ W, np.abs(D) @ np.abs(W)), (D.T @ X, np.abs(D).T @ np.abs(X))


def check_layer(y, dx, dw, x, w, dy):
    Y, DX, DW = layer_formula(x, w, dy)
    dt = NAME[x.dtype]
    assert (np.abs(wide(y) - Y) <= R.product_bound(Y, dt)).all()
    for got, (want, size), n, kind in ((dx, DX, w.shape[0], x.dtype), (dw, DW, x.shape[0], w.dtype)):
        if got is None:
            continue
        unit = 0 if NAME[kind] == "f32" else R.UNIT[NAME[kind]]
        bound = n * 2.0 ** -23 * size + unit * np.abs(want) * 1.01 + R.LEAST[NAME[kind]]
        assert got.dtype == kind and (np.abs(wide(got) - want) <= bound).all()


@GPU
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,I,O", [(1, 64, 32), (7, 100, 33), (77, 520, 260), (300, 257, 130), (2000, 64, 1100)])
def test_linear_and_its_gradients_match_the_formula(gpu, T, I, O, dt, kind):
    g = generator(T)
    make = lambda d, *s: torch.randn(*s, generator=g, device="cuda").to(DT[d])  # noqa: E731
    x, w, dy = make(dt, T, I).requires_grad_(), (make(kind, O, I) * 0.05).requires_grad_(), make(dt, T, O) * 0.01
    y = qcp.int8_linear(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), dy, retain_graph=True)
    check_layer(y, dx, dw, x, w, dy)
    again = torch.autograd.grad(y, (x, w), dy)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    # the payload as the weight: the same output and the same gradient of x
    z = qcp.int8_linear(x, qcp.int8_quantize(w.detach()))
    assert torch.equal(z, y) and torch.equal(torch.autograd.grad(z, x, dy)[0], dx)
    with torch.no_grad():
        assert torch.equal(qcp.int8_linear(x, w), y) and torch.equal(qcp.int8_linear(x, qcp.int8_quantize(w)), y)


@GPU
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("I", [1, 100, 128, 1000, 4096, 6144, 6145, 12000, 20001, 49152, 49153])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9])
def test_linear_of_few_rows_is_the_quantize_and_the_product(gpu, T, I, dt):
    """Up to 8 rows of a frozen layer take one launch where they fit, with the same bytes; rows of
    zeros, with NaN and of any size among them."""
    x = values(T, I, dt, T * I)
    if T > 3:
        x[3, I // 2] = float("nan")
    for O in (1, 16, 70, 1001):
        w = random_payload(O, I, O)
        with torch.no_grad():
            y = qcp.int8_linear(x, w)
        want = qcp.int8_matmul(*qcp.int8_quantize(x), *w, dtype=DT[dt])
        assert torch.equal(y.view(torch.int16), want.view(torch.int16)), (O, qcp.library().qcp_int8_linear_rows_fit(T, O, I))


@GPU
def test_c_entry_for_few_rows_takes_strides(gpu):
    """Rows of x and y apart; what lies between them is neither read into the sums nor written."""
    big = torch.full((5, 700), float("nan"), device="cuda").to(torch.bfloat16)
    x = values(5, 300, "bf16", 1)
    big[:, 3:303] = x
    w = random_payload(90, 300, 2)
    y = torch.full((5, 100), 7.0, device="cuda", dtype=torch.bfloat16)
    rc = qcp.library().int8_linear_rows(big[:, 3:].data_ptr(), 2, 5, 300, 700, w[0].data_ptr(), w[1].data_ptr(), 90, y.data_ptr(), 100,
                                        torch.cuda.current_stream().cuda_stream)
    want = qcp.int8_matmul(*qcp.int8_quantize(x), *w)
    assert rc == 0 and torch.equal(y[:, :90], want) and (y[:, 90:] == 7).all()


@GPU
def test_linear_gradients_match_differences(gpu):
    """On rows whose largest value is 127 and whose values are integers the payload is the
    matrix itself, so the layer is the plain linear map, and differences of a whole step equal
    its gradients: all sums are integers below 2^24 (70 * 9 * 9 + 2 * 9 * 127 at most), exact in
    fp32, and what the layer returns is those sums rounded once to fp16 (whole numbers above
    2048 do not all fit its 11 bits).  The differences are taken of the product before that
    rounding."""
    g = generator(1)
    T, I, O = 24, 70, 40
    draw = lambda *s: torch.randint(-9, 10, s, generator=g, device="cuda").float()  # noqa: E731
    x, w, dy = draw(T, I), draw(O, I), draw(T, O)
    x[:, 5], w[:, 6] = 127.0, -127.0
    x, w, dy = (t.to(torch.float16) for t in (x, w, dy))
    x.requires_grad_(), w.requires_grad_()

    def loss(a, b):
        product = qcp.int8_matmul(*qcp.int8_quantize(a.detach()), *qcp.int8_quantize(b.detach()), dtype=torch.float32)
        return (product.double() * dy.double()).sum().item()
    y = qcp.int8_linear(x, w)
    assert torch.equal(y, (x.double() @ w.double().t()).to(torch.float16))
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    base = loss(x, w)
    for t, grad, name in ((x, dx, "x"), (w, dw, "w")):
        for r, c in ((0, 1), (3, 7), (23, 69), (16, 33)):
            for step in (1.0, -2.0):
                moved = t.detach().clone()
                moved[r, c] += step
                change = (loss(moved, w) if name == "x" else loss(x, moved)) - base
                assert torch.tensor(change / step).to(torch.float16).item() == grad[r, c].item(), (name, r, c, step)


@GPU
def test_linear_shapes_and_partial_gradients(gpu):
    x = torch.randn(2, 3, 40, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(50, 40, device="cuda", dtype=torch.bfloat16)
    flat = qcp.int8_linear(x.view(6, 40), w)
    assert torch.equal(qcp.int8_linear(x, w), flat.view(2, 3, 50))
    assert torch.equal(qcp.int8_linear(x[0, 0], w), flat[0])
    a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
    qcp.int8_linear(a, b).float().square().sum().backward()
    c = x.clone().requires_grad_()
    qcp.int8_linear(c, w).float().square().sum().backward()
    d = w.clone().requires_grad_()
    qcp.int8_linear(x, d).float().square().sum().backward()
    assert torch.equal(a.grad, c.grad) and torch.equal(b.grad, d.grad)
    e = x.clone().requires_grad_()                 # a broadcast input: its gradient sums over the copies
    qcp.int8_linear(e[:1].expand(5, 3, 40), w).sum().backward()
    assert e.grad[0].abs().sum() > 0 and not e.grad[1:].any()
    f = w.clone().requires_grad_()                 # a transposed weight, and a weight used twice
    torch.stack([qcp.int8_linear(x, f), qcp.int8_linear(x, f)]).float().square().sum().backward()
    assert torch.allclose(f.grad.float(), 2 * b.grad.float(), rtol=2.0 ** -7)
    t = w.t().contiguous().requires_grad_()
    qcp.int8_linear(x, t.t()).float().square().sum().backward()
    assert torch.equal(t.grad.t(), b.grad)


@GPU
def test_linear_keeps_eight_bits_of_its_input(gpu):
    """What waits for the backward pass is one byte and a share of a scale for each value, and
    only what a gradient needs."""
    T, I, O = 64, 256, 128
    x = torch.randn(T, I, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(O, I, device="cuda", dtype=torch.bfloat16)
    frozen = qcp.int8_quantize(w)

    def kept(x, w):
        sizes = []
        with torch.autograd.graph.saved_tensors_hooks(lambda t: (sizes.append(t.numel() * t.element_size()), t)[1], lambda t: t):
            qcp.int8_linear(x, w)
        return sorted(sizes)
    grad = lambda t: t.clone().requires_grad_()  # noqa: E731
    assert kept(grad(x), grad(w)) == sorted([T * (I + 4), O * (I + 4)])
    assert kept(x, grad(w)) == [T * (I + 4)] and kept(grad(x), w) == [O * (I + 4)] and kept(x, w) == []
    assert kept(grad(x), frozen) == sorted([O * I, O * 4]) and kept(x, frozen) == []


@GPU
def test_linear_backward_after_its_inputs_changed(gpu):
    """Of the tensors themselves nothing is kept; a frozen payload that was written to since is refused by autograd."""
    x, w = values(40, 300, "bf16", 1).requires_grad_(), values(60, 300, "bf16", 2).requires_grad_()
    dy = values(40, 60, "bf16", 3)
    want = torch.autograd.grad(qcp.int8_linear(x, w), (x, w), dy)
    y = qcp.int8_linear(x, w)
    with torch.no_grad():
        x.zero_(), w.zero_()
    assert all(map(torch.equal, torch.autograd.grad(y, (x, w), dy), want))
    payload = qcp.int8_quantize(values(60, 300, "bf16", 2))
    y = qcp.int8_linear(x, payload)
    payload[0].zero_()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(y, x, dy)


@GPU
def test_linear_passes_on_what_is_not_finite(gpu):
    """A token with a NaN has a NaN output; its neighbours do not, and the gradient of a
    weight, which sums over the tokens, does."""
    x, w = torch.randn(5, 64, device="cuda").to(torch.bfloat16), torch.randn(7, 64, device="cuda").to(torch.bfloat16).requires_grad_()
    clean = qcp.int8_linear(x, w).detach()
    x[2, 3] = float("inf")
    x.requires_grad_()
    y = qcp.int8_linear(x, w)
    assert torch.isnan(y[2]).all() and torch.equal(y[[0, 1, 3, 4]], clean[[0, 1, 3, 4]])
    dx, dw = torch.autograd.grad(y, (x, w), torch.ones_like(y))
    assert torch.isfinite(dx).all() and torch.isnan(dw).all()


@GPU
def test_training_steps_of_a_small_network(gpu):
    """Two layers, their gradients and AdamW, three steps: each step's products against the
    formula in 64 bits on the very tensors they were given."""
    g = generator(9)
    make = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    T, I, H, O = 130, 200, 390, 70
    master = [make(H, I) / I ** 0.5, make(O, H) / H ** 0.5]
    copies = [p.to(torch.bfloat16) for p in master]
    optimizer = qcp.AdamW([p.view(-1) for p in master], copies=[c.view(-1) for c in copies])
    for step in range(1, 4):
        x, target = make(T, I).to(torch.bfloat16), make(T, O)
        w = [c.detach().requires_grad_() for c in copies]
        a = qcp.int8_linear(x, w[0])
        h = torch.nn.functional.gelu(a.float()).to(torch.bfloat16)
        y = qcp.int8_linear(h, w[1])
        loss = (y.float() - target).square().mean()
        grads = torch.autograd.grad(loss, (w[0], w[1], a, h, y), retain_graph=True)
        check_layer(a, None, grads[0], x, w[0], grads[2])
        check_layer(y, grads[3], grads[1], h, w[1], grads[4])
        qcp.adamw_step(optimizer, [t.reshape(-1) for t in grads[:2]], step, 3e-3)
        assert all(torch.isfinite(p).all() for p in master)
        assert all(torch.equal(c, p.to(torch.bfloat16)) for c, p in zip(copies, master))


@GPU
def test_linear_captured_in_a_graph(gpu):
    """Forward and backward of a step, captured: replays on new inputs equal the eager step."""
    x, w = values(90, 300, "bf16", 1).requires_grad_(), values(140, 300, "bf16", 2).requires_grad_()
    dy = values(90, 140, "bf16", 3)

    def step():
        y = qcp.int8_linear(x, w)
        return (y.detach(), *torch.autograd.grad(y, (x, w), dy))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(4):
        with torch.no_grad():
            x.copy_(values(90, 300, "bf16", 10 + k))
            dy.copy_(values(90, 140, "bf16", 20 + k))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step())), k


@GPU
def test_linear_refuses_a_captured_backward_beside_a_living_graph_on_the_gpu(gpu):
    """The refusal leaves the capture and the leaves usable: without the living graph the same
    capture replays the eager step's gradients."""
    x, w = values(90, 300, "bf16", 1).requires_grad_(), values(140, 300, "bf16", 2).requires_grad_()
    dy = values(90, 140, "bf16", 3)
    alive = qcp.int8_linear(x, w)
    want = torch.autograd.grad(alive, (x, w), dy)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="default stream, lives"):
        with torch.cuda.graph(graph):
            torch.autograd.grad(qcp.int8_linear(x, w), (x, w), dy)
    del alive, graph
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(qcp.int8_linear(x, w), (x, w), dy)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ refusals (CPU)

OK, EINVAL, EALIGN, EUNSUP = 0, -1, -2, -3
A = 0x7f0000000000
S = 1 << 32


@pytest.fixture()
def lib():
    if not os.path.exists(qcp.LIB_PATH):
        pytest.fail(f"{qcp.LIB_PATH} not built")
    return qcp.library()


def test_c_entries_refuse(lib):
    def quant(x=A, xt=2, rows=64, cols=256, ld=256, c=A + S, s=A + 2 * S):
        return lib.int8_quantize(x, xt, rows, cols, ld, c, s, None)

    def dequant(c=A, s=A + S, rows=64, cols=256, y=A + 2 * S, yt=2, ld=256):
        return lib.int8_dequantize(c, s, rows, cols, y, yt, ld, None)
    assert quant(rows=0) == OK and dequant(rows=0) == OK and dequant(cols=0, ld=0) == OK
    for f in (quant, dequant):
        for bad in (dict(rows=-1), dict(cols=-1), dict(ld=255), dict(c=0), dict(s=0), dict(rows=1 << 40),
                    dict(rows=1 << 29, cols=256), dict(rows=1, cols=(1 << 31) + 1, ld=1 << 32), dict(ld=1 << 40), dict(ld=1 << 62)):
            assert f(**bad) == EINVAL, (f, bad)
        for bad in (dict(c=A + S + 8), dict(s=A + 2 * S + 4)):
            assert f(**bad) == EALIGN, (f, bad)
    for bad in (dict(xt=0), dict(xt=4), dict(x=0), dict(c=A + 1024), dict(s=A + 1024), dict(s=A + S + 512), dict(cols=0, ld=0, s=0)):
        assert quant(**bad) == EINVAL, bad
    assert quant(x=A + 1) == EALIGN and quant(x=A + 2, xt=3) == EALIGN
    for bad in (dict(yt=0), dict(y=0), dict(y=A + 64), dict(y=A + S)):
        assert dequant(**bad) == EINVAL, bad
    assert dequant(y=A + 2 * S + 1) == EALIGN and dequant(y=A + 2 * S + 2, yt=3) == EALIGN


def test_c_entry_of_the_product_refuses(lib):
    work = lib.qcp_int8_matmul_work
    need = work(64, 64, 9000)
    assert need > 0 and need % (4 * 64 * 64) == 0 and work(8, 512, 28672) == 0 and work(64, 64, 200) == 0
    assert work(0, 64, 28672) == work(64, 64, 0) == 0
    assert work(-1, 64, 8192) == work(64, 1 << 40, 8192) == work(64, 64, 130945) == -1

    def mul(a=A, sa=A + S, b=A + 2 * S, sb=A + 3 * S, M=64, N=64, K=9000, c=A + 4 * S, ct=2, ldc=64, w=A + 5 * S, n=need):
        return lib.int8_matmul(a, sa, b, sb, M, N, K, c, ct, ldc, w, n, None)
    assert mul(M=0) == OK and mul(N=0, ldc=0) == OK and mul(M=0, w=None, n=0) == OK
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(K=130945), dict(ldc=63), dict(ct=0), dict(a=0), dict(sa=0), dict(b=0),
                dict(sb=0), dict(c=0), dict(M=1 << 30), dict(c=A), dict(c=A + 2 * S + 64), dict(c=A + 3 * S), dict(sb=0, K=0),
                dict(M=1 << 22, N=1 << 22, K=128, ldc=1 << 22), dict(n=need - 1), dict(n=-1), dict(w=A), dict(w=A + 4 * S),
                dict(w=A + 3 * S + 16)):
        assert mul(**bad) == EINVAL, bad
    for bad in (dict(a=A + 8), dict(sa=A + S + 4), dict(sb=A + 3 * S + 4), dict(c=A + 4 * S + 1), dict(c=A + 4 * S + 2, ct=3),
                dict(w=A + 5 * S + 4)):
        assert mul(**bad) == EALIGN, bad


def test_c_entry_for_few_rows_refuses(lib):
    fit = lib.qcp_int8_linear_rows_fit
    assert fit(1, 14336, 4096) == fit(1, 28672, 8192) == fit(8, 4096, 4096) == fit(8, 1000, 6144) == fit(1, 1, 49152) == 1
    assert fit(8, 14336, 4096) == fit(4, 14336, 4096) == 0                  # as quick in two launches
    assert fit(9, 64, 64) == fit(8, 1000, 6145) == fit(1, 1, 49153) == fit(0, 4, 4) == fit(4, 0, 4) == fit(4, 4, 0) == fit(1, 4, 1 << 40) == 0

    def call(x=A, xt=2, M=4, K=256, ldx=256, w=A + S, s=A + 2 * S, N=64, y=A + 3 * S, ldy=64):
        return lib.int8_linear_rows(x, xt, M, K, ldx, w, s, N, y, ldy, None)
    assert call(M=0) == OK and call(N=0, ldy=0) == OK
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(xt=3), dict(xt=0), dict(ldx=255), dict(ldy=63), dict(x=0), dict(w=0), dict(s=0),
                dict(y=0), dict(y=A), dict(y=A + S), dict(y=A + 2 * S), dict(K=130945, ldx=130945), dict(N=1 << 30, ldy=1 << 30)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(M=9), dict(K=0, ldx=0), dict(K=50000, ldx=50000), dict(M=8, N=14336, ldy=14336, K=4096, ldx=4096)):
        assert call(**bad) == EUNSUP, bad
    for bad in (dict(x=A + 1), dict(y=A + 3 * S + 1), dict(w=A + S + 8), dict(s=A + 2 * S + 4)):
        assert call(**bad) == EALIGN, bad


def test_rows_below_the_bound_have_no_slices(lib):
    """The binding asks for scratch memory only above this length."""
    from quantized_collective_payloads_amd.int8 import _UNSLICED
    work = lib.qcp_int8_matmul_work
    shapes = [(M, N) for M in (17, 32, 33, 64, 128, 200, 500, 2048, 8192) for N in (1, 16, 64, 500, 700, 2048, 4096, 8192)]
    assert not any(work(M, N, K) for M, N in shapes for K in (128, 1000, 4096, _UNSLICED - 127, _UNSLICED))
    assert work(64, 64, _UNSLICED + 1) > 0


def test_c_entry_of_the_mixed_product_refuses(lib):
    work = lib.qcp_int8_mixed_work
    need = work(64, 64, 9000, 0, 1)
    assert need > 0 and need % (4 * 64 * 64) == 0
    assert work(4096, 4096, 28672, 0, 1) == work(64, 64, 200, 0, 1) == work(0, 64, 9000, 0, 1) == work(64, 64, 0, 1, 1) == 0
    assert work(-1, 64, 8192, 0, 1) == work(64, 1 << 40, 8192, 0, 1) == work(64, 64, 64, 2, 1) == work(64, 64, 64, 0, 2) == -1
    copied = work(4096, 4096, 4100, 0, 0)                                # a's rows to 16 bytes: 4104 elements each
    assert copied == 4096 * 4104 * 2 and work(4096, 4096, 4100, 0, 1) == copied and work(4096, 4096, 4096, 0, 1) == 0
    assert work(1 << 36, 64, 1 << 36, 0, 0) >= -1 and work(1 << 36, 64, 1 << 36, 1, 0) >= -1
    assert work(50257, 4096, 8192, 1, 0) == 0                            # more than 256 MB is not copied

    def mul(a=A, at=2, lda=9000, t=0, x=A + S, s=A + 2 * S, M=64, N=64, K=9000, c=A + 3 * S, ct=2, ldc=64, w=A + 4 * S, n=need):
        return lib.int8_matmul_mixed(a, at, lda, t, x, s, M, N, K, c, ct, ldc, w, n, None)
    assert mul(M=0) == OK and mul(N=0, ldc=0) == OK and mul(M=0, w=None, n=0) == OK
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(t=2), dict(t=-1), dict(at=3), dict(at=0), dict(ct=0), dict(lda=8999),
                dict(t=1, lda=63), dict(ldc=63), dict(a=0), dict(x=0), dict(s=0), dict(c=0), dict(c=A), dict(c=A + S), dict(c=A + 2 * S),
                dict(N=(1 << 24) + 1, ldc=1 << 25), dict(lda=(1 << 23) + 1), dict(K=1 << 30), dict(n=need - 1), dict(w=A), dict(w=A + S),
                dict(w=A + 3 * S), dict(M=1 << 30, N=1 << 20, K=1, lda=1, ldc=1 << 20)):
        assert mul(**bad) == EINVAL, bad
    assert mul(ct=1) == EUNSUP and mul(at=1, ct=2) == EUNSUP
    for bad in (dict(a=A + 1), dict(x=A + S + 8), dict(s=A + 2 * S + 4), dict(c=A + 3 * S + 1), dict(c=A + 3 * S + 2, ct=3),
                dict(w=A + 4 * S + 4)):
        assert mul(**bad) == EALIGN, bad


def test_binding_refuses(lib):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    one = torch.ones

    def raises(match, fn, *a, **kw):
        with pytest.raises(ValueError, match=match):
            fn(*a, **kw)
    raises("x: 1 dimensions", qcp.int8_quantize, torch.zeros(64))
    raises("x: dtype", qcp.int8_quantize, torch.zeros(4, 64, dtype=torch.float64))
    raises("x: expected", qcp.int8_quantize, None)
    raises("codes: shape", qcp.int8_quantize, torch.zeros(4, 64), codes=u8(4, 64))
    raises("codes: dtype", qcp.int8_quantize, torch.zeros(4, 64), codes=torch.zeros(4, 128, dtype=torch.int8))
    raises("scales: shape", qcp.int8_quantize, torch.zeros(4, 64), scales=one(5))
    raises("scales: dtype", qcp.int8_quantize, torch.zeros(4, 64), scales=u8(4))
    raises("GPU tensors only", qcp.int8_quantize, torch.zeros(4, 64))
    raises("codes: rows of 100 bytes", qcp.int8_dequantize, u8(4, 100), one(4), 100)
    raises("codes: 1 dimensions", qcp.int8_dequantize, u8(128), one(1), 100)
    raises("scales: shape", qcp.int8_dequantize, u8(4, 128), one(4, 1), 100)
    raises("scales: dtype", qcp.int8_dequantize, u8(4, 128), one(4).double(), 100)
    raises("codes: rows of 128 values for 129", qcp.int8_dequantize, u8(4, 128), one(4), 129)
    raises("codes: rows of 128 values for -1", qcp.int8_dequantize, u8(4, 128), one(4), -1)
    raises("out: shape", qcp.int8_dequantize, u8(4, 128), one(4), 100, out=torch.zeros(4, 99))
    raises("unsupported dtype", qcp.int8_dequantize, u8(4, 128), one(4), 100, torch.float64)
    raises("must be contiguous", qcp.int8_dequantize, u8(4, 256)[:, :128], one(4), 100)
    raises("must be contiguous", qcp.int8_dequantize, u8(4, 128), one(8)[::2], 100)
    raises("GPU tensors only", qcp.int8_dequantize, u8(4, 128), one(4), 100)
    raises("b_codes: rows of 256", qcp.int8_matmul, u8(4, 128), one(4), u8(4, 256), one(4))
    raises("a_scales: shape", qcp.int8_matmul, u8(4, 128), one(3), u8(4, 128), one(4))
    raises("out: shape", qcp.int8_matmul, u8(4, 128), one(4), u8(5, 128), one(5), out=torch.zeros(5, 4))
    raises("GPU tensors only", qcp.int8_matmul, u8(4, 128), one(4), u8(5, 128), one(5))
    half = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    raises("a: dtype", qcp.int8_matmul_mixed, torch.zeros(3, 4), u8(4, 128), one(4), 100)
    raises("a: 1 dimensions", qcp.int8_matmul_mixed, half(4), u8(4, 128), one(4), 100)
    raises("payload of 4 rows", qcp.int8_matmul_mixed, half(4, 3), u8(4, 128), one(4), 100)
    raises("payload of 4 rows", qcp.int8_matmul_mixed, half(3, 4), u8(4, 128), one(4), 100, transpose=True)
    raises("for 200 columns", qcp.int8_matmul_mixed, half(3, 4), u8(4, 128), one(4), 200)
    raises("dtype torch.float16", qcp.int8_matmul_mixed, half(3, 4), u8(4, 128), one(4), 100, dtype=torch.float16)
    raises("out: shape", qcp.int8_matmul_mixed, half(3, 4), u8(4, 128), one(4), 100, out=half(3, 99))
    raises("GPU tensors only", qcp.int8_matmul_mixed, half(3, 4), u8(4, 128), one(4), 100)
    raises("last dimension 63", qcp.int8_linear, half(4, 63), half(8, 64))
    raises("last dimension 129", qcp.int8_linear, half(4, 129), (u8(8, 128), one(8)))
    raises("weight: 1 dimensions", qcp.int8_linear, half(4, 63), half(8))
    raises("weight scales: shape", qcp.int8_linear, half(4, 63), (u8(8, 128), one(7)))
    raises("weight: expected a tensor or a payload", qcp.int8_linear, half(4, 63), (u8(8, 128),))
    raises("x: dtype", qcp.int8_linear, torch.zeros(4, 64), half(8, 64))
    raises("x: expected", qcp.int8_linear, None, half(8, 64))
    raises("GPU tensors only", qcp.int8_linear, half(4, 64), half(8, 64))


@pytest.fixture()
def layer_on_cpu(monkeypatch):
    """The layer on CPU tensors, its launches replaced: quantizing does nothing and products are zero."""
    from quantized_collective_payloads_amd import int8
    monkeypatch.setattr(int8, "_same_gpu", lambda index, *ts: None)
    monkeypatch.setattr(int8, "_quantized", lambda index, x: x.new_empty(x.shape[0] * (R.padded(x.shape[1]) + 4), dtype=torch.uint8))
    monkeypatch.setattr(int8, "_multiply", lambda index, a, sa, b, sb, M, N, K, c: c.zero_())
    monkeypatch.setattr(int8, "_frozen_product", lambda index, x, codes, scales: x.new_zeros((x.shape[0], codes.shape[0])))
    monkeypatch.setattr(int8, "_mixed", lambda index, a, codes, scales, M, N, K, transpose, c: c.zero_())


@pytest.mark.parametrize("which", ["x", "weight", "both"])
@pytest.mark.parametrize("grad", [True, False])
def test_linear_refuses_forward_mode_tangents(layer_on_cpu, grad, which):
    from torch.autograd import forward_ad
    x, w = torch.ones(3, 32, dtype=torch.bfloat16), torch.ones(4, 32, dtype=torch.bfloat16)
    payload = torch.zeros(4, 128, dtype=torch.uint8), torch.ones(4)
    with torch.set_grad_enabled(grad), forward_ad.dual_level():
        a = forward_ad.make_dual(x, x) if which != "weight" else x
        b = forward_ad.make_dual(w, w) if which != "x" else w
        for v in (a, a.view(3, 1, 32), a.t().contiguous().t()):
            with pytest.raises(NotImplementedError):
                qcp.int8_linear(v, b)
            if which != "weight":
                with pytest.raises(NotImplementedError):
                    qcp.int8_linear(v, payload)
        assert qcp.int8_linear(x, w).shape == (3, 4)
    assert qcp.int8_linear(x, payload).shape == (3, 4)


@pytest.mark.parametrize("kind", ["tensor", "cast", "frozen"])
@pytest.mark.parametrize("stream,refused", [(0, True), (7, False)])
def test_linear_refuses_a_captured_backward_beside_a_living_graph(layer_on_cpu, monkeypatch, kind, stream, refused):
    from quantized_collective_payloads_amd import int8
    streams = {"now": stream}
    monkeypatch.setattr(int8, "_raw_stream", lambda index: streams["now"])
    monkeypatch.setattr(int8, "_captured", lambda index: streams["now"] == 9)
    w = torch.ones(4, 32, requires_grad=True)
    payload = torch.zeros(4, 128, dtype=torch.uint8), torch.ones(4)

    def layer(x, on):
        streams["now"] = on
        return qcp.int8_linear(x, payload if kind == "frozen" else w.to(torch.bfloat16) if kind == "cast" else w)
    for shape in ((6, 32), (2, 3, 32)):
        for grad in (True, False) if kind != "frozen" else (True,):
            x = torch.ones(shape, dtype=torch.bfloat16, requires_grad=grad)
            alive = layer(x, stream)
            y = layer(x, 9)
            if refused:
                with pytest.raises(RuntimeError, match="default stream, lives"):
                    y.sum().backward()
            else:
                y.sum().backward()
            del alive, y
            layer(x, 9).sum().backward()


EMPTY = [(2, 3, 0), (0,), (3, 0), (0, 3, 0), (0, 0), (2, 0, 64), (0, 64), (64,), (2, 1, 3, 64)]


def like_torch(shape, device):
    """y and the gradients have the shapes of torch's own layer, and its zeros where there is nothing to sum."""
    x, w = (torch.ones(s, device=device, dtype=torch.bfloat16, requires_grad=True) for s in (shape, (5, shape[-1])))
    y = qcp.int8_linear(x, w)
    want = torch.nn.functional.linear(x, w)
    assert y.shape == want.shape
    with torch.no_grad():
        assert qcp.int8_linear(x, w).shape == want.shape
    dx, dw = torch.autograd.grad(y.sum(), (x, w))
    assert dx.shape == x.shape and dw.shape == w.shape
    return y, dx, dw, x.numel() == 0


@pytest.mark.parametrize("shape", EMPTY)
def test_linear_shapes_without_elements(layer_on_cpu, shape):
    like_torch(shape, "cpu")


@GPU
@pytest.mark.parametrize("shape", EMPTY)
def test_linear_of_nothing_is_zero(gpu, shape):
    y, dx, dw, nothing = like_torch(shape, "cuda")
    torch.cuda.synchronize()
    if nothing:
        assert not y.any() and not dx.any() and not dw.any()
    else:                                          # y = 127 * 127 * (1 / 127)^2 * I, a rounding of 1/127 off twice
        assert torch.allclose(y.float(), torch.tensor(float(shape[-1]), device="cuda"), rtol=2.0 ** -7)
        assert torch.allclose(dx.float(), torch.tensor(5.0, device="cuda"), rtol=2.0 ** -7)
        assert torch.allclose(dw.float(), torch.tensor(y.numel() / 5, device="cuda"), rtol=2.0 ** -7)
