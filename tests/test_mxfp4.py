"""The MXFP4 payload byte for byte against its definition, the product and the
linear layer against float64, and the refusals."""
import os

import numpy as np
import pytest
import torch

import quantized_collective_payloads_amd as qcp
from tests import operator_reference as R

GPU = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture()
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    qcp.library()


def wide(t):
    return t.detach().to(torch.float64).cpu().numpy()


def values(rows, cols, dt, seed):
    """Normal values over many binades, with zero blocks, signed zeros, exact ties
    and single outliers."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    k = torch.randint(-14 if dt == "f16" else -40, 9, (rows, -(-cols // 32)), generator=g, device="cuda")
    x = x * torch.exp2(k.float()).repeat_interleave(32, 1)[:, :cols]
    x[torch.rand(rows, cols, generator=g, device="cuda") < 0.01] *= 30
    ties = torch.rand(rows, cols, generator=g, device="cuda") < 0.2
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 4.0, -0.0, 0.0], device="cuda")
    pick = grid[torch.randint(0, 11, (rows, cols), generator=g, device="cuda")]
    x = torch.where(ties, pick * torch.exp2(k.float()).repeat_interleave(32, 1)[:, :cols], x)
    if rows > 2:
        x[1] = 0
        x[2, :32] = -0.0
    return x.to(DT[dt])


def check_payload(x, transpose, what):
    codes, scales = qcp.mxfp4_quantize(x, transpose=transpose)
    ref = wide(x).T if transpose else wide(x)
    wc, ws, ok = R.mx_payload(np.ascontiguousarray(ref))
    gc, gs = codes.cpu().numpy(), scales.cpu().numpy()
    assert gs.shape == ws.shape and np.array_equal(gs, ws), (what, np.argwhere(gs != ws)[:4])
    live = np.repeat(ok, 16, axis=1)                       # codes of a NaN block are unspecified
    bad = np.argwhere((gc != wc) & live)
    assert gc.shape == wc.shape and bad.size == 0, (what, bad[:4])
    return codes, scales


SHAPES = [(1, 1), (1, 31), (3, 32), (2, 33), (5, 127), (4, 128), (37, 1003), (128, 64), (129, 65), (255, 130),
          (256, 128), (257, 384), (1, 5000), (5000, 1), (300, 2048)]


@GPU
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_and_back(gpu, rows, cols, dt, transpose):
    x = values(rows, cols, dt, rows * 7 + cols)
    codes, scales = check_payload(x, transpose, (rows, cols, dt, transpose))
    n = rows if transpose else cols
    stands = R.mx_values(codes.cpu().numpy(), scales.cpu().numpy())
    assert not stands[:, n:].any()
    for yt in DT:
        y = qcp.mxfp4_dequantize(codes, scales, n, DT[yt])
        want = torch.from_numpy(stands[:, :n]).to(DT[yt])           # one rounding
        assert torch.equal(y.cpu(), want), (rows, cols, dt, yt)


@GPU
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES + [(513, 449), (1024, 192)])
def test_both_payloads_in_one_pass(gpu, rows, cols, dt):
    x = values(rows, cols, dt, rows + 3 * cols)
    wide_rows = values(rows + 1, cols + 7, dt, 5)[1:, 3:3 + cols]        # rows apart, unaligned
    for v in (x, x.t(), wide_rows, wide_rows.t(), x[:1].expand(5, cols), x[:, ::2]):
        for got, want in zip(qcp.mxfp4_quantize_both(v), (qcp.mxfp4_quantize(v), qcp.mxfp4_quantize(v, transpose=True))):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (tuple(v.shape), v.stride())


@GPU
@pytest.mark.parametrize("rows,cols,dt", [(16390, 8211, "bf16"), (16391, 8210, "f16"), (8201, 8291, "f32")])
def test_matrices_beyond_the_last_cache(gpu, rows, cols, dt):
    """Above 256 MB the column-wise pass streams: the same bytes as of the parts."""
    x = values(rows, cols, dt, 7)
    assert x.numel() * x.element_size() > 256 << 20
    straight, across = qcp.mxfp4_quantize_both(x)
    for a, b in zip(straight, qcp.mxfp4_quantize(x)):
        assert torch.equal(a, b)
    alone = qcp.mxfp4_quantize(x, transpose=True)
    for c in range(0, cols, 2100):
        for a, b, part in zip(across, alone, qcp.mxfp4_quantize(x[:, c:c + 2100], transpose=True)):
            assert torch.equal(a[c:c + 2100], part) and torch.equal(b[c:c + 2100], part)


@GPU
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_every_16_bit_value(gpu, dt):
    """All 65,536 patterns, each the largest of its block and each beside a larger
    one; infinities and NaN make their block NaN."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(DT[dt]).cuda()
    alone = torch.zeros(65536, 32, dtype=DT[dt], device="cuda")
    alone[:, 5] = bits
    alone[:, 9] = bits / 3
    check_payload(alone, False, "alone")
    check_payload(alone.t().contiguous(), True, "alone, transposed")
    for top in (6.0, 1.0, 448.0, 2.0 ** -13):
        beside = torch.full((2048, 64), top, dtype=DT[dt], device="cuda")
        beside[:, 1:33] = bits.view(2048, 32)
        codes, scales = check_payload(beside, False, ("beside", top))
        y = wide(qcp.mxfp4_dequantize(codes, scales, 64, torch.float32))
        nan = ~np.isfinite(wide(beside)).reshape(2048, 2, 32).all(2)
        assert np.array_equal(np.isnan(y).reshape(2048, 2, 32).all(2), nan)
        assert not np.isnan(y.reshape(2048, 2, 32)[~nan]).any()


@GPU
def test_fp32_extremes(gpu):
    x = torch.tensor([0.0, -0.0, 1e-45, -1e-45, 2.0 ** -149, 2.0 ** -130, 2.0 ** -127, 2.0 ** -126, 3e38, -3.4028e38,
                      float("inf"), float("-inf"), float("nan"), 1.0, 6.0, 6.0001, 7.999, 8.0], device="cuda")
    a = torch.zeros(18, 64, device="cuda")
    a[:, 0], a[:, 33], a[:, 34] = x, x, x / 5
    check_payload(a, False, "extremes")
    check_payload(a.t().contiguous(), True, "extremes, transposed")


@GPU
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_strides(gpu, dt):
    """Row strides, unaligned starts, transposed views, overlapping and reversed
    inputs: all as their contiguous copy."""
    base = values(70, 301, dt, 3).reshape(-1)
    views = [base[1:1 + 60 * 301].view(60, 301)[:, 3:200], base[:70 * 301].view(70, 301).t(),
             base[5:5 + 20 * 600].view(20, 600)[:, ::2], base[:256].expand(9, 256), base[3:4 * 129 + 3].view(4, 129)[:, :128],
             base[:70 * 301].view(70, 301)[::3, 1:], base[:300].view(300, 1), base[:300].view(1, 300).t()]
    for i, v in enumerate(views):
        for transpose in (False, True):
            got = qcp.mxfp4_quantize(v, transpose=transpose)
            want = qcp.mxfp4_quantize(v.contiguous(), transpose=transpose)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (i, transpose)
            check_payload(v.contiguous(), transpose, (i, transpose))


@GPU
def test_nothing_outside_the_payload_is_written(gpu):
    for rows, cols, transpose in ((37, 1003, False), (37, 1003, True), (300, 65, True), (129, 127, False)):
        x = values(rows, cols, "bf16", 1)
        lines, n = (cols, rows) if transpose else (rows, cols)
        P = qcp.mxfp4_padded(n)
        code = torch.full((lines * P // 2 + 4096,), 0xAA, dtype=torch.uint8, device="cuda")
        mark = torch.full((lines * P // 32 + 4096,), 0xAA, dtype=torch.uint8, device="cuda")
        c, m = code[:lines * P // 2].view(lines, -1), mark[:lines * P // 32].view(lines, -1)
        qcp.mxfp4_quantize(x, transpose=transpose, codes=c, scales=m)
        assert (code[lines * P // 2:] == 0xAA).all() and (mark[lines * P // 32:] == 0xAA).all()
        out = torch.full((lines * n + 512,), 7.0, device="cuda")
        qcp.mxfp4_dequantize(c, m, n, out=out[:lines * n].view(lines, n))
        assert (out[lines * n:] == 7.0).all()


@GPU
def test_empty(gpu):
    for shape in ((0, 5), (5, 0), (0, 0)):
        for (c, s), n in zip(qcp.mxfp4_quantize_both(torch.zeros(shape, device="cuda")), (shape[1], shape[0])):
            assert c.shape[1] == qcp.mxfp4_padded(n) // 2
        for transpose in (False, True):
            c, s = qcp.mxfp4_quantize(torch.zeros(shape, device="cuda"), transpose=transpose)
            lines, n = shape[::-1] if transpose else shape
            assert c.shape == (lines, qcp.mxfp4_padded(n) // 2)
            assert qcp.mxfp4_dequantize(c, s, n).shape == (lines, n)
    a, b = qcp.mxfp4_quantize(torch.zeros(3, 0, device="cuda")), qcp.mxfp4_quantize(torch.zeros(70, 0, device="cuda"))
    assert torch.equal(qcp.mxfp4_matmul(*a, *b), torch.zeros(3, 70, dtype=torch.bfloat16, device="cuda"))
    z = qcp.mxfp4_quantize(torch.zeros(0, 64, device="cuda"))
    one = qcp.mxfp4_quantize(torch.ones(5, 64, device="cuda"))
    assert qcp.mxfp4_matmul(*z, *one).shape == (0, 5) and qcp.mxfp4_matmul(*one, *z).shape == (5, 0)


# ------------------------------------------------------------------ product

def random_payload(lines, n, seed, lo=115, hi=130):
    """Random codes and scales, zero past column n: every payload is valid input."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    P = qcp.mxfp4_padded(n)
    c = torch.randint(0, 256, (lines, P // 2), generator=g, dtype=torch.uint8, device="cuda")
    s = torch.randint(lo, hi, (lines, P // 32), generator=g, dtype=torch.uint8, device="cuda")
    c[:, (n + 1) // 2:] = 0
    if n % 2:
        c[:, n // 2] &= 15
    return c, s


def check_product(a, b, out, dt, what):
    """fp32 accumulation in any order: K roundings of at most the sum of
    magnitudes; then one rounding to the output's type."""
    av, bv = (torch.from_numpy(R.mx_values(c.cpu().numpy(), s.cpu().numpy())).cuda() for c, s in (a, b))
    want, size = av @ bv.T, av.abs() @ bv.abs().T
    bound = av.shape[1] * 2.0 ** -24 * size + (0 if dt == "f32" else UNIT[dt]) * want.abs()
    if dt == "f16":
        bound = bound + 2.0 ** -25                       # subnormal results
    err = (out.to(torch.float64) - want).abs()
    bad = (~(err <= bound)).nonzero()
    assert bad.numel() == 0, (what, bad[:4].tolist())


MATMULS = [(1, 1, 1), (1, 16, 32), (1, 257, 4096), (2, 100, 33), (5, 1000, 1111), (16, 64, 640), (17, 129, 255),
           (31, 31, 129), (32, 4096, 512), (33, 300, 2049), (64, 64, 64), (65, 63, 127), (77, 1001, 1111),
           (96, 2048, 384), (128, 128, 128), (129, 257, 385), (200, 520, 8192), (255, 511, 1000), (256, 256, 256),
           (257, 1000, 260), (300, 5, 300), (512, 768, 1280), (1000, 1, 100), (1030, 1290, 600)]


@GPU
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", MATMULS)
def test_product(gpu, M, N, K, dt):
    lo, hi = (115, 124) if dt == "f16" else (115, 130)
    a, b = random_payload(M, K, M + K, lo, hi), random_payload(N, K, N * 3 + K, lo, hi)
    # guard: what lies around the result stays
    buf = torch.full((M * N + 1024,), 3.0, dtype=DT[dt], device="cuda")
    out = buf[512:512 + M * N].view(M, N)
    qcp.mxfp4_matmul(*a, *b, out=out)
    assert (buf[:512] == 3).all() and (buf[512 + M * N:] == 3).all()
    check_product(a, b, out, dt, (M, N, K, dt))
    again = qcp.mxfp4_matmul(*a, *b, dtype=DT[dt])
    assert torch.equal(again, out)                       # the same bytes on every run


# several rounds of tiles with ragged edges: 256 x 256 and 128 x 128 work-groups that walk
# more than one tile, with an odd number of granules and with few of them
@GPU
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(4100, 4130, 4200), (3000, 3010, 1111), (700, 3000, 520), (65, 8200, 900), (5121, 2050, 640)])
def test_product_over_several_rounds_of_tiles(gpu, M, N, K, dt):
    a, b = random_payload(M, K, 1), random_payload(N, K, 2)
    buf = torch.full((M * N + 1024,), 3.0, dtype=DT[dt], device="cuda")
    out = buf[512:512 + M * N].view(M, N)
    for _ in range(2):
        out.fill_(5.0)
        qcp.mxfp4_matmul(*a, *b, out=out)
        assert (buf[:512] == 3).all() and (buf[512 + M * N:] == 3).all()
        check_product(a, b, out, dt, (M, N, K, dt))


@GPU
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(700, 900, 1), (1100, 1000, 128), (1025, 1290, 200), (129, 4097, 256), (2049, 700, 384), (1300, 1301, 300)])
def test_product_over_a_short_k(gpu, M, N, K, dt):
    a, b = random_payload(M, K, M, 110, 126), random_payload(N, K, N, 110, 126)
    a[1][M // 2, 0] = 255
    out = qcp.mxfp4_matmul(*a, *b, dtype=DT[dt])
    assert out[M // 2].isnan().all()
    keep = [i for i in range(M) if i != M // 2]
    check_product((a[0][keep], a[1][keep]), b, out[keep], dt, (M, N, K))


@GPU
def test_product_over_a_very_long_k(gpu):
    """K = 2^25, zeros but for the last 128: as the product of these."""
    K, M, N = 1 << 25, 40, 33
    parts, wide_ones = [], []
    for lines, seed in ((M, 5), (N, 6)):
        tail = random_payload(lines, 128, seed, 120, 125)
        codes = torch.zeros(lines, K // 2, dtype=torch.uint8, device="cuda")
        scales = torch.full((lines, K // 32), 127, dtype=torch.uint8, device="cuda")
        codes[:, -64:], scales[:, -4:] = tail
        parts.append(tail)
        wide_ones += [codes, scales]
    check_product(*parts, qcp.mxfp4_matmul(*wide_ones, dtype=torch.float32), "f32", K)


SLICED = [(33, 100, 12288), (100, 200, 20000), (64, 512, 28672), (17, 50, 16400), (500, 700, 10000), (128, 4096, 8200),
          (40, 33, 12161), (129, 257, 13001), (1000, 31, 12345)]


@GPU
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SLICED)
def test_product_in_slices_of_k(gpu, M, N, K, dt):
    assert 0 < qcp.library().qcp_mxfp4_matmul_work(M, N, K) <= 4 << 20
    a, b = random_payload(M, K, M, 110, 124), random_payload(N, K, N, 110, 124)
    out = qcp.mxfp4_matmul(*a, *b, dtype=DT[dt])
    check_product(a, b, out, dt, (M, N, K))
    assert torch.equal(out, qcp.mxfp4_matmul(*a, *b, dtype=DT[dt]))
    a[1][M // 2, -1] = 255                               # in the last slice, of one row
    bad = qcp.mxfp4_matmul(*a, *b, dtype=DT[dt])
    assert bad[M // 2].isnan().all() and torch.equal(bad[:M // 2], out[:M // 2])
    # without scratch memory: one sum, within the same bound
    a[1][M // 2, -1] = 120
    whole = torch.empty(M, N, dtype=DT[dt], device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert qcp.library().mxfp4_matmul(a[0].data_ptr(), a[1].data_ptr(), b[0].data_ptr(), b[1].data_ptr(), M, N, K,
                                      whole.data_ptr(), qcp.DTYPES[DT[dt]], N, stream) == 0
    check_product(a, b, whole, dt, (M, N, K))


@GPU
def test_slices_stay_in_their_scratch_memory_and_rows(gpu):
    M, N, K, ldc = 70, 130, 13000, 137
    a, b = random_payload(M, K, 1, 110, 124), random_payload(N, K, 2, 110, 124)
    need = qcp.library().qcp_mxfp4_matmul_work(M, N, K)
    work = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    c = torch.full((M, ldc), 7.0, device="cuda")
    assert qcp.library().mxfp4_matmul_sliced(
        a[0].data_ptr(), a[1].data_ptr(), b[0].data_ptr(), b[1].data_ptr(), M, N, K, c.data_ptr(), qcp.DTYPES[c.dtype],
        ldc, work.data_ptr(), need, torch.cuda.current_stream().cuda_stream) == 0
    check_product(a, b, c[:, :N], "f32", "rows apart")
    assert (c[:, N:] == 7).all() and (work[need:] == 0x5a).all()


@GPU
def test_slices_in_a_graph(gpu):
    M, N, K = 48, 96, 12288
    a, b = random_payload(M, K, 1, 110, 124), random_payload(N, K, 2, 110, 124)
    out = torch.empty(M, N, device="cuda")
    qcp.mxfp4_matmul(*a, *b, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qcp.mxfp4_matmul(*a, *b, out=out)
    for seed in (3, 4, 5):
        for t, new in zip(a, random_payload(M, K, seed, 110, 124)):
            t.copy_(new)
        graph.replay()
        assert torch.equal(out, qcp.mxfp4_matmul(*a, *b, dtype=torch.float32))


@GPU
def test_product_of_integers_is_exact(gpu):
    """Codes at scale 1: every partial sum is a multiple of 1/4 below 2^22, so any
    order of fp32 sums is exact -- each element and each k lands where it should."""
    for M, N, K in ((3, 50, 700), (40, 40, 1000), (130, 260, 2000), (300, 300, 4096), (520, 1100, 300), (4100, 4100, 2050)):
        a, b = random_payload(M, K, 1, 127, 128), random_payload(N, K, 2, 127, 128)
        want = torch.from_numpy(R.mx_values(*(t.cpu().numpy() for t in a)) @ R.mx_values(*(t.cpu().numpy() for t in b)).T)
        assert torch.equal(qcp.mxfp4_matmul(*a, *b, dtype=torch.float32).cpu().double(), want), (M, N, K)


@GPU
def test_product_extreme_scales(gpu):
    """A NaN scale spoils its own row or column only; the smallest and largest
    scales multiply as they should."""
    for M, N in ((5, 70), (150, 300), (300, 520)):
        a, b = random_payload(M, 512, 5, 127, 128), random_payload(N, 512, 6, 127, 128)
        clean = qcp.mxfp4_matmul(*a, *b, dtype=torch.float32)
        a[1][3, 5] = 255
        b[1][N - 1, 0] = 255
        got = qcp.mxfp4_matmul(*a, *b, dtype=torch.float32)
        keep = torch.ones(M, N, dtype=torch.bool, device="cuda")
        keep[3], keep[:, N - 1] = False, False
        assert torch.isnan(got[~keep]).all() and torch.equal(got[keep], clean[keep])
        lo, hi = random_payload(M, 256, 7, 0, 1), random_payload(N, 256, 8, 254, 255)
        check_product(lo, hi, qcp.mxfp4_matmul(*lo, *hi, dtype=torch.float32), "f32", "2^-127 x 2^127")


@GPU
def test_long_rows_and_offsets_past_32_bits(gpu):
    """B's payload of more than 2^32 bytes: the last rows come out right."""
    K, N = 65536, (1 << 17) + 5
    b = (torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda"), torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda"))
    tail = random_payload(64, K, 3, 120, 125)
    b[0][-64:], b[1][-64:] = tail
    for M in (1, 40):
        a = random_payload(M, K, 4, 120, 125)
        out = qcp.mxfp4_matmul(*a, *b, dtype=torch.float32)
        assert not out[:, :-64].any()
        check_product(a, tail, out[:, -64:], "f32", M)


@GPU
def test_streams_and_graph(gpu):
    x = values(300, 1000, "bf16", 1)
    w = values(520, 1000, "bf16", 2)

    def chain():
        a, b = qcp.mxfp4_quantize(x), qcp.mxfp4_quantize(w)
        t = qcp.mxfp4_quantize(x, transpose=True)
        one = qcp.mxfp4_matmul(a[0][:1], a[1][:1], *b)
        return [*a, *b, *t, qcp.mxfp4_matmul(*a, *b, dtype=torch.float32), one, qcp.mxfp4_dequantize(*a, 1000)]
    want = [t.clone() for t in chain()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = chain()
    torch.cuda.synchronize()
    assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain()
    for k in range(4):
        for t in got:
            t.zero_()
        x.mul_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(got, want)), k
        chain()


# ------------------------------------------------------------------ linear

def rounded(t):
    c, s, _ = R.mx_payload(np.ascontiguousarray(t))
    return R.mx_values(c, s)[:, :t.shape[1]]


@GPU
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,I,O", [(1, 64, 32), (7, 100, 33), (77, 520, 260), (300, 257, 130)])
def test_linear_and_its_gradients_match_the_formula(gpu, T, I, O, dt):
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    make = lambda *s: torch.randn(*s, generator=g, device="cuda").to(DT[dt])  # noqa: E731
    x, w, dy = make(T, I).requires_grad_(), (make(O, I) * 0.05).requires_grad_(), make(T, O) * 0.01
    y = qcp.mxfp4_linear(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    X, W, D = wide(x), wide(w), wide(dy)
    for got, a, b in ((y, rounded(X), rounded(W)), (dx, rounded(D), rounded(W.T)), (dw, rounded(D.T), rounded(X.T))):
        want, size = a @ b.T, np.abs(a) @ np.abs(b).T
        bound = a.shape[1] * 2.0 ** -24 * size + UNIT[dt] * np.abs(want) + 2.0 ** -25
        assert got.dtype == DT[dt] and (np.abs(wide(got) - want) <= bound).all()


@GPU
def test_linear_gradients_match_differences(gpu):
    """On inputs that MXFP4 represents exactly the layer is the plain linear map,
    so differences along the grid (a step from one representable value to the
    next) equal its gradients exactly: all sums are small multiples of 1/4."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    T, I, O = 32, 64, 32
    pick = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, -0.5, -1.0, -2.0, -3.0], device="cuda")
    draw = lambda *s: pick[torch.randint(0, 10, s, generator=g, device="cuda")]  # noqa: E731
    x, w, dy = draw(T, I), draw(O, I), draw(T, O)
    for t in (x, w, dy):                                  # one 4 in each block of 32, along either axis
        k = torch.arange(t.shape[0], device="cuda")
        for c in range(0, t.shape[1], 32):
            t[k, c + k % 32] = 4.0
    x.requires_grad_(), w.requires_grad_()
    y = qcp.mxfp4_linear(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    base = (y.detach() * dy).sum()
    for t, grad, name in ((x, dx, "x"), (w, dw, "w")):
        for r, c in ((0, 1), (3, 7), (31, 60), (16, 33)):
            old = t.detach()[r, c].item()
            if old == 4.0:
                continue
            new = {3.0: 2.0, -3.0: -2.0}.get(old, old + 0.5 if old not in (1.5, 2.0, -2.0) else (2.0 if old == 1.5 else old + 1.0))
            moved = t.detach().clone()
            moved[r, c] = new
            y2 = qcp.mxfp4_linear(moved, w.detach()) if name == "x" else qcp.mxfp4_linear(x.detach(), moved)
            assert ((y2 * dy).sum() - base).item() == grad[r, c].item() * (new - old), (name, r, c)


@GPU
def test_linear_shapes_and_partial_gradients(gpu):
    x = torch.randn(2, 3, 40, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(50, 40, device="cuda", dtype=torch.bfloat16)
    flat = qcp.mxfp4_linear(x.view(6, 40), w)
    assert torch.equal(qcp.mxfp4_linear(x, w), flat.view(2, 3, 50))
    assert torch.equal(qcp.mxfp4_linear(x[0, 0], w), flat[0])
    a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
    qcp.mxfp4_linear(a, b).float().square().sum().backward()
    c = x.clone().requires_grad_()
    qcp.mxfp4_linear(c, w).float().square().sum().backward()
    d = w.clone().requires_grad_()
    qcp.mxfp4_linear(x, d).float().square().sum().backward()
    assert torch.equal(a.grad, c.grad) and torch.equal(b.grad, d.grad)
    e = x.clone().requires_grad_()                        # a broadcast input: its gradient sums over the copies
    qcp.mxfp4_linear(e[:1].expand(5, 3, 40), w).sum().backward()
    assert e.grad[0].abs().sum() > 0 and not e.grad[1:].any()


@GPU
def test_linear_without_gradients_does_only_the_product(gpu, monkeypatch):
    from quantized_collective_payloads_amd import mxfp4
    calls = []
    enqueue = mxfp4._enqueue
    monkeypatch.setattr(mxfp4, "_enqueue", lambda name, *a: (calls.append(name), enqueue(name, *a))[1])
    x = torch.randn(6, 40, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(50, 40, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    y = qcp.mxfp4_linear(x, w)
    assert calls == ["mxfp4_quantize_both", "mxfp4_quantize", "mxfp4_matmul"] and y.requires_grad
    for mode in (torch.no_grad, torch.inference_mode):
        calls.clear()
        with mode():
            z = qcp.mxfp4_linear(x, w)
        assert torch.equal(y, z) and not z.requires_grad
        assert calls == ["mxfp4_quantize", "mxfp4_quantize", "mxfp4_matmul"]


# ------------------------------------------------------------------ refusals (CPU)

OK, EINVAL, EALIGN = 0, -1, -2
A = 0x7f0000000000
S = 1 << 32


@pytest.fixture()
def lib():
    if not os.path.exists(qcp.LIB_PATH):
        pytest.fail(f"{qcp.LIB_PATH} not built")
    return qcp.library()


def test_c_entries_refuse(lib):
    def quant(x=A, xt=2, rows=64, cols=256, ld=256, t=0, c=A + S, s=A + 2 * S):
        return lib.mxfp4_quantize(x, xt, rows, cols, ld, t, c, s, None)

    def dequant(c=A, s=A + S, rows=64, cols=256, y=A + 2 * S, yt=2, ld=256):
        return lib.mxfp4_dequantize(c, s, rows, cols, y, yt, ld, None)

    def mul(a=A, sa=A + S, b=A + 2 * S, sb=A + 3 * S, M=64, N=64, K=256, c=A + 4 * S, ct=2, ldc=64):
        return lib.mxfp4_matmul(a, sa, b, sb, M, N, K, c, ct, ldc, None)
    def both(x=A, xt=2, rows=64, cols=256, ld=256, c=A + S, s=A + 2 * S, ct=A + 3 * S, st=A + 4 * S):
        return lib.mxfp4_quantize_both(x, xt, rows, cols, ld, c, s, ct, st, None)
    assert both(rows=0) == OK and both(cols=0, ld=0) == OK
    for bad in (dict(x=0), dict(xt=5), dict(ct=0), dict(st=0), dict(ld=255), dict(ct=A + S + 64), dict(st=A + 3 * S),
                dict(s=A), dict(st=A + 2 * S + 16), dict(rows=1 << 33, cols=1, ld=1), dict(cols=1 << 32, ld=1 << 32, rows=1)):
        assert both(**bad) == EINVAL, bad
    for bad in (dict(x=A + 1), dict(c=A + S + 8), dict(st=A + 4 * S + 4)):
        assert both(**bad) == EALIGN, bad
    for f in (quant, dequant):
        assert f(rows=0) == OK and f(cols=0, ld=0) == OK
        for bad in (dict(rows=-1), dict(cols=-1), dict(ld=255), dict(c=0), dict(s=0), dict(rows=1 << 40),
                    dict(rows=1 << 30, cols=256), dict(rows=1, cols=(1 << 31) + 1, ld=1 << 32),
                    dict(ld=1 << 40), dict(ld=1 << 62)):
            assert f(**bad) == EINVAL, (f, bad)
        for bad in (dict(c=A + S + 8), dict(s=A + 2 * S + 4)):
            assert f(**bad) == EALIGN, (f, bad)
    for bad in (dict(xt=0), dict(xt=4), dict(t=2), dict(x=0), dict(c=A + 1024), dict(s=A + 1024), dict(s=A + S + 512)):
        assert quant(**bad) == EINVAL, bad
    assert quant(x=A + 1) == EALIGN and quant(x=A + 2, xt=3) == EALIGN
    for bad in (dict(yt=0), dict(y=0), dict(y=A + 64), dict(y=A + S)):
        assert dequant(**bad) == EINVAL, bad
    assert dequant(y=A + 2 * S + 1) == EALIGN and dequant(y=A + 2 * S + 2, yt=3) == EALIGN
    assert mul(M=0) == OK and mul(N=0, ldc=0) == OK
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(ldc=63), dict(ct=0), dict(a=0), dict(sa=0), dict(b=0),
                dict(sb=0), dict(c=0), dict(M=1 << 30), dict(K=1 << 32), dict(c=A), dict(c=A + 2 * S + 64),
                dict(c=A + 3 * S), dict(M=1 << 22, N=1 << 22, K=128, ldc=1 << 22)):
        assert mul(**bad) == EINVAL, bad
    for bad in (dict(a=A + 8), dict(sb=A + 3 * S + 4), dict(c=A + 4 * S + 1), dict(c=A + 4 * S + 2, ct=3)):
        assert mul(**bad) == EALIGN, bad
    assert [qcp.mxfp4_padded(n) for n in (0, 1, 128, 129)] == [0, 128, 128, 256]
    assert lib.qcp_mxfp4_padded(-1) == -1 and lib.qcp_mxfp4_padded(1 << 40) == -1


def test_binding_refuses(lib):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731

    def raises(match, fn, *a, **kw):
        with pytest.raises(ValueError, match=match):
            fn(*a, **kw)
    raises("x: 1 dimensions", qcp.mxfp4_quantize, torch.zeros(64))
    raises("x: dtype", qcp.mxfp4_quantize, torch.zeros(4, 64, dtype=torch.float64))
    raises("x: expected", qcp.mxfp4_quantize, None)
    raises("codes: shape", qcp.mxfp4_quantize, torch.zeros(4, 64), codes=u8(4, 32))
    raises("scales: dtype", qcp.mxfp4_quantize, torch.zeros(4, 64), scales=torch.zeros(4, 4))
    raises("GPU tensors only", qcp.mxfp4_quantize, torch.zeros(4, 64))
    raises("x: 3 dimensions", qcp.mxfp4_quantize_both, torch.zeros(2, 4, 64))
    raises("GPU tensors only", qcp.mxfp4_quantize_both, torch.zeros(4, 64))
    raises("codes: rows of 60 bytes", qcp.mxfp4_dequantize, u8(4, 60), u8(4, 4), 100)
    raises("scales: shape", qcp.mxfp4_dequantize, u8(4, 64), u8(4, 8), 100)
    raises("codes: rows of 128 values for 129", qcp.mxfp4_dequantize, u8(4, 64), u8(4, 4), 129)
    raises("out: shape", qcp.mxfp4_dequantize, u8(4, 64), u8(4, 4), 100, out=torch.zeros(4, 99))
    raises("must be contiguous", qcp.mxfp4_dequantize, u8(4, 128)[:, :64], u8(4, 4), 100)
    raises("GPU tensors only", qcp.mxfp4_dequantize, u8(4, 64), u8(4, 4), 100)
    raises("b_codes: rows of 256", qcp.mxfp4_matmul, u8(4, 64), u8(4, 4), u8(4, 128), u8(4, 8))
    raises("a_scales: shape", qcp.mxfp4_matmul, u8(4, 64), u8(3, 4), u8(4, 64), u8(4, 4))
    raises("out: shape", qcp.mxfp4_matmul, u8(4, 64), u8(4, 4), u8(5, 64), u8(5, 4), out=torch.zeros(5, 4))
    raises("GPU tensors only", qcp.mxfp4_matmul, u8(4, 64), u8(4, 4), u8(5, 64), u8(5, 4))
    raises("last dimension 63", qcp.mxfp4_linear, torch.zeros(4, 63), torch.zeros(8, 64))
    raises("weight: 1 dimensions", qcp.mxfp4_linear, torch.zeros(4, 63), torch.zeros(8))
    raises("GPU tensors only", qcp.mxfp4_linear, torch.zeros(4, 64), torch.zeros(8, 64))


def test_c_entry_of_the_sliced_product_refuses(lib):
    work = lib.qcp_mxfp4_matmul_work
    assert work(64, 512, 28672) == 4 * 8 * 64 * 512 and work(64, 512, 4096) == 0 and work(8, 512, 28672) == 0
    assert work(0, 64, 28672) == work(64, 64, 0) == 0 and work(-1, 64, 8192) == work(64, 1 << 40, 8192) == -1
    need = work(64, 64, 12288)

    def mul(a=A, sa=A + S, b=A + 2 * S, sb=A + 3 * S, M=64, N=64, K=12288, c=A + 4 * S, ct=2, ldc=64, w=A + 5 * S, n=need):
        return lib.mxfp4_matmul_sliced(a, sa, b, sb, M, N, K, c, ct, ldc, w, n, None)
    assert need > 0 and mul(M=0) == OK and mul(N=0, ldc=0, w=None, n=0) == OK
    for bad in (dict(n=need - 1), dict(n=-1), dict(w=A), dict(w=A + 4 * S), dict(w=A + 3 * S + 16), dict(K=-1), dict(c=0),
                dict(a=0), dict(ldc=63), dict(ct=9)):
        assert mul(**bad) == EINVAL, bad
    assert mul(w=A + 5 * S + 4) == EALIGN and mul(c=A + 4 * S + 1) == EALIGN


@pytest.fixture()
def layer_on_cpu(monkeypatch):
    """The layer on CPU tensors, its launches replaced: quantizing does nothing and a product is zero."""
    from quantized_collective_payloads_amd import mxfp4
    monkeypatch.setattr(mxfp4, "_same_gpu", lambda index, *ts: None)
    monkeypatch.setattr(mxfp4, "_quantize_to", lambda *args: None)
    monkeypatch.setattr(mxfp4, "_product", lambda index, a, b, M, N, K, dtype, like: like.new_zeros((M, N), dtype=dtype))


@pytest.mark.parametrize("which", ["x", "weight", "both"])
@pytest.mark.parametrize("grad", [True, False])
def test_linear_refuses_forward_mode_tangents(layer_on_cpu, grad, which):
    """With and without gradients: it has no rule for them, and an output without a tangent
    would say that the derivative is zero."""
    from torch.autograd import forward_ad
    x, w = torch.ones(3, 32), torch.ones(4, 32)
    with torch.set_grad_enabled(grad), forward_ad.dual_level():
        a = forward_ad.make_dual(x, x) if which != "weight" else x
        b = forward_ad.make_dual(w, w) if which != "x" else w
        for v in (a, a.view(3, 1, 32), a.t().contiguous().t()):
            with pytest.raises(NotImplementedError):
                qcp.mxfp4_linear(v, b)
        assert qcp.mxfp4_linear(x, w).shape == (3, 4)
    assert qcp.mxfp4_linear(x, w).shape == (3, 4)


EMPTY = [(2, 3, 0), (0,), (3, 0), (0, 3, 0), (0, 0), (2, 0, 64), (0, 64), (64,), (2, 1, 3, 64)]


def like_torch(shape, device):
    """y and the gradients have the shapes of torch's own layer, and its zeros where there is nothing to sum."""
    x, w = (torch.ones(s, device=device, requires_grad=True) for s in (shape, (5, shape[-1])))
    y = qcp.mxfp4_linear(x, w)
    want = torch.nn.functional.linear(x, w)
    assert y.shape == want.shape
    with torch.no_grad():
        assert qcp.mxfp4_linear(x, w).shape == want.shape
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
    else:                                                  # ones are exact
        assert (y == shape[-1]).all() and (dx == 5).all() and (dw == y.numel() / 5).all()


def test_rows_below_the_bound_have_no_slices(lib):
    """The binding asks for scratch memory only above this length: the library has no use for
    it at any shape up to there, and one right above."""
    from quantized_collective_payloads_amd.mxfp4 import _UNSLICED
    work = qcp.library().qcp_mxfp4_matmul_work
    shapes = [(M, N) for M in (17, 32, 33, 64, 128, 200, 500, 2048, 8192) for N in (1, 16, 64, 500, 700, 2048, 4096, 8192)]
    for K in (1, 128, 4096, _UNSLICED - 127, _UNSLICED):
        assert not any(work(M, N, K) for M, N in shapes), K
    for K in (_UNSLICED + 1, 7950, 7999, 8000, 8064):
        assert work(128, 2048, K) > 0 and work(500, 700, K) > 0, K


@GPU
@pytest.mark.parametrize("K", [7936, 7937, 7950, 7999, 8000])
def test_layer_and_product_agree_bit_for_bit(gpu, K):
    """A layer passes the length of its rows, a product of payloads the padded one: the same
    kernel for both."""
    x, w = values(128, K, "bf16", 3), values(2048, K, "bf16", 4)
    y = qcp.mxfp4_linear(x, w)
    c = qcp.mxfp4_matmul(*qcp.mxfp4_quantize(x), *qcp.mxfp4_quantize(w))
    assert torch.equal(y.view(torch.int16), c.view(torch.int16))
    x32, w32 = x.float(), w.float()                        # every bit of the fp32 sums
    assert torch.equal(qcp.mxfp4_linear(x32, w32), qcp.mxfp4_matmul(*qcp.mxfp4_quantize(x), *qcp.mxfp4_quantize(w), torch.float32))
