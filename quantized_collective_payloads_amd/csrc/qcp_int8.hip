// qcp_int8.hip -- the INT8 payload with one scale per row (a token of an activation, an
// output channel of a weight): quantize and dequantize.
//
// s = absmax / 127 over the row, a code is the fp32 quotient x / s rounded to the nearest
// integer, ties to even, within +-127; a row of zeros has s = 0.  A row with an infinity or
// a NaN has a NaN scale and codes 0.  Rows of codes are padded with zeros to whole 128s, so
// that every row begins on a cache line and the products never see a short one.
//
// The scale has to be known before the first code, so a team of lanes (16, a wave, or a
// work-group) keeps a whole row in registers: x is read once.  A piece is 16 bytes of x:
// 8 values of 16 bits or 4 of 32, whose codes are 8 or 4 consecutive bytes.
//
// Bound: HBM, 3 bytes per 16-bit value each way.  8192 x 28672 bf16: quantize 114 to 122 us (6.2
// to 5.8 TB/s), dequantize 100 (7.0); 28672 x 8192 107 us; a copy runs at 5.1 TB/s.  x is read past
// the caches (ordinary loads: 126 and 125 us); the codes stay there for the product.
#include <algorithm>

#include "qcp_int8.h"
#include "qcp_ops.h"

namespace qcp {

namespace {

template <int XT>
__device__ __forceinline__ void store_codes(uint8_t *p, u32x2_t c) {
    if constexpr (XT == F32) *(uint32_t *)p = c.x;
    else *(u32x2_t *)p = c;
}

// A row per team of LANES lanes, V pieces a lane.  LONG: rows of more pieces than that, in
// rounds, read twice.
template <int XT, int LANES, int V, bool LONG>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void k_int8_quantize(
    const void *__restrict__ x, int64_t rows, int64_t cols, int64_t ld, uint32_t pieces, uint32_t groups,
    uint8_t *__restrict__ codes, float *__restrict__ scales) {
    constexpr int U = unit<XT>(), B = dtype_traits<XT>::bytes, ROWS = LANES < 256 ? 256 / LANES : 1;
    __shared__ uint32_t maxima[2][(LANES + 63) / 64];
    const uint32_t tid = __builtin_amdgcn_workitem_id_x(), team = tid / LANES, t = tid % LANES;
    uint32_t turn = 0;
    for (int64_t row = (int64_t)__builtin_amdgcn_workgroup_id_x() * ROWS + team; row < rows;
         row += (int64_t)groups * ROWS, turn ^= 1) {
        const uint8_t *const from = (const uint8_t *)x + row * ld * B;
        u32x4_t v[V];
        // piece k of a round; beyond the row it is zero
        auto load = [&](uint32_t first, int k) __attribute__((always_inline)) {
            const uint32_t p = first + k * LANES + t;
            const int64_t left = cols - (int64_t)p * U;
            v[k] = u32x4_t{0, 0, 0, 0};
            if (left > 0) v[k] = load_piece<XT>(from + (int64_t)p * 16, left > U ? U : (int)left);
        };
        uint32_t m = 0;
        for (uint32_t first = 0; first < (LONG ? pieces : 1); first += V * LANES) {
#pragma unroll
            for (int k = 0; k < V; k++) load(first, k);
#pragma unroll
            for (int k = 0; k < V; k++) m = largest<XT>(m, v[k]);
        }
        m = group_max_u32<(LANES < 64 ? LANES : 64)>(as_f32_bits<XT>(m));
        if constexpr (LANES > 64) {
            if ((tid & 63) == 0) maxima[turn][tid / 64] = m;
            __syncthreads();
            m = maxima[turn][0];
#pragma unroll
            for (int w = 1; w < LANES / 64; w++) m = max(m, maxima[turn][w]);
        }
        BlockScale<INT8> b;
        const bool finite = row_scale(m, b);
        const RecipBracket rb = recip_bracket(b.r);
        for (uint32_t first = 0; first < (LONG ? pieces : 1); first += V * LANES) {
            if constexpr (LONG) {
#pragma unroll
                for (int k = 0; k < V; k++) load(first, k);
            }
#pragma unroll
            for (int k = 0; k < V; k++) {
                const uint32_t p = first + k * LANES + t;
                if (p >= pieces) continue;
                u32x2_t c = {0, 0};
                if (finite) c = encode<XT>(v[k], b, rb);
                store_codes<XT>(codes + ((int64_t)row * pieces + p) * U, c);
            }
        }
        if (t == 0) scales[row] = scale_value(finite, b);
    }
}

template <int XT, int LANES, int V, bool LONG = false>
hipError_t run_quantize(const void *x, int64_t rows, int64_t cols, int64_t ld, int64_t pieces, uint8_t *codes,
                        float *scales, hipStream_t st) {
    constexpr int ROWS = LANES < 256 ? 256 / LANES : 1;
    const unsigned groups = (unsigned)std::min<int64_t>((rows + ROWS - 1) / ROWS, 1 << 20);
    hipLaunchKernelGGL((k_int8_quantize<XT, LANES, V, LONG>), dim3(groups), dim3(LANES < 256 ? 256 : LANES), 0, st, x,
                       rows, cols, ld, (uint32_t)pieces, groups, codes, scales);
    return hipGetLastError();
}

template <int XT>
hipError_t quantize_rows(const void *x, int64_t rows, int64_t cols, int64_t ld, uint8_t *codes, float *scales,
                         hipStream_t st) {
    const int64_t pieces = (cols + 127) / 128 * 128 / unit<XT>();
    // The fewest lanes that hold a row in 2 to 8 pieces each.  us of bf16 (fp32), read past the
    // caches: 8192 x 28672 512 x 8 114, 256 x 16 119, 1024 x 4 135; 28672 x 8192 256 x 4 107
    // (512 x 4 179), 512 x 4 123 (256 x 8 185); 4096 x 14336 512 x 4 31, 256 x 8 32; 14336 x 4096
    // 256 x 2 30 (256 x 4 48), 64 x 8 31.5; 5000 x 520 64 x 2 4.8, 256 x 2 7.3.  Few long rows do
    // not fill the GPU, and more lanes a row make each quicker: 1 x 28672 1024 x 4 4.0, 512 x 8 4.8.
    if (pieces <= 16 * 2) return run_quantize<XT, 16, 2>(x, rows, cols, ld, pieces, codes, scales, st);
    if (pieces <= 64 * 2) return run_quantize<XT, 64, 2>(x, rows, cols, ld, pieces, codes, scales, st);
    if (pieces <= 64 * 4) return run_quantize<XT, 64, 4>(x, rows, cols, ld, pieces, codes, scales, st);
    if (pieces <= 256 * 2) return run_quantize<XT, 256, 2>(x, rows, cols, ld, pieces, codes, scales, st);
    if (pieces <= 256 * 4) return run_quantize<XT, 256, 4>(x, rows, cols, ld, pieces, codes, scales, st);
    if (pieces <= 512 * 4) return run_quantize<XT, 512, 4>(x, rows, cols, ld, pieces, codes, scales, st);
    if (pieces <= 1024 * 4 && rows < 256) return run_quantize<XT, 1024, 4>(x, rows, cols, ld, pieces, codes, scales, st);
    if (pieces <= 512 * 8) return run_quantize<XT, 512, 8>(x, rows, cols, ld, pieces, codes, scales, st);
    if (pieces <= 1024 * 8) return run_quantize<XT, 1024, 8>(x, rows, cols, ld, pieces, codes, scales, st);
    return run_quantize<XT, 1024, 8, true>(x, rows, cols, ld, pieces, codes, scales, st);
}

// codes -> values: a piece of y a lane, kVecs of them a wave's stride apart
constexpr int kVecs = 4;

template <int YT>
__global__ __launch_bounds__(kThreads) void k_int8_dequantize(const uint8_t *__restrict__ codes,
                                                              const float *__restrict__ scales, int64_t vecs,
                                                              uint32_t pieces, int64_t cols, int64_t ld,
                                                              void *__restrict__ y) {
    constexpr int U = unit<YT>(), B = dtype_traits<YT>::bytes;
    const int64_t v0 = wave_id() * (64 * kVecs);
    if (v0 >= vecs) return;
    const int64_t row0 = v0 / pieces;
    const uint32_t col0 = (uint32_t)(v0 - row0 * pieces);
    u32x2_t c[kVecs];
    float s[kVecs];
    uint32_t col[kVecs];
    int64_t row[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; k++) {
        const uint32_t step = k * 64 + lane_id(), q = (col0 + step) / pieces;
        row[k] = row0 + q;
        col[k] = col0 + step - q * pieces;
        c[k] = u32x2_t{0, 0};
        s[k] = 0;
        if (v0 + step >= vecs) continue;
        const uint8_t *p = codes + (v0 + step) * U;
        if constexpr (YT == F32) c[k].x = *(const uint32_t *)p;
        else c[k] = *(const u32x2_t *)p;
        s[k] = scales[row[k]];
    }
#pragma unroll
    for (int k = 0; k < kVecs; k++) {
        const int64_t left = v0 + k * 64 + lane_id() < vecs ? cols - (int64_t)col[k] * U : 0;
        float f[U];
        static_for<4>([&](auto I) __attribute__((always_inline)) {
            constexpr int i = I;
            f[i] = cvt_sbyte<i>(c[k].x) * s[k];
            if constexpr (YT != F32) f[4 + i] = cvt_sbyte<i>(c[k].y) * s[k];
        });
        u32x4_t w;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if constexpr (YT == F32) w[i] = __float_as_uint(f[i]);
            else w[i] = narrow2<YT>(f[2 * i], f[2 * i + 1]);
        }
        uint8_t *to = (uint8_t *)y + (row[k] * ld + (int64_t)col[k] * U) * B;
        if (left >= U) {
            __builtin_nontemporal_store(w, (u32x4_any *)to);
        } else {
#pragma unroll
            for (int i = 0; i < U; i++) {
                if (i >= left) continue;
                if constexpr (YT == F32) ((uint32_t *)to)[i] = w[i];
                else ((uint16_t *)to)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
            }
        }
    }
}

template <int YT>
hipError_t dequantize_rows(const uint8_t *codes, const float *scales, int64_t rows, int64_t cols, void *y, int64_t ld,
                           hipStream_t st) {
    const int64_t pieces = (cols + 127) / 128 * 128 / unit<YT>(), vecs = rows * pieces;
    const unsigned grid = grid_for_waves((vecs + 64 * kVecs - 1) / (64 * kVecs));
    if (grid == 0) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_int8_dequantize<YT>), dim3(grid), dim3(kThreads), 0, st, codes, scales, vecs,
                       (uint32_t)pieces, cols, ld, y);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_quantize(const void *x, int xt, int64_t rows, int64_t cols, int64_t ld, uint8_t *codes,
                                float *scales, hipStream_t st) {
    switch (xt) {
    case F16: return quantize_rows<F16>(x, rows, cols, ld, codes, scales, st);
    case BF16: return quantize_rows<BF16>(x, rows, cols, ld, codes, scales, st);
    case F32: return quantize_rows<F32>(x, rows, cols, ld, codes, scales, st);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_int8_dequantize(const uint8_t *codes, const float *scales, int64_t rows, int64_t cols, void *y,
                                  int yt, int64_t ld, hipStream_t st) {
    switch (yt) {
    case F16: return dequantize_rows<F16>(codes, scales, rows, cols, y, ld, st);
    case BF16: return dequantize_rows<BF16>(codes, scales, rows, cols, y, ld, st);
    case F32: return dequantize_rows<F32>(codes, scales, rows, cols, y, ld, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qcp
