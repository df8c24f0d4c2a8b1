// qcp_mxfp4.hip -- the MXFP4 payload: quantize along the rows or along the
// columns of a matrix, and dequantize.
//
// A block is 32 values of one payload row.  With E the exponent field of the
// block's fp32 absmax, the scale byte is e = max(E - 2, 0) (the OCP MX rule: the
// largest E2M1 value is 6 = 1.5 * 2^2), and a code is x * 2^(127-e) rounded to the
// nearest of {0, 0.5, 1, 1.5, 2, 3, 4, 6}, ties to the even code, 6 beyond, sign
// kept.  gfx950's v_cvt_scalef32_pk_fp4_* does exactly that from fp32, bf16 and
// fp16, two values an instruction, and v_cvt_scalef32_pk_*_fp4 the way back.  A
// block with an infinity or a NaN has e = 255 and dequantizes to NaN throughout.
//
// A payload row holds its values padded with zeros to whole 128s: 64 code bytes
// and 4 scale bytes per 128, so every row of codes starts on 64 bytes, every row
// of scales on 4, and the matrix instructions never see a short block.
//
// Bound: HBM; 2 + 0.53 bytes per 16-bit value for a few instructions.  Measured on
// 14336 x 4096 bf16: quantize 24.6 us (6.0 TB/s), its transpose 31 (4.8; 25 from cache), both 39 (34),
// dequantize 22.9 (6.5); a copy of that matrix runs at 5.3 TB/s.
//
// Along the rows: a lane owns 8 consecutive values (one 16-byte load of 16-bit
// input, one dword of codes), so a block is 4 lanes and its absmax two DPP steps,
// on the 16-bit patterns where the input has them.  Output positions are the same
// whether rows are padded or not: vector i of the padded matrix has its codes at
// byte 4i.  A matrix that is one run of whole 128s needs no row arithmetic (FLAT).
// fp32 moves 4 values a lane (a block is 8 lanes), so that every access of a wave is
// one contiguous run: 32-byte pieces a lane cost the dequantize to fp32 a third of
// its rate (28672 x 8192: 317 us).
//
// Along the columns: a work-group takes 256 rows x 64 columns.  A lane owns two
// neighbouring columns of 32 rows, so its two blocks need no other lane: absmax,
// scale and codes all come from its own registers.  One input row of the tile and
// one output row are both 128 bytes; the codes pass through LDS to be stored so.
// For both payloads at once the tile (of 16 bits: 256 x 128) also goes through LDS as
// it is, to be taken by rows, a block of 32 values per thread: memory sees the matrix
// once.  Read again from L2 instead, fp32 took 358 us at 28672 x 8192 against 239.
#include "qcp_device.h"
#include "qcp_ops.h"

namespace qcp {

namespace {

typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
typedef u32x4_t u32x4_any __attribute__((aligned(2)));     // at an element's alignment
typedef unsigned int u32_any __attribute__((aligned(2)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef u32x2_t u32x2_any __attribute__((aligned(4)));

constexpr int kMxPad = 128;       // values of a row's granule
constexpr int kMxVecs = 4;        // vectors of 8 values per lane

template <int XT> constexpr int words8() { return XT == F32 ? 8 : 4; }   // dwords of 8 values

// 8 values of 16 bits from p, of which `count` exist (the others are zero)
__device__ __forceinline__ void load8(const uint16_t *x, int64_t i, int count, uint32_t *w) {
    const uint16_t *p = x + i;
    if (count >= 8) {
        const u32x4_any v = __builtin_nontemporal_load((const u32x4_any *)p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const uint32_t lo = 2 * k < count ? p[2 * k] : 0, hi = 2 * k + 1 < count ? p[2 * k + 1] : 0;
            w[k] = lo | (hi << 16);
        }
    }
}

// 4 fp32 values from p, of which `count` exist
__device__ __forceinline__ void load4(const float *x, int64_t i, int count, uint32_t *w) {
    if (count >= 4) {
        const u32x4_any v = __builtin_nontemporal_load((const u32x4_any *)(x + i));
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++) w[k] = k < count ? __float_as_uint(x[i + k]) : 0;
    }
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    const u16x2_t m = __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b));
    return __builtin_bit_cast(uint32_t, m);
}

// |x| maximum of one or two values' bit patterns: 16-bit types keep two maxima
template <int XT>
__device__ __forceinline__ uint32_t absmax_of(uint32_t m, uint32_t w) {
    if constexpr (XT == F32) return max(m, w & 0x7fffffffu);
    else return max_u16x2(m, w & 0x7fff7fffu);
}

// scale byte from the absmax of a block
template <int XT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
    uint32_t field;
    if constexpr (XT == F32) {
        field = m >> 23;
    } else {
        m = max(m & 0xffffu, m >> 16);
        field = XT == BF16 ? m >> 7 : __float_as_uint(f16_lo(m)) >> 23;
    }
    return field == 255u ? 255u : field < 2u ? 0u : field - 2u;
}

// 2^(e-127); 2^-127 is a subnormal
__device__ __forceinline__ float scale_of(uint32_t e) {
    return __uint_as_float(e == 0 ? 0x00400000u : e << 23);
}

// two values -> two codes in byte K of w
template <int XT, int K>
__device__ __forceinline__ uint32_t encode2(uint32_t w, uint32_t a, uint32_t b, float s) {
    if constexpr (XT == F32)
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(a), __uint_as_float(b), s, K);
    else if constexpr (XT == BF16)
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, a), s, K);
    else
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(f16x2_t, a), s, K);
}

template <int XT>
__device__ __forceinline__ uint32_t encode8(const uint32_t (&w)[words8<XT>()], float s) {
    uint32_t c = 0;
    if constexpr (XT == F32) {
        c = encode2<XT, 0>(c, w[0], w[1], s);
        c = encode2<XT, 1>(c, w[2], w[3], s);
        c = encode2<XT, 2>(c, w[4], w[5], s);
        c = encode2<XT, 3>(c, w[6], w[7], s);
    } else {
        c = encode2<XT, 0>(c, w[0], 0, s);
        c = encode2<XT, 1>(c, w[1], 0, s);
        c = encode2<XT, 2>(c, w[2], 0, s);
        c = encode2<XT, 3>(c, w[3], 0, s);
    }
    return c;
}

// where the wave's vectors lie in rows of `width` vectors: the first one's row and
// column from one division per wave, a lane's from a small one
struct RowPlace {
    int64_t row;
    uint32_t col;     // in vectors
};
__device__ __forceinline__ RowPlace place(int64_t row0, uint32_t col0, uint32_t step, uint32_t width) {
    const uint32_t c = col0 + step, q = c / width;
    return RowPlace{row0 + q, c - q * width};
}

// how many of the `unit` values at place p of a row exist
__device__ __forceinline__ int values_left(bool inside, int64_t cols, uint32_t col, int unit) {
    const int64_t left = inside ? cols - (int64_t)col * unit : 0;
    return left > unit ? unit : left < 0 ? 0 : (int)left;
}

// fp32 moves as 4 values a lane, 16 bytes, in two runs of 256 values a wave; a lane
// then has 16 bits of codes of each run (low: the first).  Lanes 2i and 2i+1 trade
// halves, and hold 8 codes of the first and of the second run, whole dwords.  The
// trade is its own inverse.
__device__ __forceinline__ uint32_t trade(uint32_t w, int lane) {
    const uint32_t other = dpp_u32<0xB1>(w);
    return lane & 1 ? (other >> 16) | (w & 0xffff0000u) : (w & 0xffffu) | (other << 16);
}

template <int XT, bool FLAT>
__global__ __launch_bounds__(kThreads) void k_mx_quantize(const void *__restrict__ x, int64_t vecs,
                                                          uint32_t width, int64_t cols, int64_t ld,
                                                          uint32_t *__restrict__ codes,
                                                          uint8_t *__restrict__ scales) {
    constexpr int UNIT = XT == F32 ? 4 : 8;                  // values of a lane's run
    const int lane = lane_id();
    const int64_t v0 = wave_id() * (64 * kMxVecs);
    if (v0 >= vecs) return;
    const int64_t row0 = FLAT ? 0 : v0 / width;
    const uint32_t col0 = FLAT ? 0 : (uint32_t)(v0 - row0 * width);
    uint32_t w[kMxVecs][words8<XT>()];
    // where run h of vector group u begins for this lane, in units, and whether inside
    auto load = [&](int u, int h, uint32_t *to) __attribute__((always_inline)) {
        constexpr int per = 8 / UNIT;
        const uint32_t step = (uint32_t)(u * 64 * per + h * 64 + lane);
        const bool inside = v0 * per + step < vecs * per;
        int64_t at = (v0 * per + step) * UNIT;
        int count = inside ? UNIT : 0;
        if constexpr (!FLAT) {
            const RowPlace p = place(row0, col0 * per, step, width * per);
            at = p.row * ld + (int64_t)p.col * UNIT;
            count = values_left(inside, cols, p.col, UNIT);
        }
        if constexpr (XT == F32) load4((const float *)x, at, count, to);
        else load8((const uint16_t *)x, at, count, to);
    };
#pragma unroll
    for (int u = 0; u < kMxVecs; u++) {
        load(u, 0, w[u]);
        if constexpr (XT == F32) load(u, 1, w[u] + 4);
    }
#pragma unroll
    for (int u = 0; u < kMxVecs; u++) {
        const int64_t v = v0 + u * 64 + lane;
        if constexpr (XT == F32) {
            // a block is 8 lanes of either run
            uint32_t e[2], c = 0;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                uint32_t m = 0;
#pragma unroll
                for (int k = 0; k < 4; k++) m = absmax_of<XT>(m, w[u][4 * h + k]);
                e[h] = scale_byte<XT>(group_max_u32<8>(m));
            }
            c = encode2<XT, 0>(c, w[u][0], w[u][1], scale_of(e[0]));
            c = encode2<XT, 1>(c, w[u][2], w[u][3], scale_of(e[0]));
            c = encode2<XT, 2>(c, w[u][4], w[u][5], scale_of(e[1]));
            c = encode2<XT, 3>(c, w[u][6], w[u][7], scale_of(e[1]));
            c = trade(c, lane);
            // vectors of 8: the first run's are v0 + 64u + 0..31, the second's 32..63
            const int64_t at = v0 + u * 64 + (lane & 1) * 32 + (lane >> 1);
            if (at < vecs) codes[at] = c;
            const int64_t block = (v0 + u * 64) / 4 + (lane >> 3);
            if ((lane & 7) == 0) {
                if (block * 4 < vecs) scales[block] = (uint8_t)e[0];
                if (block * 4 + 32 < vecs) scales[block + 8] = (uint8_t)e[1];
            }
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < words8<XT>(); k++) m = absmax_of<XT>(m, w[u][k]);
            m = absmax_of<XT>(m, dpp_u32<0xB1>(m));
            m = absmax_of<XT>(m, dpp_u32<0x4E>(m));
            const uint32_t e = scale_byte<XT>(m);
            const uint32_t c = encode8<XT>(w[u], scale_of(e));
            // the scale bytes of 4 blocks (16 lanes) in one dword
            uint32_t d = e << (8 * ((lane >> 2) & 3));
            d |= dpp_u32<0x141>(d);
            d |= dpp_u32<0x140>(d);
            if (v < vecs) {
                codes[v] = c;
                if ((lane & 15) == 0) ((uint32_t *)scales)[v >> 4] = d;
            }
        }
    }
}

// codes 2k, 2k+1 and their scale -> two values of 16 bits, or one of 32 each
template <int YT, int K>
__device__ __forceinline__ void decode2(uint32_t c, float s, uint32_t *w) {
    if constexpr (YT == F32) {
        const f32x2_t v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, K);
        w[0] = __float_as_uint(v.x);
        w[1] = __float_as_uint(v.y);
    } else if constexpr (YT == BF16) {
        w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, K));
    } else {
        w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, K));
    }
}
template <int YT> constexpr uint32_t nan_word() {
    return YT == F32 ? 0x7fc00000u : YT == BF16 ? 0x7fc07fc0u : 0x7e007e00u;
}

template <int YT>
__device__ __forceinline__ void store8(void *y, int64_t i, int count, const uint32_t (&w)[words8<YT>()]) {
    constexpr int B = dtype_traits<YT>::bytes;
    uint8_t *p = (uint8_t *)y + i * B;
    if (count >= 8) {
#pragma unroll
        for (int k = 0; k < words8<YT>() / 4; k++)
            __builtin_nontemporal_store(u32x4_any{w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]},
                                        (u32x4_any *)p + k);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) {
            if (j >= count) continue;
            if constexpr (YT == F32) ((uint32_t *)p)[j] = w[j];
            else ((uint16_t *)p)[j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
        }
    }
}

__device__ __forceinline__ void store4(float *y, int64_t i, int count, const uint32_t *w) {
    if (count >= 4) {
        __builtin_nontemporal_store(u32x4_any{w[0], w[1], w[2], w[3]}, (u32x4_any *)(y + i));
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (j < count) y[i + j] = __uint_as_float(w[j]);
    }
}

template <int YT, bool FLAT>
__global__ __launch_bounds__(kThreads) void k_mx_dequantize(const uint32_t *__restrict__ codes,
                                                            const uint8_t *__restrict__ scales,
                                                            int64_t vecs, uint32_t width, int64_t cols,
                                                            int64_t ld, void *__restrict__ y) {
    constexpr int UNIT = YT == F32 ? 4 : 8, per = 8 / UNIT;
    const int lane = lane_id();
    const int64_t v0 = wave_id() * (64 * kMxVecs);
    if (v0 >= vecs) return;
    const int64_t row0 = FLAT ? 0 : v0 / width;
    const uint32_t col0 = FLAT ? 0 : (uint32_t)(v0 - row0 * width);
    uint32_t c[kMxVecs], e[kMxVecs][per];
#pragma unroll
    for (int u = 0; u < kMxVecs; u++) {
        // fp32: as in the quantize, two runs of 256 values and a trade between lanes
        const int64_t v = v0 + u * 64 + (YT == F32 ? (lane & 1) * 32 + (lane >> 1) : lane);
        c[u] = v < vecs ? codes[v] : 0;
#pragma unroll
        for (int h = 0; h < per; h++) {
            const int64_t block = YT == F32 ? (v0 + u * 64) / 4 + h * 8 + (lane >> 3) : (v0 + u * 64 + lane) >> 2;
            e[u][h] = block * 4 < vecs ? scales[block] : 0;
        }
    }
#pragma unroll
    for (int u = 0; u < kMxVecs; u++) {
        uint32_t w[words8<YT>()];
        if constexpr (YT == F32) c[u] = trade(c[u], lane);
        static_for<4>([&](auto K) __attribute__((always_inline)) {
            constexpr int k = K, step = YT == F32 ? 2 : 1;
            decode2<YT, k>(c[u], scale_of(e[u][k * per / 4]), w + k * step);
#pragma unroll
            for (int j = k * step; j < (k + 1) * step; j++)
                if (e[u][k * per / 4] == 255u) w[j] = nan_word<YT>();
        });
        static_for<per>([&](auto H) __attribute__((always_inline)) {
            constexpr int h = H;
            const uint32_t step = (uint32_t)(u * 64 * per + h * 64 + lane);
            const bool inside = v0 * per + step < vecs * per;
            int64_t at = (v0 * per + step) * UNIT;
            int count = inside ? UNIT : 0;
            if constexpr (!FLAT) {
                const RowPlace p = place(row0, col0 * per, step, width * per);
                at = p.row * ld + (int64_t)p.col * UNIT;
                count = values_left(inside, cols, p.col, UNIT);
            }
            if constexpr (YT == F32) store4((float *)y, at, count, w + 4 * h);
            else store8<YT>(y, at, count, w);
        });
    }
}

// A matrix above the 256 MB of the last cache is read past it, which leaves the codes
// there: 28672 x 8192 fp16 with the dequantize behind it 211 -> 198 us, both payloads and
// a product 268 -> 236; fp32 408 -> 365 and 352 -> 315.  (Codes written past it too: the
// quantize alone 119 -> 114, the pair 211.)  A smaller matrix may lie there already:
// 8192 x 4096 bf16, just written, 15.9 us and 21.6 (both) against 17.5 and 24.4;
// 16384 x 5120 37 and 46 against 45 and 56.
constexpr int64_t kStreamBytes = (int64_t)256 << 20;
constexpr int kTRows = 256;                    // tile of the column-wise quantize
template <int XT, bool BOTH> constexpr int tile_cols() { return XT != F32 && BOTH ? 128 : 64; }

// the codes and the scale byte of one block of a row
template <int XT>
__device__ __forceinline__ uint4 row_block(const uint32_t (&w)[4][words8<XT>()], uint32_t &e) {
    uint32_t c[4], m = 0;
#pragma unroll
    for (int k = 0; k < 4; k++)
#pragma unroll
        for (int j = 0; j < words8<XT>(); j++) m = absmax_of<XT>(m, w[k][j]);
    e = scale_byte<XT>(m);
#pragma unroll
    for (int k = 0; k < 4; k++) c[k] = encode8<XT>(w[k], scale_of(e));
    return make_uint4(c[0], c[1], c[2], c[3]);
}

// STREAM: the matrix passes the caches by
template <bool STREAM, typename T>
__device__ __forceinline__ T load_words(const T *p) {
    if constexpr (STREAM) return __builtin_nontemporal_load(p);
    else return *p;
}

template <int XT, bool BOTH, bool STREAM>
__global__ __launch_bounds__((4 * tile_cols<XT, BOTH>())) void k_mx_quantize_t(const void *__restrict__ x, int64_t rows,
                                                            int64_t cols, int64_t ld, uint32_t col_tiles, uint32_t groups,
                                                            int64_t pad_rows, uint8_t *__restrict__ codes,
                                                            uint8_t *__restrict__ scales, int64_t pad_cols,
                                                            uint8_t *__restrict__ row_codes,
                                                            uint8_t *__restrict__ row_scales) {
    constexpr int B = dtype_traits<XT>::bytes, kTCols = tile_cols<XT, BOTH>();
    constexpr int kLine = 128 + 16;            // bytes per column in LDS: a shift of 4 banks
    // for both payloads the tile itself lies here first, rows 16 bytes more than their
    // 256 apart, which spreads the row pass over all banks
    constexpr int kRow = 256 + 16, kNeed = kTCols * (kLine + 8);
    __shared__ __attribute__((aligned(16))) uint8_t lds[BOTH ? kTRows * kRow : kNeed];
    uint8_t *const lines = lds, *const marks = lds + kTCols * kLine;
    // Work-groups are dealt round-robin to the 8 XCDs.  16 neighbouring tiles, 2 KB of
    // a 16-bit row, go to one XCD, so that its reads spread over all its L2 channels;
    // in launch order they would lie 1 KB apart, a quarter of the channels.
    uint32_t wg = __builtin_amdgcn_workgroup_id_x();
    if (wg < (groups & ~127u)) wg = (wg & ~127u) + (wg & 7) * 16 + ((wg >> 3) & 15);
    const int64_t tr = (int64_t)(wg / col_tiles) * kTRows, tc = (int64_t)(wg % col_tiles) * kTCols;
    const int tid = (int)__builtin_amdgcn_workitem_id_x();
    const int block = tid / (kTCols / 2);      // which 32 rows of the tile
    const int pair = tid % (kTCols / 2);       // which two columns
    const int64_t r0 = tr + block * 32, c0 = tc + pair * 2;
    const int64_t have = rows - r0;            // rows of this block that exist (may be <= 0)
    const int two = cols - c0 >= 2 ? 2 : cols - c0 == 1 ? 1 : 0;

    uint32_t a[32], b[XT == F32 ? 32 : 1];     // 16-bit: both columns of a row in a[r]
    const uint8_t *p = (const uint8_t *)x + (r0 * ld + c0) * B;
#pragma unroll
    for (int r = 0; r < 32; r++) {
        const uint8_t *q = p + (int64_t)r * ld * B;
        if constexpr (XT == F32) {
            a[r] = b[r] = 0;
            if (r < have && two == 2) {
                const u32x2_any v = load_words<STREAM>((const u32x2_any *)q);
                a[r] = v.x;
                b[r] = v.y;
            } else if (r < have && two == 1) {
                a[r] = *(const uint32_t *)q;
            }
        } else {
            a[r] = 0;
            if (r < have && two == 2) a[r] = load_words<STREAM>((const u32_any *)q);
            else if (r < have && two == 1) a[r] = *(const uint16_t *)q;
        }
    }
    // the tile along its rows: a thread takes a block of 32 at a time; the scales of a
    // row, 4 bytes (fp32: 2), go out at once
    if constexpr (BOTH) {
        constexpr int per = kTCols / 32;       // blocks of a row
#pragma unroll
        for (int r = 0; r < 32; r++) {
            uint8_t *at = lds + (block * 32 + r) * kRow + pair * 2 * B;
            if constexpr (XT == F32) *(u32x2_t *)at = u32x2_t{a[r], b[r]};
            else *(uint32_t *)at = a[r];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const int unit = tid + 4 * kTCols * k, line = unit / per, place = unit % per;
            const int64_t r = tr + line;
            uint32_t w[4][words8<XT>()], e;
#pragma unroll
            for (int q = 0; q < 4; q++)
#pragma unroll
                for (int j = 0; j < words8<XT>(); j += 4) {
                    const uint4 v = *(const uint4 *)(lds + line * kRow + place * 32 * B + 8 * B * q + 4 * j);
                    w[q][j] = v.x; w[q][j + 1] = v.y; w[q][j + 2] = v.z; w[q][j + 3] = v.w;
                }
            const uint4 v = row_block<XT>(w, e);
            uint32_t d = e << (8 * place);
            d |= dpp_u32<0xB1>(d);
            if constexpr (per == 4) d |= dpp_u32<0x4E>(d);
            if (r >= rows) continue;
            *(uint4 *)(row_codes + r * (pad_cols / 2) + tc / 2 + 16 * place) = v;
            uint8_t *at = row_scales + r * (pad_cols / 32) + tc / 32;
            if (place == 0) {
                if constexpr (per == 4) *(uint32_t *)at = d;
                else *(uint16_t *)at = (uint16_t)d;
            }
        }
        __syncthreads();
    }
    uint32_t ma = 0, mb = 0;
#pragma unroll
    for (int r = 0; r < 32; r++) {
        ma = absmax_of<XT>(ma, a[r]);
        if constexpr (XT == F32) mb = absmax_of<XT>(mb, b[r]);
    }
    if constexpr (XT != F32) {
        mb = ma >> 16;
        ma &= 0xffffu;
    }
    const uint32_t ea = scale_byte<XT>(ma), eb = scale_byte<XT>(mb);
    const float sa = scale_of(ea), sb = scale_of(eb);
    uint32_t ca[4], cb[4];
    static_for<4>([&](auto W) {
        constexpr int w = W;
        ca[w] = cb[w] = 0;
        static_for<4>([&](auto K) {
            constexpr int k = K, r = 8 * w + 2 * k;
            if constexpr (XT == F32) {
                ca[w] = encode2<XT, k>(ca[w], a[r], a[r + 1], sa);
                cb[w] = encode2<XT, k>(cb[w], b[r], b[r + 1], sb);
            } else {                           // rows r, r+1 of one column side by side
                ca[w] = encode2<XT, k>(ca[w], __builtin_amdgcn_perm(a[r + 1], a[r], 0x05040100u), 0, sa);
                cb[w] = encode2<XT, k>(cb[w], __builtin_amdgcn_perm(a[r + 1], a[r], 0x07060302u), 0, sb);
            }
        });
    });
    *(uint4 *)(lines + (2 * pair) * kLine + 16 * block) = make_uint4(ca[0], ca[1], ca[2], ca[3]);
    *(uint4 *)(lines + (2 * pair + 1) * kLine + 16 * block) = make_uint4(cb[0], cb[1], cb[2], cb[3]);
    marks[(2 * pair) * 8 + block] = (uint8_t)ea;
    marks[(2 * pair + 1) * 8 + block] = (uint8_t)eb;
    __syncthreads();

    // output rows of 128 bytes: 8 threads a row; the padded height may end halfway
    const int64_t wide = pad_rows - tr;        // 128 or at least 256
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const int line = (tid >> 3) + kTCols / 2 * k, piece = tid & 7;
        const int64_t c = tc + line;
        if (c < cols && 32 * piece < wide)
            *(uint4 *)(codes + c * (pad_rows / 2) + tr / 2 + 16 * piece) =
                *(const uint4 *)(lines + line * kLine + 16 * piece);
    }
    if (tid < 2 * kTCols) {
        const int line = tid >> 1, half = tid & 1;
        const int64_t c = tc + line;
        if (c < cols && 128 * half < wide)
            *(uint32_t *)(scales + c * (pad_rows / 32) + tr / 32 + 4 * half) =
                *(const uint32_t *)(marks + line * 8 + 4 * half);
    }
}

// along the columns, and with BOTH also along the rows
template <int XT, bool BOTH>
hipError_t run_quantize_t(const void *x, int64_t rows, int64_t cols, int64_t ld, uint8_t *codes,
                          uint8_t *scales, uint8_t *row_codes, uint8_t *row_scales, hipStream_t st) {
    constexpr int TC = tile_cols<XT, BOTH>();
    const int64_t pr = (rows + kMxPad - 1) / kMxPad * kMxPad, pc = (cols + kMxPad - 1) / kMxPad * kMxPad;
    const int64_t ct = ((BOTH ? pc : cols) + TC - 1) / TC, rt = (rows + kTRows - 1) / kTRows;
    const bool stream = rows * cols * dtype_traits<XT>::bytes > kStreamBytes;
    const dim3 grid((unsigned)(ct * rt)), threads(4 * TC);
    if (stream)
        hipLaunchKernelGGL((k_mx_quantize_t<XT, BOTH, true>), grid, threads, 0, st, x, rows, cols, ld, (uint32_t)ct,
                           (uint32_t)(ct * rt), pr, codes, scales, pc, row_codes, row_scales);
    else
        hipLaunchKernelGGL((k_mx_quantize_t<XT, BOTH, false>), grid, threads, 0, st, x, rows, cols, ld, (uint32_t)ct,
                           (uint32_t)(ct * rt), pr, codes, scales, pc, row_codes, row_scales);
    return hipGetLastError();
}

template <int XT>
hipError_t run_quantize(const void *x, int64_t rows, int64_t cols, int64_t ld, int transpose,
                        uint8_t *codes, uint8_t *scales, hipStream_t st) {
    if (transpose)
        return run_quantize_t<XT, false>(x, rows, cols, ld, codes, scales, nullptr, nullptr, st);
    const int64_t pad = (cols + kMxPad - 1) / kMxPad * kMxPad;
    const bool flat = cols == pad && (ld == cols || rows == 1);
    const int64_t vecs = rows * pad / 8;
    const unsigned grid = grid_for_waves((vecs + 64 * kMxVecs - 1) / (64 * kMxVecs));
    if (flat)
        hipLaunchKernelGGL((k_mx_quantize<XT, true>), dim3(grid), dim3(kThreads), 0, st, x, vecs, 1u, cols,
                           ld, (uint32_t *)codes, scales);
    else
        hipLaunchKernelGGL((k_mx_quantize<XT, false>), dim3(grid), dim3(kThreads), 0, st, x, vecs,
                           (uint32_t)(pad / 8), cols, ld, (uint32_t *)codes, scales);
    return hipGetLastError();
}

template <int YT>
hipError_t run_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols,
                          void *y, int64_t ld, hipStream_t st) {
    const int64_t pad = (cols + kMxPad - 1) / kMxPad * kMxPad;
    const bool flat = cols == pad && (ld == cols || rows == 1);
    const int64_t vecs = rows * pad / 8;
    const unsigned grid = grid_for_waves((vecs + 64 * kMxVecs - 1) / (64 * kMxVecs));
    if (flat)
        hipLaunchKernelGGL((k_mx_dequantize<YT, true>), dim3(grid), dim3(kThreads), 0, st,
                           (const uint32_t *)codes, scales, vecs, 1u, cols, ld, y);
    else
        hipLaunchKernelGGL((k_mx_dequantize<YT, false>), dim3(grid), dim3(kThreads), 0, st,
                           (const uint32_t *)codes, scales, vecs, (uint32_t)(pad / 8), cols, ld, y);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const void *x, int xt, int64_t rows, int64_t cols, int64_t ld,
                              int transpose, uint8_t *codes, uint8_t *scales, hipStream_t st) {
    switch (xt) {
    case F16: return run_quantize<F16>(x, rows, cols, ld, transpose, codes, scales, st);
    case BF16: return run_quantize<BF16>(x, rows, cols, ld, transpose, codes, scales, st);
    case F32: return run_quantize<F32>(x, rows, cols, ld, transpose, codes, scales, st);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_mx_quantize_both(const void *x, int xt, int64_t rows, int64_t cols, int64_t ld,
                                   uint8_t *codes, uint8_t *scales, uint8_t *codes_t, uint8_t *scales_t,
                                   hipStream_t st) {
    switch (xt) {
    case F16: return run_quantize_t<F16, true>(x, rows, cols, ld, codes_t, scales_t, codes, scales, st);
    case BF16: return run_quantize_t<BF16, true>(x, rows, cols, ld, codes_t, scales_t, codes, scales, st);
    case F32: return run_quantize_t<F32, true>(x, rows, cols, ld, codes_t, scales_t, codes, scales, st);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows,
                                int64_t cols, void *y, int yt, int64_t ld, hipStream_t st) {
    switch (yt) {
    case F16: return run_dequantize<F16>(codes, scales, rows, cols, y, ld, st);
    case BF16: return run_dequantize<BF16>(codes, scales, rows, cols, y, ld, st);
    case F32: return run_dequantize<F32>(codes, scales, rows, cols, y, ld, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qcp
