// qcp_int8_mixed.hip -- the product of a 16-bit matrix with an INT8 payload over whose rows
// is summed: C[m, n] = sum over k of a[m, k] * x[k, n], where x[k, n] = code * scale of row k,
// rounded to fp32 and then to a's type, as the payload is read everywhere.  A backward
// pass has two such products: dx = dy W (the payload of W, k its output channels) and
// dW = dy^T x (the payload of x, k the tokens; a is given as its transpose).
//
// The matrix cores want 8 consecutive k of a row from each lane, but the payload, and a
// transposed a, have n (or m) along their rows.  So operands go through registers: a thread
// reads 4 columns of 8 rows, decodes them (a conversion, a product with the row's scale and
// half a rounding a code), and has 8 k of each column, 16 bytes to write to LDS; of a 16-bit
// matrix the same with byte moves.  Both operands then lie in LDS with k along the rows.
#include <algorithm>

#include "qcp_matmul.h"
#include "qcp_ops.h"

namespace qcp {

namespace {

typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef u32x4_t u32x4_any __attribute__((aligned(2)));       // at an element's alignment
typedef u32x2_t u32x2_any __attribute__((aligned(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

template <int T>
__device__ __forceinline__ f32x16_t mma16bit(u32x4_t a, u32x4_t b, f32x16_t c) {
    if constexpr (T == BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// TM x TN of C per work-group, KS of k per stage, WM x WN waves
template <int TM_, int TN_, int KS_, int WM_, int WN_> struct MixedTile {
    static constexpr int TM = TM_, TN = TN_, KS = KS_, WM = WM_, WN = WN_;
    static constexpr int threads = 64 * WM * WN;
    static constexpr int FM = TM / WM / 32, FN = TN / WN / 32;   // fragments of a wave
    static constexpr int row = 2 * KS;                           // bytes of a row in LDS
    static constexpr int slot = (TM + TN) * row;
    static constexpr int octets = KS / 8;
    static_assert(TM == TN && TN / 4 * octets == threads && TM * octets == 4 * threads, "one unit of B, 4 of A a thread");
    static_assert(KS == 64 || KS == 128, "the order in LDS");
    // Where octet p (16 bytes) of a row lies.  A fragment read takes the same octet of 16
    // consecutive rows, a write after the transposition that of every fourth row of 64: in
    // both the 16 lie in different banks.
    __device__ static __forceinline__ uint32_t at(uint32_t r, uint32_t p) {
        if constexpr (KS == 64) return (r ^ ((r >> 5) & 1)) * 128 + ((p ^ ((r >> 1) & 7) ^ ((r >> 4) & 1)) * 16);
        else return r * 256 + ((p ^ (r & 15) ^ ((r >> 4) & 3)) * 16);
    }
};

// The stages of one slice of k of one tile.  TRANS: a is given as [K, M].
template <class G, int AT, bool TRANS, int CT, bool SLICED>
__global__ __launch_bounds__(G::threads, (G::slot > 40960 ? 2 : 2)) void k_int8_mixed(
    const uint16_t *__restrict__ a, int64_t lda, const uint8_t *__restrict__ codes, const float *__restrict__ scales,
    int64_t M, int64_t N, int64_t K, uint32_t pad, uint32_t slices, uint32_t m_tiles, uint32_t n_tiles,
    void *__restrict__ c, int64_t ldc) {
    constexpr int KS = G::KS, FM = G::FM, FN = G::FN;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * G::slot];
    const uint32_t tid = __builtin_amdgcn_workitem_id_x();
    const int wave = __builtin_amdgcn_readfirstlane((int)(tid >> 6)), lane = lane_id();
    uint32_t t = __builtin_amdgcn_workgroup_id_x(), slice = 0;
    if constexpr (SLICED) {
        slice = t / (m_tiles * n_tiles);
        t -= slice * (m_tiles * n_tiles);
    }
    const TilePlace place = tile_place(t, m_tiles, n_tiles);
    const int64_t m0 = (int64_t)place.m * G::TM, n0 = (int64_t)place.n * G::TN;
    const uint32_t m_rows = (uint32_t)min(M - m0, (int64_t)G::TM);
    // the slice's stages
    const int64_t all = (K + KS - 1) / KS;
    int64_t first = 0, last = all;
    if constexpr (SLICED) {
        const int64_t each = all / slices, over = all % slices;
        first = slice * each + min((int64_t)slice, over);
        last = first + each + (slice < over ? 1 : 0);
    }

    // what this thread brings: 4 columns of 8 rows of the payload, and of a transposed a ...
    constexpr uint32_t groups = G::TN / 4;
    const uint32_t col = 4 * (tid % groups), octet = groups == 64 ? (uint32_t)wave : tid / groups;
    const uint32_t b_off = octet * 8 * pad + (uint32_t)min(n0 + col, (int64_t)pad - 4);
    const uint32_t at_off = TRANS ? octet * 8 * (uint32_t)lda + col : 0;   // in elements
    const bool m_whole = m_rows == G::TM;
    // ... or 8 of k of 4 rows of a
    constexpr uint32_t row_step = G::threads / G::octets;
    const uint32_t a_row = tid / G::octets, a_oct = tid % G::octets;

    uint32_t wb[8];
    float sb[8];
    u32x2_t wt[8];
    u32x4_t wa[4];
    auto load = [&](int64_t s) __attribute__((always_inline)) {
        const int64_t k0 = s * KS;
        const uint8_t *const pb = codes + k0 * pad;
        const float *const ps = scales + k0 + octet * 8;
        const bool k_whole = k0 + KS <= K;
        if (k_whole) {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                wb[j] = *(const uint32_t *)(pb + (int64_t)j * pad + b_off);
                sb[j] = ps[j];
            }
        } else {
            const int left = (int)(K - k0) - (int)octet * 8;
#pragma unroll
            for (int j = 0; j < 8; j++) {
                wb[j] = 0;
                sb[j] = 0;
                if (j < left) {
                    wb[j] = *(const uint32_t *)(pb + (int64_t)j * pad + b_off);
                    sb[j] = ps[j];
                }
            }
        }
        if constexpr (TRANS) {
            const uint16_t *const pa = a + k0 * lda + m0;
            if (k_whole && m_whole) {
#pragma unroll
                for (int j = 0; j < 8; j++) wt[j] = *(const u32x2_any *)(pa + (int64_t)j * lda + at_off);
            } else {
                const int left = (int)min(K - k0, (int64_t)KS) - (int)octet * 8, width = (int)m_rows - (int)col;
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    wt[j] = u32x2_t{0, 0};
                    if (j >= left) continue;
                    const uint16_t *const p = pa + (int64_t)j * lda + at_off;
                    if (width >= 4) {
                        wt[j] = *(const u32x2_any *)p;
                    } else {
                        if (width > 0) wt[j].x = p[0];
                        if (width > 1) wt[j].x |= (uint32_t)p[1] << 16;
                        if (width > 2) wt[j].y = p[2];
                    }
                }
            }
        } else {
            const uint16_t *const pa = a + m0 * lda + k0;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint32_t r = min(a_row + i * row_step, m_rows - 1);
                const uint16_t *const p = pa + (r * (uint32_t)lda + a_oct * 8);
                if (k_whole) {
                    wa[i] = *(const u32x4_any *)p;
                } else {
                    const int left = (int)(K - k0) - (int)a_oct * 8;
                    wa[i] = u32x4_t{0, 0, 0, 0};
                    if (left >= 8) {
                        wa[i] = *(const u32x4_any *)p;
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; e++)
                            if (e < left) wa[i][e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
                    }
                }
            }
        }
    };
    typedef __attribute__((address_space(3))) uint8_t lds_byte;
    lds_byte *const base = (lds_byte *)lds;
    typedef __attribute__((address_space(3))) u32x4_t lds_piece;
    auto write = [&](uint32_t slot) __attribute__((always_inline)) {
        lds_byte *const to = base + slot * G::slot;
        if constexpr (TRANS) {
#pragma unroll
            for (int e = 0; e < 4; e++) {
                u32x4_t w;
#pragma unroll
                for (int j = 0; j < 4; j++)
                    w[j] = __builtin_amdgcn_perm(e < 2 ? wt[2 * j + 1].x : wt[2 * j + 1].y, e < 2 ? wt[2 * j].x : wt[2 * j].y,
                                                 e & 1 ? 0x07060302u : 0x05040100u);
                *(lds_piece *)(to + G::at(col + e, octet)) = w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) *(lds_piece *)(to + G::at(a_row + i * row_step, a_oct)) = wa[i];
        }
        static_for<4>([&](auto E) __attribute__((always_inline)) {
            constexpr int e = E;
            u32x4_t w;
#pragma unroll
            for (int j = 0; j < 4; j++)
                w[j] = narrow2<AT>(cvt_sbyte<e>(wb[2 * j]) * sb[2 * j], cvt_sbyte<e>(wb[2 * j + 1]) * sb[2 * j + 1]);
            *(lds_piece *)(to + G::TM * G::row + G::at(col + e, octet)) = w;
        });
    };

    const int r = lane & 31, half = lane >> 5;
    const uint32_t arow = (wave % G::WM) * (G::TM / G::WM) + r, brow = (wave / G::WM) * (G::TN / G::WN) + r;
    f32x16_t acc[FM][FN] = {};
    auto multiply = [&](uint32_t slot) __attribute__((always_inline)) {
        const lds_byte *const from = base + slot * G::slot;
#pragma unroll
        for (int q = 0; q < KS / 16; q++) {
            u32x4_t fa[FM], fb[FN];
#pragma unroll
            for (int j = 0; j < FN; j++) fb[j] = *(const lds_piece *)(from + G::TM * G::row + G::at(brow + 32 * j, 2 * q + half));
#pragma unroll
            for (int i = 0; i < FM; i++) fa[i] = *(const lds_piece *)(from + G::at(arow + 32 * i, 2 * q + half));
            // B first: a lane then holds 4 consecutive n of one m per group of registers
#pragma unroll
            for (int i = 0; i < FM; i++)
#pragma unroll
                for (int j = 0; j < FN; j++) acc[i][j] = mma16bit<AT>(fb[j], fa[i], acc[i][j]);
        }
    };

    if (first < last) {
        load(first);
        write(0);
        if (first + 1 < last) load(first + 1);
        wait_lds_and_meet();
        for (int64_t s = first; s < last; s++) {
            const uint32_t slot = (uint32_t)(s - first) & 1;
            if (s + 1 < last) write(slot ^ 1);
            if (s + 2 < last) load(s + 2);
            multiply(slot);
            wait_lds_and_meet();
        }
    }
    const bool whole = m0 + G::TM <= M && n0 + G::TN <= N;
    void *const to = SLICED ? (float *)c + slice * M * N : c;
    static_for<FM * FN>([&](auto I) __attribute__((always_inline)) {
        constexpr int i = I / FN, j = I % FN;
        store_fragment<CT>(acc[i][j], to, ldc, m0 + arow + 32 * i, n0 + (brow - r) + 32 * j, half, M, N, whole);
    });
}

// The sum of the slices, in their order, rounded once: 4 columns a lane.
template <int CT>
__global__ __launch_bounds__(kThreads) void k_int8_mixed_join(const float *__restrict__ parts, int slices, int64_t M,
                                                              int64_t N, void *__restrict__ c, int64_t ldc) {
    const int64_t quads = (N + 3) / 4, total = M * quads;
    const int64_t id = (int64_t)__builtin_amdgcn_workgroup_id_x() * kThreads + __builtin_amdgcn_workitem_id_x();
    if (id >= total) return;
    const int64_t m = id / quads, n = (id - m * quads) * 4;
    const int count = N - n < 4 ? (int)(N - n) : 4;
    const float *p = parts + m * N + n;
    float v[4] = {};
    for (int s = 0; s < slices; s++, p += M * N) {
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (j < count) v[j] += p[j];
    }
    store4<CT>(c, m * ldc + n, count, v);
}

using Tile256 = MixedTile<256, 256, 64, 2, 4>;
using Tile128 = MixedTile<128, 128, 64, 2, 2>;
using Tile64 = MixedTile<64, 64, 128, 2, 2>;

struct MixedArgs {
    const uint16_t *a;
    int64_t lda;
    const uint8_t *codes;
    const float *scales;
    int64_t M, N, K;
    void *c;
    int64_t ldc;
    hipStream_t st;
};

template <class G, int AT, bool TRANS, int CT, bool SLICED = false>
hipError_t run(const MixedArgs &p, int slices = 1) {
    const int64_t mt = (p.M + G::TM - 1) / G::TM, nt = (p.N + G::TN - 1) / G::TN;
    const uint32_t pad = (uint32_t)((p.N + 127) / 128 * 128);
    hipLaunchKernelGGL((k_int8_mixed<G, AT, TRANS, CT, SLICED>), dim3((unsigned)(mt * nt * slices)), dim3(G::threads), 0,
                       p.st, p.a, p.lda, p.codes, p.scales, p.M, p.N, p.K, pad, (uint32_t)slices, (uint32_t)mt,
                       (uint32_t)nt, p.c, p.ldc);
    return hipGetLastError();
}

template <int AT, bool TRANS, int CT>
hipError_t run_mixed(const MixedArgs &p, float *work) {
    const int slices = work ? int8_mixed_slices(p.M, p.N, p.K) : 1;
    if (slices > 1) {
        MixedArgs q = p;
        q.c = work;
        q.ldc = p.N;
        const hipError_t e = run<Tile64, AT, TRANS, F32, true>(q, slices);
        if (e != hipSuccess) return e;
        const int64_t total = p.M * ((p.N + 3) / 4);
        hipLaunchKernelGGL((k_int8_mixed_join<CT>), dim3((unsigned)((total + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                           p.st, work, slices, p.M, p.N, p.c, p.ldc);
        return hipGetLastError();
    }
    const auto tiles = [&](int64_t side) { return ((p.M + side - 1) / side) * ((p.N + side - 1) / side); };
    if (tiles(64) <= 512) return run<Tile64, AT, TRANS, CT>(p);
    if (tiles(256) < 192) return run<Tile128, AT, TRANS, CT>(p);
    return run<Tile256, AT, TRANS, CT>(p);
}

template <int AT, bool TRANS>
hipError_t by_result(const MixedArgs &p, int ct, float *work) {
    return ct == F32 ? run_mixed<AT, TRANS, F32>(p, work) : run_mixed<AT, TRANS, AT>(p, work);
}

}  // namespace

int int8_mixed_slices(int64_t M, int64_t N, int64_t K) {
    const int64_t stages = (K + 127) / 128, rows = (M + 63) / 64, cols = (N + 63) / 64;
    if (M < 1 || N < 1 || rows > 128 || cols > 128 || rows * cols > 128 || stages < 8) return 1;
    return (int)std::min<int64_t>(std::min<int64_t>(8, stages / 4), 256 / (rows * cols));
}

hipError_t launch_int8_mixed(const void *a, int at, int64_t lda, int transpose, const uint8_t *codes,
                             const float *scales, int64_t M, int64_t N, int64_t K, void *c, int ct, int64_t ldc,
                             float *work, hipStream_t st) {
    const MixedArgs p = {(const uint16_t *)a, lda, codes, scales, M, N, K, c, ldc, st};
    if (at == BF16) return transpose ? by_result<BF16, true>(p, ct, work) : by_result<BF16, false>(p, ct, work);
    if (at == F16) return transpose ? by_result<F16, true>(p, ct, work) : by_result<F16, false>(p, ct, work);
    return hipErrorInvalidValue;
}

}  // namespace qcp
