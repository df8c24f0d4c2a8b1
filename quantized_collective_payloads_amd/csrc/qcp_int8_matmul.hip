// qcp_int8_matmul.hip -- C = A B^T on INT8 payloads with one scale per row: A is [M, K], B
// is [N, K], both with K along their rows, C [M, N] in fp32, bf16 or fp16.
//
// c = sa sb sum(qa qb): v_mfma_i32_32x32x32_i8 and _16x16x64_i8 add up the products of codes
// in 32-bit integers, exactly (the entry point bounds K so that no sum leaves them), whatever
// the order; only then come the two scales, in fp32, and one rounding to C's type.
// Which 16 of K a lane brings is free as long as both operands agree.
//
// Measured, by the GPU's clock: 8192 x 8192, K = 28672 1550 to 1650 us (2.5 to 2.3 POP/s), with all
// codes zero 1370; 2048 x 14336, K = 4096 118; 2048 x 2048, K = 2048 15; 1 x 14336, K = 4096 13.5
// with B in the last cache, 15.3 from HBM (3.8 TB/s); 1 x 128256, K = 4096 95 (5.5 TB/s).
#include <algorithm>

#include "qcp_int8.h"
#include "qcp_matmul.h"
#include "qcp_ops.h"

namespace qcp {

namespace {

typedef int i32x16_t __attribute__((ext_vector_type(16)));

// Scales whose product, and whose product with any sum, is a normal number or a true
// overflow: 0, or 2^-62 to 2^62
__device__ __forceinline__ bool tame(float s) { return s == 0.0f || (s >= 0x1p-62f && s <= 0x1p62f); }

// sum * sa * sb.  Outside the tame range the mantissas are multiplied and the exponents
// added, so that nothing overflows or underflows on the way to a result that does not.
template <bool TAME>
__device__ __forceinline__ float scaled(int sum, float sa, float sb) {
    if constexpr (TAME) return (float)sum * (sa * sb);
    const float m = __builtin_amdgcn_frexp_mantf(sa) * __builtin_amdgcn_frexp_mantf(sb);
    return __builtin_amdgcn_ldexpf((float)sum * m, __builtin_amdgcn_frexp_expf(sa) + __builtin_amdgcn_frexp_expf(sb));
}

// ---------------------------------------------------------------------------
// 64*FM x 64*FN of C per work-group, staged through LDS.
// ---------------------------------------------------------------------------
// Four waves, 2 x 2, hold 32*FM x 32*FN each.  A stage is 128 bytes of each operand row,
// whole cache lines, copied from memory to LDS without registers into one of `slots`; the
// lower half-wave takes the first 64 bytes of its rows, the upper one the others.  A stage is
// two phases; while a phase's products issue, the fragments of the next one are read, and in
// the second the copies of a later stage go into the slot that the barrier between the two
// has freed.  The order written is kept (sched_barrier).
//
// LDS holds a row's 8 pieces of 16 bytes in the order piece ^ (row / 2 % 8): the copy
// permutes its source addresses, so that a fragment read, 16 rows of 128 bytes at the same
// piece a cycle, touches each of the 64 banks once.
//
// A work-group walks several tiles: the copies of the next one's first stages, and of its
// scales, go out before the results of this one.  Rows past the end repeat the last row.
//
// Bound: the power that the matrix cores draw and, on zeros too, the waits of one wave a SIMD; 4 x
// 4 holds 256 accumulators and keeps up to 7 registers around a tile in scratch memory, none in the
// loop.
template <int FM, int FN> struct igeom {
    static constexpr int TM = 64 * FM, TN = 64 * FN;       // C per work-group
    static constexpr int slots = FM * FN == 1 ? 4 : 2;     // stages in LDS
    static constexpr int rows = TM + TN;
    static constexpr int slot = rows * 128;                // codes of A and B, one stage
    static constexpr int marks = rows * 4;                 // scales of A and B, one tile
    static constexpr int lds = slots * slot + 2 * marks;   // 132 KB at 4 x 4, 66 KB at 2 x 2, 65 KB at 1 x 1
    static constexpr int ops = 2 * FM * FN;                // products per phase and wave
    static constexpr int reads = 2 * (FM + FN);            // fragment pieces per phase
    static constexpr int copies = rows / 32;               // per stage and wave, 8 rows each
    static constexpr int waves_per_simd = FM * FN <= 4 ? 2 : 1;
    // 16-byte stores of a wave's whole results
    template <int CT> static constexpr int stores() { return FM * FN * 16 * dtype_traits<CT>::bytes / 16; }
    static constexpr int ahead = (slots - 2) * copies;     // copies of stages beyond the next
};

template <int FM, int FN> struct IntFragments {
    i32x4_t a[FM][2], b[FN][2];
};

__device__ __forceinline__ i32x4_t lds_codes(uint32_t at) { return __builtin_bit_cast(i32x4_t, lds16(at)); }

// SLICED: the tiles are those of `slices` parts of K, one part after the other; c is int32,
// an M x N for each, and the scales are left to the join.
template <int FM, int FN, int CT, bool SLICED>
__global__ __launch_bounds__(kThreads, (igeom<FM, FN>::waves_per_simd)) void k_int8_matmul_tiled(
    const uint8_t *__restrict__ a, const float *__restrict__ as, const uint8_t *__restrict__ b,
    const float *__restrict__ bs, int64_t M, int64_t N, uint32_t row_stages, uint32_t slices, uint32_t m_tiles,
    uint32_t n_tiles, uint32_t groups, void *__restrict__ c, int64_t ldc) {
    using Gm = igeom<FM, FN>;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[Gm::lds];
    const int tid = (int)__builtin_amdgcn_workitem_id_x();
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = lane_id();

    const uint32_t tiles = m_tiles * n_tiles * (SLICED ? slices : 1);
    const uint32_t row_bytes = row_stages * 128;
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
    constexpr uint32_t kMarks = Gm::slots * Gm::slot;      // where the scales begin
    uint32_t stages = row_stages, slice = 0;               // of the tile

    // the tile that is being copied: a wave brings a quarter of each operand's rows, 8 rows
    // at a time
    int64_t m0, n0;
    i32x4_t ra, rb;
    uint32_t m_rows, n_rows;
    auto set_tile = [&](uint32_t t) __attribute__((always_inline)) {
        uint32_t skip = 0;                                   // stages before the slice
        if constexpr (SLICED) {
            slice = t / (m_tiles * n_tiles);
            t -= slice * (m_tiles * n_tiles);
            const uint32_t each = row_stages / slices, over = row_stages % slices;
            skip = slice * each + min(slice, over);
            stages = each + (slice < over ? 1 : 0);
        }
        const TilePlace at = tile_place(t, m_tiles, n_tiles);
        m0 = (int64_t)at.m * Gm::TM;
        n0 = (int64_t)at.n * Gm::TN;
        m_rows = (uint32_t)min(M - m0, (int64_t)Gm::TM);
        n_rows = (uint32_t)min(N - n0, (int64_t)Gm::TN);
        ra = buffer_of(a + m0 * row_bytes + skip * 128, (uint64_t)m_rows * row_bytes - skip * 128);
        rb = buffer_of(b + n0 * row_bytes + skip * 128, (uint64_t)n_rows * row_bytes - skip * 128);
    };
    // the tile's scales, 64 rows a wave
    auto copy_marks = [&](uint32_t to) __attribute__((always_inline)) {
        if constexpr (SLICED) return;
        if (wave < FM)
            copy4_to_lds(to + wave * 256, min((uint32_t)(wave * 64 + lane), m_rows - 1) * 4,
                         buffer_of(as + m0, (uint64_t)m_rows * 4));
        if (wave < FN)
            copy4_to_lds(to + Gm::TM * 4 + wave * 256, min((uint32_t)(wave * 64 + lane), n_rows - 1) * 4,
                         buffer_of(bs + n0, (uint64_t)n_rows * 4));
    };

    // the n-th copy of a stage into the slot at `to`, from byte k of the rows
    const uint32_t copy_row = lane >> 3, copy_piece = ((lane & 7) ^ (lane >> 4)) * 16;
    auto copy = [&](auto I, uint32_t to, uint32_t k) __attribute__((always_inline)) {
        constexpr int n = I;
        constexpr bool of_a = n < 2 * FM;
        constexpr int i = of_a ? n : n - 2 * FM, rows = 16 * (of_a ? FM : FN);   // this wave's rows begin at wave * rows
        // three operations a copy instead of a register each (the asm keeps them from
        // being made once): row < 2^8, row_bytes < 2^24
        uint32_t row = copy_row;
        asm volatile("" : "+v"(row));
        row = min(wave * rows + i * 8 + row, (of_a ? m_rows : n_rows) - 1);
        const uint32_t at = (row & 0xffu) * (row_bytes & 0xffffffu) + (copy_piece ^ (i & 1 ? 64 : 0));
        copy_to_lds(to + (of_a ? 0 : Gm::TM * 128) + wave * rows * 128 + i * 1024, at, of_a ? ra : rb, k);
    };
    auto slot_of = [&](uint32_t s) __attribute__((always_inline)) { return (s & (Gm::slots - 1)) * Gm::slot; };
    auto copy_stage = [&](uint32_t s) __attribute__((always_inline)) {
        static_for<Gm::copies>([&](auto I) __attribute__((always_inline)) { copy(I, base + slot_of(s), s * 128); });
    };

    // fragments: wave w computes rows 32*FM*(w&1) of A against rows 32*FN*(w>>1) of B
    const int r = lane & 31, half = lane >> 5, x = (lane >> 1) & 7;
    const uint32_t arow = (wave & 1) * 32 * FM + r, brow = Gm::TM + (wave >> 1) * 32 * FN + r;
    // where piece 4 * half of the first fragment lies in slot 0; pieces p and q of a row
    // differ by the bits of 16 * (p ^ q)
    const uint32_t a_at = base + arow * 128 + ((4 * half) ^ x) * 16;
    const uint32_t b_at = base + brow * 128 + ((4 * half) ^ x) * 16;
    // the n-th of the fragments' pieces at la, lb and those at the piece beside, in the
    // order the products use them
    using Frag = IntFragments<FM, FN>;
    auto read = [&](auto I, uint32_t la, uint32_t lb, Frag &f) __attribute__((always_inline)) {
        constexpr int n = I, u = n / (FM + FN), q = n % (FM + FN);
        if constexpr (q < FN) f.b[q][u] = lds_codes((lb ^ (16 * u)) + q * 4096);
        else f.a[q - FN][u] = lds_codes((la ^ (16 * u)) + (q - FN) * 4096);
    };
    // pieces p and p ^ 1 beyond 4 * half of the slot of stage s
    auto read_all = [&](uint32_t s, uint32_t p, Frag &f) __attribute__((always_inline)) {
        const uint32_t la = (a_at ^ (16 * p)) + slot_of(s), lb = (b_at ^ (16 * p)) + slot_of(s);
        static_for<Gm::reads>([&](auto I) __attribute__((always_inline)) { read(I, la, lb, f); });
    };

    i32x16_t acc[FM][FN];
    Frag f, h;
    // the n-th product of a phase.  B first: a lane then holds 4 consecutive n of one m per
    // group of registers
    auto product = [&](auto I, const Frag &v) __attribute__((always_inline)) {
        constexpr int n = I, u = n / (FM * FN), i = n / FN % FM, j = n % FN;
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(v.b[j][u], v.a[i][u], acc[i][j], 0, 0, 0);
    };
    auto products = [&](const Frag &v) __attribute__((always_inline)) {
        static_for<Gm::ops>([&](auto I) __attribute__((always_inline)) { product(I, v); });
    };
    // the products of phase P of a stage, in the order written: between them the reads of the
    // next phase's fragments, from the slot at `from`, and with COPY the copies of stage
    // `next`, so the matrix cores never wait for the rest to issue.
    auto phase = [&](auto P, const Frag &now, Frag &then, uint32_t from, auto COPY, uint32_t next)
        __attribute__((always_inline)) {
        constexpr int S = Gm::ops;
        const uint32_t to = base + slot_of(next), k = next * 128;
        uint32_t la = a_at, lb = b_at;
        asm volatile("" : "+v"(la), "+v"(lb));   // addresses made here, not kept for every phase
        la = (la ^ (P ? 0 : 32)) + from;
        lb = (lb ^ (P ? 0 : 32)) + from;
        static_for<S>([&](auto I) __attribute__((always_inline)) {
            constexpr int n = I;
            product(I, now);
            // reads in the first half of the phase, copies too
            constexpr int r0 = n * 2 * Gm::reads / S, r1 = (n + 1) * 2 * Gm::reads / S;
            static_for<r1 - r0>([&](auto Q) __attribute__((always_inline)) {
                constexpr int q = r0 + Q;
                if constexpr (q < Gm::reads) read(std::integral_constant<int, q>{}, la, lb, then);
            });
            if constexpr (COPY) {
                constexpr int c0 = n * 2 * Gm::copies / S, c1 = (n + 1) * 2 * Gm::copies / S;
                static_for<c1 - c0>([&](auto Q) __attribute__((always_inline)) {
                    constexpr int q = c0 + Q;
                    if constexpr (q < Gm::copies) copy(std::integral_constant<int, q>{}, to, k);
                });
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    using no = std::integral_constant<int, 0>;
    using yes = std::integral_constant<int, 1>;

    uint32_t turn = 0;                                       // which of the scales' two places
    auto copy_first = [&]() __attribute__((always_inline)) {
        copy_marks(base + kMarks + turn * Gm::marks);
        static_for<Gm::slots>([&](auto Q) __attribute__((always_inline)) {
            if ((uint32_t)Q < stages) copy_stage((uint32_t)Q);
        });
    };
    uint32_t tile = __builtin_amdgcn_workgroup_id_x();
    set_tile(tile);
    copy_first();
    wait_and_meet<0>();
    for (;;) {
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int j = 0; j < FN; j++) acc[i][j] = i32x16_t{};
        if (stages) read_all(0, 0, f);
        uint32_t s = 0;
        for (; s + Gm::slots < stages; s++) {
            phase(no{}, f, h, slot_of(s), no{}, 0);
            wait_and_meet<Gm::ahead>();
            phase(yes{}, h, f, slot_of(s + 1), yes{}, s + Gm::slots);
        }
        for (; s < stages; s++) {
            read_all(s, 2, h);
            products(f);
            wait_and_meet<0>();
            products(h);
            if (s + 1 < stages) read_all(s + 1, 0, f);
        }

        // the next tile's first copies go out before this one's results
        const int64_t m_done = m0 + (wave & 1) * 32 * FM + r, n_done = n0 + (wave >> 1) * 32 * FN;
        const bool whole = m0 + Gm::TM <= M && n0 + Gm::TN <= N;
        void *const to = SLICED ? (int *)c + slice * M * N : c;
        const uint32_t marks = base + kMarks + turn * Gm::marks;
        tile += groups;
        const bool more = tile < tiles;
        if (more) {
            wait_lds_and_meet();                             // every wave is done with the slots
            set_tile(tile);
            turn ^= 1;
            copy_first();
        }
        if constexpr (SLICED) {
            static_for<FM * FN>([&](auto I) __attribute__((always_inline)) {
                constexpr int i = I / FN, j = I % FN;
                store_fragment<F32>(__builtin_bit_cast(f32x16_t, acc[i][j]), to, ldc, m_done + 32 * i, n_done + 32 * j,
                                    half, M, N, whole);
            });
        } else {
            const uint32_t at_a = marks + arow * 4, at_b = marks + (brow - r + 4 * half) * 4;
            float sa[FM];
            bool ok = true;
#pragma unroll
            for (int i = 0; i < FM; i++) {
                sa[i] = __uint_as_float(lds4(at_a + i * 128));
                ok = ok && tame(sa[i]);
            }
            static_for<FN>([&](auto J) __attribute__((always_inline)) {
                constexpr int j = J;
                float sb[16];
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const u32x4_t w = lds16(at_b + j * 128 + q * 32);
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        sb[4 * q + e] = __uint_as_float(w[e]);
                        ok = ok && tame(sb[4 * q + e]);
                    }
                }
                auto put = [&](auto T) __attribute__((always_inline)) {
                    static_for<FM>([&](auto I) __attribute__((always_inline)) {
                        constexpr int i = I;
                        f32x16_t v;
#pragma unroll
                        for (int e = 0; e < 16; e++) v[e] = scaled<T>(acc[i][j][e], sa[i], sb[e]);
                        store_fragment<CT>(v, to, ldc, m_done + 32 * i, n_done + 32 * j, half, M, N, whole);
                    });
                };
                if (__all(ok)) put(yes{});
                else put(no{});
            });
        }
        if (!more) break;
        // the copies are older than the stores, of which a whole tile has `stores` at least
        constexpr int stores = SLICED ? Gm::template stores<F32>() : Gm::template stores<CT>();
        if (whole) wait_and_meet<(stores < 63 ? stores : 63)>();
        else wait_and_meet<0>();
    }
}

template <int FM, int FN, int CT, bool SLICED = false>
hipError_t run_tiled(const uint8_t *a, const float *as, const uint8_t *b, const float *bs, int64_t M, int64_t N,
                     int64_t stages, void *c, int64_t ldc, hipStream_t st, int slices = 1) {
    using Gm = igeom<FM, FN>;
    const int64_t mt = (M + Gm::TM - 1) / Gm::TM, nt = (N + Gm::TN - 1) / Gm::TN;
    // as many work-groups as the GPU holds walk the tiles (a multiple of 8, so that each
    // stays on its XCD's tiles)
    const unsigned groups = (unsigned)std::min<int64_t>(mt * nt * slices, kCUs * Gm::waves_per_simd);
    hipLaunchKernelGGL((k_int8_matmul_tiled<FM, FN, CT, SLICED>), dim3(groups), dim3(kThreads), 0, st, a, as, b, bs, M,
                       N, (uint32_t)stages, (uint32_t)slices, (uint32_t)mt, (uint32_t)nt, groups, c, ldc);
    return hipGetLastError();
}

// The sum of the slices, and the scales: 4 columns a lane.
template <int CT>
__global__ __launch_bounds__(kThreads) void k_int8_matmul_join(const int *__restrict__ parts, int slices,
                                                               const float *__restrict__ as,
                                                               const float *__restrict__ bs, int64_t M, int64_t N,
                                                               void *__restrict__ c, int64_t ldc) {
    const int64_t m = group_y();
    const int64_t n = ((int64_t)__builtin_amdgcn_workgroup_id_x() * kThreads + __builtin_amdgcn_workitem_id_x()) * 4;
    if (n >= N) return;
    const int count = N - n < 4 ? (int)(N - n) : 4;
    const int *p = parts + m * N + n;
    int sum[4] = {};
    for (int s = 0; s < slices; s++, p += M * N) {
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (j < count) sum[j] += p[j];
    }
    const float sa = as[m];
    float v[4] = {};
#pragma unroll
    for (int j = 0; j < 4; j++)
        if (j < count) v[j] = scaled<false>(sum[j], sa, bs[n + j]);
    store4<CT>(c, m * ldc + n, count, v);
}

// ---------------------------------------------------------------------------
// Few rows of A (a token, a small batch): 16*FA rows against 16*FB rows of B.
// ---------------------------------------------------------------------------
// Bound: reading B once, and some 3 us that the smallest calls take.  N/16 work-groups; the WV waves of one deal out K in steps of 256
// bytes and add their sums in LDS, so a few rows still fill the GPU, without a second
// launch.  A load takes 64 consecutive bytes of 16 rows, a quarter-wave 16 of them (a lane 64
// consecutive bytes in four loads: 14.8 us for 1 x 14336, K = 4096, so 13.4).  Operands go
// straight to registers, a whole step's loads at a time (two steps at a time: 2 to 10% slower).
template <int FA, int FB, int WV, int CT>
__global__ __launch_bounds__(64 * WV) void k_int8_matmul_rows(
    const uint8_t *__restrict__ a, const float *__restrict__ as, const uint8_t *__restrict__ b,
    const float *__restrict__ bs, int64_t M, int64_t N, int64_t granules, void *__restrict__ c, int64_t ldc) {
    __shared__ i32x4_t sums[WV][FA * FB][64];
    const int wave = __builtin_amdgcn_readfirstlane((int)(__builtin_amdgcn_workitem_id_x() >> 6)), lane = lane_id();
    const int row = lane & 15, quarter = lane >> 4;
    const int64_t n0 = (int64_t)__builtin_amdgcn_workgroup_id_x() * (16 * FB), m0 = group_y() * (16 * FA);
    // rows of A past the end are not read (their sums are not stored), those of B repeat the last
    const uint8_t *pa[FA], *pb[FB];
    bool there[FA];
#pragma unroll
    for (int i = 0; i < FA; i++) {
        there[i] = m0 + 16 * i + row < M;
        pa[i] = a + (m0 + 16 * i + row) * granules * 64 + 16 * quarter;
    }
#pragma unroll
    for (int i = 0; i < FB; i++) pb[i] = b + min(n0 + 16 * i + row, N - 1) * granules * 64 + 16 * quarter;
    // granules are even, and so is where a step may end
    auto load = [&](int64_t g, i32x4_t (&v)[4], const uint8_t *p) __attribute__((always_inline)) {
        const bool all = g + 2 < granules;
#pragma unroll
        for (int t = 0; t < 4; t++) v[t] = t < 2 || all ? *(const i32x4_t *)(p + (g + t) * 64) : i32x4_t{0, 0, 0, 0};
    };
    i32x4_t acc[FA][FB] = {};
    for (int64_t g = 4 * wave; g < granules; g += 4 * WV) {
        i32x4_t fa[FA][4] = {}, fb[FB][4];
#pragma unroll
        for (int i = 0; i < FB; i++) load(g, fb[i], pb[i]);
#pragma unroll
        for (int i = 0; i < FA; i++)
            if (there[i]) load(g, fa[i], pa[i]);
#pragma unroll
        for (int t = 0; t < 4; t++)
#pragma unroll
            for (int i = 0; i < FA; i++)
#pragma unroll
                for (int j = 0; j < FB; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j][t], fa[i][t], acc[i][j], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < FA; i++)
#pragma unroll
        for (int j = 0; j < FB; j++) sums[wave][i * FB + j][lane] = acc[i][j];
    __syncthreads();
    // a lane's 4 sums are consecutive n of one m
    for (int k = wave; k < FA * FB; k += WV) {
        i32x4_t v = sums[0][k][lane];
#pragma unroll
        for (int w = 1; w < WV; w++) v += sums[w][k][lane];
        const int64_t m = m0 + 16 * (k / FB) + row, n = n0 + 16 * (k % FB) + 4 * quarter;
        if (m >= M || n >= N) continue;
        const int count = N - n < 4 ? (int)(N - n) : 4;
        const float sa = as[m];
        float r[4] = {};
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (j < count) r[j] = scaled<false>(v[j], sa, bs[n + j]);
        store4<CT>(c, m * ldc + n, count, r);
    }
}

template <int FA, int FB, int CT>
hipError_t run_rows(const uint8_t *a, const float *as, const uint8_t *b, const float *bs, int64_t M, int64_t N,
                    int64_t granules, void *c, int64_t ldc, hipStream_t st) {
    const dim3 grid((unsigned)((N + 16 * FB - 1) / (16 * FB)), (unsigned)((M + 16 * FA - 1) / (16 * FA)));
    if (granules <= 16)
        hipLaunchKernelGGL((k_int8_matmul_rows<FA, FB, 4, CT>), grid, dim3(256), 0, st, a, as, b, bs, M, N, granules, c, ldc);
    else
        hipLaunchKernelGGL((k_int8_matmul_rows<FA, FB, 8, CT>), grid, dim3(512), 0, st, a, as, b, bs, M, N, granules, c, ldc);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// The layer for few rows, in one launch: y = Q(x) W^T, up to 8 rows of x in 16 bits.
// ---------------------------------------------------------------------------
// Bound: reading W once; what a launch of its own for Q(x) takes, 2.6 us of the GPU and 6 of the
// host, is as much as a small product.  Every work-group makes Q(x) for itself, in LDS: a team
// of its lanes keeps a row in registers, V pieces a lane, as the quantize does and with its
// results.  Its first loads of W go out before (those of two steps: 1 x 4096, K = 4096 9.2 us from HBM and
// 9.8, 1 x 14336, K = 4096 19.1 and 17.9).
//
// LDS holds a row's pieces of 16 bytes in the order piece ^ (row % 8), so that the reads of a
// piece of 8 rows touch different banks.
constexpr int kFewWaves = 8, kFewThreads = 64 * kFewWaves, kFewBytes = 48 << 10;

template <int XT, int V>
__global__ __launch_bounds__(kFewThreads) void k_int8_linear_rows(const void *__restrict__ x, int64_t ldx, int M, int64_t K,
                                                                  const uint8_t *__restrict__ b,
                                                                  const float *__restrict__ bs, int64_t N,
                                                                  uint32_t granules, void *__restrict__ y, int64_t ldy) {
    extern __shared__ __attribute__((aligned(16))) uint8_t codes[];          // M rows of 64 * granules bytes
    __shared__ i32x4_t sums[kFewWaves][64];
    __shared__ uint32_t maxima[kFewWaves];
    __shared__ float marks[8];
    const uint32_t tid = __builtin_amdgcn_workitem_id_x(), P = granules * 64;
    const int wave = __builtin_amdgcn_readfirstlane((int)(tid >> 6)), lane = lane_id();
    const int row = lane & 15, quarter = lane >> 4;
    const int64_t n0 = (int64_t)__builtin_amdgcn_workgroup_id_x() * 16;
    const uint8_t *const pb = b + min(n0 + row, N - 1) * P + 16 * quarter;
    auto load = [&](uint32_t g, i32x4_t (&v)[4]) __attribute__((always_inline)) {
#pragma unroll
        for (uint32_t t = 0; t < 4; t++)
            v[t] = g + t < granules ? *(const i32x4_t *)(pb + (uint64_t)(g + t) * 64) : i32x4_t{0, 0, 0, 0};
    };
    i32x4_t fb[4];
    load(4 * wave, fb);

    // 1, 2, 4 or 8 teams of at least a wave, a row each
    const uint32_t teams = M <= 1 ? 1 : M <= 2 ? 2 : M <= 4 ? 4 : 8, lanes = kFewThreads / teams;
    const uint32_t m = tid / lanes, t = tid % lanes, pieces = P / 8;
    const bool mine = m < (uint32_t)M;
    const uint8_t *const from = (const uint8_t *)x + (mine ? m : 0) * ldx * 2;
    u32x4_t v[V];
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < V; k++) {
        const int64_t p = k * lanes + t, left = mine ? K - p * 8 : 0;
        v[k] = u32x4_t{0, 0, 0, 0};
        if (left > 0) v[k] = load_piece<XT>(from + p * 16, left > 8 ? 8 : (int)left);
    }
#pragma unroll
    for (int k = 0; k < V; k++) top = largest<XT>(top, v[k]);
    top = group_max_u32<64>(as_f32_bits<XT>(top));
    if (lane == 0) maxima[wave] = top;
    __syncthreads();
    const uint32_t first = wave & ~(lanes / 64 - 1);
    for (uint32_t w = 0; w < lanes / 64; w++) top = max(top, maxima[first + w]);
    BlockScale<INT8> s;
    const bool finite = row_scale(top, s);
    const RecipBracket rb = recip_bracket(s.r);
#pragma unroll
    for (int k = 0; k < V; k++) {
        const uint32_t p = k * lanes + t;
        if (!mine || p >= pieces) continue;
        u32x2_t c = {0, 0};
        if (finite) c = encode<XT>(v[k], s, rb);
        *(u32x2_t *)(codes + m * P + ((p / 2) ^ (m & 7)) * 16 + 8 * (p & 1)) = c;
    }
    if (mine && t == 0) marks[m] = scale_value(finite, s);
    __syncthreads();

    // rows past the end repeat the last one and are not stored
    const uint32_t ra = min(row, M - 1);
    const uint8_t *const pa = codes + ra * P;
    i32x4_t acc = {};
    for (uint32_t g = 4 * wave; g < granules; g += 4 * kFewWaves) {
        i32x4_t next[4];
        load(g + 4 * kFewWaves, next);
#pragma unroll
        for (uint32_t t4 = 0; t4 < 4; t4++) {
            // past the end of the row fb is zeros
            const uint32_t piece = 4 * min(g + t4, granules - 1) + quarter;
            const i32x4_t fa = *(const i32x4_t *)(pa + (piece ^ (ra & 7)) * 16);
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[t4], fa, acc, 0, 0, 0);
        }
#pragma unroll
        for (int t4 = 0; t4 < 4; t4++) fb[t4] = next[t4];
    }
    sums[wave][lane] = acc;
    __syncthreads();
    if (wave != 0) return;
    // a lane's 4 sums are consecutive n of one m
#pragma unroll
    for (int w = 1; w < kFewWaves; w++) acc += sums[w][lane];
    const int64_t n = n0 + 4 * quarter;
    if (row >= M || n >= N) return;
    const int count = N - n < 4 ? (int)(N - n) : 4;
    float r[4] = {};
#pragma unroll
    for (int j = 0; j < 4; j++)
        if (j < count) r[j] = scaled<false>(acc[j], marks[row], bs[n + j]);
    store4<XT>(y, row * ldy + n, count, r);
}

template <int XT, int V>
hipError_t run_few(const void *x, int64_t ldx, int64_t M, int64_t K, const uint8_t *b, const float *bs, int64_t N,
                   int64_t granules, void *y, int64_t ldy, hipStream_t st) {
    hipLaunchKernelGGL((k_int8_linear_rows<XT, V>), dim3((unsigned)((N + 15) / 16)), dim3(kFewThreads),
                       (unsigned)(M * granules * 64), st, x, ldx, (int)M, K, b, bs, N, (uint32_t)granules, y, ldy);
    return hipGetLastError();
}

template <int XT>
hipError_t few_rows(const void *x, int64_t ldx, int64_t M, int64_t K, const uint8_t *b, const float *bs, int64_t N,
                    int64_t stages, void *y, int64_t ldy, hipStream_t st) {
    const int64_t granules = 2 * stages, teams = M <= 1 ? 1 : M <= 2 ? 2 : M <= 4 ? 4 : 8;
    const int64_t each = (granules * 8 + kFewThreads / teams - 1) / (kFewThreads / teams);   // pieces a lane
    if (each <= 1) return run_few<XT, 1>(x, ldx, M, K, b, bs, N, granules, y, ldy, st);
    if (each <= 2) return run_few<XT, 2>(x, ldx, M, K, b, bs, N, granules, y, ldy, st);
    if (each <= 4) return run_few<XT, 4>(x, ldx, M, K, b, bs, N, granules, y, ldy, st);
    if (each <= 8) return run_few<XT, 8>(x, ldx, M, K, b, bs, N, granules, y, ldy, st);
    if (each <= 16) return run_few<XT, 16>(x, ldx, M, K, b, bs, N, granules, y, ldy, st);
    return hipErrorInvalidValue;
}

// which form takes a product that is not one for few rows: the cheapest
constexpr Form kForms[] = {
    {64, 128, 512, 29, 44, 300},       // 512 x 4096, K = 4096: 18.7 us, tiles of 128 24.4
    {128, 128, 512, 75, 103, 400},     // 2048 x 4096, K = 14336: 120 us, tiles of 64 201, of 256 152
    {256, 128, 256, 125, 170, 1100},   // 4096 x 4096, K = 4096: 65 us, tiles of 128 76
};

template <int CT>
hipError_t run_matmul(const uint8_t *a, const float *as, const uint8_t *b, const float *bs, int64_t M, int64_t N,
                      int64_t stages, void *c, int64_t ldc, int *work, hipStream_t st) {
    const int slices = work ? int8_matmul_slices(M, N, stages) : 1;
    if (slices > 1) {
        const hipError_t e = run_tiled<1, 1, F32, true>(a, as, b, bs, M, N, stages, work, N, st, slices);
        if (e != hipSuccess) return e;
        const dim3 grid((unsigned)((N + 4 * kThreads - 1) / (4 * kThreads)), (unsigned)M);
        hipLaunchKernelGGL((k_int8_matmul_join<CT>), grid, dim3(kThreads), 0, st, work, slices, as, bs, M, N, c, ldc);
        return hipGetLastError();
    }
    // Few rows: one pass over B by as many work-groups as it has 16 rows, unless that many
    // rows of A make it the slower (us warm and cold, and with tiles of 64: 1 x 14336, K = 4096
    // 13.3 and 15.3, 12.2 and 17.9; 16 x 14336, K = 4096 17.4 and 19.9, 12.6 and 18.1; 16 x 4096,
    // K = 4096 6.4 and 7.9, 10.5 and 12.9); also for more rows where the tiles would leave most
    // of the GPU idle and K is short (77 x 1001, K = 1111: 4.2 and 4.7, 6.0 and 6.5; 48 x 4096,
    // K = 4096: 12.7, 11.1 warm).
    const int64_t small = kForms[0].tiles(M, N), granules = 2 * stages;
    const bool rows = (N + 15) / 16 <= kMaxGroups / 2;
    if (rows && (M <= 8 || (M <= 16 && small < 160))) return run_rows<1, 1, CT>(a, as, b, bs, M, N, granules, c, ldc, st);
    if (rows && ((M <= 32 && small < 160) || (small <= 64 && stages <= 16)))
        return run_rows<2, 1, CT>(a, as, b, bs, M, N, granules, c, ldc, st);
    const auto price = [&](int f) { return kForms[f].price(kForms[f].tiles(M, N), stages); };
    const int64_t p64 = price(0), p128 = price(1), p256 = price(2);
    if (p64 <= p128 && p64 <= p256) return run_tiled<1, 1, CT>(a, as, b, bs, M, N, stages, c, ldc, st);
    if (p128 <= p256) return run_tiled<2, 2, CT>(a, as, b, bs, M, N, stages, c, ldc, st);
    return run_tiled<4, 4, CT>(a, as, b, bs, M, N, stages, c, ldc, st);
}

}  // namespace

// A long K and too few tiles for the GPU: slices of K, each a share of the work-groups,
// added up in a second launch (us without and with: 64 x 4096, K = 14336 29 and 18.5; 128 x
// 4096, K = 14336 29.5 and 23; 32 x 4096, K = 14336 22 and 17.5; 64 x 512, K = 28672 30 and 16.3;
// 320 x 1000, K = 9000 20.4 and 16.7; but 64 x 4096, K = 4096 11 both; 256 x 4096, K = 14336 32
// and 33).
int int8_matmul_slices(int64_t M, int64_t N, int64_t stages) {
    const int64_t rows = (M + 63) / 64, cols = (N + 63) / 64;
    if (M <= 16 || N < 1 || rows > 128 || cols > 128 || rows * cols > 128 || stages < 64) return 1;
    return (int)std::min<int64_t>(8, 256 / (rows * cols));
}

// Up to 8 rows that fit LDS, while what every work-group repeats (M P codes, N / 16 times) takes
// about what the launch does that it saves.  us in one launch and in two, in a graph with W in
// the last cache, there from HBM, and called eagerly, where two are bound by the host:
//   1 x 4096, K = 4096    6.6 and 7.6
//   1 x 14336, K = 4096   15.5 and 16.2
//   2 x 4096, K = 4096    6.3 and 7.2    8.6 and 9.5     6.1 and 12.2
//   4 x 8192, K = 4096    9.4 and 10.7   12.2 and 12.6   9.0 and 11.6
//   8 x 1024, K = 4096    7.1 and 7.8    8.6 and 8.6     7.2 and 11.5
//   8 x 4096, K = 4096    8.5 and 8.4    10.9 and 9.9    8.3 and 11.6
//   8 x 2048, K = 6144    9.8 and 9.5    13.4 and 11.1   9.7 and 12.2
// beyond the bound on N:
//   8 x 6144, K = 4096    12.1 and 11.9  13.3 and 12.7   11.9 and 12.3
//   8 x 14336, K = 4096   22.9 and 18.3  25.1 and 19.0   22.4 and 17.8
//   4 x 14336, K = 4096   17.6 and 17.2  19.0 and 17.9   17.2 and 16.9
// So 8 rows at the bound give up a tenth (a fifth where K is longest) in a graph with W from HBM
// for a quarter of an eager call.
bool int8_linear_few(int64_t M, int64_t N, int64_t stages) {
    const int64_t teams = M <= 1 ? 1 : M <= 2 ? 2 : M <= 4 ? 4 : 8, P = stages * 128;
    if (M < 1 || M > 8 || stages < 1 || teams * P > kFewBytes || (N + 15) / 16 > kMaxGroups / 2) return false;
    return M == 1 || N <= ((int64_t)1 << 27) / (M * P);
}

hipError_t launch_int8_linear_rows(const void *x, int xt, int64_t ldx, int64_t M, int64_t K, const uint8_t *b,
                                   const float *bs, int64_t N, int64_t stages, void *y, int64_t ldy, hipStream_t st) {
    if (xt == BF16) return few_rows<BF16>(x, ldx, M, K, b, bs, N, stages, y, ldy, st);
    if (xt == F16) return few_rows<F16>(x, ldx, M, K, b, bs, N, stages, y, ldy, st);
    return hipErrorInvalidValue;
}

hipError_t launch_int8_matmul(const uint8_t *a, const float *as, const uint8_t *b, const float *bs, int64_t M,
                              int64_t N, int64_t stages, void *c, int ct, int64_t ldc, int *work, hipStream_t st) {
    switch (ct) {
    case F16: return run_matmul<F16>(a, as, b, bs, M, N, stages, c, ldc, work, st);
    case BF16: return run_matmul<BF16>(a, as, b, bs, M, N, stages, c, ldc, work, st);
    case F32: return run_matmul<F32>(a, as, b, bs, M, N, stages, c, ldc, work, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qcp
