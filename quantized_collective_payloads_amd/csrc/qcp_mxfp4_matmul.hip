// qcp_mxfp4_matmul.hip -- C = A B^T on MXFP4 payloads: A is [M, K], B is [N, K],
// both with K along their rows, C [M, N] in fp32, bf16 or fp16.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies two 32 x 64 pieces of E2M1 codes,
// each lane supplying 32 codes of one row (16 bytes) and that block's E8M0 scale;
// it accumulates in fp32, and its products carry the scales, so the payload is
// never decoded.  Which 32 of K a lane brings is free as long as both operands
// agree: of a granule of 128 (64 bytes of a row), the lower half-wave takes the
// first 32 bytes and the upper one the last, and two instructions use them up.
// The row's 4 scale bytes are one dword; its half is shifted down once per
// granule, and the instruction picks the byte.
//
// Measured, by the GPU's clock: 8192 x 8192, K = 28672 850 to 960 us (4.5 to 4.0 PFLOP/s);
// 2048 x 14336, K = 4096 78 us (3.1), 81 with operands from HBM; 1 x 14336, K = 4096 7.4 us
// with B in the last cache, 8.7 from HBM (3.6 TB/s).
#include <algorithm>

#include "qcp_matmul.h"
#include "qcp_ops.h"

namespace qcp {

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

template <int T>
__device__ __forceinline__ f32x16_t mma(u32x4_t a, uint32_t sa, u32x4_t b, uint32_t sb, f32x16_t c) {
    const i32x8_t av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const i32x8_t bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, T, (int)sa, T, (int)sb);
}

// A wave's 64 x 64 of C from fragments of 32 rows
template <int CT>
__device__ __forceinline__ void store_wave(const f32x16_t (&acc)[2][2], void *c, int64_t ldc, int64_t m0, int64_t n0,
                                           int lane, int64_t M, int64_t N) {
    const bool whole = m0 + 64 <= M && n0 + 64 <= N;
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++)
            store_fragment<CT>(acc[i][j], c, ldc, m0 + 32 * i + (lane & 31), n0 + 32 * j, lane >> 5, M, N, whole);
}

// K of G = 1 to 3 granules: 128 x 128 of C per work-group.  The payload rows of a tile are
// one run of memory, 16 KB of A and B per granule, that goes to LDS at once; 4 waves,
// 2 x 2, then compute 64 x 64 each from fragments there.  Rows past the end repeat the last
// one and are not stored.
// Bound: writing C.  14336 x 4096 to bf16, 23 us of writing: K = 128, 256, 384 27, 32 and
// 36 us; with fragments straight from memory 31, 48 and 56 (both operands read twice, in
// pieces of 16 bytes), and that a granule at a time with 8-byte stores 47, 63 and 70.
//
// LDS holds a row's pieces of 16 bytes in an order that gives the 16 rows that a fragment
// read touches in a cycle all 64 banks: rows are 64 G bytes apart, so for odd G 4
// consecutive rows lie side by side in the banks, and the low bits of the piece follow row / 4;
// for G = 2 2 rows do, and the piece's 3 bits follow row / 2.
template <int G, int CT>
__global__ __launch_bounds__(kThreads) void k_mx_matmul_short(
    const uint8_t *__restrict__ a, const uint8_t *__restrict__ as, const uint8_t *__restrict__ b,
    const uint8_t *__restrict__ bs, int64_t M, int64_t N, uint32_t m_tiles, uint32_t n_tiles, void *__restrict__ c,
    int64_t ldc) {
    constexpr int kPieces = 4 * G, kSide = 128 * 64 * G;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kSide];
    const TilePlace t = tile_place(__builtin_amdgcn_workgroup_id_x(), m_tiles, n_tiles);
    const int64_t mt = (int64_t)t.m * 128, nt = (int64_t)t.n * 128;
    const int tid = (int)__builtin_amdgcn_workitem_id_x(), wave = tid >> 6, lane = lane_id();
    auto where = [](int row, int piece) __attribute__((always_inline)) {
        const int x = G == 2 ? (row >> 1) & 7 : (row >> 2) & 3;
        return row * 64 * G + (piece ^ x) * 16;
    };
    u32x4_t v[2][2 * G];
#pragma unroll
    for (int k = 0; k < 2 * G; k++) {
        const int at = tid + kThreads * k, row = at / kPieces, piece = at % kPieces;
        v[0][k] = *(const u32x4_t *)(a + min(mt + row, M - 1) * (64 * G) + piece * 16);
        v[1][k] = *(const u32x4_t *)(b + min(nt + row, N - 1) * (64 * G) + piece * 16);
    }
    const int row = lane & 31, half = lane >> 5, ra = (wave & 1) * 64 + row, rb = (wave >> 1) * 64 + row;
    uint32_t sa[2][G], sb[2][G];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int g = 0; g < G; g++) {
            sa[i][g] = *(const uint32_t *)(as + min(mt + ra + 32 * i, M - 1) * (4 * G) + 4 * g) >> (16 * half);
            sb[i][g] = *(const uint32_t *)(bs + min(nt + rb + 32 * i, N - 1) * (4 * G) + 4 * g) >> (16 * half);
        }
#pragma unroll
    for (int k = 0; k < 2 * G; k++) {
        const int at = tid + kThreads * k, to = where(at / kPieces, at % kPieces);
        *(u32x4_t *)(lds + to) = v[0][k];
        *(u32x4_t *)(lds + kSide + to) = v[1][k];
    }
    __syncthreads();
    f32x16_t acc[2][2] = {};
#pragma unroll
    for (int g = 0; g < G; g++) {
        u32x4_t fa[2][2], fb[2][2];
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int u = 0; u < 2; u++) {
                fa[i][u] = *(const u32x4_t *)(lds + where(ra + 32 * i, 4 * g + 2 * half + u));
                fb[i][u] = *(const u32x4_t *)(lds + kSide + where(rb + 32 * i, 4 * g + 2 * half + u));
            }
        // B first: a lane then holds 4 consecutive n of one m per group of registers
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int j = 0; j < 2; j++) {
                acc[i][j] = mma<0>(fb[j][0], sb[j][g], fa[i][0], sa[i][g], acc[i][j]);
                acc[i][j] = mma<1>(fb[j][1], sb[j][g], fa[i][1], sa[i][g], acc[i][j]);
            }
    }
    store_wave<CT>(acc, c, ldc, mt + (wave & 1) * 64, nt + (wave >> 1) * 64, lane, M, N);
}

// The plain form, for K from 2^25 on, whose rows are beyond the 32-bit offsets within a
// tile of the kernels below, and for more than 2^24 tiles of 64 x 64: a wave computes 64 x 64 of C from 2 + 2 fragments per granule,
// read straight from memory; a work-group's 4 waves make 128 x 128.
template <int CT>
__global__ __launch_bounds__(kThreads) void k_mx_matmul(const uint8_t *__restrict__ a,
                                                        const uint8_t *__restrict__ as,
                                                        const uint8_t *__restrict__ b,
                                                        const uint8_t *__restrict__ bs, int64_t M,
                                                        int64_t N, int64_t granules, uint32_t m_tiles,
                                                        void *__restrict__ c, int64_t ldc) {
    const uint32_t wg = __builtin_amdgcn_workgroup_id_x();
    const int wave = (int)(__builtin_amdgcn_workitem_id_x() >> 6), lane = lane_id();
    const int64_t m0 = (int64_t)(wg % m_tiles) * 128 + (wave & 1) * 64;
    const int64_t n0 = (int64_t)(wg / m_tiles) * 128 + (wave >> 1) * 64;
    if (m0 >= M || n0 >= N) return;
    const int row = lane & 31, half = lane >> 5;
    const uint8_t *pa[2], *pb[2], *qa[2], *qb[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int64_t m = min(m0 + 32 * i + row, M - 1), n = min(n0 + 32 * i + row, N - 1);
        pa[i] = a + m * granules * 64 + 32 * half;
        pb[i] = b + n * granules * 64 + 32 * half;
        qa[i] = as + m * granules * 4;
        qb[i] = bs + n * granules * 4;
    }
    f32x16_t acc[2][2] = {};
    for (int64_t g = 0; g < granules; g++) {
        u32x4_t fa[2][2], fb[2][2];
        uint32_t sa[2], sb[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
#pragma unroll
            for (int t = 0; t < 2; t++) {
                fa[i][t] = *(const u32x4_t *)(pa[i] + g * 64 + 16 * t);
                fb[i][t] = *(const u32x4_t *)(pb[i] + g * 64 + 16 * t);
            }
            sa[i] = *(const uint32_t *)(qa[i] + g * 4) >> (16 * half);
            sb[i] = *(const uint32_t *)(qb[i] + g * 4) >> (16 * half);
        }
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int j = 0; j < 2; j++) {
                acc[i][j] = mma<0>(fb[j][0], sb[j], fa[i][0], sa[i], acc[i][j]);
                acc[i][j] = mma<1>(fb[j][1], sb[j], fa[i][1], sa[i], acc[i][j]);
            }
    }
    store_wave<CT>(acc, c, ldc, m0, n0, lane, M, N);
}

// ---------------------------------------------------------------------------
// 64*FM x 64*FN of C per work-group, staged through LDS.
// ---------------------------------------------------------------------------
// Bound: the matrix cores' clock and the waits between their instructions.  Normal values
// multiplied in registers alone reach 6.5 PFLOP/s, zeros 9.7: the clock follows the energy
// (here 1.3 to 1.8 GHz against 2.1).  8192 x 8192, K = 28672 takes 860 us and 710 (4.5 and
// 5.4): in cycles the cores are busy 59 to 65% and 57%, and a wave waits at barriers and
// for memory 20% and 25% of the time.  Four waves, 2 x 2, hold 32*FM x 32*FN each.  At
// 4 x 4 that is 256 x 256 per work-group and 256 accumulators, one wave per SIMD: a
// phase is 32 instructions of 32 cycles on 16 KB of operands, a quarter of what LDS
// gives.  At 2 x 2, 128 x 128, two work-groups share a CU: twice the operand traffic
// per product, but four times as many tiles, and one's stores run beside the
// other's products.  A stage is 256 of K: 128 bytes of each operand row, whole cache
// lines, in one of two slots; with two, the barrier of each stage waits for all copies
// in flight (1 x 1 has four slots, and two stages' copies stay in flight).
//
// Within a stage the lower half-wave takes the first granule (64 bytes of its row)
// and the upper one the second, so a lane's four blocks have their scales in one
// dword and the instruction picks the byte.  A stage is two phases of 128 of K.
//
// Copies go from memory to LDS without registers (buffer_load ... lds), and run beside
// the matrix instructions of a stage or more: with the
// fragments of phase 0 in registers a wave issues its products and reads those of
// phase 1; one barrier, at which every wave has read this stage and holds no
// outstanding copy of the next; the copies of the stage after that go into the
// slot just freed; and the products of phase 1 run beside the reads of the next
// stage's phase 0.
//
// LDS holds a row's 8 pieces of 16 bytes in the order piece ^ (row / 2 % 8): the
// copy permutes its source addresses, so that a fragment read, 16 rows of 128 bytes
// at the same piece a cycle, touches each of the 64 banks once.  Scales are copied
// for 4 granules at a time, 16 bytes a row, into slots of their own.
//
// A work-group walks several tiles: the copies of the next one's first stages go out
// before the results of this one, and its stores stay in flight into the next tile
// (14336 x 4096, K = 2048: 119 us for a work-group per tile with 8-byte stores, 109 so).
// At 4 x 4 less overlaps than this order says: the compiler keeps 41 vector registers (66
// with fp32 results) in scratch memory around a tile.  None is reloaded in the loop of
// stages, but each reload elsewhere waits for everything in flight, so the results
// follow the copies' arrival and the next tile's first products that of the results.
// The forms of 1 x 1 and 2 x 2 keep all in registers.
//
// Rows past the end repeat the last row.  Windows in K are pulled back to end
// with the row: a last odd granule comes as the second one of its window, and is
// multiplied by itself as in the kernel above.
template <int FM, int FN> struct tgeom {
    static constexpr int TM = 64 * FM, TN = 64 * FN;       // C per work-group
    static constexpr int slots = FM * FN == 1 ? 4 : 2;     // stages in LDS
    static constexpr int rows = TM + TN;
    static constexpr int slot = rows * 128;                // codes of A and B, one stage
    static constexpr int mark_slot = rows * 16;            // scales of A and B, 4 granules
    static constexpr int lds = slots * (slot + mark_slot); // 144 KB at 4 x 4, 72 KB at 2 x 2 and 1 x 1
    static constexpr int ops = 2 * FM * FN;                // products per phase and wave
    static constexpr int reads = 2 * (FM + FN);            // fragment pieces per phase
    static constexpr int copies = rows / 32;               // per stage and wave, 8 rows each
    static constexpr int waves_per_simd = FM * FN <= 4 ? 2 : 1;
    // 16-byte stores of a wave's whole results
    template <int CT> static constexpr int stores() { return FM * FN * 16 * dtype_traits<CT>::bytes / 16; }
    static constexpr int ahead = (slots - 2) * copies;     // copies of stages beyond the next
};

template <int FM, int FN> struct Fragments {
    u32x4_t a[FM][2], b[FN][2];
};
template <int FM, int FN> struct Scales {
    uint32_t a[FM], b[FN];
};

// SLICED: the tiles are those of `slices` parts of K, one part after the other; c is fp32,
// an M x N for each.
template <int FM, int FN, int CT, bool SLICED>
__global__ __launch_bounds__(kThreads, (tgeom<FM, FN>::waves_per_simd)) void k_mx_matmul_tiled(
    const uint8_t *__restrict__ a, const uint8_t *__restrict__ as, const uint8_t *__restrict__ b,
    const uint8_t *__restrict__ bs, int64_t M, int64_t N, uint32_t row_granules, uint32_t slices, uint32_t m_tiles,
    uint32_t n_tiles, uint32_t groups, void *__restrict__ c, int64_t ldc) {
    using Gm = tgeom<FM, FN>;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[Gm::lds];
    const int tid = (int)__builtin_amdgcn_workitem_id_x();
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = lane_id();

    const uint32_t tiles = m_tiles * n_tiles * (SLICED ? slices : 1);
    const uint32_t row_bytes = row_granules * 64, mark_bytes = row_granules * 4;
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
    uint32_t granules = row_granules, stages = (granules + 1) / 2, slice = 0;   // of the tile

    // the tile that is being copied.  Copies: a wave brings a quarter of each operand's
    // rows, 8 rows at a time.  Scales: 64 rows at a time, FM pieces of A, then FN of B,
    // dealt to the waves (the last piece twice where they do not divide).  No branches:
    // the loop below stays one basic block, in which the order written is kept.
    constexpr int mark_rounds = (FM + FN + 3) / 4;
    int64_t m0, n0;
    i32x4_t ra, rb, rs[mark_rounds];
    uint32_t vs[mark_rounds], mark_at[mark_rounds], m_rows, n_rows;
    auto set_tile = [&](uint32_t t) __attribute__((always_inline)) {
        uint32_t skip = 0;                                   // granules before the slice
        if constexpr (SLICED) {
            slice = t / (m_tiles * n_tiles);
            t -= slice * (m_tiles * n_tiles);
            const uint32_t pairs = row_granules / 2, each = pairs / slices, over = pairs % slices;
            skip = 2 * (slice * each + min(slice, over));
            granules = slice + 1 == slices ? row_granules - skip : 2 * (each + (slice < over ? 1 : 0));
            stages = (granules + 1) / 2;
        }
        const TilePlace at = tile_place(t, m_tiles, n_tiles);
        m0 = (int64_t)at.m * Gm::TM;
        n0 = (int64_t)at.n * Gm::TN;
        m_rows = (uint32_t)min(M - m0, (int64_t)Gm::TM);
        n_rows = (uint32_t)min(N - n0, (int64_t)Gm::TN);
        ra = buffer_of(a + m0 * row_bytes + skip * 64, (uint64_t)m_rows * row_bytes - skip * 64);
        rb = buffer_of(b + n0 * row_bytes + skip * 64, (uint64_t)n_rows * row_bytes - skip * 64);
        const i32x4_t rsa = buffer_of(as + m0 * mark_bytes + skip * 4, (uint64_t)m_rows * mark_bytes - skip * 4);
        const i32x4_t rsb = buffer_of(bs + n0 * mark_bytes + skip * 4, (uint64_t)n_rows * mark_bytes - skip * 4);
        static_for<mark_rounds>([&](auto I) __attribute__((always_inline)) {
            constexpr int k = I;
            const int q = min(wave + 4 * k, FM + FN - 1);
            const bool of_a = FM >= 4 * k + 4 || (FM > 4 * k && q < FM);
            mark_at[k] = q * 1024;
            vs[k] = (of_a ? min((uint32_t)(64 * q + lane), m_rows - 1) : min((uint32_t)(64 * (q - FM) + lane), n_rows - 1)) * mark_bytes;
            rs[k] = of_a ? rsa : rsb;
        });
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
    auto copy_marks = [&](uint32_t to, uint32_t k) __attribute__((always_inline)) {
        static_for<mark_rounds>([&](auto I) __attribute__((always_inline)) {
            copy_to_lds(to + mark_at[I], vs[I], rs[I], k);
        });
    };
    constexpr uint32_t kMarks = Gm::slots * Gm::slot;      // where the scales begin
    auto slot_of = [&](uint32_t s) __attribute__((always_inline)) { return (s & (Gm::slots - 1)) * Gm::slot; };
    auto mark_slot_of = [&](uint32_t s) __attribute__((always_inline)) {
        return kMarks + ((s >> 1) & (Gm::slots - 1)) * Gm::mark_slot;
    };
    auto copy_stage = [&](uint32_t s) __attribute__((always_inline)) {
        const uint32_t k = min(2 * s, granules - 2) * 64;
        static_for<Gm::copies>([&](auto I) __attribute__((always_inline)) { copy(I, base + slot_of(s), k); });
        if ((s & 1) == 0) copy_marks(base + mark_slot_of(s), min(2 * s, granules - 4) * 4);
    };

    // fragments: wave w computes rows 32*FM*(w&1) of A against rows 32*FN*(w>>1) of B
    const int r = lane & 31, half = lane >> 5, x = (lane >> 1) & 7;
    const uint32_t arow = (wave & 1) * 32 * FM + r, brow = Gm::TM + (wave >> 1) * 32 * FN + r;
    // where piece 4 * half of the first fragment lies in slot 0; pieces p and q of a row
    // differ by the bits of 16 * (p ^ q)
    const uint32_t a_at = base + arow * 128 + ((4 * half) ^ x) * 16;
    const uint32_t b_at = base + brow * 128 + ((4 * half) ^ x) * 16;
    const uint32_t a_marks = base + arow * 16, b_marks = base + brow * 16;   // + mark_slot_of
    // the n-th of the fragments' pieces at la, lb and those at the piece beside, in the
    // order the products use them
    using Frag = Fragments<FM, FN>;
    using Scale = Scales<FM, FN>;
    auto read = [&](auto I, uint32_t la, uint32_t lb, Frag &f) __attribute__((always_inline)) {
        constexpr int n = I, u = n / (FM + FN), q = n % (FM + FN);
        if constexpr (q < FN) f.b[q][u] = lds16((lb ^ (16 * u)) + q * 4096);
        else f.a[q - FN][u] = lds16((la ^ (16 * u)) + (q - FN) * 4096);
    };
    // pieces p and p ^ 1 beyond 4 * half of the slot of stage s
    auto read_all = [&](uint32_t s, uint32_t p, Frag &f) __attribute__((always_inline)) {
        const uint32_t la = (a_at ^ (16 * p)) + slot_of(s), lb = (b_at ^ (16 * p)) + slot_of(s);
        static_for<Gm::reads>([&](auto I) __attribute__((always_inline)) { read(I, la, lb, f); });
    };
    // the scales of one granule, at dword k of the group of stage s
    auto read_scales = [&](uint32_t s, uint32_t k, Scale &e) __attribute__((always_inline)) {
        const uint32_t at = mark_slot_of(s) + 4 * k;
#pragma unroll
        for (int i = 0; i < FM; i++) e.a[i] = lds4(a_marks + at + i * 512);
#pragma unroll
        for (int i = 0; i < FN; i++) e.b[i] = lds4(b_marks + at + i * 512);
    };
    const uint32_t upper = half ? ~0u : 0u;                // all bits in the upper half-wave
    auto pick = [&](uint32_t lo, uint32_t up) __attribute__((always_inline)) { return (lo & ~upper) | (up & upper); };
    auto window = [&](uint32_t s) __attribute__((always_inline)) { return min((2 * s) & ~3u, granules - 4); };   // first granule of s's scales

    f32x16_t acc[FM][FN];
    Frag f, h;
    Scale e;
    u32x4_t ga[FM], gb[FN];
    // the n-th product of phase P
    auto product = [&](auto P, auto I, const Frag &v) __attribute__((always_inline)) {
        constexpr int ph = P, n = I, u = n / (FM * FN), i = n / FN % FM, j = n % FN;
        acc[i][j] = mma<2 * ph + u>(v.b[j][u], e.b[j], v.a[i][u], e.a[i], acc[i][j]);
    };
    auto products = [&](auto P, const Frag &v) __attribute__((always_inline)) {
        static_for<Gm::ops>([&](auto I) __attribute__((always_inline)) { product(P, I, v); });
    };
    // the products of phase P of a stage, in the order written: between them the
    // reads of the next phase's fragments, from the slot at `from`, and with COPY the
    // copies of stage `next`, so the matrix cores never wait for the rest to issue.
    // GROUP_READ: also the scales of the group at `marks`; GROUP_COPY: the copy of
    // those of stage `next`.
    auto phase = [&](auto P, const Frag &now, Frag &then, uint32_t from, auto COPY, uint32_t next,
                     auto GROUP_READ, uint32_t marks, auto GROUP_COPY) __attribute__((always_inline)) {
        constexpr int S = Gm::ops;
        const uint32_t to = base + slot_of(next), k = next * 128;
        uint32_t la = a_at, lb = b_at;
        asm volatile("" : "+v"(la), "+v"(lb));   // addresses made here, not kept for every phase
        la = (la ^ (P ? 0 : 32)) + from;
        lb = (lb ^ (P ? 0 : 32)) + from;
        static_for<S>([&](auto I) __attribute__((always_inline)) {
            constexpr int n = I;
            product(P, I, now);
            // reads in the first half of the phase, copies too
            constexpr int r0 = n * 2 * Gm::reads / S, r1 = (n + 1) * 2 * Gm::reads / S;
            static_for<r1 - r0>([&](auto Q) __attribute__((always_inline)) {
                constexpr int q = r0 + Q, g = q - Gm::reads;
                if constexpr (q < Gm::reads) read(std::integral_constant<int, q>{}, la, lb, then);
                else if constexpr (GROUP_READ && g < FN) gb[g] = lds16(b_marks + marks + g * 512);
                else if constexpr (GROUP_READ && g < FN + FM) ga[g - FN] = lds16(a_marks + marks + (g - FN) * 512);
            });
            if constexpr (COPY) {
                constexpr int c0 = n * 2 * Gm::copies / S, c1 = (n + 1) * 2 * Gm::copies / S;
                static_for<c1 - c0>([&](auto Q) __attribute__((always_inline)) {
                    constexpr int q = c0 + Q;
                    if constexpr (q < Gm::copies) copy(std::integral_constant<int, q>{}, to, k);
                });
                if constexpr (GROUP_COPY && n == S / 2) copy_marks(base + mark_slot_of(next), k / 16);
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    using no = std::integral_constant<int, 0>;
    using yes = std::integral_constant<int, 1>;

    auto copy_first = [&]() __attribute__((always_inline)) {
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
            for (int j = 0; j < FN; j++) acc[i][j] = f32x16_t{};
        read_all(0, 0, f);
        read_scales(0, half, e);

        // two stages at a time while there are enough more to copy: every window then lies
        // where the stage number says, and `ahead` copies follow those waited for
        uint32_t s = 0;
        const uint32_t full = granules / 2;
        if (full >= 2 + Gm::slots) {
#pragma unroll
            for (int i = 0; i < FM; i++) ga[i] = lds16(a_marks + kMarks + i * 512);
#pragma unroll
            for (int i = 0; i < FN; i++) gb[i] = lds16(b_marks + kMarks + i * 512);
            for (; s + 2 + Gm::slots <= full; s += 2) {
                const uint32_t s0 = slot_of(s), s1 = slot_of(s + 1), s2 = slot_of(s + 2);
                phase(no{}, f, h, s0, no{}, 0, no{}, 0, no{});
                wait_and_meet<Gm::ahead>();
                phase(yes{}, h, f, s1, yes{}, s + Gm::slots, no{}, 0, yes{});
#pragma unroll
                for (int i = 0; i < FM; i++) e.a[i] = pick(ga[i].z, ga[i].w);
#pragma unroll
                for (int i = 0; i < FN; i++) e.b[i] = pick(gb[i].z, gb[i].w);
                phase(no{}, f, h, s1, no{}, 0, no{}, 0, no{});
                wait_and_meet<Gm::ahead>();
                phase(yes{}, h, f, s2, yes{}, s + 1 + Gm::slots, yes{}, mark_slot_of(s + 2), no{});
#pragma unroll
                for (int i = 0; i < FM; i++) e.a[i] = pick(ga[i].x, ga[i].y);
#pragma unroll
                for (int i = 0; i < FN; i++) e.b[i] = pick(gb[i].x, gb[i].y);
            }
            // the group's scales may have come from a window that is pulled back
            read_scales(s, 2 * s - window(s) + half, e);
        }
        for (; s < full; s++) {
            read_all(s, 2, h);
            products(no{}, f);
            wait_and_meet<0>();
            if (s + Gm::slots < stages) copy_stage(s + Gm::slots);
            products(yes{}, h);
            if (s + 1 < full) {
                read_all(s + 1, 0, f);
                read_scales(s + 1, 2 * s + 2 - window(s + 1) + half, e);
            }
        }
        if (granules & 1) {                                  // the last granule, alone: pieces 4 + 2 * half
            read_all(full, 4 ^ (6 * half), f);
            read_scales(full, granules - 1 - window(full), e);
#pragma unroll
            for (int i = 0; i < FM; i++) e.a[i] >>= 16 * half;
#pragma unroll
            for (int i = 0; i < FN; i++) e.b[i] >>= 16 * half;
            products(no{}, f);
        }

        // the next tile's first copies go out before this one's results
        const int64_t m_done = m0 + (wave & 1) * 32 * FM + r, n_done = n0 + (wave >> 1) * 32 * FN;
        const bool whole = m0 + Gm::TM <= M && n0 + Gm::TN <= N;
        void *const to = SLICED ? (float *)c + slice * M * N : c;
        tile += groups;
        const bool more = tile < tiles;
        if (more) {
            wait_lds_and_meet();                             // every wave is done with the slots
            set_tile(tile);
            copy_first();
        }
        static_for<FM * FN>([&](auto I) __attribute__((always_inline)) {
            constexpr int i = I / FN, j = I % FN;
            store_fragment<CT>(acc[i][j], to, ldc, m_done + 32 * i, n_done + 32 * j, half, M, N, whole);
        });
        if (!more) break;
        // the copies are older than the stores, of which a whole tile has `stores` at least
        if (whole) wait_and_meet<(Gm::template stores<CT>() < 63 ? Gm::template stores<CT>() : 63)>();
        else wait_and_meet<0>();
    }
}

template <int FM, int FN, int CT, bool SLICED = false>
hipError_t run_tiled(const uint8_t *a, const uint8_t *as, const uint8_t *b, const uint8_t *bs, int64_t M,
                     int64_t N, int64_t granules, void *c, int64_t ldc, hipStream_t st, int slices = 1) {
    using Gm = tgeom<FM, FN>;
    const int64_t mt = (M + Gm::TM - 1) / Gm::TM, nt = (N + Gm::TN - 1) / Gm::TN;
    // as many work-groups as the GPU holds walk the tiles (a multiple of 8, so that each
    // stays on its XCD's tiles)
    const unsigned groups = (unsigned)std::min<int64_t>(mt * nt * slices, kCUs * Gm::waves_per_simd);
    hipLaunchKernelGGL((k_mx_matmul_tiled<FM, FN, CT, SLICED>), dim3(groups), dim3(kThreads), 0, st, a, as, b, bs, M,
                       N, (uint32_t)granules, (uint32_t)slices, (uint32_t)mt, (uint32_t)nt, groups, c, ldc);
    return hipGetLastError();
}

// The sum of the slices, in their order, rounded once: 4 columns a lane.
template <int CT>
__global__ __launch_bounds__(kThreads) void k_mx_matmul_join(const float *__restrict__ parts, int slices, int64_t M,
                                                             int64_t N, void *__restrict__ c, int64_t ldc) {
    typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
    const int64_t m = group_y();
    const int64_t n = ((int64_t)__builtin_amdgcn_workgroup_id_x() * kThreads + __builtin_amdgcn_workitem_id_x()) * 4;
    if (n >= N) return;
    const int count = N - n < 4 ? (int)(N - n) : 4;
    const float *p = parts + m * N + n;
    float v[4] = {};
    for (int s = 0; s < slices; s++, p += M * N) {
        if (count == 4) {
            const f32x4_any x = *(const f32x4_any *)p;
            v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        } else {
#pragma unroll
            for (int j = 0; j < 3; j++)
                if (j < count) v[j] += p[j];
        }
    }
    store4<CT>(c, m * ldc + n, count, v);
}

// ---------------------------------------------------------------------------
// Few rows of A (a token, a small batch): 16*FA rows against 16*FB rows of B.
// ---------------------------------------------------------------------------
// Bound: reading B once, at these sizes the latency of it (1 x 14336, K = 4096: 31 MB in
// 7.4 us from the last cache, 8.7 from HBM; the smallest calls take 2.5).  v_mfma_scale_f32_16x16x128_f8f6f4 takes 16 rows, so N/16
// work-groups; the WV waves of one deal out K in steps of 512 and add their sums in
// LDS in a fixed order, so a few rows still fill the GPU, without a second launch.  Of a step's 4 granules
// a quarter-wave takes one: a lane reads 64 consecutive bytes of its row and one
// dword of scales, a row of the fragment 256.  Operands go straight to registers, a
// whole step's loads at a time.
template <int T>
__device__ __forceinline__ f32x4_t mma16(u32x4_t a, uint32_t sa, u32x4_t b, uint32_t sb, f32x4_t c) {
    const i32x8_t av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const i32x8_t bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, T, (int)sa, T, (int)sb);
}

template <int F> struct StepOf {
    u32x4_t v[F][4];
    uint32_t s[F];
};

template <int FA, int FB, int WV, int CT>
__global__ __launch_bounds__(64 * WV) void k_mx_matmul_rows(
    const uint8_t *__restrict__ a, const uint8_t *__restrict__ as, const uint8_t *__restrict__ b,
    const uint8_t *__restrict__ bs, int64_t M, int64_t N, int64_t granules, void *__restrict__ c, int64_t ldc) {
    __shared__ f32x4_t sums[WV][FA * FB][64];
    const int wave = __builtin_amdgcn_readfirstlane((int)(__builtin_amdgcn_workitem_id_x() >> 6)), lane = lane_id();
    const int row = lane & 15, quarter = lane >> 4;
    const int64_t n0 = (int64_t)__builtin_amdgcn_workgroup_id_x() * (16 * FB), m0 = group_y() * (16 * FA);
    const uint8_t *pa[FA], *qa[FA], *pb[FB], *qb[FB];
#pragma unroll
    for (int i = 0; i < FA; i++) {
        const int64_t m = min(m0 + 16 * i + row, M - 1) * granules + quarter;
        pa[i] = a + m * 64;
        qa[i] = as + m * 4;
    }
#pragma unroll
    for (int i = 0; i < FB; i++) {
        const int64_t n = min(n0 + 16 * i + row, N - 1) * granules + quarter;
        pb[i] = b + n * 64;
        qb[i] = bs + n * 4;
    }
    auto load = [&](int64_t g, auto &f, const uint8_t *const *p, const uint8_t *const *q, auto F) __attribute__((always_inline)) {
        static_for<F>([&](auto I) __attribute__((always_inline)) {
            constexpr int i = I;
            if (g + quarter < granules) {
#pragma unroll
                for (int t = 0; t < 4; t++) f.v[i][t] = *(const u32x4_t *)(p[i] + g * 64 + 16 * t);
                f.s[i] = *(const uint32_t *)(q[i] + g * 4);
            } else {
#pragma unroll
                for (int t = 0; t < 4; t++) f.v[i][t] = u32x4_t{0, 0, 0, 0};
                f.s[i] = 0;
            }
        });
    };
    f32x4_t acc[FA][FB] = {};
    for (int64_t g = 4 * wave; g < granules; g += 4 * WV) {
        StepOf<FA> fa;
        StepOf<FB> fb;
        load(g, fb, pb, qb, std::integral_constant<int, FB>{});
        load(g, fa, pa, qa, std::integral_constant<int, FA>{});
        static_for<4>([&](auto T) __attribute__((always_inline)) {
            constexpr int t = T;
#pragma unroll
            for (int i = 0; i < FA; i++)
#pragma unroll
                for (int j = 0; j < FB; j++) acc[i][j] = mma16<t>(fb.v[j][t], fb.s[j], fa.v[i][t], fa.s[i], acc[i][j]);
        });
    }
#pragma unroll
    for (int i = 0; i < FA; i++)
#pragma unroll
        for (int j = 0; j < FB; j++) sums[wave][i * FB + j][lane] = acc[i][j];
    __syncthreads();
    // a lane's 4 sums are consecutive n of one m
    for (int k = wave; k < FA * FB; k += WV) {
        f32x4_t v = sums[0][k][lane];
#pragma unroll
        for (int w = 1; w < WV; w++) v += sums[w][k][lane];
        const int64_t m = m0 + 16 * (k / FB) + row, n = n0 + 16 * (k % FB) + 4 * quarter;
        const float r[4] = {v.x, v.y, v.z, v.w};
        if (m < M && n < N) store4<CT>(c, m * ldc + n, N - n < 4 ? (int)(N - n) : 4, r);
    }
}

template <int FA, int FB, int CT>
hipError_t run_rows(const uint8_t *a, const uint8_t *as, const uint8_t *b, const uint8_t *bs, int64_t M,
                    int64_t N, int64_t granules, void *c, int64_t ldc, hipStream_t st) {
    const dim3 grid((unsigned)((N + 16 * FB - 1) / (16 * FB)), (unsigned)((M + 16 * FA - 1) / (16 * FA)));
    // A wave for each step of K up to 4, else 8 (us with 4 and with 8, warm and cold): 1 x
    // 14336, K = 512 2.6 and 2.7, 3.4 and 3.5; 1 x 28672, K = 1024 4.3 and 4.6, 5.5 and 6.6; but
    // 1 x 256, K = 2560 2.7 and 2.7, 3.3 and 3.1; 1 x 4096, K = 14336 7.5 and 6.8, 10.6 and 8.2;
    // 32 x 4096, K = 4096 5.4 and 5.5, 6.8 and 6.4; 1 x 28672, K = 8192 23.9 both, 27.7 and 27.5.
    // 16 waves took 2 to 5% more than 8 from 1 to 512 work-groups (1 x 1024, K = 14336 6.7
    // and 7.6 against 6.5 and 7.4) and a third more beyond, where K is short.  (8 waves: rows
    // of more than 2048 values, of which a payload holds fewer than 2^25, so the grid is small.)
    if (granules <= 16)
        hipLaunchKernelGGL((k_mx_matmul_rows<FA, FB, 4, CT>), grid, dim3(256), 0, st, a, as, b, bs, M, N, granules, c, ldc);
    else
        hipLaunchKernelGGL((k_mx_matmul_rows<FA, FB, 8, CT>), grid, dim3(512), 0, st, a, as, b, bs, M, N, granules, c, ldc);
    return hipGetLastError();
}

template <int CT>
hipError_t run_matmul(const uint8_t *a, const uint8_t *as, const uint8_t *b, const uint8_t *bs,
                      int64_t M, int64_t N, int64_t granules, void *c, int64_t ldc, float *work, hipStream_t st) {
    const int slices = work ? mx_matmul_slices(M, N, granules) : 1;
    if (slices > 1) {
        const hipError_t e = run_tiled<1, 1, F32, true>(a, as, b, bs, M, N, granules, work, N, st, slices);
        if (e != hipSuccess) return e;
        const dim3 grid((unsigned)((N + 4 * kThreads - 1) / (4 * kThreads)), (unsigned)M);
        hipLaunchKernelGGL((k_mx_matmul_join<CT>), grid, dim3(kThreads), 0, st, work, slices, M, N, c, ldc);
        return hipGetLastError();
    }
    const auto tiles = [&](int64_t m, int64_t n) { return ((M + m - 1) / m) * ((N + n - 1) / n); };
    // Few rows: one pass over B by as many work-groups as it has 16 rows; also for more
    // rows of A where 64 x 64 tiles would leave most of the GPU idle and K is short
    // (64 x 4096, K = 4096: 8.2 us warm and 8.9 cold against 7.3 and 10.9; 32 x 4096, the
    // same K: 5.7 and 6.4 against 7.3 and 9.8; 77 x 1001, K = 1111: 3.6 and 3.5 against 4.7
    // and 5.0; but 200 x 520, K = 8192: 13.6 and 14.4 against 11.2 and 14.1).  32 x 28672,
    // K = 8192 is 1792 work-groups of rows and 448 tiles: 49 us and 52 against 22 and 32.
    const int64_t small = tiles(64, 64), middle = tiles(128, 128), large = tiles(256, 256);
    const bool staged = granules >= 4 && granules < (1 << 18) && small <= kMaxGroups;
    const bool rows = (N + 15) / 16 <= kMaxGroups;
    if (rows && M <= 16) return run_rows<1, 1, CT>(a, as, b, bs, M, N, granules, c, ldc, st);
    if (rows && M <= 32 && (small < 128 || !staged)) return run_rows<2, 1, CT>(a, as, b, bs, M, N, granules, c, ldc, st);
    if (rows && small <= 64 && granules <= 32) return run_rows<4, 1, CT>(a, as, b, bs, M, N, granules, c, ldc, st);
    if (staged) {
        // 64 x 64 while they fit the GPU twice over (512 x 4096, K = 4096: 11.2 us
        // against 12.6 with 128 x 128); then 128 x 128, 512 at a time, or 256 x 256, 256
        // at a time, by what their rounds take: 1.35 us a stage and 3.5 more, or 2.05 and
        // 11 (measured, 128 and 256: 8192 x 8192, K = 28672: 1116 us and 865;
        // 4096 x 4096, K = 4096: 47 and 42; 14336 x 4096, K = 2048: 89 and 107;
        // 2048 x 4096, K = 14336: 74 and 90; 2048 x 14336, K = 4096: 80 and 82)
        const int64_t stages = (granules + 1) / 2;
        if (small <= 512) return run_tiled<1, 1, CT>(a, as, b, bs, M, N, granules, c, ldc, st);
        if ((middle + 511) / 512 * (27 * stages + 70) < (large + 255) / 256 * (41 * stages + 220))
            return run_tiled<2, 2, CT>(a, as, b, bs, M, N, granules, c, ldc, st);
        return run_tiled<4, 4, CT>(a, as, b, bs, M, N, granules, c, ldc, st);
    }
    if (middle > kMaxGroups) return hipErrorInvalidValue;
    const dim3 grid((unsigned)middle);
    const uint32_t mt = (uint32_t)((M + 127) / 128), nt = (uint32_t)((N + 127) / 128);
    switch (granules) {
    case 1: hipLaunchKernelGGL((k_mx_matmul_short<1, CT>), grid, dim3(kThreads), 0, st, a, as, b, bs, M, N, mt, nt, c, ldc); break;
    case 2: hipLaunchKernelGGL((k_mx_matmul_short<2, CT>), grid, dim3(kThreads), 0, st, a, as, b, bs, M, N, mt, nt, c, ldc); break;
    case 3: hipLaunchKernelGGL((k_mx_matmul_short<3, CT>), grid, dim3(kThreads), 0, st, a, as, b, bs, M, N, mt, nt, c, ldc); break;
    default: hipLaunchKernelGGL((k_mx_matmul<CT>), grid, dim3(kThreads), 0, st, a, as, b, bs, M, N, granules, mt, c, ldc);
    }
    return hipGetLastError();
}

}  // namespace

// A long K and too few tiles for the GPU: slices of K, each a share of the work-groups,
// added up in a second launch.  256 work-groups measured best (128 and 512 a tenth to a
// third slower), up to 8 slices, by the GPU's clock: 64 x 512, K = 28672 30 us and 12; 256 x
// 256 30 and 12; 64 x 4096, K = 14336 18.5 and 13, K = 8192 11.2 and 10.8 (cold 17 and 14).  The
// second launch and the scratch memory take the host 4 us: 128 x 1024, K = 8192 11.9 and
// 13.7.  Against the kernel for few rows: 32 x 512, K = 28672 27 and 14; 32 x 4096,
// K = 14336 15 and 15.5; 16 x 4096, K = 28672 19.5 and 18.8 at best.  Slices of 128 x 128
// for more tiles gain up to a fifth (384 x 4096, K = 14336: 41 and 33) for six times the
// scratch memory, and are left out.
int mx_matmul_slices(int64_t M, int64_t N, int64_t granules) {
    const int64_t stages = (granules + 1) / 2, rows = (M + 63) / 64, cols = (N + 63) / 64;
    if (M <= 16 || N < 1 || rows > 128 || cols > 128 || rows * cols > 128 || granules >= (1 << 18)) return 1;
    if (stages < (M <= 32 ? 64 : rows * cols < 48 ? 48 : 32)) return 1;
    return (int)std::min<int64_t>(8, 256 / (rows * cols));
}

hipError_t launch_mx_matmul(const uint8_t *a, const uint8_t *as, const uint8_t *b, const uint8_t *bs,
                            int64_t M, int64_t N, int64_t granules, void *c, int ct, int64_t ldc,
                            float *work, hipStream_t st) {
    switch (ct) {
    case F16: return run_matmul<F16>(a, as, b, bs, M, N, granules, c, ldc, work, st);
    case BF16: return run_matmul<BF16>(a, as, b, bs, M, N, granules, c, ldc, work, st);
    case F32: return run_matmul<F32>(a, as, b, bs, M, N, granules, c, ldc, work, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qcp
