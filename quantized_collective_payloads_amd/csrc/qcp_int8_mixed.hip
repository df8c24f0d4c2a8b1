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
// Where a's rows are aligned (or it is large, and a copy with aligned rows is cheap), larger
// products take the form below instead, which leaves the transposition to reads of LDS.
//
// Bound, of this form: the latency of a stage's load, decode, write and read where there are few
// tiles (77 x 520, K = 1033 11 us, the smallest 5 to 6), and the decoding beside few products in
// small tiles.
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

// TM x TN of C per work-group, KS of k per stage, WM x WN waves; the loads of AHEAD stages are in
// flight beside the one that is multiplied.  TEAMS of so many waves take the stages in turn, and
// their sums are added in LDS at the end.
template <int TM_, int TN_, int KS_, int WM_, int WN_, int AHEAD_, int TEAMS_> struct MixedTile {
    static constexpr int TM = TM_, TN = TN_, KS = KS_, WM = WM_, WN = WN_, AHEAD = AHEAD_, TEAMS = TEAMS_;
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

constexpr int64_t kJoinRows = 32768;                         // rows of work-groups, of the kernels that have one for each row

// The stages of one slice of k of one tile.  TRANS: a is given as [K, M].
template <class G, int AT, bool TRANS, int CT, bool SLICED>
__global__ __launch_bounds__(G::threads * G::TEAMS, 2) void k_int8_mixed(
    const uint16_t *__restrict__ a, int64_t lda, const uint8_t *__restrict__ codes, const float *__restrict__ scales,
    int64_t M, int64_t N, int64_t K, uint32_t pad, uint32_t slices, uint32_t m_tiles, uint32_t n_tiles,
    void *__restrict__ c, int64_t ldc) {
    constexpr int KS = G::KS, FM = G::FM, FN = G::FN;
    constexpr int TEAMS = G::TEAMS;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[TEAMS * 2 * G::slot];
    const uint32_t tid = __builtin_amdgcn_workitem_id_x() % G::threads;
    const int team = TEAMS == 1 ? 0 : __builtin_amdgcn_readfirstlane((int)(__builtin_amdgcn_workitem_id_x() / G::threads));
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
    // ... (columns past the end repeat the last four that begin within), or 8 of k of 4 rows of a
    const uint32_t a_col = min(col, (m_rows - 1) & ~3u);
    const uint32_t t_off = octet * 8 * (uint32_t)lda + a_col;              // in elements
    constexpr uint32_t row_step = G::threads / G::octets;
    const uint32_t a_row = tid / G::octets, a_oct = tid % G::octets;
    uint32_t s_off[4];
#pragma unroll
    for (int i = 0; i < 4; i++) s_off[i] = min(a_row + i * row_step, m_rows - 1) * (uint32_t)lda + a_oct * 8;

    struct Loaded {
        uint32_t b[8];
        float s[8];
        u32x2_t t[8];
        u32x4_t a[4];
    };
    Loaded regs[G::AHEAD];
    // A stage all of whose rows exist.  Where M is no multiple of 4, 4 columns of a transposed a may
    // reach 3 elements past its row: 3 more rows have to follow.
    const bool fours = TRANS ? M % 4 == 0 : true;
    const int beyond = fours ? 0 : 3;
    auto load = [&](int64_t s, Loaded &w) __attribute__((always_inline)) {
        const int64_t k0 = s * KS;
        const uint8_t *const pb = codes + k0 * pad;
        const float *const ps = scales + k0 + octet * 8;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            w.b[j] = *(const uint32_t *)(pb + (int64_t)j * pad + b_off);
            w.s[j] = ps[j];
        }
        if constexpr (TRANS) {
            const uint16_t *const pa = a + k0 * lda + m0;
#pragma unroll
            for (int j = 0; j < 8; j++) w.t[j] = *(const u32x2_any *)(pa + (int64_t)j * lda + t_off);
        } else {
            const uint16_t *const pa = a + m0 * lda + k0;
#pragma unroll
            for (int i = 0; i < 4; i++) w.a[i] = *(const u32x4_any *)(pa + s_off[i]);
        }
    };
    // the last ones: rows past the end repeat the last one and become zeros.  No branch that
    // differs between lanes, so that the loads are in flight together.
    auto load_last = [&](int64_t s, Loaded &w) __attribute__((always_inline)) {
        const int64_t k0 = s * KS, last_k = K - 1;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int64_t k = k0 + octet * 8 + j, row = min(k, last_k);
            w.b[j] = *(const uint32_t *)(codes + row * pad + (b_off - octet * 8 * pad));
            const float mark = scales[row];
            w.s[j] = k <= last_k ? mark : 0.0f;
        }
        if constexpr (TRANS) {
            const uint16_t *const pa = a + m0;
            if (fours) {
#pragma unroll
                for (int j = 0; j < 8; j++) w.t[j] = *(const u32x2_any *)(pa + min(k0 + octet * 8 + j, last_k) * lda + a_col);
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const uint16_t *const p = pa + min(k0 + octet * 8 + j, last_k) * lda;
                    uint32_t h[4];
#pragma unroll
                    for (uint32_t e = 0; e < 4; e++) h[e] = p[min(a_col + e, m_rows - 1)];
                    w.t[j] = u32x2_t{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
                }
            }
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (k0 + octet * 8 + j > last_k) w.t[j] = u32x2_t{0, 0};
        } else {
            const int64_t k = k0 + a_oct * 8;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint16_t *const p = a + m0 * lda + (s_off[i] - a_oct * 8);
                if (K % 8 == 0) {
                    w.a[i] = *(const u32x4_any *)(p + min(k, K - 8));
                    if (k > last_k) w.a[i] = u32x4_t{0, 0, 0, 0};
                } else {
                    w.a[i] = u32x4_t{0, 0, 0, 0};
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const uint32_t h = p[min(k + e, last_k)];
                        w.a[i][e / 2] |= k + e <= last_k ? h << (16 * (e & 1)) : 0;
                    }
                }
            }
        }
    };
    typedef __attribute__((address_space(3))) uint8_t lds_byte;
    lds_byte *const base = (lds_byte *)lds + team * 2 * G::slot;
    typedef __attribute__((address_space(3))) u32x4_t lds_piece;
    auto write = [&](uint32_t slot, const Loaded &w) __attribute__((always_inline)) {
        lds_byte *const to = base + slot * G::slot;
        if constexpr (TRANS) {
#pragma unroll
            for (int e = 0; e < 4; e++) {
                u32x4_t v;
#pragma unroll
                for (int j = 0; j < 4; j++)
                    v[j] = __builtin_amdgcn_perm(e < 2 ? w.t[2 * j + 1].x : w.t[2 * j + 1].y, e < 2 ? w.t[2 * j].x : w.t[2 * j].y,
                                                 e & 1 ? 0x07060302u : 0x05040100u);
                *(lds_piece *)(to + G::at(col + e, octet)) = v;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) *(lds_piece *)(to + G::at(a_row + i * row_step, a_oct)) = w.a[i];
        }
        static_for<4>([&](auto E) __attribute__((always_inline)) {
            constexpr int e = E;
            u32x4_t v;
#pragma unroll
            for (int j = 0; j < 4; j++)
                v[j] = narrow2<AT>(cvt_sbyte<e>(w.b[2 * j]) * w.s[2 * j], cvt_sbyte<e>(w.b[2 * j + 1]) * w.s[2 * j + 1]);
            *(lds_piece *)(to + G::TM * G::row + G::at(col + e, octet)) = v;
        });
    };

    const int r = lane & 31, half = lane >> 5;
    const uint32_t arow = (wave % G::WM) * (G::TM / G::WM) + r, brow = (wave / G::WM) * (G::TN / G::WN) + r;
    f32x16_t acc[FM][FN] = {};
    auto multiply = [&](uint32_t slot) __attribute__((always_inline)) {
        const lds_byte *const from = base + slot * G::slot;
        u32x4_t fa[2][FM], fb[2][FN];
        auto read = [&](int q) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < FN; j++) fb[q & 1][j] = *(const lds_piece *)(from + G::TM * G::row + G::at(brow + 32 * j, 2 * q + half));
#pragma unroll
            for (int i = 0; i < FM; i++) fa[q & 1][i] = *(const lds_piece *)(from + G::at(arow + 32 * i, 2 * q + half));
        };
        read(0);
#pragma unroll
        for (int q = 0; q < KS / 16; q++) {
            if (q + 1 < KS / 16) read(q + 1);
            // B first: a lane then holds 4 consecutive n of one m per group of registers
#pragma unroll
            for (int i = 0; i < FM; i++)
#pragma unroll
                for (int j = 0; j < FN; j++) acc[i][j] = mma16bit<AT>(fb[q & 1][j], fa[q & 1][i], acc[i][j]);
        }
    };

    // the team's turns: stage first + TEAMS i + team.  Those of `load` come first, then those of
    // load_last.
    constexpr int D = G::AHEAD;
    const int64_t mine = first + team, whole_k = min((K - beyond) / KS, last);
    auto fill = [&](int64_t s, Loaded &w) __attribute__((always_inline)) {
        if (s < whole_k) load(s, w);
        else if (s < last) load_last(s, w);
    };
    // stage s, in slot P: the next one is written, the one D turns after it loaded
    auto stage = [&](int64_t s, auto P, auto MAIN) __attribute__((always_inline)) {
        Loaded &w = regs[(D - 1) & (P ^ 1)];
        if (MAIN || s + TEAMS < last) write(P ^ 1, w);
        if constexpr (MAIN) load(s + TEAMS * (1 + D), w);
        else fill(s + TEAMS * (1 + D), w);
        if (MAIN || s < last) multiply(P);
        wait_lds_and_meet();
    };
    if (first < last) {
        fill(mine, regs[0]);
        if (mine < last) write(0, regs[0]);
        static_for<D>([&](auto I) __attribute__((always_inline)) { fill(mine + TEAMS * (1 + I), regs[(1 + I) % D]); });
        wait_lds_and_meet();
        int64_t s = first;                                   // of team 0, the longest
        if constexpr (D == 1) {
            uint32_t slot = 0;
            for (; s + TEAMS * 3 <= whole_k; s += TEAMS, slot ^= 1) stage(s + team, slot, std::true_type{});
            for (; s < last; s += TEAMS, slot ^= 1) stage(s + team, slot, std::false_type{});
        } else {
            using even = std::integral_constant<uint32_t, 0>;
            using odd = std::integral_constant<uint32_t, 1>;
            for (; s + TEAMS * (3 + D) <= whole_k; s += 2 * TEAMS) {
                stage(s + team, even{}, std::true_type{});
                stage(s + team + TEAMS, odd{}, std::true_type{});
            }
            for (; s < last; s += 2 * TEAMS) {
                stage(s + team, even{}, std::false_type{});
                if (s + TEAMS < last) stage(s + team + TEAMS, odd{}, std::false_type{});
            }
        }
    }
    if constexpr (TEAMS == 2) {
        // the second team's sums to LDS; the first adds and stores them
        typedef __attribute__((address_space(3))) f32x4_t lds_sums;
        lds_byte *const at = (lds_byte *)lds + tid * 16;
        static_for<FM * FN * 4>([&](auto I) __attribute__((always_inline)) {
            constexpr int f = I / 4, q = I % 4;
            const f32x16_t &v = acc[f / FN][f % FN];
            if (team == 1) *(lds_sums *)(at + I * G::threads * 16) = f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
        });
        wait_lds_and_meet();
        if (team == 1) return;
        static_for<FM * FN * 4>([&](auto I) __attribute__((always_inline)) {
            constexpr int f = I / 4, q = I % 4;
            const f32x4_t v = *(const lds_sums *)(at + I * G::threads * 16);
#pragma unroll
            for (int e = 0; e < 4; e++) acc[f / FN][f % FN][4 * q + e] += v[e];
        });
    }
    const bool whole = m0 + G::TM <= M && n0 + G::TN <= N;
    void *const to = SLICED ? (float *)c + slice * M * N : c;
    static_for<FM * FN>([&](auto I) __attribute__((always_inline)) {
        constexpr int i = I / FN, j = I % FN;
        store_fragment<CT>(acc[i][j], to, ldc, m0 + arow + 32 * i, n0 + (brow - r) + 32 * j, half, M, N, whole);
    });
}

// ---------------------------------------------------------------------------
// 256 x 256 or 128 x 128 of C per work-group, operands copied to LDS as they lie in memory.
// ---------------------------------------------------------------------------
// For an a whose rows are aligned to 16 bytes.  Eight waves hold 256 x 32 each (four 128 x 32), so
// that a column of the payload is decoded once in a work-group; a's fragments are read by all of
// them.  A stage is 64 of k: 32 KB of a, 16 KB of codes and 64 scales, in one of three slots.
// LDS gives 8 k of a column to a lane: ds_read_b64_tr_b8 turns 8 rows x 16 bytes for 16 lanes,
// _tr_b16 4 rows x 16 values of a transposed a.  A register holds the scales of two steps of 16,
// each row of 16 lanes its own 16, and the products with them take one lane's for all
// (row_newbcast).
//
// A step is 8 products (4 in tiles of 128); between them, in the order written, the fragment just
// used is read for the next step, and that step's codes are read and decoded.  Before a stage's
// last step, whose fragments were read by then, the waves meet: the next stage has arrived, and the
// one before this was multiplied by all, so the copies of the stage after the next go into its slot.
// In tiles of 128, whose stages are half as long, copies go a stage further ahead, into the slot
// just read, and the waves wait for those reads as well (1024 x 4096, K = 4096 46 us and 52; in
// tiles of 256 that is 1% the slower).
//
// Bound: the cycles in which the matrix cores wait, two fifths of them, and on normal values the
// power that they draw, which takes the clock from 2.4 GHz to 1.9.  8192 x 8192, K = 4096 takes 460
// us (1.2 PFLOP/s; the cores are busy in 60% of the cycles and LDS in 33%, the waves wait in 31% of
// their time for a barrier or a count, and 80 of 142 vector instructions a wave and stage are the
// decoding) and on zeros 320 to 334 (1.7 PFLOP/s).  4096 x 4096, K = 4096 119 to 124 us; 2048 x 4096,
// K = 14336 in two slices 207 and 13 for the join; 14336 x 4096, K = 2048 to fp32 240 to 253, whose
// 3.5 rounds of tiles take 4; 2048 x 2048, K = 2048 in tiles of 128 28 to 29.
//
// Pieces of 16 bytes lie in LDS in an order that spreads what a read touches in a cycle over all
// banks: of a row by row, piece ^ (row / 2 % 8); of a transposed, piece ^ 4 (row % 4); of the
// payload, piece ^ 2 (row % 8), or where its rows are 128 bytes 2 (row / 2 % 4).  What is read past
// the end of a buffer counts for nothing: results past the end are not stored, and in the last stage
// of a K that is no multiple of 64 the values of a and the scales past the end are made zeros in LDS.
namespace direct {

constexpr int kStage = 64, kSlots = 3;
constexpr int kCopies = 7;                                   // of a wave and stage
constexpr int64_t kMaxLd = (int64_t)1 << 22;                 // 256 rows of a are within 32 bits

// 32*FM x 32*NW of C per work-group of NW waves
template <int FM_, int NW_> struct Tile {
    static constexpr int FM = FM_, NW = NW_, TM = 32 * FM, TN = 32 * NW, threads = 64 * NW;
    static constexpr uint32_t ahead = NW == 8 ? 2 : 3;           // stages copied before the first is multiplied
    static constexpr uint32_t codes_at = TM * kStage * 2, scales_at = codes_at + TN * kStage, slot = scales_at + 256;
    static constexpr uint32_t t_row = 2 * TM, t_pieces = TM / 8; // of a row of a transposed a, in LDS
    static constexpr uint32_t b_row = TN, b_pieces = TN / 16;    // of a row of codes
    static_assert(FM == NW && (NW == 8 || NW == 4), "7 copies a wave; the order of the pieces");
    // what a piece of the payload's row k is moved by
    __device__ static __forceinline__ uint32_t turn(uint32_t k) { return NW == 8 ? 2 * (k & 7) : k & 6; }
};

typedef __attribute__((address_space(3))) uint8_t lds_byte;

__device__ __forceinline__ u32x2_t read_tr8(uint32_t at) {
    typedef int i32x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2_t *)at));
}
__device__ __forceinline__ u32x2_t read_tr16(uint32_t at) {
    typedef short i16x4_t __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t *)at));
}
// lane J of each row of 16 lanes, to all of the row
template <int J>
__device__ __forceinline__ float of_lane(float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x150 + J, 0xf, 0xf, true));
}
// until at most N of this wave's copies and stores are in flight, reads of LDS not counted; then
// with the other waves
template <int N>
__device__ __forceinline__ void wait_copies_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

// width: elements of a row of a as it is given, a multiple of 8
template <class G, int AT, bool TRANS, int CT, bool SLICED>
__global__ __launch_bounds__(G::threads, 2) void k_int8_mixed_direct(
    const uint16_t *__restrict__ a, int64_t lda, const uint8_t *__restrict__ codes, const float *__restrict__ scales,
    int64_t M, int64_t N, int64_t K, int64_t width, uint32_t pad, uint32_t slices, uint32_t m_tiles, uint32_t n_tiles,
    uint32_t groups, void *__restrict__ c, int64_t ldc) {
    constexpr int FM = G::FM;
    constexpr uint32_t kSlot = G::slot, kCodesAt = G::codes_at, kScalesAt = G::scales_at;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kSlots * kSlot];
    const int tid = (int)__builtin_amdgcn_workitem_id_x();
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t lane = (uint32_t)lane_id(), r = lane & 31, half = lane >> 5, t16 = lane & 15, side = (lane >> 4) & 1;
    const uint32_t base = (uint32_t)(uintptr_t)(lds_byte *)lds;
    const uint32_t tiles = m_tiles * n_tiles * (SLICED ? slices : 1);

    // the tile that is being copied, and the next of its stages to be
    int64_t m0, n0, k_next, k_end;
    uint32_t m_rows, stages, slice = 0, b_voff[2], to_slot;
    auto set_tile = [&](uint32_t t) __attribute__((always_inline)) {
        const int64_t all = (K + kStage - 1) / kStage;
        int64_t first = 0, count = all;
        if constexpr (SLICED) {
            slice = t / (m_tiles * n_tiles);
            t -= slice * (m_tiles * n_tiles);
            const int64_t each = all / slices, over = all % slices;
            first = slice * each + min((int64_t)slice, over);
            count = each + (slice < over ? 1 : 0);
        }
        stages = (uint32_t)count;
        const TilePlace at = tile_place(t, m_tiles, n_tiles);
        m0 = (int64_t)at.m * G::TM;
        n0 = (int64_t)at.n * G::TN;
        m_rows = (uint32_t)min(M - m0, (int64_t)G::TM);
        k_next = first * kStage;
        k_end = min((first + count) * kStage, K);
        to_slot = 0;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint32_t row = kStage / G::NW * wave + (kStage / G::NW / 2) * i + lane / G::b_pieces;
            const uint32_t piece = lane % G::b_pieces ^ G::turn(row);
            b_voff[i] = row * pad + (uint32_t)min(n0 + 16 * piece, (int64_t)pad - 16);
        }
    };
    // the n-th copy of the next stage, the scales first
    auto copy = [&](auto I) __attribute__((always_inline)) {
        constexpr int n = I;
        const uint32_t to = base + to_slot;
        if constexpr (n == 0) {
            copy4_to_lds(to + kScalesAt, lane * 4, buffer_of(scales + k_next, (uint64_t)(K - k_next) * 4));
        } else if constexpr (n <= 2) {
            copy_to_lds(to + kCodesAt + wave * 2048 + (n - 1) * 1024, b_voff[n - 1],
                        buffer_of(codes + k_next * pad, (uint64_t)(K - k_next) * pad), 0);
        } else if constexpr (TRANS) {
            constexpr int i = n - 3;
            const uint32_t row = kStage / G::NW * wave + (kStage / G::NW / 4) * i + lane / G::t_pieces;
            const uint32_t piece = lane % G::t_pieces ^ (4 * (row & 3));
            copy_to_lds(to + wave * 4096 + i * 1024, row * (uint32_t)lda * 2 + piece * 16,
                        buffer_of(a + k_next * lda + m0, (uint64_t)((K - 1 - k_next) * lda + (width - m0)) * 2), 0);
        } else {
            constexpr int i = n - 3;
            const uint32_t row = min(32 * wave + 8 * i + (lane >> 3), m_rows - 1);
            const uint32_t piece = (lane & 7) ^ (lane >> 4) ^ (4 * (i & 1));
            copy_to_lds(to + wave * 4096 + i * 1024, row * (uint32_t)lda * 2 + piece * 16,
                        buffer_of(a + m0 * lda + k_next, (uint64_t)((m_rows - 1) * lda + width - k_next) * 2), 0);
        }
    };
    auto copied = [&]() __attribute__((always_inline)) {
        k_next += kStage;
        to_slot = to_slot == (kSlots - 1) * kSlot ? 0 : to_slot + kSlot;
    };

    // where this lane reads in slot 0
    const uint32_t a_at = base + (TRANS ? (8 * half + (t16 >> 2)) * G::t_row + ((4 * (t16 >> 2) + 2 * side + ((t16 & 3) >> 1)) * 16) + 8 * (t16 & 1)
                                        : r * 128 + ((half ^ ((r >> 1) & 7)) * 16));
    const uint32_t b_at = base + kCodesAt + (8 * half + (t16 >> 1)) * G::b_row + (((2 * wave + side) ^ G::turn(t16 >> 1)) * 16) + 8 * (t16 & 1);
    const uint32_t s_at = base + kScalesAt + 4 * (16 * (t16 >> 3) + 8 * half + (t16 & 7));

    f32x16_t acc[FM];
    u32x4_t fa[FM], fb;
    u32x2_t raw;
    float mark[2];
    uint32_t from = 0;                                       // the slot that is being read
    auto read_a = [&](auto I, auto Q) __attribute__((always_inline)) {
        constexpr int i = I, q = Q;
        if constexpr (TRANS) {
            const uint32_t at = (a_at ^ (64 * (i & 3))) + from;
            const u32x2_t lo = read_tr16(at + 256 * (i >> 2) + 16 * G::t_row * q), hi = read_tr16(at + 256 * (i >> 2) + 16 * G::t_row * q + 4 * G::t_row);
            fa[i] = u32x4_t{lo.x, lo.y, hi.x, hi.y};
        } else {
            fa[i] = lds16((a_at ^ (32 * q)) + from + 4096 * i);
        }
    };
    auto read_codes = [&](auto Q) __attribute__((always_inline)) { raw = read_tr8(b_at + from + 16 * G::b_row * Q); };
    auto read_marks = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 2; i++) mark[i] = __uint_as_float(lds4(s_at + from + 128 * i));
    };
    // values 2J and 2J + 1 of step Q
    auto decode = [&](auto J, auto Q, u32x4_t &to) __attribute__((always_inline)) {
        constexpr int j = J, q = Q, l = 8 * (q & 1) + 2 * j;
        const uint32_t w = j < 2 ? raw.x : raw.y;
        to[j] = narrow2<AT>(cvt_sbyte<2 * (j & 1)>(w) * of_lane<l>(mark[q >> 1]),
                            cvt_sbyte<2 * (j & 1) + 1>(w) * of_lane<l + 1>(mark[q >> 1]));
    };
    using std::integral_constant;
    using zero = integral_constant<int, 0>;
    // what lies past the end of K in the slot at `at`, `left` of whose k exist, becomes zeros: a's
    // values and the scales.  Of a row by row these are whole pieces of 8 k; where K ends inside
    // one, the rows are the aligned copy's, which holds zeros from K to the end of that piece
    auto clear = [&](uint32_t at, uint32_t left) __attribute__((always_inline)) {
        typedef __attribute__((address_space(3))) u32x4_t lds_piece;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t n = i * G::threads + tid;
            const uint32_t k = TRANS ? n / G::t_pieces : n % 8 * 8;
            const uint32_t to = TRANS ? n * 16 : n / 8 * 128 + ((n ^ (n / 16)) & 7) * 16;
            if (k >= left) *(lds_piece *)(at + to) = u32x4_t{0, 0, 0, 0};
        }
        if (tid < kStage && (uint32_t)tid >= left) *(__attribute__((address_space(3))) float *)(at + kScalesAt + tid * 4) = 0;
        wait_lds_and_meet();
    };
    // a stage.  COPY: the next stage is copied beside it.  LAST: nothing follows.  meet: before the
    // next stage's slot, which it is given, is read.
    auto stage = [&](auto COPY, auto LAST, auto meet) __attribute__((always_inline)) {
        static_for<4>([&](auto Q) __attribute__((always_inline)) {
            constexpr int q = Q, then = (q + 1) % 4;
            constexpr bool more = q < 3 || !LAST;
            u32x4_t fn;
            if constexpr (q == 3 && !LAST) {
                from = from == (kSlots - 1) * kSlot ? 0 : from + kSlot;
                meet(from);
            }
            static_for<FM>([&](auto I) __attribute__((always_inline)) {
                constexpr int i = I;
                // B first: a lane then holds 4 consecutive n of one m per group of registers
                acc[i] = mma16bit<AT>(fb, fa[i], acc[i]);
                if constexpr (more) {
                    if constexpr (i == 0) {
                        read_codes(integral_constant<int, then>{});
                        if constexpr (then == 0) read_marks();
                    }
                    read_a(I, integral_constant<int, then>{});
                    if constexpr (i >= FM / 2)
                        static_for<8 / FM>([&](auto J) __attribute__((always_inline)) {
                            decode(integral_constant<int, (i - FM / 2) * (8 / FM) + J>{}, integral_constant<int, then>{}, fn);
                        });
                }
                if constexpr (COPY && q == 3)
                    static_for<8 / FM>([&](auto J) __attribute__((always_inline)) {
                        constexpr int n = i * (8 / FM) + J - 1;
                        if constexpr (n >= 0) copy(integral_constant<int, n>{});
                    });
                __builtin_amdgcn_sched_barrier(0);
            });
            if constexpr (more) fb = fn;
            if constexpr (COPY && q == 3) copied();
        });
    };
    auto begin = [&]() __attribute__((always_inline)) {
        from = 0;
        read_codes(zero{});
        read_marks();
        static_for<FM>([&](auto I) __attribute__((always_inline)) { read_a(I, zero{}); });
        static_for<4>([&](auto J) __attribute__((always_inline)) { decode(J, zero{}, fb); });
    };
    auto copy_first = [&]() __attribute__((always_inline)) {
        for (uint32_t s = 0; s < min(stages, G::ahead); s++) {
            static_for<kCopies>(copy);
            copied();
        }
    };
    using no = integral_constant<int, 0>;
    using yes = integral_constant<int, 1>;
    // 16-byte stores of a wave's whole results
    constexpr int stores = FM * 16 * dtype_traits<CT>::bytes / 16;

    uint32_t tile = __builtin_amdgcn_workgroup_id_x();
    set_tile(tile);
    copy_first();
    wait_and_meet<0>();
    int behind = 0;                                          // stages whose copies are older than the last tile's stores
    constexpr int later = (G::ahead - 2) * kCopies;          // copies of stages beyond the next, in flight where the waves meet
    auto arrive = [&](auto N) __attribute__((always_inline)) {
        if constexpr (G::ahead == kSlots) wait_and_meet<N>();
        else wait_copies_and_meet<N>();
    };
    for (;;) {
#pragma unroll
        for (int i = 0; i < FM; i++) acc[i] = f32x16_t{};
        if (stages) {
            const uint32_t tail = (uint32_t)(k_end - (k_end - 1) / kStage * kStage);   // rows of the last stage
            if (stages == 1 && tail < kStage) clear(base, tail);
            begin();
            uint32_t s = 0;
            for (; s + G::ahead < stages; s++)
                stage(yes{}, no{}, [&](uint32_t) __attribute__((always_inline)) {
                    if (behind > 0) {
                        behind--;
                        arrive(integral_constant<int, later + stores>{});
                    } else {
                        arrive(integral_constant<int, later>{});
                    }
                });
            for (; s + 1 < stages; s++)
                stage(no{}, no{}, [&](uint32_t slot) __attribute__((always_inline)) {
                    wait_and_meet<0>();
                    if (s + 2 == stages && tail < kStage) clear(base + slot, tail);
                });
            stage(no{}, yes{}, [](uint32_t) __attribute__((always_inline)) {});
        }

        // the next tile's first copies go out before this one's results
        const int64_t m_done = m0 + r, n_done = n0 + 32 * wave;
        const bool whole = m0 + G::TM <= M && n0 + G::TN <= N;
        void *const to = SLICED ? (float *)c + slice * M * N : c;
        tile += groups;
        const bool more = tile < tiles;
        if (more) {
            wait_lds_and_meet();                             // every wave is done with the slots
            set_tile(tile);
            copy_first();
        }
        static_for<FM>([&](auto I) __attribute__((always_inline)) {
            constexpr int i = I;
            store_fragment<CT>(acc[i], to, ldc, m_done + 32 * i, n_done, (int)half, M, N, whole);
        });
        if (!more) break;
        behind = whole && stages >= G::ahead ? (int)G::ahead - 1 : 0;
        if (behind) wait_and_meet<later + kCopies + stores>();
        else wait_and_meet<0>();
    }
}

}  // namespace direct

// The sum of the slices, in their order, rounded once: 4 columns a lane, a row of work-groups for
// each row of C.  (A division per lane to find its row in one long grid took as long as the
// memory: 2048 x 4096, 2 slices, 22 us.)
template <int CT>
__global__ __launch_bounds__(kThreads) void k_int8_mixed_join(const float *__restrict__ parts, int slices, int64_t part,
                                                              int64_t M, int64_t N, void *__restrict__ c, int64_t ldc) {
    typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
    const int64_t n = ((int64_t)__builtin_amdgcn_workgroup_id_x() * kThreads + __builtin_amdgcn_workitem_id_x()) * 4;
    if (n >= N) return;
    const int count = N - n < 4 ? (int)(N - n) : 4;
    for (int64_t m = group_y(); m < M; m += kJoinRows) {
        const float *p = parts + m * N + n;
        float v[4] = {};
        if (count == 4) {
            // 2, 4, 8 or 16 slices: several loads in flight
#pragma unroll 4
            for (int s = 0; s < slices; s += 2) {
                f32x4_any x[2];
#pragma unroll
                for (int k = 0; k < 2; k++, p += part) x[k] = *(const f32x4_any *)p;
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    v[0] += x[k].x; v[1] += x[k].y; v[2] += x[k].z; v[3] += x[k].w;
                }
            }
        } else {
            for (int s = 0; s < slices; s++, p += part)
#pragma unroll
                for (int j = 0; j < 3; j++)
                    if (j < count) v[j] += p[j];
        }
        store4<CT>(c, m * ldc + n, count, v);
    }
}

// a with rows of whole 16 bytes, the rest of a row's last 16 zeros: what the kernel above can copy.
// A row of work-groups for each row.
__global__ __launch_bounds__(kThreads) void k_int8_mixed_align(const uint16_t *__restrict__ a, int64_t lda, int64_t rows,
                                                               int64_t width, uint16_t *__restrict__ to) {
    const int64_t at = ((int64_t)__builtin_amdgcn_workgroup_id_x() * kThreads + __builtin_amdgcn_workitem_id_x()) * 8;
    const int64_t whole = (width + 7) / 8 * 8, left = width - at;
    if (left <= 0) return;
    for (int64_t r = group_y(); r < rows; r += kJoinRows) {
        const uint16_t *const p = a + r * lda + at;
        u32x4_t w = {0, 0, 0, 0};
        if (left >= 8) {
            w = __builtin_nontemporal_load((const u32x4_any *)p);
        } else {
#pragma unroll
            for (int e = 0; e < 7; e++)
                if (e < left) w[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
        }
        *(u32x4_t *)(to + r * whole + at) = w;
    }
}

using Tile256 = MixedTile<256, 256, 64, 2, 4, 1, 1>;
using Tile128 = MixedTile<128, 128, 64, 2, 2, 2, 1>;
using Tile64 = MixedTile<64, 64, 128, 2, 2, 1, 1>;
using Tile64x2 = MixedTile<64, 64, 128, 2, 2, 1, 2>;

struct MixedArgs {
    const uint16_t *a;
    int64_t lda, width;          // elements between its rows, and of a row
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
    hipLaunchKernelGGL((k_int8_mixed<G, AT, TRANS, CT, SLICED>), dim3((unsigned)(mt * nt * slices)), dim3(G::threads * G::TEAMS), 0,
                       p.st, p.a, p.lda, p.codes, p.scales, p.M, p.N, p.K, pad, (uint32_t)slices, (uint32_t)mt,
                       (uint32_t)nt, p.c, p.ldc);
    return hipGetLastError();
}

template <class G, int AT, bool TRANS, int CT, bool SLICED>
hipError_t run_direct(const MixedArgs &p, int slices, int resident) {
    const int64_t mt = (p.M + G::TM - 1) / G::TM, nt = (p.N + G::TN - 1) / G::TN;
    const uint32_t pad = (uint32_t)((p.N + 127) / 128 * 128);
    const unsigned groups = (unsigned)std::min<int64_t>(mt * nt * slices, resident);
    hipLaunchKernelGGL((direct::k_int8_mixed_direct<G, AT, TRANS, CT, SLICED>), dim3(groups), dim3(G::threads), 0, p.st,
                       p.a, p.lda, p.codes, p.scales, p.M, p.N, p.K, p.width, pad, (uint32_t)slices, (uint32_t)mt,
                       (uint32_t)nt, groups, p.c, p.ldc);
    return hipGetLastError();
}

// which form takes a product: the cheapest
constexpr Form kForms[] = {
    {64, 256, 256, 110, 130, 380},     // two teams; 512 x 512, K = 512: 6.1 us, one team 6.7
    {64, 128, 512, 85, 130, 330},      // 1000 x 1500, K = 1000: 15 us, two teams 18.6, tiles of 128 18.8
    {128, 64, 512, 85, 134, 400},      // 2048 x 2048, K = 2048: 33 us, tiles of 64 44, of 256 46
    {256, 64, 256, 200, 215, 1000},    // 4000 x 4000, K = 300: 24 us, tiles of 128 29
    {128, 64, 512, 66, 112, 400},      // an aligned a: 2048 x 2048, K = 2048 26 us, without copies to LDS 30
    {256, 64, 256, 120, 170, 800},     // the same: 4096 x 4096, K = 4096 119 us, the form above 146, tiles of 128 168
};
constexpr int kPlain256 = 3, kDirect128 = 4, kDirect256 = 5;

struct Choice {
    int form, slices;
    bool copy;                   // of a, to aligned rows
    int64_t copy_bytes, work;    // of that copy, and all scratch memory
};
constexpr int64_t kMostCopied = (int64_t)256 << 20;
// Slices of K (up to 16, each of at least 256) fill the GPU where there are few tiles: 512 x
// 4096, K = 14336 80 us with 4 (tiles of 128), 140 without; 2048 x 4096, K = 14336 222 with 2, 283
// without.  They cost a second launch, and the sums a trip to memory and back.  A copy of an a
// that is not aligned costs the same: 14335 x 4095, K = 2047 272 us with it and 328 without;
// scratch: scratch memory may be used.
Choice choose(int64_t M, int64_t N, int64_t K, bool transpose, bool aligned, bool scratch) {
    Choice best = {0, 1, false, 0, 0};
    int64_t least = INT64_MAX;
    const int64_t width = transpose ? M : K, rows = transpose ? K : M, wide = (width + 7) / 8 * 8;
    aligned = aligned && width % 8 == 0 && wide <= direct::kMaxLd;
    const bool copy = !aligned && scratch && K > 0 && wide <= direct::kMaxLd && rows <= kMostCopied / (2 * wide);
    const int64_t copied = copy ? 2 * wide * rows : 0;
    for (int f = 0; f <= kDirect256; f++) {
        if (f >= kDirect128 ? !aligned && !copy : aligned && f == kPlain256) continue;
        const Form &m = kForms[f];
        const int64_t tiles = m.tiles(M, N), stages = (K + m.stage - 1) / m.stage;
        if (tiles > kMaxGroups / 2) continue;
        const bool with = f >= kDirect128 && copy;
        for (int s = 1; s <= (scratch ? 16 : 1); s *= 2) {
            if (s > 1 && (K / s < 256 || tiles * s > m.resident + m.resident / 4)) break;
            int64_t price = m.price(tiles * s, (stages + s - 1) / s);
            if (s > 1) price += 550 + (8 * s - 1) * M * N / 50000;   // fp32 sums out at 4 TB/s, in at 6.2
            if (with) price += 700 + copied / 22500;                 // out and in at 4.5 TB/s
            if (price < least) {
                least = price;
                const int64_t bytes = with ? (copied + 255) / 256 * 256 : 0;
                best = {f, s, with, bytes, bytes + (s > 1 ? 4 * s * M * N : 0)};
            }
        }
    }
    return best;
}

template <int AT, bool TRANS, int CT, bool SLICED>
hipError_t run_form(const MixedArgs &p, Choice which) {
    switch (which.form) {
    case 0: return run<Tile64x2, AT, TRANS, CT, SLICED>(p, which.slices);
    case 1: return run<Tile64, AT, TRANS, CT, SLICED>(p, which.slices);
    case 2: return run<Tile128, AT, TRANS, CT, SLICED>(p, which.slices);
    case kPlain256: return run<Tile256, AT, TRANS, CT, SLICED>(p, which.slices);
    case kDirect128: return run_direct<direct::Tile<4, 4>, AT, TRANS, CT, SLICED>(p, which.slices, kForms[kDirect128].resident);
    default: return run_direct<direct::Tile<8, 8>, AT, TRANS, CT, SLICED>(p, which.slices, kForms[kDirect256].resident);
    }
}

// is a, with rows lda apart, as the copies to LDS need it (where their width is, too)
bool is_aligned(const void *a, int64_t lda) { return (uintptr_t)a % 16 == 0 && lda % 8 == 0 && lda <= direct::kMaxLd; }

template <int AT, bool TRANS, int CT>
hipError_t run_mixed(MixedArgs p, uint8_t *work) {
    const Choice which = choose(p.M, p.N, p.K, TRANS, is_aligned(p.a, p.lda), work != nullptr);
    if (which.copy) {
        const int64_t rows = TRANS ? p.K : p.M;
        const dim3 grid((unsigned)((p.width + 8 * kThreads - 1) / (8 * kThreads)), (unsigned)std::min<int64_t>(rows, kJoinRows));
        hipLaunchKernelGGL(k_int8_mixed_align, grid, dim3(kThreads), 0, p.st, p.a, p.lda, rows, p.width, (uint16_t *)work);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        p.a = (const uint16_t *)work;
        p.lda = p.width = (p.width + 7) / 8 * 8;
    }
    if (which.slices == 1) return run_form<AT, TRANS, CT, false>(p, which);
    float *const sums = (float *)(work + which.copy_bytes);
    MixedArgs q = p;
    q.c = sums;
    q.ldc = p.N;
    const hipError_t e = run_form<AT, TRANS, F32, true>(q, which);
    if (e != hipSuccess) return e;
    // a C that is one run of whole fours is one row
    const bool flat = p.ldc == p.N && p.N % 4 == 0;
    const int64_t rows = flat ? 1 : p.M, cols = flat ? p.M * p.N : p.N;
    const dim3 grid((unsigned)((cols + 4 * kThreads - 1) / (4 * kThreads)), (unsigned)std::min<int64_t>(rows, kJoinRows));
    hipLaunchKernelGGL((k_int8_mixed_join<CT>), grid, dim3(kThreads), 0, p.st, sums, which.slices, p.M * p.N, rows, cols,
                       p.c, p.ldc);
    return hipGetLastError();
}

template <int AT, bool TRANS>
hipError_t by_result(const MixedArgs &p, int ct, uint8_t *work) {
    return ct == F32 ? run_mixed<AT, TRANS, F32>(p, work) : run_mixed<AT, TRANS, AT>(p, work);
}

}  // namespace

int64_t int8_mixed_work(int64_t M, int64_t N, int64_t K, int transpose, bool aligned) {
    if (M < 1 || N < 1 || K < 1) return 0;
    return choose(M, N, K, transpose, aligned, true).work;
}
bool int8_mixed_aligned(const void *a, int64_t lda) { return is_aligned(a, lda); }

hipError_t launch_int8_mixed(const void *a, int at, int64_t lda, int transpose, const uint8_t *codes,
                             const float *scales, int64_t M, int64_t N, int64_t K, void *c, int ct, int64_t ldc,
                             void *work, hipStream_t st) {
    const MixedArgs p = {(const uint16_t *)a, lda, transpose ? M : K, codes, scales, M, N, K, c, ldc, st};
    uint8_t *const w = (uint8_t *)work;
    if (at == BF16) return transpose ? by_result<BF16, true>(p, ct, w) : by_result<BF16, false>(p, ct, w);
    if (at == F16) return transpose ? by_result<F16, true>(p, ct, w) : by_result<F16, false>(p, ct, w);
    return hipErrorInvalidValue;
}

}  // namespace qcp
