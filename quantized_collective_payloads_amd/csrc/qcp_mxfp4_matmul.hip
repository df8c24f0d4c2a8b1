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
#include "qcp_device.h"
#include "qcp_launch.h"

namespace qcp {

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

template <int T>
__device__ __forceinline__ f32x16_t mma(uint4 a, uint32_t sa, uint4 b, uint32_t sb, f32x16_t c) {
    const i32x8_t av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const i32x8_t bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, T, (int)sa, T, (int)sb);
}

template <int CT>
__device__ __forceinline__ void store4(void *c, int64_t at, int count, const float (&v)[4]) {
    if constexpr (CT == F32) {
        float *p = (float *)c + at;
        typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
        if (count >= 4) *(f32x4_any *)p = f32x4_any{v[0], v[1], v[2], v[3]};
        else
#pragma unroll
            for (int j = 0; j < 4; j++)
                if (j < count) p[j] = v[j];
    } else {
        uint16_t *p = (uint16_t *)c + at;
        typedef unsigned int u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
        const uint32_t lo = narrow2<CT>(v[0], v[1]), hi = narrow2<CT>(v[2], v[3]);
        if (count >= 4) *(u32x2_any *)p = u32x2_any{lo, hi};
        else
#pragma unroll
            for (int j = 0; j < 4; j++)
                if (j < count) p[j] = (uint16_t)((j < 2 ? lo : hi) >> (16 * (j & 1)));
    }
}

// A wave computes 64 x 64 of C from 2 + 2 fragments per granule, read straight
// from memory; a work-group's 4 waves make 128 x 128.  Rows past the end repeat
// the last one and are not stored.
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
        uint4 fa[2][2], fb[2][2];
        uint32_t sa[2], sb[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
#pragma unroll
            for (int t = 0; t < 2; t++) {
                fa[i][t] = *(const uint4 *)(pa[i] + g * 64 + 16 * t);
                fb[i][t] = *(const uint4 *)(pb[i] + g * 64 + 16 * t);
            }
            sa[i] = *(const uint32_t *)(qa[i] + g * 4) >> (16 * half);
            sb[i] = *(const uint32_t *)(qb[i] + g * 4) >> (16 * half);
        }
        // B first: a lane then holds 4 consecutive n of one m per group of registers
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int j = 0; j < 2; j++) {
                acc[i][j] = mma<0>(fb[j][0], sb[j], fa[i][0], sa[i], acc[i][j]);
                acc[i][j] = mma<1>(fb[j][1], sb[j], fa[i][1], sa[i], acc[i][j]);
            }
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int64_t m = m0 + 32 * i + row;
        if (m >= M) continue;
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int64_t n = n0 + 32 * j + 8 * q + 4 * half;
                const float v[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                store4<CT>(c, m * ldc + n, N - n < 4 ? (int)(N - n) : 4, v);
            }
    }
}

// ---------------------------------------------------------------------------
// 256 x 256 of C per work-group, for shapes whose tiles fill the GPU.
// ---------------------------------------------------------------------------
// Bound: the matrix cores.  Four waves, one per SIMD, hold 128 x 128 each in 256
// accumulators; a granule of 128 is then 32 instructions of 32 cycles on 16 KB of
// operands per wave, 64 bytes of LDS a cycle for the whole CU, half of what it
// gives.  A stage is 256 of K: 128 bytes of each of the 512 operand rows, whole
// cache lines, in one of two 64 KB slots.
//
// Within a stage the lower half-wave takes the first granule (64 bytes of its row)
// and the upper one the second, so a lane's four blocks have their scales in one
// dword and the instruction picks the byte.  A stage is two phases of 128 of K.
//
// Copies go from memory to LDS without registers (buffer_load ... lds), so their
// latency is covered by the matrix instructions of a whole stage: with the
// fragments of phase 0 in registers a wave issues its products and reads those of
// phase 1; one barrier, at which every wave has read this stage and holds no
// outstanding copy of the next; the copies of the stage after that go into the
// slot just freed; and the products of phase 1 run beside the reads of the next
// stage's phase 0.
//
// LDS holds a row's 8 pieces of 16 bytes in the order piece ^ (row / 2 % 8): the
// copy permutes its source addresses, so that a fragment read, 16 rows of 128 bytes
// at the same piece a cycle, touches each of the 64 banks once.  Scales are copied for 4 granules at a time,
// 16 bytes a row, into two slots of their own.
//
// Rows past the end repeat the last row.  Windows in K are pulled back to end
// with the row: a last odd granule comes as the second one of its window, and is
// multiplied by itself as in the kernel above.
constexpr int kTile = 256;
constexpr int kSlot = 2 * kTile * 128;                 // codes of A and B, one stage
constexpr int kMarkSlot = 2 * kTile * 16;              // scales of A and B, 4 granules
constexpr int kBigLds = 2 * kSlot + 2 * kMarkSlot;     // 144 KB

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// 64 lanes x 16 bytes from rsrc[voff + soff] to LDS at `lds` + 16 * lane.  The
// caller waits for it with wait_copies; no register is written.
__device__ __forceinline__ void copy_to_lds(uint32_t lds, uint32_t voff, i32x4_t rsrc, uint32_t soff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory", "m0");
}

__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ i32x4_t buffer_of(const void *p, uint64_t bytes) {
    const uint64_t at = (uint64_t)p;
    const uint32_t n = bytes > 0xfffffffcull ? 0xfffffffcu : (uint32_t)bytes;
    return i32x4_t{__builtin_amdgcn_readfirstlane((int)(uint32_t)at),
                   __builtin_amdgcn_readfirstlane((int)(uint32_t)(at >> 32)),
                   __builtin_amdgcn_readfirstlane((int)n), 0x00020000};
}

struct Fragments {
    uint4 a[4][2], b[4][2];
};
struct Scales {
    uint32_t a[4], b[4];
};

// the 32 products of phase P, four rows of instructions at a time
template <int P>
__device__ __forceinline__ void products(const Fragments &f, const Scales &e, f32x16_t (&acc)[4][4]) {
    static_for<32>([&](auto S) {
        constexpr int s = S, t = s / 16, i = s / 4 % 4, n = s % 4;
        acc[i][n] = mma<2 * P + t>(f.b[n][t], e.b[n], f.a[i][t], e.a[i], acc[i][n]);
    });
}

template <int CT>
__global__ __launch_bounds__(kThreads, 1) void k_mx_matmul_big(
    const uint8_t *__restrict__ a, const uint8_t *__restrict__ as, const uint8_t *__restrict__ b,
    const uint8_t *__restrict__ bs, int64_t M, int64_t N, uint32_t granules, uint32_t m_tiles,
    uint32_t n_tiles, void *__restrict__ c, int64_t ldc) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kBigLds];
    const int tid = (int)__builtin_amdgcn_workitem_id_x();
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = lane_id();

    // work-groups are dealt round-robin to the 8 XCDs: give each XCD a contiguous
    // run of tiles, and walk it 4 tiles of M by N, so that the 32 tiles an XCD works
    // on at a time share 4 + 8 operand panels in its L2
    const uint32_t tiles = m_tiles * n_tiles;
    uint32_t t = __builtin_amdgcn_workgroup_id_x();
    const uint32_t per = tiles / 8, extra = tiles % 8, xcd = t % 8, slot8 = t / 8;
    t = xcd * per + min(xcd, extra) + slot8;
    const uint32_t band = 4 * n_tiles, first = t / band * 4, height = min(4u, m_tiles - first);
    const uint32_t in = t - t / band * band;
    const int64_t m0 = (int64_t)(first + in % height) * kTile, n0 = (int64_t)(in / height) * kTile;

    const uint32_t row_bytes = granules * 64, mark_bytes = granules * 4;
    const int64_t m_left = M - m0, n_left = N - n0;
    const i32x4_t ra = buffer_of(a + m0 * row_bytes, (uint64_t)min(m_left, (int64_t)kTile) * row_bytes);
    const i32x4_t rb = buffer_of(b + n0 * row_bytes, (uint64_t)min(n_left, (int64_t)kTile) * row_bytes);
    const i32x4_t rsa = buffer_of(as + m0 * mark_bytes, (uint64_t)min(m_left, (int64_t)kTile) * mark_bytes);
    const i32x4_t rsb = buffer_of(bs + n0 * mark_bytes, (uint64_t)min(n_left, (int64_t)kTile) * mark_bytes);
    const uint32_t m_last = (uint32_t)min(m_left, (int64_t)kTile) - 1;
    const uint32_t n_last = (uint32_t)min(n_left, (int64_t)kTile) - 1;

    // copies: wave w brings rows 64w .. 64w+63 of both operands, 8 rows at a time
    uint32_t va[8], vb[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t row = wave * 64 + i * 8 + (lane >> 3);
        const uint32_t piece = ((lane & 7) ^ ((row >> 1) & 7)) * 16;
        va[i] = min(row, m_last) * row_bytes + piece;
        vb[i] = min(row, n_last) * row_bytes + piece;
    }
    const uint32_t vsa = min((uint32_t)(wave * 64 + lane), m_last) * mark_bytes;
    const uint32_t vsb = min((uint32_t)(wave * 64 + lane), n_last) * mark_bytes;
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
    const uint32_t stages = (granules + 1) / 2;

    auto copy_stage = [&](uint32_t s) {
        const uint32_t at = base + (s & 1) * kSlot + wave * 64 * 128;
        const uint32_t k = min(2 * s, granules - 2) * 64;
#pragma unroll
        for (int i = 0; i < 8; i++) copy_to_lds(at + i * 1024, va[i], ra, k);
#pragma unroll
        for (int i = 0; i < 8; i++) copy_to_lds(at + kTile * 128 + i * 1024, vb[i], rb, k);
        if ((s & 1) == 0) {
            const uint32_t mark = base + 2 * kSlot + ((s >> 1) & 1) * kMarkSlot + wave * 64 * 16;
            const uint32_t ks = min(2 * s, granules - 4) * 4;
            copy_to_lds(mark, vsa, rsa, ks);
            copy_to_lds(mark + kTile * 16, vsb, rsb, ks);
        }
    };

    // fragments: wave w computes rows 128*(w&1) of A against rows 128*(w>>1) of B
    const int r = lane & 31, half = lane >> 5, x = (lane >> 1) & 7;
    const uint32_t arow = (wave & 1) * 128 + r, brow = kTile + (wave >> 1) * 128 + r;
    // 16-byte pieces p and p + 1 of the fragments' rows
    auto read = [&](const uint8_t *codes, uint32_t p, Fragments &f) {
        static_for<4>([&](auto I) {
            constexpr int i = I;
#pragma unroll
            for (int t = 0; t < 2; t++) {
                f.a[i][t] = *(const uint4 *)(codes + (arow + 32 * i) * 128 + ((p ^ x) ^ t) * 16);
                f.b[i][t] = *(const uint4 *)(codes + (brow + 32 * i) * 128 + ((p ^ x) ^ t) * 16);
            }
        });
    };
    // the scales of one granule, at dword k of the group's 4
    auto read_scales = [&](const uint8_t *marks, uint32_t k, Scales &e) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            e.a[i] = *(const uint32_t *)(marks + (arow + 32 * i) * 16 + 4 * k);
            e.b[i] = *(const uint32_t *)(marks + (brow + 32 * i) * 16 + 4 * k);
        }
    };
    auto marks_of = [&](uint32_t s) { return lds + 2 * kSlot + ((s >> 1) & 1) * kMarkSlot; };
    auto window = [&](uint32_t s) { return min(2 * s & ~3u, granules - 4); };   // first granule of s's scales

    f32x16_t acc[4][4] = {};
    copy_stage(0);
    if (stages > 1) copy_stage(1);
    wait_and_meet();
    Fragments f, h;
    Scales e;
    read(lds, 4 * half, f);
    read_scales(marks_of(0), half, e);

    // the 32 products of phase P of a stage, in the order written: after product n
    // come the n-th read of the next phase's fragments, and with COPY the n-th copy
    // of the stage at byte k of the rows, so the matrix cores never wait for the rest
    // to issue.  GROUP: also the scales of the next 4 granules, and the copy of those
    // after them.
    uint4 ga[4], gb[4];
    auto phase = [&](auto P, const Fragments &now, Fragments &then, const uint8_t *codes, auto COPY,
                     uint32_t to, uint32_t k, auto READ_GROUP, const uint8_t *marks, auto COPY_GROUP,
                     uint32_t marks_to) {
        constexpr int ph = P;
        const uint32_t p0 = ((4 * half + (ph ? 0 : 2)) ^ x) * 16;
        static_for<32>([&](auto S) {
            constexpr int s = S, t = s / 16, i = s / 4 % 4, n = s % 4;
            acc[i][n] = mma<2 * ph + t>(now.b[n][t], e.b[n], now.a[i][t], e.a[i], acc[i][n]);
            if constexpr (s < 16) {
                constexpr int u = s / 8, r4 = s % 4;
                if constexpr (s % 8 < 4) then.b[r4][u] = *(const uint4 *)(codes + (brow + 32 * r4) * 128 + (p0 ^ (16 * u)));
                else then.a[r4][u] = *(const uint4 *)(codes + (arow + 32 * r4) * 128 + (p0 ^ (16 * u)));
            } else if constexpr (READ_GROUP && s < 20) {
                gb[s - 16] = *(const uint4 *)(marks + (brow + 32 * (s - 16)) * 16);
            } else if constexpr (READ_GROUP && s < 24) {
                ga[s - 20] = *(const uint4 *)(marks + (arow + 32 * (s - 20)) * 16);
            }
            if constexpr (COPY) {
                if constexpr (s < 8) copy_to_lds(to + s * 1024, va[s], ra, k);
                else if constexpr (s < 16) copy_to_lds(to + kTile * 128 + (s - 8) * 1024, vb[s - 8], rb, k);
                else if constexpr (COPY_GROUP && s == 16) copy_to_lds(marks_to, vsa, rsa, k / 16);
                else if constexpr (COPY_GROUP && s == 17) copy_to_lds(marks_to + kTile * 16, vsb, rsb, k / 16);
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    using no = std::integral_constant<int, 0>;
    using yes = std::integral_constant<int, 1>;

    // two stages at a time while there are two more to copy: every window then lies
    // where the stage number says
    uint32_t s = 0;
    const uint32_t full = granules / 2;
    if (full >= 4) {
        const uint32_t codes_to = base + wave * 64 * 128, marks_to = base + 2 * kSlot + wave * 64 * 16;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            ga[i] = *(const uint4 *)(marks_of(0) + (arow + 32 * i) * 16);
            gb[i] = *(const uint4 *)(marks_of(0) + (brow + 32 * i) * 16);
        }
        for (; s + 4 <= full; s += 2) {
            const uint32_t next = ((s >> 1) & 1) ^ 1;
            phase(no{}, f, h, lds, no{}, 0, 0, no{}, lds, no{}, 0);
            wait_and_meet();
            phase(yes{}, h, f, lds + kSlot, yes{}, codes_to, (s + 2) * 128, no{}, lds, yes{},
                  marks_to + next * kMarkSlot);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                e.a[i] = half ? ga[i].w : ga[i].z;
                e.b[i] = half ? gb[i].w : gb[i].z;
            }
            phase(no{}, f, h, lds + kSlot, no{}, 0, 0, no{}, lds, no{}, 0);
            wait_and_meet();
            phase(yes{}, h, f, lds, yes{}, codes_to + kSlot, (s + 3) * 128, yes{},
                  lds + 2 * kSlot + next * kMarkSlot, no{}, 0);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                e.a[i] = half ? ga[i].y : ga[i].x;
                e.b[i] = half ? gb[i].y : gb[i].x;
            }
        }
        // the group's scales may have come from a window that is pulled back
        read_scales(marks_of(s), 2 * s - window(s) + half, e);
    }
    for (; s < full; s++) {
        read(lds + (s & 1) * kSlot, 4 * half + 2, h);
        products<0>(f, e, acc);
        wait_and_meet();
        if (s + 2 < stages) copy_stage(s + 2);
        products<1>(h, e, acc);
        if (s + 1 < full) {
            read(lds + ((s + 1) & 1) * kSlot, 4 * half, f);
            read_scales(marks_of(s + 1), 2 * s + 2 - window(s + 1) + half, e);
        }
    }
    if (granules & 1) {                                  // the last granule, alone
        read(lds + (full & 1) * kSlot, 4 + 2 * half, f);
        read_scales(marks_of(full), granules - 1 - window(full), e);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            e.a[i] >>= 16 * half;
            e.b[i] >>= 16 * half;
        }
        products<0>(f, e, acc);
    }

#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int64_t m = m0 + (wave & 1) * 128 + 32 * i + r;
        if (m >= M) continue;
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int64_t n = n0 + (wave >> 1) * 128 + 32 * j + 8 * q + 4 * half;
                const float v[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                store4<CT>(c, m * ldc + n, N - n < 4 ? (int)(N - n) : 4, v);
            }
    }
}

template <int CT>
hipError_t run_matmul(const uint8_t *a, const uint8_t *as, const uint8_t *b, const uint8_t *bs,
                      int64_t M, int64_t N, int64_t granules, void *c, int64_t ldc, hipStream_t st) {
    if (M > 128 && N > 128 && granules >= 4 && granules < (1 << 18)) {
        const int64_t bm = (M + kTile - 1) / kTile, bn = (N + kTile - 1) / kTile;
        hipLaunchKernelGGL((k_mx_matmul_big<CT>), dim3((unsigned)(bm * bn)), dim3(kThreads), 0, st, a, as, b,
                           bs, M, N, (uint32_t)granules, (uint32_t)bm, (uint32_t)bn, c, ldc);
        return hipGetLastError();
    }
    const int64_t mt = (M + 127) / 128, nt = (N + 127) / 128;
    if (mt * nt > kMaxGroups) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_mx_matmul<CT>), dim3((unsigned)(mt * nt)), dim3(kThreads), 0, st, a, as, b, bs, M,
                       N, granules, (uint32_t)mt, c, ldc);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_matmul(const uint8_t *a, const uint8_t *as, const uint8_t *b, const uint8_t *bs,
                            int64_t M, int64_t N, int64_t granules, void *c, int ct, int64_t ldc,
                            hipStream_t st) {
    switch (ct) {
    case F16: return run_matmul<F16>(a, as, b, bs, M, N, granules, c, ldc, st);
    case BF16: return run_matmul<BF16>(a, as, b, bs, M, N, granules, c, ldc, st);
    case F32: return run_matmul<F32>(a, as, b, bs, M, N, granules, c, ldc, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qcp
