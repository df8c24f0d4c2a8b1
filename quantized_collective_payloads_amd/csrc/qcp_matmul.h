// qcp_matmul.h -- what the products on the matrix cores share: how tiles of C are dealt
// to the XCDs, copies from memory to LDS, and the stores of a fragment of C.
#pragma once

#include <algorithm>

#include "qcp_device.h"
#include "qcp_launch.h"

namespace qcp {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int kCUs = 256;

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

// What a product takes in a kernel of square tiles, in units of 10 ns, from measured parts: a
// stage while the GPU is half full and when it is full (where the clock gives way to the power
// that the matrix cores draw, and the caches are shared), and a round beside its stages.
struct Form {
    int side, stage, resident;   // of its tiles, bytes or values of K in a stage, work-groups that the GPU holds
    int half, full, beside;
    int64_t tiles(int64_t M, int64_t N) const { return ((M + side - 1) / side) * ((N + side - 1) / side); }
    int64_t price(int64_t groups, int64_t stages) const {
        const int64_t last = groups % resident, over = std::max<int64_t>(0, 2 * last - resident);
        const int64_t step = half + (full - half) * over / resident;
        return groups / resident * (stages * full + beside) + (last ? stages * step + beside : 0);
    }
};

// Which tile of C work-group t takes.  Work-groups are dealt round-robin to the 8 XCDs:
// each gets a contiguous run of tiles and walks it 4 tiles of M by N, so that the tiles
// an XCD works on at a time share few operand panels in its L2.
struct TilePlace {
    uint32_t m, n;
};
__device__ __forceinline__ TilePlace tile_place(uint32_t t, uint32_t m_tiles, uint32_t n_tiles) {
    const uint32_t tiles = m_tiles * n_tiles, per = tiles / 8, extra = tiles % 8, xcd = t % 8;
    t = xcd * per + min(xcd, extra) + t / 8;
    const uint32_t band = 4 * n_tiles, first = t / band * 4, height = min(4u, m_tiles - first);
    const uint32_t in = t - t / band * band;
    return TilePlace{first + in % height, in / height};
}

// A fragment of C: lane r of a half-wave has row m, and of columns n + 8q + 4 * half + 0..3
// register group q.  16-bit results go out 16 bytes a lane: the half-waves swap groups, so
// that the lower one has columns n + 16k + 0..7 and the upper one 8..15.
template <int CT>
__device__ __forceinline__ void store_fragment(const f32x16_t &v, void *c, int64_t ldc, int64_t m, int64_t n,
                                               int half, int64_t M, int64_t N, bool whole) {
    if constexpr (CT == F32) {
        if (!whole && m >= M) return;
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int64_t at = n + 8 * q + 4 * half;
            const float r[4] = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            store4<CT>(c, m * ldc + at, whole || N - at >= 4 ? 4 : (int)(N - at), r);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 2; k++) {
            uint32_t w[4];
#pragma unroll
            for (int d = 0; d < 2; d++) {
                const uint32_t lo = narrow2<CT>(v[8 * k + 2 * d], v[8 * k + 2 * d + 1]);
                const uint32_t hi = narrow2<CT>(v[8 * k + 4 + 2 * d], v[8 * k + 5 + 2 * d]);
                const auto swapped = __builtin_amdgcn_permlane32_swap(lo, hi, false, false);
                w[d] = swapped[0];
                w[2 + d] = swapped[1];
            }
            const int64_t at = n + 16 * k + 8 * half;
            uint16_t *p = (uint16_t *)c + m * ldc + at;
            typedef u32x4_t u32x4_any __attribute__((aligned(2)));
            if (whole || (m < M && N - at >= 8)) {
                *(u32x4_any *)p = u32x4_t{w[0], w[1], w[2], w[3]};
            } else if (m < M) {
#pragma unroll
                for (int e = 0; e < 8; e++)
                    if (at + e < N) p[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
            }
        }
    }
}

// 64 lanes x 16 bytes from rsrc[voff + soff] to LDS at `lds` + 16 * lane.  The
// caller waits for it with wait_and_meet; no vector register is written.  The
// instruction takes the LDS address from m0, which is an operand here, so that the
// compiler knows what it holds.  The compiler does not count wait states into an asm
// statement: the s_nop holds the five that a scalar register needs between a vector
// instruction that writes it (v_readlane, which restores a spilled one) and a memory
// instruction that reads it, and the one that m0 needs.  The range check, which reads zeros
// past the end of the buffer, is relied on for voff alone: with a soff other than 0 their sum
// has to end within the buffer by itself.
__device__ __forceinline__ void copy_to_lds(uint32_t lds, uint32_t voff, i32x4_t rsrc, uint32_t soff) {
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :
                 : "v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane((int)soff)),
                   "{m0}"(__builtin_amdgcn_readfirstlane((int)lds))
                 : "memory");
}

// until at most N of this wave's copies are in flight; then with the other waves
template <int N>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __forceinline__ void wait_lds_and_meet() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ i32x4_t buffer_of(const void *p, uint64_t bytes) {
    const uint64_t at = (uint64_t)p;
    const uint32_t n = bytes > 0xfffffffcull ? 0xfffffffcu : (uint32_t)bytes;
    return i32x4_t{__builtin_amdgcn_readfirstlane((int)(uint32_t)at),
                   __builtin_amdgcn_readfirstlane((int)(uint32_t)(at >> 32)),
                   __builtin_amdgcn_readfirstlane((int)n), 0x00020000};
}

// as copy_to_lds, 4 bytes a lane
__device__ __forceinline__ void copy4_to_lds(uint32_t lds, uint32_t voff, i32x4_t rsrc) {
    asm volatile("s_nop 4\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 :
                 : "v"(voff), "s"(rsrc), "{m0}"(__builtin_amdgcn_readfirstlane((int)lds))
                 : "memory");
}

// 16 bytes and 4 bytes of LDS at a byte address
__device__ __forceinline__ u32x4_t lds16(uint32_t at) {
    return *(const __attribute__((address_space(3))) u32x4_t *)at;
}
__device__ __forceinline__ uint32_t lds4(uint32_t at) {
    return *(const __attribute__((address_space(3))) uint32_t *)at;
}

}  // namespace qcp
