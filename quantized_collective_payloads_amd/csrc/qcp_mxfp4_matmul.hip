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

template <int CT>
hipError_t run_matmul(const uint8_t *a, const uint8_t *as, const uint8_t *b, const uint8_t *bs,
                      int64_t M, int64_t N, int64_t granules, void *c, int64_t ldc, hipStream_t st) {
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
