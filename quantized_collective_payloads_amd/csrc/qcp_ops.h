// qcp_ops.h -- internal launchers of the optimizer step and of the MXFP4 and INT8 payloads.
// As in qcp_launch.h, arguments are already validated by the caller (qcp_ops_api.hip).
#pragma once

#include "qcp_launch.h"

namespace qcp {

// AdamW over n tensors (tensors without elements left out); see qcp_adamw.hip
struct AdamwTensor {
    float *param;
    const void *grad;
    void *copy;            // null: no 16-bit copy
    int64_t n;
    int64_t offset;        // first element's place in the moments
};
struct AdamwConst {
    void *m, *v;           // fp32, or E4M3 codes of m and sqrt(v)
    float *m_scales, *v_scales;
    const float *grad_scale;
    float beta1, one_beta1, beta2, one_beta2, decay, step_size, root_scale, eps;
    uint32_t key;
    int copy_type;
};
template <int CAP> struct AdamwTable {
    AdamwTensor t[CAP];
    uint32_t first[CAP];   // first work-group of each tensor; ~0 past the last
};
hipError_t launch_adamw(const AdamwTensor *t, int n, int gt, int state, int G, const AdamwConst &c,
                        hipStream_t st);

// the MXFP4 payload of x (transpose: of x^T), and back; see qcp_mxfp4.hip
hipError_t launch_mx_quantize(const void *x, int xt, int64_t rows, int64_t cols, int64_t ld,
                              int transpose, uint8_t *codes, uint8_t *scales, hipStream_t st);
hipError_t launch_mx_quantize_both(const void *x, int xt, int64_t rows, int64_t cols, int64_t ld,
                                   uint8_t *codes, uint8_t *scales, uint8_t *codes_t, uint8_t *scales_t,
                                   hipStream_t st);
hipError_t launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows,
                                int64_t cols, void *y, int yt, int64_t ld, hipStream_t st);

// C[M, N] = A B^T, rows of `granules` times 128 values; see qcp_mxfp4_matmul.hip.
// work: null, or room for slices * M * N floats, slices of K as many as said here
int mx_matmul_slices(int64_t M, int64_t N, int64_t granules);
hipError_t launch_mx_matmul(const uint8_t *a, const uint8_t *as, const uint8_t *b, const uint8_t *bs,
                            int64_t M, int64_t N, int64_t granules, void *c, int ct, int64_t ldc,
                            float *work, hipStream_t st);

// the INT8 payload of x with one scale per row, and back; see qcp_int8.hip
hipError_t launch_int8_quantize(const void *x, int xt, int64_t rows, int64_t cols, int64_t ld, uint8_t *codes,
                                float *scales, hipStream_t st);
hipError_t launch_int8_dequantize(const uint8_t *codes, const float *scales, int64_t rows, int64_t cols, void *y,
                                  int yt, int64_t ld, hipStream_t st);

// C[M, N] = A B^T, rows of `stages` times 128 codes; see qcp_int8_matmul.hip.
// work: null, or room for slices * M * N integers, slices of K as many as said here
int int8_matmul_slices(int64_t M, int64_t N, int64_t stages);
hipError_t launch_int8_matmul(const uint8_t *a, const float *as, const uint8_t *b, const float *bs, int64_t M,
                              int64_t N, int64_t stages, void *c, int ct, int64_t ldc, int *work, hipStream_t st);

// Y[M, N] = Q(x) B^T for few rows of 16 bits, in one launch; `few`: whether they are
bool int8_linear_few(int64_t M, int64_t N, int64_t stages);
hipError_t launch_int8_linear_rows(const void *x, int xt, int64_t ldx, int64_t M, int64_t K, const uint8_t *b,
                                   const float *bs, int64_t N, int64_t stages, void *y, int64_t ldy, hipStream_t st);

// C[M, N] = A X for a 16-bit A (transpose: given as [K, M]) and the payload of X [K, N];
// see qcp_int8_mixed.hip.  work: null, or as many bytes as said here; aligned: what the other
// function says of a
int64_t int8_mixed_work(int64_t M, int64_t N, int64_t K, int transpose, bool aligned);
bool int8_mixed_aligned(const void *a, int64_t lda);
hipError_t launch_int8_mixed(const void *a, int at, int64_t lda, int transpose, const uint8_t *codes,
                             const float *scales, int64_t M, int64_t N, int64_t K, void *c, int ct, int64_t ldc,
                             void *work, hipStream_t st);

// the counter hash of the stochastic rounding: an invertible scramble of 32 bits
// (two rounds of xor-shift and an odd multiplier, the fractions of sqrt 2 and sqrt 3)
__host__ __device__ inline uint32_t adamw_mix(uint32_t x) {
    x ^= x >> 16;
    x *= 0x6a09e667u;
    x ^= x >> 15;
    x *= 0xbb67ae85u;
    return x ^ (x >> 16);
}

}  // namespace qcp
