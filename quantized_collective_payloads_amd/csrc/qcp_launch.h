// qcp_launch.h -- internal launchers behind the C-ABI (one per kernel family).
// Arguments are already validated by the caller (qcp_api.hip); each launcher
// picks the template instance for (dtype, format, G) and enqueues it on `st`.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qcp {

// blockwise quantize + pack: x[n] of dtype xt -> codes (fmt), scales
hipError_t launch_encode(const void *x, int xt, int64_t n, int G, int fmt, uint8_t *codes,
                         float *scales, hipStream_t st);

// qgZ sender: tensor-slice reordering of x[n] (n_nodes x gpus_per_node chunks)
// fused with the quantization of the gpus_per_node slices it produces
hipError_t launch_encode_reorder(const void *x, int xt, int64_t n, int n_nodes,
                                 int gpus_per_node, int G, int fmt, uint8_t *codes,
                                 int64_t slice_stride, float *scales, int64_t scale_stride,
                                 hipStream_t st);

// sub-byte pack / unpack with interleaved metadata: one record per block,
// [fp32 scale][G*b/8 code bytes]
hipError_t launch_encode_records(const void *x, int xt, int64_t n, int G, int b, uint8_t *records,
                                 hipStream_t st);
hipError_t launch_decode_records(const uint8_t *records, int64_t n, int G, int b, void *y, int yt,
                                 hipStream_t st);

// unpack + dequantize: codes (fmt), scales -> y[n] of dtype yt
hipError_t launch_decode(const uint8_t *codes, const float *scales, int fmt, int64_t n, int G,
                         void *y, int yt, hipStream_t st);

// N-slice dequantize -> fp32 fmaf chain -> requantize
hipError_t launch_reduce(const uint8_t *codes_in, int64_t slice_stride, const float *scales_in,
                         int64_t scale_stride, int n_slices, int64_t L, int G, int fmt_in,
                         int fmt_out, uint8_t *codes_out, float *scales_out, float *sum_out,
                         hipStream_t st);

// in-place FP8 main-gradient accumulate
hipError_t launch_accum(uint8_t *state_codes, float *state_scales, const void *grad, int gt,
                        int64_t n, int G, hipStream_t st);

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

// C[M, N] = A B^T, rows of `granules` times 128 values; see qcp_mxfp4_matmul.hip
hipError_t launch_mx_matmul(const uint8_t *a, const uint8_t *as, const uint8_t *b, const uint8_t *bs,
                            int64_t M, int64_t N, int64_t granules, void *c, int ct, int64_t ldc,
                            hipStream_t st);

// the counter hash of the stochastic rounding: an invertible scramble of 32 bits
// (two rounds of xor-shift and an odd multiplier, the fractions of sqrt 2 and sqrt 3)
__host__ __device__ inline uint32_t adamw_mix(uint32_t x) {
    x ^= x >> 16;
    x *= 0x6a09e667u;
    x ^= x >> 15;
    x *= 0xbb67ae85u;
    return x ^ (x >> 16);
}

// workgroups of 4 waves; each kernel derives its wave index from the
// work-group and work-item ids
constexpr int kThreads = 256;
constexpr int kWavesPerGroup = kThreads / 64;

// Work-item and work-group ids read through the compiler builtins.  (HIP's
// threadIdx / blockIdx / gridDim go through device-library functions that are
// compiled with different floating-point attributes than this library, so
// they are not inlined: every kernel would start with two function calls.)
__device__ __forceinline__ int lane_id() { return (int)(__builtin_amdgcn_workitem_id_x() & 63u); }
__device__ __forceinline__ int64_t wave_id() {
    return (int64_t)__builtin_amdgcn_workgroup_id_x() * kWavesPerGroup +
           (__builtin_amdgcn_workitem_id_x() >> 6);
}
__device__ __forceinline__ int64_t group_y() { return (int64_t)__builtin_amdgcn_workgroup_id_y(); }

// Work-groups per launch: a dispatch holds at most 2^32 - 1 work-items.  The
// entry points reject element counts whose grid would exceed this (QCP_EINVAL)
// before any launch; grid_for_waves returns 0 -- a launch the runtime refuses --
// should a grid still be too large.
constexpr int64_t kMaxGroups = ((int64_t)1 << 32) / kThreads - 1;

inline unsigned grid_for_waves(int64_t waves) {
    const int64_t groups = (waves + kWavesPerGroup - 1) / kWavesPerGroup;
    return groups <= kMaxGroups ? (unsigned)groups : 0u;
}

}  // namespace qcp
