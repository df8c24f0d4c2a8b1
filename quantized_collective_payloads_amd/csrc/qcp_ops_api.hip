// qcp_ops_api.hip -- the extern "C" entry points of the optimizer step and of the
// MXFP4 and INT8 payloads and their products (include/qcp.h).
//
// As in qcp_api.hip: each validates its arguments on the host (no HIP call is made for
// a rejected call or one without work), enqueues on the caller's stream (one kernel;
// adamw_step one per 64 tensors, a sliced product two) and maps a launch error to
// QCP_EHIP.  Nothing is allocated on the device and no state is kept between calls.
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <new>

#include "qcp.h"
#include "qcp_ops.h"

namespace {

// the library's limit on elements, as in qcp_api.hip
constexpr int64_t kMaxElems = qcp::kMaxGroups * 4096;

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
bool valid_g(int32_t G) { return G >= 32 && G <= 1024 && (G & (G - 1)) == 0; }
bool valid_dtype(int t) { return t == QCP_F16 || t == QCP_BF16 || t == QCP_F32; }
int64_t dtype_bytes(int t) { return t == QCP_F32 ? 4 : 2; }
int64_t n_blocks(int64_t n, int32_t G) { return (n + G - 1) / G; }
int status_of(hipError_t e) { return e == hipSuccess ? QCP_OK : QCP_EHIP; }

// do [a, a+na) and [b, b+nb) intersect?
bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return na > 0 && nb > 0 && a0 < b0 + (uintptr_t)nb && b0 < a0 + (uintptr_t)na;
}

// a range of memory that a call touches
struct Range {
    uintptr_t at, end;
    bool written;
};

// does any written range meet another one?  The ranges are sorted by where they
// begin; then a range meets an earlier one exactly if it begins before the
// furthest end so far (of all ranges, or of the written ones if it is only read).
bool ranges_clash(Range *r, int64_t n) {
    std::sort(r, r + n, [](const Range &a, const Range &b) { return a.at < b.at; });
    uintptr_t all = 0, written = 0;
    for (int64_t i = 0; i < n; i++) {
        if (r[i].at < (r[i].written ? all : written)) return true;
        all = std::max(all, r[i].end);
        if (r[i].written) written = std::max(written, r[i].end);
    }
    return false;
}

// a matrix of rows x cols elements with ld elements between rows: its bytes from
// the first element to the last
int check_matrix(int64_t rows, int64_t cols, int64_t ld, int t, int64_t *bytes) {
    if (rows < 0 || cols < 0 || rows > kMaxElems || cols > kMaxElems || !valid_dtype(t)) return QCP_EINVAL;
    if (ld < cols || ld > kMaxElems) return QCP_EINVAL;
    *bytes = 0;
    if (rows == 0 || cols == 0) return QCP_OK;
    if (rows > 1 && ld > 0 && (rows - 1) > (INT64_MAX / 8 - cols) / ld) return QCP_EINVAL;
    *bytes = ((rows - 1) * ld + cols) * dtype_bytes(t);
    return QCP_OK;
}

// a payload of `lines` rows of n values: the padded row length.  Rows of at most
// 2^31 values keep every position within a row in 32 bits and the column-wise
// quantize's grid (one work-group per 256 x 64 values) within one launch.
bool mx_payload(int64_t lines, int64_t n, int64_t *pad) {
    *pad = (n + 127) / 128 * 128;
    return *pad == 0 || (n <= (int64_t)1 << 31 && lines <= kMaxElems / *pad);
}

// an INT8 payload of `lines` rows of n codes: the padded row length.  As above, positions
// within a row are 32 bits.
bool int8_payload(int64_t lines, int64_t n, int64_t *pad) { return mx_payload(lines, n, pad); }

// sums of products of codes stay within 32 bits: 130944 * 128 * 128 < 2^31
constexpr int64_t kInt8MaxK = 130944;
// the mixed product: 128 rows of the payload and 256 of a, in bytes, are 32-bit offsets
constexpr int64_t kMixedMaxN = (int64_t)1 << 24, kMixedMaxLd = (int64_t)1 << 23;
// and its tiles of C, 256 x 256, a launch's work-groups
bool mixed_tiles(int64_t M, int64_t N) {
    return N <= 0 || (M + 255) / 256 <= qcp::kMaxGroups / 2 / ((N + 255) / 256);
}

// The arguments that adamw_step checks, by their names there
struct AdamwArgs {
    float *const *params;
    const void *const *grads;
    void *const *copies;
    const int64_t *sizes, *offsets;
    int64_t n_tensors;
    int gt, ct, state;
    void *m;
    float *m_scales;
    void *v;
    float *v_scales;
    int64_t n_state;
    int32_t G;
    int64_t step;
    double lr, beta1, beta2, eps, weight_decay;
    const float *grad_scale;
};

// ranges that a step over n tensors touches, at most
constexpr int64_t adamw_ranges(int64_t n) { return 3 * n + 5; }

// All but the overlaps.  *live: tensors with elements; *past: the end of the last
// tensor's blocks in the moments
int check_adamw(const AdamwArgs &a, int64_t *live, int64_t *past) {
    *live = *past = 0;
    if (a.n_tensors < 0 || a.n_state < 0 || !valid_g(a.G)) return QCP_EINVAL;
    if (!valid_dtype(a.gt) || (a.state != QCP_F32 && a.state != QCP_E4M3)) return QCP_EINVAL;
    if (a.copies && a.ct != QCP_F16 && a.ct != QCP_BF16) return QCP_EINVAL;
    // the denominator is at least eps, and the device's reciprocal takes what is below
    // the least normal number for 0
    const bool scalars = a.step >= 1 && isfinite(a.lr) && a.lr >= 0 && a.beta1 >= 0 && a.beta1 < 1 && a.beta2 >= 0 &&
                         a.beta2 < 1 && isfinite(a.eps) && (float)a.eps >= 0x1p-126f && isfinite(a.weight_decay) &&
                         a.weight_decay >= 0;
    if (!scalars) return QCP_EINVAL;
    if (a.n_tensors == 0) return QCP_OK;
    if (!a.params || !a.grads || !a.sizes || !a.offsets) return QCP_EINVAL;
    const bool eight = a.state == QCP_E4M3;
    for (int64_t i = 0; i < a.n_tensors; i++) {
        const int64_t n = a.sizes[i];
        if (n < 0 || n > kMaxElems) return QCP_EINVAL;
        if (a.offsets[i] < *past || a.offsets[i] % a.G != 0) return QCP_EINVAL;
        if (a.offsets[i] > a.n_state || n_blocks(n, a.G) > (a.n_state - a.offsets[i]) / a.G) return QCP_EINVAL;
        *past = a.offsets[i] + n_blocks(n, a.G) * a.G;
        if (n == 0) continue;
        ++*live;
        if (!a.params[i] || !a.grads[i] || (a.copies && !a.copies[i])) return QCP_EINVAL;
        if ((uintptr_t)a.params[i] % 4 || (uintptr_t)a.grads[i] % dtype_bytes(a.gt)) return QCP_EALIGN;
        if (a.copies && (uintptr_t)a.copies[i] % 2) return QCP_EALIGN;
    }
    if (*live == 0) return QCP_OK;
    if (!a.m || !a.v || (eight && (!a.m_scales || !a.v_scales))) return QCP_EINVAL;
    if (!aligned16(a.m) || !aligned16(a.v)) return QCP_EALIGN;
    if (eight && (!aligned16(a.m_scales) || !aligned16(a.v_scales))) return QCP_EALIGN;
    if ((uintptr_t)a.grad_scale % 4) return QCP_EALIGN;
    return QCP_OK;
}

// does a buffer that a step writes meet another one?  r: room for adamw_ranges(n_tensors)
bool adamw_clash(const AdamwArgs &a, int64_t past, Range *r) {
    const bool eight = a.state == QCP_E4M3;
    int64_t k = 0;
    auto range = [&](const void *p, int64_t bytes, bool written) {
        if (p && bytes > 0) r[k++] = Range{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, written};
    };
    for (int64_t i = 0; i < a.n_tensors; i++) {
        const int64_t n = a.sizes[i];
        if (n == 0) continue;
        range(a.params[i], 4 * n, true);
        range(a.grads[i], n * dtype_bytes(a.gt), false);
        if (a.copies) range(a.copies[i], 2 * n, true);
    }
    range(a.m, eight ? past : 4 * past, true);
    range(a.v, eight ? past : 4 * past, true);
    if (eight) {
        range(a.m_scales, past / a.G * 4, true);
        range(a.v_scales, past / a.G * 4, true);
    }
    range(a.grad_scale, 4, false);
    return ranges_clash(r, k);
}

}  // namespace

extern "C" {

int qcp_adamw_check(float *const *params, const void *const *grads, void *const *copies,
                    const int64_t *sizes, const int64_t *offsets, int64_t n_tensors, int gt, int ct,
                    int state, void *m, float *m_scales, void *v, float *v_scales, int64_t n_state,
                    int32_t G, int64_t step, double lr, double beta1, double beta2, double eps,
                    double weight_decay, const float *grad_scale) {
    const AdamwArgs a = {params, grads, copies, sizes, offsets, n_tensors, gt, ct, state, m, m_scales, v, v_scales,
                         n_state, G, step, lr, beta1, beta2, eps, weight_decay, grad_scale};
    int64_t live, past;
    const int rc = check_adamw(a, &live, &past);
    if (rc != QCP_OK || live == 0) return rc;
    // live tensors were all looked at, so their number is that of a real array
    Range *r = new (std::nothrow) Range[adamw_ranges(n_tensors)];
    if (!r) return QCP_EUNSUPPORTED;
    const bool clash = adamw_clash(a, past, r);
    delete[] r;
    return clash ? QCP_EINVAL : QCP_OK;
}

int adamw_step(float *const *params, const void *const *grads, void *const *copies,
               const int64_t *sizes, const int64_t *offsets, int32_t n_tensors, int gt, int ct,
               int state, void *m, float *m_scales, void *v, float *v_scales, int64_t n_state,
               int32_t G, int64_t step, double lr, double beta1, double beta2, double eps,
               double weight_decay, const float *grad_scale, uint64_t seed, void *stream) {
    if (n_tensors > QCP_ADAMW_MAX_TENSORS) return QCP_EINVAL;
    const AdamwArgs a = {params, grads, copies, sizes, offsets, n_tensors, gt, ct, state, m, m_scales, v, v_scales,
                         n_state, G, step, lr, beta1, beta2, eps, weight_decay, grad_scale};
    int64_t live, past;
    const int rc = check_adamw(a, &live, &past);
    if (rc != QCP_OK || live == 0) return rc;

    // 41 KB and 74 KB of the caller's stack
    qcp::AdamwTensor t[QCP_ADAMW_MAX_TENSORS];
    Range r[adamw_ranges(QCP_ADAMW_MAX_TENSORS)];
    if (adamw_clash(a, past, r)) return QCP_EINVAL;
    for (int32_t i = 0, at = 0; i < n_tensors; i++)
        if (sizes[i] > 0)
            t[at++] = qcp::AdamwTensor{params[i], grads[i], copies ? copies[i] : nullptr, sizes[i], offsets[i]};

    uint32_t key = 0;
    for (uint32_t word : {(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)step, (uint32_t)((uint64_t)step >> 32)})
        key = qcp::adamw_mix(key + word + 0x9e3779b9u);
    qcp::AdamwConst c = {};
    c.m = m;
    c.v = v;
    c.m_scales = m_scales;
    c.v_scales = v_scales;
    c.grad_scale = grad_scale;
    c.beta1 = (float)beta1;
    c.one_beta1 = (float)(1 - beta1);
    c.beta2 = (float)beta2;
    c.one_beta2 = (float)(1 - beta2);
    c.decay = (float)(1 - lr * weight_decay);
    c.step_size = (float)(lr / (1 - pow(beta1, (double)step)));
    c.root_scale = (float)(1 / sqrt(1 - pow(beta2, (double)step)));
    c.eps = (float)eps;
    c.key = key;
    c.copy_type = ct;
    return status_of(qcp::launch_adamw(t, (int)live, gt, state, G, c, (hipStream_t)stream));
}

int mxfp4_quantize(const void *x, int xt, int64_t rows, int64_t cols, int64_t ld, int32_t transpose,
                   uint8_t *codes, uint8_t *scales, void *stream) {
    int64_t xb, pad;
    int rc = check_matrix(rows, cols, ld, xt, &xb);
    if (rc != QCP_OK) return rc;
    if (transpose != 0 && transpose != 1) return QCP_EINVAL;
    if (rows == 0 || cols == 0) return QCP_OK;
    const int64_t lines = transpose ? cols : rows;
    if (!mx_payload(lines, transpose ? rows : cols, &pad)) return QCP_EINVAL;
    if (!x || !codes || !scales) return QCP_EINVAL;
    if ((uintptr_t)x % dtype_bytes(xt) || !aligned16(codes) || !aligned16(scales)) return QCP_EALIGN;
    const int64_t cb = lines * pad / 2, sb = lines * pad / 32;
    if (overlap(x, xb, codes, cb) || overlap(x, xb, scales, sb) || overlap(codes, cb, scales, sb))
        return QCP_EINVAL;
    return status_of(qcp::launch_mx_quantize(x, xt, rows, cols, ld, transpose, codes, scales,
                                             (hipStream_t)stream));
}

int mxfp4_quantize_both(const void *x, int xt, int64_t rows, int64_t cols, int64_t ld, uint8_t *codes,
                        uint8_t *scales, uint8_t *codes_t, uint8_t *scales_t, void *stream) {
    int64_t xb, pad, pad_t;
    int rc = check_matrix(rows, cols, ld, xt, &xb);
    if (rc != QCP_OK) return rc;
    if (rows == 0 || cols == 0) return QCP_OK;
    if (!mx_payload(rows, cols, &pad) || !mx_payload(cols, rows, &pad_t)) return QCP_EINVAL;
    if (!x || !codes || !scales || !codes_t || !scales_t) return QCP_EINVAL;
    if ((uintptr_t)x % dtype_bytes(xt) || !aligned16(codes) || !aligned16(scales) || !aligned16(codes_t) ||
        !aligned16(scales_t))
        return QCP_EALIGN;
    const void *at[5] = {x, codes, scales, codes_t, scales_t};
    const int64_t bytes[5] = {xb, rows * pad / 2, rows * pad / 32, cols * pad_t / 2, cols * pad_t / 32};
    for (int i = 0; i < 5; i++)
        for (int j = i + 1; j < 5; j++)
            if (overlap(at[i], bytes[i], at[j], bytes[j])) return QCP_EINVAL;
    return status_of(qcp::launch_mx_quantize_both(x, xt, rows, cols, ld, codes, scales, codes_t, scales_t,
                                                  (hipStream_t)stream));
}

int mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, void *y,
                     int yt, int64_t ld, void *stream) {
    int64_t yb, pad;
    int rc = check_matrix(rows, cols, ld, yt, &yb);
    if (rc != QCP_OK) return rc;
    if (rows == 0 || cols == 0) return QCP_OK;
    if (!mx_payload(rows, cols, &pad)) return QCP_EINVAL;
    if (!codes || !scales || !y) return QCP_EINVAL;
    if (!aligned16(codes) || !aligned16(scales) || (uintptr_t)y % dtype_bytes(yt)) return QCP_EALIGN;
    if (overlap(y, yb, codes, rows * pad / 2) || overlap(y, yb, scales, rows * pad / 32)) return QCP_EINVAL;
    return status_of(qcp::launch_mx_dequantize(codes, scales, rows, cols, y, yt, ld, (hipStream_t)stream));
}

int mxfp4_matmul_sliced(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *b_codes,
                        const uint8_t *b_scales, int64_t M, int64_t N, int64_t K, void *c, int ct,
                        int64_t ldc, void *work, int64_t work_bytes, void *stream) {
    int64_t cb, pad;
    int rc = check_matrix(M, N, ldc, ct, &cb);
    if (rc != QCP_OK) return rc;
    if (K < 0) return QCP_EINVAL;
    if (M == 0 || N == 0) return QCP_OK;
    if (!mx_payload(M, K, &pad) || !mx_payload(N, K, &pad)) return QCP_EINVAL;
    if ((M + 127) / 128 > qcp::kMaxGroups / ((N + 127) / 128)) return QCP_EINVAL;   // tiles of C
    if (!c || (K > 0 && (!a_codes || !a_scales || !b_codes || !b_scales))) return QCP_EINVAL;
    const int64_t need = work ? qcp_mxfp4_matmul_work(M, N, K) : 0;
    if (work_bytes < need) return QCP_EINVAL;
    if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(b_codes) || !aligned16(b_scales) ||
        !aligned16(work) || (uintptr_t)c % dtype_bytes(ct))
        return QCP_EALIGN;
    const void *in[4] = {a_codes, a_scales, b_codes, b_scales};
    const int64_t bytes[4] = {M * pad / 2, M * pad / 32, N * pad / 2, N * pad / 32};
    if (overlap(c, cb, work, need)) return QCP_EINVAL;
    for (int i = 0; i < 4; i++)
        if (overlap(c, cb, in[i], bytes[i]) || overlap(work, need, in[i], bytes[i])) return QCP_EINVAL;
    return status_of(qcp::launch_mx_matmul(a_codes, a_scales, b_codes, b_scales, M, N, pad / 128, c, ct,
                                           ldc, need ? (float *)work : nullptr, (hipStream_t)stream));
}

int mxfp4_matmul(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *b_codes,
                 const uint8_t *b_scales, int64_t M, int64_t N, int64_t K, void *c, int ct, int64_t ldc,
                 void *stream) {
    return mxfp4_matmul_sliced(a_codes, a_scales, b_codes, b_scales, M, N, K, c, ct, ldc, nullptr, 0, stream);
}

int64_t qcp_mxfp4_matmul_work(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0 || M > kMaxElems || N > kMaxElems || K > kMaxElems) return -1;
    const int slices = qcp::mx_matmul_slices(M, N, (K + 127) / 128);
    return slices > 1 ? 4 * slices * M * N : 0;
}

int64_t qcp_mxfp4_padded(int64_t n) { return n < 0 || n > kMaxElems ? -1 : (n + 127) / 128 * 128; }

int int8_quantize(const void *x, int xt, int64_t rows, int64_t cols, int64_t ld, uint8_t *codes, float *scales,
                  void *stream) {
    int64_t xb, pad;
    int rc = check_matrix(rows, cols, ld, xt, &xb);
    if (rc != QCP_OK) return rc;
    if (rows == 0) return QCP_OK;
    if (!int8_payload(rows, cols, &pad)) return QCP_EINVAL;
    if (!scales || (cols > 0 && (!x || !codes))) return QCP_EINVAL;
    if ((uintptr_t)x % dtype_bytes(xt) || !aligned16(codes) || !aligned16(scales)) return QCP_EALIGN;
    if (overlap(x, xb, codes, rows * pad) || overlap(x, xb, scales, rows * 4) ||
        overlap(codes, rows * pad, scales, rows * 4))
        return QCP_EINVAL;
    return status_of(qcp::launch_int8_quantize(x, xt, rows, cols, ld, codes, scales, (hipStream_t)stream));
}

int int8_dequantize(const uint8_t *codes, const float *scales, int64_t rows, int64_t cols, void *y, int yt,
                    int64_t ld, void *stream) {
    int64_t yb, pad;
    int rc = check_matrix(rows, cols, ld, yt, &yb);
    if (rc != QCP_OK) return rc;
    if (rows == 0 || cols == 0) return QCP_OK;
    if (!int8_payload(rows, cols, &pad)) return QCP_EINVAL;
    if (!codes || !scales || !y) return QCP_EINVAL;
    if (!aligned16(codes) || !aligned16(scales) || (uintptr_t)y % dtype_bytes(yt)) return QCP_EALIGN;
    if (overlap(y, yb, codes, rows * pad) || overlap(y, yb, scales, rows * 4)) return QCP_EINVAL;
    return status_of(qcp::launch_int8_dequantize(codes, scales, rows, cols, y, yt, ld, (hipStream_t)stream));
}

int int8_matmul(const uint8_t *a_codes, const float *a_scales, const uint8_t *b_codes, const float *b_scales,
                int64_t M, int64_t N, int64_t K, void *c, int ct, int64_t ldc, void *work, int64_t work_bytes,
                void *stream) {
    int64_t cb, pad;
    int rc = check_matrix(M, N, ldc, ct, &cb);
    if (rc != QCP_OK) return rc;
    if (K < 0 || K > kInt8MaxK) return QCP_EINVAL;
    if (M == 0 || N == 0) return QCP_OK;
    if (!int8_payload(M, K, &pad) || !int8_payload(N, K, &pad)) return QCP_EINVAL;
    if ((M + 127) / 128 > qcp::kMaxGroups / ((N + 127) / 128)) return QCP_EINVAL;   // tiles of C
    if (!c || !a_scales || !b_scales || (K > 0 && (!a_codes || !b_codes))) return QCP_EINVAL;
    const int64_t need = work ? qcp_int8_matmul_work(M, N, K) : 0;
    if (work_bytes < need) return QCP_EINVAL;
    if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(b_codes) || !aligned16(b_scales) ||
        !aligned16(work) || (uintptr_t)c % dtype_bytes(ct))
        return QCP_EALIGN;
    const void *in[4] = {a_codes, a_scales, b_codes, b_scales};
    const int64_t bytes[4] = {M * pad, M * 4, N * pad, N * 4};
    if (overlap(c, cb, work, need)) return QCP_EINVAL;
    for (int i = 0; i < 4; i++)
        if (overlap(c, cb, in[i], bytes[i]) || overlap(work, need, in[i], bytes[i])) return QCP_EINVAL;
    return status_of(qcp::launch_int8_matmul(a_codes, a_scales, b_codes, b_scales, M, N, pad / 128, c, ct, ldc,
                                             need ? (int *)work : nullptr, (hipStream_t)stream));
}

int64_t qcp_int8_matmul_work(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0 || M > kMaxElems || N > kMaxElems || K > kInt8MaxK) return -1;
    const int slices = qcp::int8_matmul_slices(M, N, (K + 127) / 128);
    return slices > 1 ? 4 * slices * M * N : 0;
}

int int8_linear_rows(const void *x, int xt, int64_t M, int64_t K, int64_t ldx, const uint8_t *w_codes,
                     const float *w_scales, int64_t N, void *y, int64_t ldy, void *stream) {
    int64_t xb, yb, pad;
    if (xt != QCP_F16 && xt != QCP_BF16) return QCP_EINVAL;
    int rc = check_matrix(M, K, ldx, xt, &xb);
    if (rc != QCP_OK) return rc;
    rc = check_matrix(M, N, ldy, xt, &yb);
    if (rc != QCP_OK) return rc;
    if (K > kInt8MaxK) return QCP_EINVAL;
    if (M == 0 || N == 0) return QCP_OK;
    if (!int8_payload(N, K, &pad)) return QCP_EINVAL;
    if (!qcp_int8_linear_rows_fit(M, N, K)) return QCP_EUNSUPPORTED;
    if (!x || !y || !w_codes || !w_scales) return QCP_EINVAL;
    if (!aligned16(w_codes) || !aligned16(w_scales) || (uintptr_t)x % 2 || (uintptr_t)y % 2) return QCP_EALIGN;
    if (overlap(y, yb, x, xb) || overlap(y, yb, w_codes, N * pad) || overlap(y, yb, w_scales, N * 4)) return QCP_EINVAL;
    return status_of(qcp::launch_int8_linear_rows(x, xt, ldx, M, K, w_codes, w_scales, N, pad / 128, y, ldy,
                                                  (hipStream_t)stream));
}

int qcp_int8_linear_rows_fit(int64_t M, int64_t N, int64_t K) {
    if (M < 1 || N < 1 || K < 1 || N > kMaxElems || K > kInt8MaxK) return 0;
    return qcp::int8_linear_few(M, N, (K + 127) / 128) ? 1 : 0;
}

int int8_matmul_mixed(const void *a, int at, int64_t lda, int32_t transpose, const uint8_t *codes,
                      const float *scales, int64_t M, int64_t N, int64_t K, void *c, int ct, int64_t ldc,
                      void *work, int64_t work_bytes, void *stream) {
    int64_t ab, cb, pad;
    if (transpose != 0 && transpose != 1) return QCP_EINVAL;
    if (at != QCP_F16 && at != QCP_BF16) return QCP_EINVAL;
    if (valid_dtype(ct) && ct != QCP_F32 && ct != at) return QCP_EUNSUPPORTED;
    int rc = transpose ? check_matrix(K, M, lda, at, &ab) : check_matrix(M, K, lda, at, &ab);
    if (rc != QCP_OK) return rc;
    rc = check_matrix(M, N, ldc, ct, &cb);
    if (rc != QCP_OK) return rc;
    if (M == 0 || N == 0) return QCP_OK;
    if (N > kMixedMaxN || lda > kMixedMaxLd || !int8_payload(K, N, &pad)) return QCP_EINVAL;
    if (!mixed_tiles(M, N)) return QCP_EINVAL;
    if (!c || (K > 0 && (!a || !codes || !scales))) return QCP_EINVAL;
    const int64_t need = work ? qcp_int8_mixed_work(M, N, K, transpose, qcp::int8_mixed_aligned(a, lda) ? 1 : 0) : 0;
    if (work_bytes < need) return QCP_EINVAL;
    if (!aligned16(codes) || !aligned16(scales) || !aligned16(work) || (uintptr_t)a % 2 ||
        (uintptr_t)c % dtype_bytes(ct))
        return QCP_EALIGN;
    const void *in[3] = {a, codes, scales};
    const int64_t bytes[3] = {ab, K * pad, K * 4};
    if (overlap(c, cb, work, need)) return QCP_EINVAL;
    for (int i = 0; i < 3; i++)
        if (overlap(c, cb, in[i], bytes[i]) || overlap(work, need, in[i], bytes[i])) return QCP_EINVAL;
    return status_of(qcp::launch_int8_mixed(a, at, lda, transpose, codes, scales, M, N, K, c, ct, ldc,
                                            need ? work : nullptr, (hipStream_t)stream));
}

int64_t qcp_int8_mixed_work(int64_t M, int64_t N, int64_t K, int32_t transpose, int32_t aligned) {
    if (M < 0 || N < 0 || K < 0 || M > kMaxElems || N > kMixedMaxN || K > kMaxElems) return -1;
    if ((transpose != 0 && transpose != 1) || (aligned != 0 && aligned != 1)) return -1;
    if (!mixed_tiles(M, N)) return -1;
    return qcp::int8_mixed_work(M, N, K, transpose, aligned != 0);
}

}  // extern "C"
