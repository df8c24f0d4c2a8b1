// qcp_api.hip -- the extern "C" entry points declared in include/qcp.h.
//
// Each entry point validates its arguments on the host (pure checks: no HIP
// call is made for a rejected call or for n == 0), then enqueues one kernel on
// the caller's stream (adamw_step one per 64 tensors) and maps a launch error to
// QCP_EHIP.  No device memory is allocated and no state is kept between calls.
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <new>

#include "qcp.h"
#include "qcp_launch.h"

namespace {

// Largest element count (per tensor, or per slice of a reduce) any entry point
// accepts.  A dispatch holds at most 2^32 - 1 work-items, i.e. kMaxGroups
// work-groups of 256; every kernel gives a work-group at least 4096 elements
// (4 waves, each at least 64 lanes x 16 codes), so kMaxGroups * 4096 elements
// always fit in one launch.  That is 2^36 - 4096 elements: 137 GB of bf16 input.
constexpr int64_t kMaxElems = qcp::kMaxGroups * 4096;

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
bool valid_g(int32_t G) { return G >= 32 && G <= 1024 && (G & (G - 1)) == 0; }
bool valid_dtype(int t) { return t == QCP_F16 || t == QCP_BF16 || t == QCP_F32; }
bool valid_fmt(int f) {
    return f == QCP_INT2 || f == QCP_INT4 || f == QCP_INT6 || f == QCP_INT8 || f == QCP_E4M3;
}
int fmt_bits(int f) { return f == QCP_E4M3 ? 8 : f; }
int64_t dtype_bytes(int t) { return t == QCP_F32 ? 4 : 2; }
int64_t code_bytes(int64_t n, int fmt) { return (n * fmt_bits(fmt) + 7) / 8; }
int64_t n_blocks(int64_t n, int32_t G) { return (n + G - 1) / G; }

// do [a, a+na) and [b, b+nb) intersect?
bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return na > 0 && nb > 0 && a0 < b0 + (uintptr_t)nb && b0 < a0 + (uintptr_t)na;
}

int status_of(hipError_t e) { return e == hipSuccess ? QCP_OK : QCP_EHIP; }

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

int check_common(int64_t n, int32_t G) {
    if (n < 0 || n > kMaxElems) return QCP_EINVAL;
    if (!valid_g(G)) return QCP_EINVAL;
    return QCP_OK;
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

}  // namespace

extern "C" {

int quantize_blockwise(const void *x, int xt, int64_t n, int32_t G, int fmt, void *codes,
                       float *scales, void *stream) {
    int rc = check_common(n, G);
    if (rc != QCP_OK) return rc;
    if (!valid_dtype(xt) || !valid_fmt(fmt)) return QCP_EINVAL;
    if (n == 0) return QCP_OK;
    if (!x || !codes || !scales) return QCP_EINVAL;
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return QCP_EALIGN;
    int64_t xb = n * dtype_bytes(xt), cb = code_bytes(n, fmt), sb = 4 * n_blocks(n, G);
    if (overlap(x, xb, codes, cb) || overlap(x, xb, scales, sb) || overlap(codes, cb, scales, sb))
        return QCP_EINVAL;
    return status_of(qcp::launch_encode(x, xt, n, G, fmt, (uint8_t *)codes, scales,
                                        (hipStream_t)stream));
}

int reorder_quantize(const void *x, int xt, int64_t n, int32_t n_nodes, int32_t gpus_per_node,
                     int32_t G, int fmt, void *codes, int64_t slice_stride_bytes, float *scales,
                     int64_t scale_stride, void *stream) {
    int rc = check_common(n, G);
    if (rc != QCP_OK) return rc;
    if (!valid_dtype(xt) || !valid_fmt(fmt)) return QCP_EINVAL;
    if (n_nodes < 1 || n_nodes > 65536 || gpus_per_node < 1 || gpus_per_node > 64) return QCP_EINVAL;
    const int64_t W = (int64_t)n_nodes * gpus_per_node;
    if (n % W != 0 || (n / W) % 8 != 0) return QCP_EINVAL;
    if (n == 0) return QCP_OK;
    if (!x || !codes || !scales) return QCP_EINVAL;
    const int64_t L = n / gpus_per_node, cb = code_bytes(L, fmt), nb = n_blocks(L, G);
    if (slice_stride_bytes < cb || scale_stride < nb) return QCP_EINVAL;
    if (slice_stride_bytes % 16 != 0 || scale_stride % 4 != 0) return QCP_EALIGN;
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return QCP_EALIGN;
    const int64_t xb = n * dtype_bytes(xt);
    const int64_t ob = (int64_t)(gpus_per_node - 1) * slice_stride_bytes + cb;
    const int64_t sb = 4 * ((int64_t)(gpus_per_node - 1) * scale_stride + nb);
    if (overlap(x, xb, codes, ob) || overlap(x, xb, scales, sb) || overlap(codes, ob, scales, sb))
        return QCP_EINVAL;
    return status_of(qcp::launch_encode_reorder(x, xt, n, n_nodes, gpus_per_node, G, fmt,
                                                (uint8_t *)codes, slice_stride_bytes, scales,
                                                scale_stride, (hipStream_t)stream));
}

int dequantize_blockwise(const void *codes, const float *scales, int fmt, int64_t n, int32_t G,
                         void *y, int yt, void *stream) {
    int rc = check_common(n, G);
    if (rc != QCP_OK) return rc;
    if (!valid_dtype(yt) || !valid_fmt(fmt)) return QCP_EINVAL;
    if (n == 0) return QCP_OK;
    if (!codes || !scales || !y) return QCP_EINVAL;
    if (!aligned16(codes) || !aligned16(scales) || !aligned16(y)) return QCP_EALIGN;
    int64_t yb = n * dtype_bytes(yt), cb = code_bytes(n, fmt), sb = 4 * n_blocks(n, G);
    if (overlap(y, yb, codes, cb) || overlap(y, yb, scales, sb)) return QCP_EINVAL;
    return status_of(qcp::launch_decode((const uint8_t *)codes, scales, fmt, n, G, y, yt,
                                        (hipStream_t)stream));
}

int pack_subbyte(const void *x, int xt, int64_t n, int32_t b, int32_t G, uint8_t *packed,
                 float *scales, void *stream) {
    if (b != 2 && b != 4 && b != 6 && b != 8) return QCP_EINVAL;
    return quantize_blockwise(x, xt, n, G, b, packed, scales, stream);
}

int unpack_subbyte(const uint8_t *packed, const float *scales, int64_t n, int32_t b, int32_t G,
                   void *y, int yt, void *stream) {
    if (b != 2 && b != 4 && b != 6 && b != 8) return QCP_EINVAL;
    return dequantize_blockwise(packed, scales, b, n, G, y, yt, stream);
}

int pack_subbyte_records(const void *x, int xt, int64_t n, int32_t b, int32_t G,
                         uint8_t *records, void *stream) {
    int rc = check_common(n, G);
    if (rc != QCP_OK) return rc;
    if (!valid_dtype(xt) || (b != 2 && b != 4 && b != 6 && b != 8)) return QCP_EINVAL;
    if (n == 0) return QCP_OK;
    if (!x || !records) return QCP_EINVAL;
    if (!aligned16(x) || !aligned16(records)) return QCP_EALIGN;
    if (overlap(x, n * dtype_bytes(xt), records, qcp_payload_bytes(n, b, G))) return QCP_EINVAL;
    return status_of(qcp::launch_encode_records(x, xt, n, G, b, records, (hipStream_t)stream));
}

int unpack_subbyte_records(const uint8_t *records, int64_t n, int32_t b, int32_t G, void *y,
                           int yt, void *stream) {
    int rc = check_common(n, G);
    if (rc != QCP_OK) return rc;
    if (!valid_dtype(yt) || (b != 2 && b != 4 && b != 6 && b != 8)) return QCP_EINVAL;
    if (n == 0) return QCP_OK;
    if (!records || !y) return QCP_EINVAL;
    if (!aligned16(records) || !aligned16(y)) return QCP_EALIGN;
    if (overlap(y, n * dtype_bytes(yt), records, qcp_payload_bytes(n, b, G))) return QCP_EINVAL;
    return status_of(qcp::launch_decode_records(records, n, G, b, y, yt, (hipStream_t)stream));
}

int dequant_reduce_requant(const void *codes_in, int64_t in_slice_stride_bytes,
                           const float *scales_in, int64_t in_scale_stride, int32_t n_slices,
                           int64_t slice_len, int32_t G, int fmt_in, int fmt_out,
                           void *codes_out, float *scales_out, float *sum_out, void *stream) {
    int rc = check_common(slice_len, G);
    if (rc != QCP_OK) return rc;
    if (!valid_fmt(fmt_in) || !valid_fmt(fmt_out)) return QCP_EINVAL;
    if (n_slices < 1 || n_slices > 64) return QCP_EINVAL;
    if (slice_len == 0) return QCP_OK;
    if (!codes_in || !scales_in || !codes_out || !scales_out) return QCP_EINVAL;
    int64_t in_cb = code_bytes(slice_len, fmt_in), nb = n_blocks(slice_len, G);
    if (in_slice_stride_bytes < in_cb || in_scale_stride < nb) return QCP_EINVAL;
    if (in_slice_stride_bytes % 16 != 0 || in_scale_stride % 4 != 0) return QCP_EALIGN;
    if (!aligned16(codes_in) || !aligned16(scales_in) || !aligned16(codes_out) ||
        !aligned16(scales_out) || (sum_out && !aligned16(sum_out)))
        return QCP_EALIGN;
    int64_t in_b = (int64_t)(n_slices - 1) * in_slice_stride_bytes + in_cb;
    int64_t in_sb = 4 * ((int64_t)(n_slices - 1) * in_scale_stride + nb);
    int64_t out_cb = code_bytes(slice_len, fmt_out), out_sb = 4 * nb, sum_b = 4 * slice_len;
    const void *outs[3] = {codes_out, scales_out, sum_out};
    int64_t out_len[3] = {out_cb, out_sb, sum_out ? sum_b : 0};
    for (int i = 0; i < 3; i++) {
        if (overlap(outs[i], out_len[i], codes_in, in_b) ||
            overlap(outs[i], out_len[i], scales_in, in_sb))
            return QCP_EINVAL;
        for (int j = i + 1; j < 3; j++)
            if (overlap(outs[i], out_len[i], outs[j], out_len[j])) return QCP_EINVAL;
    }
    return status_of(qcp::launch_reduce((const uint8_t *)codes_in, in_slice_stride_bytes,
                                        scales_in, in_scale_stride, n_slices, slice_len, G,
                                        fmt_in, fmt_out, (uint8_t *)codes_out, scales_out,
                                        sum_out, (hipStream_t)stream));
}

int fp8_accum_requant(uint8_t *state_codes, float *state_scales, const void *grad, int gt,
                      int64_t n, int32_t G, void *stream) {
    int rc = check_common(n, G);
    if (rc != QCP_OK) return rc;
    if (!valid_dtype(gt)) return QCP_EINVAL;
    if (n == 0) return QCP_OK;
    if (!state_codes || !state_scales || !grad) return QCP_EINVAL;
    if (!aligned16(state_codes) || !aligned16(state_scales) || !aligned16(grad)) return QCP_EALIGN;
    int64_t cb = n, sb = 4 * n_blocks(n, G), gb = n * dtype_bytes(gt);
    if (overlap(state_codes, cb, state_scales, sb) || overlap(grad, gb, state_codes, cb) ||
        overlap(grad, gb, state_scales, sb))
        return QCP_EINVAL;
    return status_of(qcp::launch_accum(state_codes, state_scales, grad, gt, n, G,
                                       (hipStream_t)stream));
}

int adamw_step(float *const *params, const void *const *grads, void *const *copies,
               const int64_t *sizes, const int64_t *offsets, int32_t n_tensors, int gt, int ct,
               int state, void *m, float *m_scales, void *v, float *v_scales, int64_t n_state,
               int32_t G, int64_t step, double lr, double beta1, double beta2, double eps,
               double weight_decay, const float *grad_scale, uint64_t seed, void *stream) {
    if (n_tensors < 0 || n_tensors > QCP_ADAMW_MAX_TENSORS || n_state < 0 || !valid_g(G)) return QCP_EINVAL;
    if (!valid_dtype(gt) || (state != QCP_F32 && state != QCP_E4M3)) return QCP_EINVAL;
    if (copies && ct != QCP_F16 && ct != QCP_BF16) return QCP_EINVAL;
    const bool scalars = step >= 1 && isfinite(lr) && lr >= 0 && beta1 >= 0 && beta1 < 1 && beta2 >= 0 &&
                         beta2 < 1 && isfinite(eps) && (float)eps > 0 && isfinite(weight_decay) &&
                         weight_decay >= 0;
    if (!scalars) return QCP_EINVAL;
    if (n_tensors == 0) return QCP_OK;
    if (!params || !grads || !sizes || !offsets) return QCP_EINVAL;
    const bool eight = state == QCP_E4M3;
    int64_t past = 0;                                       // end of the last tensor's blocks
    int32_t live = 0;
    for (int32_t i = 0; i < n_tensors; i++) {
        const int64_t n = sizes[i];
        if (n < 0 || n > kMaxElems) return QCP_EINVAL;
        if (offsets[i] < past || offsets[i] % G != 0) return QCP_EINVAL;
        if (offsets[i] > n_state || n_blocks(n, G) > (n_state - offsets[i]) / G) return QCP_EINVAL;
        past = offsets[i] + n_blocks(n, G) * G;
        if (n == 0) continue;
        live++;
        if (!params[i] || !grads[i] || (copies && !copies[i])) return QCP_EINVAL;
        if ((uintptr_t)params[i] % 4 || (uintptr_t)grads[i] % dtype_bytes(gt)) return QCP_EALIGN;
        if (copies && (uintptr_t)copies[i] % 2) return QCP_EALIGN;
    }
    if (live == 0) return QCP_OK;
    if (!m || !v || (eight && (!m_scales || !v_scales))) return QCP_EINVAL;
    if (!aligned16(m) || !aligned16(v)) return QCP_EALIGN;
    if (eight && (!aligned16(m_scales) || !aligned16(v_scales))) return QCP_EALIGN;
    if ((uintptr_t)grad_scale % 4) return QCP_EALIGN;

    qcp::AdamwTensor *t = new (std::nothrow) qcp::AdamwTensor[live];
    Range *r = new (std::nothrow) Range[3 * (int64_t)live + 5];
    int rc = t && r ? QCP_OK : QCP_ENOMEM;
    if (rc == QCP_OK) {
        int64_t k = 0, at = 0;
        auto range = [&](const void *p, int64_t bytes, bool written) {
            if (p && bytes > 0) r[k++] = Range{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, written};
        };
        for (int32_t i = 0; i < n_tensors; i++) {
            const int64_t n = sizes[i];
            if (n == 0) continue;
            void *copy = copies ? copies[i] : nullptr;
            t[at++] = qcp::AdamwTensor{params[i], grads[i], copy, n, offsets[i]};
            range(params[i], 4 * n, true);
            range(grads[i], n * dtype_bytes(gt), false);
            range(copy, 2 * n, true);
        }
        range(m, eight ? past : 4 * past, true);
        range(v, eight ? past : 4 * past, true);
        if (eight) {
            range(m_scales, past / G * 4, true);
            range(v_scales, past / G * 4, true);
        }
        range(grad_scale, 4, false);
        if (ranges_clash(r, k)) rc = QCP_EINVAL;
    }
    if (rc == QCP_OK) {
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
        rc = status_of(qcp::launch_adamw(t, live, gt, state, G, c, (hipStream_t)stream));
    }
    delete[] t;
    delete[] r;
    return rc;
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

int mxfp4_matmul(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *b_codes,
                 const uint8_t *b_scales, int64_t M, int64_t N, int64_t K, void *c, int ct, int64_t ldc,
                 void *stream) {
    int64_t cb, pad;
    int rc = check_matrix(M, N, ldc, ct, &cb);
    if (rc != QCP_OK) return rc;
    if (K < 0) return QCP_EINVAL;
    if (M == 0 || N == 0) return QCP_OK;
    if (!mx_payload(M, K, &pad) || !mx_payload(N, K, &pad)) return QCP_EINVAL;
    if ((M + 127) / 128 > qcp::kMaxGroups / ((N + 127) / 128)) return QCP_EINVAL;   // tiles of C
    if (!c || (K > 0 && (!a_codes || !a_scales || !b_codes || !b_scales))) return QCP_EINVAL;
    if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(b_codes) || !aligned16(b_scales) ||
        (uintptr_t)c % dtype_bytes(ct))
        return QCP_EALIGN;
    if (overlap(c, cb, a_codes, M * pad / 2) || overlap(c, cb, a_scales, M * pad / 32) ||
        overlap(c, cb, b_codes, N * pad / 2) || overlap(c, cb, b_scales, N * pad / 32))
        return QCP_EINVAL;
    return status_of(qcp::launch_mx_matmul(a_codes, a_scales, b_codes, b_scales, M, N, pad / 128, c, ct,
                                           ldc, (hipStream_t)stream));
}

int64_t qcp_mxfp4_padded(int64_t n) { return n < 0 || n > kMaxElems ? -1 : (n + 127) / 128 * 128; }

int64_t qcp_payload_bytes(int64_t n, int32_t bits, int32_t G) {
    if (n < 0 || G < 1 || bits < 1 || bits > 32) return -1;
    return (n * bits + 7) / 8 + 4 * ((n + G - 1) / G);
}

double qcp_aquavit_target(int64_t t, int64_t T, double a, double c) {
    if (T <= 0 || t < 0 || t > T) return -1.0;
    return 8.0 - 6.0 / (a + c * (double)t / (double)T);   // (c*t)/T, left to right
}

int qcp_aquavit_level(int64_t t, int64_t T, double a, double c, int32_t *b, int32_t *G) {
    if (T <= 0 || t < 0 || t > T || !b || !G) return QCP_EINVAL;
    const double want = qcp_aquavit_target(t, T, a, c);
    // levels b + 32/G in increasing bpw: within each b, G from 1024 down to 32
    double best = 0.0;
    bool have = false;
    for (int32_t bb = 2; bb <= 8; bb += 2) {
        for (int32_t gg = 1024; gg >= 32; gg /= 2) {
            const double level = bb + 32.0 / gg;
            const double d = level > want ? level - want : want - level;
            // strictly closer wins; on a tie the earlier (smaller) level stays
            if (!have || d < best) {
                best = d;
                *b = bb;
                *G = gg;
                have = true;
            }
        }
    }
    return QCP_OK;
}

const char *qcp_strerror(int status) {
    switch (status) {
    case QCP_OK: return "success";
    case QCP_EINVAL: return "invalid argument (size, block size, bit width, format, dtype, stride, null or overlapping buffer)";
    case QCP_EALIGN: return "pointer or stride not aligned to 16 bytes";
    case QCP_EUNSUPPORTED: return "unsupported combination";
    case QCP_ENOMEM: return "out of host memory";
    case QCP_EHIP: return "HIP runtime error at kernel launch";
    default: return "unknown status";
    }
}

const char *qcp_version(void) { return "0.2.0"; }

int64_t qcp_max_elements(void) { return kMaxElems; }

}  // extern "C"
