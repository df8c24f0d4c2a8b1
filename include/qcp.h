/*
 * qcp.h -- quantized collective payloads: the C-ABI of libqcp.so.
 *
 * The data-parallel hot path of quantized ZeRO-3 communication, on one
 * gfx950 (MI355X) GPU: the kernels that sit on either side of the collectives
 * (quantize before an all-gather or all-to-all, dequantize or reduce after it).
 *
 * Sources (web pages, cited by title and section):
 *  [ZPP]  "Quantized LLM Training at Scale with ZeRO++" (talk summary):
 *         "Blockwise weight quantization cuts forward-gather traffic in half" (qwZ),
 *         "QGZ keeps reductions in full precision while sending quantized gradients",
 *         "The implementation combines kernel fusion with communication overlap" (qgZ).
 *  [AQV]  "Aquavit: Ascending Quantization for Communication-Efficient Vast-Scale
 *         Distributed Training" (review): granularity modulation, bpw = b + 32/G
 *         (Eq. 6, Table 1), b in {2,4,6,8}, sub-byte packing kernels (Section 5.2).
 *  [AGOQ] "AGoQ: Activation and Gradient Quantization for Memory-Efficient
 *         Distributed Training of LLMs", Section 2.B (QuanGrad): local accumulation
 *         of FP8 gradients, and the local-reduce step of the precision-preserved
 *         all-reduce.
 *
 * Conventions shared by every entry point
 *  - Pointers are device pointers (HBM), except where a comment says otherwise.
 *    The caller allocates and frees every buffer; the library allocates nothing,
 *    keeps no pointer after returning and holds no mutable global state.
 *  - `stream` is a hipStream_t (NULL = the legacy default stream).  Every call
 *    enqueues its kernel(s) on `stream` and returns without synchronizing; the
 *    status reports argument validation and launch errors only.
 *  - Element types (qcp_dtype): fp16, bf16, fp32.  A payload format (qcp_fmt) is
 *    INT2/INT4/INT6/INT8 (symmetric two's-complement codes in [-qmax, qmax],
 *    qmax = 2^(b-1)-1) or E4M3 (OCP E4M3FN, largest finite value 448).
 *  - Blocks: element i of a tensor (or of one slice) belongs to block i / G; the
 *    last block may be short.  Each block has one fp32 scale s = absmax / qmax
 *    (IEEE division; a block of zeros has s = +0 and all codes 0).
 *  - Codes: q = IEEE fp32 quotient x / s; INT code = round-half-even(q) clamped
 *    to [-qmax, qmax]; E4M3 code = nearest E4M3FN value to q, ties to even
 *    mantissa (sign of zero kept, NaN never produced).
 *  - Code layout: an LSB-first bitstream; element i occupies bits [b*i, b*i+b)
 *    and bit 8j+t of the stream is bit t of byte j.  So INT8 and E4M3 are one
 *    byte per code, INT4 puts the even element in the low nibble, INT6 packs 4
 *    codes in 3 bytes.  The stream is ceil(n*b/8) bytes, zero-padded at the end.
 *    Scales are a separate fp32 array of ceil(n/G) entries.
 *  - Preconditions: 0 <= n <= qcp_max_elements() (n == 0 is a no-op returning
 *    QCP_OK; for a reduce, n is the slice length); G a power of two in
 *    [32, 1024]; every pointer non-null and 16-byte aligned when there is work;
 *    inputs finite (non-finite inputs give unspecified codes, never a fault);
 *    outputs do not overlap inputs (except the in-place state of
 *    fp8_accum_requant) and do not overlap each other.
 *  - Results are a pure function of the inputs: no atomics, a fixed order of
 *    summation, byte-identical on every run.
 */
#ifndef QCP_H
#define QCP_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    QCP_OK = 0,
    QCP_EINVAL = -1,        /* bad size, G, b, format, dtype, stride, null or overlapping pointer */
    QCP_EALIGN = -2,        /* a pointer or stride is not a multiple of 16 bytes */
    QCP_EUNSUPPORTED = -3,  /* a combination this library does not implement */
    QCP_EHIP = -4           /* the HIP runtime reported an error at launch */
} qcp_status;

typedef enum { QCP_F16 = 1, QCP_BF16 = 2, QCP_F32 = 3 } qcp_dtype;

typedef enum { QCP_INT2 = 2, QCP_INT4 = 4, QCP_INT6 = 6, QCP_INT8 = 8, QCP_E4M3 = 0x43 } qcp_fmt;

/*
 * Blockwise quantize [ZPP qwZ: per-block 8-bit weight quantization of the
 * forward all-gather payload; AGOQ: per-block E4M3].
 *   x       n elements of type xt
 *   codes   out: ceil(n*b/8) bytes in format fmt (b = 8 for INT8/E4M3)
 *   scales  out: ceil(n/G) fp32
 * Any qcp_fmt is accepted; INT8 is the qwZ payload, E4M3 the FP8 one.
 */
int quantize_blockwise(const void *x, int xt, int64_t n, int32_t G, int fmt,
                       void *codes, float *scales, void *stream);

/*
 * Blockwise dequantize [ZPP qwZ: the gathered 8-bit payload becomes 16-bit
 * values again before compute]:  y_i = cast(fl(value(code_i) * s_{i/G})) with
 * one round-to-nearest-even cast to yt (fp32 output is the product itself).
 *   codes   ceil(n*b/8) bytes;  scales ceil(n/G) fp32;  y out: n elements of yt
 */
int dequantize_blockwise(const void *codes, const float *scales, int fmt, int64_t n,
                         int32_t G, void *y, int yt, void *stream);

/*
 * Sub-byte pack [AQV granularity modulation, Section 5.1-5.2]: fused blockwise
 * quantize + pack to b bits, b in {2,4,6,8}; identical to
 * quantize_blockwise(fmt = b).  Payload = ceil(n*b/8) + 4*ceil(n/G) bytes, so
 * bpw = b + 32/G when G divides n.
 */
int pack_subbyte(const void *x, int xt, int64_t n, int32_t b, int32_t G,
                 uint8_t *packed, float *scales, void *stream);

/* Sub-byte unpack + dequantize [AQV]: identical to dequantize_blockwise(fmt = b). */
int unpack_subbyte(const uint8_t *packed, const float *scales, int64_t n, int32_t b,
                   int32_t G, void *y, int yt, void *stream);

/*
 * Fused dequantize -> fp32 sum over N slices -> requantize.
 * [ZPP qgZ: the slices one rank receives from its N peers after the all-to-all
 * are dequantized, reduced in full precision and requantized for the next hop,
 * in one kernel.  AGOQ precision-preserved all-reduce, step 2 "Local Reduce":
 * dequantize received FP8 to FP32, sum, requantize to FP8.]
 *   codes_in   slice j (j = 0..n_slices-1) starts at codes_in + j*in_slice_stride_bytes
 *              and holds slice_len codes in fmt_in (ceil(slice_len*b_in/8) bytes)
 *   scales_in  slice j's ceil(slice_len/G) scales start at scales_in + j*in_scale_stride
 *   For each element i:  acc = -0.0;  acc = fmaf(value(c_ji), s_j[i/G], acc) for
 *   j = 0..n_slices-1 in order;  sum_i = acc.
 *   The sums are quantized blockwise with the same G in fmt_out:
 *   codes_out  ceil(slice_len*b_out/8) bytes;  scales_out ceil(slice_len/G) fp32
 *   sum_out    nullable; if given, slice_len fp32 sums
 *   1 <= n_slices <= 64; in_slice_stride_bytes is a multiple of 16 and at least
 *   one slice's code bytes; in_scale_stride (in floats) is a multiple of 4 and
 *   at least ceil(slice_len/G).
 */
int dequant_reduce_requant(const void *codes_in, int64_t in_slice_stride_bytes,
                           const float *scales_in, int64_t in_scale_stride,
                           int32_t n_slices, int64_t slice_len, int32_t G,
                           int fmt_in, int fmt_out, void *codes_out, float *scales_out,
                           float *sum_out, void *stream);

/*
 * Sub-byte pack / unpack with interleaved metadata [AQV Section 5.2, metadata
 * interleaving]: the payload of n elements at b bits with block size G as one
 * record per block, records back to back:
 *   record k = [fp32 scale s_k (4 bytes)][codes of block k, LSB-first b-bit
 *              fields: G*b/8 bytes, ceil(len*b/8) for the short last block]
 * so record k starts at byte k*(4 + G*b/8) and the whole stream has exactly
 * qcp_payload_bytes(n, b, G) bytes.  Codes and scales are those of
 * pack_subbyte / unpack_subbyte; only the layout differs.
 *   records   output of pack / input of unpack, 16-byte aligned.
 * Errors: as pack_subbyte / unpack_subbyte.
 */
int pack_subbyte_records(const void *x, int xt, int64_t n, int32_t b, int32_t G,
                         uint8_t *records, void *stream);
int unpack_subbyte_records(const uint8_t *records, int64_t n, int32_t b, int32_t G, void *y,
                           int yt, void *stream);

/*
 * Aquavit ascending precision schedule [AQV key idea, Section 5.1, Table 1]:
 * the target bits per weight at step t of T is 8 - 6/(a + c*t/T) ((a, c) =
 * (0.9, 5) on the pages); qcp_aquavit_level writes the granularity-modulation
 * level (b in {2,4,6,8}, G in {32, ..., 1024}) whose b + 32/G is nearest the
 * target (ties: the smaller b + 32/G).  From t = 0 to t = T this runs from
 * 2-bit/G=1024 (2.03 bpw) to 6-bit/G=32 (7.00 bpw).  Host only.
 * qcp_aquavit_target returns -1 and qcp_aquavit_level QCP_EINVAL unless
 * 0 <= t <= T and T > 0 (and b, G non-null).
 */
double qcp_aquavit_target(int64_t t, int64_t T, double a, double c);
int qcp_aquavit_level(int64_t t, int64_t T, double a, double c, int32_t *b, int32_t *G);

/*
 * qgZ sender: tensor-slice reordering fused with the quantization of the
 * intra-node all-to-all's send slices [ZPP "Tensor-slice reordering fixes
 * incorrect gradient placement"; "The implementation combines kernel fusion
 * with communication overlap": reordering fused with intra-node quantization].
 *   x               one rank's gradient bucket, n elements of type xt; it is
 *                   W = n_nodes*gpus_per_node chunks of C = n/W elements, chunk
 *                   c being the part global rank c (node c/N, GPU c%N) owns
 *                   after the reduce-scatter (N = gpus_per_node, K = n_nodes)
 *   codes, scales   N slices: slice j holds chunks b*N + j for b = 0..K-1 in
 *                   node order (L = n/N elements), quantized blockwise in fmt
 *                   with blocks restarting at each slice.  Its codes start at
 *                   codes + j*slice_stride_bytes (ceil(L*b/8) bytes), its
 *                   ceil(L/G) scales at scales + j*scale_stride.
 * With this order, after the intra-node reduce (dequant_reduce_requant on the
 * N received slices) and the inter-node exchange, every rank holds its own
 * chunk.  Equivalent to reordering x and calling quantize_blockwise on each
 * slice.  Preconditions beyond the shared ones: 1 <= n_nodes <= 65536,
 * 1 <= gpus_per_node <= 64, n divisible by W with C a multiple of 8;
 * slice_stride_bytes a multiple of 16 and >= ceil(L*b/8); scale_stride a
 * multiple of 4 and >= ceil(L/G).  Errors: QCP_EINVAL, QCP_EALIGN, QCP_EHIP.
 */
int reorder_quantize(const void *x, int xt, int64_t n, int32_t n_nodes, int32_t gpus_per_node,
                     int32_t G, int fmt, void *codes, int64_t slice_stride_bytes, float *scales,
                     int64_t scale_stride, void *stream);

/*
 * FP8 main-gradient accumulation, in place [AGOQ QuanGrad "Local Accumulation":
 * dequantize the FP8 main gradient to 16 bits, add the micro-batch gradient,
 * requantize the sum to FP8]:
 *   d_i = bf16(fl(value(e_i) * s_{i/G}));  t_i = bf16(fl(d_i + g_i));
 *   (state_codes, state_scales) <- E4M3 blockwise quantization of t.
 *   state_codes  n E4M3 bytes (read and overwritten)
 *   state_scales ceil(n/G) fp32 (read and overwritten)
 *   grad         n elements of type gt
 * The all-zero state (codes 0x00, scales +0) is the empty accumulator.
 */
int fp8_accum_requant(uint8_t *state_codes, float *state_scales, const void *grad, int gt,
                      int64_t n, int32_t G, void *stream);

/*
 * AdamW over the tensors of an optimizer shard, in place: the step between the
 * gradient reduce-scatter (whose last reduce leaves fp32 sums, sum_out above)
 * and the weight all-gather.  For every element, in fp32, with
 * g = grad * grad_scale, t = step:
 *   m <- beta1*m + (1-beta1)*g         v <- beta2*v + (1-beta2)*g^2
 *   p <- p*(1 - lr*weight_decay) - lr/(1-beta1^t) * m / (sqrt(v)/sqrt(1-beta2^t) + eps)
 *   params    host array of n_tensors pointers to fp32 elements (4-byte aligned)
 *   grads     host array of pointers to elements of type gt, aligned to them
 *   copies    null, or a host array of pointers that receive p rounded to the
 *             16-bit type ct (QCP_F16 or QCP_BF16), 2-byte aligned
 *   sizes, offsets   host arrays: elements of each tensor, and the place of its
 *             first element in the moments: a multiple of G, ascending, each
 *             tensor's ceil(size/G)*G places apart from the next one's
 *   state     QCP_F32: m and v hold n_state fp32 values; the scales are ignored.
 *             QCP_E4M3: m and v hold n_state codes of m and of sqrt(v) with
 *             one fp32 scale per G (value = code * scale).  The scale is 2^k, the
 *             smallest k >= -126 at which the block's absmax is at most
 *             448 * 2^k; a block of zeros has scale +0.  A value is rounded to one
 *             of its two neighbours at random: up in magnitude when its fraction of
 *             their distance plus u/2^16 reaches 1, where u is 16 bits of a hash of
 *             (place, step, seed): the low half for m, the high half for sqrt(v).
 *             A positive sqrt(v) never becomes 0.  All zeros is the state before
 *             the first step.  Places that pad a tensor's last block stay 0.  A block
 *             in which m or v is infinite or NaN (from such a gradient, or from one
 *             whose square overflows) has a NaN scale, from then on.
 *   step >= 1; lr, weight_decay >= 0; 0 <= beta1, beta2 < 1; eps >= 2^-126
 *   grad_scale   null (1), or a device pointer to one fp32 factor: the clipping
 *             or unscaling factor, read when the kernel runs
 *   seed      of the hash; unused with QCP_F32
 * The host arrays are read before the call returns.  m, v and the scales are
 * 16-byte aligned.  At most QCP_ADAMW_MAX_TENSORS tensors a call; tensors without
 * elements are skipped.  No two buffers overlap, except that gradients may.
 * One kernel launch per 64 tensors.  Errors: QCP_EINVAL, QCP_EALIGN, QCP_EHIP.
 */
#define QCP_ADAMW_MAX_TENSORS 1024
int adamw_step(float *const *params, const void *const *grads, void *const *copies,
               const int64_t *sizes, const int64_t *offsets, int32_t n_tensors, int gt, int ct,
               int state, void *m, float *m_scales, void *v, float *v_scales, int64_t n_state,
               int32_t G, int64_t step, double lr, double beta1, double beta2, double eps,
               double weight_decay, const float *grad_scale, uint64_t seed, void *stream);

/*
 * What adamw_step would refuse, for any number of tensors: a step over more than
 * QCP_ADAMW_MAX_TENSORS is several calls, each of which sees its own tensors only, so
 * its caller asks here first and makes none of them where one would be refused.
 * Host only.  Errors: QCP_EINVAL, QCP_EALIGN; QCP_EUNSUPPORTED where the host has no
 * memory to compare the buffers.
 */
int qcp_adamw_check(float *const *params, const void *const *grads, void *const *copies,
                    const int64_t *sizes, const int64_t *offsets, int64_t n_tensors, int gt, int ct,
                    int state, void *m, float *m_scales, void *v, float *v_scales, int64_t n_state,
                    int32_t G, int64_t step, double lr, double beta1, double beta2, double eps,
                    double weight_decay, const float *grad_scale);

/*
 * The MXFP4 payload of a matrix (OCP Microscaling: E2M1 codes, one E8M0 scale per
 * 32): 4.25 bits per weight, which the matrix cores multiply as it is
 * (mxfp4_matmul).  A payload of `lines` rows of n values holds each row padded
 * with zeros to P = qcp_mxfp4_padded(n) values (whole 128s):
 *   codes    lines x P/2 bytes; value 2i of a row in the low four bits of its
 *            byte i, value 2i+1 in the high ones; sign, 2 exponent bits, 1 mantissa
 *            bit: +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}
 *   scales   lines x P/32 bytes: e stands for 2^(e-127), 255 for NaN
 * Quantize: E = exponent field of a block's fp32 absmax, e = max(E - 2, 0); a code
 * is the value nearest to x * 2^(127-e), ties to the even code, 6 beyond, the sign
 * of zero kept.  A block with an infinity or a NaN has e = 255 and unspecified
 * codes.
 *   x          rows x cols elements of type xt (aligned to them), rows ld
 *              elements apart, ld >= cols
 *   transpose  0: the payload of x (lines = rows, blocks along its rows);
 *              1: the payload of x^T (lines = cols, blocks along its columns)
 * Both: the payloads of x (codes, scales) and of x^T (codes_t, scales_t), reading
 * x once: what the forward and the backward product of a layer take.
 * Dequantize: y (rows x cols of type yt, rows ld apart) is code * 2^(e-127) rounded
 * once to yt.
 *   codes, scales   16-byte aligned; lines * P <= qcp_max_elements(), n <= 2^31
 * Errors: QCP_EINVAL, QCP_EALIGN, QCP_EHIP.
 */
int mxfp4_quantize(const void *x, int xt, int64_t rows, int64_t cols, int64_t ld, int32_t transpose,
                   uint8_t *codes, uint8_t *scales, void *stream);
int mxfp4_quantize_both(const void *x, int xt, int64_t rows, int64_t cols, int64_t ld, uint8_t *codes,
                        uint8_t *scales, uint8_t *codes_t, uint8_t *scales_t, void *stream);
int mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, void *y,
                     int yt, int64_t ld, void *stream);

/*
 * Product of two MXFP4 payloads: c[m, n] = sum over k of a[m, k] * b[n, k],
 * accumulated in fp32 and rounded once to type ct (rows ldc elements apart).
 *   a_codes, a_scales   the payload of A, M rows of K values
 *   b_codes, b_scales   the payload of B, N rows of K values (a weight stored as
 *                       [out, in], as the forward pass has it)
 * K = 0 gives zeros.  A scale of 255 makes its row (or column) of c NaN.  Forward,
 * y = x W^T: A = x, B = W.  Backward: dx = dy W takes the payloads of dy and of
 * W^T, dW = dy^T x those of dy^T and x^T (transpose = 1).
 */
int mxfp4_matmul(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *b_codes,
                 const uint8_t *b_scales, int64_t M, int64_t N, int64_t K, void *c, int ct, int64_t ldc,
                 void *stream);

/*
 * The same with scratch memory of at least qcp_mxfp4_matmul_work(M, N, K) bytes,
 * 16-byte aligned, on the device.  Where that is not 0 (few tiles of C and a long K)
 * slices of K are multiplied side by side into fp32 sums there and added up, always in
 * the same order, in a second launch; else `work` is not used and may be null.  The
 * order of the sums, and with it their last bits, differs from mxfp4_matmul's.
 */
int mxfp4_matmul_sliced(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *b_codes,
                        const uint8_t *b_scales, int64_t M, int64_t N, int64_t K, void *c, int ct,
                        int64_t ldc, void *work, int64_t work_bytes, void *stream);

/* Bytes of scratch memory for mxfp4_matmul_sliced, at most 4 MB; -1 for a negative or
 * too large size.  Host only. */
int64_t qcp_mxfp4_matmul_work(int64_t M, int64_t N, int64_t K);

/* n rounded up to whole 128s, the row length of an MXFP4 payload; -1 if n is
 * negative or above qcp_max_elements().  Host only. */
int64_t qcp_mxfp4_padded(int64_t n);

/*
 * The INT8 payload of a matrix with one scale per row: a token of an activation, an
 * output channel of a weight.  The rows of n codes are padded with zeros to
 * P = qcp_mxfp4_padded(n) (whole 128s):
 *   codes    rows x P bytes, two's complement
 *   scales   one fp32 per row
 * Quantize: as quantize_blockwise with the row as its block: s = absmax / 127 (IEEE; a
 * row of zeros, or one whose quotient underflows, has s = +0 and codes 0), a code is
 * the fp32 quotient x / s rounded half to even within [-127, 127].  A row with an
 * infinity or a NaN has a NaN scale and codes 0.
 *   x          rows x cols elements of type xt (aligned to them), rows ld elements
 *              apart, ld >= cols; rows without elements get the scale 0
 * Dequantize: y (rows x cols of type yt, rows ld apart) is the fp32 product code * s,
 * rounded once to yt.
 *   codes, scales   16-byte aligned; rows * P <= qcp_max_elements(), n <= 2^31
 * Errors: QCP_EINVAL, QCP_EALIGN, QCP_EHIP.
 */
int int8_quantize(const void *x, int xt, int64_t rows, int64_t cols, int64_t ld, uint8_t *codes,
                  float *scales, void *stream);
int int8_dequantize(const uint8_t *codes, const float *scales, int64_t rows, int64_t cols, void *y, int yt,
                    int64_t ld, void *stream);

/*
 * Product of two such payloads: c[m, n] = sa[m] * sb[n] * sum over k of qa[m, k] * qb[n, k],
 * rounded to type ct (rows ldc elements apart).  The sum is exact (any codes of 8 bits,
 * -128 too); the sum, the scales and their products are rounded to fp32.
 *   a_codes, a_scales   the payload of A, M rows of K codes (tokens)
 *   b_codes, b_scales   the payload of B, N rows of K codes (a weight, [out, in])
 *   K <= 130944, within which no sum leaves 32 bits; K = 0 gives zeros (times the scales)
 *   work     null, or scratch memory on the device of at least qcp_int8_matmul_work(M, N,
 *            K) bytes, 16-byte aligned.  Where that is not 0 (few tiles of C and a long K)
 *            slices of K are multiplied side by side and added up in a second launch.
 *            The result is the same with and without.
 */
int int8_matmul(const uint8_t *a_codes, const float *a_scales, const uint8_t *b_codes, const float *b_scales,
                int64_t M, int64_t N, int64_t K, void *c, int ct, int64_t ldc, void *work, int64_t work_bytes,
                void *stream);

/* Bytes of scratch memory for int8_matmul, at most 4 MB; -1 for a negative or too large
 * size.  Host only. */
int64_t qcp_int8_matmul_work(int64_t M, int64_t N, int64_t K);

/*
 * A linear layer for few rows (the tokens of a decoding step) in one launch: y = Q(x) W^T,
 * what int8_quantize of x and int8_matmul give.
 *   x          M x K elements of type xt (QCP_F16 or QCP_BF16), rows ldx apart
 *   w_codes, w_scales   the payload of W, N rows of K codes
 *   y          M x N of type xt, rows ldy apart
 * Where qcp_int8_linear_rows_fit(M, N, K) is 0 (more than 8 rows, rows too long for a
 * work-group to hold, or a product that is as quick in two launches), QCP_EUNSUPPORTED;
 * that function is host only.
 */
int int8_linear_rows(const void *x, int xt, int64_t M, int64_t K, int64_t ldx, const uint8_t *w_codes,
                     const float *w_scales, int64_t N, void *y, int64_t ldy, void *stream);
int qcp_int8_linear_rows_fit(int64_t M, int64_t N, int64_t K);

/*
 * Product of a 16-bit matrix with an INT8 payload over whose rows is summed, as a
 * backward pass has them: c[m, n] = sum over k of a[m, k] * x[k, n], where x[k, n] is
 * what int8_dequantize gives for the payload in a's type.  Accumulated in fp32, rounded
 * once to ct.
 *   a          transpose 0: M x K elements of type at (QCP_F16 or QCP_BF16), rows lda
 *              apart; 1: its transpose, K x M.  lda <= 2^23
 *   codes, scales   the payload of X, K rows of N codes; N <= 2^24
 *   c          M x N of type ct, which is QCP_F32 or at (else QCP_EUNSUPPORTED), rows
 *              ldc apart; K = 0 gives zeros
 *   work       null, or scratch memory on the device of at least qcp_int8_mixed_work(...)
 *              bytes, 16-byte aligned: for slices of a long K side by side, added up in a
 *              fixed order in a second launch, and for a copy of a large a whose rows are
 *              not aligned to 16 bytes (at most 80 and 256 MiB).  The order of the sums,
 *              and with it their last bits, differs from the product without.
 * dx = dy W: a = dy, the payload of W [out, in].  dW = dy^T x: a = dy with transpose, the
 * payload of x [tokens, in], which is all that a layer keeps of its input.  In fp16 a value
 * of the payload above 65504 is an infinity, and small ones are subnormal.
 */
int int8_matmul_mixed(const void *a, int at, int64_t lda, int32_t transpose, const uint8_t *codes,
                      const float *scales, int64_t M, int64_t N, int64_t K, void *c, int ct, int64_t ldc,
                      void *work, int64_t work_bytes, void *stream);

/* Bytes of scratch memory for int8_matmul_mixed; `aligned` is 1 for an a that is 16-byte
 * aligned with lda a multiple of 8 and at most 2^22, else 0.  -1 for a negative or too
 * large size.  Host only. */
int64_t qcp_int8_mixed_work(int64_t M, int64_t N, int64_t K, int32_t transpose, int32_t aligned);

/* Payload bytes of n codes at `bits` bits with one fp32 scale per G elements:
 * ceil(n*bits/8) + 4*ceil(n/G); -1 for invalid arguments.  Host only. */
int64_t qcp_payload_bytes(int64_t n, int32_t bits, int32_t G);

/* Static, human-readable text for a qcp_status value.  Host only. */
const char *qcp_strerror(int status);

/* Library version as "major.minor.patch".  Host only. */
const char *qcp_version(void);

/* Largest element count an entry point accepts (per tensor, or per slice of a
 * reduce): 2^36 - 4096, the most one kernel launch covers (a dispatch holds at
 * most 2^32 - 1 work-items).  Larger counts return QCP_EINVAL without a
 * launch; split such payloads into several calls.  Host only. */
int64_t qcp_max_elements(void);

#ifdef __cplusplus
}
#endif

#endif /* QCP_H */
