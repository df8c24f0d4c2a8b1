// qcp_adamw.hip -- AdamW over the many tensors of an optimizer shard, 64 to a launch.
//
// The step that stands between the gradient reduce-scatter (whose last reduce
// leaves fp32 sums on each rank) and the weight all-gather.  Per element, with
// g = grad * grad_scale:
//   m <- beta1*m + (1-beta1)*g          v <- beta2*v + (1-beta2)*g^2
//   p <- p*(1 - lr*wd) - lr/(1-beta1^t) * m / (sqrt(v)/sqrt(1-beta2^t) + eps)
// and, where wanted, a 16-bit copy of p.  Everything is computed in fp32.
//
// Moments are fp32, or 8 bits: m and r = sqrt(v) as E4M3 codes with one
// power-of-two scale per block of G.  sqrt(v) rather than v doubles the exponent
// range that 8 bits cover.  The codes are rounded stochastically: with beta2 =
// 0.999 a step moves r by about 5e-4 of itself, far below half an E4M3 spacing
// (1/16 to 1/8), so rounding to nearest would freeze it.  The scale is a power of
// two so that the grid of representable values stays where it is when a block's
// absmax drifts: a value that does not move is then not rounded again, and the
// only noise is that of the moves.  A positive r never rounds to 0, so a
// denominator never falls below the smallest step of its block while m is alive.
//
// Bound: HBM.  An element moves 8 (p) + 2 or 4 (gradient) + 2 (copy) + 4 (8-bit
// moments) or 16 (fp32 moments) bytes for about 60 operations.
//
// Layout: a work-group owns 4096 consecutive elements of one tensor, a wave 1024
// of them as 4 vectors of 256, a lane 4 consecutive elements of each vector, so
// every access of a wave is one contiguous run: 16 bytes a lane for fp32, 8 for
// 16-bit types, 4 for codes.  A block of G <= 256 lies within one vector (G/4
// lanes), G = 512 and 1024 take 2 and 4 vectors of the same lanes.  Which tensor
// a work-group belongs to is found in one step: lane i compares the work-group
// number with tensor i's first, and the ballot's population count is the answer.
// The table of tensors is a kernel argument: nothing is allocated or copied.
//
// Everything is read and written once, so loads and stores are non-temporal: 27.3M
// elements with fp32 moments 153 -> 134 us, with 8-bit ones 86 -> 70, 369M 1105 -> 1042
// (5.7 TB/s).  Only the 16-bit copies, which are read next, stay in the last cache where
// the moments are fp32 and the copies of a call are at most half of it: 27.3M elements
// 134 -> 128 us and with a quantize of the copy behind it 147 -> 140; 58.7M with the
// quantize 316 -> 293, alone 289 -> 271 on the same tensors again and 289 -> 297 on three
// sets in turn.  Beside 8-bit moments the step alone loses by it (27.3M 70 -> 73, 50.3M
// 138 -> 144; with the quantize 82 -> 81 and 160 -> 150), so there they pass it by.
#include "qcp_device.h"
#include "qcp_ops.h"

namespace qcp {

namespace {

// vectors of 4 elements at addresses aligned to their element only: tensors are
// views of larger buffers at any offset
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

template <int GT>
__device__ __forceinline__ void load4(const void *p, int64_t i, float (&x)[4]) {
    if constexpr (GT == F32) {
        const f32x4_any v = __builtin_nontemporal_load((const f32x4_any *)((const float *)p + i));
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
        const u32x2_any v = __builtin_nontemporal_load((const u32x2_any *)((const uint16_t *)p + i));
        x[0] = widen_lo<GT>(v.x); x[1] = widen_hi<GT>(v.x);
        x[2] = widen_lo<GT>(v.y); x[3] = widen_hi<GT>(v.y);
    }
}

template <int GT>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
    if constexpr (GT == F32) return ((const float *)p)[i];
    else return widen_lo<GT>(((const uint16_t *)p)[i]);
}

__device__ __forceinline__ void store4(float *p, int64_t i, const float (&x)[4]) {
    __builtin_nontemporal_store(f32x4_any{x[0], x[1], x[2], x[3]}, (f32x4_any *)(p + i));
}

template <int YT, bool KEEP>
__device__ __forceinline__ void copy4(void *p, int64_t i, const float (&x)[4]) {
    const u32x2_any v = {narrow2<YT>(x[0], x[1]), narrow2<YT>(x[2], x[3])};
    u32x2_any *to = (u32x2_any *)((uint16_t *)p + i);
    if constexpr (KEEP) *to = v;
    else __builtin_nontemporal_store(v, to);
}

template <int YT>
__device__ __forceinline__ void copy1(void *p, int64_t i, float x) {
    ((uint16_t *)p)[i] = (uint16_t)narrow2<YT>(x, x);
}

// |q| <= 448 to the E4M3 grid, up with a probability of (position between the two
// neighbours) to 16 bits: `up` holds the random bits in positions 4..19, right
// below the three mantissa bits that stay.  Below 2^-6 the spacing stays 2^-9:
// there 2^-6 is added first and taken off again.
__device__ __forceinline__ float round_e4m3(float a, uint32_t up) {
    const float small = a < 0x1p-6f ? 0x1p-6f : 0.0f;
    const uint32_t t = (__float_as_uint(a + small) + up) & 0xfff00000u;
    return __uint_as_float(t) - small;
}

// scale exponent (biased) of a block: the smallest 2^k, k >= -126, with
// absmax * 2^-k <= 448 = 1.75 * 2^8
__device__ __forceinline__ uint32_t pow2_scale(uint32_t absmax_bits) {
    const int e = (int)((absmax_bits + 0x1fffffu) >> 23) - 8;
    return (uint32_t)(e < 1 ? 1 : e);
}

// the scale that is stored: 0 for a block of zeros; NaN where a value is NaN or
// infinite (E4M3 codes could lose it, and the block with it: NaN stays for good)
__device__ __forceinline__ float block_scale(uint32_t absmax_bits, uint32_t e) {
    return absmax_bits >= 0x7f800000u ? __builtin_nanf("") : absmax_bits ? __uint_as_float(e << 23) : 0.0f;
}

template <int G> struct ogeom {
    static constexpr int GL = G >= 256 ? 64 : G / 4;        // lanes per block
    static constexpr int VB = G > 256 ? G / 256 : 1;        // vectors per block
};

constexpr int64_t kKeepCopies = (int64_t)128 << 20;        // bytes
constexpr int kVec = 4;                                     // vectors per wave
constexpr int kWaveElems = 256 * kVec;
constexpr int kGroupElems = kWaveElems * kWavesPerGroup;

// a wave's 1024 elements; FULL: all of them lie within the tensor; KEEP: the copies are
// not written past the caches
template <int GT, int G, bool KEEP, bool FULL>
__device__ __forceinline__ void adamw_wave(const AdamwTensor &t, const AdamwConst &c, float gs,
                                           int64_t base) {
    constexpr bool EIGHT = G != 0;
    const int lane = lane_id();
    float p[kVec][4], g[kVec][4], m[kVec][4], v[kVec][4];
    uint32_t mc[kVec], vc[kVec];
    float ms[kVec], vs[kVec];
    int64_t at[kVec];
    int left[kVec];                                         // elements of the vector inside, 0..4
#pragma unroll
    for (int u = 0; u < kVec; u++) {
        at[u] = base + u * 256 + lane * 4;
        if constexpr (FULL) {
            left[u] = 4;
            load4<F32>(t.param, at[u], p[u]);
            load4<GT>(t.grad, at[u], g[u]);
        } else {
            const int64_t k = t.n - at[u];
            left[u] = k < 0 ? 0 : k > 4 ? 4 : (int)k;
            if (left[u] == 4) {
                load4<F32>(t.param, at[u], p[u]);
                load4<GT>(t.grad, at[u], g[u]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    p[u][j] = j < left[u] ? t.param[at[u] + j] : 0.0f;
                    g[u][j] = j < left[u] ? load1<GT>(t.grad, at[u] + j) : 0.0f;
                }
            }
        }
        const int64_t i = t.offset + at[u];                 // place in the moments
        if constexpr (EIGHT) {
            mc[u] = vc[u] = 0;
            ms[u] = vs[u] = 0.0f;
            if (FULL || left[u] > 0) {
                mc[u] = *(const uint32_t *)((const uint8_t *)c.m + i);
                vc[u] = *(const uint32_t *)((const uint8_t *)c.v + i);
                ms[u] = c.m_scales[i / G];
                vs[u] = c.v_scales[i / G];
            }
        } else {
            if (FULL || left[u] > 0) {
                const f32x4_t a = __builtin_nontemporal_load((const f32x4_t *)((const float *)c.m + i));
                const f32x4_t b = __builtin_nontemporal_load((const f32x4_t *)((const float *)c.v + i));
                m[u][0] = a.x; m[u][1] = a.y; m[u][2] = a.z; m[u][3] = a.w;
                v[u][0] = b.x; v[u][1] = b.y; v[u][2] = b.z; v[u][3] = b.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++) m[u][j] = v[u][j] = 0.0f;
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kVec; u++) {
        if constexpr (EIGHT) {
            static_for<4>([&](auto J) {
                constexpr int j = J;
                m[u][j] = e4m3_value<j>(mc[u]) * ms[u];
                const float r = e4m3_value<j>(vc[u]) * vs[u];
                v[u][j] = r * r;
            });
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float gj = g[u][j] * gs;
            m[u][j] = m[u][j] * c.beta1 + gj * c.one_beta1;
            v[u][j] = v[u][j] * c.beta2 + (gj * gj) * c.one_beta2;
            if (!FULL && j >= left[u]) m[u][j] = v[u][j] = 0.0f;   // what pads a block stays 0
            const float r = sqrtf(v[u][j]);
            // the reciprocal's last bit only reaches the update, 2^-23 of itself
            p[u][j] = p[u][j] * c.decay -
                      (m[u][j] * c.step_size) * __builtin_amdgcn_rcpf(r * c.root_scale + c.eps);
            if constexpr (EIGHT) v[u][j] = r;
        }
        if (FULL || left[u] == 4) {
            store4(t.param, at[u], p[u]);
            if (t.copy) {
                if (c.copy_type == BF16) copy4<BF16, KEEP>(t.copy, at[u], p[u]);
                else copy4<F16, KEEP>(t.copy, at[u], p[u]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (j >= left[u]) continue;
                t.param[at[u] + j] = p[u][j];
                if (!t.copy) continue;
                if (c.copy_type == BF16) copy1<BF16>(t.copy, at[u] + j, p[u][j]);
                else copy1<F16>(t.copy, at[u] + j, p[u][j]);
            }
        }
        if constexpr (!EIGHT) {
            if (FULL || left[u] > 0) {
                const int64_t i = t.offset + at[u];
                __builtin_nontemporal_store(f32x4_t{m[u][0], m[u][1], m[u][2], m[u][3]}, (f32x4_t *)((float *)c.m + i));
                __builtin_nontemporal_store(f32x4_t{v[u][0], v[u][1], v[u][2], v[u][3]}, (f32x4_t *)((float *)c.v + i));
            }
        }
    }
    if constexpr (EIGHT) {
        using Gm = ogeom<G ? G : 32>;
#pragma unroll
        for (int u0 = 0; u0 < kVec; u0 += Gm::VB) {
            uint32_t ma = 0, va = 0;
#pragma unroll
            for (int u = u0; u < u0 + Gm::VB; u++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    ma = max(ma, __float_as_uint(m[u][j]) & 0x7fffffffu);
                    va = max(va, __float_as_uint(v[u][j]));
                }
            ma = group_max_u32<Gm::GL>(ma);
            va = group_max_u32<Gm::GL>(va);
            const uint32_t me = pow2_scale(ma), ve = pow2_scale(va);
            const float mr = __uint_as_float((254u - me) << 23), vr = __uint_as_float((254u - ve) << 23);
#pragma unroll
            for (int u = u0; u < u0 + Gm::VB; u++) {
                const int64_t i = t.offset + at[u];
                float mq[4], vq[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const uint32_t h = adamw_mix((uint32_t)(i + j) ^ (c.key + (uint32_t)(i >> 32) * 0x9e3779b9u));
                    const float a = m[u][j] * mr;
                    mq[j] = __builtin_copysignf(round_e4m3(__builtin_fabsf(a), (h & 0xffffu) << 4), a);
                    const float b = round_e4m3(v[u][j] * vr, (h >> 16) << 4);
                    vq[j] = v[u][j] > 0.0f ? __builtin_fmaxf(b, 0x1p-9f) : 0.0f;
                }
                if (FULL || left[u] > 0) {
                    __builtin_nontemporal_store(e4m3_pack4(mq[0], mq[1], mq[2], mq[3]), (uint32_t *)((uint8_t *)c.m + i));
                    __builtin_nontemporal_store(e4m3_pack4(vq[0], vq[1], vq[2], vq[3]), (uint32_t *)((uint8_t *)c.v + i));
                }
            }
            const int64_t i = t.offset + at[u0];
            if ((lane & (Gm::GL - 1)) == 0 && (FULL || left[u0] > 0)) {
                c.m_scales[i / G] = block_scale(ma, me);
                c.v_scales[i / G] = block_scale(va, ve);
            }
        }
    }
}

template <int GT, int G, bool KEEP, int CAP>
__global__ __launch_bounds__(kThreads) void k_adamw(const AdamwTable<CAP> table, const AdamwConst c) {
    const uint32_t wg = __builtin_amdgcn_workgroup_id_x();
    const int lane = lane_id();
    const uint32_t first = lane < CAP ? table.first[lane] : 0xffffffffu;
    const int which = __builtin_amdgcn_readfirstlane(__popcll(__ballot(first <= wg)) - 1);
    const AdamwTensor t = table.t[which];
    const int wave = __builtin_amdgcn_readfirstlane((int)(__builtin_amdgcn_workitem_id_x() >> 6));
    const int64_t base = (int64_t)(wg - table.first[which]) * kGroupElems + wave * kWaveElems;
    if (base >= t.n) return;
    const float gs = c.grad_scale ? *c.grad_scale : 1.0f;
    if (base + kWaveElems <= t.n) adamw_wave<GT, G, KEEP, true>(t, c, gs, base);
    else adamw_wave<GT, G, KEEP, false>(t, c, gs, base);
}

template <int GT, int G, bool KEEP, int CAP>
hipError_t run_cap(const AdamwTensor *t, int n, const AdamwConst &c, hipStream_t st) {
    AdamwTable<CAP> table;
    uint32_t groups = 0;
    for (int i = 0; i < CAP; i++) {
        table.first[i] = i < n ? groups : 0xffffffffu;
        table.t[i] = i < n ? t[i] : AdamwTensor{};
        if (i < n) groups += (uint32_t)((t[i].n + kGroupElems - 1) / kGroupElems);
    }
    hipLaunchKernelGGL((k_adamw<GT, G, KEEP, CAP>), dim3(groups), dim3(kThreads), 0, st, table, c);
    return hipGetLastError();
}

// as few launches as the table's 64 places and the grid's limit allow
template <int GT, int G, bool KEEP>
hipError_t run_tables(const AdamwTensor *t, int n, const AdamwConst &c, hipStream_t st) {
    for (int at = 0; at < n;) {
        int64_t groups = 0;
        int k = 0;
        while (at + k < n && k < 64) {
            const int64_t more = (t[at + k].n + kGroupElems - 1) / kGroupElems;
            if (k && groups + more > kMaxGroups) break;
            groups += more;
            k++;
        }
        const hipError_t e = k <= 8 ? run_cap<GT, G, KEEP, 8>(t + at, k, c, st)
                                    : run_cap<GT, G, KEEP, 64>(t + at, k, c, st);
        if (e != hipSuccess) return e;
        at += k;
    }
    return hipSuccess;
}

template <int GT, int G>
hipError_t run_adamw(const AdamwTensor *t, int n, const AdamwConst &c, hipStream_t st) {
    if constexpr (G == 0) {
        int64_t copies = 0;
        for (int i = 0; i < n; i++) copies += t[i].copy ? 2 * t[i].n : 0;
        if (copies && copies <= kKeepCopies) return run_tables<GT, G, true>(t, n, c, st);
    }
    return run_tables<GT, G, false>(t, n, c, st);
}

template <int GT>
hipError_t run_state(const AdamwTensor *t, int n, int state, int G, const AdamwConst &c, hipStream_t st) {
    if (state == F32) return run_adamw<GT, 0>(t, n, c, st);
    switch (G) {
    case 32: return run_adamw<GT, 32>(t, n, c, st);
    case 64: return run_adamw<GT, 64>(t, n, c, st);
    case 128: return run_adamw<GT, 128>(t, n, c, st);
    case 256: return run_adamw<GT, 256>(t, n, c, st);
    case 512: return run_adamw<GT, 512>(t, n, c, st);
    case 1024: return run_adamw<GT, 1024>(t, n, c, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_adamw(const AdamwTensor *t, int n, int gt, int state, int G, const AdamwConst &c,
                        hipStream_t st) {
    switch (gt) {
    case F16: return run_state<F16>(t, n, state, G, c, st);
    case BF16: return run_state<BF16>(t, n, state, G, c, st);
    case F32: return run_state<F32>(t, n, state, G, c, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qcp
