// Expert choice from router logits: softmax or sigmoid scores, a balance bias
// that moves the choice but not the weight, groups of experts, top-k, weights
// renormalised over the chosen and scaled.  The layer's own rule ("softmax
// after top-k") is the case softmax, no bias, one group, renormalised; "GPT-OSS
// on Day 0" (perplexity.ai hub blog, MoE routing) names the scheme as the main
// thing that differs between MoE models, with softmax over all experts for
// others.
//
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e))        c_e = s_e + bias_e
//   group score = sum of the group_top (1 or 2) largest c of the group
//   the top_groups best groups stay open; the k largest c in them are chosen
//   w_j = s_j  [/ (sum_j s_j + 1e-20)]  * scale
//
// Ties go to the lower index, and choices are those of the formula in 64 bits:
// without a bias c orders like the logits, so the logits themselves are
// compared (exact); with one, fp32 scores are compared, and a row in which a
// different candidate lies within the fp32 error of the border (about one row
// in 10^4) is chosen again in 64 bits by the same warp.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "moe_device.cuh"
#include "moe_internal.h"
#include "moe_scan.cuh"

namespace moe {

constexpr int kGateWarps = 8;
constexpr uint32_t kFull = 0xffffffffu;

// Unsigned key that orders like the float (-inf lowest); 0 stands below every
// key: experts past E, in closed groups, or taken already.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kFull, v); }

// One logit; -0 is 0 (they tie), NaN counts as -inf and +inf as the largest
// finite value, so that no comparison or difference below is undefined.
__device__ __forceinline__ float clean(float x) {
    x = x + 0.0f;
    if (!(x == x)) return -INFINITY;
    return fminf(x, 3.402823466e38f);
}
template <int DT>
__device__ __forceinline__ float logit_at(const void* row, int e) {
    if (DT == kDtFp32) return clean(static_cast<const float*>(row)[e]);
    if (DT == kDtFp16) return clean(__half2float(static_cast<const __half*>(row)[e]));
    return clean(bf16_bits_to_f32(static_cast<const uint16_t*>(row)[e]));
}

// Lane l holds experts [l*VPL, (l+1)*VPL), so the lowest lane and then the
// lowest register of a tie is the lowest expert, and a row is one or two wide
// loads per lane when its start is aligned and no lane straddles E.
template <int VPL, int DT>
__device__ __forceinline__ void load_row(const GateParams& p, const void* row, int lane, float (&x)[VPL]) {
    const int e0 = lane * VPL;
    if (p.vec) {
        constexpr int BYTES = VPL * (DT == kDtFp32 ? 4 : 2);
        constexpr int W = (BYTES + 3) / 4;
        uint32_t w[W];
        if (e0 < p.E) {
            const uint8_t* src = static_cast<const uint8_t*>(row) + (size_t)lane * BYTES;
            if constexpr (BYTES >= 16) {
#pragma unroll
                for (int i = 0; i < BYTES / 16; ++i) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i);
                    w[4 * i] = v.x;
                    w[4 * i + 1] = v.y;
                    w[4 * i + 2] = v.z;
                    w[4 * i + 3] = v.w;
                }
            } else if constexpr (BYTES == 8) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
                w[0] = v.x;
                w[1] = v.y;
            } else if constexpr (BYTES == 4) {
                w[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
            } else {
                w[0] = __ldg(reinterpret_cast<const uint16_t*>(src));
            }
        }
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            float v;
            if (DT == kDtFp32) {
                v = __uint_as_float(w[j]);
            } else {
                const uint16_t h = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
                v = DT == kDtFp16 ? __half2float(__ushort_as_half(h)) : bf16_bits_to_f32(h);
            }
            x[j] = e0 < p.E ? clean(v) : -INFINITY;
        }
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) x[j] = e0 + j < p.E ? logit_at<DT>(row, e0 + j) : -INFINITY;
    }
}

// The k chosen experts of one row in 64 bits, expert of round r in lane r.
// Same rules as the fp32 path; slow and rare, so kept small: every reduction
// is a full butterfly.
template <int VPL, int DT>
__device__ __noinline__ int choose_64(const GateParams& p, const void* row, int lane) {
    double c[VPL];
    double m = -INFINITY;
    for (int j = 0; j < VPL; ++j) {
        const int e = lane * VPL + j;
        c[j] = e < p.E ? (double)logit_at<DT>(row, e) : -INFINITY;
        m = fmax(m, c[j]);
    }
    if (p.score == 0) {
        for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kFull, m, o));
        double z = 0.0;
        for (int j = 0; j < VPL; ++j) {
            c[j] = m == -INFINITY ? 0.0 : exp(c[j] - m);
            z += lane * VPL + j < p.E ? c[j] : 0.0;
        }
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
        for (int j = 0; j < VPL; ++j) c[j] = z > 0.0 ? c[j] / z : 0.0;
    } else {
        for (int j = 0; j < VPL; ++j) c[j] = 1.0 / (1.0 + exp(-c[j]));
    }
    for (int j = 0; j < VPL; ++j) {
        const int e = lane * VPL + j;
        if (e < p.E && p.bias) c[j] += (double)p.bias[e];
        if (e >= p.E) c[j] = -INFINITY;
    }
    uint32_t open = kFull;
    if (p.groups > 1) {
        const int gs = p.E / p.groups;
        double mine = -INFINITY;  // group `lane`'s score
        for (int g = 0; g < p.groups; ++g) {
            double a = -INFINITY, b = -INFINITY;
            for (int j = 0; j < VPL; ++j) {
                const int e = lane * VPL + j;
                if (e < g * gs || e >= (g + 1) * gs) continue;
                b = fmax(b, fmin(a, c[j]));
                a = fmax(a, c[j]);
            }
            for (int o = 16; o > 0; o >>= 1) {
                const double oa = __shfl_xor_sync(kFull, a, o), ob = __shfl_xor_sync(kFull, b, o);
                b = fmax(fmin(a, oa), fmax(b, ob));
                a = fmax(a, oa);
            }
            if (lane == g) mine = p.group_top == 2 ? a + b : a;
        }
        int rank = 0;
        for (int g = 0; g < p.groups; ++g) {
            const double v = __shfl_sync(kFull, mine, g);
            rank += v > mine || (v == mine && g < lane);
        }
        open = __ballot_sync(kFull, lane < p.groups && rank < p.top_groups);
    }
    uint32_t live = 0;
    for (int j = 0; j < VPL; ++j) {
        const int e = lane * VPL + j;
        if (e < p.E && !p.bias) c[j] = (double)logit_at<DT>(row, e);  // scores order like the logits
        if (e < p.E && (p.groups == 1 || ((open >> (e / (p.E / p.groups))) & 1u))) live |= 1u << j;
    }
    int got = 0;
    for (int r = 0; r < p.k; ++r) {
        double v = -INFINITY;
        int be = 0x7fffffff;
        for (int j = 0; j < VPL; ++j)
            if (((live >> j) & 1u) && (be == 0x7fffffff || c[j] > v)) {
                v = c[j];
                be = lane * VPL + j;
            }
        for (int o = 16; o > 0; o >>= 1) {
            const double ov = __shfl_xor_sync(kFull, v, o);
            const int oe = __shfl_xor_sync(kFull, be, o);
            if (oe != 0x7fffffff && (be == 0x7fffffff || ov > v || (ov == v && oe < be))) {
                v = ov;
                be = oe;
            }
        }
        if (lane == r) got = be;
        if (be / VPL == lane) live &= ~(1u << (be % VPL));
    }
    return got;
}

// One warp per token.  p.r.hist != nullptr: the layer's routing step, which
// also counts the chunk histogram and lets the last CTA scan it.
template <int VPL, int DT>
__global__ void __launch_bounds__(kGateWarps * 32) gate_kernel(GateParams p) {
    __shared__ int s_scan[kGateWarps * VPL * 36];  // the choices of each warp's row (groups); later the scan's staging
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * kGateWarps + warp;
    if (t < p.T) {
        const uint8_t* row = static_cast<const uint8_t*>(p.logits) + (size_t)t * p.ld_bytes;
        float x[VPL], c[VPL];
        load_row<VPL, DT>(p, row, lane, x);
        const int e0 = lane * VPL;
        const bool scored = p.bias != nullptr || (p.groups > 1 && p.group_top == 2);  // fp32 scores are compared
        float m = 0.f, z = 1.f;
        if (p.score == 0 && (scored || !p.renorm)) {  // softmax over all experts
            float mx = x[0];
#pragma unroll
            for (int j = 1; j < VPL; ++j) mx = fmaxf(mx, x[j]);
            m = key_value(warp_max(order_key(mx)));
            z = 0.f;
#pragma unroll
            for (int j = 0; j < VPL; ++j) z += m == -INFINITY ? 0.f : expf(x[j] - m);  // past E: exp(-inf) = 0
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
        }
        const float rz = z > 0.f ? 1.0f / z : 0.f;
        if (scored) {
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                // sigmoid: ex2 and rcp approximations, absolute error below 2^-22 (the error of
                // exp(-x) enters times s (1 - s))
                const float s = p.score == 0 ? (m == -INFINITY ? 0.f : __expf(x[j] - m) * rz)
                                             : __fdividef(1.0f, 1.0f + __expf(-fmaxf(x[j], -80.f)));
                c[j] = s + (p.bias && e0 + j < p.E ? __ldg(p.bias + e0 + j) : 0.f);
            }
        } else {
#pragma unroll
            for (int j = 0; j < VPL; ++j) c[j] = x[j];
        }
        bool unsure = false;
        uint32_t open = kFull;
        const int gs = p.gsize;
        if (p.groups > 1) {
            // P lanes to a group, members dealt round; the choices pass through shared memory
            // (a pad of 4 per 32 spreads groups of 32 over the banks)
            float* sc = reinterpret_cast<float*>(s_scan) + warp * VPL * 36;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int e = e0 + j;
                sc[e + ((e >> 5) << 2)] = c[j];
            }
            __syncwarp();
            const int P = p.lanes_per_group;
            const int g = lane / P;
            float a = -INFINITY, b = -INFINITY;
            if (g < p.groups)
                for (int i = lane % P; i < gs; i += P) {
                    const int e = g * gs + i;
                    const float v = sc[e + ((e >> 5) << 2)];
                    b = fmaxf(b, fminf(a, v));
                    a = fmaxf(a, v);
                }
            for (int o = P >> 1; o > 0; o >>= 1) {
                const float oa = __shfl_xor_sync(kFull, a, o), ob = __shfl_xor_sync(kFull, b, o);
                b = fmaxf(fminf(a, oa), fmaxf(b, ob));
                a = fmaxf(a, oa);
            }
            const float mine = p.group_top == 2 ? a + b : a;
            int rank = 0;
            for (int q = 0; q < p.groups; ++q) {
                const float v = __shfl_sync(kFull, mine, q * P);
                rank += v > mine || (v == mine && q < g);
            }
            const bool lead = g < p.groups && lane % P == 0;
            if (scored) {
                // another group within the error of the last open one's score (two choices of
                // absolute error 2^-20 (1 + |c|) each at most)
                const float last = key_value(warp_max(lead && rank == p.top_groups - 1 ? order_key(mine) : 0u));
                const float mag = 2.f + fabsf(a) + (p.group_top == 2 ? fabsf(b) : 0.f);
                const float err = 0x1p-20f * key_value(warp_max(lead ? order_key(mag) : 0u));
                unsure = __any_sync(kFull, lead && rank != p.top_groups - 1 && fabsf(mine - last) <= 2.f * err);
            }
            const uint32_t bits = __ballot_sync(kFull, lead && rank < p.top_groups);
            open = bits;  // bit q * P: group q is open
            __syncwarp();
        }
        uint32_t key[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = e0 + j;
            bool in = e < p.E;
            if (p.groups > 1) in = in && ((open >> ((e / gs) * p.lanes_per_group)) & 1u);
            // with groups by sums and no bias the experts still order like their logits
            key[j] = in ? order_key(p.bias ? c[j] : x[j]) : 0u;
        }
        int mine = 0;  // lane r: the expert of round r
        uint32_t last = 0;
        if (!unsure) {
            uint32_t left[VPL];
#pragma unroll
            for (int j = 0; j < VPL; ++j) left[j] = key[j];
            for (int r = 0; r < p.k; ++r) {
                uint32_t best = left[0];
#pragma unroll
                for (int j = 1; j < VPL; ++j) best = max(best, left[j]);
                last = warp_max(best);
                int at = 0;
#pragma unroll
                for (int j = VPL - 1; j >= 0; --j) at = left[j] == last ? j : at;
                const int w = __ffs(__ballot_sync(kFull, best == last)) - 1;
                const int e = __shfl_sync(kFull, e0 + at, w);
                if (lane == r) mine = e;
#pragma unroll
                for (int j = 0; j < VPL; ++j) left[j] = e == e0 + j ? 0u : left[j];
            }
            if (p.bias) {
                // a candidate within the error of the border that is not the same logit and bias?
                const float ck = key_value(last);
                const int ek = __shfl_sync(kFull, mine, p.k - 1);
                const float xk = logit_at<DT>(row, ek), bk = p.bias[ek];
                const float err = 0x1p-20f * (1.f + fabsf(ck));
                bool near = false;
#pragma unroll
                for (int j = 0; j < VPL; ++j)
                    if (key[j] != 0u && fabsf(c[j] - ck) <= 2.f * err)
                        near = near || x[j] != xk || __ldg(p.bias + e0 + j) != bk;
                unsure = __any_sync(kFull, near);
            }
        }
        if (unsure) mine = choose_64<VPL, DT>(p, row, lane);

        // weights: lane r < k has one chosen expert
        const bool has = lane < p.k;
        const float xe = has ? logit_at<DT>(row, mine) : -INFINITY;
        float s;
        if (p.score == 0) {
            if (!scored && p.renorm) {  // the sum over all experts cancels
                m = key_value(warp_max(has ? order_key(xe) : 0u));
                s = has && m != -INFINITY ? expf(xe - m) : 0.f;
            } else {
                s = has && m != -INFINITY ? expf(xe - m) * rz : 0.f;
            }
        } else {
            s = has ? 1.0f / (1.0f + expf(-xe)) : 0.f;
        }
        if (p.renorm) {
            float sum = s;
#pragma unroll
            for (int o = kMaxTopK / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
            s = s / (sum + 1e-20f);
        }
        s *= p.scale;
        int slot = 0;
        for (int q = 0; q < p.k; ++q) slot += __shfl_sync(kFull, mine, q) < mine;
        if (has) {
            const size_t o = (size_t)t * p.k + slot;
            p.r.topk_idx[o] = mine;
            p.r.topk_w[o] = s;
            if (p.r.hist) {
                __nv_bfloat16 wb = __float2bfloat16_rn(s);
                p.r.topk_wb[o] = *reinterpret_cast<uint16_t*>(&wb);
                atomicAdd(&p.r.hist[(size_t)(t / kChunkTokens) * p.E + mine], 1);
            }
        }
    }
    if (p.r.hist && last_to_arrive(p.r.done, gridDim.x)) finish_scan(p.r, s_scan, kGateWarps * VPL * 36);
}

template <int VPL>
static cudaError_t launch_gate_v(const GateParams& p, int dtype, cudaStream_t st) {
    const int grid = (p.T + kGateWarps - 1) / kGateWarps;
    if (dtype == kDtFp32)
        gate_kernel<VPL, kDtFp32><<<grid, kGateWarps * 32, 0, st>>>(p);
    else if (dtype == kDtFp16)
        gate_kernel<VPL, kDtFp16><<<grid, kGateWarps * 32, 0, st>>>(p);
    else
        gate_kernel<VPL, kDtBf16><<<grid, kGateWarps * 32, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_gate(const GateParams& p_in, int dtype, cudaStream_t st) {
    GateParams p = p_in;
    const int vpl = p.E <= 32 ? 1 : p.E <= 64 ? 2 : p.E <= 128 ? 4 : 8;
    const size_t lane_bytes = (size_t)vpl * (dtype == kDtFp32 ? 4 : 2);
    const size_t al = lane_bytes < 16 ? lane_bytes : 16;
    p.vec = p.E % vpl == 0 && reinterpret_cast<uintptr_t>(p.logits) % al == 0 && p.ld_bytes % al == 0;
    p.gsize = p.E / p.groups;
    int P = 32;
    while (P * p.groups > 32) P >>= 1;
    p.lanes_per_group = P;
    switch (vpl) {
        case 1: return launch_gate_v<1>(p, dtype, st);
        case 2: return launch_gate_v<2>(p, dtype, st);
        case 4: return launch_gate_v<4>(p, dtype, st);
        default: return launch_gate_v<8>(p, dtype, st);
    }
}

}  // namespace moe
