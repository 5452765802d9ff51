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
// Ties go to the lower index.  Without a bias c rises with the logit, so experts
// (and groups by one best) are ordered by the logits themselves, whole -- also
// where 64 bits would round two scores to one.  With a bias, and for sums of two,
// choices are those of the formula in 64 bits: fp32 scores are compared, and where
// a candidate lies within the fp32 error of the border the same warp ranks those
// few again in 64 bits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "moe_device.cuh"
#include "moe_internal.h"
#include "moe_scan.cuh"

namespace moe {

constexpr int kGateWarps = 8;
constexpr int kGateCtas = 3;  // per SM at most
constexpr uint32_t kFull = 0xffffffffu;
// Words of shared memory of a warp: up to 32 VPL 64-bit values and as many
// expert numbers (or 36 VPL choices).
template <int VPL>
constexpr int kListAt = 64 * VPL;
template <int VPL>
constexpr int kScratch = 96 * VPL;

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
__device__ __forceinline__ float warp_max(float v) {  // of numbers; -0 stays below 0
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// One logit; -0 is 0 (they tie), NaN counts as -inf and +inf as the largest
// finite value, so that no comparison or difference below is undefined.
__device__ __forceinline__ float clean(float x) {
    return fminf(fmaxf(x + 0.0f, -INFINITY), 3.402823466e38f);  // fmaxf takes the number of a number and a NaN
}
template <int DT>
__device__ __forceinline__ float logit_at(const void* row, int e) {
    if (DT == kDtFp32) return clean(static_cast<const float*>(row)[e]);
    if (DT == kDtFp16) return clean(__half2float(static_cast<const __half*>(row)[e]));
    return clean(bf16_bits_to_f32(static_cast<const uint16_t*>(row)[e]));
}

// Lane l holds experts [l*VPL, (l+1)*VPL), so the lowest lane and then the
// lowest register of a tie is the lowest expert, and a row is one or two wide
// loads per lane when its start is aligned and no lane straddles E.  What is past
// E holds -inf: set once by clear(), and left alone by the wide loads.
template <int VPL, int DT>
struct RawRow {
    static constexpr int BYTES = VPL * (DT == kDtFp32 ? 4 : 2);
    // -inf
    static constexpr uint32_t kAbsent = DT == kDtFp32 ? 0xff800000u : DT == kDtFp16 ? 0xfc00fc00u : 0xff80ff80u;
    uint32_t w[(BYTES + 3) / 4];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < (BYTES + 3) / 4; ++i) w[i] = kAbsent;
    }
};
template <int VPL, int DT>
__device__ __forceinline__ void load_row(const GateParams& p, const uint8_t* row, int lane, RawRow<VPL, DT>& v) {
    constexpr int BYTES = RawRow<VPL, DT>::BYTES;
    const int e0 = lane * VPL;
    if (p.vec) {
        if (e0 >= p.E) return;
        const uint8_t* src = row + lane * BYTES;
        if constexpr (BYTES >= 16) {
#pragma unroll
            for (int i = 0; i < BYTES / 16; ++i) {
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(src) + i);
                v.w[4 * i] = u.x;
                v.w[4 * i + 1] = u.y;
                v.w[4 * i + 2] = u.z;
                v.w[4 * i + 3] = u.w;
            }
        } else if constexpr (BYTES == 8) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(src));
            v.w[0] = u.x;
            v.w[1] = u.y;
        } else if constexpr (BYTES == 4) {
            v.w[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
        } else {
            v.w[0] = __ldg(reinterpret_cast<const uint16_t*>(src));
        }
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            if (DT == kDtFp32) {
                v.w[j] = e0 + j < p.E ? reinterpret_cast<const uint32_t*>(row)[e0 + j] : RawRow<VPL, DT>::kAbsent;
            } else {
                const uint32_t h = e0 + j < p.E ? reinterpret_cast<const uint16_t*>(row)[e0 + j]
                                                : RawRow<VPL, DT>::kAbsent & 0xffffu;
                v.w[j / 2] = j & 1 ? v.w[j / 2] | (h << 16) : h;
            }
        }
    }
}
template <int VPL, int DT>
__device__ __forceinline__ void unpack_row(const RawRow<VPL, DT>& v, float (&x)[VPL]) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        float f;
        if (DT == kDtFp32) {
            f = __uint_as_float(v.w[j]);
        } else {
            const uint16_t h = (uint16_t)(v.w[j / 2] >> (16 * (j & 1)));
            f = DT == kDtFp16 ? __half2float(__ushort_as_half(h)) : bf16_bits_to_f32(h);
        }
        x[j] = f;
    }
}

// Two largest of what a group of `width` lanes hold, in every lane of it.
template <typename T>
__device__ __forceinline__ void top2_lanes(T& a, T& b, int width) {
    for (int o = width >> 1; o > 0; o >>= 1) {
        const T oa = __shfl_xor_sync(kFull, a, o), ob = __shfl_xor_sync(kFull, b, o);
        const T low = a < oa ? a : oa, nb = b > ob ? b : ob;
        b = low > nb ? low : nb;
        a = a > oa ? a : oa;
    }
}

// fp32 choices of a lane's experts: scores and bias, or the logits themselves.
// A score's error: sigmoid -- exp (2 + 1.2 |x| steps of 2^-23, times s (1 - s)),
// the sum and the reciprocal: below 2^-21.7; softmax -- relative, 2 + 1.2 d
// steps of exp(-d), 8 of the sum z, 2 more: below 2^-19.4 of the largest.
template <int VPL>
__device__ __forceinline__ void choices(const GateParams& p, const float (&x)[VPL], const float (&bias)[VPL],
                                        bool scored, float m, float rz, float (&c)[VPL]) {
    if (!scored) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) c[j] = x[j];
    } else if (p.score == 0) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) c[j] = (m == -INFINITY ? 0.f : __expf(x[j] - m) * rz) + bias[j];
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) c[j] = rcp_approx(1.0f + __expf(-x[j])) + bias[j];
    }
}
// A bias, and the sum of a group, count as at most kMostBias either way (NaN as the
// least): sums and differences of choices stay finite, all masked experts (-inf) tie,
// and so do the groups that have one among their best.
constexpr float kMostBias = 0x1p126f;
__device__ __forceinline__ float bounded(float b) { return fminf(fmaxf(b, -kMostBias), kMostBias); }
__device__ __forceinline__ float pair_sum(float a, float b) { return a >= kMostBias ? kMostBias : bounded(a + b); }
__device__ __forceinline__ double pair_sum(double a, double b) {
    const double most = kMostBias;
    return a >= most ? most : fmin(fmax(a + b, -most), most);
}
template <int VPL>
__device__ __forceinline__ void load_bias(const GateParams& p, int e0, float (&bias)[VPL]) {
#pragma unroll
    for (int j = 0; j < VPL; ++j)  // -inf past E: so are the choices
        bias[j] = e0 + j >= p.E ? -INFINITY : p.bias ? bounded(__ldg(p.bias + e0 + j)) : 0.f;
}
// Bound of the error of an fp32 choice of size |c|; rz: the largest softmax score.
// c less its bound grows with c, and so does c with it added: a choice that is clear
// of the border by the border's bound is clear by its own.
__device__ __forceinline__ float choice_error(const GateParams& p, float rz, float c) {
    return (p.score == 0 ? 0x1p-19f * rz : 0x1p-21f) + 0x1p-23f * fabsf(c);
}

// One score in 64 bits; out of line, so that its registers are paid for once.
__device__ __noinline__ double score_64(float x, float m, double z, int score) {
    if (score == 0) return m == -INFINITY ? 0.0 : exp((double)x - (double)m) / z;
    return 1.0 / (1.0 + exp(-(double)x));
}

// The 64-bit choices of the experts flagged in `want` (bit j: expert e0 + j),
// dealt one to a lane so that the warp evaluates them together; list and value
// are the warp's shared memory, the count is returned.
template <int VPL, int DT>
__device__ __forceinline__ int choices_64(const GateParams& p, const uint8_t* row, int lane, uint32_t want, float m,
                                          double z64, int* list, double* value) {
    int at = __popc(want);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, at, o);
        if (lane >= o) at += v;
    }
    const int n = __shfl_sync(kFull, at, 31);
    at -= __popc(want);
    for (uint32_t w = want; w; w &= w - 1) list[at++] = lane * VPL + __ffs(w) - 1;
    __syncwarp();
    for (int i = lane; i < n; i += 32) {
        const int e = list[i];
        const double s = score_64(logit_at<DT>(row, e), m, z64, p.score);
        value[i] = p.bias ? s + (double)bounded(p.bias[e]) : s;
    }
    __syncwarp();
    return n;
}

// The k chosen experts of a row with candidates too close for the fast path,
// expert of round r in lane r.  Logits are compared whole; of fp32 scores, the
// groups and experts within the error of the border (as a rule two of them)
// are ranked again in 64 bits, the others are settled by the fp32 values.
// open: the lane's experts in open groups, or settle_groups to choose those too.
template <int VPL, int DT>
__device__ __noinline__ int choose_close(const GateParams& p, const uint8_t* row, int lane, float m, float rz,
                                         uint32_t live, bool settle_groups, int* scratch) {
    // the warp's kScratch words: 64-bit values, then (kListAt) the list of their experts
    double* value = reinterpret_cast<double*>(scratch);
    int* list = scratch + kListAt<VPL>;
    float x[VPL], c[VPL];
    const int e0 = lane * VPL;
    {
        RawRow<VPL, DT> raw;
        raw.clear();
        load_row<VPL, DT>(p, row, lane, raw);
        unpack_row<VPL, DT>(raw, x);
#pragma unroll
        for (int j = 0; j < VPL; ++j) x[j] = clean(x[j]);
    }
    const bool scored = p.bias != nullptr || (p.groups > 1 && p.group_top == 2);
    {
        float bias[VPL];
        load_bias<VPL>(p, e0, bias);
        choices<VPL>(p, x, bias, scored, m, rz, c);
    }
    double z64 = 1.0;
    if (scored && p.score == 0) {
        z64 = 0.0;
#pragma unroll
        for (int j = 0; j < VPL; ++j) z64 += e0 + j < p.E ? score_64(x[j], m, 1.0, 0) : 0.0;
        for (int o = 16; o > 0; o >>= 1) z64 += __shfl_xor_sync(kFull, z64, o);
    }
    const int gs = p.gsize;
    if (settle_groups) {
        float mine = -INFINITY, second = -INFINITY, err = 0.f;  // of group `lane`
        for (int g = 0; g < p.groups; ++g) {
            float a = -INFINITY, b = -INFINITY;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int e = e0 + j;
                if (e < g * gs || e >= (g + 1) * gs) continue;
                b = fmaxf(b, fminf(a, c[j]));
                a = fmaxf(a, c[j]);
            }
            top2_lanes(a, b, 32);
            if (lane == g) {
                mine = p.group_top == 2 ? pair_sum(a, b) : a;
                second = p.group_top == 2 ? b : a;
                err = 2.f * choice_error(p, rz, fabsf(a) + (p.group_top == 2 ? fabsf(b) : 0.f));
            }
        }
        int rank = 0;
        for (int g = 0; g < p.groups; ++g) {
            const float v = __shfl_sync(kFull, mine, g);
            rank += v > mine || (v == mine && g < lane);
        }
        uint32_t open = __ballot_sync(kFull, lane < p.groups && rank < p.top_groups);
        if (scored && p.top_groups < p.groups) {
            // near: groups that their errors may bring past one on the other side of the border
            const bool in = (open >> lane) & 1u, out = lane < p.groups && !in;
            const float lowest = -warp_max(in ? err - mine : -INFINITY);
            const float highest = warp_max(out ? mine + err : -INFINITY);
            const bool clear = in && mine - err > highest;
            const uint32_t sure = __ballot_sync(kFull, clear);
            const uint32_t near = __ballot_sync(kFull, (in && !clear) || (out && mine + err >= lowest));
            const float from = second - 2.f * err;
            uint32_t want = 0;  // members of near groups that may be among their largest
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int g = e0 + j < p.E ? (e0 + j) / gs : 0;
                const float least = __shfl_sync(kFull, from, g);
                if (e0 + j < p.E && ((near >> g) & 1u) && c[j] >= least) want |= 1u << j;
            }
            const int n = choices_64<VPL, DT>(p, row, lane, want, m, z64, list, value);
            double a = -INFINITY, b = -INFINITY;
            if ((near >> lane) & 1u)
                for (int i = 0; i < n; ++i) {
                    if (list[i] / gs != lane) continue;
                    b = fmax(b, fmin(a, value[i]));
                    a = fmax(a, value[i]);
                }
            __syncwarp();
            const double exact = p.group_top == 2 ? pair_sum(a, b) : a;
            int before = __popc(sure);
            for (uint32_t left = near; left; left &= left - 1) {
                const int g = __ffs(left) - 1;
                const double v = __shfl_sync(kFull, exact, g);
                before += v > exact || (v == exact && g < lane);
            }
            open = sure | __ballot_sync(kFull, ((near >> lane) & 1u) && before < p.top_groups);
        }
        live = 0;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (e0 + j < p.E && ((open >> ((e0 + j) / gs)) & 1u)) live |= 1u << j;
    }
    // the k largest whole keys; without a bias the experts order like their logits
    uint32_t left = live, last = 0;
    int mine = 0;
    for (int r = 0; r < p.k; ++r) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int j = VPL - 1; j >= 0; --j) {
            const uint32_t key = (left >> j) & 1u ? order_key(p.bias ? c[j] : x[j]) : 0u;
            if (key >= best) best = key, at = j;
        }
        last = warp_max(best);
        const int w = __ffs(__ballot_sync(kFull, best == last)) - 1;
        const int e = __shfl_sync(kFull, e0 + at, w);
        if (lane == r) mine = e;
        if (lane == w) left &= ~(1u << at);
    }
    if (!p.bias) return mine;
    const float ck = key_value(last);
    const float err = choice_error(p, rz, ck);
    int sure = 0;
    uint32_t near = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        if (!((live >> j) & 1u)) continue;
        const float above = c[j] - ck;
        if (above > 2.f * err)
            ++sure;
        else if (above >= -2.f * err)
            near |= 1u << j;
    }
    sure = __reduce_add_sync(kFull, sure);  // they were the first rounds
    if (__reduce_add_sync(kFull, __popc(near)) == p.k - sure) return mine;  // all of the near are in
    const int n = choices_64<VPL, DT>(p, row, lane, near, m, z64, list, value);
    // a near expert with r near ones before it takes round sure + r
    for (int i = lane; i < (n + 31) / 32 * 32; i += 32) {
        int before = 0;
        if (i < n)
            for (int q = 0; q < n; ++q)
                before += value[q] > value[i] || (value[q] == value[i] && list[q] < list[i]);
        for (int r = sure; r < p.k; ++r) {
            const uint32_t who = __ballot_sync(kFull, i < n && before == r - sure);
            const int e = __shfl_sync(kFull, i < n ? list[i] : 0, who ? __ffs(who) - 1 : 0);
            if (who && lane == r) mine = e;
        }
    }
    return mine;
}

// Keys carry their index: 23 or 24 bits of the choice above 255 - expert (or
// 31 - group), so that one warp maximum finds value and index of the next choice
// and ties fall to the lower index.  bf16 and fp16 logits fit whole (upper bits
// of their order key).  fp32 values are laid on a grid of 2^23 steps below the
// row's largest, `reach` wide, monotone (two roundings of a monotone function);
// equal steps, steps that the scores' error can bridge, or a border below the
// grid send the row to choose_close.  With the grid that is about ten times
// rarer than with the upper bits of a float.
constexpr float kReachLogit = 16.f, kReachScore = 2.f, kReachGroup = 4.f;
constexpr uint32_t kGridFloor = 8;  // steps up to this hold what lies below the grid
__device__ __forceinline__ uint32_t grid_key(float v, float top, float reach, uint32_t tag) {
    const float d = fmaxf(v - top, reach * (0x1p-20f - 1.f));  // NaN (both -inf): the floor
    // 2^24 - 1 for the largest, 2^23 + 7 at the floor: the step is the float's mantissa
    return (__float_as_uint(fmaf(d, 0x1p23f / reach, 16777215.f)) << 9) + tag;
}
// Whether keys `w` and the next below it may be in the wrong order, for values
// off by at most e: 2e in steps, and 3 for the roundings.
__device__ __forceinline__ bool grid_close(uint32_t w, uint32_t next, float reach, float e) {
    const uint32_t apart = e > 0.f ? 3u + __float2uint_ru(fminf(2.f * e * (0x1p23f / reach), 1e9f)) : 1u;
    return (w >> 9) <= kGridFloor || (w >> 9) - (next >> 9) < apart;
}

// A CTA's warps take its tokens as they come free (a close row holds up one warp
// only), the next token's logits in flight.
// 16384 rows of 256 fp32 experts, sigmoid, bias, 4 of 8 groups, top-8: 21 us, 0.8 TB/s:
// ~800 instructions a row bound it (63 % of issue slots, ALU pipe 50 %); the tail of its
// 5 close rows is 3 us of that. Softmax without bias or groups: 11.5 us. 256 rows of
// 128: 2.4 us, of which a launch is most. Rows dealt out beforehand: 26 us (a close row
// delays what its warp has left); 4 or 5 CTAs an SM spill: 22.5 and 30 us.
// p.r.hist != nullptr: the layer's routing step, which also counts the chunk
// histogram and lets the last CTA scan it.
template <int VPL, int DT>
__global__ void __launch_bounds__(kGateWarps * 32, kGateCtas) gate_kernel(GateParams p) {
    // odd groups: a row's choices; close rows: their 64-bit values; later the scan's staging
    __shared__ __align__(16) int s_scan[kGateWarps * kScratch<VPL>];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e0 = lane * VPL;
    int* scratch = s_scan + warp * kScratch<VPL>;
    __shared__ int s_next;
    const bool scored = p.bias != nullptr || (p.groups > 1 && p.group_top == 2);  // fp32 scores are compared
    const bool gridded = DT == kDtFp32 || p.bias;  // of experts
    pdl_wait();
    pdl_allow_dependents();  // one wave: what follows may take its place beside it
    const float reach = p.bias ? kReachScore : kReachLogit;
    float bias[VPL];
    load_bias<VPL>(p, e0, bias);
    if (threadIdx.x == 0) s_next = kGateWarps;
    __syncthreads();
    int t = warp * gridDim.x + blockIdx.x, ahead = 0;
    auto take = [&]() {  // the next of the CTA's tokens that no warp has
        int j = 0;
        if (lane == 0) j = atomicAdd(&s_next, 1);
        return (int)min((long long)__shfl_sync(kFull, j, 0) * gridDim.x + blockIdx.x, (long long)p.T);
    };
    RawRow<VPL, DT> raw;
    raw.clear();
    // Without scores and with a grid a NaN needs no care (maxima pass it over, grid_key puts it on the
    // floor) and +inf puts the whole row there; elsewhere logits are made finite first
    const bool clean_first = scored || !gridded || (p.score == 0 && !p.renorm);
    auto row_of = [&](int i) { return static_cast<const uint8_t*>(p.logits) + (size_t)i * p.ld_bytes; };
    if (t < p.T) load_row<VPL, DT>(p, row_of(t), lane, raw);
    for (; t < p.T; t = ahead) {
        const uint8_t* row = row_of(t);
        ahead = take();
        float x[VPL], c[VPL];
        unpack_row<VPL, DT>(raw, x);
        if (clean_first) {
#pragma unroll
            for (int j = 0; j < VPL; ++j) x[j] = clean(x[j]);
        }
        if (ahead < p.T) load_row<VPL, DT>(p, row_of(ahead), lane, raw);
        float m = 0.f, rz = 1.f;
        if (p.score == 0 && (scored || !p.renorm)) {  // softmax over all experts
            float mx = x[0];
#pragma unroll
            for (int j = 1; j < VPL; ++j) mx = fmaxf(mx, x[j]);
            m = warp_max(mx);
            float z = 0.f;
#pragma unroll
            for (int j = 0; j < VPL; ++j) z += m == -INFINITY ? 0.f : expf(x[j] - m);  // past E: exp(-inf) = 0
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
            rz = z > 0.f ? 1.0f / z : 0.f;
        }
        choices<VPL>(p, x, bias, scored, m, rz, c);
        bool close = false;
        uint32_t in = kFull;  // the lane's experts in open groups
        bool open = true;     // all of them
        if (p.groups > 1) {
            const int P = p.lanes_per_group;
            float a = -INFINITY, b = -INFINITY;
            if (p.aligned) {  // a group is P whole lanes
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    b = fmaxf(b, fminf(a, c[j]));
                    a = fmaxf(a, c[j]);
                }
            } else {
                // P lanes to a group, members dealt round, through shared memory (a pad of 4
                // per 32 spreads the groups over the banks)
                float* sc = reinterpret_cast<float*>(scratch);
#pragma unroll
                for (int j = 0; j < VPL; ++j) sc[e0 + j + (((e0 + j) >> 5) << 2)] = c[j];
                __syncwarp();
                const int g = lane / P;
                if (g < p.groups)
                    for (int i = lane % P; i < p.gsize; i += P) {
                        const int e = g * p.gsize + i;
                        const float v = sc[e + ((e >> 5) << 2)];
                        b = fmaxf(b, fminf(a, v));
                        a = fmaxf(a, v);
                    }
                __syncwarp();
            }
            top2_lanes(a, b, P);
            const int g = lane / P;
            const float score = p.group_top == 2 ? pair_sum(a, b) : a;
            uint32_t gkey = 0;
            float top = 0.f;
            if (DT == kDtFp32 || scored) {
                top = warp_max(score);
                if (g < p.groups) gkey = grid_key(score, top, kReachGroup, 31u - g);
            } else if (g < p.groups) {
                gkey = (order_key(score) & ~31u) | (31u - g);
            }
            uint32_t w = kFull;
            for (int r = 0; r < p.top_groups; ++r) w = warp_max(gkey < w ? gkey : 0u);
            if ((DT == kDtFp32 || scored) && p.top_groups < p.groups) {
                // close: the errors may bring a group left out past one taken (or equal steps hide their order)
                const float err =
                    scored ? 2.f * choice_error(p, rz, fabsf(a) + (p.group_top == 2 ? fabsf(b) : 0.f)) : 0.f;
                const float lowest = -warp_max(g < p.groups && gkey >= w ? err - score : -INFINITY);
                const float highest = warp_max(g < p.groups && gkey < w ? score + err : -INFINITY);
                close = lowest <= highest;
            }
            if (p.aligned) {
                open = gkey >= w;
                in = open ? kFull : 0u;
            } else {
                const uint32_t groups = __ballot_sync(kFull, lane % P == 0 && gkey >= w);  // bit g * P
                in = 0;
#pragma unroll
                for (int j = 0; j < VPL; ++j)  // (e * ceil(2^16 / gsize)) >> 16 = e / gsize for e < 256
                    in |= ((groups >> ((((e0 + j) * p.inv_gsize) >> 16) * P)) & 1u) << j;
            }
        }
        const bool settle = close;
        uint32_t key[VPL];
        float top = 0.f;
        if (gridded) {
            float v[VPL];
            if (p.bias) {
#pragma unroll
                for (int j = 0; j < VPL; ++j) v[j] = c[j];
            } else {
#pragma unroll
                for (int j = 0; j < VPL; ++j) v[j] = x[j];
            }
            if (p.groups > 1) {
                if (p.aligned) {
                    const float shut = open ? 0.f : -INFINITY;
#pragma unroll
                    for (int j = 0; j < VPL; ++j) v[j] += shut;
                } else {
#pragma unroll
                    for (int j = 0; j < VPL; ++j) v[j] = (in >> j) & 1u ? v[j] : -INFINITY;
                }
            }
            top = v[0];
#pragma unroll
            for (int j = 1; j < VPL; ++j) top = fmaxf(top, v[j]);
            top = warp_max(top);
            // what is closed or absent lies on the floor with what is below the grid
#pragma unroll
            for (int j = 0; j < VPL; ++j) key[j] = grid_key(v[j], top, reach, 255u - (e0 + j));
        } else {
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                key[j] = (in >> j) & 1u && e0 + j < p.E ? (order_key(x[j]) & ~255u) | (255u - (e0 + j)) : 0u;
        }
        // each lane's keys in falling order, then k rounds of the warp's largest head
        if constexpr (VPL == 2) {
            const uint32_t hi = max(key[0], key[1]), lo = min(key[0], key[1]);
            key[0] = hi, key[1] = lo;
        } else if constexpr (VPL >= 4) {
            auto order = [&](int i, int j) {
                const uint32_t hi = max(key[i], key[j]), lo = min(key[i], key[j]);
                key[i] = hi, key[j] = lo;
            };
#pragma unroll
            for (int h = 0; h < VPL; h += 4) {  // sort each four (5 comparators)
                order(h, h + 1), order(h + 2, h + 3);
                order(h, h + 2), order(h + 1, h + 3);
                order(h + 1, h + 2);
            }
            if constexpr (VPL == 8) {  // odd-even merge of the two fours (9 comparators)
                order(0, 4), order(1, 5), order(2, 6), order(3, 7);
                order(2, 4), order(3, 5);
                order(1, 2), order(3, 4), order(5, 6);
            }
        }
        int mine = 0, slot = 0;  // lane r: the expert of round r, and its place in ascending order
        uint32_t w = 0;
#pragma unroll
        for (int r = 0; r < kMaxTopK; ++r) {
            if (r < p.k) {
                w = warp_max(key[0]);
                const bool pop = key[0] == w;
#pragma unroll
                for (int j = 0; j < VPL && j + r < kMaxTopK; ++j)  // what later rounds and the border can see
                    key[j] = pop ? (j + 1 < VPL ? key[j + 1] : 0u) : key[j];
                if (lane == r) mine = (int)w;
            }
        }
        mine = 255 - (mine & 255);
        if (gridded) {
            const uint32_t next = warp_max(key[0]);
            const float mag = fmaxf(fabsf(top), fabsf(top - reach));
            close = close || grid_close(w, next, reach, p.bias ? choice_error(p, rz, mag) : 0.f);
        }
        if (close) {
            if (e0 + VPL > p.E) in &= (1u << max(p.E - e0, 0)) - 1u;
            mine = choose_close<VPL, DT>(p, row, lane, m, rz, in, settle, scratch);
        }
        for (int q = 0; q < p.k; ++q) slot += __shfl_sync(kFull, mine, q) < mine;

        // weights: lane r < k has one chosen expert
        const bool has = lane < p.k;
        const float xe = has ? logit_at<DT>(row, mine) : -INFINITY;
        float s;
        if (p.score == 0) {
            if (!scored && p.renorm) {  // the sum over all experts cancels
                m = warp_max(xe);
                s = has && m != -INFINITY ? __expf(xe - m) : 0.f;
            } else {
                s = has && m != -INFINITY ? __expf(xe - m) * rz : 0.f;
            }
        } else {
            s = has ? rcp_approx(1.0f + __expf(-xe)) : 0.f;
        }
        if (p.renorm) {
            float sum = s;
#pragma unroll
            for (int o = kMaxTopK / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
            s = __fdividef(s, sum + 1e-20f);
        }
        s *= p.scale;
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
    if (p.r.hist && last_to_arrive(p.r.done, gridDim.x)) finish_scan(p.r, s_scan, kGateWarps * kScratch<VPL>);
}

template <int VPL>
static cudaError_t launch_gate_v(const GateParams& p, int dtype, int sms, cudaStream_t st) {
    const int want = (p.T + kGateWarps - 1) / kGateWarps;
    const int grid = want < kGateCtas * sms ? want : kGateCtas * sms;
    if (dtype == kDtFp32)
        return launch_pdl(gate_kernel<VPL, kDtFp32>, dim3(grid), dim3(kGateWarps * 32), 0, st, p);
    else if (dtype == kDtFp16)
        return launch_pdl(gate_kernel<VPL, kDtFp16>, dim3(grid), dim3(kGateWarps * 32), 0, st, p);
    else
        return launch_pdl(gate_kernel<VPL, kDtBf16>, dim3(grid), dim3(kGateWarps * 32), 0, st, p);
}

cudaError_t launch_gate(const GateParams& p_in, int dtype, int sms, cudaStream_t st) {
    GateParams p = p_in;
    const int vpl = p.E <= 32 ? 1 : p.E <= 64 ? 2 : p.E <= 128 ? 4 : 8;
    const size_t lane_bytes = (size_t)vpl * (dtype == kDtFp32 ? 4 : 2);
    const size_t al = lane_bytes < 16 ? lane_bytes : 16;
    p.vec = p.E % vpl == 0 && reinterpret_cast<uintptr_t>(p.logits) % al == 0 && p.ld_bytes % al == 0;
    p.gsize = p.E / p.groups;
    p.inv_gsize = (65536 + p.gsize - 1) / p.gsize;
    // groups of whole lanes, a power of two of them, stay in registers
    const int per = p.gsize / vpl;
    p.aligned = p.gsize % vpl == 0 && (per & (per - 1)) == 0 && per > 0;
    int P = 32;
    while (P * p.groups > 32) P >>= 1;
    p.lanes_per_group = p.aligned ? per : P;
    switch (vpl) {
        case 1: return launch_gate_v<1>(p, dtype, sms, st);
        case 2: return launch_gate_v<2>(p, dtype, sms, st);
        case 4: return launch_gate_v<4>(p, dtype, sms, st);
        default: return launch_gate_v<8>(p, dtype, sms, st);
    }
}

}  // namespace moe
