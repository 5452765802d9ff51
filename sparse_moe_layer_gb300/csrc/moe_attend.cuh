// What the attention kernels over a paged cache share: asynchronous copies, 16-bit
// packing, the bounds of the running sums, and the end of a softmax row.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_device.cuh"

namespace moe {

constexpr uint32_t kAllLanes = 0xffffffffu;
enum : int { kKvBf16 = 0, kKvFp16 = 1, kKvE4m3 = 2 };

// 16-bit caches: powers of two that a score may stand above the maximum that its row's sums
// are about, and that these lie below that maximum: fp16 probabilities start at 2^7, reach
// 2^15, and keep their 11 bits down to 2^-21 of the largest (without it a flat tail of
// probabilities below 2^-25 was lost, however long).
constexpr float kSlack = 8.f;
template <int KV>
constexpr float kLift = KV == kKvFp16 ? 7.f : 0.f;
// e4m3: a weight is probability times value scale, and the row's sums and accumulators are
// about a power of two that makes the largest weight so far at least 2^kNewWeight when it is
// set (but kMostLift powers of two below the scores' maximum at most, where all weights are
// tiny). While a tile's largest probability times its largest scale, as they stand to that,
// is at most 2^kMostWeight the weights fit fp16; else they are looked at and it is set again.
constexpr float kNewWeight = 5.f, kMostLift = 104.f, kMostWeight = 15.f;
constexpr float kLeastScale = 0x1p-89f;  // 2^(kMostWeight - kMostLift): the sums' room where scales are smaller
constexpr float kNoWeights = -0x1p127f;  // the power of two before a row's first

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16z(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async4z(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Two e4m3 codes (low half of v) -> two fp16 values, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
    return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
    if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&v));
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// a = a f + b h
__device__ __forceinline__ void add_scaled(float4& a, float f, const float4& b, float h) {
    a.x = a.x * f + b.x * h;
    a.y = a.y * f + b.y * h;
    a.z = a.z * f + b.z * h;
    a.w = a.w * f + b.w * h;
}

// 1 / (sum with the head's sink, where there is one), about the larger of the two exponents: what
// sums taken about m are multiplied by.  0 for a row without tokens; NaN stays NaN.
__device__ __forceinline__ float final_weight(bool sinks, float sink, float m, float l) {
    float w = 1.f;
    if (sinks) {
        const float k = sink * 1.4426950408889634f;
        const float n = fmaxf(m, k);
        w = n == -INFINITY ? 0.f : ex2_approx(m - n);
        l = n == -INFINITY ? 0.f : l * w + (k == n ? 1.f : ex2_approx(k - n));  // (an infinite sink too)
    }
    return l == 0.f ? 0.f : w / l;
}
__device__ __forceinline__ float final_weight(const float* sinks, int head, float m, float l) {
    return final_weight(sinks != nullptr, sinks ? __ldg(sinks + head) : 0.f, m, l);
}

}  // namespace moe
