// Rotation of q and k by position, and k, v appended to a paged cache in the
// same pass.  The pages name the pieces: rotary positions with a YaRN scale
// ("GPT-OSS on Day 0", perplexity.ai hub blog, architecture list) and a cache
// kept heads-major, tokens contiguous ("Hosting Qwen on Blackwell").
//
//   a_i = position * inv_freq_i   (64 bits), i < rot / 2; with several axes (time,
//         height, width of images and video) the position is that of pair i's axis
//   (x_i, y_i) -> m (x_i cos a_i - y_i sin a_i, x_i sin a_i + y_i cos a_i)
//   pairs (i, i + rot/2), or neighbours (2i, 2i+1); dims past rot unchanged
//   16-bit cache: the rotated k and v, rounded once
//   e4m3 cache:   per token and head s = amax / 448 (1 if all zero), codes
//                 e4m3(value / s) of the unrounded fp32 values: the layer's
//                 1 x 128 group quantiser on a head
//
// Bound by memory: every value is read and written once.  A row (one head of
// one token) belongs to a run of lanes, 16 values each -- both halves of its
// pairs, so the rotation needs no exchange and in-place q is safe -- moved by
// two 16-byte loads and stores.  A lane has the same pairs in every row, so a
// warp computes its token's angles once, keeps them in registers and streams
// rows with kAppendBatch groups of them in flight and no barrier; small batches
// split a token's rows over more warps.
//
// 8192 tokens of 72 heads of 128 into an e4m3 cache: 54.4 us, 5.4 TB/s (80 % of a copy);
// 256 tokens of 80 heads of 64, 16-bit cache: 3.1 us, 1 token 2.1; 8192 tokens of 80 heads of
// 128 with three axes, 16-bit cache: 60.7 us, 5.5 TB/s (81 %). A CTA per token with
// its angles in shared memory took 83 us (a barrier, one round of rows in flight); 2 or
// 3 groups in flight 60 and 56; more CTAs an SM have fewer registers (58 to 84).
// Equal runs of batches over the borders of tokens gain where tokens just pass a wave
// of warps (2600 tokens 21.2 -> 18.5) and lose below one (1200 tokens 8.3 -> 9.3).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

constexpr int kAppendWarps = 4;  // per CTA
constexpr int kAppendBatch = 4;  // row groups in flight per warp

template <bool FP16>
__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (FP16) {
            const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        } else {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
template <bool FP16>
__device__ __forceinline__ uint4 pack8(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (FP16) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool FP16, bool E4M3, bool NEIGHBOURS>
__global__ void __launch_bounds__(kAppendWarps * 32) rotate_append_kernel(AppendParams p) {
    __shared__ __align__(16) float2 s_cs[kAppendWarps][128];  // m (cos, sin) of a warp's token
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long job = (long long)blockIdx.x * kAppendWarps + warp;
    const int n = (int)(job / p.parts), part = (int)(job - (long long)n * p.parts);
    pdl_wait();
    if (n >= p.N) return;
    const int rows = p.Hq + 2 * p.Hkv;
    const int lpr = 1 << p.lpr_shift;
    const int unit = lane & (lpr - 1), sub = lane >> p.lpr_shift;
    const int rpg = 32 >> p.lpr_shift;  // rows of a group
    const bool has = unit < (p.D >> 4);
    // this lane's 16 values: both halves of 8 pairs, or 16 in a row
    const bool turns = unit < (p.rot >> 4);
    const int half = p.rot >> 1;
    const int ca = NEIGHBOURS || !turns ? 16 * unit : 8 * unit;
    const int cb = NEIGHBOURS || !turns ? ca + 8 : ca + half;
    const int r_end = min(rows, (part + 1) * p.groups_per_part * rpg);
    int r0 = part * p.groups_per_part * rpg + sub;

    auto load = [&](int r, uint4& a, uint4& b) {
        if (r >= r_end || !has) return;
        const uint16_t* src = r < p.Hq           ? p.q + n * p.q_token + (long long)r * p.q_head
                              : r < p.Hq + p.Hkv ? p.k + n * p.k_token + (long long)(r - p.Hq) * p.k_head
                                                 : p.v + n * p.v_token + (long long)(r - p.Hq - p.Hkv) * p.v_head;
        a = __ldcs(reinterpret_cast<const uint4*>(src + ca));
        b = __ldcs(reinterpret_cast<const uint4*>(src + cb));
    };
    uint4 va[kAppendBatch], vb[kAppendBatch];
#pragma unroll
    for (int i = 0; i < kAppendBatch; ++i) {
        va[i] = vb[i] = make_uint4(0, 0, 0, 0);
        load(r0 + i * rpg, va[i], vb[i]);  // in flight while the angles are computed
    }
    const long long slot = p.slots[n];
    const double at_n = (double)p.positions[n];  // (axes: of axis 0)
    for (int i = lane; i < half; i += 32) {
        double pos = at_n;
        if (p.axes) {
            const int axis = __ldg(p.axes + i);
            if ((uint32_t)axis < (uint32_t)p.n_axes)
                pos = (double)__ldg(p.positions + axis * p.axis_ld + n);
            else if (p.status)
                atomicOr(p.status, kErrBadIndex);
        }
        // whole turns drop out in 64 bits: a float keeps only 2^-24 of the angle, not of its fraction
        const double turn = pos * p.inv_freq[i] * 0.15915494309189533577;
        float s, c;
        sincospif(2.0f * (float)(turn - rint(turn)), &s, &c);
        s_cs[warp][i] = make_float2(c * p.rope_scale, s * p.rope_scale);
    }
    int page = -1, off = 0;  // page -1: nothing appended
    if (slot >= 0 && slot < (long long)p.num_pages * p.page_size) {
        page = (int)((uint32_t)slot / (uint32_t)p.page_size);
        off = (int)((uint32_t)slot - (uint32_t)page * (uint32_t)p.page_size);
    } else if (slot >= 0 && p.status && lane == 0) {
        atomicOr(p.status, kErrBadIndex);
    }
    __syncwarp();
    float2 cs[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float4 v = make_float4(1.f, 0.f, 1.f, 0.f);
        if (turns) v = *reinterpret_cast<const float4*>(&s_cs[warp][8 * unit + 2 * i]);
        cs[2 * i] = make_float2(v.x, v.y);
        cs[2 * i + 1] = make_float2(v.z, v.w);
    }
    const KvCache& kv = p.cache;
    const long long k_at = page * kv.k_page + off * kv.k_token, v_at = page * kv.v_page + off * kv.v_token;
    const long long s_at = page * kv.s_page + off * kv.s_token;

    for (; r0 - sub < r_end; r0 += kAppendBatch * rpg) {
#pragma unroll
        for (int i = 0; i < kAppendBatch; ++i) {
            const int r = r0 + i * rpg;
            if (r - sub >= r_end) break;
            float x[8], y[8];
            unpack8<FP16>(va[i], x);
            unpack8<FP16>(vb[i], y);
            load(r + kAppendBatch * rpg, va[i], vb[i]);
            const bool act = r < r_end && has;
            if (turns && r < p.Hq + p.Hkv) {
                if (NEIGHBOURS) {  // 4 pairs in x, 4 in y
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 u = cs[j], w = cs[j + 4];
                        const float x0 = x[2 * j], y0 = y[2 * j];
                        x[2 * j] = x0 * u.x - x[2 * j + 1] * u.y;
                        x[2 * j + 1] = x0 * u.y + x[2 * j + 1] * u.x;
                        y[2 * j] = y0 * w.x - y[2 * j + 1] * w.y;
                        y[2 * j + 1] = y0 * w.y + y[2 * j + 1] * w.x;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float x0 = x[j];
                        x[j] = x0 * cs[j].x - y[j] * cs[j].y;
                        y[j] = x0 * cs[j].y + y[j] * cs[j].x;
                    }
                }
            }
            if (r - sub + rpg > p.Hq) {  // a group with key or value rows (the whole warp)
                float amax = 0.f;
                if (E4M3) {
                    if (act) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fmaxf(fabsf(x[j]), fabsf(y[j])));
                    }
                    for (int o = lpr >> 1; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                }
                if (act && r >= p.Hq && page >= 0) {
                    const bool is_k = r < p.Hq + p.Hkv;
                    const int h = is_k ? r - p.Hq : r - p.Hq - p.Hkv;
                    void* base = is_k ? kv.k : kv.v;
                    const long long at = is_k ? k_at + h * kv.k_head : v_at + h * kv.v_head;
                    if (E4M3) {
                        const float s = group_scale(amax), rs = recip_rn(s);
                        uint8_t* dst = static_cast<uint8_t*>(base) + at;
                        *reinterpret_cast<uint2*>(dst + ca) = make_uint2(quant4(x[0], x[1], x[2], x[3], amax, s, rs),
                                                                         quant4(x[4], x[5], x[6], x[7], amax, s, rs));
                        *reinterpret_cast<uint2*>(dst + cb) = make_uint2(quant4(y[0], y[1], y[2], y[3], amax, s, rs),
                                                                         quant4(y[4], y[5], y[6], y[7], amax, s, rs));
                        if (unit == 0) (is_k ? kv.k_scale : kv.v_scale)[s_at + h * kv.s_head] = s;
                    } else {
                        uint16_t* dst = static_cast<uint16_t*>(base) + at;
                        *reinterpret_cast<uint4*>(dst + ca) = pack8<FP16>(x);
                        *reinterpret_cast<uint4*>(dst + cb) = pack8<FP16>(y);
                    }
                }
            }
            if (act && r < p.Hq) {
                uint16_t* dst = p.q_out + n * p.o_token + (long long)r * p.o_head;
                *reinterpret_cast<uint4*>(dst + ca) = pack8<FP16>(x);
                *reinterpret_cast<uint4*>(dst + cb) = pack8<FP16>(y);
            }
        }
    }
}

template <bool FP16, bool E4M3>
static cudaError_t launch_append_t(const AppendParams& p, int grid, cudaStream_t st) {
    const dim3 g(grid), b(kAppendWarps * 32);
    return p.neighbours ? launch_pdl(rotate_append_kernel<FP16, E4M3, true>, g, b, 0, st, p)
                        : launch_pdl(rotate_append_kernel<FP16, E4M3, false>, g, b, 0, st, p);
}

cudaError_t launch_rotate_append(const AppendParams& p_in, bool fp16, bool e4m3, int sms, cudaStream_t st) {
    AppendParams p = p_in;
    const int rows = p.Hq + 2 * p.Hkv;
    p.lpr_shift = 0;
    while ((16 << p.lpr_shift) < p.D) ++p.lpr_shift;
    // one warp a token where that gives every SM 8 of them, else its rows are split (each part
    // computes the angles again): 256 tokens of 80 rows take 3.4 us with 8 warps an SM, 4.7 with
    // 24; 777 of 28 rows 4.3, 4.8 with 4 and 6.1 with 24
    const int rpg = 32 >> p.lpr_shift, groups = (rows + rpg - 1) / rpg;
    const long long even = (8LL * sms + p.N - 1) / p.N;  // (N may be close to 2^31)
    const int parts = even < groups ? (int)even : groups;
    p.groups_per_part = (groups + parts - 1) / parts;
    p.parts = (groups + p.groups_per_part - 1) / p.groups_per_part;
    const int grid = (int)(((long long)p.N * p.parts + kAppendWarps - 1) / kAppendWarps);
    if (fp16) return e4m3 ? launch_append_t<true, true>(p, grid, st) : launch_append_t<true, false>(p, grid, st);
    return e4m3 ? launch_append_t<false, true>(p, grid, st) : launch_append_t<false, false>(p, grid, st);
}

}  // namespace moe
