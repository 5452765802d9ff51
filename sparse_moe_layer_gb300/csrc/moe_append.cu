// Rotation of q and k by position, and k, v appended to a paged cache in the
// same pass.  The pages name the pieces: rotary positions with a YaRN scale
// ("GPT-OSS on Day 0", perplexity.ai hub blog, architecture list) and a cache
// kept heads-major, tokens contiguous ("Hosting Qwen on Blackwell").
//
//   a_i = position * inv_freq_i   (64 bits), i < rot / 2
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
// two 16-byte loads and stores.  The angles of a token are computed once by
// its CTA.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

constexpr int kAppendMaxTokens = 8;  // tokens per CTA

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
__global__ void __launch_bounds__(512) rotate_append_kernel(AppendParams p) {
    extern __shared__ float2 s_cs[];  // [tokens][rot / 2] m (cos, sin)
    __shared__ int s_page[kAppendMaxTokens], s_off[kAppendMaxTokens];  // page -1: nothing appended
    const int n0 = blockIdx.x * p.tokens_per_cta;
    const int nt = min(p.tokens_per_cta, p.N - n0);
    const int half = p.rot >> 1;
    const int rows = p.Hq + 2 * p.Hkv;
    const int lpr = 1 << p.lpr_shift;
    const int unit = threadIdx.x & (lpr - 1);
    const bool has = unit < (p.D >> 4);
    // this lane's 16 values: both halves of 8 pairs, or 16 in a row
    const int turned = p.rot >> 4;  // units that rotate
    const bool turns = unit < turned;
    const int ca = NEIGHBOURS || !turns ? 16 * unit : 8 * unit;
    const int cb = NEIGHBOURS || !turns ? ca + 8 : ca + half;
    const int step = blockDim.x >> p.lpr_shift;
    const int items = nt * rows;
    const int rounds = (items + step - 1) / step;

    // the values of one row
    auto load = [&](int item, uint4& a, uint4& b) {
        if (item >= items || !has) return;
        const int tt = item / rows, r = item - tt * rows;
        const long long n = n0 + tt;
        const uint16_t* src = r < p.Hq             ? p.q + n * p.q_token + (long long)r * p.q_head
                              : r < p.Hq + p.Hkv   ? p.k + n * p.k_token + (long long)(r - p.Hq) * p.k_head
                                                   : p.v + n * p.v_token + (long long)(r - p.Hq - p.Hkv) * p.v_head;
        a = __ldcs(reinterpret_cast<const uint4*>(src + ca));
        b = __ldcs(reinterpret_cast<const uint4*>(src + cb));
    };
    uint4 va = make_uint4(0, 0, 0, 0), vb = va;
    int item = threadIdx.x >> p.lpr_shift;
    load(item, va, vb);  // in flight while the angles are computed

    for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
        const int tt = i / half;
        // whole turns drop out in 64 bits: a float keeps only 2^-24 of the angle, not of its fraction
        const double turn = (double)p.positions[n0 + tt] * p.inv_freq[i - tt * half] * 0.15915494309189533577;
        float s, c;
        sincospif(2.0f * (float)(turn - rint(turn)), &s, &c);
        s_cs[i] = make_float2(c * p.rope_scale, s * p.rope_scale);
    }
    if (threadIdx.x < nt) {
        const long long slot = p.slots[n0 + threadIdx.x];
        int page = -1, off = 0;
        if (slot >= 0 && slot < (long long)p.num_pages * p.page_size) {
            page = (int)((uint32_t)slot / (uint32_t)p.page_size);
            off = (int)((uint32_t)slot - (uint32_t)page * (uint32_t)p.page_size);
        } else if (slot >= 0 && p.status) {
            atomicOr(p.status, kErrBadIndex);
        }
        s_page[threadIdx.x] = page;
        s_off[threadIdx.x] = off;
    }
    __syncthreads();

    for (int round = 0; round < rounds; ++round, item += step) {
        uint4 na = va, nb = vb;
        if (round + 1 < rounds) load(item + step, na, nb);
        const int tt = item < items ? item / rows : 0, r = item - tt * rows;
        const bool act = item < items && has;
        float x[8], y[8];
        unpack8<FP16>(va, x);
        unpack8<FP16>(vb, y);
        if (act && turns && r < p.Hq + p.Hkv) {
            const float2* cs = s_cs + tt * half + 8 * unit;
            if (NEIGHBOURS) {  // 4 pairs in x, 4 in y
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 u = cs[i], w = cs[i + 4];
                    const float x0 = x[2 * i], y0 = y[2 * i];
                    x[2 * i] = x0 * u.x - x[2 * i + 1] * u.y;
                    x[2 * i + 1] = x0 * u.y + x[2 * i + 1] * u.x;
                    y[2 * i] = y0 * w.x - y[2 * i + 1] * w.y;
                    y[2 * i + 1] = y0 * w.y + y[2 * i + 1] * w.x;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 u = cs[i];
                    const float x0 = x[i];
                    x[i] = x0 * u.x - y[i] * u.y;
                    y[i] = x0 * u.y + y[i] * u.x;
                }
            }
        }
        float amax = 0.f;
        if (E4M3) {
            if (act) {
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(x[i]), fabsf(y[i])));
            }
            for (int o = lpr >> 1; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        }
        if (act) {
            if (r < p.Hq) {
                uint16_t* dst = p.q_out + (n0 + tt) * p.o_token + (long long)r * p.o_head;
                *reinterpret_cast<uint4*>(dst + ca) = pack8<FP16>(x);
                *reinterpret_cast<uint4*>(dst + cb) = pack8<FP16>(y);
            } else if (s_page[tt] >= 0) {
                const bool is_k = r < p.Hq + p.Hkv;
                const int h = is_k ? r - p.Hq : r - p.Hq - p.Hkv;
                const KvCache& kv = p.cache;
                void* base = is_k ? kv.k : kv.v;
                const long long at = is_k ? s_page[tt] * kv.k_page + h * kv.k_head + s_off[tt] * kv.k_token
                                          : s_page[tt] * kv.v_page + h * kv.v_head + s_off[tt] * kv.v_token;
                if (E4M3) {
                    const float s = group_scale(amax), rs = recip_rn(s);
                    uint8_t* dst = static_cast<uint8_t*>(base) + at;
                    *reinterpret_cast<uint2*>(dst + ca) =
                        make_uint2(quant4(x[0], x[1], x[2], x[3], amax, s, rs), quant4(x[4], x[5], x[6], x[7], amax, s, rs));
                    *reinterpret_cast<uint2*>(dst + cb) =
                        make_uint2(quant4(y[0], y[1], y[2], y[3], amax, s, rs), quant4(y[4], y[5], y[6], y[7], amax, s, rs));
                    if (unit == 0) {
                        float* sc = is_k ? kv.k_scale : kv.v_scale;
                        sc[s_page[tt] * kv.s_page + h * kv.s_head + s_off[tt] * kv.s_token] = s;
                    }
                } else {
                    uint16_t* dst = static_cast<uint16_t*>(base) + at;
                    *reinterpret_cast<uint4*>(dst + ca) = pack8<FP16>(x);
                    *reinterpret_cast<uint4*>(dst + cb) = pack8<FP16>(y);
                }
            }
        }
        va = na;
        vb = nb;
    }
}

template <bool FP16, bool E4M3>
static void launch_append_t(const AppendParams& p, int grid, int block, size_t smem, cudaStream_t st) {
    if (p.neighbours)
        rotate_append_kernel<FP16, E4M3, true><<<grid, block, smem, st>>>(p);
    else
        rotate_append_kernel<FP16, E4M3, false><<<grid, block, smem, st>>>(p);
}

cudaError_t launch_rotate_append(const AppendParams& p_in, bool fp16, bool e4m3, int sms, cudaStream_t st) {
    AppendParams p = p_in;
    const int rows = p.Hq + 2 * p.Hkv;
    p.lpr_shift = 0;
    while ((16 << p.lpr_shift) < p.D) ++p.lpr_shift;
    // several tokens to a CTA where one would leave most of 256 threads idle and there are
    // tokens enough for two CTAs on every SM anyway
    int tpc = 256 / (rows << p.lpr_shift);
    tpc = tpc < 1 ? 1 : (tpc > kAppendMaxTokens ? kAppendMaxTokens : tpc);
    if ((long long)p.N < 2LL * sms * tpc) tpc = p.N / (2 * sms) > 1 ? p.N / (2 * sms) : 1;
    p.tokens_per_cta = tpc;
    // as many threads as values, in equal rounds of at most 512
    const long long lanes = (long long)tpc * rows << p.lpr_shift;
    const long long rounds = (lanes + 511) / 512;
    const int block = (int)(((lanes + rounds - 1) / rounds + 31) / 32 * 32);
    const int grid = (p.N + tpc - 1) / tpc;
    const size_t smem = (size_t)tpc * (p.rot / 2) * sizeof(float2);
    if (fp16)
        e4m3 ? launch_append_t<true, true>(p, grid, block, smem, st) : launch_append_t<true, false>(p, grid, block, smem, st);
    else
        e4m3 ? launch_append_t<false, true>(p, grid, block, smem, st)
             : launch_append_t<false, false>(p, grid, block, smem, st);
    return cudaGetLastError();
}

}  // namespace moe
