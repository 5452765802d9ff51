// Attention of one new token per sequence over a paged key-value cache, with
// grouped query heads, an optional sink logit per head and an optional sliding
// window ("GPT-OSS on Day 0", perplexity.ai hub blog: GQA, sink attention --
// the sink enters the softmax sum once per row -- and alternating windows).
//
//   o = sum_t p_t v_t / (sum_t p_t + 2^(sink log2 e - m)),  p_t = 2^(s_t - m),
//   s_t = (q . k_t) scale log2 e,  t over the last `window` of `length` tokens
//
// Bound by the cache's bytes: each key and value is read once, for all (up to
// 16) query heads that share it, so the products need G flops a byte (8 to 16,
// above what the fp32 pipes give at full bandwidth, far below the matrix
// instructions): m16n8k16 with the group's heads as the 16 rows, scores and
// probabilities staying in registers between the two products.  A 64- or
// 128-row tcgen05 tile would be 4 to 16 times padding here and hand the scores
// through tensor memory.
//
// Every warp works alone: the (sequence, key head, token tile) list is cut into
// equal runs, one per resident warp, so a batch of very different lengths loads
// all SMs alike; a warp streams its tiles through its own cp.async ring with
// running maximum and sum, and only a row cut by a run's border leaves fp32
// partials, which a second, dependent launch joins in a fixed order (results
// do not depend on scheduling).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr uint32_t kAllLanes = 0xffffffffu;
constexpr int kAttWarps = 4;  // warps per CTA
constexpr int kAttRows = 16;  // query heads per row (m16 of the products)
enum : int { kKvBf16 = 0, kKvFp16 = 1, kKvE4m3 = 2 };

template <int DP, int KV>
struct AttCfg {
    static constexpr int ES = KV == kKvE4m3 ? 1 : 2;       // bytes of a cached value
    static constexpr int TT = KV == kKvE4m3 || DP == 64 ? 32 : 16;  // tokens per tile
    static constexpr int ROW = DP * ES;                    // bytes of a token's row in shared memory
    static constexpr int CH = ROW / 16;                    // its 16-byte chunks
    static constexpr int STAGES = DP == 64 && KV == kKvE4m3 ? 4 : DP == 256 && KV == kKvE4m3 ? 2 : 3;
    static constexpr int TILE = TT * ROW;                  // bytes of a K (or V) tile
    static constexpr int SC = KV == kKvE4m3 ? 2 * TT * 4 : 0;
    static constexpr int STAGE = 2 * TILE + SC + 16;       // + meta
    static constexpr int QS = DP == 256 ? DP / 16 * 512 : 0;  // Q fragments, where registers do not hold them
    static constexpr int WARP = (STAGES * STAGE + QS + 127) / 128 * 128;
    static constexpr int SMEM = kAttWarps * WARP;
    static constexpr int CTAS = DP == 64 && KV == kKvE4m3 ? 3 : DP == 256 ? 1 : 2;  // resident per SM
};

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
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Byte of chunk c (16 bytes) of token row r in a tile: 8 rows of one chunk
// column fall on 8 different bank groups, for the loads and for ldmatrix.
template <int CH>
__device__ __forceinline__ uint32_t swz(int r, int c) {
    if (CH >= 8) return (uint32_t)(r * CH + ((c & ~7) | ((c ^ r) & 7))) * 16u;
    return (uint32_t)(r * CH + (c ^ ((r >> 1) & 3))) * 16u;  // CH == 4: two rows per 128 bytes
}

__device__ __forceinline__ int seen_tokens(const AttendParams& p, int b, int* start) {
    const int raw = __ldg(p.lengths + b);
    const int len = min(max(raw, 0), p.max_tokens);
    if (len != raw && p.status) atomicOr(p.status, kErrBadIndex);
    *start = p.window > 0 && len > p.window ? len - p.window : 0;
    return len;
}

// Tiles of a row: tokens [tile0, tile0 + TT) and on, tile0 = start rounded down
// to TT, so that a tile's groups of 16 tokens never straddle a page of 16 n.
template <int TT>
__device__ __forceinline__ int tiles_of(int start, int len) {
    return max(1, (len + TT - 1) / TT - start / TT);
}

// Where a warp stands in the list of tiles: sequence b, row h of it (key head
// and block of 16 query heads), tile of the row.  step: tiles apart (a team's
// warps take a row's tiles in turn).
template <int TT>
struct TileIt {
    int b, h, tile, ntiles, start, len;
    __device__ __forceinline__ void seq(const AttendParams& p) {
        len = seen_tokens(p, b, &start);
        ntiles = tiles_of<TT>(start, len);
    }
    __device__ __forceinline__ void next(const AttendParams& p, int step) {
        tile += step;
        if (tile < ntiles) return;
        tile = 0;
        if (++h < p.rows_per_seq) return;
        h = 0;
        if (++b < p.B) seq(p);
    }
};

// 1 / (sum with the head's sink), about the larger of the two exponents: what
// sums taken about m are multiplied by.  0 for a row without tokens.
__device__ __forceinline__ float final_weight(const AttendParams& p, int head, float m, float l) {
    float w = 1.f;
    if (p.sinks) {
        const float k = __ldg(p.sinks + head) * 1.4426950408889634f;
        const float n = fmaxf(m, k);
        w = n == -INFINITY ? 0.f : ex2_approx(m - n);
        l = n == -INFINITY ? 0.f : l * w + ex2_approx(k - n);
    }
    return l > 0.f ? w / l : 0.f;
}

}  // namespace

template <int DP, int KV, bool QF16>
__global__ void __launch_bounds__(kAttWarps * 32, AttCfg<DP, KV>::CTAS) attend_kernel(AttendParams p) {
    using C = AttCfg<DP, KV>;
    constexpr bool F16 = KV != kKvBf16;  // type of the products
    constexpr int TT = C::TT, NT = TT / 8, KT = TT / 16, KS = DP / 16, S = C::STAGES;
    constexpr uint32_t kAllTokens = TT == 32 ? 0xffffffffu : 0xffffu;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_pre[kAttWarps * 32 + 1];
    __shared__ int s_wsum[kAttWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    const int nwarps = gridDim.x * kAttWarps;
    const int gw = warp * gridDim.x + blockIdx.x;  // neighbouring runs on different SMs
    pdl_allow_dependents();

    // --- this warp's run of the tile list ---
    TileIt<TT> it;
    int left;  // tiles of the run
    int step = 1;
    if (p.team) {
        // few rows, none long: a CTA per row, its warps take the tiles in turn
        it.b = blockIdx.x / p.rows_per_seq;
        it.h = blockIdx.x - it.b * p.rows_per_seq;
        it.seq(p);
        it.tile = warp;
        step = kAttWarps;
        left = it.ntiles > warp ? (it.ntiles - warp + kAttWarps - 1) / kAttWarps : 0;
    } else if (p.by_row) {  // whole rows
        const int rows = p.B * p.rows_per_seq, n = rows < nwarps ? rows : nwarps;
        if (gw >= n) return;
        const int u0 = (int)((long long)rows * gw / n), u1 = (int)((long long)rows * (gw + 1) / n);
        it.b = u0 / p.rows_per_seq;
        it.h = u0 - it.b * p.rows_per_seq;
        it.seq(p);
        it.tile = 0;
        left = 0;
        TileIt<TT> t = it;
        for (int r = u1 - u0; r > 0; --r) {
            left += t.ntiles;
            t.tile = t.ntiles - 1;
            t.next(p, 1);
        }
    } else {
        // each thread sums the tiles of a slice of the sequences (rows_per_seq rows each)
        const int slice = (p.B + kAttWarps * 32 - 1) / (kAttWarps * 32);
        int mine = 0;
        for (int i = 0; i < slice; ++i) {
            const int b = tid * slice + i;
            if (b < p.B) {
                int st;
                const int len = seen_tokens(p, b, &st);
                mine += tiles_of<TT>(st, len);
            }
        }
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kAllLanes, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) s_wsum[warp] = inc;
        __syncthreads();
        int before = 0;
#pragma unroll
        for (int w = 0; w < kAttWarps; ++w)
            if (w < warp) before += s_wsum[w];
        s_pre[tid + 1] = before + inc;
        if (tid == 0) s_pre[0] = 0;
        __syncthreads();
        const long long total = (long long)s_pre[kAttWarps * 32] * p.rows_per_seq;
        const long long want = (total + p.min_units - 1) / p.min_units;
        const int n = (int)(want < nwarps ? want : nwarps);
        if (gw >= n) {
            if (lane == 0) p.cont[gw] = -1;
            return;
        }
        const long long u0 = total * gw / n, u1 = total * (gw + 1) / n;
        // the slice, then the sequence, that holds u0
        int sl = 0;
        for (int base = 0; base < kAttWarps * 32; base += 32) {
            const bool past = (long long)s_pre[base + lane + 1] * p.rows_per_seq <= u0;
            sl += __popc(__ballot_sync(kAllLanes, past));
        }
        long long u = u0 - (long long)s_pre[sl] * p.rows_per_seq;
        it.b = sl * slice;
        while (true) {
            it.seq(p);
            const long long here = (long long)it.ntiles * p.rows_per_seq;
            if (u < here) break;
            u -= here;
            ++it.b;
        }
        it.h = (int)(u / it.ntiles);
        it.tile = (int)(u - (long long)it.h * it.ntiles);
        left = (int)(u1 - u0);
        if (lane == 0) p.cont[gw] = it.tile ? it.b * p.rows_per_seq + it.h : -1;
    }

    // --- the ring ---
    uint8_t* ring = smem + warp * C::WARP;
    const uint32_t ring_s = smem_u32(ring);
    constexpr int RPS = 32 / (C::CH < 32 ? C::CH : 32);  // token rows per step of the warp
    const int ch = lane % C::CH, r0 = lane / C::CH;
    const bool in = ch * (16 / C::ES) < p.D;
    // byte offsets of the lane's chunk in a group of 16 tokens, and of a step
    const long long k_lane = (long long)r0 * p.cache.k_token * C::ES + ch * 16, k_step = RPS * p.cache.k_token * C::ES;
    const long long v_lane = (long long)r0 * p.cache.v_token * C::ES + ch * 16, v_step = RPS * p.cache.v_token * C::ES;
    // tile `it`: tokens of the lanes and their pages, fetched one tile ahead of the copies
    int f_pid = -1, f_off = 0;
    bool f_ok = false;
    auto fetch = [&]() {
        const int tok = (it.start / TT + it.tile) * TT + (lane & (TT - 1));
        f_pid = -1;
        if (tok < it.len) {
            const int pi = p.page_shift >= 0 ? tok >> p.page_shift : tok / p.page_size;
            f_off = tok - pi * p.page_size;
            // a token before the window shares its group's page; with smaller pages it is not looked up
            if (tok >= it.start || p.page16) f_pid = __ldg(p.table + (long long)it.b * p.table_ld + pi);
        }
        f_ok = tok >= it.start && tok < it.len;
    };
    auto issue = [&](int slot) {
        const uint32_t dst = ring_s + slot * C::STAGE;
        const int kvh = p.head_blocks == 1 ? it.h : it.h / p.head_blocks;
        if ((uint32_t)f_pid >= (uint32_t)p.num_pages) {
            if (f_ok && p.status) atomicOr(p.status, kErrBadIndex);
            f_pid = 0;
            f_ok = false;
        }
        const uint32_t mask = __ballot_sync(kAllLanes, f_ok);
        const uint8_t* kb = static_cast<const uint8_t*>(p.cache.k) + (long long)kvh * p.cache.k_head * C::ES;
        const uint8_t* vb = static_cast<const uint8_t*>(p.cache.v) + (long long)kvh * p.cache.v_head * C::ES;
        if (p.page16) {  // a group of 16 tokens lies on one page
#pragma unroll
            for (int hh = 0; hh < KT; ++hh) {
                const long long pid = __shfl_sync(kAllLanes, f_pid, hh * 16), off = __shfl_sync(kAllLanes, f_off, hh * 16);
                const uint8_t* ks = kb + (pid * p.cache.k_page + off * p.cache.k_token) * C::ES + k_lane;
                const uint8_t* vs = vb + (pid * p.cache.v_page + off * p.cache.v_token) * C::ES + v_lane;
                if (((mask >> (16 * hh)) & 0xffffu) == 0xffffu) {
                    if (in) {
#pragma unroll
                        for (int i = 0; i < 16 / RPS; ++i) {
                            const uint32_t at = dst + swz<C::CH>(16 * hh + r0 + i * RPS, ch);
                            cp_async16(at, ks + i * k_step);
                            cp_async16(at + C::TILE, vs + i * v_step);
                        }
                    }
                } else if (in) {
#pragma unroll
                    for (int i = 0; i < 16 / RPS; ++i) {
                        const int r = 16 * hh + r0 + i * RPS;
                        const uint32_t at = dst + swz<C::CH>(r, ch);
                        const bool ok = (mask >> r) & 1u;
                        cp_async16z(at, ok ? ks + i * k_step : kb, ok);
                        cp_async16z(at + C::TILE, ok ? vs + i * v_step : vb, ok);
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < TT / RPS; ++i) {
                const int r = r0 + i * RPS;
                const long long pid = __shfl_sync(kAllLanes, f_pid, r), off = __shfl_sync(kAllLanes, f_off, r);
                const bool ok = (mask >> r) & 1u;
                const uint32_t at = dst + swz<C::CH>(r, ch);
                if (in) {
                    cp_async16z(at, ok ? kb + (pid * p.cache.k_page + off * p.cache.k_token) * C::ES + ch * 16 : kb, ok);
                    cp_async16z(at + C::TILE, ok ? vb + (pid * p.cache.v_page + off * p.cache.v_token) * C::ES + ch * 16 : vb, ok);
                }
            }
        }
        if constexpr (KV == kKvE4m3) {  // lane = token (TT == 32)
            const long long at =
                f_ok ? f_pid * p.cache.s_page + kvh * p.cache.s_head + f_off * p.cache.s_token : 0;
            cp_async4z(dst + 2 * C::TILE + lane * 4, p.cache.k_scale + at, f_ok);
            cp_async4z(dst + 2 * C::TILE + TT * 4 + lane * 4, p.cache.v_scale + at, f_ok);
        }
        if (lane == 0) {
            // b, h, valid tokens, flags: 1 first tile of its row, 2 last tile of its row
            int4 m;
            m.x = it.b;
            m.y = it.h;
            m.z = (int)(mask & kAllTokens);
            m.w = (it.tile == 0 ? 1 : 0) | (it.tile == it.ntiles - 1 ? 2 : 0);
            *reinterpret_cast<int4*>(ring + slot * C::STAGE + 2 * C::TILE + C::SC) = m;
        }
    };
    // dims past D (D < DP) are products of zeros: no branch in the tile loop
    if (p.D < DP)
        for (int i = lane * 16; i < S * C::STAGE; i += 32 * 16) *reinterpret_cast<uint4*>(ring + i) = make_uint4(0, 0, 0, 0);
    __syncwarp();
    int to_issue = left;
    if (left > 0) fetch();
    auto issue_next = [&](int slot) {
        if (to_issue > 0) {
            issue(slot);
            if (--to_issue > 0) {
                it.next(p, step);
                fetch();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int row_b = it.b, row_h = it.h;  // a team's row
#pragma unroll
    for (int s = 0; s < S - 1; ++s) issue_next(s);

    float o[DP / 8][4];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // rows g and g + 8
    float qf0 = p.scale_log2, qf1 = p.scale_log2;              // times the query row's power of two (e4m3)
    float vref = 0x1p-100f;                                    // e4m3: the accumulator's value scale
    uint32_t qr[DP <= 128 ? KS : 1][4];
    uint32_t* qs = reinterpret_cast<uint32_t*>(ring + S * C::STAGE);
    auto qfrag = [&](int k, uint32_t (&a)[4]) {
        if constexpr (DP <= 128) {
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] = qr[k][j];
        } else {
            const uint4 v = *reinterpret_cast<const uint4*>(qs + (k * 32 + lane) * 4);
            a[0] = v.x, a[1] = v.y, a[2] = v.z, a[3] = v.w;
        }
    };
    auto set_qfrag = [&](int k, const uint32_t (&a)[4]) {
        if constexpr (DP <= 128) {
#pragma unroll
            for (int j = 0; j < 4; ++j) qr[k][j] = a[j];
        } else {
            *reinterpret_cast<uint4*>(qs + (k * 32 + lane) * 4) = make_uint4(a[0], a[1], a[2], a[3]);
        }
    };
    // the queries of a row as A fragments, as they are in memory
    auto load_q = [&](int b, int h) {
        const int kvh = p.head_blocks == 1 ? h : h / p.head_blocks, hb = h - kvh * p.head_blocks;
        const int heads = min(kAttRows, p.group - hb * kAttRows);
        const uint16_t* q0 = p.q + b * p.q_token + (long long)(kvh * p.group + hb * kAttRows + g) * p.q_head;
        const uint16_t* q1 = q0 + 8 * p.q_head;
        const bool h0 = g < heads, h1 = g + 8 < heads;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            uint32_t a[4] = {0u, 0u, 0u, 0u};
            if (k * 16 < p.D) {
                // columns 2c, 2c+1 and 2c+8, 2c+9 of the k16 step; for e4m3 keys a lane has
                // dims 4c..4c+3 of both operands instead (any order of the dims will do)
                const int ca = k * 16 + (KV == kKvE4m3 ? 4 * c : 2 * c), cb = ca + (KV == kKvE4m3 ? 2 : 8);
                if (h0) {
                    a[0] = *reinterpret_cast<const uint32_t*>(q0 + ca);
                    a[2] = *reinterpret_cast<const uint32_t*>(q0 + cb);
                }
                if (h1) {
                    a[1] = *reinterpret_cast<const uint32_t*>(q1 + ca);
                    a[3] = *reinterpret_cast<const uint32_t*>(q1 + cb);
                }
            }
            set_qfrag(k, a);
        }
    };
    auto meta_at = [&](int slot) { return *reinterpret_cast<const int4*>(ring + slot * C::STAGE + 2 * C::TILE + C::SC); };
    __syncwarp();
    if (left > 0) load_q(row_b, row_h);  // in flight with the first tiles
#pragma unroll
    for (int d = 0; d < DP / 8; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[d][j] = 0.f;
    bool fresh = true, whole = true;
    int slot = 0, fill = S - 1;
    for (int i = 0; i < left; ++i) {
        cp_async_wait<S - 2>();
        __syncwarp();
        issue_next(fill);
        fill = fill + 1 == S ? 0 : fill + 1;
        const uint8_t* stage = ring + slot * C::STAGE;
        const uint32_t ks_s = ring_s + slot * C::STAGE, vs_s = ks_s + C::TILE;
        const int4 meta = meta_at(slot);
        if (fresh) {  // a new row
            fresh = false;
            whole = (meta.w & 1) != 0;
            if constexpr (KV == kKvE4m3) {
                // the products run in fp16: each query row is scaled by a power of two to
                // below 2 (exact but for values 2^-24 below the largest)
                float a0 = 0.f, a1 = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t a[4];
                    qfrag(k, a);
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        const float2 x = unpack2<QF16>(a[j]), y = unpack2<QF16>(a[j + 1]);
                        a0 = fmaxf(a0, fmaxf(fabsf(x.x), fabsf(x.y)));
                        a1 = fmaxf(a1, fmaxf(fabsf(y.x), fabsf(y.y)));
                    }
                }
                a0 = fmaxf(a0, __shfl_xor_sync(kAllLanes, a0, 1));
                a0 = fmaxf(a0, __shfl_xor_sync(kAllLanes, a0, 2));
                a1 = fmaxf(a1, __shfl_xor_sync(kAllLanes, a1, 1));
                a1 = fmaxf(a1, __shfl_xor_sync(kAllLanes, a1, 2));
                // 2^-floor(log2 amax), exponent field kept within [1, 253]
                const uint32_t e0 = min(max(__float_as_uint(a0) >> 23, 1u), 253u);
                const uint32_t e1 = min(max(__float_as_uint(a1) >> 23, 1u), 253u);
                const float f0 = __uint_as_float((254u - e0) << 23), f1 = __uint_as_float((254u - e1) << 23);
                qf0 = p.scale_log2 * __uint_as_float(e0 << 23);
                qf1 = p.scale_log2 * __uint_as_float(e1 << 23);
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t a[4];
                    qfrag(k, a);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 x = unpack2<QF16>(a[j]);
                        const float f = j & 1 ? f1 : f0;
                        a[j] = pack2<true>(x.x * f, x.y * f);
                    }
                    set_qfrag(k, a);
                }
            }
        }

        // --- scores of the tile: S[16 heads, TT tokens] ---
        float s[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[t][j] = 0.f;
        if constexpr (KV != kKvE4m3) {
            // matrices of a load: tokens 0-7 and 8-15, dims 0-7 and 8-15 of the step
            const int r = (lane & 7) + ((lane >> 4) << 3), hi = (lane >> 3) & 1;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t a[4];
                qfrag(k, a);
#pragma unroll
                for (int t = 0; t < KT; ++t) {
                    uint32_t b[4];
                    ldsm4(ks_s + swz<C::CH>(16 * t + r, 2 * k + hi), b);
                    mma16816<F16>(s[2 * t], a, b[0], b[1]);
                    mma16816<F16>(s[2 * t + 1], a, b[2], b[3]);
                }
            }
        } else {
            // a matrix: 8 tokens x 16 dims of codes; a load takes 4 groups of 8 tokens
            const int r = lane;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t a[4], b[4];
                qfrag(k, a);
                ldsm4(ks_s + swz<C::CH>(r, k), b);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    mma16816<F16>(s[t], a, e4m3x2_to_f16x2(b[t]), e4m3x2_to_f16x2(b[t] >> 16));
            }
        }
        // --- scale, mask, running maximum ---
        float vr[NT][2];  // e4m3: value scale of the lane's tokens over the accumulator's
        float vmax = 0.f;
        if constexpr (KV == kKvE4m3) {
            const float* sck = reinterpret_cast<const float*>(stage + 2 * C::TILE);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float2 kk = *reinterpret_cast<const float2*>(sck + t * 8 + 2 * c);
                const float2 vv = *reinterpret_cast<const float2*>(sck + TT + t * 8 + 2 * c);
                s[t][0] *= kk.x * qf0;
                s[t][1] *= kk.y * qf0;
                s[t][2] *= kk.x * qf1;
                s[t][3] *= kk.y * qf1;
                vr[t][0] = vv.x;
                vr[t][1] = vv.y;
                vmax = fmaxf(vmax, fmaxf(vv.x, vv.y));
            }
        } else {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[t][j] *= p.scale_log2;
        }
        const uint32_t valid = (uint32_t)meta.z;
        if (valid != kAllTokens) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (!((valid >> (t * 8 + 2 * c + (j & 1))) & 1u)) s[t][j] = -INFINITY;
        }
        float t0 = m0, t1 = m1;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            t0 = fmaxf(t0, fmaxf(s[t][0], s[t][1]));
            t1 = fmaxf(t1, fmaxf(s[t][2], s[t][3]));
        }
        t0 = fmaxf(t0, __shfl_xor_sync(kAllLanes, t0, 1));
        t1 = fmaxf(t1, __shfl_xor_sync(kAllLanes, t1, 1));
        t0 = fmaxf(t0, __shfl_xor_sync(kAllLanes, t0, 2));
        t1 = fmaxf(t1, __shfl_xor_sync(kAllLanes, t1, 2));
        float vnew = vref;
        if constexpr (KV == kKvE4m3) {
            vmax = fmaxf(vmax, __shfl_xor_sync(kAllLanes, vmax, 1));
            vmax = fmaxf(vmax, __shfl_xor_sync(kAllLanes, vmax, 2));
            vnew = fmaxf(vref, vmax);
        }
        const float b0 = t0 == -INFINITY ? 0.f : t0, b1 = t1 == -INFINITY ? 0.f : t1;
        if (__any_sync(kAllLanes, t0 != m0 || t1 != m1 || vnew != vref)) {
            const float c0 = ex2_approx(m0 - b0), c1 = ex2_approx(m1 - b1);
            const float cv = KV == kKvE4m3 ? vref / vnew : 1.f;
            l0 *= c0;
            l1 *= c1;
#pragma unroll
            for (int d = 0; d < DP / 8; ++d) {
                o[d][0] *= c0 * cv;
                o[d][1] *= c0 * cv;
                o[d][2] *= c1 * cv;
                o[d][3] *= c1 * cv;
            }
            m0 = t0;
            m1 = t1;
            vref = vnew;
        }
        // --- probabilities (fp32 sums; rounded to 16 bits for the second product) ---
        uint32_t pa[KT][4];
        const float ivref = KV == kKvE4m3 ? 1.0f / vref : 1.f;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float e[4];
            e[0] = ex2_approx(s[t][0] - b0);
            e[1] = ex2_approx(s[t][1] - b0);
            e[2] = ex2_approx(s[t][2] - b1);
            e[3] = ex2_approx(s[t][3] - b1);
            l0 += e[0] + e[1];
            l1 += e[2] + e[3];
            if constexpr (KV == kKvE4m3) {
                const float x = vr[t][0] * ivref, y = vr[t][1] * ivref;
                e[0] *= x;
                e[1] *= y;
                e[2] *= x;
                e[3] *= y;
            }
            pa[t >> 1][(t & 1) * 2] = pack2<F16>(e[0], e[1]);
            pa[t >> 1][(t & 1) * 2 + 1] = pack2<F16>(e[2], e[3]);
        }
        // --- O += P V ---
        if constexpr (KV != kKvE4m3) {
            const int r = (lane & 7) + (((lane >> 3) & 1) << 3), hi = lane >> 4;
#pragma unroll
            for (int d = 0; d < KS; ++d) {
#pragma unroll
                for (int t = 0; t < KT; ++t) {
                    uint32_t b[4];
                    ldsm4_t(vs_s + swz<C::CH>(16 * t + r, 2 * d + hi), b);
                    mma16816<F16>(o[2 * d], pa[t], b[0], b[1]);
                    mma16816<F16>(o[2 * d + 1], pa[t], b[2], b[3]);
                }
            }
        } else {
            // a transposed matrix hands a lane dims 2g, 2g+1 of tokens 2c, 2c+1: one product
            // takes the even dims of a 16-dim block, one the odd
            const int r = lane;
#pragma unroll
            for (int d = 0; d < KS; ++d) {
                uint32_t b[4];
                ldsm4_t(vs_s + swz<C::CH>(r, d), b);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t lo = __byte_perm(b[2 * k], 0, 0x3120), hi = __byte_perm(b[2 * k + 1], 0, 0x3120);
                    mma16816<F16>(o[2 * d], pa[k], e4m3x2_to_f16x2(lo), e4m3x2_to_f16x2(hi));
                    mma16816<F16>(o[2 * d + 1], pa[k], e4m3x2_to_f16x2(lo >> 16), e4m3x2_to_f16x2(hi >> 16));
                }
            }
        }
        slot = slot + 1 == S ? 0 : slot + 1;

        if (p.team) continue;  // joined after the loop
        const bool row_ends = (meta.w & 2) != 0;
        if (!row_ends && i + 1 < left) continue;
        // --- the row, or the run's part of it, is done ---
        if (i + 1 < left) {  // the next row's queries come while this one is written
            __syncwarp();
            const int4 nm = meta_at(slot);
            load_q(nm.x, nm.y);
        }
        const int kvh = p.head_blocks == 1 ? meta.y : meta.y / p.head_blocks, hb = meta.y - kvh * p.head_blocks;
        const int head0 = kvh * p.group + hb * kAttRows;           // first query head of the row
        const int heads = min(kAttRows, p.group - hb * kAttRows);  // of 16 rows used
        fresh = true;
        l0 += __shfl_xor_sync(kAllLanes, l0, 1);
        l1 += __shfl_xor_sync(kAllLanes, l1, 1);
        l0 += __shfl_xor_sync(kAllLanes, l0, 2);
        l1 += __shfl_xor_sync(kAllLanes, l1, 2);
        const bool done = whole && row_ends;
        float w0 = 1.f, w1 = 1.f;
        float* part = nullptr;
        if (done) {
            w0 = g < heads ? final_weight(p, head0 + g, m0, l0) : 0.f;
            w1 = g + 8 < heads ? final_weight(p, head0 + g + 8, m1, l1) : 0.f;
        } else {
            part = p.partial + ((long long)gw * 2 + (whole ? 1 : 0)) * (kAttRows * (p.D + 2));
            if (c == 0) {
                if (g < heads) part[2 * g] = m0, part[2 * g + 1] = l0;
                if (g + 8 < heads) part[2 * g + 16] = m1, part[2 * g + 17] = l1;
            }
            part += 2 * kAttRows;
        }
        if constexpr (KV == kKvE4m3) {
            w0 *= vref;
            w1 *= vref;
        }
#pragma unroll
        for (int d = 0; d < KS; ++d) {
            if (d * 16 >= p.D) continue;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int row = g + 8 * half;
                const float w = half ? w1 : w0;
                if (row >= heads) continue;
                // a lane's dims: 16 d + 2c, + 1 and 8 on, or (e4m3) 16 d + 4c .. + 3
                const float lo = o[2 * d][2 * half] * w, hi = o[2 * d + 1][2 * half + 1] * w;
                const float u = (KV == kKvE4m3 ? o[2 * d + 1][2 * half] : o[2 * d][2 * half + 1]) * w;
                const float v = (KV == kKvE4m3 ? o[2 * d][2 * half + 1] : o[2 * d + 1][2 * half]) * w;
                const int d0 = d * 16 + (KV == kKvE4m3 ? 4 * c : 2 * c), d1 = d0 + (KV == kKvE4m3 ? 2 : 8);
                if (done) {
                    uint16_t* dst = p.out + meta.x * p.o_token + (long long)(head0 + row) * p.o_head;
                    *reinterpret_cast<uint32_t*>(dst + d0) = pack2<QF16>(lo, u);
                    *reinterpret_cast<uint32_t*>(dst + d1) = pack2<QF16>(v, hi);
                } else {
                    *reinterpret_cast<float2*>(part + row * p.D + d0) = make_float2(lo, u);
                    *reinterpret_cast<float2*>(part + row * p.D + d1) = make_float2(v, hi);
                }
            }
        }
        // the run that a row begins in, for the join (-1: it ends there too)
        if (p.by_row_join && whole && lane == 0) p.first[meta.x * p.rows_per_seq + meta.y] = row_ends ? -1 : gw;
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
        vref = 0x1p-100f;
#pragma unroll
        for (int d = 0; d < DP / 8; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[d][j] = 0.f;
    }
    if (!p.team) return;

    // --- a team: the warps' parts of the row meet in the ring's memory ---
    l0 += __shfl_xor_sync(kAllLanes, l0, 1);
    l1 += __shfl_xor_sync(kAllLanes, l1, 1);
    l0 += __shfl_xor_sync(kAllLanes, l0, 2);
    l1 += __shfl_xor_sync(kAllLanes, l1, 2);
    cp_async_wait<0>();
    __syncthreads();
    float2* s_ml = reinterpret_cast<float2*>(smem);                      // [warps][16]
    float* s_o = reinterpret_cast<float*>(smem + kAttWarps * 16 * 8);    // [warps][16][D + 4]: rows on other banks
    const int ld = p.D + 4;
    if (c == 0) {
        s_ml[warp * 16 + g] = make_float2(m0, l0);
        s_ml[warp * 16 + g + 8] = make_float2(m1, l1);
    }
    const float f = KV == kKvE4m3 ? vref : 1.f;
#pragma unroll
    for (int d = 0; d < KS; ++d) {
        if (d * 16 >= p.D) continue;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float* dst = s_o + (warp * 16 + g + 8 * half) * ld + d * 16 + (KV == kKvE4m3 ? 4 * c : 2 * c);
            const float lo = o[2 * d][2 * half] * f, hi = o[2 * d + 1][2 * half + 1] * f;
            const float u = (KV == kKvE4m3 ? o[2 * d + 1][2 * half] : o[2 * d][2 * half + 1]) * f;
            const float v = (KV == kKvE4m3 ? o[2 * d][2 * half + 1] : o[2 * d + 1][2 * half]) * f;
            *reinterpret_cast<float2*>(dst) = make_float2(lo, u);
            *reinterpret_cast<float2*>(dst + (KV == kKvE4m3 ? 2 : 8)) = make_float2(v, hi);
        }
    }
    __syncthreads();
    const int kvh = row_h / p.head_blocks, hb = row_h - kvh * p.head_blocks;
    const int head0 = kvh * p.group + hb * kAttRows, heads = min(kAttRows, p.group - hb * kAttRows);
    for (int row = warp; row < heads; row += kAttWarps) {
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < kAttWarps; ++w) m = fmaxf(m, s_ml[w * 16 + row].x);
        float e[kAttWarps];
#pragma unroll
        for (int w = 0; w < kAttWarps; ++w) {
            e[w] = m == -INFINITY ? 0.f : ex2_approx(s_ml[w * 16 + row].x - m);
            l += e[w] * s_ml[w * 16 + row].y;
        }
        const float fw = final_weight(p, head0 + row, m, l);
        uint16_t* dst = p.out + row_b * p.o_token + (long long)(head0 + row) * p.o_head;
        for (int d = 2 * lane; d < p.D; d += 64) {
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int w = 0; w < kAttWarps; ++w) {
                const float2 v = *reinterpret_cast<const float2*>(s_o + (w * 16 + row) * ld + d);
                x += e[w] * v.x;
                y += e[w] * v.y;
            }
            *reinterpret_cast<uint32_t*>(dst + d) = pack2<QF16>(x * fw, y * fw);
        }
    }
}

// Joins the parts of rows cut by a run's border.  Job j: row j (by_row_join: its
// first run in first[j], -1 if one run did it all), or the row that run j
// continues as the first to do so.  Parts: slot 1 of the first run, slot 0 of
// the runs that continue the row.  A CTA takes heads_per_cta heads, its 8 warps
// split over heads and, where those are fewer, over the parts.
template <bool QF16>
__global__ void __launch_bounds__(256) attend_join_kernel(AttendParams p) {
    __shared__ float s_m[8], s_l[8];
    __shared__ float s_o[8 * 256];
    pdl_wait();
    const int j = blockIdx.x;
    const int nruns = p.runs;
    int run0, row;
    if (p.by_row_join) {
        run0 = p.first[j];
        row = j;
        if (run0 < 0) return;
    } else {
        row = p.cont[j];
        if (row < 0 || p.cont[j - 1] == row) return;  // run 0 starts a row: cont[0] is -1
        run0 = j - 1;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int nparts = 1;
    for (uint32_t same = kAllLanes; same == kAllLanes;) {
        const int r = run0 + nparts + lane;
        same = __ballot_sync(kAllLanes, r < nruns && p.cont[r] == row);
        nparts += same == kAllLanes ? 32 : __ffs(~same) - 1;
    }
    const int b = row / p.rows_per_seq, h = row - b * p.rows_per_seq;
    const int hb = h % p.head_blocks, head0 = (h / p.head_blocks) * p.group + hb * kAttRows;
    const int heads = min(kAttRows, p.group - hb * kAttRows);
    const int psize = kAttRows * (p.D + 2);
    auto part = [&](int i) { return p.partial + ((long long)(run0 + i) * 2 + (i == 0 ? 1 : 0)) * psize; };
    const int pw = p.heads_per_cta >= 8 ? 1 : 8 / p.heads_per_cta;  // warps per head
    const int hw = 8 / pw;
    const int h_end = min(heads, ((int)blockIdx.y + 1) * p.heads_per_cta);
    for (int hh = blockIdx.y * p.heads_per_cta; hh < h_end; hh += hw) {
        const int head = hh + warp / pw, sub = warp % pw;
        float m = -INFINITY, l = 0.f;
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (head < h_end) {
            const int i0 = nparts * sub / pw, i1 = nparts * (sub + 1) / pw;
            for (int i = i0 + lane; i < i1; i += 32) m = fmaxf(m, part(i)[2 * head]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAllLanes, m, o));
            const float base = m == -INFINITY ? 0.f : m;
#pragma unroll 4
            for (int i = i0; i < i1; ++i) {
                const float* q = part(i);
                const float w = ex2_approx(q[2 * head] - base);
                l += w * q[2 * head + 1];
                const float* src = q + 2 * kAttRows + head * p.D;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k * 32 + lane < p.D) acc[k] += w * src[k * 32 + lane];
            }
        }
        if (pw > 1) {  // the warps of a head join in shared memory, in order
            if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k * 32 + lane < p.D) s_o[warp * 256 + k * 32 + lane] = acc[k];
            __syncthreads();
            if (sub == 0 && head < h_end) {
                float top = -INFINITY;
                for (int w = 0; w < pw; ++w) top = fmaxf(top, s_m[warp + w]);
                m = top;
                l = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] = 0.f;
                for (int w = 0; w < pw; ++w) {
                    const float f = top == -INFINITY ? 0.f : ex2_approx(s_m[warp + w] - top);
                    l += f * s_l[warp + w];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k * 32 + lane < p.D) acc[k] += f * s_o[(warp + w) * 256 + k * 32 + lane];
                }
            }
            __syncthreads();
        }
        if (sub == 0 && head < h_end) {
            const float w = final_weight(p, head0 + head, m, l);
            uint16_t* dst = p.out + b * p.o_token + (long long)(head0 + head) * p.o_head;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k * 32 + lane < p.D) dst[k * 32 + lane] = (uint16_t)pack2<QF16>(acc[k] * w, 0.f);
        }
    }
}

namespace {

// Runs are at least this many tokens; rows of at most this many are not cut; a
// CTA takes a row of its own where all rows fit at once and none is longer.
constexpr int kMinTokens = 64;
constexpr int kWholeTokens = 128;
constexpr int kTeamTokens = 512;

int dp_of(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
int ctas_per_sm(int dp, bool e4m3) { return dp == 64 && e4m3 ? 3 : dp == 256 ? 1 : 2; }
int tile_tokens(int dp, bool e4m3) { return e4m3 || dp == 64 ? 32 : 16; }

template <int DP, int KV, bool QF16>
cudaError_t launch_attend_t(const AttendParams& p, int grid, cudaStream_t st) {
    using C = AttCfg<DP, KV>;
    static_assert(C::SMEM * C::CTAS <= 226 * 1024, "shared memory of the resident CTAs");
    cudaError_t e = cudaFuncSetAttribute(attend_kernel<DP, KV, QF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    attend_kernel<DP, KV, QF16><<<grid, kAttWarps * 32, C::SMEM, st>>>(p);
    return cudaGetLastError();
}
template <int KV, bool QF16>
cudaError_t launch_attend_d(const AttendParams& p, int grid, cudaStream_t st) {
    switch (dp_of(p.D)) {
        case 64: return launch_attend_t<64, KV, QF16>(p, grid, st);
        case 128: return launch_attend_t<128, KV, QF16>(p, grid, st);
        default: return launch_attend_t<256, KV, QF16>(p, grid, st);
    }
}

}  // namespace

// How the rows are given to warps; the workspace is for the parts of cut rows.
void attend_plan(int B, int Hq, int Hkv, int D, bool e4m3, int most, int sms, AttendPlan* w) {
    const int ctas = sms * ctas_per_sm(dp_of(D), e4m3), runs = ctas * kAttWarps;
    const long long rows = (long long)B * Hkv * ((Hq / Hkv + kAttRows - 1) / kAttRows);
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    w->runs = runs;
    w->team = rows <= ctas && most <= kTeamTokens;
    w->by_row = !w->team && most <= kWholeTokens;
    w->by_row_join = rows <= runs;
    w->cont = 0;
    w->first = up((size_t)runs * 4);
    w->partial = w->first + up((size_t)(rows <= runs ? rows : 1) * 4);
    w->total = w->team || w->by_row ? 0 : w->partial + (size_t)runs * 2 * kAttRows * (D + 2) * 4;
}

cudaError_t launch_attend(const AttendParams& p_in, const AttendPlan& w, int kv_dtype, bool fp16, void* workspace,
                          cudaStream_t st) {
    AttendParams p = p_in;
    const bool e4m3 = kv_dtype == kDtE4m3;
    p.runs = w.runs;
    p.team = w.team;
    p.by_row = w.by_row;
    p.group = p.Hq / p.Hkv;
    p.head_blocks = (p.group + kAttRows - 1) / kAttRows;
    p.rows_per_seq = p.Hkv * p.head_blocks;
    p.page16 = p.page_size % 16 == 0;
    p.page_shift = -1;
    if ((p.page_size & (p.page_size - 1)) == 0)
        for (p.page_shift = 0; (1 << p.page_shift) < p.page_size;) ++p.page_shift;
    const long long rows = (long long)p.B * p.rows_per_seq;
    p.min_units = kMinTokens / tile_tokens(dp_of(p.D), e4m3);
    if (w.total) {
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        p.by_row_join = w.by_row_join;
        p.cont = reinterpret_cast<int32_t*>(ws + w.cont);
        p.first = reinterpret_cast<int32_t*>(ws + w.first);
        p.partial = reinterpret_cast<float*>(ws + w.partial);
    }
    const int grid = p.team ? (int)rows : w.runs / kAttWarps;
    cudaError_t e;
    if (e4m3)
        e = fp16 ? launch_attend_d<kKvE4m3, true>(p, grid, st) : launch_attend_d<kKvE4m3, false>(p, grid, st);
    else
        e = fp16 ? launch_attend_d<kKvFp16, true>(p, grid, st) : launch_attend_d<kKvBf16, false>(p, grid, st);
    if (e != cudaSuccess || p.by_row || p.team) return e;
    // few rows: a CTA per head, its warps over the parts; many: a CTA per row
    const int heads = p.group < kAttRows ? p.group : kAttRows;
    const int jobs = p.by_row_join ? (int)rows : p.runs;
    p.heads_per_cta = jobs <= 256 ? 1 : 8;
    const dim3 jg(jobs, (heads + p.heads_per_cta - 1) / p.heads_per_cta);
    return fp16 ? launch_pdl(attend_join_kernel<true>, jg, dim3(256), 0, st, p)
                : launch_pdl(attend_join_kernel<false>, jg, dim3(256), 0, st, p);
}

}  // namespace moe
