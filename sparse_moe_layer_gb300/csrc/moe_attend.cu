// Attention of one new token per sequence over a paged key-value cache, with
// grouped query heads, an optional sink logit per head and an optional sliding
// window ("GPT-OSS on Day 0", perplexity.ai hub blog: GQA, sink attention --
// the sink enters the softmax sum once per row -- and alternating windows).
//
//   o = sum_t p_t v_t / (sum_t p_t + 2^(sink log2 e - m)),  p_t = 2^(s_t - m),
//   s_t = (q . k_t) scale log2 e,  t over the last `window` of `length` tokens
//
// Bound by the cache's bytes: each key and value is read once for (up to 16)
// query heads that share it, so the products need G flops a byte (8 to 16,
// above what the fp32 pipes give at full bandwidth, far below the matrix
// instructions): m16n8k16 with the group's heads as the 16 rows, scores and
// probabilities staying in registers between the two products.  A 64- or
// 128-row tcgen05 tile would be 4 to 16 times padding here and hand the scores
// through tensor memory.
//
// The (sequence, key head, token tile) list is cut into equal runs, one per
// resident CTA, so a batch of very different lengths loads all SMs alike.  A
// CTA's warps take the run's tiles in turn, each through its own cp.async ring
// (the copies run on over the borders of rows) with its own running maximum and
// sum; where a row or the run ends they join in shared memory.  Only a row cut by
// a run's border leaves fp32 parts, which a second, dependent launch joins in a
// fixed order (results do not depend on scheduling).  Short rows are not cut: a
// CTA or a warp takes whole ones (attend_plan).
//
// 64 sequences of 1 to 16384 tokens, 8 key heads of 64, bf16: 164 us, 6.3 TB/s (92 % of a
// copy). 4 sequences of 100000 to 131072 tokens, 4 key heads of 128, e4m3: 89 us, 5.5 TB/s;
// 6.8 TB/s while it streams, and 15 us of launch, first tiles, row ends and the join.
// 256 sequences, window 128, 8 key heads of 64, bf16: 16 us, 4.5 TB/s: latency of the 8
// tiles that a warp has. One sequence of 90 tokens: 3.5 us, latency.
// A run per warp instead of per CTA lost 4 % on 128 rows and more; 16-token tiles on
// e4m3 took 149 us, 12 warps an SM with two stages 132 where this shape took 123.
// More than 16 heads to a key: a row per 16, which reads the cache again (4 x 60000 tokens,
// 4 key heads of 128, bf16: 64 heads 88 us, 128 heads 166).
#include "moe_attend.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kAttWarps = 4;  // warps per CTA
constexpr int kAttRows = 16;  // query heads per row (m16 of the products)

// How the rows are given out: equal runs of tiles, one per CTA; a row per CTA; rows
// per warp.  attend_plan chooses.
enum : int { kRuns = 0, kTeam = 1, kRows = 2 };

// Tokens per tile and CTAs per SM.  light (16-bit caches of up to 64 dims): half the
// tile and twice the warps, for whole rows that one wave of these takes.
constexpr int tile_tokens(int dp, bool e4m3, bool light) { return e4m3 || (dp == 64 && !light) ? 32 : 16; }
constexpr int ctas_per_sm(int dp, bool e4m3, bool light) {
    return dp == 64 ? (e4m3 ? 3 : light ? 4 : 2) : dp == 256 ? 1 : 2;
}

// Rows of at most kWholeTokens are not cut where that costs little.  A CTA takes a
// row, all rows resident at once: up to one wave of the wide kernel if the tiles
// that its idle CTAs miss are few (kTeamTiles each on average), up to one of the
// light kernel (between the two, us of the light team / warps with rows / cut: 320 rows
// of 128 tokens 6.3 / 7.0 / 11.2, 600 of 512 15.9 / 19.8 / 23.3, of 1000 27.9 / 35.7 / 34.6;
// below, the wide team wins: 256 rows of 300 7.1 / 7.7).  Else a warp takes rows, if the
// tiles that the busiest has beyond the average are fewer than what the alternative
// costs: borders, joins and the second launch (kRowTiles) and a meeting of the
// CTA's warps at every row's end (kEndTiles), both twice as many where a warp's
// tile counts half (light) or a CTA has the SM for itself (more than 128 dims).
// us whole / cut, bf16, D = 64: 1024 rows of 128 tokens 8.1 / 19.2, of 1000 45.5 / 52.2; 2600
// of 256 38.5 / 46.8, of 512 69.6 / 68.1, of 1000 130 / 111; light: 1296 of 128 11.1 / 20.6, of
// 1000 60.9 / 62.8; D = 128, e4m3: 320 of 256 15.9 / 19.3, of 512 27.2 / 22.5, 4096 of 512 116 / 158;
// D = 256: 320 of 512 42.9 / 56.9, 1300 of 1000 277 / 251.
// kRowTilesFound: the same in a kernel that was launched for long rows and finds short
// ones, with more rows than CTAs; what it was launched with costs the join's launch either
// way. us whole / cut, table of 16000 tokens more: bf16, D = 64: 2048 rows of 1-128 tokens
// 17.1 / 36.9, of 256 32.0 / 38.1, 320 of 64 8.7 / 8.6, of 256 14.2 / 12.8, 64 of 256 12.7 / 7.9;
// D = 128, e4m3: 2048 of 1-128 23.7 / 71.5, of 1000 111 / 128.
constexpr int kWholeTokens = 1024;
constexpr int kTeamTiles = 24;
constexpr int kRowTiles = 9, kEndTiles = 4;
constexpr int kRowTilesFound = 4;
// Whether warps of n CTAs take whole rows of up to `tiles` tiles (allowance, weight: as above).
__host__ __device__ inline bool rows_fit(long long tiles, long long rows, int n, int allowance, int weight) {
    const long long warps = (long long)n * kAttWarps, waves = (rows + warps - 1) / warps;
    return tiles * (waves * warps - rows) <= weight * (allowance * warps + kEndTiles * rows);
}

template <int DP, int KV, bool LIGHT>
struct AttCfg {
    static constexpr int ES = KV == kKvE4m3 ? 1 : 2;       // bytes of a cached value
    static constexpr int TT = tile_tokens(DP, KV == kKvE4m3, LIGHT);  // tokens per tile
    static constexpr int CH = DP * ES / 16;                // 16-byte chunks of a token's row
    static constexpr int LANES = CH <= 4 ? 4 : CH <= 8 ? 8 : CH <= 16 ? 16 : 32;  // lanes that copy it
    static constexpr int PITCH = DP == 96 ? CH | 1 : CH;   // chunks from row to row in shared memory
    static constexpr int ROW = PITCH * 16;
    static constexpr int STAGES = DP == 64 && KV == kKvE4m3 ? 4 : DP == 256 && KV == kKvE4m3 ? 2 : 3;
    static constexpr int TILE = TT * ROW;                  // bytes of a K (or V) tile
    static constexpr int SC = KV == kKvE4m3 ? 2 * TT * 4 : 0;
    static constexpr int STAGE = 2 * TILE + SC + 16;       // + the mask of valid tokens
    static constexpr int QS = DP == 256 ? DP / 16 * 512 : 0;  // Q fragments, where registers do not hold them
    static constexpr int WARP = (STAGES * STAGE + QS + 127) / 128 * 128;
    static constexpr int SMEM = kAttWarps * WARP;
    static constexpr int CTAS = ctas_per_sm(DP, KV == kKvE4m3, LIGHT);
};

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
// Byte of chunk c (16 bytes) of token row r in a tile: 8 rows of one chunk
// column fall on 8 different bank groups, for the loads and for ldmatrix.
template <typename C>
__device__ __forceinline__ uint32_t swz(int r, int c) {
    if (C::PITCH & 1) return (uint32_t)(r * C::PITCH + c) * 16u;  // an odd pitch does it alone
    if (C::CH >= 8) return (uint32_t)(r * C::CH + ((c & ~7) | ((c ^ r) & 7))) * 16u;
    return (uint32_t)(r * C::CH + (c ^ ((r >> 1) & 3))) * 16u;  // CH == 4: two rows per 128 bytes
}

// a / b of numbers >= 0: 32-bit where they fit, as they nearly always do (the
// 64-bit division is a routine of a few hundred cycles)
__device__ __forceinline__ long long quotient(long long a, int b) {
    return a >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
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

// A place in the list of tiles: sequence b, row h of it (key head and block of
// 16 query heads), tile of the row.
template <int TT>
struct TileIt {
    int b, h, tile, ntiles, start, len;
    __device__ __forceinline__ void seq(const AttendParams& p) {
        len = seen_tokens(p, b, &start);
        ntiles = tiles_of<TT>(start, len);
    }
    __device__ __forceinline__ void advance(const AttendParams& p, int step) {
        tile += step;
        while (tile >= ntiles) {
            tile -= ntiles;
            if (++h < p.rows_per_seq) continue;
            h = 0;
            if (++b >= p.B) return;
            seq(p);
        }
    }
};

// A lane's four values of a 16-dim block of one row (half 0: row g, 1: row g + 8)
// from its two accumulators, times w, in memory order: dims quad_at, + 1 and, 8
// on (e4m3: 2 on), two more.
struct Quad {
    float a, b, c, d;
};
template <int KV>
__device__ __forceinline__ Quad quad(const float (&u)[4], const float (&v)[4], int half, float w) {
    if (KV == kKvE4m3) return {u[2 * half] * w, v[2 * half] * w, u[2 * half + 1] * w, v[2 * half + 1] * w};
    return {u[2 * half] * w, u[2 * half + 1] * w, v[2 * half] * w, v[2 * half + 1] * w};
}
template <int KV>
__device__ __forceinline__ int quad_at(int c) {
    return KV == kKvE4m3 ? 4 * c : 2 * c;
}

}  // namespace

template <int DP, int KV, bool QF16, int MODE, bool LIGHT>
__global__ void __launch_bounds__(kAttWarps * 32, AttCfg<DP, KV, LIGHT>::CTAS) attend_kernel(AttendParams p) {
    using C = AttCfg<DP, KV, LIGHT>;
    bool by_row = MODE == kRows;  // kRuns: if the lengths found are all short
    constexpr bool F16 = KV != kKvBf16;  // type of the products
    constexpr int TT = C::TT, NT = TT / 8, KT = TT / 16, KS = DP / 16, S = C::STAGES;
    constexpr uint32_t kAllTokens = TT == 32 ? 0xffffffffu : 0xffffu;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_pre[kAttWarps * 32 + 1];
    __shared__ int s_wsum[kAttWarps], s_wmax[kAttWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    __shared__ float2 s_ml[kAttWarps][kAttRows];  // a segment's maxima and sums
    __shared__ int s_slot[kAttWarps];             // and the ring slot of its values
    pdl_wait();
    pdl_allow_dependents();

    // --- the run: tiles that the CTA's warps take in turn, or whole rows of one warp ---
    TileIt<TT> it;  // of the copies
    int rem;        // tiles of the run
    const int run = blockIdx.x;
    auto whole_rows = [&]() {  // a warp's rows, neighbouring warps' on different SMs; false: none
        const int nwarps = gridDim.x * kAttWarps, w = warp * gridDim.x + blockIdx.x;
        const int rows = p.B * p.rows_per_seq, n = rows < nwarps ? rows : nwarps;
        if (w >= n) return false;
        const int u0 = (int)((long long)rows * w / n), u1 = (int)((long long)rows * (w + 1) / n);
        it.b = u0 / p.rows_per_seq;
        it.h = u0 - it.b * p.rows_per_seq;
        it.tile = 0;
        it.seq(p);
        rem = 0;
        TileIt<TT> t = it;
        for (int r = u1 - u0; r > 0; --r) {
            rem += t.ntiles;
            t.advance(p, t.ntiles);
        }
        return true;
    };
    if constexpr (MODE == kRows) {
        if (!whole_rows()) return;
    } else if constexpr (MODE == kTeam) {  // few rows, none long: one to a CTA
        it.b = run / p.rows_per_seq;
        it.h = run - it.b * p.rows_per_seq;
        it.tile = 0;
        it.seq(p);
        rem = it.ntiles;
    } else {
        // each thread sums the tiles of a slice of the sequences (rows_per_seq rows each)
        const int slice = (p.B + kAttWarps * 32 - 1) / (kAttWarps * 32);
        int mine = 0, longest = 0;
        for (int i = 0; i < slice; ++i) {
            const int b = tid * slice + i;
            if (b < p.B) {
                int st;
                const int len = seen_tokens(p, b, &st);
                const int nt = tiles_of<TT>(st, len);
                mine += nt;
                longest = max(longest, nt);
            }
        }
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kAllLanes, inc, o);
            if (lane >= o) inc += v;
        }
        longest = __reduce_max_sync(kAllLanes, longest);
        if (lane == 31) s_wsum[warp] = inc, s_wmax[warp] = longest;
        __syncthreads();
        int before = 0;
#pragma unroll
        for (int w = 0; w < kAttWarps; ++w) {
            if (w < warp) before += s_wsum[w];
            longest = max(longest, s_wmax[w]);
        }
        // a wide table whose rows turn out short: whole rows by warps after all (kRowTilesFound)
        const int rows = p.B * p.rows_per_seq;
        by_row = longest * TT <= kWholeTokens && rows >= (int)gridDim.x &&
                 rows_fit(longest, rows, gridDim.x, kRowTilesFound, DP == 256 ? 2 : 1);
        s_pre[tid + 1] = before + inc;
        if (tid == 0) s_pre[0] = 0;
        __syncthreads();
        if (by_row) {
            if (tid == 0) p.cont[run] = -1;
            if (!whole_rows()) return;
        } else {
            const long long total = (long long)s_pre[kAttWarps * 32] * p.rows_per_seq;
            const long long want = (total + kAttWarps - 1) / kAttWarps;
            const int n = (int)(want < (int)gridDim.x ? want : gridDim.x);
            if (run >= n) {
                if (tid == 0) p.cont[run] = -1;
                return;
            }
            // run r starts at total * r / n: longer runs spread evenly, not first (2 us on 16 rows of 8000)
            const long long each = quotient(total, n);
            const int more = (int)(total - each * n), from = more * run / n;  // n <= runs: small products
            const long long u0 = each * run + from;
            rem = (int)each + more * (run + 1) / n - from;
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
            it.h = (int)quotient(u, it.ntiles);
            it.tile = (int)(u - (long long)it.h * it.ntiles);
            if (tid == 0) p.cont[run] = it.tile ? it.b * p.rows_per_seq + it.h : -1;
        }
    }
    TileIt<TT> row = it;  // of the products: the tile that the current segment (a row's tiles in the run) begins with
    const int step = by_row ? 1 : kAttWarps;
    int to_issue = by_row ? rem : rem > warp ? (rem - warp + kAttWarps - 1) / kAttWarps : 0;  // tiles of this warp
    if (!by_row && to_issue > 0) it.advance(p, warp);

    // --- the ring ---
    uint8_t* ring = smem + warp * C::WARP;
    const uint32_t ring_s = smem_u32(ring);
    constexpr int RPS = 32 / C::LANES;  // token rows per step of the warp
    const int ch = lane % C::LANES, r0 = lane / C::LANES;
    const bool in = ch * (16 / C::ES) < p.D;
    // byte offsets of the lane's chunk in a group of 16 tokens, and of a step
    const long long k_lane = (long long)r0 * p.cache.k_token * C::ES + ch * 16, k_step = RPS * p.cache.k_token * C::ES;
    const long long v_lane = (long long)r0 * p.cache.v_token * C::ES + ch * 16, v_step = RPS * p.cache.v_token * C::ES;
    // tile `it`: tokens of the lanes and their pages, looked up before the copies need them
    struct Fetched {
        int h, pid, off;
        bool ok;
    };
    auto fetch = [&]() {
        Fetched f = {it.h, -1, 0, false};
        const int tok = (it.start / TT + it.tile) * TT + (lane & (TT - 1));
        if (tok < it.len) {
            const int pi = p.page_shift >= 0 ? tok >> p.page_shift : tok / p.page_size;
            f.off = tok - pi * p.page_size;
            // a token before the window shares its group's page; with smaller pages it is not looked up
            if (tok >= it.start || p.page16) f.pid = __ldg(p.table + (long long)it.b * p.table_ld + pi);
        }
        f.ok = tok >= it.start && tok < it.len;
        return f;
    };
    auto issue = [&](int slot, Fetched f) {
        const uint32_t dst = ring_s + slot * C::STAGE;
        const int kvh = p.head_blocks == 1 ? f.h : f.h / p.head_blocks;
        if ((uint32_t)f.pid >= (uint32_t)p.num_pages) {
            if (f.ok && p.status) atomicOr(p.status, kErrBadIndex);
            f.pid = 0;
            f.ok = false;
        }
        const uint32_t mask = __ballot_sync(kAllLanes, f.ok);
        const uint8_t* kb = static_cast<const uint8_t*>(p.cache.k) + (long long)kvh * p.cache.k_head * C::ES;
        const uint8_t* vb = static_cast<const uint8_t*>(p.cache.v) + (long long)kvh * p.cache.v_head * C::ES;
        if (p.page16) {  // a group of 16 tokens lies on one page
#pragma unroll
            for (int hh = 0; hh < KT; ++hh) {
                const long long pid = __shfl_sync(kAllLanes, f.pid, hh * 16);
                const long long off = __shfl_sync(kAllLanes, f.off, hh * 16);
                const uint8_t* ks = kb + (pid * p.cache.k_page + off * p.cache.k_token) * C::ES + k_lane;
                const uint8_t* vs = vb + (pid * p.cache.v_page + off * p.cache.v_token) * C::ES + v_lane;
                if (((mask >> (16 * hh)) & 0xffffu) == 0xffffu) {
                    if (in) {
#pragma unroll
                        for (int i = 0; i < 16 / RPS; ++i) {
                            const uint32_t at = dst + swz<C>(16 * hh + r0 + i * RPS, ch);
                            cp_async16(at, ks + i * k_step);
                            cp_async16(at + C::TILE, vs + i * v_step);
                        }
                    }
                } else if (in) {
#pragma unroll
                    for (int i = 0; i < 16 / RPS; ++i) {
                        const int r = 16 * hh + r0 + i * RPS;
                        const uint32_t at = dst + swz<C>(r, ch);
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
                const long long pid = __shfl_sync(kAllLanes, f.pid, r), off = __shfl_sync(kAllLanes, f.off, r);
                const bool ok = (mask >> r) & 1u;
                const uint32_t at = dst + swz<C>(r, ch);
                const long long k_at = (pid * p.cache.k_page + off * p.cache.k_token) * C::ES + ch * 16;
                const long long v_at = (pid * p.cache.v_page + off * p.cache.v_token) * C::ES + ch * 16;
                if (in) {
                    cp_async16z(at, ok ? kb + k_at : kb, ok);
                    cp_async16z(at + C::TILE, ok ? vb + v_at : vb, ok);
                }
            }
        }
        if constexpr (KV == kKvE4m3) {  // lane = token (TT == 32)
            const long long at =
                f.ok ? f.pid * p.cache.s_page + kvh * p.cache.s_head + f.off * p.cache.s_token : 0;
            cp_async4z(dst + 2 * C::TILE + lane * 4, p.cache.k_scale + at, f.ok);
            cp_async4z(dst + 2 * C::TILE + TT * 4 + lane * 4, p.cache.v_scale + at, f.ok);
        }
        if (lane == 0)  // valid tokens
            *reinterpret_cast<uint32_t*>(ring + slot * C::STAGE + 2 * C::TILE + C::SC) = mask & kAllTokens;
    };
    // dims past D (D < DP) are products of zeros: no branch in the tile loop
    auto zero_pad = [&](int slot) {
        if (p.D < DP)
            for (int i = lane * 16; i < 2 * C::TILE; i += 32 * 16)
                *reinterpret_cast<uint4*>(ring + slot * C::STAGE + i) = make_uint4(0, 0, 0, 0);
        __syncwarp();
    };
    for (int s = 0; s < S; ++s) zero_pad(s);
    Fetched next = {0, -1, 0, false};
    if (to_issue > 0) next = fetch();
    auto issue_next = [&](int slot) {
        if (to_issue > 0) {
            issue(slot, next);
            if (--to_issue > 0) {
                it.advance(p, step);
                next = fetch();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1  // (a tile's pages are in the cache line of the one before, as a rule)
    for (int s = 0; s < S - 1; ++s) issue_next(s);

    float o[DP / 8][4];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // rows g and g + 8; e4m3: a lane's share of the sums
    float ls[4] = {0.f, 0.f, 0.f, 0.f};                        // 16-bit caches: the sums, [0] and [2]
    // positive factors of the scores: |scale| log2 e, times the query row's power of two (e4m3)
    float qf0 = p.scale_log2, qf1 = p.scale_log2;
    float b0 = 0.f, b1 = 0.f;  // powers of two that sums and accumulators are about
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
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] ^= p.q_sign;
            set_qfrag(k, a);
        }
    };
    int slot = 0, fill = S - 1, pos = 0;
    int b = 0, h = 0;  // the segment done last
    bool starts = false, ends = false;
    for (bool first = true;; first = false) {
        // the row's queries come with its first tiles, or while the row before is written
        if (rem > 0) load_q(row.b, row.h);
        if (!first) {
            const int kvh = p.head_blocks == 1 ? h : h / p.head_blocks, hb = h - kvh * p.head_blocks;
            const int head0 = kvh * p.group + hb * kAttRows;           // first query head of the row
            const int heads = min(kAttRows, p.group - hb * kAttRows);  // of 16 rows used
            if constexpr (KV == kKvE4m3) {
                l0 += __shfl_xor_sync(kAllLanes, l0, 1);
                l1 += __shfl_xor_sync(kAllLanes, l1, 1);
                l0 += __shfl_xor_sync(kAllLanes, l0, 2);
                l1 += __shfl_xor_sync(kAllLanes, l1, 2);
            } else {
                l0 = ls[0];
                l1 = ls[2];
            }
            m0 = m0 * qf0 - kLift<KV>;  // from here on in powers of two, what the sums are about
            m1 = m1 * qf1 - kLift<KV>;
            // e4m3: sums and accumulators about the maximum
            const float f0 = KV != kKvE4m3 ? 1.f : m0 == -INFINITY ? 0.f : ex2_approx(b0 - m0);
            const float f1 = KV != kKvE4m3 ? 1.f : m1 == -INFINITY ? 0.f : ex2_approx(b1 - m1);
            l0 *= f0;
            l1 *= f1;
            const bool done = MODE != kRuns || (starts && ends);
            float* part = done ? nullptr : p.partial + ((long long)run * 2 + (starts ? 1 : 0)) * (kAttRows * (p.D + 2));
            // the runs that a row begins and ends in, for the join (first -1: one run has all of it)
            if (MODE == kRuns && p.by_row_join && (by_row ? lane : tid) == 0) {
                const int at = b * p.rows_per_seq + h;
                if (starts) p.first[at] = ends ? -1 : run;
                if (ends && !starts) p.last[at] = run;
            }
            if (by_row) {
                float w0 = g < heads ? final_weight(p.sinks, head0 + g, m0, l0) : 0.f;
                float w1 = g + 8 < heads ? final_weight(p.sinks, head0 + g + 8, m1, l1) : 0.f;
                if constexpr (KV == kKvE4m3) {
                    w0 *= f0;
                    w1 *= f1;
                }
#pragma unroll
                for (int d = 0; d < KS; ++d) {
                    if (d * 16 >= p.D) continue;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int r = g + 8 * half;
                        if (r >= heads) continue;
                        const Quad q = quad<KV>(o[2 * d], o[2 * d + 1], half, half ? w1 : w0);
                        uint16_t* dst =
                            p.out + b * p.o_token + (long long)(head0 + r) * p.o_head + d * 16 + quad_at<KV>(c);
                        *reinterpret_cast<uint32_t*>(dst) = pack2<QF16>(q.a, q.b);
                        *reinterpret_cast<uint32_t*>(dst + (KV == kKvE4m3 ? 2 : 8)) = pack2<QF16>(q.c, q.d);
                    }
                }
            } else {
                // the warps' parts meet in the ring slots that hold no tile (one of each warp); columns of a
                // row are moved by 4 (row mod 8) to spread the rows over the banks
                if (lane == 0) s_slot[warp] = fill;
                if (c == 0) {
                    s_ml[warp][g] = make_float2(m0, l0);
                    s_ml[warp][g + 8] = make_float2(m1, l1);
                }
                {
                    float* mine = reinterpret_cast<float*>(ring + fill * C::STAGE);
#pragma unroll
                    for (int d = 0; d < KS; ++d) {
                        if (d * 16 >= p.D) continue;
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            if (g + 8 * half >= heads) continue;
                            const Quad q = quad<KV>(o[2 * d], o[2 * d + 1], half, half ? f1 : f0);
                            float* dst = mine + (g + 8 * half) * DP;
                            const int d0 = d * 16 + quad_at<KV>(c), d1 = d0 + (KV == kKvE4m3 ? 2 : 8);
                            *reinterpret_cast<float2*>(dst + (d0 ^ (g << 2))) = make_float2(q.a, q.b);
                            *reinterpret_cast<float2*>(dst + (d1 ^ (g << 2))) = make_float2(q.c, q.d);
                        }
                    }
                }
                __syncthreads();
                constexpr int LPR = DP == 64 ? 16 : 32;  // lanes of a row, 4 dims each
                constexpr int RPW = 32 / LPR;
#pragma unroll 4
                for (int r0 = 0; r0 < kAttRows; r0 += kAttWarps * RPW) {
                    const int r = r0 + warp * RPW + lane / LPR;
                    if (r >= heads) break;
                    float m = -INFINITY, l = 0.f, e[kAttWarps];
                    const float* src[kAttWarps];
#pragma unroll
                    for (int w = 0; w < kAttWarps; ++w) {
                        m = fmaxf(m, s_ml[w][r].x);
                        src[w] = reinterpret_cast<const float*>(smem + w * C::WARP + s_slot[w] * C::STAGE) + r * DP;
                    }
#pragma unroll
                    for (int w = 0; w < kAttWarps; ++w) {
                        e[w] = m == -INFINITY ? 0.f : ex2_approx(s_ml[w][r].x - m);
                        l += e[w] * s_ml[w][r].y;
                    }
                    const float fw = done ? final_weight(p.sinks, head0 + r, m, l) : 1.f;
                    if (!done && lane % LPR == 0) *reinterpret_cast<float2*>(part + 2 * r) = make_float2(m, l);
#pragma unroll
                    for (int q = 0; q < (DP + 127) / 128; ++q) {
                        const int d = 4 * (lane % LPR) + 128 * q;
                        if (d >= p.D) continue;
                        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int w = 0; w < kAttWarps; ++w)
                            add_scaled(x, 1.f, *reinterpret_cast<const float4*>(src[w] + (d ^ ((r & 7) << 2))), e[w]);
                        if (done) {
                            uint16_t* dst = p.out + b * p.o_token + (long long)(head0 + r) * p.o_head + d;
                            *reinterpret_cast<uint32_t*>(dst) = pack2<QF16>(x.x * fw, x.y * fw);
                            *reinterpret_cast<uint32_t*>(dst + 2) = pack2<QF16>(x.z * fw, x.w * fw);
                        } else {
                            *reinterpret_cast<float4*>(part + 2 * kAttRows + r * p.D + d) = x;
                        }
                    }
                }
                if (rem > 0) {
                    __syncthreads();  // the slots are free again
                    zero_pad(fill);
                }
            }
        }
        if (rem == 0) return;
        // --- a segment ---
        const int nseg = min(row.ntiles - row.tile, rem);
        m0 = m1 = -INFINITY;
        l0 = l1 = ls[0] = ls[2] = 0.f;
        b0 = b1 = KV == kKvE4m3 ? kNoWeights : 0.f;
#pragma unroll
        for (int d = 0; d < DP / 8; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[d][j] = 0.f;
        if constexpr (KV == kKvE4m3) {
            // the products run in fp16: each query row is scaled by a power of two to below 2^15, fp16's
            // upper end, so that every fp16 value and bf16 values down to 2^-30 of the largest are exact (its
            // smallest step is 2^-39 of the largest; sums of 256 products by codes stay below 2^32)
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
            // 2^(14 - floor(log2 amax)) and its inverse, exponent fields kept within [1, 253]
            const uint32_t e0 = min(max(__float_as_uint(a0) >> 23, 15u), 253u);
            const uint32_t e1 = min(max(__float_as_uint(a1) >> 23, 15u), 253u);
            const float f0 = __uint_as_float((268u - e0) << 23), f1 = __uint_as_float((268u - e1) << 23);
            // not 0, which would make NaN of a masked score
            qf0 = fmaxf(p.scale_log2 * __uint_as_float((e0 - 14u) << 23), 0x1p-126f);
            qf1 = fmaxf(p.scale_log2 * __uint_as_float((e1 - 14u) << 23), 0x1p-126f);
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
        // a warp's tiles of the segment: places of the run that are its own modulo the warps
        for (int j = by_row ? 0 : (warp - pos) & (kAttWarps - 1); j < nseg; j += step) {
            cp_async_wait<S - 2>();
            __syncwarp();
            issue_next(fill);
            fill = fill + 1 == S ? 0 : fill + 1;
            const uint8_t* stage = ring + slot * C::STAGE;
            const uint32_t ks_s = ring_s + slot * C::STAGE, vs_s = ks_s + C::TILE;

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
                        ldsm4(ks_s + swz<C>(16 * t + r, 2 * k + hi), b);
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
                    ldsm4(ks_s + swz<C>(r, k), b);
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        mma16816<F16>(s[t], a, e4m3x2_to_f16x2(b[t]), e4m3x2_to_f16x2(b[t] >> 16));
                }
            }
            // --- key scales, mask, running maximum (of scores before the positive factors qf) ---
            float vr[NT][2];  // e4m3: value scales of the lane's tokens
            float vmax = kLeastScale;
            if constexpr (KV == kKvE4m3) {
                const float* sck = reinterpret_cast<const float*>(stage + 2 * C::TILE);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const float2 kk = *reinterpret_cast<const float2*>(sck + t * 8 + 2 * c);
                    const float2 vv = *reinterpret_cast<const float2*>(sck + TT + t * 8 + 2 * c);
                    s[t][0] *= kk.x;
                    s[t][1] *= kk.y;
                    s[t][2] *= kk.x;
                    s[t][3] *= kk.y;
                    vr[t][0] = vv.x;
                    vr[t][1] = vv.y;
                    vmax = fmaxf(vmax, fmaxf(fabsf(vv.x), fabsf(vv.y)));
                }
            }
            const float room = kMostWeight - __log2f(vmax);  // for the tile's probabilities
            const uint32_t valid = *reinterpret_cast<const uint32_t*>(stage + 2 * C::TILE + C::SC);
            if (valid != kAllTokens) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (!((valid >> (t * 8 + 2 * c + (j & 1))) & 1u)) s[t][j] = -INFINITY;
            }
            float t0 = KV == kKvE4m3 ? -INFINITY : m0, t1 = KV == kKvE4m3 ? -INFINITY : m1;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                t0 = fmaxf(t0, fmaxf(s[t][0], s[t][1]));
                t1 = fmaxf(t1, fmaxf(s[t][2], s[t][3]));
            }
            t0 = fmaxf(t0, __shfl_xor_sync(kAllLanes, t0, 1));
            t1 = fmaxf(t1, __shfl_xor_sync(kAllLanes, t1, 1));
            t0 = fmaxf(t0, __shfl_xor_sync(kAllLanes, t0, 2));
            t1 = fmaxf(t1, __shfl_xor_sync(kAllLanes, t1, 2));
            float c0, c1;  // what a rescaling multiplies sums and accumulators by
            bool rescale;
            if constexpr (KV == kKvE4m3) {
                m0 = fmaxf(m0, t0);
                m1 = fmaxf(m1, t1);
                rescale = __any_sync(kAllLanes, fmaxf(fmaf(t0, qf0, -b0), fmaf(t1, qf1, -b1)) > room);
                if (rescale) {
                    // The power of two rises with the weights seen, not with the scales: a large scale
                    // without probability costs the others no bits.  A head of zeros, which the append stores
                    // with a scale of 1 however small the others are, has no weight.
                    bool one = false;
#pragma unroll
                    for (int t = 0; t < NT; ++t) one = one || vr[t][0] == 1.f || vr[t][1] == 1.f;
                    if (__any_sync(kAllLanes, one)) {
                        uint4 any = make_uint4(0, 0, 0, 0);
#pragma unroll 4
                        for (int i = 0; i < C::CH; ++i) {  // lane = token
                            const uint4 v = *reinterpret_cast<const uint4*>(stage + C::TILE + swz<C>(lane, i));
                            any.x |= v.x | v.y;
                            any.y |= v.z | v.w;
                        }
                        const uint32_t some = __ballot_sync(kAllLanes, ((any.x | any.y) & 0x7f7f7f7fu) != 0u);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                if (!((some >> (t * 8 + 2 * c + j)) & 1u)) vr[t][j] = 0.f;
                    }
                    float top0 = -INFINITY, top1 = -INFINITY;  // of the weights, in powers of two
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float v = __log2f(fabsf(vr[t][j]));
                            top0 = fmaxf(top0, fmaf(s[t][j], qf0, v));
                            top1 = fmaxf(top1, fmaf(s[t][2 + j], qf1, v));
                        }
                    top0 = fmaxf(top0, __shfl_xor_sync(kAllLanes, top0, 1));
                    top1 = fmaxf(top1, __shfl_xor_sync(kAllLanes, top1, 1));
                    top0 = fmaxf(top0, __shfl_xor_sync(kAllLanes, top0, 2));
                    top1 = fmaxf(top1, __shfl_xor_sync(kAllLanes, top1, 2));
                    // (rows without tokens, m = -inf, stay)
                    const float r0 = fmaxf(b0, fmaxf(top0 - kNewWeight, m0 * qf0 - kMostLift));
                    const float r1 = fmaxf(b1, fmaxf(top1 - kNewWeight, m1 * qf1 - kMostLift));
                    c0 = ex2_approx(b0 - r0);
                    c1 = ex2_approx(b1 - r1);
                    b0 = r0;
                    b1 = r1;
                }
            } else {
                // The sums stay about an older maximum until a score passes it by kSlack powers of two (one
                // warp-wide rescaling then): probabilities reach 2^kSlack, exact in the same number of bits.
                // (NaN, both -inf: no)
                rescale = __any_sync(kAllLanes, (t0 - m0) * qf0 > kSlack || (t1 - m1) * qf1 > kSlack);
                if (rescale) {
                    const float n0 = t0 == -INFINITY ? 0.f : t0 * qf0, n1 = t1 == -INFINITY ? 0.f : t1 * qf1;
                    c0 = ex2_approx(m0 * qf0 - n0);
                    c1 = ex2_approx(m1 * qf1 - n1);
                    b0 = n0 - kLift<KV>;
                    b1 = n1 - kLift<KV>;
                    m0 = t0;
                    m1 = t1;
                }
            }
            if (rescale) {
                l0 *= c0;
                l1 *= c1;
                ls[0] *= c0;
                ls[2] *= c1;
#pragma unroll
                for (int d = 0; d < DP / 8; ++d) {
                    o[d][0] *= c0;
                    o[d][1] *= c0;
                    o[d][2] *= c1;
                    o[d][3] *= c1;
                }
            }
            // --- probabilities (e4m3: weights), rounded to 16 bits for the second product; e4m3 caches sum
            // them before (fp32), 16-bit ones after (below) ---
            uint32_t pa[KT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float e[4];
                e[0] = ex2_approx(fmaf(s[t][0], qf0, -b0));
                e[1] = ex2_approx(fmaf(s[t][1], qf0, -b0));
                e[2] = ex2_approx(fmaf(s[t][2], qf1, -b1));
                e[3] = ex2_approx(fmaf(s[t][3], qf1, -b1));
                if constexpr (KV == kKvE4m3) {
                    l0 += e[0] + e[1];
                    l1 += e[2] + e[3];
                    e[0] *= vr[t][0];
                    e[1] *= vr[t][1];
                    e[2] *= vr[t][0];
                    e[3] *= vr[t][1];
                }
                pa[t >> 1][(t & 1) * 2] = pack2<F16>(e[0], e[1]);
                pa[t >> 1][(t & 1) * 2 + 1] = pack2<F16>(e[2], e[3]);
            }
            // --- O += P V ---
            if constexpr (KV != kKvE4m3) {
                // the sums (fp32) are of the rounded probabilities, P times a column of ones: a weight's
                // rounding then cancels where it dominates its row (relative error of a window of 128
                // tokens against 64 bits 2.2e-3 -> 2.0e-3, of which 1.7e-3 is the output type)
                constexpr uint32_t kOnes = F16 ? 0x3c003c00u : 0x3f803f80u;
#pragma unroll
                for (int t = 0; t < KT; ++t) mma16816<F16>(ls, pa[t], kOnes, kOnes);
                const int r = (lane & 7) + (((lane >> 3) & 1) << 3), hi = lane >> 4;
#pragma unroll
                for (int d = 0; d < KS; ++d) {
#pragma unroll
                    for (int t = 0; t < KT; ++t) {
                        uint32_t b[4];
                        ldsm4_t(vs_s + swz<C>(16 * t + r, 2 * d + hi), b);
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
                    ldsm4_t(vs_s + swz<C>(r, d), b);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t lo = __byte_perm(b[2 * k], 0, 0x3120), hi = __byte_perm(b[2 * k + 1], 0, 0x3120);
                        mma16816<F16>(o[2 * d], pa[k], e4m3x2_to_f16x2(lo), e4m3x2_to_f16x2(hi));
                        mma16816<F16>(o[2 * d + 1], pa[k], e4m3x2_to_f16x2(lo >> 16), e4m3x2_to_f16x2(hi >> 16));
                    }
                }
            }
            slot = slot + 1 == S ? 0 : slot + 1;
        }

        // --- the segment is done: the row, or the run's part of it ---
        b = row.b;
        h = row.h;
        starts = row.tile == 0;
        ends = row.tile + nseg == row.ntiles;
        rem -= nseg;
        pos += nseg;
        row.advance(p, nseg);
    }
}

// Joins the parts of rows cut by a run's border.  Job j: row j (by_row_join: its
// first and last run), or the row that run j continues as the first to do so.
// Parts: slot 1 of the first run, slot 0 of the runs that continue the row.  A job's
// head is the work of join_warps warps: a lane has 4 dims (two times 4 past 128)
// of every n-th part, and the lanes' running sums meet by shuffles, then in
// shared memory, always in the same order.  Bound by latency: the parts of 304 runs
// are 1 to 2.5 MB in L2, and the join takes 2 to 3 us behind the first kernel (6.8
// to 8.5 with cold caches).
constexpr int kJoinWarps = 8;  // per CTA

struct Sums {
    float m, l;
    float4 v[2];
};
// a += b, each about its own maximum
__device__ __forceinline__ void join(Sums& a, const Sums& b) {
    const float m = fmaxf(a.m, b.m);
    const float f = m == -INFINITY ? 0.f : ex2_approx(a.m - m), h = m == -INFINITY ? 0.f : ex2_approx(b.m - m);
    a.m = m;
    a.l = a.l * f + b.l * h;
    add_scaled(a.v[0], f, b.v[0], h);
    add_scaled(a.v[1], f, b.v[1], h);
}

template <bool QF16>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_kernel(AttendParams p) {
    __shared__ float s_ml[kJoinWarps][2];
    __shared__ __align__(16) float s_v[kJoinWarps][256];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = min(kAttRows, p.group);  // heads of a row
    const int item = (blockIdx.x * kJoinWarps + warp) / p.join_warps, sub = warp % p.join_warps;
    const int j = item / per, head = item - j * per;
    int run0 = -1, row = -1, nparts = 0;
    if (j < p.jobs) {
        if (p.by_row_join) {
            run0 = p.first[j];
            row = j;
            if (run0 >= 0) nparts = p.last[j] - run0 + 1;  // (not set where one run has the row)
        } else {
            row = p.cont[j];
            if (row >= 0 && p.cont[j - 1] != row) {  // run 0 starts a row: cont[0] is -1
                run0 = j - 1;
                nparts = 1;
                for (uint32_t same = kAllLanes; same == kAllLanes;) {
                    const int r = run0 + nparts + lane;
                    same = __ballot_sync(kAllLanes, r < p.runs && p.cont[r] == row);
                    nparts += same == kAllLanes ? 32 : __ffs(~same) - 1;
                }
            }
        }
    }
    const int b = nparts ? row / p.rows_per_seq : 0, h = nparts ? row - b * p.rows_per_seq : 0;
    const int hb = h % p.head_blocks, head0 = (h / p.head_blocks) * p.group + hb * kAttRows;
    if (head >= p.group - hb * kAttRows) nparts = 0;  // a last block of fewer heads
    const int psize = kAttRows * (p.D + 2);
    // lanes of a part: a power of two of 4 dims each, at most the warp
    const int lp = p.D <= 16 ? 4 : p.D <= 32 ? 8 : p.D <= 64 ? 16 : 32;
    const int d = (lane & (lp - 1)) * 4, splits = (32 / lp) * p.join_warps, at = sub * (32 / lp) + lane / lp;
    Sums a = {-INFINITY, 0.f, {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)}};
#pragma unroll 4
    for (int i = at; i < nparts; i += splits) {
        const float* q = p.partial + ((long long)(run0 + i) * 2 + (i == 0 ? 1 : 0)) * psize;
        const float2 ml = *reinterpret_cast<const float2*>(q + 2 * head);
        const float* src = q + 2 * kAttRows + head * p.D + d;
        Sums x = {ml.x, ml.y, {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)}};
        if (d < p.D) x.v[0] = *reinterpret_cast<const float4*>(src);
        if (d + 128 < p.D) x.v[1] = *reinterpret_cast<const float4*>(src + 128);
        join(a, x);
    }
    for (int o = lp; o < 32; o <<= 1) {
        Sums x;
        x.m = __shfl_xor_sync(kAllLanes, a.m, o);
        x.l = __shfl_xor_sync(kAllLanes, a.l, o);
        x.v[0] = make_float4(__shfl_xor_sync(kAllLanes, a.v[0].x, o), __shfl_xor_sync(kAllLanes, a.v[0].y, o),
                             __shfl_xor_sync(kAllLanes, a.v[0].z, o), __shfl_xor_sync(kAllLanes, a.v[0].w, o));
        x.v[1] = a.v[1];  // only past 128 dims, where a part takes the warp
        join(a, x);
    }
    if (p.join_warps > 1) {
        if (lane == 0) s_ml[warp][0] = a.m, s_ml[warp][1] = a.l;
        if (lane < lp && d < p.D) *reinterpret_cast<float4*>(&s_v[warp][d]) = a.v[0];
        if (d + 128 < p.D) *reinterpret_cast<float4*>(&s_v[warp][d + 128]) = a.v[1];
        __syncthreads();
        if (sub == 0 && d < p.D)
            for (int w = 1; w < p.join_warps; ++w) {
                const float* v = s_v[warp + w] + d;
                Sums x = {s_ml[warp + w][0], s_ml[warp + w][1], {*reinterpret_cast<const float4*>(v), a.v[1]}};
                if (d + 128 < p.D) x.v[1] = *reinterpret_cast<const float4*>(v + 128);
                join(a, x);
            }
    }
    if (nparts && sub == 0 && lane < lp) {
        const float w = final_weight(p.sinks, head0 + head, a.m, a.l);
        uint16_t* dst = p.out + b * p.o_token + (long long)(head0 + head) * p.o_head + d;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (d + 128 * k < p.D) {
                *reinterpret_cast<uint32_t*>(dst + 128 * k) = pack2<QF16>(a.v[k].x * w, a.v[k].y * w);
                *reinterpret_cast<uint32_t*>(dst + 128 * k + 2) = pack2<QF16>(a.v[k].z * w, a.v[k].w * w);
            }
    }
}

namespace {

int dp_of(int D) { return D <= 64 ? 64 : D <= 96 ? 96 : D <= 128 ? 128 : 256; }

template <int DP, int KV, bool QF16, int MODE, bool LIGHT>
cudaError_t launch_attend_m(const AttendParams& p, int grid, cudaStream_t st) {
    using C = AttCfg<DP, KV, LIGHT>;
    static_assert(C::SMEM * C::CTAS <= 226 * 1024, "shared memory of the resident CTAs");
    const auto kernel = attend_kernel<DP, KV, QF16, MODE, LIGHT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(grid), dim3(kAttWarps * 32), C::SMEM, st, p);
}
template <int DP, int KV, bool QF16>
cudaError_t launch_attend_t(const AttendParams& p, const AttendPlan& w, cudaStream_t st) {
    if constexpr (DP == 64 && KV != kKvE4m3) {
        if (w.light)
            return w.mode == kRows ? launch_attend_m<DP, KV, QF16, kRows, true>(p, w.ctas, st)
                                   : launch_attend_m<DP, KV, QF16, kTeam, true>(p, w.ctas, st);
    }
    return w.mode == kRows   ? launch_attend_m<DP, KV, QF16, kRows, false>(p, w.ctas, st)
           : w.mode == kTeam ? launch_attend_m<DP, KV, QF16, kTeam, false>(p, w.ctas, st)
                             : launch_attend_m<DP, KV, QF16, kRuns, false>(p, w.ctas, st);
}
template <int KV, bool QF16>
cudaError_t launch_attend_d(const AttendParams& p, const AttendPlan& w, cudaStream_t st) {
    switch (dp_of(p.D)) {
        case 64: return launch_attend_t<64, KV, QF16>(p, w, st);
        case 96: return launch_attend_t<96, KV, QF16>(p, w, st);
        case 128: return launch_attend_t<128, KV, QF16>(p, w, st);
        default: return launch_attend_t<256, KV, QF16>(p, w, st);
    }
}

}  // namespace

// The workspace is for the parts of cut rows.
void attend_plan(int B, int Hq, int Hkv, int D, bool e4m3, int most, int sms, AttendPlan* w) {
    const int dp = dp_of(D);
    const long long rows = (long long)B * Hkv * ((Hq / Hkv + kAttRows - 1) / kAttRows);
    const int ctas = sms * ctas_per_sm(dp, e4m3, false), light_ctas = sms * ctas_per_sm(dp, e4m3, true);
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    auto tiles = [&](bool light) {
        const int tt = tile_tokens(dp, e4m3, light);
        return (long long)((most + tt - 1) / tt);
    };
    auto waves = [&](long long n) { return (rows + n * kAttWarps - 1) / (n * kAttWarps); };
    w->mode = kRuns;
    w->light = false;
    w->ctas = ctas;
    if (most <= kWholeTokens) {
        if (rows <= ctas) {
            if (tiles(false) * (ctas - rows) <= (long long)kTeamTiles * ctas) w->mode = kTeam;
        } else if (rows <= light_ctas) {
            w->mode = kTeam;
            w->light = true;
        }
        if (w->mode == kTeam) {
            w->ctas = (int)rows;
        } else {
            // twice the warps at half the speed: 2048 rows of 128 tokens 14.8 us light, 16.2 not (one
            // wave against two), 1024 rows 10.0, 8.1 (one against one)
            const bool light = light_ctas > ctas && 2 * waves(light_ctas) <= waves(ctas);
            const int n = light ? light_ctas : ctas;
            if (rows_fit(tiles(light), rows, n, kRowTiles, light || dp == 256 ? 2 : 1)) {
                w->mode = kRows;
                w->light = light;
                w->ctas = n;
            }
        }
    }
    const int runs = ctas;
    w->runs = runs;
    w->by_row_join = rows <= runs;
    w->cont = 0;
    w->first = up((size_t)runs * 4);
    w->last = w->first + up((size_t)(rows <= runs ? rows : 1) * 4);
    w->partial = w->last + up((size_t)(rows <= runs ? rows : 1) * 4);
    w->total = w->mode != kRuns ? 0 : w->partial + (size_t)runs * 2 * kAttRows * (D + 2) * 4;
}

cudaError_t launch_attend(const AttendParams& p_in, const AttendPlan& w, int kv_dtype, bool fp16, void* workspace,
                          cudaStream_t st) {
    AttendParams p = p_in;
    const bool e4m3 = kv_dtype == kDtE4m3;
    p.runs = w.runs;
    p.group = p.Hq / p.Hkv;
    p.head_blocks = (p.group + kAttRows - 1) / kAttRows;
    p.rows_per_seq = p.Hkv * p.head_blocks;
    p.page16 = p.page_size % 16 == 0;
    p.page_shift = -1;
    if ((p.page_size & (p.page_size - 1)) == 0)
        for (p.page_shift = 0; (1 << p.page_shift) < p.page_size;) ++p.page_shift;
    const long long rows = (long long)p.B * p.rows_per_seq;
    if (w.total) {
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        p.by_row_join = w.by_row_join;
        p.cont = reinterpret_cast<int32_t*>(ws + w.cont);
        p.first = reinterpret_cast<int32_t*>(ws + w.first);
        p.last = reinterpret_cast<int32_t*>(ws + w.last);
        p.partial = reinterpret_cast<float*>(ws + w.partial);
    }
    cudaError_t e;
    if (e4m3)
        e = fp16 ? launch_attend_d<kKvE4m3, true>(p, w, st) : launch_attend_d<kKvE4m3, false>(p, w, st);
    else
        e = fp16 ? launch_attend_d<kKvFp16, true>(p, w, st) : launch_attend_d<kKvBf16, false>(p, w, st);
    if (e != cudaSuccess || w.mode != kRuns) return e;
    // warps per head by the parts that a row can have on average
    const int heads = p.group < kAttRows ? p.group : kAttRows;
    p.jobs = p.by_row_join ? (int)rows : p.runs;
    p.join_warps = 1;
    while (p.join_warps < kJoinWarps && (long long)p.join_warps * 8 * p.jobs <= p.runs) p.join_warps *= 2;
    const dim3 jg((unsigned)(((long long)p.jobs * heads * p.join_warps + kJoinWarps - 1) / kJoinWarps));
    return fp16 ? launch_pdl(attend_join_kernel<true>, jg, dim3(kJoinWarps * 32), 0, st, p)
                : launch_pdl(attend_join_kernel<false>, jg, dim3(kJoinWarps * 32), 0, st, p);
}

}  // namespace moe
