// Attention of a step's drafted tokens over a paged key-value cache: each sequence
// has a few drafts that form a tree (or a chain) behind its context, their keys and
// values already in the cache, and every draft sees the context, its ancestors and
// itself ("GPT-OSS on Day 0", perplexity.ai hub blog: grouped heads, sink attention,
// sliding windows).
//
//   draft i of n, depth d_i, context of c tokens: sees token t < c if t > c + d_i - window,
//   and draft j (token c + j) if j is i or an ancestor and d_i - d_j < window
//   o = sum_t p_t v_t / (sum_t p_t + 2^(sink log2 e - m)),  p_t = 2^(s_t - m),
//   s_t = (q . k_t) scale log2 e
//
// Drafts and query heads share a key, so the rows of the products are the n x group
// (draft, head) pairs: 128 of them are the rows of a tcgen05 tile.  A key is read once for
// 256 rows (two row tiles), or for 128 with more than 128 dims or where the batch's
// sequences have at most 128 on average.  S = Q K^T goes to tensor memory, where a thread has a whole row: no
// exchange for maximum and sum.  Probabilities go back in 16 bits beside the scores and
// are the first operand of P V, whose sums stay in tensor memory; they are rescaled only
// when a row's maximum rises by more than 2^kSlack, after its first time by a whole power of
// two, so that probabilities are rounded once.
//
// One CTA: a warp that issues the products, a warp that copies keys and values by TMA
// (pieces of tokens that lie on one page), warps that turn e4m3 codes into fp16, and a
// warpgroup for each row tile.  Pages of which 8 is no divisor are copied 16 bytes a
// thread, by as many warps.  One row tile: two score buffers, so that the next scores are
// there when the exponentials of the last are done.  Two row tiles (more than 128 rows)
// share the keys and values in shared memory, and their scores are made anew as soon as
// a row tile has read its own.
//
// A wait on a barrier takes 100 to 150 cycles even when it has come, so there are few: one
// for a tile's keys and values, one for its scores, one for its probabilities.
//
// Measured (one GB300): chains of 4 drafts of 64 heads on 8 of 64, 64 sequences of 1 to
// 16384 tokens: 176 us for 1.08 GB, 6.1 TB/s, 90 % of a copy. Trees of 48 to 64 drafts of
// the same heads, 32 sequences of 2000 to 8192 tokens: 236 us, 635 TFLOP/s; two row tiles
// are in turn at their exponentials, 3.1 thousand cycles for 128 tokens of 256 rows where the
// exponential unit needs 1.0 (without softmax 143 us). 16 drafts of 64 heads on 4 of 128, 4
// sequences of 100000 to 131072 tokens, e4m3: 286 us, 845 TFLOP/s, bound by conversion and
// exponentials together (without softmax 245 us). A window of 128 over 256 sequences: 44.8
// us, a tile's and a row end's latency after another. One short sequence: 7.0 us.
// One row tile for all: 239 and 446 us for the two wide cases. Copies by threads, which pages
// of odd sizes take: 286, 322, 304 and 54 us for these four.
//
// e4m3 caches with few rows stay behind bf16 ones of the same shape (8 rows, 32 sequences of 8000
// tokens, 8 key heads of 64: 122 us, bf16 92): a warp converts the codes of 32 tokens by itself.
//
// A value that is infinite or NaN makes NaN of its product with a weight of 0, so a draft's would
// reach its siblings, and that of a window's first token those that have passed it.  A row's end
// looks whether its sums are finite (windows 43.8 -> 44.3 us, one short sequence 6.8 -> 7.0); if some are
// not, the CTA ends with tree_mend, which computes the rows anew that such a value spoilt. A look at every
// value of the tiles that hold such tokens took 51 us for the windows, 304 for the e4m3 case, a second
// run of the CTA with that look where it is needed, 45 and 296: registers of the common path.
//
// The list of items (sequence, key head, row tiles) and their token tiles is cut into
// equal runs, one per CTA; an item cut by a run's border leaves fp32 parts that a second,
// dependent launch joins in a fixed order.
#pragma once
#include <type_traits>

#include "moe_attend.cuh"
#include "moe_internal.h"

namespace moe {

constexpr int kTreeRows = 128;  // rows of a tile
// Token tiles of a run, at least, where there are so many (8: one sequence of 1000 tokens 24.4 us for 20.0; 2: the same).
constexpr int kMinTiles = 4;
// What an item costs beside its tiles (queries, the place in the tree, the row's end), in tiles: runs are cut into
// equal sums of both.  (1: ragged lengths up to 16384 204 us, up to 3000 35; 4: 182 and 28; 2: 196; 8: 180, wide trees
// +2 %.)
constexpr int kItemTiles = 4;
// What cutting items adds to every run beside a second item's cost (parts written, the join), in tiles: items stay whole
// where equal numbers of them take no longer.  (16 sequences of 1000 and 2000 tokens, 8 key heads of 128: cut 33.8 and
// 49.0 us, whole 21.0 and 36.0; one sequence: cut 20.0 and 22.1, whole 19.6 and 31.6.  3 cuts 64 sequences of 500: 59.4
// us for 53.3; 12 leaves one of 2000 with 256 rows whole: 32.9 for 24.1.)
constexpr int kCutTiles = 7;
// Tables for so few tiles are never cut, so without workspace and join: 64 sequences of 500 tokens 22.4 us, cut 24.7;
// one short sequence 7.5, cut 14.0.
constexpr int kWholeTiles = 8;

// KV: the cache's type; TILES: row tiles of a CTA; TMA: copies by tensor maps.
template <int DP, int KV, int TILES, bool TMA>
struct TreeCfg {
    static constexpr bool E4M3 = KV == kKvE4m3;
    static constexpr int TT = DP == 256 ? 32 : TILES == 2 && DP == 64 ? 128 : 64;  // tokens of a tile
    static constexpr int CTAS = TILES == 1 && DP == 64 ? 2 : 1;
    // warps: row tiles, then those that copy or convert (a token a lane), a TMA warp, the products' warp
    static constexpr int LOADERS = E4M3 || !TMA ? TT / 32 : 0;
    static constexpr int TMA_WARP = TILES * 4 + LOADERS, MMA_WARP = TMA_WARP + (TMA ? 1 : 0);
    static constexpr int THREADS = (MMA_WARP + 1) * 32;
    // scores that a thread works on at a time, by its registers
    static constexpr int WARPS_EACH = ((MMA_WARP + 1) * CTAS + 3) / 4;  // of a scheduler
    static constexpr int WIDE = TT < 64 || WARPS_EACH > 3 ? 32 : 64;
    static constexpr int Q_TILE = kTreeRows * DP * 2;
    static constexpr int KV_TILE = TT * DP * 2;     // 16-bit keys (or values) of a token tile
    static constexpr int RAW_TILE = TT * DP;        // their codes
    static constexpr int STAGE = 2 * KV_TILE;       // keys, values
    // stages of keys and values: as many as fit (one row tile, 16 bits: 5 where 4 took 181 us, now 176, for the 1.08 GB of
    // 64 sequences of up to 16384 tokens)
    static constexpr int NS = E4M3 ? 3 : DP == 64 || (DP == 128 && TILES == 1) ? 5 : 4;
    // the raw codes' ring; by threads also scales and valid tokens
    static constexpr int NR = !E4M3 ? 0 : DP == 64 && TILES == 2 ? 4 : DP == 64 && !TMA ? 2 : 3;
    static constexpr int RAW_STAGE = 2 * RAW_TILE + (TMA ? 0 : 2 * TT * 4 + 16);
    // what the softmax knows of a tile: valid tokens; e4m3: each loading warp's largest value scale, scales
    static constexpr int META = E4M3 ? 32 + 2 * TT * 4 : 32;
    static constexpr int ANC = TILES * kTreeRows * (kMaxDrafts / 32) * 4;
    // Few rows of e4m3 caches stand 2 or 4 times in their tile, each copy with a part of the tokens, so that conversion
    // and exponentials share the schedulers evenly (8 rows, 32 sequences of 8000 tokens, 8 key heads of 64: 122 us, once
    // each 127). 16-bit caches have them once (a window of 128 over 256 sequences: 44.8 us, four times 50.7).
    // Where the copies meet: each one's sums in fp32, over the queries and behind them.
    static constexpr bool COPIES = E4M3 && TILES == 1 && TT == 64;
    static constexpr int MEET = COPIES ? kTreeRows * DP * 4 - Q_TILE : 0;
    static constexpr int Q_AT = 0;
    static constexpr int KV_AT = TILES * Q_TILE + MEET;
    static constexpr int RAW_AT = KV_AT + NS * STAGE;
    static constexpr int META_AT = RAW_AT + NR * RAW_STAGE;
    static constexpr int ANC_AT = META_AT + NS * META;
    static constexpr int SMEM = ANC_AT + ANC + 1024;  // (aligned to 1024 in the kernel)
    // tensor memory: two score buffers (a row tile's own, or in turn), the sums of each row tile, two of
    // probabilities (16 bits)
    static constexpr int O_AT = 2 * TT, P_AT = O_AT + TILES * DP;
    static constexpr int COLS = P_AT + TT <= 256 ? 256 : 512;
};

struct TreeSeq {
    int first;         // first row of q
    int n, len, ctx;   // drafts, tokens, tokens before the drafts
    int lo;            // first token that any draft sees
    int start, ntiles; // first token of the first tile (a multiple of 16), token tiles
    int rtiles;        // row tiles (of TILES * 128 rows)
};

template <int TT, int TILES>
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int b) {
    TreeSeq s;
    const int lo = __ldg(p.starts + b), hi = __ldg(p.starts + b + 1), raw = __ldg(p.lengths + b);
    const bool fine = lo >= 0 && hi >= lo && hi <= p.N && hi - lo <= kMaxDrafts;
    s.first = lo;
    s.n = fine ? hi - lo : 0;
    s.len = min(max(raw, 0), p.max_tokens);
    s.ctx = max(s.len - s.n, 0);
    if ((!fine || s.len != raw || s.len < s.n) && p.status) atomicOr(p.status, kErrBadIndex);
    s.lo = p.window > 0 && s.ctx >= p.window ? s.ctx - p.window + 1 : 0;
    s.start = s.lo & ~15;
    s.ntiles = max(1, (int)((unsigned)(s.len - s.start + TT - 1) / TT));
    s.rtiles = (s.n * p.group + TILES * kTreeRows - 1) / (TILES * kTreeRows);
    return s;
}

// Where a run begins, and what it has: token tiles and items' costs, or items where they are not cut.
struct TreeWork {
    int b, h, rt, tile;
    int lead, rem;  // what the item costs before its first tile; what the run has left, of both
};
// A part of an item: token tiles [tile, tile + n) of it.
struct TreeSeg {
    TreeSeq s;
    int b, h, rt, tile, n;
    bool starts, ends;
};

// Where a run is: the sequence of its next part, and what is left.
struct TreeWalk {
    TreeWork w;
    TreeSeq s;
};
// The next part of the run; false: none.
template <int TT, int TILES>
__device__ __forceinline__ bool tree_next(const TreeParams& p, bool whole, TreeWalk& k, TreeSeg& g) {
    TreeWork& w = k.w;
    const int have = w.rem - w.lead;  // (none: the next run begins the item)
    if (have <= 0) return false;
    const int left = k.s.ntiles - w.tile;
    g.s = k.s;
    g.b = w.b;
    g.h = w.h;
    g.rt = w.rt;
    g.tile = w.tile;
    g.n = whole || left < have ? left : have;
    g.starts = w.tile == 0;
    g.ends = g.n == left;
    w.rem = have - (whole ? 1 : g.n);
    w.lead = whole ? 0 : kItemTiles;
    w.tile += g.n;
    if (g.ends) {
        w.tile = 0;
        if (++w.rt == k.s.rtiles) {
            w.rt = 0;
            if (++w.h == p.Hkv) {
                w.h = 0;
                while (w.rem > 0) {
                    if (++w.b >= p.B) {  // (starts that descend can make sums of work that overflow)
                        w.rem = 0;
                        break;
                    }
                    k.s = tree_seq<TT, TILES>(p, w.b);
                    if (k.s.rtiles) break;
                }
            }
        }
    }
    return true;
}

// A place in a ring of N stages.
template <int N>
struct TreeRing {
    int at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++at == N) at = 0, phase ^= 1u;
    }
};

// Draft of row `at` of a sequence (rounded once, and far from a border: rows are below 2^20).
__device__ __forceinline__ int tree_draft(const TreeParams& p, int at) { return (int)(((float)at + 0.5f) * p.inv_group); }

// Bits lo and on of 32.
__device__ __forceinline__ uint32_t bits_from(int lo) { return lo <= 0 ? kAllLanes : lo >= 32 ? 0u : kAllLanes << lo; }

// Byte of 16-byte chunk c of row r in a block of `rows` rows: blocks of 64 values a row, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_at(int rows, int r, int c) {
    return (uint32_t)((c >> 3) * rows * 128 + r * 128 + ((c ^ r) & 7) * 16);
}

// Rows of the CTA's run whose sums are not finite because of a value that other rows see and they do not (a draft of
// another branch, a token before their window): computed anew, a warp each, in fp32, over what they see.  All of the CTA's
// threads, seldom, and no faster than it has to be (one such draft in each of 64 sequences of 8000 tokens, 4 drafts of 8
// heads: 10 ms for 0.19; a bad value that all rows see: 0.22).
template <int KV, int TT, int TILES>
static __device__ __noinline__ void tree_mend(const TreeParams& p, const TreeWork* work, bool whole) {
    constexpr bool E4M3 = KV == kKvE4m3;
    constexpr int ROWS = TILES * kTreeRows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int group = 2;  // lanes that have a token's dims, 8 each
    while (group * 8 < p.D) group *= 2;
    const int groups = 32 / group, ch = lane % group;
    const bool in = ch * 8 < p.D;
    const bool qf16 = E4M3 ? p.fp16 : KV == kKvFp16;
    TreeWalk walk;
    TreeSeg g;
    walk.w = *work;
    if (walk.w.rem > 0) walk.s = tree_seq<TT, TILES>(p, walk.w.b);
    auto wide = [](uint16_t v, bool f16) { return f16 ? unpack2<true>(v).x : unpack2<false>(v).x; };
#pragma unroll 1
    while (tree_next<TT, TILES>(p, whole, walk, g)) {
        const TreeSeq& s = g.s;
        const bool done = g.starts && g.ends;
        const int rows = min(ROWS, s.n * p.group - g.rt * ROWS);
        const int t_end = min(s.start + (g.tile + g.n) * TT, s.len), t_begin = max(s.start + g.tile * TT, s.lo);
        // tokens from here to the context's end are seen by all rows
        const int edge = p.window > 0 ? s.ctx + s.n - p.window : 0;
        float* part = p.partial + ((long long)blockIdx.x * 2 + (g.starts ? 1 : 0)) * (ROWS * (p.D + 2));
#pragma unroll 1
        for (int row = warp; row < rows; row += warps) {
            const int at = g.rt * ROWS + row, draft = tree_draft(p, at), head = g.h * p.group + at - draft * p.group;
            uint16_t* dst = p.out + (s.first + draft) * p.o_token + (long long)head * p.o_head;
            auto sum = [&](int d) { return part + 2 * ROWS + ((d / 4) * ROWS + row) * 4 + d % 4; };
            bool odd = false;
            for (int d = lane; d < p.D; d += 32) odd = odd || !isfinite(done ? wide(dst[d], qf16) : *sum(d));
            if (!__any_sync(kAllLanes, odd)) continue;
            // the draft's place; ancestors, and itself: 32 of them a lane
            uint32_t path = 0;
            int depth = -1;
#pragma unroll 1
            for (int a = draft; a >= 0;) {
                ++depth;
                if (a >> 5 == lane && (p.window <= 0 || depth < p.window)) path |= 1u << (a & 31);
                const int up = p.parents ? __ldg(p.parents + s.first + a) : a - 1;
                a = up < a && up >= -1 ? up : -1;
            }
            const int since = p.window > 0 ? s.ctx + depth - p.window + 1 : 0;
            // a lane has a token: its page (-1: none, or out of range), whether the row sees it
            auto page = [&](int t) {
                const int pid = t < t_end ? __ldg(p.table + (long long)g.b * p.table_ld + t / p.page_size) : -1;
                return (uint32_t)pid < (uint32_t)p.num_pages ? pid : -1;
            };
            auto sees = [&](int t) {
                const int o = t - s.ctx;
                const uint32_t word = __shfl_sync(kAllLanes, path, (o >> 5) & 31);
                return o < 0 ? t >= since : o < kMaxDrafts && ((word >> (o & 31)) & 1u);
            };
            auto scale = [&](const float* of, int pid, int t) {
                if constexpr (!E4M3) return 1.f;
                return __ldg(of + pid * p.cache.s_page + g.h * p.cache.s_head + t % p.page_size * p.cache.s_token);
            };
            auto k_at = [&](int pid, int t) {
                return pid * p.cache.k_page + g.h * p.cache.k_head + t % p.page_size * p.cache.k_token;
            };
            auto v_at = [&](int pid, int t) {
                return pid * p.cache.v_page + g.h * p.cache.v_head + t % p.page_size * p.cache.v_token;
            };
            auto load8 = [&](const void* of, long long i, float (&y)[8]) {
                uint32_t u[4];
                if constexpr (E4M3) {
                    const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(of) + i);
                    u[0] = e4m3x2_to_f16x2(c.x), u[1] = e4m3x2_to_f16x2(c.x >> 16);
                    u[2] = e4m3x2_to_f16x2(c.y), u[3] = e4m3x2_to_f16x2(c.y >> 16);
                } else {
                    const uint4 c = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(of) + i);
                    u[0] = c.x, u[1] = c.y, u[2] = c.z, u[3] = c.w;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x = unpack2<KV != kKvBf16>(u[j]);
                    y[2 * j] = x.x, y[2 * j + 1] = x.y;
                }
            };
            odd = false;
#pragma unroll 1
            for (int t0 = t_begin; t0 < t_end; t0 += 32) {
                if (t0 >= edge && t0 + 32 <= s.ctx) {  // (all are seen)
                    t0 += (s.ctx - t0) / 32 * 32 - 32;
                    continue;
                }
                const int t = t0 + lane, pid = page(t);
                if (sees(t) || pid < 0) continue;
                odd = odd || !isfinite(scale(p.cache.v_scale, pid, t));
#pragma unroll 1
                for (int d = 0; d < p.D; d += 8) {
                    float y[8];
                    load8(p.cache.v, v_at(pid, t) + d, y);
#pragma unroll
                    for (int j = 0; j < 8; ++j) odd = odd || !isfinite(y[j]);
                }
            }
            if (!__any_sync(kAllLanes, odd)) continue;
            // over what it sees, 32 tokens at a time: groups of lanes take a token's key, then its value, 8 dims a lane
            const float factor = p.q_sign ? -p.scale_log2 : p.scale_log2;
            float m = -INFINITY, l = 0.f, x[8] = {}, acc[8] = {};  // l: the lane's part
            if (in) {
                const uint4 c = *reinterpret_cast<const uint4*>(p.q + (s.first + draft) * p.q_token +
                                                                (long long)head * p.q_head + 8 * ch);
                const uint32_t u[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 y = qf16 ? unpack2<true>(u[j]) : unpack2<false>(u[j]);
                    x[2 * j] = y.x, x[2 * j + 1] = y.y;
                }
            }
#pragma unroll 1
            for (int t0 = t_begin; t0 < t_end; t0 += 32) {
                const int t = t0 + lane, pid = page(t);
                const bool seen = sees(t) && pid >= 0;
                const uint32_t any = __ballot_sync(kAllLanes, seen);
                const long long k = seen ? k_at(pid, t) : 0, v = seen ? v_at(pid, t) : 0;
                float y = 0.f;
#pragma unroll 4
                for (int i = 0; i < group; ++i) {
                    float z[8] = {}, r = 0.f;
                    const long long at = __shfl_sync(kAllLanes, k, i * groups + lane / group);
                    if (in) load8(p.cache.k, at + 8 * ch, z);  // (of the first token where none is seen)
#pragma unroll
                    for (int j = 0; j < 8; ++j) r = fmaf(x[j], z[j], r);
                    for (int o = group / 2; o; o >>= 1) r += __shfl_xor_sync(kAllLanes, r, o);
                    r = __shfl_sync(kAllLanes, r, lane % groups * group);
                    if (lane / groups == i) y = r;
                }
                y = seen ? y * (scale(p.cache.k_scale, pid, t) * factor) : -INFINITY;
                float n = y;
#pragma unroll
                for (int o = 16; o; o >>= 1) n = fmaxf(n, __shfl_xor_sync(kAllLanes, n, o));
                n = fmaxf(m, n);
                const float f = m == -INFINITY ? 0.f : ex2_approx(m - n), e = y == -INFINITY ? 0.f : ex2_approx(y - n);
                const float w = seen ? e * scale(p.cache.v_scale, pid, t) : 0.f;
                m = n;
                l = l * f + e;
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] *= f;
#pragma unroll 4
                for (int i = 0; i < group; ++i) {
                    const int from = i * groups + lane / group;
                    float z[8] = {};
                    const long long at = __shfl_sync(kAllLanes, v, from);
                    const float h = __shfl_sync(kAllLanes, w, from);
                    if (in) load8(p.cache.v, at + 8 * ch, z);
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[j] = (any >> from) & 1u ? fmaf(h, z[j], acc[j]) : acc[j];
                }
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(kAllLanes, l, o);
            for (int o = 16; o >= group; o >>= 1)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] += __shfl_xor_sync(kAllLanes, acc[j], o);
            const float fw = done ? final_weight(p.sinks, head, m, l) : 1.f;
            if (!done && lane == 0) reinterpret_cast<float2*>(part)[row] = make_float2(m, l);
            if (in && lane < group)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (done)
                        dst[8 * ch + j] = (uint16_t)(qf16 ? pack2<true>(acc[j] * fw, 0.f) : pack2<false>(acc[j] * fw, 0.f));
                    else
                        *sum(8 * ch + j) = acc[j];
                }
        }
    }
}

template <int DP, int KV, int TILES, bool TMA>
__global__ void __launch_bounds__(TreeCfg<DP, KV, TILES, TMA>::THREADS, TreeCfg<DP, KV, TILES, TMA>::CTAS)
    tree_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const __grid_constant__ TreeParams p) {
    using C = TreeCfg<DP, KV, TILES, TMA>;
    constexpr bool E4M3 = C::E4M3, F16 = KV != kKvBf16;  // F16: type of the products
    const bool qf16 = E4M3 ? p.fp16 : F16;               // of q and out
    constexpr int TT = C::TT, NS = C::NS, NR = C::NR ? C::NR : 1, THREADS = C::THREADS;
    constexpr int kFillers = C::LOADERS ? C::LOADERS : 1;  // arrivals that fill a stage
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[NS], empty_bar[NS], q_bar[TILES], s_bar[2], p_bar[2], o_bar[TILES], end_bar,
        raw_full_bar[NR], raw_empty_bar[NR], read_bar[TILES], x_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag, s_sum[3];  // (all runs': units, items, tiles of the longest)
    __shared__ int s_odd;                 // a row's sums were not finite
    __shared__ TreeWork s_work;
    __shared__ float s_qf[TILES][kTreeRows];
    __shared__ int16_t s_up[TILES][kMaxDrafts];  // parents
    __shared__ float2 s_ml[TILES == 1 ? kTreeRows : 1];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t smem_s = smem_u32(smem);
    int* s_pre = reinterpret_cast<int*>(smem);  // [THREADS + 1], before the tiles come

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(smem_u32(&full_bar[i]), kFillers);
            mbar_init(smem_u32(&empty_bar[i]), 1);
        }
        for (int i = 0; i < NR; ++i) {
            mbar_init(smem_u32(&raw_full_bar[i]), 1);
            mbar_init(smem_u32(&raw_empty_bar[i]), kFillers);
        }
        for (int i = 0; i < TILES; ++i) {
            mbar_init(smem_u32(&q_bar[i]), kTreeRows);
            mbar_init(smem_u32(&o_bar[i]), 1);
            mbar_init(smem_u32(&read_bar[i]), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&s_bar[i]), 1);
            mbar_init(smem_u32(&p_bar[i]), 4);
        }
        mbar_init(smem_u32(&end_bar), 1);
        mbar_init(smem_u32(&x_bar), kTreeRows);
        abort_flag = s_odd = 0;
        fence_barrier_init();
    }
    if (warp == C::MMA_WARP) tmem_alloc(smem_u32(&tmem_slot), C::COLS);
    pdl_wait();
    pdl_allow_dependents();

    // --- the run: each thread counts a slice of the sequences ---
    const int slice = (p.B + THREADS - 1) / THREADS;
    if (tid < 3) s_sum[tid] = 0;
    __syncthreads();
    int mine = 0, items = 0, longest = 0;
#pragma unroll 1
    for (int i = 0; i < slice; ++i) {
        const int b = tid * slice + i;
        if (b < p.B) {
            const TreeSeq s = tree_seq<TT, TILES>(p, b);
            items += p.Hkv * s.rtiles;
            mine += p.Hkv * s.rtiles * (s.ntiles + kItemTiles);
            if (s.rtiles) longest = max(longest, s.ntiles);
        }
    }
    const int warp_units = __reduce_add_sync(kAllLanes, mine), warp_items = __reduce_add_sync(kAllLanes, items);
    longest = __reduce_max_sync(kAllLanes, longest);
    if (lane == 0) {
        atomicAdd(&s_sum[0], warp_units);
        atomicAdd(&s_sum[1], warp_items);
        atomicMax(&s_sum[2], longest);
        if (warp == 0) s_pre[0] = 0;
    }
    __syncthreads();
    bool whole = p.whole;
    if (!whole) {
        const int least = kMinTiles + kItemTiles, n = min((s_sum[0] + least - 1) / least, p.runs);
        const float each = (float)((s_sum[1] + p.runs - 1) / p.runs) * (float)(s_sum[2] + kItemTiles);
        whole = each <= (float)s_sum[0] / (float)max(n, 1) + (float)(kItemTiles + kCutTiles);
    }
    s_pre[tid + 1] = whole ? items : mine;
    __syncthreads();
    if (warp == 0) {  // prefix sums, 32 at a time
        int before = 0;
        const int slices = (p.B + slice - 1) / slice;
#pragma unroll 1
        for (int base = 0; base < slices; base += 32) {
            int v = s_pre[base + lane + 1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(kAllLanes, v, o);
                if (lane >= o) v += u;
            }
            v += before;
            s_pre[base + lane + 1] = v;
            before = __shfl_sync(kAllLanes, v, 31);
        }
        __syncwarp();
        const int least = whole ? 1 : kMinTiles + kItemTiles;
        const int total = before, n = min((total + least - 1) / least, p.runs), run = blockIdx.x;
        TreeWork w = {0, 0, 0, 0, 0, 0};
        if (run < n) {
            const int most = total / n, more = total - most * n, from = more * run / n;  // (n is small)
            int u = most * run + from;
            w.rem = most + more * (run + 1) / n - from;
            int sl = 0;
#pragma unroll 1
            for (int base = 0; base < slices; base += 32)
                sl += __popc(__ballot_sync(kAllLanes, s_pre[base + lane + 1] <= u));
            u -= s_pre[sl];
            w.b = sl * slice;
#pragma unroll 1
            for (bool found = false; !found;) {
                if (u < 0 || w.b >= p.B) {  // (as in tree_next)
                    w.rem = 0;
                    break;
                }
                const TreeSeq s = tree_seq<TT, TILES>(p, w.b);
                const int each = whole ? 1 : s.ntiles + kItemTiles;
                const int here = p.Hkv * s.rtiles * each;
                if (u < here) {
                    const int item = u / each, at = u - item * each;
                    w.lead = whole ? 0 : max(kItemTiles - at, 0);
                    w.tile = whole ? 0 : max(at - kItemTiles, 0);
                    w.h = item / s.rtiles;
                    w.rt = item - w.h * s.rtiles;
                    found = true;
                } else {
                    u -= here;
                    ++w.b;
                }
            }
        }
        if (lane == 0) {
            s_work = w;
            // (a run whose part of an item is all cost has none of it)
            if (!p.whole) p.cont[run] = make_int4(w.b, w.h, w.rt, w.tile > 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    volatile int* abort_p = &abort_flag;
    TreeWalk walk;
    TreeSeg g;
    walk.w = s_work;
    if (walk.w.rem > 0) walk.s = tree_seq<TT, TILES>(p, walk.w.b);
    auto next_part = [&]() { return tree_next<TT, TILES>(p, whole, walk, g); };

    if (warp == C::MMA_WARP) {
        // ------------------------------------------------ the products
        // (the warp stays together, one lane issues: what describes the operands is uniform)
        constexpr uint32_t ID_S = idesc_f16_f32(F16, kTreeRows, TT, false);
        const uint32_t id_o = idesc_f16_f32(F16, kTreeRows, p.D, true);
        const int ksteps = p.D / 16;
        const bool issuer = elect_one();
        TreeRing<NS> c, ahead;  // stages of the tile whose values are next, and whose keys are
        uint32_t q_phase = 0, p_phase = 0, read_phase = 0;  // bit i: phase of row tile (score buffer) i
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t phase) {
            const bool r = mbar_wait_on(smem_u32(bar), phase & 1u, abort_p, p.status, kErrTimeoutMma);
            return __all_sync(kAllLanes, r) != 0;
        };
        auto full = [&]() { return wait(&full_bar[ahead.at], ahead.phase); };
        // descriptors: a start address in 16-byte units in the low bits, so steps are additions
        const uint64_t q_desc = smem_desc_sw128(smem_s + C::Q_AT), k_desc = smem_desc_sw128(smem_s + C::KV_AT),
                       v_desc = smem_desc_sw128_mn(smem_s + C::KV_AT + C::KV_TILE, TT * 128);
        auto scores = [&](int w, int buf) {
            if (issuer) {
                const uint64_t a = q_desc + w * (C::Q_TILE >> 4), b = k_desc + ahead.at * (C::STAGE >> 4);
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    if (k < ksteps)
                        mma_bf16(tmem + buf * TT, a + (((k >> 2) * kTreeRows * 128 + (k & 3) * 32) >> 4),
                                 b + (((k >> 2) * TT * 128 + (k & 3) * 32) >> 4), ID_S, k != 0);
                mma_commit(smem_u32(&s_bar[buf]));
            }
        };
        auto values = [&](int w, int buf, bool first) {
            if (issuer) {
                const uint64_t b = v_desc + c.at * (C::STAGE >> 4);
#pragma unroll
                for (int k = 0; k < TT / 16; ++k)
                    mma_16bit_tmem_a(tmem + C::O_AT + w * DP, tmem + C::P_AT + buf * (TT / 2) + 8 * k,
                                     b + ((k * 2048) >> 4), id_o, k > 0 || !first);
                mma_commit(smem_u32(&o_bar[w]));
            }
        };
        auto probabilities = [&](int buf) {
            const bool r = wait(&p_bar[buf], p_phase >> buf);
            p_phase ^= 1u << buf;
            return r;
        };
        while (ok && next_part()) {
            const int act = TILES == 2 && g.s.n * p.group - g.rt * 2 * kTreeRows > kTreeRows ? 2 : 1;
#pragma unroll
            for (int w = 0; w < TILES; ++w)
                if (w < act && ok) {
                    ok = wait(&q_bar[w], q_phase >> w);
                    q_phase ^= 1u << w;
                }
            if (!ok || !(ok = full())) break;
            tc_fence_after();
#pragma unroll
            for (int w = 0; w < TILES; ++w)
                if (w < act) scores(w, w);
            ahead.next();
            // Products of different accumulators keep no order: what a product writes over has been read, by
            // the row tile's threads (scores), or by products that they waited for (probabilities).
#pragma unroll 1
            for (int j = 0; j < g.n && ok; ++j) {
                const bool more = j + 1 < g.n;
                if constexpr (TILES == 1) {
                    if (more) {
                        if (!(ok = full())) break;
                        tc_fence_after();
                        scores(0, (j + 1) & 1);
                        ahead.next();
                    }
                    if (!(ok = probabilities(j & 1))) break;
                    tc_fence_after();
                    values(0, j & 1, j == 0);
                } else {
#pragma unroll
                    for (int w = 0; w < TILES; ++w) {
                        if (w >= act || !ok) continue;
                        ok = wait(&read_bar[w], read_phase >> w) && (w > 0 || !more || full());
                        read_phase ^= 1u << w;
                        if (!ok || !more) continue;
                        tc_fence_after();
                        scores(w, w);
                    }
                    if (more) ahead.next();
#pragma unroll
                    for (int w = 0; w < TILES; ++w) {
                        if (w >= act || !ok) continue;
                        if (!(ok = probabilities(w))) continue;
                        tc_fence_after();
                        values(w, w, j == 0);
                    }
                    if (!ok) break;
                }
                if (issuer) mma_commit(smem_u32(&empty_bar[c.at]));
                c.next();
            }
        }
        // every issued product has finished once this commit lands
        if (issuer) mma_commit(smem_u32(&end_bar));
        int dummy = 0;
        mbar_wait_on(smem_u32(&end_bar), 0, &dummy, p.status, kErrTimeoutMma);
        __syncwarp();
    } else if (warp >= TILES * 4) {
        // ------------------------------------------------ keys and values
        constexpr int ES = E4M3 ? 1 : 2, CH = DP * ES / 16;  // 16-byte chunks of a token's head
        constexpr int RPS = 32 / CH, STEPS = 32 / RPS;       // tokens of a step of a loading warp
        const int lw = warp - TILES * 4, ch = lane % CH, r0 = lane / CH;
        const bool in = ch * (16 / ES) < p.D;
        TreeRing<NS> c;  // the stage to fill
        int filled = 0;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t phase) {
            const bool r = mbar_wait_on(smem_u32(bar), phase & 1u, abort_p, p.status, kErrTimeoutProducer);
            return __all_sync(kAllLanes, r) != 0;
        };
        auto wait_empty = [&]() { return filled < NS || wait(&empty_bar[c.at], c.phase ^ 1u); };
        // a stage is filled (all lanes did, or waited for, their part)
        auto signal = [&](int at) {
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&full_bar[at]));
        };
        auto stage = [&]() { return smem_s + C::KV_AT + c.at * C::STAGE; };
        auto meta = [&]() { return smem + C::META_AT + c.at * C::META; };
        // a lane's token, its page looked up before the copies need it
        struct Token {
            int pid, off, h;
            bool in;
        };
        int tile = 0;
        bool any = next_part();
        // token `at` of the next tile
        auto take = [&](bool& has, int at) {
            Token t = {-1, 0, 0, false};
            has = any;
            if (!any) return t;
            t.h = g.h;
            const int tok = g.s.start + (g.tile + tile) * TT + at;
            if (tok >= g.s.lo && tok < g.s.len) {
                const int pi = p.page_shift >= 0 ? tok >> p.page_shift : tok / p.page_size;
                t.off = tok - pi * p.page_size;
                t.pid = __ldg(p.table + (long long)g.b * p.table_ld + pi);
                t.in = true;
            }
            if (++tile == g.n) {
                tile = 0;
                any = next_part();
            }
            return t;
        };
        // false, and reported, where the page is out of range
        auto on_page = [&](const Token& t) {
            const bool good = (uint32_t)t.pid < (uint32_t)p.num_pages;
            if (t.in && !good && p.status) atomicOr(p.status, kErrBadIndex);
            return t.in && good;
        };

        if (TMA && warp == C::TMA_WARP) {
            // pieces of box tokens; 32 of them, a lane's each, are looked up together, a batch of tiles ahead
            const int pieces = TT / p.box, per = 32 / pieces;
            const int blocks = E4M3 ? 1 : (p.D + 63) / 64;
            const bool issuer = elect_one();
            TreeRing<NR> raw;
            struct Batch {
                int pid, off, h, t0, lo, len, n;
                bool in;
            };
            auto look_up = [&]() {
                Batch t;
                t.n = 0;
                if (!any) return t;
                t.n = min(per, g.n - tile);
                t.t0 = g.s.start + (g.tile + tile) * TT;
                t.lo = g.s.lo;
                t.len = g.s.len;
                t.h = g.h;
                t.pid = t.off = 0;
                const int tok = t.t0 + lane * p.box;
                t.in = lane < t.n * pieces && tok + p.box > t.lo && tok < t.len;
                if (t.in) {
                    const int pi = p.page_shift >= 0 ? tok >> p.page_shift : tok / p.page_size;
                    t.off = tok - pi * p.page_size;
                    t.pid = __ldg(p.table + (long long)g.b * p.table_ld + pi);
                }
                tile += t.n;
                if (tile == g.n) {
                    tile = 0;
                    any = next_part();
                }
                return t;
            };
            Batch u;
            u.n = 0;
#pragma unroll 1
            while (true) {
                const Batch following = look_up();
                const bool there = u.n && u.in && (uint32_t)u.pid < (uint32_t)p.num_pages;
                if (u.n && u.in && !there && p.status) atomicOr(p.status, kErrBadIndex);
                uint32_t copied = __ballot_sync(kAllLanes, there), bad = __ballot_sync(kAllLanes, u.n && u.in && !there);
#pragma unroll 1
                for (int j = 0; j < u.n; ++j) {
                    ok = E4M3 ? filled < NR || wait(&raw_empty_bar[raw.at], raw.phase ^ 1u) : wait_empty();
                    if (!ok) break;
                    const uint32_t mine = pieces == 32 ? kAllLanes : (1u << pieces) - 1u;
                    if (!E4M3) {
                        if (lane < TT / 32) {  // valid tokens, 32 a lane
                            const int w0 = u.t0 + j * TT + 32 * lane;
                            uint32_t v = bits_from(u.lo - w0) & ~bits_from(u.len - w0);
#pragma unroll 1
                            for (uint32_t b = bad & mine; b; b &= b - 1) {
                                const int at = (__ffs(b) - 1) * p.box - 32 * lane;
                                v &= ~(bits_from(at) & ~bits_from(at + p.box));
                            }
                            reinterpret_cast<uint32_t*>(meta())[lane] = v;
                        }
                        __syncwarp();
                    }
                    const uint32_t bar = smem_u32(E4M3 ? &raw_full_bar[raw.at] : &full_bar[c.at]);
                    const uint32_t to = E4M3 ? smem_s + C::RAW_AT + raw.at * C::RAW_STAGE : stage();
                    if (issuer)
                        mbar_arrive_expect_tx(bar, 2 * __popc(copied & mine) * p.box * (E4M3 ? p.D : 128 * blocks));
                    // one lane issues all (lanes that issue a piece each take 100 cycles a piece), four at a time
#pragma unroll 1
                    for (int i0 = 0; i0 < pieces; i0 += 4) {
                        int pid[4], off[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            pid[i] = __shfl_sync(kAllLanes, u.pid, j * pieces + i0 + i);
                            off[i] = __shfl_sync(kAllLanes, u.off, j * pieces + i0 + i);
                        }
                        if (issuer) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (!(((copied & mine) >> (i0 + i)) & 1u)) continue;
                                if (E4M3) {
                                    const uint32_t at = to + (i0 + i) * p.box * p.D;
                                    tma_load_4d(at, &tmK, 0, off[i], u.h, pid[i], bar);
                                    tma_load_4d(at + C::RAW_TILE, &tmV, 0, off[i], u.h, pid[i], bar);
                                } else {
                                    const uint32_t at = to + (i0 + i) * p.box * 128;
#pragma unroll
                                    for (int k = 0; k < DP / 64; ++k) {
                                        if (k >= blocks) continue;
                                        tma_load_4d(at + k * TT * 128, &tmK, k * 64, off[i], u.h, pid[i], bar);
                                        tma_load_4d(at + C::KV_TILE + k * TT * 128, &tmV, k * 64, off[i], u.h, pid[i], bar);
                                    }
                                }
                            }
                        }
                    }
                    __syncwarp();
                    copied = pieces == 32 ? 0u : copied >> pieces;
                    bad = pieces == 32 ? 0u : bad >> pieces;
                    ++filled;
                    if (E4M3)
                        raw.next();
                    else
                        c.next();
                }
                u = following;
                if (!ok || u.n == 0) break;
            }
            // the last copies have landed before the CTA may exit
            constexpr int LAST = E4M3 ? NR : NS;
            int dummy = 0;
#pragma unroll 1
            for (int i = max(0, filled - LAST); i < filled; ++i)
                mbar_wait_on(smem_u32(E4M3 ? &raw_full_bar[i % LAST] : &full_bar[i % LAST]), (uint32_t)(i / LAST) & 1u, &dummy,
                             p.status, kErrTimeoutProducer);
        } else if constexpr (!E4M3) {
            // copies of tiles in flight behind the one issued last: a stage is free again once the products that
            // read it are done, which wait for no tile but the next
            constexpr int DEPTH = NS - 2;
            TreeRing<NS> landed;
            bool has = false;
            Token t = {};
#pragma unroll 1
            while (true) {
                Token u = t;
                const bool had = has;
                t = take(has, lw * 32 + lane);
                if (!had) {
                    if (!has) break;
                    continue;
                }
                u.in = on_page(u);
                const uint32_t mask = __ballot_sync(kAllLanes, u.in);  // valid tokens of the warp
                if (!u.in) u.pid = u.off = 0;
                if (!(ok = wait_empty())) break;
                if (lane == 0) reinterpret_cast<uint32_t*>(meta())[lw] = mask;
                const uint8_t* kb = static_cast<const uint8_t*>(p.cache.k) + (u.h * p.cache.k_head) * 2 + ch * 16;
                const uint8_t* vb = static_cast<const uint8_t*>(p.cache.v) + (u.h * p.cache.v_head) * 2 + ch * 16;
                const long long k_off = u.pid * p.cache.k_page + u.off * p.cache.k_token,
                                v_off = u.pid * p.cache.v_page + u.off * p.cache.v_token;
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    const int r = i * RPS + r0;
                    const long long ko = __shfl_sync(kAllLanes, k_off, r), vo = __shfl_sync(kAllLanes, v_off, r);
                    const uint32_t at = stage() + tile_at(TT, lw * 32 + r, ch);
                    if (in) {
                        cp_async16z(at, kb + ko * 2, (mask >> r) & 1u);
                        cp_async16z(at + C::KV_TILE, vb + vo * 2, (mask >> r) & 1u);
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                cp_async_wait<DEPTH>();
                if (filled >= DEPTH) {
                    signal(landed.at);
                    landed.next();
                }
                ++filled;
                c.next();
                if (!has) break;
            }
            cp_async_wait<0>();
            if (ok)
#pragma unroll 1
                for (int i = min(DEPTH, filled); i > 0; --i) {
                    signal(landed.at);
                    landed.next();
                }
        } else {
            // e4m3: raw codes become fp16.  By TMA: [token][D].  By threads: a lane copies, and later converts,
            // pieces of its own, [step][lane] 16 bytes.
            constexpr int LANES = C::LOADERS * 32, BATCH = STEPS < 8 ? STEPS : 8;
            TreeRing<NR> raw;  // the slot to convert
            auto slot = [&](int at) { return smem + C::RAW_AT + at * C::RAW_STAGE; };
            // the keys (values) of a stage from a raw slot; sc: the scale of the lane's token, mask: the warp's
            // valid tokens
            auto convert = [&](bool is_k, float sc, uint32_t mask) {
                const uint8_t* at = slot(raw.at) + (is_k ? 0 : C::RAW_TILE);
                uint8_t* dst = smem + C::KV_AT + c.at * C::STAGE + (is_k ? 0 : C::KV_TILE);
                auto codes = [&](int r, int k) {  // 16 of token r of the warp
                    return *reinterpret_cast<const uint4*>(
                        at + (TMA ? (lw * 32 + r) * p.D + k * 16 : (r / RPS * LANES + lw * 32 + r % RPS * CH + k) * 16));
                };
#pragma unroll
                for (int i0 = 0; i0 < STEPS; i0 += BATCH) {
                    uint4 v[BATCH];
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        const int r = (i0 + i) * RPS + r0;
                        v[i] = make_uint4(0, 0, 0, 0);
                        if (in && ((mask >> r) & 1u)) v[i] = codes(r, ch);
                    }
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        const int r = lw * 32 + (i0 + i) * RPS + r0;
                        if (!in) continue;
                        *reinterpret_cast<uint4*>(dst + tile_at(TT, r, 2 * ch)) =
                            make_uint4(e4m3x2_to_f16x2(v[i].x), e4m3x2_to_f16x2(v[i].x >> 16), e4m3x2_to_f16x2(v[i].y),
                                       e4m3x2_to_f16x2(v[i].y >> 16));
                        *reinterpret_cast<uint4*>(dst + tile_at(TT, r, 2 * ch + 1)) =
                            make_uint4(e4m3x2_to_f16x2(v[i].z), e4m3x2_to_f16x2(v[i].z >> 16), e4m3x2_to_f16x2(v[i].w),
                                       e4m3x2_to_f16x2(v[i].w >> 16));
                    }
                }
                uint8_t* m = meta();
                // a head of zeros, which the append stores with a scale of 1 however small the others are,
                // has no weight
                if (!is_k && __any_sync(kAllLanes, sc == 1.f)) {
                    uint32_t some = 0;
#pragma unroll 1
                    for (int k = 0; k < p.D / 16; ++k) {
                        const uint4 v = codes(lane, k);
                        some |= (v.x | v.y | v.z | v.w) & 0x7f7f7f7fu;
                    }
                    if (sc == 1.f && !some) sc = 0.f;
                }
                reinterpret_cast<float*>(m + 32)[(is_k ? 0 : TT) + lw * 32 + lane] = sc;
                if (is_k) {
                    if (lane == 0) reinterpret_cast<uint32_t*>(m)[lw] = mask;
                } else {
                    // (floats of one sign order as whole numbers do; NaN above all)
                    const uint32_t top = __reduce_max_sync(kAllLanes, __float_as_uint(sc) & 0x7fffffffu);
                    if (lane == 0) reinterpret_cast<uint32_t*>(m)[4 + lw] = top;
                }
            };
            if constexpr (TMA) {
                struct Scales {
                    float k, v;
                    bool in;
                };
                // (pages two tiles, scales one tile ahead)
                auto scales = [&](const Token& t) {
                    Scales s = {0.f, 0.f, on_page(t)};
                    if (s.in) {
                        const long long at = t.pid * p.cache.s_page + t.h * p.cache.s_head + t.off * p.cache.s_token;
                        s.k = __ldg(p.cache.k_scale + at);
                        s.v = __ldg(p.cache.v_scale + at);
                    }
                    return s;
                };
                bool has_t = false, has_s = false;
                Token t = {};
                Scales s = {};
#pragma unroll 1
                while (true) {
                    const Scales u = s;
                    const bool now = has_s;
                    has_s = has_t;
                    if (has_s) s = scales(t);
                    t = take(has_t, lw * 32 + lane);
                    if (!now) {
                        if (!has_s && !has_t) break;
                        continue;
                    }
                    const uint32_t mask = __ballot_sync(kAllLanes, u.in);
                    ok = wait_empty() && wait(&raw_full_bar[raw.at], raw.phase);
                    if (!ok) break;
                    convert(true, u.k, mask);
                    convert(false, u.v, mask);
                    signal(c.at);
                    if (lane == 0) mbar_arrive(smem_u32(&raw_empty_bar[raw.at]));
                    ++filled;
                    c.next();
                    raw.next();
                    if (!has_s) break;
                }
            } else {
                bool has;
                Token t = take(has, lw * 32 + lane);
                TreeRing<NR> issued;
                int ahead = 0;  // tiles whose copies are issued
                auto issue_next = [&]() {
                    if (has) {
                        Token u = t;
                        t = take(has, lw * 32 + lane);
                        u.in = on_page(u);
                        const uint32_t mask = __ballot_sync(kAllLanes, u.in);
                        if (!u.in) u.pid = u.off = 0;
                        const uint8_t* kb = static_cast<const uint8_t*>(p.cache.k) + u.h * p.cache.k_head;
                        const uint8_t* vb = static_cast<const uint8_t*>(p.cache.v) + u.h * p.cache.v_head;
                        const long long k_off = u.pid * p.cache.k_page + u.off * p.cache.k_token,
                                        v_off = u.pid * p.cache.v_page + u.off * p.cache.v_token;
                        uint8_t* at = slot(issued.at);
                        const uint32_t dst = smem_u32(at);
#pragma unroll
                        for (int i = 0; i < STEPS; ++i) {
                            const int r = i * RPS + r0;
                            const long long ko = __shfl_sync(kAllLanes, k_off, r), vo = __shfl_sync(kAllLanes, v_off, r);
                            const uint32_t to = dst + (i * LANES + lw * 32 + lane) * 16;
                            const bool there = in && ((mask >> r) & 1u);
                            cp_async16z(to, in ? kb + ko + ch * 16 : kb, there);
                            cp_async16z(to + C::RAW_TILE, in ? vb + vo + ch * 16 : vb, there);
                        }
                        const long long s_off = u.pid * p.cache.s_page + u.h * p.cache.s_head + u.off * p.cache.s_token;
                        const uint32_t sc = dst + 2 * C::RAW_TILE + (lw * 32 + lane) * 4;
                        cp_async4z(sc, p.cache.k_scale + s_off, u.in);
                        cp_async4z(sc + TT * 4, p.cache.v_scale + s_off, u.in);
                        if (lane == 0) *reinterpret_cast<uint32_t*>(at + 2 * C::RAW_TILE + 2 * TT * 4 + lw * 4) = mask;
                        ++ahead;
                        issued.next();
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");  // (empty where nothing is left)
                };
#pragma unroll 1
                for (int i = 0; i < NR - 1; ++i) issue_next();
#pragma unroll 1
                while (filled < ahead) {
                    cp_async_wait<NR - 2>();
                    __syncwarp();
                    if (!(ok = wait_empty())) break;
                    const uint8_t* sc = slot(raw.at) + 2 * C::RAW_TILE;
                    const uint32_t mask = *reinterpret_cast<const uint32_t*>(sc + 2 * TT * 4 + lw * 4);
                    convert(true, *reinterpret_cast<const float*>(sc + (lw * 32 + lane) * 4), mask);
                    convert(false, *reinterpret_cast<const float*>(sc + (TT + lw * 32 + lane) * 4), mask);
                    signal(c.at);  // (and the warp is done with the raw slot)
                    ++filled;
                    c.next();
                    raw.next();
                    issue_next();
                }
                cp_async_wait<0>();
            }
        }
    } else {
        // ------------------------------------------------ softmax: a thread has a row
        const int w = warp >> 2, r = tid & (kTreeRows - 1);
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_o = tmem + C::O_AT + w * DP + lanes;
        uint32_t q_phase = 0, s_phase = 0, x_phase = 0;
        // products with values: of the tiles so far, and those known to have reached the accumulators
        uint32_t tiles_done = 0, reached = 0;
        TreeRing<NS> c;  // the tile's stage
        uint32_t* anc = reinterpret_cast<uint32_t*>(smem + C::ANC_AT) + w * kTreeRows + r;  // words 128 * TILES apart
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t phase) {
            const bool r = mbar_wait_on(smem_u32(bar), phase & 1u, abort_p, p.status, kErrTimeoutEpilogue);
            return __all_sync(kAllLanes, r) != 0;
        };
        // all of the row tile's threads (one row tile) have come so far
        auto come = [&]() {
            mbar_arrive(smem_u32(&x_bar));
            x_phase ^= 1u;
        };
        auto met = [&]() { return wait(&x_bar, x_phase ^ 1u); };
        bool to_meet = false;  // copies of the part before may still be read where the queries go
        constexpr int LPR = DP / 8, RPI = kTreeRows / LPR;  // lanes of a row of queries, rows of a round
        constexpr int BATCH = 8;                            // rounds in flight
        const int q_ch = r % LPR;
        int rows = 0;  // of the part's row tile
        // how often the rows stand in the tile (e4m3): each copy's warps take a part of the tokens, with sums of their own
        // that meet at the end
        auto copies = [&]() { return !C::COPIES || rows > 64 ? 1 : rows > 32 ? 2 : 4; };
        // the next part that has rows in this tile
        auto advance = [&]() {
            while (next_part()) {
                rows = g.s.n * p.group - (g.rt * TILES + w) * kTreeRows;
                if (rows > 0) return true;
                for (int i = g.n % (2 * NS); i > 0; --i) c.next();
            }
            return false;
        };
        // rounds i0 and on of its queries, 16 bytes a lane; rows come again `every` so many (a power of two)
        auto load_q = [&](int i0, int every, uint4 (&q)[BATCH]) {
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int row = (r / LPR + (i0 + i) * RPI) & (every - 1);
                q[i] = make_uint4(0, 0, 0, 0);
                if (q_ch * 8 < p.D && row < rows) {
                    const int at = (g.rt * TILES + w) * kTreeRows + row, d = tree_draft(p, at);
                    q[i] = *reinterpret_cast<const uint4*>(p.q + (g.s.first + d) * p.q_token +
                                                           (long long)(g.h * p.group + at - d * p.group) * p.q_head + q_ch * 8);
                }
            }
        };
        auto store_q = [&](int i0, const uint4 (&q)[BATCH]) {
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int row = r / LPR + (i0 + i) * RPI;
                uint4 v = q[i];
                v.x ^= p.q_sign, v.y ^= p.q_sign, v.z ^= p.q_sign, v.w ^= p.q_sign;
                if constexpr (E4M3) {
                    // the products run in fp16: each row is scaled by a power of two to below 2^15, so that
                    // fp16 values, and bf16 values down to 2^-30 of the largest, are exact
                    uint32_t u[4] = {v.x, v.y, v.z, v.w};
                    float a = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 x = (qf16 ? unpack2<true>(u[j]) : unpack2<false>(u[j]));
                        a = fmaxf(a, fmaxf(fabsf(x.x), fabsf(x.y)));
                    }
#pragma unroll
                    for (int o = LPR / 2; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(kAllLanes, a, o));
                    const uint32_t e = min(max(__float_as_uint(a) >> 23, 15u), 253u);
                    const float f = __uint_as_float((268u - e) << 23);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 x = (qf16 ? unpack2<true>(u[j]) : unpack2<false>(u[j]));
                        u[j] = pack2<true>(x.x * f, x.y * f);
                    }
                    v = make_uint4(u[0], u[1], u[2], u[3]);
                    // not 0, which would make NaN of a masked score
                    if (q_ch == 0)
                        s_qf[w][row] = fmaxf(p.scale_log2 * __uint_as_float((e - 14u) << 23), 0x1p-126f);
                }
                *reinterpret_cast<uint4*>(smem + C::Q_AT + w * C::Q_TILE + tile_at(kTreeRows, row, q_ch)) = v;
            }
        };
        // parents of drafts r and on, the lane's draft's where there are few
        auto load_up = [&](int (&up)[2]) {
            const int from = g.s.n <= 32 ? lane : r;
            up[0] = p.parents && from < g.s.n ? __ldg(p.parents + g.s.first + from) : -1;
            up[1] = p.parents && from == r && r + kTreeRows < g.s.n ? __ldg(p.parents + g.s.first + r + kTreeRows) : -1;
        };
        while (ok && advance()) {
            const int rep = copies(), fold = kTreeRows / rep - 1, lr = r & fold;  // lr: the thread's row
            const int cols = TT / rep, col0 = r / (fold + 1) * cols;
            // --- the queries; the parents ---
            int up[2];
            load_up(up);
#pragma unroll 1
            for (int i0 = 0; i0 < LPR && (rep > 1 || i0 * RPI < rows); i0 += BATCH) {
                // (rows past the last have any values)
                uint4 q[BATCH];
                load_q(i0, fold + 1, q);
                if (C::COPIES && to_meet) {
                    if (!(ok = met())) break;
                    to_meet = false;
                }
                store_q(i0, q);
            }
            if (!ok) break;
            const bool few = g.s.n <= 32;  // drafts: a warp has their parents in its lanes
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int d = (few ? lane : r) + i * kTreeRows;
                if (up[i] >= d || up[i] < -1) {
                    if (d < g.s.n && p.status) atomicOr(p.status, kErrBadIndex);
                    up[i] = -1;
                }
                if (!few) s_up[w][d] = (int16_t)up[i];
            }
            fence_async_shared();
            mbar_arrive(smem_u32(&q_bar[w]));
            // --- the row's place in the tree ---
            const bool act = lr < rows, warp_act = (lr & ~31) < rows;
            const int at = (g.rt * TILES + w) * kTreeRows + min(lr, rows - 1), draft = tree_draft(p, at);
            const int head = g.h * p.group + at - draft * p.group;
            const float sink = TILES == 1 && p.sinks ? __ldg(p.sinks + head) : 0.f;  // (in time; two row tiles: registers)
            const bool sees_drafts = g.s.start + (long long)(g.tile + g.n) * TT > g.s.ctx;
            if (E4M3 || !few) {
                if (!(ok = wait(&q_bar[w], q_phase))) break;
            }
            q_phase ^= 1u;
            int depth = draft;
            if (p.parents && (sees_drafts || p.window > 0)) {
                depth = -1;
                if (few) {
                    uint32_t bits = 0;
                    int a = draft;
                    while (__any_sync(kAllLanes, a >= 0)) {
                        if (a >= 0) {
                            ++depth;
                            if (p.window <= 0 || depth < p.window) bits |= 1u << a;
                        }
                        const int above = __shfl_sync(kAllLanes, up[0], a & 31);
                        a = a >= 0 ? above : -1;
                    }
                    anc[0] = bits;  // (what follows is of tokens that are not there)
                } else {
                    uint32_t bits[kMaxDrafts / 32];
#pragma unroll
                    for (int k = 0; k < kMaxDrafts / 32; ++k) bits[k] = 0;
#pragma unroll 1
                    for (int a = draft; a >= 0; a = s_up[w][a]) {
                        ++depth;
                        if (p.window <= 0 || depth < p.window) {
#pragma unroll
                            for (int k = 0; k < kMaxDrafts / 32; ++k)
                                if (a >> 5 == k) bits[k] |= 1u << (a & 31);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < kMaxDrafts / 32; ++k) anc[k * TILES * kTreeRows] = bits[k];
                }
            }
            // the first token that the row sees of the context (of all, in a chain)
            const int since = p.window > 0 ? max(g.s.ctx + depth - p.window + 1, 0) : 0;
            const float qf = E4M3 ? s_qf[w][lr] : p.scale_log2;  // positive factor of the scores
            if (rep > 1) {  // probabilities of the other copies' tokens
                const uint32_t z[16] = {};
#pragma unroll 1
                for (int k = 0; k < TT; k += 16) tmem_st16(tmem + C::P_AT + lanes + k, z);
                tmem_st_wait();
            }

            float m = -INFINITY;  // e4m3: largest score (before qf)
            float base = kNoWeights;       // the power of two that sums are about
            uint64_t sum[4] = {0, 0, 0, 0};  // in eight parts
            // all products so far have reached the accumulators (a parity tells only neighbours apart: each phase is
            // waited for, or known to have passed)
            auto reach = [&]() {
#pragma unroll 1
                for (; reached != tiles_done && ok; ++reached) ok = wait(&o_bar[w], reached);
            };
#pragma unroll 1
            for (int j = 0; j < g.n; ++j, c.next()) {
                const int buf = TILES == 2 ? w : j & 1;
                ok = wait(&s_bar[buf], s_phase >> buf);
                s_phase ^= 1u << buf;
                if (!ok) break;
                tc_fence_after();
                // The tile's keys, values and scales are there (its scores waited for them), and the products issued
                // before its scores, up to those of the tile before the last, are done.
                if (j > 0) reached = tiles_done - 1;
                const uint8_t* meta = smem + C::META_AT + c.at * C::META;
                bool all = true;  // the tile's tokens are there
#pragma unroll
                for (int k = 0; k < TT / 32; ++k) all = all && reinterpret_cast<const uint32_t*>(meta)[k] == kAllLanes;
                if (TMA && !E4M3 && !all && w == 0) {
                    // a copied piece may hold anything behind the last token (before the first, on a bad page):
                    // such values become 0, whose product with a probability of 0 is 0
                    if (!(ok = wait(&full_bar[c.at], c.phase))) break;
                    if (r < TT && !((reinterpret_cast<const uint32_t*>(meta)[r >> 5] >> (r & 31)) & 1u))
#pragma unroll 1
                        for (int k = 0; k < p.D / 8; ++k)
                            *reinterpret_cast<uint4*>(smem + C::KV_AT + c.at * C::STAGE + C::KV_TILE + tile_at(TT, r, k)) =
                                make_uint4(0, 0, 0, 0);
                    fence_async_shared();
                }
                if (warp_act) {
                    const uint32_t t_s = tmem + buf * TT + lanes, t_p = tmem + C::P_AT + buf * (TT / 2) + lanes;
                    const int t0 = g.s.start + (g.tile + j) * TT;
                    const bool masked = g.s.ctx - t0 < TT || !all || __any_sync(kAllLanes, since > t0);
                    const float* scales = reinterpret_cast<const float*>(meta + 32);
                    float room = kSlack + kLift<KV>;  // above base, for a score (e4m3: for a weight, less the scales)
                    if constexpr (E4M3) {
                        const float* v = reinterpret_cast<const float*>(meta + 16);  // largest, of each loading warp
                        float most = kLeastScale;
#pragma unroll
                        for (int i = 0; i < C::LOADERS; ++i) most = fmaxf(most, v[i]);
                        room = kMostWeight - __log2f(most);
                    }
                    // the row tile's next scores may come (two row tiles)
                    auto read_scores = [&]() {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&read_bar[w]));
                    };
                    // W scores from column c0 on: what the sums are about, seldom moved; probabilities (e4m3: weights),
                    // rounded to 16 bits
                    auto part = [&](auto wide, int c0) {
                        constexpr int W = decltype(wide)::value;
                        uint32_t y[W];
                        if constexpr (W == 16) tmem_ld16(t_s + c0, y);
                        if constexpr (W == 32) tmem_ld32(t_s + c0, y);
                        if constexpr (W == 64) tmem_ld64(t_s + c0, y);
                        if (TILES == 2 && c0 + W == TT) read_scores();
                        auto score = [&](int i) { return __uint_as_float(y[i]); };
                        auto pair = [&](int i) { return f32x2(__uint_as_float(y[i]), __uint_as_float(y[i + 1])); };
                        if constexpr (E4M3) {
#pragma unroll
                            for (int i = 0; i < W; i += 4) {
                                const float4 f = *reinterpret_cast<const float4*>(scales + c0 + i);
                                const float2 u = f32x2_get(f32x2_mul(pair(i), f32x2(f.x, f.y))),
                                             v = f32x2_get(f32x2_mul(pair(i + 2), f32x2(f.z, f.w)));
                                y[i] = __float_as_uint(u.x), y[i + 1] = __float_as_uint(u.y);
                                y[i + 2] = __float_as_uint(v.x), y[i + 3] = __float_as_uint(v.y);
                            }
                        }
                        if (masked) {
#pragma unroll
                            for (int k = 0; k < W; k += 32) {
                                // the tokens that the row sees, from t on
                                const int t = t0 + c0 + k, past = g.s.ctx - t;  // bits from `past` on are drafts
                                uint32_t see = bits_from(since - t);
                                if (past < 32) {
                                    if (p.parents) {
                                        const int o = -past;  // draft of bit 0
                                        uint32_t d = 0;
                                        if (o < 0) {
                                            d = anc[0] << -o;
                                        } else if (o < kMaxDrafts) {
                                            const uint32_t lo = anc[(o >> 5) * TILES * kTreeRows];
                                            const uint32_t hi =
                                                o < kMaxDrafts - 32 ? anc[((o >> 5) + 1) * TILES * kTreeRows] : 0u;
                                            d = __funnelshift_r(lo, hi, o & 31);
                                        }
                                        const uint32_t drafts = bits_from(past);
                                        see = (see & ~drafts) | (d & drafts);
                                    } else {
                                        see &= ~bits_from(past + draft + 1);
                                    }
                                }
                                const uint16_t* there = reinterpret_cast<const uint16_t*>(meta) + (c0 + k) / 16;
                                see &= W == 16 ? there[0] : there[0] | (uint32_t)there[1] << 16;
#pragma unroll
                                for (int i = 0; i < (W < 32 ? W : 32); ++i)
                                    if (!((see >> i) & 1u)) y[k + i] = __float_as_uint(-INFINITY);
                            }
                        }
                        float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int i = 0; i < W / 2; ++i) t[i & 3] = max3(t[i & 3], score(2 * i), score(2 * i + 1));
                        const float top = fmaxf(max3(t[0], t[1], t[2]), t[3]);
                        if (E4M3) m = fmaxf(m, top);
                        const bool over = fmaf(top, qf, -base) > room;  // (NaN, -inf: no)
                        if (__any_sync(kAllLanes, over)) {
                            // After the first time it moves by whole powers of two, so that the tile's probabilities so
                            // far, of which some may be as large as the new ones, keep their bits.  (e4m3: down to
                            // the weights' place, up to the least that it may have; none where the bound was too high.)
                            float n = base, steps = 0.f;
                            const bool first = base == kNoWeights;
                            if constexpr (!E4M3) {
                                const float to = top * qf - kLift<KV>;
                                if (over) steps = rintf(to - base), n = first ? to : base + steps;
                            } else {
                                float best = -INFINITY;  // of the weights, in powers of two
#pragma unroll
                                for (int i = 0; i < W; ++i)
                                    best = fmaxf(best, fmaf(score(i), qf, __log2f(fabsf(scales[TT + c0 + i]))));
                                const float to = best - kNewWeight, least = m * qf - kMostLift;
                                if (over) {
                                    steps = fmaxf(fmaxf(floorf(to - base), ceilf(least - base)), 0.f);
                                    n = first ? fmaxf(base, fmaxf(to, least)) : base + steps;
                                }
                            }
                            // (sums take the difference as it was rounded, probabilities the whole power)
                            const float f = ex2_approx(base - n), fp = steps < 127.f ? __uint_as_float((127u - (uint32_t)steps) << 23) : 0.f;
                            base = n;
#pragma unroll
                            for (int i = 0; i < 4; ++i) sum[i] = f32x2_mul(sum[i], f32x2(f, f));
                            reach();
                            if (!ok) return;
                            tc_fence_after();
                            // what an earlier part of the tile stored, probabilities and rescaled sums, is there
                            // before it is loaded
                            tmem_st_wait();
                            if (j > 0) {
#pragma unroll 1
                                for (int d = 0; d < p.D; d += 16) {
                                    uint32_t z[16];
                                    tmem_ld16(t_o + d, z);
#pragma unroll
                                    for (int i = 0; i < 16; ++i) z[i] = __float_as_uint(__uint_as_float(z[i]) * f);
                                    tmem_st16(t_o + d, z);
                                }
                            }
                            if (c0 > col0) {  // and the tile's probabilities so far
#pragma unroll 1
                                for (int d = col0 / 2; d < c0 / 2; d += 16) {
                                    uint32_t z[16];
                                    tmem_ld16(t_p + d, z);
#pragma unroll
                                    for (int i = 0; i < 16; ++i) {
                                        const float2 v = unpack2<F16>(z[i]);
                                        z[i] = pack2<F16>(v.x * fp, v.y * fp);
                                    }
                                    tmem_st16(t_p + d, z);
                                }
                            }
                        }
                        const uint64_t qq = f32x2(qf, qf), bb = f32x2(-base, -base);
                        if (TILES == 2) {  // the columns of the probabilities are read by the products of the tile before
                            reach();
                            if (!ok) return;
                            tc_fence_after();
                        }
                        uint32_t z[W / 2];
#pragma unroll
                        for (int i = 0; i < W / 2; i += 2) {
                            const float2 a = f32x2_get(f32x2_fma(pair(2 * i), qq, bb)),
                                         b = f32x2_get(f32x2_fma(pair(2 * i + 2), qq, bb));
                            uint64_t e0 = f32x2(ex2_approx(a.x), ex2_approx(a.y)),
                                     e1 = f32x2(ex2_approx(b.x), ex2_approx(b.y));
                            sum[i & 2] = f32x2_add(sum[i & 2], e0);
                            sum[(i & 2) + 1] = f32x2_add(sum[(i & 2) + 1], e1);
                            if constexpr (E4M3) {
                                const float4 v = *reinterpret_cast<const float4*>(scales + TT + c0 + 2 * i);
                                e0 = f32x2_mul(e0, f32x2(v.x, v.y));
                                e1 = f32x2_mul(e1, f32x2(v.z, v.w));
                            }
                            const float2 u0 = f32x2_get(e0), u1 = f32x2_get(e1);
                            z[i] = pack2<F16>(u0.x, u0.y);
                            z[i + 1] = pack2<F16>(u1.x, u1.y);
                        }
                        if constexpr (W == 16) tmem_st8(t_p + c0 / 2, z);
                        if constexpr (W == 32) tmem_st16(t_p + c0 / 2, z);
                        if constexpr (W == 64) tmem_st32(t_p + c0 / 2, z);
                    };
                    if constexpr (C::COPIES) {
                        if (rep == 4) {
                            part(std::integral_constant<int, 16>(), col0);
                        } else if (rep == 2) {
                            part(std::integral_constant<int, 32>(), col0);
                        }
                    }
                    if (rep == 1) {
#pragma unroll
                        for (int c0 = 0; c0 < TT; c0 += C::WIDE)
                            if (ok) part(std::integral_constant<int, C::WIDE>(), c0);
                    }
                    if (!ok) break;
                    tmem_st_wait();
                    tc_fence_before();
                }
                if (TILES == 2 && !warp_act && lane == 0) mbar_arrive(smem_u32(&read_bar[w]));
                // Two row tiles: the next scores may come before the others' probabilities, a warp without rows keeps
                // behind them.  The last tile: one phase is left to wait for afterwards.
                if (TILES == 2 || j == g.n - 1) reach();
                if (!ok) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&p_bar[buf]));
                ++tiles_done;
            }
            if (!ok) break;
            // --- the row, or the run's part of it ---
            constexpr int ROWS = TILES * kTreeRows;
            const float2 halves = f32x2_get(f32x2_add(f32x2_add(sum[0], sum[1]), f32x2_add(sum[2], sum[3])));
            float l = halves.x + halves.y;
            if (base == kNoWeights) base = -INFINITY;  // no tokens
            const bool done = g.starts && g.ends;
            uint16_t* dst = p.out + (g.s.first + draft) * p.o_token + (long long)head * p.o_head;
            float* part = p.partial + ((long long)blockIdx.x * 2 + (g.starts ? 1 : 0)) * (ROWS * (p.D + 2));
            float4* sums = reinterpret_cast<float4*>(part + 2 * ROWS) + w * kTreeRows + lr;
            reach();
            if (!ok) break;
            tc_fence_after();
            auto pack = [&](float a, float b) { return qf16 ? pack2<true>(a, b) : pack2<false>(a, b); };
            uint64_t odd = 0;  // NaN where a sum is not finite
            if (rep == 1) {
                if (warp_act) {
                    const float fw = !done        ? 1.f
                                     : TILES == 1 ? final_weight(p.sinks != nullptr, sink, base, l)
                                                  : final_weight(p.sinks, head, base, l);
                    if (!done && act) reinterpret_cast<float2*>(part)[w * kTreeRows + r] = make_float2(base, l);
#pragma unroll 1
                    for (int d = 0; d < p.D; d += 16) {
                        uint32_t x[16];
                        tmem_ld16(t_o + d, x);
                        float v[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(x[i]) * fw;
#pragma unroll
                        for (int i = 0; i < 16; i += 2)
                            odd = f32x2_fma(f32x2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), 0, odd);
                        if (act && done) {
                            *reinterpret_cast<uint4*>(dst + d) =
                                make_uint4(pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7]));
                            *reinterpret_cast<uint4*>(dst + d + 8) =
                                make_uint4(pack(v[8], v[9]), pack(v[10], v[11]), pack(v[12], v[13]), pack(v[14], v[15]));
                        } else if (act) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                sums[(d / 4 + i) * ROWS] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        }
                    }
                }
            } else if constexpr (C::COPIES) {
                // the copies of a row meet where the queries were; sums are in the order of the copies
                const int mine = r / (fold + 1);
                // [four dims, copy, row]; eight dims in turn are a copy's to add up
                float4* room = reinterpret_cast<float4*>(smem + C::Q_AT);
                s_ml[r] = make_float2(base, l);
#pragma unroll 1
                for (int d = 0; d < p.D; d += 32) {
                    uint32_t x[32];
                    tmem_ld32(t_o + d, x);
                    if (act) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            room[(d / 4 + i) * kTreeRows + r] =
                                make_float4(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1]),
                                            __uint_as_float(x[4 * i + 2]), __uint_as_float(x[4 * i + 3]));
                    }
                    __syncwarp();
                }
                come();
                if (!(ok = met())) break;
                float f[4];  // what each copy's sums are multiplied by
                float top = -INFINITY;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f[k] = k < rep ? s_ml[k * (fold + 1) + lr].x : -INFINITY;
                    top = fmaxf(top, f[k]);
                }
                l = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f[k] = top == -INFINITY ? 0.f : ex2_approx(f[k] - top);
                    if (k < rep) l += s_ml[k * (fold + 1) + lr].y * f[k];
                }
                const float fw = done ? final_weight(p.sinks != nullptr, sink, top, l) : 1.f;
                if (!done && act && mine == 0) reinterpret_cast<float2*>(part)[lr] = make_float2(top, l);
                if (act) {
#pragma unroll 1
                    for (int e = 2 * mine; e < p.D / 4; e += 2 * rep) {  // 8 dims
                        float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (k >= rep) continue;
                            add_scaled(u, 1.f, room[e * kTreeRows + k * (fold + 1) + lr], f[k]);
                            add_scaled(v, 1.f, room[(e + 1) * kTreeRows + k * (fold + 1) + lr], f[k]);
                        }
                        odd = f32x2_fma(f32x2(u.x, u.y), 0, f32x2_fma(f32x2(u.z, u.w), 0, odd));
                        odd = f32x2_fma(f32x2(v.x, v.y), 0, f32x2_fma(f32x2(v.z, v.w), 0, odd));
                        u = make_float4(u.x * fw, u.y * fw, u.z * fw, u.w * fw);
                        v = make_float4(v.x * fw, v.y * fw, v.z * fw, v.w * fw);
                        if (done) {
                            *reinterpret_cast<uint4*>(dst + 4 * e) =
                                make_uint4(pack(u.x, u.y), pack(u.z, u.w), pack(v.x, v.y), pack(v.z, v.w));
                        } else {
                            sums[e * ROWS] = u;
                            sums[(e + 1) * ROWS] = v;
                        }
                    }
                }
                come();
                to_meet = true;
            }
            const float2 o = f32x2_get(odd);
            if (act && o.x + o.y != 0.f) s_odd = 1;
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == C::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, C::COLS);
    }
    if (s_odd && !abort_flag && !p.once) tree_mend<KV, TT, TILES>(p, &s_work, whole);
}

template <int DP, int KV, int TILES, bool TMA>
cudaError_t launch_tree_t(const CUtensorMap& tmK, const CUtensorMap& tmV, const TreeParams& p, int ctas,
                          cudaStream_t st) {
    using C = TreeCfg<DP, KV, TILES, TMA>;
    // (a CTA's fixed arrays and what the system keeps of its shared memory: 1 KB each)
    static_assert((C::SMEM + 2048) * C::CTAS <= 228 * 1024, "shared memory of the resident CTAs");
    static_assert(C::P_AT + C::TT <= C::COLS && C::COLS * C::CTAS <= 512, "tensor memory");
    const auto kernel = tree_kernel<DP, KV, TILES, TMA>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(ctas), dim3(C::THREADS), C::SMEM, st, tmK, tmV, p);
}
template <int DP, int KV>
cudaError_t launch_tree_w(const CUtensorMap& tmK, const CUtensorMap& tmV, const TreeParams& p, const TreePlan& w,
                          cudaStream_t st) {
    if constexpr (DP <= 128)
        if (w.tiles == 2)
            return p.box ? launch_tree_t<DP, KV, 2, true>(tmK, tmV, p, w.ctas, st)
                         : launch_tree_t<DP, KV, 2, false>(tmK, tmV, p, w.ctas, st);
    return p.box ? launch_tree_t<DP, KV, 1, true>(tmK, tmV, p, w.ctas, st)
                 : launch_tree_t<DP, KV, 1, false>(tmK, tmV, p, w.ctas, st);
}
template <int KV>
cudaError_t launch_tree_d(const CUtensorMap& tmK, const CUtensorMap& tmV, const TreeParams& p, const TreePlan& w,
                          cudaStream_t st) {
    return p.D <= 64    ? launch_tree_w<64, KV>(tmK, tmV, p, w, st)
           : p.D <= 128 ? launch_tree_w<128, KV>(tmK, tmV, p, w, st)
                        : launch_tree_w<256, KV>(tmK, tmV, p, w, st);
}

}  // namespace moe
