// Keys and values moved within a paged cache, in all layers of a model by one
// launch: whole pages or their first places (a fork's last page, pages moved
// together), and the kept ones of a step's drafted tokens, which close up behind
// the context ("Hosting Qwen on Blackwell", perplexity.ai hub blog: a paged cache,
// heads-major; "GPT-OSS on Day 0": the layers' own caches).
//
// Bound by memory: what moves is read once and written once, in 16-byte pieces.
// 256 pages of 64 tokens, 4 heads of 128 e4m3 codes, 36 layers: 187.6 us for 1.25 GB,
// 6.66 TB/s, 98 % of a copy. The used places of 64 last pages of 16, 8 heads of 64, 24
// layers: 10.0 us for 53 MB. Up to 7 of 24 drafts of 128 sequences, e4m3, 36 layers: 10.2
// us for 19.5 MB in tokens of 128 bytes, latency; 4 of 8 of one sequence: 2.9.
#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyPieces = 4;  // 16-byte pieces that a thread has in flight (2: 193 and 12.9 us, 8: 189.5 and 13.0)
constexpr int kCopyBlock = kCopyThreads * kCopyPieces;
constexpr int kMoveWarps = 4;   // per CTA
constexpr int kMoveLayers = 4;  // layers that a warp has in flight (2: 9.8 us, 8: 10.8)

}  // namespace

// A CTA copies kCopyBlock pieces of one page's keys or values in one layer.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(CopyPagesParams p) {
    pdl_wait();
    pdl_allow_dependents();
    unsigned at = blockIdx.x;
    const int part = at % p.parts;
    at /= p.parts;
    const bool is_k = (at & 1) == 0;
    at >>= 1;
    const int layer = at % p.layers, i = at / p.layers;
    const int from = __ldg(p.src + i), to = __ldg(p.dst + i);
    const int named = p.tokens ? __ldg(p.tokens + i) : p.page_size;
    const int n = min(max(named, 0), p.page_size);
    if (from < 0 || to < 0) return;
    const bool bad = from >= p.num_pages || to >= p.num_pages;
    if ((bad || n != named) && p.status && threadIdx.x == 0) atomicOr(p.status, kErrBadIndex);
    if (bad) return;
    const KvCache& c = p.cache;
    const long long page = is_k ? c.k_page : c.v_page, head = is_k ? c.k_head : c.v_head,
                    token = is_k ? c.k_token : c.v_token;
    uint8_t* base = static_cast<uint8_t*>(is_k ? c.k : c.v) + layer * (is_k ? p.k_layer : p.v_layer) * p.elem;
    const uint8_t* src = base + from * page * p.elem;
    uint8_t* dst = base + to * page * p.elem;
    const unsigned row = p.row_pieces, run = n * row, total = run * p.Hkv;
    uint4 v[kCopyPieces];
    long long off[kCopyPieces];
#pragma unroll
    for (int j = 0; j < kCopyPieces; ++j) {
        const unsigned k = part * kCopyBlock + j * kCopyThreads + threadIdx.x;
        off[j] = -1;
        if (k < total) {
            const unsigned h = k / run, r = k - h * run, t = r / row;
            off[j] = (h * head + t * token) * p.elem + (r - t * row) * 16;
            v[j] = __ldcs(reinterpret_cast<const uint4*>(src + off[j]));
        }
    }
#pragma unroll
    for (int j = 0; j < kCopyPieces; ++j)
        if (off[j] >= 0) __stcs(reinterpret_cast<uint4*>(dst + off[j]), v[j]);
    if (c.k_scale) {  // the page's scales, dealt to its CTAs
        float* s = (is_k ? c.k_scale : c.v_scale) + layer * p.s_layer;
        for (unsigned k = part * kCopyThreads + threadIdx.x; k < (unsigned)(n * p.Hkv); k += p.parts * kCopyThreads) {
            const unsigned h = k / n, t = k - h * n;
            const long long o = h * c.s_head + t * c.s_token;
            s[to * c.s_page + o] = s[from * c.s_page + o];
        }
    }
}

// A warp moves the kept drafts of one sequence, key or value head, in a part of
// the layers.  Kept drafts ascend, so draft j comes from place j or a later one:
// a batch of tokens is read before it is written, and no batch reads what an
// earlier one wrote.
__global__ void __launch_bounds__(kMoveWarps * 32) compact_drafts_kernel(CompactParams p) {
    pdl_wait();
    pdl_allow_dependents();
    const int lane = threadIdx.x & 31;
    const long long job = (long long)blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
    const long long per_seq = 2LL * p.Hkv * p.layer_parts;
    if (job >= p.B * per_seq) return;
    const int b = (int)(job / per_seq);
    int at = (int)(job - b * per_seq);
    const int part = at % p.layer_parts;
    at /= p.layer_parts;
    const bool is_k = at < p.Hkv;
    const int h = is_k ? at : at - p.Hkv;
    const bool reports = part == 0 && at == 0;

    const int raw = __ldg(p.lengths + b), lo = __ldg(p.starts + b), hi = __ldg(p.starts + b + 1);
    const int drafts = (int)((long long)hi - lo);
    if (lo < 0 || hi < lo || raw < drafts || raw > p.max_tokens) {
        if (reports && lane == 0) {
            p.out[b] = raw;
            if (p.status) atomicOr(p.status, kErrBadIndex);
        }
        return;
    }
    const int first = raw - drafts;
    const int32_t* kept = p.kept + (long long)b * p.kept_ld;
    const KvCache& c = p.cache;
    const int lpr = 1 << p.lpr_shift, sub = lane >> p.lpr_shift, piece = lane & (lpr - 1), rows = 32 >> p.lpr_shift;
    const long long page = is_k ? c.k_page : c.v_page, token = is_k ? c.k_token : c.v_token;
    const long long layer = (is_k ? p.k_layer : p.v_layer) * p.elem;
    uint8_t* base = static_cast<uint8_t*>(is_k ? c.k : c.v) + h * (is_k ? c.k_head : c.v_head) * p.elem;
    float* scales = c.k_scale ? (is_k ? c.k_scale : c.v_scale) + h * c.s_head : nullptr;
    const int l0 = (int)((long long)p.layers * part / p.layer_parts),
              l1 = (int)((long long)p.layers * (part + 1) / p.layer_parts);

    int count = 0;      // leading entries that are drafts, ascending
    int last = -1;
    bool bad = false;
    for (int j0 = 0; j0 < p.K; j0 += 32) {
        // a lane has one entry; the list ends at the first that is negative or bad
        const int mine = j0 + lane < p.K ? __ldg(kept + j0 + lane) : -1;
        int before = __shfl_up_sync(0xffffffffu, mine, 1);
        if (lane == 0) before = last;
        const bool fine = mine > before && mine < drafts;
        const uint32_t stop = __ballot_sync(0xffffffffu, !fine);
        const int n = stop ? __ffs(stop) - 1 : 32;
        if (n < 32 && __shfl_sync(0xffffffffu, mine, n) >= 0) bad = true;
        last = __shfl_sync(0xffffffffu, mine, 31);
        count = j0 + n;
        // where each lane's token is and goes
        long long from = -1, to = -1, s_from = 0, s_to = 0;
        if (lane < n && mine != j0 + lane) {
            const int t0 = first + mine, t1 = first + j0 + lane;
            const int p0 = t0 / p.page_size, p1 = t1 / p.page_size;
            const int a = __ldg(p.table + (long long)b * p.table_ld + p0), d = __ldg(p.table + (long long)b * p.table_ld + p1);
            if ((uint32_t)a < (uint32_t)p.num_pages && (uint32_t)d < (uint32_t)p.num_pages) {
                const int o0 = t0 - p0 * p.page_size, o1 = t1 - p1 * p.page_size;
                from = (a * page + o0 * token) * p.elem;
                to = (d * page + o1 * token) * p.elem;
                s_from = a * c.s_page + o0 * c.s_token;
                s_to = d * c.s_page + o1 * c.s_token;
            } else {
                bad = true;
            }
        }
        for (int r0 = 0; r0 < n; r0 += rows) {
            const int r = r0 + sub;
            const long long f = __shfl_sync(0xffffffffu, from, r & 31), t = __shfl_sync(0xffffffffu, to, r & 31);
            const long long sf = __shfl_sync(0xffffffffu, s_from, r & 31), st = __shfl_sync(0xffffffffu, s_to, r & 31);
            const bool act = r < n && f >= 0 && piece < p.row_pieces;
            if (!__any_sync(0xffffffffu, act)) continue;
            for (int l = l0; l < l1; l += kMoveLayers) {
                uint4 v[kMoveLayers];
                float s[kMoveLayers];
#pragma unroll
                for (int k = 0; k < kMoveLayers; ++k)
                    if (act && l + k < l1) {
                        v[k] = *reinterpret_cast<const uint4*>(base + (l + k) * layer + f + piece * 16);
                        if (scales && piece == 0) s[k] = scales[(l + k) * p.s_layer + sf];
                    }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < kMoveLayers; ++k)
                    if (act && l + k < l1) {
                        *reinterpret_cast<uint4*>(base + (l + k) * layer + t + piece * 16) = v[k];
                        if (scales && piece == 0) scales[(l + k) * p.s_layer + st] = s[k];
                    }
            }
            __syncwarp();
        }
        if (n < 32) break;
    }
    bad = __any_sync(0xffffffffu, bad);
    if (reports && lane == 0) {
        p.out[b] = first + count;
        if (bad && p.status) atomicOr(p.status, kErrBadIndex);
    }
}

cudaError_t launch_copy_pages(const CopyPagesParams& p_in, cudaStream_t st) {
    CopyPagesParams p = p_in;
    const long long pieces = (long long)p.page_size * p.row_pieces * p.Hkv;
    p.parts = (int)((pieces + kCopyBlock - 1) / kCopyBlock);
    const long long grid = (long long)p.N * p.layers * 2 * p.parts;
    if (grid >= (1LL << 31)) return cudaErrorInvalidValue;
    return launch_pdl(copy_pages_kernel, dim3((unsigned)grid), dim3(kCopyThreads), 0, st, p);
}

cudaError_t launch_compact_drafts(const CompactParams& p_in, int sms, cudaStream_t st) {
    CompactParams p = p_in;
    p.lpr_shift = 0;
    while ((1 << p.lpr_shift) < p.row_pieces) ++p.lpr_shift;
    // a warp's layers share its index arithmetic; fewer each where that leaves SMs without warps (one sequence 2.6 us, all
    // layers in one warp 3.8; 128 sequences 9.7, in one warp 18.2, always in parts of four layers 10.6)
    const long long warps = 2LL * p.B * p.Hkv, most = (p.layers + kMoveLayers - 1) / kMoveLayers;
    const long long parts = (32LL * sms + warps - 1) / warps;
    p.layer_parts = (int)(parts < 1 ? 1 : parts < most ? parts : most);
    const long long grid = (warps * p.layer_parts + kMoveWarps - 1) / kMoveWarps;
    if (grid >= (1LL << 31)) return cudaErrorInvalidValue;
    return launch_pdl(compact_drafts_kernel, dim3((unsigned)grid), dim3(kMoveWarps * 32), 0, st, p);
}

}  // namespace moe
