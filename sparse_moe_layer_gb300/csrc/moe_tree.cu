// Attention of drafted tokens: how the work is split, the launches, and the join of cut items (moe_tree.cuh has
// the kernel).
#include "moe_tree.cuh"

namespace moe {

// Joins the parts of items cut by a run's border.  blockIdx.x: a run that continues an
// item as the first to do so; blockIdx.y: 32 rows, one a lane; a warp has every 8th
// four dims.  Parts: slot 1 of the run before, slot 0 of the runs that continue the item.
constexpr int kTreeJoinWarps = 8;

template <bool QF16>
__global__ void __launch_bounds__(kTreeJoinWarps * 32) tree_join_kernel(TreeParams p, int ROWS) {
    pdl_wait();
    pdl_allow_dependents();
    const int j = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto same = [](const int4& a, const int4& b) { return a.w && b.w && a.x == b.x && a.y == b.y && a.z == b.z; };
    const int4 item = p.cont[j];
    if (!item.w || same(item, p.cont[j - 1])) return;
    // (a workspace that overlapping calls share holds anything: wrong sums, but no stray access)
    if ((unsigned)item.x >= (unsigned)p.B || (unsigned)item.y >= (unsigned)p.Hkv || item.z < 0 || item.z > kMaxDrafts * 32)
        return;
    const int lo = __ldg(p.starts + item.x), hi = __ldg(p.starts + item.x + 1);
    if (lo < 0 || hi < lo || hi > p.N || hi - lo > kMaxDrafts) return;
    const int n = hi - lo;
    const int row = blockIdx.y * 32 + lane, at = item.z * ROWS + row;
    if (blockIdx.y * 32 + item.z * ROWS >= n * p.group) return;
    int parts = 1;
    for (bool more = true; more;) {
        const int r = j + parts - 1 + lane;
        const uint32_t s = __ballot_sync(kAllLanes, r < p.runs && same(p.cont[r], item));
        parts += s == kAllLanes ? 32 : __ffs(~s) - 1;
        more = s == kAllLanes;
    }
    const long long size = (long long)ROWS * (p.D + 2);
    auto part = [&](int i) { return p.partial + ((long long)(j - 1 + i) * 2 + (i == 0 ? 1 : 0)) * size; };
    if (at >= n * p.group) return;
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < parts; ++i) {
        const float2 ml = reinterpret_cast<const float2*>(part(i))[row];
        const float t = fmaxf(m, ml.x);
        l = t == -INFINITY ? 0.f : l * ex2_approx(m - t) + ml.y * ex2_approx(ml.x - t);
        m = t;
    }
    const int d = at / p.group, head = item.y * p.group + at - d * p.group;
    const float fw = final_weight(p.sinks, head, m, l);
    uint16_t* dst = p.out + (lo + d) * p.o_token + (long long)head * p.o_head;
    for (int c = warp; c < p.D / 4; c += kTreeJoinWarps) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < parts; ++i) {
            const float* q = part(i);
            const float e = m == -INFINITY ? 0.f : ex2_approx(reinterpret_cast<const float2*>(q)[row].x - m);
            add_scaled(x, 1.f, reinterpret_cast<const float4*>(q + 2 * ROWS)[c * ROWS + row], e);
        }
        *reinterpret_cast<uint2*>(dst + 4 * c) = make_uint2(pack2<QF16>(x.x * fw, x.y * fw), pack2<QF16>(x.z * fw, x.w * fw));
    }
}

void tree_plan(int N, int B, int Hq, int Hkv, int D, int page_size, int window, int most, int sms, TreePlan* w) {
    const long long rows = ((long long)N * (Hq / Hkv) + B - 1) / B;  // of a sequence and key head, on average
    // two row tiles share a tile of keys and values (they fit to 128 dims): 64 drafts of 8 heads 236 us, one by one 239;
    // 16 drafts of 16 heads of 128, e4m3, converted once instead of twice: 286, 446.  By the batch's average: one large
    // tree among many single drafts has one row tile at a time.
    w->tiles = D <= 128 && rows > kTreeRows ? 2 : 1;
    w->ctas = w->tiles == 2 || D > 64 ? sms : 2 * sms;
    const int tt = D > 128 ? 32 : w->tiles == 2 && D <= 64 ? 128 : 64;
    // (a window of `most` tokens begins anywhere in 16, and drafts come behind it)
    w->whole = (long long)most + 16 + kMaxDrafts <= kWholeTiles * tt;
    // TMA pieces of tokens that divide a page, and tiles, which start at a multiple of 16 in a window; from 8 on: pieces
    // cost the copying warp 17 cycles each (64 sequences of up to 16384 tokens, pages of 16: 176 us, by threads 286)
    const int largest = window > 0 ? 16 : tt;
    w->box = page_size & -page_size;
    if (w->box > largest) w->box = largest;
    if (w->box < 8) w->box = 0;
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    w->cont = 0;
    w->partial = up((size_t)w->ctas * 16);
    w->total = w->whole ? 0 : w->partial + (size_t)w->ctas * 2 * w->tiles * kTreeRows * (D + 2) * 4;
}

cudaError_t launch_tree(const CUtensorMap& tmK, const CUtensorMap& tmV, const TreeParams& p_in, const TreePlan& w,
                        int kv_dtype, bool fp16, void* workspace, cudaStream_t st) {
    TreeParams p = p_in;
    p.box = w.box;
    p.fp16 = fp16;
    p.group = p.Hq / p.Hkv;
    p.inv_group = 1.f / (float)p.group;
    p.whole = w.whole;
    p.runs = w.ctas;
    p.page_shift = -1;
    if ((p.page_size & (p.page_size - 1)) == 0)
        for (p.page_shift = 0; (1 << p.page_shift) < p.page_size;) ++p.page_shift;
    if (w.total) {
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        p.cont = reinterpret_cast<int4*>(ws + w.cont);
        p.partial = reinterpret_cast<float*>(ws + w.partial);
    }
    cudaError_t e;
    if (kv_dtype == kDtE4m3)
        e = launch_tree_e4m3(tmK, tmV, p, w, st);
    else
        e = fp16 ? launch_tree_fp16(tmK, tmV, p, w, st) : launch_tree_bf16(tmK, tmV, p, w, st);
    if (e != cudaSuccess || w.whole || p.runs < 2) return e;
    const int rows = w.tiles * kTreeRows;
    const dim3 grid(p.runs - 1, rows / 32), block(kTreeJoinWarps * 32);
    return fp16 ? launch_pdl(tree_join_kernel<true>, grid, block, 0, st, p, rows)
                : launch_pdl(tree_join_kernel<false>, grid, block, 0, st, p, rows);
}

}  // namespace moe
