// The end of a routing kernel: the last CTA to arrive turns the (chunk, expert)
// histogram into row offsets, chunk bases and GEMM tile lists.  Shared by the
// routers and the gate kernel.
#pragma once
#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

// Run by the last CTA (blockDim 256): counts, offsets, chunk bases, tile lists.
// The (chunk, expert) histogram is first copied into `buf` (the CTA's shared
// memory, free by then) with coalesced loads when it fits in `cap` ints, so
// the per-expert sums over the chunks run from shared memory instead of one
// dependent L2 round trip per chunk.
__device__ inline void finish_scan(const RouteParams& p, int* buf, int cap) {
    __shared__ int s_count[kMaxExperts], s_off[kMaxExperts];
    const int n = p.nchunks * p.E;
    const bool staged = n <= cap;
    if (staged)
        for (int i = threadIdx.x; i < n; i += blockDim.x) buf[i] = __ldcg(&p.hist[i]);
    __syncthreads();
    auto h = [&](int c, int e) { return staged ? buf[(size_t)c * p.E + e] : __ldcg(&p.hist[(size_t)c * p.E + e]); };
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        int run = 0;
        for (int c = 0; c < p.nchunks; ++c) run += h(c, e);
        s_count[e] = run;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        // exclusive scans of the counts and of the m-tiles over the experts by
        // one warp: lane l owns experts [8l, 8l+8) (E <= 256)
        const int lane = threadIdx.x;
        int cnt[8], mt[8];
        int tc = 0, tm = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = lane * 8 + i;
            cnt[i] = e < p.E ? s_count[e] : 0;
            mt[i] = (cnt[i] + p.bm - 1) / p.bm;
            tc += cnt[i];
            tm += mt[i];
        }
        int ic = tc, im = tm;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int vc = __shfl_up_sync(0xffffffffu, ic, o);
            const int vm = __shfl_up_sync(0xffffffffu, im, o);
            if (lane >= o) {
                ic += vc;
                im += vm;
            }
        }
        int off = ic - tc, mts = im - tm;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = lane * 8 + i;
            if (e < p.E) {
                s_off[e] = off;
                p.offset[e] = off;
                p.count[e] = cnt[i];
                p.tiles1[e] = mts * p.nt1;
                p.tiles2[e] = mts * p.nt2;
            }
            off += cnt[i];
            mts += mt[i];
        }
        if (lane == 31) {
            p.offset[p.E] = off;
            p.tiles1[p.E] = mts * p.nt1;
            p.tiles2[p.E] = mts * p.nt2;
            p.status[kStatusTiles1] = (uint32_t)(mts * p.nt1);
            p.status[kStatusTiles2] = (uint32_t)(mts * p.nt2);
            p.status[kStatusTileRows] = (uint32_t)p.bm;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        int run = s_off[e];
        for (int c = 0; c < p.nchunks; ++c) {
            p.chunk_base[(size_t)c * p.E + e] = run;
            run += h(c, e);
        }
    }
}

// True in every thread of the CTA that is the `total`-th to arrive on *ctr.
// The barrier orders every thread's earlier writes before thread 0's
// GPU-scope fence, which (fences are cumulative) orders them before its
// count; in the last CTA thread 0 fences again after the count, and the
// barrier behind it orders the other threads' reads after that.
__device__ __forceinline__ bool last_to_arrive(int* ctr, int total) {
    __shared__ int s_last;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        const bool last = atomicAdd(ctr, 1) == total - 1;
        if (last) __threadfence();
        s_last = last;
    }
    __syncthreads();
    return s_last != 0;
}

}  // namespace moe
