// dan_attn_plan.cuh -- the tile kernel's work list, made by one block of the
// step kernel, so that it costs no launch and runs beside the step's work.
#pragma once

#include "dan_attn.cuh"
#include "dan_device.cuh"
#include "dan_ring.cuh"

namespace dan {

// Items (sequence, tile, split, -) longest first, and the tiles that are
// split.  plan_head: [0] items, [1] split tiles, [2] next item * Hkv + u.
constexpr int kPlanThreads = 128;

struct PlanShared {
    int first[kPlanThreads + 1]; // first tile of each sequence of a chunk of them
    int warp[kPlanThreads / 32];
    int hist[kPlanBuckets];
    int split;
};

// Sum over the block's threads up to and with this one.
__device__ __forceinline__ int plan_scan(int x, int *s_warp)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    for (int w = 0; w < warp; ++w) x += s_warp[w];
    __syncthreads();
    return x;
}

// Largest x of the block's threads before this one (0 for the first); all: of
// every thread.  Only for x >= 0.
__device__ __forceinline__ int plan_max_before(int x, int *s_warp, int &all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x = max(x, y);
    }
    if (lane == 31) s_warp[warp] = x;
    int before = __shfl_up_sync(kFull, x, 1);
    if (lane == 0) before = 0;
    __syncthreads();
    all = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) before = max(before, s_warp[w]);
        all = max(all, s_warp[w]);
    }
    __syncthreads();
    return before;
}

// A sequence that begins before an earlier one's end is left out.  So the
// planned sequences share no row, and their tiles are at most N / tile_tokens
// and one for each: the counts below fit 32 bits and the lists the places
// that the host gave them, whatever the query starts are, and the block's
// work is bounded by N and S.
__device__ __noinline__ void plan_tiles(const AttnParams &p, PlanShared &S)
{
    const int tid = threadIdx.x;
    for (int i = tid; i < kPlanBuckets; i += kPlanThreads) S.hist[i] = 0;
    if (tid == 0) S.split = 0;
    __syncthreads();
    for (int pass = 0; pass < 2; ++pass) { // count by length, then place
        int reach = 0; // where the furthest of the sequences before s0 ends
        for (int s0 = 0; s0 < p.S; s0 += kPlanThreads) {
            int tiles = 0, first = 0, end = 0;
            if (s0 + tid < p.S) {
                const SeqInfo q = seq_info(p, s0 + tid);
                tiles = q.n * p.g > kStepRows ? seq_tiles(p, q) : 0;
                if (q.n > 0) first = q.q0, end = q.q0 + q.n;
            }
            int furthest;
            const int before = max(reach, plan_max_before(end, S.warp, furthest));
            reach = max(reach, furthest);
            if (tiles && first < before) {
                tiles = 0;
                set_status(p.status, kStatusIndex);
            }
            const int upto = plan_scan(tiles, S.warp);
            S.first[tid + 1] = upto;
            if (tid == 0) S.first[0] = 0;
            __syncthreads();
            const int total = S.first[kPlanThreads];
            for (int e = tid; e < total; e += kPlanThreads) {
                int lo = 0, hi = kPlanThreads; // the sequence whose tiles hold e
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (S.first[mid] <= e) lo = mid;
                    else hi = mid;
                }
                const int seq = s0 + lo, tile = e - S.first[lo];
                const SeqInfo q = seq_info(p, seq);
                const RowRange all = tile_union(p, q, tile);
                const KeyBlocks<7> kb(all);
                const int per = tile_split_blocks(p, seq_tiles(p, q), kb.count);
                const int nsplit = max(1, (kb.count + per - 1) / per);
                const int tok0 = tile * tile_tokens(p.g), ntok = min(tile_tokens(p.g), q.n - tok0);
                const int cost = min(per, kb.count); // a block takes as long with one row tile as with two
                const int bucket = kPlanBuckets - 1 - min(kPlanBuckets - 1, cost);
                if (pass == 0) {
                    atomicAdd(&S.hist[bucket], nsplit);
                } else {
                    // (past the lists only where a caller changes the arrays meanwhile)
                    const int at = atomicAdd(&S.hist[bucket], nsplit);
                    const int sp = nsplit > 1 ? atomicAdd(&S.split, 1) : 0;
                    if (at + nsplit <= p.items_cap && (nsplit == 1 || sp < p.split_tiles_cap)) {
                        TileItem it = {seq, 0, 0, nsplit, q.q0, q.n, q.L, tok0, ntok, 0, 0, q.L - q.n,
                                       all.sink, all.lo, all.hi, kb.nsink, kb.first, {0, 0, 0}};
                        for (int k = 0; k < nsplit; ++k) {
                            it.split = k;
                            it.b0 = k * per;
                            it.b1 = min(kb.count, it.b0 + per);
                            p.items[at + k] = it;
                        }
                        if (nsplit > 1) p.split_tiles[sp] = make_int2(seq, tile);
                    } else {
                        set_status(p.status, kStatusIndex);
                        for (int k = at; k < min(at + nsplit, p.items_cap); ++k)
                            p.items[k].s = -2;
                        if (nsplit > 1 && sp < p.split_tiles_cap) p.split_tiles[sp] = make_int2(-1, 0);
                    }
                }
            }
            __syncthreads();
        }
        if (pass == 0) { // first place of each bucket
            constexpr int NB = kPlanBuckets / kPlanThreads;
            int v[NB], sum = 0;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                v[i] = S.hist[tid * NB + i];
                sum += v[i];
            }
            int before = plan_scan(sum, S.warp) - sum;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                S.hist[tid * NB + i] = before;
                before += v[i];
            }
            if (tid == kPlanThreads - 1) p.plan_head[0] = min(before, p.items_cap);
            __syncthreads();
        }
    }
    if (tid == 0) {
        p.plan_head[1] = min(S.split, p.split_tiles_cap);
        p.plan_head[2] = 0;
    }
}

} // namespace dan
