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

// Sum over the block's threads up to and with this one; any: whether one of
// them has the flag.
__device__ __forceinline__ int plan_scan(int x, int *s_warp, bool flag, bool &any)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    any = __syncthreads_or(flag);
    for (int w = 0; w < warp; ++w) x += s_warp[w];
    __syncthreads();
    return x;
}

// Whether the sequence of this thread, rows first .. end-1, begins before the
// end of one before it: of an earlier thread's, or of what any thread has seen
// in earlier turns (`reach`).  Apart from the plan, which seldom needs it.
__device__ __noinline__ bool plan_overlaps(int first, int end, int reach, int *s_warp)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        reach = max(reach, __shfl_xor_sync(kFull, reach, o));
        const int y = __shfl_up_sync(kFull, end, o);
        if (lane >= o) end = max(end, y);
    }
    // ends >= 0 up to and with this thread's; the warp's own, and of earlier turns
    const int before = __shfl_up_sync(kFull, end, 1);
    if (lane == 0) s_warp[warp] = reach;
    __syncthreads();
    for (int w = 0; w < kPlanThreads / 32; ++w) reach = max(reach, s_warp[w]);
    __syncthreads();
    if (lane == 31) s_warp[warp] = end;
    __syncthreads();
    if (lane > 0) reach = max(reach, before);
    for (int w = 0; w < warp; ++w) reach = max(reach, s_warp[w]);
    __syncthreads();
    return first < reach;
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
        // An earlier end lies past a later start only where a start lies past the
        // next one: until one does, no sequence is compared with the others
        // (always comparing cost the call of a prompt 0.8 us, this 0.3).
        bool descended = false, any;
        int reach = 0; // furthest end that this thread has seen in earlier turns
        for (int s0 = 0; s0 < p.S; s0 += kPlanThreads) {
            int tiles = 0, first = 0, end = 0;
            bool down = false;
            if (s0 + tid < p.S) {
                const SeqInfo q = seq_info(p, s0 + tid);
                tiles = q.n * p.g > kStepRows ? seq_tiles(p, q) : 0;
                if (q.n > 0) first = q.q0, end = q.q0 + q.n;
                down = q.down;
            }
            int upto = plan_scan(tiles, S.warp, down, any);
            descended = descended || any;
            if (descended) { // the whole block
                if (plan_overlaps(first, end, reach, S.warp) && tiles) {
                    tiles = 0;
                    set_status(p.status, kStatusIndex);
                }
                upto = plan_scan(tiles, S.warp, false, any);
            }
            reach = max(reach, end);
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
            int before = plan_scan(sum, S.warp, false, any) - sum;
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
