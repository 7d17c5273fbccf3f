// dan_attn_tile.cu -- attention over the paged cache for sequences with more
// than 16 query rows (n_s * heads/kv_heads): prompts, chunks, long drafts.
//
// Mathematics: the same one-pass softmax as the step kernel.  Rows are
// (token, query head of the group) pairs, tokens outermost, so that a tile
// of rows shares its keys; 4 * hd flops per (row, key) against 2 * 2 * hd
// bytes per key for 256 rows: the bound is the tensor cores, and beside them
// one exponential per (row, key).  Measured on one GB300: a prompt of 4216
// tokens, 32 query and 8 key heads of 128, 114 us, 1.27 PFLOP/s, 0.65 of a
// large library product's rate; the tensor pipe is busy 79% of the time in the
// middle of an item.
//
// One persistent CTA per SM, work items (sequence, tile, split, key head) from
// a list that a block of the step kernel wrote, longest first, taken in turn
// from a counter.  Roles:
//   warps 0-3, 4-7  softmax of row tiles A and B (128 rows each, a row per
//                   thread): scores out of TMEM, probabilities back into it
//   warp 8          issues every tcgen05 product
//   warp 9          takes the items and brings K and V by TMA (128 keys each)
//   warp 10         brings the item's query rows by TMA
//   warp 11         follows the blocks: clears value rows that no query sees,
//                   vouches for a block's K and V, gives its stages back
// Per 128 keys and row tile: S = Q K^T (operands in shared memory, result in
// TMEM), softmax, P (bf16) over S's columns in TMEM, O += P V with P read
// from TMEM.  The tensor pipe runs in issue order: O_A(j), S_A(j+1), O_B(j),
// S_B(j+1), so each tile's softmax has the other tile's two products to hide
// behind.  The completion of S(j+1) implies that of O(j).
//
// The reference m of a row's exponentials need not be its maximum, only near
// enough for fp32 and bf16 range.  It is the maximum of the first block of
// which the row sees a key.  Where a later block sums to more than 2^10, m
// rises after it by that sum's exponent, and the row's sum and output are
// scaled by the same power of two, exactly; where it sums to more than 2^24,
// the block's maximum is found and the block taken again.  Each choice is the
// row's own, so bits do not depend on its neighbours.  Finding every block's
// maximum first cost a third of the softmax's time.
#include "dan_device.cuh"
#include "dan_internal.h"
#include "dan_attn.cuh"
#include "dan_attn_tma.cuh"
#include "dan_ring.cuh"

namespace dan {

constexpr int kTileThreads = 384;
constexpr int kTileItems = 2; // item slots between warp 9 and the others
constexpr int kTileBarBytes = 768;

template <int HD>
struct TileShape {
    static constexpr int HALVES = HD / 64;
    static constexpr int HALF = 128 * 128;       // 128 rows of 128 bytes
    static constexpr int MAT = HALVES * HALF;    // Q tile, K tile or V tile
    static constexpr int STAGES = HD == 128 ? 5 : 10;
    static constexpr int Q_OFF = 0;
    static constexpr int KV_OFF = 2 * MAT;
    static constexpr int BAR_OFF = KV_OFF + STAGES * MAT;
    static constexpr int SMEM = BAR_OFF + kTileBarBytes + 1024;
    // TMEM columns
    static constexpr int S_COL = 0;   // S_A, S_B: 128 each; P over the first 64 of each
    static constexpr int O_COL = 256; // O_A, O_B: HD each
};

struct TileBars {
    uint64_t kv_full[10], kv_empty[10];
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], o_empty[2];
    uint64_t item_full[kTileItems], item_empty[kTileItems];
    uint64_t drain;
    TileItem item[kTileItems];
    uint32_t tmem, dead; // dead: a wait ran out
};
static_assert(sizeof(TileBars) <= kTileBarBytes, "barrier area");

// ------------------------------------------------------- tcgen05 primitives

__device__ __forceinline__ void tc_fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// One lane of the converged warp, the same one each time.  The compiler knows
// that this picks one lane and keeps descriptors in uniform registers: with a
// branch on the lane number each product took 130 cycles to issue instead of
// its 64 (128 x 128 x 16, measured on GB300).
__device__ __forceinline__ bool elect_one()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(e));
    return e != 0;
}
// Arrive on `bar` when every product issued so far by this thread is done.
__device__ __forceinline__ void tc_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
                 : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
                 : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle.  sbo: bytes between
// groups of 8 rows of 128 bytes; lbo: bytes between 64-column blocks of a
// matrix whose columns are the contiguous dimension (else unused).
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(lbo >> 4) << 16) |
           ((uint64_t)(sbo >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: bf16 x bf16 -> fp32, M = 128; b_cols: B's columns
// are its contiguous dimension.
__host__ __device__ constexpr uint32_t tc_idesc(int n, bool b_cols)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_cols ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           (8u << 24);
}

#define DAN_R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), \
                     "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define DAN_I8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), \
                     "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])

// 32 columns of this warp's 32 lanes (a lane per thread).
__device__ __forceinline__ void tc_ld32(uint32_t *r, uint32_t addr)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : DAN_R8(r, 0), DAN_R8(r, 8), DAN_R8(r, 16), DAN_R8(r, 24)
                 : "r"(addr));
}
__device__ __forceinline__ void tc_ld16(uint32_t *r, uint32_t addr)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : DAN_R8(r, 0), DAN_R8(r, 8)
                 : "r"(addr));
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
                 DAN_I8(r, 0), DAN_I8(r, 8)
                 : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pk2(a)), "l"(pk2(b)), "l"(pk2(c)));
    return upk2(r);
}

// ------------------------------------------------------------------- main

// A wait of a role, each lane by itself.  One that runs out marks the CTA dead;
// from then on every wait returns at once and the roles run to their end (on
// whatever the buffers hold; no address depends on it but an item's, and no
// item is taken any more).
__device__ __forceinline__ void role_wait(const AttnParams &p, TileBars &B, uint64_t *bar, unsigned parity)
{
    if (mbar_try_wait(bar, parity)) return;
    const unsigned long long t0 = global_ns();
    volatile uint32_t *dead = &B.dead;
#pragma unroll 1
    while (!*dead) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return;
        if (global_ns() - t0 > p.limit_ns) {
            *dead = 1;
            set_status(p.status, kStatusWaitFull);
        }
    }
}

// The same for a whole warp, converged afterwards.
__device__ __forceinline__ void warp_wait(const AttnParams &p, TileBars &B, uint64_t *bar, unsigned parity)
{
    role_wait(p, B, bar, parity);
    __syncwarp();
}

__device__ __forceinline__ bool is_dead(TileBars &B)
{
    return __any_sync(kFull, *reinterpret_cast<volatile uint32_t *>(&B.dead) != 0);
}

// A word whose lowest n bits are set (n of any size).
__device__ __forceinline__ uint32_t low_bits(int n)
{
    return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}

// Take the next item from its slot; false when there is none or the wait ran out.
__device__ __forceinline__ bool next_item(const AttnParams &p, TileBars &B, int k, TileItem &it)
{
    const int slot = k % kTileItems;
    warp_wait(p, B, &B.item_full[slot], (k / kTileItems) & 1);
    if (is_dead(B)) return false;
    it = B.item[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&B.item_empty[slot]);
    return it.s >= 0;
}

// Four lanes with four 16-byte chunks each of their own row: afterwards v[k]
// is chunk (lane & 3) of the row of lane k of the four.
__device__ __forceinline__ void transpose4(uint4 (&v)[4])
{
    const int lane = threadIdx.x & 31;
    auto swap = [&](uint4 &a, uint4 &b, int bit) { // lanes with the bit clear give b for the other's a
        const bool up = lane & bit;
        uint4 s = up ? a : b;
        s.x = __shfl_xor_sync(kFull, s.x, bit);
        s.y = __shfl_xor_sync(kFull, s.y, bit);
        s.z = __shfl_xor_sync(kFull, s.z, bit);
        s.w = __shfl_xor_sync(kFull, s.w, bit);
        if (up) a = s;
        else b = s;
    };
    swap(v[0], v[1], 1);
    swap(v[2], v[3], 1);
    swap(v[0], v[2], 2);
    swap(v[1], v[3], 2);
}

// Keys of a block that a row sees: below `sink` or in [lo, hi), and below hi.
struct BlockMask {
    int hi, lo, sink;
    __device__ __forceinline__ bool whole() const { return hi >= 128 && (lo <= 0 || sink >= 128); }
    __device__ __forceinline__ bool some() const { return hi > 0 && (sink > 0 || lo < min(hi, 128)); }
    // keys 32c .. 32c+31, a bit each
    __device__ __forceinline__ uint32_t bits(int c) const
    {
        return low_bits(hi - 32 * c) & (low_bits(sink - 32 * c) | ~low_bits(lo - 32 * c));
    }
};

// -infinity in place of the scores that the row does not see: a bit per key
// and no branch per key (measured: branches took about 9000 cycles a block).
__device__ __forceinline__ void mask_chunk(uint32_t *x, uint32_t see)
{
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = (see >> e) & 1u ? x[e] : 0xFF800000u;
}

// Half a row's block: probabilities 2^(x * scale - z) of 64 scores, in pairs
// rounded to bf16 for the product with V, on their way into TMEM when it
// returns; the sum of the unrounded ones.  (The product takes two operands of
// one type, and V is bf16: relative 2^-8 at most each, as in the step kernel.)
__device__ __forceinline__ float half_exp(uint32_t p_addr, const uint32_t *x, float scale_log2, float z)
{
    const float2 scale = dup2(scale_log2), minus_z = dup2(-z);
    float2 sum0 = make_float2(0, 0), sum1 = make_float2(0, 0);
    uint32_t pk[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        float2 v = fma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), scale, minus_z);
        v.x = exp2_fast(v.x);
        v.y = exp2_fast(v.y);
        if (e & 1) sum1 = add2(sum1, v);
        else sum0 = add2(sum0, v);
        pk[e] = pack_bf16(v.x, v.y);
    }
    tc_st16(p_addr, pk);
    tc_st16(p_addr + 16, pk + 16);
    sum0 = add2(sum0, sum1);
    return sum0.x + sum0.y;
}

// A block's sum above which m rises after it, and above which the block is taken
// again.  They bound the row's sum: at most 2^10 from each block that leaves m
// where it is, 2^24 from one after which it rises (which then divides what is
// there by 2^10 or more), so 2^24 + 8 kv_len in all and 16 times 2^24 over joined
// splits.  Outputs are that times the largest value before the division, bf16's
// rounding of the probabilities included: with values up to 2^99 at most
// 2^99 * (2^28 + 2^27) * 1.004 < 2^128 for 2^24 keys, and with 2^94 likewise for 2^30.
constexpr float kRiseSum = 1024.0f;
constexpr float kAgainSum = 16777216.0f;

template <int HD>
__device__ __forceinline__ void tile_softmax(const AttnParams &p, TileBars &B, uint32_t tmem)
{
    using Sh = TileShape<HD>;
    const int t = threadIdx.x >> 7, wq = (threadIdx.x >> 5) & 3;
    const int lane = threadIdx.x & 31, trow = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t s_addr = tmem + lanes + Sh::S_COL + t * 128;
    const uint32_t o_addr = tmem + lanes + Sh::O_COL + t * HD;
    const int tq = 128 / p.g, tl = trow / p.g, head = trow - tl * p.g; // the row's token and head
    unsigned s_phase = 0, o_phase = 0;
    TileItem it;
    for (int k = 0; next_item(p, B, k, it); ++k) {
        if (t == 1 && it.ntok <= tq) continue; // no rows in tile B
        const int tok = it.tok0 + t * tq + tl; // token of the sequence
        const bool live = tl < tq && t * tq + tl < it.ntok;
        const RowRange rr = live ? row_range(p, it.pos0 + tok, it.L) : RowRange{0, 0, 0};
        float m = -INFINITY, l = 0.0f;
        int rise = 0; // by which m goes up before the next block
        for (int j = it.b0; j < it.b1; ++j) {
            const int key0 = it.key_of(j);
            const BlockMask bm = {rr.hi - key0, rr.lo - key0, rr.sink - key0};
            const bool part = __any_sync(kFull, live && !bm.whole()), some = live && bm.some();
            warp_wait(p, B, &B.s_full[t], s_phase);
            s_phase ^= 1;
            tc_fence_after();
            // O(j-1) is complete (see above)
            auto scale_output = [&](float f) {
                l *= f;
#pragma unroll 1
                for (int c = 0; c < HD; c += 16) {
                    uint32_t o[16];
                    tc_ld16(o, o_addr + c);
                    tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                    tc_st16(o_addr + c, o);
                }
            };
            if (__any_sync(kFull, rise != 0)) {
                scale_output(__uint_as_float((uint32_t)(127 - rise) << 23));
                m += (float)rise;
                rise = 0;
            }
            uint32_t x[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tc_ld32(x + 32 * c, s_addr + 32 * c);
            tc_wait_ld();
            if (part) {
#pragma unroll
                for (int c = 0; c < 4; ++c) mask_chunk(x + 32 * c, bm.bits(c));
            }
            // P goes over the scores, which stay in registers
            auto block_exp = [&] {
                const float z = m == -INFINITY ? 0.0f : m;
                const float a = half_exp(s_addr, x, p.scale_log2, z);
                return a + half_exp(s_addr + 32, x + 64, p.scale_log2, z);
            };
            float sum = 0.0f;
            bool again = m == -INFINITY && some;
            if (j > it.b0) { // (a first block always looks for its maximum)
                sum = block_exp();
                again = again || (live && sum > kAgainSum);
            }
            if (j == it.b0 || __any_sync(kFull, again)) {
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < 128; ++c) top = fmaxf(top, __uint_as_float(x[c]));
                top *= p.scale_log2;
                again = again && top > m;
                tc_wait_st();
                if (j > it.b0) scale_output(again ? exp2_fast(m - top) : 1.0f);
                if (again) m = top;
                sum = block_exp();
            }
            if (live && sum > kRiseSum && sum <= kAgainSum) rise = (int)(__float_as_uint(sum) >> 23) - 127;
            l += sum;
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.p_full[t]);
        }
        // The row's output, straight from TMEM: whole, or a split's part.
        const bool any = it.b1 > it.b0, part = it.nsplit > 1;
        const float inv = part ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
        const SeqInfo q = {it.q0, it.n, it.L, false};
        const int64_t orow = live ? (int64_t)(it.q0 + tok) * p.H + it.u * p.g + head : -1;
        const int64_t prow =
            live ? part_base(p, p.tile_part, it.s, q, it.u) + (int64_t)it.split * it.n * p.g + tok * p.g + head : -1;
        const int64_t base = part ? prow : orow;
        if (live) {
            if (part) p.part_ml[prow] = make_float2(m, l);
            else if (p.lse) p.lse[orow] = row_lse(m, l);
        }
        if (any) {
            warp_wait(p, B, &B.o_full[t], o_phase);
            o_phase ^= 1;
            tc_fence_after();
        }
        int64_t rows4[4]; // the rows that this lane's four stores go to
#pragma unroll
        for (int i = 0; i < 4; ++i) rows4[i] = __shfl_sync(kFull, base, (lane & ~3) + i);
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
            uint32_t o[32];
            __syncwarp();
            if (any) { // warp-uniform
                tc_ld32(o, o_addr + c);
                tc_wait_ld();
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0u;
            }
            // Four lanes trade chunks so that each store writes 64 bytes of a row
            // (a row per lane wrote 16 at a time: an item's epilogue took 6600 cycles,
            // now 2600).
            if (part) {
#pragma unroll
                for (int hc = 0; hc < 2; ++hc) {
                    uint4 v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = make_uint4(o[16 * hc + 4 * i], o[16 * hc + 4 * i + 1],
                                          o[16 * hc + 4 * i + 2], o[16 * hc + 4 * i + 3]);
                    transpose4(v);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (rows4[i] >= 0)
                            *reinterpret_cast<uint4 *>(p.part_o + rows4[i] * HD + c + 16 * hc +
                                                       4 * (lane & 3)) = v[i];
                }
            } else {
                uint4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        set_word(v[i], e, pack_bf16(__uint_as_float(o[8 * i + 2 * e]) * inv,
                                                    __uint_as_float(o[8 * i + 2 * e + 1]) * inv));
                transpose4(v);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (rows4[i] >= 0) p.out[(rows4[i] * HD + c) / 8 + (lane & 3)] = v[i];
            }
        }
        if (any) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.o_empty[t]);
        }
    }
}

// All of it in one elected lane, and as little as can be between a wait and
// its products.  A commit holds the lane until the products before it have
// been taken up (about 300 cycles), so each tile's block has one: the scores'.
template <int HD>
__device__ __forceinline__ void tile_mma(const AttnParams &p, TileBars &B, char *smem, uint32_t tmem)
{
    using Sh = TileShape<HD>;
    constexpr uint32_t id_s = tc_idesc(128, false), id_o = tc_idesc(HD, true);
    const uint32_t base = smem_addr(smem);
    const uint64_t q0 = tc_desc(base + Sh::Q_OFF, 16, 1024);
    const uint64_t k0 = tc_desc(base + Sh::KV_OFF, 16, 1024);
    const uint64_t v0 = tc_desc(base + Sh::KV_OFF, Sh::HALF, 1024);
    unsigned stage = 0, kv_phase = 0;               // of the next block, keys or values
    unsigned q_phase = 0, p_phase = 0, o_phase = 3; // a bit for each row tile
    auto wait_tile = [&](uint64_t *bars, int t, unsigned &phase) {
        role_wait(p, B, bars + t, (phase >> t) & 1);
        phase ^= 1u << t;
    };
    auto advance = [&] {
        const unsigned st = stage;
        if (++stage == Sh::STAGES) stage = 0, kv_phase ^= 1;
        return st;
    };
    auto product_s = [&](int t, unsigned st) {
        const uint64_t qd = q0 + (uint64_t)((t * Sh::MAT) >> 4), kd = k0 + (uint64_t)((st * Sh::MAT) >> 4);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
            const uint64_t off = (uint64_t)(((k >> 2) * Sh::HALF + (k & 3) * 32) >> 4);
            tc_mma_ss(tmem + Sh::S_COL + t * 128, qd + off, kd + off, id_s, k > 0);
        }
        tc_commit(&B.s_full[t]);
    };
    TileItem it;
    for (int n = 0; next_item(p, B, n, it); ++n) {
        const int nt = it.b1 - it.b0, last = it.ntok > 128 / p.g ? 1 : 0; // last active row tile
        if (elect_one()) {
            if (nt > 0) role_wait(p, B, &B.kv_full[stage], kv_phase);
            unsigned kst = nt > 0 ? advance() : 0; // the key block's stage
            // every loaded query tile is released, used or not
            for (int t = 0; t <= last; ++t) {
                wait_tile(B.q_full, t, q_phase);
                if (nt <= 0) {
                    mbar_arrive(&B.q_empty[t]);
                    continue;
                }
                tc_fence_after();
                product_s(t, kst);
                if (nt == 1) tc_commit(&B.q_empty[t]);
            }
            for (int j = 0; j < nt; ++j) {
                const unsigned vst = advance();
                const bool more = j + 1 < nt;
                if (more) kst = advance();
                const uint64_t vd = v0 + (uint64_t)((vst * Sh::MAT) >> 4);
                for (int t = 0; t <= last; ++t) {
                    if (j == 0) wait_tile(B.o_empty, t, o_phase); // the previous item's output has been read
                    wait_tile(B.p_full, t, p_phase); // P, and V(j) and K(j+1) too
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        tc_mma_ts(tmem + Sh::O_COL + t * HD, tmem + Sh::S_COL + t * 128 + k * 8,
                                  vd + (uint64_t)(k * 2048 >> 4), id_o, j > 0 || k > 0);
                    if (more) {
                        product_s(t, kst);
                        if (j + 2 == nt) tc_commit(&B.q_empty[t]);
                    } else {
                        tc_commit(&B.o_full[t]);
                    }
                }
            }
        }
        __syncwarp();
    }
    // every product is done before the TMEM is given back
    if (elect_one()) tc_commit(&B.drain); // the lane that issued them
    __syncwarp();
    if (!mbar_wait(&B.drain, 0, p.limit_ns)) set_status(p.status, kStatusWaitDrain);
}

// Follows the blocks of an item.  Before the products of block j may run (its
// arrival on p_full beside the softmax's): V(j) and K(j+1) have landed, and
// value rows that no row of the tile sees, which may hold anything, are zeros.
// When the last tile's scores of block j are there, its products have read
// K(j) and V(j-1): those stages go back to the loader.
template <int HD>
__device__ __forceinline__ void tile_follow(const AttnParams &p, TileBars &B, char *smem)
{
    using Sh = TileShape<HD>;
    const int lane = threadIdx.x & 31;
    unsigned stage = 0, phase = 0;                  // of the next block that lands
    unsigned given = 0;                             // the next stage to give back
    unsigned s_phase = 0, o_phase = 0;              // a bit for each row tile
    auto landed = [&] {
        warp_wait(p, B, &B.kv_full[stage], phase);
        const unsigned st = stage;
        if (++stage == Sh::STAGES) stage = 0, phase ^= 1;
        return st;
    };
    auto give_back = [&] {
        if (lane == 0) mbar_arrive(&B.kv_empty[given]);
        if (++given == Sh::STAGES) given = 0;
    };
    TileItem it;
    for (int n = 0; next_item(p, B, n, it); ++n) {
        const int last = it.ntok > 128 / p.g ? 1 : 0;
        if (it.b0 < it.b1) landed(); // K of the first block
        for (int j = it.b0; j < it.b1; ++j) {
            const unsigned vst = landed();
            const int key0 = it.key_of(j);
            if (key0 + 128 > it.hi || (key0 < it.lo && key0 + 128 > it.sink)) {
                char *v = smem + Sh::KV_OFF + vst * Sh::MAT;
                for (int r = lane; r < 128; r += 32) {
                    const int key = key0 + r;
                    if (key >= it.hi || (key >= it.sink && key < it.lo))
                        for (int c = 0; c < Sh::HALVES * 8; ++c)
                            *reinterpret_cast<uint4 *>(v + (c >> 3) * Sh::HALF + r * 128 + (c & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            }
            if (j + 1 < it.b1) landed();
            for (int t = 0; t <= last; ++t) {
                warp_wait(p, B, &B.s_full[t], (s_phase >> t) & 1);
                s_phase ^= 1u << t;
                if (lane == 0) mbar_arrive(&B.p_full[t]);
            }
            if (j > it.b0) give_back(); // V(j-1)
            give_back();                // K(j)
        }
        if (it.b0 < it.b1) {
            warp_wait(p, B, &B.o_full[last], (o_phase >> last) & 1);
            give_back(); // the last V
            o_phase ^= last ? 3 : 1;
        }
    }
}

template <int HD>
__device__ __forceinline__ void tile_load(const AttnParams &p, TileBars &B, char *smem,
                                          const CUtensorMap &kmap, const CUtensorMap &vmap)
{
    using Sh = TileShape<HD>;
    const int lane = threadIdx.x & 31;
    const int total = p.plan_head[0] * p.Hkv;
    const int box = min(128, 1 << p.page_shift), per = 128 / box; // pages of a key block
    const int rows_total = (p.num_pages * p.Hkv) << p.page_shift;
    unsigned kv = 0;
    // Take the next item off the list and put it in its slot, one ahead of the
    // loads, so that the other roles have it when they are done with theirs.
    auto post = [&](int k) {
        int4 raw; // lane l < 5: the item's l-th 16 bytes
        do {      // (-2: one that the plan left out)
            int w = 0;
            if (lane == 0) w = atomicAdd(p.plan_head + 2, 1);
            w = __shfl_sync(kFull, w, 0);
            raw = make_int4(-1, 0, 0, 0);
            if (w < total && lane < 5) {
                raw = reinterpret_cast<const int4 *>(p.items + w / p.Hkv)[lane];
                if (lane == 0) raw.y = w % p.Hkv;
            }
        } while (__shfl_sync(kFull, raw.x, 0) == -2);
        const int slot = k % kTileItems;
        warp_wait(p, B, &B.item_empty[slot], ((k / kTileItems) & 1) ^ 1);
        if (is_dead(B)) return; // the slot may still be read
        if (lane < 5) reinterpret_cast<int4 *>(&B.item[slot])[lane] = raw;
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.item_full[slot]);
    };
    post(0);
    for (int k = 0; !is_dead(B); ++k) {
        const TileItem it = B.item[k % kTileItems]; // (this warp wrote it)
        if (it.s < 0) break;
        post(k + 1);
        const int32_t *trow = p.table + (int64_t)it.s * p.table_stride;
        // Lane l < per: first cache row of page l of key block j (a page that no
        // row sees, or an id out of range: past the end, where the copy gives zeros)
        auto cache_row = [&](int j) {
            if (lane >= per || j >= it.b1) return rows_total;
            const int key = it.key_of(j) + lane * box, end = key + box;
            const bool see = (it.lo < it.hi && key < it.hi && end > it.lo) || key < it.sink;
            if (!see) return rows_total;
            const int page = __ldg(trow + (key >> p.page_shift));
            if (page < 0 || page >= p.num_pages) {
                set_status(p.status, kStatusIndex);
                return rows_total;
            }
            return ((page * p.Hkv + it.u) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
        };
        int rows = cache_row(it.b0);
        for (int j = it.b0; j < it.b1; ++j) {
            const int next = cache_row(j + 1); // in flight while this block's copies start
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int st = kv % Sh::STAGES;
                warp_wait(p, B, &B.kv_empty[st], ((kv / Sh::STAGES) & 1) ^ 1);
                if (is_dead(B)) break;
                if (lane == 0) mbar_arrive_expect_tx(&B.kv_full[st], Sh::MAT);
                __syncwarp();
                if (lane < per) {
                    char *dst = smem + Sh::KV_OFF + st * Sh::MAT + lane * box * 128;
#pragma unroll
                    for (int h = 0; h < Sh::HALVES; ++h)
                        tma_load_2d(dst + h * Sh::HALF, m ? &vmap : &kmap, h * 64, rows, &B.kv_full[st]);
                }
                ++kv;
                __syncwarp();
            }
            rows = next;
        }
    }
    // copies still in flight (after a wait that ran out) land before the CTA ends
    for (unsigned i = kv > Sh::STAGES ? kv - Sh::STAGES : 0; i < kv; ++i)
        if (!mbar_wait(&B.kv_full[i % Sh::STAGES], (i / Sh::STAGES) & 1, p.limit_ns))
            set_status(p.status, kStatusWaitDrain);
}

// Query rows into the swizzled tiles: whole tokens of the key head's group.
// Rows of tokens past the tile's own are another sequence's or zeros, and the
// last 128 % g rows whatever stood there; none of them is looked at.
template <int HD>
__device__ __forceinline__ void tile_queries(const AttnParams &p, TileBars &B, char *smem,
                                             const CUtensorMap &qmap)
{
    using Sh = TileShape<HD>;
    const int lane = threadIdx.x & 31, tq = 128 / p.g;
    unsigned phase[2] = {1, 1};
    TileItem it;
    for (int k = 0; next_item(p, B, k, it); ++k)
        for (int t = 0; t < (it.ntok > tq ? 2 : 1); ++t) {
            warp_wait(p, B, &B.q_empty[t], phase[t]);
            phase[t] ^= 1;
            if (lane == 0) {
                mbar_arrive_expect_tx(&B.q_full[t], (unsigned)(Sh::HALVES * tq * p.g * 128));
                for (int h = 0; h < Sh::HALVES; ++h)
                    tma_load_3d(smem + Sh::Q_OFF + t * Sh::MAT + h * Sh::HALF, &qmap, h * 64, it.u * p.g,
                                it.q0 + it.tok0 + t * tq, &B.q_full[t]);
            }
            __syncwarp();
        }
    // copies still in flight (after a wait that ran out) land before the CTA ends
    for (int t = 0; t < 2; ++t)
        if (is_dead(B) && !mbar_wait(&B.q_full[t], phase[t], p.limit_ns))
            set_status(p.status, kStatusWaitDrain);
}

template <int HD>
__global__ void __launch_bounds__(kTileThreads, 1)
    window_attention_tile_kernel(const AttnParams p, const __grid_constant__ CUtensorMap qmap,
                                 const __grid_constant__ CUtensorMap kmap,
                                 const __grid_constant__ CUtensorMap vmap)
{
    using Sh = TileShape<HD>;
    extern __shared__ char smem_raw[];
    char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    TileBars &B = *reinterpret_cast<TileBars *>(smem + Sh::BAR_OFF);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        prefetch_map(&qmap);
        prefetch_map(&kmap);
        prefetch_map(&vmap);
        for (int i = 0; i < Sh::STAGES; ++i) {
            mbar_init(&B.kv_full[i], 1);
            mbar_init(&B.kv_empty[i], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&B.q_full[t], 1);
            mbar_init(&B.q_empty[t], 1);
            mbar_init(&B.s_full[t], 1);
            mbar_init(&B.p_full[t], 5); // the four softmax warps and warp 11
            mbar_init(&B.o_full[t], 1);
            mbar_init(&B.o_empty[t], 4);
        }
        for (int i = 0; i < kTileItems; ++i) {
            mbar_init(&B.item_full[i], 1);
            mbar_init(&B.item_empty[i], 11); // every warp but 9
        }
        mbar_init(&B.drain, 1);
        B.dead = 0;
        mbar_init_fence();
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_addr(&B.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = B.tmem;
    grid_dependency_wait(); // the plan, and what came before it
    allow_dependents();
    // Registers from the third warpgroup to the softmax: 128 * (208 + 208 + 88) =
    // 384 * 168, what the block was launched with (kTileRegs, checked before the launch).
    if (warp < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp < 8) {
        tile_softmax<HD>(p, B, tmem);
    } else if (warp == 8) {
        tile_mma<HD>(p, B, smem, tmem);
    } else if (warp == 9) {
        tile_load<HD>(p, B, smem, kmap, vmap);
    } else if (warp == 10) {
        tile_queries<HD>(p, B, smem, qmap);
    } else {
        tile_follow<HD>(p, B, smem);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

namespace {

// The registers that the kernel's split takes from and gives to its warps: with
// fewer at launch the split would wait for ever.  The count is asked for until
// it is known (a failed query is not kept).
constexpr int kTileRegs = 168;

template <int HD>
cudaError_t ready_tile_hd()
{
    const void *fn = reinterpret_cast<const void *>(window_attention_tile_kernel<HD>);
    static DeviceCache<int> regs;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int n = cached_per_device(regs, dev, [&] {
        cudaFuncAttributes at = {};
        e = cudaFuncGetAttributes(&at, fn);
        return e == cudaSuccess ? at.numRegs : 0;
    });
    if (e != cudaSuccess) return e;
    if (n != kTileRegs) return cudaErrorInvalidConfiguration;
    return allow_dynamic_smem(fn, TileShape<HD>::SMEM);
}

template <int HD>
cudaError_t launch_tile_hd(const AttnParams &p, const CUtensorMap &qmap, const CUtensorMap &kmap,
                           const CUtensorMap &vmap, cudaStream_t s)
{
    const int64_t work = (int64_t)p.items_cap * p.Hkv;
    const int grid = (int)(work < sm_count() ? work : sm_count());
    return launch_overlapped_2d(window_attention_tile_kernel<HD>, dim3((unsigned)grid), kTileThreads,
                                TileShape<HD>::SMEM, s, p, qmap, kmap, vmap);
}

} // namespace

cudaError_t ready_attention_tile(int head_dim)
{
    return head_dim == 64 ? ready_tile_hd<64>() : ready_tile_hd<128>();
}

cudaError_t launch_attention_tile(const AttnParams &p, int head_dim, const CUtensorMap &qmap,
                                  const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t s)
{
    return head_dim == 64 ? launch_tile_hd<64>(p, qmap, kmap, vmap, s)
                          : launch_tile_hd<128>(p, qmap, kmap, vmap, s);
}

} // namespace dan
