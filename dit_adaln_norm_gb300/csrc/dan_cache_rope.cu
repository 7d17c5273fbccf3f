// dan_cache_rope.cu -- QK-RMSNorm + RoPE at given positions, with K and V
// stored into a paged cache.
//
// Mathematics, per token and head of Q and K: rstd = 1/sqrt(mean x^2 + eps),
// n = x * rstd * w, then pairs (a, b) of n turned by the angle of their
// column at the token's position; V is copied.  About 8 flops per 4 bytes
// moved: the bound is memory (and, for a few tokens, latency).  Measured on
// one GB300: 65536 tokens of 32 + 2 x 8 heads of 128, 259 us, 6.35 TB/s, 0.95
// of the copy bandwidth; 4216 tokens of 3 x 32 heads, 38 us, 5.5 TB/s.
//
// A token's heads are one list, Q then K then V.  A unit of work is kSteps
// consecutive steps of it, each step 32/LPH heads of LPH = hd/8 lanes with a
// 16-byte fragment per lane; a warp has a unit's loads in flight together.  The
// sums of squares of its kSteps heads are folded over their lanes by recursive
// halving, so that each lane ends with one head's sum and takes one reciprocal
// square root; a head's fold is the same adjacent-pair tree whatever step it
// falls in.  For the rotation of halves the lanes of the two
// halves trade fragments of two heads, so that each has both halves of one.
#include "dan_device.cuh"
#include "dan_internal.h"
#include "dan_attn.cuh"
#include "dan_ring.cuh"

namespace dan {

struct CacheRopeParams {
    const uint4 *q, *k, *v;
    int64_t N, q_stride8, kv_stride8, qo_stride8; // strides in 16-byte fragments
    int H, Hkv, steps_per_token;                  // units of work of a token
    const uint4 *wq, *wk;
    const float4 *rope;
    int64_t table_rows, slots_total;
    const int32_t *positions, *slots;
    float eps;
    uint4 *q_out, *k_cache, *v_cache;
    int page_shift;
    unsigned *status;
    unsigned long long limit_ns;
};

constexpr int kCacheRopeWarps = 2; // (direct form) small blocks: an SM is refilled by the warp pair
constexpr int kSteps = 8; // steps of a warp (two heads each at hd 128, four at 64)

__device__ __forceinline__ uint4 select4(bool c, const uint4 &a, const uint4 &b)
{
    return make_uint4(c ? a.x : b.x, c ? a.y : b.y, c ? a.z : b.z, c ? a.w : b.w);
}

// What a warp has in hand of a unit: kSteps fragments a lane, and the lane's
// columns of the token's cosines and sines.
template <int HD, bool NEOX>
struct RopeUnit {
    static constexpr int LPH = HD / 8, GPS = 32 / LPH, HALF = LPH / 2;
    static constexpr int NV = NEOX ? 2 : 1, NC = 4 * NV;
    uint4 x[kSteps];
    float cs[NC], sn[NC];
    int64_t t;
    int first; // the warp's first head
    int pos, slot;

    // Columns of the lane's rotation from a row of the table: pairs 4fl ..
    // 4fl+3, or columns 8 fh .. 8 fh + 7 of both halves (neox).
    __device__ __forceinline__ void take_row(const float4 *row, int fl)
    {
        row += NEOX ? 2 * (fl % HALF) : fl;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float4 c4 = row[i], s4 = row[HD / 8 + i];
            cs[4 * i] = c4.x, cs[4 * i + 1] = c4.y, cs[4 * i + 2] = c4.z, cs[4 * i + 3] = c4.w;
            sn[4 * i] = s4.x, sn[4 * i + 1] = s4.y, sn[4 * i + 2] = s4.z, sn[4 * i + 3] = s4.w;
        }
    }
};

template <int HD, bool NEOX>
__device__ __forceinline__ void rope_unit(const CacheRopeParams &p, const RopeUnit<HD, NEOX> &U)
{
    using Un = RopeUnit<HD, NEOX>;
    constexpr int LPH = Un::LPH, GPS = Un::GPS, HALF = Un::HALF;
    const int lane = threadIdx.x & 31, hs = lane / LPH, fl = lane % LPH, fh = fl % HALF;
    const int HQK = p.H + p.Hkv, HT = HQK + p.Hkv;
    const int64_t t = U.t;
    const int first = U.first, pos = U.pos, slot = U.slot;
    const uint4(&x)[kSteps] = U.x;
    const float(&cs)[Un::NC] = U.cs, (&sn)[Un::NC] = U.sn;
    if (pos < 0 || pos >= p.table_rows) {
        if (lane == 0) set_status(p.status, kStatusIndex);
        return; // the whole warp: one token
    }
    if (slot >= p.slots_total && lane == 0) set_status(p.status, kStatusIndex);
    const bool store = slot >= 0 && slot < p.slots_total;
    // the slot's first head in the caches, in fragments
    const int64_t cbase = store ? (((int64_t)(slot >> p.page_shift) * p.Hkv << p.page_shift) +
                                   (slot & ((1 << p.page_shift) - 1))) * LPH
                                : 0;
    // where fragment f of head h goes, or nullptr
    auto place = [&](int h, int f) -> uint4 * {
        if (h < p.H) return p.q_out + t * p.qo_stride8 + h * LPH + f;
        if (!store || h >= HT) return nullptr;
        const bool key = h < HQK;
        return (key ? p.k_cache : p.v_cache) + cbase + ((int64_t)(h - (key ? p.H : HQK)) << p.page_shift) * LPH + f;
    };
    if (first + GPS * kSteps > HQK) { // values: copied as they are
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int h = first + hs + GPS * i;
            if (h >= HQK) {
                uint4 *dst = place(h, fl);
                if (dst) st_stream(dst, x[i]);
            }
        }
        if (first >= HQK) return;
    }

    // Sums of squares over the lane's columns in order, two heads at a time.
    float ps[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; i += 2) {
        float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 v = make_float2(elem(x[i], e), elem(x[i + 1], e));
            acc = addmul2(acc, v, v);
        }
        ps[i] = acc.x;
        ps[i + 1] = acc.y;
    }
    // Fold over the head's lanes at xor offset 1, 2, 4 (, 8); afterwards the
    // lane holds the sum of step 4 b0 + 2 b1 + b2, bi the bits of its number.
#pragma unroll
    for (int lvl = 0, n = kSteps; lvl < 3; ++lvl, n >>= 1) {
        const bool upper = (fl >> lvl) & 1;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float send = upper ? ps[i] : ps[i + n / 2];
            const float keep = upper ? ps[i + n / 2] : ps[i];
            ps[i] = __fadd_rn(keep, __shfl_xor_sync(kFull, send, 1 << lvl));
        }
    }
    if (LPH == 16) ps[0] = __fadd_rn(ps[0], __shfl_xor_sync(kFull, ps[0], 8));
    const float mine = defined_rsqrt(__fadd_rn(div_by<HD>(ps[0]), p.eps));
    auto rstd = [&](int i) {
        return __shfl_sync(kFull, mine, hs * LPH + (((i >> 2) & 1) | (i & 2) | ((i & 1) << 2)));
    };

    if constexpr (NEOX) {
        const uint4 wq[2] = {ld_vec(p.wq + fh), ld_vec(p.wq + fh + HALF)};
        const uint4 wk[2] = {ld_vec(p.wk + fh), ld_vec(p.wk + fh + HALF)};
        const bool upper = fl >= HALF;
#pragma unroll
        for (int i = 0; i < kSteps; i += 2) {
            if (first + GPS * i >= HQK) break; // warp-uniform: values from here on
            const float r0 = rstd(i), r1 = rstd(i + 1), r = upper ? r1 : r0;
            // the lower lanes take both halves of step i's head, the upper of step i+1's
            const uint4 give = select4(upper, x[i], x[i + 1]);
            uint4 got;
            got.x = __shfl_xor_sync(kFull, give.x, HALF);
            got.y = __shfl_xor_sync(kFull, give.y, HALF);
            got.z = __shfl_xor_sync(kFull, give.z, HALF);
            got.w = __shfl_xor_sync(kFull, give.w, HALF);
            const uint4 a = select4(upper, got, x[i]), b = select4(upper, x[i + 1], got);
            const int h = first + hs + GPS * (upper ? i + 1 : i);
            const uint4 wa = select4(h < p.H, wq[0], wk[0]), wb = select4(h < p.H, wq[1], wk[1]);
            const float2 r2 = dup2(r);
            uint4 oa, ob;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                float ra[2], rb[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int e = 2 * m + k;
                    // (first half, second half) of column e
                    const float2 n = mul2(mul2(make_float2(elem(a, e), elem(b, e)), r2),
                                          make_float2(elem(wa, e), elem(wb, e)));
                    const float2 pc = mul2(n, dup2(cs[e])), pn = mul2(n, dup2(sn[e]));
                    ra[k] = __fsub_rn(pc.x, pn.y);
                    rb[k] = __fadd_rn(pn.x, pc.y);
                }
                set_word(oa, m, pack_bf16(ra[0], ra[1]));
                set_word(ob, m, pack_bf16(rb[0], rb[1]));
            }
            if (h < HQK) {
                uint4 *dst = place(h, fh);
                if (dst) {
                    st_stream(dst, oa);
                    st_stream(dst + HALF, ob);
                }
            }
        }
    } else {
        const uint4 wq = ld_vec(p.wq + fl), wk = ld_vec(p.wk + fl);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int h = first + hs + GPS * i;
            if (first + GPS * i >= HQK) break; // warp-uniform: values from here on
            const uint4 w = select4(h < p.H, wq, wk);
            const float2 r2 = dup2(rstd(i));
            uint4 out;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float2 n = mul2(mul2(wide2(word(x[i], m)), r2), wide2(word(w, m)));
                const float2 pc = mul2(n, dup2(cs[m])), pn = mul2(n, dup2(sn[m]));
                set_word(out, m, pack_bf16(__fsub_rn(pc.x, pn.y), __fadd_rn(pn.x, pc.y)));
            }
            if (h < HQK) {
                uint4 *dst = place(h, fl);
                if (dst) st_stream(dst, out);
            }
        }
    }
}

// A warp per unit, straight from global memory: the shortest way for a few
// tokens.
template <int HD, bool NEOX>
__global__ void __launch_bounds__(32 * kCacheRopeWarps, 8) qk_norm_rope_cache_kernel(const CacheRopeParams p)
{
    using Un = RopeUnit<HD, NEOX>;
    const int lane = threadIdx.x & 31, hs = lane / Un::LPH, fl = lane % Un::LPH;
    const int64_t unit = (int64_t)blockIdx.x * kCacheRopeWarps + (threadIdx.x >> 5);
    Un U;
    U.t = unit / p.steps_per_token;
    U.first = (int)(unit - U.t * p.steps_per_token) * (Un::GPS * kSteps);
    grid_dependency_wait();
    allow_dependents();
    if (U.t >= p.N) return;
    const int HQK = p.H + p.Hkv, HT = HQK + p.Hkv;
    const uint4 *qrow = p.q + U.t * p.q_stride8;
    const uint4 *krow = p.k + U.t * p.kv_stride8;
    const uint4 *vrow = p.v + U.t * p.kv_stride8;
    U.pos = __ldg(p.positions + U.t);
    U.slot = __ldg(p.slots + U.t);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int h = U.first + hs + Un::GPS * i;
        const uint4 *src = h < p.H ? qrow + h * Un::LPH
                           : h < HQK ? krow + (h - p.H) * Un::LPH
                                     : vrow + (h - HQK) * Un::LPH;
        U.x[i] = h < HT ? ld_stream(src + fl) : make_uint4(0, 0, 0, 0);
    }
    const bool known = U.pos >= 0 && U.pos < p.table_rows;
    if (U.first < HQK) U.take_row(p.rope + (int64_t)(known ? U.pos : 0) * (HD / 4), fl);
    rope_unit<HD, NEOX>(p, U);
}

// Persistent CTAs, each warp with a ring of slots that bulk copies fill while
// it works (dan_ring.cuh): for many tokens, where it keeps more of the loads
// in flight.  Measured, ring against direct form: 65536 tokens of 48 heads of
// 128 (81 units a warp) 259 us against 315 to 365, 4216 tokens of 96 heads (10
// units) 38.4 against 42.9; with two units a warp they are equal, and below
// that the ring only adds the copy's latency.  12 warps with two slots took
// 287 us, 6 with four 308.
constexpr int kRingWarps = 8, kRingSlots = 3, kRingFrom = 2;

template <int HD>
struct RopeRing {
    static constexpr int DATA = 32 * kSteps;        // fragments of a unit's heads (4 KB)
    static constexpr int SLOT = DATA + HD / 4 + 1;  // with the table row, and position and slot
    static constexpr int SMEM = kRingWarps * kRingSlots * (SLOT * 16 + 8);
};

template <int HD, bool NEOX>
__global__ void __launch_bounds__(32 * kRingWarps, 2) qk_norm_rope_cache_ring_kernel(const CacheRopeParams p)
{
    using Un = RopeUnit<HD, NEOX>;
    using Ring = RopeRing<HD>;
    using Pipe = WarpPipe<kRingSlots>;
    extern __shared__ __align__(128) uint4 rope_smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(rope_smem + kRingWarps * kRingSlots * Ring::SLOT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, fl = lane % Un::LPH;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRingWarps * kRingSlots; ++i) mbar_init(full + i, 1);
        mbar_init_fence();
    }
    __syncthreads();
    grid_dependency_wait();
    allow_dependents();
    const int HQK = p.H + p.Hkv, HT = HQK + p.Hkv;
    const int64_t total = p.N * p.steps_per_token;
    const int64_t w0 = (int64_t)blockIdx.x * kRingWarps + warp, W = (int64_t)gridDim.x * kRingWarps;
    const int units = w0 < total ? (int)((total - w0 + W - 1) / W) : 0;
    uint4 *slots = rope_smem + warp * kRingSlots * Ring::SLOT;
    uint64_t *bar = full + warp * kRingSlots;
    auto locate = [&](int i, int64_t &t, int &first) {
        const int64_t u = w0 + W * i;
        t = u / p.steps_per_token;
        first = (int)(u - t * p.steps_per_token) * (Un::GPS * kSteps);
    };
    // Lane l holds position and slot of the warp's unit 32 r + l for the round
    // r of the next request.
    int my_pos = 0, my_slot = 0;
    auto look_up = [&](int i) {
        if (i >= units) return;
        int64_t t;
        int first;
        locate(i, t, first);
        my_pos = __ldg(p.positions + t);
        my_slot = __ldg(p.slots + t);
    };
    auto request = [&](int i) { // the whole warp
        if (i >= units) return;
        const int pos = __shfl_sync(kFull, my_pos, i & 31), slot = __shfl_sync(kFull, my_slot, i & 31);
        if (lane == 0) {
            int64_t t;
            int first;
            locate(i, t, first);
            const int last = min(HT, first + Un::GPS * kSteps);
            uint4 *dst = slots + Pipe::slot(i) * Ring::SLOT;
            uint64_t *b = bar + Pipe::slot(i);
            *reinterpret_cast<int2 *>(dst + Ring::SLOT - 1) = make_int2(pos, slot);
            const bool turn = first < HQK;
            mbar_arrive_expect_tx(b, (unsigned)((last - first) * HD * 2 + (turn ? HD * 4 : 0)));
            auto piece = [&](const uint4 *row, int from, int to, int base) { // heads from .. to-1 of the list
                from = max(from, first);
                to = min(to, last);
                if (from < to)
                    bulk_load(dst + (from - first) * Un::LPH, row + (int64_t)(from - base) * Un::LPH,
                              (unsigned)((to - from) * HD * 2), b);
            };
            piece(p.q + t * p.q_stride8, 0, p.H, 0);
            piece(p.k + t * p.kv_stride8, p.H, HQK, p.H);
            piece(p.v + t * p.kv_stride8, HQK, HT, HQK);
            if (turn) {
                const bool known = pos >= 0 && pos < p.table_rows;
                bulk_load(dst + Ring::DATA, p.rope + (int64_t)(known ? pos : 0) * (HD / 4), HD * 4, b);
            }
        }
    };
    look_up(lane);
    for (int i = 0; i < kRingSlots; ++i) request(i);
    for (int i = 0; i < units; ++i) {
        if (!__all_sync(kFull, Pipe::wait(bar, i, p.limit_ns))) {
            Pipe::abort(bar, i, units, p.status, p.limit_ns);
            return;
        }
        Un U;
        locate(i, U.t, U.first);
        const uint4 *src = slots + Pipe::slot(i) * Ring::SLOT;
        const int n = (HT - U.first) * Un::LPH; // fragments there are
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            U.x[s] = 32 * s + lane < n ? src[32 * s + lane] : make_uint4(0, 0, 0, 0);
        if (U.first < HQK) U.take_row(reinterpret_cast<const float4 *>(src + Ring::DATA), fl);
        const int2 at = *reinterpret_cast<const int2 *>(src + Ring::SLOT - 1);
        U.pos = at.x;
        U.slot = at.y;
        slot_reads_done();
        const int next = i + kRingSlots;
        if ((next & 31) == 0) look_up(next + lane);
        request(next);
        rope_unit<HD, NEOX>(p, U);
    }
}

namespace {

template <int HD, bool NEOX>
cudaError_t launch_shape(CacheRopeParams p, cudaStream_t s)
{
    constexpr int heads = 32 / (HD / 8) * kSteps;
    p.steps_per_token = (p.H + 2 * p.Hkv + heads - 1) / heads;
    const int64_t units = p.N * p.steps_per_token;
    // more units than kRingFrom for each warp that the ring has
    if (units >= (int64_t)kRingFrom * 2 * kRingWarps * sm_count()) {
        if (units / (2 * kRingWarps * sm_count()) > 0x7FFFFFF0) return cudaErrorInvalidConfiguration;
        auto fn = qk_norm_rope_cache_ring_kernel<HD, NEOX>;
        const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(fn), RopeRing<HD>::SMEM);
        if (e != cudaSuccess) return e;
        return launch_overlapped(fn, 2 * sm_count(), 32 * kRingWarps, RopeRing<HD>::SMEM, s, p);
    }
    const int64_t blocks = (units + kCacheRopeWarps - 1) / kCacheRopeWarps;
    return launch_overlapped(qk_norm_rope_cache_kernel<HD, NEOX>, (int)blocks, 32 * kCacheRopeWarps, 0, s,
                             p);
}

} // namespace

cudaError_t launch_qk_norm_rope_cache(const CacheRopeProblem &c, cudaStream_t s)
{
    CacheRopeParams p = {};
    p.q = static_cast<const uint4 *>(c.q);
    p.k = static_cast<const uint4 *>(c.k);
    p.v = static_cast<const uint4 *>(c.v);
    p.N = c.N;
    p.q_stride8 = c.q_stride / 8;
    p.kv_stride8 = c.kv_stride / 8;
    p.qo_stride8 = c.qo_stride / 8;
    p.H = (int)c.heads;
    p.Hkv = (int)c.kv_heads;
    p.wq = static_cast<const uint4 *>(c.wq);
    p.wk = static_cast<const uint4 *>(c.wk);
    p.rope = reinterpret_cast<const float4 *>(c.rope);
    p.table_rows = c.table_rows;
    p.slots_total = c.num_pages << page_shift(c.page_size);
    p.positions = c.positions;
    p.slots = c.slots;
    p.eps = c.eps;
    p.q_out = static_cast<uint4 *>(c.q_out);
    p.k_cache = static_cast<uint4 *>(c.k_cache);
    p.v_cache = static_cast<uint4 *>(c.v_cache);
    p.page_shift = page_shift(c.page_size);
    p.status = device_status();
    p.limit_ns = 1000000000ull;
    if (c.head_dim == 64) return c.neox ? launch_shape<64, true>(p, s) : launch_shape<64, false>(p, s);
    return c.neox ? launch_shape<128, true>(p, s) : launch_shape<128, false>(p, s);
}

} // namespace dan
