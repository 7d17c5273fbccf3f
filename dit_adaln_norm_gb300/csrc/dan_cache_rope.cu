// dan_cache_rope.cu -- QK-RMSNorm + RoPE at given positions, with K and V
// stored into a paged cache.
//
// Mathematics, per token and head of Q and K: rstd = 1/sqrt(mean x^2 + eps),
// n = x * rstd * w, then pairs (a, b) of n turned by the angle of their
// column at the token's position; V is copied.  About 8 flops per 4 bytes
// moved: the bound is memory (and, for a few tokens, latency).
//
// A token's heads are one list, Q then K then V.  A warp takes kSteps
// consecutive steps of it, each step 32/LPH heads of LPH = hd/8 lanes with a
// 16-byte fragment per lane, and has all its loads in flight before the first
// use.  The sums of squares of its kSteps heads are folded over their lanes
// by recursive halving, so that each lane ends with one head's sum and takes
// one reciprocal square root; a head's fold is the same adjacent-pair tree
// whatever step it falls in.  For the rotation of halves the lanes of the two
// halves trade fragments of two heads, so that each has both halves of one.
#include "dan_device.cuh"
#include "dan_internal.h"
#include "dan_attn.cuh"
#include "dan_ring.cuh"

namespace dan {

struct CacheRopeParams {
    const uint4 *q, *k, *v;
    int64_t N, q_stride8, kv_stride8, qo_stride8; // strides in 16-byte fragments
    int H, Hkv, steps_per_token;                  // warps per token
    const uint4 *wq, *wk;
    const float4 *rope;
    int64_t table_rows, slots_total;
    const int32_t *positions, *slots;
    float eps;
    uint4 *q_out, *k_cache, *v_cache;
    int page_shift;
    unsigned *status;
};

constexpr int kCacheRopeWarps = 2; // small blocks: an SM is refilled by the warp pair
constexpr int kSteps = 8; // steps of a warp (two heads each at hd 128, four at 64)

__device__ __forceinline__ uint4 select4(bool c, const uint4 &a, const uint4 &b)
{
    return make_uint4(c ? a.x : b.x, c ? a.y : b.y, c ? a.z : b.z, c ? a.w : b.w);
}

template <int HD, bool NEOX>
__global__ void __launch_bounds__(32 * kCacheRopeWarps, 12) qk_norm_rope_cache_kernel(const CacheRopeParams p)
{
    constexpr int LPH = HD / 8, GPS = 32 / LPH, HALF = LPH / 2;
    const int lane = threadIdx.x & 31, hs = lane / LPH, fl = lane % LPH;
    const int64_t unit = (int64_t)blockIdx.x * kCacheRopeWarps + (threadIdx.x >> 5);
    const int64_t t = unit / p.steps_per_token;
    const int first = (int)(unit - t * p.steps_per_token) * (GPS * kSteps); // the warp's first head
    grid_dependency_wait();
    allow_dependents();
    if (t >= p.N) return;

    const int HQK = p.H + p.Hkv, HT = HQK + p.Hkv;
    const uint4 *qrow = p.q + t * p.q_stride8;
    const uint4 *krow = p.k + t * p.kv_stride8;
    const uint4 *vrow = p.v + t * p.kv_stride8;
    const int pos = __ldg(p.positions + t), slot = __ldg(p.slots + t);
    uint4 x[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int h = first + hs + GPS * i;
        const uint4 *src = h < p.H ? qrow + h * LPH : h < HQK ? krow + (h - p.H) * LPH : vrow + (h - HQK) * LPH;
        x[i] = h < HT ? ld_stream(src + fl) : make_uint4(0, 0, 0, 0);
    }
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

    // Columns of the lane's rotation: pairs 4fl .. 4fl+3, or columns 8 fh ..
    // 8 fh + 7 of both halves (neox).
    const int fh = fl % HALF;
    constexpr int NV = NEOX ? 2 : 1, NC = 4 * NV;
    const float4 *row = p.rope + (int64_t)pos * (HD / 4) + (NEOX ? 2 * fh : fl);
    float cs[NC], sn[NC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const float4 c4 = ld_vec(row + i), s4 = ld_vec(row + HD / 8 + i);
        cs[4 * i] = c4.x, cs[4 * i + 1] = c4.y, cs[4 * i + 2] = c4.z, cs[4 * i + 3] = c4.w;
        sn[4 * i] = s4.x, sn[4 * i + 1] = s4.y, sn[4 * i + 2] = s4.z, sn[4 * i + 3] = s4.w;
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

namespace {

template <int HD, bool NEOX>
cudaError_t launch_shape(CacheRopeParams p, cudaStream_t s)
{
    constexpr int heads = 32 / (HD / 8) * kSteps;
    p.steps_per_token = (p.H + 2 * p.Hkv + heads - 1) / heads;
    const int64_t blocks = (p.N * p.steps_per_token + kCacheRopeWarps - 1) / kCacheRopeWarps;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
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
    if (c.head_dim == 64) return c.neox ? launch_shape<64, true>(p, s) : launch_shape<64, false>(p, s);
    return c.neox ? launch_shape<128, true>(p, s) : launch_shape<128, false>(p, s);
}

} // namespace dan
