// dan_cache_rope.cu -- QK-RMSNorm + RoPE at given positions, with K and V
// stored into a paged cache.
//
// Mathematics, per token and head of Q and K: rstd = 1/sqrt(mean x^2 + eps),
// n = x * rstd * w, then pairs (a, b) of n turned by the angle of their
// column at the token's position; V is copied.  About 8 flops per 4 bytes
// moved: the bound is memory (and, for a few tokens, latency).
//
// A token's heads are one list, Q then K then V.  A warp takes STEPS
// consecutive steps of it, each step 32/LPH heads of LPH = hd/8 lanes with a
// 16-byte fragment per lane, and has all its loads in flight before the
// first use.  A head's sum of squares is folded over its own LPH lanes, so
// its bits do not depend on which warp or step it falls in.
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

constexpr int kCacheRopeWarps = 8;

template <int HD, bool NEOX, int STEPS>
__global__ void __launch_bounds__(32 * kCacheRopeWarps) qk_norm_rope_cache_kernel(const CacheRopeParams p)
{
    constexpr int LPH = HD / 8, GPS = 32 / LPH;
    const int lane = threadIdx.x & 31, hs = lane / LPH, fl = lane % LPH;
    const int64_t unit = (int64_t)blockIdx.x * kCacheRopeWarps + (threadIdx.x >> 5);
    const int64_t t = unit / p.steps_per_token;
    const int h0 = (int)(unit - t * p.steps_per_token) * (GPS * STEPS) + hs;
    grid_dependency_wait();
    allow_dependents();
    if (t >= p.N) return;

    const int HQK = p.H + p.Hkv, HT = HQK + p.Hkv;
    const uint4 *qrow = p.q + t * p.q_stride8 + fl;
    const uint4 *krow = p.k + t * p.kv_stride8 + fl;
    const uint4 *vrow = p.v + t * p.kv_stride8 + fl;
    const int pos = __ldg(p.positions + t), slot = __ldg(p.slots + t);
    uint4 x[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int h = h0 + GPS * i;
        const uint4 *src = h < p.H ? qrow + h * LPH
                           : h < HQK ? krow + (h - p.H) * LPH
                                     : vrow + (h - HQK) * LPH;
        x[i] = h < HT ? ld_stream(src) : make_uint4(0, 0, 0, 0);
    }
    const uint4 wq = ld_vec(p.wq + fl), wk = ld_vec(p.wk + fl);
    if (pos < 0 || pos >= p.table_rows) {
        if (lane == 0) set_status(p.status, kStatusIndex);
        return; // the whole warp: one token
    }
    if (slot >= p.slots_total && lane == 0) set_status(p.status, kStatusIndex);
    const bool store = slot >= 0 && slot < p.slots_total;
    // the lane's columns: pairs 4fl .. 4fl+3, or columns of one half (neox)
    const float4 *row = p.rope + (int64_t)pos * (HD / 4);
    float cs[8], sn[8];
    {
        constexpr int NV = NEOX ? 2 : 1;
        const int b = NEOX ? 2 * (fl % (LPH / 2)) : fl;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float4 c4 = ld_vec(row + b + i), s4 = ld_vec(row + HD / 8 + b + i);
            cs[4 * i] = c4.x, cs[4 * i + 1] = c4.y, cs[4 * i + 2] = c4.z, cs[4 * i + 3] = c4.w;
            sn[4 * i] = s4.x, sn[4 * i + 1] = s4.y, sn[4 * i + 2] = s4.z, sn[4 * i + 3] = s4.w;
        }
        if (NEOX && fl < LPH / 2) // first half: own*c - other*s
#pragma unroll
            for (int e = 0; e < 8; ++e) sn[e] = -sn[e];
    }
    // fragment offset of the slot's first head in the caches
    const int64_t cbase =
        store ? (((int64_t)(slot >> p.page_shift) * p.Hkv << p.page_shift) +
                 (slot & ((1 << p.page_shift) - 1))) * LPH + fl
              : 0;

#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int h = h0 + GPS * i;
        if (h - hs >= HT) break; // warp-uniform: no head left in any lane
        const uint4 f = x[i];
        float acc = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float v = elem(f, e);
            acc = __fadd_rn(acc, __fmul_rn(v, v));
        }
#pragma unroll
        for (int off = 1; off < LPH; off <<= 1)
            acc = __fadd_rn(acc, __shfl_xor_sync(kFull, acc, off));
        const float r = defined_rsqrt(__fadd_rn(div_by<HD>(acc), p.eps));
        const uint4 w = h < p.H ? wq : wk;
        float n[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] = __fmul_rn(__fmul_rn(elem(f, e), r), elem(w, e));
        uint4 out;
        if (NEOX) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float o0 = __shfl_xor_sync(kFull, n[2 * m], LPH / 2);
                const float o1 = __shfl_xor_sync(kFull, n[2 * m + 1], LPH / 2);
                // the second half's sum rn(a s) + rn(b c) has its terms the other
                // way round here, and the sum of two values is the same either way
                set_word(out, m,
                         pack_bf16(__fadd_rn(__fmul_rn(n[2 * m], cs[2 * m]), __fmul_rn(o0, sn[2 * m])),
                                   __fadd_rn(__fmul_rn(n[2 * m + 1], cs[2 * m + 1]),
                                             __fmul_rn(o1, sn[2 * m + 1]))));
            }
        } else {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float a = n[2 * m], b = n[2 * m + 1];
                set_word(out, m,
                         pack_bf16(__fsub_rn(__fmul_rn(a, cs[m]), __fmul_rn(b, sn[m])),
                                   __fadd_rn(__fmul_rn(a, sn[m]), __fmul_rn(b, cs[m]))));
            }
        }
        if (h < p.H) {
            st_stream(p.q_out + t * p.qo_stride8 + h * LPH + fl, out);
        } else if (h < HT && store) {
            const bool key = h < HQK;
            const int64_t u = key ? h - p.H : h - HQK;
            st_stream((key ? p.k_cache : p.v_cache) + cbase + (u << p.page_shift) * LPH,
                      key ? out : f);
        }
    }
}

namespace {

template <int HD, bool NEOX, int STEPS>
cudaError_t launch_steps(CacheRopeParams p, cudaStream_t s)
{
    constexpr int heads = 32 / (HD / 8) * STEPS;
    p.steps_per_token = (p.H + 2 * p.Hkv + heads - 1) / heads;
    const int64_t blocks = (p.N * p.steps_per_token + kCacheRopeWarps - 1) / kCacheRopeWarps;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return launch_overlapped(qk_norm_rope_cache_kernel<HD, NEOX, STEPS>, (int)blocks,
                             32 * kCacheRopeWarps, 0, s, p);
}

template <int HD>
cudaError_t launch_hd(const CacheRopeParams &p, bool neox, cudaStream_t s)
{
    return neox ? launch_steps<HD, true, 4>(p, s) : launch_steps<HD, false, 4>(p, s);
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
    return c.head_dim == 64 ? launch_hd<64>(p, c.neox, s) : launch_hd<128>(p, c.neox, s);
}

} // namespace dan
