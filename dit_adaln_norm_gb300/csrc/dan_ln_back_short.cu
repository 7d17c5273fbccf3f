// dan_ln_back_short.cu -- gradients of LayerNorm + modulate for many short batches
// (include/dan_train.h): scale and shift of a token each, or of a few.
//
// In dan_ln_back.cu a batch's column sums cross a CTA's teams, the memory and a
// second kernel, and the rows in flight end with the batch.  Here a team (or,
// of narrow rows, a row's lanes) has whole batches to itself: its column sums are
// the batch's, stored as they are, without a workspace.
#include "dan_ln_back.cuh"

namespace dan {
namespace {

constexpr int kShortThreads = 256;
// CTAs that share an SM, by the registers of K fragments a thread.
__host__ __device__ constexpr int short_blocks(int K) { return K == 1 ? 3 : K == 2 ? 2 : 1; }

// R: the rows at a time of ln_back_kernel at this width, whose order of sums is kept.
template <int K, int R, bool CKPT, bool RES, bool MULTI>
__global__ void __launch_bounds__(kShortThreads, short_blocks(K))
    ln_back_short_kernel(const LnBackParams p, int64_t B, uint4 *dscale, uint4 *dshift, int64_t gs8)
{
    using XWord = typename std::conditional<CKPT, uint2, uint4>::type;
    constexpr int kWarps = kShortThreads / 32, LV = 16 / R; // lanes that add a value's warps together
    __shared__ float2 s_red[2][kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int W = p.W, L = MULTI ? p.L : 32, F = p.F;
    const int team = warp / W;
    const int sub = MULTI ? lane / L : 0, per = MULTI ? 32 / L : 1; // batches side by side in a warp
    const int width = MULTI ? L : 32 * W;
    const int col = MULTI ? lane - sub * L : (warp - team * W) * 32 + lane;
    const int64_t units = (int64_t)gridDim.x * p.teams * per;
    const bool in_team = team < p.teams, has_last = col + width * (K - 1) < F;
    auto has = [&](int k) { return k < K - 1 || has_last; };
    grid_dependency_wait();
    allow_dependents();
    if (!in_team) return; // (a whole warp)
    int parity = 0;
    // (a warp's batches go on together: the first one tells whether there are any)
    for (int64_t b0 = ((int64_t)blockIdx.x * p.teams + team) * per; b0 < B; b0 += units) {
        const int64_t b = b0 + sub;
        const bool live = b < B;
        float2 sum_n[K][4], sum_1[K][4], o[K][4]; // o: 1 + scale
#pragma unroll
        for (int k = 0; k < K; ++k) {
            uint4 sc = make_uint4(0, 0, 0, 0);
            if (live && has(k) && p.T > 0) sc = ld_stream(p.scale + b * p.vs8 + col + width * k);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                o[k][w] = add2(dup2(1.0f), wide2(word(sc, w)));
                sum_n[k][w] = sum_1[k][w] = make_float2(0.0f, 0.0f);
            }
        }
        for (int64_t row = b * p.T, end = row + p.T; row < end; ++row) { // (as often for each of a warp's batches)
            uint4 dy[K], res[K];
            XWord xv[K];
            unsigned code[K];
            float2 st = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                dy[k] = res[k] = make_uint4(0, 0, 0, 0);
                xv[k] = XWord();
                code[k] = 127;
                if (live && has(k)) {
                    const int64_t at = row * F + col + width * k;
                    dy[k] = ld_stream(p.dy + at);
                    if (RES) res[k] = ld_stream(p.dres + at);
                    if constexpr (CKPT) {
                        xv[k] = __ldg(p.codes + at);
                        code[k] = __ldg(p.block_scales + row * p.blocks + ((col + width * k) >> 2));
                    } else {
                        xv[k] = ld_stream(p.x + at);
                    }
                }
            }
            if (live) st = __ldg(p.stats + row);
            float2 n[K][4], g[K][4], s1 = make_float2(0.0f, 0.0f), s2 = s1;
            const float2 neg_mean = dup2(-st.x), rstd = dup2(st.y);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float2 v[4];
                if constexpr (CKPT) {
                    const float2 s = dup2(block_scale_value(code[k]));
                    v[0] = fma2(e4m3_pair(xv[k].x & 0xFFFFu), s, neg_mean);
                    v[1] = fma2(e4m3_pair(xv[k].x >> 16), s, neg_mean);
                    v[2] = fma2(e4m3_pair(xv[k].y & 0xFFFFu), s, neg_mean);
                    v[3] = fma2(e4m3_pair(xv[k].y >> 16), s, neg_mean);
                } else {
#pragma unroll
                    for (int w = 0; w < 4; ++w) v[w] = add2(wide2(word(xv[k], w)), neg_mean);
                }
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float2 d = wide2(word(dy[k], w));
                    n[k][w] = mul2(v[w], rstd);
                    if (!(live && has(k))) n[k][w] = make_float2(0.0f, 0.0f); // whatever the statistics
                    g[k][w] = mul2(d, o[k][w]);
                    sum_1[k][w] = add2(sum_1[k][w], d);
                    sum_n[k][w] = fma2(d, n[k][w], sum_n[k][w]);
                    s1 = add2(s1, g[k][w]);
                    s2 = fma2(g[k][w], n[k][w], s2);
                }
            }
            float2 sum = make_float2(__fadd_rn(s1.x, s1.y), __fadd_rn(s2.x, s2.y));
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1)
                if (!MULTI || off < L) {
                    sum.x = __fadd_rn(sum.x, __shfl_xor_sync(kFull, sum.x, off));
                    sum.y = __fadd_rn(sum.y, __shfl_xor_sync(kFull, sum.y, off));
                }
            if (!MULTI && W > 1) {
                float2 *red = s_red[parity];
                parity ^= 1; // (the other warps may still read the last row's)
                if (lane == 0) red[warp] = sum;
                team_barrier(team, 32 * W);
                sum = make_float2(0.0f, 0.0f);
                for (int j = lane % LV; j < W; j += LV) sum = add2(sum, red[team * W + j]);
#pragma unroll
                for (int off = 1; off < LV; off *= 2) {
                    sum.x = __fadd_rn(sum.x, __shfl_xor_sync(kFull, sum.x, off));
                    sum.y = __fadd_rn(sum.y, __shfl_xor_sync(kFull, sum.y, off));
                }
            }
            // dx = g * rstd - mean(g) * rstd - n * (mean(g * n) * rstd)
            const float2 m1 = dup2(-__fmul_rn(__fmul_rn(sum.x, p.inv_d), st.y));
            const float2 m2 = dup2(-__fmul_rn(__fmul_rn(sum.y, p.inv_d), st.y));
#pragma unroll
            for (int k = 0; k < K; ++k) {
                uint4 out;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    float2 v = fma2(n[k][w], m2, fma2(g[k][w], rstd, m1));
                    if (RES) v = add2(v, wide2(word(res[k], w)));
                    set_word(out, w, pack_bf16(v.x, v.y));
                }
                if (live && has(k)) st_stream(p.dx + row * F + col + width * k, out);
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            uint4 u, v;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                set_word(u, w, pack_bf16(sum_n[k][w].x, sum_n[k][w].y));
                set_word(v, w, pack_bf16(sum_1[k][w].x, sum_1[k][w].y));
            }
            if (!(live && has(k))) continue;
            st_stream(dscale + b * gs8 + col + width * k, u);
            st_stream(dshift + b * gs8 + col + width * k, v);
        }
    }
}

template <int K, int R, bool CKPT, bool RES, bool MULTI>
cudaError_t launch_short(LnBackParams p, const LnBackProblem &q, cudaStream_t s)
{
    p.teams = kShortThreads / 32 / p.W;
    const int64_t of_cta = p.teams * (int64_t)(MULTI ? 32 / p.L : 1), ctas = (q.B + of_cta - 1) / of_cta;
    const int64_t most = (int64_t)short_blocks(K) * sm_count();
    const auto fn = ln_back_short_kernel<K, R, CKPT, RES, MULTI>;
    const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(fn), 0);
    if (e != cudaSuccess) return e;
    return launch_overlapped(fn, (int)(ctas < most ? ctas : most), kShortThreads, 0, s, p, q.B,
                             static_cast<uint4 *>(q.dscale), static_cast<uint4 *>(q.dshift), q.gs / 8);
}

} // namespace

// By what the two took, in us: here a row of each team's in turn, 1.0 to 1.9 by the
// fragments of a thread (rows of one warp, or of a team); there a batch's end 2.2 and
// 1 / 800 a column, and the rows.  Replayed, from checkpoints, there and here:
//   65536 x 1 x 64      970  12.6     1953 x 8 x 1024    48.6 24.6     3906 x 1 x 4096   171 41.6
//   4096 x 16 x 8      68.9  14.2     488 x 16 x 256     12.3 12.9     488 x 4 x 8192   48.2 37.9
//   2048 x 32 x 64     35.6  28.0     488 x 32 x 1024    27.5 39.6     304 x 64 x 8192   175  246
bool ln_back_is_short(int64_t B, int64_t T, int64_t D)
{
    if (T == 0) return true; // zeros
    const int64_t sms = sm_count();
    if (B < 2 * sms || T > 64) return false;
    const LnBackCut c = ln_back_cut((int)(D / 8));
    const int64_t units = sms * short_blocks(c.K) * (kShortThreads / 32 / c.W) * (32 / c.L);
    const double row = c.K <= 2 ? 1.0 : c.W == 1 ? 1.2 : c.K == 3 ? 1.5 : 1.9;
    const double here = row * (double)((B + units - 1) / units * T);
    const double there = (double)B / (double)sms * (2.2 + (double)D / 800 + (double)(T * D) / 9000);
    return here < there;
}

cudaError_t launch_ln_back_short(const LnBackProblem &q, cudaStream_t s)
{
    const LnBackParams p = ln_back_params(q);
    const bool ckpt = !p.x, res = p.dres != nullptr;
    return with_cut(ln_back_cut(p.F), [&](auto k, auto rows, auto multi) {
        constexpr int K = decltype(k)::value, R = decltype(rows)::value;
        constexpr bool M = decltype(multi)::value;
        if (ckpt) return res ? launch_short<K, R, true, true, M>(p, q, s) : launch_short<K, R, true, false, M>(p, q, s);
        return res ? launch_short<K, R, false, true, M>(p, q, s) : launch_short<K, R, false, false, M>(p, q, s);
    });
}

} // namespace dan
