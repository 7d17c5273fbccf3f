// dan_ln_back.cu -- gradients of LayerNorm + modulate for sm_103a
// (include/dan_train.h).
//
// With n = (x - mean) * rstd and g = dy * (1 + scale), a row's
//   dx = rstd * (g - mean(g) - n * mean(g * n)) [+ dres]
// needs two sums over the row, and dscale, dshift are sums of dy * n and dy
// over a batch's rows: one pass over the data, bound by HBM.
//
// A CTA per SM takes a contiguous block of rows.  Its 16 warps form teams of W
// warps (narrow rows: several rows share a warp); every thread has the same
// columns of each of its team's rows, so the column sums stay in its registers
// until the batch ends.  Each thread copies its own columns of the next rows
// into shared memory with cp.async, kAhead rows ahead, and nobody else reads
// them: the only exchange per row is that of the two sums.  At the end of a
// batch, or of the CTA's rows, the teams' column sums are added in order and
// stored as one partial of the batch; a second kernel adds the partials in
// order.
#include "dan_train.cuh"

namespace dan {
namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kAhead = 4; // rows (of each team) in flight

struct LnBackParams {
    const uint4 *dy, *x;
    const uint2 *codes;
    const uint8_t *block_scales;
    const float2 *stats;
    const uint4 *scale;
    const uint4 *dres;
    uint4 *dx;
    float *part; // [grid + B][2][D] partial column sums; CTA c's of batch b is number c + b
    int64_t rows, T, vs8;
    int F;      // fragments (of eight columns) per row
    int blocks; // checkpoint blocks per row
    int W;      // warps per team
    int L;      // lanes per row (32 with W > 1)
    int teams;
    float inv_d;
};

// First row of CTA c of G.
__host__ __device__ inline int64_t first_row(int64_t c, int64_t rows, int64_t G) { return c * rows / G; }

__device__ __forceinline__ void team_barrier(int team, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(threads) : "memory");
}

// K fragments per thread.
template <int K, bool CKPT, bool RES>
__global__ void __launch_bounds__(kThreads, 1) ln_back_kernel(const LnBackParams p)
{
    using XWord = typename std::conditional<CKPT, uint2, uint4>::type;
    extern __shared__ __align__(16) uint4 smem[];
    uint4 *s_dy = smem;                                                     // [kAhead][K][kThreads]
    uint4 *s_res = s_dy + kAhead * K * kThreads;                            // likewise (RES)
    XWord *s_x = reinterpret_cast<XWord *>(s_res + (RES ? kAhead * K * kThreads : 0));
    float2 *s_red = reinterpret_cast<float2 *>(s_x + kAhead * K * kThreads); // [2][kWarps]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int W = p.W, L = p.L, F = p.F;
    const int team = warp / W;
    const bool in_team = team < p.teams;
    const int sub = lane / L, per_warp = 32 / L; // this lane's row of its warp's
    const int width = W == 1 ? L : 32 * W;       // threads of a row
    const int col = W == 1 ? lane - sub * L : (warp - team * W) * 32 + lane;
    const int step = p.teams * per_warp; // rows of a CTA's step
    const int64_t c = blockIdx.x, G = gridDim.x;
    const int64_t r_end = first_row(c + 1, p.rows, G);
    bool has[K];
#pragma unroll
    for (int k = 0; k < K; ++k) has[k] = in_team && col + width * k < F;

    grid_dependency_wait();
    allow_dependents();

    for (int64_t r0 = first_row(c, p.rows, G); r0 < r_end;) {
        const int64_t b = r0 / p.T;
        const int64_t r1 = min(r_end, (b + 1) * p.T);
        const int steps = (int)((r1 - r0 + step - 1) / step);
        const int64_t mine = r0 + team * per_warp + sub; // this lane's row of step 0

        float2 o[K][4]; // 1 + scale
        float2 sum_n[K][4], sum_1[K][4];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            uint4 sc = make_uint4(0, 0, 0, 0);
            if (has[k]) sc = ld_vec(p.scale + b * p.vs8 + col + width * k);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                o[k][w] = add2(dup2(1.0f), wide2(word(sc, w)));
                sum_n[k][w] = sum_1[k][w] = make_float2(0.0f, 0.0f);
            }
        }
        auto request = [&](int i) {
            const int64_t row = mine + (int64_t)i * step;
            const int slot = i % kAhead;
            if (i < steps && row < r1) {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (has[k]) {
                        const int64_t at = row * F + col + width * k;
                        const int to = (slot * K + k) * kThreads + tid;
                        cp_async16(s_dy + to, p.dy + at);
                        if (RES) cp_async16(s_res + to, p.dres + at);
                        if (CKPT) cp_async8(s_x + to, p.codes + at);
                        else cp_async16(s_x + to, p.x + at);
                    }
                if (CKPT && (lane & 31) == 0 && has[0])
                    prefetch_l2_line(p.block_scales + row * p.blocks + (col >> 2));
            }
            cp_async_commit();
        };
        float2 next_stats = make_float2(0.0f, 0.0f);
        unsigned next_code[K];
        auto fetch = [&](int i) { // the row's statistics and block scales, a row ahead
            const int64_t row = mine + (int64_t)i * step;
#pragma unroll
            for (int k = 0; k < K; ++k) next_code[k] = 127;
            if (i < steps && row < r1 && in_team) {
                next_stats = __ldg(p.stats + row);
                if (CKPT)
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        if (has[k]) next_code[k] = __ldg(p.block_scales + row * p.blocks + ((col + width * k) >> 2));
            }
        };
        for (int i = 0; i < kAhead; ++i) request(i);
        fetch(0);

        for (int i = 0; i < steps; ++i) {
            const int64_t row = mine + (int64_t)i * step;
            const bool live = row < r1;
            const float2 st = next_stats;
            float bs[K];
#pragma unroll
            for (int k = 0; k < K; ++k) bs[k] = block_scale_value(next_code[k]);
            fetch(i + 1);
            cp_async_wait<kAhead - 1>();
            float2 n[K][4], g[K][4];
            float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
            const float2 neg_mean = dup2(-st.x), rstd = dup2(st.y);
            uint4 res[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int at = ((i % kAhead) * K + k) * kThreads + tid;
                uint4 dy = make_uint4(0, 0, 0, 0);
                XWord xv = XWord();
                res[k] = dy;
                if (has[k] && live) {
                    dy = s_dy[at];
                    xv = s_x[at];
                    if (RES) res[k] = s_res[at];
                }
                float2 v[4];
                if constexpr (CKPT) {
                    decode8(xv, bs[k], v);
                } else {
#pragma unroll
                    for (int w = 0; w < 4; ++w) v[w] = wide2(word(xv, w));
                }
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float2 d = wide2(word(dy, w));
                    n[k][w] = mul2(add2(v[w], neg_mean), rstd);
                    if (!(has[k] && live)) n[k][w] = make_float2(0.0f, 0.0f);
                    g[k][w] = mul2(d, o[k][w]);
                    sum_1[k][w] = add2(sum_1[k][w], d);
                    sum_n[k][w] = fma2(d, n[k][w], sum_n[k][w]);
                    s1 = add2(s1, g[k][w]);
                    s2 = fma2(g[k][w], n[k][w], s2);
                }
            }
            request(i + kAhead); // into the slot that was just read
            float a = __fadd_rn(s1.x, s1.y), q = __fadd_rn(s2.x, s2.y);
            for (int off = L >> 1; off >= 1; off >>= 1) {
                a = __fadd_rn(a, __shfl_xor_sync(kFull, a, off));
                q = __fadd_rn(q, __shfl_xor_sync(kFull, q, off));
            }
            if (W > 1 && in_team) {
                if (lane == 0) s_red[(i & 1) * kWarps + warp] = make_float2(a, q);
                team_barrier(team, 32 * W);
                a = q = 0.0f;
                for (int j = 0; j < W; ++j) {
                    const float2 t = s_red[(i & 1) * kWarps + team * W + j];
                    a = __fadd_rn(a, t.x);
                    q = __fadd_rn(q, t.y);
                }
            }
            // dx = g * rstd - mean(g) * rstd - n * (mean(g * n) * rstd)
            const float2 m1 = dup2(-__fmul_rn(__fmul_rn(a, p.inv_d), st.y));
            const float2 m2 = dup2(-__fmul_rn(__fmul_rn(q, p.inv_d), st.y));
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!(has[k] && live)) continue;
                uint4 out;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    float2 v = fma2(n[k][w], m2, fma2(g[k][w], rstd, m1));
                    if (RES) v = add2(v, wide2(word(res[k], w)));
                    set_word(out, w, pack_bf16(v.x, v.y));
                }
                st_stream(p.dx + row * F + col + width * k, out);
            }
        }
        cp_async_wait_all();

        // the batch's column sums: of a warp's rows, then of the teams, in order
        for (int off = L; off < 32; off <<= 1)
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    sum_n[k][w].x = __fadd_rn(sum_n[k][w].x, __shfl_xor_sync(kFull, sum_n[k][w].x, off));
                    sum_n[k][w].y = __fadd_rn(sum_n[k][w].y, __shfl_xor_sync(kFull, sum_n[k][w].y, off));
                    sum_1[k][w].x = __fadd_rn(sum_1[k][w].x, __shfl_xor_sync(kFull, sum_1[k][w].x, off));
                    sum_1[k][w].y = __fadd_rn(sum_1[k][w].y, __shfl_xor_sync(kFull, sum_1[k][w].y, off));
                }
        __syncthreads(); // every thread has read its slots
        float2 *s_sum = reinterpret_cast<float2 *>(smem); // [team][K][8][width]
        if (in_team && sub == 0)
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    s_sum[((team * K + k) * 8 + w) * width + col] = sum_n[k][w];
                    s_sum[((team * K + k) * 8 + 4 + w) * width + col] = sum_1[k][w];
                }
        __syncthreads();
        float *part = p.part + (c + b) * 2 * (8 * (int64_t)F);
        for (int i = tid; i < K * 2 * width; i += kThreads) {
            const int k = i / (2 * width), which = i / width & 1, at = i % width;
            const int f = at + width * k;
            if (f >= F) continue;
            float2 v[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) v[w] = make_float2(0.0f, 0.0f);
            for (int t = 0; t < p.teams; ++t)
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    v[w] = add2(v[w], s_sum[((t * K + k) * 8 + 4 * which + w) * width + at]);
            float4 *to = reinterpret_cast<float4 *>(part + (int64_t)which * 8 * F + 8 * f);
            to[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
            to[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
        }
        __syncthreads(); // the sums are read: the slots may be filled again
        r0 = r1;
    }
}

// dscale and dshift of batch b: the partials c + b of the CTAs c that had rows
// of it, added in order (eight threads a share of them each, then the shares).
// A block has 32 groups of four columns of [dscale | dshift].
constexpr int kJoinLanes = 8;
__global__ void __launch_bounds__(32 * kJoinLanes)
    ln_back_join_kernel(const float4 *part, uint2 *dscale, uint2 *dshift, int64_t gs4, int64_t rows,
                        int64_t T, int64_t G, int D4, int tiles)
{
    __shared__ float4 s_sum[kJoinLanes][32];
    const int64_t b = blockIdx.x / tiles;
    const int quad = (int)(blockIdx.x - b * tiles) * 32 + (threadIdx.x & 31);
    const int share = threadIdx.x >> 5;
    grid_dependency_wait();
    allow_dependents();
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (quad < 2 * D4 && rows > 0) {
        // the CTAs of the batch's first and last rows
        auto cta_of = [&](int64_t row) {
            int64_t c = row * G / rows;
            while (first_row(c + 1, rows, G) <= row) ++c;
            while (first_row(c, rows, G) > row) --c;
            return c;
        };
        const int64_t c0 = cta_of(b * T), c1 = cta_of((b + 1) * T - 1);
#pragma unroll 4
        for (int64_t c = c0 + share; c <= c1; c += kJoinLanes) {
            const float4 t = __ldg(part + (c + b) * 2 * D4 + quad);
            v.x = __fadd_rn(v.x, t.x);
            v.y = __fadd_rn(v.y, t.y);
            v.z = __fadd_rn(v.z, t.z);
            v.w = __fadd_rn(v.w, t.w);
        }
    }
    s_sum[share][threadIdx.x & 31] = v;
    __syncthreads();
    if (share != 0 || quad >= 2 * D4) return;
#pragma unroll
    for (int j = 1; j < kJoinLanes; ++j) {
        const float4 t = s_sum[j][threadIdx.x];
        v.x = __fadd_rn(v.x, t.x);
        v.y = __fadd_rn(v.y, t.y);
        v.z = __fadd_rn(v.z, t.z);
        v.w = __fadd_rn(v.w, t.w);
    }
    uint2 *to = quad < D4 ? dscale + b * gs4 + quad : dshift + b * gs4 + quad - D4;
    *to = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

int64_t back_grid(int64_t rows) { return rows < sm_count() ? rows : sm_count(); }

template <int K, bool CKPT, bool RES>
cudaError_t launch_back(const LnBackParams &p, int grid, cudaStream_t s)
{
    const int smem = kAhead * K * kThreads * (16 + (CKPT ? 8 : 16) + (RES ? 16 : 0)) +
                     2 * kWarps * (int)sizeof(float2);
    const auto fn = ln_back_kernel<K, CKPT, RES>;
    const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(fn), smem);
    return e != cudaSuccess ? e : launch_overlapped(fn, grid, kThreads, smem, s, p);
}

} // namespace

int64_t ln_modulate_backward_workspace(int64_t B, int64_t T, int64_t D)
{
    const int64_t rows = B * T;
    return rows == 0 ? 0 : (back_grid(rows) + B) * 2 * D * (int64_t)sizeof(float);
}

cudaError_t launch_ln_modulate_backward(const LnBackProblem &q, cudaStream_t s)
{
    LnBackParams p = {};
    p.dy = static_cast<const uint4 *>(q.dy);
    p.x = static_cast<const uint4 *>(q.x);
    p.codes = static_cast<const uint2 *>(q.codes);
    p.block_scales = static_cast<const uint8_t *>(q.block_scales);
    p.stats = static_cast<const float2 *>(q.stats);
    p.scale = static_cast<const uint4 *>(q.scale);
    p.dres = static_cast<const uint4 *>(q.dres);
    p.dx = static_cast<uint4 *>(q.dx);
    p.part = static_cast<float *>(q.workspace);
    p.rows = q.B * q.T;
    p.T = q.T;
    p.vs8 = q.vs / 8;
    p.F = (int)(q.D / 8);
    p.blocks = (int)((q.D + 31) / 32);
    p.inv_d = 1.0f / (float)q.D;
    const int64_t G = back_grid(p.rows);
    if (p.rows > 0) {
        const int K = p.F <= 256 ? 1 : 2;
        p.W = (p.F + 32 * K - 1) / (32 * K);
        p.teams = kWarps / p.W;
        p.L = 32;
        while (p.W == 1 && p.L / 2 >= p.F) p.L /= 2;
        const bool ckpt = q.x == nullptr, res = q.dres != nullptr;
        auto go = [&](auto k) {
            constexpr int KK = decltype(k)::value;
            if (ckpt) return res ? launch_back<KK, true, true>(p, (int)G, s) : launch_back<KK, true, false>(p, (int)G, s);
            return res ? launch_back<KK, false, true>(p, (int)G, s) : launch_back<KK, false, false>(p, (int)G, s);
        };
        const cudaError_t e = K == 1 ? go(std::integral_constant<int, 1>()) : go(std::integral_constant<int, 2>());
        if (e != cudaSuccess) return e;
    }
    const int D4 = (int)(q.D / 4), tiles = (2 * D4 + 31) / 32;
    if (q.B > (int64_t(1) << 30) / tiles) return cudaErrorInvalidConfiguration;
    return launch_overlapped(ln_back_join_kernel, (int)(q.B * tiles), 32 * kJoinLanes, 0, s,
                             static_cast<const float4 *>(q.workspace), static_cast<uint2 *>(q.dscale),
                             static_cast<uint2 *>(q.dshift), q.gs / 4, p.rows, p.T, G, D4, tiles);
}

} // namespace dan
