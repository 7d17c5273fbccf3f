// dan_ln_back.cu -- gradients of LayerNorm + modulate for sm_103a
// (include/dan_train.h).
//
// With n = (x - mean) * rstd and g = dy * (1 + scale), a row's
//   dx = rstd * (g - mean(g) - n * mean(g * n)) [+ dres]
// needs two sums over the row, and dscale, dshift are sums of dy * n and dy
// over a batch's rows: one pass over the data, bound by HBM.
//
// A CTA per SM takes a contiguous block of rows.  Its warps form teams of W warps
// (narrow rows: several rows share a warp) that take R rows at a time; every
// thread has the same K fragments of eight columns of each of its team's rows, so
// the column sums stay in its registers until the batch ends.  K * R is large, up
// to eight fragments, on eight warps of up to 255 registers: what a step costs
// apart from its elements, the exchange of the rows' sums above all, is spread
// over 32 to 64 elements of a thread, and the rows' chains of shuffles and
// barriers run side by side (4216 x 4096: 24.0 us, 0.53 of the copy rate, some 8 us
// of it the call's two ends; 33 with one or two fragments on sixteen warps; one row
// at a time by two teams of four warps is no slower than four rows by one of eight).
// Each thread copies its own columns of the next rows into shared memory with
// cp.async and nobody else reads them.  At the end
// of a batch, or of the CTA's rows, the teams' column sums are added in order and
// stored as one partial of the batch; a second kernel adds the partials in order.
// Many short batches go to dan_ln_back_short.cu.
#include "dan_ln_back.cuh"

namespace dan {
namespace {

// Threads of a CTA: large shares take the registers of two threads.
__host__ __device__ constexpr int threads_of(int K, int R) { return K * R <= 2 ? 512 : 256; }

// Steps (of R rows of each team) in flight: four, or what shared memory has room for.
__host__ __device__ constexpr int ahead_of(int K, int R, bool ckpt, bool res)
{
    const int step = R * K * threads_of(K, R) * (16 + (ckpt ? 8 : 16) + (res ? 16 : 0));
    return 4 * step <= 220 * 1024 ? 4 : 3 * step <= 220 * 1024 ? 3 : 2;
}

// Bytes of a hint.
constexpr int kHint = 8192;

// First row of CTA c of G.
__host__ __device__ inline int64_t first_row(int64_t c, int64_t rows, int64_t G) { return c * rows / G; }

// K fragments per thread, R rows at a time.  MULTI: several rows share a warp
// (K == R == W == 1).
template <int K, int R, bool CKPT, bool RES, bool MULTI>
__global__ void __launch_bounds__(threads_of(K, R), 1) ln_back_kernel(const LnBackParams p)
{
    using XWord = typename std::conditional<CKPT, uint2, uint4>::type;
    constexpr int NT = threads_of(K, R), A = ahead_of(K, R, CKPT, RES), NV = 2 * R;
    extern __shared__ __align__(16) uint4 smem[];
    uint4 *s_dy = smem;                   // [A][R][K][NT]
    uint4 *s_res = s_dy + A * R * K * NT; // likewise (RES)
    XWord *s_x = reinterpret_cast<XWord *>(s_res + (RES ? A * R * K * NT : 0));
    float *s_red = reinterpret_cast<float *>(s_x + A * R * K * NT); // [2][warps][NV]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int W = p.W, L = MULTI ? p.L : 32, F = p.F;
    const int team = warp / W;
    const bool in_team = team < p.teams;
    const int sub = MULTI ? lane / L : 0, per_warp = MULTI ? 32 / L : R; // this lane's row of its team's
    const int width = MULTI ? L : 32 * W;                                // threads of a row
    const int col = MULTI ? lane - sub * L : (warp - team * W) * 32 + lane;
    const int step = p.teams * per_warp; // rows of a CTA's step
    const int64_t c = blockIdx.x, G = gridDim.x;
    const int64_t r_begin = first_row(c, p.rows, G), r_end = first_row(c + 1, p.rows, G);
    // every fragment but a thread's last is there for sure
    const bool has_last = in_team && col + width * (K - 1) < F;
    auto has = [&](int k) { return k < K - 1 || has_last; };
    const bool whole = F == width * K; // all threads have all theirs

    // the CTA's first rows, those of two steps, hinted into the L2 before the dependency
    // wait (prefetch_l2: it returns nothing).  Several rows a warp: up to 1024 of
    // them, one piece of each tensor (a hint a row made 600000 rows of 8 columns take
    // 19.7 us, so 9.6).  Else a warp a row (in pieces, rows of 4096 took 0.4 us more).
    if (MULTI) {
        const int rows = (int)min(r_end - r_begin, (int64_t)2 * step), bytes = rows * F * 16, turn = lane * (NT / 32) + warp;
        const int64_t first = r_begin * F * 16;
        for (int i = turn * kHint; i < bytes; i += NT * kHint) {
            const unsigned n = min(kHint, bytes - i);
            prefetch_l2(reinterpret_cast<const char *>(p.dy) + first + i, n);
            if (RES) prefetch_l2(reinterpret_cast<const char *>(p.dres) + first + i, n);
            if (!CKPT) prefetch_l2(reinterpret_cast<const char *>(p.x) + first + i, n);
            if (CKPT && p.hint_codes) prefetch_l2(reinterpret_cast<const char *>(p.codes) + (first + i) / 2, n / 2);
        }
        const char *scales = reinterpret_cast<const char *>(p.block_scales) + r_begin * p.blocks;
        if (CKPT)
            for (int i = turn * 128; i < rows * p.blocks; i += NT * 128) prefetch_l2_line(scales + i);
        for (int i = turn * 16; i < rows; i += NT * 16) prefetch_l2_line(p.stats + r_begin + i);
    } else {
        for (int64_t row = r_begin + warp; row < min(r_end, r_begin + 2 * step); row += NT / 32) {
            if (lane == 0) prefetch_l2(p.dy + row * F, F * 16);
            if (RES && lane == 1) prefetch_l2(p.dres + row * F, F * 16);
            if (!CKPT && lane == 2) prefetch_l2(p.x + row * F, F * 16);
            if (CKPT && lane == 2 && p.hint_codes) prefetch_l2(p.codes + row * F, F * 8);
            if (CKPT && lane == 3) prefetch_l2_line(p.block_scales + row * p.blocks);
            if (lane == 4) prefetch_l2_line(p.stats + row);
        }
    }
    grid_dependency_wait();
    allow_dependents();

    for (int64_t r0 = r_begin; r0 < r_end;) {
        const int64_t b = r0 / p.T;
        const int64_t r1 = min(r_end, (b + 1) * p.T);
        const int64_t first = r0 + team * per_warp + sub; // this lane's first row
        const int64_t team_first = r0 + team * per_warp;
        const int steps = in_team && team_first < r1 ? (int)((r1 - team_first + step - 1) / step) : 0;

        // this lane's rows: those of a step begin at `row`, with `left` from there on
        // (what is requested or fetched ahead follows from the two)
        int64_t row = first;
        int left = in_team ? (int)(r1 - first) : 0;
        auto request = [&](int ahead, int slot) { // of the step `ahead` of this one
            const int64_t at0 = (row + ahead * step) * F + col;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r < left - ahead * step) {
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        if (has(k)) {
                            const int64_t at = at0 + (int64_t)r * F + width * k;
                            const int to = ((slot * R + r) * K + k) * NT + tid;
                            cp_async16(s_dy + to, p.dy + at);
                            if (RES) cp_async16(s_res + to, p.dres + at);
                            if (CKPT) cp_async8(s_x + to, p.codes + at);
                            else cp_async16(s_x + to, p.x + at);
                        }
                }
            cp_async_commit();
        };
        float2 next_stats[R];
        unsigned next_code[R][K];
        auto fetch = [&](int ahead) { // its statistics and block scales
            const int64_t next = row + ahead * step;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r < left - ahead * step) {
                    next_stats[r] = __ldg(p.stats + next + r);
                    if (CKPT) {
                        const uint8_t *scales = p.block_scales + (next + r) * p.blocks + (col >> 2);
#pragma unroll
                        for (int k = 0; k < K; ++k)
                            if (has(k)) next_code[r][k] = __ldg(scales + (width >> 2) * k);
                    }
                }
        };
#pragma unroll
        for (int r = 0; r < R; ++r) {
            next_stats[r] = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < K; ++k) next_code[r][k] = 127;
        }
        for (int i = 0; i < A; ++i) request(i, i);
        fetch(0);

        float2 sum_n[K][4], sum_1[K][4], o[K][4]; // o: 1 + scale
#pragma unroll
        for (int k = 0; k < K; ++k) {
            uint4 sc = make_uint4(0, 0, 0, 0);
            if (in_team && has(k)) sc = ld_vec(p.scale + b * p.vs8 + col + width * k);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                o[k][w] = add2(dup2(1.0f), wide2(word(sc, w)));
                sum_n[k][w] = sum_1[k][w] = make_float2(0.0f, 0.0f);
            }
        }
        int slot = 0;
        for (int i = 0; i < steps; ++i) {
            float2 st[R], n[R][K][4], g[R][K][4];
            float bs[R][K], sums[NV];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                st[r] = next_stats[r];
#pragma unroll
                for (int k = 0; k < K; ++k) bs[r][k] = block_scale_value(next_code[r][k]);
            }
            fetch(1);
            cp_async_wait<A - 1>();
            // one row at a time, a step's row is there
            auto live = [&](int r) { return (!MULTI && R == 1) || r < left; };
            // The elements' n and g, and the sums.  MASKED: some rows or columns may
            // not be there; they count as zeros, and are rare.
            auto take = [&](auto masked) {
                constexpr bool MASKED = decltype(masked)::value;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
                    const float2 neg_mean = dup2(-st[r].x), rstd = dup2(st[r].y);
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        const int at = ((slot * R + r) * K + k) * NT + tid;
                        uint4 dy = make_uint4(0, 0, 0, 0);
                        XWord xv = XWord();
                        const bool here = !MASKED || (has(k) && live(r));
                        if (here) {
                            dy = s_dy[at];
                            xv = s_x[at];
                        }
                        float2 v[4];
                        if constexpr (CKPT) {
                            const float2 s = dup2(bs[r][k]);
                            v[0] = fma2(e4m3_pair(xv.x & 0xFFFFu), s, neg_mean);
                            v[1] = fma2(e4m3_pair(xv.x >> 16), s, neg_mean);
                            v[2] = fma2(e4m3_pair(xv.y & 0xFFFFu), s, neg_mean);
                            v[3] = fma2(e4m3_pair(xv.y >> 16), s, neg_mean);
                        } else {
#pragma unroll
                            for (int w = 0; w < 4; ++w) v[w] = add2(wide2(word(xv, w)), neg_mean);
                        }
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const float2 d = wide2(word(dy, w));
                            n[r][k][w] = mul2(v[w], rstd);
                            if (MASKED && !here) n[r][k][w] = make_float2(0.0f, 0.0f); // whatever the statistics
                            g[r][k][w] = mul2(d, o[k][w]);
                            sum_1[k][w] = add2(sum_1[k][w], d);
                            sum_n[k][w] = fma2(d, n[r][k][w], sum_n[k][w]);
                            s1 = add2(s1, g[r][k][w]);
                            s2 = fma2(g[r][k][w], n[r][k][w], s2);
                        }
                    }
                    sums[2 * r] = __fadd_rn(s1.x, s1.y);
                    sums[2 * r + 1] = __fadd_rn(s2.x, s2.y);
                }
            };
            if (!MULTI && whole && left >= R) take(std::false_type());
            else take(std::true_type());
            if (MULTI) {
                for (int off = L >> 1; off >= 1; off >>= 1) {
                    sums[0] = __fadd_rn(sums[0], __shfl_xor_sync(kFull, sums[0], off));
                    sums[1] = __fadd_rn(sums[1], __shfl_xor_sync(kFull, sums[1], off));
                }
            } else {
                constexpr int LV = 32 / NV; // lanes per value
                float v = warp_sums<NV>(sums, lane);
                if (W > 1) {
                    float *red = s_red + (i & 1) * (NT / 32) * NV;
                    if (lane % LV == 0) red[warp * NV + lane / LV] = v;
                    team_barrier(team, 32 * W);
                    v = 0.0f; // a value's lanes take every LV-th warp's
                    for (int k = lane % LV; k < W; k += LV) v = __fadd_rn(v, red[(team * W + k) * NV + lane / LV]);
#pragma unroll
                    for (int off = 1; off < LV; off *= 2) v = __fadd_rn(v, __shfl_xor_sync(kFull, v, off));
                }
#pragma unroll
                for (int k = 0; k < NV; ++k) sums[k] = __shfl_sync(kFull, v, k * LV);
            }
            // dx = g * rstd - mean(g) * rstd - n * (mean(g * n) * rstd)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float2 rstd = dup2(st[r].y);
                const float2 m1 = dup2(-__fmul_rn(__fmul_rn(sums[2 * r], p.inv_d), st[r].y));
                const float2 m2 = dup2(-__fmul_rn(__fmul_rn(sums[2 * r + 1], p.inv_d), st[r].y));
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    uint4 out, res = make_uint4(0, 0, 0, 0);
                    if (RES) res = s_res[((slot * R + r) * K + k) * NT + tid];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        float2 v = fma2(n[r][k][w], m2, fma2(g[r][k][w], rstd, m1));
                        if (RES) v = add2(v, wide2(word(res, w)));
                        set_word(out, w, pack_bf16(v.x, v.y));
                    }
                    if (has(k) && live(r)) st_stream(p.dx + (row + r) * F + col + width * k, out);
                }
            }
            request(A, slot); // into the slot that was read
            slot = slot + 1 == A ? 0 : slot + 1;
            row += step;
            left -= step;
        }
        cp_async_wait_all();

        // the batch's column sums: of a warp's rows, then of the teams, in order
        if (MULTI)
            for (int off = L; off < 32; off <<= 1)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    sum_n[0][w].x = __fadd_rn(sum_n[0][w].x, __shfl_xor_sync(kFull, sum_n[0][w].x, off));
                    sum_n[0][w].y = __fadd_rn(sum_n[0][w].y, __shfl_xor_sync(kFull, sum_n[0][w].y, off));
                    sum_1[0][w].x = __fadd_rn(sum_1[0][w].x, __shfl_xor_sync(kFull, sum_1[0][w].x, off));
                    sum_1[0][w].y = __fadd_rn(sum_1[0][w].y, __shfl_xor_sync(kFull, sum_1[0][w].y, off));
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
        for (int i = tid; i < K * 2 * width; i += NT) {
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
// of it, added in order: SHARES threads a share of them each (a few, all under way at
// once), then the shares of a warp, then the warps'.  A block has 256 / SHARES
// groups of four columns of [dscale | dshift].  With 64 shares whatever their number, a
// batch of 4096 columns had 512 blocks: 22 us for 16 batches, 85 for 61.
constexpr int kJoinThreads = 256;
template <int SHARES>
__global__ void __launch_bounds__(kJoinThreads)
    ln_back_join_kernel(const float4 *part, uint2 *dscale, uint2 *dshift, int64_t gs4, int64_t rows,
                        int64_t T, int64_t G, int D4, int tiles)
{
    constexpr int kQuads = kJoinThreads / SHARES, kWarps = kJoinThreads / 32, kAcross = kQuads < 32 ? kQuads : 32;
    __shared__ float4 s_sum[SHARES > 1 ? kWarps : 1][kAcross];
    __shared__ int64_t s_cta[2];
    const unsigned b = blockIdx.x / (unsigned)tiles;
    const int tid = threadIdx.x, mine = tid % kQuads, share = tid / kQuads;
    const int quad = (int)(blockIdx.x - b * tiles) * kQuads + mine;
    // the CTAs of the batch's first and last rows
    if (tid < 2) {
        const int64_t row = (b + tid) * T - tid;
        int64_t c = row * G / rows;
        while (first_row(c + 1, rows, G) <= row) ++c;
        while (first_row(c, rows, G) > row) --c;
        s_cta[tid] = c;
    }
    __syncthreads();
    const int64_t c0 = s_cta[0], c1 = s_cta[1];
    grid_dependency_wait();
    allow_dependents();
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](const float4 &t) {
        v.x = __fadd_rn(v.x, t.x);
        v.y = __fadd_rn(v.y, t.y);
        v.z = __fadd_rn(v.z, t.z);
        v.w = __fadd_rn(v.w, t.w);
    };
    if (quad < 2 * D4) {
        const float4 *from = part + b * (int64_t)(2 * D4) + quad;
#pragma unroll 3
        for (int64_t c = c0 + share; c <= c1; c += SHARES) add(__ldcg(from + c * 2 * D4));
    }
#pragma unroll
    for (int off = kQuads; off < 32; off *= 2)
        add(make_float4(__shfl_xor_sync(kFull, v.x, off), __shfl_xor_sync(kFull, v.y, off),
                        __shfl_xor_sync(kFull, v.z, off), __shfl_xor_sync(kFull, v.w, off)));
    if (SHARES > 1) {
        if ((tid & 31) < kAcross) s_sum[tid >> 5][mine] = v;
        __syncthreads();
        if (tid >= kQuads) return;
#pragma unroll
        for (int j = 1; j < kWarps; ++j) add(s_sum[j][mine]);
    }
    if (quad >= 2 * D4) return;
    uint2 *to = quad < D4 ? dscale + b * gs4 + quad : dshift + b * gs4 + quad - D4;
    *to = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

int64_t back_grid(int64_t rows) { return rows < sm_count() ? rows : sm_count(); }

// Calls f with the shares of a batch's partials: up to G / B + 2 of them.
template <typename F>
cudaError_t with_shares(int64_t B, int64_t G, F f)
{
    const int64_t most = (G + B - 1) / B + 1;
    if (most > 16) return f(std::integral_constant<int, 64>());
    if (most > 4) return f(std::integral_constant<int, 8>());
    return f(std::integral_constant<int, 1>());
}

template <int K, int R, bool CKPT, bool RES, bool MULTI>
cudaError_t launch_back(LnBackParams p, int grid, cudaStream_t s)
{
    constexpr int NT = threads_of(K, R);
    p.teams = NT / 32 / p.W;
    const int smem = ahead_of(K, R, CKPT, RES) * R * K * NT * (16 + (CKPT ? 8 : 16) + (RES ? 16 : 0)) +
                     2 * (NT / 32) * 2 * R * (int)sizeof(float);
    const auto fn = ln_back_kernel<K, R, CKPT, RES, MULTI>;
    const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(fn), smem);
    return e != cudaSuccess ? e : launch_overlapped(fn, grid, NT, smem, s, p);
}

} // namespace

LnBackParams ln_back_params(const LnBackProblem &q)
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
    p.hint_codes = p.F % 2 == 0 && reinterpret_cast<uintptr_t>(q.codes) % 16 == 0;
    const LnBackCut c = ln_back_cut(p.F);
    p.W = c.W;
    p.L = c.L;
    return p;
}

int64_t ln_modulate_backward_workspace(int64_t B, int64_t T, int64_t D)
{
    return ln_back_is_short(B, T, D) ? 0 : (back_grid(B * T) + B) * 2 * D * (int64_t)sizeof(float);
}

cudaError_t launch_ln_modulate_backward(const LnBackProblem &q, cudaStream_t s)
{
    if (ln_back_is_short(q.B, q.T, q.D)) return launch_ln_back_short(q, s);
    const LnBackParams p = ln_back_params(q);
    const int64_t G = back_grid(p.rows);
    const int D4 = (int)(q.D / 4);
    return with_shares(q.B, G, [&](auto shares) {
        constexpr int kQuads = kJoinThreads / decltype(shares)::value;
        const auto join = ln_back_join_kernel<decltype(shares)::value>;
        const int tiles = (2 * D4 + kQuads - 1) / kQuads;
        // the call's kernels are made ready before the first launch
        cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(join), 0);
        if (e != cudaSuccess) return e;
        e = with_cut(ln_back_cut(p.F), [&](auto k, auto rows, auto multi) {
            constexpr int K = decltype(k)::value, R = decltype(rows)::value;
            constexpr bool M = decltype(multi)::value;
            if (!p.x) return p.dres ? launch_back<K, R, true, true, M>(p, (int)G, s) : launch_back<K, R, true, false, M>(p, (int)G, s);
            return p.dres ? launch_back<K, R, false, true, M>(p, (int)G, s) : launch_back<K, R, false, false, M>(p, (int)G, s);
        });
        if (e != cudaSuccess) return e;
        return launch_overlapped(join, (int)(q.B * tiles), kJoinThreads, 0, s, static_cast<const float4 *>(q.workspace),
                                 static_cast<uint2 *>(q.dscale), static_cast<uint2 *>(q.dshift), q.gs / 4, p.rows, p.T, G,
                                 D4, tiles);
    });
}

} // namespace dan
