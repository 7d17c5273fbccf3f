// dan_gn_back.cu -- gradients of the group norm of channels-last images, for
// sm_103a (include/dan_train.h).
//
// With the forward pass's mean and rstd at hand, everything that dx needs of
// the rest of its group, and all the parameters' gradients, follow from two
// sums per image and channel, s0 = sum dz and s1 = sum dz * n.  So: a kernel
// that reads dy and x (or its checkpoint) once and stores the sums of each chunk
// of rows; one that joins the chunks, per group; one that reads both again (the
// chunks in the opposite order, the last ones still in the L2) and writes dx;
// and for several images one that adds their shares of dweight and dbias.
#include "dan_gn.cuh"

namespace dan {
namespace {

struct GnBackParams {
    const char *dy, *x;
    const uint2 *codes;
    const uint8_t *block_scales;
    const float2 *stats;
    char *dx;
    float2 *part; // [N][P][C] (s0, s1) of a chunk
    float2 *sums; // [N][C]    (s0, s1)
    float2 *mean; // [N][groups] means of a * dz and a * dz * n
    void *dweight, *dbias, *dscale, *dshift;
    Gains gains;
    int64_t gs;
    int64_t S, R, P;
    int F, Ft, tiles, RL;
    int per, groups;
    int act;
};

// A row's fragment of x: its own values, or its checkpoint's.
template <int TYPE, bool CKPT>
struct Input {
    Fragment<TYPE> f;
    __device__ __forceinline__ void load(const GnBackParams &p, int64_t at)
    {
        f.load(p.x + at * Fragment<TYPE>::kBytes);
    }
    __device__ __forceinline__ void values(float2 (&v)[4]) const { f.values(v); }
};
template <int TYPE>
struct Input<TYPE, true> {
    uint2 c;
    unsigned scale;
    __device__ __forceinline__ void load(const GnBackParams &p, int64_t at)
    {
        c = __ldg(p.codes + at);
        scale = __ldg(p.block_scales + (at >> 2));
    }
    __device__ __forceinline__ void values(float2 (&v)[4]) const { decode8(c, block_scale_value(scale), v); }
};

// A thread's eight channels: n = (x - mean) * rstd, z = n * a + b.  UNI: they lie
// in one group.
template <bool UNI>
struct Channels {
    static constexpr int K = UNI ? 1 : 4;
    float2 mean[K], rstd[K], a[4], b[4];
    __device__ __forceinline__ void get(const GnBackParams &p, int64_t n, int f)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = 8 * f + e;
            float g, h;
            p.gains.get(n, c, g, h);
            if (e & 1) a[e / 2].y = g, b[e / 2].y = h;
            else a[e / 2].x = g, b[e / 2].x = h;
            if (UNI && e > 0) continue;
            const float2 st = p.stats[n * p.groups + c / p.per];
            if (UNI) mean[0] = dup2(st.x), rstd[0] = dup2(st.y);
            else if (e & 1) mean[e / 2 % K].y = st.x, rstd[e / 2 % K].y = st.y;
            else mean[e / 2 % K].x = st.x, rstd[e / 2 % K].x = st.y;
        }
    }
    // n of pair w, and dz of dy.
    __device__ __forceinline__ void pair(int w, int act, float2 x, float2 dy, float2 &n, float2 &dz) const
    {
        n = mul2(sub2(x, mean[w % K]), rstd[w % K]);
        dz = dy;
        if (act) {
            const float2 z = fma2(n, a[w], b[w]);
            const float2 p = make_float2(sigmoid(z.x), sigmoid(z.y));
            // the derivative, p * (1 + z * (1 - p))
            dz = mul2(dy, fma2(mul2(z, p), sub2(dup2(1.0f), p), p));
        }
    }
};

struct Where {
    int64_t n, chunk;
    int tile;
    __device__ __forceinline__ Where(int64_t id, int tiles, int64_t P)
    {
        chunk = id % P;
        const int64_t rest = id / P;
        tile = (int)(rest % tiles);
        n = rest / tiles;
    }
};

template <int TYPE, bool CKPT, bool UNI>
__global__ void __launch_bounds__(kGnMost, 1) gn_sums_kernel(const GnBackParams p)
{
    using Frag = Fragment<TYPE>;
    extern __shared__ float2 s_sums[]; // [RL][8 channels of the fragments]
    const int tid = threadIdx.x;
    const Where at(blockIdx.x, p.tiles, p.P);
    const int f0 = at.tile * p.Ft, Ft = min(p.Ft, p.F - f0);
    const int r = tid / p.Ft, f = tid - r * p.Ft;
    const bool here = r < p.RL && f < Ft;
    const int64_t row0 = at.chunk * p.R;
    const int rows = (int)min(p.R, p.S - row0);
    grid_dependency_wait();
    allow_dependents();
    if (here) {
        Channels<UNI> ch;
        ch.get(p, at.n, f0 + f);
        float2 s0[4], s1[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) s0[w] = s1[w] = make_float2(0.0f, 0.0f);
        const int64_t base = (at.n * p.S + row0) * p.F + f0 + f;
        constexpr int U = 4;
        for (int i = r; i < rows; i += U * p.RL) {
            Frag dy[U];
            Input<TYPE, CKPT> x[U];
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (i + j * p.RL < rows) {
                    const int64_t k = base + (int64_t)(i + j * p.RL) * p.F;
                    dy[j].load(p.dy + k * Frag::kBytes);
                    x[j].load(p, k);
                }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (i + j * p.RL >= rows) break;
                float2 v[4], d[4];
                dy[j].values(d);
                x[j].values(v);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    float2 n, dz;
                    ch.pair(w, p.act, v[w], d[w], n, dz);
                    s0[w] = add2(s0[w], dz);
                    s1[w] = fma2(dz, n, s1[w]);
                }
            }
        }
        float4 *to = reinterpret_cast<float4 *>(s_sums + (r * Ft + f) * 8);
#pragma unroll
        for (int w = 0; w < 4; ++w) to[w] = make_float4(s0[w].x, s1[w].x, s0[w].y, s1[w].y);
    }
    __syncthreads();
    for (int c = tid; c < Ft * 8; c += blockDim.x) {
        float2 t = s_sums[c];
        for (int k = 1; k < p.RL; ++k) t = add2(t, s_sums[k * Ft * 8 + c]);
        p.part[(at.n * p.P + at.chunk) * (8 * (int64_t)p.F) + 8 * f0 + c] = t;
    }
}

// Joins the chunks of a group's channels; then what follows from the sums.
constexpr int kJoin = 256;
__global__ void __launch_bounds__(kJoin) gn_back_join_kernel(const GnBackParams p, bool last)
{
    __shared__ float2 s_part[kJoin];
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t n = blockIdx.x / p.groups;
    const int g = (int)(blockIdx.x - n * p.groups);
    const int64_t C = 8 * (int64_t)p.F;
    const int cols = min(p.per, kJoin), shares = kJoin / cols;
    const int col = tid % cols, share = tid / cols;
    grid_dependency_wait();
    allow_dependents();
    float2 all = make_float2(0.0f, 0.0f); // sums of a * s0 and a * s1 over this thread's channels
    for (int j0 = 0; j0 < p.per; j0 += cols) {
        const int64_t c = g * (int64_t)p.per + j0 + col;
        const bool here = share < shares && j0 + col < p.per;
        float2 t = make_float2(0.0f, 0.0f);
        if (here)
#pragma unroll 8
            for (int64_t k = share; k < p.P; k += shares) t = add2(t, __ldcg(p.part + (n * p.P + k) * C + c));
        s_part[tid] = t;
        __syncthreads();
        if (here && share == 0) {
            for (int k = 1; k < shares; ++k) t = add2(t, s_part[k * cols + col]);
            float a, b;
            p.gains.get(n, c, a, b);
            all = fma2(dup2(a), t, all);
            p.sums[n * C + c] = t;
            if (p.dscale) {
                const float w = p.gains.weight ? load_as(p.gains.weight, p.gains.param_type, c) : 1.0f;
                const float v = p.gains.bias ? load_as(p.gains.bias, p.gains.param_type, c) : 0.0f;
                store_as(p.dscale, p.gains.type, n * p.gs + c, __fmaf_rn(w, t.y, __fmul_rn(v, t.x)));
                store_as(p.dshift, p.gains.type, n * p.gs + c, t.x);
            }
            if (last && p.dweight) { // the call's only image
                const float o = p.gains.scale ? __fadd_rn(1.0f, load_as(p.gains.scale, p.gains.type, c)) : 1.0f;
                store_as(p.dweight, p.gains.param_type, c, __fmul_rn(o, t.y));
                store_as(p.dbias, p.gains.param_type, c, __fmul_rn(o, t.x));
            }
        }
        __syncthreads();
    }
    // the group's means
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        all.x = __fadd_rn(all.x, __shfl_xor_sync(kFull, all.x, off));
        all.y = __fadd_rn(all.y, __shfl_xor_sync(kFull, all.y, off));
    }
    if (lane == 0) s_part[tid >> 5] = all;
    __syncthreads();
    if (tid != 0) return;
    for (int k = 1; k < kJoin / 32; ++k) all = add2(all, s_part[k]);
    const float count = (float)(p.S * p.per);
    p.mean[n * p.groups + g] = make_float2(__fdiv_rn(all.x, count), __fdiv_rn(all.y, count));
}

template <int TYPE, bool CKPT, bool UNI>
__global__ void __launch_bounds__(kGnMost, 1) gn_dx_kernel(const GnBackParams p)
{
    using Frag = Fragment<TYPE>;
    const int tid = threadIdx.x;
    const Where at(gridDim.x - 1 - blockIdx.x, p.tiles, p.P); // the last chunk first
    const int f0 = at.tile * p.Ft, Ft = min(p.Ft, p.F - f0);
    const int r = tid / p.Ft, f = f0 + tid - r * p.Ft;
    const int64_t row0 = at.chunk * p.R;
    const int rows = (int)min(p.R, p.S - row0);
    grid_dependency_wait();
    allow_dependents();
    if (r >= p.RL || f - f0 >= Ft) return;
    Channels<UNI> ch;
    ch.get(p, at.n, f);
    constexpr int K = Channels<UNI>::K;
    float2 m1[K], m2[K]; // minus the means, times rstd
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = 8 * f + 2 * k;
        const float2 u = p.mean[at.n * p.groups + c / p.per];
        const float2 v = UNI ? u : p.mean[at.n * p.groups + (c + 1) / p.per];
        m1[k] = mul2(make_float2(-u.x, -v.x), ch.rstd[k]);
        m2[k] = mul2(make_float2(-u.y, -v.y), ch.rstd[k]);
    }
    const int64_t base = (at.n * p.S + row0) * p.F + f;
    constexpr int U = 4;
    for (int i = r; i < rows; i += U * p.RL) {
        Frag dy[U];
        Input<TYPE, CKPT> x[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (i + j * p.RL < rows) {
                const int64_t k = base + (int64_t)(i + j * p.RL) * p.F;
                dy[j].load(p.dy + k * Frag::kBytes);
                x[j].load(p, k);
            }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (i + j * p.RL >= rows) break;
            float2 v[4], d[4];
            dy[j].values(d);
            x[j].values(v);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                float2 n, dz;
                ch.pair(w, p.act, v[w], d[w], n, dz);
                d[w] = fma2(n, m2[w % K], fma2(mul2(dz, ch.a[w]), ch.rstd[w % K], m1[w % K]));
            }
            Frag::store(p.dx + (base + (int64_t)(i + j * p.RL) * p.F) * Frag::kBytes, d);
        }
    }
}

// dweight and dbias from the images' sums, in order; eight threads a channel.
__global__ void __launch_bounds__(256) gn_params_kernel(const GnBackParams p, int64_t N)
{
    __shared__ float2 s_sum[8][32];
    const int share = threadIdx.x >> 5;
    const int64_t C = 8 * (int64_t)p.F, c = blockIdx.x * (int64_t)32 + (threadIdx.x & 31);
    grid_dependency_wait();
    allow_dependents();
    float2 t = make_float2(0.0f, 0.0f);
    if (c < C)
        for (int64_t n = share; n < N; n += 8) {
            const float o = p.gains.scale ? __fadd_rn(1.0f, load_as(p.gains.scale, p.gains.type, n * p.gains.vs + c)) : 1.0f;
            t = fma2(dup2(o), __ldcg(p.sums + n * C + c), t);
        }
    s_sum[share][threadIdx.x & 31] = t;
    __syncthreads();
    if (share != 0 || c >= C) return;
    for (int k = 1; k < 8; ++k) t = add2(t, s_sum[k][threadIdx.x]);
    store_as(p.dweight, p.gains.param_type, c, t.y);
    store_as(p.dbias, p.gains.param_type, c, t.x);
}

GnCut backward_cut(int64_t S, int64_t C, int64_t groups, int type, bool checkpoint)
{
    return gn_cut(S, C, groups, type, checkpoint, 65536, 1024);
}

template <int TYPE, bool CKPT, bool UNI>
cudaError_t launch_passes(const GnBackParams &p, const GnProblem &q, const GnCut &c, int64_t grid, bool last,
                          cudaStream_t s)
{
    const int smem = c.RL * c.Ft * 8 * (int)sizeof(float2);
    cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(gn_sums_kernel<TYPE, CKPT, UNI>), smem);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(gn_sums_kernel<TYPE, CKPT, UNI>, (int)grid, c.threads, smem, s, p);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(gn_back_join_kernel, (int)(q.N * q.groups), kJoin, 0, s, p, last);
    if (e != cudaSuccess) return e;
    return launch_overlapped(gn_dx_kernel<TYPE, CKPT, UNI>, (int)grid, c.threads, 0, s, p);
}

template <int TYPE>
cudaError_t launch_type(const GnBackParams &p, const GnProblem &q, const GnCut &c, int64_t grid, bool last,
                        cudaStream_t s)
{
    const bool uni = p.per % 8 == 0;
    if (q.x == nullptr)
        return uni ? launch_passes<TYPE, true, true>(p, q, c, grid, last, s)
                   : launch_passes<TYPE, true, false>(p, q, c, grid, last, s);
    return uni ? launch_passes<TYPE, false, true>(p, q, c, grid, last, s)
               : launch_passes<TYPE, false, false>(p, q, c, grid, last, s);
}

} // namespace

int64_t group_norm_backward_workspace(int64_t N, int64_t S, int64_t C, int64_t groups, int type, bool checkpoint)
{
    const GnCut c = backward_cut(S, C, groups, type, checkpoint);
    return N * (C * (c.P + 1) + groups) * (int64_t)sizeof(float2);
}

cudaError_t launch_group_norm_backward(const GnProblem &q, cudaStream_t s)
{
    const bool ckpt = q.x == nullptr;
    const GnCut c = backward_cut(q.S, q.C, q.groups, q.type, ckpt);
    GnBackParams p = {};
    p.dy = static_cast<const char *>(q.dy);
    p.x = static_cast<const char *>(q.x);
    p.codes = static_cast<const uint2 *>(q.codes);
    p.block_scales = static_cast<const uint8_t *>(q.block_scales);
    p.stats = static_cast<const float2 *>(q.stats);
    p.dx = static_cast<char *>(q.dx);
    p.part = static_cast<float2 *>(q.workspace);
    p.sums = p.part + q.N * c.P * q.C;
    p.mean = p.sums + q.N * q.C;
    p.dweight = q.dweight;
    p.dbias = q.dbias;
    p.dscale = q.dscale;
    p.dshift = q.dshift;
    p.gains = Gains{q.weight, q.bias, q.scale, q.shift, q.param_type, q.type, q.vs};
    p.gs = q.gs;
    p.S = q.S;
    p.R = c.R;
    p.P = c.P;
    p.F = c.F;
    p.Ft = c.Ft;
    p.tiles = c.tiles;
    p.RL = c.RL;
    p.per = (int)(q.C / q.groups);
    p.groups = (int)q.groups;
    p.act = q.act;
    const bool last = q.N == 1;
    const int64_t grid = q.N * c.tiles * c.P, joins = q.N * q.groups;
    if (grid > 0x7FFFFFFF || joins > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaSuccess;
    if (grid > 0)
        e = q.type == kBf16   ? launch_type<kBf16>(p, q, c, grid, last, s)
            : q.type == kFp16 ? launch_type<kFp16>(p, q, c, grid, last, s)
                              : launch_type<kFp32>(p, q, c, grid, last, s);
    else if (joins > 0) // no positions: sums of nothing
        e = launch_overlapped(gn_back_join_kernel, (int)joins, kJoin, 0, s, p, last);
    if (e != cudaSuccess || last || !q.dweight) return e;
    return launch_overlapped(gn_params_kernel, (int)((q.C + 31) / 32), 256, 0, s, p, q.N);
}

} // namespace dan
