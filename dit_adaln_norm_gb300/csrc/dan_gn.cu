// dan_gn.cu -- group norm of channels-last images with an activation, for
// sm_103a (include/dan_train.h).
//
// A group's mean and variance need all of an image's rows before the first
// output can be written.  Three launches: the moments of each chunk of rows
// (x read once), their join per group, and the normalisation, which reads x
// again, the chunks in the opposite order so that what the first kernel read
// last still lies in the L2.
//
// Moments: a thread sums d and d^2 of its values' differences d from its first
// one (so that a level far above the spread costs no accuracy), turns them into
// a mean and a sum of squares about it, and these are joined pairwise in a fixed
// order.
#include "dan_gn.cuh"

namespace dan {
namespace {

struct GnParams {
    const char *x;
    char *y;
    float2 *part;  // [N][groups][P] mean and squared sum of a chunk
    float2 *stats; // [N][groups] mean and rstd
    uint2 *codes;
    uint8_t *block_scales;
    Gains gains;
    int64_t S, R, P;
    int F, Ft, tiles, RL;
    int per;    // channels per group
    int groups;
    int unit;   // channels of a fragment that are sure to lie in one group: gcd(per, 8)
    int act;
    float eps;
};

// The CTA's image, tile and chunk.
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

// ----------------------------------------------------------------- moments

// A thread's sums of differences from a pivot (for eight channels).
struct Sums {
    float2 pivot[4], s1[4], s2[4];
    __device__ __forceinline__ void start(const float2 (&v)[4], int unit)
    {
        pivot[0] = unit == 1 ? v[0] : dup2(v[0].x);
        pivot[1] = unit == 1 ? v[1] : unit == 2 ? dup2(v[1].x) : dup2(v[0].x);
        pivot[2] = unit == 1 ? v[2] : unit == 8 ? dup2(v[0].x) : dup2(v[2].x);
        pivot[3] = unit == 1 ? v[3] : unit == 2 ? dup2(v[3].x) : unit == 4 ? dup2(v[2].x) : dup2(v[0].x);
#pragma unroll
        for (int w = 0; w < 4; ++w) s1[w] = s2[w] = make_float2(0.0f, 0.0f);
    }
    __device__ __forceinline__ void add(const float2 (&v)[4])
    {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float2 d = sub2(v[w], pivot[w]);
            s1[w] = add2(s1[w], d);
            s2[w] = fma2(d, d, s2[w]);
        }
    }
    // Mean and squared sum of each unit of `unit` channels over `rows` rows, to
    // `to` (8 / unit of them).
    __device__ __forceinline__ void finish(int unit, int rows, float2 *to) const
    {
        float a[8], q[8], p[8];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            a[2 * w] = s1[w].x, a[2 * w + 1] = s1[w].y;
            q[2 * w] = s2[w].x, q[2 * w + 1] = s2[w].y;
            p[2 * w] = pivot[w].x, p[2 * w + 1] = pivot[w].y;
        }
#pragma unroll
        for (int k = 1; k < 8; k *= 2)
            if (k < unit) {
#pragma unroll
                for (int i = 0; i < 8; i += 2 * k) {
                    a[i] = __fadd_rn(a[i], a[i + k]);
                    q[i] = __fadd_rn(q[i], q[i + k]);
                }
            }
        const float inv = 1.0f / (float)(rows * unit);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i % unit == 0) {
                const float d = __fmul_rn(a[i], inv);
                to[i / unit] = make_float2(__fadd_rn(p[i], d), fmaxf(__fmaf_rn(-a[i], d, q[i]), 0.0f));
            }
    }
};

template <int TYPE>
__global__ void __launch_bounds__(kGnMost, 2) gn_moments_kernel(const GnParams p)
{
    using Frag = Fragment<TYPE>;
    extern __shared__ float2 s_units[]; // [RL][units of the tile]
    const int tid = threadIdx.x, lane = tid & 31;
    const Where at(blockIdx.x, p.tiles, p.P);
    const int f0 = at.tile * p.Ft, Ft = min(p.Ft, p.F - f0);
    const int r = tid / p.Ft, f = tid - r * p.Ft;
    const int64_t row0 = at.chunk * p.R;
    const int rows = (int)min(p.R, p.S - row0); // of the chunk
    const int mine = r < p.RL && f < Ft && r < rows ? (rows - r + p.RL - 1) / p.RL : 0;
    const int64_t row_bytes = (int64_t)p.F * Frag::kBytes, step = row_bytes * p.RL;
    const char *x = p.x + ((at.n * p.S + row0 + r) * p.F + f0 + f) * Frag::kBytes;
    grid_dependency_wait();
    allow_dependents();
    const int per_frag = 8 / p.unit, units = Ft * per_frag;
    if (mine > 0) {
        Sums sums;
        float2 v[4];
        Frag a[4];
        a[0].load(x);
        a[0].values(v);
        sums.start(v, p.unit);
        int i = 0;
        for (; i + 4 <= mine; i += 4, x += 4 * step) {
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j].load(x + j * step);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a[j].values(v);
                sums.add(v);
            }
        }
        for (; i < mine; ++i, x += step) {
            a[0].load(x);
            a[0].values(v);
            sums.add(v);
        }
        sums.finish(p.unit, mine, s_units + r * units + f * per_frag);
    }
    __syncthreads();
    // a warp joins a group's entries: its units of every row lane
    const int per_group = p.per / p.unit, groups = Ft * 8 / p.per;
    const int lanes = min(p.RL, rows);
    for (int g = tid >> 5; g < groups; g += blockDim.x >> 5) {
        Moments m{0.0f, 0.0f, 0.0f};
        for (int e = lane; e < lanes * per_group; e += 32) {
            const int rl = e / per_group, u = e - rl * per_group;
            const float2 t = s_units[rl * units + g * per_group + u];
            m = join(m, Moments{(float)((rows - rl + p.RL - 1) / p.RL * p.unit), t.x, t.y});
        }
        m = join_warp(m, lane);
        if (lane == 0)
            p.part[(at.n * p.groups + f0 * 8 / p.per + g) * p.P + at.chunk] = make_float2(m.mean, m.m2);
    }
}

// Mean and rstd of each group (a warp's) from its chunks' moments.
__global__ void __launch_bounds__(128)
    gn_join_kernel(const float2 *part, float2 *stats, int64_t total, int64_t P, int64_t S, int64_t R, int per,
                   float eps)
{
    const int lane = threadIdx.x & 31;
    const int64_t g = blockIdx.x * (int64_t)4 + (threadIdx.x >> 5);
    grid_dependency_wait();
    allow_dependents();
    if (g >= total) return;
    Moments m{0.0f, 0.0f, 0.0f};
    for (int64_t c = lane; c < P; c += 32) {
        const float2 t = __ldg(part + g * P + c);
        m = join(m, Moments{(float)((c + 1 < P ? R : S - c * R) * per), t.x, t.y});
    }
    m = join_warp(m, lane);
    if (lane == 0) stats[g] = make_float2(m.mean, defined_rsqrt(__fadd_rn(__fdiv_rn(m.m2, (float)(S * per)), eps)));
}

// --------------------------------------------------------------- normalise

// What a thread needs of its eight channels: z = (x - mean) * a + b.
struct Norm {
    float2 mean[4], a[4], b[4];
    __device__ __forceinline__ void get(const GnParams &p, int64_t n, int f)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = 8 * f + e;
            const float2 st = p.stats[n * p.groups + c / p.per];
            float g, h;
            p.gains.get(n, c, g, h);
            g = __fmul_rn(g, st.y);
            if (e & 1) mean[e / 2].y = st.x, a[e / 2].y = g, b[e / 2].y = h;
            else mean[e / 2].x = st.x, a[e / 2].x = g, b[e / 2].x = h;
        }
    }
    __device__ __forceinline__ void apply(const float2 (&v)[4], int act, float2 (&z)[4]) const
    {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            z[w] = fma2(sub2(v[w], mean[w]), a[w], b[w]);
            if (act) z[w] = mul2(z[w], make_float2(sigmoid(z[w].x), sigmoid(z[w].y)));
        }
    }
};

// The checkpoint of a fragment: four neighbouring lanes have a block of 32
// channels (tiles start at a block, and a block's lanes are all here or none).
__device__ __forceinline__ void store_codes(uint2 *codes, uint8_t *block_scale, const float2 (&v)[4], bool here,
                                            int f)
{
    float x[8];
#pragma unroll
    for (int w = 0; w < 4; ++w) x[2 * w] = v[w].x, x[2 * w + 1] = v[w].y;
    float top = here ? top8(x) : 0.0f;
    top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
    top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
    if (!here) return;
    const unsigned code = block_scale_code(top);
    st_stream8(codes, e4m3x8(x, block_scale_inverse(code)));
    if ((f & 3) == 0) *block_scale = (uint8_t)code;
}

template <int TYPE, bool CKPT>
__global__ void __launch_bounds__(kGnMost, 2) gn_apply_kernel(const GnParams p)
{
    using Frag = Fragment<TYPE>;
    const int tid = threadIdx.x;
    const Where at(gridDim.x - 1 - blockIdx.x, p.tiles, p.P); // the last chunk first
    const int f0 = at.tile * p.Ft, Ft = min(p.Ft, p.F - f0);
    const int r = tid / p.Ft, f = f0 + tid - r * p.Ft;
    const bool here = r < p.RL && f - f0 < Ft;
    const int64_t row0 = at.chunk * p.R;
    const int rows = (int)min(p.R, p.S - row0);
    grid_dependency_wait();
    allow_dependents();
    Norm norm = {};
    if (here) norm.get(p, at.n, f);
    constexpr int U = CKPT ? 2 : 4; // rows in flight
    for (int i = r; i - r < rows; i += U * p.RL) {
        Frag a[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (here && i + j * p.RL < rows)
                a[j].load(p.x + ((at.n * p.S + row0 + i + j * p.RL) * p.F + f) * Frag::kBytes);
            else a[j].zero();
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const bool live = here && i + j * p.RL < rows;
            const int64_t to = (at.n * p.S + row0 + i + j * p.RL) * p.F + f;
            float2 v[4], z[4];
            a[j].values(v);
            norm.apply(v, p.act, z);
            if (live) Frag::store(p.y + to * Frag::kBytes, z);
            if (CKPT) store_codes(p.codes + to, p.block_scales + (to >> 2), v, live, f);
        }
    }
}

GnCut forward_cut(int64_t S, int64_t C, int64_t groups, int type, bool checkpoint)
{
    return gn_cut(S, C, groups, type, checkpoint, 65536, 1024);
}

template <int TYPE>
cudaError_t launch_type(const GnParams &p, const GnProblem &q, const GnCut &c, cudaStream_t s)
{
    const int64_t grid = q.N * c.tiles * c.P, total = q.N * q.groups;
    if (grid > 0x7FFFFFFF || total > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const int smem = c.RL * c.Ft * (8 / p.unit) * (int)sizeof(float2);
    cudaError_t e = launch_overlapped(gn_moments_kernel<TYPE>, (int)grid, c.threads, smem, s, p);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(gn_join_kernel, (int)((total + 3) / 4), 128, 0, s, static_cast<const float2 *>(p.part),
                          p.stats, total, c.P, q.S, c.R, p.per, q.eps);
    if (e != cudaSuccess) return e;
    return p.codes ? launch_overlapped(gn_apply_kernel<TYPE, true>, (int)grid, c.threads, 0, s, p)
                   : launch_overlapped(gn_apply_kernel<TYPE, false>, (int)grid, c.threads, 0, s, p);
}

} // namespace

int64_t group_norm_workspace(int64_t N, int64_t S, int64_t C, int64_t groups, int type, bool checkpoint)
{
    if (N * S == 0) return 0;
    const GnCut c = forward_cut(S, C, groups, type, checkpoint);
    return N * groups * (c.P + 1) * (int64_t)sizeof(float2);
}

cudaError_t launch_group_norm(const GnProblem &q, cudaStream_t s)
{
    const GnCut c = forward_cut(q.S, q.C, q.groups, q.type, q.codes != nullptr);
    GnParams p = {};
    p.x = static_cast<const char *>(q.x);
    p.y = static_cast<char *>(q.y);
    p.part = static_cast<float2 *>(q.workspace);
    p.stats = q.stats ? static_cast<float2 *>(q.stats) : p.part + q.N * q.groups * c.P;
    p.codes = static_cast<uint2 *>(q.codes);
    p.block_scales = static_cast<uint8_t *>(q.block_scales);
    p.gains = Gains{q.weight, q.bias, q.scale, q.shift, q.param_type, q.type, q.vs};
    p.S = q.S;
    p.R = c.R;
    p.P = c.P;
    p.F = c.F;
    p.Ft = c.Ft;
    p.tiles = c.tiles;
    p.RL = c.RL;
    p.per = (int)(q.C / q.groups);
    p.groups = (int)q.groups;
    p.unit = (int)gcd64(p.per, 8);
    p.act = q.act;
    p.eps = q.eps;
    return q.type == kBf16   ? launch_type<kBf16>(p, q, c, s)
           : q.type == kFp16 ? launch_type<kFp16>(p, q, c, s)
                             : launch_type<kFp32>(p, q, c, s);
}

} // namespace dan
