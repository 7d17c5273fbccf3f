// dan_gn_back.cu -- gradients of the group norm of channels-last images, for
// sm_103a (include/dan_train.h).
//
// With the forward pass's mean and rstd at hand, everything that dx needs of
// the rest of its group, and all the parameters' gradients, follow from two
// sums per image and channel, s0 = sum dz and s1 = sum dz * n.  Where a cluster of
// CTAs can hold a slab of whole groups of dy and x in shared memory, one launch
// reads both once.  Else: a kernel that reads dy and x (or its checkpoint) once
// and stores the sums of each chunk of rows; one that joins the chunks, per group;
// and one that reads both again, in the opposite order (the last rows still lie in
// the L2), and writes dx.  For several images one more (for over 256, a few) adds
// their shares of dweight and dbias.
//
// Large images are bound by memory: at [1, 512 x 512, 256] bf16 the sums take 45 us
// (268 MB read from DRAM, 6.0 TB/s), dx 58 (403 MB asked for and stored, 7.0 TB/s;
// of them 356 in DRAM, 6.2 TB/s, the last stores still lying in the L2); both by ncu's
// clock, cold.  Batches of images of some MB are bound by their instructions
// ([16, 64 x 64, 320] from checkpoints: 25 and 20 us, half the issue slots).
//
// In the loops n = (x - mean) * rstd appears as t = x - mean, with rstd in the
// factors of a channel: z = t * (a * rstd) + b, s1 = rstd * sum dz * t.
#include "dan_gn.cuh"

namespace dan {
namespace {

struct GnBackParams {
    GnGrid g;
    const char *dy, *x;
    const char *codes;
    const uint8_t *block_scales;
    const float2 *stats;
    char *dx;
    float2 *part; // [N][P][C] (s0, s1) of a chunk
    float2 *sums; // [N][C]    (s0, s1)
    float2 *mean; // [N][groups] means of a * dz and a * dz * n
    void *dweight, *dbias, *dscale, *dshift;
    Gains gains;
    int64_t gs;
    int act;
    bool last;     // the call's only image
    float count;   // values of a group
    int chunks;    // of a CTA of the first kernel
    float keep;    // share of a chunk's rows that the L2 is to hold
    int log_cs, M; // slabs: CTAs of a cluster, rows of a thread at most
    int log_join;  // slabs: log2 of the lanes that add up a group's channels together
};

// A thread's P pairs of channels.  UNI: they lie in one group.
template <int P, bool UNI>
struct Channels {
    static constexpr int K = UNI ? 1 : P;
    float2 minus[K], a[P], b[P]; // minus the mean, the gain times rstd, the offset
    // stats: of the groups from the tile's channel 0 on; c: the thread's first channel of it
    template <int TYPE>
    __device__ __forceinline__ void get(const GnBackParams &p, int64_t n, int f, const float2 *stats, int c)
    {
        GroupOf group(p.g, c);
        p.gains.get<TYPE>(n, f, a, b);
        float2 rstd[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float2 s = stats[group.next()];
            const float2 t = UNI ? s : stats[group.next()];
            minus[k] = make_float2(-s.x, -t.x);
            rstd[k] = make_float2(s.y, t.y);
        }
#pragma unroll
        for (int w = 0; w < P; ++w) a[w] = mul2(a[w], rstd[w % K]);
    }
    // rstd alone (it would only take registers in the loops).
    __device__ __forceinline__ static void rstds(const GnGrid &q, const float2 *stats, int c, float2 (&rstd)[K])
    {
        GroupOf group(q, c);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            rstd[k].x = stats[group.next()].y;
            rstd[k].y = UNI ? rstd[k].x : stats[group.next()].y;
        }
    }
    // dz of dy.
    __device__ __forceinline__ float2 dz(int w, int act, float2 t, float2 dy) const
    {
        if (!act) return dy;
        const float2 z = fma2(t, a[w], b[w]);
        const float2 p = sigmoid2(z);
        // the derivative, p * (1 + z * (1 - p))
        return mul2(dy, fma2(mul2(z, p), sub2(dup2(1.0f), p), p));
    }
    // Minus the means of a * dz (times rstd) and of a * dz * n (times rstd^2).
    __device__ __forceinline__ static void means(const GnGrid &q, const float2 *means, const float2 *stats, int c,
                                                 float2 (&m1)[K], float2 (&m2)[K])
    {
        float2 rstd[K];
        rstds(q, stats, c, rstd);
        GroupOf group(q, c);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float2 u = means[group.next()];
            const float2 v = UNI ? u : means[group.next()];
            m1[k] = mul2(make_float2(-u.x, -v.x), rstd[k]);
            m2[k] = mul2(mul2(make_float2(-u.y, -v.y), rstd[k]), rstd[k]);
        }
    }
    // dx of pair w.
    __device__ __forceinline__ float2 dx(int w, float2 t, float2 dz, const float2 (&m1)[K], const float2 (&m2)[K]) const
    {
        return fma2(t, m2[w % K], fma2(dz, a[w], m1[w % K]));
    }
};

// Rows of dy and x (or its checkpoint) in flight of a thread, through shared
// memory that it alone uses: as many as 48 KB of 256 threads hold.  Their number A
// and the CTA's threads are known to the compiler, so that a row's slots and what
// is left are constants of an unrolled round of A rows.
template <int TYPE, bool CKPT, bool UNI, int NT>
struct Ring {
    using Frag = Fragment<TYPE>;
    using XWord = typename std::conditional<CKPT, typename Frag::Codes, uint4>::type;
    static constexpr int kBytes = 16 + (int)sizeof(XWord);
    static constexpr int A = 48 * 1024 / 256 / kBytes;
    const char *dy, *x;   // this thread's first row of the round
    const uint8_t *scale; // and its block's scale
    int step;             // fragments from a row to the next
    int left;             // rows from the round's first on
    int keep;             // of them the last ones that the L2 is to hold (others are to go first)
    uint64_t first, normal;
    uint4 *s_dy;          // [A][NT]
    XWord *s_x;           // [A][NT]
    unsigned scales[A];   // of the rows in flight

    // `rows` rows from fragment `at` on, `step` fragments apart.
    __device__ __forceinline__ Ring(const GnBackParams &p, uint4 *smem, int64_t at, int step_, int rows, int keep_)
    {
        keep = keep_;
        first = evict_first();
        normal = evict_normal();
        s_dy = smem + threadIdx.x;
        s_x = reinterpret_cast<XWord *>(smem + A * NT) + threadIdx.x;
        step = step_;
        left = rows;
        dy = p.dy + at * 16;
        x = (CKPT ? p.codes : p.x) + at * (int64_t)sizeof(XWord);
        scale = p.block_scales + at / Frag::kBlock;
#pragma unroll
        for (int j = 0; j < A; ++j) {
            scales[j] = 127;
            ask(j, j);
        }
    }
    // Row `ahead` of the round into slot j.
    __device__ __forceinline__ void ask(int j, int ahead)
    {
        if (left > ahead) {
            const uint64_t policy = left - ahead > keep ? first : normal;
            cp_async16(s_dy + j * NT, dy + ahead * (int64_t)(step * 16), policy);
            if constexpr (CKPT) cp_async_word(s_x + j * NT, x + ahead * (int64_t)(step * (int)sizeof(XWord)));
            else cp_async16(s_x + j * NT, x + ahead * (int64_t)(step * 16), policy);
            // (a row's fragments, and so the step, are whole blocks)
            if (CKPT) scales[j] = __ldg(scale + ahead * (int64_t)(step / Frag::kBlock));
        }
        cp_async_commit();
    }
    // Row j of the round, x - mean and dy; the slot is filled again.
    __device__ __forceinline__ void take(int j, const Channels<Frag::kP, UNI> &ch, float2 (&t)[Frag::kP], float2 (&d)[Frag::kP])
    {
        cp_async_wait<A - 1>();
        const uint4 a = s_dy[j * NT];
        const XWord c = s_x[j * NT];
        if constexpr (CKPT) {
            const float2 s = dup2(block_scale_value(scales[j]));
            Frag::codes(c, t);
#pragma unroll
            for (int w = 0; w < Frag::kP; ++w) t[w] = fma2(t[w], s, ch.minus[w % ch.K]);
        } else {
            Frag::values(c, t);
#pragma unroll
            for (int w = 0; w < Frag::kP; ++w) t[w] = add2(t[w], ch.minus[w % ch.K]);
        }
        ask(j, j + A);
        Frag::values(a, d);
    }
    // On to the next round.
    __device__ __forceinline__ void round()
    {
        dy += A * (int64_t)(step * 16);
        x += A * (int64_t)(step * (int)sizeof(XWord));
        scale += A * (int64_t)(step / Frag::kBlock);
        left -= A;
    }
};

// CTAs of 256 threads that share an SM (three, of 80 registers, spill and took
// 128 us for the gradient of [1, 512 x 512, 256] images against 109).
constexpr int kBackBlocks = 2;
// Buffers for the sums of a chunk (the widest tiles leave room for one).
__host__ __device__ constexpr int halves_of(int threads) { return threads <= 256 ? 2 : 1; }

template <int TYPE, bool CKPT, bool UNI, int NT>
__global__ void __launch_bounds__(NT, NT > 256 ? 1 : kBackBlocks) gn_sums_kernel(const GnBackParams p)
{
    using Frag = Fragment<TYPE>;
    using R = Ring<TYPE, CKPT, UNI, NT>;
    constexpr int P = Frag::kP, kHalves = halves_of(NT);
    extern __shared__ __align__(16) uint4 s_ring[];
    float2 *s_sums = reinterpret_cast<float2 *>(s_ring + R::A * R::kBytes * NT / 16); // [kHalves][RL][channels]
    const int64_t n = blockIdx.x;
    const int chunk0 = blockIdx.y * p.chunks;
    const GnPlace at(p.g, blockIdx.z, chunk0, p.chunks);
    grid_dependency_wait();
    allow_dependents();
    R ring(p, s_ring, at.first(p.g, n), p.g.RL * p.g.F, at.mine, (int)((float)at.mine * p.keep));
    Channels<P, UNI> ch = {};
    const float2 *stats = p.stats + n * p.g.groups + at.g0;
    if (at.mine > 0) ch.template get<TYPE>(p, n, at.f0 + at.f, stats, at.f * Frag::kE);
    const int channels = at.Ft * Frag::kE;
    for (int c = 0; at.rows > c * p.g.R; ++c) {
        float2 s0[P], s1[P];
#pragma unroll
        for (int w = 0; w < P; ++w) s0[w] = s1[w] = make_float2(0.0f, 0.0f);
        for (int rows = at.part(p.g, c).mine; rows > 0; rows -= R::A, ring.round()) {
#pragma unroll
            for (int j = 0; j < R::A; ++j) {
                if (rows <= j) break;
                float2 t[P], d[P];
                ring.take(j, ch, t, d);
#pragma unroll
                for (int w = 0; w < P; ++w) {
                    const float2 dz = ch.dz(w, p.act, t[w], d[w]);
                    s0[w] = add2(s0[w], dz);
                    s1[w] = fma2(dz, t[w], s1[w]);
                }
            }
        }
        float2 *sums = s_sums + c % kHalves * p.g.RL * channels;
        if (at.r < p.g.RL && at.f < at.Ft) {
            float4 *to = reinterpret_cast<float4 *>(sums + at.r * channels + at.f * Frag::kE);
            float2 rstd[ch.K];
            ch.rstds(p.g, stats, at.f * Frag::kE, rstd);
#pragma unroll
            for (int w = 0; w < P; ++w) {
                s1[w] = mul2(s1[w], rstd[w % ch.K]);
                to[w] = make_float4(s0[w].x, s1[w].x, s0[w].y, s1[w].y);
            }
        }
        __syncthreads(); // (with two halves, the other one may still be read)
        float2 *to = p.part + (n * p.g.P + chunk0 + c) * ((int64_t)p.g.F * Frag::kE) + at.f0 * Frag::kE;
        for (int k = threadIdx.x; k < channels; k += NT) {
            float2 t = sums[k];
            for (int r = 1; r < p.g.RL; ++r) t = add2(t, sums[r * channels + k]);
            to[k] = t;
        }
        if (kHalves == 1) __syncthreads();
    }
    cp_async_wait_all();
}

// What follows from an image's sums t = (s0, s1) of channel c with the gains g.
template <int TYPE>
__device__ __forceinline__ void store_sums(const GnBackParams &p, int64_t n, int64_t c, const Gains::One &g, float2 t)
{
    if (p.dscale) {
        store_as(p.dscale, TYPE, n * p.gs + c, __fmaf_rn(g.w, t.y, __fmul_rn(g.b, t.x)));
        store_as(p.dshift, TYPE, n * p.gs + c, t.x);
    }
    if (!p.dweight) return;
    if (p.last) {
        store_as(p.dweight, p.gains.param_type, c, __fmul_rn(g.o, t.y));
        store_as(p.dbias, p.gains.param_type, c, __fmul_rn(g.o, t.x));
    } else {
        p.sums[n * ((int64_t)p.g.F * Fragment<TYPE>::kE) + c] = t;
    }
}

// Joins the chunks of a group's channels; then what follows from the sums.
constexpr int kJoin = 256;
template <int TYPE>
__global__ void __launch_bounds__(kJoin) gn_back_join_kernel(const GnBackParams p)
{
    __shared__ float2 s_part[kJoin];
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t n = blockIdx.x / (unsigned)p.g.groups;
    const int g = blockIdx.x - (unsigned)n * p.g.groups;
    const int64_t C = (int64_t)p.g.F * Fragment<TYPE>::kE;
    const int cols = min(p.g.per, kJoin), shares = kJoin / cols;
    const int share = tid / cols, col = tid - share * cols;
    float2 all = make_float2(0.0f, 0.0f); // sums of a * s0 and a * s1 over this thread's channels
    for (int j0 = 0; j0 < p.g.per; j0 += cols) {
        const int64_t c = g * (int64_t)p.g.per + j0 + col;
        const bool here = share < shares && j0 + col < p.g.per;
        float2 t = make_float2(0.0f, 0.0f);
        Gains::One gain = {};
        if (here && share == 0) gain = p.gains.one<TYPE>(n, c); // (an input: complete before the sums began)
        if (j0 == 0) {
            grid_dependency_wait();
            allow_dependents();
        }
        if (here) {
            const float2 *from = p.part + n * p.g.P * C + c;
            constexpr int U = 16; // loads under way at once
            for (int k = share; k < p.g.P; k += U * shares) {
                float2 u[U];
#pragma unroll
                for (int j = 0; j < U; ++j)
                    u[j] = k + j * shares < p.g.P ? __ldcg(from + (k + j * shares) * C) : make_float2(0.0f, 0.0f);
#pragma unroll
                for (int j = 0; j < U; ++j) t = add2(t, u[j]);
            }
        }
        s_part[tid] = t;
        __syncthreads();
        if (here && share == 0) {
            for (int k = 1; k < shares; ++k) t = add2(t, s_part[k * cols + col]);
            all = fma2(dup2(gain.gain()), t, all);
            store_sums<TYPE>(p, n, c, gain, t);
        }
        __syncthreads();
    }
    // the group's means
    all.x = lane_sum(all.x, 32);
    all.y = lane_sum(all.y, 32);
    if (lane == 0) s_part[tid >> 5] = all;
    __syncthreads();
    if (tid != 0) return;
    for (int k = 1; k < kJoin / 32; ++k) all = add2(all, s_part[k]);
    p.mean[n * p.g.groups + g] = make_float2(__fdiv_rn(all.x, p.count), __fdiv_rn(all.y, p.count));
}

template <int TYPE, bool CKPT, bool UNI, int NT>
__global__ void __launch_bounds__(NT, NT > 256 ? 1 : kBackBlocks) gn_dx_kernel(const GnBackParams p)
{
    using Frag = Fragment<TYPE>;
    using R = Ring<TYPE, CKPT, UNI, NT>;
    constexpr int P = Frag::kP;
    extern __shared__ __align__(16) uint4 s_ring[];
    // the last chunk first, and of it the last rows
    const int64_t n = gridDim.x - 1 - blockIdx.x;
    const GnPlace at(p.g, gridDim.z - 1 - blockIdx.z, gridDim.y - 1 - blockIdx.y);
    const int step = -p.g.RL * p.g.F;
    const int64_t to = at.first(p.g, n) - (at.mine - 1) * (int64_t)step;
    char *dx = p.dx + to * 16;
    // dy, x, the statistics and the gains were complete before the kernel whose
    // results are waited for below let this one start
    R ring(p, s_ring, to, step, at.mine, 0); // (read for the last time)
    Channels<P, UNI> ch = {};
    if (at.mine > 0) ch.template get<TYPE>(p, n, at.f0 + at.f, p.stats + n * p.g.groups + at.g0, at.f * Frag::kE);
    grid_dependency_wait();
    allow_dependents();
    if (at.mine == 0) return;
    float2 m1[ch.K], m2[ch.K];
    ch.means(p.g, p.mean + n * p.g.groups + at.g0, p.stats + n * p.g.groups + at.g0, at.f * Frag::kE, m1, m2);
    for (; ring.left > 0; ring.round(), dx += R::A * (int64_t)(step * 16)) {
#pragma unroll
        for (int j = 0; j < R::A; ++j) {
            if (ring.left <= j) break;
            float2 t[P], d[P];
            ring.take(j, ch, t, d);
#pragma unroll
            for (int w = 0; w < P; ++w) d[w] = ch.dx(w, t[w], ch.dz(w, p.act, t[w], d[w]), m1, m2);
            Frag::store(dx + j * (int64_t)(step * 16), d, ring.first);
        }
    }
}

// dweight and dbias from the images' sums, in order; eight threads a channel add
// up to 256 of them.  Of more images each 256's sum takes the place of its first
// image's, and a further launch adds those (of the gradient of
// [65536, 1, 64], 0.29 ms, a chain of N / 8 loads instead was 2.8 ms more).  FIRST: the sums are the images', still
// without their factor 1 + scale.  `step`: images from an entry to the next.
constexpr int64_t kParamImages = 256;
template <int TYPE, bool FIRST>
__global__ void __launch_bounds__(256) gn_params_kernel(const GnBackParams p, int64_t entries, int64_t step)
{
    __shared__ float2 s_sum[8][32];
    const int share = threadIdx.x >> 5;
    const int64_t C = (int64_t)p.g.F * Fragment<TYPE>::kE, c = blockIdx.y * (int64_t)32 + (threadIdx.x & 31);
    const int64_t from = blockIdx.x * kParamImages, end = min(entries, from + kParamImages);
    grid_dependency_wait();
    allow_dependents();
    float2 t = make_float2(0.0f, 0.0f);
    if (c < C)
#pragma unroll 4
        for (int64_t i = from + share; i < end; i += 8) {
            const int64_t n = FIRST ? i : i * step;
            const float2 u = __ldcg(p.sums + n * C + c);
            if (FIRST) {
                const float s = p.gains.scale ? Gains::value<TYPE>(p.gains.scale, n * p.gains.vs + c) : 0.0f;
                t = fma2(dup2(__fadd_rn(1.0f, s)), u, t);
            } else {
                t = add2(t, u);
            }
        }
    s_sum[share][threadIdx.x & 31] = t;
    __syncthreads(); // (this part's entries are read)
    if (share != 0 || c >= C) return;
    for (int k = 1; k < 8; ++k) t = add2(t, s_sum[k][threadIdx.x]);
    if (entries > kParamImages) {
        p.sums[from * step * C + c] = t;
    } else {
        store_as(p.dweight, p.gains.param_type, c, t.y);
        store_as(p.dbias, p.gains.param_type, c, t.x);
    }
}

template <int TYPE>
cudaError_t ready_params(int64_t N)
{
    const cudaError_t e = ready(gn_params_kernel<TYPE, true>, 0);
    return e != cudaSuccess || N <= kParamImages ? e : ready(gn_params_kernel<TYPE, false>, 0);
}
template <int TYPE>
cudaError_t launch_params(const GnBackParams &p, int64_t N, int64_t C, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    for (int64_t entries = N, step = 1, parts; e == cudaSuccess && entries > 0; entries = parts > 1 ? parts : 0, step *= kParamImages) {
        parts = (entries + kParamImages - 1) / kParamImages;
        const dim3 grid((unsigned)parts, (unsigned)((C + 31) / 32));
        e = step == 1 ? launch_grid(gn_params_kernel<TYPE, true>, grid, 1, 256, 0, s, p, entries, step)
                      : launch_grid(gn_params_kernel<TYPE, false>, grid, 1, 256, 0, s, p, entries, step);
    }
    return e;
}

// The parameters' gradients of images without positions, or of no images: zeros,
// whatever the parameters are (they are not read).
__global__ void __launch_bounds__(256) gn_zeros_kernel(const GnBackParams p, int type, int64_t N, int64_t C)
{
    grid_dependency_wait();
    allow_dependents();
    const int64_t most = (N > 0 ? N : 1) * C;
    for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < most; i += gridDim.x * (int64_t)256) {
        const int64_t n = i / C, c = i - n * C;
        if (p.dscale && n < N) {
            store_as(p.dscale, type, n * p.gs + c, 0.0f);
            store_as(p.dshift, type, n * p.gs + c, 0.0f);
        }
        if (p.dweight && i < C) {
            store_as(p.dweight, p.gains.param_type, i, 0.0f);
            store_as(p.dbias, p.gains.param_type, i, 0.0f);
        }
    }
}

// ------------------------------------------------------------------- slabs

// One launch, one read of dy and x: a cluster holds a slab (whole groups of an
// image) of both in its CTAs' shared memory.  Each thread copies its own
// fragments there and nobody else reads them; the channels' sums are joined in
// the CTA, then over the cluster, each CTA for itself in the same order.  From x, one
// image and 16, in us: [8 x 8, 1280] 5.3 and 7.7 (passes 8.6 and 12.0), [16 x 16, 1280]
// 7.0 and 18.7 (8.9 and 19.2), [32 x 32, 640] 7.6 and 38 (9.6 and 25: many large slabs
// lose, of 13 to 16 warps an SM, and which form it is may not follow the batch).
// Bound by the chain of latencies, of many images by their instructions.
template <int TYPE, bool CKPT, bool UNI>
__global__ void __launch_bounds__(512, 1) gn_back_slab_kernel(const GnBackParams p)
{
    using Frag = Fragment<TYPE>;
    constexpr int P = Frag::kP, E = Frag::kE;
    using XWord = typename std::conditional<CKPT, typename Frag::Codes, uint4>::type;
    extern __shared__ __align__(16) uint4 s_dy[]; // [M][threads]
    const int tid = threadIdx.x, lane = tid & 31, NT = blockDim.x, cs = 1 << p.log_cs;
    float2 *s_sums = reinterpret_cast<float2 *>(s_dy + p.M * NT); // [RL][channels]
    XWord *s_x = reinterpret_cast<XWord *>(s_sums + NT * E);      // [M][threads]
    float2 *s_ch = reinterpret_cast<float2 *>(s_x + p.M * NT);    // [channels] this CTA's sums
    float2 *s_all = s_ch + E * p.g.Ft;                            // [channels] the slab's, times the gain
    float2 *s_mean = s_all + E * p.g.Ft;                          // [groups]
    uint8_t *s_scale = reinterpret_cast<uint8_t *>(s_mean + E * p.g.Ft); // [M][threads] (CKPT)

    const int rank = blockIdx.x & (cs - 1); // (clusters lie along x)
    const int64_t n = blockIdx.x >> p.log_cs;
    const GnPlace at(p.g, blockIdx.y, rank);
    const int64_t base = at.first(p.g, n), step = (int64_t)p.g.RL * p.g.F;

    grid_dependency_wait();
    allow_dependents();
    constexpr int kParts = 4; // the rows arrive in parts, the first is summed while the others are under way
    const int part = (p.M + kParts - 1) / kParts;
    {
        const char *dy = p.dy + base * 16, *x = (CKPT ? p.codes : p.x) + base * (int64_t)sizeof(XWord);
        int i = 0;
#pragma unroll
        for (int k = 1; k <= kParts; ++k) {
            for (const int end = min(at.mine, k * part); i < end; ++i) {
                cp_async16(s_dy + i * NT + tid, dy);
                cp_async_word(s_x + i * NT + tid, x);
                dy += step * 16;
                x += step * (int64_t)sizeof(XWord);
            }
            cp_async_commit();
        }
    }
    if (CKPT) {
        const uint8_t *scale = p.block_scales + base / Frag::kBlock;
#pragma unroll 4
        for (int i = 0; i < at.mine; ++i) s_scale[i * NT + tid] = __ldg(scale + i * (step / Frag::kBlock));
    }
    const int channels = at.Ft * E, c0 = at.f0 * E;
    Channels<P, UNI> ch = {};
    if (at.mine > 0) ch.template get<TYPE>(p, n, at.f0 + at.f, p.stats + n * p.g.groups + at.g0, at.f * E);
    Gains::One gain = {}; // of this thread's channel of the slab (the first, where it has several)
    if (tid < channels) gain = p.gains.one<TYPE>(n, c0 + tid);
    auto get = [&](int i, float2 (&t)[P], float2 (&d)[P]) {
        Frag::values(s_dy[i * NT + tid], d);
        if constexpr (CKPT) {
            const float2 s = dup2(block_scale_value(s_scale[i * NT + tid]));
            Frag::codes(s_x[i * NT + tid], t);
#pragma unroll
            for (int w = 0; w < P; ++w) t[w] = fma2(t[w], s, ch.minus[w % ch.K]);
        } else {
            Frag::values(s_x[i * NT + tid], t);
#pragma unroll
            for (int w = 0; w < P; ++w) t[w] = add2(t[w], ch.minus[w % ch.K]);
        }
    };
    float2 s0[P], s1[P];
#pragma unroll
    for (int w = 0; w < P; ++w) s0[w] = s1[w] = make_float2(0.0f, 0.0f);
    int i = 0;
#pragma unroll
    for (int k = 1; k <= kParts; ++k) {
        if (k == 1) cp_async_wait<3>();
        if (k == 2) cp_async_wait<2>();
        if (k == 3) cp_async_wait<1>();
        if (k == 4) cp_async_wait<0>();
        for (const int end = min(at.mine, k * part); i < end; ++i) {
            float2 t[P], d[P];
            get(i, t, d);
#pragma unroll
            for (int w = 0; w < P; ++w) {
                const float2 dz = ch.dz(w, p.act, t[w], d[w]);
                s0[w] = add2(s0[w], dz);
                s1[w] = fma2(dz, t[w], s1[w]);
            }
        }
    }
    // the CTA's sums: of every `shares`-th row lane, then those
    if (at.r < p.g.RL && at.f < at.Ft) {
        float4 *to = reinterpret_cast<float4 *>(s_sums + at.r * channels + at.f * E);
        float2 rstd[ch.K];
        ch.rstds(p.g, p.stats + n * p.g.groups + at.g0, at.f * E, rstd);
#pragma unroll
        for (int w = 0; w < P; ++w) {
            s1[w] = mul2(s1[w], rstd[w % ch.K]);
            to[w] = make_float4(s0[w].x, s1[w].x, s0[w].y, s1[w].y);
        }
    }
    __syncthreads();
    const int shares = min(p.g.RL, max(1, NT / channels));
    for (int c = tid; c < channels * shares; c += NT) {
        const int share = c / channels;
        float2 t = make_float2(0.0f, 0.0f);
        for (int k = share; k < p.g.RL; k += shares) t = add2(t, s_sums[k * channels + c - share * channels]);
        s_sums[c] = t; // (an entry that nobody else reads)
    }
    __syncthreads();
    for (int c = tid; c < channels; c += NT) {
        float2 t = s_sums[c];
        for (int k = 1; k < shares; ++k) t = add2(t, s_sums[k * channels + c]);
        s_ch[c] = t;
    }
    if (cs > 1) {
        cluster_arrive();
        cluster_wait();
    } // else each thread goes on with the channels that it has just summed
    for (int c = tid; c < channels; c += NT) {
        float2 t = s_ch[c];
        if (cs > 1) {
            t = make_float2(0.0f, 0.0f);
            for (int k = 0; k < cs; ++k) t = add2(t, ld_cluster(s_ch + c, k));
        }
        if (c != tid) gain = p.gains.one<TYPE>(n, c0 + c);
        s_all[c] = mul2(dup2(gain.gain()), t);
        if (rank == 0) store_sums<TYPE>(p, n, c0 + c, gain, t);
    }
    if (cs > 1) cluster_arrive(); // nobody reads this CTA's sums after the wait below
    __syncthreads();
    // a group's means, by a warp or, of up to 16 channels, by 2^log_join lanes (with a
    // warp each, groups of one channel took most of a CTA's time: the gradient of
    // [1, 8 x 8, 64] in 64 groups 16.1 us, so 6.3)
    auto finish = [&](int g, float2 t) { s_mean[g] = make_float2(__fdiv_rn(t.x, p.count), __fdiv_rn(t.y, p.count)); };
    if (p.log_join == 5) {
        for (int g = tid >> 5; g < at.groups; g += NT >> 5) {
            float2 t = make_float2(0.0f, 0.0f);
            for (int c = lane; c < p.g.per; c += 32) t = add2(t, s_all[g * p.g.per + c]);
            t.x = lane_sum(t.x, 32);
            t.y = lane_sum(t.y, 32);
            if (lane == 0) finish(g, t);
        }
    } else {
        const int lanes = 1 << p.log_join, c = lane & (lanes - 1);
        for (int g0 = tid - lane; g0 < at.groups << p.log_join; g0 += NT) {
            const int g = (g0 + lane) >> p.log_join;
            const bool here = g < at.groups && c < p.g.per;
            float2 t = here ? s_all[g * p.g.per + c] : make_float2(0.0f, 0.0f);
            t.x = lane_sum(t.x, lanes);
            t.y = lane_sum(t.y, lanes);
            if (here && c == 0) finish(g, t);
        }
    }
    __syncthreads();
    if (at.mine > 0) {
        float2 m1[ch.K], m2[ch.K];
        ch.means(p.g, s_mean, p.stats + n * p.g.groups + at.g0, at.f * E, m1, m2);
        char *dx = p.dx + base * 16;
        for (int k = 0; k < at.mine; ++k, dx += step * 16) {
            float2 t[P], d[P];
            get(k, t, d);
#pragma unroll
            for (int w = 0; w < P; ++w) d[w] = ch.dx(w, t[w], ch.dz(w, p.act, t[w], d[w]), m1, m2);
            Frag::store(dx, d);
        }
    }
    if (cs > 1) cluster_wait();
}

GnSlab backward_slab(int64_t S, int64_t C, int64_t groups, int type, bool checkpoint)
{
    const int E = (int)type_channels(type);
    // (a slab need not hold whole blocks: their scales are read only)
    // (wider ones where there are few rows gained in many images, [16384, 1, 1024] 0.88 ->
    // 0.42 ms, but lost in one, 3.8 -> 10.8 us: a thread's channels go one by one)
    return gn_slab(S, C, groups, type, false, checkpoint ? 16 + E + 1 : 32, E * (int)sizeof(float2), 0);
}

// Rows of a thread's ring (Ring::A).
constexpr int ring_rows(int type, bool ckpt) { return 48 * 1024 / 256 / (16 + (ckpt ? (type == kFp32 ? 4 : 8) : 16)); }

GnCut backward_cut(int64_t S, int64_t C, int64_t groups, int type, bool checkpoint)
{
    return gn_cut(S, C, groups, type, false, ring_rows(type, checkpoint), 2, 304);
}

template <int TYPE, bool CKPT, bool UNI>
cudaError_t launch_slab(GnBackParams p, const GnProblem &q, const GnSlab &c, cudaStream_t s)
{
    p.g = gn_grid(q.S, q.C, q.groups, TYPE, c.Ft, c.R, 1 << c.log_cs, c.RL);
    p.log_cs = c.log_cs;
    p.M = c.M;
    while (p.log_join < 5 && (1 << p.log_join) < p.g.per) ++p.log_join;
    p.sums = static_cast<float2 *>(q.workspace);
    const cudaError_t e = ready(gn_back_slab_kernel<TYPE, CKPT, UNI>, c.smem);
    if (e != cudaSuccess) return e;
    return launch_grid(gn_back_slab_kernel<TYPE, CKPT, UNI>, dim3((unsigned)(q.N << c.log_cs), c.slabs), 1 << c.log_cs,
                       c.threads, c.smem, s, p);
}

// The workspace of the passes: the chunks' sums, the images', the means.
void set_passes(GnBackParams &p, const GnProblem &q, const GnCut &c)
{
    p.g = gn_grid(q.S, q.C, q.groups, q.type, c.Ft, c.R, c.P, c.RL);
    p.part = static_cast<float2 *>(q.workspace);
    p.sums = p.part + q.N * c.P * q.C;
    p.mean = p.sums + q.N * q.C;
}

template <int TYPE, bool CKPT, bool UNI>
cudaError_t launch_passes(GnBackParams p, const GnProblem &q, const GnCut &c, cudaStream_t s)
{
    using R = Ring<TYPE, CKPT, UNI, 256>;
    static_assert(R::A == ring_rows(TYPE, CKPT), "chunks are whole rounds");
    const int ring = R::A * R::kBytes * c.threads, sums = halves_of(c.threads) * c.RL * c.Ft * Fragment<TYPE>::kE * (int)sizeof(float2);
    // Of all that the first kernel reads, what the L2 is found to hold for the
    // second: some 64 MB.
    const float all = (float)(q.N * q.S) * (float)q.C * (float)(type_bytes(TYPE) + (CKPT ? 1 : type_bytes(TYPE)));
    p.keep = all > 64e6f ? 64e6f / all : 1.0f;
    const int blocks = c.threads <= 256 ? kBackBlocks : 1;
    const int64_t slots = (int64_t)sm_count() * blocks / c.tiles;
    // the second kernel's rows need not be whole chunks
    const int64_t round = (int64_t)R::A * c.RL, second = gn_share(q.N, slots, (q.S + round - 1) / round);
    GnBackParams a = p;
    a.g.R = (int)((q.S + second - 1) / second);
    p.chunks = c.rounds ? (int)((c.P + gn_share(q.N, slots, c.P) - 1) / gn_share(q.N, slots, c.P)) : 1;
    const dim3 one((unsigned)q.N, (unsigned)((c.P + p.chunks - 1) / p.chunks), c.tiles);
    const dim3 two((unsigned)q.N, (unsigned)((q.S + a.g.R - 1) / a.g.R), c.tiles);
    const dim3 joins((unsigned)(q.N * q.groups));
    const auto go = [&](auto threads) {
        constexpr int NT = decltype(threads)::value;
        const auto first = gn_sums_kernel<TYPE, CKPT, UNI, NT>, last = gn_dx_kernel<TYPE, CKPT, UNI, NT>;
        const int smem1 = room_for(blocks, ring + sums), smem2 = room_for(blocks, ring);
        cudaError_t e = ready(first, smem1);
        if (e == cudaSuccess) e = ready(gn_back_join_kernel<TYPE>, 0);
        if (e == cudaSuccess) e = ready(last, smem2);
        if (e == cudaSuccess) e = launch_grid(first, one, 1, NT, smem1, s, p);
        if (e == cudaSuccess) e = launch_grid(gn_back_join_kernel<TYPE>, joins, 1, kJoin, 0, s, p);
        if (e == cudaSuccess) e = launch_grid(last, two, 1, NT, smem2, s, a);
        return e;
    };
    if (c.threads <= 256) return go(std::integral_constant<int, 256>());
    return go(std::integral_constant<int, gn_threads(TYPE)>());
}

} // namespace

int64_t group_norm_backward_workspace(int64_t N, int64_t S, int64_t C, int64_t groups, int type, bool checkpoint)
{
    if (N * S == 0) return 0;
    if (backward_slab(S, C, groups, type, checkpoint).Ft) // the images' sums, to be added
        return N > 1 ? N * C * (int64_t)sizeof(float2) : 0;
    const GnCut c = backward_cut(S, C, groups, type, checkpoint);
    return N * (C * (c.P + 1) + groups) * (int64_t)sizeof(float2);
}

cudaError_t launch_group_norm_backward(const GnProblem &q, cudaStream_t s)
{
    const bool ckpt = q.x == nullptr;
    const int64_t E = type_channels(q.type), per = q.C / q.groups;
    GnBackParams p = {};
    p.dy = static_cast<const char *>(q.dy);
    p.x = static_cast<const char *>(q.x);
    p.codes = static_cast<const char *>(q.codes);
    p.block_scales = static_cast<const uint8_t *>(q.block_scales);
    p.stats = static_cast<const float2 *>(q.stats);
    p.dx = static_cast<char *>(q.dx);
    p.dweight = q.dweight;
    p.dbias = q.dbias;
    p.dscale = q.dscale;
    p.dshift = q.dshift;
    p.gains = Gains{q.weight, q.bias, q.scale, q.shift, q.param_type, q.vs};
    p.gs = q.gs;
    p.act = q.act;
    p.last = q.N == 1;
    p.count = (float)(q.S * per);
    if (q.N * q.S == 0) {
        if (!q.dweight && (!q.dscale || q.N == 0)) return cudaSuccess;
        const cudaError_t e = ready(gn_zeros_kernel, 0);
        const int64_t blocks = ((q.N > 0 ? q.N : 1) * q.C + 255) / 256, most = 8 * (int64_t)sm_count();
        if (e != cudaSuccess) return e;
        return launch_grid(gn_zeros_kernel, dim3((unsigned)(blocks < most ? blocks : most)), 1, 256, 0, s, p, q.type, q.N, q.C);
    }
    const GnSlab slab = backward_slab(q.S, q.C, q.groups, q.type, ckpt);
    const GnCut cut = backward_cut(q.S, q.C, q.groups, q.type, ckpt);
    set_passes(p, q, cut);
    if (slab.Ft) p.sums = p.part;
    return with_type(q.type, [&](auto type) -> cudaError_t {
        constexpr int T = decltype(type)::value;
        const bool params = !p.last && q.dweight;
        cudaError_t e = params ? ready_params<T>(q.N) : cudaSuccess;
        if (e != cudaSuccess) return e;
        e = with_bool(ckpt, [&](auto codes) {
            return with_bool(per % E == 0, [&](auto uni) {
                constexpr bool K = decltype(codes)::value, U = decltype(uni)::value;
                return slab.Ft ? launch_slab<T, K, U>(p, q, slab, s) : launch_passes<T, K, U>(p, q, cut, s);
            });
        });
        if (e != cudaSuccess || !params) return e;
        return launch_params<T>(p, q.N, q.C, s);
    });
}

} // namespace dan
