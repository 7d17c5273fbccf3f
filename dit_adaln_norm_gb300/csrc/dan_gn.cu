// dan_gn.cu -- group norm of channels-last images with an activation, for
// sm_103a (include/dan_train.h).
//
// A group's mean and variance need all of an image's rows before the first
// output can be written.  Where a cluster of CTAs can hold a slab of whole groups
// in shared memory, one launch reads x once.  Else passes: the moments of each
// chunk of rows (x read once), their join per group (a kernel, or where there are
// few of them a part of the next one), and the normalisation, which reads x again,
// in the opposite order so that what the first kernel read last still lies in the
// L2.  Large images are bound by memory: at [1, 1024 x 1024, 128] bf16 the moments
// take 46 us (5.8 TB/s) and the normalisation 82 (6.5 TB/s); images of some MB by
// their instructions and the launches' latencies.
//
// Moments: a thread sums d and d^2 of its values' differences d from its first
// one, turns them into a mean and a sum of squares about it, and these are joined in
// a fixed order: first the means, then the squares about the joint mean.  Means
// too are summed as differences from the first one of those that are joined.  So
// a level far above the spread costs what a mean's own rounding does, half a step
// of the level at each of up to three joins, and equal values have no spread.
#include "dan_gn.cuh"

namespace dan {
namespace {

struct GnParams {
    GnGrid g;
    const char *x;
    char *y;
    float2 *part;  // [N][groups][P] mean and squared sum of a chunk
    float2 *stats; // [N][groups] mean and rstd
    char *codes;
    uint8_t *block_scales;
    Gains gains;
    int unit;      // channels of a fragment that are sure to lie in one group: gcd(per, its channels)
    int per_frag;  // units of a fragment
    int per_group; // units of a group
    int join;      // lanes that add up a group's entries together: a power of two
    int wide, deep; // of them `wide` units at once of `deep` row lanes
    Divisor by_wide;
    int act;
    float eps;
    float count;   // values of a group
    float keep;    // share of a chunk's rows that the L2 is to hold
    int chunks;    // of a CTA of the first kernel
    bool few;      // so few chunks that each CTA of the second kernel joins them itself
    int chunk_R;   // rows of a chunk (the second kernel's R is its own)
    int log_cs, M; // slabs: CTAs of a cluster, rows of a thread at most
};

// ----------------------------------------------------------------- moments

// A thread's sums of differences from a pivot, for the kP pairs of a fragment.
template <int P>
struct Sums {
    float2 pivot[P], s1[P], s2[P];
    __device__ __forceinline__ void start(const float2 (&v)[P], int unit)
    {
#pragma unroll
        for (int w = 0; w < P; ++w) {
            // the unit's first channel
            const float2 half = dup2(v[w & ~1].x), all = dup2(v[0].x);
            pivot[w] = unit == 1 ? v[w] : unit == 2 ? dup2(v[w].x) : unit == 4 ? half : all;
            s1[w] = s2[w] = make_float2(0.0f, 0.0f);
        }
    }
    __device__ __forceinline__ void add(const float2 (&v)[P])
    {
#pragma unroll
        for (int w = 0; w < P; ++w) {
            const float2 d = sub2(v[w], pivot[w]);
            s1[w] = add2(s1[w], d);
            s2[w] = fma2(d, d, s2[w]);
        }
    }
    // Mean and squared sum of each unit of `unit` channels over `rows` rows, to
    // `to`.
    __device__ __forceinline__ void finish(int unit, int rows, float2 *to) const
    {
        const float inv = __fdividef(1.0f, (float)(rows * unit));
        auto one = [&](float a, float q, float p) {
            const float d = __fmul_rn(a, inv);
            return make_float2(__fadd_rn(p, d), fmaxf(__fmaf_rn(-a, d, q), 0.0f));
        };
        if (unit == 1) {
#pragma unroll
            for (int w = 0; w < P; ++w) {
                to[2 * w] = one(s1[w].x, s2[w].x, pivot[w].x);
                to[2 * w + 1] = one(s1[w].y, s2[w].y, pivot[w].y);
            }
            return;
        }
        float a[P], q[P];
#pragma unroll
        for (int w = 0; w < P; ++w) a[w] = __fadd_rn(s1[w].x, s1[w].y), q[w] = __fadd_rn(s2[w].x, s2[w].y);
        if (unit == 2) {
#pragma unroll
            for (int w = 0; w < P; ++w) to[w] = one(a[w], q[w], pivot[w].x);
            return;
        }
#pragma unroll
        for (int w = 0; w < P; w += 2) a[w] = __fadd_rn(a[w], a[w + 1]), q[w] = __fadd_rn(q[w], q[w + 1]);
        if (unit == 4) {
#pragma unroll
            for (int w = 0; w < P; w += 2) to[w / 2] = one(a[w], q[w], pivot[w].x);
            return;
        }
        to[0] = one(__fadd_rn(a[0], a[P / 2]), __fadd_rn(q[0], q[P / 2]), pivot[0].x);
    }
};

// Mean and squared sum of each of a CTA's groups from its entries (the groups'
// units of every row lane): their mean, from the first one on, then the squared
// sums about it.
__device__ __forceinline__ void join_units(const GnParams &p, const GnPlace &at, const float2 *s_units, float2 *to,
                                           int64_t step)
{
    const int units = at.Ft * p.per_frag, lane = threadIdx.x & 31, mine = lane & (p.join - 1);
    const int at_once = 32 / p.join; // groups of a warp
    const int rl0 = p.by_wide.of(mine), u0 = mine - rl0 * p.wide;
    const int end = rl0 < p.deep ? min(p.g.RL, at.rows) : 0;
    const float inv = __fdividef(1.0f, (float)(at.rows * p.per_group)); // units weigh alike
    for (int g0 = (threadIdx.x >> 5) * at_once; g0 < at.groups; g0 += (blockDim.x >> 5) * at_once) {
        const int g = g0 + lane / p.join;
        const float2 *from = s_units + g * p.per_group;
        const int last = g < at.groups ? end : 0;
        const float pivot = last > 0 ? from->x : 0.0f; // (of a lane that has entries)
        float sum = 0.0f;
        for (int rl = rl0; rl < last; rl += p.deep)
            for (int u = u0; u < p.per_group; u += p.wide)
                sum = __fmaf_rn(__fsub_rn(from[rl * units + u].x, pivot), (float)(at.whole + (rl < at.rest)), sum);
        const float off = __fmul_rn(lane_sum(sum, p.join), inv); // the mean's, from the pivot
        float m2 = 0.0f;
        for (int rl = rl0; rl < last; rl += p.deep)
            for (int u = u0; u < p.per_group; u += p.wide) {
                const float2 t = from[rl * units + u];
                const float d = __fsub_rn(__fsub_rn(t.x, pivot), off);
                m2 = __fadd_rn(m2, __fmaf_rn(__fmul_rn(d, d), (float)((at.whole + (rl < at.rest)) * p.unit), t.y));
            }
        m2 = lane_sum(m2, p.join);
        if (mine == 0 && g < at.groups) to[g * step] = make_float2(__fadd_rn(pivot, off), m2);
    }
}

// Rows in flight of a thread, through shared memory that it alone uses: copied
// there asynchronously, so that they take no registers.
constexpr int kRing = 8;

// (NT threads: their number and kRing's are known to the compiler, so that a row's
// slot and what is left are constants of an unrolled round of rows.)
template <int TYPE, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) gn_moments_kernel(const GnParams p)
{
    using Frag = Fragment<TYPE>;
    extern __shared__ __align__(16) uint4 s_ring[]; // [kRing][NT]
    float2 *s_units = reinterpret_cast<float2 *>(s_ring + kRing * NT); // [2][RL][units of the tile]
    const int chunk0 = blockIdx.y * p.chunks;
    const GnPlace at(p.g, blockIdx.z, chunk0, p.chunks);
    const int64_t n = blockIdx.x;
    const int step = p.g.RL * p.g.F * 16;
    const char *x = p.x + at.first(p.g, n) * 16;
    uint4 *slot = s_ring + threadIdx.x;
    grid_dependency_wait();
    allow_dependents();
    // the last rows are read again first, and are to stay in the L2
    const int keep = (int)((float)at.mine * p.keep);
    const uint64_t first = evict_first(), normal = evict_normal();
    int left = at.mine;
    auto ask = [&](int j, int ahead) {
        if (left > ahead) cp_async16(slot + j * NT, x + ahead * (int64_t)step, left - ahead > keep ? first : normal);
        cp_async_commit();
    };
#pragma unroll
    for (int j = 0; j < kRing; ++j) ask(j, j);
    for (int c = 0; at.rows > c * p.g.R; ++c) {
        const GnPlace part = at.part(p.g, c);
        float2 *units = s_units + (c & 1) * p.g.RL * p.g.Ft * p.per_frag;
        if (part.mine > 0) {
            Sums<Frag::kP> sums;
            float2 v[Frag::kP];
            cp_async_wait<kRing - 1>();
            Frag::values(slot[0], v);
            sums.start(v, p.unit);
            for (int rows = part.mine; rows > 0; rows -= kRing, left -= kRing, x += kRing * (int64_t)step) {
#pragma unroll
                for (int j = 0; j < kRing; ++j) {
                    if (rows <= j) break;
                    cp_async_wait<kRing - 1>();
                    Frag::values(slot[j * NT], v);
                    sums.add(v);
                    ask(j, j + kRing);
                }
            }
            sums.finish(p.unit, part.mine, units + (at.r * at.Ft + at.f) * p.per_frag);
        }
        __syncthreads(); // (the other half of s_units may still be read)
        join_units(p, part, units, p.part + (n * p.g.groups + at.g0) * p.g.P + chunk0 + c, p.g.P);
    }
    cp_async_wait_all();
}

// Mean and rstd of each group (a block's) from its chunks' moments: up to kU
// chunks a thread, in registers.
constexpr int kJoin = 128, kU = 5;
__global__ void __launch_bounds__(kJoin) gn_join_kernel(const GnParams p)
{
    __shared__ float s_warp[2][kJoin / 32];
    const int tid = threadIdx.x;
    const int64_t g = blockIdx.x;
    float n[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
        const int k = tid + j * kJoin;
        n[j] = k >= p.g.P ? 0.0f : (float)((k + 1 < p.g.P ? p.g.R : p.g.S - (int64_t)k * p.g.R) * p.g.per);
    }
    grid_dependency_wait();
    allow_dependents();
    float2 t[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j)
        t[j] = __ldcg(p.part + g * p.g.P + (tid + j * kJoin < p.g.P ? tid + j * kJoin : 0)); // (n is 0 of no chunk)
    const float pivot = __ldcg(p.part + g * p.g.P).x;
    auto block_sum = [&](float v, int at) {
        v = lane_sum(v, 32);
        if ((tid & 31) == 0) s_warp[at][tid >> 5] = v;
        __syncthreads();
        v = s_warp[at][0];
#pragma unroll
        for (int k = 1; k < kJoin / 32; ++k) v = __fadd_rn(v, s_warp[at][k]);
        return v;
    };
    float v = 0.0f;
#pragma unroll
    for (int j = 0; j < kU; ++j) v = __fmaf_rn(__fsub_rn(t[j].x, pivot), n[j], v);
    const float off = __fdiv_rn(block_sum(v, 0), p.count); // the mean's, from the pivot
    v = 0.0f;
#pragma unroll
    for (int j = 0; j < kU; ++j) {
        const float d = __fsub_rn(__fsub_rn(t[j].x, pivot), off);
        v = __fadd_rn(v, __fmaf_rn(__fmul_rn(d, d), n[j], n[j] > 0.0f ? t[j].y : 0.0f));
    }
    v = __fdiv_rn(block_sum(v, 1), p.count);
    if (tid == 0) p.stats[g] = make_float2(__fadd_rn(pivot, off), defined_rsqrt(__fadd_rn(v, p.eps)));
}

// --------------------------------------------------------------- normalise

// What a thread needs of its P pairs of channels: z = (x - mean) * a + b.  UNI:
// they lie in one group.
template <int P, bool UNI>
struct Norm {
    static constexpr int K = UNI ? 1 : P;
    float2 mean[K], a[P], b[P];
    // With a and b the gains: the moments of the channels' groups, stats those from
    // the tile's channel 0 on, c the thread's first channel of the tile.
    __device__ __forceinline__ void moments(const GnGrid &q, const float2 *stats, int c)
    {
        GroupOf group(q, c);
        if (UNI) {
            const float2 st = stats[group.next()];
            mean[0] = dup2(st.x);
#pragma unroll
            for (int w = 0; w < P; ++w) a[w] = mul2(a[w], dup2(st.y));
        } else {
#pragma unroll
            for (int w = 0; w < P; ++w) {
                const float2 s = stats[group.next()], t = stats[group.next()];
                mean[w % K] = make_float2(s.x, t.x);
                a[w] = mul2(a[w], make_float2(s.y, t.y));
            }
        }
    }
    __device__ __forceinline__ void apply(const float2 (&v)[P], int act, float2 (&z)[P]) const
    {
#pragma unroll
        for (int w = 0; w < P; ++w) {
            z[w] = fma2(sub2(v[w], mean[w % K]), a[w], b[w]);
            if (act) z[w] = mul2(z[w], sigmoid2(z[w]));
        }
    }
};

// The checkpoint of fragment `at`: neighbouring lanes have a block of 32 channels
// (tiles start at a block, and a block's lanes are all here or none).  All lanes
// of a warp call this.
template <int TYPE>
__device__ __forceinline__ void store_codes(const GnParams &p, int64_t at, const float2 (&v)[Fragment<TYPE>::kP], bool here)
{
    using Frag = Fragment<TYPE>;
    float top = 0.0f; // (a NaN counts as nothing)
#pragma unroll
    for (int w = 0; w < Frag::kP; ++w) top = fmaxf(top, fmaxf(fabsf(v[w].x), fabsf(v[w].y)));
    if (!here) top = 0.0f;
#pragma unroll
    for (int off = 1; off < Frag::kBlock; off *= 2) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
    if (!here) return;
    const unsigned code = block_scale_code(top);
    const float2 inv = dup2(block_scale_inverse(code));
    uint32_t c[Frag::kP];
#pragma unroll
    for (int w = 0; w < Frag::kP; ++w) c[w] = fp8x2_e4m3(mul2(v[w], inv));
    if constexpr (TYPE == kFp32) {
        reinterpret_cast<uint32_t *>(p.codes)[at] = c[0] | (c[1] << 16);
    } else {
        st_stream8(reinterpret_cast<uint2 *>(p.codes) + at, make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16)));
    }
    if (at % Frag::kBlock == 0) p.block_scales[at / Frag::kBlock] = (uint8_t)code;
}

// A launch less, where an image's groups have few chunks (up to 128, and 4096 in
// all): each CTA joins them itself, eight lanes a group, from sums about the first
// chunk's mean.  `stats`: those of the CTA's groups; stored by the CTAs that say so.
constexpr int kFewLanes = 8, kFewChunks = 128, kFewAll = 4096;
__device__ __forceinline__ void join_few(const GnParams &p, const GnPlace &at, int64_t n, bool store, float2 *stats)
{
    const int lane = threadIdx.x & 31, from = lane % kFewLanes, at_once = 32 / kFewLanes, P = p.g.P;
    const float last = (float)((p.g.S - (int64_t)(P - 1) * p.chunk_R) * p.g.per), whole = (float)p.chunk_R * p.g.per;
    for (int g0 = (threadIdx.x >> 5) * at_once; g0 < at.groups; g0 += (blockDim.x >> 5) * at_once) {
        const int g = g0 + lane / kFewLanes;
        const float2 *part = p.part + (n * p.g.groups + at.g0 + min(g, at.groups - 1)) * P;
        const float pivot = __ldcg(part).x;
        float a = 0.0f, b = 0.0f;
        constexpr int U = 8; // loads under way at once
        for (int k = from; k < P; k += U * kFewLanes) {
            float2 t[U];
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (k + j * kFewLanes < P) t[j] = __ldcg(part + k + j * kFewLanes);
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (k + j * kFewLanes < P) {
                    const float rows = k + j * kFewLanes + 1 < P ? whole : last;
                    const float d = __fsub_rn(t[j].x, pivot), e = __fmul_rn(d, rows);
                    a = __fadd_rn(a, e);
                    b = __fadd_rn(b, __fmaf_rn(d, e, t[j].y));
                }
        }
        a = lane_sum(a, kFewLanes);
        b = lane_sum(b, kFewLanes);
        const float d = __fdiv_rn(a, p.count);
        float m2 = __fmaf_rn(-a, d, b);
        if (m2 < 0.0f) m2 = 0.0f; // (not fmaxf: what is not a number stays that)
        const float2 st = make_float2(__fadd_rn(pivot, d), defined_rsqrt(__fadd_rn(__fdiv_rn(m2, p.count), p.eps)));
        if (from == 0 && g < at.groups) {
            stats[g] = st;
            if (store) p.stats[n * p.g.groups + at.g0 + g] = st;
        }
    }
}

template <int TYPE, bool CKPT, bool UNI, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) gn_apply_kernel(const GnParams p)
{
    using Frag = Fragment<TYPE>;
    extern __shared__ __align__(16) uint4 s_ring[]; // [kRing][NT]
    // the last chunk first, and of it the last rows
    const int64_t n = gridDim.x - 1 - blockIdx.x;
    const GnPlace at(p.g, gridDim.z - 1 - blockIdx.z, gridDim.y - 1 - blockIdx.y);
    const int step = p.g.RL * p.g.F;
    int left = at.whole + (at.rest > 0); // rows of row lane 0; this thread has those up to `mine`
    int64_t to = at.first(p.g, n) + (left - 1) * (int64_t)step;
    const char *x = p.x + to * 16;
    char *y = p.y + to * 16;
    uint4 *slot = s_ring + threadIdx.x;
    // x is read for the last time, y is not read again here: neither displaces what
    // is still to be read
    const uint64_t first = evict_first();
    auto ask = [&](int j, int ahead) {
        if (left > ahead && left - ahead <= at.mine) cp_async16(slot + j * NT, x - ahead * (int64_t)(step * 16), first);
        cp_async_commit();
    };
    // x and the gains were complete before the kernel whose results are waited
    // for below let this one start
#pragma unroll
    for (int j = 0; j < kRing; ++j) ask(j, j);
    Norm<Frag::kP, UNI> norm = {};
    if (at.mine > 0) p.gains.get<TYPE>(n, at.f0 + at.f, norm.a, norm.b);
    grid_dependency_wait();
    allow_dependents();
    const float2 *stats = p.stats + n * p.g.groups + at.g0;
    if (p.few) {
        float2 *s_stats = reinterpret_cast<float2 *>(s_ring + kRing * NT);
        join_few(p, at, n, p.stats && at.row0 == 0, s_stats);
        __syncthreads();
        stats = s_stats;
    }
    if (at.mine > 0) norm.moments(p.g, stats, at.f * Frag::kE);
    for (; left > 0; left -= kRing, to -= kRing * (int64_t)step, x -= kRing * (int64_t)(step * 16), y -= kRing * (int64_t)(step * 16)) {
#pragma unroll
        for (int j = 0; j < kRing; ++j) {
            if (left <= j) break;
            const bool live = left - j <= at.mine;
            cp_async_wait<kRing - 1>();
            uint4 a = make_uint4(0, 0, 0, 0);
            if (live) a = slot[j * NT];
            ask(j, j + kRing);
            float2 v[Frag::kP], z[Frag::kP];
            Frag::values(a, v);
            norm.apply(v, p.act, z);
            if (live) Frag::store(y - j * (int64_t)(step * 16), z, first);
            if (CKPT) store_codes<TYPE>(p, to - j * (int64_t)step, v, live);
        }
    }
}

// ------------------------------------------------------------------- slabs

// One launch, one read of x (4.9 us for [1, 8 x 8, 1280], where the passes took
// 10): a cluster holds a slab (whole groups of an image) in
// its CTAs' shared memory.  Each thread copies its own fragments there, all at
// once, and nobody else reads them; the CTAs exchange their groups' moments
// through the cluster's shared memory.
template <int TYPE, bool CKPT, bool UNI>
__global__ void __launch_bounds__(512, 2) gn_slab_kernel(const GnParams p)
{
    using Frag = Fragment<TYPE>;
    extern __shared__ __align__(16) uint4 s_data[]; // [M][threads]
    const int tid = threadIdx.x, lane = tid & 31, NT = blockDim.x, cs = 1 << p.log_cs;
    float2 *s_units = reinterpret_cast<float2 *>(s_data + p.M * NT); // [RL][units]
    float2 *s_group = s_units + NT * p.per_frag;                     // [groups] mean, m2 (this CTA's)
    float2 *s_stats = s_group + Frag::kE * p.g.Ft;                   // [groups] mean, rstd

    const int rank = blockIdx.x & (cs - 1); // (clusters lie along x)
    const int64_t n = blockIdx.x >> p.log_cs;
    const GnPlace at(p.g, blockIdx.y, rank);
    const int64_t step = (int64_t)p.g.RL * p.g.F;
    int64_t to = at.first(p.g, n);
    uint4 *slot = s_data + tid;

    grid_dependency_wait();
    allow_dependents();
    constexpr int kParts = 4; // the rows arrive in parts, the first is summed while the others are under way
    const int part = (p.M + kParts - 1) / kParts;
    {
        const char *x = p.x + to * 16;
        int i = 0;
#pragma unroll
        for (int k = 1; k <= kParts; ++k) {
            for (const int end = min(at.mine, k * part); i < end; ++i, x += step * 16) cp_async16(slot + i * NT, x);
            cp_async_commit();
        }
    }
    Norm<Frag::kP, UNI> norm = {};
    if (at.mine > 0) p.gains.get<TYPE>(n, at.f0 + at.f, norm.a, norm.b);
    Sums<Frag::kP> sums;
    int i = 0;
#pragma unroll
    for (int k = 1; k <= kParts; ++k) {
        if (k == 1) cp_async_wait<3>();
        if (k == 2) cp_async_wait<2>();
        if (k == 3) cp_async_wait<1>();
        if (k == 4) cp_async_wait<0>();
        float2 v[Frag::kP];
        if (k == 1 && at.mine > 0) {
            Frag::values(slot[0], v);
            sums.start(v, p.unit);
        }
        for (const int end = min(at.mine, k * part); i < end; ++i) {
            Frag::values(slot[i * NT], v);
            sums.add(v);
        }
    }
    if (at.mine > 0) sums.finish(p.unit, at.mine, s_units + (at.r * at.Ft + at.f) * p.per_frag);
    __syncthreads();
    if (at.rows > 0) join_units(p, at, s_units, s_group, 1);
    auto finish = [&](int g, float mean, float m2) {
        const float2 st = make_float2(mean, defined_rsqrt(__fadd_rn(__fdiv_rn(m2, p.count), p.eps)));
        s_stats[g] = st;
        if (rank == 0 && p.stats) p.stats[n * p.g.groups + at.g0 + g] = st;
    };
    if (cs == 1) {
        __syncthreads();
        for (int g = tid; g < at.groups; g += NT) finish(g, s_group[g].x, s_group[g].y);
    } else {
        cluster_arrive();
        cluster_wait();
        // cs lanes have a group, a CTA's moments each
        const int from = lane & (cs - 1), at_once = 32 >> p.log_cs;
        const float share = (float)(max((int64_t)0, min((int64_t)p.g.R, p.g.S - (int64_t)from * p.g.R)) * p.g.per);
        for (int g0 = (tid >> 5) * at_once; g0 < at.groups; g0 += (NT >> 5) * at_once) {
            const int g = g0 + (lane >> p.log_cs);
            const bool here = g < at.groups && share > 0.0f;
            const float2 t = here ? ld_cluster(s_group + g, from) : make_float2(0.0f, 0.0f);
            const float pivot = __shfl_sync(kFull, t.x, lane - from); // the first CTA's (it has rows)
            const float e = here ? __fsub_rn(t.x, pivot) : 0.0f;
            const float off = __fdiv_rn(lane_sum(__fmul_rn(e, share), cs), p.count); // the mean's, from the pivot
            const float d = here ? __fsub_rn(e, off) : 0.0f;
            const float m2 = lane_sum(__fmaf_rn(__fmul_rn(d, d), share, t.y), cs);
            if (from == 0 && g < at.groups) finish(g, __fadd_rn(pivot, off), m2);
        }
        cluster_arrive(); // nobody reads this CTA's moments after the wait below
    }
    __syncthreads();
    if (at.mine > 0) norm.moments(p.g, s_stats, at.f * Frag::kE);
    const int loops = CKPT ? at.whole + (at.rest > 0) : at.mine;
    for (int k = 0; k < loops; ++k, to += step) {
        const bool live = !CKPT || k < at.mine;
        uint4 a = make_uint4(0, 0, 0, 0);
        if (live) a = slot[k * NT];
        float2 v[Frag::kP], z[Frag::kP];
        Frag::values(a, v);
        norm.apply(v, p.act, z);
        if (live) Frag::store(p.y + to * 16, z);
        if (CKPT) store_codes<TYPE>(p, to, v, live);
    }
    if (cs > 1) cluster_wait();
}

GnSlab forward_slab(int64_t S, int64_t C, int64_t groups, int type, bool checkpoint)
{
    const int64_t E = type_channels(type), unit = gcd64(C / groups, E);
    // (a fragment for each thread of the smallest CTA: [16384, 1, 1024] took 0.45 ms, fp32
    // 0.72, with the eight fragments of a segment, and 0.08 and 0.09 so)
    return gn_slab(S, C, groups, type, checkpoint, 16, (int)(E / unit * sizeof(float2)), 64);
}

GnCut forward_cut(int64_t S, int64_t C, int64_t groups, int type, bool checkpoint)
{
    return gn_cut(S, C, groups, type, checkpoint, kRing, 2, 608);
}

// Lanes of a group's join: one per entry of RL row lanes if there are fewer than a warp's.
void set_join(GnParams &p)
{
    p.join = 1;
    while (p.join < 32 && p.join < p.g.RL * p.per_group) p.join *= 2;
    p.wide = p.per_group < p.join ? p.per_group : p.join;
    p.deep = p.join / p.wide;
    p.by_wide = Divisor(p.wide);
}

template <int TYPE, bool CKPT, bool UNI>
cudaError_t launch_slab(GnParams p, const GnProblem &q, const GnSlab &c, cudaStream_t s)
{
    p.g = gn_grid(q.S, q.C, q.groups, TYPE, c.Ft, c.R, 1 << c.log_cs, c.RL);
    set_join(p);
    p.log_cs = c.log_cs;
    p.M = c.M;
    p.stats = static_cast<float2 *>(q.stats);
    const cudaError_t e = ready(gn_slab_kernel<TYPE, CKPT, UNI>, c.smem);
    if (e != cudaSuccess) return e;
    return launch_grid(gn_slab_kernel<TYPE, CKPT, UNI>, dim3((unsigned)(q.N << c.log_cs), c.slabs), 1 << c.log_cs,
                       c.threads, c.smem, s, p);
}

template <int TYPE, bool CKPT, bool UNI>
cudaError_t launch_passes(GnParams p, const GnProblem &q, const GnCut &c, cudaStream_t s)
{
    p.g = gn_grid(q.S, q.C, q.groups, TYPE, c.Ft, c.R, c.P, c.RL);
    set_join(p);
    p.part = static_cast<float2 *>(q.workspace);
    p.few = c.P <= kFewChunks && c.P * p.g.tile_groups <= kFewAll;
    p.chunk_R = (int)c.R;
    p.stats = q.stats || p.few ? static_cast<float2 *>(q.stats) : p.part + q.N * q.groups * c.P;
    // Of all that the first kernel reads, what the L2 is found to hold for the
    // second: some 64 MB.
    const float all = (float)(q.N * q.S) * (float)q.C * (float)type_bytes(TYPE);
    p.keep = all > 64e6f ? 64e6f / all : 1.0f;
    const int ring = kRing * 16 * c.threads, units = 2 * c.RL * c.Ft * p.per_frag * (int)sizeof(float2);
    const int64_t slots = (int64_t)sm_count() * (1024 / c.threads) / c.tiles;
    // the second kernel's rows need not be whole chunks
    const int64_t round = (int64_t)kRing * c.RL, second = gn_share(q.N, slots, (q.S + round - 1) / round);
    GnParams a = p;
    a.g.R = (int)((q.S + second - 1) / second);
    p.chunks = c.rounds ? (int)((c.P + gn_share(q.N, slots, c.P) - 1) / gn_share(q.N, slots, c.P)) : 1;
    const dim3 one((unsigned)q.N, (unsigned)((c.P + p.chunks - 1) / p.chunks), c.tiles);
    const dim3 two((unsigned)q.N, (unsigned)((q.S + a.g.R - 1) / a.g.R), c.tiles);
    auto go = [&](auto threads) {
        constexpr int NT = decltype(threads)::value;
        const auto moments = gn_moments_kernel<TYPE, NT>;
        const auto apply = gn_apply_kernel<TYPE, CKPT, UNI, NT>;
        const int smem1 = room_for(1024 / NT, ring + units);
        const int smem2 = room_for(1024 / NT, ring + (p.few ? p.g.tile_groups * (int)sizeof(float2) : 0));
        cudaError_t e = ready(moments, smem1);
        if (e == cudaSuccess) e = ready(gn_join_kernel, 0);
        if (e == cudaSuccess) e = ready(apply, smem2);
        if (e == cudaSuccess) e = launch_grid(moments, one, 1, NT, smem1, s, p);
        if (e == cudaSuccess && !p.few) e = launch_grid(gn_join_kernel, dim3((unsigned)(q.N * q.groups)), 1, kJoin, 0, s, p);
        if (e == cudaSuccess) e = launch_grid(apply, two, 1, NT, smem2, s, a);
        return e;
    };
    if (c.threads <= 256) return go(std::integral_constant<int, 256>());
    return go(std::integral_constant<int, gn_threads(TYPE)>());
}

} // namespace

int64_t group_norm_workspace(int64_t N, int64_t S, int64_t C, int64_t groups, int type, bool checkpoint)
{
    if (N * S == 0 || forward_slab(S, C, groups, type, checkpoint).Ft) return 0;
    const GnCut c = forward_cut(S, C, groups, type, checkpoint);
    return N * groups * (c.P + 1) * (int64_t)sizeof(float2);
}

cudaError_t launch_group_norm(const GnProblem &q, cudaStream_t s)
{
    const bool ckpt = q.codes != nullptr;
    const GnSlab slab = forward_slab(q.S, q.C, q.groups, q.type, ckpt);
    GnParams p = {};
    p.x = static_cast<const char *>(q.x);
    p.y = static_cast<char *>(q.y);
    p.codes = static_cast<char *>(q.codes);
    p.block_scales = static_cast<uint8_t *>(q.block_scales);
    p.gains = Gains{q.weight, q.bias, q.scale, q.shift, q.param_type, q.vs};
    const int64_t E = type_channels(q.type), per = q.C / q.groups;
    p.unit = (int)gcd64(per, E);
    p.per_frag = (int)E / p.unit;
    p.per_group = (int)per / p.unit;
    p.act = q.act;
    p.eps = q.eps;
    p.count = (float)(q.S * per);
    return with_type(q.type, [&](auto type) {
        return with_bool(ckpt, [&](auto codes) {
            return with_bool(p.unit == E, [&](auto uni) {
                constexpr int T = decltype(type)::value;
                constexpr bool K = decltype(codes)::value, U = decltype(uni)::value;
                if (slab.Ft) return launch_slab<T, K, U>(p, q, slab, s);
                return launch_passes<T, K, U>(p, q, forward_cut(q.S, q.C, q.groups, q.type, ckpt), s);
            });
        });
    });
}

} // namespace dan
