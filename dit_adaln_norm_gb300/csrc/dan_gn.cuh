// dan_gn.cuh -- what the group norm's forward and backward kernels share: how
// an image is cut up, fragments of 16 bytes of the three types, the gains and the
// activation.
//
// An image is S positions (rows) of C channels.  Every thread keeps to one
// fragment of neighbouring channels and visits rows: Ft threads of a CTA cover a
// tile of a row (whole groups), RL rows at a time.  All of these cuts follow from
// S, C, the groups, the type and whether there is a checkpoint, never from N, so
// that an image's bits do not depend on the others (batch invariance).
#pragma once

#include "dan_train.cuh"

#include <type_traits>

namespace dan {

// ------------------------------------------------------------- fragments

// 16 bytes of neighbouring channels of `TYPE` (a lane's 16 bytes lie beside the
// next lane's; with eight fp32 channels a thread, in two accesses, half of each
// 32-byte sector went unused at a time and the fp32 kernels took twice as long).
template <int TYPE>
struct Fragment {
    static constexpr int kE = TYPE == kFp32 ? 4 : 8; // channels
    static constexpr int kP = kE / 2;                // pairs
    static constexpr int kBlock = 32 / kE;           // fragments of a checkpoint's block
    // a fragment's codes
    using Codes = typename std::conditional<TYPE == kFp32, uint32_t, uint2>::type;

    // The fp32 pairs of a fragment.
    __device__ __forceinline__ static void values(const uint4 &w, float2 (&v)[kP])
    {
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            if constexpr (TYPE == kFp32) v[i] = make_float2(__uint_as_float(word(w, 2 * i)), __uint_as_float(word(w, 2 * i + 1)));
            else if constexpr (TYPE == kBf16) v[i] = wide2(word(w, i));
            else {
                const uint32_t u = word(w, i);
                v[i] = __half22float2(*reinterpret_cast<const __half2 *>(&u));
            }
        }
    }
    __device__ __forceinline__ static void store(char *p, const float2 (&v)[kP], uint64_t policy)
    {
        uint4 o;
        pack(v, o);
        asm volatile("st.global.L1::no_allocate.L2::cache_hint.v4.u32 [%0], {%1,%2,%3,%4}, %5;" ::"l"(p), "r"(o.x), "r"(o.y), "r"(o.z), "r"(o.w), "l"(policy) : "memory");
    }
    __device__ __forceinline__ static void store(char *p, const float2 (&v)[kP])
    {
        uint4 o;
        pack(v, o);
        st_stream(reinterpret_cast<uint4 *>(p), o);
    }
    __device__ __forceinline__ static void pack(const float2 (&v)[kP], uint4 &out)
    {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            if constexpr (TYPE == kFp32) {
                o[2 * i] = __float_as_uint(v[i].x);
                o[2 * i + 1] = __float_as_uint(v[i].y);
            } else if constexpr (TYPE == kBf16) {
                o[i] = pack_bf16(v[i].x, v[i].y);
            } else {
                const __half2 h = __floats2half2_rn(v[i].x, v[i].y);
                o[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        out = make_uint4(o[0], o[1], o[2], o[3]);
    }
    // The codes' values without their block's scale.
    __device__ __forceinline__ static void codes(const Codes &c, float2 (&v)[kP])
    {
        if constexpr (TYPE == kFp32) {
            v[0] = e4m3_pair(c & 0xFFFFu);
            v[1] = e4m3_pair(c >> 16);
        } else {
            v[0] = e4m3_pair(c.x & 0xFFFFu);
            v[1] = e4m3_pair(c.x >> 16);
            v[2] = e4m3_pair(c.y & 0xFFFFu);
            v[3] = e4m3_pair(c.y >> 16);
        }
    }
};

// One value of an output whose type is known at run time (a few per CTA).
__device__ __forceinline__ void store_as(void *p, int type, int64_t i, float v)
{
    if (type == kBf16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else if (type == kFp16) static_cast<__half *>(p)[i] = __float2half_rn(v);
    else static_cast<float *>(p)[i] = v;
}

// 1 / (1 + exp(-z)) of a pair, each within (4 + |z|) * 2^-23 of it relatively (0
// where exp(-z) passes 2^126): the function units' power of two and reciprocal in
// the forms that flush subnormal numbers, which neither meets on the way to a
// value that counts (the others take three times the instructions).
__device__ __forceinline__ float2 sigmoid2(float2 z)
{
    const float2 p = mul2(z, dup2(-1.4426950408889634f));
    float2 e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(p.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(p.y));
    const float2 q = add2(e, dup2(1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(q.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(q.y));
    return s;
}

// The gains of image n's channels: z = normalised * a + b.  weight and bias are
// of TYPE or fp32.  The loads of a call do not wait for one another: behind a
// branch each they cost a trip to memory each (32 of them took 8 us of a kernel).
struct Gains {
    const void *weight, *bias, *scale, *shift;
    int param_type;
    int64_t vs;

    // weight, bias, 1 + scale and shift of channel c.
    struct One {
        float w, b, o, t;
        __device__ __forceinline__ float gain() const { return __fmul_rn(w, o); }
    };
    template <int TYPE>
    __device__ __forceinline__ static float value(const void *p, int64_t i)
    {
        if constexpr (TYPE == kBf16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
        else if constexpr (TYPE == kFp16) return __half2float(static_cast<const __half *>(p)[i]);
        else return static_cast<const float *>(p)[i];
    }
    template <int TYPE>
    __device__ __forceinline__ One one(int64_t n, int64_t c) const
    {
        One g{1.0f, 0.0f, 1.0f, 0.0f};
        float s = 0.0f;
        if (scale) {
            s = value<TYPE>(scale, n * vs + c);
            g.t = value<TYPE>(shift, n * vs + c);
        }
        if (weight) {
            if (param_type == kFp32) {
                g.w = value<kFp32>(weight, c);
                g.b = value<kFp32>(bias, c);
            } else {
                g.w = value<TYPE>(weight, c);
                g.b = value<TYPE>(bias, c);
            }
        }
        g.o = __fadd_rn(1.0f, s);
        return g;
    }

    // a and b of the channels of fragment f.
    template <int TYPE, int P = Fragment<TYPE>::kP>
    __device__ __forceinline__ void get(int64_t n, int f, float2 (&a)[P], float2 (&b)[P]) const
    {
        using Frag = Fragment<TYPE>;
        auto load = [](const void *p, int64_t i) { return ld_stream(static_cast<const uint4 *>(p) + i); };
        uint4 s = make_uint4(0, 0, 0, 0), t = s;
        if (scale) {
            const int64_t at = n * (vs / Frag::kE) + f;
            s = load(scale, at);
            t = load(shift, at);
        }
        if (!weight) {
#pragma unroll
            for (int w = 0; w < P; ++w) a[w] = dup2(1.0f), b[w] = dup2(0.0f);
        } else if (TYPE != kFp32 && param_type == kFp32) {
            uint4 u[P / 2], v[P / 2];
#pragma unroll
            for (int i = 0; i < P / 2; ++i) {
                u[i] = load(weight, f * (P / 2) + i);
                v[i] = load(bias, f * (P / 2) + i);
            }
#pragma unroll
            for (int i = 0; i < P; ++i) {
                a[i] = make_float2(__uint_as_float(word(u[i / 2], 2 * (i & 1))), __uint_as_float(word(u[i / 2], 2 * (i & 1) + 1)));
                b[i] = make_float2(__uint_as_float(word(v[i / 2], 2 * (i & 1))), __uint_as_float(word(v[i / 2], 2 * (i & 1) + 1)));
            }
        } else {
            Frag::values(load(weight, f), a);
            Frag::values(load(bias, f), b);
        }
        float2 o[P], u[P];
        Frag::values(s, o);
        Frag::values(t, u);
#pragma unroll
        for (int w = 0; w < P; ++w) {
            o[w] = add2(dup2(1.0f), o[w]);
            a[w] = mul2(a[w], o[w]);
            b[w] = fma2(b[w], o[w], u[w]);
        }
    }
};

// ---------------------------------------------------------------- geometry

// x / d for the divisors that a launch fixes: an integer division takes some 35
// instructions, and a kernel's dozen of them as many as eight rows of its work.
// Exact for x < 2^32 / d.
struct Divisor {
    unsigned magic; // ceil(2^32 / d), or 0 for d == 1
    __host__ __device__ Divisor() : magic(0) {}
    __host__ explicit Divisor(int64_t d) : magic(d > 1 ? (unsigned)(((int64_t(1) << 32) + d - 1) / d) : 0) {}
    __device__ __forceinline__ int of(int x) const { return magic ? (int)__umulhi((unsigned)x, magic) : x; }
};

// What the kernels know of the cut: tiles of Ft fragments (the last one may be
// narrower), R rows of a chunk (or of a cluster's CTA).
struct GnGrid {
    int64_t S;
    int F, Ft;       // fragments of a row, of a tile
    int R, P;        // rows of a chunk, chunks
    int RL;          // rows that a CTA visits at once
    int per, groups; // channels of a group, groups of an image
    int tile_groups; // groups of a (whole) tile
    Divisor by_Ft, by_RL, by_per;
};

// A CTA's part of it, and this thread's: rows r, r + RL, ... of fragment f.
struct GnPlace {
    int f0, Ft, groups, g0; // the tile's fragments and groups
    int64_t row0;
    int rows, whole, rest; // rows; row lanes below `rest` have whole + 1 of them, the others whole
    int r, f;
    int mine; // this thread's rows
    // `chunk`: the first one; `chunks` of them.
    __device__ __forceinline__ GnPlace(const GnGrid &g, int tile, int chunk, int chunks = 1)
    {
        f0 = tile * g.Ft;
        Ft = min(g.Ft, g.F - f0);
        g0 = tile * g.tile_groups;
        groups = min(g.tile_groups, g.groups - g0);
        row0 = (int64_t)chunk * g.R;
        rows = (int)max((int64_t)0, min((int64_t)g.R * chunks, g.S - row0));
        whole = g.by_RL.of(rows);
        rest = rows - whole * g.RL;
        r = g.by_Ft.of(threadIdx.x);
        f = threadIdx.x - r * g.Ft;
        mine = r < g.RL && f < Ft ? whole + (r < rest) : 0;
    }
    // Their rows in chunk i of several (whole rounds, so that the row lanes go on alike).
    __device__ __forceinline__ GnPlace part(const GnGrid &g, int i) const
    {
        GnPlace q = *this;
        q.rows = min(g.R, rows - i * g.R);
        q.whole = g.by_RL.of(q.rows);
        q.rest = q.rows - q.whole * g.RL;
        q.mine = r < g.RL && f < Ft ? q.whole + (r < q.rest) : 0;
        return q;
    }
    // The thread's first fragment of image n.
    __device__ __forceinline__ int64_t first(const GnGrid &g, int64_t n) const
    {
        return (n * g.S + row0 + r) * g.F + f0 + f;
    }
};

// The groups of a thread's channels, from channel c of a tile on.
struct GroupOf {
    int g, rest, per;
    __device__ __forceinline__ GroupOf(const GnGrid &q, int c) : g(q.by_per.of(c)), per(q.per) { rest = c - g * per; }
    __device__ __forceinline__ int next()
    {
        const int now = g;
        if (++rest == per) rest = 0, ++g;
        return now;
    }
};

inline int64_t gcd64(int64_t a, int64_t b) { return b ? gcd64(b, a % b) : a; }
// Channels that tiles are made of: whole groups and fragments (and checkpoint blocks).
inline int64_t gn_step(int64_t per, bool checkpoint)
{
    const int64_t k = checkpoint ? 32 : 8;
    return per / gcd64(per, k) * k;
}

// Threads of the largest CTA: 4096 channels of a row.
__host__ __device__ constexpr int gn_threads(int type) { return type == kFp32 ? 1024 : 512; }
constexpr int64_t kGnWidest = 4096; // channels of the widest tile
inline int64_t type_bytes(int type) { return type == kFp32 ? 4 : 2; }
inline int64_t type_channels(int type) { return type == kFp32 ? 4 : 8; } // of a fragment

// How an image is cut for the kernels that read it in passes: tiles, and chunks
// of rows whose sums are kept one by one.
struct GnCut {
    int Ft, tiles, threads, RL;
    int64_t R, P;
    bool rounds; // chunks are whole rounds: a CTA may take several on end
};

// Shared memory that lets `blocks` CTAs share an SM and no more.  A wave is one CTA
// in each of these places; where the registers would let another one in, some SMs
// took three of a wave of two per SM and others one (the gradient of a [1, 512 x
// 512, 256] image: 120 us, with two each 109).
inline int room_for(int blocks, int smem)
{
    const int least = 228 * 1024 / (blocks + 1);
    return smem > least ? smem : least;
}

// Tiles of whole rows where they have up to 256 fragments, else of as many
// whole steps; chunks of `rounds` rounds of `ring` rows of each thread (a round of
// eight rows of 256 threads is 32 KB), or where there would be over `most`, that many.
inline GnCut gn_cut(int64_t S, int64_t C, int64_t groups, int type, bool checkpoint, int64_t ring, int64_t rounds,
                    int64_t most)
{
    GnCut c;
    const int64_t E = type_channels(type), F = C / E, step = gn_step(C / groups, checkpoint) / E;
    c.Ft = (int)(F <= 256 ? F : step >= 256 ? step : 256 / step * step);
    c.tiles = (int)((F + c.Ft - 1) / c.Ft);
    c.threads = c.Ft <= 256 ? 256 : gn_threads(type);
    c.RL = c.threads / c.Ft;
    const int64_t round = ring * c.RL, all = (S + round - 1) / round;
    c.rounds = all <= rounds * most;
    c.R = c.rounds ? rounds * round : (S + most - 1) / most;
    c.P = (S + c.R - 1) / c.R;
    return c;
}

// CTAs of an image (at most `most`) such that all images' come to whole waves of
// `slots`: the last, part-filled wave of a few costs as much as a full one.
inline int64_t gn_share(int64_t N, int64_t slots, int64_t most)
{
    int64_t q = slots / N;
    if (q * N * 20 < slots * 17) q = (4 * slots + N - 1) / N; // not 85% of a wave: several waves
    return q < 1 ? 1 : q < most ? q : most;
}

// How an image is cut into slabs of whole groups that a cluster of CTAs holds in
// shared memory: each CTA has R of the slab's rows.
struct GnSlab {
    int Ft;      // 0: no slab fits
    int slabs;
    int log_cs;  // CTAs of a cluster
    int64_t R;   // rows of each (the last ones may have fewer or none)
    int threads, RL;
    int M;       // rows of a thread at most
    int smem;    // bytes
};

constexpr int kSlabCluster = 3; // log2 of the largest portable cluster

// The shared memory of a CTA: up to 64 KB of rows and what joins them.
constexpr int64_t kSlabRows = 64 * 1024, kSlabRoom = 80 * 1024;

// bytes: of a fragment in shared memory; extra: further bytes per thread; fill: a
// slab of fewer fragments than that is made wider.  A warp has up to 32 (65536 images
// of [1, 64] 114 us with two, 68 so).
// Segments of 128 bytes of a row where such slabs fit, else of 64 (of 32 they took
// 17.6 us for a [1, 128 x 128, 512] image, the passes 11.7); as few CTAs, and as
// few threads of eight fragments, as do: many small ones did better for one image
// (a [1, 32 x 32, 640] one: 6.7 us with 32 KB and four fragments, 7.7 so), worse
// for many (16 of them: 20.3 and 15.8), and which it is may not count.
inline GnSlab gn_slab(int64_t S, int64_t C, int64_t groups, int type, bool checkpoint, int bytes, int extra,
                      int64_t fill)
{
    GnSlab c = {};
    const int64_t E = type_channels(type), F = C / E, step = gn_step(C / groups, checkpoint) / E;
    for (int64_t segment = 128; segment >= 64; segment /= 2) {
        int64_t Ft = (segment / 16 + step - 1) / step * step;
        while (Ft < F && 2 * Ft * S <= fill) Ft *= 2;
        if (Ft > F) Ft = F;
        if (Ft > 256 || (F + Ft - 1) / Ft > 65535) continue; // (slabs lie along a grid's y)
        int log_cs = 0;
        while (log_cs < kSlabCluster && (2 << log_cs) <= S && S * Ft * bytes > (kSlabRows << log_cs)) ++log_cs;
        const int64_t rows = (S + (1 << log_cs) - 1) >> log_cs;
        int threads = rows * Ft <= 32 && (fill > 0 || E * Ft <= 32) ? 32 : 64; // (a channel each in the gradients)
        while (threads < 512 && (threads < Ft || rows * Ft > threads * (threads < 256 ? 8 : 16))) threads *= 2;
        const int64_t RL = threads / Ft, M = (rows + RL - 1) / RL;
        const int64_t smem = M * threads * bytes + (int64_t)threads * extra + E * Ft * 48;
        if (smem > kSlabRoom) continue;
        c.Ft = (int)Ft;
        c.slabs = (int)((F + Ft - 1) / Ft);
        c.log_cs = log_cs;
        c.R = rows;
        c.threads = threads;
        c.RL = (int)RL;
        c.M = (int)M;
        c.smem = (int)smem;
        return c;
    }
    return c;
}

// The kernels' view of a cut.
inline GnGrid gn_grid(int64_t S, int64_t C, int64_t groups, int type, int64_t Ft, int64_t R, int64_t P, int64_t RL)
{
    GnGrid g;
    const int64_t E = type_channels(type), per = C / groups;
    g.S = S;
    g.F = (int)(C / E);
    g.Ft = (int)Ft;
    g.R = (int)R;
    g.P = (int)P;
    g.RL = (int)RL;
    g.per = (int)per;
    g.groups = (int)groups;
    g.tile_groups = (int)(Ft * E / per);
    g.by_Ft = Divisor(Ft);
    g.by_RL = Divisor(RL);
    g.by_per = Divisor(per);
    return g;
}

// What a kernel's launch may fail on beforehand: a call makes sure of all its
// kernels before it launches the first.
template <typename... KArgs>
cudaError_t ready(void (*fn)(KArgs...), int smem)
{
    return allow_dynamic_smem(reinterpret_cast<const void *>(fn), smem);
}

// A launch with programmatic stream serialization on a grid of three dimensions,
// in clusters of `cs` CTAs along x (of a kernel that is ready).
template <typename... KArgs, typename... Args>
cudaError_t launch_grid(void (*fn)(KArgs...), dim3 grid, int cs, int block, int smem, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cs;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cs > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

// Calls f with a type's, or a truth value's, constant.
template <typename F>
cudaError_t with_type(int type, F f)
{
    return type == kBf16   ? f(std::integral_constant<int, kBf16>())
           : type == kFp16 ? f(std::integral_constant<int, kFp16>())
                           : f(std::integral_constant<int, kFp32>());
}
template <typename F>
cudaError_t with_bool(bool b, F f)
{
    return b ? f(std::true_type()) : f(std::false_type());
}

// ------------------------------------------------------------------ cluster

// The cluster's barrier, in two halves, and a read of another CTA's shared memory.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ float2 ld_cluster(const float2 *p, int rank)
{
    unsigned at;
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}

// L2 policies: what goes first, and the usual one.
__device__ __forceinline__ uint64_t evict_first()
{
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint64_t evict_normal()
{
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void cp_async16(void *smem_dst, const void *gmem_src, uint64_t policy)
{
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(smem_addr(smem_dst)),
                 "l"(gmem_src), "l"(policy)
                 : "memory");
}

// Over each `lanes` neighbouring lanes of a warp (a power of two).
__device__ __forceinline__ float lane_sum(float v, int lanes)
{
    for (int off = lanes >> 1; off >= 1; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kFull, v, off));
    return v;
}

// Asynchronous copy of 4, 8 or 16 bytes to shared memory.
__device__ __forceinline__ void cp_async_word(uint4 *to, const void *from) { cp_async16(to, from); }
__device__ __forceinline__ void cp_async_word(uint2 *to, const void *from) { cp_async8(to, from); }
__device__ __forceinline__ void cp_async_word(uint32_t *to, const void *from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}

} // namespace dan
