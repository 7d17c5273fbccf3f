// dan_gn.cuh -- what the group norm's forward and backward kernels share: how
// an image is cut up, fragments of eight channels of the three types, and the
// activation.
//
// An image is S positions (rows) of C channels.  Every thread keeps to one
// fragment of eight neighbouring channels and visits rows: Ft threads of a CTA
// cover a tile of 8 * Ft channels (whole groups) of a row, RL rows at a time.
// All of these cuts follow from S, C, the groups and the type, never from N, so
// that an image's bits do not depend on the others (batch invariance).
#pragma once

#include "dan_train.cuh"

namespace dan {

// ------------------------------------------------------------- fragments

// Eight neighbouring channels of `TYPE`: loads, four fp32 pairs, stores.
template <int TYPE>
struct Fragment {
    static constexpr int kBytes = TYPE == kFp32 ? 32 : 16;
    static constexpr int kWords = kBytes / 16; // 16-byte words
    uint4 w[kWords];

    __device__ __forceinline__ static float2 pair(uint32_t v)
    {
        if constexpr (TYPE == kBf16) return wide2(v);
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    }
    __device__ __forceinline__ void load(const char *p)
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = ld_stream(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void values(float2 (&v)[4]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (TYPE == kFp32)
                v[i] = make_float2(__uint_as_float(word(w[i / 2], 2 * (i & 1))),
                                   __uint_as_float(word(w[i / 2], 2 * (i & 1) + 1)));
            else v[i] = pair(word(w[0], i));
        }
    }
    __device__ __forceinline__ static void store(char *p, const float2 (&v)[4])
    {
        uint4 *to = reinterpret_cast<uint4 *>(p);
        if constexpr (TYPE == kFp32) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                st_stream(to + i, make_uint4(__float_as_uint(v[2 * i].x), __float_as_uint(v[2 * i].y),
                                             __float_as_uint(v[2 * i + 1].x), __float_as_uint(v[2 * i + 1].y)));
        } else {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (TYPE == kBf16) o[i] = pack_bf16(v[i].x, v[i].y);
                else {
                    const __half2 h = __floats2half2_rn(v[i].x, v[i].y);
                    o[i] = *reinterpret_cast<const uint32_t *>(&h);
                }
            }
            st_stream(to, make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
};

// One value of a vector whose type is known at run time (read a few times per CTA).
__device__ __forceinline__ float load_as(const void *p, int type, int64_t i)
{
    if (type == kBf16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    if (type == kFp16) return __half2float(static_cast<const __half *>(p)[i]);
    return static_cast<const float *>(p)[i];
}

__device__ __forceinline__ void store_as(void *p, int type, int64_t i, float v)
{
    if (type == kBf16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else if (type == kFp16) static_cast<__half *>(p)[i] = __float2half_rn(v);
    else static_cast<float *>(p)[i] = v;
}

// 1 / (1 + exp(-z)), within some 2^-21 of it relatively (and 0 where exp(-z)
// leaves fp32): the function units' exponential and reciprocal.
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.0f, __fadd_rn(1.0f, __expf(-z))); }

// The gains of channel c of image n: z = normalised * a + b.
struct Gains {
    const void *weight, *bias, *scale, *shift;
    int param_type, type;
    int64_t vs;
    __device__ __forceinline__ void get(int64_t n, int64_t c, float &a, float &b) const
    {
        a = weight ? load_as(weight, param_type, c) : 1.0f;
        b = bias ? load_as(bias, param_type, c) : 0.0f;
        if (scale) {
            const float o = __fadd_rn(1.0f, load_as(scale, type, n * vs + c));
            a = __fmul_rn(a, o);
            b = __fmaf_rn(b, o, load_as(shift, type, n * vs + c));
        }
    }
};

// ---------------------------------------------------------------- geometry

// How an image is cut: tiles of Ft fragments, chunks of R rows.
struct GnCut {
    int F;     // fragments of a row
    int Ft;    // fragments of a tile (whole groups; the last tile may be narrower)
    int tiles;
    int threads, RL; // per CTA; rows that a CTA visits at once
    int64_t R, P;    // rows of a chunk, chunks
};

inline int64_t gcd64(int64_t a, int64_t b) { return b ? gcd64(b, a % b) : a; }
// Channels that tiles are made of: whole groups and fragments (and checkpoint blocks).
inline int64_t gn_step(int64_t per, bool checkpoint)
{
    const int64_t k = checkpoint ? 32 : 8;
    return per / gcd64(per, k) * k;
}

constexpr int kGnMost = 512; // fragments of the widest tile

inline int64_t type_bytes(int type) { return type == kFp32 ? 4 : 2; }

// Tiles of whole rows where they have up to 256 fragments, else of as many
// whole steps; chunks of `bytes` (of `type`) at least, `most` chunks at most.
inline GnCut gn_cut(int64_t S, int64_t C, int64_t groups, int type, bool checkpoint, int64_t bytes,
                    int64_t most)
{
    GnCut c;
    const int64_t step = gn_step(C / groups, checkpoint) / 8;
    c.F = (int)(C / 8);
    c.Ft = (int)(c.F <= 256 ? c.F : step >= 256 ? step : 256 / step * step);
    c.tiles = (c.F + c.Ft - 1) / c.Ft;
    c.threads = c.Ft <= 256 ? 256 : kGnMost;
    c.RL = c.threads / c.Ft;
    const int64_t row = c.Ft * 8 * type_bytes(type);
    c.R = (bytes + row - 1) / row;
    if (c.R < c.RL) c.R = c.RL;
    if (c.R < (S + most - 1) / most) c.R = (S + most - 1) / most;
    c.P = (S + c.R - 1) / c.R;
    return c;
}

// --------------------------------------------------- means and squared sums

// Count, mean and sum of squared differences from it of a set of values.
struct Moments {
    float n, mean, m2;
};

// Those of two sets together.
__device__ __forceinline__ Moments join(const Moments &a, const Moments &b)
{
    if (b.n == 0.0f) return a;
    if (a.n == 0.0f) return b;
    Moments o;
    o.n = __fadd_rn(a.n, b.n);
    const float w = __fdividef(b.n, o.n), d = __fsub_rn(b.mean, a.mean);
    o.mean = __fmaf_rn(d, w, a.mean);
    o.m2 = __fmaf_rn(__fmul_rn(__fmul_rn(d, d), a.n), w, __fadd_rn(a.m2, b.m2));
    return o;
}

// Those of a warp's lanes together, in every lane.
__device__ __forceinline__ Moments join_warp(Moments m, int lane)
{
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        Moments o;
        o.n = __shfl_xor_sync(kFull, m.n, off);
        o.mean = __shfl_xor_sync(kFull, m.mean, off);
        o.m2 = __shfl_xor_sync(kFull, m.m2, off);
        m = (lane & off) ? join(o, m) : join(m, o);
    }
    return m;
}

} // namespace dan
