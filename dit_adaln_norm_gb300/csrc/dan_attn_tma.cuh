// dan_attn_tma.cuh -- device primitives of the attention kernels: TMA tile
// loads, warp matrix products, base-2 exponential, and the row epilogue.
#pragma once

#include "dan_attn.cuh"
#include "dan_device.cuh"
#include "dan_ring.cuh"

namespace dan {

// Tile at (column x, row y) of a 2-D tensor map into shared memory, counted
// in bytes on `bar`.  x is a multiple of 64 elements here (128 bytes); rows
// past the map's extent arrive as zeros and are counted all the same.
__device__ __forceinline__ void tma_load_2d(void *smem_dst, const CUtensorMap *map, int x, int y,
                                            uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(smem_dst)),
                 "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
                 : "memory");
}

// Fetch a tensor map before its first use (it is a kernel argument: it does
// not depend on the kernel before).
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Box at (column x, y, z) of a 3-D tensor map, likewise.
__device__ __forceinline__ void tma_load_3d(void *smem_dst, const CUtensorMap *map, int x, int y, int z,
                                            uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(smem_dst)),
                 "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const void *p)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_addr(p))
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], const void *p)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_addr(p))
                 : "memory");
}

// d += a (16 x 16, rows) * b (16 x 8, columns), bf16 products summed in fp32.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                 "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 2^x by the hardware's approximation (relative error about 2^-22; -infinity
// gives 0, NaN gives NaN).
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Natural-log statistic of a row from its base-2 maximum and sum.
__device__ __forceinline__ float row_lse(float m, float l)
{
    constexpr float kLn2 = 0.693147180559945309f;
    return l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Columns c .. c+3 of query head h of token t: the accumulated row over its
// sum (a row that saw no key: zeros), rounded once; column 0's writer also
// stores the statistic.
template <int HD>
__device__ __forceinline__ void write_row(const AttnParams &p, int t, int h, int c, const float4 &a,
                                          float m, float l)
{
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t row = (int64_t)t * p.H + h;
    uint2 w;
    w.x = pack_bf16(a.x * inv, a.y * inv);
    w.y = pack_bf16(a.z * inv, a.w * inv);
    *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(p.out) + row * HD + c) = w;
    if (c == 0 && p.lse) p.lse[row] = row_lse(m, l);
}

} // namespace dan
