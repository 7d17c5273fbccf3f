// dan_ln_back.cuh -- what the two kernels of LayerNorm + modulate's gradients
// share: a row's cut into threads, and its sums.  A row's dx has the same bits from
// both: the cut and the order of a row's sums follow from the width alone.
#pragma once

#include "dan_train.cuh"

#include <type_traits>

namespace dan {

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
    bool hint_codes; // the codes' rows begin and end on 16 bytes, as the bulk hint wants them
};

__device__ __forceinline__ void team_barrier(int team, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(threads) : "memory");
}

// Sums of N values over a warp: each step halves the lanes' values, the lanes of
// the one half of a pair going on with the one half of them.  Value i ends in the
// lanes whose upper bits are i (32 / N lanes each).
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N], int lane)
{
    int off = 16;
#pragma unroll
    for (int n = N; n > 1; n /= 2, off /= 2) {
        const bool upper = lane & off;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float mine = upper ? v[i + n / 2] : v[i], other = upper ? v[i] : v[i + n / 2];
            v[i] = __fadd_rn(mine, __shfl_xor_sync(kFull, other, off));
        }
    }
    float s = v[0];
#pragma unroll
    for (int k = 32 / N / 2; k >= 1; k /= 2) s = __fadd_rn(s, __shfl_xor_sync(kFull, s, k));
    return s;
}

// Threads of a row: K fragments each, W warps (or, with W == 1, L lanes).  R: the rows
// that ln_back_kernel takes at a time.
struct LnBackCut {
    int K, R, W, L;
};
// A warp per row up to five fragments a lane; else teams of up to eight warps,
// several rows at a time where the registers last.  Replayed, in us, 16M elements from
// checkpoints and from rows with dres (floor 12 and 19), this cut and the next best:
//    264 (K 2)  27 29   K 1  44 44        2048 (K 2, R 4)  22 26   K 4  21 26
//    520 (K 3)  25 28   K 2  31 32        2056 (K 3, R 2)  28 29   K 5  26 28   K 2  32 32
//   1032 (K 5)  22 27   K 3  28 29        3072 (K 3, R 2)  22 27   K 2  25 27
//   1288 (K 2, R 4)  29 29   K 3  24 28   4096 (K 2, R 4)  24 28   K 4  23 27
//   4104 (K 4)  35 37   K 5  27 30        8192 (K 4)  26 31   K 5  28 31
// Several rows a warp, 100000 rows of 8 and of 128 columns: 5.5 and 21 us, a warp a
// row 27 and 33.
inline LnBackCut ln_back_cut(int F)
{
    LnBackCut c;
    c.K = F <= 160 ? (F + 31) / 32 : F <= 256 ? 2 : F <= 384 ? 3 : F <= 512 ? 2 : 4;
    c.W = (F + 32 * c.K - 1) / (32 * c.K);
    c.R = c.W == 1 || c.K == 4 ? 1 : c.K == 2 ? 4 : 2;
    c.L = 32;
    while (c.W == 1 && c.L / 2 >= F) c.L /= 2;
    return c;
}

LnBackParams ln_back_params(const LnBackProblem &q);

// Calls f with the constants (K, R, several rows a warp) of a cut.
template <typename F>
cudaError_t with_cut(const LnBackCut &c, F f)
{
    const std::false_type no;
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    const std::integral_constant<int, 3> three;
    const std::integral_constant<int, 4> four;
    const std::integral_constant<int, 5> five;
    return c.L < 32              ? f(one, one, std::true_type())
           : c.K == 1            ? f(one, one, no)
           : c.K == 2 && c.W > 1 ? f(two, four, no)
           : c.K == 2            ? f(two, one, no)
           : c.K == 3 && c.W > 1 ? f(three, two, no)
           : c.K == 3            ? f(three, one, no)
           : c.K == 4            ? f(four, one, no)
                                 : f(five, one, no);
}

// Short batches (dan_ln_back_short.cu): whether a call goes there, and its launch.
bool ln_back_is_short(int64_t B, int64_t T, int64_t D);
cudaError_t launch_ln_back_short(const LnBackProblem &q, cudaStream_t s);

} // namespace dan
