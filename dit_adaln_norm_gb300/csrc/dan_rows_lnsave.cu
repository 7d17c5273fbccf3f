// dan_rows_lnsave.cu -- launches of LayerNorm + modulate that keeps what the
// gradient needs (include/dan_train.h): the row kernel of dan_rows.cuh from 1024
// columns on, and below them a kernel for short rows.
//
// A row of up to 1024 columns is the one fragment of eight columns of each of up
// to 128 threads in ln_modulate's Welford tree.  The row kernel gives such a row
// a warp, one at a time, and where they are not whole folds all four logical warps
// with a division at each of their merges, however few lanes have columns: 2.3 us
// and more a row and warp.  Here
//  - a row of up to 256 columns takes L lanes, a power of two, and several share a
//    warp.  Merging with lanes that hold nothing changes nothing, so the L lanes'
//    folds in the same order have ln_modulate's bits;
//  - a wider one takes the J fragments per lane that it has;
//  - how many values a lane's state stands for at each merge follows from the
//    width alone, so each merge's weight is divided once per kernel, not per row;
//  - U rows a lane are under way at once, of three CTAs an SM (80 registers; of
//    four, 64, they spill).
// With checkpoints, row kernel against this one: 593750 rows of 64 columns 1891 and
// 57 us (floor 29), 16000 of 264 59.0 and 14.2 (3.2), 16000 of 1000 78.4 and 24.0
// (12); one row of 8 to 1000 columns 4.6 to 6.5 and 2.1 to 3.1.  Bound by the issue of
// instructions (64 to 73% of the slots): Welford's chain takes six an element, the
// store and the codes as many, and where L or 32 J is not all of a row's fragments
// the other lanes' are for nothing.  Rows of 1024 are whole: the row kernel folds
// them without divisions, 7.2 us for 4216 of them where this one takes 8.1.
#include "dan_rows.cuh"

namespace dan {
namespace {

struct ShortRows {
    const uint4 *x, *scale, *shift;
    uint4 *y;
    float2 *stats;
    uint2 *codes; // or nullptr
    uint8_t *block_scales;
    int64_t rows, T, vs8;
    int F;
    float eps;
    float inv_d; // 1 / D where D is a power of two, else 0
};

constexpr int kShortThreads = 256, kShortBlocks = 3; // of a CTA; CTAs of an SM

__host__ __device__ constexpr int log2_of(int n) { return n <= 1 ? 0 : 1 + log2_of(n / 2); }

// The merges of one logical warp's fold, lane l with lane l + off for off = L / 2,
// ..., 1: the weights of `combine`, for the lanes whose results count.
template <int L>
struct Merges {
    static constexpr int S = log2_of(L);
    float n[S + 1], c[S + 1]; // values of the lower side; rn(upper / both)
    unsigned none;            // bit s: the upper side of merge s is empty
    __device__ __forceinline__ void plan(float count)
    {
        none = 0;
#pragma unroll
        for (int s = 0, off = L / 2; s < S; ++s, off /= 2) {
            const float other = __shfl_down_sync(kFull, count, off, L), both = __fadd_rn(count, other);
            n[s] = count;
            c[s] = count == other ? 0.5f : other == 0.0f ? 0.0f : __fdiv_rn(other, both);
            if (other == 0.0f) none |= 1u << s;
            count = both;
        }
    }
    // FULL: every lane has its eight values, so that all weights are 1/2.
    template <bool FULL>
    __device__ __forceinline__ void fold(float &mean, float &m2) const
    {
#pragma unroll
        for (int s = 0, off = L / 2; s < S; ++s, off /= 2) {
            const float mb = __shfl_down_sync(kFull, mean, off, L), m2b = __shfl_down_sync(kFull, m2, off, L);
            if (FULL) {
                combine_eq1(mean, m2, mb, m2b, (float)(8 << s));
            } else {
                const float delta = __fsub_rn(mb, mean);
                const float a = __fadd_rn(mean, __fmul_rn(delta, c[s]));
                const float b = __fadd_rn(__fadd_rn(m2, m2b), __fmul_rn(__fmul_rn(__fmul_rn(delta, delta), n[s]), c[s]));
                if (!(none >> s & 1u)) mean = a, m2 = b;
            }
        }
        mean = __shfl_sync(kFull, mean, 0, L);
        m2 = __shfl_sync(kFull, m2, 0, L);
    }
};

// Welford's mean and squares of a fragment's eight values, in order.
__device__ __forceinline__ void welford8(const float (&x)[8], float &mean, float &m2)
{
    mean = m2 = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float d = __fsub_rn(x[e], mean);
        mean = __fadd_rn(mean, __fmul_rn(d, 1.0f / (float)(e + 1)));
        m2 = __fadd_rn(m2, __fmul_rn(d, __fsub_rn(x[e], mean)));
    }
}

// L lanes a row (32 where J > 1), J fragments of a row a lane, U rows of a lane at once.
template <int L, int J, int U>
__global__ void __launch_bounds__(kShortThreads, kShortBlocks) ln_save_short_kernel(const ShortRows p)
{
    static_assert(L == 32 || J == 1, "a warp a row, or several rows a warp");
    constexpr int per = 32 / L; // rows side by side in a warp
    const int lane = threadIdx.x & 31, sub = lane / L, col = lane % L, F = p.F;
    const int64_t warps = (int64_t)gridDim.x * (kShortThreads / 32);
    const int64_t first = ((int64_t)blockIdx.x * (kShortThreads / 32) + (threadIdx.x >> 5)) * (per * U);
    const bool last_here = col + 32 * (J - 1) < F; // (the fragments before the last one are all there)
    auto here = [&](int j) { return j < J - 1 || last_here; };
    Merges<L> merges;
    merges.plan(last_here ? 8.0f : 0.0f);

    // this lane's rows: row + u * per.  A batch further on each `per` rows, and each
    // round of all warps, without a division.
    int64_t row = first + sub, b = row / p.T, t = row - b * p.T;
    const int64_t round = warps * per * U, per_b = per / p.T, per_t = per - per_b * p.T;
    const int64_t round_b = round / p.T, round_t = round - round_b * p.T;
    grid_dependency_wait();
    allow_dependents();
    for (int64_t base = first; base < p.rows; base += round, row += round) { // (the same for a whole warp)
        uint4 v[U][J];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                v[u][j] = make_uint4(0, 0, 0, 0);
                if (here(j) && row + u * per < p.rows) v[u][j] = ld_stream(p.x + (row + u * per) * F + col + 32 * j);
            }
        int64_t bu = b, tu = t;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = row + u * per;
            const bool live = r < p.rows;
            float x[J][8];
            Welford w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = Welford{0.0f, 0.0f, 0.0f};
                if (j >= J) continue;
                widen8(v[u][j], x[j]);
                welford8(x[j], w[j].mean, w[j].m2);
                if (j < J - 1) merges.template fold<true>(w[j].mean, w[j].m2);
                else merges.template fold<false>(w[j].mean, w[j].m2);
                w[j].n = j < J - 1 ? 256.0f : (float)(8 * (F - 32 * (J - 1)));
            }
            float mean, m2;
            ln_final<true>(w, mean, m2);
            const float var = p.inv_d != 0.0f ? __fmul_rn(m2, p.inv_d) : __fdiv_rn(m2, (float)(8 * F));
            const float rstd = defined_rsqrt(__fadd_rn(var, p.eps));
            if (live && col == 0) p.stats[r] = make_float2(mean, rstd);
            const int64_t vec = bu * p.vs8 + col;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const bool mine = live && here(j);
                const int f = col + 32 * j;
                if (mine) {
                    const uint4 sc = ld_vec(p.scale + vec + 32 * j), sh = ld_vec(p.shift + vec + 32 * j);
                    uint4 out;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 n = mul2(sub2(make_float2(x[j][2 * e], x[j][2 * e + 1]), dup2(mean)), dup2(rstd));
                        const float2 z = fma2(n, add2(dup2(1.0f), wide2(word(sc, e))), wide2(word(sh, e)));
                        set_word(out, e, pack_bf16(z.x, z.y));
                    }
                    st_stream(p.y + r * F + f, out);
                }
                if (p.codes == nullptr) continue;
                float top = mine ? top8(x[j]) : 0.0f; // (a block is up to four lanes of the row)
                if (L >= 2) top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
                if (L >= 4) top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
                if (!mine) continue;
                const unsigned code = block_scale_code(top);
                st_stream8(p.codes + r * F + f, e4m3x8(x[j], block_scale_inverse(code)));
                if ((f & 3) == 0) p.block_scales[r * ((F + 3) >> 2) + (f >> 2)] = (uint8_t)code;
            }
            bu += per_b;
            tu += per_t;
            if (tu >= p.T) tu -= p.T, ++bu;
        }
        b += round_b;
        t += round_t;
        if (t >= p.T) t -= p.T, ++b;
    }
}

template <int L, int J, int U>
cudaError_t launch_short(const RowProblem &q, cudaStream_t s)
{
    ShortRows p;
    p.x = static_cast<const uint4 *>(q.x);
    p.scale = static_cast<const uint4 *>(q.scale);
    p.shift = static_cast<const uint4 *>(q.shift);
    p.y = static_cast<uint4 *>(q.y);
    p.stats = static_cast<float2 *>(q.stats);
    p.codes = static_cast<uint2 *>(q.q);
    p.block_scales = static_cast<uint8_t *>(q.block_scales);
    p.rows = q.B * q.T;
    p.T = q.T;
    p.vs8 = q.vs / 8;
    p.F = (int)(q.D / 8);
    p.eps = q.eps;
    p.inv_d = (q.D & (q.D - 1)) == 0 ? 1.0f / (float)q.D : 0.0f;
    const int64_t rows_of_cta = kShortThreads / L * U, ctas = (p.rows + rows_of_cta - 1) / rows_of_cta;
    const int64_t most = (int64_t)kShortBlocks * sm_count();
    const auto fn = ln_save_short_kernel<L, J, U>;
    const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(fn), 0);
    return e != cudaSuccess ? e : launch_overlapped(fn, (int)(ctas < most ? ctas : most), kShortThreads, 0, s, p);
}

} // namespace

cudaError_t launch_ln_modulate_save(const RowProblem &q, cudaStream_t s)
{
    const int64_t F = q.D / 8;
    if (F <= 1) return launch_short<1, 1, 4>(q, s);
    if (F <= 2) return launch_short<2, 1, 4>(q, s);
    if (F <= 4) return launch_short<4, 1, 4>(q, s);
    if (F <= 8) return launch_short<8, 1, 4>(q, s);
    if (F <= 16) return launch_short<16, 1, 4>(q, s);
    if (F <= 32) return launch_short<32, 1, 4>(q, s);
    if (F <= 64) return launch_short<32, 2, 2>(q, s);
    if (F <= 96) return launch_short<32, 3, 1>(q, s);
    if (F < 128) return launch_short<32, 4, 1>(q, s);
    return (q.D % 1024) ? launch_ln_fpt<kLnSave, true>(q, s) : launch_ln_fpt<kLnSave, false>(q, s);
}

} // namespace dan
