// dan_attn_step.cu -- attention over the paged cache for sequences with few
// query rows (n_s * heads/kv_heads <= 16): a decoded token, or a few drafted
// ones; and the join of split results of both kernels.
//
// Mathematics: o = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m) with
// x_j = scale * log2(e) * q.k_j and a running maximum m, one pass over the
// keys.  Every key and value is read once for all query heads that share it;
// at 16 rows the arithmetic per byte is small and the bound is memory.  Measured
// on one GB300: 64 tokens over up to 32768 keys, 32 query and 8 key heads of
// 128, 618 us, 7.0 TB/s (a copy reaches 6.7); 96 sequences of one to three
// tokens over 2112 keys of 8 heads of 64, 76 us, 5.0 TB/s; one token over 1028
// keys 10 us, launches and dependent loads.
//
// One CTA has one (sequence, key head, split); where the tile kernel follows,
// one more plans its work.  Its four warps take blocks of 16 keys (32 at
// head_dim 64) in turn, each with its own ring of TMA-filled slots, its own
// running maximum, sum and output; nothing but the end joins them.  The 16
// query rows are the rows of m16n8k16 products.  TMA brings a block's K and V
// with the 128-byte swizzle, so that the matrix loads are free of bank
// conflicts.
#include "dan_device.cuh"
#include "dan_internal.h"
#include "dan_attn.cuh"
#include "dan_attn_plan.cuh"
#include "dan_attn_tma.cuh"
#include "dan_ring.cuh"

namespace dan {

constexpr int kStepWarps = 4;
// Three slots leave fewer CTAs per SM: 96 sequences of 2112 keys of 8 heads of 64
// take 84 us with them and 76 with two, 64 over up to 32768 keys 627 and 619.
constexpr int kStepSlots = 2;
template <int HD>
struct StepShape {
    static constexpr int HALVES = HD / 64;               // 128-byte columns of a row
    static constexpr int KEYS = 1 << kStepShift<HD>;     // of a block
    static constexpr int BOXES = KEYS / kSmallestPage;   // a box lies in one page
    static constexpr int BOX = kSmallestPage * 128;      // bytes of one box
    static constexpr int HALF = BOXES * BOX;
    static constexpr int TILE = HALVES * HALF;           // K or V of a block
    static constexpr int SLOT = 2 * TILE;
    static constexpr int RING = kStepWarps * kStepSlots * SLOT;
    static constexpr int SMEM = RING + kStepWarps * kStepSlots * 8 + kStepWarps * 16 * 8 + 1024;
};

template <int HD>
__global__ void __launch_bounds__(32 * kStepWarps)
    window_attention_step_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                                 const __grid_constant__ CUtensorMap vmap)
{
    using Sh = StepShape<HD>;
    using Pipe = WarpPipe<kStepSlots>;
    constexpr int KS = HD / 16; // products over the head's columns
    constexpr int NT = HD / 8;  // output column tiles
    extern __shared__ char smem_raw[];
    char *ring = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    uint64_t *full = reinterpret_cast<uint64_t *>(ring + Sh::RING);
    float2 *s_ml = reinterpret_cast<float2 *>(full + kStepWarps * kStepSlots);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStepWarps * kStepSlots; ++i) mbar_init(full + i, 1);
        mbar_init_fence();
    }
    grid_dependency_wait();
    allow_dependents();

    const int u = blockIdx.x % p.Hkv;
    const int s = blockIdx.x / p.Hkv, split = blockIdx.y;
    if (s == p.S) { // the block past the sequences: the tile kernel's plan
        if (u == 0 && split == 0) plan_tiles(p, *reinterpret_cast<PlanShared *>(ring));
        return;
    }
    const SeqInfo q = seq_info(p, s);
    if (q.bad && split == 0 && u == 0 && threadIdx.x == 0) set_status(p.status, kStatusIndex);
    const int R = q.n * p.g;
    if (R == 0 || R > kStepRows) return;
    const int pos0 = q.L - q.n;
    const RowRange all = rows_union(p, pos0, q.L - 1, q.L);
    const KeyBlocks<kStepShift<HD>> kb(all);
    const int per = step_split_blocks<HD>(kb.count);
    const int nsplit = max(1, (kb.count + per - 1) / per);
    if (split >= nsplit) return;
    const int b0 = split * per, b1 = min(kb.count, b0 + per);

    // the lane's two rows of the products, and its two columns of each tile
    const int r0 = lane >> 2, r1 = r0 + 8, c2 = (lane & 3) * 2;
    const RowRange rr0 = r0 < R ? row_range(p, pos0 + r0 / p.g, q.L) : RowRange{0, 0, 0};
    const RowRange rr1 = r1 < R ? row_range(p, pos0 + r1 / p.g, q.L) : RowRange{0, 0, 0};

    uint32_t qf[KS][4];
    {
        const uint32_t *qb = reinterpret_cast<const uint32_t *>(p.q);
        const int64_t a0 = ((int64_t)(q.q0 + r0 / p.g) * p.q_stride8 + (u * p.g + r0 % p.g) * (HD / 8)) * 4;
        const int64_t a1 = ((int64_t)(q.q0 + r1 / p.g) * p.q_stride8 + (u * p.g + r1 % p.g) * (HD / 8)) * 4;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const int c = k * 8 + (lane & 3);
            qf[k][0] = r0 < R ? __ldg(qb + a0 + c) : 0u;
            qf[k][1] = r1 < R ? __ldg(qb + a1 + c) : 0u;
            qf[k][2] = r0 < R ? __ldg(qb + a0 + c + 4) : 0u;
            qf[k][3] = r1 < R ? __ldg(qb + a1 + c + 4) : 0u;
        }
    }
    __syncthreads(); // barriers initialised

    char *slots = ring + warp * kStepSlots * Sh::SLOT;
    uint64_t *bar = full + warp * kStepSlots;
    const int nblk = b1 - b0 > warp ? (b1 - b0 - warp + kStepWarps - 1) / kStepWarps : 0;
    const int32_t *trow = p.table + (int64_t)s * p.table_stride;
    const int rows_total = (p.num_pages * p.Hkv) << p.page_shift; // < 2^31 (host)
    auto my_block = [&](int i) { return kb.block(b0 + warp + i * kStepWarps); };
    constexpr int ROUND = 32 / Sh::BOXES; // blocks whose rows the lanes hold
    // Lane l: first cache row of box l % BOXES of the warp's block i + l / BOXES;
    // rows_total (filled with zeros by the copy) where no query sees the box or
    // its page id is out of range.
    auto cache_rows = [&](int i) {
        i += lane / Sh::BOXES;
        if (i >= nblk) return rows_total;
        const int key = (my_block(i) << kStepShift<HD>) + lane % Sh::BOXES * kSmallestPage;
        const bool see = (all.lo < all.hi && key < all.hi && key + kSmallestPage > all.lo) || key < all.sink;
        if (!see) return rows_total;
        const int page = __ldg(trow + (key >> p.page_shift));
        if (page < 0 || page >= p.num_pages) {
            set_status(p.status, kStatusIndex);
            return rows_total;
        }
        return ((page * p.Hkv + u) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
    };
    int rows = cache_rows(0);
    auto request = [&](int i) { // the whole warp
        uint64_t *b = bar + Pipe::slot(i);
        char *dst = slots + Pipe::slot(i) * Sh::SLOT;
        if (lane == 0 && i < nblk) mbar_arrive_expect_tx(b, Sh::SLOT);
#pragma unroll
        for (int x = 0; x < Sh::BOXES; ++x) {
            const int row = __shfl_sync(kFull, rows, i % ROUND * Sh::BOXES + x);
            if (lane == 0 && i < nblk)
#pragma unroll
                for (int hf = 0; hf < Sh::HALVES; ++hf) {
                    tma_load_2d(dst + hf * Sh::HALF + x * Sh::BOX, &kmap, hf * 64, row, b);
                    tma_load_2d(dst + Sh::TILE + hf * Sh::HALF + x * Sh::BOX, &vmap, hf * 64, row, b);
                }
        }
    };
    for (int i = 0; i < kStepSlots; ++i) request(i);

    float o[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
    for (int i = 0; i < nblk; ++i) {
        if (!__all_sync(kFull, Pipe::wait(bar, i, p.limit_ns))) {
            Pipe::abort(bar, i, nblk, p.status, p.limit_ns);
            break;
        }
        char *kt = slots + Pipe::slot(i) * Sh::SLOT, *vt = kt + Sh::TILE;
        const int key0 = my_block(i) << kStepShift<HD>;
        // value rows that no query of the sequence sees may hold anything: zeros
        if (key0 + Sh::KEYS > all.hi || (key0 < all.lo && key0 + Sh::KEYS > all.sink)) {
            for (int r = lane; r < Sh::KEYS; r += 32) {
                const int key = key0 + r;
                if (key >= all.hi || (key >= all.sink && key < all.lo))
                    for (int c = 0; c < Sh::HALVES * 8; ++c)
                        *reinterpret_cast<uint4 *>(vt + (c >> 3) * Sh::HALF + r * 128 + (c & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
        }
        constexpr int KT = Sh::KEYS / 8; // score tiles of 8 keys
        float x[KT][4];                  // keys 8t + c2, +1 of rows r0 and r1
#pragma unroll
        for (int t = 0; t < KT; ++t) x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int t = 0; t < KT; t += 2) {
                // matrices: keys 8t..+7 and 8t+8..+15, columns 16k..+7 and +8..+15
                const int key = 8 * t + (lane & 7) + ((lane >> 4) << 3);
                const int chunk = (2 * k + ((lane >> 3) & 1)) & 7;
                uint32_t b[4];
                ldmatrix4(b, kt + (k >> 2) * Sh::HALF + key * 128 + ((chunk ^ (key & 7)) << 4));
                mma_bf16(x[t], qf[k], b[0], b[1]);
                mma_bf16(x[t + 1], qf[k], b[2], b[3]);
            }
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = key0 + 8 * t + c2 + (e & 1);
                const RowRange &r = e < 2 ? rr0 : rr1;
                const bool see = key < r.hi && (key < r.sink || key >= r.lo);
                x[t][e] = see ? __fmul_rn(x[t][e], p.scale_log2) : -INFINITY;
            }
        float a0 = fmaxf(x[0][0], x[0][1]), a1 = fmaxf(x[0][2], x[0][3]);
#pragma unroll
        for (int t = 1; t < KT; ++t) {
            a0 = fmaxf(fmaxf(a0, x[t][0]), x[t][1]);
            a1 = fmaxf(fmaxf(a1, x[t][2]), x[t][3]);
        }
        a0 = fmaxf(a0, __shfl_xor_sync(kFull, a0, 1));
        a1 = fmaxf(a1, __shfl_xor_sync(kFull, a1, 1));
        a0 = fmaxf(a0, __shfl_xor_sync(kFull, a0, 2));
        a1 = fmaxf(a1, __shfl_xor_sync(kFull, a1, 2));
        const float n0 = fmaxf(m0, a0), n1 = fmaxf(m1, a1);
        // a row that has seen no key yet keeps -infinity and adds zeros
        const float z0 = n0 == -INFINITY ? 0.0f : n0, z1 = n1 == -INFINITY ? 0.0f : n1;
        if (__any_sync(kFull, n0 != m0 || n1 != m1)) {
            const float f0 = exp2_fast(m0 - z0), f1 = exp2_fast(m1 - z1);
            l0 *= f0;
            l1 *= f1;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                o[n][0] *= f0;
                o[n][1] *= f0;
                o[n][2] *= f1;
                o[n][3] *= f1;
            }
            m0 = n0;
            m1 = n1;
        }
        // Probabilities, rounded to bf16 for the product with V, whose operands
        // are of one type (relative 2^-8 at most each, of either sign: against 64
        // bits outputs are off by 0.0020 to 0.0023 of their size, 0.0017 of it their
        // own rounding); the sums are of the unrounded ones, of this lane's keys
        // (the quad's are added at the end).
#pragma unroll
        for (int t = 0; t < KT; t += 2) {
            float e0[4], e1[4]; // keys 8t + c2, +1 and 8t + 8 + c2, +1
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    e0[2 * i + e] = exp2_fast(x[t + i][e] - z0);
                    e1[2 * i + e] = exp2_fast(x[t + i][2 + e] - z1);
                }
            l0 += (e0[0] + e0[1]) + (e0[2] + e0[3]);
            l1 += (e1[0] + e1[1]) + (e1[2] + e1[3]);
            const uint32_t pf[4] = {pack_bf16(e0[0], e0[1]), pack_bf16(e1[0], e1[1]),
                                    pack_bf16(e0[2], e0[3]), pack_bf16(e1[2], e1[3])};
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                // matrices: keys 8t..+7 and 8t+8..+15 of columns 8n..+7, then of 8n+8..+15
                const int key = 8 * t + (lane & 15), chunk = (n + (lane >> 4)) & 7;
                uint32_t b[4];
                ldmatrix4_trans(b, vt + (n >> 3) * Sh::HALF + key * 128 + ((chunk ^ (key & 7)) << 4));
                mma_bf16(o[n], pf, b[0], b[1]);
                mma_bf16(o[n + 1], pf, b[2], b[3]);
            }
        }
        slot_reads_done();
        const int nx = i + kStepSlots;
        if (nx % ROUND == 0) rows = cache_rows(nx);
        request(nx);
    }
    l0 += __shfl_xor_sync(kFull, l0, 1);
    l1 += __shfl_xor_sync(kFull, l1, 1);
    l0 += __shfl_xor_sync(kFull, l0, 2);
    l1 += __shfl_xor_sync(kFull, l1, 2);

    // Join the warps in shared memory, in warp order: each puts its output in
    // its own ring (its copies have all landed), [row][column] fp32.
    __syncwarp();
    float *mine = reinterpret_cast<float *>(slots);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        *reinterpret_cast<float2 *>(mine + r0 * HD + 8 * n + c2) = make_float2(o[n][0], o[n][1]);
        *reinterpret_cast<float2 *>(mine + r1 * HD + 8 * n + c2) = make_float2(o[n][2], o[n][3]);
    }
    if ((lane & 3) == 0) {
        s_ml[warp * 16 + r0] = make_float2(m0, l0);
        s_ml[warp * 16 + r1] = make_float2(m1, l1);
    }
    __syncthreads();
    constexpr int CT = HD / 4; // threads of a row, four columns each
    const int64_t base = part_base(p, p.step_part, s, q, u) + (int64_t)split * R;
    for (int r = threadIdx.x / CT; r < R; r += 32 * kStepWarps / CT) {
        const int c = (threadIdx.x % CT) * 4;
        float m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int w = 0; w < kStepWarps; ++w) m = fmaxf(m, s_ml[w * 16 + r].x);
        const float z = m == -INFINITY ? 0.0f : m;
        float4 a = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int w = 0; w < kStepWarps; ++w) {
            const float2 ml = s_ml[w * 16 + r];
            const float f = exp2_fast(ml.x - z);
            const float4 v = *reinterpret_cast<const float4 *>(
                reinterpret_cast<const float *>(ring + w * kStepSlots * Sh::SLOT) + r * HD + c);
            l = fmaf(f, ml.y, l);
            a.x = fmaf(f, v.x, a.x);
            a.y = fmaf(f, v.y, a.y);
            a.z = fmaf(f, v.z, a.z);
            a.w = fmaf(f, v.w, a.w);
        }
        if (nsplit == 1) {
            write_row<HD>(p, q.q0 + r / p.g, u * p.g + r % p.g, c, a, m, l);
        } else {
            *reinterpret_cast<float4 *>(p.part_o + (base + r) * HD + c) = a;
            if (c == 0) p.part_ml[base + r] = make_float2(m, l);
        }
    }
}

// Join one row's split results, in split order: HD / 4 threads, four columns
// each.
template <int HD>
__device__ __forceinline__ void join_row(const AttnParams &p, const PartRoom &room, int s, const SeqInfo &q,
                                         int u, int r, int nsplit, int c)
{
    const int R = q.n * p.g;
    const int64_t base = part_base(p, room, s, q, u) + r;
    float m = -INFINITY;
#pragma unroll 4
    for (int k = 0; k < nsplit; ++k) m = fmaxf(m, p.part_ml[base + (int64_t)k * R].x);
    const float z = m == -INFINITY ? 0.0f : m;
    float l = 0.0f;
    float4 a = make_float4(0, 0, 0, 0);
#pragma unroll 4
    for (int k = 0; k < nsplit; ++k) {
        const float2 ml = p.part_ml[base + (int64_t)k * R];
        const float4 v = *reinterpret_cast<const float4 *>(p.part_o + (base + (int64_t)k * R) * HD + c);
        const float f = exp2_fast(ml.x - z);
        l = fmaf(f, ml.y, l);
        a.x = fmaf(f, v.x, a.x);
        a.y = fmaf(f, v.y, a.y);
        a.z = fmaf(f, v.z, a.z);
        a.w = fmaf(f, v.w, a.w);
    }
    write_row<HD>(p, q.q0 + r / p.g, u * p.g + r % p.g, c, a, m, l);
}

constexpr int kJoinThreads = 128;

// The first step_blocks blocks take the rows of a (sequence, key head) of the
// step kernel each; the others the split tiles of the tile kernel.
template <int HD>
__global__ void __launch_bounds__(kJoinThreads) window_attention_join_kernel(const AttnParams p, int step_blocks)
{
    constexpr int CT = HD / 4, RB = kJoinThreads / CT; // threads of a row, rows of a block
    grid_dependency_wait();
    allow_dependents();
    const int br = threadIdx.x / CT, c = threadIdx.x % CT * 4;
    if ((int)blockIdx.x < step_blocks) {
        const int u = blockIdx.x % p.Hkv, s = blockIdx.x / p.Hkv;
        const SeqInfo q = seq_info(p, s);
        const int R = q.n * p.g;
        if (R > kStepRows) return;
        const KeyBlocks<kStepShift<HD>> kb(rows_union(p, q.L - q.n, q.L - 1, q.L));
        const int per = step_split_blocks<HD>(kb.count);
        const int nsplit = (kb.count + per - 1) / per;
        if (nsplit > 1)
            for (int r = br; r < R; r += RB) join_row<HD>(p, p.step_part, s, q, u, r, nsplit, c);
        return;
    }
    constexpr int TB = kTileRows / RB; // blocks of a tile's rows
    const int64_t work = (int64_t)p.plan_head[1] * p.Hkv * TB;
    for (int64_t w = blockIdx.x - step_blocks; w < work; w += gridDim.x - step_blocks) {
        const int2 st = p.split_tiles[w / TB / p.Hkv];
        if (st.x < 0) continue;
        const int u = (int)(w / TB % p.Hkv);
        const SeqInfo q = seq_info(p, st.x);
        const int rows = tile_tokens(p.g) * p.g, rt = (int)(w % TB) * RB + br, r = st.y * rows + rt;
        if (rt >= rows || r >= q.n * p.g) continue;
        const int count = KeyBlocks<7>(tile_union(p, q, st.y)).count;
        const int per = tile_split_blocks(p, seq_tiles(p, q), count);
        join_row<HD>(p, p.tile_part, st.x, q, u, r, (count + per - 1) / per, c);
    }
}

namespace {

template <int HD>
cudaError_t launch_step_hd(const AttnParams &p, const CUtensorMap &kmap, const CUtensorMap &vmap,
                           int splits, bool plan, cudaStream_t s)
{
    static_assert(32 * kStepWarps == kPlanThreads && sizeof(PlanShared) <= StepShape<HD>::RING, "plan");
    return launch_overlapped_2d(window_attention_step_kernel<HD>,
                                dim3((unsigned)(p.S * p.Hkv + (plan ? 1 : 0)), (unsigned)splits),
                                32 * kStepWarps, StepShape<HD>::SMEM, s, p, kmap, vmap);
}

template <int HD>
cudaError_t launch_join_hd(const AttnParams &p, bool tiles, cudaStream_t s)
{
    const int64_t step = (int64_t)p.S * p.Hkv;
    const int64_t grid = step + (tiles ? 12 * sm_count() : 0);
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return launch_overlapped_2d(window_attention_join_kernel<HD>, dim3((unsigned)grid), kJoinThreads, 0, s, p,
                                (int)step);
}

} // namespace

cudaError_t ready_attention_step(int head_dim)
{
    return head_dim == 64 ? allow_dynamic_smem(reinterpret_cast<const void *>(window_attention_step_kernel<64>),
                                               StepShape<64>::SMEM)
                          : allow_dynamic_smem(reinterpret_cast<const void *>(window_attention_step_kernel<128>),
                                               StepShape<128>::SMEM);
}

cudaError_t launch_attention_step(const AttnParams &p, int head_dim, const CUtensorMap &kmap,
                                  const CUtensorMap &vmap, int splits, bool plan, cudaStream_t s)
{
    return head_dim == 64 ? launch_step_hd<64>(p, kmap, vmap, splits, plan, s)
                          : launch_step_hd<128>(p, kmap, vmap, splits, plan, s);
}

cudaError_t launch_attention_join(const AttnParams &p, int head_dim, bool tiles, cudaStream_t s)
{
    return head_dim == 64 ? launch_join_hd<64>(p, tiles, s) : launch_join_hd<128>(p, tiles, s);
}

} // namespace dan
