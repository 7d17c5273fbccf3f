// dan_attn.cuh -- what the paged-cache operators share: their problems as
// the shim validated them, which keys a query row sees, how a sequence's
// keys are split, and the partial results of the splits.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dan {

constexpr unsigned kStatusIndex = 8u; // an index in a caller's array was out of its range

constexpr int kSmallestPage = 16;

inline int page_shift(int64_t page_size)
{
    int s = 0;
    while ((int64_t(1) << s) < page_size) ++s;
    return s;
}

struct CacheRopeProblem {
    const void *q, *k, *v;
    int64_t N, q_stride, kv_stride, heads, kv_heads, head_dim;
    const void *wq, *wk;
    const float *rope;
    int64_t table_rows;
    const int32_t *positions, *slots;
    float eps;
    bool neox;
    void *q_out;
    int64_t qo_stride;
    void *k_cache, *v_cache;
    int64_t num_pages, page_size;
};

struct AttnProblem {
    const void *q;
    int64_t N, q_stride;
    const void *k_cache, *v_cache;
    int64_t num_pages, page_size;
    const int32_t *page_table;
    int64_t table_stride, max_pages;
    const int32_t *q_start, *kv_len;
    int64_t S, heads, kv_heads, head_dim, window, sinks, chunk, max_q;
    float scale;
    void *out;
    float *lse;
    void *workspace;
};

cudaError_t launch_qk_norm_rope_cache(const CacheRopeProblem &p, cudaStream_t s);
cudaError_t launch_window_attention(const AttnProblem &p, cudaStream_t s);
int64_t window_attention_workspace(const AttnProblem &p); // its sizes alone

// Launch with programmatic stream serialization (see launch_overlapped) on a
// two-dimensional grid.
template <typename... KArgs, typename... Args>
cudaError_t launch_overlapped_2d(void (*fn)(KArgs...), dim3 grid, int block, int smem,
                                 cudaStream_t s, const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

// ----------------------------------------------------------- device side

// One piece of work of the tile kernel: a split of the keys of a tile of
// query tokens, for one key head.
struct __align__(16) TileItem {
    int s, u, split, nsplit; // sequence, key head (set when taken); s < 0: none
    int q0, n, L, tok0;      // the sequence; the tile's first token in it
    int ntok, b0, b1, pos0;  // tokens of the tile, its split's key blocks, first query's position
    int sink, lo, hi, nsink; // keys that some row sees, blocks of the sinks
    int first, pad[3];       // first block of the window

    // first key of block j
    __host__ __device__ int key_of(int j) const { return (j < nsink ? j : j - nsink + first) << 7; }
};

// Where the partial results of a kernel's split sequences lie in the workspace,
// in rows from `first`: `cap` rows for each (sequence, key head) or, with cap 0,
// `splits` rows for each row of a query head.
struct PartRoom {
    int64_t first, cap;
    int splits;
};

struct AttnParams {
    const uint4 *q;
    int64_t N, q_stride8; // query row stride in 16-byte fragments
    const int32_t *table;
    int64_t table_stride;
    int max_pages, num_pages, page_shift;
    const int32_t *q_start, *kv_len;
    int S, H, Hkv, g; // g = H / Hkv query heads share a key head
    int window, sinks, chunk;
    int max_q;
    float scale_log2; // scale * log2(e): the softmax is taken in base 2
    uint4 *out;
    float *lse;
    // partial results: rows of outputs, and of (maximum, sum)
    float *part_o;
    float2 *part_ml;
    PartRoom step_part, tile_part;
    // work of the tile kernel (see its plan)
    TileItem *items;
    int2 *split_tiles;
    int *plan_head;
    int items_cap, split_tiles_cap;
    unsigned *status;
    unsigned long long limit_ns;
};

// A sequence as the arrays say it, with what is out of range cut off; n == 0
// where nothing is to be done.
struct SeqInfo {
    int q0, n, L;
    bool bad;  // an entry was out of its range
    bool down; // its start lies past the next one's
};

__device__ __forceinline__ SeqInfo seq_info(const AttnParams &p, int s)
{
    SeqInfo q;
    const int a = __ldg(p.q_start + s), b = __ldg(p.q_start + s + 1);
    int L = __ldg(p.kv_len + s);
    const int cap = p.max_pages << p.page_shift;
    q.bad = L < 0 || L > cap;
    q.L = L < 0 ? 0 : L > cap ? cap : L;
    q.q0 = a;
    q.n = b - a;
    q.down = b < a;
    if (a < 0 || b < a || b > p.N || q.n > p.max_q) {
        q.bad = true;
        q.n = 0;
    }
    return q;
}

// Keys that the query at position `pos` sees: [0, sink) and [lo, hi).
struct RowRange {
    int sink, lo, hi;
};

__device__ __forceinline__ RowRange row_range(const AttnParams &p, int pos, int L)
{
    RowRange r = {0, 0, 0};
    if (pos < 0) return r;
    const int p0 = pos - pos % p.chunk;
    r.hi = min(L, p0 + p.chunk);
    r.sink = min(p.sinks, r.hi);
    r.lo = p.window ? min(r.hi, max(0, p0 + 1 - p.window)) : r.hi;
    return r;
}

// Keys that some query at positions first..last of one sequence sees.  The
// ranges of successive positions overlap or touch (lo never passes the
// previous hi when there is a window), so their union is again [0, sink) and
// [lo, hi).
__device__ __forceinline__ RowRange rows_union(const AttnParams &p, int first, int last, int L)
{
    if (last < 0) return RowRange{0, 0, 0};
    RowRange r = row_range(p, last, L);
    if (p.window) r.lo = row_range(p, max(first, 0), L).lo;
    return r;
}

// The union's keys in blocks of 2^SHIFT, each block once: the sinks' blocks
// from 0, then the window's.
template <int SHIFT>
struct KeyBlocks {
    int nsink, first, count; // block i is i < nsink ? i : i - nsink + first
    __device__ __forceinline__ explicit KeyBlocks(const RowRange &r)
    {
        constexpr int M = (1 << SHIFT) - 1;
        nsink = (r.sink + M) >> SHIFT;
        first = max(r.lo >> SHIFT, nsink);
        const int end = r.lo < r.hi ? (r.hi + M) >> SHIFT : 0;
        count = nsink + max(0, end - first);
    }
    __device__ __forceinline__ int block(int i) const { return i < nsink ? i : i - nsink + first; }
};

// How a step sequence's keys are split: by its own number of blocks alone, so
// that a row's bits do not depend on the batch, and never more than 32 ways.
// At head_dim 64 splits have 768 keys at least, at 128 they have 512, or down
// to 256 where that makes at most nine.  Measured (replayed, keys not in L2): at
// head_dim 64, 96 sequences of up to 2112 visible keys take 81 us with splits of
// 512 keys at least, 75 with 768 and 74 with 1024, one sequence of 1028 keys
// 9.5, 10.9 and 12.9.  At head_dim 128 one sequence of 1028 keys takes 10.2 us
// with 256 and 12.1 with 512, eight of up to 4216 take 23.5 and 22.8.
constexpr int kStepRows = 16;     // query rows (tokens x g) that the step kernel takes
constexpr int kMaxSplits = 32;
template <int HD>
constexpr int kStepShift = HD == 64 ? 5 : 4; // its key blocks: 32 or 16 keys, 4 KB of each cache
template <int HD>
constexpr int kStepBlocks = 512 >> kStepShift<HD>;
template <int HD>
constexpr int kStepMinBlocks = HD == 64 ? kStepBlocks<HD> * 3 / 2 : kStepBlocks<HD> / 2;

template <int HD>
__device__ __forceinline__ int step_split_blocks(int count)
{
    return max(max(kStepMinBlocks<HD>, min(count / 8, kStepBlocks<HD>)), (count + kMaxSplits - 1) / kMaxSplits);
}

// First partial row of (sequence, key head); its rows are [split][row].
__device__ __forceinline__ int64_t part_base(const AttnParams &p, const PartRoom &room, int s,
                                             const SeqInfo &q, int u)
{
    if (room.cap) return room.first + ((int64_t)s * p.Hkv + u) * room.cap;
    return room.first + ((int64_t)q.q0 * p.H + (int64_t)u * q.n * p.g) * room.splits;
}

// The tile kernel's rows: two row tiles of 128 / g whole tokens each, at most
// 256 (token, query head) rows.
constexpr int kTileRows = 256;
constexpr int kMaxGroup = 128; // most query heads of a key head
constexpr int kPlanBuckets = 2048;

__host__ __device__ __forceinline__ int tile_tokens(int g) { return 2 * (128 / g); }

// Keys that some row of a tile sees:
__device__ __forceinline__ RowRange tile_union(const AttnParams &p, const SeqInfo &q, int tile)
{
    const int nt = tile_tokens(p.g), first = tile * nt, end = min(q.n, first + nt), pos0 = q.L - q.n;
    return rows_union(p, pos0 + first, pos0 + end - 1, q.L);
}

__device__ __forceinline__ int seq_tiles(const AttnParams &p, const SeqInfo &q)
{
    const int nt = tile_tokens(p.g);
    return (q.n + nt - 1) / nt;
}

// Key blocks (128 keys) of a split of a tile that sees `count` of them, in a
// sequence of `tiles` tiles: split only where the sequence alone has fewer
// than half of kTileSplitTarget items, and not below 8 blocks.
constexpr int kTileSplitTarget = 64;
constexpr int kTileMaxSplits = 16;
constexpr int kTileMinBlocks = 8;

__device__ __forceinline__ int tile_split_blocks(const AttnParams &p, int tiles, int count)
{
    const int64_t items = (int64_t)tiles * p.Hkv;
    int n = items > kTileSplitTarget ? 1 : min(kTileMaxSplits, kTileSplitTarget / (int)items);
    n = min(n, count / kTileMinBlocks);
    return n <= 1 ? max(1, count) : (count + n - 1) / n;
}

// What the step and the tile kernel need before their first launch on the
// current device.  A call asks for all that it will launch before its first
// launch: one that cannot run whole writes nothing.
cudaError_t ready_attention_step(int head_dim);
cudaError_t ready_attention_tile(int head_dim);

// Launch one kernel each: sequences of at most kStepRows rows, split at most
// `splits` ways (and the plan of the others); the others; the join of splits.
cudaError_t launch_attention_step(const AttnParams &p, int head_dim, const CUtensorMap &kmap,
                                  const CUtensorMap &vmap, int splits, bool plan, cudaStream_t s);
cudaError_t launch_attention_tile(const AttnParams &p, int head_dim, const CUtensorMap &qmap,
                                  const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t s);
cudaError_t launch_attention_join(const AttnParams &p, int head_dim, bool tiles, cudaStream_t s);

} // namespace dan
