// dan_cache_abi.cu -- the extern "C" boundary of the paged-cache operators
// (include/dan_cache.h): argument validation, tensor maps, launches.
#include "../../include/dan_cache.h"
#include "dan_attn.cuh"
#include "dan_internal.h"

#include <cmath>
#include <mutex>

namespace dan {
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once (the library does not link
// the driver, so that it loads on machines without one).
EncodeTiled encode_tiled()
{
    static std::mutex mu;
    static EncodeTiled fn = nullptr;
    std::lock_guard<std::mutex> lk(mu);
    if (!fn) {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &found) == cudaSuccess &&
            found == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(ptr);
    }
    return fn;
}

// A cache as a matrix of `rows` token rows of one head, read in boxes of 64
// columns x box_rows tokens with the 128-byte swizzle.
bool cache_map(CUtensorMap *map, const void *cache, int64_t rows, int64_t hd, int box_rows)
{
    const EncodeTiled enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)hd, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)hd * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    const cuuint32_t step[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(cache), dims, strides, box,
               step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as [token][head][column], read in boxes of the 128 / g tokens by
// g heads of a row tile, 64 columns each.
bool query_map(CUtensorMap *map, const AttnProblem &a, int g)
{
    const EncodeTiled enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.heads, (cuuint64_t)a.N};
    const cuuint64_t strides[2] = {(cuuint64_t)a.head_dim * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)g, (cuuint32_t)(128 / g)};
    const cuuint32_t step[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q), dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Most splits that a step sequence that sees at most `keys` keys can have.
int step_splits(int64_t keys, int64_t head_dim)
{
    // the first tokens' last block and the window's first and last may be partly seen
    const int64_t blocks = (keys >> (head_dim == 64 ? kStepShift<64> : kStepShift<128>)) + 3;
    const int64_t least = head_dim == 64 ? kStepMinBlocks<64> : kStepMinBlocks<128>;
    const int64_t n = (blocks + least - 1) / least;
    return (int)(n < kMaxSplits ? n : kMaxSplits);
}

// Keys that `tokens` successive tokens of a sequence can see together: the
// first ones, and their windows and chunks.
int64_t keys_seen(const AttnProblem &a, int64_t tokens)
{
    const int64_t seen = a.sinks + (a.window ? a.window + 2 * a.chunk + tokens : 0);
    const int64_t cap = a.max_pages * a.page_size;
    return seen < cap ? seen : cap;
}

// Most splits that a tile of the tile kernel can have.
int tile_splits(int64_t keys, int64_t kv_heads)
{
    const int64_t n = kTileSplitTarget / kv_heads, blocks = keys / 128 + 3;
    const int64_t most = blocks / kTileMinBlocks < kTileMaxSplits ? blocks / kTileMinBlocks : kTileMaxSplits;
    return (int)(n < most ? (n < 1 ? 1 : n) : most < 1 ? 1 : most);
}

// Most partial rows of a (sequence, key head) that the tile kernel splits, whose
// sequence has `tiles` tiles: a tile's splits are as many as the items allow.
int64_t tile_part_rows(int64_t tiles, int64_t g, int64_t kv_heads, int64_t max_q, int most)
{
    const int64_t n = kTileSplitTarget / (tiles * kv_heads), splits = n < most ? n : most;
    const int64_t tokens = tiles * tile_tokens((int)g);
    return splits > 1 ? (tokens < max_q ? tokens : max_q) * g * splits : 0;
}

// What a call needs of the workspace: partial results of splits, and the tile
// kernel's work lists.  Partial results have room by (sequence, key head) or
// by query row, whichever is least: the same for both kernels, as a sequence
// is one kernel's alone, or the step kernel's by sequence (it takes 16 rows of
// one at most) and after it the tile kernel's by row (it splits less).  At 32
// query and 8 key heads of 128 over a table of 32768 keys, 256 sequences with
// 4096 rows: 1040 MiB, one room for both 2080; 64 single tokens: 32 MiB.
struct Room {
    int step_splits = 1, tile_splits = 1; // most splits of a sequence of either kernel
    bool tiles = false; // a sequence may have more rows than the step kernel takes
    PartRoom step = {}, tile = {};
    int64_t part_rows = 0, items = 0, split_tiles = 0;
    int64_t part_bytes = 0, bytes = 0;
};

Room room_for(const AttnProblem &a)
{
    Room r;
    if (a.N == 0 || a.S == 0) return r;
    const int64_t g = a.heads / a.kv_heads, max_q = a.max_q < a.N ? a.max_q : a.N;
    // rows of a step sequence's key head
    const int64_t step_rows = kStepRows / g < max_q ? kStepRows / g * g : max_q * g;
    if (step_rows) r.step_splits = step_splits(keys_seen(a, kStepRows), a.head_dim);
    const int64_t step_cap = r.step_splits > 1 ? step_rows * r.step_splits : 0;
    r.tiles = max_q * g > kStepRows;
    int64_t tile_cap = 0;
    if (r.tiles) {
        // sequences that the tile kernel takes, and the tiles of one that may be split
        const int64_t long_seqs = a.S < a.N * g / kStepRows ? a.S : a.N * g / kStepRows;
        const int64_t split_target = kTileSplitTarget / a.kv_heads;
        r.items = a.N / tile_tokens((int)g) + long_seqs * (1 + split_target);
        r.split_tiles = long_seqs * (1 + split_target / 2);
        r.tile_splits = tile_splits(keys_seen(a, kTileRows), a.kv_heads);
        for (int64_t t = 1; t <= split_target / 2 && (t - 1) * tile_tokens((int)g) < max_q; ++t) {
            const int64_t rows = tile_part_rows(t, g, a.kv_heads, max_q, r.tile_splits);
            if (rows > tile_cap) tile_cap = rows;
        }
        if (!tile_cap) r.tile_splits = 1;
    }
    const int64_t seqs = a.S * a.kv_heads, rows = a.N * a.heads;
    const int64_t cap = step_cap > tile_cap ? step_cap : tile_cap;
    const int splits = r.step_splits > r.tile_splits ? r.step_splits : r.tile_splits;
    const int64_t by_seq = seqs * cap, by_row = splits > 1 ? rows * splits : 0;
    const int64_t apart = seqs * step_cap + rows * r.tile_splits;
    r.part_rows = by_seq < by_row ? by_seq : by_row;
    if (step_cap && tile_cap && apart < r.part_rows) {
        r.step = {0, step_cap, r.step_splits};
        r.tile = {seqs * step_cap, 0, r.tile_splits};
        r.part_rows = apart;
    } else {
        r.step = r.tile = {0, by_seq < by_row ? cap : 0, splits};
    }
    r.part_bytes = (r.part_rows * (a.head_dim * 4 + 8) + 15) / 16 * 16;
    r.bytes = r.part_bytes + (r.tiles ? 16 + (int64_t)sizeof(TileItem) * r.items + 8 * r.split_tiles : 0);
    return r;
}

} // namespace

int64_t window_attention_workspace(const AttnProblem &a) { return room_for(a).bytes; }

cudaError_t launch_window_attention(const AttnProblem &a, cudaStream_t s)
{
    AttnParams p = {};
    p.q = static_cast<const uint4 *>(a.q);
    p.N = a.N;
    p.q_stride8 = a.q_stride / 8;
    p.table = a.page_table;
    p.table_stride = a.table_stride;
    p.max_pages = (int)a.max_pages;
    p.num_pages = (int)a.num_pages;
    p.page_shift = page_shift(a.page_size);
    p.q_start = a.q_start;
    p.kv_len = a.kv_len;
    p.S = (int)a.S;
    p.H = (int)a.heads;
    p.Hkv = (int)a.kv_heads;
    p.g = (int)(a.heads / a.kv_heads);
    const int64_t big = int64_t(1) << 30; // past every position
    p.window = (int)(a.window < big ? a.window : big);
    p.sinks = (int)(a.sinks < big ? a.sinks : big);
    p.chunk = (int)(a.chunk < big ? a.chunk : big);
    p.max_q = (int)(a.max_q < a.N ? a.max_q : a.N);
    p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
    p.out = static_cast<uint4 *>(a.out);
    p.lse = a.lse;
    const Room room = room_for(a);
    if (room.items > 0x7FFFFFFF || room.split_tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
    p.part_o = static_cast<float *>(a.workspace);
    p.part_ml = reinterpret_cast<float2 *>(p.part_o + room.part_rows * a.head_dim);
    p.step_part = room.step;
    p.tile_part = room.tile;
    p.plan_head = reinterpret_cast<int *>(static_cast<char *>(a.workspace) + room.part_bytes);
    p.items = reinterpret_cast<TileItem *>(p.plan_head + 4);
    p.split_tiles = reinterpret_cast<int2 *>(p.items + room.items);
    p.items_cap = (int)room.items;
    p.split_tiles_cap = (int)room.split_tiles;
    p.status = device_status();
    // a second, and what an item with every key of the table takes: some waits are
    // for a whole item (a block of 128 keys takes about 1.4 us)
    p.limit_ns = 1000000000ull + 30ull * (unsigned long long)(a.max_pages * a.page_size);
    const int64_t rows = a.num_pages * a.kv_heads * a.page_size;
    const int hd = (int)a.head_dim, box = (int)(a.page_size < 128 ? a.page_size : 128);
    CUtensorMap kmap, vmap, tile_q, tile_k, tile_v;
    cudaError_t e = ready_attention_step(hd);
    if (e == cudaSuccess && room.tiles) e = ready_attention_tile(hd);
    if (e != cudaSuccess) return e;
    if (!cache_map(&kmap, a.k_cache, rows, hd, kSmallestPage) ||
        !cache_map(&vmap, a.v_cache, rows, hd, kSmallestPage) ||
        (room.tiles && (!query_map(&tile_q, a, p.g) || !cache_map(&tile_k, a.k_cache, rows, hd, box) ||
                        !cache_map(&tile_v, a.v_cache, rows, hd, box))))
        return cudaErrorInvalidValue;
    e = launch_attention_step(p, hd, kmap, vmap, room.step_splits, room.tiles, s);
    if (e == cudaSuccess && room.tiles) e = launch_attention_tile(p, hd, tile_q, tile_k, tile_v, s);
    if (e != cudaSuccess || room.part_rows == 0) return e;
    return launch_attention_join(p, hd, room.tiles, s);
}

} // namespace dan

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxCacheRows = (int64_t(1) << 31) - 256;
constexpr int64_t kMaxInt = 0x7FFFFFFF;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Range {
    uintptr_t lo, hi;
    Range(const void *p, int64_t bytes)
        : lo(reinterpret_cast<uintptr_t>(p)), hi(lo + static_cast<uintptr_t>(bytes))
    {
    }
};

bool overlap(const Range &a, const Range &b)
{
    return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

// Shared checks of sizes: heads, head_dim, pages.
int check_cache(int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t num_pages,
                int64_t page_size)
{
    if (head_dim != 64 && head_dim != 128) return DAN_EUNSUPPORTED;
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
        return DAN_EUNSUPPORTED;
    if (heads < 1 || kv_heads < 1 || num_pages < 1 || heads % kv_heads) return DAN_EINVAL;
    if (heads > 1024) return DAN_EUNSUPPORTED;
    if (num_pages > kMaxCacheRows / (kv_heads * page_size)) return DAN_EUNSUPPORTED;
    return DAN_OK;
}

// Bytes of N rows of `width` elements at `stride`; -1 if out of bounds.
int64_t rows_bytes(int64_t N, int64_t width, int64_t stride)
{
    if (stride < width || stride > kMaxElems || N > kMaxElems / stride) return -1;
    return ((N - 1) * stride + width) * 2;
}

int validate_rope(const dan_bf16 *q, const dan_bf16 *k, const dan_bf16 *v, int64_t N,
                  int64_t q_row_stride, int64_t kv_row_stride, int64_t heads, int64_t kv_heads,
                  int64_t hd, const dan_bf16 *wq, const dan_bf16 *wk, const float *rope,
                  int64_t table_rows, const int32_t *positions, const int32_t *slots, float eps,
                  const dan_bf16 *q_out, int64_t qo_row_stride, const dan_bf16 *k_cache,
                  const dan_bf16 *v_cache, int64_t num_pages, int64_t page_size)
{
    const int st = check_cache(heads, kv_heads, hd, num_pages, page_size);
    if (st != DAN_OK) return st;
    if (N < 0 || table_rows < 1 || table_rows > kMaxInt || !std::isfinite(eps) || eps < 0.0f)
        return DAN_EINVAL;
    if (N == 0) return DAN_OK;
    const int64_t qb = rows_bytes(N, heads * hd, q_row_stride);
    const int64_t kb = rows_bytes(N, kv_heads * hd, kv_row_stride);
    const int64_t ob = rows_bytes(N, heads * hd, qo_row_stride);
    if (qb < 0 || kb < 0 || ob < 0) return DAN_EINVAL;
    if (!q || !k || !v || !wq || !wk || !rope || !positions || !slots || !q_out || !k_cache || !v_cache)
        return DAN_EINVAL;
    const void *p16[] = {q, k, v, wq, wk, rope, q_out, k_cache, v_cache};
    for (const void *p : p16)
        if (!aligned(p, 16)) return DAN_EALIGN;
    if (!aligned(positions, 4) || !aligned(slots, 4)) return DAN_EALIGN;
    if (q_row_stride % 8 || kv_row_stride % 8 || qo_row_stride % 8) return DAN_EALIGN;
    const int64_t cb = num_pages * kv_heads * page_size * hd * 2;
    const Range outs[] = {{q_out, ob}, {k_cache, cb}, {v_cache, cb}};
    const Range ins[] = {{q, qb},         {k, kb},          {v, kb},        {wq, hd * 2},
                         {wk, hd * 2},    {rope, table_rows * hd * 4}, {positions, N * 4}, {slots, N * 4}};
    const bool in_place = q_out == q && qo_row_stride == q_row_stride;
    for (int o = 0; o < 3; ++o) {
        for (int i = 0; i < 8; ++i) {
            if (o == 0 && i == 0 && in_place) continue;
            // the columns of one packed buffer, in any order: in-place q rows lie beside
            // k and v rows of the same stride
            if (o == 0 && in_place && (i == 1 || i == 2) && q_row_stride == kv_row_stride) {
                const uintptr_t row = (uintptr_t)(heads * hd * 2), krow = (uintptr_t)(kv_heads * hd * 2);
                const uintptr_t step = (uintptr_t)q_row_stride * 2;
                const uintptr_t at = ins[i].lo >= outs[0].lo // where k's rows begin behind q's, below step
                                         ? (ins[i].lo - outs[0].lo) % step
                                         : (step - (outs[0].lo - ins[i].lo) % step) % step;
                if (at >= row && at + krow <= step) continue;
            }
            if (overlap(outs[o], ins[i])) return DAN_EALIAS;
        }
        for (int o2 = o + 1; o2 < 3; ++o2)
            if (overlap(outs[o], outs[o2])) return DAN_EALIAS;
    }
    return DAN_OK;
}

int validate_attention(const dan_bf16 *q, int64_t N, int64_t q_row_stride, const dan_bf16 *k_cache,
                       const dan_bf16 *v_cache, int64_t num_pages, int64_t page_size,
                       const int32_t *page_table, int64_t table_stride, int64_t max_pages,
                       const int32_t *q_start, const int32_t *kv_len, int64_t S, int64_t heads,
                       int64_t kv_heads, int64_t hd, int64_t window, int64_t sinks, int64_t chunk,
                       int64_t max_q, float scale, const dan_bf16 *out, const float *lse,
                       const void *workspace, int64_t workspace_bytes)
{
    const int st = check_cache(heads, kv_heads, hd, num_pages, page_size);
    if (st != DAN_OK) return st;
    if (N < 0 || S < 0 || max_pages < 1 || max_q < 0) return DAN_EINVAL;
    if (window < 0 || window > kMaxInt || sinks < 0 || sinks > kMaxInt || chunk < 1 || chunk > kMaxInt)
        return DAN_EINVAL;
    if (!std::isfinite(scale) || scale <= 0.0f) return DAN_EINVAL;
    if (heads / kv_heads > dan::kMaxGroup || q_row_stride >= (int64_t(1) << 39)) return DAN_EUNSUPPORTED;
    if (N > (int64_t(1) << 30) || S > (int64_t(1) << 20) ||
        N > (int64_t(1) << 30) / heads || max_pages > (int64_t(1) << 30) / page_size)
        return DAN_EUNSUPPORTED;
    if (N == 0 || S == 0) return DAN_OK;
    if (table_stride < max_pages || table_stride > kMaxElems / S) return DAN_EINVAL;
    const int64_t qb = rows_bytes(N, heads * hd, q_row_stride);
    if (qb < 0) return DAN_EINVAL;
    if (!q || !k_cache || !v_cache || !page_table || !q_start || !kv_len || !out) return DAN_EINVAL;
    const int64_t need = dan_window_attention_workspace(N, S, heads, kv_heads, hd, max_pages, page_size,
                                                        window, sinks, chunk, max_q);
    if (workspace_bytes < need || (need > 0 && !workspace)) return DAN_EINVAL;
    const void *p16[] = {q, k_cache, v_cache, out, workspace};
    for (const void *p : p16)
        if (!aligned(p, 16)) return DAN_EALIGN;
    const void *p4[] = {page_table, q_start, kv_len, lse};
    for (const void *p : p4)
        if (!aligned(p, 4)) return DAN_EALIGN;
    if (q_row_stride % 8) return DAN_EALIGN;
    const int64_t cb = num_pages * kv_heads * page_size * hd * 2;
    const Range outs[] = {{out, N * heads * hd * 2},
                          {lse, lse ? N * heads * 4 : 0},
                          {workspace, need}};
    const Range ins[] = {{q, qb},
                         {k_cache, cb},
                         {v_cache, cb},
                         {page_table, ((S - 1) * table_stride + max_pages) * 4},
                         {q_start, (S + 1) * 4},
                         {kv_len, S * 4}};
    for (int o = 0; o < 3; ++o) {
        for (const Range &in : ins)
            if (overlap(outs[o], in)) return DAN_EALIAS;
        for (int o2 = o + 1; o2 < 3; ++o2)
            if (overlap(outs[o], outs[o2])) return DAN_EALIAS;
    }
    return DAN_OK;
}

// A launch's status.  What it keeps on the host (a map, a lock) may throw, and
// no exception may pass the C boundary.
template <typename F>
int status_of(F launch)
{
    try {
        return launch() == cudaSuccess ? DAN_OK : DAN_ECUDA;
    } catch (...) {
        return DAN_ECUDA;
    }
}

} // namespace

extern "C" {

int dan_can_use_qk_norm_rope_cache(const dan_bf16 *q, const dan_bf16 *k, const dan_bf16 *v,
                                   int64_t N, int64_t q_row_stride, int64_t kv_row_stride,
                                   int64_t heads, int64_t kv_heads, int64_t head_dim,
                                   const dan_bf16 *wq, const dan_bf16 *wk, const float *rope,
                                   int64_t table_rows, const int32_t *positions,
                                   const int32_t *slots, float eps, int neox,
                                   const dan_bf16 *q_out, int64_t qo_row_stride,
                                   const dan_bf16 *k_cache, const dan_bf16 *v_cache,
                                   int64_t num_pages, int64_t page_size)
{
    (void)neox;
    return validate_rope(q, k, v, N, q_row_stride, kv_row_stride, heads, kv_heads, head_dim, wq, wk,
                         rope, table_rows, positions, slots, eps, q_out, qo_row_stride, k_cache,
                         v_cache, num_pages, page_size);
}

int dan_qk_norm_rope_cache(const dan_bf16 *q, const dan_bf16 *k, const dan_bf16 *v, int64_t N,
                           int64_t q_row_stride, int64_t kv_row_stride, int64_t heads,
                           int64_t kv_heads, int64_t head_dim, const dan_bf16 *wq,
                           const dan_bf16 *wk, const float *rope, int64_t table_rows,
                           const int32_t *positions, const int32_t *slots, float eps, int neox,
                           dan_bf16 *q_out, int64_t qo_row_stride, dan_bf16 *k_cache,
                           dan_bf16 *v_cache, int64_t num_pages, int64_t page_size, void *stream)
{
    const int st = validate_rope(q, k, v, N, q_row_stride, kv_row_stride, heads, kv_heads, head_dim,
                                 wq, wk, rope, table_rows, positions, slots, eps, q_out,
                                 qo_row_stride, k_cache, v_cache, num_pages, page_size);
    if (st != DAN_OK || N == 0) return st;
    const dan::CacheRopeProblem c{q, k, v, N, q_row_stride, kv_row_stride, heads, kv_heads, head_dim,
                                  wq, wk, rope, table_rows, positions, slots, eps, neox != 0, q_out,
                                  qo_row_stride, k_cache, v_cache, num_pages, page_size};
    return status_of([&] { return dan::launch_qk_norm_rope_cache(c, static_cast<cudaStream_t>(stream)); });
}

int64_t dan_window_attention_workspace(int64_t N, int64_t S, int64_t heads, int64_t kv_heads,
                                       int64_t head_dim, int64_t max_pages, int64_t page_size,
                                       int64_t window, int64_t sinks, int64_t chunk, int64_t max_q)
{
    if (N < 0 || S < 0 || N > (int64_t(1) << 30) || S > (int64_t(1) << 20) || max_q < 0 || window < 0 ||
        window > kMaxInt || sinks < 0 || sinks > kMaxInt || chunk < 1 || chunk > kMaxInt ||
        check_cache(heads, kv_heads, head_dim, 1, page_size) != DAN_OK || max_pages < 1 ||
        heads / kv_heads > dan::kMaxGroup || N > (int64_t(1) << 30) / heads ||
        max_pages > (int64_t(1) << 30) / page_size)
        return 0; // the call itself refuses these sizes
    dan::AttnProblem a = {};
    a.N = N, a.S = S, a.heads = heads, a.kv_heads = kv_heads, a.head_dim = head_dim;
    a.max_pages = max_pages, a.page_size = page_size, a.max_q = max_q;
    a.window = window, a.sinks = sinks, a.chunk = chunk;
    return dan::window_attention_workspace(a);
}

int dan_can_use_window_attention(const dan_bf16 *q, int64_t N, int64_t q_row_stride,
                                 const dan_bf16 *k_cache, const dan_bf16 *v_cache,
                                 int64_t num_pages, int64_t page_size, const int32_t *page_table,
                                 int64_t table_stride, int64_t max_pages, const int32_t *q_start,
                                 const int32_t *kv_len, int64_t S, int64_t heads, int64_t kv_heads,
                                 int64_t head_dim, int64_t window, int64_t sinks, int64_t chunk,
                                 int64_t max_q, float scale, const dan_bf16 *out, const float *lse,
                                 const void *workspace, int64_t workspace_bytes)
{
    return validate_attention(q, N, q_row_stride, k_cache, v_cache, num_pages, page_size, page_table,
                              table_stride, max_pages, q_start, kv_len, S, heads, kv_heads, head_dim,
                              window, sinks, chunk, max_q, scale, out, lse, workspace,
                              workspace_bytes);
}

int dan_window_attention(const dan_bf16 *q, int64_t N, int64_t q_row_stride,
                         const dan_bf16 *k_cache, const dan_bf16 *v_cache, int64_t num_pages,
                         int64_t page_size, const int32_t *page_table, int64_t table_stride,
                         int64_t max_pages, const int32_t *q_start, const int32_t *kv_len,
                         int64_t S, int64_t heads, int64_t kv_heads, int64_t head_dim,
                         int64_t window, int64_t sinks, int64_t chunk, int64_t max_q, float scale,
                         dan_bf16 *out, float *lse, void *workspace, int64_t workspace_bytes,
                         void *stream)
{
    const int st = validate_attention(q, N, q_row_stride, k_cache, v_cache, num_pages, page_size,
                                      page_table, table_stride, max_pages, q_start, kv_len, S, heads,
                                      kv_heads, head_dim, window, sinks, chunk, max_q, scale, out, lse,
                                      workspace, workspace_bytes);
    if (st != DAN_OK || N == 0 || S == 0) return st;
    const dan::AttnProblem a{q, N, q_row_stride, k_cache, v_cache, num_pages, page_size, page_table,
                             table_stride, max_pages, q_start, kv_len, S, heads, kv_heads, head_dim,
                             window, sinks, chunk, max_q, scale, out, lse, workspace};
    return status_of([&] { return dan::launch_window_attention(a, static_cast<cudaStream_t>(stream)); });
}

} // extern "C"
