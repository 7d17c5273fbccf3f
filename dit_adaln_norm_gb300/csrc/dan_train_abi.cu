// dan_train_abi.cu -- the extern "C" boundary of the training operators
// (include/dan_train.h): argument validation and launches.
#include "../../include/dan_train.h"
#include "dan_gn.cuh"

#include <cmath>

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;

static_assert((int)DAN_BF16 == dan::kBf16 && (int)DAN_FP16 == dan::kFp16 && (int)DAN_FP32 == dan::kFp32, "types");

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool eps_ok(float eps) { return std::isfinite(eps) && eps >= 0.0f; }

// A buffer of a call: bytes at an address that must be aligned (0 bytes: not there).
struct Buf {
    const void *p;
    int64_t bytes;
    uintptr_t align;
};

bool overlap(const Buf &a, const Buf &b)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.bytes > 0 && b.bytes > 0 && x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// Every buffer there is non-null and aligned; no output overlaps an input or
// another output, but for outs[0] (of the same bytes) exactly on one of the first
// `in_place` inputs.
template <int I, int O>
int check_buffers(const Buf (&ins)[I], const Buf (&outs)[O], int in_place)
{
    for (const Buf &b : ins)
        if (b.bytes > 0 && !b.p) return DAN_EINVAL;
    for (const Buf &b : outs)
        if (b.bytes > 0 && !b.p) return DAN_EINVAL;
    for (const Buf &b : ins)
        if (b.bytes > 0 && !aligned(b.p, b.align)) return DAN_EALIGN;
    for (const Buf &b : outs)
        if (b.bytes > 0 && !aligned(b.p, b.align)) return DAN_EALIGN;
    for (int o = 0; o < O; ++o) {
        for (int i = 0; i < I; ++i) {
            if (o == 0 && i < in_place && outs[0].p == ins[i].p && outs[0].bytes == ins[i].bytes) continue;
            if (overlap(outs[o], ins[i])) return DAN_EALIAS;
        }
        for (int o2 = o + 1; o2 < O; ++o2)
            if (overlap(outs[o], outs[o2])) return DAN_EALIAS;
    }
    return DAN_OK;
}

// B rows of D at a stride, in elements; -1 where the stride is out of bounds.
int64_t strided(int64_t B, int64_t D, int64_t stride)
{
    if (B == 0) return 0;
    if (stride < D || stride > kMaxElems || B - 1 > kMaxElems / stride) return -1;
    return (B - 1) * stride + D;
}

int check_ln(int64_t B, int64_t T, int64_t D)
{
    if (B < 0 || T < 0 || D < 0) return DAN_EINVAL;
    if (D < 8 || D > 8192 || D % 8) return DAN_EUNSUPPORTED;
    if ((B > 0 && T > kMaxElems / B) || B > kMaxElems / D || B * T > kMaxElems / D) return DAN_EINVAL;
    return DAN_OK;
}

int validate_save(const dan_bf16 *x, const dan_bf16 *scale, const dan_bf16 *shift, int64_t vs,
                  const dan_bf16 *y, const float *stats, const uint8_t *codes, const uint8_t *scales,
                  int64_t B, int64_t T, int64_t D, float eps)
{
    const int st = check_ln(B, T, D);
    if (st != DAN_OK) return st;
    if (!eps_ok(eps) || (codes == nullptr) != (scales == nullptr)) return DAN_EINVAL;
    const int64_t rows = B * T;
    if (rows == 0) return DAN_OK;
    const int64_t vec = strided(B, D, vs);
    if (vec < 0) return DAN_EINVAL;
    if (vs % 8) return DAN_EALIGN;
    const Buf ins[] = {{x, rows * D * 2, 16}, {scale, vec * 2, 16}, {shift, vec * 2, 16}};
    const Buf outs[] = {{y, rows * D * 2, 16},
                        {stats, rows * 8, 8},
                        {codes, codes ? rows * D : 0, 8},
                        {scales, scales ? rows * ((D + 31) / 32) : 0, 1}};
    return check_buffers(ins, outs, 1);
}

int validate_ln_back(const dan_bf16 *dy, const dan_bf16 *x, const uint8_t *codes, const uint8_t *scales,
                     const float *stats, const dan_bf16 *scale, int64_t vs, const dan_bf16 *dres,
                     const dan_bf16 *dx, const dan_bf16 *dscale, const dan_bf16 *dshift, int64_t gs,
                     int64_t B, int64_t T, int64_t D, const void *workspace, int64_t workspace_bytes)
{
    const int st = check_ln(B, T, D);
    if (st != DAN_OK || B == 0) return st;
    if (B > (int64_t(1) << 30) / D) return DAN_EUNSUPPORTED; // blocks of the join
    const int64_t vec = strided(B, D, vs), grad = strided(B, D, gs);
    if (vec < 0 || grad < 0) return DAN_EINVAL;
    if (vs % 8 || gs % 8) return DAN_EALIGN;
    const int64_t rows = B * T, need = dan::ln_modulate_backward_workspace(B, T, D);
    if (workspace_bytes < need) return DAN_EINVAL;
    // dx is outs[0], and dy and dres the inputs that it may be
    const Buf ins[] = {{dy, rows * D * 2, 16},
                       {dres, dres ? rows * D * 2 : 0, 16},
                       {x, x ? rows * D * 2 : 0, 16},
                       {codes, x ? 0 : rows * D, 8},
                       {scales, x ? 0 : rows * ((D + 31) / 32), 1},
                       {stats, rows * 8, 8},
                       {scale, rows ? vec * 2 : 0, 16}};
    // the two gradients may be slices of one buffer, side by side: their rows are compared below
    const Buf outs[] = {{dx, rows * D * 2, 16}, {dscale, grad * 2, 16}, {workspace, need, 16}};
    int bad = check_buffers(ins, outs, 2);
    if (bad != DAN_OK) return bad;
    const Buf outs2[] = {{dx, rows * D * 2, 16}, {dshift, grad * 2, 16}, {workspace, need, 16}};
    bad = check_buffers(ins, outs2, 2);
    if (bad != DAN_OK) return bad;
    if (overlap(outs[1], outs2[1])) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(dscale), b = reinterpret_cast<uintptr_t>(dshift);
        const uintptr_t step = (uintptr_t)gs * 2, row = (uintptr_t)D * 2;
        const uintptr_t behind = a < b ? (b - a) % step : (step - (a - b) % step) % step;
        if (behind < row || behind + row > step) return DAN_EALIAS;
    }
    return DAN_OK;
}

// Sizes and types of a group norm; `checkpoint`: its blocks are written or read.
int check_gn(int64_t N, int64_t S, int64_t C, int64_t groups, int type, bool checkpoint)
{
    if (N < 0 || S < 0 || C < 0 || groups < 1 || type < 0 || type > 2) return DAN_EINVAL;
    if (C < 8 || C % 8 || C > (int64_t(1) << 20) || C % groups || (checkpoint && C % 32)) return DAN_EUNSUPPORTED;
    if (dan::gn_step(C / groups, checkpoint) > dan::kGnWidest) return DAN_EUNSUPPORTED;
    if (S > 0x7FFFFFFF || N >= (int64_t(1) << 28) || N * groups > 0x7FFFFFFF) return DAN_EUNSUPPORTED;
    if (S > 0 && N > kMaxElems / S) return DAN_EINVAL;
    if (N * S > kMaxElems / C || N > kMaxElems / C) return DAN_EINVAL;
    return DAN_OK;
}

// The vectors of a group norm: bytes of weight (and bias) and of scale (and shift).
int check_gn_vectors(const void *weight, const void *bias, int param_type, const void *scale, const void *shift,
                     int64_t vs, int type, int act, int64_t N, int64_t C, int64_t &params, int64_t &vec)
{
    if (act != DAN_NO_ACT && act != DAN_SILU) return DAN_EINVAL;
    if ((weight == nullptr) != (bias == nullptr) || (scale == nullptr) != (shift == nullptr)) return DAN_EINVAL;
    params = vec = 0;
    if (weight) {
        if (param_type != type && param_type != DAN_FP32) return DAN_EINVAL;
        params = C * dan::type_bytes(param_type);
    }
    if (scale) {
        vec = strided(N, C, vs);
        if (vec < 0) return DAN_EINVAL;
        if (vs * dan::type_bytes(type) % 16) return DAN_EALIGN;
        vec *= dan::type_bytes(type);
    }
    return DAN_OK;
}

struct GnArgs {
    const void *x;
    int type;
    const void *weight, *bias;
    int param_type;
    const void *scale, *shift;
    int64_t vs;
    int act;
    const void *y;
    const float *stats;
    const uint8_t *codes, *scales;
    int64_t N, S, C, groups;
    float eps;
    const void *workspace;
    int64_t workspace_bytes;
};

int validate_gn(const GnArgs &a)
{
    if ((a.codes == nullptr) != (a.scales == nullptr) || (a.codes && !a.stats)) return DAN_EINVAL;
    int st = check_gn(a.N, a.S, a.C, a.groups, a.type, a.codes != nullptr);
    if (st != DAN_OK) return st;
    int64_t params, vec;
    st = check_gn_vectors(a.weight, a.bias, a.param_type, a.scale, a.shift, a.vs, a.type, a.act, a.N, a.C, params, vec);
    if (st != DAN_OK) return st;
    if (!eps_ok(a.eps)) return DAN_EINVAL;
    const int64_t elems = a.N * a.S * a.C, bytes = elems * dan::type_bytes(a.type);
    if (elems == 0) return DAN_OK;
    const int64_t need = dan::group_norm_workspace(a.N, a.S, a.C, a.groups, a.type, a.codes != nullptr);
    if (a.workspace_bytes < need) return DAN_EINVAL;
    const Buf ins[] = {{a.x, bytes, 16}, {a.weight, params, 16}, {a.bias, params, 16}, {a.scale, vec, 16}, {a.shift, vec, 16}};
    const Buf outs[] = {{a.y, bytes, 16},
                        {a.stats, a.stats ? a.N * a.groups * 8 : 0, 8},
                        {a.codes, a.codes ? elems : 0, 8},
                        {a.scales, a.scales ? elems / 32 : 0, 1},
                        {a.workspace, need, 16}};
    return check_buffers(ins, outs, 1);
}

struct GnBackArgs {
    const void *dy, *x;
    int type;
    const uint8_t *codes, *scales;
    const float *stats;
    const void *weight, *bias;
    int param_type;
    const void *scale, *shift;
    int64_t vs;
    int act;
    const void *dx, *dweight, *dbias, *dscale, *dshift;
    int64_t gs;
    int64_t N, S, C, groups;
    const void *workspace;
    int64_t workspace_bytes;
};

int validate_gn_back(const GnBackArgs &a)
{
    const bool ckpt = a.x == nullptr;
    int st = check_gn(a.N, a.S, a.C, a.groups, a.type, ckpt);
    if (st != DAN_OK) return st;
    int64_t params, vec;
    st = check_gn_vectors(a.weight, a.bias, a.param_type, a.scale, a.shift, a.vs, a.type, a.act, a.N, a.C, params, vec);
    if (st != DAN_OK) return st;
    // each gradient with its parameter, and none without
    if ((a.weight == nullptr) != (a.dweight == nullptr) || (a.bias == nullptr) != (a.dbias == nullptr)) return DAN_EINVAL;
    if (a.N > 0 && ((a.scale == nullptr) != (a.dscale == nullptr) || (a.shift == nullptr) != (a.dshift == nullptr)))
        return DAN_EINVAL;
    const int es = (int)dan::type_bytes(a.type);
    int64_t grad = 0;
    if (a.dscale) {
        grad = strided(a.N, a.C, a.gs);
        if (grad < 0) return DAN_EINVAL;
        if (a.gs * es % 16) return DAN_EALIGN;
        grad *= es;
    }
    const int64_t elems = a.N * a.S * a.C;
    const int64_t need = dan::group_norm_backward_workspace(a.N, a.S, a.C, a.groups, a.type, ckpt);
    if (a.workspace_bytes < need) return DAN_EINVAL;
    const Buf ins[] = {{a.dy, elems * es, 16},
                       {a.x, a.x ? elems * es : 0, 16},
                       {a.codes, a.x ? 0 : elems, 8},
                       {a.scales, a.x ? 0 : elems / 32, 1},
                       {a.stats, a.N * a.groups * 8 * (a.S > 0), 8},
                       {a.weight, params, 16},
                       {a.bias, params, 16},
                       {a.scale, vec, 16},
                       {a.shift, vec, 16}};
    const Buf dx{a.dx, elems * es, 16}, dw{a.dweight, params, 16}, db{a.dbias, params, 16}, ws{a.workspace, need, 16};
    const Buf dsc{a.dscale, grad, 16}, dsh{a.dshift, grad, 16};
    // dscale and dshift may be slices of one buffer, side by side: compared by rows
    const Buf one[] = {dx, dw, db, dsc, ws}, two[] = {dx, dw, db, dsh, ws};
    st = check_buffers(ins, one, 1);
    if (st == DAN_OK) st = check_buffers(ins, two, 1);
    if (st != DAN_OK) return st;
    if (overlap(dsc, dsh)) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.dscale), y = reinterpret_cast<uintptr_t>(a.dshift);
        const uintptr_t step = (uintptr_t)(a.gs * es), row = (uintptr_t)(a.C * es);
        const uintptr_t behind = x < y ? (y - x) % step : (step - (x - y) % step) % step;
        if (behind < row || behind + row > step) return DAN_EALIAS;
    }
    return DAN_OK;
}

// A launch's status; no exception passes the C boundary.
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

int dan_can_use_ln_modulate_save(const dan_bf16 *x, const dan_bf16 *scale, const dan_bf16 *shift,
                                 int64_t vec_bstride, const dan_bf16 *y, const float *stats,
                                 const uint8_t *codes, const uint8_t *scales, int64_t B, int64_t T,
                                 int64_t D, float eps)
{
    return validate_save(x, scale, shift, vec_bstride, y, stats, codes, scales, B, T, D, eps);
}

int dan_ln_modulate_save(const dan_bf16 *x, const dan_bf16 *scale, const dan_bf16 *shift,
                         int64_t vec_bstride, dan_bf16 *y, float *stats, uint8_t *codes, uint8_t *scales,
                         int64_t B, int64_t T, int64_t D, float eps, void *stream)
{
    const int st = validate_save(x, scale, shift, vec_bstride, y, stats, codes, scales, B, T, D, eps);
    if (st != DAN_OK || B * T == 0) return st;
    dan::RowProblem p{x, nullptr, nullptr, nullptr, scale, shift, vec_bstride, y, nullptr, B, T, D, eps};
    p.q = codes;
    p.stats = stats;
    p.block_scales = scales;
    return status_of([&] { return dan::launch_ln_modulate_save(p, static_cast<cudaStream_t>(stream)); });
}

int64_t dan_ln_modulate_backward_workspace(int64_t B, int64_t T, int64_t D)
{
    return check_ln(B, T, D) == DAN_OK ? dan::ln_modulate_backward_workspace(B, T, D) : 0;
}

int dan_can_use_ln_modulate_backward(const dan_bf16 *dy, const dan_bf16 *x, const uint8_t *codes,
                                     const uint8_t *scales, const float *stats, const dan_bf16 *scale,
                                     int64_t vec_bstride, const dan_bf16 *dres, const dan_bf16 *dx,
                                     const dan_bf16 *dscale, const dan_bf16 *dshift, int64_t grad_bstride,
                                     int64_t B, int64_t T, int64_t D, const void *workspace,
                                     int64_t workspace_bytes)
{
    return validate_ln_back(dy, x, codes, scales, stats, scale, vec_bstride, dres, dx, dscale, dshift,
                            grad_bstride, B, T, D, workspace, workspace_bytes);
}

int dan_ln_modulate_backward(const dan_bf16 *dy, const dan_bf16 *x, const uint8_t *codes,
                             const uint8_t *scales, const float *stats, const dan_bf16 *scale,
                             int64_t vec_bstride, const dan_bf16 *dres, dan_bf16 *dx, dan_bf16 *dscale,
                             dan_bf16 *dshift, int64_t grad_bstride, int64_t B, int64_t T, int64_t D,
                             void *workspace, int64_t workspace_bytes, void *stream)
{
    const int st = validate_ln_back(dy, x, codes, scales, stats, scale, vec_bstride, dres, dx, dscale, dshift,
                                    grad_bstride, B, T, D, workspace, workspace_bytes);
    if (st != DAN_OK || B == 0) return st;
    const dan::LnBackProblem q{dy, x, codes, scales, stats, scale, vec_bstride, dres, dx, dscale, dshift,
                               grad_bstride, B, T, D, workspace};
    return status_of([&] { return dan::launch_ln_modulate_backward(q, static_cast<cudaStream_t>(stream)); });
}

int64_t dan_group_norm_workspace(int64_t N, int64_t S, int64_t C, int64_t groups, int type, int checkpoint)
{
    if (check_gn(N, S, C, groups, type, checkpoint != 0) != DAN_OK) return 0;
    return dan::group_norm_workspace(N, S, C, groups, type, checkpoint != 0);
}

int dan_can_use_group_norm(const void *x, int type, const void *weight, const void *bias, int param_type,
                           const void *scale, const void *shift, int64_t vec_bstride, int act, const void *y,
                           const float *stats, const uint8_t *codes, const uint8_t *scales, int64_t N,
                           int64_t S, int64_t C, int64_t groups, float eps, const void *workspace,
                           int64_t workspace_bytes)
{
    return validate_gn(GnArgs{x, type, weight, bias, param_type, scale, shift, vec_bstride, act, y, stats, codes,
                              scales, N, S, C, groups, eps, workspace, workspace_bytes});
}

int dan_group_norm(const void *x, int type, const void *weight, const void *bias, int param_type,
                   const void *scale, const void *shift, int64_t vec_bstride, int act, void *y, float *stats,
                   uint8_t *codes, uint8_t *scales, int64_t N, int64_t S, int64_t C, int64_t groups, float eps,
                   void *workspace, int64_t workspace_bytes, void *stream)
{
    const int st = validate_gn(GnArgs{x, type, weight, bias, param_type, scale, shift, vec_bstride, act, y, stats,
                                      codes, scales, N, S, C, groups, eps, workspace, workspace_bytes});
    if (st != DAN_OK || N * S == 0) return st;
    dan::GnProblem q = {};
    q.x = x, q.type = type, q.weight = weight, q.bias = bias, q.param_type = param_type;
    q.scale = scale, q.shift = shift, q.vs = vec_bstride, q.act = act, q.y = y, q.stats = stats;
    q.codes = codes, q.block_scales = scales;
    q.N = N, q.S = S, q.C = C, q.groups = groups, q.eps = eps, q.workspace = workspace;
    return status_of([&] { return dan::launch_group_norm(q, static_cast<cudaStream_t>(stream)); });
}

int64_t dan_group_norm_backward_workspace(int64_t N, int64_t S, int64_t C, int64_t groups, int type,
                                          int checkpoint)
{
    if (check_gn(N, S, C, groups, type, checkpoint != 0) != DAN_OK) return 0;
    return dan::group_norm_backward_workspace(N, S, C, groups, type, checkpoint != 0);
}

int dan_can_use_group_norm_backward(const void *dy, const void *x, int type, const uint8_t *codes,
                                    const uint8_t *scales, const float *stats, const void *weight,
                                    const void *bias, int param_type, const void *scale, const void *shift,
                                    int64_t vec_bstride, int act, const void *dx, const void *dweight,
                                    const void *dbias, const void *dscale, const void *dshift,
                                    int64_t grad_bstride, int64_t N, int64_t S, int64_t C, int64_t groups,
                                    const void *workspace, int64_t workspace_bytes)
{
    return validate_gn_back(GnBackArgs{dy, x, type, codes, scales, stats, weight, bias, param_type, scale, shift,
                                       vec_bstride, act, dx, dweight, dbias, dscale, dshift, grad_bstride, N, S, C,
                                       groups, workspace, workspace_bytes});
}

int dan_group_norm_backward(const void *dy, const void *x, int type, const uint8_t *codes, const uint8_t *scales,
                            const float *stats, const void *weight, const void *bias, int param_type,
                            const void *scale, const void *shift, int64_t vec_bstride, int act, void *dx,
                            void *dweight, void *dbias, void *dscale, void *dshift, int64_t grad_bstride,
                            int64_t N, int64_t S, int64_t C, int64_t groups, void *workspace,
                            int64_t workspace_bytes, void *stream)
{
    const int st = validate_gn_back(GnBackArgs{dy, x, type, codes, scales, stats, weight, bias, param_type, scale,
                                               shift, vec_bstride, act, dx, dweight, dbias, dscale, dshift,
                                               grad_bstride, N, S, C, groups, workspace, workspace_bytes});
    if (st != DAN_OK) return st;
    dan::GnProblem q = {};
    q.x = x, q.type = type, q.weight = weight, q.bias = bias, q.param_type = param_type;
    q.scale = scale, q.shift = shift, q.vs = vec_bstride, q.act = act;
    q.stats = const_cast<float *>(stats);
    q.codes = const_cast<uint8_t *>(codes), q.block_scales = const_cast<uint8_t *>(scales);
    q.N = N, q.S = S, q.C = C, q.groups = groups, q.workspace = workspace;
    q.dy = dy, q.dx = dx, q.dweight = dweight, q.dbias = dbias, q.dscale = dscale, q.dshift = dshift;
    q.gs = grad_bstride;
    return status_of([&] { return dan::launch_group_norm_backward(q, static_cast<cudaStream_t>(stream)); });
}

} // extern "C"
