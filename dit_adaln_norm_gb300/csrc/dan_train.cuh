// dan_train.cuh -- launch interface of the training operators
// (include/dan_train.h), and the device helpers that they share.
#pragma once

#include "dan_device.cuh"
#include "dan_internal.h"
#include "dan_ring.cuh"

namespace dan {

// Gradients of LayerNorm + modulate.  Validated by the shim.
struct LnBackProblem {
    const void *dy, *x; // x: bf16 rows, or nullptr: codes and block_scales
    const void *codes, *block_scales;
    const void *stats, *scale;
    int64_t vs;
    const void *dres; // or nullptr
    void *dx, *dscale, *dshift;
    int64_t gs; // batch stride of dscale and dshift
    int64_t B, T, D;
    void *workspace;
};

int64_t ln_modulate_backward_workspace(int64_t B, int64_t T, int64_t D);
cudaError_t launch_ln_modulate_backward(const LnBackProblem &q, cudaStream_t s);

// Group norm of channels-last images, and its gradients.  Validated by the shim.
enum : int { kBf16 = 0, kFp16 = 1, kFp32 = 2 }; // dan_type
struct GnProblem {
    const void *x; // backward: or nullptr, codes and block_scales
    int type;
    const void *weight, *bias; // or both nullptr
    int param_type;
    const void *scale, *shift; // or both nullptr
    int64_t vs;
    int act;
    void *y;            // forward
    void *stats;        // [N, groups] (mean, rstd): written, or read by the backward pass
    void *codes, *block_scales; // the checkpoint, or both nullptr
    int64_t N, S, C, groups;
    float eps;
    void *workspace;
    const void *dy; // backward
    void *dx, *dweight, *dbias, *dscale, *dshift;
    int64_t gs;
};

int64_t group_norm_workspace(int64_t N, int64_t S, int64_t C, int64_t groups, int type, bool checkpoint);
int64_t group_norm_backward_workspace(int64_t N, int64_t S, int64_t C, int64_t groups, int type,
                                      bool checkpoint);
cudaError_t launch_group_norm(const GnProblem &q, cudaStream_t s);
cudaError_t launch_group_norm_backward(const GnProblem &q, cudaStream_t s);

// Asynchronous 8-byte global -> shared copy.
__device__ __forceinline__ void cp_async8(void *smem_dst, const void *gmem_src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(smem_dst)), "l"(gmem_src) : "memory");
}

} // namespace dan
