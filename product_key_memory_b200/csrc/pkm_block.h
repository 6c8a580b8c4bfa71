// pkm_block.h -- internal launcher interface of the transformer-block operators (layer
// norm, dense layer, AdamW) between pkm_block_api.cu and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/pkm.h"

namespace pkm {

// Launches a kernel that may be scheduled before the stream's previous kernel has ended, where
// that one allows it (as the operators' own kernels do: each lets the next in, most when
// they start). Such a kernel calls wait_for_previous() before it touches global memory, which
// waits on the device for the end of the previous kernel and its writes.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, int cluster,
                         cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

#ifdef __CUDACC__
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_in() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
#endif

// Adds n to the library's launch counter (pkm_trace_read).
void count_launches(int n);

// ---------------------------------------------------------------- layer norm
constexpr int kNormMaxD = 16384;

struct NormArgs {
  int64_t rows;
  int d;
  int x_dtype, add_dtype, y_dtype, grad_dtype;
  float eps;
};

cudaError_t launch_layernorm_forward(const NormArgs& a, const void* x, const void* add,
                                     const float* gamma, const float* beta, void* y, void* sum,
                                     float* mean, float* rstd, cudaStream_t st);

// Partial column sums of the backward: [2][d] fp32 for each of at most so many blocks. Never more
// for fewer rows (the blocks themselves may be, in narrow rows: their groups are whole warps).
int norm_workspace_blocks(int64_t rows);
cudaError_t launch_layernorm_backward(const NormArgs& a, const void* grad_y, const void* x,
                                      const float* mean, const float* rstd, const float* gamma,
                                      const void* grad_sum, void* grad_x, float* grad_gamma,
                                      float* grad_beta, float* part, cudaStream_t st);

// --------------------------------------------------------------------- AdamW
using AdamWTensor = pkm_adamw_tensor;
using AdamWHyper = pkm_adamw_hyper;
// Adds the kernels launched to *launches.
cudaError_t launch_adamw(const AdamWTensor* t, int64_t count, const AdamWHyper& h,
                         const float* dyn, int* launches, cudaStream_t st);

}  // namespace pkm
