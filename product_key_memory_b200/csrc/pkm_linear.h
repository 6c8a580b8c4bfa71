// pkm_linear.h -- internal interface of the dense layer: the tensor-core product
// (pkm_linear_tc.cu), the passes around it and the small-batch kernel (pkm_linear.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/pkm.h"

namespace pkm {

// What becomes of an output element v: pre = v + bias, y = act(pre) + residual; with `part`
// the raw v is kept for linear_finish instead ([split][M][ldp] fp32).
struct LinearEpilogue {
  void* y;
  const float* bias;
  const void* residual;   // y's type
  void* pre;
  float* part;
  int64_t ldp;
  int y_f32, pre_f32, act;
};

enum LinearLayout { kForward, kGradX, kGradW };
// Tile shapes: 256 x 256, 192 and 128 on a pair of CTAs, 128 x 128 and 128 x 64 on one.
enum LinearTile { kTile256, kTile192, kTilePair128, kTile128, kTile64 };

// One product C[M][N] over K. A: K-major [a_count][M][lda] (forward, grad_x) or MN-major
// [a_count][K][lda] (grad_W); B: K-major [b_count][N][ldb] (forward) or MN-major
// [b_count][K][ldb]. Plane pair i of the sum is A's nibble i of a_planes with B's nibble i
// of b_planes. Leading dimensions are multiples of 8.
struct LinearGemm {
  LinearLayout layout;
  LinearTile tile;
  const void *a, *b;
  int64_t lda, ldb;
  int M, N, K;
  uint32_t a_count, b_count;
  uint32_t a_planes, b_planes;
  int pairs, ksplit;
  LinearEpilogue epi;
  int* status;
  int clear;   // clear the status word first
};
cudaError_t launch_linear_gemm(const LinearGemm& g, cudaStream_t st);

struct LinearArgs {
  int64_t M;
  int N, K;
  int dtype, out_dtype, act;
};

constexpr int kLinearMaxWidth = 1 << 20;   // N and K

bool linear_small(const LinearArgs& a);    // the forward's small-batch kernel takes it
size_t linear_workspace_bytes(const LinearArgs& a, bool backward);
cudaError_t launch_linear_forward(const LinearArgs& a, const void* x, const void* W,
                                  const float* bias, const void* residual, void* y, void* pre,
                                  void* workspace, int* launches, cudaStream_t st);
cudaError_t launch_linear_backward(const LinearArgs& a, const void* x, const void* W,
                                   const void* grad_y, const void* pre, void* grad_x,
                                   float* grad_W, float* grad_bias, void* workspace,
                                   int* launches, cudaStream_t st);

}  // namespace pkm
