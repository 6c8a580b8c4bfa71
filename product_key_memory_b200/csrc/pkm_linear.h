// pkm_linear.h -- internal interface of the dense layer: the tensor-core product
// (pkm_linear_tc.cu), the passes around it and the small-batch kernel (pkm_linear.cu), the products
// of small fp32 layers (pkm_linear_f32.cu).
#pragma once

#include "pkm_block.h"

namespace pkm {

// What becomes of an output element v: pre = v + bias, y = act(pre) + residual.
struct LinearEpilogue {
  void* y;
  const float* bias;
  const void* residual;   // y's type
  void* pre;
  int y_f32, pre_f32, act;
};

enum LinearLayout { kForward, kGradX, kGradW };
constexpr int kLinearTileM = 256, kLinearTileN = 256;   // of a pair of CTAs

// How a product's tiles are shared out over `pairs` pairs of CTAs: the first `whole` tiles go
// round; the K blocks of the `cut` tiles after them, end to end, are dealt in equal ranges.
struct LinearWork {
  int pairs, whole, cut, kblocks;
  // First K block of pair c's range.
  __host__ __device__ int64_t begin(int c) const {
    return static_cast<int64_t>(cut) * kblocks * c / pairs;
  }
  // The pair whose range holds K block p: the largest c with begin(c) <= p.
  __host__ __device__ int owner(int64_t p) const {
    return static_cast<int>(((p + 1) * pairs - 1) / (static_cast<int64_t>(cut) * kblocks));
  }
};

// The plane products of one K block: step i (16 bits from bit 16 i) multiplies up to three planes
// of A (nibbles 0..2 in this order, their number in bits 14..15) with one of B (bits 12..13).
struct LinearSteps {
  uint64_t packed;
  int count, products;
};

// One product C[M][N] over K. A: K-major [a_count][M][lda] (forward, grad_x) or MN-major
// [a_count][K][lda] (grad_W); B: K-major [b_count][N][ldb] (forward) or MN-major
// [b_count][K][ldb]. Leading dimensions are multiples of 8.
struct LinearGemm {
  LinearLayout layout;
  const void *a, *b;
  int64_t lda, ldb;
  int M, N, K;
  uint32_t a_count, b_count;
  LinearSteps steps;
  LinearWork work;
  float* part;     // [2 pairs][256][256] fp32 when tiles are cut, else NULL
  LinearEpilogue epi;
  int* status;
  int clear;   // clear the status word first
};
cudaError_t launch_linear_gemm(const LinearGemm& g, int* launches, cudaStream_t st);

struct LinearArgs {
  int64_t M;
  int N, K;
  int dtype, out_dtype, act;
};

constexpr int kLinearMaxWidth = 1 << 20;   // N and K

bool linear_small(const LinearArgs& a);    // the forward's small-batch kernel takes it

// Small fp32 layers on the CUDA cores (pkm_linear_f32.cu).
bool linear_f32(const LinearArgs& a, bool backward);
cudaError_t launch_f32_forward(const LinearArgs& a, const float* x, const float* W,
                               const LinearEpilogue& epi, int* status, int* launches,
                               cudaStream_t st);
cudaError_t launch_f32_backward(const LinearArgs& a, const float* x, const float* W,
                                const float* grad_y, const float* pre, void* grad_x, float* grad_W,
                                float* grad_bias, int* status, int* launches, cudaStream_t st);
size_t linear_workspace_bytes(const LinearArgs& a, bool backward);
cudaError_t launch_linear_forward(const LinearArgs& a, const void* x, const void* W,
                                  const float* bias, const void* residual, void* y, void* pre,
                                  void* workspace, int* launches, cudaStream_t st);
cudaError_t launch_linear_backward(const LinearArgs& a, const void* x, const void* W,
                                   const void* grad_y, const void* pre, void* grad_x,
                                   float* grad_W, float* grad_bias, void* workspace,
                                   int* launches, cudaStream_t st);

}  // namespace pkm
