// pkm_linear_epi.cuh -- activations of the dense layer and the epilogue of its outputs.
#pragma once

#include <math.h>

#include "pkm_elem.cuh"
#include "pkm_linear.h"

namespace pkm {

// gelu is v Phi(v) with Phi(v) = erfc(-v / sqrt 2) / 2 (no cancellation for negative v);
// silu is v / (1 + exp(-v)). relu keeps a NaN.
__device__ __forceinline__ float act_value(float v, int act) {
  if (act == PKM_ACT_RELU) return v <= 0.f ? 0.f : v;
  if (act == PKM_ACT_GELU) return 0.5f * v * erfcf(v * -0.70710678118654752f);
  if (act == PKM_ACT_SILU) return v / (1.f + expf(-v));
  return v;
}

// d act / d v. gelu' = Phi(v) + v phi(v), silu' = s (1 + v (1 - s)) with s = 1/(1 + exp(-v)).
__device__ __forceinline__ float act_slope(float v, int act) {
  if (act == PKM_ACT_RELU) return v <= 0.f ? 0.f : (v > 0.f ? 1.f : v);
  if (act == PKM_ACT_GELU)
    return fmaf(v * 0.39894228040143268f, expf(-0.5f * v * v),
                0.5f * erfcf(v * -0.70710678118654752f));
  if (act == PKM_ACT_SILU) {
    const float s = 1.f / (1.f + expf(-v));
    return s * fmaf(v, 1.f - s, 1.f);
  }
  return 1.f;
}

__device__ __forceinline__ void linear_store1(const LinearEpilogue& e, int64_t at, int col,
                                              float v) {
  if (e.bias) v += __ldg(e.bias + col);
  if (e.pre) {
    if (e.pre_f32) static_cast<float*>(e.pre)[at] = v;
    else static_cast<__nv_bfloat16*>(e.pre)[at] = __float2bfloat16_rn(v);
  }
  v = act_value(v, e.act);
  if (e.y_f32) {
    if (e.residual) v += static_cast<const float*>(e.residual)[at];
    static_cast<float*>(e.y)[at] = v;
  } else {
    if (e.residual) v += __bfloat162float(static_cast<const __nv_bfloat16*>(e.residual)[at]);
    static_cast<__nv_bfloat16*>(e.y)[at] = __float2bfloat16_rn(v);
  }
}

// Eight consecutive columns of one row; `at` and `col` are multiples of 8.
__device__ __forceinline__ void linear_store8(const LinearEpilogue& e, int64_t at, int col,
                                              float* v) {
  if (e.bias) {
    float b[8];
    load_param<8>(e.bias, col, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
  }
  if (e.pre) {
    if (e.pre_f32) Out<F32, 8>::store(e.pre, at, v);
    else Out<BF16, 8>::store(e.pre, at, v);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = act_value(v[i], e.act);
  if (e.residual) {
    float r[8];
    if (e.y_f32) {
      Raw<F32, 8> q;
      q.load(e.residual, at);
      q.get(r);
    } else {
      Raw<BF16, 8> q;
      q.load(e.residual, at);
      q.get(r);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
  }
  if (e.y_f32) Out<F32, 8>::store(e.y, at, v);
  else Out<BF16, 8>::store(e.y, at, v);
}

// 32 consecutive columns from `col` (a multiple of 32) of one row; columns from N on do
// not exist.
__device__ __forceinline__ void linear_store_row32(const LinearEpilogue& e, int row, int col,
                                                   int M, int N, int split, float* v) {
  if (e.part) {
    float* p = e.part + (static_cast<int64_t>(split) * M + row) * e.ldp + col;
#pragma unroll
    for (int i = 0; i < 8; ++i)   // ldp covers the last group of four
      if (col + 4 * i < N)
        reinterpret_cast<float4*>(p)[i] =
            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    return;
  }
  const int64_t at = static_cast<int64_t>(row) * N + col;
  if ((N & 7) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + 8 * i < N) linear_store8(e, at + 8 * i, col + 8 * i, v + 8 * i);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (col + i < N) linear_store1(e, at + i, col + i, v[i]);
  }
}

}  // namespace pkm
