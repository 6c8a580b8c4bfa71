// pkm_linear_epi.cuh -- activations of the dense layer and the epilogue of its outputs.
#pragma once

#include <math.h>

#include "pkm_elem.cuh"
#include "pkm_linear.h"

namespace pkm {

// 2^x and 1 / x by the special function unit, flushing subnormal numbers: 2 ulp and 1 ulp,
// without the range steps around __expf and __fdividef.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// erfc(x) / 2 and exp(-x^2) for x >= 0 by Abramowitz and Stegun 7.1.26: a polynomial of
// t = 1 / (1 + p x) times exp(-x^2), within 0.75e-7 (a rounding of the 1 + erf(x) that it
// stands for) and falling with exp(-x^2). A third of erfcf's instructions: the epilogue of
// a product has about 32 per element before it takes longer than the product.
__device__ __forceinline__ float half_erfc(float x, float* gauss) {
  const float t = rcp_fast(fmaf(0.3275911f, x, 1.f));
  float q = fmaf(0.5f * 1.061405429f, t, 0.5f * -1.453152027f);
  q = fmaf(q, t, 0.5f * 1.421413741f);
  q = fmaf(q, t, 0.5f * -0.284496736f);
  q = fmaf(q, t, 0.5f * 0.254829592f);
  *gauss = exp2_fast(x * x * -kLog2e);
  return q * t * *gauss;
}

// gelu is v Phi(v) with Phi(v) = erfc(-v / sqrt 2) / 2, mirrored for v > 0; silu is
// v / (1 + exp(-v)). relu keeps a NaN.
__device__ __forceinline__ float act_value(float v, int act) {
  if (act == PKM_ACT_RELU) return v <= 0.f ? 0.f : v;
  if (act == PKM_ACT_GELU) {
    float gauss;
    const float q = half_erfc(fabsf(v) * 0.70710678118654752f, &gauss);
    return v * (v > 0.f ? 1.f - q : q);
  }
  if (act == PKM_ACT_SILU) return v * rcp_fast(1.f + exp2_fast(v * -kLog2e));
  return v;
}

// d act / d v. gelu' = Phi(v) + v phi(v), silu' = s (1 + v (1 - s)) with s = 1/(1 + exp(-v)).
__device__ __forceinline__ float act_slope(float v, int act) {
  if (act == PKM_ACT_RELU) return v <= 0.f ? 0.f : (v > 0.f ? 1.f : v);
  if (act == PKM_ACT_GELU) {
    float gauss;
    const float q = half_erfc(fabsf(v) * 0.70710678118654752f, &gauss);
    return fmaf(v * 0.39894228040143268f, gauss, v > 0.f ? 1.f - q : q);
  }
  if (act == PKM_ACT_SILU) {
    const float s = rcp_fast(1.f + exp2_fast(v * -kLog2e));
    return s * fmaf(v, 1.f - s, 1.f);
  }
  return 1.f;
}

__device__ __forceinline__ float load_as(const void* p, int64_t at, int f32) {
  return f32 ? static_cast<const float*>(p)[at]
             : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
}
__device__ __forceinline__ void store_as(void* p, int64_t at, int f32, float v) {
  if (f32) static_cast<float*>(p)[at] = v;
  else static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ void linear_store1(const LinearEpilogue& e, int64_t at, int col,
                                              float v) {
  if (e.bias) v += __ldg(e.bias + col);
  if (e.pre) store_as(e.pre, at, e.pre_f32, v);
  v = act_value(v, e.act);
  if (e.residual) v += load_as(e.residual, at, e.y_f32);
  store_as(e.y, at, e.y_f32, v);
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

}  // namespace pkm
