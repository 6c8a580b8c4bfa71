// pkm_linear_epi.cuh -- activations of the dense layer and the epilogue of its outputs.
#pragma once

#include <math.h>

#include "pkm_elem.cuh"
#include "pkm_linear.h"

namespace pkm {

// 2^x and 1 / x by the special function unit, flushing subnormal numbers: 2^-22 and 1 ulp,
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

// exp(c x) with log2(e) c given as its fp32 value hi and the rest lo. FINE (results that are kept
// in fp32): the product's rounding, which the power multiplies by |c x|, is put back; without it a
// result that is rounded to bf16 loses nothing.
template <bool FINE>
__device__ __forceinline__ float exp_scaled(float x, float hi, float lo) {
  const float e = x * hi;
  const float y = exp2_fast(e);
  if (!FINE) return y;
  const float rest = fmaf(x, lo, fmaf(x, hi, -e)) * 0.69314718056f;
  return fabsf(e) < 126.f ? fmaf(y, rest, y) : y;   // y is 0 or infinite outside
}
constexpr float kLog2e = 1.4426950408889634f, kLog2eLo = 1.92596303e-8f;

// Phi(-x) and exp(-x^2 / 2) for x >= 0. Phi(-x) exp(x^2 / 2) is a smooth function that falls
// like 1 / x, so it is a polynomial of t = 1 / (1 + p x) times t: these eight coefficients (a least
// largest relative error on 0 <= x <= 13.4) leave 1.2e-7 of it. Phi is then good relative to
// itself however small it is; 1 - Phi(-x) stands for Phi(x). erfcf and expf take three times
// the instructions: the epilogue of a product has about 32 per element before it takes
// longer than the product.
template <bool FINE>
__device__ __forceinline__ float normal_tail(float x, float* gauss) {
  const float t = rcp_fast(fmaf(0.304055929f, x, 1.f));
  float q = fmaf(0.0368539616f, t, -0.155186698f);
  q = fmaf(q, t, 0.191852868f);
  q = fmaf(q, t, -0.0428629071f);
  q = fmaf(q, t, 0.123422243f);
  q = fmaf(q, t, 0.102475539f);
  q = fmaf(q, t, 0.122187726f);
  q = fmaf(q, t, 0.121257305f);
  const float s = x * x;
  *gauss = exp_scaled<FINE>(s, -0.5f * kLog2e, -0.5f * kLog2eLo);
  if (FINE && s < 174.f) *gauss = fmaf(*gauss, -0.5f * fmaf(x, x, -s), *gauss);   // s as rounded
  return q * t * *gauss;
}

// gelu is v Phi(v) with Phi(v) = 1 - Phi(-v) for v > 0; silu is v / (1 + exp(-v)). relu keeps
// a NaN. FINE: within 2^-19 of themselves while Phi or exp(v) is above 2^-126.
template <bool FINE>
__device__ __forceinline__ float act_value(float v, int act) {
  if (act == PKM_ACT_RELU) return v <= 0.f ? 0.f : v;
  if (act == PKM_ACT_GELU) {
    float gauss;
    const float q = normal_tail<FINE>(fabsf(v), &gauss);
    return v * (v > 0.f ? 1.f - q : q);
  }
  if (act == PKM_ACT_SILU) return v * rcp_fast(1.f + exp_scaled<FINE>(v, -kLog2e, -kLog2eLo));
  return v;
}

// d act / d v, which fp32 gradients are made of, so always FINE. gelu' = Phi(v) + v phi(v), silu' =
// s (1 + v (1 - s)) with s = 1/(1 + exp(-v)).
__device__ __forceinline__ float act_slope(float v, int act) {
  if (act == PKM_ACT_RELU) return v <= 0.f ? 0.f : (v > 0.f ? 1.f : v);
  if (act == PKM_ACT_GELU) {
    float gauss;
    const float q = normal_tail<true>(fabsf(v), &gauss);
    return fmaf(v * 0.39894228040143268f, gauss, v > 0.f ? 1.f - q : q);
  }
  if (act == PKM_ACT_SILU) {
    const float s = rcp_fast(1.f + exp_scaled<true>(v, -kLog2e, -kLog2eLo));
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
  v = act_value<true>(v, e.act);
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
  for (int i = 0; i < 8; ++i) v[i] = act_value<true>(v[i], e.act);
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
