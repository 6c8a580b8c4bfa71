// pkm_adamw.cu -- one AdamW step over a list of tensors, states in fp32 or in 8 bits.
//
//   m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2,
//   p <- p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Every element is read once and written once, so the step is bound by HBM. The list
// travels in the kernel's parameters (no device copy of it, nothing to keep alive, and a
// captured launch holds its own). A launch takes the tensors of one kind (types, states), so
// nothing is decided per element. The tensors' elements are cut into units of kUnit; a
// block takes units b, b + grid, ... and finds a unit's tensor by its first unit. A
// warp owns 256 consecutive elements, 8 per lane, which is also the block that shares
// a scale of 8-bit states: its largest magnitude is one warp reduction of the fp32 bits
// (ordered like the magnitudes, NaN above all). m, v, the codes and the scales are
// computed in single operations rounded to nearest (no fused multiply-add, but for the dither's
// sum, whose product is exact), so they are the same bits as the formula evaluated step by
// step in fp32.
//
// Measured on the tensors of a 512^2 layer with their vectors, 271 M elements: 1.35 ms with
// fp32 states and masters (6.8 TB/s), 0.66 ms with 8-bit states (5.0 TB/s).
//
// With 8-bit states an element has 12 to 22 bytes and the arithmetic comes near the issue
// rate (66 % of it, and 53 % of the DRAM's time), so it is kept short: a code's scale is
// folded into beta (powers of two: exact, for the squares while they are normal numbers) and an
// element's quotient is the special function unit's (2^-23). Its root decides a code and is
// rounded to nearest: with the special function unit's, 5 % faster, 4 codes in a million fell
// the other way. With fp32 states, whose root only moves p, that one is used.
#include <cuda_fp8.h>

#include <math.h>

#include "pkm_block.h"
#include "pkm_elem.cuh"
#include "pkm_tc.h"

namespace pkm {

namespace {

constexpr int kThreads = 256;
constexpr int kUnit = kThreads * 8;

// The kind of a tensor.
enum : int { kParamBf16 = 1, kGradBf16 = 2, kEight = 4, kMaster = 8 };

struct Tensor {
  void* param;
  void* grad;
  float* master;
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t n;
  uint32_t first;      // first unit of the launch that belongs to it
  uint32_t key;        // index in the list times the odd constant of the dither's key
  float keep, step;    // 1 - lr wd and lr / (1 - b1^t); with dyn: wd and lr_scale
};

template <int CAP>
struct List {
  Tensor t[CAP];
  int count;
  uint32_t units;
  float b1, c1, b2, c2, eps, root, grad_scale;   // c = 1 - b, root = 1 / sqrt(1 - b2^t)
  double db1, db2;
  uint32_t seed, step32;
  int zero;
  const float* dyn;
};

__host__ __device__ __forceinline__ uint32_t mix32(uint32_t h) {
  h ^= h >> 16;
  h *= 0x85ebca6bu;
  h ^= h >> 13;
  h *= 0xc2b2ae35u;
  return h ^ (h >> 16);
}

constexpr uint32_t kGolden = 0x9e3779b9u;

// Bits of the smallest power of two s >= 2^-100 with |x| <= 448 s, 448 = 1.75 2^8, for the
// largest |x| of the block by its bits: a mantissa above 1.75 carries into the exponent.
__device__ __forceinline__ uint32_t scale_bits(uint32_t most) {
  if (most >= 0x7f800000u) return 0x7fc00000u;
  const uint32_t b = (most + 0x1fffffu) & 0x7f800000u;
  const uint32_t low = 27u << 23;   // 2^-100
  return b < low + (8u << 23) ? low : b - (8u << 23);
}

__device__ __forceinline__ float inverse_pow2(uint32_t sbits) {
  return sbits == 0x7fc00000u ? __uint_as_float(sbits) : __uint_as_float((254u << 23) - sbits);
}

__device__ __forceinline__ void widen8(uint2 codes, float* f) {
  const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 x = __half22float2(__half2(h));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}

__device__ __forceinline__ float sqrt_fast(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// max(a, |b|, |c|), NaN if one is (a is not negative).
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ __forceinline__ float min3(float a, float b, float c) {
  float y;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ __forceinline__ Pair operator*(Pair a, Pair b) { return mul(a, b); }
// One at a time: the compiler fuses an addition of pairs with the product before it.
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  const float2 x = a.get(), y = b.get();
  return Pair(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}

__device__ __forceinline__ uint2 narrow8(const float* f) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i], f[4 * i + 1]),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2], f[4 * i + 3]),
                                                 __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

// q = r / s >= 0 with its dither: q + u ulp, ulp being e4m3's spacing at q (2^-9 below 2^-6)
// and u = (b - 32767.5) / 65536 from 16 bits of the pair's hash, rounded once; the nearest
// code is taken of it. For two values of 2^-6 <= q at a time.
__device__ __forceinline__ Pair dithered(Pair q, uint32_t h) {
  // 2^23 + b as bits; b and u are exact.
  const Pair b = add(Pair(__uint_as_float(__byte_perm(h, 0x4b000000u, 0x7610)),
                          __uint_as_float(__byte_perm(h, 0x4b000000u, 0x7632))),
                     Pair(-8388608.f));
  const Pair u = fma(b, Pair(1.f / 65536.f), Pair(-32767.5f / 65536.f));
  const float2 f = q.get();
  const Pair ulp(__uint_as_float((__float_as_uint(f.x) & 0x7f800000u) - (3u << 23)),
                 __uint_as_float((__float_as_uint(f.y) & 0x7f800000u) - (3u << 23)));
  return fma(u, ulp, q);
}
// Any q. What is above 0 stays at least the smallest code.
__device__ __forceinline__ float dithered_any(float q, uint32_t b16) {
  const float u = fmaf(static_cast<float>(b16), 1.f / 65536.f, -32767.5f / 65536.f);
  const uint32_t e = max(__float_as_uint(q) & 0x7f800000u, 121u << 23);
  const float near = fmaf(u, __uint_as_float(e - (3u << 23)), q);
  return q > 0.f ? fmaxf(near, 0x1p-9f) : q;
}

// Eight elements as loaded.
struct Eight {
  uint4 a, b;
};

// Codes of eight elements; as load16, in program order: all of an element group's loads are
// in flight before the first is used.
__device__ __forceinline__ uint2 load_codes(const void* p, int64_t i) {
  uint2 r;
  asm volatile("ld.global.cs.v2.u32 {%0, %1}, [%2];"
               : "=r"(r.x), "=r"(r.y)
               : "l"(static_cast<const uint8_t*>(p) + i)
               : "memory");
  return r;
}

__device__ __forceinline__ Eight load8(const void* p, int64_t i, const bool bf16) {
  Eight r;
  if (bf16) {
    r.a = load16(static_cast<const uint16_t*>(p) + i);
    r.b = make_uint4(0, 0, 0, 0);
  } else {
    r.a = load16(static_cast<const float*>(p) + i);
    r.b = load16(static_cast<const float*>(p) + i + 4);
  }
  return r;
}

__device__ __forceinline__ void widen(const Eight& r, bool bf16, float* f) {
  if (bf16) {
    Vec<uint16_t>::widen(r.a, f);
  } else {
    Vec<float>::widen(r.a, f);
    Vec<float>::widen(r.b, f + 4);
  }
}

__device__ __forceinline__ void store8(void* p, int64_t i, bool bf16, const float* f) {
  if (bf16) {
    __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i),
           make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                      pack_bf16(f[6], f[7])));
  } else {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    __stcs(q, make_float4(f[0], f[1], f[2], f[3]));
    __stcs(q + 1, make_float4(f[4], f[5], f[6], f[7]));
  }
}

__device__ __forceinline__ float load1(const void* p, int64_t i, bool bf16) {
  return bf16 ? load_elem(static_cast<const uint16_t*>(p), i)
              : load_elem(static_cast<const float*>(p), i);
}

__device__ __forceinline__ void store1(void* p, int64_t i, bool bf16, float f) {
  if (bf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(f);
  else static_cast<float*>(p)[i] = f;
}

template <int CAP, int KIND>
__global__ void __launch_bounds__(kThreads, 4) adamw_kernel(const __grid_constant__ List<CAP> list) {
  constexpr bool kWideMaster = (KIND & kMaster) != 0, eight = (KIND & kEight) != 0;
  constexpr bool gb = (KIND & kGradBf16) != 0, param_bf16 = (KIND & kParamBf16) != 0;
  constexpr bool pb = param_bf16 && !kWideMaster;   // type of what carries the parameter
  __shared__ float dynamic[2];   // 1 / (1 - b1^t), 1 / sqrt(1 - b2^t)
  let_next_in();
  wait_for_previous();
  float root = list.root, grad_scale = list.grad_scale, lr = 0.f, over = 1.f;
  uint32_t step32 = list.step32;
  if (list.dyn) {
    if (threadIdx.x == 0) {
      const double t = static_cast<double>(list.dyn[1]);
      dynamic[0] = static_cast<float>(1.0 / (1.0 - pow(list.db1, t)));
      dynamic[1] = static_cast<float>(1.0 / sqrt(1.0 - pow(list.db2, t)));
    }
    __syncthreads();
    lr = list.dyn[0];
    grad_scale = list.dyn[2];
    step32 = static_cast<uint32_t>(static_cast<int64_t>(list.dyn[1]));
    over = dynamic[0];
    root = dynamic[1];
  }
  const uint32_t key0 = mix32(list.seed + kGolden * step32);
  const int lane = threadIdx.x & 31;
  int cur = 0;
  uint32_t begin = 0, end = 0;
  for (uint32_t u = blockIdx.x; u < list.units; u += gridDim.x) {
    if (u >= end) {   // the last tensor whose first unit is at most u
      int lo = cur, hi = list.count;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (list.t[mid].first <= u) lo = mid;
        else hi = mid;
      }
      cur = lo;
      begin = list.t[cur].first;
      end = cur + 1 < list.count ? list.t[cur + 1].first : list.units;
    }
    const Tensor& T = list.t[cur];
    const int64_t n = T.n;
    const int64_t i = static_cast<int64_t>(u - begin) * kUnit + threadIdx.x * 8;
    const int64_t block = i >> 8;
    if (block * 256 >= n) continue;   // warp-uniform
    void* carrier = kWideMaster ? static_cast<void*>(T.master) : T.param;
    const bool whole = i + 8 <= n;
    float p[8], g[8], m[8], v[8];
    // 8-bit states: m and v (r then) hold the codes, their scales are in these factors.
    float bm = list.b1, bv = list.b2;
    if (eight) {
      const float ms = T.ms[block], vs = T.vs[block];
      bm *= ms;
      bv *= vs * vs;
    }
    if (whole) {
      const Eight rg = load8(T.grad, i, gb);
      const Eight rp = load8(carrier, i, pb);
      if (eight) {
        const uint2 rm = load_codes(T.m, i), rv = load_codes(T.v, i);
        widen8(rm, m);
        widen8(rv, v);
      } else {
        const Eight rm = load8(T.m, i, false), rv = load8(T.v, i, false);
        widen(rm, false, m);
        widen(rv, false, v);
      }
      widen(rg, gb, g);
      widen(rp, pb, p);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = i + j < n;
        g[j] = in ? load1(T.grad, i + j, gb) : 0.f;
        p[j] = in ? load1(carrier, i + j, pb) : 0.f;
        if (eight) {
          const uint32_t cm = in ? static_cast<const uint8_t*>(T.m)[i + j] : 0u;
          const uint32_t cv = in ? static_cast<const uint8_t*>(T.v)[i + j] : 0u;
          m[j] = __half2float(__half(__nv_cvt_fp8_to_halfraw(cm, __NV_E4M3)));
          v[j] = __half2float(__half(__nv_cvt_fp8_to_halfraw(cv, __NV_E4M3)));
        } else {
          m[j] = in ? static_cast<const float*>(T.m)[i + j] : 0.f;
          v[j] = in ? static_cast<const float*>(T.v)[i + j] : 0.f;
        }
      }
    }
    float keep = T.keep, step = T.step;
    if (list.dyn) {
      const float mine = lr * step;            // lr lr_scale
      keep = 1.f - mine * keep;
      step = mine * over;
    }
    float most_m = 0.f, most_v = 0.f;
    const Pair b1(bm), b2(bv), c1(list.c1), c2(list.c2), gs(grad_scale);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const Pair gj = Pair(g[j], g[j + 1]) * gs;
      Pair v2(v[j], v[j + 1]);
      if (eight) v2 = v2 * v2;                           // of a code: exact
      const Pair m2 = b1 * Pair(m[j], m[j + 1]) + c1 * gj;
      v2 = b2 * v2 + c2 * gj * gj;
      m[j] = m2.lo(), m[j + 1] = m2.hi();
      v[j] = v2.lo(), v[j + 1] = v2.hi();
      if (eight) {
        most_m = max_nan(most_m, m[j], m[j + 1]);
        most_v = max_nan(most_v, v[j], v[j + 1]);
      }
    }
    // r[j] is the root of v[j], or (fast) that over its scale.
    float r[8], scale_r = 1.f;
    uint32_t sm = 0, sr = 0;
    bool fast = false;
    if (eight) {
      sm = scale_bits(__reduce_max_sync(0xffffffffu, __float_as_uint(most_m)));
      sr = scale_bits(__float_as_uint(__fsqrt_rn(__uint_as_float(
          __reduce_max_sync(0xffffffffu, __float_as_uint(most_v))))) & 0x7fffffffu);
      // Fast: every r / s is at least 2^-6 (none 2^14 below the block's largest, no zeros) and
      // 1 / s^2 is a number.
      const float ir = inverse_pow2(sr), over2 = ir * ir;
      float least = v[0];
#pragma unroll
      for (int j = 2; j < 8; j += 2) least = min3(least, v[j - 1], v[j]);
      least = fminf(least, v[7]);
      fast = __all_sync(0xffffffffu, least * over2 >= 0x1p-12f && over2 < INFINITY &&
                                         most_v < INFINITY);
      if (fast) {
        scale_r = __uint_as_float(sr);
        const Pair o(over2);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const Pair q = Pair(v[j], v[j + 1]) * o;
          r[j] = __fsqrt_rn(q.lo());
          r[j + 1] = __fsqrt_rn(q.hi());
        }
      }
    }
    if (!fast) {
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = eight ? __fsqrt_rn(v[j]) : sqrt_fast(v[j]);
    }
    const Pair roots(root * scale_r), eps(list.eps), keeps(keep), steps(-step);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const Pair den = fma(Pair(r[j], r[j + 1]), roots, eps);
      const Pair up = Pair(m[j], m[j + 1]) * Pair(rcp_fast(den.lo()), rcp_fast(den.hi()));
      const Pair p2 = fma(up, steps, Pair(p[j], p[j + 1]) * keeps);
      p[j] = p2.lo(), p[j + 1] = p2.hi();
    }
    if (whole) {
      if (!eight) {
        store8(T.m, i, false, m);
        store8(T.v, i, false, v);
      }
      if (kWideMaster) store8(T.master, i, false, p);
      store8(T.param, i, param_bf16, p);
      if (list.zero) {
        const float z[8] = {};
        store8(T.grad, i, gb, z);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (i + j >= n) continue;
        if (!eight) {
          static_cast<float*>(T.m)[i + j] = m[j];
          static_cast<float*>(T.v)[i + j] = v[j];
        }
        if (kWideMaster) T.master[i + j] = p[j];
        store1(T.param, i + j, param_bf16, p[j]);
        if (list.zero) store1(T.grad, i + j, gb, 0.f);
      }
    }
    if (eight) {
      const uint32_t key = mix32(key0 ^ T.key);
      const uint32_t pair = static_cast<uint32_t>(i >> 1);
      const Pair ims(inverse_pow2(sm));
      const float ir = inverse_pow2(sr);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const Pair q = Pair(m[j], m[j + 1]) * ims;
        m[j] = q.lo(), m[j + 1] = q.hi();
      }
      const uint2 cm = narrow8(m);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const uint32_t h = mix32((pair + j / 2) ^ key);
        if (fast) {
          const Pair q = dithered(Pair(r[j], r[j + 1]), h);
          r[j] = q.lo(), r[j + 1] = q.hi();
        } else {
          r[j] = dithered_any(r[j] * ir, h & 0xffffu);
          r[j + 1] = dithered_any(r[j + 1] * ir, h >> 16);
        }
      }
      const uint2 cv = narrow8(r);                       // saturates at 448
      const int64_t block = i >> 8;
      if (lane == 0) {
        T.ms[block] = __uint_as_float(sm);
        T.vs[block] = __uint_as_float(sr);
      }
      if (whole) {
        __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(T.m) + i), cm);
        __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(T.v) + i), cv);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (i + j < n) {
            static_cast<uint8_t*>(T.m)[i + j] =
                static_cast<uint8_t>((j < 4 ? cm.x : cm.y) >> (8 * (j & 3)));
            static_cast<uint8_t*>(T.v)[i + j] =
                static_cast<uint8_t>((j < 4 ? cv.x : cv.y) >> (8 * (j & 3)));
          }
      }
    }
  }
}

// Tensors of a launch, whose parameters (96 bytes a tensor) the host copies at each call: 48
// vectors take 6.5 us of it with 64, 8.8 with 256.
constexpr int kSmallList = 16;
constexpr int kMediumList = 64;
constexpr int kLargeList = 256;    // 25 KB (32,764 bytes is the limit)

template <int CAP, int KIND>
cudaError_t launch_kind(const List<CAP>& list, cudaStream_t st) {
  // fp32 states: a block per unit (8 blocks an SM going round took 12 % longer). 8-bit states:
  // 32 blocks an SM going round, which spares most units the block's setup.
  const unsigned most = (KIND & kEight) ? static_cast<unsigned>(sm_count()) * 32 : 1u << 30;
  const unsigned grid = list.units < most ? list.units : most;
  return launch_after(adamw_kernel<CAP, KIND>, dim3(grid), dim3(kThreads), 0, 1, st, list);
}

constexpr int kKinds = 16;

template <int CAP>
cudaError_t launch_list(const List<CAP>& list, int kind, cudaStream_t st) {
  switch (kind) {
#define PKM_KIND(k) \
  case k: return launch_kind<CAP, k>(list, st);
    PKM_KIND(0) PKM_KIND(kGradBf16) PKM_KIND(kEight) PKM_KIND(kEight | kGradBf16)
    PKM_KIND(kParamBf16) PKM_KIND(kParamBf16 | kGradBf16) PKM_KIND(kParamBf16 | kEight)
    PKM_KIND(kParamBf16 | kEight | kGradBf16) PKM_KIND(kParamBf16 | kMaster)
    PKM_KIND(kParamBf16 | kMaster | kGradBf16) PKM_KIND(kParamBf16 | kMaster | kEight)
    PKM_KIND(kParamBf16 | kMaster | kEight | kGradBf16)
#undef PKM_KIND
  }
  return cudaErrorInvalidValue;   // a master goes with a bf16 parameter (checked by the caller)
}

int kind_of(const AdamWTensor& t) {
  return (t.param_dtype ? kParamBf16 : 0) | (t.grad_dtype ? kGradBf16 : 0) |
         (t.state_bits == 8 ? kEight : 0) | (t.master ? kMaster : 0);
}

template <int CAP>
cudaError_t run_lists(const AdamWTensor* t, int64_t count, const AdamWHyper& h, const float* dyn,
                      int* launches, cudaStream_t st) {
  static_assert(sizeof(List<CAP>) <= 32764, "kernel parameters");
  List<CAP> list;
  const double fix1 = 1.0 - pow(h.beta1, static_cast<double>(h.step));
  const double fix2 = 1.0 - pow(h.beta2, static_cast<double>(h.step));
  list.b1 = static_cast<float>(h.beta1);
  list.c1 = static_cast<float>(1.0 - h.beta1);
  list.b2 = static_cast<float>(h.beta2);
  list.c2 = static_cast<float>(1.0 - h.beta2);
  list.eps = static_cast<float>(h.eps);
  list.root = static_cast<float>(1.0 / sqrt(fix2));
  list.grad_scale = static_cast<float>(h.grad_scale);
  list.db1 = h.beta1;
  list.db2 = h.beta2;
  list.seed = h.seed;
  list.step32 = static_cast<uint32_t>(h.step);
  list.zero = h.zero_grad;
  list.dyn = dyn;
  unsigned present = 0;
  for (int64_t i = 0; i < count; ++i)
    if (t[i].n > 0) present |= 1u << kind_of(t[i]);
  for (int kind = 0; kind < kKinds; ++kind) {
    if (!(present >> kind & 1)) continue;
    list.count = 0;
    list.units = 0;
    for (int64_t i = 0; i < count; ++i) {
      if (t[i].n > 0 && kind_of(t[i]) == kind) {
        Tensor& d = list.t[list.count++];
        d.param = t[i].param;
        d.grad = t[i].grad;
        d.master = t[i].master;
        d.m = t[i].m;
        d.v = t[i].v;
        d.ms = t[i].m_scale;
        d.vs = t[i].v_scale;
        d.n = t[i].n;
        d.first = list.units;
        d.key = static_cast<uint32_t>(i) * kGolden;
        if (dyn) {
          d.keep = t[i].weight_decay;
          d.step = t[i].lr_scale;
        } else {
          const double lr = h.lr * t[i].lr_scale;
          d.keep = static_cast<float>(1.0 - lr * t[i].weight_decay);
          d.step = static_cast<float>(lr / fix1);
        }
        list.units += static_cast<uint32_t>((d.n + kUnit - 1) / kUnit);
      }
      // A launch holds CAP tensors and 2^31 units; a tensor has at most 2^27.
      if (list.count && (list.count == CAP || i + 1 == count || list.units >= 1u << 30)) {
        const cudaError_t e = launch_list(list, kind, st);
        if (e != cudaSuccess) return e;
        ++*launches;
        list.count = 0;
        list.units = 0;
      }
    }
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_adamw(const AdamWTensor* t, int64_t count, const AdamWHyper& h,
                         const float* dyn, int* launches, cudaStream_t st) {
  if (count <= kSmallList) return run_lists<kSmallList>(t, count, h, dyn, launches, st);
  if (count <= kMediumList) return run_lists<kMediumList>(t, count, h, dyn, launches, st);
  return run_lists<kLargeList>(t, count, h, dyn, launches, st);
}

}  // namespace pkm
