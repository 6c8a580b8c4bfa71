// pkm_elem.cuh -- typed vector loads and stores of the transformer-block kernels: V
// consecutive elements (8 and 4: 16-byte accesses to fp32, 16 and 8 to bf16; 1: any alignment) of fp32 or bf16 arrays,
// widened to fp32. Loads are ordinary (not the read-only path): several operators may
// run in place.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pkm_common.cuh"

namespace pkm {

struct F32 {
  using T = float;
};
struct BF16 {
  using T = __nv_bfloat16;
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// V elements of type E in their stored form (a load in flight costs only its bytes).
template <typename E, int V> struct Raw;
template <> struct Raw<F32, 8> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    a = __ldcs(q);
    b = __ldcs(q + 1);
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};
template <> struct Raw<BF16, 8> {
  uint4 a;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    a = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
  }
  __device__ __forceinline__ void load_again(const void* p, int64_t i) {
    a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  }
  __device__ __forceinline__ void get(float* f) const { Vec<uint16_t>::widen(a, f); }
};
template <> struct Raw<F32, 4> {
  float4 a;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    a = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
  }
  __device__ __forceinline__ void load_again(const void* p, int64_t i) {
    a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  }
};
template <> struct Raw<BF16, 4> {
  uint2 a;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    a = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i));
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = bf16_lo(a.x); f[1] = bf16_hi(a.x);
    f[2] = bf16_lo(a.y); f[3] = bf16_hi(a.y);
  }
};
template <> struct Raw<F32, 1> {
  float a;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    a = __ldcs(static_cast<const float*>(p) + i);
  }
  __device__ __forceinline__ void load_again(const void* p, int64_t i) {
    a = static_cast<const float*>(p)[i];
  }
  __device__ __forceinline__ void get(float* f) const { f[0] = a; }
};
template <> struct Raw<BF16, 1> {
  uint16_t a;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    a = __ldcs(static_cast<const unsigned short*>(p) + i);
  }
  __device__ __forceinline__ void load_again(const void* p, int64_t i) {
    a = static_cast<const uint16_t*>(p)[i];
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = __uint_as_float(static_cast<uint32_t>(a) << 16);
  }
};

template <typename E, int V> struct Out;
template <> struct Out<F32, 8> {
  __device__ __forceinline__ static void store(void* p, int64_t i, const float* f) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};
template <> struct Out<BF16, 8> {
  __device__ __forceinline__ static void store(void* p, int64_t i, const float* f) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                   pack_bf16(f[6], f[7]));
  }
};
template <> struct Out<F32, 4> {
  __device__ __forceinline__ static void store(void* p, int64_t i, const float* f) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <> struct Out<BF16, 4> {
  __device__ __forceinline__ static void store(void* p, int64_t i, const float* f) {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
        make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
  }
};
template <> struct Out<F32, 1> {
  __device__ __forceinline__ static void store(void* p, int64_t i, const float* f) {
    static_cast<float*>(p)[i] = f[0];
  }
};
template <> struct Out<BF16, 1> {
  __device__ __forceinline__ static void store(void* p, int64_t i, const float* f) {
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(f[0]);
  }
};

// fp32 parameter vectors, read by every row (cached).
template <int V>
__device__ __forceinline__ void load_param(const float* p, int i, float* f) {
  if (V == 8) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p + i));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p + i) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else if (V == 4) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p + i));
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  } else {
    f[0] = __ldg(p + i);
  }
}

// A streaming load that stays where it is written: loads meant to be in flight together or
// ahead of their use are not moved behind other arithmetic.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 r;
  asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// Two fp32 values and their operations (one instruction for both), each rounded to nearest.
struct Pair {
  unsigned long long v;
  Pair() = default;
  __device__ __forceinline__ Pair(float a, float b) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  }
  __device__ __forceinline__ explicit Pair(float a) : Pair(a, a) {}
  __device__ __forceinline__ float lo() const { return get().x; }
  __device__ __forceinline__ float hi() const { return get().y; }
  __device__ __forceinline__ float2 get() const {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
  }
};
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
// May be fused with a product before it.
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// The value as an array of type E holds it.
template <typename E> __device__ __forceinline__ float rounded(float x);
template <> __device__ __forceinline__ float rounded<F32>(float x) { return x; }
template <> __device__ __forceinline__ float rounded<BF16>(float x) {
  return __bfloat162float(__float2bfloat16_rn(x));
}

}  // namespace pkm
