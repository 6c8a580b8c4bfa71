// pkm_linear.cu -- the dense layer around its tensor-core product: the small-batch
// forward, operand planes, the backward's d = grad_y act'(pre), column sums, and how a
// product's tiles are shared out.
#include "pkm_linear.h"

#include <type_traits>

#include "pkm_block.h"
#include "pkm_linear_epi.cuh"
#include "pkm_tc.h"
#include "pkm_tcgen05.cuh"

namespace pkm {

namespace {

constexpr int kSmallM = 8;          // rows of the small-batch kernel

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
int64_t pad8(int64_t x) { return (x + 7) / 8 * 8; }

// A call's status word is cleared by its first kernel: one operation less in the stream.
__device__ __forceinline__ void clear_status(int* status) {
  if (status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *status = 0;
}

// v as bf16 planes hi, mid, lo (rounded to nearest, so the sum is v to 2^-24; a hi that would
// round up to infinity is cut). Infinities and NaN leave zeros below them.
__device__ __forceinline__ void split(float v, float* p) {
  const float inf = __uint_as_float(0x7f800000u);
  p[0] = rounded<BF16>(v);
  if (fabsf(p[0]) == inf) p[0] = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
  const bool fine = fabsf(p[0]) < inf;
  p[1] = fine ? rounded<BF16>(v - p[0]) : 0.f;
  p[2] = fine ? rounded<BF16>(v - p[0] - p[1]) : 0.f;
}

// ---------------------------------------------------------------- small batches
constexpr int kSmallCols = 4;

// Sums of NV values over a warp, NV a power of two up to 32: each exchange halves the values a
// lane keeps. Returns the sum of value lane / (32 / NV).
template <int NV>
__device__ __forceinline__ float warp_sums(float* v, int lane) {
  int o = 16;
#pragma unroll
  for (int n = NV / 2; n > 0; n /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  float s = v[0];
  for (; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// A warp has four columns, so that a piece of x (from L1 or L2) serves four rows of W, and one
// of `slices` shares of K; the lanes' sums are added by a tree, the slices' in order. With few
// rows W's bytes bound it (16384 x 16384 bf16, 1 row: 86 us, 6.2 TB/s), with 8 the reading of
// x, M / 4 times W's bytes from L1 (166 us; 2 columns a warp 169, and slower with fewer
// rows). 1024 -> 4096 bf16, 1 row: 3.2 us; 5590 -> 2972 fp32, 4 rows: 16 us.
template <typename E, int V, int M>
__global__ void __launch_bounds__(256) linear_small_kernel(const void* x, const void* W, int N,
                                                           int K, int slices,
                                                           const LinearEpilogue epi,
                                                           int* status) {
  constexpr int C = kSmallCols;
  constexpr int NV = C * M <= 4 ? 4 : C * M <= 8 ? 8 : C * M <= 16 ? 16 : 32;
  // Accesses of a W row in flight. More rows hold more of x in registers; of single elements,
  // four times as many cost one row's sectors their place in L1 (17 -> 38 us at 5591 -> 2972).
  constexpr int kDepth = V == 1 ? (M <= 2 ? 4 : 8) : M <= 2 ? 2 : 1;
  __shared__ float sums[8][NV];
  let_next_in();
  wait_for_previous();
  clear_status(status);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = 8 / slices;
  const int col0 = (blockIdx.x * groups + warp / slices) * C;
  float acc[NV] = {};   // [m][c]
  constexpr int stride = 32 * V;
  const int share = (K + stride * slices - 1) / (stride * slices) * stride;
  int k0 = warp % slices * share;
  const int k1 = min(K, k0 + share);
  k0 += lane * V;
  const auto pieces = [&](auto depth) {
    constexpr int kDepth = decltype(depth)::value;
    Raw<E, V> w[kDepth][C];
#pragma unroll
    for (int u = 0; u < kDepth; ++u)
#pragma unroll
      for (int c = 0; c < C; ++c)
        w[u][c].load(W, static_cast<int64_t>(min(col0 + c, N - 1)) * K + k0 + u * stride);
#pragma unroll
    for (int u = 0; u < kDepth; ++u) {
      Raw<E, V> xr[M];
#pragma unroll
      for (int m = 0; m < M; ++m) xr[m].load_again(x, static_cast<int64_t>(m) * K + k0 + u * stride);
      float wf[C][V];
#pragma unroll
      for (int c = 0; c < C; ++c) w[u][c].get(wf[c]);
#pragma unroll
      for (int m = 0; m < M; ++m) {
        float xf[V];
        xr[m].get(xf);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int v = 0; v < V; ++v) acc[m * C + c] = fmaf(wf[c][v], xf[v], acc[m * C + c]);
      }
    }
    k0 += stride * kDepth;
  };
  while (k0 + (kDepth - 1) * stride < k1) pieces(std::integral_constant<int, kDepth>());
  while (k0 < k1) pieces(std::integral_constant<int, 1>());
  __syncwarp();
  const float s = warp_sums<NV>(acc, lane);
  if (lane % (32 / NV) == 0) sums[warp][lane / (32 / NV)] = s;
  __syncthreads();
  const int g = threadIdx.x / NV, i = threadIdx.x % NV;
  const int col = (blockIdx.x * groups + g) * C + i % C;
  if (g >= groups || i >= C * M || col >= N) return;
  float total = 0.f;
  for (int j = 0; j < slices; ++j) total += sums[g * slices + j][i];
  linear_store1(epi, static_cast<int64_t>(i / C) * N + col, col, total);
}

template <typename E, int V>
cudaError_t run_small(int M, const void* x, const void* W, int N, int K,
                      const LinearEpilogue& epi, int* status, cudaStream_t st) {
  // K is shared out until there are 16 warps an SM or a slice has one access a row.
  const int64_t warps = (N + kSmallCols - 1) / kSmallCols;
  int slices = 1;
  while (slices < 8 && slices * 32 * V < K && warps * slices < 16 * sm_count()) slices *= 2;
  const int per = 8 / slices * kSmallCols;
  const unsigned grid = static_cast<unsigned>((N + per - 1) / per);
  const auto run = [&](auto* kernel) {
    return launch_after(kernel, grid, 256, 0, 1, st, x, W, N, K, slices, epi, status);
  };
  switch (M) {
    case 1: return run(linear_small_kernel<E, V, 1>);
    case 2: return run(linear_small_kernel<E, V, 2>);
    case 3: return run(linear_small_kernel<E, V, 3>);
    case 4: return run(linear_small_kernel<E, V, 4>);
  }
  if constexpr (V == 8) {                    // bf16: linear_rows_kernel takes more
    return cudaErrorInvalidValue;
  } else {
    switch (M) {
      case 5: return run(linear_small_kernel<E, V, 5>);
      case 6: return run(linear_small_kernel<E, V, 6>);
      case 7: return run(linear_small_kernel<E, V, 7>);
      default: return run(linear_small_kernel<E, V, 8>);
    }
  }
}

// --------------------------------------------------------------------- few rows
// y^T = W x^T in bf16 on the warps' matrix instructions (m16n8k16): a warp has 16 rows of W, NT
// tiles of 8 rows of x, and one of `slices` shares of K. Which k an instruction's
// places stand for is free as long as W and x agree, so a lane's fragments are 16 bytes of a
// row as they lie in memory: each lane copies its own into shared memory kStages pieces of 32
// k ahead, with no barrier, which keeps enough of W in flight (two pieces ahead in registers
// took twice as long). The accumulators are taken out every 4 pieces, as the tensor-core
// kernel does; the slices' sums are added in order. Bound by W's bytes and, with
// few of them, by latency: 16 rows, 1024 -> 4096: 4.7 us (256-row tiles 9.6), 4096 -> 4096 10 us,
// 16384 -> 16384 106 us, 5.0 TB/s.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int NT> struct RowsTile {
  static constexpr int kPieces = 2 + NT;                       // 512 bytes of a warp each
  static constexpr int kStages = NT == 1 ? 8 : NT == 2 ? 6 : 4;
  static constexpr int kValues = NT * 4;                       // sums of a lane
  static constexpr size_t kSmem = kStages * kPieces * 512;     // of a warp
  static_assert(kSmem >= kValues * 32 * sizeof(float), "the sums take the ring's place");
};

template <int NT>
__global__ void __launch_bounds__(512) linear_rows_kernel(const uint16_t* x, const uint16_t* W,
                                                          int M, int N, int K, int slices,
                                                          const LinearEpilogue epi, int* status) {
  using T = RowsTile<NT>;
  extern __shared__ __align__(16) uint8_t ring_raw[];
  let_next_in();
  wait_for_previous();
  clear_status(status);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int groups = (blockDim.x >> 5) / slices, slice = warp % slices;
  const int n0 = (blockIdx.x * groups + warp / slices) * 16;
  const int share = (K + 32 * slices - 1) / (32 * slices) * 32;
  const int begin = min(K, slice * share), end = min(K, begin + share);
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(ring_raw)) +
                        warp * static_cast<uint32_t>(T::kSmem) + lane * 16;
  // Rows past the end are the last one again; their sums are not stored.
  const uint16_t *pw[2], *px[NT];
#pragma unroll
  for (int i = 0; i < 2; ++i) pw[i] = W + static_cast<int64_t>(min(n0 + i * 8 + g, N - 1)) * K;
#pragma unroll
  for (int j = 0; j < NT; ++j) px[j] = x + static_cast<int64_t>(min(j * 8 + g, M - 1)) * K;
  int next = begin + q * 8;                            // this lane's next k to copy
  uint32_t fill = 0;
  const auto prefetch = [&] {
    const int bytes = next < end ? 16 : 0;             // 0: zeros, nothing is read
    const int at = next < end ? next : 0;
    const uint32_t to = ring + fill * (T::kPieces * 512);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + i * 512),
                   "l"(pw[i] + at), "r"(bytes)
                   : "memory");
#pragma unroll
    for (int j = 0; j < NT; ++j)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(to + (2 + j) * 512),
                   "l"(px[j] + at), "r"(bytes)
                   : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
    next += 32;
    if (++fill == T::kStages) fill = 0;
  };
  const auto piece = [&](uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
  };
#pragma unroll
  for (int i = 0; i < T::kStages - 1; ++i) prefetch();
  float sum[NT][4] = {}, c[NT][4] = {};
  uint32_t slot = 0;
  const int steps = (end - begin + 31) / 32;
  for (int s = 0; s < steps; ++s) {
    asm volatile("cp.async.wait_group %0;" ::"n"(T::kStages - 2) : "memory");
    const uint32_t at = ring + slot * (T::kPieces * 512);
    const uint4 lo = piece(at), hi = piece(at + 512);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint4 b = piece(at + (2 + j) * 512);
      mma16816(c[j], lo.x, hi.x, lo.y, hi.y, b.x, b.y);
      mma16816(c[j], lo.z, hi.z, lo.w, hi.w, b.z, b.w);
    }
    prefetch();                                        // into the slot before this one
    if (++slot == T::kStages) slot = 0;
    if ((s & 3) == 3 || s + 1 == steps) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[j][i] += c[j][i], c[j][i] = 0.f;
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();                                     // the ring is free
  float* sums = reinterpret_cast<float*>(ring_raw);    // [warp][value][lane]
  float* mine = sums + warp * T::kValues * 32 + lane;
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) mine[(j * 4 + i) * 32] = sum[j][i];
  __syncthreads();
  // The slices share the values of their group out.
  const float* from = sums + (warp - slice) * T::kValues * 32 + lane;
  for (int v = slice; v < T::kValues; v += slices) {
    const int i = v & 3, j = v >> 2;
    const int col = n0 + (i >> 1) * 8 + g, m = j * 8 + 2 * q + (i & 1);
    if (col >= N || m >= M) continue;
    float total = 0.f;
    for (int w = 0; w < slices; ++w) total += from[(w * T::kValues + v) * 32];
    linear_store1(epi, static_cast<int64_t>(m) * N + col, col, total);
  }
}

template <int NT>
cudaError_t run_rows(const void* x, const void* W, int M, int N, int K, const LinearEpilogue& epi,
                     int* status, cudaStream_t st) {
  // K is shared out until there are 8 warps an SM or a slice has less than 256 k; blocks of 16
  // warps where all of them share a group's K (6400 -> 1600, 8 rows: 7.6 us, with 8 warps 9.5;
  // 1600 -> 6400, which has 4 slices: 10.1 and 7.3).
  const int64_t tiles = (N + 15) / 16;
  int slices = 1;
  while (slices < 16 && slices * 256 <= K && tiles * slices < 8 * sm_count()) slices *= 2;
  const int warps = slices == 16 ? 16 : 8;
  const int per = warps / slices * 16;
  const size_t smem = warps * RowsTile<NT>::kSmem;
  auto* kernel = linear_rows_kernel<NT>;
  cudaError_t e = set_max_smem(reinterpret_cast<const void*>(kernel), 16 * RowsTile<NT>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_after(kernel, dim3((N + per - 1) / per), dim3(32 * warps), smem, 1, st,
                      static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(W), M, N, K,
                      slices, epi, status);
}

// --------------------------------------------------------------- operand planes
// Eight columns of a row from `col` (a multiple of 8) as loaded; columns from `cols` on are 0.
// V = 8: the row is 16-byte aligned and the eight exist.
template <typename E, int V> struct Chunk;
template <typename E> struct Chunk<E, 8> {
  Raw<E, 8> r;
  __device__ __forceinline__ void load(const void* p, int64_t at, int, int) { r.load(p, at); }
  __device__ __forceinline__ void get(float* f) const { r.get(f); }
};
template <typename E> struct Chunk<E, 1> {
  Raw<E, 1> r[8];
  int n;
  __device__ __forceinline__ void load(const void* p, int64_t at, int col, int cols) {
    n = cols - col;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) r[j].load(p, at + j);
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[j] = 0.f;
      if (j < n) r[j].get(f + j);
    }
  }
};

template <int NP>
__device__ __forceinline__ void store_planes(uint16_t* dst, int64_t plane, int64_t at,
                                             const float* f) {
  float p[3][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float q[3];
    if (NP == 1) {
      q[0] = f[j];
    } else {
      split(f[j], q);
    }
#pragma unroll
    for (int n = 0; n < NP; ++n) p[n][j] = q[n];
  }
#pragma unroll
  for (int n = 0; n < NP; ++n) Out<BF16, 8>::store(dst + n * plane, at, p[n]);
}

// [rows][cols] of E -> NP planes [rows][ld] of bf16, ld a multiple of 8; two arrays of as many
// columns at a time (the second may have no rows).
struct PlanesOf {
  const void* src;
  uint16_t* dst;
  int64_t rows;
};
template <typename E, int V, int NP>
__global__ void __launch_bounds__(256) linear_planes_kernel(const PlanesOf a, const PlanesOf b,
                                                            int cols, int64_t ld, int* status) {
  let_next_in();
  wait_for_previous();
  clear_status(status);
  const int chunks = static_cast<int>(ld / 8);
  const int64_t total = (a.rows + b.rows) * chunks;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    int64_t r = i / chunks;
    const int col = static_cast<int>(i - r * chunks) * 8;
    const bool second = r >= a.rows;
    if (second) r -= a.rows;
    const int64_t rows = second ? b.rows : a.rows;
    float f[8];
    Chunk<E, V> c;
    c.load(second ? b.src : a.src, r * cols + col, col, cols);
    c.get(f);
    store_planes<NP>(second ? b.dst : a.dst, rows * ld, r * ld + col, f);
  }
}

cudaError_t make_planes(const PlanesOf& a, const PlanesOf& b, int dtype, int cols, int* status,
                        cudaStream_t st) {
  const int64_t ld = pad8(cols);
  const int64_t blocks = ((a.rows + b.rows) * (ld / 8) + 255) / 256;
  const unsigned grid = static_cast<unsigned>(blocks < 148 * 32 ? blocks : 148 * 32);
  const bool vec = cols % 8 == 0;
  auto* kernel = dtype == PKM_BF16 ? linear_planes_kernel<BF16, 1, 1>
                 : vec             ? linear_planes_kernel<F32, 8, 3>
                                   : linear_planes_kernel<F32, 1, 3>;
  return launch_after(kernel, grid, 256, 0, 1, st, a, b, cols, ld, status);
}

// ------------------------------------------------------------ d = grad_y act'(pre)
// Block: 256 columns (32 lanes of 8) x `per` rows (8 warps, every eighth row each). d is
// written as NP planes (NP = 0: not needed) and its column sums as one partial row per block
// row (part NULL: not needed). Bound by HBM and the slope's arithmetic together: 4096 x 6400
// bf16, gelu, three planes, 262 MB: 58 us with four blocks an SM (two, of which
// each thread has two rows in flight, took 5 us more).
// Rows of a block: 64, or fewer (a warp then has fewer one after the other) until there are two
// blocks for each of the 148 SMs (the whole backward of 777 x 4096 -> 1024 bf16 gelu: 58 us on the
// device, with 64 rows 69).
int slope_rows(int64_t rows, int cols) {
  int per = 64;
  while (per > 8 && (rows + per - 1) / per * ((cols + 255) / 256) < 2 * 148) per /= 2;
  return per;
}
int64_t slope_blocks(int64_t rows, int cols) {
  const int per = slope_rows(rows, cols);
  return (rows + per - 1) / per;
}

template <typename E, int V, int NP>
__global__ void __launch_bounds__(256, 4) linear_slope_kernel(const void* gy, const void* pre,
                                                           int act, uint16_t* dst, float* part,
                                                           int64_t rows, int cols, int64_t ld,
                                                           int per, int* status) {
  __shared__ float sh[8][256];
  let_next_in();
  wait_for_previous();
  clear_status(status);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.y * 256 + lane * 8;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * per;
  float sum[8] = {};
  if (col < cols) {
    const int64_t r1 = r0 + per < rows ? r0 + per : rows;
    for (int64_t r = r0 + warp; r < r1; r += 8) {
      float g[8], t[8];
      Chunk<E, V> gc, tc;
      gc.load(gy, r * cols + col, col, cols);
      if (act != PKM_ACT_NONE) tc.load(pre, r * cols + col, col, cols);
      gc.get(g);
      if (act != PKM_ACT_NONE) {
        tc.get(t);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] *= act_slope(t[j], act);
      }
      if (NP > 0) store_planes<NP>(dst, rows * ld, r * ld + col, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += g[j];
    }
  }
  if (!part) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) sh[warp][lane * 8 + j] = sum[j];
  __syncthreads();
  const int c = blockIdx.y * 256 + threadIdx.x;
  if (c < cols) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sh[w][threadIdx.x];
    part[static_cast<int64_t>(blockIdx.x) * cols + c] = s;
  }
}

__global__ void __launch_bounds__(256) linear_bias_kernel(const float* part, int64_t blocks,
                                                          int cols, float* out) {
  let_next_in();
  wait_for_previous();
  __shared__ float sh[8][33];
  const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  float s = 0.f;
  if (col < cols)
    for (int64_t r = k; r < blocks; r += 8) s += part[r * cols + col];
  sh[k][c] = s;
  __syncthreads();
  if (k == 0 && col < cols) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a += sh[i][c];
    out[col] = a;
  }
}

template <typename E, int V>
cudaError_t run_slope(int planes, const void* gy, const void* pre, int act, uint16_t* dst,
                      float* part, int64_t rows, int cols, int* status, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(slope_blocks(rows, cols)),
                  static_cast<unsigned>((cols + 255) / 256));
  const int64_t ld = pad8(cols);
  auto* kernel = planes == 0 ? linear_slope_kernel<E, V, 0> : linear_slope_kernel<E, V, 3>;
  if constexpr (sizeof(typename E::T) == 2) {   // fp32 layers use all planes
    if (planes == 1) kernel = linear_slope_kernel<E, V, 1>;
    if (planes == 2) kernel = linear_slope_kernel<E, V, 2>;
  }
  return launch_after(kernel, grid, 256, 0, 1, st, gy, pre, act, dst, part, rows, cols, ld,
                      slope_rows(rows, cols), status);
}

// ------------------------------------------------------------------- host side
// How a product is shared out over the 74 pairs of CTAs of a B200 (fixed, because the
// workspace's size depends on it), counted in K steps of a tile (0.3 us). More tiles than
// pairs: whole rounds, and the tiles of the last one cut along K over all pairs where that
// saves more than the parts cost (below). Fewer: cut for more pairs where that takes less
// time: the longest range, the join kernel (12), and each pair's part, written and read at
// about 5 TB/s (256 rows: a third). 777 x 4096 -> 1024 takes 20.8 us cut and 28.5 whole, 2048 x
// 2048 -> 2048 27 and 19.7; grad_W of 4096 x 1600 -> 6400 gelu, 175 tiles, 265 us with the last
// 27 cut and 305 whole.
constexpr int kPairs = 74;
constexpr int kMinSteps = 8;      // of a range

LinearWork share_out(int64_t M, int64_t N, int64_t K, int products) {
  const int kblocks = static_cast<int>((K + 63) / 64);
  const int64_t tiles = ((M + kLinearTileM - 1) / kLinearTileM) *
                        ((N + kLinearTileN - 1) / kLinearTileN);
  const int64_t steps = static_cast<int64_t>(kblocks) * products;   // of one tile
  LinearWork best{static_cast<int>(tiles < kPairs ? tiles : kPairs), static_cast<int>(tiles), 0,
                  kblocks};
  if (tiles > kPairs) {
    const int rest = static_cast<int>(tiles % kPairs);
    const double idle = static_cast<double>(steps) * (kPairs - rest) / kPairs;
    if (rest && rest * steps >= kPairs * kMinSteps && idle > 12 + kPairs / 3.0) {
      best.cut = rest;
      best.whole -= rest;
    }
    return best;
  }
  double least = static_cast<double>(steps);
  const double rows = M < kLinearTileM ? static_cast<double>(M) / kLinearTileM : 1.0;
  for (int64_t ways = 2; ways <= 32; ++ways) {
    const int64_t pairs = ways * tiles < kPairs ? ways * tiles : kPairs;
    // No range is empty, or too short to be worth it.
    if (pairs > tiles * kblocks || pairs * kMinSteps > tiles * steps) break;
    const double cost = static_cast<double>(tiles * steps) / pairs + 12 + rows * pairs / 3;
    if (cost < least) {
      least = cost;
      best = {static_cast<int>(pairs), 0, static_cast<int>(tiles), kblocks};
    }
    if (pairs == kPairs) break;
  }
  return best;
}

// The products of a's and b's planes, p + q below the larger plane count, smallest first.
LinearSteps plane_steps(int a, int b) {
  const auto step = [](int pb, int count, int p0, int p1, int p2) {
    return static_cast<uint64_t>(p0 | p1 << 4 | p2 << 8 | pb << 12 | count << 14);
  };
  if (a == 3 && b == 3)
    return {step(2, 1, 0, 0, 0) | step(1, 2, 1, 0, 0) << 16 | step(0, 2, 2, 1, 0) << 32 |
                step(0, 1, 0, 0, 0) << 48, 4, 6};
  if (a == 3) return {step(0, 3, 2, 1, 0), 1, 3};
  if (a == 2) return {step(0, 2, 1, 0, 0), 1, 2};
  return {step(0, 1, 0, 0, 0), 1, 1};
}

// Number of planes of an operand of the layer's type; in place (0 bytes) for bf16 rows of
// 16-byte multiples.
int input_planes(int dtype) { return dtype == PKM_F32 ? 3 : 1; }
bool in_place(int dtype, int cols) { return dtype == PKM_BF16 && cols % 8 == 0; }
size_t planes_bytes(int dtype, int64_t rows, int cols) {
  return in_place(dtype, cols) ? 0 : align256(static_cast<size_t>(rows) * pad8(cols) * 2 *
                                              input_planes(dtype));
}

size_t part_bytes(const LinearWork& w) {
  return w.cut ? static_cast<size_t>(2 * w.pairs) * kLinearTileM * kLinearTileN * 4 : 0;
}

// The backward's d: planes written (0: grad_y itself is the operand).
int slope_planes(const LinearArgs& a) {
  if (a.dtype == PKM_F32 || a.act != PKM_ACT_NONE) return 3;
  return a.N % 8 == 0 ? 0 : 1;
}
// Those that grad_x takes. In bf16 two are enough: they are d to 2^-16, 1 / 256 of grad_x's own
// rounding (one plane alone is as large as that: 2.35e-3 of grad_x where 1.66e-3 is its rounding;
// the second takes 385 us to 479 for the backward of 4096 x 1600 -> 6400 gelu). relu's d is
// grad_y or 0: one.
int grad_x_planes(const LinearArgs& a) {
  const int d = slope_planes(a);
  if (d < 3 || a.dtype == PKM_F32 || a.out_dtype == PKM_F32) return d;
  return a.act == PKM_ACT_RELU ? 1 : 2;
}

// The forward of few rows on the warps' matrix instructions: from 5 rows of bf16 on (4 rows, 4096
// -> 1024: 5.4 us, the small-batch kernel 4.4), up to 16, or 32 where W is small enough that the
// rereading of x (M / 16 times W's bytes) is hidden (32 rows, 4096 -> 4096: 15.3 us, the tensor-core
// kernel 15.8; 4096 -> 8192: 24.6 and 21.5).
bool linear_rows(const LinearArgs& a) {
  return a.dtype == PKM_BF16 && a.K % 8 == 0 && a.M > 4 &&
         (a.M <= 16 || (a.M <= 32 && static_cast<int64_t>(a.N) * a.K <= 1 << 24));
}

struct Layout {
  size_t x, W, d, part, bias, total;   // offsets; total = bytes
  LinearWork fwd, gx, gw;
  LinearSteps fwd_p, gx_p, gw_p;
};

Layout layout(const LinearArgs& a, bool backward) {
  Layout l{};
  size_t off = kStatusBytes;
  const int in = input_planes(a.dtype);
  l.x = off;
  off += planes_bytes(a.dtype, a.M, a.K);
  l.W = off;
  off += planes_bytes(a.dtype, a.N, a.K);
  l.part = off;
  if (!backward) {
    l.fwd_p = plane_steps(in, in);
    l.fwd = share_out(a.M, a.N, a.K, l.fwd_p.products);
    off += part_bytes(l.fwd);
  } else {
    const int d = slope_planes(a), dx = grad_x_planes(a);
    l.gx_p = plane_steps(dx ? dx : 1, in);
    l.gw_p = plane_steps(d ? d : 1, in);
    l.gx = share_out(a.M, a.K, a.N, l.gx_p.products);
    l.gw = share_out(a.N, a.K, a.M, l.gw_p.products);
    const size_t px = part_bytes(l.gx), pw = part_bytes(l.gw);
    off += px > pw ? px : pw;    // the two products run one after the other
    l.d = off;
    off += align256(static_cast<size_t>(a.M) * pad8(a.N) * 2 * d);
    l.bias = off;
    off += align256(static_cast<size_t>(slope_blocks(a.M, a.N)) * a.N * 4);
  }
  l.total = off;
  return l;
}

}  // namespace

bool linear_small(const LinearArgs& a) { return a.M <= kSmallM || linear_rows(a); }

size_t linear_workspace_bytes(const LinearArgs& a, bool backward) {
  if (a.M == 0 || (!backward && linear_small(a)) || linear_f32(a, backward)) return kStatusBytes;
  return layout(a, backward).total;
}

cudaError_t launch_linear_forward(const LinearArgs& a, const void* x, const void* W,
                                  const float* bias, const void* residual, void* y, void* pre,
                                  void* workspace, int* launches, cudaStream_t st) {
  LinearEpilogue epi{y, bias, residual, pre, a.out_dtype == PKM_F32,
                     a.dtype == PKM_F32, a.act};
  int* status = static_cast<int*>(workspace);
  int* first = status;   // what the next kernel clears: only the call's first one does
  cudaError_t e = cudaSuccess;
  if (linear_small(a)) {
    ++*launches;
    const int M = static_cast<int>(a.M);
    const bool vec = a.K % (a.dtype == PKM_F32 ? 4 : 8) == 0;   // rows of whole 16 bytes
    if (linear_rows(a)) {
      if (M <= 8) return run_rows<1>(x, W, M, a.N, a.K, epi, first, st);
      if (M <= 16) return run_rows<2>(x, W, M, a.N, a.K, epi, first, st);
      return run_rows<4>(x, W, M, a.N, a.K, epi, first, st);
    }
    if (a.dtype == PKM_F32)
      return vec ? run_small<F32, 4>(M, x, W, a.N, a.K, epi, first, st)
                 : run_small<F32, 1>(M, x, W, a.N, a.K, epi, first, st);
    return vec ? run_small<BF16, 8>(M, x, W, a.N, a.K, epi, first, st)
               : run_small<BF16, 1>(M, x, W, a.N, a.K, epi, first, st);
  }
  if (linear_f32(a, false))
    return launch_f32_forward(a, static_cast<const float*>(x), static_cast<const float*>(W), epi,
                              status, launches, st);
  const Layout l = layout(a, false);
  char* ws = static_cast<char*>(workspace);
  const int64_t ld = pad8(a.K);
  if (!in_place(a.dtype, a.K)) {
    e = make_planes({x, reinterpret_cast<uint16_t*>(ws + l.x), a.M},
                    {W, reinterpret_cast<uint16_t*>(ws + l.W), a.N}, a.dtype, a.K, first, st);
    if (e != cudaSuccess) return e;
    first = nullptr;
    x = ws + l.x;
    W = ws + l.W;
    ++*launches;
  }
  const uint32_t in = static_cast<uint32_t>(input_planes(a.dtype));
  const LinearGemm g{kForward, x, W, ld, ld, static_cast<int>(a.M), a.N, a.K, in, in, l.fwd_p, l.fwd,
                     l.fwd.cut ? reinterpret_cast<float*>(ws + l.part) : nullptr, epi, status,
                     first != nullptr};
  return launch_linear_gemm(g, launches, st);
}

cudaError_t launch_linear_backward(const LinearArgs& a, const void* x, const void* W,
                                   const void* grad_y, const void* pre, void* grad_x,
                                   float* grad_W, float* grad_bias, void* workspace,
                                   int* launches, cudaStream_t st) {
  if (linear_f32(a, true))
    return launch_f32_backward(a, static_cast<const float*>(x), static_cast<const float*>(W),
                               static_cast<const float*>(grad_y), static_cast<const float*>(pre),
                               grad_x, grad_W, grad_bias, static_cast<int*>(workspace), launches, st);
  const Layout l = layout(a, true);
  char* ws = static_cast<char*>(workspace);
  int* status = static_cast<int*>(workspace);
  int* first = status;   // what the next kernel clears: only the call's first one does
  cudaError_t e = cudaSuccess;
  const int dp = slope_planes(a);
  const int64_t ldn = pad8(a.N), ldk = pad8(a.K);
  uint16_t* d = reinterpret_cast<uint16_t*>(ws + l.d);
  const bool want_d = grad_x || grad_W;
  if (grad_bias || (want_d && dp > 0)) {
    float* part = grad_bias ? reinterpret_cast<float*>(ws + l.bias) : nullptr;
    const int planes = !want_d ? 0 : grad_W ? dp : grad_x_planes(a);
    const bool vec = a.N % 8 == 0;
    if (a.dtype == PKM_F32)
      e = vec ? run_slope<F32, 8>(planes, grad_y, pre, a.act, d, part, a.M, a.N, first, st)
              : run_slope<F32, 1>(planes, grad_y, pre, a.act, d, part, a.M, a.N, first, st);
    else
      e = vec ? run_slope<BF16, 8>(planes, grad_y, pre, a.act, d, part, a.M, a.N, first, st)
              : run_slope<BF16, 1>(planes, grad_y, pre, a.act, d, part, a.M, a.N, first, st);
    if (e != cudaSuccess) return e;
    first = nullptr;
    ++*launches;
    if (grad_bias) {
      e = launch_after(linear_bias_kernel, (a.N + 31) / 32, 256, 0, 1, st, part,
                       slope_blocks(a.M, a.N), a.N, grad_bias);
      if (e != cudaSuccess) return e;
      ++*launches;
    }
  }
  if (!want_d) return cudaSuccess;
  const void* dop = dp ? static_cast<const void*>(d) : grad_y;
  const uint32_t dcount = dp ? dp : 1, in = static_cast<uint32_t>(input_planes(a.dtype));
  const bool inpl = in_place(a.dtype, a.K);
  float* part = reinterpret_cast<float*>(ws + l.part);
  if (!inpl) {   // W's planes for grad_x, x's for grad_W
    e = make_planes({W, reinterpret_cast<uint16_t*>(ws + l.W), grad_x ? a.N : 0},
                    {x, reinterpret_cast<uint16_t*>(ws + l.x), grad_W ? a.M : 0}, a.dtype, a.K,
                    first, st);
    if (e != cudaSuccess) return e;
    first = nullptr;
    W = ws + l.W;
    x = ws + l.x;
    ++*launches;
  }
  if (grad_x) {
    const LinearEpilogue epi{grad_x, nullptr, nullptr, nullptr, a.out_dtype == PKM_F32, 0,
                             PKM_ACT_NONE};
    const LinearGemm g{kGradX, dop, W, ldn, ldk, static_cast<int>(a.M), a.K, a.N, dcount, in,
                       l.gx_p, l.gx, l.gx.cut ? part : nullptr, epi,
                       status, first != nullptr};
    e = launch_linear_gemm(g, launches, st);
    if (e != cudaSuccess) return e;
    first = nullptr;
  }
  if (grad_W) {
    const LinearEpilogue epi{grad_W, nullptr, nullptr, nullptr, 1, 0, PKM_ACT_NONE};
    const LinearGemm g{kGradW, dop, x, ldn, ldk, a.N, a.K, static_cast<int>(a.M), dcount, in,
                       l.gw_p, l.gw, l.gw.cut ? part : nullptr, epi,
                       status, first != nullptr};
    e = launch_linear_gemm(g, launches, st);
  }
  return e;
}

}  // namespace pkm
