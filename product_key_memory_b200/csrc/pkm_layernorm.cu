// pkm_layernorm.cu -- layer norm (with the residual addition before it) and its backward.
//
// Forward, per row:  h = x + add, mean = sum h / d, rstd = 1/sqrt(sum (h - mean)^2 / d + eps),
// y = (h - mean) rstd gamma + beta. The row is read once and stays in registers for the
// three uses; a row belongs to T threads (a part of a warp, a warp, or several warps). Bound
// by HBM: 16384 rows of 1024, fp32 x, add and h, bf16 y: 40 us, 5.9 TB/s.
//
// Backward, per row, with xhat = (x - mean) rstd and t = grad_y gamma:
//   grad_x = rstd (t - sum t / d - xhat sum (t xhat) / d) + grad_sum
// and over the rows grad_gamma = sum grad_y xhat, grad_beta = sum grad_y. A group of T
// threads keeps the same columns for all of its rows, so the column sums stay in its
// registers; each block writes one partial row, and a second kernel adds the partial
// rows in a fixed order. 16384 rows of 1600, fp32 grad_y, the others bf16: 60 us, 4.4 TB/s;
// the row's reduction, between its reads and its writes, keeps it from the copy's rate.
#include "pkm_block.h"
#include "pkm_elem.cuh"
#include "pkm_kernels.h"
#include "pkm_tc.h"

namespace pkm {

namespace {

constexpr int kMaxNormThreads = 512;

// Barrier of the `threads` threads of group g of a block (whole warps).
__device__ __forceinline__ void group_barrier(int g, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(threads) : "memory");
}

// Sum over the lanes of a row and its warps; `red` holds a float for each of those. Callers take
// turns with two arrays.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, int wide, int group, int w, float* red) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (wide > 1) {
    if ((threadIdx.x & 31) == 0) red[w] = v;
    group_barrier(group, wide * 32);
    v = 0.f;
    for (int i = 0; i < wide; ++i) v += red[i];
  }
  return v;
}

// V = 4: rows of a multiple of 4 columns, four at a time, contiguous over the lanes. V = 1: any.
// A row belongs to LANES lanes of `wide` warps (1 where LANES < 32), H accesses each.
template <typename X, typename Y, int V, int H, int LANES>
__global__ void __launch_bounds__(kMaxNormThreads)
layernorm_forward_kernel(const void* x, const void* add, int add_f32,
                         const float* __restrict__ gamma, const float* __restrict__ beta, void* y,
                         void* sum, float* mean_out, float* rstd_out, int64_t rows, int d, int wide,
                         float eps) {
  __shared__ float red[2][kMaxNormThreads / 32];
  let_next_in();
  wait_for_previous();
  const int lane = threadIdx.x & (LANES - 1), part = threadIdx.x / LANES;
  const int group = part / wide, w = part - group * wide;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / (LANES * wide)) + group;
  const bool live = row < rows;   // all lanes and warps stay for shuffles and barriers
  constexpr int kHop = LANES * V;
  const int col0 = w * (H * kHop) + lane * V;
  const int64_t base = row * d + col0;
  float h[H][V];
  Raw<X, V> rx[H];
#pragma unroll
  for (int c = 0; c < H; ++c)
    if (live && col0 + c * kHop < d) rx[c].load(x, base + c * kHop);
  const auto widen_sum = [&](auto& ra) {
#pragma unroll
    for (int c = 0; c < H; ++c)
      if (live && col0 + c * kHop < d) ra[c].load(add, base + c * kHop);
#pragma unroll
    for (int c = 0; c < H; ++c) {
      float f[V];
      rx[c].get(h[c]);
      ra[c].get(f);
#pragma unroll
      for (int v = 0; v < V; ++v) h[c][v] = rounded<X>(h[c][v] + f[v]);
      if (live && col0 + c * kHop < d) Out<X, V>::store(sum, base + c * kHop, h[c]);
    }
  };
  if (!add) {
#pragma unroll
    for (int c = 0; c < H; ++c) rx[c].get(h[c]);
  } else if (add_f32) {
    Raw<F32, V> ra[H];
    widen_sum(ra);
  } else {
    Raw<BF16, V> ra[H];
    widen_sum(ra);
  }
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < H; ++c) {
    const bool in = live && col0 + c * kHop < d;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!in) h[c][v] = 0.f;
      s += h[c][v];
    }
  }
  const float mean = row_sum<LANES>(s, wide, group, w, &red[0][group * wide]) / static_cast<float>(d);
  float q = 0.f;
#pragma unroll
  for (int c = 0; c < H; ++c) {
    const bool in = live && col0 + c * kHop < d;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[c][v] -= mean;
      if (in) q = fmaf(h[c][v], h[c][v], q);
    }
  }
  const float rstd = 1.f / sqrtf(row_sum<LANES>(q, wide, group, w, &red[1][group * wide]) /
                                     static_cast<float>(d) + eps);
  if (live && w == 0 && lane == 0) {
    if (mean_out) mean_out[row] = mean;
    if (rstd_out) rstd_out[row] = rstd;
  }
#pragma unroll
  for (int c = 0; c < H; ++c) {
    const int col = col0 + c * kHop;
    if (!live || col >= d) continue;
    float g[V], b[V];
    load_param<V>(gamma, col, g);
    if (beta) load_param<V>(beta, col, b);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float n = h[c][v] * rstd * g[v];
      h[c][v] = beta ? n + b[v] : n;
    }
    Out<Y, V>::store(y, base + c * kHop, h[c]);
  }
}

int round32(int x) { return (x + 31) / 32 * 32; }

struct FwdLaunch {
  int64_t rows;
  int d, add_f32;
  const void *x, *add;
  const float *gamma, *beta;
  void *y, *sum;
  float *mean, *rstd;
  float eps;
  cudaStream_t st;
};

template <typename X, typename Y, int V, int H, int LANES = 32>
cudaError_t run_fwd(const FwdLaunch& l) {
  const int wide = (l.d + LANES * V * H - 1) / (LANES * V * H);
  // Blocks of 256 threads, or of one row that is wider.
  const int per = LANES * wide >= 256 ? 1 : 256 / (LANES * wide);
  const int threads = round32(LANES * wide * per);
  const int64_t blocks = (l.rows + per - 1) / per;
  return launch_after(layernorm_forward_kernel<X, Y, V, H, LANES>, dim3(static_cast<unsigned>(blocks)),
                      dim3(threads), 0, 1, l.st, l.x, l.add, l.add_f32, l.gamma, l.beta, l.y, l.sum,
                      l.mean, l.rstd, l.rows, l.d, wide, l.eps);
}

template <typename X, typename Y>
cudaError_t pick_fwd(const FwdLaunch& l) {
  const int d = l.d;
  if (d % 4 == 0) {
    const int pieces = (d + 127) / 128;   // of a warp's access
    if (d <= 64) return run_fwd<X, Y, 4, 2, 8>(l);
    // Few rows: more warps for each, for latency. Else a warp for up to 512 columns (16384 fp32
    // rows of 1600: 39 us, with 1024 columns 45), or 1024 where that is too many warps.
    if (pieces <= 1 || (l.rows <= 4 * sm_count() && pieces <= 16)) return run_fwd<X, Y, 4, 1>(l);
    if (pieces <= 2) return run_fwd<X, Y, 4, 2>(l);
    if (pieces <= 32) return run_fwd<X, Y, 4, 4>(l);
    return run_fwd<X, Y, 4, 8>(l);
  }
  if (d <= 32) return run_fwd<X, Y, 1, 4, 8>(l);
  if (d <= 128) return run_fwd<X, Y, 1, 4>(l);
  if (d <= 256) return run_fwd<X, Y, 1, 8>(l);
  // 512 columns a warp (65280 bf16 rows of 257: 45 us, with 256 columns 65; fp32 rows of 2001:
  // 33 and 41).
  if (d <= 16 * 32 * 16) return run_fwd<X, Y, 1, 16>(l);
  return run_fwd<X, Y, 1, 32>(l);
}

// ------------------------------------------------------------------ backward
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <typename E> constexpr int kSize = sizeof(typename E::T);

// Four elements from shared memory as pairs.
struct Four {
  Pair a, b;
};
template <bool F32_>
__device__ __forceinline__ Four lds_four(uint32_t addr) {
  Four f;
  if (F32_) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    f.a = Pair(v.x, v.y), f.b = Pair(v.z, v.w);
  } else {
    uint32_t x, y;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(addr) : "memory");
    f.a = Pair(bf16_lo(x), bf16_hi(x)), f.b = Pair(bf16_lo(y), bf16_hi(y));
  }
  return f;
}

template <typename O>
__device__ __forceinline__ void store_four(void* base, int64_t i, Pair a, Pair b) {
  const float2 x = a.get(), y = b.get();
  if (kSize<O> == 4)
    *reinterpret_cast<float4*>(static_cast<float*>(base) + i) = make_float4(x.x, x.y, y.x, y.y);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + i) =
        make_uint2(pack_bf16(x.x, x.y), pack_bf16(y.x, y.y));
}

// (-1/d) sums over the T threads of a row (or of two rows, R = 2) of s1 and s2, T <= 32 a power
// of two (lanes of a warp) or a multiple of 32 (warps; `red` is then the half of the
// group's array that this step uses: the halves alternate, so one barrier is enough).
template <int R, bool WARPS>
__device__ __forceinline__ void row_sums(float (&s1)[R], float (&s2)[R], int T, int group, int w,
                                         float4* red, float ninv_d) {
  if constexpr (WARPS) {
    // The lanes' upper half goes on with s2; with two rows, the upper quarters with the second.
    const bool up = threadIdx.x & 16, second = threadIdx.x & 8;
    float v[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      v[r] = (up ? s2[r] : s1[r]) + __shfl_xor_sync(0xffffffffu, up ? s1[r] : s2[r], 16);
    float q;
    if constexpr (R == 2)
      q = (second ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, second ? v[0] : v[1], 8);
    else
      q = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
    if ((threadIdx.x & 7) == 0) reinterpret_cast<float*>(red + w)[(second ? 2 : 0) + up] = q;
    group_barrier(group, T);
    const int warps = T >> 5;
    float4 f = red[0];
#pragma unroll 4
    for (int i = 1; i < warps; ++i) {
      const float4 g = red[i];
      f.x += g.x, f.y += g.y, f.z += g.z, f.w += g.w;
    }
    s1[0] = f.x * ninv_d, s2[0] = f.y * ninv_d;
    if constexpr (R == 2) s1[1] = f.z * ninv_d, s2[1] = f.w * ninv_d;
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      for (int o = T >> 1; o > 0; o >>= 1) {
        s1[r] += __shfl_xor_sync(0xffffffffu, s1[r], o);
        s2[r] += __shfl_xor_sync(0xffffffffu, s2[r], o);
      }
      s1[r] *= ninv_d, s2[r] *= ninv_d;
    }
  }
}

// A block's partial column sums, added over its groups in order by way of sh[group][2][d], into
// its row of `part`. Thread values are put in place by `put(destination of [2][d])`.
template <typename Put>
__device__ __forceinline__ void store_part(float* part, float* sh, int d, int group, int per,
                                           const Put& put) {
  float* pg = part + static_cast<int64_t>(blockIdx.x) * 2 * d;
  put(per == 1 ? pg : sh + group * 2 * d);
  if (per == 1) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * d; i += blockDim.x) {
    float s = 0.f;
    for (int g = 0; g < per; ++g) s += sh[g * 2 * d + i];
    pg[i] = s;
  }
}

// Rows of 16-byte multiples (d a multiple of 8). A block holds `per` groups of T threads, group
// g of the grid takes R rows at a time (two of up to 4096 columns: the reduction, the
// barrier and the addresses, most of the instructions, come once for both). A warp (or, T <
// 32, a group) owns spans of 8 columns a lane, each lane the four at 4 l and the four half
// a span further, so that its accesses to fp32 and to bf16 arrays are both contiguous over
// the lanes. It copies its spans of the next rows into shared memory ahead of time, 16
// bytes a lane and contiguous (16 of every 32 bytes at a time took 71 us where this took 48,
// 16384 fp32 rows of 1024), so memory stays busy across the reduction and barrier.
template <typename X, typename G, typename O, int C, bool WARPS>
__global__ void __launch_bounds__(kMaxNormThreads, 1)
layernorm_backward_kernel(const void* gy, const void* x, const float* __restrict__ mean,
                          const float* __restrict__ rstd, const float* __restrict__ gamma,
                          const void* gsum, int gsum_f32, void* gx, float* part, int64_t rows,
                          int d, int T, int per, int stages) {
  extern __shared__ __align__(16) float sh[];   // the ring; at the end the groups' column sums
  __shared__ float4 red[2][kMaxNormThreads / 32];
  wait_for_previous();
  constexpr int R = C == 1 ? 2 : 1;
  constexpr int kX = kSize<X>, kG = kSize<G>, kO = kSize<O>;
  const int group = threadIdx.x / T;
  const int t = threadIdx.x - group * T;
  const int lanes = WARPS ? 32 : T;                    // of a span
  const int l = t & (lanes - 1);
  const int half = lanes * 4;                          // columns
  const float ninv_d = -1.f / static_cast<float>(d);
  const int ks = gsum ? (gsum_f32 ? 4 : 2) : 0;
  const int span = lanes * 8 * (kX + kG + ks);         // bytes of one span of all arrays
  const int at_g = lanes * 8 * kX, at_s = lanes * 8 * (kX + kG);
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(sh)) +
                        static_cast<uint32_t>(threadIdx.x / lanes) * (stages * R * C * span);
  const uint32_t ring_end = ring + stages * R * C * span;
  const uint32_t nrows = static_cast<uint32_t>(rows), stride = gridDim.x * per * R;
  const int first_col = (t / lanes) * 2 * half;        // of this warp's span, access 0
  const int hop = T * 8;                               // columns from one access to the next
  const uint32_t row_step = stride * d;                // elements

  // Cursors of the copies (16 bytes a lane, two for fp32) and of the results.
  uint32_t frow = (blockIdx.x * per + group) * R;      // the next row to copy
  const int64_t start = static_cast<int64_t>(frow) * d + first_col;
  const int lane16 = l * 16, wide = lanes * 16;        // bytes
  const char* px = static_cast<const char*>(x) + start * kX + lane16;
  const char* pg = static_cast<const char*>(gy) + start * kG + lane16;
  const char* ps = static_cast<const char*>(gsum) + start * ks + lane16;
  char* po = static_cast<char*>(gx) + (start + 4 * l) * kO;
  const auto copy = [&](uint32_t dst, const char* p, int left, int size) {
    if (left > 0) copy_async16(dst, p);
    if (size == 4 && left > wide) copy_async16(dst + wide, p + wide);
  };
  uint32_t fslot = ring + lane16;
  const auto prefetch = [&]() {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (frow + r < nrows) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int left = d - first_col - c * hop;    // columns
          const uint32_t dst = fslot + (r * C + c) * span;
          copy(dst, px + (c * hop + r * d) * kX, left * kX - lane16, kX);
          copy(dst + at_g, pg + (c * hop + r * d) * kG, left * kG - lane16, kG);
          if (ks == 4) copy(dst + at_s, ps + (c * hop + r * d) * 4, left * 4 - lane16, 4);
          else if (ks == 2) copy(dst + at_s, ps + (c * hop + r * d) * 2, left * 2 - lane16, 2);
        }
      }
    }
    copy_commit();                                     // empty groups keep the count
    px += static_cast<int64_t>(row_step) * kX;
    pg += static_cast<int64_t>(row_step) * kG;
    ps += static_cast<int64_t>(row_step) * ks;
    frow += stride;
    fslot += R * C * span;
    if (fslot >= ring_end) fslot -= stages * R * C * span;
  };

  // [c][h]: columns first_col + c hop + h half + 4 l.
  Pair ag[C][2][2], ab[C][2][2], gm[C][2][2];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = first_col + c * hop + h * half + 4 * l;
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (col < d) f = __ldg(reinterpret_cast<const float4*>(gamma + col));
      gm[c][h][0] = Pair(f.x, f.y), gm[c][h][1] = Pair(f.z, f.w);
      ag[c][h][0] = ag[c][h][1] = ab[c][h][0] = ab[c][h][1] = Pair(0.f);
    }
  uint32_t row = frow;
  const float* pm = mean + row;
  const float* pr = rstd + row;
  for (int k = 0; k < stages - 1; ++k) prefetch();
  float mu[R] = {}, rstd_row[R] = {};
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (row + r < nrows) mu[r] = __ldg(pm + r), rstd_row[r] = __ldg(pr + r);
  float4* my_red = &red[0][group * (T >> 5)];
  uint32_t slot = ring;
  // Block-uniform trip count: every thread takes part in the reductions.
  for (uint32_t r0 = blockIdx.x * per * R; r0 < nrows; r0 += stride, row += stride) {
    __syncwarp();                                      // the slot has been read by every lane
    prefetch();
    pm += stride, pr += stride;
    float mu_next[R] = {}, rs_next[R] = {};
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (row + stride + r < nrows) mu_next[r] = __ldg(pm + r), rs_next[r] = __ldg(pr + r);
    if (stages == 3) copy_wait<2>();
    else if (stages == 2) copy_wait<1>();
    else copy_wait<0>();
    __syncwarp();
    Pair xh[R][C][2][2], tt[R][C][2][2];
    float s1[R], s2[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      Pair p1(0.f), p2(0.f);
      if (row + r < nrows) {
        // xhat = (x - mean) rstd, the difference first: fma(x, rstd, -mean rstd) would keep the
        // rounding of a product as large as the mean in deviations.
        const Pair rs(rstd_row[r]), off(-mu[r]);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (first_col + c * hop + h * half + 4 * l >= d) continue;
            const uint32_t at = slot + (r * C + c) * span;
            const Four fx = lds_four<kX == 4>(at + (h * half + 4 * l) * kX);
            const Four fg = lds_four<kG == 4>(at + at_g + (h * half + 4 * l) * kG);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const Pair g = v ? fg.b : fg.a;
              const Pair q = mul(add(v ? fx.b : fx.a, off), rs);
              const Pair w = mul(g, gm[c][h][v]);
              ag[c][h][v] = fma(g, q, ag[c][h][v]);
              ab[c][h][v] = add(g, ab[c][h][v]);
              p1 = add(w, p1);
              p2 = fma(w, q, p2);
              xh[r][c][h][v] = q;
              tt[r][c][h][v] = w;
            }
          }
      }
      s1[r] = p1.lo() + p1.hi(), s2[r] = p2.lo() + p2.hi();
    }
    row_sums<R, WARPS>(s1, s2, T, group, t >> 5, my_red, ninv_d);
    my_red = my_red >= red[1] ? my_red - kMaxNormThreads / 32 : my_red + kMaxNormThreads / 32;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row + r >= nrows) continue;
      const Pair rs(rstd_row[r]), m1(s1[r]), m2(s2[r]);
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (first_col + c * hop + h * half + 4 * l >= d) continue;
          Pair o[2];
#pragma unroll
          for (int v = 0; v < 2; ++v) o[v] = add(fma(xh[r][c][h][v], m2, tt[r][c][h][v]), m1);
          if (ks) {
            const uint32_t as = slot + (r * C + c) * span + at_s + (h * half + 4 * l) * ks;
            const Four f = ks == 4 ? lds_four<true>(as) : lds_four<false>(as);
            o[0] = fma(o[0], rs, f.a), o[1] = fma(o[1], rs, f.b);
          } else {
            o[0] = mul(o[0], rs), o[1] = mul(o[1], rs);
          }
          store_four<O>(po, r * d + c * hop + h * half, o[0], o[1]);
        }
    }
    po += static_cast<int64_t>(row_step) * kO;
#pragma unroll
    for (int r = 0; r < R; ++r) mu[r] = mu_next[r], rstd_row[r] = rs_next[r];
    slot += R * C * span;
    if (slot == ring_end) slot = ring;
  }
  let_next_in();
  if (!part) return;
  copy_wait<0>();
  __syncthreads();                                     // the ring is free
  store_part(part, sh, d, group, per, [&](float* to) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int col = first_col + c * hop + h * half + 4 * l;
        if (col >= d) continue;
        store_four<F32>(to, col, ag[c][h][0], ag[c][h][1]);
        store_four<F32>(to, d + col, ab[c][h][0], ab[c][h][1]);
      }
  });
}

// Rows of other lengths up to 4096: one element at a time, straight into registers (a warp's
// accesses are contiguous). 16760 bf16 rows of 1001: 52 us; by way of shared memory, as
// below, 58.
template <typename X, typename G, typename O, int C, bool WARPS>
__global__ void __launch_bounds__(kMaxNormThreads)
layernorm_backward_odd_kernel(const void* gy, const void* x, const float* __restrict__ mean,
                              const float* __restrict__ rstd, const float* __restrict__ gamma,
                              const void* gsum, int gsum_f32, void* gx, float* part, int64_t rows,
                              int d, int T, int per) {
  extern __shared__ float sh[];   // the groups' column sums
  __shared__ float4 red[2][kMaxNormThreads / 32];
  wait_for_previous();
  const int group = threadIdx.x / T;
  const int t = threadIdx.x - group * T;
  const float inv_d = 1.f / static_cast<float>(d);
  float ag[C], ab[C];
#pragma unroll
  for (int c = 0; c < C; ++c) ag[c] = ab[c] = 0.f;
  int flip = 0;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * per;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * per; r0 < rows; r0 += stride, flip ^= 1) {
    const int64_t row = r0 + group;
    const bool live = row < rows;
    const int64_t base = row * d;
    Raw<X, 1> rx[C];
    Raw<G, 1> rg[C];
    float s[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = c * T + t;
      if (live && col < d) {
        rx[c].load(x, base + col);
        rg[c].load(gy, base + col);
        s[c] = gsum ? (gsum_f32 ? load_elem(static_cast<const float*>(gsum), base + col)
                                : load_elem(static_cast<const uint16_t*>(gsum), base + col))
                    : 0.f;
      }
    }
    const float mu = live ? mean[row] : 0.f, rs = live ? rstd[row] : 0.f;
    float s1 = 0.f, s2 = 0.f;
    float xh[C], tt[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = c * T + t;
      if (live && col < d) {
        float xv, gv;
        rx[c].get(&xv);
        rg[c].get(&gv);
        xh[c] = (xv - mu) * rs;
        tt[c] = gv * __ldg(gamma + col);
        s1 += tt[c];
        s2 = fmaf(tt[c], xh[c], s2);
        ag[c] = fmaf(gv, xh[c], ag[c]);
        ab[c] += gv;
      }
    }
    float a1[1] = {s1}, a2[1] = {s2};
    row_sums<1, WARPS>(a1, a2, T, group, t >> 5, &red[flip][group * (T >> 5)], -inv_d);
    s1 = -a1[0], s2 = -a2[0];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = c * T + t;
      if (!live || col >= d) continue;
      const float o = rs * (tt[c] - s1 - xh[c] * s2) + s[c];
      Out<O, 1>::store(gx, base + col, &o);
    }
  }
  let_next_in();
  if (!part) return;
  store_part(part, sh, d, group, per, [&](float* to) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = c * T + t;
      if (col >= d) continue;
      to[col] = ag[c];
      to[d + col] = ab[c];
    }
  });
}

// Rows of other lengths above 4096, a block each: it copies the 16-byte pieces that its next rows
// touch into shared memory ahead of time, then works on single elements, contiguous over the
// threads (3354 bf16 rows of 5001: 54 us; straight into registers, 16 at a time, 299). A row
// begins anywhere in a piece.
__host__ __device__ constexpr int row_window(int d, int size) {
  return (d * size + 14) / 16 * 16 + 16;   // d * size bytes that start at most 15 into a block
}
// The blocks that hold `bytes` bytes from p, of an array that ends at `end`.
__device__ __forceinline__ void copy_row(uint32_t dst, const char* p, int bytes, const char* end,
                                         int t, int T) {
  const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
  for (int i = t * 16; i < shift + bytes; i += T * 16) {
    const char* q = p - shift + i;
    const int64_t left = end - q;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i), "l"(q),
                 "r"(left < 16 ? static_cast<int>(left) : 16)
                 : "memory");
  }
}
template <typename E> __device__ __forceinline__ float lds_elem(uint32_t at) {
  if constexpr (kSize<E> == 4) {
    float f;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(at) : "memory");
    return f;
  } else {
    uint16_t h;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(at) : "memory");
    return __uint_as_float(static_cast<uint32_t>(h) << 16);
  }
}

template <typename X, typename G, typename O, int C>
__global__ void __launch_bounds__(kMaxNormThreads)
layernorm_backward_wide_kernel(const void* gy, const void* x, const float* __restrict__ mean,
                              const float* __restrict__ rstd, const float* __restrict__ gamma,
                              const void* gsum, int gsum_f32, void* gx, float* part, int64_t rows,
                              int d, int stages) {
  extern __shared__ __align__(16) float sh[];   // the ring
  __shared__ float4 red[2][kMaxNormThreads / 32];
  wait_for_previous();
  constexpr int kX = kSize<X>, kG = kSize<G>;
  constexpr bool kHold = C <= 16;   // xhat and t stay in registers; else they are made twice
  constexpr int T = kMaxNormThreads;
  const int t = threadIdx.x;
  const float ninv_d = -1.f / static_cast<float>(d);
  const int ks = gsum ? (gsum_f32 ? 4 : 2) : 0;
  const int at_g = row_window(d, kX), at_s = at_g + row_window(d, kG);
  const int stage = at_s + (ks ? row_window(d, ks) : 0);
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(sh));
  float ag[C], ab[C];
#pragma unroll
  for (int c = 0; c < C; ++c) ag[c] = ab[c] = 0.f;
  const int64_t stride = gridDim.x;
  const char *cx = static_cast<const char*>(x), *cg = static_cast<const char*>(gy),
             *cs = static_cast<const char*>(gsum);
  int fill = 0;                                  // the slot that the next copy goes to
  const auto prefetch = [&](int64_t row) {
    if (row < rows) {
      const uint32_t to = ring + fill * stage;
      const int64_t at = row * d, n = rows * d;
      copy_row(to, cx + at * kX, d * kX, cx + n * kX, t, T);
      copy_row(to + at_g, cg + at * kG, d * kG, cg + n * kG, t, T);
      if (ks) copy_row(to + at_s, cs + at * ks, d * ks, cs + n * ks, t, T);
    }
    copy_commit();                               // empty groups keep the count
    if (++fill == stages) fill = 0;
  };
  int64_t row = blockIdx.x;
  for (int k = 0; k < stages - 1; ++k) prefetch(row + k * stride);
  float mu = __ldg(mean + row), rs = __ldg(rstd + row);   // no more blocks than rows
  int slot = 0, flip = 0;
  for (; row < rows; row += stride) {
    if (stages == 1) {
      __syncthreads();                                 // the row before has been read
      prefetch(row);
      copy_wait<0>();
    } else if (stages == 2) {
      copy_wait<0>();
    } else {
      copy_wait<1>();
    }
    __syncthreads();                                   // all threads' copies; the row before is free
    if (stages > 1) prefetch(row + (stages - 1) * stride);
    const bool more = row + stride < rows;
    const float mu_next = more ? __ldg(mean + row + stride) : 0.f;
    const float rs_next = more ? __ldg(rstd + row + stride) : 0.f;
    const int64_t base = row * d;
    // The element of column t.
    const uint32_t in = ring + slot * stage;
    const uint32_t sx = in + (static_cast<uint32_t>(base * kX) & 15) + t * kX;
    const uint32_t sg = in + at_g + (static_cast<uint32_t>(base * kG) & 15) + t * kG;
    const uint32_t ss = in + at_s + (static_cast<uint32_t>(base * ks) & 15) + t * ks;
    float s1 = 0.f, s2 = 0.f;
    float xh[kHold ? C : 1], tt[kHold ? C : 1];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = c * T + t;
      if (col >= d) break;
      const float q = (lds_elem<X>(sx + c * T * kX) - mu) * rs;
      const float g = lds_elem<G>(sg + c * T * kG);
      const float w = g * __ldg(gamma + col);
      s1 += w;
      s2 = fmaf(w, q, s2);
      ag[c] = fmaf(g, q, ag[c]);
      ab[c] += g;
      if (kHold) xh[kHold ? c : 0] = q, tt[kHold ? c : 0] = w;
    }
    float a1[1] = {s1}, a2[1] = {s2};
    row_sums<1, true>(a1, a2, T, 0, t >> 5, red[flip], ninv_d);
    flip ^= 1;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = c * T + t;
      if (col >= d) break;
      const float q = kHold ? xh[kHold ? c : 0] : (lds_elem<X>(sx + c * T * kX) - mu) * rs;
      const float w = kHold ? tt[kHold ? c : 0]
                            : lds_elem<G>(sg + c * T * kG) * __ldg(gamma + col);
      float o = rs * (w + a1[0] + q * a2[0]);
      if (ks == 4) o += lds_elem<F32>(ss + c * T * 4);
      else if (ks == 2) o += lds_elem<BF16>(ss + c * T * 2);
      Out<O, 1>::store(gx, base + col, &o);
    }
    mu = mu_next, rs = rs_next;
    if (++slot == stages) slot = 0;
  }
  let_next_in();
  if (!part) return;
  float* to = part + static_cast<int64_t>(blockIdx.x) * 2 * d;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = c * T + t;
    if (col >= d) break;
    to[col] = ag[c];
    to[d + col] = ab[c];
  }
}

// grad_gamma / grad_beta = column sums of the partial rows [blocks][2 d]: 32 columns a
// block, 32 strands of rows per column, added in order.
constexpr int kStrands = 32;
__global__ void __launch_bounds__(32 * kStrands) layernorm_columns_kernel(const float* part,
                                                                         int blocks, int d,
                                                                         float* gg, float* gb) {
  wait_for_previous();
  __shared__ float sh[kStrands][33];
  const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  float s = 0.f;
  if (col < 2 * d) {
#pragma unroll 4
    for (int r = k; r < blocks; r += kStrands) s += part[static_cast<int64_t>(r) * 2 * d + col];
  }
  sh[k][c] = s;
  __syncthreads();
  if (k == 0 && col < 2 * d) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < kStrands; ++i) a += sh[i][c];
    if (col < d) {
      if (gg) gg[col] = a;
    } else if (gb) {
      gb[col - d] = a;
    }
  }
}

// How the backward's rows are shared out: groups of T threads with C accesses of 8 (or, odd
// widths, 1) elements each and R rows at a time, `per` groups a block of at most 512
// threads, and at most one block for each of the 148 SMs of a B200.
struct NormGroups {
  int T, C, R, per, blocks;
};

NormGroups norm_groups(int64_t rows, int d) {
  NormGroups n;
  n.R = 1;
  if (d % 8 == 0) {
    const int chunks = d / 8;
    n.C = chunks <= kMaxNormThreads ? 1 : (chunks <= 2 * kMaxNormThreads ? 2 : 4);
    n.T = chunks <= 8 ? 8 : round32((chunks + n.C - 1) / n.C);
    if (n.C == 1) n.R = 2;
  } else {
    n.C = d <= 64 ? 2 : (d <= 8 * kMaxNormThreads ? 8 : (d <= 16 * kMaxNormThreads ? 16 : 32));
    n.T = n.C > 8 ? kMaxNormThreads : round32((d + n.C - 1) / n.C);
  }
  n.per = kMaxNormThreads / n.T;
  if (n.T > 32 && n.per > 8) n.per = 8;                  // barriers: one for each group
  while (n.per > 1 && (rows + n.per * n.R - 1) / (n.per * n.R) < 148) --n.per;   // every SM first
  while (n.T * n.per % 32) ++n.per;                      // whole warps
  const int64_t want = (rows + n.per * n.R - 1) / (n.per * n.R);
  n.blocks = static_cast<int>(want < 148 ? (want > 0 ? want : 1) : 148);
  return n;
}

struct BwdLaunch {
  int64_t rows;
  int d, gsum_f32, blocks;
  const void *gy, *x, *gsum;
  const float *mean, *rstd, *gamma;
  void* gx;
  float* part;
  cudaStream_t st;
};

constexpr size_t kRingBytes = 220 * 1024;                // one block an SM

template <typename X, typename G, typename O, int C, bool WARPS>
cudaError_t run_bwd(const BwdLaunch& l, const NormGroups& n) {
  const int threads = n.T * n.per;
  const size_t sums = n.per > 1 ? static_cast<size_t>(n.per) * 2 * l.d * sizeof(float) : 0;
  const size_t row = static_cast<size_t>(C == 1 ? 2 : C) * threads * 8 *
                     (kSize<X> + kSize<G> + (l.gsum ? (l.gsum_f32 ? 4 : 2) : 0));
  int stages = 1;                                        // 1: rows of 16384 in fp32, not ahead
  while (stages < 3 && (stages + 1) * row <= kRingBytes) ++stages;
  const size_t smem = stages * row > sums ? stages * row : sums;
  auto* kernel = layernorm_backward_kernel<X, G, O, C, WARPS>;
  cudaError_t e = set_max_smem(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  return launch_after(kernel, dim3(n.blocks), dim3(threads), smem, 1, l.st, l.gy, l.x, l.mean, l.rstd,
                      l.gamma, l.gsum, l.gsum_f32, l.gx, l.part, l.rows, l.d, n.T, n.per, stages);
}

template <typename X, typename G, typename O, int C, bool WARPS>
cudaError_t run_bwd_odd(const BwdLaunch& l, const NormGroups& n) {
  const size_t smem = n.per > 1 ? static_cast<size_t>(n.per) * 2 * l.d * sizeof(float) : 0;
  return launch_after(layernorm_backward_odd_kernel<X, G, O, C, WARPS>, dim3(n.blocks),
                      dim3(n.T * n.per), smem, 1, l.st, l.gy, l.x, l.mean, l.rstd, l.gamma, l.gsum,
                      l.gsum_f32, l.gx, l.part, l.rows, l.d, n.T, n.per);
}

template <typename X, typename G, typename O, int C>
cudaError_t run_bwd_wide(const BwdLaunch& l, const NormGroups& n) {
  const size_t row = row_window(l.d, kSize<X>) + row_window(l.d, kSize<G>) +
                     (l.gsum ? row_window(l.d, l.gsum_f32 ? 4 : 2) : 0);
  int stages = 1;                                        // 1: the widest rows, not ahead
  while (stages < 3 && (stages + 1) * row <= kRingBytes) ++stages;
  auto* kernel = layernorm_backward_wide_kernel<X, G, O, C>;
  cudaError_t e = set_max_smem(reinterpret_cast<const void*>(kernel), stages * row);
  if (e != cudaSuccess) return e;
  return launch_after(kernel, dim3(n.blocks), dim3(kMaxNormThreads), stages * row, 1, l.st, l.gy, l.x,
                      l.mean, l.rstd, l.gamma, l.gsum, l.gsum_f32, l.gx, l.part, l.rows, l.d, stages);
}

template <typename X, typename G, typename O>
cudaError_t pick_bwd(const BwdLaunch& l) {
  const NormGroups n = norm_groups(l.rows, l.d);
  if (l.d % 8 == 0) {
    if (n.T <= 32) return run_bwd<X, G, O, 1, false>(l, n);
    if (n.C == 1) return run_bwd<X, G, O, 1, true>(l, n);
    if (n.C == 2) return run_bwd<X, G, O, 2, true>(l, n);
    return run_bwd<X, G, O, 4, true>(l, n);
  }
  if (n.C == 2) return run_bwd_odd<X, G, O, 2, false>(l, n);
  if (n.C == 8 && n.T == 32) return run_bwd_odd<X, G, O, 8, false>(l, n);   // a warp: no barrier
  if (n.C == 8) return run_bwd_odd<X, G, O, 8, true>(l, n);
  if (n.C == 16) return run_bwd_wide<X, G, O, 16>(l, n);
  return run_bwd_wide<X, G, O, 32>(l, n);
}

}  // namespace

cudaError_t launch_layernorm_forward(const NormArgs& a, const void* x, const void* add,
                                     const float* gamma, const float* beta, void* y, void* sum,
                                     float* mean, float* rstd, cudaStream_t st) {
  FwdLaunch l{a.rows, a.d, a.add_dtype == 0, x, add, gamma, beta, y, sum, mean, rstd, a.eps, st};
  const bool xf = a.x_dtype == 0, yf = a.y_dtype == 0;
  if (xf) return yf ? pick_fwd<F32, F32>(l) : pick_fwd<F32, BF16>(l);
  return yf ? pick_fwd<BF16, F32>(l) : pick_fwd<BF16, BF16>(l);
}

int norm_workspace_blocks(int64_t rows) {
  return static_cast<int>(rows < 1 ? 1 : (rows < 148 ? rows : 148));
}

cudaError_t launch_layernorm_backward(const NormArgs& a, const void* grad_y, const void* x,
                                      const float* mean, const float* rstd, const float* gamma,
                                      const void* grad_sum, void* grad_x, float* grad_gamma,
                                      float* grad_beta, float* part, cudaStream_t st) {
  const bool sums = grad_gamma || grad_beta;
  BwdLaunch l{a.rows, a.d, a.add_dtype == 0, norm_groups(a.rows, a.d).blocks, grad_y, x,
              grad_sum, mean, rstd, gamma, grad_x, sums ? part : nullptr, st};
  const bool xf = a.x_dtype == 0, gf = a.y_dtype == 0, of = a.grad_dtype == 0;
  cudaError_t e;
  if (xf) {
    if (gf) e = of ? pick_bwd<F32, F32, F32>(l) : pick_bwd<F32, F32, BF16>(l);
    else e = of ? pick_bwd<F32, BF16, F32>(l) : pick_bwd<F32, BF16, BF16>(l);
  } else {
    if (gf) e = of ? pick_bwd<BF16, F32, F32>(l) : pick_bwd<BF16, F32, BF16>(l);
    else e = of ? pick_bwd<BF16, BF16, F32>(l) : pick_bwd<BF16, BF16, BF16>(l);
  }
  if (e != cudaSuccess || !sums) return e;
  // Scheduled while the last rows are written; waits on the device for their end.
  return launch_after(layernorm_columns_kernel, dim3((2 * a.d + 31) / 32), dim3(32 * kStrands), 0, 1,
                      st, static_cast<const float*>(part), l.blocks, a.d, grad_gamma, grad_beta);
}

}  // namespace pkm
