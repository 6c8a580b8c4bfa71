// pkm_layernorm.cu -- layer norm (with the residual addition before it) and its backward.
//
// Forward, per row:  h = x + add, mean = sum h / d, rstd = 1/sqrt(sum (h - mean)^2 / d + eps),
// y = (h - mean) rstd gamma + beta. The row is read once and stays in registers for the
// three uses; a row belongs to T threads (a part of a warp, a warp, or several warps).
//
// Backward, per row, with xhat = (x - mean) rstd and t = grad_y gamma:
//   grad_x = rstd (t - sum t / d - xhat sum (t xhat) / d) + grad_sum
// and over the rows grad_gamma = sum grad_y xhat, grad_beta = sum grad_y. A group of T
// threads keeps the same columns for all of its rows, so the column sums stay in its
// registers; each block writes one partial row, and a second kernel adds the partial
// rows in a fixed order.
#include "pkm_block.h"
#include "pkm_elem.cuh"
#include "pkm_tc.h"

namespace pkm {

namespace {

// Sum over the T threads of a row (T a power of two up to 32, or a multiple of 32 that
// is the whole block). `red` holds one float per warp and is reused: callers alternate.
template <bool BLK>
__device__ __forceinline__ float row_sum(float v, int T, float* red) {
  const int w = BLK ? 32 : T;
  for (int o = w >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (BLK) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < (T >> 5); ++i) v += red[i];
  }
  return v;
}

constexpr int kMaxNormThreads = 512;

// V elements per access, C accesses per thread: thread t of a row holds the elements
// (c T + t) V ... + V - 1 for c < C.
template <typename X, typename Y, int V, int C, bool BLK>
__global__ void __launch_bounds__(BLK ? kMaxNormThreads : 256)
layernorm_forward_kernel(const void* x, const void* add, int add_f32,
                         const float* __restrict__ gamma, const float* __restrict__ beta, void* y,
                         void* sum, float* mean_out, float* rstd_out, int64_t rows, int d, int T,
                         float eps) {
  __shared__ float red[2][kMaxNormThreads / 32];
  const int t = BLK ? threadIdx.x : threadIdx.x & (T - 1);
  const int64_t row = BLK ? blockIdx.x
                          : static_cast<int64_t>(blockIdx.x) * (blockDim.x / T) + threadIdx.x / T;
  const bool live = BLK || row < rows;   // every lane stays for the shuffles
  const int64_t base = row * d;
  float h[C][V];
  Raw<X, V> rx[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * T + t) * V;
    if (live && col < d) rx[c].load(x, base + col);
  }
  if (add) {
    if (add_f32) {
      Raw<F32, V> ra[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = (c * T + t) * V;
        if (live && col < d) ra[c].load(add, base + col);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float f[V];
        rx[c].get(h[c]);
        ra[c].get(f);
#pragma unroll
        for (int v = 0; v < V; ++v) h[c][v] = rounded<X>(h[c][v] + f[v]);
      }
    } else {
      Raw<BF16, V> ra[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = (c * T + t) * V;
        if (live && col < d) ra[c].load(add, base + col);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float f[V];
        rx[c].get(h[c]);
        ra[c].get(f);
#pragma unroll
        for (int v = 0; v < V; ++v) h[c][v] = rounded<X>(h[c][v] + f[v]);
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * T + t) * V;
      if (live && col < d) Out<X, V>::store(sum, base + col, h[c]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) rx[c].get(h[c]);
  }
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const bool in = live && (c * T + t) * V < d;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!in) h[c][v] = 0.f;
      s += h[c][v];
    }
  }
  const float mean = row_sum<BLK>(s, T, red[0]) / static_cast<float>(d);
  float q = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const bool in = live && (c * T + t) * V < d;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[c][v] -= mean;
      if (in) q = fmaf(h[c][v], h[c][v], q);
    }
  }
  const float rstd = 1.f / sqrtf(row_sum<BLK>(q, T, red[1]) / static_cast<float>(d) + eps);
  if (live && t == 0) {
    if (mean_out) mean_out[row] = mean;
    if (rstd_out) rstd_out[row] = rstd;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * T + t) * V;
    if (!live || col >= d) continue;
    float g[V], b[V];
    load_param<V>(gamma, col, g);
    if (beta) load_param<V>(beta, col, b);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float n = h[c][v] * rstd * g[v];
      h[c][v] = beta ? n + b[v] : n;
    }
    Out<Y, V>::store(y, base + col, h[c]);
  }
}

struct FwdLaunch {
  int64_t rows;
  int d, T, add_f32;
  const void *x, *add;
  const float *gamma, *beta;
  void *y, *sum;
  float *mean, *rstd;
  float eps;
  cudaStream_t st;
};

template <typename X, typename Y, int V, int C, bool BLK>
cudaError_t run_fwd(const FwdLaunch& l) {
  const int threads = BLK ? l.T : 256;
  const int per = BLK ? 1 : 256 / l.T;
  const int64_t blocks = (l.rows + per - 1) / per;
  layernorm_forward_kernel<X, Y, V, C, BLK><<<static_cast<unsigned>(blocks), threads, 0, l.st>>>(
      l.x, l.add, l.add_f32, l.gamma, l.beta, l.y, l.sum, l.mean, l.rstd, l.rows, l.d, l.T, l.eps);
  return cudaGetLastError();
}

int round32(int x) { return (x + 31) / 32 * 32; }

template <typename X, typename Y>
cudaError_t pick_fwd(FwdLaunch l) {
  const int d = l.d;
  if (d % 8 == 0) {
    const int n = d / 8;   // 8-element chunks of a row
    const bool few = l.rows <= 4 * sm_count();
    if (n <= 8) { l.T = 8; return run_fwd<X, Y, 8, 1, false>(l); }
    if (n <= 32) { l.T = 32; return run_fwd<X, Y, 8, 1, false>(l); }
    if (few && n <= kMaxNormThreads) { l.T = round32(n); return run_fwd<X, Y, 8, 1, true>(l); }
    if (n <= 64) { l.T = 32; return run_fwd<X, Y, 8, 2, false>(l); }
    if (n <= 128) { l.T = 32; return run_fwd<X, Y, 8, 4, false>(l); }
    if (n <= 256) { l.T = 32; return run_fwd<X, Y, 8, 8, false>(l); }
    l.T = round32((n + 3) / 4);
    return run_fwd<X, Y, 8, 4, true>(l);
  }
  if (d <= 64) { l.T = 32; return run_fwd<X, Y, 1, 2, false>(l); }
  if (d <= 256) { l.T = 32; return run_fwd<X, Y, 1, 8, false>(l); }
  if (d <= 8 * kMaxNormThreads) { l.T = round32((d + 7) / 8); return run_fwd<X, Y, 1, 8, true>(l); }
  l.T = round32((d + 31) / 32);
  return run_fwd<X, Y, 1, 32, true>(l);
}

// ------------------------------------------------------------------ backward
// Groups of T threads (T <= 32: 256/T groups of a block, each with its own rows; else
// the block is one group); group g of the grid takes the rows g, g + groups, ...
template <typename X, typename G, typename O, int V, int C, bool BLK>
__global__ void __launch_bounds__(BLK ? kMaxNormThreads : 256)
layernorm_backward_kernel(const void* gy, const void* x, const float* __restrict__ mean,
                          const float* __restrict__ rstd, const float* __restrict__ gamma,
                          const void* gsum, int gsum_f32, void* gx, float* part, int64_t rows,
                          int d, int T) {
  extern __shared__ float sh[];   // !BLK: column sums of the block's groups
  __shared__ float red[2][2][kMaxNormThreads / 32];
  const int t = BLK ? threadIdx.x : threadIdx.x & (T - 1);
  const int per = BLK ? 1 : blockDim.x / T;
  const int group = BLK ? 0 : threadIdx.x / T;
  const float inv_d = 1.f / static_cast<float>(d);
  float ag[C][V], ab[C][V];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int v = 0; v < V; ++v) ag[c][v] = ab[c][v] = 0.f;
  int flip = 0;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * per;
  // Block-uniform trip count: every thread takes part in the reductions.
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * per; r0 < rows; r0 += stride, flip ^= 1) {
    const int64_t row = r0 + group;
    const bool live = row < rows;
    const int64_t base = row * d;
    Raw<X, V> rx[C];
    Raw<G, V> rg[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * T + t) * V;
      if (live && col < d) {
        rx[c].load(x, base + col);
        rg[c].load(gy, base + col);
      }
    }
    const float mu = live ? mean[row] : 0.f, rs = live ? rstd[row] : 0.f;
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * T + t) * V;
      if (live && col < d) {
        float xv[V], gv[V], gm[V];
        rx[c].get(xv);
        rg[c].get(gv);
        load_param<V>(gamma, col, gm);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float xh = (xv[v] - mu) * rs;
          const float tt = gv[v] * gm[v];
          s1 += tt;
          s2 = fmaf(tt, xh, s2);
          ag[c][v] = fmaf(gv[v], xh, ag[c][v]);
          ab[c][v] += gv[v];
        }
      }
    }
    const int w = BLK ? 32 : T;
    for (int o = w >> 1; o > 0; o >>= 1) {
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      s2 += __shfl_xor_sync(0xffffffffu, s2, o);
    }
    if (BLK) {
      // The two halves of `red` alternate, so one barrier per row is enough.
      if ((threadIdx.x & 31) == 0) {
        red[flip][0][threadIdx.x >> 5] = s1;
        red[flip][1][threadIdx.x >> 5] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.f;
      for (int i = 0; i < (T >> 5); ++i) {
        s1 += red[flip][0][i];
        s2 += red[flip][1][i];
      }
    }
    s1 *= inv_d;
    s2 *= inv_d;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * T + t) * V;
      if (!live || col >= d) continue;
      float xv[V], gv[V], gm[V], o[V];
      rx[c].get(xv);
      rg[c].get(gv);
      load_param<V>(gamma, col, gm);
#pragma unroll
      for (int v = 0; v < V; ++v)
        o[v] = rs * (gv[v] * gm[v] - s1 - (xv[v] - mu) * rs * s2);
      if (gsum) {
        float f[V];
        if (gsum_f32) {
          Raw<F32, V> q;
          q.load(gsum, base + col);
          q.get(f);
        } else {
          Raw<BF16, V> q;
          q.load(gsum, base + col);
          q.get(f);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] += f[v];
      }
      Out<O, V>::store(gx, base + col, o);
    }
  }
  if (!part) return;
  float* pg = part + static_cast<int64_t>(blockIdx.x) * 2 * d;
  if (BLK) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * T + t) * V;
      if (col >= d) continue;
      Out<F32, V>::store(pg, col, ag[c]);
      Out<F32, V>::store(pg + d, col, ab[c]);
    }
  } else {
    // Groups in order: sh[group][2][d]; then each column is added over the groups.
    float* mine = sh + group * 2 * d;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * T + t) * V;
      if (col >= d) continue;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        mine[col + v] = ag[c][v];
        mine[d + col + v] = ab[c][v];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * d; i += blockDim.x) {
      float s = 0.f;
      for (int g = 0; g < per; ++g) s += sh[g * 2 * d + i];
      pg[i] = s;
    }
  }
}

// grad_gamma / grad_beta = column sums of the partial rows [blocks][2 d]: 32 columns a
// block, 8 rows at a time per column, the 8 strands added in order.
__global__ void __launch_bounds__(256) layernorm_columns_kernel(const float* __restrict__ part,
                                                                int blocks, int d, float* gg,
                                                                float* gb) {
  __shared__ float sh[8][33];
  const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  float s = 0.f;
  if (col < 2 * d)
    for (int r = k; r < blocks; r += 8) s += part[static_cast<int64_t>(r) * 2 * d + col];
  sh[k][c] = s;
  __syncthreads();
  if (k == 0 && col < 2 * d) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a += sh[i][c];
    if (col < d) {
      if (gg) gg[col] = a;
    } else if (gb) {
      gb[col - d] = a;
    }
  }
}

struct BwdLaunch {
  int64_t rows;
  int d, T, gsum_f32, blocks;
  const void *gy, *x, *gsum;
  const float *mean, *rstd, *gamma;
  void* gx;
  float* part;
  cudaStream_t st;
};

template <typename X, typename G, typename O, int V, int C, bool BLK>
cudaError_t run_bwd(const BwdLaunch& l) {
  const int threads = BLK ? l.T : 256;
  const size_t smem = BLK ? 0 : static_cast<size_t>(256 / l.T) * 2 * l.d * sizeof(float);
  layernorm_backward_kernel<X, G, O, V, C, BLK><<<l.blocks, threads, smem, l.st>>>(
      l.gy, l.x, l.mean, l.rstd, l.gamma, l.gsum, l.gsum_f32, l.gx, l.part, l.rows, l.d, l.T);
  return cudaGetLastError();
}

template <typename X, typename G, typename O>
cudaError_t pick_bwd(BwdLaunch l) {
  const int d = l.d;
  if (d % 8 == 0) {
    const int n = d / 8;
    if (n <= 8) { l.T = 8; return run_bwd<X, G, O, 8, 1, false>(l); }
    if (n <= 32) { l.T = 32; return run_bwd<X, G, O, 8, 1, false>(l); }
    if (n <= kMaxNormThreads) { l.T = round32(n); return run_bwd<X, G, O, 8, 1, true>(l); }
    l.T = round32((n + 3) / 4);
    return run_bwd<X, G, O, 8, 4, true>(l);
  }
  if (d <= 64) { l.T = 32; return run_bwd<X, G, O, 1, 2, false>(l); }
  if (d <= 8 * kMaxNormThreads) { l.T = round32((d + 7) / 8); return run_bwd<X, G, O, 1, 8, true>(l); }
  l.T = round32((d + 31) / 32);
  return run_bwd<X, G, O, 1, 32, true>(l);
}

}  // namespace

cudaError_t launch_layernorm_forward(const NormArgs& a, const void* x, const void* add,
                                     const float* gamma, const float* beta, void* y, void* sum,
                                     float* mean, float* rstd, cudaStream_t st) {
  FwdLaunch l{a.rows, a.d, 0, a.add_dtype == 0, x, add, gamma, beta, y, sum, mean, rstd, a.eps, st};
  const bool xf = a.x_dtype == 0, yf = a.y_dtype == 0;
  if (xf) return yf ? pick_fwd<F32, F32>(l) : pick_fwd<F32, BF16>(l);
  return yf ? pick_fwd<BF16, F32>(l) : pick_fwd<BF16, BF16>(l);
}

// Blocks of the backward: a few per SM (148 on a B200), fewer when there are fewer
// groups of rows. The workspace is sized by it, so it depends on the sizes alone.
int norm_backward_blocks(int64_t rows, int d) {
  const bool vec = d % 8 == 0;
  const int per = vec ? (d <= 64 ? 32 : (d <= 256 ? 8 : 1)) : (d <= 64 ? 8 : 1);
  const int64_t want = (rows + per - 1) / per;
  const int64_t most = 148 * 4;
  return static_cast<int>(want < most ? (want > 0 ? want : 1) : most);
}

cudaError_t launch_layernorm_backward(const NormArgs& a, const void* grad_y, const void* x,
                                      const float* mean, const float* rstd, const float* gamma,
                                      const void* grad_sum, void* grad_x, float* grad_gamma,
                                      float* grad_beta, float* part, cudaStream_t st) {
  const bool sums = grad_gamma || grad_beta;
  BwdLaunch l{a.rows, a.d, 0, a.add_dtype == 0, norm_backward_blocks(a.rows, a.d), grad_y, x,
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
  layernorm_columns_kernel<<<(2 * a.d + 31) / 32, 256, 0, st>>>(part, l.blocks, a.d, grad_gamma,
                                                               grad_beta);
  return cudaGetLastError();
}

}  // namespace pkm
