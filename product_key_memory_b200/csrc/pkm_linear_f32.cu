// pkm_linear_f32.cu -- the products of small fp32 dense layers, each as one launch.
//
//   forward  y = act(x W^T + b) + residual,   grad_x = d W,   grad_W = d^T x, grad_b = sum_rows d
//
// with d = grad_y act'(pre) made from its two arrays as they are loaded. The tensor cores take
// fp32 operands as bf16 planes: a pass that writes the planes, the product on tiles of 256 x 256,
// and a pass that joins its parts, one after the other on a few of the SMs. In a small layer that
// chain of launches is the time, more than a plain fp32 product of a library takes. Measured
// here and there, alone on the device in a captured graph: 777 x 320 -> 93 forward 10.7 us and 14.4,
// backward 23 and 34; 16 x 64 -> 8192 backward 12.5 and 33; 1 x 2888 -> 672 backward 15 and 38.
//
// A block of 256 threads has a tile of BM x 64 results, a thread BM / 16 x 4 of them; operands come
// 32 k at a time through registers, the next ones in flight while these are multiplied, into
// shared memory as [k][m] and [k][n] (rows 4 words longer than the tile: the transposing
// stores of 8 k x 4 rows a warp then touch every bank once). K is cut over the blocks of a
// cluster until there are two blocks an SM; the cluster's blocks add their sums in order from
// one another's shared memory, each a share of the rows. Every 32 products are a sum of their
// own, added to the total in fp32: K terms round like 32 and K / 32 (2.2e-7 of a sum at K = 4096).
// Bound by latency: a step takes 1.8 us of loads, 32 products and a barrier, with one block an SM
// or two (23 TFLOP/s of the CUDA cores' 70 at 1000 x 1000 -> 1000, where the planes take a third).
#include "pkm_linear.h"

#include "pkm_linear_epi.cuh"
#include "pkm_tc.h"
#include "pkm_tcgen05.cuh"

namespace pkm {

using namespace tc;

namespace {

constexpr int kThreads = 256;
constexpr int kN = 64;             // columns of a tile
constexpr int kStep = 32;          // k at a time
constexpr int kPad = 4;

struct F32Product {
  const float *a, *pre, *b;        // pre: NULL, or a's slopes are taken from it
  int M, N, K;                     // of this product
  int cut;                         // blocks that share K
  LinearEpilogue epi;              // y NULL: only the column sums
  float* sums;                     // sum over k of a [M]: grad_bias; may be NULL
  int act;                         // of the slope
  int* status;
  int clear;
};

// Places of an operand's tile of R rows (of m or n) x kStep k that a thread loads: R / 8 of them.
// Contiguous in k: a warp's access is 8 k x 4 rows. Contiguous in the rows (R = 64): 32 rows.
template <bool K_INNER, int R> struct Places {
  static_assert(K_INNER || R == 64, "two accesses a row of 64");
  int k0, r0;
  __device__ __forceinline__ Places() {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    k0 = K_INNER ? (warp & 3) * 8 + (lane & 7) : warp >> 1;
    r0 = K_INNER ? (warp >> 2) * 4 + (lane >> 3) : (warp & 1) * 32 + lane;
  }
  __device__ __forceinline__ int k(int i) const { return K_INNER ? k0 : k0 + 4 * i; }
  __device__ __forceinline__ int r(int i) const { return K_INNER ? r0 + 8 * i : r0; }
};

// One element or, not `in`, 0. Stays where it is written: the next tile's loads are in flight while
// this one is multiplied.
__device__ __forceinline__ float load_or_zero(const float* p, bool in) {
  float v;
  asm volatile("{\n\t.reg .pred in;\n\tsetp.ne.b32 in, %2, 0;\n\tmov.f32 %0, 0f00000000;\n\t"
               "@in ld.global.f32 %0, [%1];\n\t}"
               : "=f"(v) : "l"(p), "r"(static_cast<int>(in)) : "memory");
  return v;
}

// A thread's places of an operand, rows from `row` of [rows][K] (K_INNER) or of [K][rows].
template <bool K_INNER, int R> struct Operand {
  const float* at;                 // place 0 of the next step
  int64_t hop, step;               // elements to the next place, to the next step
  uint32_t live;                   // places whose row exists
  __device__ __forceinline__ Operand(const float* p, const Places<K_INNER, R>& pl, int row, int rows,
                                     int k, int K) {
    const int m = row + pl.r0;
    const int64_t kk = k + pl.k0;
    at = p + (K_INNER ? static_cast<int64_t>(m) * K + kk : kk * rows + m);
    hop = K_INNER ? 8 * static_cast<int64_t>(K) : 4 * static_cast<int64_t>(rows);
    step = K_INNER ? kStep : static_cast<int64_t>(kStep) * rows;
    live = 0;
#pragma unroll
    for (int i = 0; i < R / 8; ++i) live |= static_cast<uint32_t>(row + pl.r(i) < rows) << i;
  }
  // `left` k are left from the step's first one.
  __device__ __forceinline__ void load(const Places<K_INNER, R>& pl, int left, float (&v)[R / 8]) {
    const float* q = at;
#pragma unroll
    for (int i = 0; i < R / 8; ++i, q += hop) v[i] = load_or_zero(q, (live >> i & 1) && pl.k(i) < left);
    at += step;
  }
};

__device__ __forceinline__ float peer_value(const float* p, uint32_t rank) {
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

template <LinearLayout L, int BM>
__global__ void __launch_bounds__(kThreads, 2) linear_f32_kernel(const F32Product p) {
  constexpr bool kAInner = L != kGradW, kBInner = L == kForward;
  constexpr int TM = BM / 16;
  using PA = Places<kAInner, BM>;
  using PB = Places<kBInner, kN>;
  __shared__ __align__(16) float sa[2][kStep][BM + kPad];
  __shared__ __align__(16) float sb[2][kStep][kN + kPad];
  __shared__ float column[BM];
  let_next_in();
  wait_for_previous();
  if (p.clear && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  const int nt = p.epi.y ? (p.N + kN - 1) / kN : 1;
  const int tile = blockIdx.x / p.cut, rank = blockIdx.x - tile * p.cut;
  const int m0 = tile / nt * BM, n0 = (tile - tile / nt * nt) * kN;
  const int steps = (p.K + kStep - 1) / kStep;
  const int begin = static_cast<int>(static_cast<int64_t>(steps) * rank / p.cut) * kStep;
  const int end = min(p.K, static_cast<int>(static_cast<int64_t>(steps) * (rank + 1) / p.cut) * kStep);
  const bool sums = p.sums && n0 == 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tn = (warp & 1) * 32 + (lane & 7) * 4, tm = ((warp >> 1) * 4 + (lane >> 3)) * TM;
  const PA at_a;
  const PB at_b;
  float va[BM / 8], vp[BM / 8], vb[kN / 8];
  Operand<kAInner, BM> oa(p.a, at_a, m0, p.M, begin, p.K);
  Operand<kAInner, BM> op(p.pre, at_a, m0, p.M, begin, p.K);
  Operand<kBInner, kN> ob(p.b, at_b, n0, p.N, begin, p.K);
  const auto load = [&](int left) {
    oa.load(at_a, left, va);
    if (L != kForward && p.pre) op.load(at_a, left, vp);
    if (p.epi.y) ob.load(at_b, left, vb);
  };
  const auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < BM / 8; ++i) {
      if (L != kForward && p.pre) va[i] *= act_slope(vp[i], p.act);
      sa[buf][at_a.k(i)][at_a.r(i)] = va[i];
    }
    if (p.epi.y) {
#pragma unroll
      for (int i = 0; i < kN / 8; ++i) sb[buf][at_b.k(i)][at_b.r(i)] = vb[i];
    }
  };
  float total[TM][4] = {};
  float column_sum = 0.f;
  if (begin < end) {
    load(end - begin);
    put(0);
  }
  __syncthreads();
  for (int k = begin, buf = 0; k < end; k += kStep, buf ^= 1) {
    const bool more = k + kStep < end;
    if (more) load(end - k - kStep);
    const int count = min(kStep, end - k);            // the tiles are 0 behind it
    if (p.epi.y) {
      float acc[TM][4] = {};
      const auto terms = [&](int j) {
        float fa[TM];
        const float* ra = &sa[buf][j][tm];
        if constexpr (TM == 4) {
          const float4 q = *reinterpret_cast<const float4*>(ra);
          fa[0] = q.x, fa[1] = q.y, fa[2] = q.z, fa[3] = q.w;
        } else if constexpr (TM == 2) {
          const float2 q = *reinterpret_cast<const float2*>(ra);
          fa[0] = q.x, fa[1] = q.y;
        } else {
          fa[0] = *ra;
        }
        const float4 q = *reinterpret_cast<const float4*>(&sb[buf][j][tn]);
        const float fb[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[i][c] = fmaf(fa[i], fb[c], acc[i][c]);
      };
      if (count == kStep) {
#pragma unroll 8
        for (int j = 0; j < kStep; ++j) terms(j);
      } else {
#pragma unroll 4
        for (int j = 0; j < (count + 3 & ~3); ++j) terms(j);
      }
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) total[i][c] += acc[i][c];
    }
    if (sums && threadIdx.x < BM) {
      float s = 0.f;
#pragma unroll 8
      for (int j = 0; j < kStep; ++j) s += sa[buf][j][threadIdx.x];
      column_sum += s;
    }
    if (more) put(buf ^ 1);
    __syncthreads();
  }
  // The block's sums take the operands' place, [BM][kN].
  float* out = &sb[0][0][0];
  static_assert(sizeof(sb) >= BM * kN * sizeof(float), "the sums take an operand's place");
#pragma unroll
  for (int i = 0; i < TM; ++i)
    *reinterpret_cast<float4*>(out + (tm + i) * kN + tn) =
        make_float4(total[i][0], total[i][1], total[i][2], total[i][3]);
  if (threadIdx.x < BM) column[threadIdx.x] = column_sum;
  if (p.cut > 1) cluster_sync_all();
  else __syncthreads();
  if (p.epi.y) {
    const int share = BM / p.cut, row0 = rank * share;
    for (int i = threadIdx.x; i < share * kN; i += kThreads) {
      const int row = row0 + i / kN, col = i % kN;
      const int m = m0 + row, n = n0 + col;
      if (m >= p.M || n >= p.N) continue;
      const float* at = out + row * kN + col;
      float v = p.cut > 1 ? peer_value(at, 0) : *at;
      for (int s = 1; s < p.cut; ++s) v += peer_value(at, s);
      linear_store1(p.epi, static_cast<int64_t>(m) * p.N + n, n, v);
    }
  }
  if (sums && rank == 0 && threadIdx.x < BM && m0 + threadIdx.x < p.M) {
    float v = column[threadIdx.x];
    for (int s = 1; s < p.cut; ++s) v += peer_value(&column[threadIdx.x], s);
    p.sums[m0 + threadIdx.x] = v;
  }
  if (p.cut > 1) cluster_sync_all();   // no block leaves while its sums are read
}

int rows_of_tile(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : 64; }

// How a product is shared out, by its sizes alone: the sums are the same whichever results are asked
// for.
struct Cut {
  int64_t tiles;
  int blocks, steps;   // that share K; of 32 k, for each of them
};
Cut cut_of(int64_t M, int64_t N, int64_t K, int bm) {
  Cut c{(M + bm - 1) / bm * ((N + kN - 1) / kN), 1, 0};
  const int64_t steps = (K + kStep - 1) / kStep;
  while (c.blocks < 8 && c.tiles * c.blocks * 2 <= 2 * 148 && steps >= 2 * c.blocks) c.blocks *= 2;
  c.steps = static_cast<int>((steps + c.blocks - 1) / c.blocks);
  return c;
}
// Steps of 1.8 us that the product takes.
double load_of(int64_t M, int64_t N, int64_t K, int bm) {
  const Cut c = cut_of(M, N, K, bm);
  const double each = static_cast<double>(c.tiles) * c.blocks / 148;
  return c.steps * (each > 1 ? each : 1);
}

template <LinearLayout L, int BM>
cudaError_t run(F32Product p, int* launches, cudaStream_t st) {
  const Cut c = cut_of(p.M, p.N, p.K, BM);
  p.cut = c.blocks;
  const int64_t tiles = p.epi.y ? c.tiles : (p.M + BM - 1) / BM;
  ++*launches;
  return launch_after(linear_f32_kernel<L, BM>, dim3(static_cast<unsigned>(tiles * p.cut)),
                      dim3(kThreads), 0, p.cut, st, p);
}

template <LinearLayout L>
cudaError_t run_rows(const F32Product& p, int* launches, cudaStream_t st) {
  switch (rows_of_tile(p.M)) {
    case 16: return run<L, 16>(p, launches, st);
    case 32: return run<L, 32>(p, launches, st);
  }
  return run<L, 64>(p, launches, st);
}

}  // namespace

// Up to 8 steps a product. Over 400 random sizes of 2^17 to 2^33 terms this is within 1 % of the faster
// of the two ways on average, forward and backward; the planes from the first size on were 30 %
// and 33 % above it, these products up to 30 steps 12 % and more.
bool linear_f32(const LinearArgs& a, bool backward) {
  constexpr double kMost = 8;
  if (a.dtype != PKM_F32) return false;
  if (!backward) return load_of(a.M, a.N, a.K, rows_of_tile(a.M)) <= kMost;
  return load_of(a.M, a.K, a.N, rows_of_tile(a.M)) + load_of(a.N, a.K, a.M, 64) <= 2 * kMost;
}

cudaError_t launch_f32_forward(const LinearArgs& a, const float* x, const float* W,
                               const LinearEpilogue& epi, int* status, int* launches,
                               cudaStream_t st) {
  return run_rows<kForward>({x, nullptr, W, static_cast<int>(a.M), a.N, a.K, 1, epi, nullptr, 0,
                             status, 1}, launches, st);
}

cudaError_t launch_f32_backward(const LinearArgs& a, const float* x, const float* W,
                                const float* grad_y, const float* pre, void* grad_x, float* grad_W,
                                float* grad_bias, int* status, int* launches, cudaStream_t st) {
  const int M = static_cast<int>(a.M);
  if (a.act == PKM_ACT_NONE) pre = nullptr;
  cudaError_t e = cudaSuccess;
  if (grad_x) {
    const LinearEpilogue epi{grad_x, nullptr, nullptr, nullptr, a.out_dtype == PKM_F32, 0,
                             PKM_ACT_NONE};
    e = run_rows<kGradX>({grad_y, pre, W, M, a.K, a.N, 1, epi, nullptr, a.act, status, 1}, launches, st);
    if (e != cudaSuccess) return e;
  }
  if (grad_W || grad_bias) {
    const LinearEpilogue epi{grad_W, nullptr, nullptr, nullptr, 1, 0, PKM_ACT_NONE};
    e = run<kGradW, 64>({grad_y, pre, x, a.N, a.K, M, 1, epi, grad_bias, a.act, status, !grad_x},
                        launches, st);
  }
  return e;
}

}  // namespace pkm
