// pkm_linear_tc.cu -- the dense layer's tensor-core product (tcgen05 / TMEM / TMA):
//
//   C[M][N] = sum over plane pairs (p, q) of A_p B_q, over K, with an epilogue
//
// in the three layouts of a dense layer (x [M][K], W [N][K], d = grad_y act'(pre)):
//   forward   y  = x W^T   A = x   K-major,  B = W  K-major
//   grad_x    gx = d W     A = d   K-major,  B = W  MN-major
//   grad_W    gW = d^T x   A = d   MN-major, B = x  MN-major
// No operand is transposed in memory; the MMA's instruction descriptor carries the
// majorness. bf16 operands are one plane. An fp32 operand arrives as bf16 planes
// hi, mid, lo whose sum is the value to 2^-24, and the products whose size is above 2^-24
// are added in one fp32 accumulator, the K loop running over (K block, plane pair).
//
// Persistent, warp-specialised, 320 threads: warp 0 TMA producer, warp 1 MMA issuer,
// warps 2..9 epilogue (two per TMEM lane quadrant, half of the columns each), the
// accumulator double-buffered in TMEM. A tile is CG x 128 rows by BN columns: with CG = 2
// a pair of CTAs shares each MMA (cta_group::2), every CTA loading half of A's rows and
// half of B's columns. Every wait is bounded as in the query kernel; the pair leaves
// through a cluster barrier, so neither CTA exits under the other's copies or MMAs.
#include "pkm_linear_epi.cuh"
#include "pkm_tc.h"
#include "pkm_tcgen05.cuh"

namespace pkm {

using namespace tc;

namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kRows = 128;               // rows of a tile per CTA
constexpr int kK = 64;                   // K per stage: one 128-byte swizzled row of bf16
constexpr uint32_t kABytes = kRows * kK * 2;
constexpr uint32_t kMnBlock = 64 * kK * 2;   // 64 MN x 64 K of an MN-major operand

template <int CG, int BN> struct Tile {
  static constexpr int kCols = BN / CG;                      // of B per CTA
  static constexpr uint32_t kBBytes = kCols * kK * 2;
  static constexpr uint32_t kStage = kABytes + kBBytes;
  static constexpr int kStages = 196608 / kStage;            // 192 KiB of stages
  static constexpr size_t kSmem = 1024 + kStages * kStage + 512;
  static constexpr uint32_t kTmemCols = 2 * BN;
};

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// MN-major operand with the 128-byte swizzle: rows of 64 MN elements of one K index, 8 K
// rows a 1024-byte atom (SBO), blocks of 64 MN elements kMnBlock apart (LBO).
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr) {
  return ((addr >> 4) & 0x3fffull) | (static_cast<uint64_t>(kMnBlock >> 4) << 16) |
         ((1024ull >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

template <bool A_MN, bool B_MN, int CG, int BN>
__global__ void __launch_bounds__(kThreads, 1) linear_tc_kernel(
    const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, int M,
    int N, int K, uint32_t a_planes, uint32_t b_planes, int pairs, int ksplit,
    const LinearEpilogue epi, int* status) {
  using T = Tile<CG, BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(stages + T::kStages * T::kStage);
  uint64_t* empty = full + T::kStages;
  uint64_t* tfull = empty + T::kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? static_cast<int>(cluster_ctarank()) : 0;
  const int mt = (M + CG * kRows - 1) / (CG * kRows);
  const int nt = (N + BN - 1) / BN;
  const int ntiles = mt * nt * ksplit;
  const int steps = (K + kK - 1) / kK * pairs;      // K blocks x plane pairs
  const int per = (steps + ksplit - 1) / ksplit;
  const int first = blockIdx.x / CG, stride = gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], CG * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tm_a);
    prefetch_tensormap(&tm_b);
  }
  if (warp == 1) tmem_alloc_cg<CG>(tmem_slot, T::kTmemCols);
  __syncwarp();
  tc_fence_before();
  if (CG == 2) cluster_sync_all();   // the peer's barriers too
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer (each CTA its own halves)
      uint32_t s = 0, ph = 0;
      int issued = 0;
      bool ok = true;
      for (int t = first; t < ntiles && ok; t += stride) {
        const int sp = t % ksplit, mn = t / ksplit;
        const int m0 = (mn / nt) * (CG * kRows) + rank * kRows;
        const int n0 = (mn % nt) * BN + rank * T::kCols;
        const int i0 = sp * per, i1 = min(steps, i0 + per);
        for (int i = i0; i < i1; ++i) {
          if (!mbar_wait(&empty[s], ph ^ 1, status, abort)) { ok = false; break; }
          uint8_t* a = stages + s * T::kStage;
          uint8_t* b = a + kABytes;
          const int kb = i / pairs, pr = i - kb * pairs;
          const int k0 = kb * kK;
          const int pa = (a_planes >> (4 * pr)) & 15, pb = (b_planes >> (4 * pr)) & 15;
          uint32_t bar;
          if (CG == 2) {
            bar = leader_addr(&full[s]);
            if (rank == 0) mbar_arrive_expect_tx(&full[s], CG * T::kStage);
          } else {
            bar = smem_addr(&full[s]);
            mbar_arrive_expect_tx(&full[s], T::kStage);
          }
          if (A_MN) {
            tma_load_3d_cg<CG>(a, &tm_a, bar, m0, k0, pa);
            tma_load_3d_cg<CG>(a + kMnBlock, &tm_a, bar, m0 + 64, k0, pa);
          } else {
            tma_load_3d_cg<CG>(a, &tm_a, bar, k0, m0, pa);
          }
          if (B_MN) {
#pragma unroll
            for (int blk = 0; blk < T::kCols / 64; ++blk)
              tma_load_3d_cg<CG>(b + blk * kMnBlock, &tm_b, bar, n0 + 64 * blk, k0, pb);
          } else {
            tma_load_3d_cg<CG>(b, &tm_b, bar, k0, n0, pb);
          }
          ++issued;
          if (++s == T::kStages) { s = 0; ph ^= 1; }
        }
      }
      if (!ok) {
        // Let the copies already issued land before the CTA exits. Rank 0 counts the
        // bytes of both CTAs and can watch them; the other one waits the full time.
        const uint64_t t0 = global_timer_ns();
        const int last = issued < T::kStages ? issued : T::kStages;
        for (int back = 1; back <= last; ++back) {
          const int idx = issued - back;
          uint64_t* bar = &full[idx % T::kStages];
          const uint32_t phase = (idx / T::kStages) & 1;
          while ((rank != 0 || !mbar_try_wait(bar, phase)) &&
                 global_timer_ns() - t0 < kDrainLimitNs) {
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ---------------- MMA issuer (of the pair)
      const uint32_t idesc = idesc_bf16_f32(CG * kRows, BN) | (B_MN ? 1u << 16 : 0u) |
                             (A_MN ? 1u << 15 : 0u);
      uint32_t s = 0, ph = 0;
      bool ok = true;
      int it = 0;
      for (int t = first; t < ntiles && ok; t += stride, ++it) {
        const int sp = t % ksplit;
        const int i0 = sp * per, i1 = min(steps, i0 + per);
        const int buf = it & 1;
        const uint32_t tph = (it >> 1) & 1;
        if (!mbar_wait(&tempty[buf], tph ^ 1, status, abort)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + buf * BN;
        for (int i = i0; i < i1; ++i) {
          if (!mbar_wait(&full[s], ph, status, abort)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a = smem_addr(stages + s * T::kStage);
          const uint32_t b = a + kABytes;
#pragma unroll
          for (int j = 0; j < kK / 16; ++j) {
            // 16 K = two 8-row atoms of an MN-major tile, 32 bytes of a K-major row.
            const uint64_t ad = A_MN ? mn_desc(a + j * 2048) : sw128_desc(a, j * 32);
            const uint64_t bd = B_MN ? mn_desc(b + j * 2048) : sw128_desc(b, j * 32);
            mma_bf16_cg<CG>(d_tmem, ad, bd, idesc, (i != i0 || j != 0) ? 1u : 0u);
          }
          mma_commit_all<CG>(&empty[s]);
          if (++s == T::kStages) { s = 0; ph ^= 1; }
        }
        if (ok) mma_commit_all<CG>(&tfull[buf]);
      }
      mma_commit_all<CG>(drain);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(drain, 0) && global_timer_ns() - t0 < kDrainLimitNs) {
      }
    }
  } else {
    // ---------------- epilogue: one thread per output row
    constexpr int kGroups = BN / 64;          // groups of 32 columns per warp
    const int quad = warp & 3;
    const int cset = (warp - 2) >> 2;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    int it = 0;
    for (int t = first; t < ntiles; t += stride, ++it) {
      const int buf = it & 1;
      const uint32_t tph = (it >> 1) & 1;
      if (!warp_wait(&tfull[buf], tph, status, abort)) break;
      tc_fence_after();
      const int sp = t % ksplit, mn = t / ksplit;
      const int row = (mn / nt) * (CG * kRows) + rank * kRows + quad * 32 + lane;
      const int n0 = (mn % nt) * BN;
#pragma unroll 1
      for (int gg = 0; gg < kGroups; ++gg) {
        const int g = cset * kGroups + gg;
        float v[32];
        __syncwarp();
        tmem_ld32(tmem_base + lane_addr + buf * BN + g * 32, v);
        if (gg == kGroups - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (CG == 2) mbar_arrive_cluster(leader_addr(&tempty[buf]));
            else mbar_arrive(&tempty[buf]);
          }
        }
        const int col = n0 + g * 32;
        if (row < M && col < N) linear_store_row32(epi, row, col, M, N, sp, v);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  if (CG == 2) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<CG>(tmem_base, T::kTmemCols);
  }
}

template <bool A_MN, bool B_MN, int CG, int BN>
cudaError_t run(const LinearGemm& g, cudaStream_t st) {
  using T = Tile<CG, BN>;
  CUtensorMap tm_a, tm_b;
  // K-major: [planes][rows][K]; MN-major: [planes][K][columns]; ld elements a row.
  const cuuint64_t al = static_cast<cuuint64_t>(g.lda) * 2, bl = static_cast<cuuint64_t>(g.ldb) * 2;
  const cuuint64_t ar = static_cast<cuuint64_t>(A_MN ? g.K : g.M);
  const cuuint64_t br = static_cast<cuuint64_t>(B_MN ? g.K : g.N);
  const cuuint64_t ad[3] = {static_cast<cuuint64_t>(A_MN ? g.M : g.K), ar, g.a_count};
  const cuuint64_t bd[3] = {static_cast<cuuint64_t>(B_MN ? g.N : g.K), br, g.b_count};
  const cuuint64_t as[2] = {al, al * ar}, bs[2] = {bl, bl * br};
  const cuuint32_t ab[3] = {64, static_cast<cuuint32_t>(A_MN ? kK : kRows), 1};
  const cuuint32_t bb[3] = {64, static_cast<cuuint32_t>(B_MN ? kK : T::kCols), 1};
  if (!make_map(&tm_a, g.a, 3, ad, as, ab) || !make_map(&tm_b, g.b, 3, bd, bs, bb))
    return cudaErrorInvalidValue;
  auto* kernel = linear_tc_kernel<A_MN, B_MN, CG, BN>;
  cudaError_t e = set_max_smem(reinterpret_cast<const void*>(kernel), T::kSmem);
  if (e != cudaSuccess) return e;
  const int tiles = ((g.M + CG * kRows - 1) / (CG * kRows)) * ((g.N + BN - 1) / BN) * g.ksplit;
  const int most = sm_count() / CG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((tiles < most ? tiles : most) * CG);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = T::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, tm_a, tm_b, g.M, g.N, g.K, g.a_planes, g.b_planes,
                            g.pairs, g.ksplit, g.epi, g.status);
}

template <bool A_MN, bool B_MN>
cudaError_t pick(const LinearGemm& g, cudaStream_t st) {
  switch (g.tile) {
    case kTile256: return run<A_MN, B_MN, 2, 256>(g, st);
    case kTile128: return run<A_MN, B_MN, 1, 128>(g, st);
    default: return run<A_MN, B_MN, 1, 64>(g, st);
  }
}

}  // namespace

cudaError_t launch_linear_gemm(const LinearGemm& g, cudaStream_t st) {
  switch (g.layout) {
    case kForward: return pick<false, false>(g, st);
    case kGradX: return pick<false, true>(g, st);
    default: return pick<true, true>(g, st);
  }
}

}  // namespace pkm
