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
// are added in one fp32 accumulator. A step of the K loop is one K block of one plane of B
// and of up to three planes of A, each multiplied with it: a B tile is loaded once for
// them. With planes a stage is one tile of one operand (10 of 16 KiB in a CTA; stages of a
// whole step, 3 of them, did not hide L2's latency).
//
// A tile is 256 x 256 outputs of a pair of CTAs that shares each MMA (cta_group::2): every
// CTA loads half of A's rows and half of B's columns. What bounds the product is the
// traffic from L2 into shared memory, 64 bytes a cycle and SM against the
// MMA's 512 cycles a K block; smaller tiles read more per product (128 x 128 on single CTAs
// took 1.5 times as long on every size measured). Persistent, warp-specialised: warp 0 TMA
// producer, warp 1 MMA issuer, the others epilogue, the accumulator double-buffered in
// TMEM. Every wait is bounded as in the query kernel; the pair leaves through a cluster
// barrier, so neither CTA exits under the other's copies or MMAs.
//
// Work: the first `whole` tiles go round the pairs. The others, where their number would
// leave pairs idle, are laid end to end as K blocks and cut into one equal range per
// pair; a pair writes the pieces of tiles that it does not have entirely as fp32 parts,
// and linear_join_kernel adds a tile's parts in order and applies the epilogue.
//
// Accumulation: the tensor cores cut the running sum at each step of 16 products, about
// 2^-24 of it towards zero, so K / 16 cuts add up (1e-5 of the result at K = 8192). Where
// the output is fp32 (PROMOTE) the accumulator is therefore taken out every kSegment K
// blocks and added to fp32 registers, rounded to nearest; the epilogue warps do that while
// the next segment is multiplied into the other half of TMEM. The steps of a segment go
// smallest products first, each over all of its K blocks: what the cuts take then is measured
// against the small sums for all but the last step (one K block after the other, all of its
// steps, left an fp32 result at 1.3e-6 instead of 3e-7 at K = 4052).
//
// Epilogue: with PROMOTE 8 warps (two per TMEM lane quadrant; their accumulators take the
// registers), else 16, whose activations hide one another's latencies. A thread owns a row
// of 32 columns at a time. Rows go through shared memory, swizzled, and leave as TMA
// stores of 32 rows x 128 bytes (a thread's own 16-byte stores would touch a line per
// lane); for `pre` and y of bf16 outputs the accumulator is read twice, so that one buffer
// serves both. Outputs whose rows are no multiple of 16 bytes go out a row at a time, lanes
// along the columns.
#include "pkm_linear_epi.cuh"
#include "pkm_tc.h"
#include "pkm_tcgen05.cuh"

namespace pkm {

using namespace tc;

namespace {

constexpr int kRows = kLinearTileM / 2;  // of a tile per CTA
constexpr int BN = kLinearTileN;
constexpr int kCols = BN / 2;            // columns of B per CTA
constexpr int kK = 64;                   // K per stage: one 128-byte swizzled row of bf16
constexpr int kSegment = 4;              // K blocks between two takings (PROMOTE)
// Terms above which bf16 results are taken out as fp32 ones are: 2^11 cuts of 2^-24 are 2^-13, 1/32 of
// half a step of bf16, and K = 2^20 would be all of it. 4096 x 40960 -> 4096 takes 1060 us so, 930
// in one piece.
constexpr int kLongSum = 1 << 15;
constexpr uint32_t kABytes = kRows * kK * 2;
constexpr uint32_t kMnBlock = 64 * kK * 2;   // 64 MN x 64 K of an MN-major operand

template <bool PLANES, bool PROMOTE> struct Tile {
  static constexpr uint32_t kBBytes = kCols * kK * 2;
  // A K block of both operands, or of one plane of either.
  static constexpr uint32_t kStage = PLANES ? kABytes : kABytes + kBBytes;
  static_assert(kABytes == kBBytes, "one size of stage");
  static constexpr int kStages = 163840 / kStage;            // up to 160 KiB of stages
  // Epilogue warps: each takes kWide columns of its quadrant's rows.
  static constexpr int kWide = PROMOTE ? BN / 2 : BN / 4;
  static constexpr int kEpi = 4 * (BN / kWide);
  static constexpr int kThreads = 64 + 32 * kEpi;
  // Staging of one epilogue warp: 32 x 32 outputs of y and pre, 4 KiB of either in fp32, 2 in
  // bf16; two sets of buffers in turn where both fit twice. Without PROMOTE all outputs
  // are bf16, or a part.
  static constexpr uint32_t kStaging = PROMOTE ? 8192 : 4096;
  static constexpr size_t kSmem = 1024 + kStages * kStage + kEpi * kStaging + 512;
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

// The steps of one K block (LinearSteps), packed into 16 bits each: A's planes in the order of
// their products, B's plane, and the number of A's planes.
__device__ __forceinline__ int step_planes(uint64_t steps, int i) {
  return static_cast<int>(steps >> (16 * i)) & 0xffff;
}

// Tiles go in groups of kGroupM rows of tiles, down the group's rows first: the tiles in
// flight at a time share their operands in both directions.
constexpr int kGroupM = 8;
struct TileAt {
  int m, n;
};
__device__ __forceinline__ TileAt tile_at(int i, int mt, int nt) {
  const int g = i / (kGroupM * nt), r = i - g * (kGroupM * nt);
  const int rows = min(kGroupM, mt - g * kGroupM);
  const int n = r / rows;
  return {g * kGroupM + r - n * rows, n};
}

// What one pair works through: whole tiles, then its range of the cut ones.
struct Piece {
  int tile, kb0, kb1;
  int slot;               // of the part, or -1 for a whole tile
};
struct Work {
  LinearWork w;
  int me, at;             // this pair; whole tiles: the next one
  int64_t lo, pos, hi;    // its range of the cut tiles' K blocks
  __device__ __forceinline__ Work(const LinearWork& work, int pair)
      : w(work), me(pair), at(pair), lo(0), pos(0), hi(0) {
    if (w.cut) {   // 64-bit divisions: a microsecond before the first load, only where needed
      pos = lo = w.begin(pair);
      hi = w.begin(pair + 1);
    }
  }
  __device__ __forceinline__ bool next(Piece* p) {
    if (at < w.whole) {
      *p = {at, 0, w.kblocks, -1};
      at += w.pairs;
      return true;
    }
    if (pos >= hi) return false;
    const int t = static_cast<int>(pos / w.kblocks);
    const int kb0 = static_cast<int>(pos - static_cast<int64_t>(t) * w.kblocks);
    const int64_t left = hi - pos;
    const int kb1 = left < w.kblocks - kb0 ? kb0 + static_cast<int>(left) : w.kblocks;
    const bool all = kb0 == 0 && kb1 == w.kblocks;
    *p = {w.whole + t, kb0, kb1, all ? -1 : 2 * me + (pos == lo ? 0 : 1)};
    pos += kb1 - kb0;
    return true;
  }
};

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

__device__ __forceinline__ float4 lds128(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Shared-memory address of the 16-byte chunk c of row r of a 32 x 32 tile: 128-byte rows
// (fp32) or 64-byte rows (bf16) with the matching TMA swizzle.
__device__ __forceinline__ uint32_t tile_chunk(uint32_t base, int r, int c, bool f32) {
  return f32 ? base + r * 128 + ((c ^ (r & 7)) << 4) : base + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ void stage_row(uint32_t base, int r, bool f32, const float* v) {
  if (f32) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      sts128(tile_chunk(base, r, c, true), __float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]),
             __float_as_uint(v[4 * c + 2]), __float_as_uint(v[4 * c + 3]));
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      sts128(tile_chunk(base, r, c, false), pack_bf16(v[8 * c], v[8 * c + 1]),
             pack_bf16(v[8 * c + 2], v[8 * c + 3]), pack_bf16(v[8 * c + 4], v[8 * c + 5]),
             pack_bf16(v[8 * c + 6], v[8 * c + 7]));
  }
}

// 32 rows of 128 bytes (WIDE: 32 fp32 or 64 bf16 columns) or of 64 (32 bf16 columns) of the residual
// into a warp's staging area, whole 16-byte chunks (the rows are multiples of 16 bytes), lanes
// along the rows' chunks. All copies are in flight at a time, beside what the warp does until
// residual_here() (14952 x 32 -> 4208 fp32 with residual: 154 us, 84 without one; a load and a store
// one after the other: 378).
template <bool WIDE, int UNROLL>
__device__ __forceinline__ void stage_residual(uint32_t base, const void* residual, bool f32,
                                               int row0, int col, int M, int N, int lane) {
  constexpr int kPer = WIDE ? 8 : 4;        // chunks a row
  const int cols = f32 ? 4 : 8;             // of a chunk
  const int c = lane & (kPer - 1);
  const char* from = static_cast<const char*>(residual) + 16 * c;
  const int64_t row = static_cast<int64_t>(N) * (f32 ? 4 : 2), col_at = static_cast<int64_t>(col) * (f32 ? 4 : 2);
#pragma unroll UNROLL   // a copy in flight holds no register, its address does
  for (int i = 0; i < kPer; ++i) {
    const int r = lane / kPer + i * (32 / kPer);
    const bool in = row0 + r < M && col + c * cols < N;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tile_chunk(base, r, c, WIDE)),
                 "l"(in ? from + (row0 + r) * row + col_at : from), "r"(in ? 16 : 0)   // 0: zeros
                 : "memory");
  }
}
__device__ __forceinline__ void residual_here() {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();                             // the other lanes' chunks of this row
}

__device__ __forceinline__ void add_residual(uint32_t base, int r, bool f32, float* v) {
  if (f32) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float4 q = lds128(tile_chunk(base, r, c, true));
      v[4 * c] += q.x; v[4 * c + 1] += q.y; v[4 * c + 2] += q.z; v[4 * c + 3] += q.w;
    }
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 q = lds128(tile_chunk(base, r, c, false));
      const uint32_t w[4] = {__float_as_uint(q.x), __float_as_uint(q.y), __float_as_uint(q.z),
                             __float_as_uint(q.w)};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[8 * c + 2 * k] += bf16_lo(w[k]);
        v[8 * c + 2 * k + 1] += bf16_hi(w[k]);
      }
    }
  }
}

// The epilogue of one warp: its staging area and what it knows of the outputs' layout.
struct Outputs {
  uint32_t staging;      // shared address, 1024-byte aligned
  uint32_t pre_at, set;  // offset of pre's block, bytes of one set of buffers
  int sets, turn;
  bool part_before;      // the last block stored was a part's
  bool tma;              // rows are multiples of 16 bytes
};

__device__ __forceinline__ void add_bias32(const float* bias, int col, int N, float* v) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    if (col + i < N) {   // N is a multiple of 4
      const float4 b = __ldg(reinterpret_cast<const float4*>(bias + col + i));
      v[i] += b.x; v[i + 1] += b.y; v[i + 2] += b.z; v[i + 3] += b.w;
    }
  }
}

template <bool FINE, int C>
__device__ __forceinline__ void activate(int act, float* v) {
  if (act == PKM_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = act_value<FINE>(v[i], PKM_ACT_RELU);
  } else if (act == PKM_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = act_value<FINE>(v[i], PKM_ACT_GELU);
  } else if (act == PKM_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = act_value<FINE>(v[i], PKM_ACT_SILU);
  }
}

// 32 rows x 32 columns of the result: this thread's row `row0 + lane` in v, columns from
// `col`. Warp-uniform arguments but v. FINE: activations for fp32 outputs.
template <bool FINE>
__device__ __forceinline__ void store_block(const CUtensorMap* tm_y, const CUtensorMap* tm_pre,
                                            const LinearEpilogue& e, Outputs& o, int row0, int col,
                                            int M, int N, int lane, float* v) {
  if (o.tma) {
    const uint32_t y = o.staging + o.turn * o.set, p = y + o.pre_at;
    // The set's previous stores have read it: all but the last group, or all of them.
    if (lane == 0) {
      if (o.sets == 2 && !o.part_before) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      else bulk_wait_read0();
    }
    o.part_before = false;
    __syncwarp();
    if (e.residual) {
      if (e.y_f32) stage_residual<true, 1>(y, e.residual, true, row0, col, M, N, lane);
      else stage_residual<false, 1>(y, e.residual, false, row0, col, M, N, lane);
    }
    if (e.bias) add_bias32(e.bias, col, N, v);
    if (e.pre) stage_row(p, lane, e.pre_f32, v);
    activate<FINE, 32>(e.act, v);
    if (e.residual) {
      residual_here();
      add_residual(y, lane, e.y_f32, v);
    }
    stage_row(y, lane, e.y_f32, v);   // the row that this thread alone has read
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d_at(tm_y, y, col, row0, 0);
      if (e.pre) tma_store_3d_at(tm_pre, p, col, row0, 0);
      bulk_commit();
    }
    if (o.sets == 2) o.turn ^= 1;
    return;
  }
  // Rows of any length: transposed through shared memory (word i of row r at i xor r, so
  // neither direction has bank conflicts), then a row at a time, lanes along the columns.
  const uint32_t base = o.staging;
  if (o.part_before && lane == 0) bulk_wait_read0();
  o.part_before = false;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 32; ++i) sts_f32(base + (lane * 32 + (i ^ lane)) * 4, v[i]);
  __syncwarp();
  const bool mine = col + lane < N;
  const float bias = e.bias && mine ? __ldg(e.bias + col + lane) : 0.f;
  const int64_t at0 = static_cast<int64_t>(row0) * N + col + lane;
  const int rows = mine ? min(32, M - row0) : 0;
#pragma unroll 1
  for (int r = 0; r < 32; r += 8) {
    float u[8], res[8] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = lds_f32(base + ((r + j) * 32 + (lane ^ (r + j))) * 4) + bias;
    if (e.residual) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (r + j < rows) res[j] = load_as(e.residual, at0 + static_cast<int64_t>(r + j) * N, e.y_f32);
    }
    if (e.pre) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (r + j < rows) store_as(e.pre, at0 + static_cast<int64_t>(r + j) * N, e.pre_f32, u[j]);
    }
    activate<FINE, 8>(e.act, u);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (r + j < rows)
        store_as(e.y, at0 + static_cast<int64_t>(r + j) * N, e.y_f32, u[j] + res[j]);
  }
}

// 32 rows x 64 columns of bf16 outputs of a whole tile, straight from TMEM columns `tmem`: the
// columns' first 32, then the others, staged as 128-byte rows. `release` is called once the
// accumulator has been read for the last time.
template <typename Release>
__device__ __forceinline__ void store_block64(uint32_t tmem, const CUtensorMap* tm_y,
                                              const CUtensorMap* tm_pre, const LinearEpilogue& e,
                                              Outputs& o, int row0, int col, int M, int N, int lane,
                                              const Release& release) {
  for (int pass = e.pre ? 0 : 1; pass < 2; ++pass) {
    if (lane == 0) bulk_wait_read0();   // the buffer's last store has left it
    __syncwarp();
    if (pass && e.residual)
      stage_residual<true, 8>(o.staging, e.residual, false, row0, col, M, N, lane);
#pragma unroll 1
    for (int g = 0; g < 2; ++g) {
      float v[32];
      __syncwarp();
      tmem_ld32(tmem + g * 32, v);
      if (pass && g) release();
      if (col + g * 32 >= N) continue;
      if (e.bias) add_bias32(e.bias, col + g * 32, N, v);
      if (pass) {
        activate<false, 32>(e.act, v);
        if (e.residual) {
          if (g == 0) residual_here();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float4 q = lds128(tile_chunk(o.staging, lane, g * 4 + c, true));
            const uint32_t w[4] = {__float_as_uint(q.x), __float_as_uint(q.y), __float_as_uint(q.z),
                                   __float_as_uint(q.w)};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              v[8 * c + 2 * k] += bf16_lo(w[k]);
              v[8 * c + 2 * k + 1] += bf16_hi(w[k]);
            }
          }
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)   // a row that this thread alone has read
        sts128(tile_chunk(o.staging, lane, g * 4 + c, true), pack_bf16(v[8 * c], v[8 * c + 1]),
               pack_bf16(v[8 * c + 2], v[8 * c + 3]), pack_bf16(v[8 * c + 4], v[8 * c + 5]),
               pack_bf16(v[8 * c + 6], v[8 * c + 7]));
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d_at(pass ? tm_y : tm_pre, o.staging, col, row0, 0);
      bulk_commit();
    }
  }
  o.part_before = true;   // the buffer is single here
}

// The same block of a part: fp32 as it is, at (col, row) of the part's 256 x BN.
__device__ __forceinline__ void store_part(const CUtensorMap* tm_part, Outputs& o, int slot,
                                           int row, int col, int lane, const float* v) {
  if (lane == 0) bulk_wait_read0();
  __syncwarp();
  stage_row(o.staging, lane, true, v);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_3d_at(tm_part, o.staging, col, row, slot);
    bulk_commit();
  }
  o.part_before = true;
}

template <bool A_MN, bool B_MN, bool PLANES, bool PROMOTE>
__global__ void __launch_bounds__(Tile<PLANES, PROMOTE>::kThreads, 1) linear_tc_kernel(
    const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
    const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ CUtensorMap tm_pre,
    const __grid_constant__ CUtensorMap tm_part, int M, int N, const uint64_t steps,
    const int nsteps, const LinearWork plan, int use_tma, const LinearEpilogue epi,
    int* status, int clear) {
  using T = Tile<PLANES, PROMOTE>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = align1024(smem_raw);
  uint8_t* staging = stages + T::kStages * T::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + T::kEpi * T::kStaging);
  uint64_t* empty = full + T::kStages;
  uint64_t* tfull = empty + T::kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int mt = (M + 2 * kRows - 1) / (2 * kRows);
  const int nt = (N + BN - 1) / BN;
  const int pair = blockIdx.x >> 1;
  // K blocks of a segment of a piece of k, and of the producer's walk, whose order only
  // matters with planes.
  static_assert(!PLANES || PROMOTE, "planes: fp32 outputs");
  const auto segment = [](int k) { return PROMOTE ? kSegment : k; };
  let_next_in();

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * T::kEpi);
    }
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tm_a);
    prefetch_tensormap(&tm_b);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, T::kTmemCols);
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();   // the peer's barriers too
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // The set-up above ran beside the previous kernel's end; global memory starts here.
  wait_for_previous();
  if (clear && blockIdx.x == 0 && threadIdx.x == 0) *status = 0;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer (each CTA its own halves)
      uint32_t s = 0, ph = 0;
      int issued = 0;
      bool ok = true;
      Work work(plan, pair);
      Piece pc;
      while (ok && work.next(&pc)) {
        const TileAt mn = tile_at(pc.tile, mt, nt);
        const int m0 = mn.m * (2 * kRows) + rank * kRows;
        const int n0 = mn.n * BN + rank * kCols;
        for (int g0 = pc.kb0; g0 < pc.kb1 && ok; g0 += kSegment) {
          const int blocks = min(kSegment, pc.kb1 - g0);
          for (int i = 0; i < blocks * nsteps; ++i) {
            const int step = i / blocks;
            const int k0 = (g0 + i - step * blocks) * kK;
            const int what = PLANES ? step_planes(steps, step) : 1 << 14;
            // B's stage (without planes A's too), then A's planes.
            for (int p = PLANES ? -1 : 0; p < what >> 14; ++p) {
              if (!mbar_wait(&empty[s], ph ^ 1, status, abort)) { ok = false; break; }
              uint8_t* to = stages + s * T::kStage;
              const uint32_t bar = leader_addr(&full[s]);
              if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * T::kStage);
              if (p >= 0) {
                const int pa = (what >> (4 * p)) & 15;
                if (A_MN) {
                  tma_load_3d_pair(to, &tm_a, bar, m0, k0, pa);
                  tma_load_3d_pair(to + kMnBlock, &tm_a, bar, m0 + 64, k0, pa);
                } else {
                  tma_load_3d_pair(to, &tm_a, bar, k0, m0, pa);
                }
              }
              if (!PLANES || p < 0) {
                const int pb = (what >> 12) & 3;
                uint8_t* b = PLANES ? to : to + kABytes;
                if (B_MN) {
#pragma unroll
                  for (int blk = 0; blk < kCols / 64; ++blk)
                    tma_load_3d_pair(b + blk * kMnBlock, &tm_b, bar, n0 + 64 * blk, k0, pb);
                } else {
                  tma_load_3d_pair(b, &tm_b, bar, k0, n0, pb);
                }
              }
              ++issued;
              if (++s == T::kStages) { s = 0; ph ^= 1; }
            }
            if (!ok) break;
          }
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
      const uint32_t idesc = idesc_bf16_f32(2 * kRows, BN) | (B_MN ? 1u << 16 : 0u) |
                             (A_MN ? 1u << 15 : 0u);
      uint32_t s = 0, ph = 0;
      bool ok = true;
      int it = 0;
      Work work(plan, pair);
      Piece pc;
      while (ok && work.next(&pc)) {
        const int kblocks = pc.kb1 - pc.kb0, seg = segment(kblocks);
        for (int k = 0; k < kblocks && ok; k += seg, ++it) {
          const int blocks = min(seg, kblocks - k);   // with planes at most kSegment
          const int buf = it & 1;
          const uint32_t tph = (it >> 1) & 1;
          if (!mbar_wait(&tempty[buf], tph ^ 1, status, abort)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + buf * BN;
          for (int i = 0; i < blocks * nsteps; ++i) {
            const int count = PLANES ? step_planes(steps, i / blocks) >> 14 : 1;
            uint32_t b = 0, b_stage = 0;
            if (PLANES) {
              if (!mbar_wait(&full[s], ph, status, abort)) { ok = false; break; }
              b = smem_addr(stages + s * T::kStage);
              b_stage = s;
              if (++s == T::kStages) { s = 0; ph ^= 1; }
            }
            for (int p = 0; p < count; ++p) {
              if (!mbar_wait(&full[s], ph, status, abort)) { ok = false; break; }
              tc_fence_after();
              const uint32_t a = smem_addr(stages + s * T::kStage);
              if (!PLANES) b = a + kABytes;
#pragma unroll
              for (int j = 0; j < kK / 16; ++j) {
                // 16 K = two 8-row atoms of an MN-major tile, 32 bytes of a K-major row.
                const uint64_t ad = A_MN ? mn_desc(a + j * 2048) : sw128_desc(a, j * 32);
                const uint64_t bd = B_MN ? mn_desc(b + j * 2048) : sw128_desc(b, j * 32);
                mma_bf16_pair(d_tmem, ad, bd, idesc, (i != 0 || p != 0 || j != 0) ? 1u : 0u);
              }
              mma_commit_pair(&empty[s]);
              if (++s == T::kStages) { s = 0; ph ^= 1; }
            }
            if (!ok) break;
            if (PLANES) mma_commit_pair(&empty[b_stage]);
          }
          if (ok) mma_commit_pair(&tfull[buf]);
        }
      }
      mma_commit_pair(drain);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(drain, 0) && global_timer_ns() - t0 < kDrainLimitNs) {
      }
    }
  } else {
    // ---------------- epilogue: one thread per output row
    constexpr int kGroups = T::kWide / 32;
    const int quad = warp & 3;
    const int cset = (warp - 2) >> 2;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    Outputs o;
    o.staging = smem_addr(staging + (warp - 2) * T::kStaging);
    o.pre_at = epi.y_f32 ? 4096 : 2048;
    o.set = o.pre_at + (epi.pre ? (epi.pre_f32 ? 4096 : 2048) : 0);
    o.sets = o.set * 2 <= T::kStaging ? 2 : 1;
    o.turn = 0;
    o.part_before = false;
    o.tma = use_tma;
    int it = 0;
    bool ok = true;
    Work work(plan, pair);
    Piece pc;
    while (ok && work.next(&pc)) {
      const TileAt mn = tile_at(pc.tile, mt, nt);
      const int prow = rank * kRows + quad * 32;           // in the tile
      const int row0 = mn.m * (2 * kRows) + prow;
      const int pcol = cset * T::kWide, n0 = mn.n * BN + pcol;
      const int kblocks = pc.kb1 - pc.kb0, seg = segment(kblocks);
      const int segments = (kblocks + seg - 1) / seg;
      float acc[PROMOTE ? kGroups : 1][32];
      if (PROMOTE) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[PROMOTE ? g : 0][i] = 0.f;
      }
      for (int k = 0; k < segments; ++k, ++it) {
        const int buf = it & 1;
        const uint32_t tph = (it >> 1) & 1;
        if (!warp_wait(&tfull[buf], tph, status, abort)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + lane_addr + buf * BN + cset * T::kWide;
        if (PROMOTE) {
#pragma unroll
          for (int h = 0; h < 2 * kGroups; ++h) {
            float v[16];
            __syncwarp();
            tmem_ld16(d_tmem + h * 16, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[PROMOTE ? h / 2 : 0][(h & 1) * 16 + i] += v[i];
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(leader_addr(&tempty[buf]));
        } else if (o.tma && pc.slot < 0 && row0 < M && n0 < N) {
          static_assert(PROMOTE || kGroups == 2, "64 columns a warp");
          store_block64(d_tmem, &tm_y, &tm_pre, epi, o, row0, n0, M, N, lane, [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(leader_addr(&tempty[buf]));
          });
        } else {
#pragma unroll 1
          for (int g = 0; g < kGroups; ++g) {
            float v[32];
            __syncwarp();
            tmem_ld32(d_tmem + g * 32, v);
            if (g == kGroups - 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster(leader_addr(&tempty[buf]));
            }
            if (row0 >= M || n0 + g * 32 >= N) continue;
            if (pc.slot < 0)
              store_block<PROMOTE>(&tm_y, &tm_pre, epi, o, row0, n0 + g * 32, M, N, lane, v);
            else
              store_part(&tm_part, o, pc.slot, prow, pcol + g * 32, lane, v);
          }
        }
      }
      if (PROMOTE && ok) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          if (row0 >= M || n0 + g * 32 >= N) continue;
          float* v = acc[PROMOTE ? g : 0];
          if (pc.slot < 0)
            store_block<PROMOTE>(&tm_y, &tm_pre, epi, o, row0, n0 + g * 32, M, N, lane, v);
          else store_part(&tm_part, o, pc.slot, prow, pcol + g * 32, lane, v);
        }
      }
    }
    if (lane == 0) bulk_wait0();   // the stores have left shared memory and landed
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, T::kTmemCols);
  }
}

// Adds the parts of the cut tiles in order and applies the epilogue. Block: kJoinRows rows of
// one tile, a warp for a row: eight columns a lane side by side, or (rows of the output that
// are no 16-byte multiples) 32 apart, so that every access is contiguous over the lanes.
constexpr int kJoinRows = 4;
template <bool APART>
__global__ void __launch_bounds__(kJoinRows* BN / 8) linear_join_kernel(
    const float* part, const LinearWork plan, int mt, int nt, int M, int N,
    const LinearEpilogue epi) {
  static_assert(BN == 256, "32 lanes of 8 columns");
  constexpr int kBlocks = 2 * kRows / kJoinRows;
  const int t = blockIdx.x / kBlocks;                    // of the cut tiles
  const int row = (blockIdx.x % kBlocks) * kJoinRows + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  const int col = APART ? lane : lane * 8;
  const TileAt mn = tile_at(plan.whole + t, mt, nt);
  const int m = mn.m * (2 * kRows) + row, n = mn.n * BN + col;
  const int64_t p0 = static_cast<int64_t>(t) * plan.kblocks, p1 = p0 + plan.kblocks;
  const int c0 = plan.owner(p0), c1 = plan.owner(p1 - 1);
  // The first pair's part is its second one when its range began in an earlier tile.
  const int first = 2 * c0 + (plan.begin(c0) >= p0 ? 0 : 1);
  let_next_in();
  wait_for_previous();
  if (m >= M || n >= N || c0 == c1) return;              // c0 == c1: one pair had it all
  constexpr int64_t kPart = static_cast<int64_t>(2 * kRows) * BN;
  const float* q = part + static_cast<int64_t>(row) * BN + col;
  const auto load = [](const float* p, float* v) {
    if (APART) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p[32 * i];
    } else {
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  };
  float v[8];
  load(q + first * kPart, v);
#pragma unroll 4
  for (int c = c0 + 1; c <= c1; ++c) {
    float u[8];
    load(q + 2 * c * kPart, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += u[i];
  }
  const int64_t at = static_cast<int64_t>(m) * N + n;
  if (!APART) {
    linear_store8(epi, at, n, v);
    return;
  }
  float res[8] = {}, bias[8] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (n + 32 * i >= N) break;
    if (epi.residual) res[i] = load_as(epi.residual, at + 32 * i, epi.y_f32);
    if (epi.bias) bias[i] = __ldg(epi.bias + n + 32 * i);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] += bias[i];
    if (epi.pre && n + 32 * i < N) store_as(epi.pre, at + 32 * i, epi.pre_f32, v[i]);
  }
  activate<true, 8>(epi.act, v);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (n + 32 * i < N) store_as(epi.y, at + 32 * i, epi.y_f32, v[i] + res[i]);
}

// [planes][rows][cols] of an output or of the parts.
bool output_map(CUtensorMap* m, const void* p, bool f32, int64_t cols, int64_t rows, int planes,
                int box_cols = 32) {
  const cuuint64_t e = f32 ? 4 : 2;
  const cuuint64_t d[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                           static_cast<cuuint64_t>(planes)};
  const cuuint64_t s[2] = {static_cast<cuuint64_t>(cols) * e,
                           static_cast<cuuint64_t>(cols * rows) * e};
  const cuuint32_t b[3] = {static_cast<cuuint32_t>(box_cols), 32, 1};
  return make_map(m, p, 3, d, s, b,
                  box_cols * e == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
}

template <bool A_MN, bool B_MN, bool PLANES, bool PROMOTE>
cudaError_t run(const LinearGemm& g, int* launches, cudaStream_t st) {
  using T = Tile<PLANES, PROMOTE>;
  CUtensorMap tm_a, tm_b;
  // K-major: [planes][rows][K]; MN-major: [planes][K][columns]; ld elements a row.
  const cuuint64_t al = static_cast<cuuint64_t>(g.lda) * 2, bl = static_cast<cuuint64_t>(g.ldb) * 2;
  const cuuint64_t ar = static_cast<cuuint64_t>(A_MN ? g.K : g.M);
  const cuuint64_t br = static_cast<cuuint64_t>(B_MN ? g.K : g.N);
  const cuuint64_t ad[3] = {static_cast<cuuint64_t>(A_MN ? g.M : g.K), ar, g.a_count};
  const cuuint64_t bd[3] = {static_cast<cuuint64_t>(B_MN ? g.N : g.K), br, g.b_count};
  const cuuint64_t as[2] = {al, al * ar}, bs[2] = {bl, bl * br};
  const cuuint32_t ab[3] = {64, static_cast<cuuint32_t>(A_MN ? kK : kRows), 1};
  const cuuint32_t bb[3] = {64, static_cast<cuuint32_t>(B_MN ? kK : kCols), 1};
  if (!make_map(&tm_a, g.a, 3, ad, as, ab) || !make_map(&tm_b, g.b, 3, bd, bs, bb))
    return cudaErrorInvalidValue;
  // TMA stores need rows of 16-byte multiples (parts have them).
  const LinearEpilogue& e = g.epi;
  const int tma = g.N % (e.y_f32 ? 4 : 8) == 0 && (!e.pre || e.pre_f32 || g.N % 8 == 0);
  CUtensorMap tm_y = tm_a, tm_pre = tm_a, tm_part = tm_a;
  const int box = PROMOTE ? 32 : 64;   // columns stored at a time
  if ((tma && !output_map(&tm_y, e.y, e.y_f32, g.N, g.M, 1, box)) ||
      (tma && e.pre && !output_map(&tm_pre, e.pre, e.pre_f32, g.N, g.M, 1, box)) ||
      (g.part && !output_map(&tm_part, g.part, true, BN, 2 * kRows, 2 * g.work.pairs)))
    return cudaErrorInvalidValue;
  auto* kernel = linear_tc_kernel<A_MN, B_MN, PLANES, PROMOTE>;
  cudaError_t rc = set_max_smem(reinterpret_cast<const void*>(kernel), T::kSmem);
  if (rc != cudaSuccess) return rc;
  rc = launch_after(kernel, dim3(2 * g.work.pairs), dim3(T::kThreads), T::kSmem, 2, st, tm_a, tm_b,
                    tm_y, tm_pre, tm_part, g.M, g.N, g.steps.packed, g.steps.count, g.work, tma,
                    g.epi, g.status, g.clear);
  if (rc != cudaSuccess) return rc;
  ++*launches;
  if (!g.part) return cudaSuccess;
  const int mt = (g.M + 2 * kRows - 1) / (2 * kRows), nt = (g.N + BN - 1) / BN;
  const unsigned blocks = static_cast<unsigned>((mt * nt - g.work.whole) * (2 * kRows / kJoinRows));
  ++*launches;
  auto* join = g.N % 8 ? linear_join_kernel<true> : linear_join_kernel<false>;
  return launch_after(join, dim3(blocks), dim3(kJoinRows * BN / 8), 0, 1, st, g.part,
                      g.work, mt, nt, g.M, g.N, g.epi);
}

template <bool A_MN, bool B_MN>
cudaError_t promoted(const LinearGemm& g, int* launches, cudaStream_t st) {
  if (g.steps.products > 1) return run<A_MN, B_MN, true, true>(g, launches, st);
  // fp32 results, and bf16 ones of very long sums; else a bf16 result's own rounding hides the cuts.
  if constexpr (!A_MN)   // grad_W is fp32
    if (!g.epi.y_f32 && !(g.epi.pre && g.epi.pre_f32) && g.K <= kLongSum)
      return run<A_MN, B_MN, false, false>(g, launches, st);
  return run<A_MN, B_MN, false, true>(g, launches, st);
}

}  // namespace

cudaError_t launch_linear_gemm(const LinearGemm& g, int* launches, cudaStream_t st) {
  switch (g.layout) {
    case kForward: return promoted<false, false>(g, launches, st);
    case kGradX: return promoted<false, true>(g, launches, st);
    default: return promoted<true, true>(g, launches, st);
  }
}

}  // namespace pkm
