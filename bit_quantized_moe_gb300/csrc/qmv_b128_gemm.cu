// qmv_b128_gemm.cu -- products of E4M3 operands with fp32 scales of 128 columns
// (rows) and blocks of 128 x 128 (weights), and their gradients, over many rows
// on the tcgen05 tensor cores:
//
//   y[r][n]     = sum_b sx[r][b] sw[n / 128][b] sum_{k in b} q[r][k] w[n][k]
//   dx[r][k]    = sum_b sd[r][b] sw[b][k / 128] sum_{n in b} d[r][n] w[n][k]
//   dW[e][n][k] = sum over e's rows r of dy[r][n] x[r][k]
//
// A pair of CTAs on two SMs takes an output tile of 256 x 256: each holds 128
// rows of one operand and half of the other in shared memory, 128 bytes of
// depth a step (128 codes, a block; 64 of the 16-bit numbers of dW), and 128 x
// 256 sums in its tensor memory. A step's MMAs start from zero, so that its sum
// can take its scales: the epilogue's threads, a row and 128 columns each, read
// it from tensor memory (two steps fit) and add it, scaled, to fp32 sums in
// registers. The scale is one number for a thread's 128 columns: its row's
// times its block's. dW goes the same way without scales, 512 rows at a time.
//
// Operands whose depth is contiguous (rows in y and dx, weights in y) lie in shared
// memory as rows of 128 bytes, swizzled; the others (weights in dx, both in dW)
// as 128 bytes of outputs at each depth, which the tensor core reads transposed:
// no operand is transposed in memory, and one copy of the weights serves both products.
//
// Warps: 0 issues the TMA copies, 1 (of the pair's first CTA) the MMAs, 2 clears
// the rows behind an expert's last one (dW), 4..11 are the epilogue.
//
// What bounds y and dx: the epilogue beside the tensor cores. 8192 x 7168 x 7168:
// MMAs alone 185 us, with the copies 220, with the epilogue's barriers 224, with
// its loads of tensor memory 244, its additions 291, its scales 320, its stores
// 345; with two loads out at once, and the sum released when half of it has been
// added, 330; with the loads of scales behind that release, and a tile's first
// before the stores of the one before, 294 (2.86 PFLOP/s, 0.64 of the nominal
// rate). Tried and slower: the next step's first loads of tensor memory before the
// last additions (337), the next step's scale there (304), four half
// sums of 128 columns (413), 16 epilogue warps of 64 columns (353), the scales
// through shared memory (384 to 433), loads of 16 columns one by one (357).
// dW is bound by the MMAs (8192 x 7168 x 7168: 470 us, 1.8 PFLOP/s) and, over experts
// of few rows, by its output and the steps that rows behind an expert's last are
// cleared in (32 x 2880 x 2880 from 16,384 rows: 300 us, 1.06 GB written; filling that
// takes 142. Rows in whole sixteens, which need no clearing: 274. With all of the
// step's 64 rows cleared and multiplied 379).
#include <cmath>
#include <type_traits>

#include "qmv_internal.h"
#include "qmv_rows.cuh"
#include "qmv_tc.cuh"

namespace qmv {

enum : int { kModeY = 0, kModeDx = 1, kModeDw = 2 };

// Steps whose MMAs add to one sum in tensor memory. y and dx: one, whose scales follow. dW has none: 512 rows, so that the
// tensor cores' truncating additions stay few (measured: within 3e-7 of the sum of magnitudes, 5e-7 of the matrix's norm)
// and the epilogue seldom (8192 x 7168 x 7168 582 -> 472 us).
template <int MODE>
constexpr int kGroup = MODE == kModeDw ? 8 : 1;

constexpr int kHalf = 128;             // rows, and columns of the other operand, of one CTA
constexpr int kPairTile = 2 * kHalf;
constexpr int kPairThreads = 384;
constexpr int kPairStages = 5;
constexpr int kBand = 8;               // row tiles that follow one another (see pair_tile)
constexpr uint32_t kOperandBytes = kHalf * 128;
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr int kEpiWarps = 8;           // a CTA's
// Bytes of a row that its thread parks in shared memory before its warp stores
// them, and the pitch of a row there (an odd number of 16 bytes: no bank conflicts).
constexpr int kParkRow = 128, kParkPitch = kParkRow + 16;
constexpr uint32_t kParkBytes = kEpiWarps * 32 * kParkPitch;
constexpr int kPairJoinSteps = 9;      // steps that take as long as joining two pairs' sums
constexpr int kJoinBytes = 32 * kHalf / 2 * 4;   // of half of a warp's sums
static_assert(kEpiWarps * kJoinBytes <= kPairStages * kStageBytes, "the sums to join");
// At least so much that no other kernel with tensor memory fits beside it on an SM (the smallest takes 10 KB): of a pair and
// a cluster of another stream's kernel, each could wait on one SM for what the other holds on the next.
constexpr size_t kPairSmemLeast = 219 * 1024;
constexpr size_t pair_smem(int n_experts) {
  const size_t used = 1024 + (size_t)kPairStages * kStageBytes + kParkBytes + 2 * ((size_t)n_experts + 1) * sizeof(int);
  return used < kPairSmemLeast ? kPairSmemLeast : used;
}
static_assert(pair_smem(QMV_MAX_SORT_EXPERTS) + 512 <= 227 * 1024, "shared memory");
// Registers of an epilogue thread and of the others, within the 168 a thread that the launch gives. (Any spilled register
// is in the steps' way: with 216 and 72 a kernel that spilled 80 bytes took 414 us instead of 345.)
constexpr int kEpiRegs = 232, kOtherRegs = 40;
static_assert(256 * kEpiRegs + 128 * kOtherRegs <= kPairThreads * 168, "what the launch gives");

struct PairParams {
  const float4* sx;           // scales of the rows [nrows][blocks of depth, rounded up to 4]
  const float* sw;            // scales of the weights [E][ceil(N / 128)][ceil(K / 128)]
  const int32_t* offsets;
  void* y;
  int64_t nrows;
  int n_experts, N, K;
  int out_n;                  // columns of the output
  int out_type;
  bool whole16;               // the output's rows are of whole 16 bytes
  int steps, per_split;       // y, dx: of depth, and of the first of two pairs
  int x_quads;                // fours of a row's scales
  int k_blocks, n_blocks;     // of the weights' scales
  int n_tiles, m_tiles;       // column tiles; dW: row tiles of a matrix
};

template <int MODE, bool F16>
__device__ __forceinline__ constexpr uint32_t pair_idesc() {
  return (1u << 4) | (MODE == kModeDw && !F16 ? (1u << 7) | (1u << 10) : 0u) | (MODE == kModeDw ? 1u << 15 : 0u) |
         (MODE != kModeY ? 1u << 16 : 0u) | ((uint32_t)(kPairTile >> 3) << 17) | ((uint32_t)(kPairTile >> 4) << 24);
}

template <int MODE>
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (MODE == kModeDw) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
  } else {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
  }
}

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
// Arrivals at a barrier of the cluster that hand over no memory written by
// threads (copies and tensor memory have their own order): releasing and
// acquiring at the cluster's scope at every step made the steps four times as
// long (8192 x 7168 x 7168: 693 us).
__device__ __forceinline__ void mbar_expect_pair(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive_pair(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The address of `addr` in the first CTA of this one's pair.
template <bool SPLIT>
__device__ __forceinline__ uint32_t pair_leader(uint32_t addr) {
  if constexpr (!SPLIT) return leader_addr(addr);
  return peer_addr(addr, (int)(cluster_rank() & ~1u));
}
// The MMAs so far, complete, arrive at a barrier of both CTAs of the pair.
template <bool SPLIT>
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  if constexpr (!SPLIT) return mma_commit_to<true>(bar);
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               :: "r"(bar), "h"((uint16_t)(3u << (cluster_rank() & ~1u))) : "memory");
}
// 16 bytes, four sums, of another CTA's shared memory.
__device__ __forceinline__ void ld_cluster4(uint32_t addr, uint64_t& a, uint64_t& b) {
  asm volatile("ld.shared::cluster.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr) : "memory");
}

// As mbar_wait_bounded, without a hint to sleep.
__device__ __forceinline__ bool wait_brisk(uint32_t bar, uint32_t parity) {
  unsigned long long t0 = 0;
  for (uint32_t i = 1;; ++i) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    if (ok != 0) return true;
    if (i % 1024 == 0) {
      const unsigned long long now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitLimitNs) return false;
    }
  }
}

// Two fp32 sums in one register pair.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ uint64_t pack2(uint32_t a, uint32_t b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(a), "r"(b));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ void fma2(uint64_t& sum, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(sum) : "l"(a), "l"(b));
}
__device__ __forceinline__ void add2(uint64_t& sum, uint64_t a) { asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum) : "l"(a)); }

// Two numbers of 16 bits in a word.
template <typename T>
__device__ __forceinline__ uint32_t two16(float a, float b) {
  if constexpr (std::is_same_v<T, __half>) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// The columns from n0 on of a warp's 32 rows, as T: parked 128 bytes a row
// at a time and stored four rows by 128 bytes an instruction. (As 32-byte stores of
// 32 rows at once: 8192 x 7168 x 7168 396 us; as bulk copies of 128 bytes: 347 us,
// but dW of 32 experts of 2880 627.) Rows are of whole 16 bytes.
template <typename T, int TWOS>
__device__ __forceinline__ void store_rows(const PairParams& p, uint8_t* park, int64_t row0, int rows, int n0, int lane,
                                           const uint64_t (&sum)[TWOS]) {
  constexpr int cols = kParkRow / (int)sizeof(T);
#pragma unroll
  for (int c = 0; c < 2 * TWOS; c += cols) {
    const int vecs = min(cols, p.out_n - n0 - c) * (int)sizeof(T) / 16;
    if (vecs <= 0) break;
    uint8_t* mine = park + lane * kParkPitch;
#pragma unroll
    for (int i = 0; i < kParkRow / 16; ++i) {
      uint4 w;
      if constexpr (sizeof(T) == 4) {
        const uint64_t a = sum[(c + 4 * i) / 2], b = sum[(c + 4 * i) / 2 + 1];
        w = make_uint4((uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32));
      } else {
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float lo, hi;
          unpack2(sum[(c + 8 * i) / 2 + k], lo, hi);
          h[k] = two16<T>(lo, hi);
        }
        w = make_uint4(h[0], h[1], h[2], h[3]);
      }
      reinterpret_cast<uint4*>(mine)[i] = w;
    }
    __syncwarp();
    uint8_t* out = static_cast<uint8_t*>(p.y) + ((row0 + lane / 8) * p.out_n + n0 + c) * (int64_t)sizeof(T) + (lane & 7) * 16;
    const uint8_t* src = park + (lane / 8) * kParkPitch + (lane & 7) * 16;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (4 * i + lane / 8 < rows && (lane & 7) < vecs) {
        *reinterpret_cast<uint4*>(out + (int64_t)(4 * i) * p.out_n * sizeof(T)) =
            *reinterpret_cast<const uint4*>(src + 4 * i * kParkPitch);
      }
    }
    __syncwarp();
  }
}

// 32 columns of a warp's 32 rows, turned round in shared memory, so that
// neighbouring lanes store neighbouring elements: rows that start anywhere. (8192 x
// 7167 x 7168 335 us; two rows of 16 columns an instruction 355.)
template <typename T>
__device__ __forceinline__ void store_turned(const PairParams& p, float* park, int64_t row0, int rows, int n0, int lane,
                                             const uint64_t* sum) {
  constexpr int pitch = 33;
  static_assert(pitch * 4 <= kParkPitch, "a row's place");
#pragma unroll
  for (int i = 0; i < 16; ++i) unpack2(sum[i], park[lane * pitch + 2 * i], park[lane * pitch + 2 * i + 1]);
  __syncwarp();
  T* y = static_cast<T*>(p.y) + row0 * p.out_n + n0 + lane;
  if (n0 + lane < p.out_n) {
#pragma unroll 8
    for (int i = 0; i < 32; ++i) {
      if (i < rows) y[(int64_t)i * p.out_n] = from_f32<T>(park[i * pitch + lane]);
    }
  }
  __syncwarp();
}

template <int TWOS>
__device__ __forceinline__ void store_tile(const PairParams& p, uint8_t* park, int64_t row0, int rows, int n0, int lane,
                                           const uint64_t (&sum)[TWOS]) {
  const auto store = [&](auto type) {
    using T = decltype(type);
    if (p.whole16) return store_rows<T>(p, park, row0, rows, n0, lane, sum);
#pragma unroll
    for (int c = 0; c < TWOS / 16; ++c) {
      if (n0 + 32 * c >= p.out_n) break;
      store_turned<T>(p, reinterpret_cast<float*>(park), row0, rows, n0 + 32 * c, lane, sum + 16 * c);
    }
  };
  if (p.out_type == QMV_BF16) store(__nv_bfloat16());
  else if (p.out_type == QMV_F16) store(__half());
  else store(0.0f);
}

// What a CTA does of one output tile.
struct PairTile {
  int expert;
  int row0, rows;    // y, dx: its first row, and rows from there on; dW: the expert's
  int m, n;          // dW: first row of the matrix; first column of the pair
  int steps;
};

// Output tile t: experts in order; of an expert, bands of up to kBand row tiles,
// column by column, so that the tiles that run at once share their rows and their
// columns alike.
template <int MODE>
__device__ __forceinline__ PairTile pair_tile(int t, const PairParams& p, const int* first_tile, const int* first_row, int rank) {
  PairTile r;
  if constexpr (MODE == kModeDw) {
    const int each = p.m_tiles * p.n_tiles;
    r.expert = t / each;
    const int i = t - r.expert * each;
    const int band = i / (kBand * p.n_tiles), in = i - band * kBand * p.n_tiles, tall = min(kBand, p.m_tiles - band * kBand);
    r.n = in / tall;
    r.m = (band * kBand + in - r.n * tall) * kPairTile + rank * kHalf;
    r.n *= kPairTile;
    r.row0 = first_row[r.expert];
    r.rows = first_row[r.expert + 1] - r.row0;
    r.steps = (r.rows + 63) / 64;
  } else {
    int lo = 0, hi = p.n_experts - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (first_tile[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    const int rows = first_row[lo + 1] - first_row[lo];
    const int mt = (rows + kPairTile - 1) / kPairTile;
    const int i = t - first_tile[lo];
    r.expert = lo;
    const int band = i / (kBand * p.n_tiles), in = i - band * kBand * p.n_tiles, tall = min(kBand, mt - band * kBand);
    r.n = in / tall;
    const int m = (band * kBand + in - r.n * tall) * kPairTile + rank * kHalf;
    r.n *= kPairTile;
    r.m = 0;
    r.row0 = first_row[lo] + m;
    r.rows = rows - m;
    r.steps = p.steps;
  }
  return r;
}

// SPLIT: the two pairs of a cluster share a tile's depth. Each thread keeps half of its columns and takes the other pair's
// sums of them from its shared memory; the first pair's come first. A cluster has one tile.
template <int MODE, bool F16, bool SPLIT>
__global__ void __launch_bounds__(kPairThreads, 1)
b128_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 const __grid_constant__ PairParams p) {
  constexpr int kStages = kPairStages;
  extern __shared__ uint8_t dyn[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
  uint8_t* park = stages + kStages * kStageBytes;
  int* first_tile = reinterpret_cast<int*>(park + kParkBytes);   // [n_experts + 1]
  int* first_row = first_tile + p.n_experts + 1;                 // [n_experts + 1]
  // Barriers. full (the first CTA's): a step's copies of both CTAs have arrived; empty: its MMAs are complete;
  // acc_full, acc_empty (the first CTA's): a sum in tensor memory is there, has been read by both CTAs; tail: dW, this
  // CTA's copies of a step that is an expert's last, ragged one.
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], tail[kStages], done;
  __shared__ uint32_t tmem_base;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0), lane = threadIdx.x & 31;
  static_assert(!SPLIT || MODE != kModeDw, "depth of y and dx");
  const int rank = SPLIT ? (int)cluster_rank() & 1 : (int)cluster_rank();
  constexpr int splits = SPLIT ? 2 : 1;
  const int part = SPLIT ? (int)cluster_rank() / 2 : 0, first_step = SPLIT ? part * p.per_split : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&full[i]), 2);
      mbar_init(smem_addr(&empty[i]), 1);
      mbar_init(smem_addr(&tail[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&acc_full[i]), 1);
      mbar_init(smem_addr(&acc_empty[i]), 2 * kEpiWarps);
    }
    mbar_init(smem_addr(&done), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_addr(&tmem_base)),
                 "r"(2u * kPairTile) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  pdl_wait();
  if (warp == 0) expert_tiles(p.offsets, (int)p.nrows, p.n_experts, kPairTile, p.n_tiles, lane, first_row, first_tile);
  tc_before_sync();
  __syncthreads();
  cluster_sync_all();   // both CTAs' barriers exist
  tc_after_sync();
  const uint32_t tmem = tmem_base;
  const int tiles = MODE == kModeDw ? p.n_experts * p.m_tiles * p.n_tiles : first_tile[p.n_experts];
  const int t0 = (int)blockIdx.x / (2 * splits), dt = (int)gridDim.x / (2 * splits);
  bool ok = true;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    const int my_tiles = __shfl_sync(0xffffffffu, t0 < tiles ? (tiles - t0 + dt - 1) / dt : 0, 0);
    const auto tile_of = [&](int t) {   // the same in all lanes, and known to be
      PairTile r = pair_tile<MODE>(t, p, first_tile, first_row, rank);
      if constexpr (SPLIT) r.steps = part == 0 ? p.per_split : r.steps - first_step;
      r.expert = __shfl_sync(0xffffffffu, r.expert, 0);
      r.row0 = __shfl_sync(0xffffffffu, r.row0, 0);
      r.rows = __shfl_sync(0xffffffffu, r.rows, 0);
      r.m = __shfl_sync(0xffffffffu, r.m, 0);
      r.n = __shfl_sync(0xffffffffu, r.n, 0);
      r.steps = __shfl_sync(0xffffffffu, r.steps, 0);
      return r;
    };
    if (warp == 0) {
      // ---- copies
      const uint32_t data0 = smem_addr(stages);
      int it = 0, st = 0;
      for (int i = 0; i < my_tiles && ok; ++i) {
        const PairTile tile = tile_of(t0 + i * dt);
        // boxes of 64 rows that have a live one; rows that are not copied keep what the stage held, and are not stored
        const int copies = max(0, min(tile.rows, kHalf) + 63) / 64;
        for (int s = 0; s < tile.steps; ++s, ++it) {
          if (it >= kStages && !__all_sync(0xffffffffu, wait_brisk(smem_addr(&empty[st]), ((it / kStages) & 1) ^ 1))) {
            ok = false;
            break;
          }
          const uint32_t a = data0 + (uint32_t)st * kStageBytes, b = a + kOperandBytes;
          const uint32_t lead = pair_leader<SPLIT>(smem_addr(&full[st]));
          if (elect_one()) {
            if constexpr (MODE == kModeDw) {
              // two panels of 64 outputs x 64 rows each
              const int row = tile.row0 + 64 * s, x0 = (tile.m) * 2, y0 = (tile.n + rank * kHalf) * 2;
              if (tile.rows - 64 * s >= 64 || (tile.rows & 15) == 0) {
                mbar_expect_pair(lead, kStageBytes);
                tma_load_2d<true>(a, &map_a, x0, row, lead);
                tma_load_2d<true>(a + kOperandBytes / 2, &map_a, x0 + 128, row, lead);
                tma_load_2d<true>(b, &map_b, y0, row, lead);
                tma_load_2d<true>(b + kOperandBytes / 2, &map_b, y0 + 128, row, lead);
              } else {   // the last 16 rows that are multiplied hold the next expert's too: warp 2 clears those, then arrives
                const uint32_t mine = smem_addr(&tail[st]);
                mbar_arrive_expect_tx(mine, kStageBytes);
                tma_load_2d<false>(a, &map_a, x0, row, mine);
                tma_load_2d<false>(a + kOperandBytes / 2, &map_a, x0 + 128, row, mine);
                tma_load_2d<false>(b, &map_b, y0, row, mine);
                tma_load_2d<false>(b + kOperandBytes / 2, &map_b, y0 + 128, row, mine);
              }
            } else {
              const int at = (first_step + s) * 128;
              mbar_expect_pair(lead, (uint32_t)copies * 64 * 128 + kOperandBytes);
              for (int c = 0; c < copies; ++c) tma_load_2d<true>(a + c * 64 * 128, &map_a, at, tile.row0 + 64 * c, lead);
              if constexpr (MODE == kModeY) tma_load_3d_pair(b, &map_b, at, tile.n + rank * kHalf, tile.expert, lead);
              else tma_load_3d_pair(b, &map_b, tile.n + rank * kHalf, at, tile.expert, lead);
            }
          }
          __syncwarp();
          if (++st == kStages) st = 0;
        }
      }
      if (!ok) {   // leave no copy in flight: they report to the first CTA, so give them their time
        const unsigned long long from = global_timer_ns();
        while (global_timer_ns() - from < kDrainLimitNs) {}
      }
    } else if (warp == 1 && rank == 0) {
      // ---- products; the same in all lanes, one issues
      const uint32_t data0 = smem_addr(stages);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      constexpr uint32_t idesc = pair_idesc<MODE, F16>();
      int st = 0, sums = 0;
      uint32_t st_phase = 0;
      for (int i = 0; i < my_tiles && ok; ++i) {
        const PairTile tile = tile_of(t0 + i * dt);
        const int steps = tile.steps;
        for (int s = 0; s < steps; ++s) {
          const int acc = sums & 1;
          if ((s % kGroup<MODE> == 0 && !__all_sync(0xffffffffu, wait_brisk(smem_addr(&acc_empty[acc]), ((sums >> 1) & 1) ^ 1))) ||
              !__all_sync(0xffffffffu, wait_brisk(smem_addr(&full[st]), st_phase))) {
            ok = false;
            break;
          }
          // What warp 2 of both CTAs cleared: the phase is complete, and is acquired at the cluster's scope. (As a fence of the
          // cluster 32 experts' dW below took 318 us.)
          if (MODE == kModeDw && s == steps - 1 && (tile.rows & 15) != 0) mbar_wait_cluster(smem_addr(&full[st]), st_phase, 0);
          tc_after_sync();
          const uint32_t a = data0 + (uint32_t)st * kStageBytes, b = a + kOperandBytes;
          const uint32_t d = tm + (uint32_t)(acc * kPairTile);
          const bool last = s % kGroup<MODE> == kGroup<MODE> - 1 || s == steps - 1;   // of the sum
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {   // 32 bytes of depth each; transposed: 32 or 16 depths
              if (MODE == kModeDw && 64 * s + 16 * j >= tile.rows) break;
              uint64_t da, db;
              if constexpr (MODE == kModeDw) {
                da = transposed_desc(a + j * 16 * 128, kOperandBytes / 2);
                db = transposed_desc(b + j * 16 * 128, kOperandBytes / 2);
              } else {
                da = operand_desc(a + j * 32);
                db = MODE == kModeY ? operand_desc(b + j * 32) : transposed_desc(b + j * 32 * 128, 1024);
              }
              pair_mma<MODE>(d, da, db, idesc, s % kGroup<MODE> > 0 || j > 0 ? 1u : 0u);
            }
            pair_commit<SPLIT>(smem_addr(&empty[st]));
            if (last) pair_commit<SPLIT>(smem_addr(&acc_full[acc]));
          }
          __syncwarp();
          sums += last;
          if (++st == kStages) {
            st = 0;
            st_phase ^= 1;
          }
        }
      }
      if (elect_one()) pair_commit<SPLIT>(smem_addr(&done));
      __syncwarp();
      if (!wait_brisk(smem_addr(&done), 0)) ok = false;
    } else if (warp == 2 && MODE == kModeDw) {
      // ---- the rows behind an expert's last one, up to a multiple of 16, cleared in both operands (0 times a NaN is one)
      int it = 0;
      uint32_t phases = 0;   // bit st: of tail[st]
      for (int i = 0; i < my_tiles && ok; ++i) {
        const PairTile tile = tile_of(t0 + i * dt);
        it += tile.steps;
        if ((tile.rows & 15) == 0) continue;
        const int st = (it - 1) % kStages;
        if (!__all_sync(0xffffffffu, wait_brisk(smem_addr(&tail[st]), (phases >> st) & 1))) {
          ok = false;
          break;
        }
        phases ^= 1u << st;
        // a row of four panels at a time, 16 bytes a lane
        uint8_t* at = stages + (uint32_t)st * kStageBytes + (lane / 8) * (kOperandBytes / 2) + (lane & 7) * 16;
        const int valid = tile.rows - 64 * (tile.steps - 1), end = (valid + 15) / 16 * 16;
        for (int row = valid; row < end; ++row) *reinterpret_cast<uint4*>(at + row * 128) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(pair_leader<SPLIT>(smem_addr(&full[st])));
      }
    }
  } else {
    // ---- epilogue: thread = row 32 (warp % 4) + lane, columns 128 * half on
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    const int quad = warp % 4, half = (warp - 4) / 4;
    const int r = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    uint8_t* warp_park = park + (uint32_t)(warp - 4) * 32 * kParkPitch;
    int it = 0;
    // The scales: the row's four steps at a time, a load ahead; the weights' blocks' 32 steps at a time, a lane each, a load
    // ahead; a tile's first before the stores of the one before. (A thread's loads under way are waited for with its next
    // load of tensor memory, so they follow a step's last: before its first, 8192 x 7168 x 7168 took 330 us.)
    int steps = 0;
    const float4* sx = nullptr;
    const float* sw = nullptr;
    float4 next4 = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    float next32 = 1.0f;
    const auto block_scales = [&](int from) {
      const int at = min(from + lane, steps - 1);
      return sw[MODE == kModeY ? (int64_t)at : (int64_t)at * p.k_blocks];
    };
    const auto begin = [&](int t) {
      const PairTile tile = pair_tile<MODE>(t, p, first_tile, first_row, rank);
      steps = (tile.steps + kGroup<MODE> - 1) / kGroup<MODE>;
      if constexpr (SPLIT) steps = part == 0 ? p.per_split : steps - first_step;
      if constexpr (MODE != kModeDw) {
        sx = p.sx + min((int64_t)tile.row0 + r, p.nrows - 1) * p.x_quads;
        const int block = min((tile.n + half * kHalf) / kB128, (MODE == kModeY ? p.n_blocks : p.k_blocks) - 1);
        sw = p.sw + (int64_t)tile.expert * p.n_blocks * p.k_blocks + (MODE == kModeY ? (int64_t)block * p.k_blocks : block);
        if constexpr (SPLIT) {   // a whole number of fours
          sx += first_step / 4;
          sw += MODE == kModeY ? (int64_t)first_step : (int64_t)first_step * p.k_blocks;
        }
        next4 = *sx;
        next32 = block_scales(0);
      }
    };
    uint64_t sum[64];
    if (t0 < tiles) begin(t0);
    for (int t = t0; t < tiles && ok; t += dt) {
      float4 x4 = next4;
      float w32 = next32;
#pragma unroll
      for (int i = 0; i < 64; ++i) sum[i] = 0;
      for (int s = 0; s < steps; ++s, ++it) {
        const int acc = it & 1;
        float scale = 1.0f;
        if constexpr (MODE != kModeDw) {
          if (s % 4 == 0) {
            x4 = next4;
            if (s % 32 == 0) w32 = next32;
          }
          const float x = (s & 2) ? ((s & 1) ? x4.w : x4.z) : ((s & 1) ? x4.y : x4.x);
          scale = x * __shfl_sync(0xffffffffu, w32, s & 31);
        }
        if (!__all_sync(0xffffffffu, wait_brisk(smem_addr(&acc_full[acc]), (it >> 1) & 1))) {
          ok = false;
          break;
        }
        tc_after_sync();
        const uint64_t scale2 = pack2(scale, scale);
        const uint32_t d = tmem + (uint32_t)(acc * kPairTile + half * kHalf) + lanes;
        // Two loads of 32 columns are out before the first is added, and the other two while the first two are: the sum
        // has been read when half of it has been added. (One load after the other: 8192 x 7168 x 7168 345 us.)
        uint32_t v[2][32];
        const auto add = [&](int c) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint64_t two = pack2(v[c & 1][2 * i], v[c & 1][2 * i + 1]);
            if constexpr (MODE == kModeDw) add2(sum[16 * c + i], two);
            else fma2(sum[16 * c + i], two, scale2);
          }
        };
        tmem_ld32(d, v[0]);
        tmem_ld32(d + 32, v[1]);
        tmem_ld_wait(v[0]);
        tmem_ld_wait(v[1]);
        add(0);
        tmem_ld32(d + 64, v[0]);
        add(1);
        tmem_ld32(d + 96, v[1]);
        tmem_ld_wait(v[0]);
        tmem_ld_wait(v[1]);
        tc_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(pair_leader<SPLIT>(smem_addr(&acc_empty[acc])));   // read
        if constexpr (MODE != kModeDw) {
          if (s % 4 == 0 && s + 4 < steps) next4 = sx[s / 4 + 1];
          if (s % 32 == 31 && s + 1 < steps) next32 = block_scales(s + 1);
        }
        add(2);
        add(3);
      }
      if (!ok) break;
      if constexpr (SPLIT) break;
      asm volatile("" : "+r"(t));   // the tile's place is worked out again, not kept in registers over the steps
      if (t + dt < tiles) begin(t + dt);
      const PairTile tile = pair_tile<MODE>(t, p, first_tile, first_row, rank);
      const int n0 = tile.n + half * kHalf;   // first column of this thread
      const int64_t row0 = MODE == kModeDw ? (int64_t)tile.expert * p.N + tile.m : (int64_t)tile.row0;   // of the CTA
      const int rows = MODE == kModeDw ? p.N - tile.m : tile.rows;
      store_tile<64>(p, warp_park, row0 + quad * 32, rows - quad * 32, n0, lane, sum);
    }
    if constexpr (SPLIT) {
      // Where the CTA's steps were: the tile's last sum is complete. 16 bytes a lane follow one another, as they cross best.
      uint4* mine = reinterpret_cast<uint4*>(stages + (warp - 4) * kJoinBytes) + lane;
      uint64_t keep[32];
      if (t0 < tiles) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const uint64_t a = part == 0 ? sum[32 + i] : sum[i], b = part == 0 ? sum[33 + i] : sum[i + 1];
          keep[i] = part == 0 ? sum[i] : sum[32 + i];
          keep[i + 1] = part == 0 ? sum[i + 1] : sum[33 + i];
          mine[i * 16] = make_uint4((uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32));
        }
      }
      cluster_sync_all();
      if (t0 < tiles && ok) {
        uint64_t other[32];
        const uint32_t from = peer_addr(smem_addr(mine), (int)cluster_rank() ^ 2);
#pragma unroll
        for (int i = 0; i < 32; i += 2) ld_cluster4(from + 256 * i, other[i], other[i + 1]);
#pragma unroll
        for (int i = 0; i < 32; ++i) add2(keep[i], other[i]);   // the same in either order
        const PairTile tile = pair_tile<MODE>(t0, p, first_tile, first_row, rank);
        const int n0 = tile.n + half * kHalf + part * (kHalf / 2);
        store_tile<32>(p, warp_park, (int64_t)tile.row0 + quad * 32, tile.rows - quad * 32, n0, lane, keep);
      }
    }
    // the first CTA's last arrivals have reached this one before it may exit
    if (ok && !wait_brisk(smem_addr(&done), 0)) ok = false;
  }
  if (SPLIT && warp < 4) cluster_sync_all();
  if (!ok && lane == 0) set_status(kStatusWaitTile);
  __syncwarp();
  pdl_launch_dependents();
  tc_before_sync();
  __syncthreads();
  cluster_sync_all();   // neither CTA's memory is in use by the other any more
  if (warp == 1) {
    tc_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(2u * kPairTile));
  }
}

QMV_DEFINE_STATUS_ACCESSOR(status_b128_gemm)

namespace {

template <int MODE, bool F16, bool SPLIT>
cudaError_t pair_go(PairParams& p, int64_t tiles, const void* a, uint64_t a_bytes, uint64_t a_stride, const void* b,
                    uint64_t b_bytes, uint64_t b_stride, cudaStream_t stream) {
  constexpr int kCluster = SPLIT ? 4 : 2;
  auto* kernel = b128_pair_kernel<MODE, F16, SPLIT>;
  // The most that any call asks for (the attribute is the function's), and before the tensor maps: it makes the device's
  // context current on a host thread whose first CUDA call this is.
  g_launch_stage = "cudaFuncSetAttribute";
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)pair_smem(QMV_MAX_SORT_EXPERTS));
  if (e != cudaSuccess) return e;
  g_launch_stage = "cuTensorMapEncodeTiled";
  if (encode_fn() == nullptr) return cudaErrorNotSupported;
  CUtensorMap ma, mb;
  {
    const cuuint64_t dims[2] = {a_bytes, (cuuint64_t)p.nrows}, strides[1] = {a_stride};
    const cuuint32_t box[2] = {128, 64};
    if (!encode(&ma, 2, a, dims, strides, box)) return cudaErrorInvalidValue;
  }
  if constexpr (MODE == kModeDw) {
    const cuuint64_t dims[2] = {b_bytes, (cuuint64_t)p.nrows}, strides[1] = {b_stride};
    const cuuint32_t box[2] = {128, 64};
    if (!encode(&mb, 2, b, dims, strides, box)) return cudaErrorInvalidValue;
  } else {
    const cuuint64_t dims[3] = {b_bytes, (cuuint64_t)p.N, (cuuint64_t)p.n_experts};
    const cuuint64_t strides[2] = {b_stride, b_stride * (cuuint64_t)p.N};
    const cuuint32_t box[3] = {128, 128, 1};
    if (!encode(&mb, 3, b, dims, strides, box)) return cudaErrorInvalidValue;
  }
  p.k_blocks = b128_blocks(p.K);
  p.n_blocks = b128_blocks(p.N);
  p.whole16 = (uint64_t)p.out_n * (p.out_type == QMV_F32 ? 4 : 2) % 16 == 0;

  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = pair_smem(p.n_experts);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // no more clusters than run at once
  static PerDevice clusters;
  int most = 0;
  g_launch_stage = "cudaOccupancyMaxActiveClusters";
  e = clusters.get(&most, [&](int* n) {
    cfg.gridDim = dim3((unsigned)(device_sm_count() / kCluster * kCluster));
    return cudaOccupancyMaxActiveClusters(n, kernel, &cfg);
  });
  if (e != cudaSuccess) return e;
  if (most < 1) return cudaErrorInvalidConfiguration;
  g_launch_stage = "launch";
  cfg.gridDim = dim3((unsigned)(kCluster * (SPLIT || tiles < most ? tiles : most)));
  cfg.numAttrs = stream != nullptr ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, ma, mb, p);
}

// Tiles that there can be of `out_n` columns: every expert has at most one partial row tile.
int64_t pair_tiles(const B128GemmArgs& a, int out_n) {
  const int64_t hit = a.nrows < a.n_experts ? a.nrows : (int64_t)a.n_experts;
  const int64_t rows = a.n_experts == 1 ? (a.nrows + kPairTile - 1) / kPairTile : a.nrows / kPairTile + hit;
  return rows * ((out_n + kPairTile - 1) / kPairTile);
}

// Steps of the first pair where two share a tile's: fours, as the rows' scales are loaded.
int first_half(int steps) { return (steps / 2 + 3) / 4 * 4; }

// Whether two pairs share a tile's depth: where all run at once and it saves more than joining costs. Measured (one pair /
// two, us): 256 x 7168 x 7168 27.6 / 21.8, 160 x 7168 x 16384 57 / 38, 1000 x 1024 x 4096 17.4 / 14.0, 256 x 8192 x 2880
// 14.6 / 14.3, 256 x 8192 x 2048 11.8 / 12.2, 512 x 2880 x 1024 8.4 / 9.3. (Three and four took as long as two, or more.)
bool pairs_split(int64_t tiles, int steps, int sms) {
  return 2 * tiles <= sms / 2 && first_half(steps) + kPairJoinSteps < steps;
}

template <int MODE>
cudaError_t product_go(const B128GemmArgs& a) {
  const int depth = MODE == kModeY ? a.K : a.N;
  PairParams p = {};
  p.sx = reinterpret_cast<const float4*>(static_cast<const uint8_t*>(a.xq) + b128_scale_offset(a.nrows, depth));
  p.x_quads = b128_scale_row(depth) / 4;
  p.sw = a.w_scales;
  p.offsets = a.offsets;
  p.y = a.y;
  p.nrows = a.nrows;
  p.n_experts = a.n_experts;
  p.N = a.N;
  p.K = a.K;
  p.out_n = MODE == kModeY ? a.N : a.K;
  p.out_type = a.out_type;
  p.steps = b128_blocks(depth);
  p.n_tiles = (p.out_n + kPairTile - 1) / kPairTile;
  const int64_t tiles = pair_tiles(a, p.out_n);
  p.per_split = first_half(p.steps);
  auto* go = pairs_split(tiles, p.steps, device_sm_count()) ? pair_go<MODE, false, true> : pair_go<MODE, false, false>;
  return go(p, tiles, a.xq, b128_row_bytes(depth), b128_row_bytes(depth), a.w,
                              (uint64_t)a.K, (uint64_t)a.K, a.stream);
}

// Whether a product takes the kernel for few rows: both times are estimated. The pairs' goes by the tiles that each pair
// has to take, 0.38 us a step, or by reading the weights, at 4 TB/s, as fitted to GB300; experts are taken as equally
// full, with half a tile more each. Measured (few / pairs, us):
//   1 x 2880 x 2880 5.8 / 13, 16 x 7168 x 7168 13.0 / 22, 64 x 7168 x 7168 16.7 / 21.5, 128 x 7168 x 7168 25.6 / 21.5,
//   256 x 7168 x 7168 39 / 21.8, 256 x 2880 x 2880 12.1 / 12.3, 333 x 1001 x 2880 9.9 / 14.5, 400 x 2880 x 2880 18.2 / 12.8,
//   512 x 2880 x 1024 9.4 / 8.4; over 32 experts of 2880 x 2880: 1024 rows 53 / 73, 2048 rows 69 / 74, 4096 rows 106 / 75
bool few_rows(const B128GemmArgs& a, int depth, int out_n) {
  const int steps = b128_blocks(depth), sms = device_sm_count();
  const double hit = a.nrows < a.n_experts ? (double)a.nrows : (double)a.n_experts, each = a.nrows / hit / kPairTile;
  const double row_tiles = a.n_experts == 1 ? ceil(each) : hit * (each > 0.5 ? each + 0.5 : 1.0);
  const double rounds = ceil(row_tiles * ((out_n + kPairTile - 1) / kPairTile) / (sms / 2));
  const double chain = pairs_split(pair_tiles(a, out_n), steps, sms) ? first_half(steps) * 0.38 + 5.0 : rounds * steps * 0.38;
  return b128_few_us(a, depth, out_n, sms) < 5.5 + fmax(chain, hit * a.N * a.K / 4e6);
}

}  // namespace

cudaError_t launch_b128_product(const B128GemmArgs& a) { return few_rows(a, a.K, a.N) ? launch_b128_few(a, false) : product_go<kModeY>(a); }
cudaError_t launch_b128_linear(const B128GemmArgs& a) {
  const bool few = few_rows(a, a.K, a.N);
  if (few) {
    const cudaError_t e = launch_b128_few_linear(a);
    if (e != cudaErrorNotSupported) return e;
    g_launch_stage = "launch";
  }
  B128QuantArgs q;
  q.type = a.x_type;
  q.x = a.x;
  q.ldx = a.ldx;
  q.nrows = a.nrows;
  q.K = a.K;
  q.xq = const_cast<void*>(a.xq);
  q.stream = a.stream;
  const cudaError_t e = launch_quantize_b128(q);
  return e != cudaSuccess ? e : few ? launch_b128_few(a, false) : product_go<kModeY>(a);
}
cudaError_t launch_b128_grad_x(const B128GemmArgs& a) { return few_rows(a, a.N, a.K) ? launch_b128_few(a, true) : product_go<kModeDx>(a); }

cudaError_t launch_b128_grad_w(const B128GradWArgs& a) {
  PairParams p = {};
  p.offsets = a.offsets;
  p.y = a.dw;
  p.nrows = a.nrows;
  p.n_experts = a.n_experts;
  p.N = a.N;
  p.K = a.K;
  p.out_n = a.K;
  p.out_type = a.out_type;
  p.m_tiles = (a.N + kPairTile - 1) / kPairTile;
  p.n_tiles = (a.K + kPairTile - 1) / kPairTile;
  const int64_t tiles = (int64_t)a.n_experts * p.m_tiles * p.n_tiles;
  const uint64_t ld_dy = (uint64_t)a.ld_dy * 2, ldx = (uint64_t)a.ldx * 2;
  if (a.type == QMV_F16) {
    return pair_go<kModeDw, true, false>(p, tiles, a.dy, (uint64_t)a.N * 2, ld_dy, a.x, (uint64_t)a.K * 2, ldx, a.stream);
  }
  return pair_go<kModeDw, false, false>(p, tiles, a.dy, (uint64_t)a.N * 2, ld_dy, a.x, (uint64_t)a.K * 2, ldx, a.stream);
}

}  // namespace qmv
