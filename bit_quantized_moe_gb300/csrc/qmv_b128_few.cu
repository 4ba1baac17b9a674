// qmv_b128_few.cu -- the products of E4M3 operands with scales of blocks of 128
// (qmv_b128_gemm.cu) where an expert has few rows: a decode token, a decode
// batch over the experts, the end of a prompt.
//
// Bound by reading the weights once. The weights take the tensor cores' 128
// rows, the activations' rows their columns (BN of them), so that a step moves
// 16 KB of weights and 2 to 8 KB of rows. Two CTAs an SM keep a ring of 4 or 5
// steps under way each. Where there are fewer tiles than SMs, a cluster of CTAs
// shares a tile's depth and adds its parts in shared memory in the order of the
// ranks: no workspace, the same bits every run.
//
// Measured (16, 32, 64 columns for as many rows of an expert): 16 x 7168 x 7168 13.0
// us, 32 rows 14.0, 64 rows 16.7 (with 32 columns 20.8), 2048 rows of 32 experts of
// 2880 x 2880 69 (80). 128 columns, one CTA an SM, four groups of epilogue warps: 128 x
// 7168 x 7168 24.9 (with 64 27.3), but 2048 rows of 32 experts 88.
//
// A step's sum starts from zero and is added in fp32 registers, scaled by its
// row's scale (one a column here) times its block's, as in qmv_b128_gemm.cu.
//
// The rows come as a quantized buffer, by TMA, or as they are (X: their type):
// where every CTA has one tile and few steps, it quantizes its rows' part of the
// depth itself while its first weights are on their way, with the arithmetic of
// the separate launch and instead of it. (Quantized step by step by two warps: 1 x
// 7168 x 7168 18.8 us with its quantization where two launches took 15.6.)
//
// Warps: 0 issues the TMA copies, 1 the MMAs, 4 and on are the epilogue, thread =
// row of the weights and 16 or 32 columns; 2..7 quantize (X) first.
#include <cmath>
#include <type_traits>

#include "qmv_b128.cuh"
#include "qmv_internal.h"
#include "qmv_tc.cuh"

namespace qmv {

constexpr int kFewCtas = 2;            // of an SM
constexpr int kFewAccs = 4;
constexpr int kFewSplits = 6;          // CTAs of a cluster, at most
constexpr int kFewJoinSteps = 5;       // steps that take as long as the cluster's start and join
constexpr uint32_t kFewW = 128 * 128;  // bytes of weights of a step

// 64 columns: registers of an epilogue thread and of the others, within the 80 a thread that the launch gives.
constexpr int kFewEpiRegs = 104, kFewOtherRegs = 32;
static_assert(256 * kFewEpiRegs + 128 * kFewOtherRegs <= 384 * 80, "what the launch gives");

constexpr int kFewQuantSteps = 16;     // X: steps of a CTA, at most
constexpr int kFewQuantWarps = 6;
// X: blocks of 128 columns of a CTA, at most (of equally full experts). Four a CTA 6.2 us with the product, in two launches
// 7.3; 48: 7.5 and 8.1; 64: 9.5 and 8.1; 192: 22.2 and 15.0 (1, 12 and 16 x 2880 x 2880, 16 x 7168 x 7168).
constexpr int kFewQuantUnits = 48;

// X: the rows' codes of all steps lie beside the ring, which holds weights only.
template <int BN, bool QUANT>
struct Few {
  static constexpr int stages = QUANT || BN == 64 ? 4 : 5;
  static constexpr int groups = BN == 64 ? 2 : 1;   // of four epilogue warps
  static constexpr int cols = BN / groups;          // columns of a group
  static constexpr int threads = 128 + 128 * groups;
  static constexpr uint32_t x_bytes = BN * 128;
  static constexpr uint32_t stage_bytes = kFewW + (QUANT ? 0 : x_bytes);
  static constexpr uint32_t quant_bytes = QUANT ? kFewQuantSteps * (x_bytes + BN * 4) : 0;
  static constexpr uint32_t scale_bytes = 4 * BN * 4;   // a warp's scales of a step
  static constexpr uint32_t tmem_cols = kFewAccs * BN;
  static constexpr size_t smem(int n_experts) {
    return 1024 + (size_t)stages * stage_bytes + quant_bytes + scale_bytes + 2 * ((size_t)n_experts + 1) * sizeof(int);
  }
  static_assert(BN * 128 * 4 <= stages * stage_bytes, "the sums to join");
  static_assert(kFewCtas * (smem(256) + 1536) <= 228 * 1024 && smem(QMV_MAX_SORT_EXPERTS) + 512 <= 227 * 1024, "shared memory");
};

struct FewParams {
  const void* x;              // X: the rows
  int64_t ldx;
  bool x_vec;                 // X: every row starts on a 16-byte boundary
  int K;
  const float4* sx;           // scales of the rows [nrows][blocks of depth, rounded up to 4]
  const float* sw;            // scales of the weights [E][ceil(N / 128)][ceil(K / 128)]
  const int32_t* offsets;
  void* y;
  int64_t nrows;
  int n_experts, out_n, out_type;
  int x_quads, k_blocks, n_blocks;
  int steps, per_split;       // of depth, and of one rank of the cluster
  int n_tiles;                // tiles of 128 outputs
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ int cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ void tmem_ld16_now(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      " tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// The epilogue's warps say that they have read their last sums; the MMAs' warp waits for it.
template <int THREADS, bool WAIT>
__device__ __forceinline__ void sums_read() {
  if constexpr (WAIT) asm volatile("bar.sync 1, %0;" :: "n"(THREADS) : "memory");
  else asm volatile("bar.arrive 1, %0;" :: "n"(THREADS) : "memory");
}

struct FewTile {
  int expert, row0, rows, n;   // first row of the tile, and rows from there on; first output
};
template <int BN>
__device__ __forceinline__ FewTile few_tile(int t, const FewParams& p, const int* first_tile, const int* first_row) {
  int lo = 0, hi = p.n_experts - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (first_tile[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const int rows = first_row[lo + 1] - first_row[lo];
  const int mt = (rows + BN - 1) / BN;   // row tiles of a tile of outputs follow one another: its weights come from L2 again
  const int i = t - first_tile[lo];
  FewTile r;
  r.expert = lo;
  r.n = i / mt * 128;
  const int m = (i % mt) * BN;
  r.row0 = first_row[lo] + m;
  r.rows = rows - m;
  return r;
}

__device__ __forceinline__ void few_store(const FewParams& p, int64_t at, float v) {
  if (p.out_type == QMV_BF16) static_cast<__nv_bfloat16*>(p.y)[at] = from_f32<__nv_bfloat16>(v);
  else if (p.out_type == QMV_F16) static_cast<__half*>(p.y)[at] = from_f32<__half>(v);
  else static_cast<float*>(p.y)[at] = v;
}

// DX: the weights' outputs are their columns, read transposed. X: element type of rows to quantize, or void.
template <int BN, bool DX, typename X>
__global__ void __launch_bounds__((Few<BN, false>::threads), kFewCtas)
b128_few_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                const __grid_constant__ FewParams p) {
  constexpr bool kQuant = !std::is_void_v<X>;
  using F = Few<BN, kQuant>;
  constexpr int kStages = F::stages;
  extern __shared__ uint8_t dyn[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
  uint8_t* quant = stages + kStages * F::stage_bytes;                         // X: [kFewQuantSteps][BN][128] codes
  float* quant_scales = reinterpret_cast<float*>(quant + (kQuant ? kFewQuantSteps * F::x_bytes : 0));   // [kFewQuantSteps][BN]
  float* scales = reinterpret_cast<float*>(quant + F::quant_bytes);           // [4 warps][BN]
  float* join = reinterpret_cast<float*>(stages);   // [BN][128] this CTA's sums, where its steps were
  int* first_tile = reinterpret_cast<int*>(scales + 4 * BN);
  int* first_row = first_tile + p.n_experts + 1;
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], acc_full[kFewAccs], acc_empty[kFewAccs], done, quantized;
  __shared__ uint32_t tmem_base;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0), lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), splits = cluster_size();

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&full[i]), 1);
      mbar_init(smem_addr(&empty[i]), 1);
    }
    mbar_init(smem_addr(&quantized), kFewQuantWarps);
    for (int i = 0; i < kFewAccs; ++i) {
      mbar_init(smem_addr(&acc_full[i]), 1);
      mbar_init(smem_addr(&acc_empty[i]), 4 * F::groups);
    }
    mbar_init(smem_addr(&done), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_addr(&tmem_base)),
                 "r"(F::tmem_cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  if (warp == 0) expert_tiles(p.offsets, (int)p.nrows, p.n_experts, BN, p.n_tiles, lane, first_row, first_tile);
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  const uint32_t tmem = tmem_base;
  const int tiles = first_tile[p.n_experts];
  const int t0 = (int)blockIdx.x / splits, dt = (int)gridDim.x / splits;
  const int s0 = min(rank * p.per_split, p.steps), s1 = min(s0 + p.per_split, p.steps);   // this rank's steps
  bool ok = true;

  if constexpr (kQuant) {
    // ---- the rows of all of this CTA's steps: a warp takes a row's 128 columns of a step, lane = four of them; eight
    // such units' loads are under way together. Only the tile's own rows: the others' columns are not stored, whatever
    // they hold.
    if (warp >= 2 && t0 < tiles) {
      static_assert(sizeof(X) == 2, "8 bytes a lane");
      const FewTile tile = few_tile<BN>(t0, p, first_tile, first_row);
      const int rows = min(tile.rows, BN), units = rows * (s1 - s0);
      constexpr int kTogether = 8;
      for (int u0 = warp - 2; u0 < units; u0 += kFewQuantWarps * kTogether) {
        uint2 v[kTogether];
        uint32_t top[kTogether];
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
          const int u = u0 + i * kFewQuantWarps, step = u / rows, row = u - step * rows;
          const int c = (s0 + step) * 128 + lane * 4;
          const X* x = static_cast<const X*>(p.x) + (int64_t)(tile.row0 + row) * p.ldx + c;
          v[i] = make_uint2(0, 0);
          if (u < units && c < p.K) {
            if (p.x_vec) {   // K is a multiple of 16
              v[i] = *reinterpret_cast<const uint2*>(x);
            } else {
              X e[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) e[k] = x[k];
              v[i] = *reinterpret_cast<const uint2*>(e);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
          const X* e = reinterpret_cast<const X*>(&v[i]);
          uint32_t m = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) m = max(m, __float_as_uint(to_f32(e[k])) & 0x7fffffffu);
          top[i] = __reduce_max_sync(0xffffffffu, m);
        }
        uint32_t mine = 0;   // lane i: the maximum of unit i, whose scale it works out
#pragma unroll
        for (int i = 0; i < kTogether; ++i) mine = lane == i ? top[i] : mine;
        const BlockScale scale = block_scale(mine);
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
          const int u = u0 + i * kFewQuantWarps, step = u / rows, row = u - step * rows;
          const float inverse = __shfl_sync(0xffffffffu, scale.inverse, i), s = __shfl_sync(0xffffffffu, scale.scale, i);
          if (u < units) {
            const X* e = reinterpret_cast<const X*>(&v[i]);
            // rows of 128 bytes as the TMA copies lay them: 16-byte pieces exchanged by the row's place among eight
            *reinterpret_cast<uint32_t*>(quant + step * F::x_bytes + row * 128 + ((lane / 4) ^ (row & 7)) * 16 + (lane & 3) * 4) =
                codes4(to_f32(e[0]), to_f32(e[1]), to_f32(e[2]), to_f32(e[3]), inverse);
            if (lane == 0) quant_scales[step * BN + row] = s;
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_one(smem_addr(&quantized));
    }
  }
  if constexpr (BN == 64) {
    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewOtherRegs));
  }
  if (warp == 0) {
    // ---- copies
    int it = 0, st = 0;
    for (int t = t0; t < tiles && ok; t += dt) {
      FewTile tile = few_tile<BN>(t, p, first_tile, first_row);
      tile.expert = __shfl_sync(0xffffffffu, tile.expert, 0);
      tile.row0 = __shfl_sync(0xffffffffu, tile.row0, 0);
      tile.n = __shfl_sync(0xffffffffu, tile.n, 0);
      for (int s = s0; s < s1; ++s, ++it) {
        if (it >= kStages && !__all_sync(0xffffffffu, wait_for<false>(smem_addr(&empty[st]), ((it / kStages) & 1) ^ 1))) {
          ok = false;
          break;
        }
        const uint32_t w = smem_addr(stages) + (uint32_t)st * F::stage_bytes, bar = smem_addr(&full[st]);
        if (elect_one()) {
          mbar_arrive_expect_tx(bar, F::stage_bytes);
          if constexpr (DX) tma_load_3d(w, &map_w, tile.n, s * 128, tile.expert, bar);
          else tma_load_3d(w, &map_w, s * 128, tile.n, tile.expert, bar);
          if constexpr (!kQuant) tma_load_2d<false>(w + kFewW, &map_x, s * 128, tile.row0, bar);
        }
        __syncwarp();
        if (++st == kStages) st = 0;
      }
    }
    if (!ok) {   // leave no copy in flight
      for (int i = it > kStages ? it - kStages : 0; i < it; ++i) {
        if (!mbar_wait_bounded(smem_addr(&full[i % kStages]), (i / kStages) & 1, kDrainLimitNs) && lane == 0) {
          set_status(kStatusDrain);
        }
      }
    }
  } else if (warp == 1) {
    // ---- products; the same in all lanes, one issues
    constexpr uint32_t idesc = (1u << 4) | (DX ? 1u << 15 : 0u) | ((uint32_t)(BN >> 3) << 17) | (8u << 24);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const int my_tiles = __shfl_sync(0xffffffffu, t0 < tiles ? (tiles - t0 + dt - 1) / dt : 0, 0);
    const int total = my_tiles * (s1 - s0);
    int st = 0;
    uint32_t st_phase = 0;
    if (kQuant && total > 0 && !__all_sync(0xffffffffu, wait_for<false>(smem_addr(&quantized), 0))) ok = false;
    for (int it = 0; it < total && ok; ++it) {
      const int acc = it % kFewAccs;
      if (!__all_sync(0xffffffffu, wait_for<false>(smem_addr(&acc_empty[acc]), ((it / kFewAccs) & 1) ^ 1)) ||
          !__all_sync(0xffffffffu, wait_for<false>(smem_addr(&full[st]), st_phase))) {
        ok = false;
        break;
      }
      tc_after_sync();
      const uint32_t w = smem_addr(stages) + (uint32_t)st * F::stage_bytes;
      const uint32_t x = kQuant ? smem_addr(quant) + (uint32_t)it * F::x_bytes : w + kFewW;   // X: one tile
      const uint32_t d = tm + (uint32_t)(acc * BN);
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t a = DX ? transposed_desc(w + j * 32 * 128, 1024) : operand_desc(w + j * 32);
          asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}"
                       :: "r"(d), "l"(a), "l"(operand_desc(x + j * 32)), "r"(idesc), "r"(j > 0 ? 1u : 0u) : "memory");
        }
        mma_commit_to<false>(smem_addr(&empty[st]));
        mma_commit_to<false>(smem_addr(&acc_full[acc]));
      }
      __syncwarp();
      if (++st == kStages) {
        st = 0;
        st_phase ^= 1;
      }
    }
    if (elect_one()) mma_commit_to<false>(smem_addr(&done));
    __syncwarp();
    if (!wait_for<false>(smem_addr(&done), 0)) ok = false;
    __syncwarp();
    // Tensor memory is given back before the ranks wait for one another: held until then, it could keep a cluster of another
    // stream's kernel from starting that holds some where this one's peers are to start.
    sums_read<F::threads - 96, true>();
    tc_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tm), "r"(F::tmem_cols));
  } else if (warp >= 4) {
    // ---- epilogue: thread = row of the weights 32 (warp % 4) + lane; the tile's rows are its columns
    if constexpr (BN == 64) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFewEpiRegs));
    constexpr int kCols = F::cols;
    const int quad = warp % 4, group = F::groups == 1 ? 0 : warp / 4 - 1, c0 = group * kCols;   // its first column
    float* mine = scales + (warp - 4) * kCols;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    int it = 0;
    for (int t = t0; t < tiles && ok; t += dt) {
      const FewTile tile = few_tile<BN>(t, p, first_tile, first_row);
      const int block = tile.n / kB128;
      const float* sw = p.sw + (int64_t)tile.expert * p.n_blocks * p.k_blocks + (DX ? block : (int64_t)block * p.k_blocks);
      const int64_t sw_stride = DX ? p.k_blocks : 1;
      // the rows' scales four steps at a time, a load ahead; the block's 32 steps at a time, a lane each (a thread's loads
      // under way are waited for with its next load of tensor memory)
      float4 x4, next4;
      float w32 = 0.0f;
      const float4* sx = nullptr;
      if constexpr (!kQuant) {
        sx = p.sx + min((int64_t)tile.row0 + c0 + lane, p.nrows - 1) * p.x_quads;
        next4 = s0 < s1 ? sx[s0 / 4] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        x4 = next4;
      }
      float sum[kCols];
#pragma unroll
      for (float& v : sum) v = 0.0f;
      for (int s = s0; s < s1; ++s, ++it) {
        const int acc = it % kFewAccs;
        if (!kQuant && (s == s0 || s % 4 == 0)) {
          x4 = next4;
          if (s / 4 * 4 + 4 < s1) next4 = sx[s / 4 + 1];
        }
        if ((s - s0) % 32 == 0) w32 = sw[min(s + lane, s1 - 1) * sw_stride];
        const float w = __shfl_sync(0xffffffffu, w32, (s - s0) & 31);
        if (kQuant && s == s0 && !__all_sync(0xffffffffu, wait_for<false>(smem_addr(&quantized), 0))) {
          ok = false;
          break;
        }
        __syncwarp();   // the step before has been read
        const float x = kQuant ? quant_scales[(s - s0) * BN + (lane & (BN - 1))] : (s & 2) ? ((s & 1) ? x4.w : x4.z) : ((s & 1) ? x4.y : x4.x);
        if (lane < kCols) mine[lane] = x * w;
        __syncwarp();
        if (!__all_sync(0xffffffffu, wait_for<false>(smem_addr(&acc_full[acc]), (it / kFewAccs) & 1))) {
          ok = false;
          break;
        }
        tc_after_sync();
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          uint32_t v[16];
          tmem_ld16_now(tmem + (uint32_t)(acc * BN + c0 + c) + lanes, v);
          if (c + 16 >= kCols) {   // read
            tc_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_one(smem_addr(&acc_empty[acc]));
          }
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(mine + c + i);
            sum[c + i] = fmaf(__uint_as_float(v[i]), f.x, sum[c + i]);
            sum[c + i + 1] = fmaf(__uint_as_float(v[i + 1]), f.y, sum[c + i + 1]);
            sum[c + i + 2] = fmaf(__uint_as_float(v[i + 2]), f.z, sum[c + i + 2]);
            sum[c + i + 3] = fmaf(__uint_as_float(v[i + 3]), f.w, sum[c + i + 3]);
          }
        }
      }
      if (!ok) break;
      if (splits == 1) {
        const int n = tile.n + quad * 32 + lane;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          if (c0 + c < tile.rows && n < p.out_n) few_store(p, ((int64_t)tile.row0 + c0 + c) * p.out_n + n, sum[c]);
        }
      } else {
        // A cluster has one tile only: its last sum is complete, so that no copy or product uses the ring any more.
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          if (c0 + c < tile.rows) join[(c0 + c) * 128 + quad * 32 + lane] = sum[c];
        }
      }
    }
    tc_before_sync();
    __syncwarp();
    sums_read<F::threads - 96, false>();
    if (splits > 1) {
      cluster_sync_all();   // every rank's sums lie in its own shared memory; each adds up the rows that are its share
      if (t0 < tiles && ok) {
        const FewTile tile = few_tile<BN>(t0, p, first_tile, first_row);
        const int n = tile.n + quad * 32 + lane, rows = min(tile.rows, BN);
        // several rows' parts are on their way together (X: seldom more than one row; by four, 1 x 2880 x 2880 takes 0.3 us more)
        constexpr int kRows = kQuant ? 1 : 4;
        const int step = splits * F::groups;
        for (int c = rank + splits * group; c < rows; c += kRows * step) {
          float part[kRows][kFewSplits];
#pragma unroll
          for (int k = 0; k < kRows; ++k) {
            const uint32_t at = smem_addr(join + (c + k * step) * 128 + quad * 32 + lane);
#pragma unroll
            for (int i = 0; i < kFewSplits; ++i) part[k][i] = i < splits && c + k * step < rows ? ld_cluster(peer_addr(at, i)) : 0.0f;
          }
#pragma unroll
          for (int k = 0; k < kRows; ++k) {
            float v = part[k][0];
#pragma unroll
            for (int i = 1; i < kFewSplits; ++i) v += part[k][i];
            if (c + k * step < rows && n < p.out_n) few_store(p, ((int64_t)tile.row0 + c + k * step) * p.out_n + n, v);
          }
        }
      }
    }
  }
  if (splits > 1 && warp < 4) cluster_sync_all();
  if (!ok && lane == 0) set_status(kStatusWaitTile);
  __syncwarp();
  pdl_launch_dependents();
  if (splits > 1) cluster_sync_all();   // no CTA's sums are being read any more
}

QMV_DEFINE_STATUS_ACCESSOR(status_b128_few)

namespace {

// Ranks that share a tile's depth: as many as there is room for on the SMs, each with two steps at least, while every tile
// has a cluster of its own and it saves more than joining them costs. Measured, us: 1 x 7168 x 7168 (56 tiles) one rank
// 20.8, two 14.3, three 13.3, five 12.6, clusters that take a second tile 16.7 and more; 64 x 2880 x 2880 five 8.2, six
// 7.9, eight 9.2; 333 x 2880 of depth 1001 (8 steps) one 7.2, two 10.5; 64 x 2880 x 512 one 5.2, two 6.8.
int few_splits(int64_t tiles, int steps, int sms) {
  int splits = 1;
  while (splits < kFewSplits && (splits + 1) * tiles <= kFewCtas * sms && (splits + 1) * 2 <= steps) ++splits;
  return (steps + splits - 1) / splits + kFewJoinSteps < steps ? splits : 1;
}

int64_t hit_experts(const B128GemmArgs& a) { return a.nrows < a.n_experts ? a.nrows : (int64_t)a.n_experts; }
// Columns of a tile, by the rows of an expert, taken as equally full.
int few_columns(const B128GemmArgs& a) {
  const int64_t hit = hit_experts(a);
  return a.nrows <= 16 * hit ? 16 : a.nrows <= 32 * hit ? 32 : 64;
}

template <int BN, bool DX, typename X>
cudaError_t few_go(const B128GemmArgs& a) {
  constexpr bool kQuant = !std::is_void_v<X>;
  using F = Few<BN, kQuant>;
  auto* kernel = b128_few_kernel<BN, DX, X>;
  const int depth = DX ? a.N : a.K;
  FewParams p = {};
  if constexpr (kQuant) {
    p.x = a.x;
    p.ldx = a.ldx;
    p.x_vec = a.ldx % (16 / (int64_t)sizeof(X)) == 0;
  } else {
    p.sx = reinterpret_cast<const float4*>(static_cast<const uint8_t*>(a.xq) + b128_scale_offset(a.nrows, depth));
  }
  p.K = a.K;
  p.sw = a.w_scales;
  p.offsets = a.offsets;
  p.y = a.y;
  p.nrows = a.nrows;
  p.n_experts = a.n_experts;
  p.out_n = DX ? a.K : a.N;
  p.out_type = a.out_type;
  p.x_quads = b128_scale_row(depth) / 4;
  p.k_blocks = b128_blocks(a.K);
  p.n_blocks = b128_blocks(a.N);
  p.steps = b128_blocks(depth);
  p.n_tiles = b128_blocks(p.out_n);
  // tiles that there can be: every expert has at most one partial row tile
  const int64_t row_tiles = a.n_experts == 1 ? (a.nrows + BN - 1) / BN : a.nrows / BN + hit_experts(a);
  const int64_t tiles = row_tiles * p.n_tiles;
  int splits = few_splits(tiles, p.steps, device_sm_count()), most = 0;
  const auto quantizes = [&] {   // X: whether a CTA's rows are few enough
    p.per_split = (p.steps + splits - 1) / splits;
    const int64_t hit = hit_experts(a);
    return p.per_split <= kFewQuantSteps && (a.nrows + hit - 1) / hit * p.per_split <= kFewQuantUnits;
  };
  if (kQuant && !quantizes()) return cudaErrorNotSupported;   // nothing is launched
  g_launch_stage = "cudaFuncSetAttribute";
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)F::smem(QMV_MAX_SORT_EXPERTS));
  if (e != cudaSuccess) return e;
  g_launch_stage = "cuTensorMapEncodeTiled";
  if (encode_fn() == nullptr) return cudaErrorNotSupported;
  CUtensorMap mw, mx;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)a.K, (cuuint64_t)a.N, (cuuint64_t)a.n_experts};
    const cuuint64_t strides[2] = {(cuuint64_t)a.K, (cuuint64_t)a.K * (cuuint64_t)a.N};
    const cuuint32_t box[3] = {128, 128, 1};
    if (!encode(&mw, 3, a.w, dims, strides, box)) return cudaErrorInvalidValue;
  }
  if constexpr (kQuant) {
    mx = mw;
  } else {
    const cuuint64_t row = b128_row_bytes(depth);
    const cuuint64_t dims[2] = {row, (cuuint64_t)a.nrows}, strides[1] = {row};
    const cuuint32_t box[2] = {128, BN};
    if (!encode(&mx, 2, a.xq, dims, strides, box)) return cudaErrorInvalidValue;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(F::threads);
  cfg.dynamicSmemBytes = F::smem(a.n_experts);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // The occupancy query counts one CTA an SM; two run (the fives of 56 tiles are 280 CTAs).
  static PerDevice clusters[kFewSplits + 1];   // of each size that run at once
  for (;; --splits) {
    attr[0].val.clusterDim.x = (unsigned)splits;
    g_launch_stage = "cudaOccupancyMaxActiveClusters";
    e = clusters[splits].get(&most, [&](int* n) {
      cfg.gridDim = dim3((unsigned)(device_sm_count() / splits * splits));
      return cudaOccupancyMaxActiveClusters(n, kernel, &cfg);
    });
    if (e != cudaSuccess) return e;
    most *= kFewCtas;
    if (splits == 1 || most >= tiles) break;
  }
  if (most < 1) return cudaErrorInvalidConfiguration;
  if (kQuant && (most < tiles || !quantizes())) return cudaErrorNotSupported;
  p.per_split = (p.steps + splits - 1) / splits;
  g_launch_stage = "launch";
  cfg.gridDim = dim3((unsigned)(splits * (tiles < most ? tiles : most)));
  cfg.numAttrs = a.stream != nullptr ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, mw, mx, p);
}

template <bool DX>
cudaError_t few_by_rows(const B128GemmArgs& a) {
  const int columns = few_columns(a);
  return columns == 16 ? few_go<16, DX, void>(a) : columns == 32 ? few_go<32, DX, void>(a) : few_go<64, DX, void>(a);
}

}  // namespace

cudaError_t launch_b128_few_linear(const B128GemmArgs& a) {
  if (a.x_type == QMV_F32 || few_columns(a) > 16) return cudaErrorNotSupported;
  return a.x_type == QMV_BF16 ? few_go<16, false, __nv_bfloat16>(a) : few_go<16, false, __half>(a);
}

// By the CTAs' steps, alone or side by side, 2 or 2.5 ns a tile's step over the whole device, or reading the weights at 5.2
// TB/s, as fitted to GB300; experts are taken as equally full, with half a tile more each.
double b128_few_us(const B128GemmArgs& a, int depth, int out_n, int sms) {
  const int columns = few_columns(a), steps = b128_blocks(depth);
  const double hit = (double)hit_experts(a), each = a.nrows / hit / columns;
  const double row_tiles = a.n_experts == 1 ? ceil(each) : hit * (each > 0.5 ? each + 0.5 : 1.0);
  const double tiles = row_tiles * b128_blocks(out_n);
  const int splits = few_splits((int64_t)ceil(tiles), steps, sms);
  const double ctas = tiles * splits, step = columns < 64 ? 0.5 : ctas > sms ? 0.68 : 0.4;   // us, of a CTA
  const double chain = ceil(ctas / (kFewCtas * sms)) * ((steps + splits - 1) / splits) * step;
  const double all = tiles * steps * (columns == 64 ? 2.5e-3 : 2e-3), read = hit * a.N * a.K / 5.2e6;
  return 4.0 + fmax(fmax(all, read), chain + (splits > 1 ? 2.5 : 0.0));
}

cudaError_t launch_b128_few(const B128GemmArgs& a, bool dx) { return dx ? few_by_rows<true>(a) : few_by_rows<false>(a); }

}  // namespace qmv
