// qmv_mxgemm.cu -- products of microscaled activations and microscaled weights
// on the tcgen05 tensor cores, over many rows: dense, and grouped by expert.
//
//   y[r][n] = sum over groups g of 2^(ex[r][g] - 127) 2^(ew[n][g] - 127)
//             sum over the 32 columns of g of q[r][k] c[n][k]
//
// MXFP4 operands take tcgen05.mma kind::mxf4 (64 columns an instruction, two
// scales a row), MXFP8 operands kind::mxf8f6f4 (32 columns, one scale a row):
// the codes go from memory into the tensor core as they are, with their E8M0
// scales, and the sums are held in fp32 in tensor memory.
//
// The weights are read in the layout the decode matvec uses (qmv_layout.h), so
// that one copy in memory serves both. A tile's rows are rows of a tensor map:
// the 8 rows of a row tile lie at the stride of a chunk's lane blocks, and a
// box of (128 bytes, 8 rows, row tiles) lands in shared memory as consecutive
// rows of 128 bytes, swizzled as the tensor core reads them. The last, ragged
// chunk has a map of its own. The scales of a row tile lie lane by lane
// ([lane][row]); a scale warp transposes them while the codes are in flight.
//
// One CTA per SM takes output tiles of 128 rows x 192 columns in turn. Warps:
//   0      issues the TMA copies of codes, kStages steps of 128 bytes deep
//   1      copies a step's scales into tensor memory (tcgen05.cp) and issues
//          its MMAs; two accumulators, so that the next tile's products run
//          while a tile is stored
//   4..7   the epilogue: a thread has a row's columns in order, so SwiGLU, a
//          group's maximum and its quantization need no other thread
//   8..11  read the scales of one step in four each, a step ahead, and write
//          them as tcgen05.cp wants them
// Tiles of an expert follow one another along its rows, so that its weights
// are read from memory once and again from L2.
#include <cuda.h>

#include "qmv_internal.h"
#include "qmv_rows.cuh"

namespace qmv {

constexpr int kTileM = 128;        // rows of activations
constexpr int kTileN = 192;        // rows of weights: the output's columns
constexpr int kGemmThreads = 384;
constexpr int kStages = 5;
constexpr int kScaleWarps = 4;

template <int FMT>
struct GemmFmt {
  static constexpr int step_k = FMT == MXFP4 ? 256 : 128;   // columns in 128 bytes of codes
  static constexpr int mma_k = FMT == MXFP4 ? 64 : 32;      // columns of one MMA
  static constexpr int atoms = step_k / 128;                // scale words of a row per step
  static constexpr int steps_per_chunk = kChunkK / step_k;
  static constexpr uint32_t a_bytes = kTileM * 128;
  static constexpr uint32_t b_bytes = kTileN * 128;
  // scales: 512 bytes hold the words of 128 rows, [row % 32][row / 32]
  static constexpr uint32_t sfa_bytes = atoms * 512;
  static constexpr uint32_t sfb_bytes = atoms * 1024;
  static constexpr uint32_t stage_bytes = (a_bytes + b_bytes + sfa_bytes + sfb_bytes + 1023) / 1024 * 1024;
  static constexpr uint32_t sf_cols = atoms * 12;           // tensor memory columns of a stage's scales
};
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSfCol0 = 2 * kTileN;   // scales follow the two accumulators
static_assert(kSfCol0 + kStages * GemmFmt<MXFP4>::sf_cols <= kTmemCols, "tensor memory");

struct GemmParams {
  const uint8_t* w;
  const uint32_t* x_scales;   // words [ceil(K / 128)][nrows]
  const int32_t* offsets;
  void* y;
  uint32_t* h_scales;         // glu
  int64_t nrows;
  uint64_t expert_stride, rowtile;
  uint32_t full_tile;
  int row_tiles, chunks_full, last_lanes;   // last_lanes: lanes of a ragged last chunk, 0: none
  int K, n_experts, out_n, out_type, n_tiles;
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
               :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int x, int r, int t, int c, int e,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
      :: "r"(dst), "l"(map), "r"(x), "r"(r), "r"(t), "r"(c), "r"(e), "r"(bar) : "memory");
}

// K-major operand in shared memory, rows of 128 bytes with the 128-byte
// swizzle, eight rows every 1024 bytes.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
// Scales in shared memory: 32 rows of 16 bytes, eight every 128 bytes, no swizzle.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}

// Instruction descriptor of the block-scaled kinds: element types (E2M1 is 1 in
// kind::mxf4; E4M3 is 0 in kind::mxf8f6f4), N / 8, E8M0 scales (bit 23), M / 128,
// and which byte of the scale words the instruction's first group uses.
template <int FMT>
__device__ __forceinline__ uint32_t block_idesc(uint32_t sf_byte) {
  constexpr uint32_t elem = FMT == MXFP4 ? 1u : 0u;
  constexpr uint32_t base = (elem << 7) | (elem << 10) | ((uint32_t)(kTileN >> 3) << 17) | (1u << 23) |
                            ((uint32_t)(kTileM >> 7) << 27);
  return base | (sf_byte << 4) | (sf_byte << 29);
}

template <int FMT>
__device__ __forceinline__ void mma_block_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                                 uint32_t sfb, uint32_t accumulate) {
  if constexpr (FMT == MXFP4) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
  } else {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
  }
}

__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" :: "r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ void mma_commit_to(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_one(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void tc_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 accumulator columns of this thread's row.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// Waits for this warp's tensor memory loads; r is not used before it.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :: "memory");
  asm volatile("" : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                    "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                    "+r"(r[30]), "+r"(r[31]) :: "memory");
}

// One lane of a converged warp, as the compiler knows it: the operands of the
// instructions it guards stay in uniform registers. (With lane == 0 in its
// place each tcgen05 instruction took about 100 cycles to issue, and the
// 8192 x 7168 x 7168 MXFP4 product 295 us.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// The 4 x 4 bytes of four words, transposed.
__device__ __forceinline__ void transpose4(const uint32_t (&a)[4], uint32_t (&t)[4]) {
  const uint32_t p = prmt(a[0], a[1], 0x5140), q = prmt(a[2], a[3], 0x5140);
  const uint32_t r = prmt(a[0], a[1], 0x7362), s = prmt(a[2], a[3], 0x7362);
  t[0] = prmt(p, q, 0x5410);
  t[1] = prmt(p, q, 0x7632);
  t[2] = prmt(r, s, 0x5410);
  t[3] = prmt(r, s, 0x7632);
}

// silu(g) * u with the special functions' exponential and reciprocal (a few
// units of the last fp32 place): h is rounded to 2 or 4 significant bits next.
__device__ __forceinline__ float swiglu_fast(float g, float u) {
  return __fdividef(g, 1.0f + __expf(-g)) * u;
}

// Where one output tile lies.
struct Tile {
  int expert;
  int row0;    // first row, and rows of the expert from there on
  int rows;
  int n;       // column tile
};

// Output tile t: experts in order, the column tiles of an expert in order, the
// row tiles of a column tile in order. first_tile[e]: tiles before expert e.
__device__ __forceinline__ Tile tile_at(int t, const int* first_tile, const int* first_row, int n_experts) {
  int lo = 0, hi = n_experts - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (first_tile[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const int rows = first_row[lo + 1] - first_row[lo];
  const int mt = (rows + kTileM - 1) / kTileM;
  const int i = t - first_tile[lo];
  Tile r;
  r.expert = lo;
  r.n = i / mt;
  const int m = i - r.n * mt;
  r.row0 = first_row[lo] + m * kTileM;
  r.rows = rows - m * kTileM;
  return r;
}

// The scales of one step as a scale warp's lane reads them: the words of four
// rows of activations per 128 columns, and 32 bytes ([lane][row], four lanes)
// of one or two row tiles of weights.
template <int FMT>
struct StepScales {
  static constexpr int kItems = kTileN / 8 * GemmFmt<FMT>::atoms;   // (row tile, 128 columns) pairs
  static constexpr int kRounds = (kItems + 31) / 32;
  uint32_t a[GemmFmt<FMT>::atoms][4];
  uint4 b[kRounds][2];

  __device__ __forceinline__ void load(const GemmParams& p, const Tile& t, int step, int lane) {
    using F = GemmFmt<FMT>;
    const int words = mx_scale_words(p.K);
#pragma unroll
    for (int k = 0; k < F::atoms; ++k) {
      const int kb = step * F::atoms + k;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = min((int64_t)t.row0 + lane + 32 * i, p.nrows - 1);   // rows past the last are not stored
        a[k][i] = kb < words ? __ldg(p.x_scales + (int64_t)kb * p.nrows + row) : 0u;
      }
    }
    const int chunk = step / F::steps_per_chunk;
    const int lanes = chunk < p.chunks_full ? 32 : p.last_lanes;
    const uint8_t* base = p.w + (uint64_t)t.expert * p.expert_stride + (uint64_t)chunk * p.full_tile +
                          tile_code_bytes(FMT, lanes);
    const int l0 = (step % F::steps_per_chunk) * (F::step_k / 32);
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int item = lane + 32 * i;
      const int rt = t.n * (kTileN / 8) + item / F::atoms;
      const int l = l0 + 4 * (item % F::atoms);
      const uint4* src = reinterpret_cast<const uint4*>(base + (uint64_t)rt * p.rowtile + (uint64_t)l * kRows);
      const bool in = item < kItems && rt < p.row_tiles;
      // two lanes of 8 rows a load; the tile's padding to 16 bytes is zero
      b[i][0] = in && l < lanes ? __ldg(src) : make_uint4(0, 0, 0, 0);
      b[i][1] = in && l + 2 < lanes ? __ldg(src + 1) : make_uint4(0, 0, 0, 0);
    }
  }

  __device__ __forceinline__ void store(uint8_t* sfa, uint8_t* sfb, int lane) const {
    using F = GemmFmt<FMT>;
#pragma unroll
    for (int k = 0; k < F::atoms; ++k) {
      *reinterpret_cast<uint4*>(sfa + k * 512 + lane * 16) = make_uint4(a[k][0], a[k][1], a[k][2], a[k][3]);
    }
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int item = lane + 32 * i;
      if (item < kItems) {
        const uint32_t lo[4] = {b[i][0].x, b[i][0].z, b[i][1].x, b[i][1].z};   // rows 0..3 of four lanes
        const uint32_t hi[4] = {b[i][0].y, b[i][0].w, b[i][1].y, b[i][1].w};   // rows 4..7
        uint32_t w[8];
        transpose4(lo, *reinterpret_cast<uint32_t(*)[4]>(w));
        transpose4(hi, *reinterpret_cast<uint32_t(*)[4]>(w + 4));
        const int row0 = item / F::atoms * 8;
        uint8_t* atom = sfb + (item % F::atoms) * 1024 + (row0 / 128) * 512 + (row0 % 128) / 32 * 4;
#pragma unroll
        for (int r = 0; r < 8; ++r) *reinterpret_cast<uint32_t*>(atom + ((row0 + r) % 32) * 16) = w[r];
      }
    }
  }
};

template <typename T>
__device__ __forceinline__ void store_columns(T* out, const uint32_t (&r)[32], int count, bool vec) {
  if (vec && count >= 32) {
    constexpr int per = 16 / (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < 32 / per; ++i) {
      uint4 v;
      T* e = reinterpret_cast<T*>(&v);
#pragma unroll
      for (int k = 0; k < per; ++k) e[k] = from_f32<T>(__uint_as_float(r[i * per + k]));
      reinterpret_cast<uint4*>(out)[i] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (i < count) out[i] = from_f32<T>(__uint_as_float(r[i]));
    }
  }
}

// HFMT < 0: y as out_type. Otherwise the columns are gate and up rows by fours
// and silu(gate) * up is stored, quantized to HFMT.
template <int FMT, int HFMT>
__global__ void __launch_bounds__(kGemmThreads, 1)
mx_gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
               const __grid_constant__ CUtensorMap map_last, const __grid_constant__ GemmParams p) {
  using F = GemmFmt<FMT>;
  extern __shared__ uint8_t dyn[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
  int* first_tile = reinterpret_cast<int*>(stages + kStages * F::stage_bytes);   // [n_experts + 1]
  int* first_row = first_tile + p.n_experts + 1;                                 // [n_experts + 1]
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], done;
  __shared__ uint32_t tmem_base;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&full[i]), 2);   // the copies' thread and the step's scale warp
      mbar_init(smem_addr(&empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&acc_full[i]), 1);
      mbar_init(smem_addr(&acc_empty[i]), 4);
    }
    mbar_init(smem_addr(&done), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_addr(&tmem_base)),
                 "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  if (warp == 0) {
    int tiles = 0;
    for (int e0 = 0; e0 < p.n_experts; e0 += 32) {
      const int e = e0 + lane;
      int lo = 0, hi = 0;
      if (e < p.n_experts) {
        lo = p.offsets != nullptr ? __ldg(p.offsets + e) : 0;
        hi = p.offsets != nullptr ? __ldg(p.offsets + e + 1) : (int)p.nrows;
        // offsets that do not name rows of this call name none
        lo = max(0, min(lo, (int)p.nrows));
        hi = max(lo, min(hi, (int)p.nrows));
        first_row[e] = lo;
        if (e == p.n_experts - 1) first_row[e + 1] = hi;
      }
      int inc = (hi - lo + kTileM - 1) / kTileM * p.n_tiles;
      const int own = inc;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        inc += lane >= o ? v : 0;
      }
      if (e < p.n_experts) first_tile[e] = tiles + inc - own;
      tiles += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) first_tile[p.n_experts] = tiles;
  }
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  const uint32_t tmem = tmem_base;
  const int tiles = first_tile[p.n_experts];
  const int steps = p.chunks_full * F::steps_per_chunk + (p.last_lanes * 32 + F::step_k - 1) / F::step_k;
  bool ok = true;

  if (warp == 0) {
    // ---- copies of codes
    int it = 0;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const Tile tile = tile_at(t, first_tile, first_row, p.n_experts);
      for (int s = 0; s < steps; ++s, ++it) {
        const int st = it % kStages;
        if (!mbar_wait_bounded(smem_addr(&empty[st]), ((it / kStages) & 1) ^ 1, kWaitLimitNs)) { ok = false; break; }
        if (elect_one()) {
          const uint32_t bar = smem_addr(&full[st]);
          const uint32_t dst = smem_addr(stages + (uint32_t)st * F::stage_bytes);
          mbar_arrive_expect_tx(bar, F::a_bytes + F::b_bytes);
          tma_load_2d(dst, &map_x, s * 128, tile.row0, bar);
          const int chunk = s / F::steps_per_chunk;
          const int x = (s % F::steps_per_chunk) * 128;
          if (chunk < p.chunks_full) {
            tma_load_5d(dst + F::a_bytes, &map_w, x, 0, tile.n * (kTileN / 8), chunk, tile.expert, bar);
          } else {
            tma_load_5d(dst + F::a_bytes, &map_last, x, 0, tile.n * (kTileN / 8), 0, tile.expert, bar);
          }
        }
        __syncwarp();
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
    // ---- products
    int it = 0, n = 0;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++n) {
      const int acc = n & 1;
      if (!mbar_wait_bounded(smem_addr(&acc_empty[acc]), ((n >> 1) & 1) ^ 1, kWaitLimitNs)) { ok = false; break; }
      tc_after_sync();
      const uint32_t d = tmem + (uint32_t)(acc * kTileN);
      for (int s = 0; s < steps; ++s, ++it) {
        const int st = it % kStages;
        if (!mbar_wait_bounded(smem_addr(&full[st]), (it / kStages) & 1, kWaitLimitNs)) { ok = false; break; }
        tc_after_sync();
        if (elect_one()) {
          const uint32_t a0 = smem_addr(stages + (uint32_t)st * F::stage_bytes);
          const uint32_t b0 = a0 + F::a_bytes, sfa = b0 + F::b_bytes, sfb = sfa + F::sfa_bytes;
          const uint32_t sf = tmem + kSfCol0 + (uint32_t)st * F::sf_cols;
#pragma unroll
          for (int k = 0; k < F::atoms; ++k) {
            scales_to_tmem(sf + (uint32_t)k * 12, scale_desc(sfa + (uint32_t)k * 512));
            scales_to_tmem(sf + (uint32_t)k * 12 + 4, scale_desc(sfb + (uint32_t)k * 1024));
            scales_to_tmem(sf + (uint32_t)k * 12 + 8, scale_desc(sfb + (uint32_t)k * 1024 + 512));
          }
          const int left = p.K - s * F::step_k;
#pragma unroll
          for (int j = 0; j < F::step_k / F::mma_k; ++j) {
            if (j * F::mma_k < left) {
              constexpr int per_atom = 128 / F::mma_k;
              const uint32_t col = sf + (uint32_t)(j / per_atom) * 12;
              mma_block_scaled<FMT>(d, operand_desc(a0 + (uint32_t)j * 32), operand_desc(b0 + (uint32_t)j * 32),
                                    block_idesc<FMT>((uint32_t)(j % per_atom) * (F::mma_k / 32)), col, col + 4,
                                    (s > 0 || j > 0) ? 1u : 0u);
            }
          }
          mma_commit_to(smem_addr(&empty[st]));
          if (s == steps - 1) mma_commit_to(smem_addr(&acc_full[acc]));
        }
        __syncwarp();
      }
    }
    if (elect_one()) mma_commit_to(smem_addr(&done));
    __syncwarp();
    if (!mbar_wait_bounded(smem_addr(&done), 0, kWaitLimitNs)) ok = false;
  } else if (warp >= 8) {
    // ---- scales: every fourth step, loaded one turn ahead of its slot in the ring
    const int mine = warp - 8;
    StepScales<FMT> cur;
    int it = 0, t = blockIdx.x, s = mine;
    Tile tile{};
    // step `mine`, `mine` + 4, ... of this CTA's steps, tile after tile
    while (t < tiles && s >= steps) { s -= steps; t += gridDim.x; }
    if (t < tiles) {
      tile = tile_at(t, first_tile, first_row, p.n_experts);
      cur.load(p, tile, s, lane);
    }
    it = mine;
    while (t < tiles) {
      int t2 = t, s2 = s + kScaleWarps;
      while (t2 < tiles && s2 >= steps) { s2 -= steps; t2 += gridDim.x; }
      StepScales<FMT> next = cur;
      if (t2 < tiles) {
        if (t2 != t) tile = tile_at(t2, first_tile, first_row, p.n_experts);
        next.load(p, tile, s2, lane);
      }
      const int st = it % kStages;
      if (!mbar_wait_bounded(smem_addr(&empty[st]), ((it / kStages) & 1) ^ 1, kWaitLimitNs)) { ok = false; break; }
      uint8_t* sfa = stages + (uint32_t)st * F::stage_bytes + F::a_bytes + F::b_bytes;
      cur.store(sfa, sfa + F::sfa_bytes, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_one(smem_addr(&full[st]));
      cur = next;
      t = t2;
      s = s2;
      it += kScaleWarps;
    }
  } else if (warp >= 4) {
    // ---- epilogue: thread = row 32 (warp - 4) + lane of the tile
    const int quad = warp - 4;
    int n = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++n) {
      const int acc = n & 1;
      const Tile tile = tile_at(t, first_tile, first_row, p.n_experts);
      if (!mbar_wait_bounded(smem_addr(&acc_full[acc]), (n >> 1) & 1, kWaitLimitNs)) { ok = false; break; }
      tc_after_sync();
      const int r = quad * 32 + lane;
      const bool live = r < tile.rows;
      const int64_t row = (int64_t)tile.row0 + r;
      const uint32_t d = tmem + (uint32_t)(acc * kTileN) + ((uint32_t)(quad * 32) << 16);
      if constexpr (HFMT < 0) {
        const int size = p.out_type == QMV_F32 ? 4 : 2;
        const bool vec = ((int64_t)p.out_n * size) % 16 == 0;
#pragma unroll 1
        for (int c = 0; c < kTileN; c += 32) {
          uint32_t v[32];
          tmem_ld32(d + (uint32_t)c, v);
          tmem_ld_wait(v);
          const int n0 = tile.n * kTileN + c;
          if (live && n0 < p.out_n) {
            const int64_t at = row * p.out_n + n0;
            if (p.out_type == QMV_BF16) store_columns(static_cast<__nv_bfloat16*>(p.y) + at, v, p.out_n - n0, vec);
            else if (p.out_type == QMV_F16) store_columns(static_cast<__half*>(p.y) + at, v, p.out_n - n0, vec);
            else store_columns(static_cast<float*>(p.y) + at, v, p.out_n - n0, vec);
          }
        }
      } else {
        const uint64_t h_bytes = mx_row_bytes(HFMT, p.out_n);
#pragma unroll 1
        for (int c = 0; c < kTileN; c += 64) {
          uint32_t v[2][32];
          tmem_ld32(d + (uint32_t)c, v[0]);
          tmem_ld32(d + (uint32_t)c + 32, v[1]);
          tmem_ld_wait(v[0]);
          tmem_ld_wait(v[1]);
          const int n0 = (tile.n * kTileN + c) / 2;   // a group of 32 columns of h
          if (live && n0 < p.out_n) {
            float h[4][8];
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                // h column 8 i + k: row tile 2 i + k / 4, gate row k % 4, up row k % 4 + 4
                const int col = (2 * i + k / 4) * 8 + k % 4;
                h[i][k] = swiglu_fast(__uint_as_float(v[col / 32][col % 32]),
                                      __uint_as_float(v[(col + 4) / 32][(col + 4) % 32]));
              }
              m = max(m, amax_bits8(h[i]));
            }
            const uint32_t e = group_e8m0<HFMT>(m);
            uint8_t* out = static_cast<uint8_t*>(p.y) + (uint64_t)row * h_bytes;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[HFMT == MXFP4 ? 1 : 2];
              mx_codes8<HFMT>(h[i], e, w);
              store_codes8<HFMT>(out, n0 + 8 * i, w);
            }
            uint8_t* sc = reinterpret_cast<uint8_t*>(p.h_scales + (int64_t)(n0 / 128) * p.nrows + row);
            const int b = n0 / 32 % 4;
            sc[b] = (uint8_t)e;
            if (n0 + 32 == p.out_n) {   // bytes past the last group are zero
              for (int i = b + 1; i < 4; ++i) sc[i] = 0;
            }
          }
        }
      }
      tc_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_one(smem_addr(&acc_empty[acc]));
    }
  }
  if (!ok && lane == 0) set_status(kStatusWaitTile);
  __syncwarp();
  pdl_launch_dependents();
  __syncthreads();
  if (warp == 1) {
    tc_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(kTmemCols));
  }
}

QMV_DEFINE_STATUS_ACCESSOR(status_mx_gemm)

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult st;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &st) != cudaSuccess ||
        st != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

bool encode(CUtensorMap* map, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box,
                     one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT, int HFMT>
cudaError_t go(const MxGemmArgs& a) {
  using F = GemmFmt<FMT>;
  const Geometry g = make_geometry(FMT, a.N, a.K);
  const int lane_bytes = lane_code_bytes(FMT);
  GemmParams p = {};
  p.w = static_cast<const uint8_t*>(a.w);
  p.nrows = a.nrows;
  p.x_scales = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.xq) + mx_scale_offset(FMT, a.nrows, a.K));
  p.offsets = a.offsets;
  p.y = a.y;
  if (HFMT >= 0) {
    p.h_scales = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.y) + mx_scale_offset(a.h_fmt, a.nrows, a.out_n));
  }
  p.expert_stride = g.expert;
  p.rowtile = g.rowtile;
  p.full_tile = g.full_tile;
  p.row_tiles = g.row_tiles;
  p.chunks_full = a.K / kChunkK;
  p.last_lanes = (a.K % kChunkK) / kLaneK;
  p.K = a.K;
  p.n_experts = a.n_experts;
  p.out_n = a.out_n;
  p.out_type = a.out_type;
  p.n_tiles = (g.row_tiles * kRows + kTileN - 1) / kTileN;

  g_launch_stage = "cuTensorMapEncodeTiled";
  if (encode_fn() == nullptr) return cudaErrorNotSupported;
  CUtensorMap mx, mw, ml;
  {
    const cuuint64_t row = mx_row_bytes(FMT, a.K);
    const cuuint64_t dims[2] = {row, (cuuint64_t)a.nrows}, strides[1] = {row};
    const cuuint32_t box[2] = {128, kTileM};
    if (!encode(&mx, 2, a.xq, dims, strides, box)) return cudaErrorInvalidValue;
  }
  const cuuint32_t box[5] = {128, kRows, kTileN / kRows, 1, 1};
  // lanes of the map's chunks, chunks, first byte
  const auto weights = [&](CUtensorMap* m, int lanes, int chunks, uint64_t at) {
    const cuuint64_t row = (cuuint64_t)lanes * lane_bytes;
    const cuuint64_t dims[5] = {row, kRows, (cuuint64_t)g.row_tiles, (cuuint64_t)chunks, (cuuint64_t)a.n_experts};
    const cuuint64_t strides[4] = {row, g.rowtile, g.full_tile, g.expert};
    return encode(m, 5, p.w + at, dims, strides, box);
  };
  if (p.chunks_full > 0 && !weights(&mw, 32, p.chunks_full, 0)) return cudaErrorInvalidValue;
  if (p.last_lanes > 0 && !weights(&ml, p.last_lanes, 1, (uint64_t)p.chunks_full * g.full_tile)) return cudaErrorInvalidValue;
  if (p.chunks_full == 0) mw = ml;
  if (p.last_lanes == 0) ml = mw;

  const size_t smem = 1024 + (size_t)kStages * F::stage_bytes + 2 * ((size_t)a.n_experts + 1) * sizeof(int);
  g_launch_stage = "cudaFuncSetAttribute";
  cudaError_t e = cudaFuncSetAttribute(mx_gemm_kernel<FMT, HFMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  // no more CTAs than tiles there can be: every expert has at most one partial row tile
  const int64_t row_tiles = a.nrows / kTileM + (a.nrows < a.n_experts ? a.nrows : (int64_t)a.n_experts);
  int64_t grid = row_tiles * p.n_tiles;
  if (grid > device_sm_count()) grid = device_sm_count();
  g_launch_stage = "launch";
  return launch_pdl(mx_gemm_kernel<FMT, HFMT>, dim3((unsigned)grid), dim3(kGemmThreads), smem, a.stream, mx, mw, ml, p);
}

template <int FMT>
cudaError_t by_h(const MxGemmArgs& a) {
  if (!a.glu) return go<FMT, -1>(a);
  return a.h_fmt == MXFP4 ? go<FMT, MXFP4>(a) : go<FMT, MXFP8>(a);
}

}  // namespace

cudaError_t launch_mx_gemm(const MxGemmArgs& a) { return a.fmt == MXFP4 ? by_h<MXFP4>(a) : by_h<MXFP8>(a); }

}  // namespace qmv
