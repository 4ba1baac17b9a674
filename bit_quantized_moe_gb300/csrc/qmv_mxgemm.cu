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
// One CTA per SM takes output tiles of 128 rows x 128 or 64 columns in turn, or
// a pair of CTAs on two SMs tiles of 256 x 192 (pick_tile). Warps:
//   0      issues the TMA copies of codes, 128 bytes of every row a step.
//          (Asking for the weights of 16 later steps in L2, by boxes or by
//          whole tiles, was slower at every size measured: 132 rows of 32
//          experts 57 -> 79 us.)
//   1      copies a step's scales into tensor memory (tcgen05.cp) and issues
//          its MMAs; two accumulators, so that the next tile's products run
//          while a tile is stored
//   4..11  the epilogue, one warpgroup an accumulator: a thread has a row's
//          columns in order, so SwiGLU, a group's maximum and its quantization
//          need no other thread
//   3, 12..19  read the scales of one step in nine each, a turn ahead, and
//          write them as tcgen05.cp wants them
//   2      tells warp 1, on the codes' barrier, that a step's scales are there
// Tiles of an expert follow one another along its rows, so that its weights
// are read from memory once and again from L2.
#include <cmath>

#include "qmv_internal.h"
#include "qmv_rows.cuh"
#include "qmv_tc.cuh"

namespace qmv {

constexpr int kTileM = 128;        // rows of activations of one CTA
constexpr int kGemmThreads = 640;
constexpr int kScaleWarps = 9;      // warps 3 and 12..19 (8192 x 7168 x 7168 MXFP4: six 152 us, nine 141, ten 143)
// Columns of 16-bit outputs that a thread parks in shared memory before its
// warp stores them row by row, and the pitch of a row there (an odd number of
// 16 bytes: no bank conflicts between rows).
constexpr int kParkCols = 32;
constexpr int kParkPitch = kParkCols * 2 + 16;

template <int FMT, int TN, bool PAIR>
struct GemmFmt {
  static constexpr int step_k = FMT == MXFP4 ? 256 : 128;   // columns in 128 bytes of codes
  static constexpr int mma_k = FMT == MXFP4 ? 64 : 32;      // columns of one MMA
  static constexpr int atoms = step_k / 128;                // scale words of a row per step
  static constexpr int steps_per_chunk = kChunkK / step_k;
  static constexpr uint32_t a_bytes = kTileM * 128;
  // Rows of one copy of activations: a CTA makes as many as its live rows need. Copies of rows that are not there are
  // not free (17 rows: boxes of 128 rows took longer than 128 rows did), and an expert's last tile is half empty.
  static constexpr int x_rows = PAIR ? 64 : 32;
  static constexpr int b_rows = PAIR ? TN / 2 : TN;         // a pair's CTAs hold half of the weights each
  static constexpr uint32_t b_bytes = b_rows * 128;
  static constexpr uint32_t stage_bytes = a_bytes + b_bytes;
  // scales: 512 bytes, and four columns of tensor memory, hold the words of 128 rows, [row % 32][row / 32]
  static constexpr int b_blocks = (TN + 127) / 128;
  static constexpr uint32_t sfa_bytes = atoms * 512;
  static constexpr uint32_t sfb_bytes = atoms * b_blocks * 512;
  static constexpr uint32_t sf_bytes = sfa_bytes + sfb_bytes;
  static constexpr uint32_t atom_cols = 4 + 4 * b_blocks;   // tensor memory columns of 128 columns' scales
  static constexpr uint32_t sf_cols = atoms * atom_cols;
  static constexpr int stages = PAIR ? 6 : (TN == 128 ? 5 : 7);
  // Steps that the scales may be ahead. At least the scale warps: a warp may then not be two uses of a place ahead of
  // the MMAs, which its barrier's phase bit could not tell from none.
  static constexpr int sf_stages = 9;
  static_assert(kScaleWarps <= sf_stages && stages <= sf_stages, "phases of the barriers");
  static constexpr uint32_t park_bytes = 2 * kTileM * kParkPitch;
  static constexpr uint32_t sf_col0 = 2 * TN;               // scales follow the two accumulators
  // Steps whose scales tensor memory holds; a step waits for the MMAs of the one whose place it takes.
  static constexpr int sf_slots = (int)((512 - sf_col0) / sf_cols) < stages ? (int)((512 - sf_col0) / sf_cols) : stages;
  static constexpr uint32_t tmem_cols = sf_col0 + sf_slots * sf_cols <= 256 ? 256 : 512;
  static_assert(sf_slots >= 4 && sf_col0 + sf_slots * sf_cols <= tmem_cols, "tensor memory");
  // Dynamic shared memory: the rings from a 1024-byte boundary on, the parked columns, two tables of the experts.
  static constexpr size_t smem_bytes(int n_experts) {
    return 1024 + (size_t)stages * stage_bytes + sf_stages * sf_bytes + park_bytes + 2 * ((size_t)n_experts + 1) * sizeof(int);
  }
  static_assert(smem_bytes(QMV_MAX_SORT_EXPERTS) + 1024 <= 227 * 1024, "shared memory, with 1 KB for the barriers");
};

struct GemmParams {
  const uint8_t* w;
  const uint32_t* x_scales;   // words [ceil(K / 128)][nrows]
  const int32_t* offsets;
  void* y;
  float* wide;                // out_type fp16: null, or where sums that fp16 does not hold are kept
  uint32_t* h_scales;         // glu
  int64_t nrows;
  uint64_t expert_stride, rowtile;
  uint32_t full_tile;
  int row_tiles, chunks_full, last_lanes;   // last_lanes: lanes of a ragged last chunk, 0: none
  int K, n_experts, out_n, out_type, n_tiles;
};

// Scales in shared memory: 32 rows of 16 bytes, eight every 128 bytes, no swizzle.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}

// Instruction descriptor of the block-scaled kinds: element types (E2M1 is 1 in
// kind::mxf4; E4M3 is 0 in kind::mxf8f6f4), N / 8, E8M0 scales (bit 23), M / 128,
// and which byte of the scale words the instruction's first group uses.
template <int FMT, int TN, bool PAIR>
__device__ __forceinline__ uint32_t block_idesc(uint32_t sf_byte) {
  constexpr uint32_t elem = FMT == MXFP4 ? 1u : 0u;
  constexpr uint32_t base = (elem << 7) | (elem << 10) | ((uint32_t)(TN >> 3) << 17) | (1u << 23) |
                            ((uint32_t)((PAIR ? 2 * kTileM : kTileM) >> 7) << 27);
  return base | (sf_byte << 4) | (sf_byte << 29);
}

#define QMV_BLOCK_MMA(GROUP, KIND)                                                              \
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n tcgen05.mma.cta_group::" GROUP       \
               ".kind::" KIND " [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d), "l"(a), "l"(b),   \
               "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                                   \
               : "memory")

template <int FMT, bool PAIR>
__device__ __forceinline__ void mma_block_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                                 uint32_t sfb, uint32_t accumulate) {
  if constexpr (FMT == MXFP4) {
    if constexpr (PAIR) QMV_BLOCK_MMA("2", "mxf4.block_scale.scale_vec::2X");
    else QMV_BLOCK_MMA("1", "mxf4.block_scale.scale_vec::2X");
  } else {
    if constexpr (PAIR) QMV_BLOCK_MMA("2", "mxf8f6f4.block_scale.scale_vec::1X");
    else QMV_BLOCK_MMA("1", "mxf8f6f4.block_scale.scale_vec::1X");
  }
}
#undef QMV_BLOCK_MMA

// PAIR: each CTA's tensor memory from the same place in its own shared memory.
template <bool PAIR>
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint64_t desc) {
  if constexpr (PAIR) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" :: "r"(taddr), "l"(desc) : "memory");
  else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" :: "r"(taddr), "l"(desc) : "memory");
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

// silu(g) * u within 12 * 2^-24 of itself for every g from about -167 up (0
// below), in the range of the result: with t = e^-|g| <= 1 as
// g * (g < 0 ? t : 1) / (1 + t) * u, whose divisor lies in [1, 2]. t is
// 2^(-|g| log2 e) by the special function, the product's rounding error made
// good to first order. Where t would leave the normal numbers its exponent is
// taken 115 higher and u's 115 lower. (The layer of 4096 x 4 slots, 32 experts
// of 2880: 284 us; with expf and an IEEE division 501.)
__device__ __forceinline__ float swiglu_range(float g, float u) {
  constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = (float)(1.4426950408889634 - (double)kLog2e);
  constexpr float kLn2 = 0.6931471805599453f;
  const float a = fabsf(g);
  float x = -a * kLog2e;
  const float low = fmaf(-a, kLog2eLow, fmaf(-a, kLog2e, -x));
  const bool far = g < -79.0f;
  if (far) {
    x += 115.0f;   // exact
    u *= 0x1p-115f;
  }
  float t, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(x));
  t = fmaf(t, low * kLn2, t);
  const float d = far ? 1.0f : 1.0f + t;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return (g < 0.0f ? g * t : g) * r * u;
}

// Where a CTA's part of one output tile lies.
struct Tile {
  int expert;
  int row0;    // first row, and rows of the expert from there on (none: 0 or less)
  int rows;
  int n;       // column tile
};

// Output tile t: experts in order, the column tiles of an expert in order, the
// row tiles of a column tile in order. first_tile[e]: tiles before expert e.
template <bool PAIR>
__device__ __forceinline__ Tile tile_at(int t, const int* first_tile, const int* first_row, int n_experts, int rank) {
  int lo = 0, hi = n_experts - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (first_tile[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const int rows = first_row[lo + 1] - first_row[lo];
  constexpr int unit = PAIR ? 2 * kTileM : kTileM;
  const int mt = (rows + unit - 1) / unit;
  const int i = t - first_tile[lo];
  Tile r;
  r.expert = lo;
  r.n = i / mt;
  const int m = i - r.n * mt;
  r.row0 = first_row[lo] + m * unit + rank * kTileM;
  r.rows = rows - m * unit - rank * kTileM;
  return r;
}

// The scales of one step as a scale warp's lane reads them: the words of four
// rows of activations per 128 columns, and 32 bytes ([lane][row], four lanes)
// of one or two row tiles of weights.
template <int FMT, int TN>
struct StepScales {
  using F = GemmFmt<FMT, TN, (TN > 128)>;   // the scales of a tile are the same for one CTA and a pair
  static constexpr int kItems = TN / 8 * F::atoms;   // (row tile, 128 columns) pairs
  static constexpr int kRounds = (kItems + 31) / 32;
  uint32_t a[F::atoms][4];
  uint4 b[kRounds][2];

  __device__ __forceinline__ void load(const GemmParams& p, const Tile& t, int step, int lane) {
    const int words = mx_scale_words(p.K);
#pragma unroll
    for (int k = 0; k < F::atoms; ++k) {
      const int kb = step * F::atoms + k;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = min((int64_t)t.row0 + lane + 32 * i, p.nrows - 1);   // rows past the last are not stored
        a[k][i] = kb < words ? p.x_scales[(int64_t)kb * p.nrows + row] : 0u;
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
      const int rt = t.n * (TN / 8) + item / F::atoms;
      const int l = l0 + 4 * (item % F::atoms);
      const uint4* src = reinterpret_cast<const uint4*>(base + (uint64_t)rt * p.rowtile + (uint64_t)l * kRows);
      const bool in = item < kItems && rt < p.row_tiles;
      // two lanes of 8 rows a load; the tile's padding to 16 bytes is zero
      b[i][0] = in && l < lanes ? __ldg(src) : make_uint4(0, 0, 0, 0);
      b[i][1] = in && l + 2 < lanes ? __ldg(src + 1) : make_uint4(0, 0, 0, 0);
    }
  }

  __device__ __forceinline__ void store(uint8_t* sfa, uint8_t* sfb, int lane) const {
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
        // Row r of every item lies in the same eighth of the banks, so lanes take the rows in orders of their own:
        // w[r] becomes the word of row r ^ x, x different in lanes whose items otherwise share banks.
        const int x = F::atoms == 2 ? lane & 7 : (lane & 3) | (lane >> 4 & 1) << 2;
#pragma unroll
        for (int bit = 1; bit < 8; bit <<= 1) {
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            if ((r & bit) == 0) {
              const uint32_t u = w[r], v = w[r | bit];
              w[r] = (x & bit) ? v : u;
              w[r | bit] = (x & bit) ? u : v;
            }
          }
        }
        const int row0 = item / F::atoms * 8;
        uint8_t* atom = sfb + ((item % F::atoms) * F::b_blocks + row0 / 128) * 512 + (row0 % 32) * 16 + (row0 % 128) / 32 * 4;
#pragma unroll
        for (int r = 0; r < 8; ++r) *reinterpret_cast<uint32_t*>(atom + (r ^ x) * 16) = w[r];
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

template <typename T>
__device__ __forceinline__ void park_columns(uint8_t* at, const uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 v;
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = from_f32<T>(__uint_as_float(r[i * 8 + k]));
    reinterpret_cast<uint4*>(at)[i] = v;
  }
}

// HFMT < 0: y as out_type. Otherwise the columns are gate and up rows by fours
// and silu(gate) * up is stored, quantized to HFMT.
// PAIR: two CTAs (a cluster) share a tile of 256 rows; the first, the leader,
// issues the MMAs of both.
template <int FMT, int HFMT, int TN, bool PAIR>
__global__ void __launch_bounds__(kGemmThreads, 1)
mx_gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
               const __grid_constant__ CUtensorMap map_last, const __grid_constant__ GemmParams p) {
  using F = GemmFmt<FMT, TN, PAIR>;
  constexpr int kStages = F::stages;
  constexpr int kCtas = PAIR ? 2 : 1;
  extern __shared__ uint8_t dyn[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
  uint8_t* scales = stages + kStages * F::stage_bytes;   // [sf_stages][sf_bytes]
  uint8_t* park = scales + F::sf_stages * F::sf_bytes;
  int* first_tile = reinterpret_cast<int*>(park + F::park_bytes);   // [n_experts + 1]
  int* first_row = first_tile + p.n_experts + 1;                    // [n_experts + 1]
  // Barriers of a step: all of it has arrived, its scales have, its MMAs are complete. The scales run up to sf_stages
  // steps ahead, the codes kStages; both wait for the MMAs of the step whose place they take.
  __shared__ __align__(8) uint64_t full[F::stages], sf_full[F::sf_stages], used[F::sf_stages];
  __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2], done;
  __shared__ uint32_t tmem_base;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0), lane = threadIdx.x & 31;
  const int rank = PAIR ? (int)cluster_rank() : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(smem_addr(&full[i]), 1);
    for (int i = 0; i < F::sf_stages; ++i) {
      mbar_init(smem_addr(&sf_full[i]), kCtas);   // every CTA's scale warp
      mbar_init(smem_addr(&used[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&acc_full[i]), 1);
      mbar_init(smem_addr(&acc_empty[i]), 4 * kCtas);
    }
    mbar_init(smem_addr(&done), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_addr(&tmem_base)),
                   "r"(F::tmem_cols) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_addr(&tmem_base)),
                   "r"(F::tmem_cols) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
  }
  pdl_wait();
  if (warp == 0) {
    constexpr int unit = kCtas * kTileM;
    expert_tiles(p.offsets, (int)p.nrows, p.n_experts, unit, p.n_tiles, lane, first_row, first_tile);
  }
  tc_before_sync();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();   // both CTAs' barriers exist
  tc_after_sync();
  const uint32_t tmem = tmem_base;
  const int tiles = first_tile[p.n_experts];
  const int steps = p.chunks_full * F::steps_per_chunk + (p.last_lanes * 32 + F::step_k - 1) / F::step_k;
  const int t0 = (int)blockIdx.x / kCtas, dt = (int)gridDim.x / kCtas;
  const auto tile_of = [&](int t) { return tile_at<PAIR>(t, first_tile, first_row, p.n_experts, rank); };
  bool ok = true;

  // Waits until the MMAs of step `it` - AHEAD are complete.
  const auto wait_used = [&](int it, int ahead) {
    const int j = it - ahead;
    return j < 0 || wait_for<false>(smem_addr(&used[j % F::sf_stages]), (j / F::sf_stages) & 1);
  };

  // Copies of F::x_rows rows that a CTA with so many rows of the tile left makes. Rows past the last copy keep what the
  // stage held: their products are not stored.
  const auto x_copies = [](int rows) { return (max(0, min(rows, kTileM)) + F::x_rows - 1) / F::x_rows; };

  if (warp == 0) {
    // ---- copies of codes (the same in all lanes, one issues; as the products' warp)
    const int my_tiles = __shfl_sync(0xffffffffu, t0 < tiles ? (tiles - t0 + dt - 1) / dt : 0, 0);
    const uint32_t code0 = smem_addr(stages);
    int it = 0, st = 0;
    for (int n = 0; n < my_tiles && ok; ++n) {
      Tile tile = tile_of(t0 + n * dt);
      tile.expert = __shfl_sync(0xffffffffu, tile.expert, 0);
      tile.row0 = __shfl_sync(0xffffffffu, tile.row0, 0);
      tile.n = __shfl_sync(0xffffffffu, tile.n, 0);
      const int copies = __shfl_sync(0xffffffffu, x_copies(tile.rows), 0);
      const int rt = tile.n * (TN / 8) + rank * (F::b_rows / 8);
      int chunk = 0, x = 0;   // of the step in the weights
      for (int s = 0; s < steps; ++s, ++it) {
        if (!__all_sync(0xffffffffu, wait_used(it, kStages))) { ok = false; break; }
        uint32_t bar = smem_addr(&full[st]);
        if constexpr (PAIR) bar = leader_addr(bar);
        const uint32_t dst = code0 + (uint32_t)st * F::stage_bytes;
        if (elect_one()) {
          if (chunk < p.chunks_full) tma_load_5d<PAIR>(dst + F::a_bytes, &map_w, x, 0, rt, chunk, tile.expert, bar);
          else tma_load_5d<PAIR>(dst + F::a_bytes, &map_last, x, 0, rt, 0, tile.expert, bar);
          for (int i = 0; i < copies; ++i) {
            tma_load_2d<PAIR>(dst + (uint32_t)i * F::x_rows * 128, &map_x, s * 128, tile.row0 + i * F::x_rows, bar);
          }
        }
        __syncwarp();
        if (++st == kStages) st = 0;
        x += 128;
        if (x == F::steps_per_chunk * 128) {
          x = 0;
          ++chunk;
        }
      }
    }
    if (!ok) {   // leave no copy in flight
      if constexpr (PAIR) {
        const unsigned long long from = global_timer_ns();   // the copies report to the leader: give them their time
        while (global_timer_ns() - from < kDrainLimitNs) {}
      } else {
        for (int i = it > kStages ? it - kStages : 0; i < it; ++i) {
          if (!mbar_wait_bounded(smem_addr(&full[i % kStages]), (i / kStages) & 1, kDrainLimitNs) && lane == 0) {
            set_status(kStatusDrain);
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---- products. Everything here is the same in all lanes, and the compiler knows it (counts come by shuffle,
    // conditions by vote): addresses and descriptors stay in uniform registers, and one lane issues.
    if (rank == 0) {
      const int my_tiles = __shfl_sync(0xffffffffu, t0 < tiles ? (tiles - t0 + dt - 1) / dt : 0, 0);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t code0 = smem_addr(stages), scale0 = smem_addr(scales);
      int st = 0, ss = 0, sl = 0;   // places of the step's codes, its scales, and these in tensor memory
      uint32_t st_phase = 0;
      // a step's barrier is looked at before the step before it is issued: the look's latency is then hidden
      bool ready = false;
      for (int n = 0; n < my_tiles && ok; ++n) {
        const int acc = n & 1;
        if (!__all_sync(0xffffffffu, wait_for<PAIR>(smem_addr(&acc_empty[acc]), ((n >> 1) & 1) ^ 1))) { ok = false; break; }
        tc_after_sync();
        const uint32_t d = tm + (uint32_t)(acc * TN);
        int left = p.K;
        for (int s = 0; s < steps; ++s, left -= F::step_k) {
          if (!ready && !__all_sync(0xffffffffu, wait_for<false>(smem_addr(&full[st]), st_phase))) {
            ok = false;
            break;
          }
          tc_after_sync();
          const uint32_t a0 = code0 + (uint32_t)st * F::stage_bytes, b0 = a0 + F::a_bytes;
          const uint32_t sfa = scale0 + (uint32_t)ss * F::sf_bytes, sfb = sfa + F::sfa_bytes;
          const uint32_t sf = tm + F::sf_col0 + (uint32_t)sl * F::sf_cols;
          const uint32_t used_bar = smem_addr(&used[ss]);
          if (++st == kStages) { st = 0; st_phase ^= 1; }
          if (++ss == F::sf_stages) ss = 0;
          if (++sl == F::sf_slots) sl = 0;
          ready = __all_sync(0xffffffffu, peek(smem_addr(&full[st]), st_phase));
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < F::atoms; ++k) {
              const uint32_t col = sf + (uint32_t)k * F::atom_cols;
              scales_to_tmem<PAIR>(col, scale_desc(sfa + (uint32_t)k * 512));
#pragma unroll
              for (int i = 0; i < F::b_blocks; ++i) {
                scales_to_tmem<PAIR>(col + 4 + 4 * i, scale_desc(sfb + (uint32_t)(k * F::b_blocks + i) * 512));
              }
            }
            const auto mma = [&](int j, uint32_t accumulate) {
              constexpr int per_atom = 128 / F::mma_k;
              const uint32_t col = sf + (uint32_t)(j / per_atom) * F::atom_cols;
              mma_block_scaled<FMT, PAIR>(d, operand_desc(a0 + (uint32_t)j * 32), operand_desc(b0 + (uint32_t)j * 32),
                                          block_idesc<FMT, TN, PAIR>((uint32_t)(j % per_atom) * (F::mma_k / 32)), col,
                                          col + 4, accumulate);
            };
            mma(0, s > 0 ? 1u : 0u);
            if (left >= F::step_k) {
#pragma unroll
              for (int j = 1; j < F::step_k / F::mma_k; ++j) mma(j, 1u);
            } else {   // the ragged end of K
#pragma unroll
              for (int j = 1; j < F::step_k / F::mma_k; ++j) {
                if (j * F::mma_k < left) mma(j, 1u);
              }
            }
            mma_commit_to<PAIR>(used_bar);
            if (s == steps - 1) mma_commit_to<PAIR>(smem_addr(&acc_full[acc]));
          }
        }
      }
      if (elect_one()) mma_commit_to<PAIR>(smem_addr(&done));
      __syncwarp();
      if (!wait_for<false>(smem_addr(&done), 0)) ok = false;
    }
  } else if (warp == 2) {
    // ---- a step's one arrival, with the bytes to wait for, once its scales are there and their place in tensor memory
    // is free: the products then look at one barrier
    if (rank == 0) {
      int it = 0;
      for (int t = t0; t < tiles && ok; t += dt) {
        const int rows = tile_of(t).rows;
        const uint32_t bytes = (uint32_t)(x_copies(rows) + (PAIR ? x_copies(rows - kTileM) : 0)) * F::x_rows * 128 +
                               kCtas * F::b_bytes;
        for (int s = 0; s < steps; ++s, ++it) {
          if (!wait_for<PAIR>(smem_addr(&sf_full[it % F::sf_stages]), (it / F::sf_stages) & 1) ||
              !wait_used(it, F::sf_slots)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(smem_addr(&full[it % kStages]), bytes);
          __syncwarp();
        }
      }
    }
  } else if (warp == 3 || warp >= 12) {
    // ---- scales: every ninth step, loaded one turn ahead of its slot in the ring
    StepScales<FMT, TN> cur;
    int it = warp == 3 ? 0 : warp - 11;
    int t = t0, s = it;
    Tile tile{};
    while (t < tiles && s >= steps) { s -= steps; t += dt; }
    if (t < tiles) {
      tile = tile_of(t);
      cur.load(p, tile, s, lane);
    }
    while (t < tiles) {
      int t2 = t, s2 = s + kScaleWarps;
      while (t2 < tiles && s2 >= steps) { s2 -= steps; t2 += dt; }
      StepScales<FMT, TN> next = cur;
      if (t2 < tiles) {
        if (t2 != t) tile = tile_of(t2);
        next.load(p, tile, s2, lane);
      }
      const int ss = it % F::sf_stages;
      if (!wait_used(it, F::sf_stages)) { ok = false; break; }
      uint8_t* sfa = scales + (uint32_t)ss * F::sf_bytes;
      cur.store(sfa, sfa + F::sfa_bytes, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_cluster(leader_addr(smem_addr(&sf_full[ss])));
        else mbar_arrive_one(smem_addr(&sf_full[ss]));
      }
      cur = next;
      t = t2;
      s = s2;
      it += kScaleWarps;
    }
  } else {
    // ---- epilogue: warps 4..7 take the first, third, ... tile, warps 8..11 the others, each its own accumulator;
    // thread = row 32 (warp % 4) + lane of this CTA's part of the tile
    const int quad = warp % 4, group = warp / 4 - 1;
    uint8_t* warp_park = park + (uint32_t)(group * kTileM + quad * 32) * kParkPitch;
    uint8_t* my_park = warp_park + lane * kParkPitch;
    const int acc = group;
    uint32_t phase = 0;
    for (int t = t0 + group * dt; t < tiles; t += 2 * dt, phase ^= 1) {
      const Tile tile = tile_of(t);
      if (!wait_for<false>(smem_addr(&acc_full[acc]), phase)) { ok = false; break; }
      tc_after_sync();
      const int r = quad * 32 + lane;
      const bool live = r < tile.rows;
      const int64_t row = (int64_t)tile.row0 + r;
      const uint32_t d = tmem + (uint32_t)(acc * TN) + ((uint32_t)(quad * 32) << 16);
      const auto release = [&] {   // the accumulator has been read
        tc_before_sync();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR) mbar_arrive_cluster(leader_addr(smem_addr(&acc_empty[acc])));
          else mbar_arrive_one(smem_addr(&acc_empty[acc]));
        }
      };
      if constexpr (HFMT < 0) {
        // 32 columns of this thread's row, where one of them rounds to an infinite fp16
        const auto keep_wide = [&](const uint32_t (&v)[32], int n0) {
          bool over = false;
#pragma unroll
          for (uint32_t e : v) over |= fabsf(__uint_as_float(e)) >= 65520.0f;
          if (over && live && n0 < p.out_n) store_columns(p.wide + row * p.out_n + n0, v, p.out_n - n0, false);
        };
        if (p.out_type != QMV_F32 && p.out_n % 8 == 0) {
          // rows of whole 16 bytes: a warp parks its 32 rows and stores them row by row
          uint8_t* out = static_cast<uint8_t*>(p.y) + ((int64_t)tile.row0 + quad * 32) * p.out_n * 2;
          const int rows = min(32, tile.rows - quad * 32);
#pragma unroll 1
          for (int c = 0; c < TN; c += kParkCols) {
#pragma unroll
            for (int i = 0; i < kParkCols; i += 32) {
              uint32_t v[32];
              tmem_ld32(d + (uint32_t)(c + i), v);
              tmem_ld_wait(v);
              if (p.out_type == QMV_BF16) park_columns<__nv_bfloat16>(my_park + i * 2, v);
              else park_columns<__half>(my_park + i * 2, v);
              if (p.wide != nullptr) keep_wide(v, tile.n * TN + c + i);
            }
            if (c + kParkCols == TN) release();
            __syncwarp();
            const int n0 = tile.n * TN + c;
            const int vecs = min(kParkCols, p.out_n - n0) / 8;   // 16 bytes each
#pragma unroll 4
            for (int i = lane; i < 32 * (kParkCols / 8); i += 32) {
              const int r = i / (kParkCols / 8), v = i % (kParkCols / 8);
              if (r < rows && v < vecs) {
                *reinterpret_cast<uint4*>(out + ((int64_t)r * p.out_n + n0) * 2 + v * 16) =
                    *reinterpret_cast<const uint4*>(warp_park + r * kParkPitch + v * 16);
              }
            }
            __syncwarp();
          }
        } else {
          const bool vec = p.out_type == QMV_F32 && p.out_n % 4 == 0;
#pragma unroll 1
          for (int c = 0; c < TN; c += 32) {
            uint32_t v[32];
            tmem_ld32(d + (uint32_t)c, v);
            tmem_ld_wait(v);
            const int n0 = tile.n * TN + c;
            if (p.wide != nullptr) keep_wide(v, n0);
            if (live && n0 < p.out_n) {
              const int64_t at = row * p.out_n + n0;
              if (p.out_type == QMV_BF16) store_columns(static_cast<__nv_bfloat16*>(p.y) + at, v, p.out_n - n0, false);
              else if (p.out_type == QMV_F16) store_columns(static_cast<__half*>(p.y) + at, v, p.out_n - n0, false);
              else store_columns(static_cast<float*>(p.y) + at, v, p.out_n - n0, vec);
            }
          }
          release();
        }
      } else {
        const uint64_t h_bytes = mx_row_bytes(HFMT, p.out_n);
#pragma unroll 1
        for (int c = 0; c < TN; c += 64) {
          uint32_t v[2][32];
          tmem_ld32(d + (uint32_t)c, v[0]);
          tmem_ld32(d + (uint32_t)c + 32, v[1]);
          tmem_ld_wait(v[0]);
          tmem_ld_wait(v[1]);
          if (c + 64 == TN) release();
          const int n0 = (tile.n * TN + c) / 2;   // a group of 32 columns of h
          if (live && n0 < p.out_n) {
            float h[4][8];
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                // h column 8 i + k: row tile 2 i + k / 4, gate row k % 4, up row k % 4 + 4
                const int col = (2 * i + k / 4) * 8 + k % 4;
                h[i][k] = swiglu_range(__uint_as_float(v[col / 32][col % 32]),
                                       __uint_as_float(v[(col + 4) / 32][(col + 4) % 32]));
              }
              m = max(m, amax_bits8(h[i]));
            }
            const uint32_t e = group_e8m0<HFMT>(m);
            uint8_t* out = static_cast<uint8_t*>(p.y) + (uint64_t)row * h_bytes;
            constexpr int kWords = HFMT == MXFP4 ? 4 : 8;   // of the group's codes
            uint32_t w[kWords];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              mx_codes8<HFMT>(h[i], e, *reinterpret_cast<uint32_t(*)[kWords / 4]>(w + i * (kWords / 4)));
            }
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
              reinterpret_cast<uint4*>(out + n0 * fmt_bits(HFMT) / 8)[i] =
                  make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
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
    }
    // the leader's last arrival has reached this CTA before it may exit
    if (PAIR && ok && !wait_for<false>(smem_addr(&done), 0)) ok = false;
  }
  if (!ok && lane == 0) set_status(kStatusWaitTile);
  __syncwarp();
  pdl_launch_dependents();
  tc_before_sync();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();   // neither CTA's memory is in use by the other any more
  if (warp == 1) {
    tc_after_sync();
    if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(F::tmem_cols));
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(F::tmem_cols));
  }
}

QMV_DEFINE_STATUS_ACCESSOR(status_mx_gemm)

namespace {

template <int FMT, int HFMT, int TN, bool PAIR>
cudaError_t go(const MxGemmArgs& a) {
  using F = GemmFmt<FMT, TN, PAIR>;
  const Geometry g = make_geometry(FMT, a.N, a.K);
  const int lane_bytes = lane_code_bytes(FMT);
  GemmParams p = {};
  p.w = static_cast<const uint8_t*>(a.w);
  p.nrows = a.nrows;
  p.x_scales = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.xq) + mx_scale_offset(FMT, a.nrows, a.K));
  p.offsets = a.offsets;
  p.y = a.y;
  p.wide = a.wide;
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
  p.n_tiles = (g.row_tiles * kRows + TN - 1) / TN;

  const size_t smem = F::smem_bytes(a.n_experts);
  // The most that any call of this kernel asks for: the attribute is the
  // function's, and another host thread may be between it and its launch.
  // Before the tensor maps: on a host thread whose first CUDA call this is, it
  // makes the device's context current, which their encoding needs.
  g_launch_stage = "cudaFuncSetAttribute";
  cudaError_t e = cudaFuncSetAttribute(mx_gemm_kernel<FMT, HFMT, TN, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)F::smem_bytes(QMV_MAX_SORT_EXPERTS));
  if (e != cudaSuccess) return e;
  g_launch_stage = "cuTensorMapEncodeTiled";
  if (encode_fn() == nullptr) return cudaErrorNotSupported;
  CUtensorMap mx, mw, ml;
  {
    const cuuint64_t row = mx_row_bytes(FMT, a.K);
    const cuuint64_t dims[2] = {row, (cuuint64_t)a.nrows}, strides[1] = {row};
    const cuuint32_t box[2] = {128, F::x_rows};
    if (!encode(&mx, 2, a.xq, dims, strides, box)) return cudaErrorInvalidValue;
  }
  const cuuint32_t box[5] = {128, kRows, F::b_rows / kRows, 1, 1};
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

  // no more CTAs than tiles there can be: every expert has at most one partial row tile
  constexpr int ctas = PAIR ? 2 : 1;
  const int64_t row_tiles = a.nrows / (ctas * kTileM) + (a.nrows < a.n_experts ? a.nrows : (int64_t)a.n_experts);
  int64_t grid = row_tiles * p.n_tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // No more pairs than run at once: the device may not place one on every two SMs, and one that starts when another
  // ends would have its share of the tiles still before it.
  int most = device_sm_count();
  if constexpr (PAIR) {
    static PerDevice pairs;
    g_launch_stage = "cudaOccupancyMaxActiveClusters";
    e = pairs.get(&most, [&cfg](int* n) {
      cfg.gridDim = dim3((unsigned)(device_sm_count() / 2 * 2));
      return cudaOccupancyMaxActiveClusters(n, mx_gemm_kernel<FMT, HFMT, TN, PAIR>, &cfg);
    });
    if (e != cudaSuccess) return e;
    if (most < 1) return cudaErrorInvalidConfiguration;
  }
  if (grid > most) grid = most;
  g_launch_stage = "launch";
  cfg.gridDim = dim3((unsigned)(grid * ctas));
  cfg.numAttrs = a.stream != nullptr ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, mx_gemm_kernel<FMT, HFMT, TN, PAIR>, mx, mw, ml, p);
}

template <int FMT, int TN, bool PAIR>
cudaError_t by_h(const MxGemmArgs& a) {
  if (!a.glu) return go<FMT, -1, TN, PAIR>(a);
  return a.h_fmt == MXFP4 ? go<FMT, MXFP4, TN, PAIR>(a) : go<FMT, MXFP8, TN, PAIR>(a);
}

// The tile of a call: a pair's 256 x 192, or one CTA's 128 x 128 or 128 x 64.
// Every CTA (pair) takes ceil(tiles / CTAs) tiles one after another, whose time
// is their steps of 128 bytes; the row tiles of a grouped product are those of
// equally full experts, each with half a tile more. A step and a launch took,
// fitted to both formats on GB300: pair 0.33 us and 7 us, 128 x 128 0.36 and
// 4.5, 128 x 64 0.27 and 4.5. Measured (pair / 128 x 128 / 128 x 64, us):
//   17 x 7168 x 7168 MXFP4       16.8 / 13.2 / 11.6
//   200 x 7168 x 7168 MXFP4      17.0 / 14.0 / 19.2
//   300 x 7168 x 7168 MXFP4      17.3 / 21.8 / 26.0
//   1001 x 7168 x 2048 MXFP8     17.9 / 19.2 / 28.9
//   132 rows of 32 experts, gate/up 2880 MXFP4    68 / 54 / 71
//   16000 rows of them                           150 / 191 / 287
int pick_tile(const MxGemmArgs& a) {
  struct Shape {
    int m, n;
    double step_us, launch_us;
  };
  const Shape shapes[3] = {{2 * kTileM, 192, 0.33, 7.0}, {kTileM, 128, 0.36, 4.5}, {kTileM, 64, 0.27, 4.5}};
  const int steps = (int)((mx_row_bytes(a.fmt, a.K) + 127) / 128);
  int best = 0;
  double best_us = 0.0;
  for (int i = 0; i < 3; ++i) {
    const Shape& s = shapes[i];
    const double hit = a.nrows < a.n_experts ? (double)a.nrows : (double)a.n_experts;
    const double each = a.nrows / hit / s.m;
    const double row_tiles = a.n_experts == 1 ? ceil(each) : hit * (each > 0.5 ? each + 0.5 : 1.0);
    const int slots = device_sm_count() / (s.m / kTileM);
    const double us = s.launch_us + ceil(row_tiles * ((a.N + s.n - 1) / s.n) / slots) * steps * s.step_us;
    if (i == 0 || us < best_us) {
      best = i;
      best_us = us;
    }
  }
  return best;
}

template <int FMT>
cudaError_t by_tile(const MxGemmArgs& a) {
  switch (pick_tile(a)) {
    case 0: return by_h<FMT, 192, true>(a);
    case 1: return by_h<FMT, 128, false>(a);
    default: return by_h<FMT, 64, false>(a);
  }
}

}  // namespace

cudaError_t launch_mx_gemm(const MxGemmArgs& a) { return a.fmt == MXFP4 ? by_tile<MXFP4>(a) : by_tile<MXFP8>(a); }

}  // namespace qmv
