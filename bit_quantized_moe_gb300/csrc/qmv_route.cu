// qmv_route.cu -- tokens sorted by expert and back: the stable sort of routed
// slots, the copies between the tokens' and the experts' row order, the
// weighted sum, and the gradients of both.
#include <type_traits>

#include <cooperative_groups.h>

#include "qmv_internal.h"
#include "qmv_rows.cuh"

namespace cg = cooperative_groups;

namespace qmv {

// ---------------------------------------------------------------------------
// Stable counting sort of slots by expert, in one launch of one cluster of up
// to 16 CTAs (65,536 slots of 256 experts: 11.7 us, 8 CTAs 17.2).
//
// Every CTA of the cluster takes a contiguous range of slots, every warp of it
// a contiguous part. A warp counts its slots per expert 32 at a time: lanes
// with the same expert find each other (__match_any_sync) and one adds their
// number to the warp's own counter, so that nothing depends on the order in
// which warps run. The counters are summed over warps, over CTAs (distributed
// shared memory) and over experts; a second walk gives every slot its rank.
// Slots whose id is outside [0, E) count as expert E, after all others.
// Bound by latency: the walks of 32 slots a warp and the few barriers.
// ---------------------------------------------------------------------------
constexpr int kSortWarps = 32;
constexpr int kSortThreads = kSortWarps * 32;
constexpr int kSortMaxCtas = 16;   // more than 8 where the device places such a cluster
// Slots that one CTA sorts alone; more CTAs share larger calls.
constexpr int64_t kSortSlotsPerCta = 1024;
constexpr int kSortKept = 8;
constexpr uint32_t kNoSlot = 0xffffu;

__global__ void __launch_bounds__(kSortThreads, 1) moe_sort_kernel(SortArgs a) {
  extern __shared__ uint32_t smem[];
  const int E1 = a.n_experts + 1;   // with the dropped slots
  uint32_t* hist = smem;                       // [kSortWarps][E1]
  uint32_t* total = hist + kSortWarps * E1;    // [E1] this CTA's count, read by the others
  uint32_t* start = total + E1;                // [E1] first row of this CTA's slots of each expert
  __shared__ uint32_t warp_sum[kSortWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;

  // this warp's slots [s0, s1), and the warps that have any
  const int nslots = (int)a.nslots;   // at most QMV_MAX_ROWS
  const int parts = ctas * kSortWarps;
  const int per = (nslots + parts * 32 - 1) / (parts * 32) * 32;
  const int used_warps = ctas > 1 ? kSortWarps : min((nslots + 31) / 32, kSortWarps);
  const int hist_rows = used_warps <= 4 ? used_warps : kSortWarps;
  for (int i = threadIdx.x; i < hist_rows * E1; i += kSortThreads) hist[i] = 0;
  __syncthreads();
  pdl_wait();

  const int s0 = min((rank * kSortWarps + warp) * per, nslots);
  const int s1 = min(s0 + per, nslots);
  uint32_t* mine = hist + warp * E1;
  auto expert_of = [&](int s) -> int {
    if (s >= s1) return -1;
    const int e = a.ids[s];
    return e >= 0 && e < a.n_experts ? e : a.n_experts;
  };
  // Counts 32 slots of a warp; the lane's own place among its warp's slots of its expert.
  auto count = [&](int e) -> uint32_t {
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const uint32_t before = e >= 0 ? mine[e] : 0u;
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] = before + __popc(same);
    __syncwarp();
    return before + __popc(same & ((1u << lane) - 1u));
  };
  // A warp with at most 32 kSortKept slots keeps their experts and places; longer walks are made again.
  uint32_t kept[kSortKept];   // expert (kNoSlot: none) | place << 16
  const bool keep = per <= 32 * kSortKept;
  if (keep) {
#pragma unroll
    for (int i = 0; i < kSortKept; ++i) kept[i] = (uint32_t)expert_of(s0 + 32 * i + lane) & kNoSlot;
#pragma unroll
    for (int i = 0; i < kSortKept; ++i) {
      if (s0 + 32 * i < s1) kept[i] |= count(kept[i] == kNoSlot ? -1 : (int)kept[i]) << 16;
    }
  } else {
    for (int s = s0; s < s1; s += 32) count(expert_of(s + lane));
  }
  __syncthreads();
  // counts of this CTA, and each warp's first place within them: one warp an expert, lane = warp
  if (used_warps <= 4) {   // few: a thread an expert
    for (int e = threadIdx.x; e < E1; e += kSortThreads) {
      uint32_t n = 0;
      for (int w = 0; w < used_warps; ++w) {
        const uint32_t c = hist[w * E1 + e];
        hist[w * E1 + e] = n;
        n += c;
      }
      total[e] = n;
    }
  } else for (int e = warp; e < E1; e += kSortWarps) {
    const uint32_t c = hist[lane * E1 + e];
    uint32_t inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
      inc += lane >= o ? v : 0u;
    }
    hist[lane * E1 + e] = inc - c;
    if (lane == 31) total[e] = inc;
  }
  cluster.sync();
  // rows before each expert: an exclusive sum over experts of the cluster's counts
  uint32_t carry = 0;
  for (int e0 = 0; e0 < E1; e0 += kSortThreads) {
    const int e = e0 + (int)threadIdx.x;
    uint32_t all = 0, before = 0;
    if (ctas == 1) {
      all = e < E1 ? total[e] : 0u;
    } else if (e < E1) {
      for (int c0 = 0; c0 < ctas; c0 += 8) {
        uint32_t n[8];   // asked for together
#pragma unroll
        for (int c = 0; c < 8; ++c) n[c] = c0 + c < ctas ? cluster.map_shared_rank(total, c0 + c)[e] : 0u;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          all += n[c];
          before += c0 + c < rank ? n[c] : 0u;
        }
      }
    }
    uint32_t inc = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
      inc += lane >= o ? v : 0u;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    uint32_t ws = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, ws, o);
      ws += lane >= o ? v : 0u;
    }
    const uint32_t below = carry + (warp > 0 ? __shfl_sync(0xffffffffu, ws, warp - 1) : 0u);
    if (e < E1) {
      const uint32_t first = below + inc - all;
      start[e] = first + before;
      if (rank == 0) a.offsets[e] = (int32_t)first;   // offsets[E] = rows of every valid slot
    }
    carry += __shfl_sync(0xffffffffu, ws, 31);
    __syncthreads();
  }
  // a slot's row: its expert's first row, then the expert's slots in earlier CTAs, in earlier warps, in this warp
  auto place = [&](int s, int e, uint32_t row) {
    if (e < 0) return;
    a.row_of_slot[s] = e < a.n_experts ? (int32_t)row : ~(int32_t)row;
    a.slot_of_row[row] = s;
  };
  if (keep) {
#pragma unroll
    for (int i = 0; i < kSortKept; ++i) {
      const uint32_t e = kept[i] & kNoSlot;
      if (e != kNoSlot) place(s0 + 32 * i + lane, (int)e, start[e] + mine[e] + (kept[i] >> 16));
    }
  } else {
    // `mine` goes on from the warp's first place
    for (int s = s0; s < s1; s += 32) {
      const int e = expert_of(s + lane);
      const uint32_t at = count(e);
      place(s + lane, e, e >= 0 ? start[e] + at : 0u);
    }
  }
  pdl_launch_dependents();
  cluster.sync();   // the others may still read this CTA's counts
}

constexpr int kSortSmemMax = (kSortWarps + 2) * (QMV_MAX_SORT_EXPERTS + 1) * 4;

cudaError_t launch_moe_sort(const SortArgs& a) {
  const int E1 = a.n_experts + 1;
  const size_t smem = (size_t)(kSortWarps + 2) * E1 * 4;
  cudaError_t e = cudaFuncSetAttribute(moe_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmemMax);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(moe_sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  int ctas = 1;
  while (ctas < kSortMaxCtas && ctas * kSortSlotsPerCta < a.nslots) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  if (ctas > 8) {
    static PerDevice wide;   // clusters of 16 with the most shared memory that the device places
    int fit = 0;
    e = wide.get(&fit, [&](int* n) {
      attr[0].val.clusterDim.x = (unsigned)kSortMaxCtas;
      cfg.gridDim = dim3((unsigned)kSortMaxCtas);
      cfg.dynamicSmemBytes = kSortSmemMax;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(n, moe_sort_kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        *n = 0;
      }
      cfg.dynamicSmemBytes = smem;
      return cudaSuccess;
    });
    if (e != cudaSuccess) return e;
    if (fit < 1) ctas = 8;
  }
  cfg.gridDim = dim3((unsigned)ctas);
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.stream != nullptr ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, moe_sort_kernel, a);
}

// ---------------------------------------------------------------------------
// Row movers. A token's columns are spread over blockDim.x threads in accesses
// of VB bytes (the widest that every row's start and width allow, so that odd
// widths and strides are taken as they are); blockDim.y tokens share a CTA.
// Every row is read once and written once; sums are fp32 in slot order, the
// same order every run, rounded once where they are stored. Bound by memory.
// ---------------------------------------------------------------------------
template <int VB>
struct Bytes;
template <>
struct Bytes<16> { using type = uint4; };
template <>
struct Bytes<8> { using type = uint2; };
template <>
struct Bytes<4> { using type = uint32_t; };
template <>
struct Bytes<2> { using type = uint16_t; };

constexpr int kTopK = QMV_MAX_TOPK;

// The row that row_of_slot names (r, or ~r of a dropped slot) if the call has
// it; -1 otherwise: such an entry is neither read from nor written to.
__device__ __forceinline__ int row_named(int r, int nslots) {
  const int row = r >= 0 ? r : ~r;
  return row < nslots ? row : -1;
}

// Slots of a token whose rows are asked for together.
constexpr int kSlotGroup = 4;
static_assert(kTopK % kSlotGroup == 0, "part[] of the gradient");

constexpr int kMoveThreads = 384;   // most threads of a mover's CTA

// Arguments of the movers beside RouteArgs: accesses of a row, and between
// rows of the token-major side; tokens of one pass of the grid; the call's rows
// (as a parameter: computed in the kernel they cost return_kernel registers,
// of which its 16-byte forms have 8 to 16 bytes too few as it is: 8191 x 4 x
// 2880 46.5 us instead of 40.0).
struct MoveShape {
  int vecs;
  int tokens;
  int nslots;
  int64_t ld;
};

template <int VB>
__global__ void __launch_bounds__(kMoveThreads, 4) dispatch_kernel(RouteArgs a, MoveShape m) {
  using U = typename Bytes<VB>::type;
  const int ntok = (int)a.ntok, top_k = a.top_k;
  pdl_wait();
  for (int t = blockIdx.x * blockDim.y + threadIdx.y; t < ntok; t += m.tokens) {
    const int32_t* rows = a.row_of_slot + (int64_t)t * top_k;
    const U* in = static_cast<const U*>(a.tok) + t * m.ld;
    for (int v = blockIdx.y * blockDim.x + threadIdx.x; v < m.vecs; v += gridDim.y * blockDim.x) {
      const U x = in[v];
      for (int j0 = 0; j0 < top_k; j0 += kSlotGroup) {
        int row[kSlotGroup];
#pragma unroll
        for (int j = 0; j < kSlotGroup; ++j) row[j] = j0 + j < top_k ? rows[j0 + j] : 0;
#pragma unroll
        for (int j = 0; j < kSlotGroup; ++j) {
          const int at = row_named(row[j], m.nslots);
          if (j0 + j < top_k && at >= 0) {
            static_cast<U*>(a.out_rows)[(int64_t)at * m.vecs + v] = row[j] >= 0 ? x : U{};
          }
        }
      }
    }
  }
  pdl_launch_dependents();
}

// EV elements of a row, read in accesses of up to 16 bytes.
template <typename R, int EV>
struct RowVec {
  static constexpr int bytes = EV * (int)sizeof(R), access = bytes < 16 ? bytes : 16, count = bytes / access;
  typename Bytes<access>::type u[count];
  __device__ __forceinline__ void load(const void* rows, int64_t at) {
    const auto* p = static_cast<const typename Bytes<access>::type*>(rows) + at * count;
#pragma unroll
    for (int i = 0; i < count; ++i) u[i] = __ldcg(p + i);
  }
  __device__ __forceinline__ float operator[](int i) const { return to_f32(reinterpret_cast<const R*>(u)[i]); }
};

// R: the element type of the experts' rows. SPLIT: blockIdx.y takes a part of
// the columns. Without it the kernel fits 40 registers and four CTAs an SM
// (8191 tokens x 4 slots of 2880: 41 us against 47). WIDE: fp16 rows whose
// infinite elements are read as a.wide has them.
template <typename R, typename T, int VB, bool SPLIT, bool WIDE>
__global__ void __launch_bounds__(kMoveThreads, SPLIT || WIDE || sizeof(R) > sizeof(T) ? 3 : 4)
return_kernel(RouteArgs a, MoveShape m) {
  using U = typename Bytes<VB>::type;
  constexpr int EV = VB / (int)sizeof(T);
  const int ntok = (int)a.ntok, top_k = a.top_k;
  pdl_wait();
  for (int t = blockIdx.x * blockDim.y + threadIdx.y; t < ntok; t += m.tokens) {
    const int32_t* rows = a.row_of_slot + (int64_t)t * top_k;
    for (int v = (SPLIT ? blockIdx.y * blockDim.x : 0u) + threadIdx.x; v < m.vecs;
         v += (SPLIT ? gridDim.y : 1u) * blockDim.x) {
      float acc[EV];
#pragma unroll
      for (int i = 0; i < EV; ++i) acc[i] = 0.0f;
      for (int j0 = 0; j0 < top_k; j0 += kSlotGroup) {
        RowVec<R, EV> x[kSlotGroup];
        uint32_t live = 0;
#pragma unroll
        for (int j = 0; j < kSlotGroup; ++j) {
          const int r = j0 + j < top_k ? rows[j0 + j] : -1;
          if ((unsigned)r < (unsigned)m.nslots) {   // a row of this call, not dropped
            x[j].load(a.rows, (int64_t)r * m.vecs + v);
            live |= 1u << j;
          }
        }
#pragma unroll
        for (int j = 0; j < kSlotGroup; ++j) {
          if (live >> j & 1u) {
            const float w = a.weights != nullptr ? a.weights[(int64_t)t * top_k + j0 + j] : 1.0f;
#pragma unroll
            for (int i = 0; i < EV; ++i) {
              float e = x[j][i];
              if constexpr (WIDE) {
                if (isinf(e)) e = a.wide[((int64_t)rows[j0 + j] * m.vecs + v) * EV + i];
              }
              acc[i] = fmaf(w, e, acc[i]);
            }
          }
        }
      }
      U out;
      T* o = reinterpret_cast<T*>(&out);
#pragma unroll
      for (int i = 0; i < EV; ++i) o[i] = from_f32<T>(acc[i]);
      static_cast<U*>(a.out_tok)[t * m.ld + v] = out;
    }
  }
  pdl_launch_dependents();
}

// dys[row] = w dy[t] and dw = <ys[row], dy[t]>: one CTA per token (or, of few
// tokens, per token and group of slots), its slots in groups, each thread's
// part of a group's dot products reduced over the CTA in a fixed order. A dropped slot's row of dys and its weight's gradient are 0.
template <typename T, int VB>
__global__ void __launch_bounds__(kMoveThreads, 3) return_grad_kernel(RouteArgs a, MoveShape m) {
  using U = typename Bytes<VB>::type;
  constexpr int EV = VB / (int)sizeof(T);
  __shared__ float part[kTopK][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int ntok = (int)a.ntok, top_k = a.top_k;
  pdl_wait();
  for (int t = blockIdx.x; t < ntok; t += m.tokens) {
    const int32_t* rows = a.row_of_slot + (int64_t)t * top_k;
    const float* weights = a.weights + (int64_t)t * top_k;
    const U* grad = static_cast<const U*>(a.tok) + t * m.ld;
    const int first = blockIdx.y * kSlotGroup, step = gridDim.y * kSlotGroup;
    for (int j0 = first; j0 < top_k; j0 += step) {
      float dot[kSlotGroup];
#pragma unroll
      for (int j = 0; j < kSlotGroup; ++j) dot[j] = 0.0f;
      for (int v = threadIdx.x; v < m.vecs; v += blockDim.x) {
        const U g = grad[v];
        U y[kSlotGroup];
        int row[kSlotGroup];
        float w[kSlotGroup];
#pragma unroll
        for (int j = 0; j < kSlotGroup; ++j) {
          row[j] = j0 + j < top_k ? rows[j0 + j] : -1;
          w[j] = j0 + j < top_k ? weights[j0 + j] : 0.0f;
          if (row[j] >= m.nslots) row[j] = ~m.nslots;   // no row of this call
          if (row[j] >= 0) y[j] = static_cast<const U*>(a.rows)[(int64_t)row[j] * m.vecs + v];
        }
        const T* ge = reinterpret_cast<const T*>(&g);
#pragma unroll
        for (int j = 0; j < kSlotGroup; ++j) {
          const int at = row_named(row[j], m.nslots);
          if (j0 + j < top_k && at >= 0) {
            U out{};
            if (row[j] >= 0) {
              const T* ye = reinterpret_cast<const T*>(&y[j]);
              T* oe = reinterpret_cast<T*>(&out);
#pragma unroll
              for (int i = 0; i < EV; ++i) {
                const float d = to_f32(ge[i]);
                dot[j] = fmaf(to_f32(ye[i]), d, dot[j]);
                oe[i] = from_f32<T>(w[j] * d);
              }
            }
            static_cast<U*>(a.out_rows)[(int64_t)at * m.vecs + v] = out;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kSlotGroup; ++j) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
        if (lane == 0) part[j0 + j][warp] = dot[j];
      }
    }
    __syncthreads();
    if ((int)threadIdx.x < top_k && (int)threadIdx.x / kSlotGroup % gridDim.y == blockIdx.y) {
      float d = 0.0f;
      for (int i = 0; i < (int)blockDim.x / 32; ++i) d += part[threadIdx.x][i];
      a.dweights[(int64_t)t * top_k + threadIdx.x] = (unsigned)rows[threadIdx.x] < (unsigned)m.nslots ? d : 0.0f;
    }
    __syncthreads();
  }
  pdl_launch_dependents();
}

namespace {

struct RowShape {
  int vb;            // bytes of an access
  MoveShape move;
  dim3 grid, block;
};

// Accesses as wide as the row's bytes and stride allow; a CTA's threads cover
// a row in as few, evenly filled rounds as kMoveThreads threads need. Where
// that makes fewer CTAs than SMs, a row's columns (or, for one_token, its
// slots) are spread over several (16 tokens x 8 slots of 7168, one CTA a token
// against several: dispatch 3.4 and 1.7 us, return 5.5 and 2.3, its gradients
// 6.2 and 4.0).
RowShape row_shape(const RouteArgs& a, int64_t ld_elems, bool one_token) {
  const int size = a.type == QMV_F32 ? 4 : 2;
  const int64_t bytes = (int64_t)a.K * size, stride = ld_elems * size;
  RowShape s;
  s.vb = 16;
  while (s.vb > size && (bytes % s.vb != 0 || stride % s.vb != 0)) s.vb /= 2;
  const int64_t vecs = bytes / s.vb;   // at most 2^20: QMV_MAX_N elements
  const int64_t rounds = (vecs + kMoveThreads - 1) / kMoveThreads;
  int64_t x = ((vecs + rounds - 1) / rounds + 31) / 32 * 32;
  const int64_t y = one_token || x >= 256 ? 1 : 256 / x;
  int64_t grid = (a.ntok + y - 1) / y, split = 1;
  if (grid < device_sm_count()) {
    if (one_token) {
      split = (a.top_k + kSlotGroup - 1) / kSlotGroup;
    } else if (y == 1) {
      x = 128;
      split = (vecs + x - 1) / x;
    }
  }
  if (grid > (1 << 20)) grid = 1 << 20;
  s.block = dim3((unsigned)x, (unsigned)y);
  s.grid = dim3((unsigned)grid, (unsigned)split);
  s.move = {(int)vecs, (int)(grid * y), (int)(a.ntok * a.top_k), stride / s.vb};
  return s;
}

template <template <typename, int> class K, typename T>
cudaError_t by_bytes(const RouteArgs& a, const RowShape& s) {
  switch (s.vb) {
    case 16: return K<T, 16>::go(a, s);
    case 8: return K<T, 8>::go(a, s);
    case 4: return K<T, 4>::go(a, s);
    default:
      if constexpr (sizeof(T) == 2) return K<T, 2>::go(a, s);
      return cudaErrorInvalidValue;
  }
}

template <template <typename, int> class K>
cudaError_t by_type(const RouteArgs& a, const RowShape& s) {
  switch (a.type) {
    case QMV_BF16: return by_bytes<K, __nv_bfloat16>(a, s);
    case QMV_F16: return by_bytes<K, __half>(a, s);
    default: return by_bytes<K, float>(a, s);
  }
}

template <typename R, typename T, int VB>
cudaError_t go_return(const RouteArgs& a, const RowShape& s) {
  return s.grid.y > 1 ? launch_pdl(return_kernel<R, T, VB, true, false>, s.grid, s.block, 0, a.stream, a, s.move)
                      : launch_pdl(return_kernel<R, T, VB, false, false>, s.grid, s.block, 0, a.stream, a, s.move);
}
template <typename T, int VB>
struct Return {
  static cudaError_t go(const RouteArgs& a, const RowShape& s) {
    if constexpr (std::is_same_v<T, __half>) {
      if (a.wide != nullptr) {
        return s.grid.y > 1 ? launch_pdl(return_kernel<T, T, VB, true, true>, s.grid, s.block, 0, a.stream, a, s.move)
                            : launch_pdl(return_kernel<T, T, VB, false, true>, s.grid, s.block, 0, a.stream, a, s.move);
      }
    }
    return a.rows_f32 ? go_return<float, T, VB>(a, s) : go_return<T, T, VB>(a, s);
  }
};
template <typename T, int VB>
struct ReturnGrad {
  static cudaError_t go(const RouteArgs& a, const RowShape& s) {
    return launch_pdl(return_grad_kernel<T, VB>, s.grid, s.block, 0, a.stream, a, s.move);
  }
};

}  // namespace

cudaError_t launch_dispatch(const RouteArgs& a) {
  const RowShape s = row_shape(a, a.ld_tok, false);
  switch (s.vb) {
    case 16: return launch_pdl(dispatch_kernel<16>, s.grid, s.block, 0, a.stream, a, s.move);
    case 8: return launch_pdl(dispatch_kernel<8>, s.grid, s.block, 0, a.stream, a, s.move);
    case 4: return launch_pdl(dispatch_kernel<4>, s.grid, s.block, 0, a.stream, a, s.move);
    default: return launch_pdl(dispatch_kernel<2>, s.grid, s.block, 0, a.stream, a, s.move);
  }
}

cudaError_t launch_return(const RouteArgs& a) { return by_type<Return>(a, row_shape(a, a.ld_out, false)); }

cudaError_t launch_return_grad(const RouteArgs& a) { return by_type<ReturnGrad>(a, row_shape(a, a.ld_tok, true)); }

}  // namespace qmv
