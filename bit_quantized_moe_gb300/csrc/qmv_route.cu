// qmv_route.cu -- tokens sorted by expert and back: the stable sort of routed
// slots, the copies between the tokens' and the experts' row order, the
// weighted sum, and the gradients of both.
#include <cooperative_groups.h>

#include "qmv_internal.h"
#include "qmv_rows.cuh"

namespace cg = cooperative_groups;

namespace qmv {

// ---------------------------------------------------------------------------
// Stable counting sort of slots by expert, in one launch of one cluster.
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
constexpr int kSortMaxCtas = 8;
// Slots that one CTA sorts alone; more CTAs share larger calls.
constexpr int64_t kSortSlotsPerCta = 4096;

__global__ void __launch_bounds__(kSortThreads) moe_sort_kernel(SortArgs a) {
  extern __shared__ uint32_t smem[];
  const int E1 = a.n_experts + 1;   // with the dropped slots
  uint32_t* hist = smem;                       // [kSortWarps][E1]
  uint32_t* total = hist + kSortWarps * E1;    // [E1] this CTA's count, read by the others
  uint32_t* start = total + E1;                // [E1] first row of this CTA's slots of each expert
  __shared__ uint32_t warp_sum[kSortWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;

  for (int i = threadIdx.x; i < kSortWarps * E1; i += kSortThreads) hist[i] = 0;
  __syncthreads();
  pdl_wait();

  // this warp's slots [s0, s1)
  const int64_t parts = (int64_t)ctas * kSortWarps;
  const int64_t per = (a.nslots + parts * 32 - 1) / (parts * 32) * 32;
  const int64_t s0 = min(((int64_t)rank * kSortWarps + warp) * per, a.nslots);
  const int64_t s1 = min(s0 + per, a.nslots);
  uint32_t* mine = hist + warp * E1;
  auto expert_of = [&](int64_t s) -> int {
    if (s >= s1) return -1;
    const int e = __ldg(a.ids + s);
    return e >= 0 && e < a.n_experts ? e : a.n_experts;
  };
  for (int64_t s = s0; s < s1; s += 32) {
    const int e = expert_of(s + lane);
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // counts of this CTA, and each warp's first place within them
  for (int e = threadIdx.x; e < E1; e += kSortThreads) {
    uint32_t n = 0;
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t c = hist[w * E1 + e];
      hist[w * E1 + e] = n;
      n += c;
    }
    total[e] = n;
  }
  cluster.sync();
  // rows before each expert: an exclusive sum over experts of the cluster's counts
  uint32_t carry = 0;
  for (int e0 = 0; e0 < E1; e0 += kSortThreads) {
    const int e = e0 + (int)threadIdx.x;
    uint32_t all = 0, before = 0;
    if (e < E1) {
      for (int c = 0; c < ctas; ++c) {
        const uint32_t n = cluster.map_shared_rank(total, c)[e];
        all += n;
        before += c < rank ? n : 0u;
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
  // ranks: the expert's first row, its slots in earlier CTAs and warps, and in this warp before this lane
  for (int64_t s = s0; s < s1; s += 32) {
    const int e = expert_of(s + lane);
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (e >= 0) {
      const uint32_t row = start[e] + mine[e] + __popc(same & ((1u << lane) - 1u));
      a.row_of_slot[s + lane] = e < a.n_experts ? (int32_t)row : ~(int32_t)row;
      a.slot_of_row[row] = (int32_t)(s + lane);
    }
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
  pdl_launch_dependents();
  cluster.sync();   // the others may still read this CTA's counts
}

cudaError_t launch_moe_sort(const SortArgs& a) {
  const int E1 = a.n_experts + 1;
  const size_t smem = (size_t)(kSortWarps + 2) * E1 * 4;
  cudaError_t e = cudaFuncSetAttribute(moe_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  int ctas = 1;
  while (ctas < kSortMaxCtas && ctas * kSortSlotsPerCta < a.nslots) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
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

// Slot values beyond the call's top_k are never used.
constexpr int kTopK = QMV_MAX_TOPK;

template <int VB>
__global__ void __launch_bounds__(512) dispatch_kernel(RouteArgs a, int64_t vecs, int64_t ld, int64_t grid_tokens) {
  using U = typename Bytes<VB>::type;
  pdl_wait();
  for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < a.ntok; t += grid_tokens) {
    int row[kTopK];
#pragma unroll
    for (int j = 0; j < kTopK; ++j) row[j] = j < a.top_k ? __ldg(a.row_of_slot + t * a.top_k + j) : 0;
    const U* in = static_cast<const U*>(a.tok) + t * ld;
    for (int64_t v = threadIdx.x; v < vecs; v += blockDim.x) {
      const U x = __ldg(in + v);
#pragma unroll
      for (int j = 0; j < kTopK; ++j) {
        if (j < a.top_k) {
          const int r = row[j];
          static_cast<U*>(a.out_rows)[(int64_t)(r >= 0 ? r : ~r) * vecs + v] = r >= 0 ? x : U{};
        }
      }
    }
  }
  pdl_launch_dependents();
}

template <typename T, int VB>
__global__ void __launch_bounds__(512) return_kernel(RouteArgs a, int64_t vecs, int64_t ld, int64_t grid_tokens) {
  using U = typename Bytes<VB>::type;
  constexpr int EV = VB / (int)sizeof(T);
  pdl_wait();
  for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < a.ntok; t += grid_tokens) {
    int row[kTopK];
    float w[kTopK];
#pragma unroll
    for (int j = 0; j < kTopK; ++j) {
      row[j] = j < a.top_k ? __ldg(a.row_of_slot + t * a.top_k + j) : -1;
      w[j] = j < a.top_k && a.weights != nullptr ? __ldg(a.weights + t * a.top_k + j) : 1.0f;
    }
    for (int64_t v = threadIdx.x; v < vecs; v += blockDim.x) {
      U x[kTopK];
#pragma unroll
      for (int j = 0; j < kTopK; ++j) {
        x[j] = row[j] >= 0 ? __ldg(static_cast<const U*>(a.rows) + (int64_t)row[j] * vecs + v) : U{};
      }
      float acc[EV];
#pragma unroll
      for (int i = 0; i < EV; ++i) acc[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < kTopK; ++j) {
        if (row[j] >= 0) {
          const T* e = reinterpret_cast<const T*>(&x[j]);
#pragma unroll
          for (int i = 0; i < EV; ++i) acc[i] = fmaf(w[j], to_f32(e[i]), acc[i]);
        }
      }
      U out;
      T* o = reinterpret_cast<T*>(&out);
#pragma unroll
      for (int i = 0; i < EV; ++i) o[i] = from_f32<T>(acc[i]);
      static_cast<U*>(a.out_tok)[t * ld + v] = out;
    }
  }
  pdl_launch_dependents();
}

// dys[row] = w dy[t] and dw = <ys[row], dy[t]>: one CTA per token (blockDim.y
// = 1), each thread's part of the top_k dot products reduced over the CTA in
// a fixed order. A dropped slot's row of dys and its weight's gradient are 0.
template <typename T, int VB>
__global__ void __launch_bounds__(512) return_grad_kernel(RouteArgs a, int64_t vecs, int64_t ld, int64_t grid_tokens) {
  using U = typename Bytes<VB>::type;
  constexpr int EV = VB / (int)sizeof(T);
  __shared__ float part[kTopK][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  pdl_wait();
  for (int64_t t = blockIdx.x; t < a.ntok; t += grid_tokens) {
    int row[kTopK];
    float w[kTopK], dot[kTopK];
#pragma unroll
    for (int j = 0; j < kTopK; ++j) {
      row[j] = j < a.top_k ? __ldg(a.row_of_slot + t * a.top_k + j) : 0;
      w[j] = j < a.top_k ? __ldg(a.weights + t * a.top_k + j) : 0.0f;
      dot[j] = 0.0f;
    }
    for (int64_t v = threadIdx.x; v < vecs; v += blockDim.x) {
      const U g = __ldg(static_cast<const U*>(a.tok) + t * ld + v);
      const T* ge = reinterpret_cast<const T*>(&g);
#pragma unroll
      for (int j = 0; j < kTopK; ++j) {
        if (j < a.top_k) {
          U out{};
          const int64_t at = (int64_t)(row[j] >= 0 ? row[j] : ~row[j]) * vecs + v;
          if (row[j] >= 0) {
            const U y = __ldg(static_cast<const U*>(a.rows) + at);
            const T* ye = reinterpret_cast<const T*>(&y);
            T* oe = reinterpret_cast<T*>(&out);
#pragma unroll
            for (int i = 0; i < EV; ++i) {
              const float d = to_f32(ge[i]);
              dot[j] = fmaf(to_f32(ye[i]), d, dot[j]);
              oe[i] = from_f32<T>(w[j] * d);
            }
          }
          static_cast<U*>(a.out_rows)[at] = out;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kTopK; ++j) {
      if (j < a.top_k) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
        if (lane == 0) part[j][warp] = dot[j];
      }
    }
    __syncthreads();
    if ((int)threadIdx.x < a.top_k) {
      const int r = __ldg(a.row_of_slot + t * a.top_k + threadIdx.x);
      float d = 0.0f;
      for (int i = 0; i < (int)blockDim.x / 32; ++i) d += part[threadIdx.x][i];
      a.dweights[t * a.top_k + threadIdx.x] = r >= 0 ? d : 0.0f;
    }
    __syncthreads();
  }
  pdl_launch_dependents();
}

namespace {

struct RowShape {
  int vb;            // bytes of an access
  int64_t vecs, ld;  // accesses of a row, and between rows of the token-major side
  dim3 grid, block;
  int64_t tokens;    // tokens of one pass of the grid
};

// Accesses as wide as the row's bytes and stride allow; a CTA's threads cover
// a row in as few, evenly filled rounds as 512 threads need.
RowShape row_shape(const RouteArgs& a, int64_t ld_elems, bool one_token) {
  const int size = a.type == QMV_F32 ? 4 : 2;
  const int64_t bytes = (int64_t)a.K * size, stride = ld_elems * size;
  RowShape s;
  s.vb = 16;
  while (s.vb > size && (bytes % s.vb != 0 || stride % s.vb != 0)) s.vb /= 2;
  s.vecs = bytes / s.vb;
  s.ld = stride / s.vb;
  const int64_t rounds = (s.vecs + 511) / 512;
  const int64_t x = ((s.vecs + rounds - 1) / rounds + 31) / 32 * 32;
  const int64_t y = one_token || x >= 256 ? 1 : 256 / x;
  s.block = dim3((unsigned)x, (unsigned)y);
  int64_t grid = (a.ntok + y - 1) / y;
  if (grid > (1 << 20)) grid = 1 << 20;
  s.grid = dim3((unsigned)grid);
  s.tokens = grid * y;
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

template <typename T, int VB>
struct Return {
  static cudaError_t go(const RouteArgs& a, const RowShape& s) {
    return launch_pdl(return_kernel<T, VB>, s.grid, s.block, 0, a.stream, a, s.vecs, s.ld, s.tokens);
  }
};
template <typename T, int VB>
struct ReturnGrad {
  static cudaError_t go(const RouteArgs& a, const RowShape& s) {
    return launch_pdl(return_grad_kernel<T, VB>, s.grid, s.block, 0, a.stream, a, s.vecs, s.ld, s.tokens);
  }
};

}  // namespace

cudaError_t launch_dispatch(const RouteArgs& a) {
  const RowShape s = row_shape(a, a.ld_tok, false);
  switch (s.vb) {
    case 16: return launch_pdl(dispatch_kernel<16>, s.grid, s.block, 0, a.stream, a, s.vecs, s.ld, s.tokens);
    case 8: return launch_pdl(dispatch_kernel<8>, s.grid, s.block, 0, a.stream, a, s.vecs, s.ld, s.tokens);
    case 4: return launch_pdl(dispatch_kernel<4>, s.grid, s.block, 0, a.stream, a, s.vecs, s.ld, s.tokens);
    default: return launch_pdl(dispatch_kernel<2>, s.grid, s.block, 0, a.stream, a, s.vecs, s.ld, s.tokens);
  }
}

cudaError_t launch_return(const RouteArgs& a) { return by_type<Return>(a, row_shape(a, a.ld_out, false)); }

cudaError_t launch_return_grad(const RouteArgs& a) { return by_type<ReturnGrad>(a, row_shape(a, a.ld_tok, true)); }

}  // namespace qmv
