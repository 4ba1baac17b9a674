// qmv_router.cu -- the router of a MoE layer: the top_k experts of each token
// and their weights, the balance loss with the slots of each expert, and the
// gradient of both.
#include <type_traits>
#include <utility>

#include <cooperative_groups.h>

#include "qmv_internal.h"
#include "qmv_rows.cuh"

namespace cg = cooperative_groups;

namespace qmv {

// ---------------------------------------------------------------------------
// A warp takes a token; lane i holds the logits of experts i, i + 32, ... (V of
// them), so that a warp reads consecutive ones. Scores are not stored: each
// kernel takes them from the logits again, which costs 2 or 4 bytes an expert
// where stored ones would cost 4 more.
//
// softmax: exp(l - max) over its sum. sigmoid: with u = e^min(l,0) / (1 + e^-|l|)
// = 1 / (1 + e^-l); quotients of sigmoids are taken of
// t = e^(min(l,0) - top) / (1 + e^-|l|), top the largest min(l,0) of the row, which
// is in range where u is not. Exponentials are __expf, documented as off by at
// most 2 + |1.173 x| units in the last place: (4 + 2.4 |x|) * 2^-24 of the value,
// where the rounding of x = l - max itself costs |x| * 2^-24. Only scores far below
// their row's largest lose by it (28 * 2^-24 at e^-10). Sums are fp32, and a row
// divides by its sum once, by multiplying with the reciprocal. (With expf and a
// division an expert the gradient of 16,384 x 256 took 16.7 us, so 14.9.)
//
// A logit of -infinity is an expert that is not there. A row with a NaN
// (softmax: or +infinity) has no scores: its weights and its gradient are NaN.
// ---------------------------------------------------------------------------
constexpr int kRouterThreads = 256;
constexpr int kRouterWarps = kRouterThreads / 32;

__device__ __forceinline__ float exp_of(float x) { return __expf(x); }
__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xff800000u); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <typename T, int V>
__device__ __forceinline__ void load_logits(const T* row, int n_experts, int lane, float (&l)[V]) {
  T raw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    raw[i] = e < n_experts ? row[e] : from_f32<T>(neg_inf());
  }
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] = to_f32(raw[i]);
}

// 1 / (1 + e^-l)
__device__ __forceinline__ float sigmoid(float l) { return exp_of(fminf(l, 0.0f)) / (1.0f + exp_of(-fabsf(l))); }
__device__ __forceinline__ float sigmoid_scaled(float l, float top) {
  return l == neg_inf() ? 0.0f : exp_of(fminf(l, 0.0f) - top) / (1.0f + exp_of(-fabsf(l)));
}

// Whether the row has no scores: a NaN, or for softmax +infinity.
template <bool SIGMOID, int V>
__device__ __forceinline__ bool row_is_bad(const float (&l)[V]) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) bad |= l[i] != l[i] || (!SIGMOID && l[i] == -neg_inf());
  return __any_sync(0xffffffffu, bad);
}

// The row's scores as shares of their sum, and whether it has any: false for a
// row of -infinities, whose shares are 0.
template <bool SIGMOID, int V>
__device__ __forceinline__ bool row_shares(const float (&l)[V], float (&p)[V]) {
  float top = neg_inf();
#pragma unroll
  for (int i = 0; i < V; ++i) top = fmaxf(top, SIGMOID ? fminf(l[i], 0.0f) : l[i]);
  top = warp_max(top);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (SIGMOID) p[i] = sigmoid_scaled(l[i], top);
    else p[i] = l[i] == neg_inf() ? 0.0f : exp_of(l[i] - top);
    sum += p[i];
  }
  sum = warp_sum(sum);
  if (sum == 0.0f) return false;
  const float inverse = 1.0f / sum;
#pragma unroll
  for (int i = 0; i < V; ++i) p[i] *= inverse;
  return true;
}

// Keys that compare as the logits do: +0 as -0, -infinity 0.
__device__ __forceinline__ uint32_t order_key(float l) {
  const uint32_t b = __float_as_uint(l == 0.0f ? 0.0f : l);
  return l == neg_inf() ? 0u : b ^ ((b >> 31) != 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return k == 0u ? neg_inf() : __uint_as_float(k ^ ((k >> 31) != 0 ? 0x80000000u : 0xffffffffu));
}

// The top_k largest logits one by one: the largest key of each lane, of the
// warp (one reduction), and the lowest expert that has it (another).
template <typename T, bool SIGMOID, int V>
__global__ void __launch_bounds__(kRouterThreads) router_kernel(RouterArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kRouterWarps + threadIdx.x / 32;
  pdl_wait();
  if (t < a.ntok) {
    const bool live = a.live == nullptr || a.live[t] != 0;
    float l[V];
    load_logits<T, V>(static_cast<const T*>(a.logits) + t * a.ldl, a.n_experts, lane, l);
    const bool bad = row_is_bad<SIGMOID, V>(l);
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = order_key(l[i]);
    int id = -1;            // lane j < top_k: the j-th expert
    float chosen = neg_inf();   // and its logit
    float first = neg_inf();    // the largest
    for (int j = 0; j < a.top_k; ++j) {
      uint32_t best = key[0];
#pragma unroll
      for (int i = 1; i < V; ++i) best = max(best, key[i]);
      const uint32_t m = __reduce_max_sync(0xffffffffu, best);
      if (m == 0u) break;   // no logit above -infinity is left
      uint32_t at = 0xffffffffu;
#pragma unroll
      for (int i = V - 1; i >= 0; --i) at = key[i] == m ? (uint32_t)(lane + 32 * i) : at;
      const int e = (int)__reduce_min_sync(0xffffffffu, at);
      if (j == 0) first = key_value(m);
      if (lane == j) {
        id = e;
        chosen = key_value(m);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = lane + 32 * i == e ? 0u : key[i];
    }
    float w;
    if (a.renorm) {
      const float v = id < 0 ? 0.0f : (SIGMOID ? sigmoid_scaled(chosen, fminf(first, 0.0f)) : exp_of(chosen - first));
      w = v / warp_sum(v);
    } else if constexpr (SIGMOID) {
      w = sigmoid(chosen);
    } else {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += l[i] == neg_inf() ? 0.0f : exp_of(l[i] - first);
      w = exp_of(chosen - first) / warp_sum(sum);
    }
    w = id < 0 ? 0.0f : w * a.scale;
    if (bad) {
      id = lane;
      w = __uint_as_float(0x7fc00000u);
    }
    if (lane < a.top_k) {
      a.ids[t * a.top_k + lane] = live ? id : -1;
      a.weights[t * a.top_k + lane] = live ? w : 0.0f;
    }
  }
  pdl_launch_dependents();
}

// ---------------------------------------------------------------------------
// Balance loss: T live tokens, n_e their slots on expert e,
//   L = E sum_e f_e P_e,   f_e = n_e / (top_k T),   P_e = 1/T sum_t p_te.
//
// A warp adds up its tokens' shares in registers, a CTA its warps' and writes a
// row of partial sums; the second launch, 128 experts a CTA, adds the rows in
// order, and its CTAs (a cluster) their parts of the loss. A batch that one CTA
// takes needs no second launch. Slots and tokens are counted in integers, so
// that every sum is the same every run.
// ---------------------------------------------------------------------------
// Warps of a CTA: as many as have the registers for V sums, shares and logits a lane.
template <int V>
constexpr int kBalanceWarps = V <= 8 ? 32 : 16;
constexpr int kBalanceAlone = 64;      // tokens that one CTA takes alone
constexpr int kBalanceParts = 152;     // CTAs of the first launch at most: one an SM
constexpr int kFinishCols = 128, kFinishGroups = 8;

// Sum over the CTA's threads, in all of them; scratch: one number a warp.
__device__ __forceinline__ float block_sum(float v, float* scratch) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x / 32] = v;
  __syncthreads();
  const int warps = (int)blockDim.x / 32, lane = threadIdx.x & 31;
  return warp_sum(lane < warps ? scratch[lane] : 0.0f);
}

template <typename T, bool SIGMOID, int V>
__global__ void __launch_bounds__(kBalanceWarps<V> * 32) balance_kernel(BalanceArgs a) {
  constexpr int kWarps = kBalanceWarps<V>, kThreads = kWarps * 32;
  extern __shared__ float sums[];   // [warps][E], then counts [E + 1]
  __shared__ float scratch[kWarps];
  const int E = a.n_experts;
  int* counts = reinterpret_cast<int*>(sums + kWarps * E);
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  for (int i = threadIdx.x; i <= E; i += kThreads) counts[i] = 0;
  __syncthreads();
  pdl_wait();
  float mine[V];
#pragma unroll
  for (int i = 0; i < V; ++i) mine[i] = 0.0f;
  int live_tokens = 0;
  const int64_t stride = (int64_t)gridDim.x * kWarps;
  // the next token's logits are on their way while this one's are added
  int64_t t = (int64_t)warp * gridDim.x + blockIdx.x;
  float next[V];
  const T* logits = static_cast<const T*>(a.logits);
  if (t < a.ntok) load_logits<T, V>(logits + t * a.ldl, E, lane, next);
  for (; t < a.ntok; t += stride) {
    float l[V], p[V];
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = next[i];
    const bool live = a.live == nullptr || a.live[t] != 0;
    const int id = lane < a.top_k ? a.ids[t * a.top_k + lane] : -1;
    if (t + stride < a.ntok) load_logits<T, V>(logits + (t + stride) * a.ldl, E, lane, next);
    if (!live || !row_shares<SIGMOID, V>(l, p)) continue;
#pragma unroll
    for (int i = 0; i < V; ++i) mine[i] += p[i];
    ++live_tokens;
    if (id >= 0 && id < E) atomicAdd(&counts[id], 1);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (lane + 32 * i < E) sums[warp * E + lane + 32 * i] = mine[i];
  }
  if (lane == 0 && live_tokens > 0) atomicAdd(&counts[E], live_tokens);
  __syncthreads();
  const bool alone = gridDim.x == 1;
  const int tokens = counts[E];
  float part_loss = 0.0f;
  for (int e = threadIdx.x; e < E; e += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += sums[w * E + e];
    if (alone) {
      const float mean = tokens > 0 ? v / (float)tokens : 0.0f;
      a.means[e] = mean;
      a.counts[e] = counts[e];
      if (tokens > 0) part_loss += (float)counts[e] / ((float)a.top_k * (float)tokens) * mean;
    } else {
      a.part_sums[(int64_t)blockIdx.x * E + e] = v;
      a.part_counts[(int64_t)blockIdx.x * (E + 1) + e] = counts[e];
    }
  }
  if (alone) {
    const float loss = block_sum(part_loss, scratch);
    if (threadIdx.x == 0) {
      a.loss[0] = (float)E * loss;
      a.counts[E] = tokens;
    }
  } else if (threadIdx.x == 0) {
    a.part_counts[(int64_t)blockIdx.x * (E + 1) + E] = tokens;
  }
  pdl_launch_dependents();
}

__global__ void __launch_bounds__(kFinishCols * kFinishGroups) balance_finish_kernel(BalanceArgs a) {
  __shared__ float group_sums[kFinishGroups][kFinishCols];
  __shared__ int group_counts[kFinishGroups][kFinishCols];
  __shared__ float scratch[32], loss_parts[8];
  __shared__ int live_tokens;
  cg::cluster_group cluster = cg::this_cluster();
  // A CTA may write to another's shared memory only once that one runs: each says so here and waits for the others behind
  // its sums, so that the barrier is out of the loads' way.
  auto running = cluster.barrier_arrive();
  const int E = a.n_experts;
  const int c = threadIdx.x % kFinishCols, group = threadIdx.x / kFinishCols;
  const int e = (int)blockIdx.x * kFinishCols + c;
  pdl_wait();
  float sum = 0.0f;
  int n = 0;
  if (e < E) {
#pragma unroll 8
    for (int g = group; g < a.parts; g += kFinishGroups) {
      sum += a.part_sums[(int64_t)g * E + e];
      n += a.part_counts[(int64_t)g * (E + 1) + e];
    }
  }
  group_sums[group][c] = sum;
  group_counts[group][c] = n;
  if (threadIdx.x < 32) {
    int live = 0;
    for (int g = threadIdx.x; g < a.parts; g += 32) live += a.part_counts[(int64_t)g * (E + 1) + E];
    live = __reduce_add_sync(0xffffffffu, live);
    if (threadIdx.x == 0) live_tokens = live;
  }
  __syncthreads();
  const int T = live_tokens;
  float part = 0.0f;
  if (group == 0 && e < E) {
    sum = 0.0f;
    n = 0;
#pragma unroll
    for (int g = 0; g < kFinishGroups; ++g) {
      sum += group_sums[g][c];
      n += group_counts[g][c];
    }
    const float mean = T > 0 ? sum / (float)T : 0.0f;
    a.means[e] = mean;
    a.counts[e] = n;
    part = T > 0 ? (float)n / ((float)a.top_k * (float)T) * mean : 0.0f;
  }
  part = block_sum(part, scratch);
  cluster.barrier_wait(std::move(running));
  if (threadIdx.x == 0) cluster.map_shared_rank(loss_parts, 0)[cluster.block_rank()] = part;
  cluster.sync();
  if (cluster.block_rank() == 0 && threadIdx.x == 0) {
    float loss = 0.0f;
    for (unsigned i = 0; i < cluster.num_blocks(); ++i) loss += loss_parts[i];
    a.loss[0] = (float)E * loss;
    a.counts[E] = T;
  }
  pdl_launch_dependents();
}

// ---------------------------------------------------------------------------
// d logits. With g_j = scale * dweights_j for the slots' experts i_j:
//   softmax           p_e (g_e - sum_j g_j p_(i_j))
//   softmax, renorm   q_j (g_j - <g, q>) at i_j, q the softmax over the chosen
//   sigmoid           g_j s_j (1 - s_j) at i_j
//   sigmoid, renorm   (1 - s_j) q_j (g_j - <g, q>) at i_j, q_j = s_j / sum s
// and from the balance loss, f constant:
//   dloss * E / T * p_e (f_e - <f, p>), times 1 - s_e for sigmoid scores.
// Slots without an expert take no part; an expert named twice takes both parts.
// ---------------------------------------------------------------------------
template <typename T, bool SIGMOID, int V>
__global__ void __launch_bounds__(kRouterThreads) router_grad_kernel(RouterGradArgs a) {
  const int lane = threadIdx.x & 31;
  const int E = a.n_experts;
  pdl_wait();
  // the loss's part: fractions of the slots, the same for every token
  float f[V], c = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = 0.0f;
  if (a.counts != nullptr) {
    const int tokens = a.counts[E];
    if (tokens > 0) {
      const float per = 1.0f / ((float)a.top_k * (float)tokens);
      c = a.dloss[0] * (float)E / (float)tokens;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        f[i] = e < E ? (float)a.counts[e] * per : 0.0f;
      }
    }
  }
  for (int64_t t = (int64_t)blockIdx.x * kRouterWarps + threadIdx.x / 32; t < a.ntok; t += (int64_t)gridDim.x * kRouterWarps) {
    const bool live = a.live == nullptr || a.live[t] != 0;
    const T* row = static_cast<const T*>(a.logits) + t * a.ldl;
    float l[V], p[V], d[V];
    load_logits<T, V>(row, E, lane, l);
    int id = a.dweights != nullptr && lane < a.top_k ? a.ids[t * a.top_k + lane] : -1;
    if (id >= E) id = -1;
    const float dw = id >= 0 ? a.dweights[t * a.top_k + lane] : 0.0f;
    float chosen = id >= 0 ? to_f32(row[id]) : neg_inf();
    const bool any = row_shares<SIGMOID, V>(l, p);
    const float none = row_is_bad<SIGMOID, V>(l) ? __uint_as_float(0x7fc00000u) : 0.0f;
    float inner = 0.0f;   // softmax: every expert's share times this goes off
    if (a.counts != nullptr && any) {
      float fp = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) fp += f[i] * p[i];
      fp = warp_sum(fp);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        d[i] = c * p[i] * (f[i] - fp);
        if constexpr (SIGMOID) d[i] *= sigmoid(-l[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = 0.0f;
    }
    if (a.dweights != nullptr) {
      const bool has = id >= 0 && any;
      const float g = has ? a.scale * dw : 0.0f;
      if (!has) chosen = neg_inf();
      float add = 0.0f;   // at the expert
      if (a.renorm) {
        const float top = warp_max(SIGMOID ? fminf(chosen, 0.0f) : chosen);
        float q = !has ? 0.0f : (SIGMOID ? sigmoid_scaled(chosen, top) : (chosen == neg_inf() ? 0.0f : exp_of(chosen - top)));
        const float sum = warp_sum(q);
        q = sum == 0.0f ? 0.0f : q / sum;
        add = q * (g - warp_sum(has ? g * q : 0.0f));
        if constexpr (SIGMOID) add *= sigmoid(-chosen);
      } else if constexpr (SIGMOID) {
        add = g * sigmoid(chosen) * sigmoid(-chosen);
      } else {
        // the lane that holds the expert's share gives it
        float share = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float v = __shfl_sync(0xffffffffu, p[i], id & 31);
          share = has && id / 32 == i ? v : share;
        }
        add = g * share;
        inner = warp_sum(add);
      }
      for (int j = 0; j < a.top_k; ++j) {
        const int e = __shfl_sync(0xffffffffu, id, j);
        const float v = __shfl_sync(0xffffffffu, add, j);
        const int at = (e & 31) == lane ? e >> 5 : -1;   // -1 of a slot without an expert matches no i
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (at == i) d[i] += v;
        }
      }
    }
    __syncwarp();   // out may be the logits: every lane has read its slot's, which another lane writes
    T* out = static_cast<T*>(a.dlogits) + t * a.ldd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 32 * i;
      if (e < E) out[e] = from_f32<T>(live ? d[i] - p[i] * inner + none : 0.0f);
    }
  }
  pdl_launch_dependents();
}

namespace {

// Calls f(type tag, sigmoid tag, values a lane).
template <typename F>
cudaError_t by_experts(int n_experts, F&& f) {
  if (n_experts <= 32) return f(std::integral_constant<int, 1>());
  if (n_experts <= 64) return f(std::integral_constant<int, 2>());
  if (n_experts <= 128) return f(std::integral_constant<int, 4>());
  if (n_experts <= 256) return f(std::integral_constant<int, 8>());
  if (n_experts <= 512) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
}
template <typename T>
struct Tag {
  using type = T;
};
template <typename F>
cudaError_t by_type(int type, F&& f) {
  switch (type) {
    case QMV_BF16: return f(Tag<__nv_bfloat16>());
    case QMV_F16: return f(Tag<__half>());
    default: return f(Tag<float>());
  }
}
template <typename F>
cudaError_t router_dispatch(int type, int score, int n_experts, F&& f) {
  return by_type(type, [&](auto t) {
    return by_experts(n_experts, [&](auto v) {
      return score == QMV_SCORE_SIGMOID ? f(t, std::true_type(), v) : f(t, std::false_type(), v);
    });
  });
}
dim3 token_grid(int64_t ntok) { return dim3((unsigned)((ntok + kRouterWarps - 1) / kRouterWarps)); }
// CTAs that take tokens in turn: several an SM, so that what they set up first is set up seldom.
dim3 turn_grid(int64_t ntok) {
  const int64_t most = 6 * (int64_t)device_sm_count(), n = (ntok + kRouterWarps - 1) / kRouterWarps;
  return dim3((unsigned)(n < most ? n : most));
}

}  // namespace

cudaError_t launch_router(const RouterArgs& a) {
  return router_dispatch(a.type, a.score, a.n_experts, [&](auto t, auto s, auto v) {
    return launch_pdl(router_kernel<typename decltype(t)::type, decltype(s)::value, decltype(v)::value>, token_grid(a.ntok),
                      dim3(kRouterThreads), 0, a.stream, a);
  });
}

cudaError_t launch_router_grad(const RouterGradArgs& a) {
  return router_dispatch(a.type, a.score, a.n_experts, [&](auto t, auto s, auto v) {
    return launch_pdl(router_grad_kernel<typename decltype(t)::type, decltype(s)::value, decltype(v)::value>,
                      turn_grid(a.ntok), dim3(kRouterThreads), 0, a.stream, a);
  });
}

int balance_parts(int64_t ntok) {
  if (ntok <= kBalanceAlone) return 1;
  const int64_t n = (ntok + 15) / 16;
  return (int)(n < kBalanceParts ? n : kBalanceParts);
}

cudaError_t launch_balance(const BalanceArgs& a) {
  cudaError_t e = router_dispatch(a.type, a.score, a.n_experts, [&](auto t, auto s, auto v) {
    auto* kernel = balance_kernel<typename decltype(t)::type, decltype(s)::value, decltype(v)::value>;
    constexpr int warps = kBalanceWarps<decltype(v)::value>;
    constexpr int most = (32 * decltype(v)::value) * warps * 4 + (32 * decltype(v)::value + 1) * 4;
    const size_t smem = (size_t)a.n_experts * warps * 4 + (a.n_experts + 1) * 4;
    if constexpr (most > 48 * 1024) {
      g_launch_stage = "cudaFuncSetAttribute";
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      if (e != cudaSuccess) return e;
      g_launch_stage = "launch";
    }
    return launch_pdl(kernel, dim3((unsigned)a.parts), dim3(warps * 32), smem, a.stream, a);
  });
  if (e != cudaSuccess || a.parts == 1) return e;
  const unsigned ctas = (unsigned)((a.n_experts + kFinishCols - 1) / kFinishCols);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kFinishCols * kFinishGroups);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.stream != nullptr ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, balance_finish_kernel, a);
}

}  // namespace qmv
