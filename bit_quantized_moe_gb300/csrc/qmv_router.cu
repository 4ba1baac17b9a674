// qmv_router.cu -- the router of a MoE layer: the top_k experts of each token
// and their weights, the balance loss with the slots of each expert, and the
// gradient of both.
#include <type_traits>

#include "qmv_internal.h"
#include "qmv_rows.cuh"

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
// is in range where u is not. expf and its sums are fp32; a row of E terms is
// within (E / 32 + 12) * 2^-24 or so of exact.
//
// A logit of -infinity is an expert that is not there. A row with a NaN
// (softmax: or +infinity) has no scores: its weights and its gradient are NaN.
// ---------------------------------------------------------------------------
constexpr int kRouterThreads = 256;
constexpr int kRouterWarps = kRouterThreads / 32;

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
__device__ __forceinline__ float sigmoid(float l) { return expf(fminf(l, 0.0f)) / (1.0f + expf(-fabsf(l))); }
__device__ __forceinline__ float sigmoid_scaled(float l, float top) {
  return l == neg_inf() ? 0.0f : expf(fminf(l, 0.0f) - top) / (1.0f + expf(-fabsf(l)));
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
    else p[i] = l[i] == neg_inf() ? 0.0f : expf(l[i] - top);
    sum += p[i];
  }
  sum = warp_sum(sum);
  if (sum == 0.0f) return false;
#pragma unroll
  for (int i = 0; i < V; ++i) p[i] /= sum;
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
      uint32_t best = 0;
      int at = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (key[i] > best) {
          best = key[i];
          at = i;
        }
      }
      const uint32_t m = __reduce_max_sync(0xffffffffu, best);
      const int e = (int)__reduce_min_sync(0xffffffffu, best == m ? (uint32_t)(lane + 32 * at) : 0xffffffffu);
      if (m == 0u) break;   // no logit above -infinity is left
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
      const float v = id < 0 ? 0.0f : (SIGMOID ? sigmoid_scaled(chosen, fminf(first, 0.0f)) : expf(chosen - first));
      w = v / warp_sum(v);
    } else if constexpr (SIGMOID) {
      w = sigmoid(chosen);
    } else {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += l[i] == neg_inf() ? 0.0f : expf(l[i] - first);
      w = expf(chosen - first) / warp_sum(sum);
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
// row of partial sums; the second launch adds the rows in order. Slots and
// tokens are counted in integers, so that every sum is the same every run.
// ---------------------------------------------------------------------------
constexpr int kBalanceThreads = 512;
constexpr int kBalanceWarps = kBalanceThreads / 32;

template <typename T, bool SIGMOID, int V>
__global__ void __launch_bounds__(kBalanceThreads) balance_kernel(BalanceArgs a) {
  extern __shared__ float sums[];   // [warps][E], then counts [E + 1]
  const int E = a.n_experts;
  int* counts = reinterpret_cast<int*>(sums + kBalanceWarps * E);
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  for (int i = threadIdx.x; i <= E; i += kBalanceThreads) counts[i] = 0;
  __syncthreads();
  pdl_wait();
  float mine[V];
#pragma unroll
  for (int i = 0; i < V; ++i) mine[i] = 0.0f;
  int live_tokens = 0;
  for (int64_t t = (int64_t)warp * gridDim.x + blockIdx.x; t < a.ntok; t += (int64_t)gridDim.x * kBalanceWarps) {
    if (a.live != nullptr && a.live[t] == 0) continue;
    float l[V], p[V];
    load_logits<T, V>(static_cast<const T*>(a.logits) + t * a.ldl, E, lane, l);
    const int id = lane < a.top_k ? a.ids[t * a.top_k + lane] : -1;
    if (!row_shares<SIGMOID, V>(l, p)) continue;
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
  float* part = a.part_sums + (int64_t)blockIdx.x * E;
  int* part_counts = a.part_counts + (int64_t)blockIdx.x * (E + 1);
  for (int e = threadIdx.x; e <= E; e += kBalanceThreads) {
    part_counts[e] = counts[e];
    if (e == E) break;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kBalanceWarps; ++w) v += sums[w * E + e];
    part[e] = v;
  }
  pdl_launch_dependents();
}

__global__ void __launch_bounds__(1024) balance_finish_kernel(BalanceArgs a) {
  __shared__ float warp_part[32];
  __shared__ int tokens;
  const int E = a.n_experts, e = threadIdx.x;
  pdl_wait();
  float sum = 0.0f;
  int n = 0;
  if (e < E) {
#pragma unroll 8
    for (int g = 0; g < a.parts; ++g) {
      sum += a.part_sums[(int64_t)g * E + e];
      n += a.part_counts[(int64_t)g * (E + 1) + e];
    }
  }
  if (threadIdx.x < 32) {
    int live = 0;
    for (int g = threadIdx.x; g < a.parts; g += 32) live += a.part_counts[(int64_t)g * (E + 1) + E];
    live = __reduce_add_sync(0xffffffffu, live);
    if (threadIdx.x == 0) tokens = live;
  }
  __syncthreads();
  const int T = tokens;
  const float mean = T > 0 ? sum / (float)T : 0.0f;
  const float f = T > 0 ? (float)n / ((float)a.top_k * (float)T) : 0.0f;
  const float part = warp_sum(e < E ? f * mean : 0.0f);
  if ((threadIdx.x & 31) == 0) warp_part[threadIdx.x / 32] = part;
  if (e < E) {
    a.means[e] = mean;
    a.counts[e] = n;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const float all = warp_sum(warp_part[threadIdx.x]);
    if (threadIdx.x == 0) {
      a.loss[0] = (float)E * all;
      a.counts[E] = T;
    }
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
  const int64_t t = (int64_t)blockIdx.x * kRouterWarps + threadIdx.x / 32;
  const int E = a.n_experts;
  pdl_wait();
  if (t < a.ntok) {
    const bool live = a.live == nullptr || a.live[t] != 0;
    const T* row = static_cast<const T*>(a.logits) + t * a.ldl;
    float l[V], p[V], d[V];
    load_logits<T, V>(row, E, lane, l);
    const bool any = row_shares<SIGMOID, V>(l, p);
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = 0.0f;
    if (a.dweights != nullptr) {
      int id = lane < a.top_k ? a.ids[t * a.top_k + lane] : -1;
      if (id >= E || !any) id = -1;
      const bool has = id >= 0;
      const float g = has ? a.scale * a.dweights[t * a.top_k + lane] : 0.0f;
      const float chosen = has ? to_f32(row[id]) : neg_inf();
      float add = 0.0f, inner = 0.0f;   // at the expert; softmax: times p everywhere
      if (a.renorm) {
        const float top = warp_max(SIGMOID ? fminf(chosen, 0.0f) : chosen);
        float q = !has ? 0.0f : (SIGMOID ? sigmoid_scaled(chosen, top) : (chosen == neg_inf() ? 0.0f : expf(chosen - top)));
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
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] += lane + 32 * i == e ? v : 0.0f;
      }
      if (!SIGMOID && !a.renorm) {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] -= p[i] * inner;
      }
    }
    if (a.counts != nullptr && any) {
      const int tokens = a.counts[E];
      const float per = tokens > 0 ? 1.0f / ((float)a.top_k * (float)tokens) : 0.0f;
      float f[V], fp = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        f[i] = e < E ? (float)a.counts[e] * per : 0.0f;
        fp += f[i] * p[i];
      }
      fp = warp_sum(fp);
      const float c = tokens > 0 ? a.dloss[0] * (float)E / (float)tokens : 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v = c * p[i] * (f[i] - fp);
        if constexpr (SIGMOID) v *= sigmoid(-l[i]);
        d[i] += v;
      }
    }
    const float none = row_is_bad<SIGMOID, V>(l) ? __uint_as_float(0x7fc00000u) : 0.0f;
    T* out = static_cast<T*>(a.dlogits) + t * a.ldd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 32 * i;
      if (e < E) out[e] = from_f32<T>(live ? d[i] + none : 0.0f);
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
                      token_grid(a.ntok), dim3(kRouterThreads), 0, a.stream, a);
  });
}

// CTAs of the first launch: few, so that the second, of one CTA, has few rows to add.
int balance_parts(int64_t ntok) {
  const int64_t n = (ntok + 2 * kBalanceWarps - 1) / (2 * kBalanceWarps);
  return (int)(n < 1 ? 1 : (n > 64 ? 64 : n));
}

cudaError_t launch_balance(const BalanceArgs& a) {
  const size_t smem = (size_t)a.n_experts * kBalanceWarps * 4 + (a.n_experts + 1) * 4;
  cudaError_t e = router_dispatch(a.type, a.score, a.n_experts, [&](auto t, auto s, auto v) {
    auto* kernel = balance_kernel<typename decltype(t)::type, decltype(s)::value, decltype(v)::value>;
    constexpr int most = (32 * decltype(v)::value) * kBalanceWarps * 4 + (32 * decltype(v)::value + 1) * 4;
    if constexpr (most > 48 * 1024) {
      g_launch_stage = "cudaFuncSetAttribute";
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      if (e != cudaSuccess) return e;
      g_launch_stage = "launch";
    }
    return launch_pdl(kernel, dim3((unsigned)a.parts), dim3(kBalanceThreads), smem, a.stream, a);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(balance_finish_kernel, dim3(1), dim3(1024), 0, a.stream, a);
}

}  // namespace qmv
