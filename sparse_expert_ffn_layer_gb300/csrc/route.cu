// Routing by scores: s = softmax(x) or 1 / (1 + exp(-x)) over a token's experts, choice c = s + bias, the
// best top_groups groups of experts by the sum of their group_top largest c, of those the k experts of
// largest c (ties to the lower index), and weights w_j = scale s_j, divided by their sum if renormalised.
//
// The order is that of the scores as real numbers.  Without a bias, and where no two scores are added,
// the logits themselves have that order.  Otherwise c is computed in 32 bits, and a row in which two
// values whose order matters are nearer than its rounding errors allow is decided again in 64 bits:
// the experts of a token do not depend on how exp or a sum was rounded.
//
// A warp takes a row: its values stay in registers (column lane + 32 v), a round of the selection is two
// warp-wide reductions over order-preserving integer keys and a pass over the lane's own values.
// Bound by these rounds' latencies and instructions, not by the 4 E bytes of a row.
#include "launch.h"

namespace moe {
namespace {

constexpr int kWarps = 4;

// Keys with the order of the values (-0 = +0); NaN has some place in it, so that an index is always valid.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return b ^ ((b >> 63) ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(0xffffffffu, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t q = __shfl_xor_sync(0xffffffffu, (unsigned long long)k, o);
    k = q > k ? q : k;
  }
  return k;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

template <typename F>
struct KeyOf {
  using type = uint32_t;
};
template <>
struct KeyOf<double> {
  using type = uint64_t;
};

// Two choices further apart than slack (unit + |c|), unit the largest score a row can have, keep their order
// in 32 bits.  With u = 2^-24: exp is good to 2 ulp = 4 u, and the sigmoid's sum and quotient to u each:
// 6 u s; the softmax's sum of E terms adds V + 5 u, x - max at most 0.4 u and the product u: (12 + V) u s.
// The bias's addition is off by u |c|.  Twice that for the two values.
__device__ __forceinline__ float slack(int sigmoid, int V) {
  return 2.f * (sigmoid ? 8.f : 14.f + V) * 5.9604645e-08f;
}

// Scores of a row in place (logits -> s); columns beyond E, and rows of -inf only, have s = 0.
template <int V, typename F>
__device__ __forceinline__ void scores(F (&x)[V], int sigmoid, F& m, F& sum) {
  if (sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = F(1) / (F(1) + exp_of(-x[v]));
    return;
  }
  m = x[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = x[v] > m ? x[v] : m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const F q = __shfl_xor_sync(0xffffffffu, m, o);
    m = q > m ? q : m;
  }
  if (m == -INFINITY) m = F(0);
  sum = F(0);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    x[v] = exp_of(x[v] - m);
    sum += x[v];
  }
  sum = warp_sum(sum);
  const F inv = sum > F(0) ? F(1) / sum : F(0);
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] *= inv;
}

// The k experts of largest choice; lane j < k gets expert j.  Returns whether the order is certain: of the
// values whose order matters no two are within tol (unit + |c|) of each other (tol = 0: not looked at).
template <int V, typename F>
__device__ __forceinline__ bool select(F (&c)[V], const ScoreArgs& a, F* sh, int lane, F tol, F unit, int& mine) {
  using K = typename KeyOf<F>::type;
  bool sure = true;
  K key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = lane + 32 * v < a.E ? key_of(c[v]) : K(0);
  if (a.n_groups > 1 && a.top_groups < a.n_groups) {
    const int M = a.E / a.n_groups;
    __syncwarp();
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane + 32 * v < a.E) sh[lane + 32 * v] = c[v];
    __syncwarp();
    // a power of two of lanes per group
    int per = 1;
    while (per * 2 * a.n_groups <= 32) per *= 2;
    const int g = lane / per, l = lane % per;
    F b1 = -INFINITY, b2 = -INFINITY;
    if (g < a.n_groups)
      for (int i = l; i < M; i += per) {
        const F q = sh[g * M + i];
        if (q > b1) {
          b2 = b1;
          b1 = q;
        } else if (q > b2) {
          b2 = q;
        }
      }
    for (int o = per / 2; o > 0; o >>= 1) {
      const F q1 = __shfl_xor_sync(0xffffffffu, b1, o), q2 = __shfl_xor_sync(0xffffffffu, b2, o);
      const F lo = q1 < b1 ? q1 : b1;
      b1 = q1 > b1 ? q1 : b1;
      b2 = b2 > q2 ? b2 : q2;
      b2 = lo > b2 ? lo : b2;
    }
    const F value = (a.group_top == 2 && M > 1) ? b1 + b2 : b1;
    // rank of this lane's group; near: another group's value is not surely on its side
    const K kv = key_of(value);
    int rank = 0;
    bool near = false;
    for (int q = 0; q < a.n_groups; ++q) {
      const F w = __shfl_sync(0xffffffffu, value, q * per);
      const K kw = key_of(w);
      rank += (kw > kv || (kw == kv && q < g)) ? 1 : 0;
      const F gap = w > value ? w - value : value - w;
      // (sums of two: twice the error)
      near |= q != g && gap <= F(2) * tol * (unit + (value < F(0) ? -value : value));
    }
    const bool in = g < a.n_groups && rank < a.top_groups;
    // only the border between the last group inside and the first outside matters
    const bool edge = g < a.n_groups && near && (rank == a.top_groups - 1 || rank == a.top_groups);
    if (tol > F(0) && __any_sync(0xffffffffu, edge)) sure = false;
    const unsigned inside = __ballot_sync(0xffffffffu, in && l == 0);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = lane + 32 * v;
      if (e < a.E && !((inside >> (e / M * per)) & 1u)) key[v] = K(0);
    }
  }
  // k rounds, and one more for the first expert that is left out
  mine = 0;
  const int rounds = (a.k < a.E && tol > F(0)) ? a.k + 1 : a.k;
  F last = F(0);
  for (int j = 0; j < rounds; ++j) {
    K best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = key[v] > best ? key[v] : best;
    const K top = warp_max(best);
    int at = 0x7fffffff;
#pragma unroll
    for (int v = V - 1; v >= 0; --v) at = key[v] == top ? lane + 32 * v : at;
    at = (int)__reduce_min_sync(0xffffffffu, (unsigned)at);
    if (j < a.k && lane == j) mine = min(at, a.E - 1);
    if (tol > F(0)) {
      F val;
      if constexpr (sizeof(F) == 4) val = value_of(top);
      else val = F(0);
      if (top == K(0)) val = -INFINITY;
      if (j > 0 && last - val <= tol * (unit + (val < F(0) ? -val : val))) sure = false;
      last = val;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane + 32 * v == at) key[v] = K(0);
  }
  return sure;
}

template <int V>
__device__ __forceinline__ void load(float (&x)[V], const float* row, int E, int lane) {
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = lane + 32 * v < E ? row[lane + 32 * v] : -INFINITY;
}

// 64 bits, from the logits: rare rows only, so it is kept out of the row loop's registers.
template <int V>
__device__ __noinline__ int route_wide(const float* row, const ScoreArgs& a, double* sh, int lane) {
  double c[V], m, sum;
#pragma unroll
  for (int v = 0; v < V; ++v) c[v] = lane + 32 * v < a.E ? (double)row[lane + 32 * v] : -INFINITY;
  scores<V, double>(c, a.sigmoid, m, sum);
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (a.bias && lane + 32 * v < a.E) c[v] += (double)a.bias[lane + 32 * v];
  int mine;
  select<V, double>(c, a, sh, lane, 0.0, 0.0, mine);
  return mine;
}

template <int V>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const ScoreArgs a, int direct) {
  extern __shared__ double shared[];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  double* sh = shared + (size_t)w * a.E;
  for (int t = blockIdx.x * kWarps + w; t < a.T; t += gridDim.x * kWarps) {
    const float* row = a.logits + (size_t)t * a.E;
    const bool on = !a.mask || a.mask[t];
    float x[V];
    load<V>(x, row, a.E, lane);
    if (a.logits_copy)
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (lane + 32 * v < a.E) a.logits_copy[(size_t)t * a.E + lane + 32 * v] = x[v];
    float m = 0.f, sum = 0.f;
    int mine = 0;
    // the scores of all columns: where they are wanted or order the row, or their sum is
    const bool all = a.scores || !direct || (!a.sigmoid && !a.renorm);
    float s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = x[v];
    if (all) scores<V, float>(s, a.sigmoid, m, sum);
    if (a.scores)
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (lane + 32 * v < a.E) a.scores[(size_t)t * a.E + lane + 32 * v] = on ? s[v] : 0.f;
    if (!on) {
      if (lane < a.k) {
        a.topk_idx[(size_t)t * a.k + lane] = -1;
        a.topk_w[(size_t)t * a.k + lane] = 0.f;
      }
      continue;
    }
    if (direct) {
      select<V, float>(x, a, reinterpret_cast<float*>(sh), lane, 0.f, 0.f, mine);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (a.bias && lane + 32 * v < a.E) s[v] += a.bias[lane + 32 * v];
      const float unit = a.sigmoid ? 1.f : (sum > 0.f ? 1.f / sum : 0.f);
      if (!select<V, float>(s, a, reinterpret_cast<float*>(sh), lane, slack(a.sigmoid, V), unit, mine))
        mine = route_wide<V>(row, a, sh, lane);
    }
    // weights of lanes 0 .. k-1 (scores of -inf: zero)
    const bool have = lane < a.k;
    const float xl = have ? row[mine] : -INFINITY;
    float u;
    if (a.renorm) {
      // a common factor drops out: taken so that the largest u is about one
      const float low = a.sigmoid ? fminf(xl, 0.f) : xl;
      float top = low;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      u = xl == -INFINITY ? 0.f : expf(low - top);
      if (a.sigmoid && u > 0.f) u /= 1.f + expf(-fabsf(xl));
      const float tot = warp_sum(u);
      u = tot > 0.f ? u / tot : (tot == 0.f ? 0.f : tot);
    } else if (a.sigmoid) {
      u = 1.f / (1.f + expf(-xl));
    } else {
      u = sum > 0.f ? expf(xl - m) / sum : (sum == 0.f ? 0.f : sum);
    }
    if (have) {
      a.topk_idx[(size_t)t * a.k + lane] = mine;
      a.topk_w[(size_t)t * a.k + lane] = u * a.scale;
    }
  }
}

}  // namespace

cudaError_t launch_route(const ScoreArgs& a, cudaStream_t s, bool pdl) {
  int dev = 0, sms = 0;
  MOE_LAUNCH(cudaGetDevice(&dev));
  MOE_LAUNCH(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  const bool limited = a.n_groups > 1 && a.top_groups < a.n_groups;
  const int direct = !a.bias && !(limited && a.group_top == 2 && a.E > a.n_groups);
  const size_t smem = limited || !direct ? sizeof(double) * kWarps * a.E : 0;
  const int grid = std::min((a.T + kWarps - 1) / kWarps, 16 * sms);
  auto go = [&](auto kern) { return launch_k(kern, grid, kWarps * 32, smem, s, pdl, a, direct); };
  if (a.E <= 32) return go(route_kernel<1>);
  if (a.E <= 64) return go(route_kernel<2>);
  if (a.E <= 128) return go(route_kernel<4>);
  if (a.E <= 256) return go(route_kernel<8>);
  if (a.E <= 512) return go(route_kernel<16>);
  return go(route_kernel<32>);
}

}  // namespace moe
