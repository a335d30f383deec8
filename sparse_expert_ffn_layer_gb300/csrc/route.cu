// Routing by scores: s = softmax(x) or 1 / (1 + exp(-x)) over a token's experts, choice c = s + bias, the
// best top_groups groups of experts by the sum of their group_top largest c, of those the k experts of
// largest c (ties to the lower index), and weights w_j = scale s_j, divided by their sum if renormalised.
//
// The order is that of the scores as real numbers.  Without a bias, and where no two scores are added,
// the logits themselves have that order.  Otherwise c is computed in 32 bits, and a row in which two
// values whose order matters are nearer than its rounding errors allow is decided again in 64 bits:
// the experts of a token do not depend on how exp or a sum was rounded.
//
// A warp takes a row, whose values stay in registers as order-preserving integer keys.  The (k + 1)th largest of the
// lanes' own largest keys is at most the row's (k + 1)th largest: only keys from there on, hardly more than k, are put
// one to a lane and ranked against each other.  (Rounds of two warp-wide reductions and a pass over a lane's values,
// which still serve rows of many equal keys, took 1320 instructions a row of 256 experts in groups, k = 8: the integer
// pipe 68 % busy.)  A lane has V neighbouring columns where a row is 32 V of them (their loads are wide, and groups of
// whole lanes need no shared memory), else every 32nd.  Bound by a warp's chain of dependent
// shuffles and ranks (no pipe above half, half of the warps resident), not by the 4 E bytes of a row: 16384 rows of 256,
// k = 8: 19 us by the logits alone, 23 with a bias, 27 with a bias and groups, cold (rounds: 22, 28, 42).
#include <type_traits>

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
template <typename K>
struct ShflOf {
  using type = K;
};
template <>
struct ShflOf<uint64_t> {
  using type = unsigned long long;
};

// Column of value v of a lane.
template <int V, bool kWide>
__device__ __forceinline__ int col_at(int v, int lane) { return kWide ? lane * V + v : lane + 32 * v; }

// Two choices further apart than slack (unit + |c|), unit the largest score a row can have, keep their order
// in 32 bits.  With u = 2^-24: the hardware's exponential is good to 2 ulp = 4 u and |x| u, its sum and quotient to u
// and 2 u, which for the sigmoid is s (|x| + 7) u where exp(-x) matters, at most 4 u; the softmax's sum of E terms adds
// V + 5 u, x - max at most 0.4 u and the product u: (12 + V) u s.  The bias's addition is off by u |c|.  Twice that for
// the two values.
__device__ __forceinline__ float slack(int sigmoid, int V) {
  return 2.f * (sigmoid ? 5.f : 14.f + V) * 5.9604645e-08f;
}

__device__ __forceinline__ float sigmoid_of(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
__device__ __forceinline__ double sigmoid_of(double x) { return 1.0 / (1.0 + exp(-x)); }

// Scores of a row in place (logits -> s); columns beyond E, and rows of -inf only, have s = 0.
template <int V, typename F>
__device__ __forceinline__ void scores(F (&x)[V], int sigmoid, F& m, F& sum) {
  if (sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = sigmoid_of(x[v]);
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

// A group's value from its two largest choices: an infinite one decides it alone (a second one of -infinity would make NaN).
template <typename F>
__device__ __forceinline__ F group_value(F b1, F b2, bool two) { return two && b1 < F(INFINITY) ? b1 + b2 : b1; }

// The ranks of the groups in 64 bits for sigmoid scores, from the experts that may count: those not surely below their
// group's group_top-th in 32 bits.  low: what that is for a lane's own group.  False if these are more than 32.
template <int V, bool kWide>
__device__ __forceinline__ bool groups_near(const float* row, const ScoreArgs& a, const float (&c)[V], float low, int M,
                                            int per, int* sh, int lane, int& rank) {
  int n = 0;
  __syncwarp();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = col_at<V, kWide>(v, lane);
    const float l = __shfl_sync(0xffffffffu, low, min(e / M, a.n_groups - 1) * per);
    const bool near = e < a.E && c[v] >= l;
    const unsigned m = __ballot_sync(0xffffffffu, near);
    const int at = n + __popc(m & ((1u << lane) - 1u));
    if (near && at < 32) sh[at] = e;
    n += __popc(m);
  }
  if (n > 32) return false;
  __syncwarp();
  const int e = lane < n ? sh[lane] : 0, ge = lane < n ? e / M : -1, g = lane / per;
  const double own = sigmoid_of((double)row[e]) + (a.bias ? (double)a.bias[e] : 0.0);
  double b1 = -INFINITY, b2 = -INFINITY;
  for (int q = 0; q < n; ++q) {
    const double x = __shfl_sync(0xffffffffu, own, q);
    if (__shfl_sync(0xffffffffu, ge, q) != g) continue;
    const double lo = x < b1 ? x : b1;
    b1 = x > b1 ? x : b1;
    b2 = lo > b2 ? lo : b2;
  }
  const uint64_t kv = key_of(group_value(b1, b2, a.group_top == 2 && M > 1));
  rank = 0;
  for (int q = 0; q < a.n_groups; ++q) {
    const uint64_t kw = __shfl_sync(0xffffffffu, (unsigned long long)kv, q * per);
    rank += (kw > kv || (kw == kv && q < g)) ? 1 : 0;
  }
  __syncwarp();
  return true;
}

// The k experts of largest choice; lane j < k gets expert j, lane k the first that is left out.  Says where the order is
// not certain, because two values whose order matters are within tol (unit + |c|) of each other (tol = 0: not looked
// at): bit 0 of the experts, bit 1 of the groups too, or in a way that needs the whole row.  key: the choices of the
// experts in the groups.  taken, floor: how many experts were taken (fewer than k + 1 where no more are in the groups) and
// the least of their choices.  sh: 64 words, and E values where groups go through it.
template <int V, bool kWide, typename F>
__device__ __forceinline__ int select(const float* row, F (&c)[V], const ScoreArgs& a, F* sh, int lane, F tol, F unit, int& mine,
                                      typename KeyOf<F>::type (&key)[V], F& floor, int& taken) {
  using K = typename KeyOf<F>::type;
  int unsure = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = kWide || lane + 32 * v < a.E ? key_of(c[v]) : K(0);
  if (a.n_groups > 1 && a.top_groups < a.n_groups) {
    const int M = a.E / a.n_groups;
    // lanes per group, a power of two: all of a group's own, or as many as there are
    const int own = kWide && M % V == 0 && ((M / V) & (M / V - 1)) == 0 ? M / V : 0;
    int per = 1;
    F b1 = -INFINITY, b2 = -INFINITY;
    auto take = [&](F q) {
      const F lo = q < b1 ? q : b1;
      b1 = q > b1 ? q : b1;
      b2 = lo > b2 ? lo : b2;
    };
    if (own) {
      per = own;
#pragma unroll
      for (int v = 0; v < V; ++v) take(c[v]);
    } else {
      while (per * 2 * a.n_groups <= 32) per *= 2;
      __syncwarp();
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (col_at<V, kWide>(v, lane) < a.E) sh[col_at<V, kWide>(v, lane)] = c[v];
      __syncwarp();
      if (lane / per < a.n_groups)
        for (int i = lane % per; i < M; i += per) take(sh[lane / per * M + i]);
    }
    const int g = lane / per, l = lane % per;
    for (int o = per / 2; o > 0; o >>= 1) {
      const F q1 = __shfl_xor_sync(0xffffffffu, b1, o), q2 = __shfl_xor_sync(0xffffffffu, b2, o);
      take(q1);
      b2 = q2 > b2 ? q2 : b2;
    }
    const F value = group_value(b1, b2, a.group_top == 2 && M > 1);
    const K kv = key_of(value);
    int rank = 0;
    for (int q = 0; q < a.n_groups; ++q) {
      const K kw = __shfl_sync(0xffffffffu, (typename ShflOf<K>::type)kv, q * per);
      rank += (kw > kv || (kw == kv && q < g)) ? 1 : 0;
    }
    if (tol > F(0)) {
      // only the border between the last group inside and the first outside matters (sums of two: twice the error)
      const unsigned last = __ballot_sync(0xffffffffu, g < a.n_groups && rank == a.top_groups - 1);
      const unsigned next = __ballot_sync(0xffffffffu, g < a.n_groups && rank == a.top_groups);
      const F in = __shfl_sync(0xffffffffu, value, __ffs(last) - 1), out = __shfl_sync(0xffffffffu, value, __ffs(next) - 1);
      // (an infinite choice is before any other, however large the bound would be)
      if (in < F(INFINITY) && in - out <= F(2) * tol * (unit + (in < F(0) ? -in : in))) {
        unsure |= 2;
        if constexpr (sizeof(F) == 4) {
          const float least = (a.group_top == 2 && M > 1) ? b2 : b1;
          const float low = isinf(least) ? least : least - 2.f * tol * (unit + fabsf(least));
          if (a.sigmoid && groups_near<V, kWide>(row, a, c, low, M, per, reinterpret_cast<int*>(sh), lane, rank))
            unsure = 0;
        }
      }
    }
    if (own) {
      if (rank >= a.top_groups)
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = K(0);
    } else {
      const unsigned inside = __ballot_sync(0xffffffffu, g < a.n_groups && rank < a.top_groups && l == 0);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = col_at<V, kWide>(v, lane);
        if (e < a.E && !((inside >> (e / M * per)) & 1u)) key[v] = K(0);
      }
    }
  }
  // k experts, and one more for the first that is left out
  mine = 0;
  const int rounds = (a.k < a.E && tol > F(0)) ? a.k + 1 : a.k;
  if constexpr (sizeof(F) == 4) {
    uint32_t sorted = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) sorted = max(sorted, key[v]);
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
      for (int o = size / 2; o > 0; o /= 2) {    // descending over the lanes
        const uint32_t q = __shfl_xor_sync(0xffffffffu, sorted, o);
        sorted = ((lane & o) == 0) == ((lane & size) == 0) ? max(sorted, q) : min(sorted, q);
      }
    const uint32_t least = max(__shfl_sync(0xffffffffu, sorted, rounds - 1), 1u);
    uint32_t* near_key = reinterpret_cast<uint32_t*>(sh);
    int* near_col = reinterpret_cast<int*>(sh) + 32;
    int n = 0;
    __syncwarp();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool in = key[v] >= least;
      const unsigned m = __ballot_sync(0xffffffffu, in);
      const int at = n + __popc(m & ((1u << lane) - 1u));
      if (in && at < 32) {
        near_key[at] = key[v];
        near_col[at] = col_at<V, kWide>(v, lane);
      }
      n += __popc(m);
    }
    if (n >= a.k && n <= 32) {
      __syncwarp();
      const uint32_t k0 = lane < n ? near_key[lane] : 0u;
      const int c0 = lane < n ? near_col[lane] : 0x7fffffff;
      int rank = 0;
      for (int q = 0; q < n; ++q) {
        const uint32_t kq = __shfl_sync(0xffffffffu, k0, q);
        const int cq = __shfl_sync(0xffffffffu, c0, q);
        rank += (kq > k0 || (kq == k0 && cq < c0)) ? 1 : 0;
      }
      __syncwarp();
      if (lane < n) {
        near_key[rank] = k0;
        near_col[rank] = c0;
      }
      __syncwarp();
      taken = min(n, rounds);
      mine = near_col[min(lane, taken - 1)];
      if (tol > F(0)) {
        floor = value_of(near_key[taken - 1]);
        const float hi = value_of(near_key[min(lane, taken - 1)]), lo = value_of(near_key[min(lane + 1, taken - 1)]);
        if (__any_sync(0xffffffffu, lane + 1 < taken && hi - lo <= tol * (unit + fabsf(lo)))) unsure |= 1;
      }
      return unsure;
    }
  }
  F last = F(0);
  taken = 0;
  for (int j = 0; j < rounds; ++j) {
    K best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = key[v] > best ? key[v] : best;
    const K top = warp_max(best);
    int at = 0x7fffffff;
#pragma unroll
    for (int v = V - 1; v >= 0; --v) at = key[v] == top ? col_at<V, kWide>(v, lane) : at;
    const int all = (int)__reduce_min_sync(0xffffffffu, (unsigned)at);
    if (lane == j) mine = min(all, a.E - 1);
    if (tol > F(0)) {
      F val;
      if constexpr (sizeof(F) == 4) val = value_of(top);
      else val = F(0);
      if (top == K(0)) break;
      ++taken;
      if (j > 0 && last - val <= tol * (unit + (val < F(0) ? -val : val))) unsure |= 1;
      last = val;
    }
    if (at == all) {                             // (one lane)
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (col_at<V, kWide>(v, lane) == all) key[v] = K(0);
    }
  }
  floor = last;
  return unsure ? unsure | 2 : 0;                // (the keys of those taken are gone)
}

template <int V, bool kWide>
__device__ __forceinline__ void load(float (&x)[V], const float* row, int E, int lane) {
  if constexpr (kWide && V % 4 == 0) {
#pragma unroll
    for (int v = 0; v < V; v += 4) {
      const float4 q = *reinterpret_cast<const float4*>(row + lane * V + v);
      x[v] = q.x; x[v + 1] = q.y; x[v + 2] = q.z; x[v + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = kWide || lane + 32 * v < E ? row[col_at<V, kWide>(v, lane)] : -INFINITY;
  }
}

// 64 bits, from the logits: rare rows only, so it is kept out of the row loop's registers.
template <int V, bool kWide>
__device__ __noinline__ int route_wide(const float* row, const ScoreArgs& a, double* sh, int lane) {
  double c[V], m, sum;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = col_at<V, kWide>(v, lane);
    c[v] = e < a.E ? (double)row[e] : -INFINITY;
  }
  scores<V, double>(c, a.sigmoid, m, sum);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = col_at<V, kWide>(v, lane);
    if (a.bias && e < a.E) c[v] += (double)a.bias[e];
  }
  int mine;
  uint64_t key[V];
  double floor;
  int taken;
  select<V, kWide, double>(row, c, a, sh, lane, 0.0, 0.0, mine, key, floor, taken);
  return mine;
}

// The same for sigmoid scores where only the order of the experts near the last one taken is not certain: a lane decides
// for each expert that was taken, or is within `margin` of the least of these (so that no other can be among the k).
// False if these are fewer than k (NaN) or more than 32.  (All columns in 64 bits take a row 3 us, of which a batch waits
// for the last.)
template <int V, bool kWide>
__device__ __forceinline__ bool route_near(const float* row, const ScoreArgs& a, const uint32_t (&key)[V], float floor,
                                           float margin, int* sh, int lane, int& mine) {
  const uint32_t least = key_of(floor - margin);
  int n = 0;
  __syncwarp();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const bool near = key[v] != 0u && key[v] >= least;
    const unsigned m = __ballot_sync(0xffffffffu, near);
    const int at = n + __popc(m & ((1u << lane) - 1u));
    if (near && at < 32) sh[at] = col_at<V, kWide>(v, lane);
    n += __popc(m);
  }
  if (n < a.k || n > 32) return false;
  __syncwarp();
  const int e = lane < n ? sh[lane] : 0;
  const uint64_t mykey = lane < n ? key_of(sigmoid_of((double)row[e]) + (a.bias ? (double)a.bias[e] : 0.0)) : 0u;
  int rank = 0;
  for (int q = 0; q < n; ++q) {
    const uint64_t k = __shfl_sync(0xffffffffu, (unsigned long long)mykey, q);
    const int i = __shfl_sync(0xffffffffu, e, q);
    rank += (k > mykey || (k == mykey && i < e)) ? 1 : 0;
  }
  __syncwarp();
  if (lane < n) sh[rank] = e;
  __syncwarp();
  mine = sh[min(lane, n - 1)];
  return true;
}

template <int V, bool kWide>
__global__ void __launch_bounds__(kWarps * 32, V <= 8 ? 8 : V <= 16 ? 4 : 2) route_kernel(const ScoreArgs a, int direct) {
  extern __shared__ double shared[];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  float bias[V];                                 // (complete: nothing but the gate kernel may still run)
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = col_at<V, kWide>(v, lane);
    bias[v] = a.bias && e < a.E ? a.bias[e] : 0.f;
  }
  pdl_wait();
  pdl_trigger();
  double* sh = shared + (size_t)w * (a.n_groups > 1 && a.top_groups < a.n_groups ? max(a.E, 32) : 32);
  for (int t = blockIdx.x * kWarps + w; t < a.T; t += gridDim.x * kWarps) {
    const float* row = a.logits + (size_t)t * a.E;
    const bool on = !a.mask || a.mask[t];
    float x[V];
    load<V, kWide>(x, row, a.E, lane);
    if (a.logits_copy)
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (col_at<V, kWide>(v, lane) < a.E) a.logits_copy[(size_t)t * a.E + col_at<V, kWide>(v, lane)] = x[v];
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
        if (col_at<V, kWide>(v, lane) < a.E) a.scores[(size_t)t * a.E + col_at<V, kWide>(v, lane)] = on ? s[v] : 0.f;
    if (!on) {
      if (lane < a.k) {
        a.topk_idx[(size_t)t * a.k + lane] = -1;
        a.topk_w[(size_t)t * a.k + lane] = 0.f;
      }
      continue;
    }
    if (direct) {
      uint32_t key[V];
      float floor;
      int taken;
      select<V, kWide, float>(row, x, a, reinterpret_cast<float*>(sh), lane, 0.f, 0.f, mine, key, floor, taken);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] += bias[v];
      const float unit = a.sigmoid ? 1.f : (sum > 0.f ? 1.f / sum : 0.f);
      uint32_t key[V];
      float floor;
      int taken;
      const float tol = slack(a.sigmoid, V);
      const int unsure = select<V, kWide, float>(row, s, a, reinterpret_cast<float*>(sh), lane, tol, unit, mine, key, floor, taken);
      if (unsure && (unsure != 1 || !a.sigmoid || taken < a.k ||
                     !route_near<V, kWide>(row, a, key, floor, 2.f * tol * (unit + fabsf(floor)), reinterpret_cast<int*>(sh),
                                           lane, mine)))
        mine = route_wide<V, kWide>(row, a, sh, lane);
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
  // 64 words a warp; the values of a row (in 64 bits where that may be needed) where groups go through shared memory
  const size_t smem = sizeof(double) * kWarps * (limited ? std::max(a.E, 32) : 32);
  const int grid = std::min((a.T + kWarps - 1) / kWarps, 16 * sms);
  auto go = [&](auto v) {
    constexpr int V = decltype(v)::value;
    return a.E == 32 * V ? launch_k(route_kernel<V, true>, grid, kWarps * 32, smem, s, pdl, a, direct)
                         : launch_k(route_kernel<V, false>, grid, kWarps * 32, smem, s, pdl, a, direct);
  };
  using std::integral_constant;
  if (a.E <= 32) return go(integral_constant<int, 1>());
  if (a.E <= 64) return go(integral_constant<int, 2>());
  if (a.E <= 128) return go(integral_constant<int, 4>());
  if (a.E <= 256) return go(integral_constant<int, 8>());
  if (a.E <= 512) return go(integral_constant<int, 16>());
  return go(integral_constant<int, 32>());
}

}  // namespace moe
