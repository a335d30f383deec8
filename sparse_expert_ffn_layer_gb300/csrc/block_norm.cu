// The end of a block and the start of the next one, and its gradient:
//   y = sum_j w_j e_j + shared,  z = gate post_w y rp,  h = residual + alpha z,  n = next_w h rn,
//   rp = 1 / sqrt(mean y^2 + eps),  rn = 1 / sqrt(mean h^2 + eps)         (include/moe.h has the gradient)
//
// A team of WPR warps takes a token's row: thread i of the team has the 16-byte pieces i, i + 32 WPR, ..., NV
// of them, in registers from the first load to the last store, so that every row crosses DRAM once.  Bound by
// DRAM: (k + 3) rows a token forward, 2 k + 4 backward.
#include "launch.h"

namespace moe {
namespace {

template <typename T>
struct Piece;                                   // 16 bytes
template <>
struct Piece<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&f)[8]) {
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Piece<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&f)[4]) {
    f[0] = __uint_as_float(r.x);
    f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z);
    f[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

template <int WPR>
constexpr int kBlockWarps = WPR > 4 ? WPR : 4;
// Rows of experts that a thread has in flight.
template <int NV>
constexpr int kFlight = NV > 1 ? 2 : 4;

// Sums over a team's threads.  red: two buffers of WPR words; one barrier per sum (a buffer is written again
// two sums later, behind the barrier of the sum between).
template <int WPR>
struct Team {
  float* red;
  int id, tl, turn;
  __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (WPR == 1) return v;
    float* b = red + turn * WPR;
    turn ^= 1;
    if ((tl & 31) == 0) b[tl >> 5] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "n"(32 * WPR) : "memory");
    float r = b[0];
#pragma unroll
    for (int w = 1; w < WPR; ++w) r += b[w];
    return r;
  }
};

// Floats of a per-column weight at piece p.
template <int N>
__device__ __forceinline__ void weights_at(const float* w, int p, float (&f)[N]) {
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(w) + p * (N / 4) + q);
    f[4 * q] = v.x;
    f[4 * q + 1] = v.y;
    f[4 * q + 2] = v.z;
    f[4 * q + 3] = v.w;
  }
}

// y: the weighted sum of the token's kept rows, a few of them in flight, and the shared row.
template <typename T, int WPR, int NV>
__device__ __forceinline__ void block_sum(const NormArgs& a, size_t t, int tl, float (&y)[NV][Piece<T>::N]) {
  constexpr int N = Piece<T>::N;
  const int pieces = a.d / N;
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int i = 0; i < N; ++i) y[n][i] = 0.f;
  constexpr int U = kFlight<NV>;
  for (int j0 = 0; j0 < a.k; j0 += U) {
    uint4 raw[U][NV];
    float w[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int s = j0 + j < a.k ? a.slot_of[t * a.k + j0 + j] : -1;
      const bool on = (unsigned)s < (unsigned)a.S_max;
      w[j] = on ? a.topk_w[t * a.k + j0 + j] : 0.f;
      const uint4* row = reinterpret_cast<const uint4*>(static_cast<const T*>(a.expert_out) + (size_t)(on ? s : 0) * a.d);
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int p = n * 32 * WPR + tl;
        raw[j][n] = on && p < pieces ? row[p] : make_uint4(0u, 0u, 0u, 0u);
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        float f[N];
        Piece<T>::unpack(raw[j][n], f);
#pragma unroll
        for (int i = 0; i < N; ++i) y[n][i] = fmaf(w[j], f[i], y[n][i]);
      }
  }
  if (a.shared) {
    const uint4* row = reinterpret_cast<const uint4*>(static_cast<const T*>(a.shared) + t * a.d);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int p = n * 32 * WPR + tl;
      if (p < pieces) {
        float f[N];
        Piece<T>::unpack(row[p], f);
#pragma unroll
        for (int i = 0; i < N; ++i) y[n][i] += f[i];
      }
    }
  }
}

template <typename T, int WPR, int NV>
__global__ void __launch_bounds__(32 * kBlockWarps<WPR>, (NV * Piece<T>::N <= 16 ? 32 : 16) / kBlockWarps<WPR>)
    block_norm_kernel(const NormArgs a) {
  constexpr int N = Piece<T>::N, TPB = kBlockWarps<WPR> / WPR;
  __shared__ float red[TPB][2 * WPR];
  pdl_wait();
  pdl_trigger();
  const int team = threadIdx.x / (32 * WPR), tl = threadIdx.x % (32 * WPR);
  const size_t t = (size_t)blockIdx.x * TPB + team;
  if (t >= (size_t)a.T) return;                  // (a whole team: no barrier is left waiting)
  Team<WPR> tm{red[team], team, tl, 0};
  const int pieces = a.d / N;
  const uint4* res = reinterpret_cast<const uint4*>(static_cast<const T*>(a.residual) + t * a.d);
  uint4 r[NV];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int p = n * 32 * WPR + tl;
    r[n] = p < pieces ? res[p] : make_uint4(0u, 0u, 0u, 0u);
  }
  float y[NV][N];
  block_sum<T, WPR, NV>(a, t, tl, y);
  float rp = 1.f;
  if (a.post_w) {
    float s = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int i = 0; i < N; ++i) s = fmaf(y[n][i], y[n][i], s);
    rp = 1.f / sqrtf(tm.sum(s) / (float)a.d + a.eps);
    if (a.rstd_post && tl == 0) a.rstd_post[t] = rp;
  }
  float s = 0.f;
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int p = n * 32 * WPR + tl;
    if (p < pieces) {
      float f[N], g[N];
      if (a.post_w) {
        weights_at<N>(a.post_w, p, f);
#pragma unroll
        for (int i = 0; i < N; ++i) y[n][i] = y[n][i] * rp * f[i];
      }
      if (a.gate) {
        weights_at<N>(a.gate, p, g);
#pragma unroll
        for (int i = 0; i < N; ++i) y[n][i] *= g[i];
      }
      Piece<T>::unpack(r[n], f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        y[n][i] = a.with_block ? fmaf(a.alpha, y[n][i], f[i]) : f[i];
        s = fmaf(y[n][i], y[n][i], s);
      }
      if (a.hidden_out)
        reinterpret_cast<uint4*>(static_cast<T*>(a.hidden_out) + t * a.d)[p] = Piece<T>::pack(y[n]);
    }
  }
  if (!a.normed_out && !a.rstd_next) return;
  const float rn = 1.f / sqrtf(tm.sum(s) / (float)a.d + a.eps);
  if (a.rstd_next && tl == 0) a.rstd_next[t] = rn;
  if (!a.normed_out) return;
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int p = n * 32 * WPR + tl;
    if (p < pieces) {
      float f[N];
      weights_at<N>(a.next_w, p, f);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] *= y[n][i] * rn;
      reinterpret_cast<uint4*>(static_cast<T*>(a.normed_out) + t * a.d)[p] = Piece<T>::pack(f);
    }
  }
}

// A team walks the rows team, team + teams, ...: its threads' columns never change, so the sums over tokens stay
// with them, in shared memory (each thread's own words: with 16 columns and more of three sums in registers an SM
// had eight warps, 2048 columns, k = 4: 192 us), and leave once, as one partial row per team and sum;
// norm_join_kernel adds these in order.  Up to eight columns are kept in registers.
template <typename T, int NV>
constexpr bool kSumsInSmem = NV * Piece<T>::N > 8;

template <typename T, int WPR, int NV>
__global__ void __launch_bounds__(32 * kBlockWarps<WPR>, (NV * Piece<T>::N <= 16 ? 20 : 16) / kBlockWarps<WPR>)
    block_norm_backward_kernel(const NormArgs a, const NormGrads b, int teams) {
  constexpr int N = Piece<T>::N, TPB = kBlockWarps<WPR> / WPR;
  constexpr bool kSmem = kSumsInSmem<T, NV>;
  __shared__ float red[TPB][2 * WPR];
  __shared__ float dots[TPB][kRouteMaxK][WPR];
  extern __shared__ float4 dyn[];              // the teams' sums
  pdl_wait();
  pdl_trigger();
  const int team = threadIdx.x / (32 * WPR), tl = threadIdx.x % (32 * WPR), lane = tl & 31, wt = tl >> 5;
  const int at = blockIdx.x * TPB + team;
  if (at >= teams) return;
  Team<WPR> tm{red[team], team, tl, 0};
  const int pieces = a.d / N;
  const float inv_d = 1.f / (float)a.d;
  // sums[0]: dpost_w, [1]: dgate, [2]: dnext_w
  float4 sums[3][kSmem ? 1 : NV][kSmem ? 1 : N / 4];
  float4* mine = dyn + (size_t)team * 3 * (N / 4) * pieces;   // [3][N / 4][pieces]: a warp's words are neighbours
  if constexpr (kSmem) {
    for (int q = tl; q < 3 * (N / 4) * pieces; q += 32 * WPR) mine[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    // (a thread's words may have been cleared by another)
    if (WPR > 1) asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(32 * WPR) : "memory");
    else __syncwarp();
  } else {
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < N / 4; ++i) sums[q][n][i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  auto add = [&](int q, int n, int p, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      float4* at = kSmem ? mine + (q * (N / 4) + i) * pieces + p : &sums[q][kSmem ? 0 : n][kSmem ? 0 : i];
      float4 s = *at;
      s.x += v[4 * i];
      s.y += v[4 * i + 1];
      s.z += v[4 * i + 2];
      s.w += v[4 * i + 3];
      *at = s;
    }
  };
  for (size_t t = at; t < (size_t)a.T; t += teams) {
    float dh[NV][N], y[NV][N];
    // dh
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int p = n * 32 * WPR + tl;
      uint4 q = make_uint4(0u, 0u, 0u, 0u);
      if (b.dhidden && p < pieces) q = reinterpret_cast<const uint4*>(static_cast<const T*>(b.dhidden) + t * a.d)[p];
      Piece<T>::unpack(q, dh[n]);
    }
    if (b.dnormed) {
      const float rn = b.rstd_next[t];
      float (&h)[NV][N] = y;                     // (y is not needed yet)
      float c = 0.f;
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int p = n * 32 * WPR + tl;
#pragma unroll
        for (int i = 0; i < N; ++i) h[n][i] = 0.f;
        if (p < pieces) {
          float dn[N], w[N];
          Piece<T>::unpack(reinterpret_cast<const uint4*>(static_cast<const T*>(b.hidden) + t * a.d)[p], h[n]);
          Piece<T>::unpack(reinterpret_cast<const uint4*>(static_cast<const T*>(b.dnormed) + t * a.d)[p], dn);
          weights_at<N>(a.next_w, p, w);
          if (b.dnext_w) {
            float s[N];
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] = dn[i] * h[n][i] * rn;
            add(2, n, p, s);
          }
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float v = dn[i] * w[i];
            c = fmaf(v, h[n][i], c);
            dh[n][i] = fmaf(rn, v, dh[n][i]);
          }
        }
      }
      c = tm.sum(c) * inv_d * rn * rn * rn;
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < N; ++i) dh[n][i] = fmaf(-c, h[n][i], dh[n][i]);
    }
    if (b.dresidual)
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int p = n * 32 * WPR + tl;
        if (p < pieces) reinterpret_cast<uint4*>(static_cast<T*>(b.dresidual) + t * a.d)[p] = Piece<T>::pack(dh[n]);
      }
    if (!b.through) continue;
    if (b.need_y) block_sum<T, WPR, NV>(a, t, tl, y);
    // dz, then dy, in dh's place
    const float rp = a.post_w ? b.rstd_post[t] : 1.f;
    float c = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int p = n * 32 * WPR + tl;
      if (p < pieces) {
        float pw[N], g[N];
#pragma unroll
        for (int i = 0; i < N; ++i) dh[n][i] *= a.alpha;
        if (a.post_w) weights_at<N>(a.post_w, p, pw);
        if (a.gate) {
          weights_at<N>(a.gate, p, g);
          if (b.dgate) {
            float s[N];
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] = dh[n][i] * (a.post_w ? y[n][i] * rp * pw[i] : y[n][i]);
            add(1, n, p, s);
          }
#pragma unroll
          for (int i = 0; i < N; ++i) dh[n][i] *= g[i];
        }
        if (a.post_w) {
          if (b.dpost_w) {
            float s[N];
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] = dh[n][i] * y[n][i] * rp;
            add(0, n, p, s);
          }
#pragma unroll
          for (int i = 0; i < N; ++i) {
            dh[n][i] *= pw[i];
            c = fmaf(dh[n][i], y[n][i], c);
          }
        }
      }
    }
    if (a.post_w) {
      c = tm.sum(c) * inv_d * rp * rp;
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < N; ++i) dh[n][i] = rp * fmaf(-c, y[n][i], dh[n][i]);
    }
    if (b.dshared)
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int p = n * 32 * WPR + tl;
        if (p < pieces) reinterpret_cast<uint4*>(static_cast<T*>(b.dshared) + t * a.d)[p] = Piece<T>::pack(dh[n]);
      }
    if (!b.dexpert_out && !b.dtopk_w) continue;
    for (int j = 0; j < a.k; ++j) {
      const int s = a.slot_of[t * a.k + j];
      const bool on = (unsigned)s < (unsigned)a.S_max;
      float dot = 0.f;
      if (on) {
        const float w = b.dexpert_out ? a.topk_w[t * a.k + j] : 0.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          const int p = n * 32 * WPR + tl;
          if (p < pieces) {
            float f[N];
            if (b.dtopk_w) {
              Piece<T>::unpack(reinterpret_cast<const uint4*>(static_cast<const T*>(a.expert_out) + (size_t)s * a.d)[p], f);
#pragma unroll
              for (int i = 0; i < N; ++i) dot = fmaf(f[i], dh[n][i], dot);
            }
            if (b.dexpert_out) {
#pragma unroll
              for (int i = 0; i < N; ++i) f[i] = w * dh[n][i];
              reinterpret_cast<uint4*>(static_cast<T*>(b.dexpert_out) + (size_t)s * a.d)[p] = Piece<T>::pack(f);
            }
          }
        }
      }
      if (b.dtopk_w) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0) dots[team][j][wt] = dot;
      }
    }
    if (b.dtopk_w) {
      if (WPR > 1) asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(32 * WPR) : "memory");
      else __syncwarp();
      if (tl < a.k) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) v += dots[team][tl][w];
        b.dtopk_w[t * a.k + tl] = v;
      }
      // the next row's dots are written behind this
      if (WPR > 1) asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(32 * WPR) : "memory");
      else __syncwarp();
    }
  }
  if (!b.partial) return;
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    if (!(q == 0 ? b.dpost_w : q == 1 ? b.dgate : b.dnext_w)) continue;
    float* dst = b.partial + ((size_t)at * 3 + q) * a.d;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int p = n * 32 * WPR + tl;
      if (p < pieces)
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
          reinterpret_cast<float4*>(dst + p * N)[i] =
              kSmem ? mine[(q * (N / 4) + i) * pieces + p] : sums[q][kSmem ? 0 : n][kSmem ? 0 : i];
    }
  }
}

// Sum of the teams' partial rows: a block takes 32 columns of one sum, a warp every eighth team.
__global__ void __launch_bounds__(256) norm_join_kernel(const float* __restrict__ partial, int teams, int d,
                                                        float* d0, float* d1, float* d2) {
  __shared__ float part[8][33];
  pdl_wait();
  float* out = blockIdx.y == 0 ? d0 : blockIdx.y == 1 ? d1 : d2;
  if (!out) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < d)
#pragma unroll 8
    for (int r = w; r < teams; r += 8) s += partial[((size_t)r * 3 + blockIdx.y) * d + c];
  part[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < d) {
#pragma unroll
    for (int q = 1; q < 8; ++q) s += part[q][lane];
    out[c] = s;
  }
}

// Warps per row: as few as hold it at two pieces a thread, 16 at most.
int warps_for(int d, bool f16) {
  const int pieces = d / (f16 ? 8 : 4);
  int w = 1;
  while (w < 16 && w * 64 < pieces) w *= 2;
  return w;
}

template <typename T, typename F>
cudaError_t with_team(int d, F f) {
  using std::integral_constant;
  const int pieces = d / Piece<T>::N;
  const int w = warps_for(d, Piece<T>::N == 8);
  if (pieces <= 32) return f(integral_constant<int, 1>(), integral_constant<int, 1>());
  switch (w) {
    case 1: return f(integral_constant<int, 1>(), integral_constant<int, 2>());
    case 2: return f(integral_constant<int, 2>(), integral_constant<int, 2>());
    case 4: return f(integral_constant<int, 4>(), integral_constant<int, 2>());
    case 8: return f(integral_constant<int, 8>(), integral_constant<int, 2>());
  }
  if (pieces <= 1024) return f(integral_constant<int, 16>(), integral_constant<int, 2>());
  if (pieces <= 2048) return f(integral_constant<int, 16>(), integral_constant<int, 4>());
  if constexpr (Piece<T>::N == 4) return f(integral_constant<int, 16>(), integral_constant<int, 8>());
  return cudaErrorInvalidValue;
}

}  // namespace

// Teams of the backward pass: 20 warps for each of 152 SMs, fewer where the sums of more would not fit shared memory.
int norm_teams(int T, int d, bool f16) {
  const int w = warps_for(d, f16), per_sm = std::max(1, std::min(20 / w, 200 * 1024 / (12 * d)));
  return std::min(T, 152 * per_sm);
}

cudaError_t launch_block_norm(const NormArgs& a, bool f16, cudaStream_t s) {
  auto go = [&](auto type) {
    using T = decltype(type);
    return with_team<T>(a.d, [&](auto wpr, auto nv) -> cudaError_t {
      constexpr int W = decltype(wpr)::value, V = decltype(nv)::value, TPB = kBlockWarps<W> / W;
      return launch_k(block_norm_kernel<T, W, V>, (unsigned)((a.T + TPB - 1) / TPB), 32 * kBlockWarps<W>, 0, s, false, a);
    });
  };
  return f16 ? go(__half()) : go(float());
}

cudaError_t launch_block_norm_backward(const NormArgs& a, const NormGrads& b, bool f16, cudaStream_t s) {
  const int teams = norm_teams(a.T, a.d, f16);
  auto go = [&](auto type) {
    using T = decltype(type);
    return with_team<T>(a.d, [&](auto wpr, auto nv) -> cudaError_t {
      constexpr int W = decltype(wpr)::value, V = decltype(nv)::value, TPB = kBlockWarps<W> / W;
      auto kern = block_norm_backward_kernel<T, W, V>;
      const size_t smem = kSumsInSmem<T, V> ? (size_t)TPB * 3 * a.d * sizeof(float) : 0;
      if (smem) MOE_LAUNCH(ensure_smem_attr(reinterpret_cast<const void*>(kern)));
      return launch_k(kern, (teams + TPB - 1) / TPB, 32 * kBlockWarps<W>, smem, s, false, a, b, teams);
    });
  };
  MOE_LAUNCH(f16 ? go(__half()) : go(float()));
  if (b.partial)
    MOE_LAUNCH(launch_k(norm_join_kernel, dim3((a.d + 31) / 32, 3), 256, 0, s, true, (const float*)b.partial, teams,
                        a.d, b.dpost_w, b.dgate, b.dnext_w));
  return cudaSuccess;
}

}  // namespace moe
