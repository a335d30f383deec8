// The end of a block and the start of the next one, and its gradient:
//   y = sum_j w_j e_j + shared,  z = gate post_w y rp,  h = residual + alpha z,  n = next_w h rn,
//   rp = 1 / sqrt(mean y^2 + eps),  rn = 1 / sqrt(mean h^2 + eps)         (include/moe.h has the gradient)
//
// A team of WPR warps takes a token's row: thread i of the team has the 16-byte pieces i, i + 32 WPR, ..., NV
// of them, in registers from the first load to the last store, so that every row crosses DRAM once.  Bound by
// DRAM, (k + 3) rows a token forward and 2 k + 4 backward, and by how many rows an SM has in work: forward 16384 x 3584,
// k = 2: 116 us, 5.1 TB/s; backward 248 us, 3.8 TB/s (the time of a row's loads, sums and stores one after another).
#include "launch.h"

namespace moe {
namespace {

template <typename T>
struct Piece;                                   // 16 bytes, as pairs of 32-bit values
template <>
struct Piece<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float2 (&f)[4]) {
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
  }
  static __device__ __forceinline__ uint4 pack(const float2 (&f)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 v = __float22half2_rn(f[i]);
      u[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Piece<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& r, float2 (&f)[2]) {
    f[0] = make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
    f[1] = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
  }
  static __device__ __forceinline__ uint4 pack(const float2 (&f)[2]) {
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                      __float_as_uint(f[1].y));
  }
};

// Two 32-bit operations at a time.
__device__ __forceinline__ unsigned long long bits2(float2 v) {
  return (unsigned long long)__float_as_uint(v.y) << 32 | __float_as_uint(v.x);
}
__device__ __forceinline__ float2 float2_of(unsigned long long r) {
  return make_float2(__uint_as_float((uint32_t)r), __uint_as_float((uint32_t)(r >> 32)));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return float2_of(r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

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
  __device__ __forceinline__ void meet() const {
    // (A block has one or two such teams.  With the barrier's number in a register a block takes all 16, and an SM held four
    // blocks: 16384 x 1024, k = 2: 49 us instead of 35, the gradient 114 instead of 77.)
    if (WPR == 1) __syncwarp();
    else if (id == 0) asm volatile("bar.sync 1, %0;" ::"n"(32 * WPR) : "memory");
    else asm volatile("bar.sync 2, %0;" ::"n"(32 * WPR) : "memory");
  }
  __device__ __forceinline__ float sum(float2 two) {
    float v = two.x + two.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (WPR == 1) return v;
    float* b = red + turn * WPR;
    turn ^= 1;
    if ((tl & 31) == 0) b[tl >> 5] = v;
    meet();
    float r = b[0];
#pragma unroll
    for (int w = 1; w < WPR; ++w) r += b[w];
    return r;
  }
};

// A per-column weight at piece p.
template <int H>
__device__ __forceinline__ void weights_at(const float* w, int p, float2 (&f)[H]) {
#pragma unroll
  for (int q = 0; q < H / 2; ++q) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(w) + p * (H / 2) + q);
    f[2 * q] = make_float2(v.x, v.y);
    f[2 * q + 1] = make_float2(v.z, v.w);
  }
}

// A row on its way to L2 while the row before it is worked on: each thread asks for the lines that start with a piece
// of its own.
template <int WPR, int NV>
__device__ __forceinline__ void fetch_row(const uint4* row, int pieces, int tl) {
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int p = n * 32 * WPR + tl;
    if (p < pieces && (p & 7) == 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + p));
  }
}

template <typename T>
__device__ __forceinline__ const uint4* row_of(const void* m, size_t r, int d) {
  return reinterpret_cast<const uint4*>(static_cast<const T*>(m) + r * d);
}
template <typename T>
__device__ __forceinline__ uint4* out_of(void* m, size_t r, int d) {
  return reinterpret_cast<uint4*>(static_cast<T*>(m) + r * d);
}

// y: the weighted sum of the token's kept rows, a few of them in flight, and the shared row.
template <typename T, int WPR, int NV>
__device__ __forceinline__ void block_sum(const NormArgs& a, size_t t, int tl, float2 (&y)[NV][Piece<T>::N / 2]) {
  constexpr int H = Piece<T>::N / 2, U = kFlight<NV>;
  const int pieces = a.d / Piece<T>::N;
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int i = 0; i < H; ++i) y[n][i] = both(0.f);
  for (int j0 = 0; j0 < a.k; j0 += U) {
    uint4 raw[U][NV];
    float w[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int s = j0 + j < a.k ? a.slot_of[t * a.k + j0 + j] : -1;
      const bool on = (unsigned)s < (unsigned)a.S_max;
      w[j] = on ? a.topk_w[t * a.k + j0 + j] : 0.f;
      const uint4* row = row_of<T>(a.expert_out, on ? s : 0, a.d);
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
        float2 f[H];
        Piece<T>::unpack(raw[j][n], f);
#pragma unroll
        for (int i = 0; i < H; ++i) y[n][i] = fma2(both(w[j]), f[i], y[n][i]);
      }
  }
  if (a.shared) {
    const uint4* row = row_of<T>(a.shared, t, a.d);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int p = n * 32 * WPR + tl;
      if (p < pieces) {
        float2 f[H];
        Piece<T>::unpack(row[p], f);
#pragma unroll
        for (int i = 0; i < H; ++i) y[n][i] = make_float2(y[n][i].x + f[i].x, y[n][i].y + f[i].y);
      }
    }
  }
}

// A row asks for the one that is this far behind it, on its way to L2, while its own norm is worked on: four for each SM.
// us without, with four and with eight for each: rows of 3584, k = 2: 124, 116, 118; of 2048, k = 4, shared: 52, 48.5, 50; of
// 4096, k = 2, shared: 79, 72, 80; of 2048, k = 2: 62, 62, 57; of 1024, k = 8: 119, 120, 114; f32, of 4096, k = 2: 74, 67, 88;
// of 8192: 71, 81, 78.
constexpr int kRowsAhead = 4 * 152;

template <typename T, int WPR, int NV>
__global__ void __launch_bounds__(32 * kBlockWarps<WPR>, (NV * Piece<T>::N <= 16 ? 32 : 16) / kBlockWarps<WPR>)
    block_norm_kernel(const NormArgs a) {
  constexpr int N = Piece<T>::N, H = N / 2, TPB = kBlockWarps<WPR> / WPR;
  __shared__ float red[TPB][2 * WPR];
  pdl_wait();
  pdl_trigger();
  const int team = threadIdx.x / (32 * WPR), tl = threadIdx.x % (32 * WPR);
  const size_t t = (size_t)blockIdx.x * TPB + team;
  if (t >= (size_t)a.T) return;                  // (a whole team: no barrier is left waiting)
  Team<WPR> tm{red[team], team, tl, 0};
  const int pieces = a.d / N;
  const uint4* res = row_of<T>(a.residual, t, a.d);
  const size_t u = t + kRowsAhead;
  const bool more = u < (size_t)a.T;
  int next_slot = -1;
  if (more && (tl & 31) < a.k) next_slot = a.slot_of[u * a.k + (tl & 31)];
  uint4 r[NV];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int p = n * 32 * WPR + tl;
    r[n] = p < pieces ? res[p] : make_uint4(0u, 0u, 0u, 0u);
  }
  float2 y[NV][H];
  block_sum<T, WPR, NV>(a, t, tl, y);
  float rp = 1.f;
  if (a.post_w) {
    float2 s = both(0.f);
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int i = 0; i < H; ++i) s = fma2(y[n][i], y[n][i], s);
    rp = 1.f / sqrtf(tm.sum(s) / (float)a.d + a.eps);
    if (a.rstd_post && tl == 0) a.rstd_post[t] = rp;
  }
  float2 s = both(0.f);
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int p = n * 32 * WPR + tl;
    if (p < pieces) {
      float2 f[H];
      if (a.post_w) {
        weights_at<H>(a.post_w, p, f);
#pragma unroll
        for (int i = 0; i < H; ++i) y[n][i] = mul2(mul2(y[n][i], both(rp)), f[i]);
      }
      if (a.gate) {
        weights_at<H>(a.gate, p, f);
#pragma unroll
        for (int i = 0; i < H; ++i) y[n][i] = mul2(y[n][i], f[i]);
      }
      Piece<T>::unpack(r[n], f);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        y[n][i] = a.with_block ? fma2(both(a.alpha), y[n][i], f[i]) : f[i];
        s = fma2(y[n][i], y[n][i], s);
      }
      if (a.hidden_out) out_of<T>(a.hidden_out, t, a.d)[p] = Piece<T>::pack(y[n]);
    }
  }
  if (more) {
    fetch_row<WPR, NV>(row_of<T>(a.residual, u, a.d), pieces, tl);
    if (a.shared) fetch_row<WPR, NV>(row_of<T>(a.shared, u, a.d), pieces, tl);
    for (int j = 0; j < a.k; ++j) {
      const int s = __shfl_sync(0xffffffffu, next_slot, j);
      if ((unsigned)s < (unsigned)a.S_max) fetch_row<WPR, NV>(row_of<T>(a.expert_out, s, a.d), pieces, tl);
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
      float2 f[H];
      weights_at<H>(a.next_w, p, f);
#pragma unroll
      for (int i = 0; i < H; ++i) f[i] = mul2(f[i], mul2(y[n][i], both(rn)));
      out_of<T>(a.normed_out, t, a.d)[p] = Piece<T>::pack(f);
    }
  }
}

// A team walks the rows team, team + teams, ...: its threads' columns never change, so the sums over tokens stay
// with them, in shared memory (each thread's own words: in registers, with 16 columns and more a thread, an SM had eight
// warps, 2048 columns, k = 4: 192 us, not 115), and leave once, as one partial row per team and sum; norm_join_kernel adds
// these in order.  Up to eight columns are kept in registers.  There are two sums: with G = sum_t rp dh . y,
//   dgate = alpha post_w . G,   dpost_w = alpha gate . G,        and   dnext_w = sum_t rn dnormed . h.
//
// Warps of a row pass on an SM: 24, and of rows that take 16 warps two teams where a thread has two pieces of a row (with 64
// registers; four pieces need more).  us with 16, 24, 32: f16, 512 columns, k = 4: 125, 125, 146; 1024, k = 2: 85, 77, 81;
// 1024, k = 8: 376, 364, 391; 2048, k = 4: 127, 125, 138; 2048, k = 2: 147, 127, 128; 3584: 296, 248, 234; 4096: 175, 159, 169;
// f32, 1024: 70, 60, 63; 2048: 221, 219, 228.  One team or two of 16 warps: f16, 8192: 189, 155; f32, 4096: 146, 117; f32, 8192
// (four pieces): 150, 174.
template <int WPR, int NV>
constexpr int kBackWarps = WPR < 16 ? 24 : NV == 2 ? 32 : 16;
template <typename T, int NV>
constexpr bool kSumsInSmem = NV * Piece<T>::N > 8;

template <typename T, int WPR, int NV>
__global__ void __launch_bounds__(32 * kBlockWarps<WPR>, kBackWarps<WPR, NV> / kBlockWarps<WPR>)
    block_norm_backward_kernel(const NormArgs a, const NormGrads b, int teams) {
  constexpr int N = Piece<T>::N, H = N / 2, TPB = kBlockWarps<WPR> / WPR;
  constexpr bool kSmem = kSumsInSmem<T, NV>;
  __shared__ float red[TPB][2 * WPR];
  __shared__ float dots[TPB][kRouteMaxK][WPR];
  extern __shared__ float4 dyn[];                // the teams' sums
  pdl_wait();
  pdl_trigger();
  const int team = threadIdx.x / (32 * WPR), tl = threadIdx.x % (32 * WPR), lane = tl & 31, wt = tl >> 5;
  const int at = blockIdx.x * TPB + team;
  if (at >= teams) return;
  Team<WPR> tm{red[team], team, tl, 0};
  const int pieces = a.d / N;
  const float inv_d = 1.f / (float)a.d;
  // sums[0]: G, [1]: dnext_w
  float4 sums[2][kSmem ? 1 : NV][kSmem ? 1 : H / 2];
  float4* mine = dyn + (size_t)team * 2 * (H / 2) * pieces;   // [2][H / 2][pieces]: a warp's words are neighbours
  if constexpr (kSmem) {
    for (int q = tl; q < 2 * (H / 2) * pieces; q += 32 * WPR) mine[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    tm.meet();                                   // (a thread's words may have been cleared by another)
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < H / 2; ++i) sums[q][n][i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // += u v f
  auto add = [&](int q, int n, int p, const float2 (&u)[H], const float2 (&v)[H], float f) {
#pragma unroll
    for (int i = 0; i < H / 2; ++i) {
      float4* to = kSmem ? mine + (q * (H / 2) + i) * pieces + p : &sums[q][kSmem ? 0 : n][kSmem ? 0 : i];
      const float4 s = *to;
      const float2 x = fma2(mul2(u[2 * i], both(f)), v[2 * i], make_float2(s.x, s.y));
      const float2 z = fma2(mul2(u[2 * i + 1], both(f)), v[2 * i + 1], make_float2(s.z, s.w));
      *to = make_float4(x.x, x.y, z.x, z.y);
    }
  };
  for (size_t t = at; t < (size_t)a.T; t += teams) {
    float2 dh[NV][H], y[NV][H];
    // the next row's inputs: with two to five rows an SM in work, each row waited for DRAM at every step
    const size_t u = t + teams;
    const bool more = u < (size_t)a.T;
    int next_slot = -1;
    if (more) {
      if (lane < a.k) next_slot = a.slot_of[u * a.k + lane];
      for (const void* m : {b.dhidden, b.dnormed, b.dnormed ? b.hidden : nullptr, a.shared})
        if (m) fetch_row<WPR, NV>(row_of<T>(m, u, a.d), pieces, tl);
    }
    // dh
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int p = n * 32 * WPR + tl;
      uint4 q = make_uint4(0u, 0u, 0u, 0u);
      if (b.dhidden && p < pieces) q = row_of<T>(b.dhidden, t, a.d)[p];
      Piece<T>::unpack(q, dh[n]);
    }
    if (b.dnormed) {
      const float rn = b.rstd_next[t];
      float2 (&h)[NV][H] = y;                    // (y is not needed yet)
      float2 c = both(0.f);
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int p = n * 32 * WPR + tl;
#pragma unroll
        for (int i = 0; i < H; ++i) h[n][i] = both(0.f);
        if (p < pieces) {
          float2 dn[H], w[H];
          Piece<T>::unpack(row_of<T>(b.hidden, t, a.d)[p], h[n]);
          Piece<T>::unpack(row_of<T>(b.dnormed, t, a.d)[p], dn);
          weights_at<H>(a.next_w, p, w);
          if (b.dnext_w) add(1, n, p, h[n], dn, rn);
#pragma unroll
          for (int i = 0; i < H; ++i) {
            const float2 v = mul2(dn[i], w[i]);
            c = fma2(v, h[n][i], c);
            dh[n][i] = fma2(both(rn), v, dh[n][i]);
          }
        }
      }
      const float f = -tm.sum(c) * inv_d * rn * rn * rn;
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < H; ++i) dh[n][i] = fma2(both(f), h[n][i], dh[n][i]);
    }
    if (b.dresidual)
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int p = n * 32 * WPR + tl;
        if (p < pieces) out_of<T>(b.dresidual, t, a.d)[p] = Piece<T>::pack(dh[n]);
      }
    if (!b.through) continue;
    for (int j = 0; more && j < a.k; ++j) {
      const int s = __shfl_sync(0xffffffffu, next_slot, j);
      if ((unsigned)s < (unsigned)a.S_max) fetch_row<WPR, NV>(row_of<T>(a.expert_out, s, a.d), pieces, tl);
    }
    if (b.need_y) block_sum<T, WPR, NV>(a, t, tl, y);
    // dz, then dy, in dh's place
    const float rp = a.post_w ? b.rstd_post[t] : 1.f;
    float2 c = both(0.f);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int p = n * 32 * WPR + tl;
      if (p < pieces) {
        if (b.dgate || b.dpost_w) add(0, n, p, dh[n], y[n], rp);
        float2 w[H], f[H];
#pragma unroll
        for (int i = 0; i < H; ++i) w[i] = both(a.alpha);
        if (a.gate) {
          weights_at<H>(a.gate, p, f);
#pragma unroll
          for (int i = 0; i < H; ++i) w[i] = mul2(w[i], f[i]);
        }
        if (a.post_w) {
          weights_at<H>(a.post_w, p, f);
#pragma unroll
          for (int i = 0; i < H; ++i) w[i] = mul2(w[i], f[i]);
        }
#pragma unroll
        for (int i = 0; i < H; ++i) {
          dh[n][i] = mul2(dh[n][i], w[i]);
          if (a.post_w) c = fma2(dh[n][i], y[n][i], c);
        }
      }
    }
    if (a.post_w) {
      const float f = -tm.sum(c) * inv_d * rp * rp * rp;
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < H; ++i) dh[n][i] = fma2(both(f), y[n][i], mul2(dh[n][i], both(rp)));
    }
    if (b.dshared)
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int p = n * 32 * WPR + tl;
        if (p < pieces) out_of<T>(b.dshared, t, a.d)[p] = Piece<T>::pack(dh[n]);
      }
    if (!b.dexpert_out && !b.dtopk_w) continue;
    for (int j = 0; j < a.k; ++j) {
      const int s = a.slot_of[t * a.k + j];
      const bool on = (unsigned)s < (unsigned)a.S_max;
      float2 dot = both(0.f);
      if (on) {
        const float w = b.dexpert_out ? a.topk_w[t * a.k + j] : 0.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          const int p = n * 32 * WPR + tl;
          if (p < pieces) {
            float2 f[H];
            if (b.dtopk_w) {
              Piece<T>::unpack(row_of<T>(a.expert_out, s, a.d)[p], f);
#pragma unroll
              for (int i = 0; i < H; ++i) dot = fma2(f[i], dh[n][i], dot);
            }
            if (b.dexpert_out) {
#pragma unroll
              for (int i = 0; i < H; ++i) f[i] = mul2(both(w), dh[n][i]);
              out_of<T>(b.dexpert_out, s, a.d)[p] = Piece<T>::pack(f);
            }
          }
        }
      }
      if (b.dtopk_w) {
        float v = dot.x + dot.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) dots[team][j][wt] = v;
      }
    }
    if (b.dtopk_w) {
      tm.meet();
      if (tl < a.k) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) v += dots[team][tl][w];
        b.dtopk_w[t * a.k + tl] = v;
      }
      tm.meet();                                 // the next row's dots are written behind this
    }
  }
  if (!b.partial) return;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (!(q == 0 ? b.dpost_w || b.dgate : b.dnext_w != nullptr)) continue;
    float* dst = b.partial + ((size_t)at * 2 + q) * a.d;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int p = n * 32 * WPR + tl;
      if (p < pieces)
#pragma unroll
        for (int i = 0; i < H / 2; ++i)
          reinterpret_cast<float4*>(dst + p * N)[i] =
              kSmem ? mine[(q * (H / 2) + i) * pieces + p] : sums[q][kSmem ? 0 : n][kSmem ? 0 : i];
    }
  }
}

// Sum of the teams' partial rows: a block takes 32 columns of one sum, a warp every 32nd team.
__global__ void __launch_bounds__(1024) norm_join_kernel(const float* __restrict__ partial, int teams, int d, float alpha,
                                                         const float* gate, const float* post_w, float* dpost_w,
                                                         float* dgate, float* dnext_w) {
  __shared__ float part[32][33];
  pdl_wait();
  const int sum = blockIdx.y;
  if (!(sum == 0 ? dpost_w || dgate : dnext_w != nullptr)) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < d)
#pragma unroll 4
    for (int r = w; r < teams; r += 32) s += partial[((size_t)r * 2 + sum) * d + c];
  part[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < d) {
#pragma unroll
    for (int q = 1; q < 32; ++q) s += part[q][lane];
    if (sum == 1) {
      dnext_w[c] = s;
    } else {
      s *= alpha;
      if (dgate) dgate[c] = post_w ? s * post_w[c] : s;
      if (dpost_w) dpost_w[c] = gate ? s * gate[c] : s;
    }
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

// Teams of the backward pass: kBackWarps for each of 152 SMs, fewer where the sums of more would not fit shared memory.
int norm_teams(int T, int d, bool f16) {
  const int w = warps_for(d, f16), pieces = d / (f16 ? 8 : 4);
  const int warps = w < 16 ? kBackWarps<1, 1> : pieces <= 1024 ? kBackWarps<16, 2> : kBackWarps<16, 4>;
  return std::min(T, 152 * std::max(1, std::min(warps / w, 200 * 1024 / (8 * d))));
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
      const size_t smem = kSumsInSmem<T, V> ? (size_t)TPB * 2 * a.d * sizeof(float) : 0;
      if (smem) MOE_LAUNCH(ensure_smem_attr(reinterpret_cast<const void*>(kern)));
      return launch_k(kern, (teams + TPB - 1) / TPB, 32 * kBlockWarps<W>, smem, s, false, a, b, teams);
    });
  };
  MOE_LAUNCH(f16 ? go(__half()) : go(float()));
  if (b.partial)
    MOE_LAUNCH(launch_k(norm_join_kernel, dim3((a.d + 31) / 32, 2), 1024, 0, s, true, (const float*)b.partial, teams,
                        a.d, a.alpha, a.gate, a.post_w, b.dpost_w, b.dgate, b.dnext_w));
  return cudaSuccess;
}

}  // namespace moe
