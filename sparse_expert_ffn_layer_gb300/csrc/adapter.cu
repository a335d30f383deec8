// Low-rank adapters of many requests beside a shared projection, and the gradient of their
// input: for the slots s of adapter n (token t = perm[s]),
//
//   h_s = x_t P_n           [r]      (forward: P = A, Q = B;  gradient: P = B^T, Q = A^T)
//   y_t = base_t + scale_n h_s Q_n   (base may be absent)
//
// Bound by DRAM: x and base are read and y written once, the weights of the adapters in use come
// once from DRAM and then from L2; 4 r operations per token and column pair stay below the
// tensor rate for r <= 128.
//
// One launch does both products.  A cluster of eight blocks takes a tile of rows of one adapter;
// each block multiplies its eighth of the input columns (so a single token's weights are pulled
// by eight SMs), the partial h are summed over the cluster through distributed shared memory in
// rank order (no atomics: equal calls give equal bits), each block receives the whole h and
// multiplies it into its eighth of the output columns.  Both products run through one ring of
// asynchronous 128-byte-wide chunks, so the first output chunks (base and Q) load while h is
// being exchanged.
//
// f16: h keeps 22 bits.  It is scaled by a power of two per row and split into two f16 parts,
// and the second product adds both (h rounded to one f16 would cost as much accuracy as the
// rounding of y does, and could overflow).  f32: fused multiply-adds on the CUDA cores.
//
// Rows per tile: 64 for long runs of one adapter (weights read from L2 once per 64 rows, the
// four warps split the rows), 16 for short ones (the warps split the columns of a chunk).
#include <cooperative_groups.h>

#include <algorithm>

#include "launch.h"
#include "mma.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kCl = 8;                  // blocks per cluster
constexpr int kRowB = 144;              // bytes per 128-byte chunk row in shared memory
constexpr int kMaxGroups = 1024;

template <typename T>
struct Elt {
  static constexpr int V = 16 / sizeof(T);        // elements per 16 bytes
  static constexpr int C = 128 / sizeof(T);       // columns per chunk
};

// Shared-memory plan of one block.
template <typename T, int MT, int R>
struct Plan {
  static constexpr int C = Elt<T>::C, V = Elt<T>::V;
  static constexpr int kLdR = R + V;                               // rows of R elements
  static constexpr int kLdC = kRowB / (int)sizeof(T);              // rows of C elements
  static constexpr int kW = (C * kLdR > R * kLdC ? C * kLdR : R * kLdC) * (int)sizeof(T);
  static constexpr int kStage = MT * kRowB + kW;
  static constexpr int kStages = MT == 64 ? (R >= 128 ? 3 : 4) : (R >= 128 ? 4 : R >= 64 ? 6 : 8);
  static constexpr int kPart = 4 * 16 * R * 4;                     // partial h, f32
  static constexpr int kH = sizeof(T) == 2 ? MT * (R + 8) * 2 * 2  // h: two f16 parts
                                           : MT * (R + 4) * 4;     // or f32
  static constexpr int kOffPart = kStages * kStage;
  static constexpr int kOffH = kOffPart + kPart;
  static constexpr int kOffMult = kOffH + kH;
  static constexpr int kOffTok = kOffMult + MT * 4;
  static constexpr int kOffTab = kOffTok + MT * 4;                 // offsets and tile starts
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// Group boundaries as the kernels use them, and the tile starts.  bound[n] = the largest of
// offsets[0 .. n], clamped to [0, S_max]: runs never overlap and no slot lies outside the
// buffers, whatever the offsets say.  start[n] = number of tiles of the groups before n.
// All threads of the block; N <= 1024.
__device__ __forceinline__ void group_table(const int32_t* __restrict__ offsets, int N, int S_max,
                                            int MT, int* bound, int* start, int* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int per = (N + 1 + kThreads - 1) / kThreads;
  for (int i = tid; i <= N; i += kThreads) bound[i] = min(max(offsets[i], 0), S_max);
  __syncthreads();
  const int i0 = min(tid * per, N + 1), i1 = min(i0 + per, N + 1);
  // inclusive running maximum
  int m = 0;
  for (int i = i0; i < i1; ++i) m = max(m, bound[i]);
  int mm = m;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, mm, o);
    if (lane >= o) mm = max(mm, v);
  }
  if (lane == 31) scratch[w] = mm;
  int run = __shfl_up_sync(0xffffffffu, mm, 1);
  if (lane == 0) run = 0;
  __syncthreads();
  for (int q = 0; q < w; ++q) run = max(run, scratch[q]);
  for (int i = i0; i < i1; ++i) {
    run = max(run, bound[i]);
    bound[i] = run;
  }
  __syncthreads();
  // exclusive sum of tile counts
  int c = 0;
  for (int i = i0; i < min(i1, N); ++i) c += (bound[i + 1] - bound[i] + MT - 1) / MT;
  int s = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += v;
  }
  if (lane == 31) scratch[8 + w] = s;
  __syncthreads();
  s -= c;
  for (int q = 0; q < w; ++q) s += scratch[8 + q];
  for (int i = i0; i < i1; ++i) {
    start[i] = s;
    if (i < N) s += (bound[i + 1] - bound[i] + MT - 1) / MT;
  }
  __syncthreads();
}

// Checks every offset and perm entry and writes the status word (one block, beside the work).
__device__ void check_indices(const int32_t* __restrict__ perm, const int32_t* __restrict__ offsets,
                              int N, int S_max, int T, int* status) {
  bool bad = false;
  for (int i = threadIdx.x; i <= N; i += kThreads) {
    const int v = offsets[i];
    bad |= v < 0 || v > S_max || (i > 0 && v < offsets[i - 1]);
  }
  const int S = min(max(offsets[N], 0), S_max);
  for (int s = min(max(offsets[0], 0), S_max) + threadIdx.x; s < S; s += kThreads)
    bad |= (unsigned)perm[s] >= (unsigned)T;
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) *status = any ? kErrBounds : kOk;
}

struct AdapterArgs {
  const void* x;             // [T, dk]
  const void* P;             // kT ? [N, r, dk] : [N, dk, r]
  const void* Q;             // kT ? [N, dn, r] : [N, r, dn]
  const void* base;          // [T, dn] or null
  void* y;                   // [T, dn]
  float* hidden;             // [S_max, r] or null
  const float* scale;        // [N]
  const int32_t* perm;
  const int32_t* offsets;
  int* status;
  int T, dk, dn, r, N, S_max;
};

template <typename T, int MT, int R, bool kT>
__global__ void __launch_bounds__(kThreads) adapter_kernel(const AdapterArgs a) {
  using PL = Plan<T, MT, R>;
  constexpr int C = PL::C, V = PL::V, NS = PL::kStages;
  constexpr int kRowGroups = MT / 16;             // warps along rows
  constexpr int WK = 4 / kRowGroups;              // warps along a chunk's columns
  constexpr bool kHalf = sizeof(T) == 2;
  extern __shared__ __align__(128) uint8_t sm[];
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank();
  const int cid = blockIdx.x / kCl, ncl = gridDim.x / kCl - 1;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (cid == ncl) {                               // the last cluster checks the indices
    if (rank == 0) check_indices(a.perm, a.offsets, a.N, a.S_max, a.T, a.status);
    return;
  }
  float* part = reinterpret_cast<float*>(sm + PL::kOffPart);      // [WK][MT][R]
  __half* hhi = reinterpret_cast<__half*>(sm + PL::kOffH);        // [MT][R + 8]
  __half* hlo = hhi + MT * (R + 8);
  float* hf = reinterpret_cast<float*>(sm + PL::kOffH);           // f32: [MT][R + 4]
  float* mult = reinterpret_cast<float*>(sm + PL::kOffMult);
  int* tok = reinterpret_cast<int*>(sm + PL::kOffTok);
  int* bound = reinterpret_cast<int*>(sm + PL::kOffTab);
  int* start = bound + a.N + 1;
  int* scratch = start + a.N + 1;
  group_table(a.offsets, a.N, a.S_max, MT, bound, start, scratch);
  const int ntiles = start[a.N];

  const int ck = (a.dk + C - 1) / C, cn = (a.dn + C - 1) / C;
  const int k0 = (int)((long long)ck * rank / kCl), k1 = (int)((long long)ck * (rank + 1) / kCl);
  const int n0 = (int)((long long)cn * rank / kCl), n1 = (int)((long long)cn * (rank + 1) / kCl);
  const int nk = k1 - k0, total = nk + n1 - n0;
  const T* X = static_cast<const T*>(a.x);
  const T* base = static_cast<const T*>(a.base);
  T* Y = static_cast<T*>(a.y);
  const int wr = (w % kRowGroups) * 16, wk = w / kRowGroups;

  for (int tile = cid; tile < ntiles; tile += ncl) {
    // the group of this tile: the last n with start[n] <= tile
    int n = 0;
    for (int step = 512; step > 0; step >>= 1)
      if (n + step < a.N && start[n + step] <= tile) n += step;
    // groups without tiles share their start with the next one: the last is the one that has it
    const int s0 = bound[n] + (tile - start[n]) * MT;
    const int rows = min(MT, bound[n + 1] - s0);
    if (tid < MT) {
      int t = tid < rows ? a.perm[s0 + tid] : -1;
      if ((unsigned)t >= (unsigned)a.T) t = -1;
      tok[tid] = t;
    }
    __syncthreads();
    const T* P = static_cast<const T*>(a.P) + (size_t)n * a.dk * a.r;
    const T* Q = static_cast<const T*>(a.Q) + (size_t)n * a.dn * a.r;

    // chunk c of the sequence: nk input chunks (x, P), then the output chunks (base, Q)
    auto load = [&](int c) {
      uint8_t* st = sm + (c % NS) * PL::kStage;
      const bool first = c < nk;
      const int col0 = (first ? k0 + c : n0 + c - nk) * C;
      const int d = first ? a.dk : a.dn;
      const T* rowsrc = first ? X : base;
      if (rowsrc) {
        for (int i = tid; i < MT * 8; i += kThreads) {
          const int row = i >> 3, col = col0 + (i & 7) * V;
          const bool on = tok[row] >= 0 && col < d;
          cp_async16(st + row * kRowB + (i & 7) * 16, rowsrc + (on ? (size_t)tok[row] * d + col : 0), on);
        }
      }
      uint8_t* ws = st + MT * kRowB;
      const T* W = first ? P : Q;
      if (first != kT) {                          // rows of the chunk's columns, r wide
        constexpr int RV = R / V;
        for (int i = tid; i < C * RV; i += kThreads) {
          const int row = i / RV, col = (i % RV) * V;
          const bool on = col0 + row < d && col < a.r;
          cp_async16(ws + (row * PL::kLdR + col) * sizeof(T),
                     W + (on ? (size_t)(col0 + row) * a.r + col : 0), on);
        }
      } else {                                    // r rows, the chunk's columns wide
        for (int i = tid; i < R * 8; i += kThreads) {
          const int row = i >> 3, col = col0 + (i & 7) * V;
          const bool on = row < a.r && col < d;
          cp_async16(ws + row * kRowB + (i & 7) * 16, W + (on ? (size_t)row * d + col : 0), on);
        }
      }
    };
    for (int c = 0; c < NS - 1; ++c) {
      if (c < total) load(c);
      cp_async_commit();
    }
    auto advance = [&](int c) {                   // chunk c is ready, the next load is issued
      cp_async_wait<NS - 2>();
      __syncthreads();
      if (c + NS - 1 < total) load(c + NS - 1);
      cp_async_commit();
    };

    // ---- first product: partial h of this block's input columns
    if constexpr (kHalf) {
      float acc[R / 8][4];
#pragma unroll
      for (int i = 0; i < R / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
      for (int c = 0; c < nk; ++c) {
        advance(c);
        const __half* xs = reinterpret_cast<const __half*>(sm + (c % NS) * PL::kStage);
        const __half* ps = xs + MT * PL::kLdC;
#pragma unroll
        for (int kk = 0; kk < 4 / WK; ++kk) {
          const int k = (kk * WK + wk) * 16;
          uint32_t fa[4];
          frag_a(fa, xs + wr * PL::kLdC + k, PL::kLdC, lane);
#pragma unroll
          for (int j = 0; j < R / 16; ++j) {
            uint32_t fb[4];
            if (kT)
              frag_b_nk(fb, ps + j * 16 * PL::kLdC + k, PL::kLdC, lane);
            else
              frag_b_kn(fb, ps + k * PL::kLdR + j * 16, PL::kLdR, lane);
            mma16816(acc[2 * j], fa, fb[0], fb[1]);
            mma16816(acc[2 * j + 1], fa, fb[2], fb[3]);
          }
        }
      }
      float* p = part + ((size_t)wk * MT + wr + (lane >> 2)) * R + 2 * (lane & 3);
#pragma unroll
      for (int j = 0; j < R / 8; ++j) {
        *reinterpret_cast<float2*>(p + 8 * j) = make_float2(acc[j][0], acc[j][1]);
        *reinterpret_cast<float2*>(p + 8 * R + 8 * j) = make_float2(acc[j][2], acc[j][3]);
      }
    } else {
      // f32: thread (row, column group) of the 16 x R block; sixteen rows, eight threads each
      constexpr int CPT = R / 8;
      const int row = tid >> 3, c0 = tid & 7;
      float acc[CPT];
#pragma unroll
      for (int j = 0; j < CPT; ++j) acc[j] = 0.f;
      for (int c = 0; c < nk; ++c) {
        advance(c);
        const float* xs = reinterpret_cast<const float*>(sm + (c % NS) * PL::kStage);
        const float* ps = xs + MT * PL::kLdC;
#pragma unroll 4
        for (int k = 0; k < C; ++k) {
          const float xv = xs[row * PL::kLdC + k];
#pragma unroll
          for (int j = 0; j < CPT; ++j)
            acc[j] = fmaf(xv, kT ? ps[(c0 + 8 * j) * PL::kLdC + k] : ps[k * PL::kLdR + c0 + 8 * j],
                          acc[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < CPT; ++j) part[row * R + c0 + 8 * j] = acc[j];
    }
    if (kHalf && WK > 1) {                        // the warps' shares of the block
      __syncthreads();
      for (int i = tid; i < MT * R; i += kThreads) {
        float v = part[i];
#pragma unroll
        for (int q = 1; q < WK; ++q) v += part[q * MT * R + i];
        part[i] = v;
      }
    }
    cl.sync();

    // ---- h: this block sums rows rank * MT / 8 .. over the cluster and gives them to all
    {
      constexpr int CPT = R / 8;                  // eight threads per row, CPT columns each
      constexpr int RO = MT / kCl;
      const int row = rank * RO + (tid >> 3), c0 = (tid & 7) * CPT;
      if ((tid >> 3) < RO) {
        float v[CPT];
#pragma unroll
        for (int j = 0; j < CPT; ++j) v[j] = 0.f;
#pragma unroll
        for (int q = 0; q < kCl; ++q) {
          const float* src = cl.map_shared_rank(part, q) + row * R + c0;
#pragma unroll
          for (int j = 0; j < CPT; j += 2) {
            const float2 u = *reinterpret_cast<const float2*>(src + j);
            v[j] += u.x;
            v[j + 1] += u.y;
          }
        }
        if (a.hidden && row < rows) {
          float* dst = a.hidden + (size_t)(s0 + row) * a.r;
#pragma unroll
          for (int j = 0; j < CPT; ++j)
            if (c0 + j < a.r) dst[c0 + j] = v[j];
        }
        const float sc = a.scale[n];
        if constexpr (kHalf) {
          float m = 0.f;
          bool odd = false;
#pragma unroll
          for (int j = 0; j < CPT; ++j) {
            m = fmaxf(m, fabsf(v[j]));
            odd |= !isfinite(v[j]);
          }
          const unsigned grp = 0xffu << (lane & 24);
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(grp, m, o));
          odd = (__ballot_sync(grp, odd) & grp) != 0;
          const int e = odd ? 0 : scale_exp(m);
          const float inv = exp2_int(-e);
          __half2 hi[CPT / 2], lo[CPT / 2];
#pragma unroll
          for (int j = 0; j < CPT; j += 2) {
            split_f16(v[j] * inv, hi[j / 2].x, lo[j / 2].x);
            split_f16(v[j + 1] * inv, hi[j / 2].y, lo[j / 2].y);
          }
          const float mu = sc * exp2_int(e);
          for (int q = 0; q < kCl; ++q) {
            __half* dh = cl.map_shared_rank(hhi, q) + row * (R + 8) + c0;
            __half* dl = cl.map_shared_rank(hlo, q) + row * (R + 8) + c0;
#pragma unroll
            for (int j = 0; j < CPT / 2; ++j) {
              reinterpret_cast<__half2*>(dh)[j] = hi[j];
              reinterpret_cast<__half2*>(dl)[j] = lo[j];
            }
            if ((tid & 7) == 0) cl.map_shared_rank(mult, q)[row] = mu;
          }
        } else {
          for (int q = 0; q < kCl; ++q) {
            float* dh = cl.map_shared_rank(hf, q) + row * (R + 4) + c0;
#pragma unroll
            for (int j = 0; j < CPT; j += 2)
              *reinterpret_cast<float2*>(dh + j) = make_float2(v[j], v[j + 1]);
            if ((tid & 7) == 0) cl.map_shared_rank(mult, q)[row] = sc;
          }
        }
      }
    }
    cl.sync();

    // ---- second product: this block's output columns
    if constexpr (kHalf) {
      constexpr int NT = 8 / WK;                  // 8-column tiles of a chunk per warp
      const int wc = wk * NT * 8;
      uint32_t fh[R / 16][4], fl[R / 16][4];
#pragma unroll
      for (int k = 0; k < R / 16; ++k) {
        frag_a(fh[k], hhi + wr * (R + 8) + k * 16, R + 8, lane);
        frag_a(fl[k], hlo + wr * (R + 8) + k * 16, R + 8, lane);
      }
      const int g = lane >> 2, q2 = 2 * (lane & 3);
      const float m0 = mult[wr + g], m1 = mult[wr + g + 8];
      for (int c = nk; c < total; ++c) {
        advance(c);
        __half* bs = reinterpret_cast<__half*>(sm + (c % NS) * PL::kStage);
        const __half* qs = bs + MT * PL::kLdC;
        float acc[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll
        for (int k = 0; k < R / 16; ++k)
#pragma unroll
          for (int j = 0; j < NT / 2; ++j) {
            uint32_t fb[4];
            if (kT)
              frag_b_nk(fb, qs + (wc + j * 16) * PL::kLdR + k * 16, PL::kLdR, lane);
            else
              frag_b_kn(fb, qs + k * 16 * PL::kLdC + wc + j * 16, PL::kLdC, lane);
            mma16816(acc[2 * j], fl[k], fb[0], fb[1]);
            mma16816(acc[2 * j + 1], fl[k], fb[2], fb[3]);
            mma16816(acc[2 * j], fh[k], fb[0], fb[1]);
            mma16816(acc[2 * j + 1], fh[k], fb[2], fb[3]);
          }
        // base + scale * sum, rounded once, in place; then 16-byte rows out
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          __half2* b0 = reinterpret_cast<__half2*>(bs + (wr + g) * PL::kLdC + wc + 8 * j + q2);
          __half2* b1 = reinterpret_cast<__half2*>(bs + (wr + g + 8) * PL::kLdC + wc + 8 * j + q2);
          float2 u = make_float2(0.f, 0.f), v = u;
          if (base) {
            u = __half22float2(*b0);
            v = __half22float2(*b1);
          }
          *b0 = __floats2half2_rn(fmaf(m0, acc[j][0], u.x), fmaf(m0, acc[j][1], u.y));
          *b1 = __floats2half2_rn(fmaf(m1, acc[j][2], v.x), fmaf(m1, acc[j][3], v.y));
        }
        __syncwarp();
        const int col0 = (n0 + c - nk) * C;
#pragma unroll
        for (int i = lane; i < 16 * NT; i += 32) {
          const int row = wr + i / NT, cc = wc + (i % NT) * 8;
          if (tok[row] >= 0 && col0 + cc < a.dn)
            *reinterpret_cast<uint4*>(Y + (size_t)tok[row] * a.dn + col0 + cc) =
                *reinterpret_cast<const uint4*>(bs + row * PL::kLdC + cc);
        }
      }
    } else {
      const int row = tid >> 3, c0 = (tid & 7) * 4;       // four columns of a chunk per thread
      const float mu = mult[row];
      const int t = tok[row];
      for (int c = nk; c < total; ++c) {
        advance(c);
        const float* bs = reinterpret_cast<const float*>(sm + (c % NS) * PL::kStage);
        const float* qs = bs + MT * PL::kLdC;
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int k = 0; k < R; ++k) {
          const float hv = hf[row * (R + 4) + k];
          if (kT) {
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = fmaf(hv, qs[(c0 + j) * PL::kLdR + k], acc[j]);
          } else {
            const float4 q = load4(qs + k * PL::kLdC + c0);
            acc[0] = fmaf(hv, q.x, acc[0]);
            acc[1] = fmaf(hv, q.y, acc[1]);
            acc[2] = fmaf(hv, q.z, acc[2]);
            acc[3] = fmaf(hv, q.w, acc[3]);
          }
        }
        const int col = (n0 + c - nk) * C + c0;
        if (t >= 0 && col < a.dn) {
          float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
          if (base) u = load4(bs + row * PL::kLdC + c0);
          u.x = fmaf(mu, acc[0], u.x);
          u.y = fmaf(mu, acc[1], u.y);
          u.z = fmaf(mu, acc[2], u.z);
          u.w = fmaf(mu, acc[3], u.w);
          *reinterpret_cast<float4*>(Y + (size_t)t * a.dn + col) = u;
        }
      }
    }
    cp_async_wait<0>();
    __syncthreads();                              // tok and the ring are free for the next tile
  }
}

template <typename T, int MT, int R, bool kT>
cudaError_t launch_one(const AdapterArgs& a, int sms, cudaStream_t s) {
  auto kern = adapter_kernel<T, MT, R, kT>;
  MOE_LAUNCH(ensure_smem_attr(reinterpret_cast<const void*>(kern)));
  const long long most = (long long)a.S_max / MT + std::min(a.N, a.S_max);   // tiles at most
  const int ncl = (int)std::min<long long>(most, std::max(1, sms * 4 / kCl));
  const size_t smem = Plan<T, MT, R>::kOffTab + sizeof(int) * (2 * ((size_t)a.N + 1) + 16);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((ncl + 1) * kCl);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCl;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, a);
  if (err == cudaSuccess) launch_counter().fetch_add(1, std::memory_order_relaxed);
  return err;
}

template <typename T, int MT, bool kT>
cudaError_t launch_rank(const AdapterArgs& a, int sms, cudaStream_t s) {
  if (a.r <= 16) return launch_one<T, MT, 16, kT>(a, sms, s);
  if (a.r <= 32) return launch_one<T, MT, 32, kT>(a, sms, s);
  if (a.r <= 64) return launch_one<T, MT, 64, kT>(a, sms, s);
  return launch_one<T, MT, 128, kT>(a, sms, s);
}

}  // namespace

cudaError_t launch_adapter(const void* x, const void* P, const void* Q, const void* base, void* y,
                           float* hidden, const float* scale, const int32_t* perm,
                           const int32_t* offsets, int* status, int dtype_f16, bool transposed,
                           int T, int dk, int dn, int r, int N, int S_max, cudaStream_t s) {
  int dev = 0, sms = 0;
  MOE_LAUNCH(cudaGetDevice(&dev));
  MOE_LAUNCH(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  const AdapterArgs a{x, P, Q, base, y, hidden, scale, perm, offsets, status, T, dk, dn, r, N, S_max};
  if (!dtype_f16)
    return transposed ? launch_rank<float, 16, true>(a, sms, s) : launch_rank<float, 16, false>(a, sms, s);
  const bool tall = S_max > 32LL * std::min(N, S_max);
  if (tall)
    return transposed ? launch_rank<__half, 64, true>(a, sms, s) : launch_rank<__half, 64, false>(a, sms, s);
  return transposed ? launch_rank<__half, 16, true>(a, sms, s) : launch_rank<__half, 16, false>(a, sms, s);
}

}  // namespace moe
