// Gradients around the gate and the adapters: products summed over token rows (weights'
// gradients), the tokens' gradient through the gate, and the combine's gradient.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "groups.cuh"
#include "launch.h"
#include "mma.cuh"

namespace moe {
namespace {

// ---------------------------------------------------------------- sums over rows
// G[n][i][j] = scale_n sum_s x[t(s)][i] h[s][j] over the rows s of group n, in 32 bits.
//
// The groups' rows are cut into segments of at most `seg` rows; a block takes one segment and 128
// columns i (f32: 64) and walks its rows in chunks of 64 (f32: 32): x and the split h by
// asynchronous copies (f32: through registers, a chunk ahead).  A group of one segment is written at once; the segments of a longer one
// leave partial sums that a second launch adds in order (no atomics: equal calls give equal bits;
// skewed groups are spread evenly, which a fixed number of blocks per group was not).
//
// f16: h is a 32-bit input of any range and the rows are the summed index, so per chunk of 64 rows
// it is scaled by one power of two (from the chunk's largest magnitude) and split into two f16
// parts, 2^-23 of each value and 2^-39 of the largest; the chunk's product is scaled back as it is added to the 32-bit running
// sums (which also ends the tensor cores' chains of truncating additions every 64 rows).  A launch
// of its own splits h, small beside x: with the split inside the loop, waiting for h and two
// barriers per chunk took most of the time (8192 rows, 2048 + 8192 columns, r = 32: 115 us; now 6 to
// 9 us for the split and 66 to 70 for the sums, bound by the latency of fragment loads and products at
// 16 warps per SM; the rows' bytes alone are 25).
struct SumJob {
  const void* x;         // [rows, di]
  const float* h;        // [rows or slots, dj]
  float* G;              // [N, di, dj], or [N, dj, di] when transposed
  float* partial;        // [slots][di dj], laid out as G
  __half* split;         // f16: [S_max][2 ldh]: high parts, low parts (ldh: dj padded)
  float* mul;            // f16: [S_max]: the power of two of the row's chunk
  int di, dj, transposed;
  int bi, blocks;        // column blocks of di; blocks of a segment in all (bi x those of dj)
};
struct SumArgs {
  SumJob job[2];
  const float* scale;    // [N] or null (1)
  const int32_t* perm;   // row of each slot, or null (the slot itself)
  const int32_t* offsets;   // [N + 1], or null (one group of all rows)
  const uint8_t* mask;   // rows that count, or null (perm == null only)
  int T, S_max, N, seg;
};

constexpr int kSumThreads = 256;
constexpr int kIT = 128;             // columns i per block (f16)
constexpr int kRows = 64;            // rows per chunk (f16)
constexpr int kLdX = kIT + 8;

// Row of slot s, -1 where it is to be left out.
__device__ __forceinline__ int row_of(const SumArgs& a, int s, int hi) {
  if (s >= hi) return -1;
  if (a.perm) {
    const int t = a.perm[s];
    return (unsigned)t < (unsigned)a.T ? t : -1;
  }
  return a.mask && !a.mask[s] ? -1 : s;
}

// Segments: a table over the groups in shared memory, or the one group of all rows.
struct Segments {
  int *bound, *start;
  int count;
};
template <int NT = kSumThreads>
__device__ __forceinline__ Segments segment_table(const SumArgs& a, int* mem) {
  Segments g;
  g.bound = mem;
  g.start = mem + a.N + 1;
  if (a.offsets) {
    group_table<NT>(a.offsets, a.N, a.S_max, a.seg, g.bound, g.start, g.start + a.N + 1);
  } else {
    if (threadIdx.x == 0) {
      g.bound[0] = g.start[0] = 0;
      g.bound[1] = a.S_max;
      g.start[1] = (a.S_max + a.seg - 1) / a.seg;
    }
    __syncthreads();
  }
  g.count = g.start[a.N];
  return g;
}

// Partial sums of a segment that starts at slot s0: in a window of `seg` slots at most one
// segment that is not its group's last one starts (it is `seg` long), and at most one last one
// of a group with several.
__device__ __forceinline__ int partial_slot(int s0, int seg, bool last) { return 2 * (s0 / seg) + last; }

// One item of a block: rows [lo, hi) of group n, columns i0.. and j0.. of a job.
struct SumItem {
  int n, lo, hi, i0, j0;
  const SumJob* jb;
  float* dst;            // G or partial sums, at the job's [i][j] = [0][0]
  float scale;
};
template <int IT, int R>
__device__ __forceinline__ SumItem sum_item(const SumArgs& a, const Segments& g, int item) {
  SumItem it;
  const int per = a.job[0].blocks + a.job[1].blocks;
  const int sgm = item / per;
  int b = item - sgm * per;
  it.n = a.offsets ? group_of(sgm, g.start, a.N) : 0;
  it.lo = g.bound[it.n] + (sgm - g.start[it.n]) * a.seg;
  it.hi = min(it.lo + a.seg, g.bound[it.n + 1]);
  it.jb = &a.job[0];
  if (b >= a.job[0].blocks) {
    b -= a.job[0].blocks;
    it.jb = &a.job[1];
  }
  it.i0 = (b % it.jb->bi) * IT;
  it.j0 = (b / it.jb->bi) * R;
  const size_t all = (size_t)it.jb->di * it.jb->dj;
  if (g.start[it.n + 1] - g.start[it.n] == 1) {
    it.dst = it.jb->G + it.n * all;
    it.scale = a.scale ? a.scale[it.n] : 1.f;
  } else {
    it.dst = it.jb->partial + partial_slot(it.lo, a.seg, it.hi == g.bound[it.n + 1]) * all;
    it.scale = 1.f;
  }
  return it;
}
// Writes v[i][j] of the fragments' layout: rows i, i + 8 of each 16, columns j, j + 1 of each 8.
template <int MI, int NJ>
__device__ __forceinline__ void store_sums(const SumItem& it, int i, int j, float (&v)[MI][NJ][4]) {
  const int di = it.jb->di, dj = it.jb->dj;
  const bool tr = it.jb->transposed, pairs = !tr && dj % 2 == 0;   // j is even
  const int64_t si = tr ? 1 : dj, sj = tr ? di : 1;
  float* p = it.dst + i * si + j * sj;
#pragma unroll
  for (int a = 0; a < MI; ++a)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (i + 16 * a + 8 * q >= di) continue;
      float* r = p + (16 * a + 8 * q) * si;
#pragma unroll
      for (int b = 0; b < NJ; ++b) {
        const float x = it.scale * v[a][b][2 * q], y = it.scale * v[a][b][2 * q + 1];
        if (pairs) {
          if (j + 8 * b < dj) *reinterpret_cast<float2*>(r + 8 * b) = make_float2(x, y);
          continue;
        }
        if (j + 8 * b < dj) r[8 * b * sj] = x;
        if (j + 8 * b + 1 < dj) r[(8 * b + 1) * sj] = y;
      }
    }
}
__device__ __forceinline__ void store_sum(const SumItem& it, int i, int j, float v) {
  if (i < it.jb->di && j < it.jb->dj)
    it.dst[it.jb->transposed ? (size_t)j * it.jb->di + i : (size_t)i * it.jb->dj + j] = it.scale * v;
}

// Groups without rows have zero sums; the grid shares them out.
__device__ __forceinline__ void clear_empty(const SumArgs& a, const Segments& g) {
  if (g.count > 0 && a.N == 1) return;
  for (int q = 0; q < 2; ++q) {
    const SumJob& jb = a.job[q];
    if (!jb.G) continue;
    const size_t all = (size_t)jb.di * jb.dj, step = (size_t)gridDim.x * blockDim.x;
    for (int n = 0; n < a.N; ++n) {
      if (g.start[n + 1] > g.start[n]) continue;
      float* G = jb.G + n * all;
      const size_t i0 = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
      if (all % 4 == 0)
        for (size_t i = i0; i < all / 4; i += step) reinterpret_cast<float4*>(G)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      else
        for (size_t i = i0; i < all; i += step) G[i] = 0.f;
    }
  }
}

// Warps of a block over the 128 x R sums: 32 x R / 2 each (R = 16: 16 x 16; R = 128, where only one
// block fits an SM: sixteen warps of 32 x 32).
template <int R>
struct SumWarps {
  static constexpr int kThreads = R >= 128 ? 512 : 256;
  static constexpr int WJ = R >= 128 ? 4 : R >= 32 ? 2 : 1, WI = kThreads / 32 / WJ;
  static constexpr int MI = kIT / WI / 16, NJ = R / WJ / 8;        // 16-row and 8-column fragments
};

// Splits h into f16 parts per chunk of 64 rows of a group; rows that are left out become zero.
// A block takes chunks; columns beyond dj are zero up to ldh.
__global__ void __launch_bounds__(kSumThreads) split_rows_kernel(const SumArgs a, int ldh) {
  const SumJob& jb = a.job[blockIdx.y];
  extern __shared__ int table[];
  __shared__ float wmax[kSumThreads / 32];
  pdl_trigger();
  pdl_wait();                                      // h may come from the launch before
  if (!jb.G) return;
  SumArgs b = a;
  b.seg = kRows;                                   // the table's tiles are the chunks
  const Segments g = segment_table(b, table);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int dj = jb.dj, n4 = ldh / 4;              // four columns at a time
  for (int c = blockIdx.x; c < g.count; c += gridDim.x) {
    const int n = a.offsets ? group_of(c, g.start, a.N) : 0;
    const int lo = g.bound[n] + (c - g.start[n]) * kRows, hi = min(lo + kRows, g.bound[n + 1]);
    auto load = [&](int q) {
      const int s = lo + q / n4, col = (q % n4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row_of(a, s, hi) < 0 || col >= dj) return v;
      const float* src = jb.h + (size_t)s * dj + col;
      if (dj % 4 == 0) return *reinterpret_cast<const float4*>(src);
      v.x = src[0];
      if (col + 1 < dj) v.y = src[1];
      if (col + 2 < dj) v.z = src[2];
      if (col + 3 < dj) v.w = src[3];
      return v;
    };
    float m = 0.f;
    for (int q = tid; q < kRows * n4; q += kSumThreads) {
      const float4 v = load(q);
      // of the finite values: infinities and NaN need no scale, and must not take the others' away
      auto mag = [](float f) { return f - f == 0.f ? fabsf(f) : 0.f; };
      m = fmaxf(m, fmaxf(fmaxf(mag(v.x), mag(v.y)), fmaxf(mag(v.z), mag(v.w))));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    __syncthreads();
    if (lane == 0) wmax[w] = m;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kSumThreads / 32; ++q) m = fmaxf(m, wmax[q]);
    const int e = split_exp(m);
    const float inv = exp2_int(-e);
    for (int q = tid; q < kRows * n4; q += kSumThreads) {
      const int s = lo + q / n4, col = (q % n4) * 4;
      if (s >= hi) break;
      const float4 v = load(q);
      __half2 h[2], l[2];
      split_f16(v.x * inv, h[0].x, l[0].x);
      split_f16(v.y * inv, h[0].y, l[0].y);
      split_f16(v.z * inv, h[1].x, l[1].x);
      split_f16(v.w * inv, h[1].y, l[1].y);
      __half* dst = jb.split + (size_t)s * 2 * ldh + col;
      *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(h);
      *reinterpret_cast<uint2*>(dst + ldh) = *reinterpret_cast<const uint2*>(l);
    }
    if (tid < hi - lo) jb.mul[lo + tid] = exp2_int(e);
  }
}

// Shared memory: a ring of chunks, x [64][kLdX] and the R columns of both parts of h [64][2 R + 8].
template <int R>
struct SumPlan {
  static constexpr int kLdH = 2 * R + 8;
  static constexpr int kStage = kRows * (kLdX + kLdH);             // halves
  static constexpr int kStages = R == 64 ? 3 : 4;                  // two blocks per SM (R = 128: one)
};

// kPerm: rows through perm.  Rows behind a segment's end then read its last one again (their h is
// zero), and entries outside [0, T) read as zeros.  Otherwise the rows are the slots, and masked ones
// read as zeros (they may hold anything).
template <int R, bool kPerm>
__global__ void __launch_bounds__(SumWarps<R>::kThreads, R >= 128 ? 1 : 2) row_sum_f16_kernel(const SumArgs a, int ldh) {
  constexpr int NT = SumWarps<R>::kThreads, XP = kRows * 16 / NT;   // 16-byte pieces of x per thread
  constexpr int kLdH = SumPlan<R>::kLdH, NS = SumPlan<R>::kStages, kStage = SumPlan<R>::kStage;
  constexpr int MI = SumWarps<R>::MI, NJ = SumWarps<R>::NJ, WI = SumWarps<R>::WI;
  constexpr int HP = kRows * R * 4 / 16 / NT;                      // and of h
  extern __shared__ __align__(128) uint8_t sm[];
  __half* ring = reinterpret_cast<__half*>(sm);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  pdl_trigger();
  pdl_wait();                                      // the split h
  const Segments g = segment_table<NT>(a, reinterpret_cast<int*>(ring + NS * kStage));
  const int items = g.count * (a.job[0].blocks + a.job[1].blocks);
  const int wi = (w % WI) * MI * 16, wj = (w / WI) * NJ * 8;
  const uint32_t ring_at = smem_u32(ring);
  // this lane's row of a fragment load: x transposed (rows = summed index), h as it lies
  const uint32_t xlane = (((lane & 7) + (lane >> 4) * 8) * kLdX + wi + ((lane >> 3) & 1) * 8) * 2;
  const uint32_t hlane = (kRows * kLdX + (lane & 15) * kLdH + wj + (lane >> 4) * 8) * 2;

  // ---- loads: chunk after chunk across the block's items, each chunk's rows fetched one early
  const int xc = (tid & 15) * 8, xr = tid >> 4;    // x: 16-byte piece, rows xr + NT / 16 p
  int li = blockIdx.x, lc = 0, llo = 0, lhi = 0, ldi = 0, lrow[XP];
  const __half *lX = nullptr, *lH = nullptr;
  bool lin = false;
  int lw = 0;                                      // columns of h that there are
  auto begin_item = [&]() {
    if (li >= items) return;
    const SumItem it = sum_item<kIT, R>(a, g, li);
    lc = 0;
    llo = it.lo;
    lhi = it.hi;
    ldi = it.jb->di;
    lin = it.i0 + xc < ldi;                        // columns behind the last are not stored
    lX = static_cast<const __half*>(it.jb->x) + (lin ? it.i0 + xc : 0);
    lH = it.jb->split + (size_t)it.lo * 2 * ldh + it.j0;
    lw = min(R, ldh - it.j0);
  };
  // The rows are looked at when they are used, a chunk later: a comparison right here would wait
  // for the load (a third of all stalls).
  auto fetch_rows = [&]() {
    if (li >= items) return;
    const int s = llo + lc * kRows + xr;
#pragma unroll
    for (int p = 0; p < XP; ++p) {
      const int r = s + NT / 16 * p;
      if (kPerm)
        lrow[p] = a.perm[min(r, lhi - 1)];
      else
        lrow[p] = r < lhi && (!a.mask || a.mask[r]) ? r : -1;
    }
  };
  auto load = [&](int stage) {
    if (li < items) {
      const uint32_t st = ring_at + stage * (kStage * 2), dst = st + (xr * kLdX + xc) * 2;
      const int left = lhi - llo - lc * kRows;     // rows of this and later chunks
      const int need = (left + 15) & ~15;          // rows that the products read
#pragma unroll
      for (int p = 0; p < XP; ++p) {
        if (xr + NT / 16 * p >= need) break;
        if (kPerm) {
          const bool on = (unsigned)lrow[p] < (unsigned)a.T;
          const uint32_t t = on ? lrow[p] : 0;
          cp_async16_at(dst + NT / 16 * p * kLdX * 2, lX + (uint64_t)t * (uint32_t)ldi, on);
        } else {
          const bool on = lin && lrow[p] >= 0;
          cp_async16_at(dst + NT / 16 * p * kLdX * 2, on ? lX + (uint64_t)(uint32_t)lrow[p] * (uint32_t)ldi : lX, on);
        }
      }
      const uint32_t hst = st + kRows * kLdX * 2;
      const __half* src = lH + (uint64_t)(uint32_t)(lc * kRows * 2) * (uint32_t)ldh;
#pragma unroll
      for (int p = 0; p < HP; ++p) {
        const int q = tid + p * NT;                // row, part, piece of R columns
        const int row = q / (R / 4), part = q / (R / 8) % 2, col = (q % (R / 8)) * 8;
        if (row >= need) break;
        const bool on = row < left && col < lw;
        cp_async16_at(hst + (row * kLdH + part * R + col) * 2, on ? src + (row * 2 + part) * ldh + col : lH, on);
      }
      if (++lc * kRows >= lhi - llo) {
        li += gridDim.x;
        begin_item();
      }
      fetch_rows();
    }
    cp_async_commit();
  };
  begin_item();
  fetch_rows();
  int stage = 0;                                   // of the next load
  for (; stage < NS - 1; ++stage) load(stage);

  int use = 0;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const SumItem it = sum_item<kIT, R>(a, g, item);
    const float* scales = it.jb->mul + it.lo;
    float acc[MI][NJ][4];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][j][q] = 0.f;
    float next = scales[0];
    for (int row = 0; row < it.hi - it.lo; row += kRows) {
      const float mul = next;
      if (row + kRows < it.hi - it.lo) next = scales[row + kRows];
      cp_async_wait<NS - 2>();
      __syncthreads();
      load(stage);
      stage = stage + 1 == NS ? 0 : stage + 1;
      const uint32_t xb = ring_at + use * (kStage * 2) + xlane, hb = ring_at + use * (kStage * 2) + hlane;
      use = use + 1 == NS ? 0 : use + 1;
      float t[MI][NJ][4];
#pragma unroll
      for (int k = 0; k < kRows; k += 16) {
        if (k > 0 && k >= it.hi - it.lo - row) break;   // short groups: no products of empty rows
        uint32_t fa[MI][4];
#pragma unroll
        for (int i = 0; i < MI; ++i) ldsm4_t_at(fa[i], xb + (k * kLdX + i * 16) * 2);
#pragma unroll
        for (int j = 0; j < NJ / 2; ++j) {
          uint32_t fh[4], fl[4];
          ldsm4_t_at(fl, hb + (k * kLdH + R + j * 16) * 2);
          ldsm4_t_at(fh, hb + (k * kLdH + j * 16) * 2);
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            if (k == 0) {
              mma16816_first(t[i][2 * j], fa[i], fl[0], fl[1]);
              mma16816_first(t[i][2 * j + 1], fa[i], fl[2], fl[3]);
            } else {
              mma16816(t[i][2 * j], fa[i], fl[0], fl[1]);
              mma16816(t[i][2 * j + 1], fa[i], fl[2], fl[3]);
            }
            mma16816(t[i][2 * j], fa[i], fh[0], fh[1]);
            mma16816(t[i][2 * j + 1], fa[i], fh[2], fh[3]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i][j][q] = fmaf(mul, t[i][j][q], acc[i][j][q]);
    }
    store_sums(it, it.i0 + wi + (lane >> 2), it.j0 + wj + 2 * (lane & 3), acc);
  }
  cp_async_wait<0>();
  clear_empty(a, g);
}

// 32-bit inputs, and f16 ones in short batches (one launch, no split): fused multiply-adds; 64
// columns i per block, chunks of 32 rows.
constexpr int kIT32 = 64;
constexpr int kRows32 = 32;

__device__ __forceinline__ float4 load_four(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load_four(const __half* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
  return make_float4(a.x, a.y, b.x, b.y);
}

template <typename T, int R>
__global__ void __launch_bounds__(kSumThreads) row_sum_fma_kernel(const SumArgs a) {
  constexpr int JT = R / 16;
  extern __shared__ __align__(16) float dyn[];     // x chunk [32][64], h chunk [32][R], table
  float* xs = dyn;
  float* hs = dyn + kRows32 * kIT32;
  const int tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();                                      // h may come from the launch before
  const Segments g = segment_table(a, reinterpret_cast<int*>(hs + kRows32 * R));
  const int items = g.count * (a.job[0].blocks + a.job[1].blocks);
  const int ti = (tid & 15) * 4, tj = tid >> 4;
  // a chunk is fetched into registers while the one before it is summed, across the block's items
  constexpr int HV = kRows32 * R / kSumThreads;
  float4 xv[2];
  float hv[HV];
  int li = blockIdx.x, lc = 0;
  SumItem nx;
  if (li < items) nx = sum_item<kIT32, R>(a, g, li);
  auto fetch = [&]() {
    if (li >= items) return;
    const T* X = static_cast<const T*>(nx.jb->x);
    const int di = nx.jb->di, dj = nx.jb->dj, s0 = nx.lo + lc * kRows32;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int q = tid + p * kSumThreads, i = (q % (kIT32 / 4)) * 4;
      const int t = row_of(a, s0 + q / (kIT32 / 4), nx.hi);
      xv[p] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t >= 0 && nx.i0 + i < di) xv[p] = load_four(X + (size_t)t * di + nx.i0 + i);
    }
#pragma unroll
    for (int p = 0; p < HV; ++p) {
      const int q = tid + p * kSumThreads, j = q % R, s = s0 + q / R;
      hv[p] = nx.j0 + j < dj && row_of(a, s, nx.hi) >= 0 ? nx.jb->h[(size_t)s * dj + nx.j0 + j] : 0.f;
    }
    if (++lc * kRows32 >= nx.hi - nx.lo) {
      lc = 0;
      li += gridDim.x;
      if (li < items) nx = sum_item<kIT32, R>(a, g, li);
    }
  };
  fetch();
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const SumItem it = sum_item<kIT32, R>(a, g, item);
    float acc[4][JT];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < JT; ++j) acc[i][j] = 0.f;
    for (int row = it.lo; row < it.hi; row += kRows32) {
      __syncthreads();
#pragma unroll
      for (int p = 0; p < 2; ++p) *reinterpret_cast<float4*>(xs + 4 * (tid + p * kSumThreads)) = xv[p];
#pragma unroll
      for (int p = 0; p < HV; ++p) hs[tid + p * kSumThreads] = hv[p];
      __syncthreads();
      fetch();
#pragma unroll 4
      for (int k = 0; k < kRows32; ++k) {
        const float4 xv = *reinterpret_cast<const float4*>(xs + k * kIT32 + ti);
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          const float h = hs[k * R + tj + 16 * j];
          acc[0][j] = fmaf(xv.x, h, acc[0][j]);
          acc[1][j] = fmaf(xv.y, h, acc[1][j]);
          acc[2][j] = fmaf(xv.z, h, acc[2][j]);
          acc[3][j] = fmaf(xv.w, h, acc[3][j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) store_sum(it, it.i0 + ti + i, it.j0 + tj + 16 * j, acc[i][j]);
  }
  clear_empty(a, g);
}

// Groups of several segments: their partial sums in order.  A block finds those groups (while the
// sums still run) and takes pieces of 1024 values of theirs; a grid over all groups, most of which may
// have one segment, took 10 us to start and end its blocks.
constexpr int kJoinThreads = 256;
__host__ __device__ inline int join_pieces(int di, int dj) {
  const size_t all = (size_t)di * dj, per = all % 4 ? kJoinThreads : 4 * kJoinThreads;
  return (int)((all + per - 1) / per);
}
__global__ void __launch_bounds__(kJoinThreads) row_sum_join_kernel(const SumArgs a) {
  extern __shared__ int table[];
  __shared__ int several;
  const int tid = threadIdx.x;
  if (tid == 0) several = 0;
  const Segments g = segment_table<kJoinThreads>(a, table);
  int* list = table + 2 * (a.N + 1) + 64;
  for (int n = tid; n < a.N; n += kJoinThreads)
    if (g.start[n + 1] - g.start[n] > 1) list[atomicAdd(&several, 1)] = n;   // each sums for itself
  __syncthreads();
  pdl_wait();                                       // on every path: completion stays transitive
  const int p0 = a.job[0].G ? join_pieces(a.job[0].di, a.job[0].dj) : 0;
  const int p1 = a.job[1].G ? join_pieces(a.job[1].di, a.job[1].dj) : 0;
  const long long items = (long long)several * (p0 + p1);
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int n = list[it / (p0 + p1)];
    int piece = (int)(it % (p0 + p1));
    const bool second = piece >= p0;
    if (second) piece -= p0;
    const SumJob& jb = a.job[second];
    const int segs = g.start[n + 1] - g.start[n];
    const float scale = a.scale ? a.scale[n] : 1.f;
    const size_t all = (size_t)jb.di * jb.dj, i = (size_t)piece * kJoinThreads + tid;
    float* G = jb.G + n * all;
    const float* first = jb.partial + partial_slot(g.bound[n], a.seg, false) * all;   // and every second after it
    if (all % 4 == 0) {
      if (i >= all / 4) continue;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      const float* p = first + 4 * i;
#pragma unroll 8
      for (int q = 0; q < segs; ++q, p += 2 * all) {
        const float4 u = *reinterpret_cast<const float4*>(q == segs - 1 ? p + all : p);
        v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
      }
      *reinterpret_cast<float4*>(G + 4 * i) = make_float4(scale * v.x, scale * v.y, scale * v.z, scale * v.w);
    } else if (i < all) {
      float v = 0.f;
      for (int q = 0; q < segs; ++q) v += first[(2 * q + (q == segs - 1)) * all + i];
      G[i] = scale * v;
    }
  }
}
cudaError_t launch_join(const SumArgs& a, int sms, cudaStream_t s) {
  long long pieces = 0;
  for (const SumJob& j : a.job)
    if (j.G) pieces += join_pieces(j.di, j.dj);
  const long long groups = std::min<long long>(a.N, a.S_max / (a.seg + 1));   // longer than a segment
  const int grid = (int)std::max<long long>(1, std::min<long long>(groups * pieces, 8 * sms));
  return launch_k(row_sum_join_kernel, grid, kJoinThreads, sizeof(int) * (3 * ((size_t)a.N + 1) + 64), s, true, a);
}

// Short f16 groups take the multiply-add form (one launch less), where its items are two rounds of
// blocks at most.  us, both gradients, multiply-adds / tensor cores: one group, 1024 columns each,
// r = 16: 64 rows 15.4 / 16.1, 128 rows 19.0 / 16.8, 512 rows 40 / 21; eight groups of 32 rows 13.8 / 15.2,
// of 64 rows 18.9 / 18.3 (skewed groups make it 40 / 21); 16 groups of 3584 columns, 32 rows in all:
// 31 / 23.
bool sum_tc(bool f16, int S_max, int N, int columns, int sms) {
  const long long n = std::min(N, S_max);
  return f16 && (S_max > std::max(64LL, 32 * n) || n * (columns / kIT32 + 2) > 4 * sms);
}

// Rows per segment: the segments of S_max rows (and half a segment more per group) times the
// column blocks take the fewest rounds of two blocks on each SM, plus what a segment
// costs in partial sums and the launch that joins them.  chunk: us of 64 rows (fused multiply-adds:
// up to six times the tensor cores'; counted as theirs, 651 x 848 rows by 67 columns took 60 us in one
// segment).
int sum_segment(int S_max, int N, int blocks, size_t words, double chunk, int sms) {
  int best = 64;
  double cost = 1e300;
  for (int p = 1; p <= sum_parts(words); ++p) {
    const int seg = std::max(64, (int)(((long long)S_max + p - 1) / p + 63) / 64 * 64);
    const double items = blocks * ((double)S_max / seg + 0.5 * std::min(N, S_max));
    const double c = ceil(items / (2 * sms)) * (seg / 64 * chunk + 2) + 0.7 * p + (seg < S_max ? 6 : 0);
    if (c < cost) {
      cost = c;
      best = seg;
    }
  }
  return best;
}

// Columns of h's parts: dj in whole fragments (16 columns) of the row sums.
int split_width(int dj) { return (dj + 15) / 16 * 16; }

template <int R>
cudaError_t launch_sum_rank(SumArgs& a, bool f16, bool tc, int sms, bool pdl, cudaStream_t s) {
  const int it = tc ? kIT : kIT32;
  int blocks = 0, ldh = 0;
  size_t widest = 0;
  for (SumJob& j : a.job) {
    j.bi = (j.di + it - 1) / it;
    j.blocks = j.G ? j.bi * ((j.dj + R - 1) / R) : 0;
    blocks += j.blocks;
    if (j.G) widest = std::max(widest, (size_t)j.di * j.dj);
    if (j.G) ldh = std::max(ldh, split_width(j.dj));
  }
  const long long segs = (long long)a.S_max / a.seg + std::min(a.N, a.S_max);
  const size_t table = sizeof(int) * (2 * ((size_t)a.N + 1) + 64);
  // empty groups are cleared by the whole grid: at least a block per 32 KB of the sums
  const long long clear = (long long)std::min(a.N, 64) * (long long)widest / 8192;
  const int grid = (int)std::min<long long>(std::max(segs * blocks, clear), (tc && R >= 128 ? 1 : 2) * sms);
  if (tc) {
    const long long chunks = (long long)a.S_max / kRows + std::min(a.N, a.S_max);
    MOE_LAUNCH(launch_k(split_rows_kernel, dim3((int)std::min<long long>(chunks, 4 * sms), 2), kSumThreads,
                        table, s, pdl, a, ldh));
    auto kern = a.perm ? row_sum_f16_kernel<R, true> : row_sum_f16_kernel<R, false>;
    MOE_LAUNCH(ensure_smem_attr(reinterpret_cast<const void*>(kern)));
    const size_t smem = 2 * (size_t)SumPlan<R>::kStages * SumPlan<R>::kStage + table;
    MOE_LAUNCH(launch_k(kern, grid, SumWarps<R>::kThreads, smem, s, true, a, ldh));
  } else {
    auto kern = f16 ? row_sum_fma_kernel<__half, R> : row_sum_fma_kernel<float, R>;
    MOE_LAUNCH(ensure_smem_attr(reinterpret_cast<const void*>(kern)));
    const size_t smem = sizeof(float) * (kRows32 * kIT32 + kRows32 * R) + table;
    MOE_LAUNCH(launch_k(kern, grid, kSumThreads, smem, s, pdl, a));
  }
  if (a.S_max <= a.seg) return cudaSuccess;        // no group has a second segment
  return launch_join(a, sms, s);
}

// Column blocks of a job of either type, as launch_sum_rank cuts them.
int sum_blocks(int di, int dj, int dj_max, bool tc) {
  const int R = dj_max <= 16 ? 16 : dj_max <= 32 ? 32 : dj_max <= 64 ? 64 : 128, it = tc ? kIT : kIT32;
  return (di + it - 1) / it * ((dj + R - 1) / R);
}

// ---------------------------------------------------------------- tokens' gradient of the gate
// out[t,i] = in[t,i] + sum_e dl[t,e] W[i,e], fused multiply-adds on tiles of 32 tokens x 64 columns,
// chunks of 32 experts whose loads are issued together and one chunk ahead: 32-bit tokens, short
// batches, and E > 256 (the other form is in gate_grad.cu).
constexpr int kDxT = 32, kDxI = 64, kDxE = 32;

template <typename T>
__global__ void __launch_bounds__(256) gate_dx_kernel(const float* __restrict__ dl,
                                                      const float* __restrict__ W,
                                                      const T* in, int rows, int d, int E, T* out) {
  __shared__ float as[kDxE][kDxT + 4], bs[kDxE][kDxI + 4];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * kDxT;
  const int i0 = blockIdx.y * kDxI, le = tid & 31, lr = tid >> 5;
  float av[4], bv[8];
  auto fetch = [&](int e0) {
    const bool on = e0 + le < E;
#pragma unroll
    for (int q = 0; q < 4; ++q) av[q] = on && t0 + lr + 8 * q < rows ? dl[(t0 + lr + 8 * q) * E + e0 + le] : 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) bv[q] = on && i0 + lr + 8 * q < d ? W[(size_t)(i0 + lr + 8 * q) * E + e0 + le] : 0.f;
  };
  float acc[2][4] = {};
  pdl_wait();                                       // dl comes from a launch before
  fetch(0);
  for (int e0 = 0; e0 < E; e0 += kDxE) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) as[le][lr + 8 * q] = av[q];
#pragma unroll
    for (int q = 0; q < 8; ++q) bs[le][lr + 8 * q] = bv[q];
    __syncthreads();
    if (e0 + kDxE < E) fetch(e0 + kDxE);
#pragma unroll
    for (int e = 0; e < kDxE; ++e) {
      const float2 u = *reinterpret_cast<const float2*>(&as[e][ty * 2]);
      const float4 v = *reinterpret_cast<const float4*>(&bs[e][tx * 4]);
      const float a2[2] = {u.x, u.y}, b4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a2[i], b4[j], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t t = t0 + ty * 2 + i;
    if (t >= rows) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = i0 + tx * 4 + j;
      if (c >= d) continue;
      float v = acc[i][j];
      if (in) v += (float)in[t * d + c];
      out[t * d + c] = (T)v;
    }
  }
}

// ---------------------------------------------------------------- combine's gradient
// dy_s = w_tj dout_t,  dw_tj = <dout_t, y_s>,  s = slot_of[t,j].  Bound by DRAM: dout, y read
// once, dy written once (16384 x 3584 top-2: 94 us, 5.75 TB/s, 0.85 of a copy's rate).  WPR warps per
// token row (8 where there are too few rows to fill the device with a warp each).

// Written once and not read here: first to leave L2 (105 us without it).
template <typename Vec>
__device__ __forceinline__ void store_stream(void* p, const Vec& v) {
  if constexpr (sizeof(Vec) == 16)
    __stcs(static_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&v));
  else
    *static_cast<Vec*>(p) = v;
}

template <typename T, int V, int WPR>
__global__ void __launch_bounds__(256) combine_backward_kernel(
    const T* __restrict__ dout, const T* __restrict__ y, const int32_t* __restrict__ slot_of,
    const float* __restrict__ topk_w, int rows, int d, int k, int S_max, T* __restrict__ dy,
    float* __restrict__ dw) {
  struct alignas(V * sizeof(T)) Vec { T v[V]; };
  __shared__ float part[2][8];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int sub = w % WPR;
  for (int64_t t0 = (int64_t)blockIdx.x * (8 / WPR); t0 < rows; t0 += (int64_t)gridDim.x * (8 / WPR)) {
    const int64_t t = t0 + w / WPR;
    int s[2] = {-1, -1};
    float g[2] = {0.f, 0.f}, acc[2] = {0.f, 0.f};
    if (t < rows) {
      for (int j = 0; j < k; ++j) {
        s[j] = slot_of[t * k + j];
        if (s[j] >= S_max) s[j] = -1;
        if (dy) g[j] = topk_w[t * k + j];
      }
      if (s[0] >= 0 || s[1] >= 0) {
#pragma unroll 2
        for (int c = (sub * 32 + lane) * V; c < d; c += WPR * 32 * V) {
          const Vec u = *reinterpret_cast<const Vec*>(dout + t * d + c);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (s[j] < 0) continue;
            if (dw) {
              const Vec q = *reinterpret_cast<const Vec*>(y + (int64_t)s[j] * d + c);
#pragma unroll
              for (int i = 0; i < V; ++i) acc[j] = fmaf((float)u.v[i], (float)q.v[i], acc[j]);
            }
            if (dy) {
              Vec o;
#pragma unroll
              for (int i = 0; i < V; ++i) o.v[i] = (T)(g[j] * (float)u.v[i]);
              store_stream(dy + (int64_t)s[j] * d + c, o);
            }
          }
        }
      }
    }
    if (!dw) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
    if (WPR > 1) {
      if (lane == 0) {
        part[0][w] = acc[0];
        part[1][w] = acc[1];
      }
      __syncthreads();
      if (sub == 0)
        for (int q = 1; q < WPR; ++q) {
          acc[0] += part[0][w + q];
          acc[1] += part[1][w + q];
        }
      __syncthreads();
    }
    if (sub == 0 && lane < k && t < rows) dw[t * k + lane] = s[lane] >= 0 ? acc[lane] : 0.f;
  }
}

int sms_of_device() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

template <typename T, int V>
cudaError_t launch_combine_backward_t(const void* dout, const void* y, const int32_t* slot_of,
                                      const float* topk_w, int T_, int d, int k, int S_max, void* dy,
                                      float* dw, int sms, cudaStream_t s) {
  const T* du = static_cast<const T*>(dout);
  const T* yy = static_cast<const T*>(y);
  // Eight warps per row while a warp each leaves the device's loads waiting for one another: f16, us
  // one / eight: 3584 columns 1024 rows 6.3 / 4.8, 2432 rows 7.3 / 8.1; 1024 columns 256 rows 3.1 / 2.4,
  // 1024 rows 3.2 / 3.6; 64 columns the same or less for one.
  if (T_ < 128LL * ((d + 32 * V - 1) / (32 * V)))
    return launch_k(combine_backward_kernel<T, V, 8>, std::min(T_, 8 * sms), 256, 0, s, false, du, yy,
                    slot_of, topk_w, T_, d, k, S_max, static_cast<T*>(dy), dw);
  return launch_k(combine_backward_kernel<T, V, 1>, std::min((T_ + 7) / 8, 8 * sms), 256, 0, s, false,
                  du, yy, slot_of, topk_w, T_, d, k, S_max, static_cast<T*>(dy), dw);
}

}  // namespace

namespace {
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
// f16: bytes of the split parts and their scales of one job
size_t split_bytes(int dj, int S_max) { return up256((size_t)S_max * split_width(dj) * 4) + up256((size_t)S_max * 4); }
}  // namespace

// G = sum over runs of `run` of T rows, in order, of partial sums in partial_slot's layout.
cudaError_t launch_sum_join(float* G, float* partial, int di, int dj, int T, int run, int sms, cudaStream_t s) {
  SumArgs a;
  memset(&a, 0, sizeof(a));
  a.job[0].G = G;
  a.job[0].partial = partial;
  a.job[0].di = di;
  a.job[0].dj = dj;
  a.T = a.S_max = T;
  a.N = 1;
  a.seg = run;
  return launch_join(a, sms, s);
}

size_t row_sums_bytes(int di0, int dj0, int di1, int dj1, bool f16, int S_max) {
  size_t most = 0;
  // either job alone may be asked for: the plan of each combination fits
  for (int q = 1; q < 4; ++q) {
    const size_t words = (q & 1 ? (size_t)di0 * dj0 : 0) + (q & 2 ? (size_t)di1 * dj1 : 0);
    if (words > 0) most = std::max(most, sum_partial_bytes(words, S_max, 64));
  }
  return up256(most) + (f16 ? split_bytes(dj0, S_max) + split_bytes(dj1, S_max) : 0);
}

cudaError_t launch_row_sums(const void* x0, const float* h0, float* G0, int di0, int dj0, int tr0,
                            const void* x1, const float* h1, float* G1, int di1, int dj1, int tr1,
                            const float* scale, const int32_t* perm, const int32_t* offsets,
                            const uint8_t* mask, void* workspace, int dtype_f16, int T, int S_max,
                            int N, bool pdl, cudaStream_t s) {
  const int sms = sms_of_device();
  if (sms < 1) return cudaErrorInvalidDevice;
  const bool tc = sum_tc(dtype_f16, S_max, N, (G0 ? di0 : 0) + (G1 ? di1 : 0), sms);
  SumArgs a;
  memset(&a, 0, sizeof(a));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  auto job = [&](SumJob& j, const void* x, const float* h, float* G, int di, int dj, int tr) {
    j.x = x;
    j.h = h;
    j.G = G;
    j.di = di;
    j.dj = dj;
    j.transposed = tr;
    if (tc) {
      j.split = reinterpret_cast<__half*>(ws);
      j.mul = reinterpret_cast<float*>(ws + up256((size_t)S_max * split_width(dj) * 4));
      ws += split_bytes(dj, S_max);
    }
  };
  if (G0) job(a.job[0], x0, h0, G0, di0, dj0, tr0);
  if (G1) job(a.job[1], x1, h1, G1, di1, dj1, tr1);
  const int dj = std::max(G0 ? dj0 : 0, G1 ? dj1 : 0);
  const int blocks = (G0 ? sum_blocks(di0, dj0, dj, tc) : 0) + (G1 ? sum_blocks(di1, dj1, dj, tc) : 0);
  a.seg = sum_segment(S_max, N, blocks, (G0 ? (size_t)di0 * dj0 : 0) + (G1 ? (size_t)di1 * dj1 : 0),
                      tc ? 1.0 : std::max(1.0, std::min(dj, 128) * (6.0 / 128)), sms);
  a.job[0].partial = a.job[1].partial = reinterpret_cast<float*>(ws);
  if (G0) a.job[1].partial += 2 * (size_t)((S_max + a.seg - 1) / a.seg) * di0 * dj0;
  a.scale = scale;
  a.perm = perm;
  a.offsets = offsets;
  a.mask = mask;
  a.T = T;
  a.S_max = S_max;
  a.N = N;
  if (dj <= 16) return launch_sum_rank<16>(a, dtype_f16, tc, sms, pdl, s);
  if (dj <= 32) return launch_sum_rank<32>(a, dtype_f16, tc, sms, pdl, s);
  if (dj <= 64) return launch_sum_rank<64>(a, dtype_f16, tc, sms, pdl, s);
  return launch_sum_rank<128>(a, dtype_f16, tc, sms, pdl, s);
}

cudaError_t launch_gate_dx(const float* dlogits, const float* Wg, const void* in, int dtype_f16, int T,
                           int d, int E, void* out, cudaStream_t s) {
  const dim3 grid((T + kDxT - 1) / kDxT, (d + kDxI - 1) / kDxI);
  if (dtype_f16)
    return launch_k(gate_dx_kernel<__half>, grid, 256, 0, s, true, dlogits, Wg,
                    static_cast<const __half*>(in), T, d, E, static_cast<__half*>(out));
  return launch_k(gate_dx_kernel<float>, grid, 256, 0, s, true, dlogits, Wg,
                  static_cast<const float*>(in), T, d, E, static_cast<float*>(out));
}

cudaError_t launch_combine_backward(const void* dout, const void* expert_out, const int32_t* slot_of,
                                    const float* topk_w, int dtype_f16, int T, int d, int k, int S_max,
                                    void* dexpert_out, float* dtopk_w, cudaStream_t s) {
  const int sms = sms_of_device();
  if (sms < 1) return cudaErrorInvalidDevice;
  if (dtype_f16)
    return d % 8 == 0 ? launch_combine_backward_t<__half, 8>(dout, expert_out, slot_of, topk_w, T, d, k,
                                                             S_max, dexpert_out, dtopk_w, sms, s)
                      : launch_combine_backward_t<__half, 1>(dout, expert_out, slot_of, topk_w, T, d, k,
                                                             S_max, dexpert_out, dtopk_w, sms, s);
  return d % 4 == 0 ? launch_combine_backward_t<float, 4>(dout, expert_out, slot_of, topk_w, T, d, k,
                                                          S_max, dexpert_out, dtopk_w, sms, s)
                    : launch_combine_backward_t<float, 1>(dout, expert_out, slot_of, topk_w, T, d, k,
                                                          S_max, dexpert_out, dtopk_w, sms, s);
}

}  // namespace moe
