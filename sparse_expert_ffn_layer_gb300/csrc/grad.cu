// Gradients around the gate and the adapters: products summed over token rows (weights'
// gradients), the tokens' gradient through the gate, and the combine's gradient.
#include <cooperative_groups.h>

#include <algorithm>

#include "launch.h"
#include "mma.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

// ---------------------------------------------------------------- sums over rows
// G[n][i][j] = scale_n sum_s x[t(s)][i] h[s][j] over the rows s of group n, in 32 bits.
//
// Bound by DRAM: x is streamed once (per 128 columns j), G written once.  A block owns 128
// columns i of one group and walks its rows in chunks of 64: x by asynchronous copies (a ring of
// four chunks), h through registers.  h is a 32-bit input of any range and the rows are the
// summed index, so per chunk it is scaled by one power of two (from the chunk's largest
// magnitude) and split into two f16 parts, 22 bits together; the chunk's product is scaled back
// as it is added to the 32-bit running sums (which also keeps a long sum out of the tensor
// cores' accumulators, whose additions truncate).
//
// Few blocks and many rows: the rows are split over a cluster of up to eight blocks, whose sums
// are joined through distributed shared memory in rank order, so results do not depend on timing.
struct SumJob {
  const void* x;         // [rows, di]
  const float* h;        // [rows or slots, dj]
  float* G;              // [N, di, dj], or [N, dj, di] when transposed
  int di, dj, transposed, blocks;
};
struct SumArgs {
  SumJob job[2];
  const float* scale;    // [N] or null (1)
  const int32_t* perm;   // row of each slot, or null (the slot itself)
  const int32_t* offsets;   // [N + 1], or null (one group of all rows)
  const uint8_t* mask;   // rows that count, or null (perm == null only)
  int T, S_max;
};

constexpr int kSumThreads = 256;
constexpr int kIT = 128;             // columns i per block (f16)
constexpr int kRows = 64;            // rows per chunk (f16)
constexpr int kLdX = kIT + 8;
constexpr int kSumStages = 4;

__device__ __forceinline__ void group_rows(const SumArgs& a, int n, int* lo, int* hi) {
  *lo = 0;
  *hi = a.S_max;
  if (a.offsets) {
    *lo = min(max(a.offsets[n], 0), a.S_max);
    *hi = max(*lo, min(max(a.offsets[n + 1], 0), a.S_max));
  }
}

// Row of slot s, -1 where it is to be left out.
__device__ __forceinline__ int row_of(const SumArgs& a, int s, int hi) {
  if (s >= hi) return -1;
  if (a.perm) {
    const int t = a.perm[s];
    return (unsigned)t < (unsigned)a.T ? t : -1;
  }
  return a.mask && !a.mask[s] ? -1 : s;
}

// Joins the cluster's sums red[IT][ld] (this block's rows i and R columns j) and writes them.
template <int IT, int R>
__device__ __forceinline__ void join_and_store(const SumJob& jb, float* red, int ld, int i0, int j0,
                                               int n, float scale) {
  cg::cluster_group cl = cg::this_cluster();
  const int ncl = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  cl.sync();
  const int per = IT / ncl, r0 = rank * per;
  const int nj = min(R, jb.dj - j0);
  float* G = jb.G + (size_t)n * jb.di * jb.dj;
  for (int q = threadIdx.x; q < per * R; q += kSumThreads) {
    const int i = r0 + (jb.transposed ? q % per : q / R), j = jb.transposed ? q / per : q % R;
    if (j >= nj || i0 + i >= jb.di) continue;
    float v = 0.f;
    for (int b = 0; b < ncl; ++b) v += cl.map_shared_rank(red, b)[i * ld + j];
    v *= scale;
    if (jb.transposed)
      G[(size_t)(j0 + j) * jb.di + i0 + i] = v;
    else
      G[(size_t)(i0 + i) * jb.dj + j0 + j] = v;
  }
  cl.sync();                                       // no block leaves while its sums are read
}

template <int R>
__global__ void __launch_bounds__(kSumThreads) row_sum_f16_kernel(const SumArgs a) {
  constexpr int kLdH = R + 8;
  constexpr int kHB = kRows * kLdH;                // halves of one f16 part
  constexpr int NV = kRows * R / kSumThreads;      // h values per thread and chunk
  extern __shared__ __align__(128) uint8_t sm[];
  __half* xs = reinterpret_cast<__half*>(sm);                         // [stages][64][kLdX]
  __half* hs = xs + kSumStages * kRows * kLdX;                        // [2][hi, lo][64][kLdH]
  __shared__ float wmax[2][kSumThreads / 32];
  cg::cluster_group cl = cg::this_cluster();
  const int ncl = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const bool second = (int)blockIdx.x >= a.job[0].blocks;
  const SumJob jb = second ? a.job[1] : a.job[0];
  const int i0 = ((int)blockIdx.x - (second ? a.job[0].blocks : 0)) * kIT;
  const int n = blockIdx.y, j0 = (blockIdx.z / ncl) * R;
  const int dj = jb.dj;
  const __half* X = static_cast<const __half*>(jb.x);
  int lo, hi;
  group_rows(a, n, &lo, &hi);
  const int chunks = (hi - lo + kRows - 1) / kRows;
  const int c0 = (int)((long long)chunks * rank / ncl), c1 = (int)((long long)chunks * (rank + 1) / ncl);

  // x: thread's pieces are column piece tid % 16 of rows tid / 16 + 16 p
  const int xc = (tid & 15) * 8;
  int rows_next[4];
  auto fetch_rows = [&](int c) {
#pragma unroll
    for (int p = 0; p < 4; ++p) rows_next[p] = row_of(a, lo + c * kRows + (tid >> 4) + 16 * p, hi);
  };
  auto load_x = [&](int c) {                       // rows_next holds chunk c's rows
    __half* dst = xs + (c % kSumStages) * kRows * kLdX;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const bool on = rows_next[p] >= 0 && i0 + xc < jb.di;
      cp_async16(dst + ((tid >> 4) + 16 * p) * kLdX + xc,
                 X + (on ? (size_t)rows_next[p] * jb.di + i0 + xc : 0), on);
    }
  };
  // h: thread holds NV consecutive values of one row
  const int hr = tid * NV / R, hc = tid * NV % R;
  float hv[NV];
  auto load_h = [&](int c) {
    const int s = lo + c * kRows + hr;
    const bool on = c < c1 && row_of(a, s, hi) >= 0;
    const float* src = jb.h + (size_t)(on ? s : 0) * dj + j0 + hc;
    if (dj % 4 == 0) {
#pragma unroll
      for (int q = 0; q < NV; q += 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (on && j0 + hc + q < dj) v = *reinterpret_cast<const float4*>(src + q);
        hv[q] = v.x; hv[q + 1] = v.y; hv[q + 2] = v.z; hv[q + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int q = 0; q < NV; ++q) hv[q] = on && j0 + hc + q < dj ? src[q] : 0.f;
    }
  };

  float acc[R / 8][4];
#pragma unroll
  for (int i = 0; i < R / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;

  for (int p = 0; p < kSumStages - 1; ++p) {
    if (c0 + p < c1) {
      fetch_rows(c0 + p);
      load_x(c0 + p);
    }
    cp_async_commit();
  }
  if (c0 + kSumStages - 1 < c1) fetch_rows(c0 + kSumStages - 1);
  load_h(c0);
  for (int c = c0; c < c1; ++c) {
    const int b = (c - c0) & 1;
    // this chunk's power of two
    float m = 0.f;
    bool odd = false;
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      m = fmaxf(m, fabsf(hv[q]));
      odd |= !isfinite(hv[q]);
    }
    if (odd) m = INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) wmax[b][w] = m;
    cp_async_wait<kSumStages - 2>();
    __syncthreads();                               // chunk c of x is in; every wmax is written
#pragma unroll
    for (int q = 0; q < kSumThreads / 32; ++q) m = fmaxf(m, wmax[b][q]);
    const int e = scale_exp(m);
    const float inv = exp2_int(-e), mul = exp2_int(e);
    __half* hhi = hs + b * 2 * kHB;
    __half* hlo = hhi + kHB;
#pragma unroll
    for (int q = 0; q < NV; q += 2) {
      __half2 u, v;
      split_f16(hv[q] * inv, u.x, v.x);
      split_f16(hv[q + 1] * inv, u.y, v.y);
      *reinterpret_cast<__half2*>(hhi + hr * kLdH + hc + q) = u;
      *reinterpret_cast<__half2*>(hlo + hr * kLdH + hc + q) = v;
    }
    if (c + 1 < c1) load_h(c + 1);
    if (c + kSumStages - 1 < c1) load_x(c + kSumStages - 1);
    cp_async_commit();
    if (c + kSumStages < c1) fetch_rows(c + kSumStages);
    __syncthreads();
    const __half* xb = xs + (c % kSumStages) * kRows * kLdX;
    float t[R / 8][4];
#pragma unroll
    for (int i = 0; i < R / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) t[i][j] = 0.f;
#pragma unroll
    for (int k = 0; k < kRows; k += 16) {
      uint32_t fa[4];
      frag_a_t(fa, xb + k * kLdX + w * 16, kLdX, lane);
#pragma unroll
      for (int j = 0; j < R / 16; ++j) {
        uint32_t fh[4], fl[4];
        frag_b_kn(fl, hlo + k * kLdH + j * 16, kLdH, lane);
        frag_b_kn(fh, hhi + k * kLdH + j * 16, kLdH, lane);
        mma16816(t[2 * j], fa, fl[0], fl[1]);
        mma16816(t[2 * j + 1], fa, fl[2], fl[3]);
        mma16816(t[2 * j], fa, fh[0], fh[1]);
        mma16816(t[2 * j + 1], fa, fh[2], fh[3]);
      }
    }
#pragma unroll
    for (int i = 0; i < R / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(mul, t[i][j], acc[i][j]);
  }
  cp_async_wait<0>();
  __syncthreads();
  float* red = reinterpret_cast<float*>(sm);       // [128][R + 4], over the ring
  constexpr int ld = R + 4;
  static_assert(kIT * ld * 4 <= kSumStages * kRows * kLdX * 2, "the sums fit over the ring");
  float* p = red + (w * 16 + (lane >> 2)) * ld + 2 * (lane & 3);
#pragma unroll
  for (int j = 0; j < R / 8; ++j) {
    *reinterpret_cast<float2*>(p + 8 * j) = make_float2(acc[j][0], acc[j][1]);
    *reinterpret_cast<float2*>(p + 8 * ld + 8 * j) = make_float2(acc[j][2], acc[j][3]);
  }
  join_and_store<kIT, R>(jb, red, ld, i0, j0, n, a.scale ? a.scale[n] : 1.f);
}

// 32-bit inputs: fused multiply-adds; 64 columns i per block, chunks of 32 rows.
constexpr int kIT32 = 64;
constexpr int kRows32 = 32;

template <int R>
__global__ void __launch_bounds__(kSumThreads) row_sum_f32_kernel(const SumArgs a) {
  constexpr int JT = R / 16;
  __shared__ __align__(16) float xs[kRows32][kIT32];
  extern __shared__ __align__(16) float dyn[];     // h chunk [32][R], then the sums [64][R + 1]
  cg::cluster_group cl = cg::this_cluster();
  const int ncl = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x;
  const bool second = (int)blockIdx.x >= a.job[0].blocks;
  const SumJob jb = second ? a.job[1] : a.job[0];
  const int i0 = ((int)blockIdx.x - (second ? a.job[0].blocks : 0)) * kIT32;
  const int n = blockIdx.y, j0 = (blockIdx.z / ncl) * R;
  const float* X = static_cast<const float*>(jb.x);
  int lo, hi;
  group_rows(a, n, &lo, &hi);
  const int chunks = (hi - lo + kRows32 - 1) / kRows32;
  const int c0 = (int)((long long)chunks * rank / ncl), c1 = (int)((long long)chunks * (rank + 1) / ncl);
  const int ti = (tid & 15) * 4, tj = tid >> 4;
  float acc[4][JT];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j) acc[i][j] = 0.f;
  for (int c = c0; c < c1; ++c) {
    __syncthreads();
    for (int q = tid; q < kRows32 * kIT32 / 4; q += kSumThreads) {
      const int r = q / (kIT32 / 4), i = (q % (kIT32 / 4)) * 4;
      const int t = row_of(a, lo + c * kRows32 + r, hi);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t >= 0 && i0 + i < jb.di) v = *reinterpret_cast<const float4*>(X + (size_t)t * jb.di + i0 + i);
      *reinterpret_cast<float4*>(&xs[r][i]) = v;
    }
    for (int q = tid; q < kRows32 * R; q += kSumThreads) {
      const int r = q / R, j = q % R, s = lo + c * kRows32 + r;
      dyn[q] = j0 + j < jb.dj && row_of(a, s, hi) >= 0 ? jb.h[(size_t)s * jb.dj + j0 + j] : 0.f;
    }
    __syncthreads();
#pragma unroll 4
    for (int k = 0; k < kRows32; ++k) {
      const float4 xv = *reinterpret_cast<const float4*>(&xs[k][ti]);
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        const float h = dyn[k * R + tj + 16 * j];
        acc[0][j] = fmaf(xv.x, h, acc[0][j]);
        acc[1][j] = fmaf(xv.y, h, acc[1][j]);
        acc[2][j] = fmaf(xv.z, h, acc[2][j]);
        acc[3][j] = fmaf(xv.w, h, acc[3][j]);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j) dyn[(ti + i) * (R + 1) + tj + 16 * j] = acc[i][j];
  join_and_store<kIT32, R>(jb, dyn, R + 1, i0, j0, n, a.scale ? a.scale[n] : 1.f);
}

template <typename Kern>
cudaError_t launch_sum(Kern kern, size_t smem, SumArgs& a, int it, int R, int N, int rows_per_group,
                       int chunk, int sms, cudaStream_t s) {
  MOE_LAUNCH(ensure_smem_attr(reinterpret_cast<const void*>(kern)));
  int blocks = 0, jb = 1;
  for (SumJob& j : a.job) {
    j.blocks = j.G ? (j.di + it - 1) / it : 0;
    blocks += j.blocks;
    if (j.G) jb = std::max(jb, (j.dj + R - 1) / R);
  }
  // rows split until the blocks fill the device twice, at two chunks per block or more
  int cl = 1;
  while (cl < 8 && (long long)blocks * N * jb * cl < 2LL * sms && rows_per_group >= 4 * chunk * cl) cl *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, N, jb * cl);
  cfg.blockDim = dim3(kSumThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = cl;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, a);
  if (err == cudaSuccess) launch_counter().fetch_add(1, std::memory_order_relaxed);
  return err;
}

template <int R>
cudaError_t launch_sum_rank(SumArgs& a, bool f16, int N, int rows, int sms, cudaStream_t s) {
  if (f16) {
    const size_t smem = 2 * (size_t)(kSumStages * kRows * kLdX + 4 * kRows * (R + 8));
    return launch_sum(row_sum_f16_kernel<R>, smem, a, kIT, R, N, rows, kRows, sms, s);
  }
  const size_t smem = sizeof(float) * std::max(kRows32 * R, kIT32 * (R + 1));
  return launch_sum(row_sum_f32_kernel<R>, smem, a, kIT32, R, N, rows, kRows32, sms, s);
}

// ---------------------------------------------------------------- tokens' gradient of the gate
// out[t,i] = in[t,i] + sum_e dl[t,e] W[i,e], fused multiply-adds on 64 x 64 tiles.
template <typename T>
__global__ void __launch_bounds__(256) gate_dx_kernel(const float* __restrict__ dl,
                                                      const float* __restrict__ W,
                                                      const T* __restrict__ in, int rows, int d,
                                                      int E, T* __restrict__ out) {
  __shared__ float as[16][68], bs[16][68];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int i0 = blockIdx.y * 64, t0 = blockIdx.x * 64;
  float acc[4][4] = {};
  for (int e0 = 0; e0 < E; e0 += 16) {
    __syncthreads();
    for (int q = tid; q < 64 * 16; q += 256) {
      const int r = q >> 4, e = q & 15;
      as[e][r] = t0 + r < rows && e0 + e < E ? dl[(size_t)(t0 + r) * E + e0 + e] : 0.f;
      bs[e][r] = i0 + r < d && e0 + e < E ? W[(size_t)(i0 + r) * E + e0 + e] : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float4 u = *reinterpret_cast<const float4*>(&as[e][ty * 4]);
      const float4 v = *reinterpret_cast<const float4*>(&bs[e][tx * 4]);
      const float av[4] = {u.x, u.y, u.z, u.w}, bv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + ty * 4 + i;
    if (t >= rows) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = i0 + tx * 4 + j;
      if (c >= d) continue;
      const size_t at = (size_t)t * d + c;
      float v = acc[i][j];
      if (in) v += (float)in[at];
      out[at] = (T)v;
    }
  }
}

// ---------------------------------------------------------------- combine's gradient
// dy_s = w_tj dout_t,  dw_tj = <dout_t, y_s>,  s = slot_of[t,j].  Bound by DRAM: dout, y read
// once, dy written once.  WPR warps per token row (8 where there are too few rows to fill the
// device with a warp each).
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
              *reinterpret_cast<Vec*>(dy + (int64_t)s[j] * d + c) = o;
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
  if (T_ < 16 * sms)
    return launch_k(combine_backward_kernel<T, V, 8>, std::min(T_, 8 * sms), 256, 0, s, false, du, yy,
                    slot_of, topk_w, T_, d, k, S_max, static_cast<T*>(dy), dw);
  return launch_k(combine_backward_kernel<T, V, 1>, std::min((T_ + 7) / 8, 8 * sms), 256, 0, s, false,
                  du, yy, slot_of, topk_w, T_, d, k, S_max, static_cast<T*>(dy), dw);
}

}  // namespace

cudaError_t launch_row_sums(const void* x0, const float* h0, float* G0, int di0, int dj0, int tr0,
                            const void* x1, const float* h1, float* G1, int di1, int dj1, int tr1,
                            const float* scale, const int32_t* perm, const int32_t* offsets,
                            const uint8_t* mask, int dtype_f16, int T, int S_max, int N,
                            cudaStream_t s) {
  const int sms = sms_of_device();
  if (sms < 1) return cudaErrorInvalidDevice;
  SumArgs a;
  a.job[0] = SumJob{x0, h0, G0, di0, dj0, tr0, 0};
  a.job[1] = SumJob{x1, h1, G1, di1, dj1, tr1, 0};
  a.scale = scale;
  a.perm = perm;
  a.offsets = offsets;
  a.mask = mask;
  a.T = T;
  a.S_max = S_max;
  const int rows = offsets ? S_max / N : S_max;
  const int dj = std::max(G0 ? dj0 : 0, G1 ? dj1 : 0);
  if (dj <= 16) return launch_sum_rank<16>(a, dtype_f16, N, rows, sms, s);
  if (dj <= 32) return launch_sum_rank<32>(a, dtype_f16, N, rows, sms, s);
  if (dj <= 64) return launch_sum_rank<64>(a, dtype_f16, N, rows, sms, s);
  return launch_sum_rank<128>(a, dtype_f16, N, rows, sms, s);
}

cudaError_t launch_gate_dx(const float* dlogits, const float* Wg, const void* in, int dtype_f16, int T,
                           int d, int E, void* out, cudaStream_t s) {
  const dim3 grid((T + 63) / 64, (d + 63) / 64);
  if (dtype_f16)
    return launch_k(gate_dx_kernel<__half>, grid, 256, 0, s, false, dlogits, Wg,
                    static_cast<const __half*>(in), T, d, E, static_cast<__half*>(out));
  return launch_k(gate_dx_kernel<float>, grid, 256, 0, s, false, dlogits, Wg,
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
