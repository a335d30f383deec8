// Router losses over the gate's logits, and the gradient of the logits.
//
//   p = softmax(x_t),  lse_t = log sum_e exp(x_te),  n = tokens that count
//   counts[e] = #{(t, j): token t counts, topk_idx[t,j] = e},   P[e] = 1/n sum_t p_te
//   balance = E sum_e counts[e] / (n k) P[e],   z = 1/n sum_t lse_t^2
//
//   dx_te = p_te (a_e - sum_e' a_e' p_te') + 2 g_z / n lse_t p_te       (tokens that count)
//         + gradient of the gate weights at the chosen experts  (0 for tokens that do not count),
//   a_e = g_balance E counts[e] / (n^2 k)
//
// Both are one pass over [T, E] in 32 bits, bound by DRAM (4 bytes read per element, 4 more
// written by the gradient).  A row is held in registers by LANES lanes with 16 (E > 512: 32) values
// each: a row's reductions are log2(LANES) shuffles (with 8 values per lane the shuffles bound the
// passes: moe_balance_loss's over 262144 x 128 logits 40 us instead of 28).  The columns of a lane
// never change, so column sums (forward) and a_e (backward) stay in registers too.
#include <cooperative_groups.h>

#include <algorithm>

#include "gate_split.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kRowThreads = 512;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kCluster = 8;
constexpr int kFinalThreads = 1024;
// Parts of a column's sum over the records (one thread adds them up: 1024 of them took 10 us).
constexpr int kJoinParts = 64;

template <int LANES>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Element e of value (j, v) in lane l of a row's group.
template <int LANES, int VEC>
__device__ __forceinline__ int col_of(int j, int l) { return (j * LANES + l) * VEC; }

// One row's values (columns beyond E and rows that do not count: -inf).
template <int LANES, int VEC, int J>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int l, bool on,
                                         float (&x)[VEC * J]) {
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = col_of<LANES, VEC>(j, l);
    if (on && c < E) {
      if (VEC == 4) {
        const float4 q = *reinterpret_cast<const float4*>(row + c);
        x[4 * j + 0] = q.x; x[4 * j + 1] = q.y; x[4 * j + 2] = q.z; x[4 * j + 3] = q.w;
      } else {
        x[j] = row[c];
      }
    } else {
#pragma unroll
      for (int v = 0; v < VEC; ++v) x[VEC * j + v] = -INFINITY;
    }
  }
}

// Softmax in place: x becomes p (exp_row: p / inv); returns lse.  The exponentials are the hardware's (2 ulp and
// 2^-23 of |x - m| relative: small where p matters); with expf the arithmetic, not DRAM, bound the
// pass over 262144 x 128 logits (31 us instead of 28).  A row of -inf only has p = 0 and lse = 0 (it
// adds nothing to either loss); NaN and +inf give NaN as the formula does.
template <int LANES, int N>
__device__ __forceinline__ float exp_row(float (&x)[N], float& inv) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
  m = group_max<LANES>(m);
  if (m == -INFINITY) m = 0.f;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = __expf(x[i] - m);
    s += x[i];
  }
  s = group_sum<LANES>(s);
  const bool empty = s == 0.f;
  inv = empty ? 0.f : 1.f / s;
  return empty ? 0.f : m + logf(s);
}
template <int LANES, int N>
__device__ __forceinline__ float softmax_row(float (&x)[N]) {
  float inv;
  const float lse = exp_row<LANES>(x, inv);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] *= inv;
  return lse;
}

// Sum of v over the block, in a fixed order; the result is valid in thread 0.
__device__ __forceinline__ float block_sum(float v, float* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = 0.f;
  if (threadIdx.x == 0)
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) r += scratch[w];
  return r;
}

// The two halves of a cluster's barrier, with work between them (every thread of every block).
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

struct LossOut {
  int32_t* counts;
  float* prob_mean;
  float* losses;
  int32_t* n_valid;
};

// Per-block partial sums, one record per block: probability sums [E], counts [E], then the sum
// of lse^2 and the number of tokens.
__host__ __device__ inline size_t record_words(int E) { return 2 * (size_t)E + 4; }

// Joins nb records (rec(b) is record b) into the outputs.  Runs in one cluster of up to kCluster
// blocks: block c owns the columns [c Ec, (c + 1) Ec); its threads sum each column in
// up to kJoinParts parts, always in the same order, and rank 0 adds the blocks' shares of the
// balance loss through distributed shared memory.
template <typename Rec>
__device__ __forceinline__ void join_records(Rec rec, int nb, int E, int k, LossOut o, float* sh_f,
                                             int* sh_i, float* share) {
  cg::cluster_group cl = cg::this_cluster();
  cluster_arrive();                                 // waited for below, behind the records' loads
  const int c = (int)cl.block_rank(), ncl = (int)cl.num_blocks();
  const int Ec = (E + ncl - 1) / ncl;                // at most blockDim
  const int parts = max(1, min((int)blockDim.x / Ec, min(nb, kJoinParts)));
  const int col = threadIdx.x % Ec, part = threadIdx.x / Ec;
  const int e = c * Ec + col;
  float ps = 0.f;
  int cs = 0, n = 0;
  if (part < parts && e < E) {
#pragma unroll 8
    for (int b = part; b < nb; b += parts) {
      const float* r = rec(b);
      ps += r[e];
      cs += __float_as_int(r[E + e]);
    }
  }
  // every block needs n; only rank 0 needs the sum of lse^2
  float z = 0.f;
  for (int b = threadIdx.x; b < nb; b += blockDim.x) {
    const float* r = rec(b);
    z += r[2 * E];
    n += __float_as_int(r[2 * E + 1]);
  }
  if (part < parts) {
    sh_f[threadIdx.x] = ps;
    sh_i[threadIdx.x] = cs;
  }
  __shared__ int n_sh;
  __shared__ float scratch[kFinalThreads / 32];
  if (threadIdx.x == 0) n_sh = 0;
  __syncthreads();
  if (n) atomicAdd(&n_sh, n);
  z = block_sum(z, scratch);                        // its barriers publish n_sh and sh_*
  const float nf = (float)max(n_sh, 1);
  float mine = 0.f;
  if (threadIdx.x < (unsigned)Ec && e < E) {
    float p = 0.f;
    int cnt = 0;
    for (int q = 0; q < parts; ++q) {
      p += sh_f[q * Ec + col];
      cnt += sh_i[q * Ec + col];
    }
    p /= nf;
    o.prob_mean[e] = p;
    o.counts[e] = cnt;
    mine = (float)cnt * p;
  }
  mine = block_sum(mine, scratch);
  cluster_wait();                                   // rank 0 has started: its shared memory is there
  if (threadIdx.x == 0) cl.map_shared_rank(share, 0)[c] = mine;
  cl.sync();
  if (c == 0 && threadIdx.x == 0) {
    float s = 0.f;
    for (int q = 0; q < ncl; ++q) s += share[q];
    o.losses[0] = (float)E * (s / (nf * (float)k));
    o.losses[1] = z / nf;
    *o.n_valid = n_sh;
  }
}

// kOne: the grid is one cluster, which keeps its records in shared memory and joins them itself
// (small batches: one launch).  Otherwise records go to the workspace and balance_join_kernel
// follows.  262144 x 128 logits: 28 us (4.8 TB/s; exponentials, shuffles and loads share the issue
// slots at 32 warps per SM), then 6 to 8 us for the join's chain of loads and one cluster exchange.
template <int LANES, int VEC, int J, bool kOne>
__global__ void __launch_bounds__(kRowThreads, VEC * J > 16 ? 1 : 2) balance_rows_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
    const uint8_t* __restrict__ mask, int T, int E, int k, float* __restrict__ records, LossOut o) {
  constexpr int V = VEC * J;
  constexpr int RPW = 32 / LANES;
  extern __shared__ float sm[];
  float* red = sm;                                            // [kRowWarps][E]
  int* hist = reinterpret_cast<int*>(sm + kRowWarps * E);     // [E]
  float* rec_s = sm + (kRowWarps + 1) * E;                    // kOne: this block's record
  __shared__ float zs[kRowWarps];
  __shared__ int ns[kRowWarps];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int l = lane % LANES, g = lane / LANES;
  for (int e = threadIdx.x; e < E; e += kRowThreads) hist[e] = 0;
  __syncthreads();
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  float z = 0.f;
  int n = 0;
  const int64_t stride = (int64_t)gridDim.x * kRowWarps * RPW;
  // (Fetching the next row ahead costs a third of the warps in registers: 32 us instead of 28.)
  for (int64_t base = ((int64_t)blockIdx.x * kRowWarps + w) * RPW; base < T; base += stride) {
    const int64_t t = base + g;
    const bool on = t < T && (!mask || mask[t]);
    float x[V];
    load_row<LANES, VEC, J>(logits + (on ? t : 0) * E, E, l, on, x);
    if (on) {
      for (int j = l; j < k; j += LANES) {
        const int e = topk_idx[t * k + j];
        if ((unsigned)e < (unsigned)E) atomicAdd(&hist[e], 1);
      }
    }
    float inv;
    const float lse = exp_row<LANES>(x, inv);                 // all zero for a row that is off
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = fmaf(x[i], inv, acc[i]);
    if (on && l == 0) {
      z += lse * lse;
      n += 1;
    }
  }
  // rows of a warp, then warps, in a fixed order
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int s = LANES; s < 32; s <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], s);
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    z += __shfl_xor_sync(0xffffffffu, z, s);
    n += __shfl_xor_sync(0xffffffffu, n, s);
  }
  if (g == 0) {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const int e = col_of<LANES, VEC>(j, l) + v;
        if (e < E) red[w * E + e] = acc[VEC * j + v];
      }
  }
  if (lane == 0) {
    zs[w] = z;
    ns[w] = n;
  }
  __syncthreads();
  float* rec = kOne ? rec_s : records + (size_t)blockIdx.x * record_words(E);
  for (int e = threadIdx.x; e < E; e += kRowThreads) {
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < kRowWarps; ++q) s += red[q * E + e];
    rec[e] = s;
    rec[E + e] = __int_as_float(hist[e]);
  }
  if (w == kRowWarps - 1) {                         // the last warp has the fewest columns
    float zz = lane < kRowWarps ? zs[lane] : 0.f;
    int nn = lane < kRowWarps ? ns[lane] : 0;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
      zz += __shfl_xor_sync(0xffffffffu, zz, s);
      nn += __shfl_xor_sync(0xffffffffu, nn, s);
    }
    if (lane == 0) {
      rec[2 * E] = zz;
      rec[2 * E + 1] = __int_as_float(nn);
    }
  }
  if (kOne) {
    __shared__ float sh_f[kRowThreads];
    __shared__ int sh_i[kRowThreads];
    __shared__ float share[kCluster];
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();                                      // every block's record is complete
    join_records([&](int b) { return (const float*)cl.map_shared_rank(rec_s, b); },
                 (int)cl.num_blocks(), E, k, o, sh_f, sh_i, share);
    // its last cluster barrier is behind every read of another block's record
  } else {
    pdl_trigger();
  }
}

__global__ void __launch_bounds__(kFinalThreads) balance_join_kernel(
    const float* __restrict__ records, int nb, int E, int k, LossOut o) {
  __shared__ float sh_f[kFinalThreads];
  __shared__ int sh_i[kFinalThreads];
  __shared__ float share[kCluster];
  pdl_wait();
  const size_t words = record_words(E);
  join_records([&](int b) { return records + b * words; }, nb, E, k, o, sh_f, sh_i, share);
}

struct DlArgs {
  const float* logits;
  const int32_t* topk_idx;
  const float *dtopk_w, *dlosses;
  const int32_t *counts, *n_valid;
  const uint8_t* mask;
  int T, E, k;
  float* dlogits;
  int* status;                 // cleared, or null
};

// What every row needs: a_e of this lane's columns and the factor of the z loss.
template <int LANES, int VEC, int J>
__device__ __forceinline__ float loss_factors(const DlArgs& d, int l, float (&a)[VEC * J]) {
  if (!d.dlosses) return 0.f;
  const float n = (float)max(*d.n_valid, 1);
  const float cb = d.dlosses[0] * (float)d.E / (n * (float)d.k) / n;
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const int e = col_of<LANES, VEC>(j, l) + v;
      a[VEC * j + v] = e < d.E ? cb * (float)d.counts[e] : 0.f;
    }
  return 2.f * d.dlosses[1] / n;
}

// The row's logits x become their gradient (zero for a row that is off).
template <int LANES, int VEC, int J>
__device__ __forceinline__ void row_gradient(const DlArgs& d, int64_t t, bool on, int l,
                                             const float (&a)[VEC * J], float gz, float (&x)[VEC * J]) {
  constexpr int V = VEC * J;
  float top[2] = {0.f, 0.f}, dw[2] = {0.f, 0.f};
  int idx[2] = {-1, -1};
  if (d.dtopk_w && on) {
    for (int j = 0; j < d.k; ++j) {
      const int e = d.topk_idx[(size_t)t * d.k + j];
      if ((unsigned)e < (unsigned)d.E) {
        idx[j] = e;
        dw[j] = d.dtopk_w[(size_t)t * d.k + j];
      }
    }
  }
  // the chosen experts' logits, from the lane that holds them
  if (d.dtopk_w) {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const int c = col_of<LANES, VEC>(j, l) + v;
        if (c == idx[0]) top[0] = x[VEC * j + v];
        if (c == idx[1]) top[1] = x[VEC * j + v];
      }
    top[0] = group_sum<LANES>(top[0]);
    top[1] = group_sum<LANES>(top[1]);
  }
  const float lse = softmax_row<LANES>(x);                   // x is p now
  float bar = 0.f;
  if (d.dlosses) {
#pragma unroll
    for (int i = 0; i < V; ++i) bar += a[i] * x[i];
  }
  bar = group_sum<LANES>(bar);
  // top-1: w = p[e1];  top-2: w_j = p[e_j] / (p[e1] + p[e2]), a softmax over the two logits
  float add[2] = {0.f, 0.f}, minus = 0.f;
  if (d.dtopk_w) {
    if (d.k == 1) {
      // a row of -inf only has no weight to differentiate (p = 0 there)
      const float p1 = idx[0] < 0 || top[0] == -INFINITY ? 0.f : expf(top[0] - lse);
      add[0] = p1 * dw[0];
      minus = add[0];
    } else if (idx[0] >= 0 && idx[1] >= 0 && idx[0] != idx[1] &&
               !(top[0] == -INFINITY && top[1] == -INFINITY)) {
      const float hi = fmaxf(top[0], top[1]);
      const float e0 = expf(top[0] - hi), e1 = expf(top[1] - hi);
      const float inv = 1.f / (e0 + e1);
      add[0] = (e0 * inv) * (e1 * inv) * (dw[0] - dw[1]);
      add[1] = -add[0];
    }
  }
  const float c0 = gz * lse - bar;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = col_of<LANES, VEC>(j, l);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float p = x[VEC * j + v];
      float r = d.dlosses ? p * (a[VEC * j + v] + c0) : 0.f;
      if (d.dtopk_w) {
        r -= p * minus;
        if (c + v == idx[0]) r += add[0];
        if (c + v == idx[1]) r += add[1];
      }
      x[VEC * j + v] = r;
    }
  }
}

template <int LANES, int VEC, int J>
__device__ __forceinline__ void store_row(const DlArgs& d, int64_t t, int l, const float (&q)[VEC * J]) {
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = col_of<LANES, VEC>(j, l);
    if (c >= d.E) continue;
    float* dst = d.dlogits + (size_t)t * d.E + c;
    if (VEC == 4)
      *reinterpret_cast<float4*>(dst) =
          make_float4(q[VEC * j], q[VEC * j + 1 % VEC], q[VEC * j + 2 % VEC], q[VEC * j + 3 % VEC]);
    else
      dst[0] = q[j];
  }
}

// Gradient of the logits, one row per group of lanes.  Rows are taken from the last to the
// first: right after moe_balance_loss the rows that it read last are still in L2.  262144 x 128
// logits: 43 us, 6.2 TB/s read and written (DRAM; streaming stores changed nothing).
template <int LANES, int VEC, int J>
__global__ void __launch_bounds__(256) dlogits_kernel(const DlArgs d) {
  if (d.status && blockIdx.x == 0 && threadIdx.x == 0) *d.status = kOk;
  constexpr int V = VEC * J, RPW = 32 / LANES;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int l = lane % LANES, g = lane / LANES;
  float a[V];
  const float gz = loss_factors<LANES, VEC, J>(d, l, a);
  const int64_t stride = (int64_t)gridDim.x * 8 * RPW;
  for (int64_t base = ((int64_t)blockIdx.x * 8 + w) * RPW; base < d.T; base += stride) {
    const int64_t t = d.T - 1 - (base + g);
    const bool in = t >= 0, on = in && (!d.mask || d.mask[t]);
    float x[V];
    load_row<LANES, VEC, J>(d.logits + (on ? t : 0) * d.E, d.E, l, on, x);
    row_gradient<LANES, VEC, J>(d, t, on, l, a, gz, x);
    if (in) store_row<LANES, VEC, J>(d, t, l, x);
  }
}

// The same with the f16 parts that the tensor-core form of the gate's gradient multiplies
// (gate_grad.cu): a block takes 128 rows, writes their gradients in 32 bits, and when it knows their
// largest magnitude also as (hi, lo) with v = (hi + 2^-11 lo) 2^e.  16384 x 128 with a Wg of 3584 rows:
// 12 us: a block's chain of loads, two block-wide steps and stores, and one block per SM (512 threads of 73
// registers), so that the last four of the 156 blocks run behind the others.
// Blocks beyond the rows split Wg in the same way.
struct SplitOut {
  __half* dl2;                 // [T][2 Ep]: hi, lo; columns beyond E are zero
  float* sT;                   // [T / 128]
  const float* Wg;             // [d, E], or null
  __half* W2;                  // [d][2 Ep], as dl2
  float* sW;                   // [d / 128]
  int d, Ep, nT;
};
constexpr int kSplitThreads = 512;

// Largest magnitude in the block (of its finite values: infinities and NaN need no scale, and must
// not take the others' away).
__device__ __forceinline__ float block_max(float m, float* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kSplitThreads / 32; ++q) m = fmaxf(m, scratch[q]);
  return m;
}
__device__ __forceinline__ float magnitude(float v) { return v - v == 0.f ? fabsf(v) : 0.f; }

__device__ __forceinline__ void split_one(float x, __half& h, __half& l) {
  h = __float2half_rn(x);
  const float b = __half2float(h);
  l = isfinite(b) ? __float2half_rn((x - b) * kGateLo) : __ushort_as_half(0);
}
__device__ __forceinline__ void split_four(const float (&f)[4], float inv, __half* hi, __half* lo) {
  __half h[4], l[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) split_one(f[v] * inv, h[v], l[v]);
  *reinterpret_cast<uint2*>(hi) = *reinterpret_cast<const uint2*>(h);
  *reinterpret_cast<uint2*>(lo) = *reinterpret_cast<const uint2*>(l);
}

// Splits rows x E values (m: their largest magnitude) into f16 parts of `ld` columns; returns the power
// of two.
// A warp takes rows; eight loads are issued before the first result is stored (the compiler cannot
// move loads over stores that might alias them).
template <int VEC>
__device__ __forceinline__ float split_block(const float* src, int rows, int E, int Ep, float m, __half* hi,
                                             __half* lo, int ld) {
  const int e = scale_exp(m);
  const float inv = exp2_int(-e);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  constexpr int kW = kSplitThreads / 32, UR = VEC == 4 ? 4 : 2, UC = VEC == 4 ? 1 : 4;
  for (int r0 = w; r0 < rows; r0 += kW * UR) {
    for (int c0 = lane * VEC; c0 < Ep; c0 += 32 * VEC * UC) {
      float f[UR][UC][VEC];
#pragma unroll
      for (int i = 0; i < UR; ++i)
#pragma unroll
        for (int j = 0; j < UC; ++j) {
          const int r = r0 + i * kW, c = c0 + j * 32 * VEC;
#pragma unroll
          for (int v = 0; v < VEC; ++v) f[i][j][v] = 0.f;
          if (r < rows && c < E) {
            if (VEC == 4)
              *reinterpret_cast<float4*>(f[i][j]) = *reinterpret_cast<const float4*>(src + r * E + c);
            else
              f[i][j][0] = src[r * E + c];
          }
        }
#pragma unroll
      for (int i = 0; i < UR; ++i)
#pragma unroll
        for (int j = 0; j < UC; ++j) {
          const int r = r0 + i * kW, c = c0 + j * 32 * VEC;
          if (r >= rows || c >= Ep) continue;
          __half* p = hi + (size_t)r * ld + c;
          if constexpr (VEC == 4) {
            split_four(f[i][j], inv, p, p + (lo - hi));
          } else {
            __half h, l;
            split_one(f[i][j][0] * inv, h, l);
            p[0] = h;
            p[lo - hi] = l;
          }
        }
    }
  }
  return exp2_int(e);
}

template <int LANES, int VEC, int J>
__global__ void __launch_bounds__(kSplitThreads) dlogits_split_kernel(const DlArgs d, const SplitOut o) {
  constexpr int V = VEC * J, RPW = 32 / LANES;
  __shared__ float scratch[kSplitThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  pdl_trigger();
  if ((int)blockIdx.x >= o.nT) {
    const int blk = blockIdx.x - o.nT, rows = min(kGateBlock, o.d - blk * kGateBlock);
    const float* src = o.Wg + (size_t)blk * kGateBlock * d.E;
    __half* dst = o.W2 + (size_t)blk * kGateBlock * 2 * o.Ep;
    float m = 0.f;
    if (VEC == 4) {
#pragma unroll 8
      for (int q = tid; q < rows * d.E / 4; q += kSplitThreads) {
        const float4 v = reinterpret_cast<const float4*>(src)[q];
        m = fmaxf(fmaxf(m, fmaxf(magnitude(v.x), magnitude(v.y))), fmaxf(magnitude(v.z), magnitude(v.w)));
      }
    } else {
#pragma unroll 8
      for (int q = tid; q < rows * d.E; q += kSplitThreads) m = fmaxf(m, magnitude(src[q]));
    }
    m = block_max(m, scratch);
    const float s = split_block<VEC>(src, rows, d.E, o.Ep, m, dst, dst + o.Ep, 2 * o.Ep);
    if (tid == 0) o.sW[blk] = s;
    return;
  }
  if (d.status && blockIdx.x == 0 && tid == 0) *d.status = kOk;
  const int l = lane % LANES, g = lane / LANES;
  float a[V];
  const float gz = loss_factors<LANES, VEC, J>(d, l, a);
  const int row0 = blockIdx.x * kGateBlock, rows = min(kGateBlock, d.T - row0);
  __half* dst = o.dl2 + (size_t)row0 * 2 * o.Ep;
  constexpr int kPass = kSplitThreads / 32 * RPW;            // rows per pass
  constexpr int NP = kPass >= kGateBlock ? 1 : kGateBlock / kPass;
  if constexpr (VEC == 4) {
    // The block's gradients stay in registers until their largest magnitude is known (read back
    // instead: 16 us, not 13, for 16384 x 128).
    float x[NP][V];
    float m = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int r = p * kPass + w * RPW + g;
      const int64_t t = (int64_t)row0 + r;
      const bool in = r < rows, on = in && (!d.mask || d.mask[t]);
      load_row<LANES, VEC, J>(d.logits + (on ? t : 0) * d.E, d.E, l, on, x[p]);
      row_gradient<LANES, VEC, J>(d, t, on, l, a, gz, x[p]);
      if (in) store_row<LANES, VEC, J>(d, t, l, x[p]);
#pragma unroll
      for (int i = 0; i < V; ++i) m = fmaxf(m, magnitude(x[p][i]));
    }
    m = block_max(m, scratch);
    const int e = scale_exp(m);
    const float inv = exp2_int(-e);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int r = p * kPass + w * RPW + g;
      if (r >= rows) continue;
      __half* hi = dst + (size_t)r * 2 * o.Ep;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = col_of<LANES, VEC>(j, l);
        if (c >= o.Ep) continue;
        float f[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) f[v] = c < d.E ? x[p][4 * j + v] : 0.f;
        split_four(f, inv, hi + c, hi + o.Ep + c);
      }
    }
    // columns up to Ep that no lane's values cover
    const int rest = (o.Ep - LANES * V) / 8;
    if (rest > 0) {
      for (int q = tid; q < rows * 2 * rest; q += kSplitThreads) {
        const int r = q / (2 * rest), c = q - r * (2 * rest);
        __half* at = dst + (size_t)r * 2 * o.Ep + (c < rest ? LANES * V + c * 8 : o.Ep + LANES * V + (c - rest) * 8);
        *reinterpret_cast<uint4*>(at) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    if (tid == 0) o.sT[blockIdx.x] = exp2_int(e);
  } else {
    // Odd row lengths: written in 32 bits and read back (the unrolled passes of scalar accesses were
    // fetched as instructions for longer than they ran: 38 us instead of 14 for 38 x 129).
    float m = 0.f;
    for (int r0 = w * RPW; r0 < rows; r0 += kPass) {
      const int r = r0 + g;
      const int64_t t = (int64_t)row0 + r;
      const bool in = r < rows, on = in && (!d.mask || d.mask[t]);
      float x[V];
      load_row<LANES, VEC, J>(d.logits + (on ? t : 0) * d.E, d.E, l, on, x);
      row_gradient<LANES, VEC, J>(d, t, on, l, a, gz, x);
      if (in) store_row<LANES, VEC, J>(d, t, l, x);
#pragma unroll
      for (int i = 0; i < V; ++i) m = fmaxf(m, magnitude(x[i]));
    }
    m = block_max(m, scratch);                     // behind its barrier the block's rows are written
    const float s = split_block<VEC>(d.dlogits + (size_t)row0 * d.E, rows, d.E, o.Ep, m, dst, dst + o.Ep, 2 * o.Ep);
    if (tid == 0) o.sT[blockIdx.x] = s;
  }
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

// Lanes per row and values per lane (see the top); four-wide accesses where a row's length allows.
template <typename F>
cudaError_t with_shape(int E, F f) {
  auto pick = [&](auto vec) -> cudaError_t {
    constexpr int VEC = decltype(vec)::value;
    constexpr int J = 16 / VEC;
    using std::integral_constant;
    if (E <= 16) return f(integral_constant<int, 1>(), vec, integral_constant<int, J>());
    if (E <= 32) return f(integral_constant<int, 2>(), vec, integral_constant<int, J>());
    if (E <= 64) return f(integral_constant<int, 4>(), vec, integral_constant<int, J>());
    if (E <= 128) return f(integral_constant<int, 8>(), vec, integral_constant<int, J>());
    if (E <= 256) return f(integral_constant<int, 16>(), vec, integral_constant<int, J>());
    if (E <= 512) return f(integral_constant<int, 32>(), vec, integral_constant<int, J>());
    return f(integral_constant<int, 32>(), vec, integral_constant<int, 2 * J>());
  };
  return E % 4 == 0 ? pick(std::integral_constant<int, 4>()) : pick(std::integral_constant<int, 1>());
}

int lanes_for(int E) {
  int lanes = 1;
  while (lanes < 32 && lanes * 16 < E) lanes <<= 1;
  return lanes;
}

// Blocks of the row pass: as many as an SM holds (see its launch bounds), fewer for short batches.
constexpr int kMaxRecords = 512;
// Rows that a block of the row pass takes at once.
int block_rows(int E) { return kRowWarps * (32 / lanes_for(E)); }
int row_blocks(int T, int E, int sms) {
  const int rows = block_rows(E);
  return std::max(1, std::min({(T + rows - 1) / rows, (E > 512 ? 1 : 2) * sms, kMaxRecords}));
}

// Up to this many passes of eight blocks over the rows one cluster does the whole call (one block where
// a pass covers the batch, else up to eight).  us on the GPU with the gradient's call after it, two launches /
// one: E = 128, 900 rows (two passes) 10.0 / 10.4, E = 16, 8000 rows (two) 10.9 / 11.5, E = 64, 2000 rows
// (two) 10.1 / 10.1, 3000 rows (three) 10.2 / 11.2, E = 60, 4099 rows (five) 10.7 / 13.8.  The second launch is
// 2.3 us of the host's time, which a captured step or a stream with work ahead does not see: so one cluster
// where the GPU takes as long either way.
constexpr int kOnePasses = 2;

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), int grid, int block, size_t smem,
                           cudaStream_t s, bool pdl, Args&&... args) {   // the grid is one cluster
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = grid;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
  if (err == cudaSuccess) launch_counter().fetch_add(1, std::memory_order_relaxed);
  return err;
}

}  // namespace

size_t balance_records_bytes(int E) { return sizeof(float) * kMaxRecords * record_words(E); }

cudaError_t launch_balance_loss(const float* logits, const int32_t* topk_idx, const uint8_t* mask,
                                int T, int E, int k, int32_t* counts, float* prob_mean,
                                float* losses, int32_t* n_valid, float* records, cudaStream_t s) {
  const int sms = sm_count();
  if (sms < 1) return cudaErrorInvalidDevice;
  const LossOut o{counts, prob_mean, losses, n_valid};
  const bool one = T <= kOnePasses * kCluster * block_rows(E);
  int blocks = row_blocks(T, E, sms);
  if (one) {                                       // a power of two, whose blocks hold E columns
    int c = 1;
    while (c < kCluster && (c < blocks || c * kRowThreads < E)) c *= 2;
    blocks = c;
  }
  const size_t smem = sizeof(float) * ((size_t)(kRowWarps + 1) * E + (one ? record_words(E) : 0));
  return with_shape(E, [&](auto lanes, auto vec, auto j) -> cudaError_t {
    constexpr int L = decltype(lanes)::value, V = decltype(vec)::value, J = decltype(j)::value;
    if (one) {
      auto kern = balance_rows_kernel<L, V, J, true>;
      MOE_LAUNCH(ensure_smem_attr(reinterpret_cast<const void*>(kern)));
      return launch_cluster(kern, blocks, kRowThreads, smem, s, false, logits, topk_idx, mask, T, E,
                            k, records, o);
    }
    auto kern = balance_rows_kernel<L, V, J, false>;
    MOE_LAUNCH(ensure_smem_attr(reinterpret_cast<const void*>(kern)));
    MOE_LAUNCH(launch_k(kern, blocks, kRowThreads, smem, s, false, logits, topk_idx, mask, T, E, k,
                        records, o));
    return launch_cluster(balance_join_kernel, kCluster, kFinalThreads, 0, s, true,
                          (const float*)records, blocks, E, k, o);
  });
}

cudaError_t launch_dlogits(const float* logits, const int32_t* topk_idx, const float* dtopk_w,
                           const float* dlosses, const int32_t* counts, const int32_t* n_valid,
                           const uint8_t* mask, int T, int E, int k, float* dlogits, int* status,
                           cudaStream_t s) {
  const int sms = sm_count();
  if (sms < 1) return cudaErrorInvalidDevice;
  const DlArgs d{logits, topk_idx, dtopk_w, dlosses, counts, n_valid, mask, T, E, k, dlogits, status};
  const int rows = 8 * (32 / lanes_for(E));
  const int grid = std::max(1, std::min((T + rows - 1) / rows, 8 * sms));
  return with_shape(E, [&](auto lanes, auto vec, auto j) -> cudaError_t {
    constexpr int L = decltype(lanes)::value, V = decltype(vec)::value, J = decltype(j)::value;
    return launch_k(dlogits_kernel<L, V, J>, grid, 256, 0, s, false, d);
  });
}

cudaError_t launch_dlogits_split(const float* logits, const int32_t* topk_idx, const float* dtopk_w,
                                 const float* dlosses, const int32_t* counts, const int32_t* n_valid,
                                 const uint8_t* mask, int T, int E, int k, float* dlogits, int* status,
                                 const float* Wg, int d, int Ep, __half* dl2, float* sT, __half* W2,
                                 float* sW, cudaStream_t s) {
  const DlArgs a{logits, topk_idx, dtopk_w, dlosses, counts, n_valid, mask, T, E, k, dlogits, status};
  const SplitOut o{dl2, sT, Wg, W2, sW, d, Ep, (T + kGateBlock - 1) / kGateBlock};
  const int grid = o.nT + (Wg ? (d + kGateBlock - 1) / kGateBlock : 0);
  return with_shape(E, [&](auto lanes, auto vec, auto j) -> cudaError_t {
    constexpr int L = decltype(lanes)::value, V = decltype(vec)::value, J = decltype(j)::value;
    if constexpr (L > 16)
      return cudaErrorInvalidValue;               // E > 256 takes the other form
    else
      return launch_k(dlogits_split_kernel<L, V, J>, grid, kSplitThreads, 0, s, false, a, o);
  });
}

}  // namespace moe
