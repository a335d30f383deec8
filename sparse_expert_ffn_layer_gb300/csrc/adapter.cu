// Low-rank adapters of many requests beside a shared projection, and the gradient of their
// input: for the slots s of adapter n (token t = perm[s]),
//
//   h_s = x_t P_n           [r]      (forward: P = A, Q = B;  gradient: P = B^T, Q = A^T)
//   y_t = base_t + scale_n h_s Q_n   (base may be absent)
//
// x and base are read and y written once, the weights of the adapters in use come once from DRAM
// and then from L2; 4 r operations per token and column pair stay below the tensor rate for
// r <= 128.  Those bytes are the floor; short runs are bound by their chain of latencies and long
// runs by fragment loads and products (see either).
//
// Short runs (a few rows per adapter: decode) and 32-bit inputs take one launch for both
// products.  A cluster of eight blocks takes a tile of 16 rows of one adapter;
// each block multiplies its eighth of the input columns (so a single token's weights are pulled
// by eight SMs), the partial h are summed over the cluster through distributed shared memory in
// rank order (no atomics: equal calls give equal bits), each block receives the whole h and
// multiplies it into its eighth of the output columns.  Both products of all tiles of a cluster
// run through one ring of asynchronous 128-byte-wide chunks, so that the first output chunks
// (base and Q) load while h is being exchanged, and the next tile's rows while this one is
// written.  Long runs (tiles of 64 rows) take two launches, see there.
//
// f16: h is kept in 32 bits (and given out so).  For the second product each row is scaled by a power
// of two, so that no h overflows or is lost below f16's range, and split into two f16 parts: together
// h to 2^-23 of itself, 2^-39 of the row's largest, so that y differs from the 32-bit form's by 32-bit
// rounding before its own 2^-11 |y|.  (One part only: the error of 8192 rows of dtokens, r = 32, was
// 1.37 times that of 32-bit sums.)  f32: fused multiply-adds on the CUDA cores.
#include <cooperative_groups.h>

#include <algorithm>
#include <cstring>
#include <map>
#include <mutex>
#include <tuple>

#include "groups.cuh"
#include "launch.h"
#include "mma.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kCl = 8;                  // blocks per cluster
constexpr int kRowB = 144;              // bytes per 128-byte chunk row in shared memory

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// Checks every offset and perm entry and writes the status word: one block, beside the work.
__device__ void check_indices(const int32_t* __restrict__ perm, const int32_t* __restrict__ offsets,
                              int N, int S_max, int T, int* status) {
  const int step = blockDim.x;
  bool bad = false;
  for (int i = threadIdx.x; i <= N; i += step) {
    const int v = offsets[i];
    bad |= v < 0 || v > S_max || (i > 0 && v < offsets[i - 1]);
  }
  const int S = min(max(offsets[N], 0), S_max);
  // eight loads in flight: this loop must not outlast the products
  for (int64_t s = min(max(offsets[0], 0), S_max) + threadIdx.x; s < S; s += 8 * step) {
    int v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = s + q * step < S ? perm[s + q * step] : 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) bad |= (unsigned)v[q] >= (unsigned)T;
  }
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

// ---------------------------------------------------------------- f16, long runs
// Two launches of persistent blocks, h between them in 32 bits (small: r of d columns); 16384 rows of
// 3584 columns, r = 64, 8 adapters: 36 + 60 us (DRAM floor 53; 36 + 51 with h in one f16 part), bound by
// fragment loads, by the products' latency at 16 warps per SM and, in the second launch, by the tensor pipe
// where the warps' products coincide (DRAM 40%, shared-memory pipe 50 to 56%, tensor 40 to 47%):
//   shrink  partial h[part] = x P over a part of the input columns, per tile of 64 rows
//   expand  h = sum of the parts in order, then y = base + scale h Q per tile and part of the
//           output columns
// (As one launch with h exchanged through a cluster's shared memory, each tile waited 15 us or
// more for two cluster-wide hand-overs: 16384 rows of 3584 columns at r = 64 took 320 us.)
//
// Eight warps multiply and copy their share of the rows (two 16-byte pieces per thread and chunk);
// weights come as boxes of three-dimensional tensors [N, rows, columns] by TMA, whose edges read
// as zeros.  Chunks are handed over by mbarriers that count both.  (Rows by TMA gathers of four
// rows were bound by the gathers' rate, about 50 cycles each: shrink 66 us.)
constexpr int kTallRows = 64;
constexpr int kTallWarps = 8, kTallThreads = 32 * kTallWarps;
constexpr int kChunk = 64;                        // columns per chunk

template <int R>
struct PlanTall {
  // Chunks per stage of the ring: two up to rank 64, where what a stage costs beside its products
  // (waits, addresses) was most of the instructions.
  static constexpr int kSub = R <= 64 ? 2 : 1;
  static constexpr int kSubB = kTallRows * 128 + kChunk * R * 2;   // rows, weights
  static constexpr int kStage = kSub * kSubB;
  static constexpr int kStages = (96 * 1024) / kStage;             // two blocks per SM
  static constexpr int kOffBar = kStages * kStage;
  static constexpr int kOffTab = kOffBar + 16 * kStages;           // abort flag, group table
  static constexpr int kBytes = kOffTab + 8 + 1024;                // with room to align
};

// Byte offset of 16-byte piece `piece` of row `row` in a swizzled tile of PITCH-byte rows
// (PITCH 32, 64 or 128: the swizzle of that span).
template <int PITCH>
__device__ __forceinline__ int swz(int row, int piece) {
  const int pat = PITCH == 128 ? row & 7 : PITCH == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
  return row * PITCH + ((piece ^ pat) << 4);
}

struct TallArgs {
  AdapterArgs a;
  float* partial;            // [parts of the first product][slots from the first group's first on][r]
  int slots_k, slots_n;      // resident blocks of the two launches
};

// Parts of a product's columns over the tiles that there are (the caller only knows a bound): the
// count that takes the fewest chunk times on `slots` resident blocks, with `start` chunk times for
// the start of an item.  Four chunks or more each, and no more than kPartItems items (which bounds
// the partial h).  Every warp computes it, a count per lane.
__device__ __forceinline__ int column_parts(int tiles, int chunks, int slots, int start) {
  const int p = (threadIdx.x & 31) + 1;
  int cost = 0x7fffffff;
  if (p == 1 || (p <= kAdapterParts && chunks >= 4 * p && (long long)tiles * p <= kPartItems))
    cost = min((tiles * p + slots - 1) / slots, 1 << 12) * ((chunks + p - 1) / p + start);
  const int best = __reduce_min_sync(0xffffffffu, cost);
  return __ffs(__ballot_sync(0xffffffffu, cost == best));
}
// Chunks of a product and the start of its items, in both launches' terms.
template <int R>
__device__ __forceinline__ int parts_of_k(const TallArgs& ta, int tiles) {
  const int w = PlanTall<R>::kSub * kChunk;
  return column_parts(tiles, (ta.a.dk + w - 1) / w, ta.slots_k, 2);
}

// Where partial h lie: a whole one (a single part) is given out at once, by its slot.  Others are counted
// from the first group's first slot: their rows are bounded by the tiles (kPartItems), which only cover
// the slots that groups own, not those before offsets[0].
struct PartialRows {
  float* at;
  int first, count;          // slot of row 0; rows of a part
};
__device__ __forceinline__ PartialRows partial_rows(const TallArgs& ta, const int* bound, int parts) {
  const int first = bound[0], count = bound[ta.a.N] - first;
  if (parts == 1 && ta.a.hidden) return {ta.a.hidden, 0, count};
  return {ta.partial, first, count};
}

// The chunks of a block's items, loaded ahead of their use.  Item i is part i % parts of tile
// i / parts; block b takes items b, b + blocks, ...  kWide: the weights' box has r-wide rows (one
// per column of the chunk), else chunk-wide rows (r of them).
template <int R, bool kWide>
struct TallRing {
  using PL = PlanTall<R>;
  static constexpr int NS = PL::kStages, MT = kTallRows, RB = R > 64 ? 64 : R;
  uint8_t* sm;
  uint64_t *full, *empty;
  int *bound, *start;
  volatile int* abort;
  int* status;
  const int32_t* perm;
  int N, T, chunks, parts, items, blocks;         // blocks: of the grid that take items
  const __half* rows;                             // [T, d], or null (an absent base)
  int d;
  const CUtensorMap* mW;
  // use
  int stage = 0;
  uint32_t phase = 0;
  // loads: thread t copies 16-byte piece t % 8 of rows t / 8 and t / 8 + 32
  int li, lc = 0, lend = 0, ln = 0, lstage = 0, lrow[2] = {-1, -1}, lnext[2] = {-1, -1};
  uint32_t lphase = 1;

  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return;
    const bool before = *abort != 0;
    // a wait that gives up marks the call; the block then runs through without further waits
    if (!mbar_wait_bounded(bar, parity, abort, nullptr, kDefaultWaitNs) && !before) *status = kErrTimeout;
  }
  __device__ __forceinline__ int part_begin(int p) const { return (int)((long long)chunks * p / parts); }
  __device__ __forceinline__ void fetch_rows(int item) {
    if (item >= items) return;
    const int tile = item / parts, n = group_of(tile, start, N);
    const int s0 = bound[n] + (tile - start[n]) * MT + (threadIdx.x >> 3);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      lnext[q] = s0 + 32 * q < bound[n + 1] ? perm[s0 + 32 * q] : -1;   // looked at when used
    }
  }
  __device__ __forceinline__ void begin_item() {
    while (li < items) {
      const int tile = li / parts, p = li - tile * parts;
      ln = group_of(tile, start, N);
      lc = part_begin(p);
      lend = part_begin(p + 1);
      lrow[0] = lnext[0];
      lrow[1] = lnext[1];
      fetch_rows(li + blocks);
      if (lc < lend) return;
      li += blocks;
    }
  }
  // The next chunk, into the stage whose turn it is (all threads).
  __device__ __forceinline__ void issue() {
    if (li >= items) return;
    const int col = lc * (PL::kSub * kChunk);
    uint8_t* st = sm + lstage * PL::kStage;
    wait(&empty[lstage], lphase);
    if (threadIdx.x == 0 && !*abort) {            // (no further loads after a wait gave up)
      mbar_expect_tx(&full[lstage], PL::kSub * kChunk * R * 2);
#pragma unroll
      for (int u = 0; u < PL::kSub; ++u) {        // (behind the last column: zeros)
        uint8_t* ws = st + u * PL::kSubB + MT * 128;
        if (kWide) {
#pragma unroll
          for (int b = 0; b < R; b += RB)
            tma_load_3d(ws + b * kChunk * 2, mW, b, col + u * kChunk, ln, &full[lstage]);
        } else {
          tma_load_3d(ws, mW, col + u * kChunk, 0, ln, &full[lstage]);
        }
      }
    }
    if (rows) {
      const int row = threadIdx.x >> 3, pc = threadIdx.x & 7;
      const uint32_t dst = smem_u32(st) + row * 128 + ((pc ^ (row & 7)) << 4);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const bool there = (unsigned)lrow[q] < (unsigned)T;
        const __half* src = rows + (there ? (uint64_t)(uint32_t)lrow[q] * (uint32_t)d + col + pc * 8 : 0);
#pragma unroll
        for (int u = 0; u < PL::kSub; ++u) {
          const bool on = there && col + u * kChunk + pc * 8 < d;
          cp_async16_at(dst + q * 32 * 128 + u * PL::kSubB, on ? src + u * kChunk : rows, on);
        }
      }
      cp_async_arrive(&full[lstage]);
    }
    if (++lstage == NS) {
      lstage = 0;
      lphase ^= 1u;
    }
    if (++lc == lend) {
      li += blocks;
      begin_item();
    }
  }
  __device__ __forceinline__ void begin() {
    li = blockIdx.x;
    fetch_rows(li);
    begin_item();
    for (int c = 0; c < NS - 2; ++c) issue();
  }
  __device__ __forceinline__ uint8_t* next() {    // the chunk that is used next
    issue();                                      // two chunks of slack between the warps
    wait(&full[stage], phase);
    return sm + stage * PL::kStage;
  }
  __device__ __forceinline__ void done() {        // this warp has read (and written) it
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[stage]);
    if (++stage == NS) {
      stage = 0;
      phase ^= 1u;
    }
  }
  // The end of a block (all threads): after a wait gave up, what is in flight lands before the shared
  // memory is released.  A stage's last load is of this round of the ring or of the one before it
  // (none yet: a phase that counts as complete).
  __device__ __forceinline__ void finish() {
    __syncthreads();
    if (!*abort) return;
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (threadIdx.x == 0)
      for (int s = 0; s < NS; ++s) mbar_drain(&full[s], s < lstage ? lphase ^ 1u : lphase);
  }
};

// Shared-memory set-up of both kernels; returns the number of tiles.
template <int R, bool kWide>
__device__ __forceinline__ int tall_setup(TallRing<R, kWide>& ring, const AdapterArgs& a, uint8_t* raw) {
  using PL = PlanTall<R>;
  // swizzled tiles start on 1024 bytes
  uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  ring.sm = sm;
  ring.full = reinterpret_cast<uint64_t*>(sm + PL::kOffBar);
  ring.empty = ring.full + PL::kStages;
  int* flag = reinterpret_cast<int*>(sm + PL::kOffTab);
  ring.abort = flag;
  ring.bound = flag + 2;
  ring.start = ring.bound + a.N + 1;
  ring.status = a.status;
  ring.perm = a.perm;
  ring.N = a.N;
  ring.T = a.T;
  if (threadIdx.x == 0) {
    for (int i = 0; i < PL::kStages; ++i) {
      mbar_init(&ring.full[i], ring.rows ? 1 + kTallThreads : 1);
      mbar_init(&ring.empty[i], kTallWarps);
    }
    fence_mbar_init();
    *flag = 0;
  }
  group_table<kTallThreads>(a.offsets, a.N, a.S_max, kTallRows, ring.bound, ring.start,
                            ring.start + a.N + 1);
  return ring.start[a.N];
}

template <int R, bool kT>
__global__ void __launch_bounds__(kTallThreads, 2)
    adapter_shrink_kernel(const __grid_constant__ CUtensorMap mP, const TallArgs ta) {
  const AdapterArgs& a = ta.a;
  using PL = PlanTall<R>;
  constexpr int MT = kTallRows, RB = R > 64 ? 64 : R;
  constexpr int WN = R >= 32 ? 2 : 1, WK = 2 / WN;   // two warps per 16 rows: along r, or the chunk
  constexpr int NF = R / WN / 8;                     // 8-column fragments of h per warp
  extern __shared__ uint8_t raw[];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  pdl_trigger();
  if (blockIdx.x == gridDim.x - 1) {              // the last block checks the indices
    check_indices(a.perm, a.offsets, a.N, a.S_max, a.T, a.status);
    return;
  }
  TallRing<R, !kT> ring;
  ring.rows = static_cast<const __half*>(a.x);
  ring.d = a.dk;
  ring.mW = &mP;
  const int ntiles = tall_setup(ring, a, raw);
  ring.chunks = (a.dk + PL::kSub * kChunk - 1) / (PL::kSub * kChunk);
  ring.parts = parts_of_k<R>(ta, ntiles);
  ring.items = ntiles * ring.parts;
  ring.blocks = gridDim.x - 1;
  const PartialRows pr = partial_rows(ta, ring.bound, ring.parts);
  ring.begin();
  const int wr = (w & 3) * 16, wc = w >> 2, h0 = WN > 1 ? wc * (R / WN) : 0;
  const int l15 = lane & 15, lh = lane >> 4, l3 = (lane >> 3) & 1, l7 = lane & 7;
  float* pair = reinterpret_cast<float*>(ring.start + a.N + 1 + 32);   // WK > 1: [MT][R]
  for (int item = blockIdx.x; item < ring.items; item += ring.blocks) {
    const int tile = item / ring.parts, part = item - tile * ring.parts;
    const int n = group_of(tile, ring.start, a.N);
    const int s0 = ring.bound[n] + (tile - ring.start[n]) * MT, s1 = ring.bound[n + 1];
    float acc[NF][4];
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    const int c1 = ring.part_begin(part + 1);
    for (int c = ring.part_begin(part); c < c1; ++c) {
      const uint8_t* st = ring.next();
#pragma unroll
      for (int u = 0; u < PL::kSub; ++u) {
      const uint8_t* xs = st + u * PL::kSubB;
      const uint8_t* ps = xs + MT * 128;
      // The tensor cores' additions truncate: a chain of n of them loses up to n / 2^23 of the
      // sum, always towards zero.  Chains end with every chunk and are added with rounding
      // (8192 columns in chains of 64: 3e-5 of the result; this way 2e-6).
      float run[NF][4];
#pragma unroll
      for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) run[i][j] = 0.f;
#pragma unroll
      for (int kk = 0; kk < 4 / WK; ++kk) {
        const int k = WK > 1 ? kk * WK + wc : kk;                // k-step of 16
        uint32_t fa[4];
        ldsm4(fa, xs + swz<128>(wr + l15, 2 * k + lh));
#pragma unroll
        for (int j = 0; j < NF / 2; ++j) {
          uint32_t fb[4];
          if (kT) {
            ldsm4(fb, ps + swz<128>(h0 + j * 16 + l7 + lh * 8, 2 * k + l3));
          } else {
            const int col = h0 + j * 16;
            ldsm4_t(fb, ps + (col / 64) * (kChunk * 128) + swz<RB * 2>(k * 16 + l15, (col % 64) / 8 + lh));
          }
          mma16816(run[2 * j], fa, fb[0], fb[1]);
          mma16816(run[2 * j + 1], fa, fb[2], fb[3]);
        }
      }
      if (u == PL::kSub - 1) ring.done();
#pragma unroll
      for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += run[i][j];
      }
    }
    if (WK > 1) {                                 // the two warps of the same rows
      float* p = pair + (wr + (lane >> 2)) * R + 2 * (lane & 3);
      if (wc == 1) {
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          *reinterpret_cast<float2*>(p + 8 * j) = make_float2(acc[j][0], acc[j][1]);
          *reinterpret_cast<float2*>(p + 8 * R + 8 * j) = make_float2(acc[j][2], acc[j][3]);
        }
      }
      __syncthreads();
      if (wc == 0) {
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          const float2 u = *reinterpret_cast<const float2*>(p + 8 * j);
          const float2 v = *reinterpret_cast<const float2*>(p + 8 * R + 8 * j);
          acc[j][0] += u.x; acc[j][1] += u.y; acc[j][2] += v.x; acc[j][3] += v.y;
        }
      }
      __syncthreads();
    }
    if (WK == 1 || wc == 0) {
      const int sa = s0 + wr + (lane >> 2), sb = sa + 8;
      float* pa = pr.at + ((size_t)part * pr.count + (sa - pr.first)) * a.r;
      float* pb = pa + (size_t)8 * a.r;
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        const int col = h0 + 8 * j + 2 * (lane & 3);
        if (col < a.r) {
          if (sa < s1) *reinterpret_cast<float2*>(pa + col) = make_float2(acc[j][0], acc[j][1]);
          if (sb < s1) *reinterpret_cast<float2*>(pb + col) = make_float2(acc[j][2], acc[j][3]);
        }
      }
    }
  }
  ring.finish();
}

template <int R, bool kT>
__global__ void __launch_bounds__(kTallThreads, R >= 128 ? 1 : 2)
    adapter_expand_kernel(const __grid_constant__ CUtensorMap mQ, const TallArgs ta) {
  const AdapterArgs& a = ta.a;
  using PL = PlanTall<R>;
  constexpr int MT = kTallRows, RB = R > 64 ? 64 : R;
  extern __shared__ uint8_t raw[];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const bool with_base = a.base != nullptr;
  TallRing<R, kT> ring;
  ring.rows = static_cast<const __half*>(a.base);
  ring.d = a.dn;
  ring.mW = &mQ;
  const int ntiles = tall_setup(ring, a, raw);
  ring.chunks = (a.dn + PL::kSub * kChunk - 1) / (PL::kSub * kChunk);
  const int parts_k = parts_of_k<R>(ta, ntiles);
  const PartialRows pr = partial_rows(ta, ring.bound, parts_k);
  // an item reads and converts its tile's h first, all its parts
  ring.parts = column_parts(ntiles, ring.chunks, ta.slots_n, 2 + (R >= 64 ? 2 : 1) * parts_k);
  ring.items = ntiles * ring.parts;
  ring.blocks = gridDim.x;
  ring.begin();                                   // base and Q are inputs of the call
  pdl_wait();                                     // the partial h are complete
  __half* Y = static_cast<__half*>(a.y);
  const int wr = (w & 3) * 16, wc = w >> 2;
  const int l15 = lane & 15, lh = lane >> 4, l3 = (lane >> 3) & 1, l7 = lane & 7;
  // Rows that this thread writes: two of the 16 that its warp and the one beside it computed, one
  // 16-byte piece each, so that eight lanes write a whole 128-byte line (four lanes on 64 bytes:
  // 58 us for 16384 x 3584 at r = 64 where this took 51; eight rows at once: 73).
  const int yrow = wr + wc * 8 + (lane >> 3), ypc = l7;
  for (int item = blockIdx.x; item < ring.items; item += ring.blocks) {
    const int tile = item / ring.parts, part = item - tile * ring.parts;
    const int n = group_of(tile, ring.start, a.N);
    const int s0 = ring.bound[n] + (tile - ring.start[n]) * MT, s1 = ring.bound[n + 1];
    int y0 = s0 + yrow < s1 ? a.perm[s0 + yrow] : -1, y1 = s0 + yrow + 4 < s1 ? a.perm[s0 + yrow + 4] : -1;
    if ((unsigned)y0 >= (unsigned)a.T) y0 = -1;
    if ((unsigned)y1 >= (unsigned)a.T) y1 = -1;
    // ---- h in the layout of the product's left operand: rows g and g + 8, columns
    // 16 k + 2 (lane % 4) + {0, 1, 8, 9}; a row's columns are spread over four lanes
    uint32_t fh[R / 16][4], fl[R / 16][4];          // high and low parts
    float m0, m1;
    {
      const int sa = s0 + wr + (lane >> 2), sb = sa + 8;
      float2 v[R / 16][4];
#pragma unroll
      for (int k = 0; k < R / 16; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q) v[k][q] = make_float2(0.f, 0.f);
      // Unconditional loads, in batches: each waited for on its own under a condition, they took
      // most of the time (3575 rows, 1808 columns, r = 96: 80 us).  A row behind the run's end reads
      // the last one and is not stored; columns behind r read the first and count as zero.
      const uint32_t ra = (uint32_t)(min(sa, s1 - 1) - pr.first), rb = (uint32_t)(min(sb, s1 - 1) - pr.first);
      for (int p = 0; p < parts_k; ++p) {
        const float* src = pr.at + (size_t)p * pr.count * a.r + 2 * (lane & 3);
        const float *pa = src + (uint64_t)ra * (uint32_t)a.r, *pb = src + (uint64_t)rb * (uint32_t)a.r;
        constexpr int KB = R / 16 < 4 ? R / 16 : 4;
#pragma unroll
        for (int k0 = 0; k0 < R / 16; k0 += KB) {
          float2 u[KB][4];
#pragma unroll
          for (int k = 0; k < KB; ++k)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int col = 16 * (k0 + k) + 8 * (q >> 1);
              u[k][q] = *reinterpret_cast<const float2*>((q & 1 ? pb : pa) + (col < a.r ? col : 0));
            }
#pragma unroll
          for (int k = 0; k < KB; ++k)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (16 * (k0 + k) + 8 * (q >> 1) < a.r) {
                v[k0 + k][q].x += u[k][q].x;
                v[k0 + k][q].y += u[k][q].y;
              }
        }
      }
      float ma = 0.f, mb = 0.f;
      bool oa = false, ob = false;
#pragma unroll
      for (int k = 0; k < R / 16; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float m = fmaxf(fabsf(v[k][q].x), fabsf(v[k][q].y));
          const bool odd = !isfinite(v[k][q].x) || !isfinite(v[k][q].y);
          if (q & 1) {
            mb = fmaxf(mb, m);
            ob |= odd;
          } else {
            ma = fmaxf(ma, m);
            oa |= odd;
          }
          if (a.hidden && part == 0 && wc == 0 && pr.at != a.hidden) {
            const int s = q & 1 ? sb : sa, col = 16 * k + 8 * (q >> 1) + 2 * (lane & 3);
            if (s < s1 && col < a.r)
              *reinterpret_cast<float2*>(a.hidden + (size_t)s * a.r + col) = v[k][q];
          }
        }
      if (oa) ma = INFINITY;                      // a row with infinities is not scaled
      if (ob) mb = INFINITY;
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, o));
        mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
      }
      const int ea = split_exp(ma), eb = split_exp(mb);
      const float ia = exp2_int(-ea), ib = exp2_int(-eb), sc = a.scale[n];
      m0 = sc * exp2_int(ea);
      m1 = sc * exp2_int(eb);
#pragma unroll
      for (int k = 0; k < R / 16; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float i = q & 1 ? ib : ia;
          __half2 h, l;
          split_f16(v[k][q].x * i, h.x, l.x);
          split_f16(v[k][q].y * i, h.y, l.y);
          fh[k][q] = *reinterpret_cast<const uint32_t*>(&h);
          fl[k][q] = *reinterpret_cast<const uint32_t*>(&l);
        }
    }
    // ---- 32 of a chunk's 64 columns per warp
    const int c1 = ring.part_begin(part + 1);
    for (int c = ring.part_begin(part); c < c1; ++c) {
      uint8_t* st = ring.next();
#pragma unroll
      for (int u = 0; u < PL::kSub; ++u) {
      uint8_t* bs = st + u * PL::kSubB;
      const uint8_t* qs = bs + MT * 128;
      float acc[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll
      for (int k = 0; k < R / 16; ++k) {
        uint32_t fb[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (kT)
            ldsm4(fb[j], qs + (k / 4) * (kChunk * 128) +
                             swz<RB * 2>(wc * 32 + j * 16 + l7 + lh * 8, 2 * (k % 4) + l3));
          else
            ldsm4_t(fb[j], qs + swz<128>(k * 16 + l15, wc * 4 + j * 2 + lh));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) mma16816(acc[j], fl[k], fb[j / 2][j % 2 * 2], fb[j / 2][j % 2 * 2 + 1]);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma16816(acc[j], fh[k], fb[j / 2][j % 2 * 2], fb[j / 2][j % 2 * 2 + 1]);
      }
      // base + scale * sum, rounded once, in place; then 16-byte rows out
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint8_t* at = bs + swz<128>(wr + l15, wc * 4 + j * 2 + lh);
        uint32_t b[4] = {0u, 0u, 0u, 0u};
        if (with_base) ldsm4(b, at);
#pragma unroll
        for (int q = 0; q < 4; ++q) {             // b[q]: rows + 8 (q & 1), columns + 8 (q >> 1)
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&b[q]));
          const float mm = q & 1 ? m1 : m0;
          const __half2 o = __floats2half2_rn(fmaf(mm, acc[2 * j + (q >> 1)][2 * (q & 1)], f.x),
                                              fmaf(mm, acc[2 * j + (q >> 1)][2 * (q & 1) + 1], f.y));
          b[q] = *reinterpret_cast<const uint32_t*>(&o);
        }
        stsm4(at, b);
      }
      asm volatile("bar.sync %0, 64;" ::"r"(1 + (w & 3)) : "memory");   // the two warps of these rows
      const int col = (c * PL::kSub + u) * kChunk + ypc * 8;
      if (col < a.dn) {
        if (y0 >= 0)
          *reinterpret_cast<uint4*>(Y + (size_t)y0 * a.dn + col) =
              *reinterpret_cast<const uint4*>(bs + swz<128>(yrow, ypc));
        if (y1 >= 0)
          *reinterpret_cast<uint4*>(Y + (size_t)y1 * a.dn + col) =
              *reinterpret_cast<const uint4*>(bs + swz<128>(yrow + 4, ypc));
      }
      }
      ring.done();
    }
  }
  ring.finish();
}

// ---------------------------------------------------------------- f16, short runs
// Tiles of 16 rows, four warps that load and multiply (64 requests with an adapter each, 3584
// columns, r = 16: 10 us, of which the weights' bytes are 2; the rest is the chain of table, loads,
// two exchanges and stores, so chunks are wide and few at low ranks).
template <int R>
struct Plan16 {
  static constexpr int MT = 16, kThreads = 128, kWarps = 4;
  static constexpr int kBlocks = R >= 128 ? 2 : 4;                 // per SM
  static constexpr int C = R <= 32 ? 128 : 64;                     // columns per chunk
  static constexpr int kLdC = C + 8, kLdR = R + 8;                 // halves per row
  static constexpr int WN = R / kWarps >= 16 ? kWarps : 1;         // first product: warps along r,
  static constexpr int WK = kWarps / WN;                           // or along a chunk's columns
  static constexpr int kW = C * kLdR > R * kLdC ? C * kLdR : R * kLdC;
  static constexpr int kStage = 2 * (MT * kLdC + kW);
  static constexpr int kStages = R >= 64 && R < 128 ? 5 : 4;       // (three blocks per SM at R = 64)
  static constexpr int kOffPart = kStages * kStage;                // partial h [WK][MT][R]
  static constexpr int kOffH = kOffPart + WK * MT * R * 4;         // h
  static constexpr int kOffMult = kOffH + 2 * MT * kLdR * 2;       // (h in two parts)
  static constexpr int kOffTab = kOffMult + MT * 4;                // offsets, tile starts, scratch
};

template <int R, bool kT>
__global__ void __launch_bounds__(128, Plan16<R>::kBlocks) adapter_f16_kernel(const AdapterArgs a) {
  using PL = Plan16<R>;
  constexpr int MT = PL::MT, NT = PL::kThreads, NS = PL::kStages, C = PL::C, WN = PL::WN, WK = PL::WK;
  constexpr int kLdC = PL::kLdC, kLdR = PL::kLdR;
  constexpr int CV = C / 8, RV = R / 8;           // 16-byte pieces of a chunk's row, of r
  constexpr int XP = MT * CV / NT;                // of x (or base) per thread and chunk
  constexpr int WP = R * CV / NT;                 // of P or Q
  extern __shared__ __align__(16) uint8_t sm[];
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank();
  const int cid = blockIdx.x / kCl, ncl = gridDim.x / kCl - 1;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (cid == ncl) {                               // the last cluster checks the indices
    if (rank == 0) check_indices(a.perm, a.offsets, a.N, a.S_max, a.T, a.status);
    return;
  }
  float* part = reinterpret_cast<float*>(sm + PL::kOffPart);
  __half* hs = reinterpret_cast<__half*>(sm + PL::kOffH);         // [MT][R + 8] high parts, then low
  float* mult = reinterpret_cast<float*>(sm + PL::kOffMult);
  int* bound = reinterpret_cast<int*>(sm + PL::kOffTab);
  int* start = bound + a.N + 1;
  group_table<NT>(a.offsets, a.N, a.S_max, MT, bound, start, start + a.N + 1);
  const int ntiles = start[a.N];

  const int ck = (a.dk + C - 1) / C, cn = (a.dn + C - 1) / C;
  const int k0 = (int)((long long)ck * rank / kCl), k1 = (int)((long long)ck * (rank + 1) / kCl);
  const int n0 = (int)((long long)cn * rank / kCl), n1 = (int)((long long)cn * (rank + 1) / kCl);
  const int nk = k1 - k0, total = nk + n1 - n0;
  const __half* X = static_cast<const __half*>(a.x);
  const __half* base = static_cast<const __half*>(a.base);
  __half* Y = static_cast<__half*>(a.y);

  // Perm entry of row `row` of a tile, -1 where there is none.
  auto token = [&](int tile, int row) {
    if (tile >= ntiles) return -1;
    const int n = group_of(tile, start, a.N);
    const int s = bound[n] + (tile - start[n]) * MT + row;
    if (s >= bound[n + 1]) return -1;
    return a.perm[s];                             // looked at when used: no wait for the load here
  };

  // ---- loader: runs NS - 1 chunks ahead, across tiles.  Its rows' tokens are fetched a tile early.
  const int lrow = tid / CV, lpc = (tid % CV) * 8;                // pieces: rows lrow + NT / CV p
  int ltile = cid, lc = 0, ls = 0, ltok[XP], lnext[XP];
  const __half *lP = nullptr, *lQ = nullptr;
  auto begin_tile = [&]() {
#pragma unroll
    for (int p = 0; p < XP; ++p) {
      ltok[p] = lnext[p];
      lnext[p] = token(ltile + ncl, lrow + p * (NT / CV));
    }
    if (ltile < ntiles) {
      const int n = group_of(ltile, start, a.N);
      lP = static_cast<const __half*>(a.P) + (size_t)n * a.dk * a.r;
      lQ = static_cast<const __half*>(a.Q) + (size_t)n * a.dn * a.r;
    }
  };
  auto issue = [&]() {
    if (ltile < ntiles && total > 0) {
      __half* st = reinterpret_cast<__half*>(sm + ls * PL::kStage);
      const bool first = lc < nk;
      const int col0 = (first ? k0 + lc : n0 + lc - nk) * C;
      const int d = first ? a.dk : a.dn;
      const __half* rowsrc = first ? X : base;
      if (rowsrc) {
        const bool in = col0 + lpc < d;
#pragma unroll
        for (int p = 0; p < XP; ++p) {
          const bool on = in && (unsigned)ltok[p] < (unsigned)a.T;
          cp_async16(st + (lrow + p * (NT / CV)) * kLdC + lpc,
                     rowsrc + (on ? (size_t)ltok[p] * d + col0 + lpc : 0), on);
        }
      }
      __half* ws = st + MT * kLdC;
      const __half* W = first ? lP : lQ;
      if (first != kT) {                          // rows of the chunk's columns, r wide
        const int row = tid / RV, col = (tid % RV) * 8;
        const __half* src = W + (size_t)(col0 + row) * a.r + col;
#pragma unroll
        for (int p = 0; p < WP; ++p) {
          const bool on = col < a.r && col0 + row + p * (NT / RV) < d;
          cp_async16(ws + (row + p * (NT / RV)) * kLdR + col,
                     on ? src + (size_t)p * (NT / RV) * a.r : W, on);
        }
      } else {                                    // r rows, the chunk's columns wide
        const bool in = col0 + lpc < d;
        const __half* src = W + (size_t)lrow * d + col0 + lpc;
#pragma unroll
        for (int p = 0; p < WP; ++p) {
          const bool on = in && lrow + p * (NT / CV) < a.r;
          cp_async16(ws + (lrow + p * (NT / CV)) * kLdC + lpc,
                     on ? src + (size_t)p * (NT / CV) * d : W, on);
        }
      }
      if (++lc == total) {
        lc = 0;
        ltile += ncl;
        begin_tile();
      }
    }
    cp_async_commit();
    ls = ls + 1 == NS ? 0 : ls + 1;
  };
#pragma unroll
  for (int p = 0; p < XP; ++p) lnext[p] = token(ltile, lrow + p * (NT / CV));
  begin_tile();
  for (int c = 0; c < NS - 1; ++c) issue();
  int cs = 0;                                     // stage of the chunk that is used next
  auto advance = [&]() {                          // it is complete; one more load is issued
    cp_async_wait<NS - 2>();
    __syncthreads();
    issue();
    const uint8_t* st = sm + cs * PL::kStage;
    cs = cs + 1 == NS ? 0 : cs + 1;
    return reinterpret_cast<const __half*>(st);
  };

  // rows that this thread writes, one 16-byte piece of its warp's columns each
  constexpr int WCOL = C / PL::kWarps, LPR = WCOL / 8, RPT = MT * LPR / 32;
  const int yrow = lane / LPR, ycol = w * WCOL + (lane % LPR) * 8;
  int ynext[RPT];
#pragma unroll
  for (int p = 0; p < RPT; ++p) ynext[p] = token(cid, yrow + p * (32 / LPR));

  for (int tile = cid; tile < ntiles; tile += ncl) {
    const int n = group_of(tile, start, a.N);
    const int s0 = bound[n] + (tile - start[n]) * MT;
    const int rows = min(MT, bound[n + 1] - s0);
    const float scale = a.scale[n];
    int ytok[RPT];
#pragma unroll
    for (int p = 0; p < RPT; ++p) {
      ytok[p] = ynext[p];
      ynext[p] = token(tile + ncl, yrow + p * (32 / LPR));
    }

    // ---- first product: partial h of this block's input columns (chains of truncating additions
    // end after four products, see adapter_shrink_kernel)
    {
      constexpr int NF = R / WN / 8;              // 8-column fragments of h per warp
      constexpr int KS = C / 16 / WK;             // k-steps per warp and chunk
      float acc[NF][4], run[NF][4];
#pragma unroll
      for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = run[i][j] = 0.f;
      const int h0 = WN > 1 ? w * (R / WN) : 0;
      for (int c = 0; c < nk; ++c) {
        const __half* xs = advance();
        const __half* ps = xs + MT * kLdC;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
          const int k = (WK > 1 ? kk * WK + w : kk) * 16;
          uint32_t fa[4];
          frag_a(fa, xs + k, kLdC, lane);
#pragma unroll
          for (int j = 0; j < NF / 2; ++j) {
            uint32_t fb[4];
            if (kT)
              frag_b_nk(fb, ps + (h0 + j * 16) * kLdC + k, kLdC, lane);
            else
              frag_b_kn(fb, ps + k * kLdR + h0 + j * 16, kLdR, lane);
            mma16816(run[2 * j], fa, fb[0], fb[1]);
            mma16816(run[2 * j + 1], fa, fb[2], fb[3]);
          }
        }
        if (c % (4 / KS) == 4 / KS - 1 || c == nk - 1) {
#pragma unroll
          for (int i = 0; i < NF; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              acc[i][j] += run[i][j];
              run[i][j] = 0.f;
            }
        }
      }
      float* p = part + ((WK > 1 ? w : 0) * MT + (lane >> 2)) * R + h0 + 2 * (lane & 3);
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        *reinterpret_cast<float2*>(p + 8 * j) = make_float2(acc[j][0], acc[j][1]);
        *reinterpret_cast<float2*>(p + 8 * R + 8 * j) = make_float2(acc[j][2], acc[j][3]);
      }
    }
    if (WK > 1) {                                 // the warps' shares of the block
      __syncthreads();
      for (int i = tid; i < MT * R; i += NT) {
        float v = part[i];
#pragma unroll
        for (int q = 1; q < WK; ++q) v += part[q * MT * R + i];
        part[i] = v;
      }
    }
    cl.sync();

    // ---- h: this block sums rows 2 rank, 2 rank + 1 over the cluster and gives them to all
    if (tid < MT) {                               // eight threads per row, R / 8 columns each
      constexpr int CPT = R / 8;
      const int row = rank * (MT / kCl) + (tid >> 3), c0 = (tid & 7) * CPT;
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
      float m = 0.f;
      bool odd = false;
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        m = fmaxf(m, fabsf(v[j]));
        odd |= !isfinite(v[j]);
      }
      if (odd) m = INFINITY;                      // such a row is not scaled
      const unsigned grp = 0xffu << (lane & 24);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(grp, m, o));
      const int e = split_exp(m);
      const float inv = exp2_int(-e);
      struct alignas(CPT >= 8 ? 16 : 2 * CPT) Halves { __half v[CPT]; } hv, lv;
#pragma unroll
      for (int j = 0; j < CPT; ++j) split_f16(v[j] * inv, hv.v[j], lv.v[j]);
      const float mu = scale * exp2_int(e);
#pragma unroll
      for (int q = 0; q < kCl; ++q) {
        __half* dh = cl.map_shared_rank(hs, q) + row * kLdR + c0;
        *reinterpret_cast<Halves*>(dh) = hv;
        *reinterpret_cast<Halves*>(dh + MT * kLdR) = lv;
        if ((tid & 7) == 0) cl.map_shared_rank(mult, q)[row] = mu;
      }
      if (a.hidden && row < rows) {
        float* dst = a.hidden + (size_t)(s0 + row) * a.r;
#pragma unroll
        for (int j = 0; j < CPT; ++j)
          if (c0 + j < a.r) dst[c0 + j] = v[j];
      }
    }
    cl.sync();

    // ---- second product: this block's output columns
    constexpr int NF = WCOL / 8;                  // 8-column fragments of a chunk per warp
    const int c0 = w * WCOL;
    uint32_t fh[R / 16][4], fl[R / 16][4];
#pragma unroll
    for (int k = 0; k < R / 16; ++k) {
      frag_a(fh[k], hs + k * 16, kLdR, lane);
      frag_a(fl[k], hs + MT * kLdR + k * 16, kLdR, lane);
    }
    const int g = lane >> 2, q2 = 2 * (lane & 3);
    const float m0 = mult[g], m1 = mult[g + 8];
    for (int c = n0; c < n1; ++c) {
      __half* bs = const_cast<__half*>(advance());
      const __half* qs = bs + MT * kLdC;
      float acc[NF][4];
#pragma unroll
      for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll
      for (int k = 0; k < R / 16; ++k)
#pragma unroll
        for (int j = 0; j < NF / 2; ++j) {
          uint32_t fb[4];
          if (kT)
            frag_b_nk(fb, qs + (c0 + j * 16) * kLdR + k * 16, kLdR, lane);
          else
            frag_b_kn(fb, qs + k * 16 * kLdC + c0 + j * 16, kLdC, lane);
          mma16816(acc[2 * j], fl[k], fb[0], fb[1]);
          mma16816(acc[2 * j + 1], fl[k], fb[2], fb[3]);
          mma16816(acc[2 * j], fh[k], fb[0], fb[1]);
          mma16816(acc[2 * j + 1], fh[k], fb[2], fb[3]);
        }
      // base + scale * sum, rounded once, in place; then 16-byte rows out
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        __half2* b0 = reinterpret_cast<__half2*>(bs + g * kLdC + c0 + 8 * j + q2);
        __half2* b1 = reinterpret_cast<__half2*>(bs + (g + 8) * kLdC + c0 + 8 * j + q2);
        float2 u = make_float2(0.f, 0.f), v = u;
        if (base) {
          u = __half22float2(*b0);
          v = __half22float2(*b1);
        }
        *b0 = __floats2half2_rn(fmaf(m0, acc[j][0], u.x), fmaf(m0, acc[j][1], u.y));
        *b1 = __floats2half2_rn(fmaf(m1, acc[j][2], v.x), fmaf(m1, acc[j][3], v.y));
      }
      __syncwarp();
      const int col = c * C + ycol;
      if (col < a.dn) {
#pragma unroll
        for (int p = 0; p < RPT; ++p)
          if ((unsigned)ytok[p] < (unsigned)a.T)
            *reinterpret_cast<uint4*>(Y + (size_t)ytok[p] * a.dn + col) =
                *reinterpret_cast<const uint4*>(bs + (yrow + p * (32 / LPR)) * kLdC + ycol);
      }
    }
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------- f32
// As the short f16 form, with fused multiply-adds; every run goes in tiles of 16 rows (1 row of 64 to
// 256 columns: 6 us of latency; long runs are bound by the multiply-adds' operands from shared memory).
template <int R>
struct Plan32 {
  static constexpr int MT = 16, kThreads = 128, C = 32;
  static constexpr int kLdC = kRowB / 4, kLdR = R + 4;
  static constexpr int kW = 4 * (C * kLdR > R * kLdC ? C * kLdR : R * kLdC);
  static constexpr int kStage = MT * kRowB + kW;
  static constexpr int kStages = R >= 128 ? 4 : R >= 64 ? 6 : 8;
  static constexpr int kOffPart = kStages * kStage;
  static constexpr int kOffH = kOffPart + MT * R * 4;
  static constexpr int kOffMult = kOffH + MT * kLdR * 4;
  static constexpr int kOffTok = kOffMult + MT * 4;
  static constexpr int kOffTab = kOffTok + MT * 4;
};

template <int R, bool kT>
__global__ void __launch_bounds__(128) adapter_f32_kernel(const AdapterArgs a) {
  using PL = Plan32<R>;
  constexpr int MT = PL::MT, C = PL::C, NS = PL::kStages, NT = PL::kThreads;
  constexpr int kLdC = PL::kLdC, kLdR = PL::kLdR;
  extern __shared__ __align__(16) uint8_t sm[];
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank();
  const int cid = blockIdx.x / kCl, ncl = gridDim.x / kCl - 1;
  const int tid = threadIdx.x;
  if (cid == ncl) {                               // the last cluster checks the indices
    if (rank == 0) check_indices(a.perm, a.offsets, a.N, a.S_max, a.T, a.status);
    return;
  }
  float* part = reinterpret_cast<float*>(sm + PL::kOffPart);      // [MT][R]
  float* hf = reinterpret_cast<float*>(sm + PL::kOffH);           // [MT][R + 4]
  float* mult = reinterpret_cast<float*>(sm + PL::kOffMult);
  int* tok = reinterpret_cast<int*>(sm + PL::kOffTok);
  int* bound = reinterpret_cast<int*>(sm + PL::kOffTab);
  int* start = bound + a.N + 1;
  group_table<NT>(a.offsets, a.N, a.S_max, MT, bound, start, start + a.N + 1);
  const int ntiles = start[a.N];

  const int ck = (a.dk + C - 1) / C, cn = (a.dn + C - 1) / C;
  const int k0 = (int)((long long)ck * rank / kCl), k1 = (int)((long long)ck * (rank + 1) / kCl);
  const int n0 = (int)((long long)cn * rank / kCl), n1 = (int)((long long)cn * (rank + 1) / kCl);
  const int nk = k1 - k0, total = nk + n1 - n0;
  const float* X = static_cast<const float*>(a.x);
  const float* base = static_cast<const float*>(a.base);
  float* Y = static_cast<float*>(a.y);

  for (int tile = cid; tile < ntiles; tile += ncl) {
    const int n = group_of(tile, start, a.N);
    const int s0 = bound[n] + (tile - start[n]) * MT;
    const int rows = min(MT, bound[n + 1] - s0);
    if (tid < MT) {
      int t = tid < rows ? a.perm[s0 + tid] : -1;
      if ((unsigned)t >= (unsigned)a.T) t = -1;
      tok[tid] = t;
    }
    __syncthreads();
    const float* P = static_cast<const float*>(a.P) + (size_t)n * a.dk * a.r;
    const float* Q = static_cast<const float*>(a.Q) + (size_t)n * a.dn * a.r;

    // chunk c of the sequence: nk input chunks (x, P), then the output chunks (base, Q)
    auto load = [&](int c) {
      uint8_t* st = sm + (c % NS) * PL::kStage;
      const bool first = c < nk;
      const int col0 = (first ? k0 + c : n0 + c - nk) * C;
      const int d = first ? a.dk : a.dn;
      const float* rowsrc = first ? X : base;
      if (rowsrc) {
        const int row = tid >> 3, col = col0 + (tid & 7) * 4;
        const bool on = tok[row] >= 0 && col < d;
        cp_async16(st + row * kRowB + (tid & 7) * 16, rowsrc + (on ? (size_t)tok[row] * d + col : 0), on);
      }
      float* ws = reinterpret_cast<float*>(st + MT * kRowB);
      const float* W = first ? P : Q;
      if (first != kT) {                          // rows of the chunk's columns, r wide
        for (int i = tid; i < C * (R / 4); i += NT) {
          const int row = i / (R / 4), col = (i % (R / 4)) * 4;
          const bool on = col0 + row < d && col < a.r;
          cp_async16(ws + row * kLdR + col, W + (on ? (size_t)(col0 + row) * a.r + col : 0), on);
        }
      } else {                                    // r rows, the chunk's columns wide
        for (int i = tid; i < R * 8; i += NT) {
          const int row = i >> 3, col = (i & 7) * 4;
          const bool on = row < a.r && col0 + col < d;
          cp_async16(ws + row * kLdC + col, W + (on ? (size_t)row * d + col0 + col : 0), on);
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
      return reinterpret_cast<const float*>(sm + (c % NS) * PL::kStage);
    };

    // ---- first product: eight threads per row, R / 8 columns each
    {
      constexpr int CPT = R / 8;
      const int row = tid >> 3, c0 = tid & 7;
      float acc[CPT];
#pragma unroll
      for (int j = 0; j < CPT; ++j) acc[j] = 0.f;
      for (int c = 0; c < nk; ++c) {
        const float* xs = advance(c);
        const float* ps = xs + MT * kLdC;
#pragma unroll 4
        for (int k = 0; k < C; ++k) {
          const float xv = xs[row * kLdC + k];
#pragma unroll
          for (int j = 0; j < CPT; ++j)
            acc[j] = fmaf(xv, kT ? ps[(c0 + 8 * j) * kLdC + k] : ps[k * kLdR + c0 + 8 * j], acc[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < CPT; ++j) part[row * R + c0 + 8 * j] = acc[j];
    }
    cl.sync();

    // ---- h: this block sums rows 2 rank, 2 rank + 1 over the cluster and gives them to all
    if (tid < MT) {
      constexpr int CPT = R / 8;
      const int row = rank * (MT / kCl) + (tid >> 3), c0 = (tid & 7) * CPT;
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
      for (int q = 0; q < kCl; ++q) {
        float* dh = cl.map_shared_rank(hf, q) + row * kLdR + c0;
#pragma unroll
        for (int j = 0; j < CPT; j += 2) *reinterpret_cast<float2*>(dh + j) = make_float2(v[j], v[j + 1]);
        if ((tid & 7) == 0) cl.map_shared_rank(mult, q)[row] = sc;
      }
    }
    cl.sync();

    // ---- second product: four columns of a chunk per thread
    const int row = tid >> 3, c0 = (tid & 7) * 4;
    const float mu = mult[row];
    const int t = tok[row];
    for (int c = nk; c < total; ++c) {
      const float* bs = advance(c);
      const float* qs = bs + MT * kLdC;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int k = 0; k < R; ++k) {
        const float hv = hf[row * kLdR + k];
        if (kT) {
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] = fmaf(hv, qs[(c0 + j) * kLdR + k], acc[j]);
        } else {
          const float4 q = load4(qs + k * kLdC + c0);
          acc[0] = fmaf(hv, q.x, acc[0]);
          acc[1] = fmaf(hv, q.y, acc[1]);
          acc[2] = fmaf(hv, q.z, acc[2]);
          acc[3] = fmaf(hv, q.w, acc[3]);
        }
      }
      const int col = (n0 + c - nk) * C + c0;
      if (t >= 0 && col < a.dn) {
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
        if (base) u = load4(bs + row * kLdC + c0);
        u.x = fmaf(mu, acc[0], u.x);
        u.y = fmaf(mu, acc[1], u.y);
        u.z = fmaf(mu, acc[2], u.z);
        u.w = fmaf(mu, acc[3], u.w);
        *reinterpret_cast<float4*>(Y + (size_t)t * a.dn + col) = u;
      }
    }
    cp_async_wait<0>();
    __syncthreads();                              // tok and the ring are free for the next tile
  }
}

// Bytes of the group table, in powers of two of the groups: few distinct launch plans.
size_t table_bytes(int N) {
  int groups = 64;
  while (groups < N + 1) groups *= 2;
  return sizeof(int) * (2 * (size_t)groups + 64);
}

// Clusters of a kernel that are resident on the device at once (asked once per kernel, device
// and size of the group table; a grid of more would leave its last clusters for a second round).
int resident_clusters(const void* kern, const cudaLaunchConfig_t& cfg) {
  static std::mutex mu;
  static std::map<std::tuple<const void*, int, size_t>, int> known;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lk(mu);
  const auto key = std::make_tuple(kern, dev, cfg.dynamicSmemBytes);
  const auto it = known.find(key);
  if (it != known.end()) return it->second;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) n = 0;
  known[key] = n;
  return n;
}

// One cluster per tile, at most as many as are resident at once, and one more for the checks.
template <typename Kern>
cudaError_t launch_plan(Kern kern, const AdapterArgs& a, int MT, int threads, size_t smem,
                        cudaStream_t s) {
  MOE_LAUNCH(ensure_smem_attr(reinterpret_cast<const void*>(kern)));
  smem += table_bytes(a.N);
  const long long most = (long long)a.S_max / MT + std::min(a.N, a.S_max);   // tiles at most
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCl);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCl;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int fit = resident_clusters(reinterpret_cast<const void*>(kern), cfg);
  if (fit < 1) return cudaErrorLaunchOutOfResources;
  cfg.gridDim = dim3(((int)std::min<long long>(most, fit) + 1) * kCl);
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, a);
  if (err == cudaSuccess) launch_counter().fetch_add(1, std::memory_order_relaxed);
  return err;
}

template <bool kT, int R>
cudaError_t launch_short(const AdapterArgs& a, cudaStream_t s) {
  using PL = Plan16<R>;
  return launch_plan(adapter_f16_kernel<R, kT>, a, PL::MT, PL::kThreads, PL::kOffTab, s);
}
// Blocks of a kernel that are resident on the device at once, asked once as resident_clusters.
int resident_blocks(const void* kern, int threads, size_t smem) {
  static std::mutex mu;
  static std::map<std::tuple<const void*, int, size_t>, int> known;
  int dev = 0, sms = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lk(mu);
  const auto key = std::make_tuple(kern, dev, smem);
  const auto it = known.find(key);
  if (it != known.end()) return it->second;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem) != cudaSuccess)
    n = 0;
  known[key] = n * sms;
  return n * sms;
}

template <bool kT, int R>
cudaError_t launch_tall(const AdapterArgs& a, float* partial, cudaStream_t s) {
  using PL = PlanTall<R>;
  const uint64_t dk = a.dk, dn = a.dn, r = a.r, N = a.N;
  const uint32_t RB = R > 64 ? 64 : R;
  const uint32_t wide[3] = {RB, 64, 1}, flat[3] = {64, R, 1};
  const size_t smem = PL::kBytes + table_bytes(a.N) + (R < 32 ? kTallRows * R * 4 : 0);
  const long long items = ((long long)a.S_max / kTallRows + std::min(a.N, a.S_max)) * kAdapterParts;
  auto shrink = adapter_shrink_kernel<R, kT>;
  auto expand = adapter_expand_kernel<R, kT>;
  MOE_LAUNCH(ensure_smem_attr(reinterpret_cast<const void*>(shrink)));
  MOE_LAUNCH(ensure_smem_attr(reinterpret_cast<const void*>(expand)));
  const TallArgs ta{a, partial, resident_blocks(reinterpret_cast<const void*>(shrink), kTallThreads, smem),
                    resident_blocks(reinterpret_cast<const void*>(expand), kTallThreads, smem)};
  if (ta.slots_k < 2 || ta.slots_n < 1) return cudaErrorLaunchOutOfResources;
  CUtensorMap mP, mQ;
  const uint64_t p_fwd[3] = {r, dk, N}, p_bwd[3] = {dk, r, N}, q_fwd[3] = {dn, r, N}, q_bwd[3] = {r, dn, N};
  if (!encode_f16_map(&mP, a.P, 3, kT ? p_bwd : p_fwd, kT ? flat : wide)) return cudaErrorInvalidValue;
  memset(&mQ, 0, sizeof(mQ));                     // not used when there is no second product
  if (a.dn && !encode_f16_map(&mQ, a.Q, 3, kT ? q_bwd : q_fwd, kT ? wide : flat)) return cudaErrorInvalidValue;
  const int grid_k = (int)std::min<long long>(items, ta.slots_k - 1) + 1;      // and the checks
  MOE_LAUNCH(launch_k(shrink, grid_k, kTallThreads, smem, s, false, mP, ta));
  const int grid_n = (int)std::min<long long>(items, ta.slots_n);
  return launch_k(expand, grid_n, kTallThreads, smem, s, true, mQ, ta);
}
template <bool kT, int R>
cudaError_t launch_f32(const AdapterArgs& a, cudaStream_t s) {
  using PL = Plan32<R>;
  return launch_plan(adapter_f32_kernel<R, kT>, a, PL::MT, PL::kThreads, PL::kOffTab, s);
}

template <bool kT, int R>
cudaError_t launch_rank(const AdapterArgs& a, bool f16, float* partial, cudaStream_t s) {
  if (!f16) return launch_f32<kT, R>(a, s);
  return adapter_tall(a.S_max, a.N, a.r, true) ? launch_tall<kT, R>(a, partial, s) : launch_short<kT, R>(a, s);
}
template <bool kT>
cudaError_t launch_adapter_t(const AdapterArgs& a, bool f16, float* partial, cudaStream_t s) {
  if (a.r <= 16) return launch_rank<kT, 16>(a, f16, partial, s);
  if (a.r <= 32) return launch_rank<kT, 32>(a, f16, partial, s);
  if (a.r <= 64) return launch_rank<kT, 64>(a, f16, partial, s);
  return launch_rank<kT, 128>(a, f16, partial, s);
}

__global__ void __launch_bounds__(1024) adapter_check_kernel(const AdapterArgs a) {
  check_indices(a.perm, a.offsets, a.N, a.S_max, a.T, a.status);
}

}  // namespace

// Two launches with tiles of 64 rows, where tiles of 16 would take the resident clusters more than
// one round (estimated, with half a tile per adapter lost; above rank 64, where long runs have one block per
// SM, two) and an adapter has more than 16 rows on average: fewer leave a tile of 64 mostly empty.  One
// adapter, 3584 columns, us short / long: r = 16, 72 tiles of 16 rows 13.4 / 13.8, 80 tiles 17.7 / 14.6;
// r = 32, 48 tiles 13.2 / 15.5, 52 tiles 18.2 / 15.6; r = 64, 48 tiles 17.2 / 19.5, 52 tiles 24.3 / 19.4;
// r = 128, 36 tiles 20 / 34, 72 tiles 37 / 38, 80 tiles 48 / 40.  64 adapters with r = 64: 16 rows each
// 30 / 34, 24 each 41 / 35.
bool adapter_tall(int S_max, int N, int r, bool f16) {
  const int n = std::min(N, S_max), round = r > 16 && r <= 64 ? 48 : 72;
  return f16 && S_max > 16LL * n && S_max / 16 + n / 2 > round;
}

size_t adapter_partial_rows(int S_max) {
  return std::max<size_t>(S_max, std::min<size_t>((size_t)kAdapterParts * S_max, (size_t)kPartItems * kTallRows));
}

cudaError_t launch_adapter(const void* x, const void* P, const void* Q, const void* base, void* y,
                           float* hidden, float* partial, const float* scale, const int32_t* perm,
                           const int32_t* offsets, int* status, int dtype_f16, bool transposed,
                           int T, int dk, int dn, int r, int N, int S_max, cudaStream_t s) {
  const AdapterArgs a{x, P, Q, base, y, hidden, scale, perm, offsets, status, T, dk, dn, r, N, S_max};
  if (dk == 0) return launch_k(adapter_check_kernel, 1, 1024, 0, s, false, a);
  return transposed ? launch_adapter_t<true>(a, dtype_f16, partial, s)
                    : launch_adapter_t<false>(a, dtype_f16, partial, s);
}

}  // namespace moe
