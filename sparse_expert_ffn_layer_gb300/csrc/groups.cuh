// Tables of slot groups (adapters) in shared memory: clamped boundaries and the tiles of rows that
// each group is cut into.
#pragma once

#include "common.cuh"

namespace moe {

// Group boundaries as the kernels use them, and the tile starts.  bound[n] = the largest of
// offsets[0 .. n], clamped to [0, S_max]: runs never overlap and no slot lies outside the
// buffers, whatever the offsets say.  start[n] = number of tiles of the groups before n.
// All threads of the block (at most 16 warps); N <= 1024; scratch: 24 words.
template <int kThreads>
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

// The group of a tile: the last n with start[n] <= tile (a group without tiles shares its start
// with the next one).
__device__ __forceinline__ int group_of(int tile, const int* start, int N) {
  int n = 0;
#pragma unroll
  for (int step = 512; step > 0; step >>= 1)
    if (n + step < N && start[n + step] <= tile) n += step;
  return n;
}

}  // namespace moe
