// Experts in 8-bit floating point (e4m3) with a scale for each block of 128: the weights' and the rows'
// quantisers, and the grouped products on the 5th-generation tensor cores (kind::f8f6f4 and kind::mxf8f6f4, TMEM, TMA).
//
//   y[s, j] = sum_b sx[s, b] sw[j / 128, b] sum_{i in b} x8[s, i] w8[j, i]          (b: blocks of 128 inputs)
//
// Scales that this library makes are powers of two, so that bringing a value to 8 bits is one rounding: the
// quotient is exact, and the same in any precision.  The products take any 32-bit scales.
//
// Products, in two forms.  In both, as in the f16 form, a weight tile is the MMA's M operand and a run of one expert's slots
// its N operand, both with their inputs side by side (K-major).
//
// Any scales, and short runs: a stage of the pipeline is one block of 128 inputs: four MMAs whose sum goes to a TMEM slot,
// from where eight warps add it, times its scale, to the running sums in their registers (column n of a tile has one
// scale, a weight tile has one for all its rows).  So the sums over blocks are in 32 bits with every scale applied before
// them, and a slot is free again as soon as it was read.  One more warp multiplies the two scales, so that the eight do
// one multiply-add a value.  They read TMEM in the shape in which a lane has two of each eight columns and four rows: with a
// row of every column a lane, each of the four lane quarters took 128 N bytes of scales from shared memory a block
// (N = 160: 1120 cycles a block, now 730).  Bound by these reads and additions: 8 experts of 2048 rows, 8192 x 8192:
// 2340 us, 1.9 PFLOP/s.
//
// Scales that are powers of two, long runs: the tensor cores apply them, and a sum leaves them every eight blocks at the
// latest (further below; 1340 us for the same, 3.3 PFLOP/s).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "launch.h"

namespace moe {
namespace {

// ---------------------------------------------------------------- values
// The smallest power of two 2^p with amax <= 448 2^p, and its inverse (448 = 1.75 x 2^8); zero: 1; infinity or NaN: NaN.
__device__ __forceinline__ void fp8_scale(uint32_t amax_bits, float& scale, float& inv) {
  // the exponent field of amax, one more above 1.75 (a carry out of the mantissa), less 8
  const int e = max(1, (int)((amax_bits + 0x1fffffu) >> 23) - 8);
  scale = __uint_as_float((uint32_t)e << 23);
  inv = __uint_as_float((uint32_t)(254 - e) << 23);
  if (amax_bits == 0u) scale = inv = 1.f;
  if (amax_bits >= 0x7f800000u) scale = inv = __uint_as_float(0x7fc00000u);
}
__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
// Two values to e4m3, nearest (ties to even): a in the low byte.
__device__ __forceinline__ uint32_t fp8_pair(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t fp8_four(float a, float b, float c, float d) {
  return fp8_pair(a, b) | fp8_pair(c, d) << 16;
}

// ---------------------------------------------------------------- weights
__device__ __forceinline__ void unpack8(const uint4& r, float (&f)[8]) {
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
__device__ __forceinline__ void load8(const __half* p, float (&f)[8]) { unpack8(*reinterpret_cast<const uint4*>(p), f); }
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// A block takes one 128 x 128 tile of W: its values stay in registers until the largest magnitude is known, and
// leave through shared memory, four inputs of an output to a word, whole 128-byte rows at a time.
template <typename T>
__global__ void __launch_bounds__(256) fp8_weights_kernel(const T* __restrict__ W, int K, int N,
                                                          uint8_t* __restrict__ Wq, float* __restrict__ scales) {
  __shared__ uint32_t tile[128 * 32];
  __shared__ uint32_t top[8];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, nk = K / 128, nn = N / 128;
  const long long b = blockIdx.x;
  const int nb = (int)(b % nn), kb = (int)(b / nn % nk);
  const long long e = b / nn / nk;
  const T* src = W + (e * K + kb * 128) * N + nb * 128;
  // rows 4 q + i and 64 + 4 q + i, columns 8 c ..
  const int c = tid & 15, q = tid >> 4;
  float f[2][4][8];
  uint32_t m = 0;
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int i = 0; i < 4; ++i) load8(src + (long long)(64 * g + 4 * q + i) * N + 8 * c, f[g][i]);
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, magnitude_bits(f[g][i][j]));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) top[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max(m, top[w]);
  float scale, inv;
  fp8_scale(m, scale, inv);
  // word (n, k / 4) at n 32 + (k / 4 ^ n / 8): the 16 columns groups of a warp's stores fall into different banks
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      tile[(8 * c + j) * 32 + ((16 * g + q) ^ c)] =
          fp8_four(f[g][0][j] * inv, f[g][1][j] * inv, f[g][2][j] * inv, f[g][3][j] * inv);
  __syncthreads();
  uint8_t* dst = Wq + (e * N + nb * 128) * K + kb * 128;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int n = r * 32 + (tid >> 3), p = tid & 7;
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = tile[n * 32 + ((4 * p + i) ^ (n >> 3))];
    *reinterpret_cast<uint4*>(dst + (long long)n * K + 16 * p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
  if (tid == 0) scales[(e * nn + nb) * nk + kb] = scale;
}

// ---------------------------------------------------------------- slots
// Boundaries of the experts' slots as every kernel here uses them, by one warp: the largest offset so far, clamped
// to [0, S_max], so that runs never overlap or leave the buffers.  prefix[e] (not null): tiles of at most `nmax`
// rows of the experts before e.  True where an offset was changed.  kAhead x 32 boundaries are loaded together (one
// after another, each load takes the latency of L2, which short batches notice).
template <int kAhead>
__device__ __forceinline__ bool slot_table(const int32_t* offsets, int E, int S_max, int nmax, int32_t* offs,
                                           int32_t* prefix) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  int run = 0, tiles = 0;
  for (int base = 0; base <= E; base += 32 * kAhead) {
    int o[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) o[i] = base + 32 * i + lane <= E ? __ldcg(offsets + base + 32 * i + lane) : 0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int e = base + 32 * i + lane;
      if (e - lane > E) break;
      int v = min(max(o[i], 0), S_max);
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const int q = __shfl_up_sync(0xffffffffu, v, k);
        if (lane >= k) v = max(v, q);
      }
      v = max(v, run);
      bad |= e <= E && v != o[i];
      if (e <= E) offs[e] = v;
      int before = __shfl_up_sync(0xffffffffu, v, 1);
      if (lane == 0) before = run;
      run = __shfl_sync(0xffffffffu, v, 31);
      if (!prefix) continue;
      int c = e >= 1 && e <= E ? (v - before + nmax - 1) / nmax : 0;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const int q = __shfl_up_sync(0xffffffffu, c, k);
        if (lane >= k) c += q;
      }
      if (e <= E) prefix[e] = tiles + c;
      tiles += __shfl_sync(0xffffffffu, c, 31);
    }
  }
  return bad;
}
// Where the scales of expert e's slots begin in a row of scales: a multiple of four, and no run reaches the next
// (rounded up to four, a run is at least three shorter than its slots; four are added for each expert).
__device__ __forceinline__ int scale_base(int first_slot, int e) { return ((first_slot + 3) & ~3) + 4 * e; }
// Where block b's exponent of a place's scale is.
__device__ __forceinline__ size_t exponent_at(int b, int place, int Sp) { return ((size_t)(b >> 2) * Sp + place) * 4 + (b & 3); }
int scale_row(int S_max, int E) { return (S_max + 3) / 4 * 4 + 4 * (E + 1); }

// ---------------------------------------------------------------- rows
// Slot s of an expert: its token's row in 8 bits.  A warp takes up to eight blocks of 128 columns (by blockIdx.y), 16 lanes
// each, of neighbouring slots: their tokens come 32 at a time, their expert is looked for once, and the scales of 16 slots
// leave together.  It clears the status word, so a block says in a word of its own whether a slot's token was out of range,
// for the first product to report (a memset before this kernel took 3 us).  32768 slots x 2048: 30 us cold (42 with a
// division, a search and a load of the token for each slot, and its scales as words and bytes of their own).
// sx is [d / 128][Sp], a slot's place in it by scale_base.
constexpr int kRowPart = 8;
constexpr int kMaxRowBlocks = 1024;
__global__ void __launch_bounds__(256, 6) fp8_rows_kernel(const __half* __restrict__ tokens, const int32_t* __restrict__ perm,
                                                       const int32_t* __restrict__ offsets, int E, int S_max, int T, int d,
                                                       int Sp, uint8_t* __restrict__ Xq, float* __restrict__ sx,
                                                       int* status, const float* __restrict__ s1,
                                                       const float* __restrict__ s2, long long ns, uint32_t* __restrict__ xexp,
                                                       int* __restrict__ bad_rows,
                                                       int* general) {
  extern __shared__ int32_t offs[];
  pdl_wait();
  pdl_trigger();
  const int block = blockIdx.y * gridDim.x + blockIdx.x;
  if (block == 0 && threadIdx.x == 0) *status = 0;
  if (threadIdx.x < 32) slot_table<8>(offsets, E, S_max, 1, offs, nullptr);   // (what is wrong there, the products report)
  __syncthreads();
  // (slots before offsets[0] belong to no expert: a plan may be a slice of a larger one)
  const int lane = threadIdx.x & 31, l = lane & 15, nb = d / 128, S0 = offs[0], S = offs[E] - S0;
  const int h = lane >> 4, b0 = blockIdx.y * kRowPart + h;
  const int warps = gridDim.x * 8, w = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int first = S0 + (int)((long long)S * w / warps), end = S0 + (int)((long long)S * (w + 1) / warps);
  bool bad = false;
  int lo = 0, hi = E;                            // the last e with offs[e] <= s
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (offs[mid] <= first) lo = mid; else hi = mid;
  }
  int next = offs[lo + 1], base = scale_base(offs[lo], lo) - offs[lo], tokens_of = 0;
  uint32_t held[kRowPart / 2] = {};              // the scales of one of up to 16 slots, which leave side by side
  int place = -1;
  for (int s = first; s < end; ++s) {
    if (((s - first) & 31) == 0) tokens_of = s + lane < end ? perm[s + lane] : 0;
    const int t = __shfl_sync(0xffffffffu, tokens_of, (s - first) & 31);
    const bool in = (unsigned)t < (unsigned)T;
    bad |= !in;
    const __half* src = tokens + (long long)(in ? t : 0) * d + l * 8;
    uint4 r[kRowPart / 2];
#pragma unroll
    for (int i = 0; i < kRowPart / 2; ++i)
      r[i] = b0 + 2 * i < nb && in ? *reinterpret_cast<const uint4*>(src + (b0 + 2 * i) * 128) : make_uint4(0u, 0u, 0u, 0u);
    while (s >= next) {                          // (s < offs[E])
      ++lo;
      next = offs[lo + 1];
      base = scale_base(offs[lo], lo) - offs[lo];
    }
    const int turn = (s - first) & 15;
    if (l == turn) place = base + s;
    uint8_t* dst = Xq + (long long)s * d + l * 8;
#pragma unroll
    for (int i = 0; i < kRowPart / 2; ++i) {
      const int b = b0 + 2 * i;
      // the largest magnitude, two at a time as integers: infinity and NaN are above all others
      uint32_t m = __vmaxu2(__vmaxu2(r[i].x & 0x7fff7fffu, r[i].y & 0x7fff7fffu),
                            __vmaxu2(r[i].z & 0x7fff7fffu, r[i].w & 0x7fff7fffu));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
      float scale, inv;
      fp8_scale(__float_as_uint(__half2float(__ushort_as_half((unsigned short)max(m & 0xffffu, m >> 16)))), scale, inv);
      float f[8];
      unpack8(r[i], f);
      if (l == turn) held[i] = __float_as_uint(scale);
      if (b < nb)
        *reinterpret_cast<uint2*>(dst + b * 128) =
            make_uint2(fp8_four(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                       fp8_four(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
    }
    if (turn < 15 && s + 1 < end) continue;
#pragma unroll
    for (int i = 0; i < kRowPart / 2; ++i)
      if (place >= 0 && b0 + 2 * i < nb) sx[(size_t)(b0 + 2 * i) * Sp + place] = __uint_as_float(held[i]);
    if (xexp) {                                  // a half has the odd or the even blocks' bytes of two words
      uint32_t e[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        e[i] = (held[2 * i] >> 23 & 0xffu) << (8 * h) | (held[2 * i + 1] >> 23 & 0xffu) << (16 + 8 * h);
        e[i] |= __shfl_xor_sync(0xffffffffu, e[i], 16);
      }
      const int word = blockIdx.y * (kRowPart / 4) + h;
      if (place >= 0 && 4 * word < nb) xexp[(size_t)word * Sp + place] = h ? e[1] : e[0];
    }
    place = -1;
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) bad_rows[block] = any;
  if (general) {                                 // (ns of each; NaN, as the quantiser writes it, has the exponent's form too)
    bool other = false;
    const long long at = block, step = (long long)gridDim.x * gridDim.y * 256;
    for (long long i = at * 256 + threadIdx.x; i < 2 * ns; i += step) {
      const uint32_t v = __float_as_uint(i < ns ? s1[i] : s2[i - ns]);
      other |= (v & 0x807fffffu) != 0u && v != 0x7fc00000u;
      other |= v == 0u || v == 0x7f800000u;
    }
    if (__any_sync(0xffffffffu, other) && lane == 0) *general = 1;
  }
}

// ---------------------------------------------------------------- products
// Warps 0 to 3 load the weight tiles, issue the products, multiply the scales and load the rows; eight more add.
// (One warp for both loads took 600 cycles a block of its own time, and bound the kernel; 16 warps for the sums are no
// faster: TMEM's reads bound them.)
constexpr int kEpiWarps = 8;                  // two column groups of the four TMEM lane quarters
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kABytes = 128 * 128;            // a weight tile: 128 outputs, 128 inputs
constexpr int kScaleSlots = 8;                // blocks whose scales are on their way
constexpr int kMaxSlots = 16;                 // sums in TMEM
constexpr int kMaxStages = 12;                // of either ring
constexpr size_t kMinSmem = 116 * 1024;       // one block per SM: each takes all of TMEM
// Weight tiles and rows have rings of their own: na tiles of 16 KB, nb runs of nmax rows.
struct Fp8Smem {
  uint32_t b_off, b_bytes, raw_off, raw_bytes, scale_off, scale_bytes, amax_off, inv_off, join_off, bars_off, misc_off, total;
};
__host__ __device__ inline Fp8Smem fp8_smem(int nmax, int na, int nb, int E, int split) {
  Fp8Smem L;
  uint32_t off = (uint32_t)(na * kABytes);
  L.b_off = off;
  L.b_bytes = (uint32_t)nmax * 128u;
  off += (uint32_t)nb * L.b_bytes;
  L.raw_off = off;                            // the rows' scales of a block, and the weight tiles'
  L.raw_bytes = (uint32_t)nmax * 4u + 16u;
  off += kScaleSlots * L.raw_bytes;
  L.scale_off = off;                          // their products, for each sum's slot
  L.scale_bytes = (uint32_t)nmax * 4u;
  const uint32_t slots = 512u / (uint32_t)nmax;
  off += (slots < kMaxSlots ? slots : kMaxSlots) * L.scale_bytes;
  L.amax_off = off;
  off += 2u * (uint32_t)nmax * 16u;           // two items' [column][lane quarter]
  L.inv_off = off;
  off += (uint32_t)(kEpiWarps / 2) * (uint32_t)nmax * 4u;   // a warp's columns are half of a tile's
  L.join_off = off;
  off += (uint32_t)(split - 1) * (uint32_t)nmax * 512u;   // the other blocks' sums
  L.bars_off = off;
  off += (4u * kMaxStages + 2u * kMaxSlots + 2u) * 8u;
  L.misc_off = off;
  off += 16u + 8u * (uint32_t)(E + 1);
  L.total = off + 1024u;                      // slack for the alignment of the rings
  return L;
}

struct Fp8Args {
  const int32_t* offsets;
  const float* wscale;         // [E][M / 128][K / 128]
  const float* xscale;         // [K / 128][Sp]
  int E, S_max, Sp, K, M, na, nb, nslots;
  int split;                   // blocks of a cluster that share an item
  uint8_t* h;                  // first product: [S_max][M], with hscale [M / 128][Sp]
  float* hscale;
  const uint32_t* xexp;        // the scales' exponents, of four blocks a word: [K / 512][Sp], and of h (by bytes)
  uint8_t* hexp;
  __half* out;                 // second: [S_max][M]
  int* status;
  const int* bad_rows;         // of the rows' blocks; first product
  int row_blocks;
  const int* general;          // not null: which of two forms runs (not 0: the one for any scales)
};

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 16 lanes x 8 X columns: of each eight columns lane l gets columns 2 (l % 4) and the next of rows l / 4 (r[0], r[1])
// and l / 4 + 8.  Valid after tmem_wait.
template <int X>
__device__ __forceinline__ void tmem_ld16(uint32_t t, uint32_t* r) {
  if constexpr (X == 4)
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t));
  else if constexpr (X == 2)
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(t));
  else
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(t));
}
// All 32 lanes of a quarter, B groups of eight columns: v[half][4 b ..].
template <int B>
__device__ __forceinline__ void tmem_ld32(uint32_t t, uint32_t (&v)[2][4 * B]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t at = t + ((uint32_t)(16 * h) << 16);
#pragma unroll
    for (int b = 0; b + 4 <= B; b += 4) tmem_ld16<4>(at + 8 * b, v[h] + 4 * b);
    if constexpr (B % 4 >= 2) tmem_ld16<2>(at + 8 * (B / 4 * 4), v[h] + 16 * (B / 4));
    if constexpr (B % 2) tmem_ld16<1>(at + 8 * (B - 1), v[h] + 4 * (B - 1));
  }
}
template <int B>
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[2][4 * B]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 4 * B; ++i) asm volatile("" : "+r"(v[h][i]));   // no use of them moves above the wait
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
// The 128 rows of a weight tile, in each 32 of them rows 4 r + j at place 8 j + r: a lane's four TMEM rows of a
// column (r + 8 j) then are four neighbouring outputs, and leave as one store.
__device__ __forceinline__ void load_weight_tile(void* smem, const CUtensorMap* m, int x, int group, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(smem)),
      "l"(m), "r"(x), "r"(0), "r"(0), "r"(group), "r"(smem_u32(bar))
      : "memory");
}
// 4 and 16 bytes global -> shared, by the thread itself.
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// Clusters: all threads meet; the first block's address of a shared-memory address; stores and arrivals there.
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t first_block(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void store_remote(uint32_t addr, float2 v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Pairs of blocks (two neighbours of a cluster, the first one issues): products of 256 weight rows, 128 in each block's
// shared memory and TMEM, with rows of which each block holds half; loads that complete on the first block's barrier;
// arrivals on the same barrier of both blocks once the products so far are done.
__device__ __forceinline__ void mma_mx_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void load_rows_pair(void* smem, const CUtensorMap* m, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(smem)),
      "l"(m), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void load_weight_tile_pair(void* smem, const CUtensorMap* m, int x, int group, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(smem)),
      "l"(m), "r"(x), "r"(0), "r"(0), "r"(group), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* holder) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(holder)) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr));
}
// 32 lanes of a quarter: a column, or eight, of 32-bit words.
__device__ __forceinline__ void tmem_st4(uint32_t t, uint32_t w) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%1,%1,%1};" ::"r"(t), "r"(w) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t t, const uint32_t (&w)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// An arrival at another block's barrier with no memory to publish but TMEM's, which the fence before it orders.
__device__ __forceinline__ void arrive_remote_tmem(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// As mbar_wait_bounded; the clock is read only by a wait that is long already.
template <bool kCluster = false>
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  uint64_t t0 = 0;
  for (uint32_t it = 1; !(kCluster ? try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)); ++it) {
    if ((it & 63u) == 0) {
      if (*abort) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kDefaultWaitNs) {
        record_status(status, kErrTimeout);
        *abort = 1;
        return false;
      }
    }
  }
  return true;
}

// Two 32-bit operations at a time.
__device__ __forceinline__ unsigned long long bits2(float2 v) {
  return (unsigned long long)__float_as_uint(v.y) << 32 | __float_as_uint(v.x);
}
__device__ __forceinline__ float2 float2_of(unsigned long long r) {
  return make_float2(__uint_as_float((uint32_t)r), __uint_as_float((uint32_t)(r >> 32)));
}
__device__ __forceinline__ float2 pair(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(r);
}
// The larger magnitude; NaN if either is (as a positive number's bits).
__device__ __forceinline__ float max_nan(float m, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
  return r;
}
__device__ __forceinline__ void add2(float2& d, float2 a) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(d)), "l"(bits2(a)));
  d = float2_of(r);
}
__device__ __forceinline__ void fma2(float2& d, float2 a, float2 b) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(d)));
  d = float2_of(r);
}

// GeLU of two values as gelu_tanh writes it, x / (1 + 2^z) with z = -2 log2(e) sqrt(2 / pi) (x + 0.044715 x^3), by the
// hardware's exponential (2 ulp and |z| 2^-24) and reciprocal (1 ulp) with subnormals taken as zero, which neither the
// sum with one nor the quotient notices.  (By the library's functions, which keep them, 128 x 160 values took 5300
// cycles, not what the two operations need, 2560: 16 a cycle.)
__device__ __forceinline__ float2 gelu2(float2 x) {
  const float2 c1 = make_float2(-0.1029432397f, -0.1029432397f), c0 = make_float2(-2.3022081985f, -2.3022081985f);
  float2 a = c0;
  fma2(a, mul2(x, x), c1);
  const float2 z = mul2(x, a);
  float2 e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(z.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(z.y));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(1.f + e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(1.f + e.y));
  return mul2(x, r);
}

// The rows by boxes of 128, 64 and 32 of them; of long runs, of 24, 48, .. 120.
struct RowMaps {
  CUtensorMap box[5];
};

struct Tile8 {
  int e, row0, n, mt;
  int sc0;                                    // its first slot's place in a row of scales
};
// Item i: an expert, a weight tile and a run of its rows; the runs of one weight tile are next to each other, on
// different SMs at the same time, and share it in L2.
__device__ __forceinline__ Tile8 tile_at(int i, const int32_t* prefix, const int32_t* offs, int E, int mt, int nmax) {
  int lo = 0, hi = E;                         // largest e with prefix[e] mt <= i
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] * mt <= i) lo = mid; else hi = mid;
  }
  const int chunks = prefix[lo + 1] - prefix[lo], local = i - prefix[lo] * mt;
  const int rows = offs[lo + 1] - offs[lo];
  const int per = ((rows + chunks - 1) / chunks + 15) & ~15;   // runs of about the same length, at most nmax
  Tile8 t;
  t.e = lo;
  t.mt = local / chunks;
  const int c = local - t.mt * chunks;
  t.row0 = offs[lo] + c * per;
  t.sc0 = scale_base(offs[lo], lo) + c * per;
  t.n = min(per, rows - c * per);
  return t;
}

// What becomes of a warp's sums: acc[c][j] has rows lr + 8 j of the quarter's 32 (four neighbouring outputs) and columns lc and
// lc + 1 of eight.  kExp: h's scales as exponents.  cw: groups of eight columns of each warp; am: [column][quarter], invs: the
// warp's columns.
template <int C8, bool kGelu, bool kExp>
__device__ __forceinline__ void finish(float2 (&acc)[C8][4], const Tile8& t, const Fp8Args& a, int cw, int col0, int q,
                                       int g, int lane, uint32_t* am, float* invs, bool ok) {
  const int lr = lane >> 2, lc = 2 * (lane & 3);
  const size_t tile0 = (size_t)t.row0 * a.M + t.mt * 128 + 32 * q + 4 * lr;   // this lane's four outputs of a slot
  if constexpr (kGelu) {
    // GeLU, the largest magnitude of each slot's 128 columns (four warps), and 8 bits
#pragma unroll
    for (int c = 0; c < C8; ++c) {
      if (c >= cw) continue;
      float m0 = 0.f, m1 = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[c][j] = gelu2(acc[c][j]);
        m0 = max_nan(m0, acc[c][j].x);
        m1 = max_nan(m1, acc[c][j].y);
      }
      uint32_t b0 = __float_as_uint(m0), b1 = __float_as_uint(m1);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        b0 = max(b0, __shfl_xor_sync(0xffffffffu, b0, o));
        b1 = max(b1, __shfl_xor_sync(0xffffffffu, b1, o));
      }
      if (lr == 0) {
        am[(col0 + c * 8 + lc) * 4 + q] = b0;
        am[(col0 + c * 8 + lc + 1) * 4 + q] = b1;
      }
    }
    asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory");
    if (!ok) return;
    // a lane makes the scale of a column, for its whole warp
    for (int c = lane; c < 8 * cw; c += 32) {
      const int col = col0 + c;
      const uint4 r = *reinterpret_cast<const uint4*>(am + col * 4);
      float scale, inv;
      fp8_scale(max(max(r.x, r.y), max(r.z, r.w)), scale, inv);
      invs[c] = inv;
      if (q == 0 && col < t.n) {
        if (kExp) a.hexp[exponent_at(t.mt, t.sc0 + col, a.Sp)] = (uint8_t)(__float_as_uint(scale) >> 23);
        else a.hscale[(size_t)t.mt * a.Sp + t.sc0 + col] = scale;
      }
    }
    __syncwarp();
    uint8_t* dst = a.h + tile0 + (size_t)(col0 + lc) * a.M;
#pragma unroll
    for (int c = 0; c < C8; ++c) {
      if (c >= cw) continue;
      const float2 inv = *reinterpret_cast<const float2*>(invs + c * 8 + lc);
      float2 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = mul2(acc[c][j], inv);
      const int col = col0 + c * 8 + lc;
      if (col < t.n) *reinterpret_cast<uint32_t*>(dst) = fp8_four(v[0].x, v[1].x, v[2].x, v[3].x);
      if (col + 1 < t.n) *reinterpret_cast<uint32_t*>(dst + a.M) = fp8_four(v[0].y, v[1].y, v[2].y, v[3].y);
      dst += 8 * (size_t)a.M;
    }
    __syncwarp();                            // (the warp's scales are written again with the next item)
  } else {
    if (!ok) return;
#pragma unroll
    for (int c = 0; c < C8; ++c) {
      if (c >= cw) continue;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int col = col0 + c * 8 + lc + p;
        if (col < t.n) {
          const float2 (&v)[4] = acc[c];
          const __half2 lo = p ? __floats2half2_rn(v[0].y, v[1].y) : __floats2half2_rn(v[0].x, v[1].x);
          const __half2 hi = p ? __floats2half2_rn(v[2].y, v[3].y) : __floats2half2_rn(v[2].x, v[3].x);
          *reinterpret_cast<uint2*>(a.out + tile0 + (size_t)col * a.M) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        }
      }
    }
  }
}

// C8: groups of eight columns per warp (a tile has up to 16 C8 rows).  kGelu: first product.  kSplit: a cluster of
// a.split blocks takes an item, each a part of its inputs; the blocks' sums go to the first block's shared memory, which
// adds them in order.  One item for each cluster at most.
template <int C8, bool kGelu, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ RowMaps tmB, const Fp8Args a) {
  constexpr int NMAX = 16 * C8;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const Fp8Smem L = fp8_smem(NMAX, a.na, a.nb, a.E, kSplit ? a.split : 1);
  uint64_t* a_full = reinterpret_cast<uint64_t*>(sm + L.bars_off);
  uint64_t *a_empty = a_full + kMaxStages, *b_full = a_empty + kMaxStages, *b_empty = b_full + kMaxStages,
           *acc_full = b_empty + kMaxStages, *acc_empty = acc_full + kMaxSlots, *spare = acc_empty + kMaxSlots, *joined = spare + 1;
  uint32_t* holder = reinterpret_cast<uint32_t*>(sm + L.misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L.misc_off + 4);
  int32_t* prefix = reinterpret_cast<int32_t*>(sm + L.misc_off + 16);
  int32_t* offs = prefix + a.E + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    if (lane < a.na) {
      mbar_init(&a_full[lane], 1);
      mbar_init(&a_empty[lane], 1);
    }
    if (lane < a.nb) {
      mbar_init(&b_full[lane], 1);
      mbar_init(&b_empty[lane], 1);
    }
    if (lane < a.nslots) {
      mbar_init(&acc_full[lane], 2);            // the sum and its scales
      mbar_init(&acc_empty[lane], kEpiWarps);
    }
    if (lane == 0) {
      mbar_init(spare, 1);
      mbar_init(joined, kSplit ? (a.split - 1) * kEpiWarps : 1);
      *abort_flag = 0;
    }
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) prefetch_tmap(&tmA);
  if (warp == 3 && lane < 3) prefetch_tmap(&tmB.box[lane]);
  if (warp == 1) tmem_alloc(holder, 512);
  pdl_wait();
  pdl_trigger();
  if (a.general && *a.general == 0) {            // (the form for scales that are powers of two has run)
    __syncthreads();
    if (warp == 1) tmem_dealloc(*holder, 512);
    return;
  }
  if (kGelu && blockIdx.x == 0 && warp == 3) {
    int bad = 0;
    for (int i = lane; i < a.row_blocks; i += 32) bad |= a.bad_rows[i];
    if (bad) record_status(a.status, kErrBounds);
  }
  if (warp == 2 && slot_table<(C8 <= 4 ? 8 : 1)>(a.offsets, a.E, a.S_max, NMAX, offs, prefix)) record_status(a.status, kErrBounds);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;
  const int mt = a.M / 128, nkb = a.K / 128;
  if constexpr (kSplit) cluster_meet();          // the first block's barrier is set up, and the block is there
  const int part = kSplit ? (int)(blockIdx.x % a.split) : 0;
  const int kb0 = kSplit ? nkb * part / a.split : 0, kb1 = kSplit ? nkb * (part + 1) / a.split : nkb;
  // this block's items (not kept in registers)
  auto first_item = [&]() { return (int)(kSplit ? blockIdx.x / a.split : blockIdx.x); };
  auto item_step = [&]() { return (int)(kSplit ? gridDim.x / a.split : gridDim.x); };
  const int total = prefix[a.E] * mt;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_for(bar, parity, abort_flag, a.status); };
  uint32_t issued = 0, issued_par = 0;           // ring places with a load in flight, for the end
  auto note = [&](int at, uint32_t par) {
    issued |= 1u << at;
    issued_par = (issued_par & ~(1u << at)) | par << at;
  };
  if (warp < 4) {
    regs_down<56>();
    if (warp == 0) {
      // ---------------------------------------------------------- weight tiles
      // (These three loops are run by whole warps, and one lane issues: their values stay uniform, and a block takes
      // half the time that it takes a lane alone.)
      int st = 0;
      uint32_t sp = 1;
      bool ok = true;
      for (int i = first_item(); i < total && ok; i += item_step()) {
        const Tile8 t = tile_at(i, prefix, offs, a.E, mt, NMAX);
        const int agroup = t.e * (a.M / 32) + t.mt * 4;
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = __all_sync(0xffffffffu, wait(&a_empty[st], sp));
          if (!ok) break;
          note(st, sp ^ 1u);
          if (elect_one()) {
            mbar_expect_tx(&a_full[st], kABytes);
            load_weight_tile(sm + st * kABytes, &tmA, kb * 128, agroup, &a_full[st]);
          }
          if (++st == a.na) {
            st = 0;
            sp ^= 1u;
          }
        }
      }
    } else if (warp == 3) {
      // ---------------------------------------------------------- rows
      int st = 0;
      uint32_t sp = 1;
      bool ok = true;
      for (int i = first_item(); i < total && ok; i += item_step()) {
        const Tile8 t = tile_at(i, prefix, offs, a.E, mt, NMAX);
        const int rows = (t.n + 31) & ~31;
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = __all_sync(0xffffffffu, wait(&b_empty[st], sp));
          if (!ok) break;
          note(st, sp ^ 1u);
          uint8_t* to = sm + L.b_off + st * L.b_bytes;
          if (elect_one()) {
            mbar_expect_tx(&b_full[st], (uint32_t)rows * 128u);
            int r = 0;
            if constexpr (NMAX >= 128)
              for (; r + 128 <= rows; r += 128) tma_load_2d(to + r * 128, &tmB.box[0], kb * 128, t.row0 + r, &b_full[st]);
            if constexpr (NMAX >= 64)
              if (rows - r >= 64) {
                tma_load_2d(to + r * 128, &tmB.box[1], kb * 128, t.row0 + r, &b_full[st]);
                r += 64;
              }
            if (r < rows) tma_load_2d(to + r * 128, &tmB.box[2], kb * 128, t.row0 + r, &b_full[st]);
          }
          if (++st == a.nb) {
            st = 0;
            sp ^= 1u;
          }
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- products
      int as = 0, bs = 0, slot = 0;
      uint32_t asp = 0, bsp = 0, ap = 1;
      bool ok = true;
      // descriptors differ only in the start address (16-byte units, bits 0..13)
      const uint64_t d0 = smem_desc(smem_u32(sm), 16, 1024, 2);
      const uint32_t b0 = L.b_off >> 4, b16 = L.b_bytes >> 4;
      for (int i = first_item(); i < total && ok; i += item_step()) {
        const Tile8 t = tile_at(i, prefix, offs, a.E, mt, NMAX);
        const uint32_t idesc = idesc_f16(128, (t.n + 15) & ~15, 0, 0);   // (e4m3 has f16's code 0)
        for (int kb = kb0; kb < kb1; ++kb) {
          // rows, weight tile and a free slot: a lane waits for each
          uint64_t* bar = lane == 0 ? &b_full[bs] : lane == 1 ? &a_full[as] : &acc_empty[slot];
          ok = __all_sync(0xffffffffu, wait(bar, lane == 0 ? bsp : lane == 1 ? asp : ap));
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = d0 + (uint64_t)(as * (kABytes >> 4)), bd = d0 + (uint64_t)(b0 + bs * b16);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f8(tmem + slot * NMAX, ad + 2 * k, bd + 2 * k, idesc, k ? 1u : 0u);
            tc_commit(&acc_full[slot]);
            tc_commit(&a_empty[as]);
            tc_commit(&b_empty[bs]);
          }
          if (++slot == a.nslots) {
            slot = 0;
            ap ^= 1u;
          }
          if (++as == a.na) {
            as = 0;
            asp ^= 1u;
          }
          if (++bs == a.nb) {
            bs = 0;
            bsp ^= 1u;
          }
        }
      }
    } else {
      // ---------------------------------------------------------- scales
      // Copies run kScaleSlots - 1 blocks ahead of their use, over the ends of items; each lane reads what it copied
      // itself, but for the weight tiles' scales.
      int li = first_item(), lkb = kb0, ls = 0;
      Tile8 lt = {};
      if (li < total) lt = tile_at(li, prefix, offs, a.E, mt, NMAX);
      auto next_copy = [&]() {
        if (li < total) {
          const uint32_t dst = smem_u32(sm + L.raw_off) + ls * L.raw_bytes;
          const float* src = a.xscale + (size_t)lkb * a.Sp + lt.sc0;
#pragma unroll
          for (int j = lane; j < NMAX / 4; j += 32)
            if (4 * j < lt.n) copy16(dst + 16 * j, src + 4 * j);
          if (lane == 0) copy4(dst + NMAX * 4, a.wscale + ((size_t)lt.e * mt + lt.mt) * nkb + lkb);
          if (++ls == kScaleSlots) ls = 0;
          if (++lkb == kb1) {
            lkb = kb0;
            li += item_step();
            if (li < total) lt = tile_at(li, prefix, offs, a.E, mt, NMAX);
          }
        }
        copies_commit();
      };
      for (int k = 0; k < kScaleSlots - 1; ++k) next_copy();
      int slot = 0, us = 0;
      uint32_t ap = 1;
      bool ok = true;
      for (int i = first_item(); i < total && ok; i += item_step()) {
        const int n = tile_at(i, prefix, offs, a.E, mt, NMAX).n;
        for (int kb = kb0; kb < kb1; ++kb) {
          copies_wait<kScaleSlots - 2>();
          __syncwarp();
          const uint8_t* raw = sm + L.raw_off + us * L.raw_bytes;
          if (++us == kScaleSlots) us = 0;
          ok = __all_sync(0xffffffffu, wait(&acc_empty[slot], ap));
          if (!ok) break;
          const float w = reinterpret_cast<const float*>(raw)[NMAX];
          float4* to = reinterpret_cast<float4*>(sm + L.scale_off + slot * L.scale_bytes);
#pragma unroll
          for (int j = lane; j < NMAX / 4; j += 32) {
            const float4 x = reinterpret_cast<const float4*>(raw)[j];
            if (4 * j < n) to[j] = make_float4(x.x * w, x.y * w, x.z * w, x.w * w);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_full[slot]);
          if (++slot == a.nslots) {
            slot = 0;
            ap ^= 1u;
          }
          next_copy();                           // into the ring's place before this one: read, behind __syncwarp
        }
      }
      copies_wait<0>();
    }
  } else {
    regs_up<224>();
    // ------------------------------------------------------------ sums
    const int q = warp & 3, g = (warp - 4) >> 2;
    const int lc = 2 * (lane & 3);
    const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
    int slot = 0;
    uint32_t ap = 0;
    bool ok = true;
    int turn = 0;
    // a warp whose wait gives up still meets the others at every item's barrier
    for (int i = first_item(); i < total; i += item_step(), turn ^= 1) {
      const Tile8 t = tile_at(i, prefix, offs, a.E, mt, NMAX);
      const int cw = (t.n + 15) >> 4;            // groups of eight columns of each warp of this tile
      const int col0 = g * cw * 8;
      float2 acc[C8][4];
#pragma unroll
      for (int c = 0; c < C8; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[c][j] = make_float2(0.f, 0.f);
      for (int kb = kb0; kb < kb1 && ok; ++kb) {
        ok = __all_sync(0xffffffffu, wait(&acc_full[slot], ap));
        if (!ok) break;
        tc_fence_after();
        const float* sc = reinterpret_cast<const float*>(sm + L.scale_off + slot * L.scale_bytes) + col0 + lc;
        const uint32_t ts = tq + slot * NMAX + col0;
        // (what is loaded beyond the tile's columns stays within the slot, and is not used)
        uint32_t v[2][4 * C8];
        float2 x[C8];
        tmem_ld32<C8>(ts, v);
#pragma unroll
        for (int c = 0; c < C8; ++c) x[c] = *reinterpret_cast<const float2*>(sc + c * 8);
        tmem_wait<C8>(v);
#pragma unroll
        for (int c = 0; c < C8; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            fma2(acc[c][j], pair(v[j >> 1][4 * c + 2 * (j & 1)], v[j >> 1][4 * c + 2 * (j & 1) + 1]), x[c]);
        tc_fence_before();                       // read: the slot may take the next sum
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[slot]);
        if (++slot == a.nslots) {
          slot = 0;
          ap ^= 1u;
        }
      }
      if constexpr (kSplit) {
        constexpr int kWords = C8 * 4 * 32 * kEpiWarps;
        const int tid = (warp - 4) * 32 + lane;
        if (part > 0) {
          if (ok) {
            const uint32_t to = first_block(smem_u32(sm + L.join_off)) + ((part - 1) * kWords + tid) * 8;
#pragma unroll
            for (int c = 0; c < C8; ++c)
#pragma unroll
              for (int j = 0; j < 4; ++j) store_remote(to + (c * 4 + j) * (32 * kEpiWarps * 8), acc[c][j]);
            __syncwarp();
            if (lane == 0) arrive_remote(first_block(smem_u32(joined)));
          }
          continue;
        }
        if (ok) ok = __all_sync(0xffffffffu, wait_for<true>(joined, 0, abort_flag, a.status));
        if (ok) {
          for (int p = 0; p + 1 < a.split; ++p) {
            const float2* from = reinterpret_cast<const float2*>(sm + L.join_off) + p * kWords + tid;
#pragma unroll
            for (int c = 0; c < C8; ++c)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 v = from[(c * 4 + j) * (32 * kEpiWarps)];
                acc[c][j] = make_float2(acc[c][j].x + v.x, acc[c][j].y + v.y);
              }
          }
        }
      }
      float* invs = reinterpret_cast<float*>(sm + L.inv_off) + (warp - 4) * (8 * C8);
      uint32_t* am = reinterpret_cast<uint32_t*>(sm + L.amax_off) + turn * (NMAX * 4);
      finish<C8, kGelu, false>(acc, t, a, cw, col0, q, g, lane, am, invs, ok);
    }
  }
  // ------------------------------------------------------------ end
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*abort_flag) {
    // what is still in flight lands before its memory is released (bounded)
    if ((warp == 0 || warp == 3) && lane == 0) {
      uint64_t* bars = warp == 0 ? a_full : b_full;
      for (int s = 0; s < kMaxStages; ++s)
        if (issued >> s & 1u) mbar_drain(&bars[s], issued_par >> s & 1u);
    }
    if (warp == 1) {
      if (elect_one()) tc_commit(spare);         // (the lane that issued the products)
      __syncwarp();
      if (lane == 0) mbar_drain(spare, 0);
    }
  }
  __syncwarp();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if constexpr (kSplit) cluster_meet();          // no block leaves while another may still write to its shared memory
}

// ---------------------------------------------------------------- products of long runs, scales that are powers of two
// The tensor cores apply such scales themselves (kind::mxf8f6f4: a scale for each 32 inputs of a row, as an exponent), so a
// tile's sum stays in TMEM over many blocks.  But their additions cut off what does not fit 24 bits, always towards zero:
// over all of 16384 inputs a sum of one sign lost 395 u (u = 2^-24; now at most 37), and hidden values next to the border of two 8-bit ones
// took the other more often than with sums that are rounded.  So a sum leaves TMEM after kLongSum blocks, for registers
// where it is added with rounding.  Outputs' distance from those of exact sums (rounded to f16 too), 2.4B top-2 layer
// at T = 16384: 1.4e-4 with all blocks in TMEM, 0.85e-4 with eight at a time (the register form 0.8e-4, sums by 32-bit matrix
// products 0.9e-4), 0.82e-4 with four; us: 2240, 2270, 2360; 64 experts of 512 rows, 2048 x 2048: 287, 292, 319 (six: 308).
// A pair of blocks takes 256 outputs and up to 240 rows: each loads its own weight tile and half of the rows, and has the
// sums of its 128 outputs in its own TMEM, in two places by turns: eight blocks' products run while the sum before is read,
// and 16 while the end of an item is worked on.
// Scales lie in TMEM as words, four blocks' exponents each: word (lane l, column i) is row 32 i + l's, in each quarter.
// Bound by the tensor cores with many inputs (490 cycles a block of 240 rows; their nominal rate is 480), by GeLU and the
// stores with few (2048: 25 % more), by DRAM where an expert has few rows.  What counts a block is what a warp issues:
// rows in four copies, not one, took 560 cycles and bound the kernel (2340 -> 1610 -> 1400 us with one copy).
constexpr int kLongRows = 240;
constexpr int kLongGroups = 3;                // of columns, each for the four warps of the TMEM lane quarters
constexpr int kLongThreads = 256 + 128 * kLongGroups;   // weight tiles, products, -, rows; four warps for scales; results
constexpr int kLongBox = 24;                  // rows are loaded by boxes of 24, 48 .. 120: each copy costs its warp 120 cycles
constexpr uint32_t kLongStage = kABytes + kLongRows / 2 * 128;
constexpr int kLongSum = 8;                   // blocks of 128 inputs, at most, whose sum stays in the tensor cores
constexpr uint32_t kScaleCols = 2 * kLongRows;   // two sets of 16 columns: four for the weight tile, eight for the rows
struct LongSmem {
  uint32_t amax_off, inv_off, bars_off, misc_off, total;
};
__host__ __device__ inline LongSmem long_smem(int stages, int E) {
  LongSmem L;
  uint32_t off = (uint32_t)stages * kLongStage;
  L.amax_off = off;
  off += 2u * kLongRows * 16u;
  L.inv_off = off;
  off += 4u * kLongRows * 4u;
  L.bars_off = off;
  off += (2u * kMaxStages + 9u) * 8u;
  L.misc_off = (off + 15u) & ~15u;
  L.total = L.misc_off + 16u + 8u * (uint32_t)(E + 1) + 1024u;
  return L;
}

template <bool kGelu>
__global__ void __launch_bounds__(kLongThreads, 1)
    fp8_long_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ RowMaps tmB, const Fp8Args a) {
  constexpr int C8 = kLongRows / 8 / kLongGroups, CH = 2, CF = 5;   // groups of eight columns: per warp, of a load, finished at once
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const LongSmem L = long_smem(a.na, a.E);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L.bars_off);
  uint64_t *empty = full + kMaxStages, *acc_full = empty + kMaxStages, *acc_empty = acc_full + 2, *sc_full = acc_empty + 2,
           *sc_empty = sc_full + 2, *spare = sc_empty + 2;
  uint32_t* holder = reinterpret_cast<uint32_t*>(sm + L.misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L.misc_off + 4);
  int32_t* prefix = reinterpret_cast<int32_t*>(sm + L.misc_off + 16);
  int32_t* offs = prefix + a.E + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = blockIdx.x & 1;
  if (warp == 0) {
    if (lane < a.na) {
      mbar_init(&full[lane], 2);                 // (the first block's two loading warps)
      mbar_init(&empty[lane], 1);
    }
    if (lane < 2) {
      mbar_init(&acc_full[lane], 1);
      mbar_init(&acc_empty[lane], 8 * kLongGroups);   // both blocks' warps
      mbar_init(&sc_full[lane], 8);
      mbar_init(&sc_empty[lane], 1);
    }
    if (lane == 0) {
      mbar_init(spare, 1);
      *abort_flag = 0;
    }
    fence_mbar_init();
    if (lane == 0) prefetch_tmap(&tmA);
  }
  if (warp == 3 && lane < 5) prefetch_tmap(&tmB.box[lane]);
  pdl_wait();
  pdl_trigger();
  if (*a.general) return;                        // (all blocks: the other form runs)
  if (warp == 1) tmem_alloc_pair(holder);
  if (kGelu && blockIdx.x == 0 && warp == 3) {
    int bad = 0;
    for (int i = lane; i < a.row_blocks; i += 32) bad |= a.bad_rows[i];
    if (bad) record_status(a.status, kErrBounds);
  }
  if (warp == 2 && slot_table<1>(a.offsets, a.E, a.S_max, kLongRows, offs, prefix)) record_status(a.status, kErrBounds);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_meet();                                // the other's barriers are set up, and it is there
  const uint32_t tmem = *holder;
  const int mt = a.M / 128, nkb = a.K / 128, pairs = gridDim.x / 2, total = prefix[a.E] * (mt / 2);
  const int segs = (nkb + kLongSum - 1) / kLongSum;   // sums of an item, of about as many blocks each
  auto item = [&](int i) {
    Tile8 t = tile_at(i, prefix, offs, a.E, mt / 2, kLongRows);
    t.mt = 2 * t.mt + part;
    return t;
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait_for(bar, parity, abort_flag, a.status)); };
  uint32_t issued = 0, issued_par = 0;           // ring places with a load in flight, for the end
  bool ok = true;
  if (warp < 8) {
    regs_down<56>();
    if (warp == 0 || warp == 3) {
      // ---------------------------------------------------------- weight tiles, rows
      // (run by whole warps, and one lane issues: the values stay uniform)
      int st = 0;
      uint32_t sp = 1;
      for (int i = blockIdx.x / 2; i < total && ok; i += pairs) {
        const Tile8 t = item(i);
        const int agroup = t.e * (a.M / 32) + t.mt * 4, half = ((t.n + 15) & ~15) / 2, y = t.row0 + part * half,
                    box = (half - 1) / kLongBox;
        for (int kb = 0; kb < nkb; ++kb) {
          ok = wait(&empty[st], sp);
          if (!ok) break;
          issued |= 1u << st;
          issued_par = (issued_par & ~(1u << st)) | (sp ^ 1u) << st;
          uint8_t* to = sm + st * kLongStage;
          if (elect_one()) {                     // (what lands before the first block expects it counts all the same)
            const uint32_t bar = first_block(smem_u32(&full[st]));
            if (warp == 0) {
              if (part == 0) mbar_expect_tx(&full[st], 2 * kABytes);
              load_weight_tile_pair(to, &tmA, kb * 128, agroup, bar);
            } else {
              if (part == 0) mbar_expect_tx(&full[st], (uint32_t)(box + 1) * (2 * kLongBox * 128));
              load_rows_pair(to + kABytes, &tmB.box[box], kb * 128, y, bar);
            }
          }
          if (++st == a.na) {
            st = 0;
            sp ^= 1u;
          }
        }
      }
      for (int n = 0; n < a.na && ok; ++n) {     // the first block's last arrivals here
        ok = wait(&empty[st], sp);
        if (++st == a.na) {
          st = 0;
          sp ^= 1u;
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- products
      int st = 0, set = 0, turn = 0;
      uint32_t fp = 0, scp = 0, ap = 1;
      const uint64_t d0 = smem_desc(smem_u32(sm), 16, 1024, 2);
      for (int i = blockIdx.x / 2; i < total && ok && part == 0; i += pairs) {
        // e4m3 both, exponents as scales, 256 outputs; which of a word's four is in bits 4 and 29
        const uint32_t idesc = 1u << 23 | (uint32_t)((item(i).n + 15) >> 4) << 18 | 16u << 24;
        for (int sg = 0, first = 0, end; sg < segs && ok; ++sg, first = end) {
          end = nkb * (sg + 1) / segs;
          for (int kb = first; kb < end; ++kb) {
            const int j = kb & 3;
            // rows and weight tiles, scales, a free place for the sum: a lane waits for each
            uint64_t* bar = lane == 1 && j == 0 ? &sc_full[set] : lane == 2 && kb == first ? &acc_empty[turn] : &full[st];
            ok = wait(bar, lane == 1 && j == 0 ? scp : lane == 2 && kb == first ? ap : fp);
            if (!ok) break;
            tc_fence_after();
            const uint64_t ad = d0 + (uint64_t)(st * (kLongStage >> 4)), bd = ad + (kABytes >> 4);
            const uint32_t id = idesc | (uint32_t)j << 4 | (uint32_t)j << 29, sc = tmem + kScaleCols + 16 * set;
            const bool group = j == 3 || kb + 1 == nkb;
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_mx_pair(tmem + turn * kLongRows, ad + 2 * k, bd + 2 * k, id, sc, sc + 4, kb - first + k ? 1u : 0u);
              commit_pair(&empty[st]);
              if (group) commit_pair(&sc_empty[set]);
              if (kb + 1 == end) commit_pair(&acc_full[turn]);
            }
            if (++st == a.na) {
              st = 0;
              fp ^= 1u;
            }
            if (group) {
              set ^= 1;
              if (set == 0) scp ^= 1u;
            }
          }
          turn ^= 1;
          if (turn == 0) ap ^= 1u;
        }
      }
    } else if (warp >= 4) {
      // ---------------------------------------------------------- scales
      // Loads run kAhead groups of four blocks ahead of their use, over the ends of items.
      constexpr int kAhead = 2;
      const uint32_t at = tmem + kScaleCols + ((uint32_t)(32 * (warp - 4)) << 16);
      int li = blockIdx.x / 2, lkb = 0, left = 0, set = 0;
      uint32_t sp = 1, w[kAhead] = {}, x[kAhead][8] = {};
      Tile8 t = {};
      if (li < total) t = item(li);
      auto load = [&](uint32_t& w, uint32_t (&x)[8]) {
        if (li >= total) return;
        ++left;
        w = lane < 4 && lkb + lane < nkb
                ? (__float_as_uint(__ldg(a.wscale + ((size_t)t.e * mt + t.mt) * nkb + lkb + lane)) >> 23) : 0u;
        const uint32_t* src = a.xexp + (size_t)(lkb / 4) * a.Sp + t.sc0 + lane;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (32 * c + lane < t.n) x[c] = __ldcg(src + 32 * c);
        lkb += 4;
        if (lkb >= nkb) {
          lkb = 0;
          li += pairs;
          if (li < total) t = item(li);
        }
      };
#pragma unroll
      for (int b = 0; b < kAhead; ++b) load(w[b], x[b]);
      while (left > 0 && ok) {
#pragma unroll
        for (int b = 0; b < kAhead; ++b) {
          if (left == 0 || !ok) break;
          --left;
          ok = wait(&sc_empty[set], sp);
          if (!ok) break;
          const uint32_t word = __reduce_or_sync(0xffffffffu, (w[b] & 0xffu) << (8 * (lane & 3)));
          tc_fence_after();
          tmem_st4(at + 16 * set, word);
          tmem_st8(at + 16 * set + 4, x[b]);
          tmem_stored();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (part == 0) mbar_arrive(&sc_full[set]);
            else arrive_remote_tmem(first_block(smem_u32(&sc_full[set])));
          }
          set ^= 1;
          if (set == 0) sp ^= 1u;
          load(w[b], x[b]);
        }
      }
      for (int n = 0; n < 2 && ok; ++n) {        // the first block's last arrivals here
        ok = wait(&sc_empty[set], sp);
        set ^= 1;
        if (set == 0) sp ^= 1u;
      }
    }
  } else {
    regs_up<112>();
    // ------------------------------------------------------------ results
    const int q = warp & 3, g = (warp - 8) >> 2;
    const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
    int turn = 0;
    uint32_t ap = 0;
    bool odd = false;
    // a warp whose wait gives up still meets the others at every item's barrier
    for (int i = blockIdx.x / 2; i < total; i += pairs) {
      const Tile8 t = item(i);
      const int cw = (t.n + 8 * kLongGroups - 1) / (8 * kLongGroups);   // groups of eight columns of each warp of this tile
      const int col0 = 8 * g * cw;
      float2 acc[C8][4];
#pragma unroll
      for (int c = 0; c < C8; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[c][j] = make_float2(0.f, 0.f);
      for (int kb = 0, sg = 0; kb < nkb && ok; kb = nkb * ++sg / segs) {   // (kb: a sum's first block)
        ok = wait(&acc_full[turn], ap);
        if (!ok) break;
        tc_fence_after();
        // (what is loaded beyond the tile's columns stays within the place, and is not used)
#pragma unroll
        for (int c = 0; c < C8; c += CH) {
          if (c >= cw) continue;
          uint32_t v[2][4 * CH];
          tmem_ld32<CH>(tq + turn * kLongRows + col0 + 8 * c, v);
          tmem_wait<CH>(v);
#pragma unroll
          for (int h = 0; h < CH; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              add2(acc[c + h][j], pair(v[j >> 1][4 * h + 2 * (j & 1)], v[j >> 1][4 * h + 2 * (j & 1) + 1]));
        }
        tc_fence_before();                       // read: the place may take the next sum
        __syncwarp();
        if (lane == 0) {
          if (part == 0) mbar_arrive(&acc_empty[turn]);
          else arrive_remote_tmem(first_block(smem_u32(&acc_empty[turn])));
        }
        turn ^= 1;
        if (turn == 0) ap ^= 1u;
      }
#pragma unroll
      for (int c = 0; c < C8; c += CF) {
        finish<CF, kGelu, true>(reinterpret_cast<float2 (&)[CF][4]>(acc[c]), t, a, min(max(cw - c, 0), CF), col0 + 8 * c, q, g,
                                lane, reinterpret_cast<uint32_t*>(sm + L.amax_off) + (odd ? kLongRows * 4 : 0),
                                reinterpret_cast<float*>(sm + L.inv_off) + (warp - 8) * (8 * C8), ok);
      }
      odd = !odd;
    }
  }
  // ------------------------------------------------------------ end
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*abort_flag) {
    // what is still in flight lands before its memory is released (bounded)
    if (part == 0 && warp == 0 && lane == 0)
      for (int st = 0; st < a.na; ++st)
        if (issued >> st & 1u) mbar_drain(&full[st], issued_par >> st & 1u);
    if (part == 0 && warp == 1) {
      if (elect_one()) commit_pair(spare);       // (the lane that issued the products)
      __syncwarp();
      if (lane == 0) mbar_drain(spare, 0);
    }
    // The other block's loads, which this one may not have expected: microseconds each, the last of them asked for before
    // the wait of kDefaultWaitNs that gave up; a pause all the same.
    if (threadIdx.x == 64) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 1000000ull) {}
    }
  }
  __syncwarp();
  cluster_meet();                                // both are done: no arrival or load is on its way to either
  if (warp == 1) tmem_dealloc_pair(tmem);
  cluster_meet();
}

// Ring lengths: as many runs of rows as fit beside as many weight tiles (at most kMaxStages), the rest for weight tiles.
bool fp8_rings(int nmax, int E, int split, int smem, int* na, int* nb) {
  const int fixed = (int)fp8_smem(nmax, 0, 0, E, split).total, row_bytes = nmax * 128;
  *nb = std::min(kMaxStages, (smem - fixed) / (kABytes + row_bytes));
  *na = std::min(kMaxStages, (smem - fixed - *nb * row_bytes) / kABytes);
  return *nb >= 2;
}

template <typename Kern>
cudaError_t launch_cluster(Kern kern, int blocks, int sms, int threads, size_t bytes, cudaStream_t s, const CUtensorMap& A,
                           const RowMaps& B, const Fp8Args& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms / blocks * blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, A, B, a);
  if (err == cudaSuccess) launch_counter().fetch_add(1, std::memory_order_relaxed);
  return err;
}

template <int C8, bool G, bool Z>
cudaError_t launch_one(const CUtensorMap& A, const RowMaps& B, Fp8Args a, int sms, int smem, cudaStream_t s) {
  auto kern = fp8_gemm_kernel<C8, G, Z>;
  MOE_LAUNCH(ensure_smem_attr(reinterpret_cast<const void*>(kern)));
  if (!fp8_rings(16 * C8, a.E, a.split, smem, &a.na, &a.nb)) return cudaErrorInvalidValue;
  a.nslots = std::min(kMaxSlots, 512 / (16 * C8));
  const size_t bytes = std::max<size_t>(fp8_smem(16 * C8, a.na, a.nb, a.E, a.split).total, kMinSmem);
  if (!Z) return launch_k(kern, sms, kThreads, bytes, s, true, A, B, a);
  return launch_cluster(kern, a.split, sms, kThreads, bytes, s, A, B, a);
}

// Where a short batch's items leave more than half of the SMs idle, clusters of two, four or eight blocks share them
// (with four blocks of inputs each at least).
template <int C8, bool G>
cudaError_t launch_short(const CUtensorMap& A, const RowMaps& B, Fp8Args a, int sms, int smem, cudaStream_t s) {
  const long long items = (long long)(std::min(a.E, a.S_max) + a.S_max / (16 * C8)) * (a.M / 128);   // at most
  while (a.split < 8 && items * 2 * a.split <= sms && a.K / 128 >= 8 * a.split) a.split *= 2;
  if (a.split > 1) return launch_one<C8, G, true>(A, B, a, sms, smem, s);
  return launch_one<C8, G, false>(A, B, a, sms, smem, s);
}

template <bool G>
cudaError_t launch_gemm(int c8, const CUtensorMap& A, const RowMaps& B, const Fp8Args& a, int sms, int smem,
                        cudaStream_t s) {
  switch (c8) {
    case 2: return launch_short<2, G>(A, B, a, sms, smem, s);
    case 4: return launch_one<4, G, false>(A, B, a, sms, smem, s);
    case 8: return launch_one<8, G, false>(A, B, a, sms, smem, s);
    case 10: return launch_one<10, G, false>(A, B, a, sms, smem, s);
    case 12: return launch_one<12, G, false>(A, B, a, sms, smem, s);
  }
  return cudaErrorInvalidValue;
}

template <bool G>
cudaError_t launch_long(const CUtensorMap& A, const RowMaps& B, Fp8Args a, int sms, int smem, cudaStream_t s) {
  auto kern = fp8_long_kernel<G>;
  MOE_LAUNCH(ensure_smem_attr(reinterpret_cast<const void*>(kern)));
  a.na = std::min(kMaxStages, (smem - (int)long_smem(0, a.E).total) / (int)kLongStage);
  if (a.na < 2) return cudaErrorInvalidValue;
  return launch_cluster(kern, 2, sms, kLongThreads, std::max<size_t>(long_smem(a.na, a.E).total, kMinSmem), s, A, B, a);
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct Fp8Ws {
  size_t bad, x, sx, h, sh, ex, eh, total;     // ex, eh: exponents of the scales
  int Sp;
};
Fp8Ws fp8_ws(int d, int f, int E, int S_max) {
  Fp8Ws w;
  const size_t S = std::max(S_max, 1);
  w.Sp = scale_row((int)S, E);
  w.bad = 256;                                  // behind the status word
  w.x = w.bad + kMaxRowBlocks * 4;
  w.sx = w.x + up256(S * d);
  w.h = w.sx + up256((size_t)w.Sp * (d / 128) * 4);
  w.sh = w.h + up256(S * f);
  w.ex = w.sh + up256((size_t)w.Sp * (f / 128) * 4);
  w.eh = w.ex + up256((size_t)w.Sp * ((d + 511) / 512) * 4);
  w.total = w.eh + up256((size_t)w.Sp * ((f + 511) / 512) * 4);
  return w;
}

}  // namespace

size_t fp8_ffn_bytes(int d, int f, int E, int S_max) { return fp8_ws(d, f, E, S_max).total; }

cudaError_t launch_fp8_weights(const void* W, bool f16, int E, int K, int N, uint8_t* Wq, float* scales,
                               cudaStream_t s) {
  const unsigned grid = (unsigned)((long long)E * (K / 128) * (N / 128));
  if (f16)
    return launch_k(fp8_weights_kernel<__half>, grid, 256, 0, s, false, static_cast<const __half*>(W), K, N, Wq, scales);
  return launch_k(fp8_weights_kernel<float>, grid, 256, 0, s, false, static_cast<const float*>(W), K, N, Wq, scales);
}

cudaError_t launch_fp8_ffn(const void* tokens, const int32_t* perm, const int32_t* offsets, const uint8_t* W1q,
                           const float* W1s, const uint8_t* W2q, const float* W2s, int T, int d, int f, int E,
                           int S_max, void* out, uint8_t* ws, cudaStream_t s) {
  int dev = 0, sms = 0, smem = 0;
  MOE_LAUNCH(cudaGetDevice(&dev));
  MOE_LAUNCH(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  MOE_LAUNCH(cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev));
  const Fp8Ws w = fp8_ws(d, f, E, S_max);
  int* status = reinterpret_cast<int*>(ws);
  int* general = status + 1;
  uint8_t *x = ws + w.x, *h = ws + w.h;
  float *sx = reinterpret_cast<float*>(ws + w.sx), *sh = reinterpret_cast<float*>(ws + w.sh);
  // Rows per tile.  Slots that are no multiple of the tokens come from a capacity, S_max / E for each expert; otherwise
  // those of an expert that is two standard deviations fuller than the average one.  us of both products: 160 slots
  // each, 128 experts of the 2.4B layer: tiles of 160 rows (three sums in TMEM) 2514, of 192 (two sums) 2810; 160 on
  // average, 64 experts of half that width: 911 and 772, since half of the experts take two tiles of 160; 256 on
  // average: 683, 723, of 256 rows 737; 512: 492, 504, 523; 1024: 247, 247, 268.  20 on average: tiles of 32 rows
  // 534, 64 517, 128 552; 40: 884, 529, 576.
  const double mean = (double)S_max / E;
  const int rows = (int)std::min<double>(S_max, S_max % T && S_max % E == 0 ? mean : mean + 2.0 * std::sqrt(mean) + 1.0);
  const int c8 = rows <= 32 ? 2 : rows <= 64 ? 4 : rows <= 128 ? 8 : rows <= 160 || rows > 192 ? 10 : 12;
  // Long runs (from 65 slots on) with enough to do: the form for scales that are powers of two, where the rows' kernel finds no
  // other scale, else the one for any; the one that does not run takes 3 us of each product.  us without and with it, S d f
  // in 10^9: 64 experts of 512 rows, 2048 x 2048 (137): 483, 295; 128 of 160, 3584 x 14336 (1050): 2840, 2270; 64 of 70,
  // 2048 x 2048 (19): 130, 125 to 130; 1 of 4096, 1024 x 4096 (17): 78, 58; 8 of 128, 4096 x 4096 (17): 79, 81.  About the border
  // (8.6): 1 of 2048, 2048 x 2048: 49, 41; 32 of 256, 1024 x 1024: 62, 62; 16 of 128, 2048 x 2048: 52, 56.  Below it: 16 of 256,
  // 1024 x 1024 (4.3): 35, 41; 8 of 128 and 1 of 1024, 2048 x 2048 (4.3): 31, 37 both; 4 of 128, 2048 x 2048 (2.1): 29, 35;
  // 8 of 128, 1024 x 1024 (1.1): 23, 32; 4 of 256, 256 x 256 (0.07): 17, 27.
  const bool long_form = c8 >= 8 && d % 256 == 0 && f % 256 == 0 && (double)S_max * d * f >= 8e9;
  const int parts = (d / 128 + kRowPart - 1) / kRowPart;
  const dim3 rows_grid((unsigned)std::max(1, std::min((S_max + 7) / 8, std::min(6 * sms, kMaxRowBlocks) / parts)), (unsigned)parts);
  int* bad_rows = reinterpret_cast<int*>(ws + w.bad);
  if (long_form) MOE_LAUNCH(cudaMemsetAsync(general, 0, sizeof(int), s));
  MOE_LAUNCH(launch_k(fp8_rows_kernel, rows_grid, 256,
                      (E + 1) * sizeof(int32_t), s,
                      false, static_cast<const __half*>(tokens), perm, offsets, E, S_max, T, d, w.Sp, x, sx, status,
                      W1s, W2s, (long long)E * (d / 128) * (f / 128),
                      long_form ? reinterpret_cast<uint32_t*>(ws + w.ex) : nullptr, bad_rows, long_form ? general : nullptr));
  CUtensorMap A1, A2;
  RowMaps B1, B2;
  bool maps = encode_weight_map(&A1, W1q, d, (uint64_t)E * f) && encode_weight_map(&A2, W2q, f, (uint64_t)E * d);
  for (int i = 0; i < 3; ++i)
    maps = maps && encode_u8_map(&B1.box[i], x, d, S_max, 128, 128 >> i) && encode_u8_map(&B2.box[i], h, f, S_max, 128, 128 >> i);
  RowMaps L1, L2;
  for (int i = 0; i < 5 && long_form; ++i)
    maps = maps && encode_u8_map(&L1.box[i], x, d, S_max, 128, kLongBox * (i + 1)) &&
           encode_u8_map(&L2.box[i], h, f, S_max, 128, kLongBox * (i + 1));
  if (!maps)
    return cudaErrorInvalidValue;
  Fp8Args g;
  memset(&g, 0, sizeof(g));
  g.offsets = offsets;
  g.E = E;
  g.S_max = S_max;
  g.Sp = w.Sp;
  g.status = status;
  g.split = 1;
  g.bad_rows = bad_rows;
  g.row_blocks = (int)(rows_grid.x * rows_grid.y);
  g.wscale = W1s;
  g.xscale = sx;
  g.K = d;
  g.M = f;
  g.h = h;
  g.hscale = sh;
  g.general = long_form ? general : nullptr;
  g.xexp = reinterpret_cast<const uint32_t*>(ws + w.ex);
  g.hexp = ws + w.eh;
  if (long_form) MOE_LAUNCH(launch_long<true>(A1, L1, g, sms, smem, s));
  MOE_LAUNCH(launch_gemm<true>(c8, A1, B1, g, sms, smem, s));
  g.wscale = W2s;
  g.xscale = sh;
  g.xexp = reinterpret_cast<const uint32_t*>(ws + w.eh);
  g.K = f;
  g.M = d;
  g.out = static_cast<__half*>(out);
  if (long_form) MOE_LAUNCH(launch_long<false>(A2, L2, g, sms, smem, s));
  return launch_gemm<false>(c8, A2, B2, g, sms, smem, s);
}

}  // namespace moe
