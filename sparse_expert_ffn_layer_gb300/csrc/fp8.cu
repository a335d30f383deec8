// Experts in 8-bit floating point (e4m3) with a scale for each block of 128: the weights' and the rows'
// quantisers, and the grouped products on the 5th-generation tensor cores (kind::f8f6f4, TMEM, TMA).
//
//   y[s, j] = sum_b sx[s, b] sw[j / 128, b] sum_{i in b} x8[s, i] w8[j, i]          (b: blocks of 128 inputs)
//
// Scales that this library makes are powers of two, so that bringing a value to 8 bits is one rounding: the
// quotient is exact, and the same in any precision.  The products take any 32-bit scales.
//
// Products: as in the f16 form a weight tile is the MMA's M = 128 operand and a run of one expert's slots its N
// operand, both with their inputs side by side (K-major).  A stage of the pipeline is one block of 128 inputs:
// four MMAs whose sum goes to a TMEM slot, from where 16 warps add it, times its scale, to the running sums in
// their registers (column n of a tile has one scale, a weight tile has one for all its rows).  So the sums over
// blocks are in 32 bits with every scale applied before them, and a slot is free again as soon as it was read.
#include <algorithm>
#include <cstring>

#include "launch.h"

namespace moe {
namespace {

// ---------------------------------------------------------------- values
// Exponent p of the smallest power of two with amax <= 448 2^p: 448 = 1.75 x 2^8.
__device__ __forceinline__ int fp8_exp(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 127;
  return max(-126, e - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0));
}
// The scale and its inverse; zero: 1; infinity or NaN: NaN.
__device__ __forceinline__ void fp8_scale(uint32_t amax_bits, float& scale, float& inv) {
  if (amax_bits >= 0x7f800000u) {
    scale = inv = __uint_as_float(0x7fc00000u);
  } else if (amax_bits == 0u) {
    scale = inv = 1.f;
  } else {
    const int p = fp8_exp(amax_bits);
    scale = __uint_as_float((uint32_t)(127 + p) << 23);
    inv = __uint_as_float((uint32_t)(127 - p) << 23);
  }
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
__device__ __forceinline__ void load8(const __half* p, float (&f)[8]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
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

// ---------------------------------------------------------------- rows
// Slot s of an expert: its token's row in 8 bits, by 16 lanes a block of 128 columns.  sx is [d / 128][Sp].
__global__ void __launch_bounds__(256) fp8_rows_kernel(const __half* __restrict__ tokens, const int32_t* __restrict__ perm,
                                                       const int32_t* __restrict__ offsets, int E, int S_max, int T, int d,
                                                       int Sp, uint8_t* __restrict__ Xq, float* __restrict__ sx,
                                                       int* status) {
  pdl_wait();
  pdl_trigger();
  const int S = min(max(offsets[E], 0), S_max);
  const int nb = d / 128, l = threadIdx.x & 15;
  const long long total = (long long)S * nb, step = (long long)gridDim.x * 16;
  bool bad = false;
  for (long long u = (long long)blockIdx.x * 16 + (threadIdx.x >> 4); __any_sync(0xffffffffu, u < total); u += step) {
    const bool on = u < total;
    const int s = on ? (int)(u / nb) : 0, b = on ? (int)(u - (long long)s * nb) : 0;
    const int t = on ? perm[s] : 0;
    const bool in = (unsigned)t < (unsigned)T;
    bad |= !in;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.f;
    if (on && in) load8(tokens + (long long)t * d + b * 128 + l * 8, f);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, magnitude_bits(f[j]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    float scale, inv;
    fp8_scale(m, scale, inv);
    if (on) {
      const uint2 r = make_uint2(fp8_four(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                                 fp8_four(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
      *reinterpret_cast<uint2*>(Xq + (long long)s * d + b * 128 + l * 8) = r;
      if (l == 0) sx[(long long)b * Sp + s] = scale;
    }
  }
  if (bad) record_status(status, kErrBounds);
}

// ---------------------------------------------------------------- products
constexpr int kEpiWarps = 16;                 // four column groups of the four TMEM lane quarters
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kABytes = 128 * 128;            // a weight tile: 128 outputs, 128 inputs
constexpr int kScaleSlots = 8;
constexpr int kMaxSlots = 16;
constexpr int kMaxStages = 16;
constexpr size_t kMinSmem = 116 * 1024;       // one block per SM: each takes all of TMEM

struct Fp8Smem {
  uint32_t stage_bytes, b_off, scale_off, scale_bytes, amax_off, bars_off, misc_off, total;
};
__host__ __device__ inline Fp8Smem fp8_smem(int nmax, int mw, int stages, int E) {
  Fp8Smem L;
  L.b_off = (uint32_t)mw * kABytes;
  L.stage_bytes = L.b_off + (uint32_t)nmax * 128u;
  uint32_t off = (uint32_t)stages * L.stage_bytes;
  L.scale_off = off;
  L.scale_bytes = (uint32_t)(nmax + 4) * 4u;
  off += kScaleSlots * L.scale_bytes;
  L.amax_off = off;
  off += 2u * (uint32_t)(mw * nmax) * 16u;    // two items' [column][lane quarter]
  L.bars_off = off;
  off += (2u * kMaxStages + 2u * kMaxSlots + 2u * kScaleSlots + 1u) * 8u;
  L.misc_off = off;
  off += 16u + 8u * (uint32_t)(E + 1);
  L.total = off + 1024u;                      // slack for the alignment of the stages
  return L;
}

struct Fp8Args {
  const int32_t* offsets;
  const float* wscale;         // [E][M / 128][K / 128]
  const float* xscale;         // [K / 128][Sp]
  int E, S_max, Sp, K, M, stages, nslots;
  uint8_t* h;                  // first product: [S_max][M], with hscale [M / 128][Sp]
  float* hscale;
  __half* out;                 // second: [S_max][M]
  int* status;
};

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 lanes x 8 columns; the values are valid after tmem_wait.
__device__ __forceinline__ void tmem_ld8(uint32_t t, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(t));
}
template <int B>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[B][8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int b = 0; b < B; ++b)
#pragma unroll
    for (int i = 0; i < 8; ++i) asm volatile("" : "+r"(r[b][i]));   // no use of them moves above the wait
}
// Untiled copy to shared memory: addresses and size are multiples of 16 bytes.
__device__ __forceinline__ void bulk_load(void* smem, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(smem)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

struct Tile8 {
  int e, row0, n, mt;
};
// Item i: an expert, MW neighbouring weight tiles and a run of its rows; the runs of one weight tile are next to
// each other, on different SMs at the same time, and share it in L2.
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
  t.n = min(per, rows - c * per);
  return t;
}

// C8: groups of eight columns per warp (a tile has up to 32 C8 rows); MW: weight tiles per item, all multiplied
// with one load of the rows.  kGelu: first product.
template <int C8, int MW, bool kGelu>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const Fp8Args a) {
  constexpr int NMAX = 32 * C8, COLS = 8 * C8;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const Fp8Smem L = fp8_smem(NMAX, MW, a.stages, a.E);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L.bars_off);
  uint64_t *empty = full + kMaxStages, *acc_full = empty + kMaxStages, *acc_empty = acc_full + kMaxSlots,
           *sc_full = acc_empty + kMaxSlots, *sc_empty = sc_full + kScaleSlots, *spare = sc_empty + kScaleSlots;
  uint32_t* holder = reinterpret_cast<uint32_t*>(sm + L.misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L.misc_off + 4);
  int32_t* prefix = reinterpret_cast<int32_t*>(sm + L.misc_off + 16);
  int32_t* offs = prefix + a.E + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < a.nslots; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], kEpiWarps);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      mbar_init(&sc_full[s], 1);
      mbar_init(&sc_empty[s], kEpiWarps);
    }
    mbar_init(spare, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) tmem_alloc(holder, 512);
  pdl_wait();
  pdl_trigger();
  if (warp == 2) {
    // boundaries: the largest so far, clamped to [0, S_max], so that runs never overlap or leave the buffers
    bool bad = false;
    int run = 0, tiles = 0;
    for (int e0 = 0; e0 <= a.E; e0 += 32) {
      const int e = e0 + lane;
      const int o = e <= a.E ? __ldcg(a.offsets + e) : 0;
      int v = min(max(o, 0), a.S_max);
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const int q = __shfl_up_sync(0xffffffffu, v, k);
        if (lane >= k) v = max(v, q);
      }
      v = max(v, run);
      bad |= e <= a.E && v != o;
      if (e <= a.E) offs[e] = v;
      int before = __shfl_up_sync(0xffffffffu, v, 1);
      if (lane == 0) before = run;
      run = __shfl_sync(0xffffffffu, v, 31);
      // tiles of the experts before e
      int c = e >= 1 && e <= a.E ? (v - before + NMAX - 1) / NMAX : 0;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const int q = __shfl_up_sync(0xffffffffu, c, k);
        if (lane >= k) c += q;
      }
      if (e <= a.E) prefix[e] = tiles + c;
      tiles += __shfl_sync(0xffffffffu, c, 31);
    }
    if (bad) record_status(a.status, kErrBounds);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;
  const int mt = a.M / (128 * MW), nkb = a.K / 128;
  const int total = prefix[a.E] * mt;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_try_wait(bar, parity) || mbar_wait_bounded(bar, parity, abort_flag, a.status, kDefaultWaitNs);
  };
  uint32_t issued = 0, issued_par = 0, sc_issued = 0, sc_par = 0;   // loads in flight, for the end
  if (warp == 0) {
    // ------------------------------------------------------------ loads
    int st = 0, ss = 0;
    uint32_t sp = 1, scp = 1;
    bool ok = true;
    for (int i = blockIdx.x; i < total && ok; i += gridDim.x) {
      const Tile8 t = tile_at(i, prefix, offs, a.E, mt, NMAX);
      const int npad = max(16, (t.n + 15) & ~15);
      const int arow = t.e * a.M + t.mt * MW * 128;
      const int r0 = t.row0 & ~3;
      const uint32_t sc_bytes = (uint32_t)((t.row0 + t.n - r0 + 3) & ~3) * 4u;
      for (int kb = 0; kb < nkb; ++kb) {
        if (lane == 0) ok = wait(&empty[st], sp) && wait(&sc_empty[ss], scp);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        uint8_t* stage = sm + (size_t)st * L.stage_bytes;
        if (lane == 0) {
          mbar_expect_tx(&full[st], MW * kABytes + (uint32_t)npad * 128u);
#pragma unroll
          for (int h = 0; h < MW; ++h)
            tma_load_2d(stage + h * kABytes, &tmA, kb * 128, arow + h * 128, &full[st]);
          mbar_expect_tx(&sc_full[ss], sc_bytes);
          bulk_load(sm + L.scale_off + ss * L.scale_bytes, a.xscale + (size_t)kb * a.Sp + r0, sc_bytes, &sc_full[ss]);
        }
        __syncwarp();
        for (int b = lane; b < npad / 16; b += 32)
          tma_load_2d(stage + L.b_off + b * 2048, &tmB, kb * 128, t.row0 + 16 * b, &full[st]);
        issued |= 1u << st;
        issued_par = (issued_par & ~(1u << st)) | (sp ^ 1u) << st;
        sc_issued |= 1u << ss;
        sc_par = (sc_par & ~(1u << ss)) | (scp ^ 1u) << ss;
        if (++st == a.stages) {
          st = 0;
          sp ^= 1u;
        }
        if (++ss == kScaleSlots) {
          ss = 0;
          scp ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    if (lane == 0) {
      int st = 0, slot = 0;
      uint32_t sp = 0, ap = 1;
      bool ok = true;
      for (int i = blockIdx.x; i < total && ok; i += gridDim.x) {
        const Tile8 t = tile_at(i, prefix, offs, a.E, mt, NMAX);
        const uint32_t idesc = idesc_f16(128, max(16, (t.n + 15) & ~15), 0, 0);   // (e4m3 has f16's code 0)
        for (int kb = 0; kb < nkb && ok; ++kb) {
          ok = wait(&full[st], sp);
          const uint32_t s0 = smem_u32(sm + (size_t)st * L.stage_bytes);
          const uint64_t bd = smem_desc(s0 + L.b_off, 16, 1024, 2);
#pragma unroll
          for (int h = 0; h < MW; ++h) {
            if (ok) ok = wait(&acc_empty[slot], ap);
            if (!ok) break;
            tc_fence_after();
            const uint64_t ad = smem_desc(s0 + h * kABytes, 16, 1024, 2);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f8(tmem + slot * NMAX, ad + 2 * k, bd + 2 * k, idesc, k ? 1u : 0u);
            tc_commit(&acc_full[slot]);
            if (++slot == a.nslots) {
              slot = 0;
              ap ^= 1u;
            }
          }
          if (!ok) break;
          tc_commit(&empty[st]);
          if (++st == a.stages) {
            st = 0;
            sp ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ sums
    const int q = warp & 3, g = (warp - 2) >> 2;
    const int m = 32 * q + lane;                 // row of the weight tile
    const uint32_t t0 = tmem + ((uint32_t)(32 * q) << 16) + g * COLS;
    int slot = 0, ss = 0;
    uint32_t ap = 0, scp = 0;
    bool ok = true;
    int turn = 0;
    // a warp whose wait gives up still meets the others at every item's barrier
    for (int i = blockIdx.x; i < total; i += gridDim.x, turn ^= 1) {
      const Tile8 t = tile_at(i, prefix, offs, a.E, mt, NMAX);
      const int shift = t.row0 & 3;
      float acc[MW][C8][8];
#pragma unroll
      for (int h = 0; h < MW; ++h)
#pragma unroll
        for (int c = 0; c < C8; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[h][c][j] = 0.f;
      const float* ws = a.wscale + ((size_t)t.e * (a.M / 128) + t.mt * MW) * nkb;
      float wnext[MW];
#pragma unroll
      for (int h = 0; h < MW; ++h) wnext[h] = __ldg(ws + (size_t)h * nkb);
      for (int kb = 0; kb < nkb && ok; ++kb) {
        float w[MW];
#pragma unroll
        for (int h = 0; h < MW; ++h) {
          w[h] = wnext[h];
          if (kb + 1 < nkb) wnext[h] = __ldg(ws + (size_t)h * nkb + kb + 1);
        }
        ok = __all_sync(0xffffffffu, wait(&sc_full[ss], scp));
        if (!ok) break;
        const float* sc = reinterpret_cast<const float*>(sm + L.scale_off + ss * L.scale_bytes) + shift + g * COLS;
#pragma unroll
        for (int h = 0; h < MW; ++h) {
          if (ok) ok = __all_sync(0xffffffffu, wait(&acc_full[slot], ap));
          if (!ok) break;
          tc_fence_after();
          constexpr int B = C8 % 2 ? 1 : 2;      // loads in flight
#pragma unroll
          for (int c = 0; c < C8; c += B) {
            uint32_t v[B][8];
#pragma unroll
            for (int b = 0; b < B; ++b) tmem_ld8(t0 + slot * NMAX + (c + b) * 8, v[b]);
            tmem_wait<B>(v);
            if (c + B >= C8) {                   // read: the slot may take the next sum
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&acc_empty[slot]);
            }
#pragma unroll
            for (int b = 0; b < B; ++b)
#pragma unroll
              for (int j = 0; j < 8; ++j)
                acc[h][c + b][j] = fmaf(__uint_as_float(v[b][j]), w[h] * sc[(c + b) * 8 + j], acc[h][c + b][j]);
          }
          if (++slot == a.nslots) {
            slot = 0;
            ap ^= 1u;
          }
        }
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&sc_empty[ss]);
        if (++ss == kScaleSlots) {
          ss = 0;
          scp ^= 1u;
        }
      }
      const int col0 = g * COLS;
      if constexpr (kGelu) {
        // GeLU, the largest magnitude of each slot's 128 columns (four warps), and 8 bits
        uint32_t* am = reinterpret_cast<uint32_t*>(sm + L.amax_off) + turn * (MW * NMAX * 4);
#pragma unroll
        for (int h = 0; h < MW; ++h)
#pragma unroll
          for (int c = 0; c < C8; ++c) {
            uint32_t keep = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              acc[h][c][j] = gelu_tanh(acc[h][c][j]);
              const uint32_t r = __reduce_max_sync(0xffffffffu, magnitude_bits(acc[h][c][j]));
              if (lane == j) keep = r;
            }
            if (lane < 8) am[(h * NMAX + col0 + c * 8 + lane) * 4 + q] = keep;
          }
        asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory");
        if (!ok) continue;
#pragma unroll
        for (int h = 0; h < MW; ++h) {
          const int mb = t.mt * MW + h;
#pragma unroll
          for (int c = 0; c < C8; ++c) {
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
              uint32_t u = 0;                    // this lane's values of four slots
#pragma unroll
              for (int k = 0; k < 4; k += 2) {
                float inv[2], scale[2];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                  const int col = col0 + c * 8 + j + k + p;
                  const uint4 r = *reinterpret_cast<const uint4*>(am + (h * NMAX + col) * 4);
                  fp8_scale(max(max(r.x, r.y), max(r.z, r.w)), scale[p], inv[p]);
                  if (m == 0 && col < t.n) a.hscale[(size_t)mb * a.Sp + t.row0 + col] = scale[p];
                }
                u |= fp8_pair(acc[h][c][j + k] * inv[0], acc[h][c][j + k + 1] * inv[1]) << (8 * k);
              }
              // four lanes trade bytes: lane 4 i + r gets slot r's values of columns 4 i .. 4 i + 3
              uint32_t o = __shfl_xor_sync(0xffffffffu, u, 1);
              u = (lane & 1) ? __byte_perm(u, o, 0x3715) : __byte_perm(u, o, 0x6240);
              o = __shfl_xor_sync(0xffffffffu, u, 2);
              u = (lane & 2) ? __byte_perm(u, o, 0x3276) : __byte_perm(u, o, 0x5410);
              const int col = col0 + c * 8 + j + (lane & 3);
              if (col < t.n)
                *reinterpret_cast<uint32_t*>(a.h + (size_t)(t.row0 + col) * a.M + mb * 128 + (m & ~3)) = u;
            }
          }
        }
      } else {
        if (!ok) continue;
        // two columns per 4-byte store: lanes 2 i and 2 i + 1 hold columns m and m + 1; for a pair of slots
        // the even lane stores the first, the odd lane the second
        const bool odd = lane & 1;
#pragma unroll
        for (int h = 0; h < MW; ++h)
#pragma unroll
          for (int c = 0; c < C8; ++c)
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              const float v0 = acc[h][c][j], v1 = acc[h][c][j + 1];
              const float recv = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
              const int col = col0 + c * 8 + j + (odd ? 1 : 0);
              if (col < t.n)
                *reinterpret_cast<__half2*>(a.out + (size_t)(t.row0 + col) * a.M + ((t.mt * MW + h) * 128 + (m & ~1))) =
                    odd ? __floats2half2_rn(recv, v1) : __floats2half2_rn(v0, recv);
            }
      }
    }
  }
  // ------------------------------------------------------------ end
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*abort_flag && lane == 0) {
    // what is still in flight lands before its memory is released (bounded)
    if (warp == 0) {
      for (int s = 0; s < a.stages; ++s)
        if (issued >> s & 1u) mbar_drain(&full[s], issued_par >> s & 1u);
      for (int s = 0; s < kScaleSlots; ++s)
        if (sc_issued >> s & 1u) mbar_drain(&sc_full[s], sc_par >> s & 1u);
    }
    if (warp == 1) {
      tc_commit(spare);
      mbar_drain(spare, 0);
    }
  }
  __syncwarp();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

int fp8_stages(int nmax, int mw, int E, int smem) {
  for (int st = kMaxStages; st >= 2; --st)
    if ((int)fp8_smem(nmax, mw, st, E).total <= smem) return st;
  return 0;
}

template <int C8, int MW, bool G>
cudaError_t launch_one(const CUtensorMap& A, const CUtensorMap& B, Fp8Args a, int sms, int smem, cudaStream_t s) {
  auto kern = fp8_gemm_kernel<C8, MW, G>;
  MOE_LAUNCH(ensure_smem_attr(reinterpret_cast<const void*>(kern)));
  a.stages = fp8_stages(32 * C8, MW, a.E, smem);
  if (a.stages < 2) return cudaErrorInvalidValue;
  a.nslots = std::min(kMaxSlots, 512 / (32 * C8));
  const size_t bytes = std::max<size_t>(fp8_smem(32 * C8, MW, a.stages, a.E).total, kMinSmem);
  return launch_k(kern, sms, kThreads, bytes, s, true, A, B, a);
}

template <bool G>
cudaError_t launch_gemm(int c8, const CUtensorMap& A, const CUtensorMap& B, const Fp8Args& a, int sms, int smem,
                        cudaStream_t s) {
  switch (c8) {
    case 1: return launch_one<1, 1, G>(A, B, a, sms, smem, s);
    case 2: return launch_one<2, 1, G>(A, B, a, sms, smem, s);
    case 4: return launch_one<4, 1, G>(A, B, a, sms, smem, s);
    case 5: return launch_one<5, 1, G>(A, B, a, sms, smem, s);
    case 6: return launch_one<6, 1, G>(A, B, a, sms, smem, s);
    case 8: return launch_one<8, 1, G>(A, B, a, sms, smem, s);
  }
  return cudaErrorInvalidValue;
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct Fp8Ws {
  size_t x, sx, h, sh, total;
  int Sp;
};
Fp8Ws fp8_ws(int d, int f, int S_max) {
  Fp8Ws w;
  const size_t S = std::max(S_max, 1);
  w.Sp = (int)((S + 3) / 4 * 4);
  w.x = 256;                                    // the status word
  w.sx = w.x + up256(S * d);
  w.h = w.sx + up256((size_t)w.Sp * (d / 128) * 4);
  w.sh = w.h + up256(S * f);
  w.total = w.sh + up256((size_t)w.Sp * (f / 128) * 4);
  return w;
}

}  // namespace

size_t fp8_ffn_bytes(int d, int f, int S_max) { return fp8_ws(d, f, S_max).total; }

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
  const Fp8Ws w = fp8_ws(d, f, S_max);
  int* status = reinterpret_cast<int*>(ws);
  MOE_LAUNCH(cudaMemsetAsync(status, 0, sizeof(int), s));
  uint8_t *x = ws + w.x, *h = ws + w.h;
  float *sx = reinterpret_cast<float*>(ws + w.sx), *sh = reinterpret_cast<float*>(ws + w.sh);
  const long long units = (long long)S_max * (d / 128);
  MOE_LAUNCH(launch_k(fp8_rows_kernel, (unsigned)std::min<long long>((units + 15) / 16, 8LL * sms), 256, 0, s, false,
                      static_cast<const __half*>(tokens), perm, offsets, E, S_max, T, d, w.Sp, x, sx, status));
  // rows per tile: those of an expert that is somewhat fuller than the average one
  const int rows = (int)std::min<long long>(S_max, (long long)S_max * 5 / (4LL * E) + 8);
  const int c8 = rows <= 32 ? 1 : rows <= 64 ? 2 : rows <= 128 ? 4 : rows <= 160 ? 5 : rows <= 192 ? 6 : 8;
  CUtensorMap A1, A2, B1, B2;
  if (!encode_u8_map(&A1, W1q, d, (uint64_t)E * f, 128, 128) || !encode_u8_map(&A2, W2q, f, (uint64_t)E * d, 128, 128) ||
      !encode_u8_map(&B1, x, d, S_max, 128, 16) || !encode_u8_map(&B2, h, f, S_max, 128, 16))
    return cudaErrorInvalidValue;
  Fp8Args g;
  memset(&g, 0, sizeof(g));
  g.offsets = offsets;
  g.E = E;
  g.S_max = S_max;
  g.Sp = w.Sp;
  g.status = status;
  g.wscale = W1s;
  g.xscale = sx;
  g.K = d;
  g.M = f;
  g.h = h;
  g.hscale = sh;
  MOE_LAUNCH(launch_gemm<true>(c8, A1, B1, g, sms, smem, s));
  g.wscale = W2s;
  g.xscale = sh;
  g.K = f;
  g.M = d;
  g.out = static_cast<__half*>(out);
  return launch_gemm<false>(c8, A2, B2, g, sms, smem, s);
}

}  // namespace moe
