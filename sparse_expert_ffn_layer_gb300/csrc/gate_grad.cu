// The gate's gradient on the 5th-generation tensor cores, for f16 tokens:
//   dWg [d, E] = X^T dL,    dX [T, d] = dX_in + dL Wg^T       (dL = dlogits, Wg: 32-bit)
//
// dL stays good to 2^-23 of itself: a block of 128 rows is scaled by one power of two and split into
// v = hi + 2^-11 lo, both f16 (lo keeps an exponent range of its own, so what is lost is 2^-23 |v| +
// 2^-36 of the block's largest magnitude).  The products with hi and with lo go to separate
// accumulators, joined as D1 + 2^-11 D2 in 32 bits.  X is f16 and exact, so dWg keeps the accuracy of
// a 32-bit sum.  Wg is split in the same way, by 128 of its rows, and D2 takes hi lo and lo hi, so that
// dX is what 32-bit sums give, rounded once (lo lo is below 2^-22 of a product).  The splits come with
// the logits' gradient (router_loss.cu).
//
// One launch computes both, a part of its blocks dWg and the rest dX, one block per SM; warp 0 loads by
// TMA, warp 1 issues the products, eight warps read the accumulators.  Every wait is bounded (common.cuh).
// 16384 x 3584 tokens, 128 experts: 71 us after the split's 12 and before the join's 5.  (Before Wg had a low
// part 64, and as two launches 32 + 44, each with SMs idle at its end: dWg waits at the hand-over of its
// accumulators and leaves DRAM half free, dX streams dX_in and dX.)  4096 x 1024: 24.2 us in all.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "gate_split.cuh"
#include "launch.h"

namespace moe {
namespace {

constexpr int kThreads = 384;             // 4 warps (2 used) + 8 accumulator warps

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, int x, int y, const void* smem) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(m),
      "r"(x), "r"(y), "r"(smem_u32(smem))
      : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// 32 lanes x 32 columns of two accumulators, one wait.
__device__ __forceinline__ void tmem_ld32x2(uint32_t t1, uint32_t t2, float (&u)[32], float (&v)[32]) {
  uint32_t a[32], b[32];
#define MOE_LD32(r, t)                                                                              \
  asm volatile(                                                                                     \
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"                                                      \
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"    \
      "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"                                                    \
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),         \
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),     \
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),  \
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),  \
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])                                          \
      : "r"(t))
  MOE_LD32(a, t1);
  MOE_LD32(b, t2);
#undef MOE_LD32
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    u[j] = __uint_as_float(a[j]);
    v[j] = __uint_as_float(b[j]);
  }
}

// What the roles of a block share.
struct Sync {
  volatile int* abort;
  int* status;
  // Bounded; false once any wait of the block gave up.
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait_bounded(bar, parity, abort, status, kDefaultWaitNs);
  }
};

// What warp 0 has in flight: the last load into each of the barriers whose bits are set, with the parity
// of its phase.
struct InFlight {
  uint32_t issued = 0, parity = 0;
  __device__ __forceinline__ void note(int bar, uint32_t p) {
    issued |= 1u << bar;
    parity = (parity & ~(1u << bar)) | p << bar;
  }
};
// The end of a block, all threads.  After a wait gave up, the loads and products that are still in
// flight land before their memory is released (bounded: 100 ms each).  bars: the barriers that loads
// count on, from InFlight's bit 0 on; spare: one of which nothing has used yet.
__device__ __forceinline__ void end_block(const Sync& sy, const InFlight& fl, uint64_t* bars, uint64_t* spare,
                                          uint32_t tmem) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*sy.abort && lane == 0) {
    if (warp == 0)
      for (int b = 0; b < 32; ++b)
        if (fl.issued >> b & 1u) mbar_drain(&bars[b], fl.parity >> b & 1u);
    if (warp == 1) {
      tc_commit(spare);
      mbar_drain(spare, 0);
    }
  }
  __syncwarp();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- dWg
// A block owns IW x 128 rows i of dWg and 128 columns j, and a run of token rows: chunks of 64 rows
// of X (as the transposed operand) and of the split dL.  The accumulators are emptied into 32-bit
// registers after every 128 rows, where the scale of dL changes (and where the chain of truncating
// additions ends).  The hand-over of an accumulator every 128 rows, not a pipe, bounds it.  IW = 2: the two accumulators share each chunk of dL (64 KB from L2 per 64 KB of
// X; with one the copies from L2 bound it); while the second is emptied the first fills again.
// IW = 1, for batches with too few blocks: two accumulators alternate.
// Rows of masked tokens may hold anything (0 x NaN is NaN): warps 2 and 3 clear them in each chunk of X
// before the products read it (16384 x 3584 x 128, 30% masked, before Wg had a low part: both gradients 85 us,
// 84 without a mask; by the row sums of grad.cu, which copy row by row, 187).
struct WgArgs {
  const float* sT;
  const uint8_t* mask;         // rows that count, or null (all)
  float* dst;                  // [slots][d][E] (one run: dWg itself)
  int T, d, E, Ep, run;        // run: token rows per block, a multiple of 128
  int direct;                  // one run only
  int* status;
};
constexpr int kWgStageBytes = 65536;
constexpr int kWgStages = 3;

template <int IW>
__device__ __forceinline__ void wgrad_block(uint8_t* sm, const CUtensorMap& mX, const CUtensorMap& mL,
                                            const WgArgs& a, int block) {
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kWgStages * kWgStageBytes);
  uint64_t *full = bars, *empty = bars + kWgStages, *clean = bars + 2 * kWgStages, *acc_full = clean + kWgStages,
           *acc_empty = acc_full + 2, *spare = acc_empty + 2;
  uint32_t* holder = reinterpret_cast<uint32_t*>(spare + 1);
  int* flag = reinterpret_cast<int*>(holder + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < kWgStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&clean[s], 2);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&acc_full[h], 1);
      mbar_init(&acc_empty[h], 256);
    }
    mbar_init(spare, 1);
    *flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(holder, 512);
  pdl_trigger();
  pdl_wait();                                       // the split dL
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;
  const Sync sy{flag, a.status};
  const int bi = (a.d + 128 * IW - 1) / (128 * IW), runs = (a.T + a.run - 1) / a.run;
  const int r_at = block / bi % runs;
  const int i0 = block % bi * 128 * IW, r0 = r_at * a.run, r1 = min(a.T, r0 + a.run);
  const int j0 = block / bi / runs * 128;
  const int nb = min(2, (a.Ep - j0) / 64);          // 64-column boxes of dL's hi (and lo)
  const int chunks = (r1 - r0 + 63) / 64;
  InFlight fl;
  if (warp < 4) {
    regs_down<40>();
    if (warp == 0) {
      int stage = 0;
      uint32_t phase = 1;
      for (int c = 0; c < chunks; ++c) {
        bool ok = true;
        if (lane == 0) {
          ok = sy.wait(&empty[stage], phase);
          if (ok) {
            uint8_t* st = sm + stage * kWgStageBytes;
            const int y = r0 + 64 * c;
            mbar_expect_tx(&full[stage], (2 * IW + 2 * nb) * 8192);
            fl.note(stage, phase ^ 1u);
            for (int b = 0; b < 2 * IW; ++b) tma_load_2d(st + b * 8192, &mX, i0 + 64 * b, y, &full[stage]);
            for (int b = 0; b < 2 * nb; ++b)
              tma_load_2d(st + 32768 + b * 8192, &mL, (b < nb ? 0 : a.Ep) + j0 + 64 * (b % nb), y, &full[stage]);
          }
        }
        if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) break;
        if (++stage == kWgStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    } else if (warp == 1) {
      const uint32_t idesc = idesc_f16(128, 128 * nb, 1, 1);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int c = 0; c < chunks && ok; ++c) {
        const int blk = c >> 1;
        if (lane == 0) {
          ok = sy.wait(&full[stage], phase) && (!a.mask || sy.wait(&clean[stage], phase));
          tc_fence_after();
          const uint32_t s0 = smem_u32(sm + stage * kWgStageBytes);
          const uint64_t bd = smem_desc(s0 + 32768, 8192, 1024, 2);
          for (int h = 0; h < IW && ok; ++h) {
            const int buf = IW == 2 ? h : blk & 1, use = IW == 2 ? blk : blk >> 1;
            if (!(c & 1)) {                         // a new block of 128 rows: the accumulator is empty
              ok = sy.wait(&acc_empty[buf], (use & 1) ^ 1u);
              if (!ok) break;
              tc_fence_after();
            }
            const uint64_t ad = smem_desc(s0 + h * 16384, 8192, 1024, 2);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma_f16(tmem + buf * 256, ad + k * 128, bd + k * 128, idesc, ((c & 1) | k) ? 1u : 0u);
            if ((c & 1) || c == chunks - 1) tc_commit(&acc_full[buf]);
          }
          if (ok) tc_commit(&empty[stage]);
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0);
        if (++stage == kWgStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    } else if (a.mask) {                            // warps 2 and 3: half of a chunk's rows each
      int stage = 0;
      uint32_t phase = 0;
      const int box = lane >> 3;                    // of 64 columns; a row of it is 128 bytes
      const int y0 = r0 + 32 * (warp - 2) + lane;   // this lane's row of the first chunk
      bool next = y0 < r1 && !a.mask[y0];
      for (int c = 0; c < chunks; ++c) {
        const uint32_t off = __ballot_sync(0xffffffffu, next);
        const int y = y0 + 64 * (c + 1);
        next = y < r1 && !a.mask[y];
        const bool ok = sy.wait(&full[stage], phase);
        if (!__all_sync(0xffffffffu, ok)) break;
        uint8_t* st = sm + stage * kWgStageBytes + box * 8192 + (warp - 2) * 4096 + (lane & 7) * 16;
        if (off && box < 2 * IW) {
#pragma unroll
          for (int row = 0; row < 32; ++row)
            if (off >> row & 1) *reinterpret_cast<uint4*>(st + row * 128) = make_uint4(0u, 0u, 0u, 0u);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&clean[stage]);
        if (++stage == kWgStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    regs_up<232>();
    const int q = warp & 3, ch = (warp - 4) >> 2;   // TMEM lanes 32 q .., half of the columns
    const int nc = 32 * nb;                         // columns of this warp
    float acc[IW][64];
#pragma unroll
    for (int h = 0; h < IW; ++h)
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[h][j] = 0.f;
    bool ok = true;
    float next = a.sT[r0 / kGateBlock];
    for (int c = 0, blk = 0; c < chunks && ok; c += 2, ++blk) {
      const float s = next, s2 = s / kGateLo;
      if (c + 2 < chunks) next = a.sT[r0 / kGateBlock + blk + 1];
#pragma unroll
      for (int h = 0; h < IW; ++h) {
        if (!ok) break;
        const int buf = IW == 2 ? h : blk & 1, use = IW == 2 ? blk : blk >> 1;
        ok = sy.wait(&acc_full[buf], use & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t t0 = tmem + ((uint32_t)(32 * q) << 16) + buf * 256 + ch * nc;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (b < nb) {
            float u[32], v[32];
            tmem_ld32x2(t0 + 32 * b, t0 + 64 * nb + 32 * b, u, v);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              acc[h][32 * b + j] = fmaf(s, u[j], fmaf(s2, v[j], acc[h][32 * b + j]));
          }
        }
        tc_fence_before();
        mbar_arrive(&acc_empty[buf]);
      }
    }
    // Out through shared memory (the last products have read it), row by row: straight from the
    // registers a lane has a row to itself, 32 lines per store (4096 x 1024 x 127, all launches: 37 us, not 28).
    constexpr int kLd = 132;
    float* tile = reinterpret_cast<float*>(sm);     // [128 IW][kLd]
#pragma unroll
    for (int h = 0; h < IW; ++h)
#pragma unroll
      for (int j = 0; j < 64; j += 4)
        if (j < nc)
          *reinterpret_cast<float4*>(tile + (128 * h + 32 * q + lane) * kLd + ch * nc + j) =
              make_float4(acc[h][j], acc[h][j + 1], acc[h][j + 2], acc[h][j + 3]);
    asm volatile("bar.sync 3, 256;" ::: "memory");
    // runs of partial sums are laid out as row_sum_join_kernel reads them
    const int slot = a.direct ? 0 : 2 * r_at + (r1 == a.T);
    const int cols = min(2 * nc, a.E - j0);
    float* out = a.dst + ((size_t)slot * a.d + i0) * a.E + j0;
#pragma unroll 4
    for (int r = warp - 4; r < min(128 * IW, a.d - i0); r += 8) {
      if (a.E % 4 == 0) {
        if (4 * lane < cols)
          *reinterpret_cast<float4*>(out + (size_t)r * a.E + 4 * lane) =
              *reinterpret_cast<const float4*>(tile + r * kLd + 4 * lane);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (lane + 32 * k < cols) out[(size_t)r * a.E + lane + 32 * k] = tile[r * kLd + lane + 32 * k];
      }
    }
  }
  end_block(sy, fl, full, spare, tmem);
}

// ---------------------------------------------------------------- dX
// A block takes one tile of 128 tokens, keeps its split dL in shared memory (E <= 256) and walks a
// part of d in tiles of 128: the split Wg comes from L2 in chunks of 64 experts, high parts and low, dX_in by TMA
// into the tile that the accumulator warps add to in place and that TMA writes out.  Bound by the
// tiles' loads and stores (dX_in and dX at 5.3 TB/s where dX has the device alone).
struct DxArgs {
  const float *sT, *sW;
  int T, d, E, Ep;
  int parts;                   // column parts per token tile
  int with_in;
  int* status;
};
constexpr int kTile = 16384;                        // 128 rows x 64 columns
template <int NKB>                                  // chunks of 64 experts
struct DxPlan {
  static constexpr int kDxB = NKB <= 2 ? 4 : 2;     // stages of Wg: 64 experts each
  // In/out tiles of 128 x 128: one being added to, one being written, the others loading (with two
  // in all, every tile waited for its load).
  static constexpr int kIo = NKB == 1 ? 4 : NKB == 2 ? 3 : 2;
  static constexpr int kOffB = NKB * 2 * kTile, kOffIo = kOffB + kDxB * kTile;
  static constexpr int kOffBar = kOffIo + kIo * 2 * kTile;
  static constexpr int kBytes = kOffBar + 256 + 1024;
};

template <int NKB>
__device__ __forceinline__ void dx_block(uint8_t* sm, const CUtensorMap& mL, const CUtensorMap& mW,
                                         const CUtensorMap& mIn, const CUtensorMap& mOut, const DxArgs& a,
                                         int block) {
  using PL = DxPlan<NKB>;
  constexpr int IO = PL::kIo, kDxB = PL::kDxB;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + PL::kOffBar);
  uint64_t *a_full = bar, *acc_full = bar + 1, *acc_empty = bar + 3, *b_full = bar + 5,
           *b_empty = b_full + kDxB, *io_full = b_empty + kDxB, *io_empty = io_full + IO, *spare = io_empty + IO;
  uint32_t* holder = reinterpret_cast<uint32_t*>(spare + 1);
  int* flag = reinterpret_cast<int*>(holder + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    mbar_init(a_full, 1);
    for (int s = 0; s < kDxB; ++s) {
      mbar_init(&b_full[s], 1);
      mbar_init(&b_empty[s], 1);
    }
    for (int s = 0; s < IO; ++s) {
      mbar_init(&io_full[s], 1);
      mbar_init(&io_empty[s], 2);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], 256);
    }
    mbar_init(spare, 1);
    *flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(holder, 512);
  pdl_trigger();
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;
  const Sync sy{flag, a.status};
  const int nit = (a.d + 127) / 128, t = block / a.parts, p = block - t * a.parts;
  const int i0 = (int)((long long)nit * p / a.parts), i1 = (int)((long long)nit * (p + 1) / a.parts);
  InFlight fl;
  if (warp == 0) {
    if (lane == 0) {
      mbar_expect_tx(a_full, NKB * 2 * kTile);
      fl.note((int)(a_full - bar), 0);
      for (int kb = 0; kb < NKB; ++kb) {
        tma_load_2d(sm + kb * 2 * kTile, &mL, 64 * kb, t * 128, a_full);
        tma_load_2d(sm + (kb * 2 + 1) * kTile, &mL, a.Ep + 64 * kb, t * 128, a_full);
      }
      int bs = 0, io = 0;
      uint32_t bp = 1, iop = 1;
      bool ok = true;
      for (int i = i0; i < i1 && ok; ++i) {
        for (int c = 0; c < 2 * NKB && ok; ++c) {   // 64 experts' high parts, then their low parts
          ok = sy.wait(&b_empty[bs], bp);
          if (!ok) break;
          mbar_expect_tx(&b_full[bs], kTile);
          fl.note((int)(b_full - bar) + bs, bp ^ 1u);
          tma_load_2d(sm + PL::kOffB + bs * kTile, &mW, (c & 1 ? a.Ep : 0) + 64 * (c >> 1), i * 128, &b_full[bs]);
          if (++bs == kDxB) {
            bs = 0;
            bp ^= 1u;
          }
        }
        if (!ok) break;
        ok = sy.wait(&io_empty[io], iop);
        if (!ok) break;
        if (a.with_in) {
          uint8_t* st = sm + PL::kOffIo + io * 2 * kTile;
          mbar_expect_tx(&io_full[io], 2 * kTile);
          fl.note((int)(io_full - bar) + io, iop ^ 1u);
          tma_load_2d(st, &mIn, i * 128, t * 128, &io_full[io]);
          tma_load_2d(st + kTile, &mIn, i * 128 + 64, t * 128, &io_full[io]);
        } else {
          mbar_arrive(&io_full[io]);
        }
        if (++io == IO) {
          io = 0;
          iop ^= 1u;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t idesc = idesc_f16(128, 128, 0, 0);
    if (lane == 0) {
      int bs = 0;
      uint32_t bp = 0;
      bool ok = sy.wait(a_full, 0);
      for (int i = i0; i < i1 && ok; ++i) {
        const int tile = i - i0, buf = tile & 1;
        ok = sy.wait(&acc_empty[buf], ((tile >> 1) & 1) ^ 1u);
        for (int c = 0; c < 2 * NKB && ok; ++c) {
          ok = sy.wait(&b_full[bs], bp);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sa = smem_u32(sm + (c >> 1) * 2 * kTile), sb = smem_u32(sm + PL::kOffB + bs * kTile);
          const uint64_t ah = smem_desc(sa, 16, 1024, 2), al = smem_desc(sa + kTile, 16, 1024, 2);
          const uint64_t bd = smem_desc(sb, 16, 1024, 2);
          const uint32_t d1 = tmem + buf * 256, d2 = d1 + 128;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t more = (c | k) ? 1u : 0u;
            if (c & 1) {
              tc_mma_f16(d2, ah + 2 * k, bd + 2 * k, idesc, 1u);
            } else {
              tc_mma_f16(d1, ah + 2 * k, bd + 2 * k, idesc, more);
              tc_mma_f16(d2, al + 2 * k, bd + 2 * k, idesc, more);
            }
          }
          tc_commit(&b_empty[bs]);
          if (++bs == kDxB) {
            bs = 0;
            bp ^= 1u;
          }
        }
        if (ok) tc_commit(&acc_full[buf]);
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int q = warp & 3, ch = (warp - 4) >> 2;   // TMEM lanes 32 q .., 64-column half
    const int row = 32 * q + lane;
    int io = 0;
    uint32_t iop = 0;
    bool ok = true;
    const bool storer = q == 0 && lane == 0;
    const float st = a.sT[t];
    for (int i = i0; i < i1; ++i) {
      const int tile = i - i0, buf = tile & 1;
      if (ok) ok = sy.wait(&acc_full[buf], (tile >> 1) & 1) && sy.wait(&io_full[io], iop);
      ok = __all_sync(0xffffffffu, ok);
      // The four warps of a half meet at the barrier below, and each learns by itself that a wait gave
      // up: it then goes on to the barrier of every tile that is left, without waits, sums or stores.
      if (ok) {
        tc_fence_after();
        const float s = st * a.sW[i], s2 = s / kGateLo;
        uint8_t* box = sm + PL::kOffIo + (io * 2 + ch) * kTile + row * 128;
        const uint32_t t0 = tmem + ((uint32_t)(32 * q) << 16) + buf * 256 + ch * 64;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float u[32], v[32];
          tmem_ld32x2(t0 + 32 * b, t0 + 128 + 32 * b, u, v);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint4* at = reinterpret_cast<uint4*>(box + (((4 * b + w) ^ (row & 7)) << 4));
            uint4 old = make_uint4(0u, 0u, 0u, 0u);
            if (a.with_in) old = *at;
            uint32_t o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&o[j]));
              const int k = 8 * w + 2 * j;
              const __half2 r = __floats2half2_rn(fmaf(s, u[k], fmaf(s2, v[k], f.x)),
                                                  fmaf(s, u[k + 1], fmaf(s2, v[k + 1], f.y)));
              o[j] = *reinterpret_cast<const uint32_t*>(&r);
            }
            *at = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        tc_fence_before();
        mbar_arrive(&acc_empty[buf]);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      asm volatile("bar.sync %0, 128;" ::"r"(1 + ch) : "memory");
      if (storer && ok) {
        const int x = i * 128 + 64 * ch;
        if (x < a.d) tma_store_2d(&mOut, x, t * 128, sm + PL::kOffIo + (io * 2 + ch) * kTile);
        bulk_commit();
        if (tile > 0) {                           // the tile before is out: its buffer is free
          bulk_wait_read<1>();
          mbar_arrive(&io_empty[io == 0 ? IO - 1 : io - 1]);
        }
      }
      if (++io == IO) {
        io = 0;
        iop ^= 1u;
      }
    }
    if (storer) bulk_wait_read<0>();
  }
  end_block(sy, fl, bar, spare, tmem);
}

// ---------------------------------------------------------------- both in one launch
// The first w_blocks blocks sum dWg, the others write dX as they find an SM free.
struct BothMaps {
  CUtensorMap X, L64, L, W, in, out;
};
template <int IW, int NKB>
__global__ void __launch_bounds__(kThreads, 1)
    gate_grad_kernel(const __grid_constant__ BothMaps m, const WgArgs wa, const DxArgs xa, int w_blocks) {
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  if ((int)blockIdx.x < w_blocks)
    wgrad_block<IW>(sm, m.X, m.L64, wa, blockIdx.x);
  else
    dx_block<NKB>(sm, m.L, m.W, m.in, m.out, xa, (int)blockIdx.x - w_blocks);
}

int pad64(int E) { return (E + 63) / 64 * 64; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// How a call is cut: token rows per block of dWg (a multiple of 128) and accumulators per block, and
// column parts per token tile of dX.  What takes least time by 2.2 us per 128 rows of dWg with two
// accumulators, 1.4 with one, 1 us and 0.3 per 64 experts (above 128: 0.8) for a 128 x 128 tile of dX, 3 us to start
// either, and the partial sums' way through L2 and the launch that joins them; the blocks of dX take
// the SMs that dWg leaves and each of the others when its block ends.
struct GatePlan {
  int run, iw, parts;
};
GatePlan gate_plan(int T, int d, int E, bool wgrad, bool dx, int sms) {
  // The search takes up to 4 us of the host, half as long as the rest of the call there: a thread keeps the
  // plans of its last shapes (two layers in turn: 11.5 us a call with one plan kept, 7.8 now; ragged batches,
  // which differ in whole tiles of 128 rows: 9.3, 8.1).
  struct Kept {
    int tt, d, E, what, sms;
    GatePlan plan;
  };
  constexpr int kKept = 256;
  thread_local Kept kept[kKept];                    // (zero: no plan has tt = 0)
  const int tt = (T + 127) / 128, nit = (d + 127) / 128, jb = (E + 127) / 128, nkb = (E + 63) / 64;
  const int what = wgrad + 2 * dx;
  Kept& mine = kept[((uint32_t)tt * 4u + what + (uint32_t)d * 2654435761u + (uint32_t)E * 40503u) % kKept];
  if (mine.tt == tt && mine.d == d && mine.E == E && mine.what == what && mine.sms == sms) return mine.plan;
  const int most = wgrad ? std::min(tt, sum_parts((size_t)d * E)) : 1;
  GatePlan best{tt * 128, 1, 1};
  double cost = 1e300;
  for (int iw = 1; iw <= (wgrad ? 2 : 1); ++iw) {
    const int cols = (d + 128 * iw - 1) / (128 * iw) * jb;
    for (int q = 1; q <= most; ++q) {
      const int run = (tt + q - 1) / q, runs = (tt + run - 1) / run;
      const long long W = wgrad ? (long long)cols * runs : 0;
      const double w = run * (iw == 2 ? 2.2 : 1.4) + 3.0;
      const double join = runs > 1 ? 2.0 + runs * (double)d * E * 1e-6 : 0.0;
      const double early = (double)(W / sms) * w;    // SMs without a last block of dWg are free then
      const long long late = W % sms;
      if (!dx) {
        const double c = early + (late ? w : 0.0) + join;
        if (c < cost) {
          cost = c;
          best = GatePlan{run * 128, iw, 1};
        }
        continue;
      }
      for (int p = 1; p <= std::min(nit, 16); p += p < 4 ? 1 : p < 8 ? 2 : 4) {
        const double us = (nit + p - 1) / p * (1.0 + (nkb <= 2 ? 0.3 : 0.8) * nkb) + 3.0;
        const long long X = (long long)tt * p;
        // n rounds of the free SMs, and what the late ones add in that time
        long long n = std::max<long long>(1, (long long)((X * us - late * us) / (sms * us)));
        double end = 0.0;
        for (int step = 0; step < 8; ++step, ++n) {
          const double t = n * us;                   // after `early`
          const long long m = t > w ? (long long)((t - w) / us) : 0;
          if ((sms - late) * n + late * m >= X) {
            end = early + std::max(t, late ? w : 0.0);
            break;
          }
          if ((sms - late) * n + late * (m + 1) >= X) {   // the late ones' next blocks end it
            end = early + std::max(w + (m + 1) * us, t);
            break;
          }
        }
        if (end == 0.0) end = early + w + n * us;
        if (end + join < cost) {
          cost = end + join;
          best = GatePlan{run * 128, iw, p};
        }
      }
    }
  }
  mine = Kept{tt, d, E, what, sms, best};
  return best;
}

struct GateWs {
  size_t dl2, W2, sT, sW, partial, total;
};
GateWs gate_ws(int T, int d, int E) {
  const size_t Ep = pad64(E);
  GateWs w;
  w.dl2 = 0;
  w.W2 = w.dl2 + up256((size_t)T * 2 * Ep * 2);
  w.sT = w.W2 + up256((size_t)d * 2 * Ep * 2);
  w.sW = w.sT + up256((size_t)(T + 127) / 128 * 4);
  w.partial = w.sW + up256((size_t)(d + 127) / 128 * 4);
  w.total = w.partial + up256(sum_partial_bytes((size_t)d * E, T, 128));
  return w;
}

template <int IW, int NKB>
cudaError_t launch_both(const BothMaps& m, const WgArgs& wa, const DxArgs& xa, int w_blocks, int x_blocks,
                        cudaStream_t s) {
  auto kern = gate_grad_kernel<IW, NKB>;
  MOE_LAUNCH(ensure_smem_attr(reinterpret_cast<const void*>(kern)));
  const size_t w_smem = (size_t)kWgStages * kWgStageBytes + 256 + 1024, x_smem = DxPlan<NKB>::kBytes;
  const size_t smem = !x_blocks ? w_smem : !w_blocks ? x_smem : std::max(w_smem, x_smem);
  return launch_k(kern, w_blocks + x_blocks, kThreads, smem, s, true, m, wa, xa, w_blocks);
}

}  // namespace

// The multiply-add kernels (grad.cu) need no split but take a launch per gradient.  us there / here: both
// gradients, 1024 columns, T = 1: E = 8 7.9 / 7.7, E = 127 15.3 / 10.6; T = 256: E = 8 12.0 / 9.4, E = 127
// 29 / 17.  dWg alone: E = 8: T = 256 9.3 / 9.6, 512 11.5 / 10.8; E = 128: T = 16 10.5 / 9.9, 128 15.3 / 12.9;
// 3584 columns, E = 256: T = 64 14.5 / 17.1, 128 20.4 / 20.3, 256 24.5 / 20.9.  dX alone: 512 x 1024 x 128
// 11.9 / 12.5, 1024 x 1024 x 128 19.8 / 12.4; above 128 experts, whose ring of Wg is short: 128 x 3584 x 256
// 19.7 / 27.1, 256 x 3584 x 256 27.6 / 26.8; odd rows, whose split is scalar: 512 x 1024 x 127 12.2 / 15.6,
// 256 x 3584 x 255 27.8 / 31.4 (16384 x 3584 x 128: 705 / 54).
bool gate_tc_ok(int T, int d, int E, bool wgrad, bool dx) {
  if (E > 256) return false;
  if (wgrad && dx) return true;
  if (wgrad) return T >= 128 && (long long)T * E >= 4096;
  return dx && (double)T * d * E >= (E % 4 || E > 128 ? 240e6 : 100e6);
}
size_t gate_tc_bytes(int T, int d, int E) { return T > 0 ? gate_ws(T, d, E).total : 0; }

cudaError_t launch_gate_tc(const float* logits, const int32_t* topk_idx, const float* dtopk_w,
                           const float* dlosses, const int32_t* counts, const int32_t* n_valid,
                           const uint8_t* mask, int k, float* dlogits, const __half* tokens,
                           const float* Wg, float* dWg, const __half* dx_in, __half* dx, uint8_t* ws,
                           int* status, int T, int d, int E, cudaStream_t s, const RouteScore* how) {
  int dev = 0, sms = 0;
  MOE_LAUNCH(cudaGetDevice(&dev));
  MOE_LAUNCH(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  const GateWs w = gate_ws(T, d, E);
  const int Ep = pad64(E);
  __half *dl2 = reinterpret_cast<__half*>(ws + w.dl2), *W2 = reinterpret_cast<__half*>(ws + w.W2);
  float *sT = reinterpret_cast<float*>(ws + w.sT), *sW = reinterpret_cast<float*>(ws + w.sW);
  MOE_LAUNCH(launch_dlogits_split(logits, topk_idx, dtopk_w, dlosses, counts, n_valid, mask, T, E, k,
                                  dlogits, status, dx ? Wg : nullptr, d, Ep, dl2, sT, W2, sW, s, how));
  const uint64_t l_dims[2] = {(uint64_t)2 * Ep, (uint64_t)T}, x_dims[2] = {(uint64_t)d, (uint64_t)T};
  const uint64_t w_dims[2] = {(uint64_t)2 * Ep, (uint64_t)d};
  const uint32_t b64[2] = {64, 64}, b128[2] = {64, 128};
  BothMaps m;
  memset(&m, 0, sizeof(m));
  const GatePlan pl = gate_plan(T, d, E, dWg != nullptr, dx != nullptr, sms);
  WgArgs wa{};
  DxArgs xa{};
  int w_blocks = 0, x_blocks = 0, runs = 0;
  float* partial = reinterpret_cast<float*>(ws + w.partial);
  if (dWg) {
    if (!encode_f16_map(&m.X, tokens, 2, x_dims, b64) || !encode_f16_map(&m.L64, dl2, 2, l_dims, b64))
      return cudaErrorInvalidValue;
    runs = (T + pl.run - 1) / pl.run;
    wa = WgArgs{sT, mask, runs == 1 ? dWg : partial, T, d, E, Ep, pl.run, runs == 1, status};
    w_blocks = (d + 128 * pl.iw - 1) / (128 * pl.iw) * runs * ((E + 127) / 128);
  }
  if (dx) {
    if (!encode_f16_map(&m.L, dl2, 2, l_dims, b128) || !encode_f16_map(&m.W, W2, 2, w_dims, b128) ||
        !encode_f16_map(&m.out, dx, 2, x_dims, b128) || (dx_in && !encode_f16_map(&m.in, dx_in, 2, x_dims, b128)))
      return cudaErrorInvalidValue;
    xa = DxArgs{sT, sW, T, d, E, Ep, pl.parts, dx_in != nullptr, status};
    x_blocks = (T + 127) / 128 * pl.parts;
  }
  auto with_iw = [&](auto nkb) {
    constexpr int K = decltype(nkb)::value;
    return pl.iw == 2 ? launch_both<2, K>(m, wa, xa, w_blocks, x_blocks, s)
                      : launch_both<1, K>(m, wa, xa, w_blocks, x_blocks, s);
  };
  using std::integral_constant;
  const int nkb = Ep / 64;
  MOE_LAUNCH(nkb == 1   ? with_iw(integral_constant<int, 1>())
             : nkb == 2 ? with_iw(integral_constant<int, 2>())
             : nkb == 3 ? with_iw(integral_constant<int, 3>())
                        : with_iw(integral_constant<int, 4>()));
  if (runs > 1) MOE_LAUNCH(launch_sum_join(dWg, partial, d, E, T, pl.run, sms, s));
  return cudaSuccess;
}

}  // namespace moe
