// Warp-level pieces of the low-rank kernels: 16-byte asynchronous copies, fragment loads and the
// 16 x 8 x 16 f16 product, and the split of a 32-bit value into two f16 parts.
//
// The low-rank products have 2 r operations per element that they stream (r <= 128), far below
// what the tensor cores can do per byte of DRAM.  A product issued by the warp that loaded the operands
// needs no tensor memory and no hand-over to an issuing thread, which short runs, chains of
// latencies, gain by.  Long runs pay for it: their operands pass through registers, and the fragment loads
// (half of the shared-memory pipe) and the products' latencies hold them rather than DRAM (adapter.cu).
#pragma once

#include "common.cuh"

namespace moe {

// 16 bytes global -> shared; `on` false writes zeros and reads nothing (src must still be a
// valid address).
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
// One arrival on `bar` once this thread's earlier copies have landed (counted in its set-up).
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p))
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p))
               : "memory");
}

__device__ __forceinline__ void stsm4(void* p, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(smem_u32(p)),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

// The same from shared-memory addresses (bytes): loops that step through a ring keep one base and
// constant offsets instead of a generic pointer per load.
__device__ __forceinline__ void ldsm4_t_at(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void cp_async16_at(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}

// d += a b: a 16 x 16 (rows), b 16 x 8 (columns), f16 operands, f32 sums.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// d = a b.
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Fragments of a 16 x 16 block whose rows are contiguous in shared memory (stride ld halves):
// `a` operand with rows = m, columns = k.
__device__ __forceinline__ void frag_a(uint32_t (&r)[4], const __half* s, int ld, int lane) {
  ldsm4(r, s + (lane & 15) * ld + (lane >> 4) * 8);
}
// Two adjacent `b` operands (16 columns): r[0..1] the first eight, r[2..3] the next.
// Stored with rows = k, columns = n:
__device__ __forceinline__ void frag_b_kn(uint32_t (&r)[4], const __half* s, int ld, int lane) {
  ldsm4_t(r, s + (lane & 15) * ld + (lane >> 4) * 8);
}
// Stored with rows = n, columns = k:
__device__ __forceinline__ void frag_b_nk(uint32_t (&r)[4], const __half* s, int ld, int lane) {
  ldsm4(r, s + ((lane & 7) + (lane >> 4) * 8) * ld + ((lane >> 3) & 1) * 8);
}

// Power of two 2^e with e = exponent of m (m >= 0, the largest magnitude of a set), kept where
// 2^-e is a normal number; 1 when m is zero or not finite.
__device__ __forceinline__ int scale_exp(float m) {
  const int e = (int)((__float_as_uint(m) >> 23) & 255u) - 127;
  return m == 0.f || e == 128 ? 0 : max(-126, min(126, e));
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The same for values that are split into two f16 parts: 2^-e brings the largest into [2^14, 2^15), the
// top of f16's range, so that the low part of a value far below it still has its bits (scaled to
// [1, 2) instead, a value 2^-17 of the largest kept eight).
__device__ __forceinline__ int split_exp(float m) {
  const int e = (int)((__float_as_uint(m) >> 23) & 255u) - 127;
  return m == 0.f || e == 128 ? 0 : max(-126, e - 14);
}

// v = hi + lo up to 2^-23 |v| and 2^-25 (|v| < 2^15 by split_exp's scale: 2^-39 of the set's largest; hi
// has 11 bits, lo the next 11, and the smallest step of either is 2^-24).
// A value whose hi is not finite keeps it and has no lo.
__device__ __forceinline__ void split_f16(float v, __half& hi, __half& lo) {
  hi = __float2half_rn(v);
  const float h = __half2float(hi);
  lo = isfinite(h) ? __float2half_rn(v - h) : __ushort_as_half(0);
}

}  // namespace moe
