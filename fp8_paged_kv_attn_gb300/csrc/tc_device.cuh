// Device code that the block-scaled cache's attention kernels share: asynchronous copies of scales,
// V scales and their undoing, and tcgen05 (5th-generation tensor cores) building blocks.
// Included after decode_attn_mma.cuh.
#pragma once

namespace kvq {

__device__ __forceinline__ void cp_async8(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(dst)), "l"(src)
               : "memory");
}

// Arrives on the barrier once this thread's async copies so far have landed
// (the arrival is one of the barrier's expected count).
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

// A V scale as 2^e times a fraction in (1/2, 1] (1 for a power of two), x the fraction and y
// e: from the bits, since 2^-e has no fp32 for the scales above 2^126, and a subnormal scale's
// weights would sit low in f16's range with e = -126.  0 is 0 times a power of two.
__device__ __forceinline__ float2 split_scale(float s) {
  const bool sub = s < 0x1p-126f;
  const uint32_t u = __float_as_uint(sub ? s * 0x1p24f : s), frac = u & 0x7FFFFFu;
  const int e = static_cast<int>(u >> 23) - (sub ? 151 : 127) + (frac ? 1 : 0);
  return make_float2(frac ? __uint_as_float(frac | 0x3F000000u) : u ? 1.f : 0.f, static_cast<float>(e));
}

// 2^t / l as two factors, to be multiplied with in turn: a sum is undone by 2^t for t = n - m
// (and the operand's scale), and neither that power nor its quotient need have an fp32 where
// V scales are very large or small, or l is, behind a maximum that grew.  Where t is harmless
// the second factor is the power of two in 1 / l, and nothing is rounded twice.
__device__ __forceinline__ float2 out_scale(float t, float l) {
  const int k = max(-126, min(126, static_cast<int>(__float_as_uint(l) >> 23) - 127));
  const float u = fminf(fmaxf(t, -100.f), 40.f);
  return make_float2(exp2f(u) / (l * pow2(-k)), exp2f(t - u - static_cast<float>(k)));
}

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory operand of 128-byte rows, 128-byte swizzle, 8-row groups 1,024
// bytes apart (bits 46-48: descriptor version 1; 61-63: the swizzle).
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) |
         (2ull << 61);
}

// One lane of the (whole) warp, always the same.  Under this test the compiler
// knows that a single thread issues an MMA or a copy; under `lane == 0` it issues them
// in a loop over lanes (an MMA every 66 cycles at least, 40 here).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

__device__ __forceinline__ void tc_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_addr(bar))
               : "memory");
}

// Consecutive columns of this warp's 32 lanes, loaded and waited for in one statement, so that no use of
// theirs moves between.
__device__ __forceinline__ void tc_ld16(float (&v)[16], uint32_t addr) {
  uint32_t *r = reinterpret_cast<uint32_t *>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
      "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}

__device__ __forceinline__ void tc_st16(uint32_t addr, const float (&v)[16]) {
  const uint32_t *r = reinterpret_cast<const uint32_t *>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}

// q's pieces of two values: e4m3, and e5m2 of what is left.  A bf16 value's eight bits
// less their rounding to four are at most eight units of the last place, and e5m2's three
// bits hold those, down to 2^-13; only a value below e4m3's smallest normal number, 2^-6,
// is off, by at most 2^-14.
__device__ __forceinline__ void tc_q_pieces(float x, float y, int shift, uint32_t &c1, uint32_t &c2) {
  const uint16_t c = f32x2_to_e4m3x2(x, y);
  const float2 p = f16x2_to_f32x2(e4m3x2_to_f16x2(c));
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y - p.y), "f"(x - p.x));
  c1 |= static_cast<uint32_t>(c) << shift;
  c2 |= static_cast<uint32_t>(r) << shift;
}

// Bit 7 of each byte that is a NaN code (0x7F or 0xFF; no carry leaves a byte).
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// 16-byte chunk c of row r in a 128-byte-swizzled tile.
__device__ __forceinline__ uint8_t *tc_chunk(uint8_t *tile, int r, int c) {
  return tile + r * 128 + ((c ^ (r & 7)) * 16);
}

}  // namespace kvq
