// 8-bit blocks: e4m3 elements with a power-of-two scale per block, held as an
// E8M0 byte u (the scale is 2^(u - 127)).
//
// A power of two costs no precision against a free scale as long as a block's
// values stay above e4m3's subnormals (2^-15 of the block's maximum): dividing
// by it is exact, so each element is rounded once, by at most 2^-4 of its
// value. It lets the tensor core apply the scales itself, and a cache block
// can move to a larger scale without touching the mantissas of its elements.
#pragma once

#include <cuda_fp8.h>

#include "q3vl_device.cuh"

namespace q3vl {

// E8M0 byte of the scale for a block maximum `amax` (finite, >= 0): the
// smallest s >= -126 with amax <= 448 2^s = 1.75 2^(s + 8). With amax =
// m 2^e, 1 <= m < 2, that is s = e - 8, or e - 7 when m > 1.75.
__device__ __forceinline__ uint32_t e8m0_of_amax(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int u = static_cast<int>(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(u < 1 ? 1 : u);
}

// 2^(u - 127) and 2^(127 - u) for u in [1, 253] (a scale made by
// e8m0_of_amax is at most 2^120).
__device__ __forceinline__ float e8m0_scale(uint32_t u) { return __uint_as_float(u << 23); }
__device__ __forceinline__ float e8m0_inverse(uint32_t u) {
  return __uint_as_float((254u - u) << 23);
}

// |x| where x is finite, else 0: what x adds to its block's maximum.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}

// Four floats (already divided by the scale) to e4m3, round to nearest even,
// element 0 in the low byte. fma(x, 0, x) turns an infinity into NaN (the
// conversion alone would saturate it) and leaves finite values as they are.
// pack_e4m3x4_finite is for values without infinities.
__device__ __forceinline__ uint32_t pack_e4m3x4_finite(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  return pack_e4m3x4_finite(fmaf(a, 0.f, a), fmaf(b, 0.f, b), fmaf(c, 0.f, c), fmaf(d, 0.f, d));
}

// Four e4m3 bytes to floats.
__device__ __forceinline__ float4 unpack_e4m3x4(uint32_t w) {
  uint32_t l, h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(l) : "h"(static_cast<uint16_t>(w & 0xffffu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w >> 16)));
  const float2 a = __half22float2(*reinterpret_cast<__half2*>(&l));
  const float2 b = __half22float2(*reinterpret_cast<__half2*>(&h));
  return make_float4(a.x, a.y, b.x, b.y);
}

// The same for e5m2 (4 mantissa steps a factor of two, from 2^-16 to 57344),
// for values of at most 57344 or NaN.
__device__ __forceinline__ uint32_t pack_e5m2x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
__device__ __forceinline__ float4 unpack_e5m2x4(uint32_t w) {
  uint32_t l, h;
  asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(l) : "h"(static_cast<uint16_t>(w & 0xffffu)));
  asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w >> 16)));
  const float2 a = __half22float2(*reinterpret_cast<__half2*>(&l));
  const float2 b = __half22float2(*reinterpret_cast<__half2*>(&h));
  return make_float4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Eight consecutive elements of a row as floats (16-byte aligned address).
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 t = unpack_bf16x2(w[j]);
    f[2 * j] = t.x;
    f[2 * j + 1] = t.y;
  }
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// Rounds to the row's type and stores; f becomes the rounded values.
__device__ __forceinline__ void store8(__nv_bfloat16* p, float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
    const float2 t = unpack_bf16x2(w[j]);
    f[2 * j] = t.x;
    f[2 * j + 1] = t.y;
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, float (&f)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

// ---------------------------------------------------------------------------
// tcgen05 with block scales (kind::mxf8f6f4: e4m3 or e5m2 operands, one E8M0
// scale per row and 32 columns, fp32 accumulation)
// ---------------------------------------------------------------------------
// Instruction descriptor: bits [4,6) and [29,31) choose the byte of B's and
// A's scale words (idesc_sf adds them), [7,10) / [10,13) A / B format
// (0 = e4m3, 1 = e5m2), [17,23) N >> 3, 23 scale type (1 = E8M0), [24,29) M >> 4.
__host__ __device__ constexpr uint32_t idesc_sf(uint32_t byte) { return (byte << 4) | (byte << 29); }
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N) {
  return (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24);
}

// D[tmem] (+)= (A 2^sa) (B 2^sb)^T, operands in shared memory, scale words in
// TMEM (one thread).
__device__ __forceinline__ void umma_mxf8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X "
      "[%0], %1, %2, %3, [%5], [%6], p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
__device__ __forceinline__ void umma_mxf8_ss_pair(uint32_t d_tmem, uint64_t a_desc,
                                                  uint64_t b_desc, uint32_t idesc, uint32_t sfa,
                                                  uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X "
      "[%0], %1, %2, %3, [%5], [%6], p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}

// Scale words of 128 operand rows: 512 bytes in shared memory, the word of row
// r at (r % 32) * 16 + (r / 32) * 4, copied to 4 TMEM columns (row r in lane
// r % 32 of column r / 32, in all four 32-lane quarters). A copy and the MMAs
// that one thread issues behind it run in that order.
constexpr uint32_t kNoScale = 0x7f7f7f7fu;  // 2^0
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
  // no swizzle; 8-row groups of 128 bytes, one 16-byte column
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128 >> 4) << 32) |
         (static_cast<uint64_t>(1u) << 46);
}
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
__device__ __forceinline__ void tmem_cp_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

// True in one lane of a converged warp, the same one each time. The TMA and
// MMA loops below run in whole warps and issue under this test: the compiler
// then knows the operands to be uniform. Measured on a loop of four 256 x 224
// x 32 MMAs and one barrier wait: 112 cycles per MMA (the tensor core's own
// time) against 138 when a single thread runs the loop.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

// Arrival on a barrier of the CTA pair without mbar_arrive_cluster's release
// at cluster scope, which waits for all of the thread's memory operations
// (about 1 us a time). For words that only the tensor core reads: the writers'
// proxy fence has put them in place before this.
__device__ __forceinline__ void mbar_arrive_peer(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// 16 bytes from a shared-memory address of any CTA of the cluster (DSMEM).
__device__ __forceinline__ float4 ld_dsmem_f32x4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

// Requests a box into L2 only: legal before the kernel's dependency is met,
// since a later write of it goes through L2 as well.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* tm, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(tm)),
               "r"(x), "r"(y)
               : "memory");
}

}  // namespace q3vl
