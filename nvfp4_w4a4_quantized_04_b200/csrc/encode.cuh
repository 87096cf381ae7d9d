// The per-block NVFP4 encode (16 bf16 or fp32 elements -> E4M3 scale, E2M1
// codes) and its load helpers, shared by the quantize, norm and KV-append
// kernels.
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"

namespace nvfp4 {

__device__ __forceinline__ uint4 ldg_nc_v4(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// max of |bf16| over the 8 halves of a uint4, as 16-bit magnitude bits
// (NaN patterns compare above inf, so a non-finite element shows up as >= 0x7F80).
__device__ __forceinline__ uint32_t absmax8_bits(uint4 v, uint32_t m) {
  m = __vmaxu2(m, v.x & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.y & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.z & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.w & 0x7FFF7FFFu);
  return m;
}

__device__ __forceinline__ uint32_t halves_max(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }

__device__ __forceinline__ uint32_t warp_max(uint32_t m) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  return m;
}

// One 16-element bf16 block: a 32-byte load when v8 (32-byte aligned), else two 16-byte loads.
__device__ __forceinline__ void load_block(const uint16_t *p, bool v8, uint4 &a, uint4 &b) {
  if (v8) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p));
  } else {
    a = ldg_nc_v4(p);
    b = ldg_nc_v4(p + 8);
  }
}

// 32-byte form of load_block for memory that the same kernel may write (an
// output that aliases its input): an ordinary load, not the read-only path.
__device__ __forceinline__ void load_block_rw(const uint16_t *p, bool v8, uint4 &a, uint4 &b) {
  if (v8) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p) : "memory");
  } else {
    a = *reinterpret_cast<const uint4 *>(p);
    b = *reinterpret_cast<const uint4 *>(p + 8);
  }
}

__device__ __forceinline__ void store_block(uint16_t *p, bool v8, const uint4 &a, const uint4 &b) {
  if (v8) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    *reinterpret_cast<uint4 *>(p) = a;
    *reinterpret_cast<uint4 *>(p + 8) = b;
  }
}

// bf16 of the exact sum hi + lo, rounded once (to nearest even).  The sum is
// first rounded to odd in fp32 -- truncated, with the last bit set when
// anything was dropped (Boldo and Melquiond, "Emulation of FMA and correctly
// rounded sums", 2008) -- so that the rounding to bf16 sees the dropped part.
// Values computed as hi + lo to about 2^-45 this way give the same bf16 as a
// 64-bit evaluation, and so the same 4-bit codes behind it.
__device__ __forceinline__ uint32_t bf16_of_sum(float hi, float lo) {
  const float r = __fadd_rn(hi, lo);
  const float v = __fsub_rn(r, hi);
  const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(r, v)), __fsub_rn(lo, v));   // Knuth's two-sum
  uint32_t bits = __float_as_uint(r);
  if (err != 0.0f && (bits & 0x7F800000u) != 0x7F800000u) {
    if ((err < 0.0f) == (r > 0.0f)) bits -= 1;
    bits |= 1;
  }
  if (lo == 0.0f || !isfinite(hi)) bits = __float_as_uint(hi);     // keeps the sign of a zero
  const __nv_bfloat16 b = __float2bfloat16_rn(__uint_as_float(bits));
  return (uint32_t)__bfloat16_as_ushort(b);
}

// Packed pairs of fp32 (first in the low word).
__device__ __forceinline__ uint64_t pair_f32(float lo, float hi) {
  return ((uint64_t)__float_as_uint(hi) << 32) | __float_as_uint(lo);
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t x, uint64_t y) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return d;
}
// Two fp32 -> bf16x2, round to nearest even.
__device__ __forceinline__ uint32_t bf16x2_of(uint64_t p) {
  uint32_t d;
  asm("{\n.reg .f32 l, h;\nmov.b64 {l, h}, %1;\ncvt.rn.bf16x2.f32 %0, h, l;\n}" : "=r"(d) : "l"(p));
  return d;
}

// Per 16-element block: the block amax in integer SIMD, one IEEE division
// for the scale and one IEEE reciprocal, the 16 products as eight packed
// f32x2 multiplies, eight e2m1x2 conversions and one 8-byte store.

// bf16 pair (element 2i in bits 0..15) -> fp32 pair (element 2i in the low word).
__device__ __forceinline__ uint64_t bf16x2_to_f32x2(uint32_t w) {
  return ((uint64_t)(w & 0xFFFF0000u) << 32) | (uint64_t)(w << 16);
}

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t x, uint64_t rr) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(rr));
  return d;
}

// Four fp32 pairs -> one word of eight E2M1 codes (element 2i in the low nibble
// of byte i), round to nearest even, saturating at +-6.
__device__ __forceinline__ uint32_t e2m1x8_from_pairs(uint64_t p0, uint64_t p1, uint64_t p2, uint64_t p3) {
  uint32_t out;
  asm("{\n.reg .b8 b0, b1, b2, b3;\n.reg .f32 l0, h0, l1, h1, l2, h2, l3, h3;\n"
      "mov.b64 {l0, h0}, %1;\nmov.b64 {l1, h1}, %2;\nmov.b64 {l2, h2}, %3;\nmov.b64 {l3, h3}, %4;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b0, h0, l0;\ncvt.rn.satfinite.e2m1x2.f32 b1, h1, l1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b2, h2, l2;\ncvt.rn.satfinite.e2m1x2.f32 b3, h3, l3;\n"
      "mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(out) : "l"(p0), "l"(p1), "l"(p2), "l"(p3));
  return out;
}

// E4M3 byte -> fp32 through the hardware E4M3 -> f16 conversion (every E4M3
// value is an f16 normal, so both steps are exact).
__device__ __forceinline__ float e4m3_to_f32_hw(uint32_t s) {
  float f;
  asm("{\n.reg .b16 b, l, h;\n.reg .b32 w;\ncvt.u16.u32 b, %1;\ncvt.rn.f16x2.e4m3x2 w, b;\n"
      "mov.b32 {l, h}, w;\ncvt.f32.f16 %0, l;\n}" : "=f"(f) : "r"(s));
  return f;
}

__device__ __forceinline__ uint64_t sanitize_pair(uint64_t d) {
  float lo = __uint_as_float((uint32_t)d), hi = __uint_as_float((uint32_t)(d >> 32));
  lo = isnan(lo) ? 0.0f : lo;
  hi = isnan(hi) ? 0.0f : hi;
  return ((uint64_t)__float_as_uint(hi) << 32) | __float_as_uint(lo);
}

__device__ __forceinline__ uint32_t block_amax_bits(const uint4 &va, const uint4 &vb) {
  return halves_max(absmax8_bits(vb, absmax8_bits(va, 0)));
}

// The block math (the definition in include/nvfp4.h) on a block already in
// fp32 pairs with its amax a_b: S = e4m3(a_b / (6 s_g)), r = 1/(S s_g) (0 when
// that product is 0), codes = e2m1(x r).
__device__ __forceinline__ uint2 encode_f32x16(const uint64_t (&xf)[8], float a_b, float s_g, float t_g,
                                               uint32_t &S) {
  S = f32_to_e4m3_satfinite(__fdiv_rn(a_b, t_g));
  const float e = __fmul_rn(e4m3_to_f32_hw(S), s_g);
  const float r = (e == 0.0f) ? 0.0f : __frcp_rn(e);
  const uint64_t rr = ((uint64_t)__float_as_uint(r) << 32) | __float_as_uint(r);
  uint64_t prod[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) prod[i] = mul_f32x2(xf[i], rr);
  if (isinf(r)) {                     // 0 * inf: the NaN encodes as +0
#pragma unroll
    for (int i = 0; i < 8; ++i) prod[i] = sanitize_pair(prod[i]);
  }
  return make_uint2(e2m1x8_from_pairs(prod[0], prod[1], prod[2], prod[3]),
                    e2m1x8_from_pairs(prod[4], prod[5], prod[6], prod[7]));
}

// Same, from the raw bf16 block; flags a non-finite element.
__device__ __forceinline__ uint2 encode_block16(const uint4 &va, const uint4 &vb, float s_g, float t_g,
                                                uint32_t &S, bool &bad) {
  const uint32_t m = block_amax_bits(va, vb);
  if (m >= 0x7F80u) bad = true;
  const uint64_t xf[8] = {bf16x2_to_f32x2(va.x), bf16x2_to_f32x2(va.y), bf16x2_to_f32x2(va.z),
                          bf16x2_to_f32x2(va.w), bf16x2_to_f32x2(vb.x), bf16x2_to_f32x2(vb.y),
                          bf16x2_to_f32x2(vb.z), bf16x2_to_f32x2(vb.w)};
  return encode_f32x16(xf, __uint_as_float(m << 16), s_g, t_g, S);
}

// Row part and block part of the MMA-tiled scale offset (they add up to
// sf_tiled_offset(r, j, nsf)).
__device__ __forceinline__ uint64_t sf_row_part(uint32_t r, uint32_t nsf) {
  return (uint64_t)(r >> 7) * (nsf >> 2) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4;
}
__device__ __forceinline__ uint32_t sf_blk_part(uint32_t j) { return (j >> 2) * 512 + (j & 3); }

}  // namespace nvfp4
