// Shared pieces of the attention kernels over the paged NVFP4 cache.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kv_paged.cuh"

namespace nvfp4 {
namespace attn {

struct Args {
  const uint16_t *q;           // bf16 [tokens, q_heads, D], token stride ld_q
  int64_t ld_q;
  int32_t tokens;
  const int32_t *offsets;      // [batch+1] query offsets, or null: one query per sequence
  const int32_t *lens;         // [batch] cached tokens
  int32_t batch, max_query;
  const int32_t *table;        // [batch, max_pages]
  int32_t max_pages, page_size;
  FastDiv by_page;             // division by page_size
  int64_t num_pages;
  const uint8_t *k_q, *k_sf, *v_q, *v_sf;
  const float *k_gs, *v_gs;
  int32_t heads_q, heads_kv, group;
  FastDiv by_group;            // division by group
  float scale_log2;            // softmax scale * log2(e)
  int32_t causal;
  void *out;                   // [tokens, q_heads, D]
  int32_t out_bf16;
  bool v8_q, v8_out;           // rows of q, of a bf16 out begin on 32 bytes
  float *lse;                  // [tokens, q_heads] or null
  int32_t *dev_status;
};

struct Seq { int32_t len, first, queries; };

// Sequence b's part of the query offsets: inside [0, tokens], not decreasing,
// at most max_query queries.  One bad entry refuses the whole call, so that the
// sequences' queries never overlap and their sum is at most `tokens`.
__device__ __forceinline__ bool offsets_ok(const Args &A, int b) {
  if (!A.offsets) return true;
  const int32_t x = A.offsets[b], y = A.offsets[b + 1];
  return x >= 0 && x <= y && y <= A.tokens && y - x <= A.max_query;
}

// Cached tokens and queries of sequence b (its offsets checked before).  A
// length outside [0, max_pages * page_size] counts as 0 and is reported.
__device__ __forceinline__ Seq load_seq(const Args &A, int b) {
  Seq s;
  s.len = A.lens[b];
  s.first = A.offsets ? A.offsets[b] : b;
  s.queries = A.offsets ? A.offsets[b + 1] - s.first : 1;
  if (s.len < 0 || (int64_t)s.len > (int64_t)A.max_pages * A.page_size) {
    s.len = 0;
    report(A.dev_status, NVFP4_ERR_INDEX);
  }
  return s;
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint4 lds_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds_v2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts_v2(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" :: "r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kN>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(kN) : "memory"); }

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The two E2M1 codes of byte kByte of w as f16x2 (low nibble in the low half).
template <int kByte>
__device__ __forceinline__ uint32_t e2m1x2_f16x2(uint32_t w) {
  uint32_t d;
  if constexpr (kByte == 0)
    asm("{.reg .b8 a,b,c,d; mov.b32 {a,b,c,d}, %1; cvt.rn.f16x2.e2m1x2 %0, a;}" : "=r"(d) : "r"(w));
  else if constexpr (kByte == 1)
    asm("{.reg .b8 a,b,c,d; mov.b32 {a,b,c,d}, %1; cvt.rn.f16x2.e2m1x2 %0, b;}" : "=r"(d) : "r"(w));
  else if constexpr (kByte == 2)
    asm("{.reg .b8 a,b,c,d; mov.b32 {a,b,c,d}, %1; cvt.rn.f16x2.e2m1x2 %0, c;}" : "=r"(d) : "r"(w));
  else
    asm("{.reg .b8 a,b,c,d; mov.b32 {a,b,c,d}, %1; cvt.rn.f16x2.e2m1x2 %0, d;}" : "=r"(d) : "r"(w));
  return d;
}

// E4M3 scale bytes (in the low byte of each half of w) as f16 times 2^-8: the
// exponent field moves from bias 7 to bias 15 unchanged, subnormals included.
// Every byte, valid or left over in an unused part of a page, gives a finite
// value (the NaN code reads as 480), so a masked key never meets a NaN.
__device__ __forceinline__ uint32_t e4m3_pair_f16x2(uint32_t w) { return (w << 7) & 0x3F803F80u; }
constexpr float kScaleFix = 256.0f;

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace attn
}  // namespace nvfp4
