// Residual addition + RMS norm + quantized output in one pass (sm_100a).
//
// What it computes, per row (all of it from the definition in include/nvfp4.h):
//   r = bf16(x + residual),  y = bf16(r * w / sqrt(mean(r^2) + eps)),
// and y as NVFP4 with a given global scale (the activation format of the W4A4
// projections, "Qwen3.8-Flash-Next-NVFP4", two-level scaling section) or as
// E4M3 with one fp32 scale per row (the W8A8 projections of "Qwen3.8-27B-NVFP4").
//
// The row is read once: its bf16 values stay in the registers of one CTA
// between the sum of squares and the encode, so a row moves 2 + 2 bytes in and
// 2 + 9/16 (or 2 + 1) bytes out per element and nothing is read again.  The
// kernel is bound by HBM.  One CTA per row, one 16-element block per thread
// (two or four blocks for long rows): a block is the unit of the NVFP4 scale,
// so the block amax needs no exchange between threads, and a thread moves 32
// bytes per load.
//
// Rounding.  The sum of squares is kept in 64 bits (one conversion and one FMA
// per element) and 1/sqrt is one Newton step in 64 bits from the fp32 estimate
// (relative error below 2^-40); y is rounded to bf16 from an interval that holds
// it, or, where the interval's ends round apart, from an unevaluated fp32 pair.
// So y is the correctly rounded value, and the codes behind it do not depend on
// the order of the sum.  The root's power of two goes into r first, so that the
// product with w leaves fp32's range only where y does; below 2^-100, or 2^-100 |w|,
// what a subnormal drops makes y less exact.  (Such elements in 64 bits cost 270 to
// 290 us instead of 217 for 32768 rows: the test for them also finds the zeros
// that a residual leaves, about one in 10^3.  Products as (r root) w: 223.)
//
// Measured with a residual, K 5120: 32768 rows to E4M3 217 us in replayed graphs, 5.4
// TB/s (82 % of a copy's rate; 237 in plain calls); 4096 rows to NVFP4 33 us; 64 rows
// 6.3 us, which is one row's latency (load, two block reductions, store) and the launch.
// Four CTAs of ten warps an SM by registers; issue slots 69 %, stalls on loads and at
// the reductions' barriers.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "encode.cuh"
#include "host_util.cuh"

namespace nvfp4 {
namespace norm {

__device__ __forceinline__ uint32_t word(const uint4 &a, const uint4 &b, int i) {
  switch (i) {
    case 0: return a.x; case 1: return a.y; case 2: return a.z; case 3: return a.w;
    case 4: return b.x; case 5: return b.y; case 6: return b.z; default: return b.w;
  }
}
__device__ __forceinline__ uint4 pack4(const uint32_t *w) { return make_uint4(w[0], w[1], w[2], w[3]); }

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two fp32 -> two E4M3 bytes (first in the low byte), round to nearest even,
// saturating.
__device__ __forceinline__ uint32_t e4m3x2(float first, float second) {
  uint16_t out;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(out) : "f"(second), "f"(first));
  return out;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

struct Args {
  const uint16_t *x, *res, *w;
  uint16_t *res_out, *y;
  int64_t ld_x, ld_res, ld_ro;
  int32_t K;
  double inv_k, eps;
  float *scale;          // NVFP4: the given global scale; E4M3: one per row, written
  uint8_t *q, *sf;
  int32_t *dev_status;
  bool v8_x, v8_res, v8_ro, v8_y, v8_w;
};

enum { kFmtNone = 0, kFmtNvfp4 = 1, kFmtE4m3 = 2 };

// kB blocks of 16 elements per thread; block index threadIdx.x + i * blockDim.x.
// Up to kThreads threads, kCtas CTAs of that size per SM.
template <int kFmt, bool kTiled, int kB, int kThreads, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) add_rmsnorm_kernel(const Args A) {
  __shared__ double s_sum[32];
  __shared__ uint32_t s_max[32];
  const int64_t row = blockIdx.x;
  const int nblk = A.K >> 4, t = threadIdx.x, lane = t & 31, warp = t >> 5, nwarps = (blockDim.x + 31) >> 5;
  uint32_t r[kB][8];
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < kB; ++i) {
    const int j = t + i * (int)blockDim.x;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (j < nblk) {
      load_block_rw(A.x + row * A.ld_x + 16 * j, A.v8_x, a, b);
      if (A.res) {
        uint4 c, d;
        load_block_rw(A.res + row * A.ld_res + 16 * j, A.v8_res, c, d);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          r[i][k] = bf16x2_of(add_f32x2(bf16x2_to_f32x2(word(a, b, k)), bf16x2_to_f32x2(word(c, d, k))));
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) r[i][k] = word(a, b, k);
      }
      if (A.res_out) store_block(A.res_out + row * A.ld_ro + 16 * j, A.v8_ro, pack4(r[i]), pack4(r[i] + 4));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const double u = (double)lo_f32(r[i][k]), v = (double)hi_f32(r[i][k]);
        sum = fma(u, u, fma(v, v, sum));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) r[i][k] = 0;
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  sum = lane < nwarps ? s_sum[lane] : 0.0;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  // 1/sqrt: the fp32 estimate and one Newton step, then split into hi + lo
  const double ms = sum * A.inv_k + A.eps;
  double rs;
  if (ms > 1e-30 && ms < 1e30) {
    const double e0 = (double)rsqrtf((float)ms);
    rs = e0 * (1.5 - 0.5 * ms * e0 * e0);
  } else {
    rs = 1.0 / sqrt(ms);                    // rows of values beyond 1e15 or below 1e-15
  }
  const int e = max(-126, min(127, (int)((__double2hiint(rs) >> 20) & 0x7FF) - 1023));
  rs *= __hiloint2double((1023 - e) << 20, 0);                 // in [1, 2), but for roots beyond 2^127 and zero rows
  const float rs_hi = (float)rs, rs_lo = (float)(rs - (double)rs_hi);
  const uint32_t power = (uint32_t)(e + 127) << 7 | (uint32_t)(e + 127) << 23;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kB; ++i) {
    const int j = t + i * (int)blockDim.x;
    if (j >= nblk) continue;
    uint4 wa, wb;
    if (A.v8_w) {
      asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=r"(wa.x), "=r"(wa.y), "=r"(wa.z), "=r"(wa.w), "=r"(wb.x), "=r"(wb.y), "=r"(wb.z), "=r"(wb.w)
                   : "l"(A.w + 16 * j));
    } else {
      wa = __ldg(reinterpret_cast<const uint4 *>(A.w + 16 * j));
      wb = __ldg(reinterpret_cast<const uint4 *>(A.w + 16 * j + 8));
    }
    // y = r w / sqrt(..): r (with the root's power of two) times w is exact in fp32, and
    // times the fp32 root it is off by less than 2^-23 of itself.  Where both ends of
    // that interval round to the same bf16 -- for all but about one element in 2^12 --
    // that is y.
    uint32_t yw[8], differ = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) r[i][k] = mul_bf16x2(r[i][k], power);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint64_t t = mul_f32x2(bf16x2_to_f32x2(r[i][k]), bf16x2_to_f32x2(word(wa, wb, k)));
      const uint64_t p = mul_f32x2(t, pair_f32(rs_hi, rs_hi));
      yw[k] = bf16x2_of(mul_f32x2(p, pair_f32(1.0f - 0x1p-22f, 1.0f - 0x1p-22f)));
      differ |= yw[k] ^ bf16x2_of(mul_f32x2(p, pair_f32(1.0f + 0x1p-22f, 1.0f + 0x1p-22f)));
    }
    if (differ) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t w = word(wa, wb, k);
        // times hi + lo as p + (its error + t lo)
        const float tl = __fmul_rn(lo_f32(r[i][k]), lo_f32(w)), th = __fmul_rn(hi_f32(r[i][k]), hi_f32(w));
        const float pl = __fmul_rn(tl, rs_hi), ph = __fmul_rn(th, rs_hi);
        const float el = __fmaf_rn(tl, rs_lo, __fmaf_rn(tl, rs_hi, -pl));
        const float eh = __fmaf_rn(th, rs_lo, __fmaf_rn(th, rs_hi, -ph));
        yw[k] = bf16_of_sum(pl, el) | (bf16_of_sum(ph, eh) << 16);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) r[i][k] = yw[k];
    const uint4 a = pack4(r[i]), b = pack4(r[i] + 4);
    if (A.y) store_block(A.y + row * (int64_t)A.K + 16 * j, A.v8_y, a, b);
    if constexpr (kFmt == kFmtNvfp4) {
      const float s_g = __ldg(A.scale), t_g = __fmul_rn(6.0f, s_g);
      uint32_t S;
      bool bad = false;
      const uint2 q = encode_block16(a, b, s_g, t_g, S, bad);
      *reinterpret_cast<uint2 *>(A.q + row * (int64_t)(A.K >> 1) + 8 * j) = q;
      if (kTiled) A.sf[sf_row_part((uint32_t)row, (uint32_t)nblk) + sf_blk_part((uint32_t)j)] = (uint8_t)S;
      else A.sf[row * (int64_t)nblk + j] = (uint8_t)S;
      if (bad) report(A.dev_status, NVFP4_ERR_NONFINITE);
    } else if constexpr (kFmt == kFmtE4m3) {
      top = max(top, block_amax_bits(a, b));
    } else {
      if (block_amax_bits(a, b) >= 0x7F80u) report(A.dev_status, NVFP4_ERR_NONFINITE);
    }
  }
  if constexpr (kFmt == kFmtNvfp4) {
    if (row == 0 && t == 0) {
      const float s_g = __ldg(A.scale);
      if (!(s_g > 0.0f) || !isfinite(s_g)) report(A.dev_status, NVFP4_ERR_INVALID_ARG);
    }
  }
  if constexpr (kFmt == kFmtE4m3) {
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) s_max[warp] = top;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, lane < nwarps ? s_max[lane] : 0u);
    if (top >= 0x7F80u && t == 0) report(A.dev_status, NVFP4_ERR_NONFINITE);
    const float amax = __uint_as_float(top << 16);
    // at least 2^-126, so that 1/s stays finite for rows of subnormal values
    const float s = amax == 0.0f ? 1.0f : fmaxf(__fdiv_rn(amax, 448.0f), 1.17549435e-38f);
    const float inv = __frcp_rn(s);
    if (t == 0) A.scale[row] = s;
#pragma unroll
    for (int i = 0; i < kB; ++i) {
      const int j = t + i * (int)blockDim.x;
      if (j >= nblk) continue;
      uint32_t q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint64_t u = mul_f32x2(bf16x2_to_f32x2(r[i][2 * k]), pair_f32(inv, inv));
        const uint64_t v = mul_f32x2(bf16x2_to_f32x2(r[i][2 * k + 1]), pair_f32(inv, inv));
        q[k] = e4m3x2(__uint_as_float((uint32_t)u), __uint_as_float((uint32_t)(u >> 32))) |
               (e4m3x2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32))) << 16);
      }
      *reinterpret_cast<uint4 *>(A.q + row * (int64_t)A.K + 16 * j) = pack4(q);
    }
  }
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <int kFmt, bool kTiled>
nvfp4_status launch(const Args &a, int64_t rows, cudaStream_t stream) {
  const int nblk = a.K >> 4;
  const int kb = nblk <= 1024 ? 1 : nblk <= 2048 ? 2 : 4;
  const int threads = ((nblk + kb - 1) / kb + 31) / 32 * 32;
  if (kb == 1 && threads <= 384) add_rmsnorm_kernel<kFmt, kTiled, 1, 384, 4><<<(unsigned)rows, threads, 0, stream>>>(a);
  else if (kb == 1) add_rmsnorm_kernel<kFmt, kTiled, 1, 1024, 1><<<(unsigned)rows, threads, 0, stream>>>(a);
  else if (kb == 2) add_rmsnorm_kernel<kFmt, kTiled, 2, 1024, 1><<<(unsigned)rows, threads, 0, stream>>>(a);
  else add_rmsnorm_kernel<kFmt, kTiled, 4, 1024, 1><<<(unsigned)rows, threads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // namespace norm
}  // namespace nvfp4

extern "C" nvfp4_status nvfp4_add_rmsnorm_quantize(const void *x, int64_t ld_x, const void *residual, int64_t ld_res,
                                                   int64_t rows, int64_t K, const void *weight, double eps,
                                                   void *residual_out, int64_t ld_ro, void *y,
                                                   nvfp4_norm_format format, float *scale, uint8_t *q, uint8_t *sf,
                                                   nvfp4_sf_layout sf_layout, int32_t *dev_status,
                                                   cudaStream_t stream) {
  using namespace nvfp4;
  using namespace nvfp4::norm;
  if (rows < 0 || K <= 0 || K % 16 != 0 || K > 65536 || rows > 0x7FFFFFFF) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (format != NVFP4_NORM_BF16 && format != NVFP4_NORM_NVFP4 && format != NVFP4_NORM_E4M3) return NVFP4_ERR_INVALID_ARG;
  if (sf_layout != NVFP4_SF_ROWMAJOR && sf_layout != NVFP4_SF_MMA_TILED) return NVFP4_ERR_INVALID_ARG;
  if (format == NVFP4_NORM_NVFP4 && sf_layout == NVFP4_SF_MMA_TILED && K % 64 != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!(eps >= 0.0) || !(eps < 1e300)) return NVFP4_ERR_INVALID_ARG;
  if (ld_x < K || ld_x % 8 || (residual && (ld_res < K || ld_res % 8)) ||
      (residual_out && (ld_ro < K || ld_ro % 8)))
    return NVFP4_ERR_INVALID_ARG;
  if (rows == 0) return NVFP4_OK;
  // in place only row by row
  if (rows > 1 && residual_out && ((residual_out == x && ld_ro != ld_x) || (residual_out == residual && ld_ro != ld_res)))
    return NVFP4_ERR_INVALID_ARG;
  if (!x || !weight || !aligned(x, 16) || !aligned(weight, 16) || !aligned(residual, 16) ||
      !aligned(residual_out, 16) || !aligned(y, 16))
    return NVFP4_ERR_INVALID_ARG;
  if (format == NVFP4_NORM_BF16 && !y) return NVFP4_ERR_INVALID_ARG;
  if (format != NVFP4_NORM_BF16 && (!scale || !q || !aligned(q, 16) || !aligned(scale, 4))) return NVFP4_ERR_INVALID_ARG;
  if (format == NVFP4_NORM_NVFP4 && !sf) return NVFP4_ERR_INVALID_ARG;
  Args a;
  a.x = static_cast<const uint16_t *>(x);
  a.res = static_cast<const uint16_t *>(residual);
  a.w = static_cast<const uint16_t *>(weight);
  a.res_out = static_cast<uint16_t *>(residual_out);
  a.y = static_cast<uint16_t *>(y);
  a.ld_x = ld_x; a.ld_res = ld_res; a.ld_ro = ld_ro;
  a.K = (int32_t)K;
  a.inv_k = 1.0 / (double)K;
  a.eps = eps;
  a.scale = scale; a.q = q; a.sf = sf; a.dev_status = dev_status;
  a.v8_x = aligned(x, 32) && ld_x % 16 == 0;
  a.v8_res = aligned(residual, 32) && ld_res % 16 == 0;
  a.v8_ro = aligned(residual_out, 32) && ld_ro % 16 == 0;
  a.v8_y = aligned(y, 32);
  a.v8_w = aligned(weight, 32);
  if (format == NVFP4_NORM_BF16) return launch<kFmtNone, false>(a, rows, stream);
  if (format == NVFP4_NORM_E4M3) return launch<kFmtE4m3, false>(a, rows, stream);
  return sf_layout == NVFP4_SF_MMA_TILED ? launch<kFmtNvfp4, true>(a, rows, stream)
                                         : launch<kFmtNvfp4, false>(a, rows, stream);
}
