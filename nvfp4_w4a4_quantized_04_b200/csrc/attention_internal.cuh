// What the decode and the prefill form of the paged attention share on top of
// attention.cuh: constants, the row scaling of Q, the output store, and the
// prefill launcher that attention.cu calls.
#pragma once

#include "attention.cuh"

namespace nvfp4 {
namespace attn {

constexpr float kFloor = -3.40282347e38f; // running maximum before the first key: the lowest fp32, below any score
constexpr int kMaxBatch = 4096;

// The power of two that brings a row of Q to f16: 2^(14 - e) for a row whose
// largest element has biased exponent e; 1 for zero, inf, NaN rows and for
// rows below 2^-112, where the factor would leave fp32.
__device__ __forceinline__ void row_power(int e, float &up, float &down) {
  const bool plain = e < 15 || e == 255;
  up = plain ? 1.0f : __uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23);
  down = plain ? 1.0f : __uint_as_float((uint32_t)(e - 14) << 23);
}

// Both global scales finite and above 0.
__device__ __forceinline__ bool scales_ok(const Args &A) {
  const float k = __ldg(A.k_gs), v = __ldg(A.v_gs);
  return k > 0.0f && k <= 3.40282347e38f && v > 0.0f && v <= 3.40282347e38f;
}
// The factor from a row's f16 score to log2 units.  Never 0, so that a masked score
// of -inf stays -inf; NaN with a bad global scale, so that it shows in the output.
__device__ __forceinline__ float score_scale(const Args &A, float k_gs, float down) {
  const float x = A.scale_log2 * k_gs * kScaleFix * down;
  return x < 1.17549435e-38f ? 1.17549435e-38f : x;
}

// A score's exponent against the running maximum m.  Right after m was raised the
// scaled score is rounded as m was, so that no weight exceeds 1: the fused form is
// off from m by the rounding of m itself, which for scores beyond 2^27 is an
// exponent that f16 does not hold.
template <bool kRaised>
__device__ __forceinline__ float exponent(float s, float sc, float m) {
  return kRaised ? __fsub_rn(__fmul_rn(s, sc), m) : fmaf(s, sc, -m);
}

// Four output elements times f at (row `at`, element d).
__device__ __forceinline__ void store_out(const Args &A, int64_t at, int D, int d, float4 acc, float f) {
  if (A.out_bf16) {
    uint32_t lo, hi;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(acc.y * f), "f"(acc.x * f));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(acc.w * f), "f"(acc.z * f));
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(A.out) + at * D + d) = make_uint2(lo, hi);
  } else {
    *reinterpret_cast<float4 *>(static_cast<float *>(A.out) + at * D + d) =
        make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
  }
}

// Launch that may be set up while the kernel before it on the stream still
// runs; the kernel itself waits for it (griddepcontrol.wait) before it reads.
template <typename Kernel, typename Params>
inline bool launch_behind(Kernel kern, dim3 grid, int threads, int smem, cudaStream_t stream, const Params &p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess;
}

inline int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// Prefill form: sequences with more than row_floor rows.
int64_t prefill_workspace(int batch, int64_t max_query, int group, int D);
nvfp4_status launch_prefill(const Args &a, int D, int row_floor, uint8_t *ws, cudaStream_t stream);

}  // namespace attn
}  // namespace nvfp4
