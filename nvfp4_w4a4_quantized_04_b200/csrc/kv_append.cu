// Append to a paged NVFP4 KV cache: rotate the new tokens' keys (and queries)
// to their positions, quantize keys and values, write them into their slots
// ("Qwen3.8-2.4T-A95B-NVFP4": NVFP4 KV cache, quantized when it is written).
//
// Rotation.  A pair (a, b) of a head becomes (a c - b s, b c + a s) with the
// fp32 cosine and sine of the token's position, rounded to bf16 once, so that
// the 4-bit codes behind it are reproducible: from an interval that holds it,
// or, where the interval's ends round apart, from the products with their errors
// (fma).  The exact form alone, 25 instructions an element against 7, kept the
// kernel from the memory rate.  The block encode is the one of nvfp4_quantize
// with a given global scale.
//
// Traffic: 2 bytes in and 9/16 out per element of k and v, 2 + 2 per
// element of q.  A thread owns 32 elements of one token: the two 16-element
// blocks that the rotation of halves couples (block u and u + rot/32), or two
// neighbouring ones.  It keeps its 32 cosines and sines in registers and walks
// over a chunk of the heads, so that long prompts read the table once per token
// and chunk; the host halves the chunk until there are 1024 threads an SM, so that
// a decode step's few tokens still spread over all SMs (about 1000 tokens end at
// one head a thread).
//
// Measured: 16384 tokens of 32 + 2 x 4 heads of 256: 139 us, 4.5 TB/s (68 % of a
// copy's rate), bound by the loads in flight of 12 warps an SM (168 registers; the
// long scoreboard is the top stall, issue slots 49 %); 1037 tokens of 32 + 2 x 8
// heads of 128: 17 us; 64 tokens 6.3 us, the latency of slot, table, load and store.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "encode.cuh"
#include "host_util.cuh"
#include "kv_paged.cuh"

namespace nvfp4 {
namespace kv {

struct AppendArgs {
  const uint16_t *k, *v, *q;
  uint16_t *q_out;
  int64_t ld_k, ld_v, ld_q, ld_qo;
  const int64_t *slots, *positions;
  const float *rope;
  int64_t rope_rows;
  int32_t rot, tokens, heads_kv, heads_q, D, page_size, chunk;
  int64_t num_pages;
  const float *k_gs, *v_gs;
  uint8_t *k_q, *k_sf, *v_q, *v_sf;
  int32_t *dev_status;
  bool v8_k, v8_v, v8_q, v8_qo;
};

__device__ __forceinline__ float half_f32(uint32_t w, int h) {
  return h ? __uint_as_float(w & 0xFFFF0000u) : __uint_as_float(w << 16);
}

// bf16(a c - b s), rounded once, in 64 bits: the products are exact there, their sum is
// truncated, and what it and the step to fp32 drop goes into the last bit.
__device__ __forceinline__ uint32_t rot_bf16(float a, float c, float b, float s) {
  const double q = (double)b * (double)s, z = __fma_rz((double)a, (double)c, -q);
  const float f = __double2float_rz(z);
  const bool dropped = (double)f != z || __fma_ru((double)a, (double)c, -q) != __fma_rd((double)a, (double)c, -q);
  return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(__float_as_uint(f) | (dropped ? 1u : 0u))));
}

// The same for the usual element: q = b s and r = fma(a, c, -q) are off by less
// than 2^-23 (|q| + |r|) and, as subnormals, 2^-149; where both ends of a wider
// interval round to the same bf16 (all but about one element in 2^12, and those below
// 2^-140), `lo` and `hi` agree.
__device__ __forceinline__ void rot_interval(float a, float c, float b, float s, float &lo, float &hi) {
  const float q = __fmul_rn(b, s), r = __fmaf_rn(a, c, -q);
  const float e = fabsf(q) + 0x1p-118f + fabsf(r);
  lo = __fmaf_rn(e, -0x1p-22f, r);
  hi = __fmaf_rn(e, 0x1p-22f, r);
}

// Rotate the two blocks x[0..7], x[8..15] (bf16 pairs).  Halves: element i of
// the first block with element i of the second.  Pairs: neighbours.
template <bool kPairs>
__device__ __forceinline__ void rotate(uint32_t (&x)[16], const float (&c)[16], const float (&s)[16]) {
  uint32_t y[16], differ = 0;
#pragma unroll
  for (int i = 0; i < (kPairs ? 16 : 8); ++i) {
    // the word pairs (a0, a1), (b0, b1) become words ya, yb
    float a0, a1, b0, b1, c0, c1, s0, s1, l[4], h[4];
    if (kPairs) {
      a0 = half_f32(x[i], 0); b0 = half_f32(x[i], 1); c0 = c[i]; s0 = s[i];
      rot_interval(a0, c0, b0, s0, l[0], h[0]);
      rot_interval(b0, c0, -a0, s0, l[1], h[1]);
      y[i] = bf16x2_of(pair_f32(l[0], l[1]));
      differ |= y[i] ^ bf16x2_of(pair_f32(h[0], h[1]));
    } else {
      a0 = half_f32(x[i], 0); a1 = half_f32(x[i], 1); b0 = half_f32(x[8 + i], 0); b1 = half_f32(x[8 + i], 1);
      c0 = c[2 * i]; c1 = c[2 * i + 1]; s0 = s[2 * i]; s1 = s[2 * i + 1];
      rot_interval(a0, c0, b0, s0, l[0], h[0]);
      rot_interval(a1, c1, b1, s1, l[1], h[1]);
      rot_interval(b0, c0, -a0, s0, l[2], h[2]);
      rot_interval(b1, c1, -a1, s1, l[3], h[3]);
      y[i] = bf16x2_of(pair_f32(l[0], l[1]));
      y[8 + i] = bf16x2_of(pair_f32(l[2], l[3]));
      differ |= (y[i] ^ bf16x2_of(pair_f32(h[0], h[1]))) | (y[8 + i] ^ bf16x2_of(pair_f32(h[2], h[3])));
    }
  }
  if (differ) {
#pragma unroll
    for (int i = 0; i < (kPairs ? 16 : 8); ++i) {
      if (kPairs) {
        const float a = half_f32(x[i], 0), b = half_f32(x[i], 1);
        y[i] = rot_bf16(a, c[i], b, s[i]) | (rot_bf16(b, c[i], -a, s[i]) << 16);
      } else {
        const float a0 = half_f32(x[i], 0), a1 = half_f32(x[i], 1);
        const float b0 = half_f32(x[8 + i], 0), b1 = half_f32(x[8 + i], 1);
        y[i] = rot_bf16(a0, c[2 * i], b0, s[2 * i]) | (rot_bf16(a1, c[2 * i + 1], b1, s[2 * i + 1]) << 16);
        y[8 + i] = rot_bf16(b0, c[2 * i], -a0, s[2 * i]) | (rot_bf16(b1, c[2 * i + 1], -a1, s[2 * i + 1]) << 16);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = y[i];
}

__device__ __forceinline__ void load2(const uint16_t *p, int b0, int b1, bool v8, uint32_t (&x)[16]) {
  uint4 a, b, c, d;
  load_block_rw(p + 16 * b0, v8, a, b);
  load_block_rw(p + 16 * b1, v8, c, d);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  x[8] = c.x; x[9] = c.y; x[10] = c.z; x[11] = c.w; x[12] = d.x; x[13] = d.y; x[14] = d.z; x[15] = d.w;
}

// Blocks b0 and b1 of one token's head into the pool at row `at`.  A block
// with a non-finite element is stored as zeros and reported, so that a cache
// never holds a value that would spread to other queries.
__device__ __forceinline__ void put(const uint32_t (&x)[16], int b0, int b1, float gs, uint8_t *q, uint8_t *sf,
                                    int64_t at, int D, int32_t *dev_status) {
  const float tg = __fmul_rn(6.0f, gs);
  uint2 codes[2];
  uint32_t S[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 a = make_uint4(x[8 * i], x[8 * i + 1], x[8 * i + 2], x[8 * i + 3]);
    const uint4 b = make_uint4(x[8 * i + 4], x[8 * i + 5], x[8 * i + 6], x[8 * i + 7]);
    bool bad = false;
    codes[i] = encode_block16(a, b, gs, tg, S[i], bad);
    if (bad) {
      codes[i] = make_uint2(0, 0);
      S[i] = 0;
      report(dev_status, NVFP4_ERR_NONFINITE);
    }
  }
  uint8_t *to = q + at * (D >> 1), *so = sf + at * (D >> 4);
  if (b1 == b0 + 1) {
    *reinterpret_cast<uint4 *>(to + 8 * b0) = make_uint4(codes[0].x, codes[0].y, codes[1].x, codes[1].y);
    *reinterpret_cast<uint16_t *>(so + b0) = (uint16_t)(S[0] | S[1] << 8);
  } else {
    *reinterpret_cast<uint2 *>(to + 8 * b0) = codes[0];
    *reinterpret_cast<uint2 *>(to + 8 * b1) = codes[1];
    so[b0] = (uint8_t)S[0];
    so[b1] = (uint8_t)S[1];
  }
}

template <bool kPairs>
__global__ void __launch_bounds__(128, 3) append_kernel(const AppendArgs A) {
  const int units = A.D >> 5;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (int64_t)A.tokens * units) return;
  const int64_t token = i / units;
  const int u = (int)(i - token * units);
  const bool turn = u < (A.rot >> 5);
  const int b0 = (turn && !kPairs) ? u : 2 * u;
  const int b1 = (turn && !kPairs) ? u + (A.rot >> 5) : 2 * u + 1;
  float c[16], s[16];
  if (A.rot) {
    const int64_t pos = A.positions[token];
    if (pos < 0 || pos >= A.rope_rows) {
      if (u == 0 && blockIdx.y == 0) report(A.dev_status, NVFP4_ERR_INDEX);
      return;
    }
    if (turn) {
      const float4 *t = reinterpret_cast<const float4 *>(A.rope + pos * A.rot + 16 * u);
      const float4 *w = reinterpret_cast<const float4 *>(A.rope + pos * A.rot + (A.rot >> 1) + 16 * u);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 a = __ldg(t + j), b = __ldg(w + j);
        c[4 * j] = a.x; c[4 * j + 1] = a.y; c[4 * j + 2] = a.z; c[4 * j + 3] = a.w;
        s[4 * j] = b.x; s[4 * j + 1] = b.y; s[4 * j + 2] = b.z; s[4 * j + 3] = b.w;
      }
    }
  }
  const int all = A.heads_q + 2 * A.heads_kv;
  const int h0 = blockIdx.y * A.chunk, h1 = min(all, h0 + A.chunk);
  int64_t page = 0;
  int row = 0;
  bool keep = false;
  float kg = 1.0f, vg = 1.0f;
  if (h1 > A.heads_q) {
    const int64_t slot = A.slots[token];
    keep = split_slot(slot, A.num_pages, A.page_size, page, row);
    if (!keep && slot >= 0 && u == 0 && blockIdx.y == gridDim.y - 1) report(A.dev_status, NVFP4_ERR_INDEX);
    kg = __ldg(A.k_gs);
    vg = __ldg(A.v_gs);
    if (i == 0 && blockIdx.y == gridDim.y - 1 && (!(kg > 0.0f) || !isfinite(kg) || !(vg > 0.0f) || !isfinite(vg)))
      report(A.dev_status, NVFP4_ERR_INVALID_ARG);
  }
  // without a slot only the query heads are walked
  const int end = keep ? h1 : min(h1, A.heads_q);
  auto load_head = [&](int h, uint32_t (&x)[16]) {
    if (h < A.heads_q) load2(A.q + token * A.ld_q + (int64_t)h * A.D, b0, b1, A.v8_q, x);
    else if (h < A.heads_q + A.heads_kv) load2(A.k + token * A.ld_k + (int64_t)(h - A.heads_q) * A.D, b0, b1, A.v8_k, x);
    else load2(A.v + token * A.ld_v + (int64_t)(h - A.heads_q - A.heads_kv) * A.D, b0, b1, A.v8_v, x);
  };
  uint32_t next[16];
  if (h0 < end) load_head(h0, next);
  for (int h = h0; h < end; ++h) {
    uint32_t x[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = next[k];
    if (h + 1 < end) load_head(h + 1, next);            // on its way while this head is turned and encoded
    if (turn && h < A.heads_q + A.heads_kv) rotate<kPairs>(x, c, s);
    if (h < A.heads_q) {
      uint16_t *o = A.q_out + token * A.ld_qo + (int64_t)h * A.D;
      store_block(o + 16 * b0, A.v8_qo, make_uint4(x[0], x[1], x[2], x[3]), make_uint4(x[4], x[5], x[6], x[7]));
      store_block(o + 16 * b1, A.v8_qo, make_uint4(x[8], x[9], x[10], x[11]), make_uint4(x[12], x[13], x[14], x[15]));
    } else if (h < A.heads_q + A.heads_kv) {
      put(x, b0, b1, kg, A.k_q, A.k_sf, pool_row(page, A.heads_kv, A.page_size, h - A.heads_q, row), A.D, A.dev_status);
    } else {
      put(x, b0, b1, vg, A.v_q, A.v_sf, pool_row(page, A.heads_kv, A.page_size, h - A.heads_q - A.heads_kv, row), A.D,
          A.dev_status);
    }
  }
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace kv
}  // namespace nvfp4

extern "C" nvfp4_status nvfp4_kv_append(const void *k, int64_t ld_k, const void *v, int64_t ld_v, int64_t tokens,
                                        int heads, int head_dim, const int64_t *slots, const void *q, int64_t ld_q,
                                        int q_heads, void *q_out, int64_t ld_qo, const int64_t *positions,
                                        const float *rope, int64_t rope_rows, int rot_dim, int interleaved,
                                        const float *k_gs, const float *v_gs, uint8_t *k_q, uint8_t *k_sf,
                                        uint8_t *v_q, uint8_t *v_sf, int64_t num_pages, int page_size,
                                        int32_t *dev_status, cudaStream_t stream) {
  using namespace nvfp4;
  using namespace nvfp4::kv;
  if (tokens < 0 || tokens > 0x7FFFFFFF / 64 || heads < 1 || heads > 1024 || head_dim < 32 || head_dim > 512 ||
      head_dim % 32 != 0)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (page_size < kPageGranule || page_size % kPageGranule != 0 || page_size > 65536 || num_pages < 0 ||
      num_pages > 0x7FFFFFFF)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 32 != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (q && (q_heads < 1 || q_heads > 4096)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if ((interleaved != 0 && interleaved != 1) || (rot_dim > 0 && (!rope || rope_rows < 1))) return NVFP4_ERR_INVALID_ARG;
  const int64_t nkv = (int64_t)heads * head_dim, nq = q ? (int64_t)q_heads * head_dim : 0;
  if (ld_k < nkv || ld_v < nkv || ld_k % 8 || ld_v % 8 || (q && (ld_q < nq || ld_qo < nq || ld_q % 8 || ld_qo % 8)))
    return NVFP4_ERR_INVALID_ARG;
  if (tokens == 0) return NVFP4_OK;
  if (tokens > 1 && q && q_out == q && ld_qo != ld_q) return NVFP4_ERR_INVALID_ARG;     // in place only row by row
  if (!k || !v || !slots || !k_gs || !v_gs || (rot_dim > 0 && !positions) || (q && !q_out)) return NVFP4_ERR_INVALID_ARG;
  if (num_pages > 0 && (!k_q || !k_sf || !v_q || !v_sf)) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) || !aligned(k_q, 16) ||
      !aligned(v_q, 16) || !aligned(k_sf, 16) || !aligned(v_sf, 16) || !aligned(rope, 16) || !aligned(slots, 8) || !aligned(positions, 8))
    return NVFP4_ERR_INVALID_ARG;
  AppendArgs a;
  a.k = static_cast<const uint16_t *>(k);
  a.v = static_cast<const uint16_t *>(v);
  a.q = static_cast<const uint16_t *>(q);
  a.q_out = static_cast<uint16_t *>(q_out);
  a.ld_k = ld_k; a.ld_v = ld_v; a.ld_q = ld_q; a.ld_qo = ld_qo;
  a.slots = slots; a.positions = positions; a.rope = rope; a.rope_rows = rope_rows;
  a.rot = rot_dim; a.tokens = (int32_t)tokens; a.heads_kv = heads; a.heads_q = q ? q_heads : 0;
  a.D = head_dim; a.page_size = page_size; a.num_pages = num_pages;
  a.k_gs = k_gs; a.v_gs = v_gs; a.k_q = k_q; a.k_sf = k_sf; a.v_q = v_q; a.v_sf = v_sf;
  a.dev_status = dev_status;
  a.v8_k = aligned(k, 32) && ld_k % 16 == 0;
  a.v8_v = aligned(v, 32) && ld_v % 16 == 0;
  a.v8_q = aligned(q, 32) && ld_q % 16 == 0;
  a.v8_qo = aligned(q_out, 32) && ld_qo % 16 == 0;
  const int64_t threads = tokens * (head_dim / 32);
  const int all = a.heads_q + 2 * heads;
  int chunk = all < 16 ? all : 16;
  while (chunk > 1 && threads * ((all + chunk - 1) / chunk) < (int64_t)host::sm_count() * 1024) chunk = (chunk + 1) / 2;
  a.chunk = chunk;
  const dim3 grid((unsigned)((threads + 127) / 128), (unsigned)((all + chunk - 1) / chunk));
  if (interleaved) append_kernel<true><<<grid, 128, 0, stream>>>(a);
  else append_kernel<false><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
