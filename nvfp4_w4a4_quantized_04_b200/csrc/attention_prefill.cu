// Attention over the paged NVFP4 cache: prefill form (sm_100a), for sequences
// with many rows (row = query * group + head of the KV group).
//
// Same mathematics as the decode form (attention.cu).  Here 128 rows share
// every key, so the products are what bounds it, and they run on the 5th
// generation tensor cores:
//   S [128 rows, T keys]  = Q K^T    tcgen05.mma kind::f16, A = Q in tensor memory,
//   O [128 rows, D]      += P V      A = P in tensor memory,
// with K and V dequantized to f16 (exactly) once per tile into shared memory.
//
// Roles of a CTA (one per SM):
//  * warps 0-7, softmax: two threads per row, each with half of a tile's keys.
//    They put Q into tensor memory (f16, a power of two per row), turn S into P
//    (f16, written over their own half of S), keep the running maximum and sum,
//    and store O at the end of an item.  The maximum is raised, and O in tensor
//    memory rescaled, only when a score exceeds it by more than 2^8.
//  * warps 8-15, converters: cache codes -> f16 tiles in shared memory in a
//    ring of six 16 or 32 KB buffers (K and V in turn).  A warp takes 8 tokens
//    x 4 sixteen-byte pieces at a time: the 16-byte shared stores of 8 lanes
//    fall on the 8 different positions of the 128-byte swizzle.  K and V tiles
//    have one layout, [64-element chunk][token][128 bytes]: K-major for S (keys
//    are N) and N-major for O (keys are K), so V needs no transposition.  The
//    codes of a tile are loaded a whole tile ahead of their conversion, and the
//    page ids a tile ahead of that.
//  * warp 16, one thread issues the MMAs: S of tile i + 1 goes ahead of P V of
//    tile i, so the tensor cores work while the softmax runs.
// Keeping Q in tensor memory instead of shared memory halves what the first
// product reads from shared memory, whose bandwidth the converters' stores and
// the B operands already fill (256 cycles each for K and V, stored and read,
// of the about 1024 that the MMAs of a tile take).
//
// Split: a plan kernel lists the (sequence, row block) pairs with their key
// tiles; the line of all (pair, head, tile) steps is cut evenly over the CTAs,
// and items that several CTAs share are joined by a third kernel.
#include "attention.cuh"
#include "attention_internal.cuh"
#include "gemm_common.cuh"
#include "host_util.cuh"

namespace nvfp4 {
namespace attn {

using gemm::mbar_arrive;
using gemm::mbar_init;
using gemm::mbar_wait_warp;
using gemm::tc_commit;
using gemm::tc_fence_after;
using gemm::tc_fence_before;

constexpr int kRows = 128;
constexpr int kPlanThreads = 1024;
constexpr int kSoft = 8, kConv = 8;           // softmax and converter warps
constexpr int W_CONV = kSoft, W_MMA_P = kSoft + kConv;
constexpr int kPreThreads = (W_MMA_P + 4) * 32;   // five warpgroups; the last has one working warp
// Registers per thread after the roles part (setmaxnreg moves them between
// warpgroups): 256 x 128 + 256 x 80 + 128 x 56 = 60416 of the 640 x 96 = 61440
// that the block is launched with.
constexpr int kLaunchRegs = 96, kSoftRegs = 128, kConvRegs = 80, kRestRegs = 56;
static_assert(32 * (kSoft * kSoftRegs + kConv * kConvRegs + 4 * kRestRegs) <= kPreThreads * kLaunchRegs, "registers");
constexpr int kBufs = 6;
// What an item costs besides its tiles (Q in, the first S, O out), in tiles:
// the line that is cut over the CTAs counts it, so that a CTA with many short
// items takes no longer than the others.
constexpr int kItemCost = 2;

template <int D> struct Pre {
  static constexpr int T = D == 256 ? 64 : 128;         // keys per tile
  static constexpr int kTile = T * D * 2;               // bytes of one f16 tile
  static constexpr uint32_t kO = 0, kQ = D, kS = D + D / 2;   // tensor memory columns
  static constexpr uint32_t kCols = 512;
  static constexpr int kBar = kBufs * kTile;
  // kv_full[6], kv_empty[6], s_full[2], p_full[2], pv_done, o_done, q_ready, drain
  static constexpr int kNumBars = 2 * kBufs + 2 + 2 + 4;
  static constexpr int kMisc = kBar + kNumBars * 8;      // tmem base, abort flag, bad-page tags[8]
  static constexpr int kXch = kMisc + 8 + 32;            // [2][2][128] floats between a row's two threads
  static constexpr int kBytes = kXch + 2 * 2 * kRows * 4 + 1024;
  static_assert(kS + 2 * T <= kCols, "tensor memory");
  static_assert(kBytes <= 232448, "shared memory");
};

struct PlanArgs {
  Args a;
  int32_t row_floor;       // sequences with at most this many rows are left to the decode kernel
  int32_t tile;
  int32_t grid;
  int32_t *count;          // [0] entries, [1] cost per CTA, [2] total cost
  int32_t *prefix;         // [entries + 1] cost of all heads before entry e: (tiles + kItemCost) each
  int2 *entry;             // [entries] (sequence, row block)
  int32_t *start;          // [grid] entry in which CTA c begins
  float *ws_ml, *ws_o;     // parts, as in the decode form, R = 128
};

// Key tiles of one item: up to the last key that the block's last row sees,
// and one (all masked) for a block that sees none, so that its rows are written.
__device__ __forceinline__ int block_steps(const Args &A, const Seq &s, int block, int T) {
  const int rows = s.queries * A.group;
  const int last = min(rows, (block + 1) * kRows) - 1;
  const int64_t see = kv::visible_keys(s.len, s.queries, last / A.group, A.causal != 0);
  return max(1, (int)((see + T - 1) / T));
}

__device__ __forceinline__ int seq_blocks(const PlanArgs &P, const Seq &s) {
  const int rows = s.queries * P.a.group;
  return rows > P.row_floor ? (rows + kRows - 1) / kRows : 0;
}

// Inclusive scan over the block of kPlanThreads threads.
__device__ __forceinline__ int block_scan(int v, int *scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += n;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += scratch[w];
  return v + before;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs P) {
  __shared__ int32_t first[kMaxBatch + 1];      // first entry of each sequence
  __shared__ int scratch[32], carry;
  const Args &A = P.a;
  const int t = threadIdx.x;
  bool bad = false;
  for (int b = t; b < A.batch; b += kPlanThreads) bad |= !offsets_ok(A, b);
  if (__syncthreads_or(bad)) {
    if (t == 0) {
      P.count[0] = 0; P.count[1] = 0; P.count[2] = 0;
      report(A.dev_status, NVFP4_ERR_INDEX);
    }
    return;
  }
  if (t == 0) carry = 0;
  __syncthreads();
  for (int b0 = 0; b0 < A.batch; b0 += kPlanThreads) {
    const int b = b0 + t;
    const int n = b < A.batch ? seq_blocks(P, load_seq(A, b)) : 0;
    const int incl = block_scan(n, scratch);
    const int base = carry;
    if (b < A.batch) first[b] = base + incl - n;
    __syncthreads();
    if (t == kPlanThreads - 1) carry = base + incl;
    __syncthreads();
  }
  const int entries = carry;
  if (t == 0) first[A.batch] = entries;
  __syncthreads();
  if (t == 0) carry = 0;
  __syncthreads();
  for (int e0 = 0; e0 < entries; e0 += kPlanThreads) {
    const int e = e0 + t;
    int n = 0;
    if (e < entries) {
      const int b = upper_group(first, A.batch, e);
      const int block = e - first[b];
      n = (block_steps(A, load_seq(A, b), block, P.tile) + kItemCost) * A.heads_kv;
      P.entry[e] = make_int2(b, block);
    }
    const int incl = block_scan(n, scratch);
    const int base = carry;
    if (e < entries) P.prefix[e] = base + incl - n;
    __syncthreads();
    if (t == kPlanThreads - 1) carry = base + incl;
    __syncthreads();
  }
  const int total = carry;
  const int per = (int)kv::steps_per_cta(total, P.grid, 1);
  if (t == 0) {
    P.prefix[entries] = total;
    P.count[0] = entries;
    P.count[1] = per;
    P.count[2] = total;
  }
  __syncthreads();                              // P.prefix is read back below
  for (int c = t; c < P.grid; c += kPlanThreads) {
    const int64_t pos = (int64_t)c * per;
    P.start[c] = pos < total ? upper_group(P.prefix, entries, pos) : 0;
  }
}

// One CTA's walk over its part of the line, the same in every role.
struct Segment {
  int head, block, s0, s1, steps;      // tiles [s0, s1) of the item's `steps`
  int b, nrows, item_start;
  Seq seq;
};

struct Walk {
  int pos, end, entry, per;
  __device__ __forceinline__ Walk(const PlanArgs &P) {
    per = P.count[1];
    const int total = P.count[2];
    pos = (int)min((int64_t)total, (int64_t)blockIdx.x * per);
    end = (int)min((int64_t)total, (int64_t)pos + per);
    entry = P.start[blockIdx.x];
  }
  __device__ __forceinline__ bool next(const PlanArgs &P, Segment &g) {
    while (pos < end) {
      while (P.prefix[entry + 1] <= pos) ++entry;
      const int2 e = P.entry[entry];
      const int base = P.prefix[entry];
      const int cost = (P.prefix[entry + 1] - base) / P.a.heads_kv;
      g.steps = cost - kItemCost;
      g.head = (pos - base) / cost;
      g.item_start = base + g.head * cost;
      kv::item_part(blockIdx.x, per, g.item_start, kItemCost, g.steps, g.s0, g.s1);
      pos = min(end, g.item_start + cost);
      if (g.s0 >= g.s1) continue;      // only the item's fixed cost falls into this range
      g.b = e.x;
      g.block = e.y;
      g.seq = load_seq(P.a, e.x);
      g.nrows = min(kRows, g.seq.queries * P.a.group - g.block * kRows);
      return true;
    }
    return false;
  }
};

// 64 columns of this warp's lanes, complete on return.
__device__ __forceinline__ void tm_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,"
      "%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr) : "memory");
}

__device__ __forceinline__ void tm_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr) : "memory");
}

__device__ __forceinline__ void tm_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr) : "memory");
}

__device__ __forceinline__ void tm_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
         "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
         "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
         "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
      :: "r"(d), "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

// kind::f16: fp32 D, f16 A (K-major) and B; bit 16: B is N-major.
__device__ __forceinline__ uint32_t idesc(int n, bool n_major) {
  return (1u << 4) | (n_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}

// N-major tile, 128-byte swizzle: 64 elements of N per 128-byte row (one row
// per K), 8 rows of K 1024 bytes apart (stride), the next 64 of N `chunk`
// bytes on (leading).
__device__ __forceinline__ uint64_t desc_n_major(uint32_t addr, uint32_t chunk) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(chunk >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Packed pairs of fp32 (first in the low word).
__device__ __forceinline__ uint64_t pair_f32(float lo, float hi) {
  return ((uint64_t)__float_as_uint(hi) << 32) | __float_as_uint(lo);
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Column of P's k-th 16 keys in a tile's S buffer: each half of the keys lies
// at the start of its half of S.
template <int T>
__device__ __forceinline__ uint32_t p_col(int k) {
  constexpr int kHalf = T / 32;                           // 16-key steps per half
  return (k / kHalf) * (T / 2) + (k % kHalf) * 8;
}

// Barrier of the two warps that share 32 rows.
__device__ __forceinline__ void pair_sync(int quadrant) {
  asm volatile("bar.sync %0, 64;" :: "r"(1 + quadrant) : "memory");
}

template <int N>
__device__ __forceinline__ void tm_ld(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 64) tm_ld64(taddr, r);
  else tm_ld32(taddr, r);
}

// N / 2 columns of packed f16 pairs.
__device__ __forceinline__ void tm_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
         "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
template <int N>
__device__ __forceinline__ void tm_st(uint32_t taddr, const uint32_t (&v)[N]) {
  if constexpr (N == 32) tm_st32(taddr, v);
  else tm_st16(taddr, v);
}

template <int D>
__global__ void __launch_bounds__(kPreThreads, 1) prefill_kernel(const PlanArgs P) {
  using L = Pre<D>;
  constexpr int T = L::T;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const Args &A = P.a;
  const uint32_t sbase = smem_addr(smem);
  const uint32_t kv_full = sbase + L::kBar, kv_empty = kv_full + 8 * kBufs, s_full = kv_empty + 8 * kBufs;
  const uint32_t p_full = s_full + 16, pv_done = p_full + 16, o_done = pv_done + 8, q_ready = o_done + 8;
  const uint32_t drain = q_ready + 8;
  volatile uint32_t *tmem_holder = reinterpret_cast<volatile uint32_t *>(smem + L::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);
  volatile int *bad_tag = reinterpret_cast<volatile int *>(smem + L::kMisc + 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < 8; ++i) bad_tag[i] = 0;
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(kv_full + 8 * i, kConv * 32);
      mbar_init(kv_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, kSoft * 32);
    }
    mbar_init(pv_done, 1);
    mbar_init(o_done, 1);
    mbar_init(q_ready, kSoft * 32);
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == W_MMA_P) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_addr((const void *)tmem_holder)), "r"(L::kCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  if (warp >= W_MMA_P) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kRestRegs));
    if (warp == W_MMA_P) {
    // ================================================================ MMA issuer
    // Buffers in the order of use: K of the first tile, then per tile i the K
    // of tile i + 1 (if any) and the V of tile i.
    Walk walk(P);
    Segment G = {};
    uint32_t buf = 0, tile = 0, item = 0;
    bool ok = true;
    auto qk = [&](uint32_t t) -> bool {             // S of tile t (global count) from the next buffer
      const uint32_t x = buf % kBufs;
      if (!mbar_wait_warp(kv_full + 8 * x, (buf / kBufs) & 1, abort_flag, A.dev_status)) return false;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t at = sbase + x * L::kTile;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ts(tmem + L::kS + (t & 1) * T, tmem + L::kQ + 8 * k,
                 gemm::desc_sw128(at + (k >> 2) * (T * 128)) + 2 * (k & 3), idesc(T, false), k > 0);
        tc_commit(kv_empty + 8 * x);
        tc_commit(s_full + 8 * (t & 1));
      }
      __syncwarp();
      ++buf;
      return true;
    };
    while (ok && walk.next(P, G)) {
      if (!mbar_wait_warp(q_ready, item & 1, abort_flag, A.dev_status)) { ok = false; break; }
      tc_fence_after();
      const int n = G.s1 - G.s0;
      if (!qk(tile)) { ok = false; break; }
      for (int i = 0; i < n; ++i, ++tile) {
        if (i + 1 < n) {
          // S buffer (tile + 1) & 1 held P of tile - 1: wait until that was read
          if (i > 0 && !mbar_wait_warp(pv_done, (tile - 1) & 1, abort_flag, A.dev_status)) { ok = false; break; }
          if (!qk(tile + 1)) { ok = false; break; }
        }
        if (!mbar_wait_warp(p_full + 8 * (tile & 1), (tile >> 1) & 1, abort_flag, A.dev_status)) { ok = false; break; }
        const uint32_t x = buf % kBufs;
        if (!mbar_wait_warp(kv_full + 8 * x, (buf / kBufs) & 1, abort_flag, A.dev_status)) { ok = false; break; }
        tc_fence_after();
        if (lane == 0) {
          const uint32_t at = sbase + x * L::kTile;
#pragma unroll
          for (int k = 0; k < T / 16; ++k)
            mma_ts(tmem + L::kO, tmem + L::kS + (tile & 1) * T + p_col<T>(k), desc_n_major(at + k * 2048, T * 128),
                   idesc(D, true), i > 0 || k > 0);
          tc_commit(kv_empty + 8 * x);
          tc_commit(pv_done);
          if (i + 1 == n) tc_commit(o_done);
        }
        __syncwarp();
        ++buf;
      }
      ++item;
    }
    if (lane == 0) {
      tc_commit(drain);
      const long long t0 = clock64();
      while (!gemm::mbar_try_wait(drain, 0) && clock64() - t0 < gemm::kWaitBudgetCycles) {}
    }
    __syncwarp();
    }
  } else if (warp >= W_CONV) {
    // ================================================================ converters
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kConvRegs));
    Walk walk(P);
    Segment G = {};
    // A warp takes 16 tokens (8 with D = 256) of a tile, all on one page; a lane
    // kPer neighbouring 16-byte pieces of one token.
    constexpr int kPer = D == 64 ? 1 : 2;
    constexpr int kTok = T / kConv;                       // tokens per warp
    const int w = __shfl_sync(0xffffffffu, warp - W_CONV, 0);
    const int t_lane = lane % kTok, p_lane = (lane / kTok) * kPer;
    const int t = w * kTok + t_lane;
    uint8_t *const dst = smem + (p_lane >> 1) * (T * 128) + t * 128;
    const int lane_q = t_lane * (D / 2) + p_lane * 16, lane_s = t_lane * (D / 16) + p_lane * 2;
    uint32_t buf = 0, tile = 0;
    bool ok = true;
    struct Piece { uint32_t code[4 * kPer], scale; };
    Piece next_k, next_v;                                 // loaded, not yet converted
    int32_t page = -1;                                    // page of the tile whose rows are next
    int64_t row = -1, row_prev = -1;                      // pool row of that tile's first token, and of the one before
    auto fetch_page = [&](int i) {                        // i: tile of the sequence
      const int tok = i * T + w * kTok;
      page = -1;
      if (i < G.s1 && tok < G.seq.len)
        page = __ldg(A.table + (int64_t)G.b * A.max_pages + fast_div((uint32_t)tok, A.by_page));
    };
    auto row_of = [&](int i, uint32_t tag) {
      const int tok = i * T + w * kTok;
      row_prev = row;
      row = -1;
      if (i < G.s1 && tok < G.seq.len) {
        if (kv::page_ok(page, A.num_pages)) {
          const int in_page = tok - (int)fast_div((uint32_t)tok, A.by_page) * A.page_size;
          row = kv::pool_row(page, A.heads_kv, A.page_size, G.head, in_page);
        } else {
          report(A.dev_status, NVFP4_ERR_INDEX);
          bad_tag[tag & 7] = (int)tag + 1;
        }
      }
    };
    // Tokens past the sequence's end on its last page come along: their codes
    // are finite, whatever the memory held, and their scores are masked.
    auto load = [&](Piece &x, const uint8_t *q, const uint8_t *sf, int64_t at) {
      if (at >= 0) {
        const uint8_t *c = q + at * (D / 2) + lane_q, *s = sf + at * (D / 16) + lane_s;
        if constexpr (kPer == 2) {
          asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(x.code[0]), "=r"(x.code[1]), "=r"(x.code[2]), "=r"(x.code[3]) : "l"(c));
          asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(x.code[4]), "=r"(x.code[5]), "=r"(x.code[6]), "=r"(x.code[7]) : "l"(c + 16));
          x.scale = __ldg(reinterpret_cast<const uint32_t *>(s));
        } else {
          asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(x.code[0]), "=r"(x.code[1]), "=r"(x.code[2]), "=r"(x.code[3]) : "l"(c));
          x.scale = __ldg(reinterpret_cast<const uint16_t *>(s));
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4 * kPer; ++k) x.code[k] = 0;
        x.scale = 0;
      }
    };
    auto put = [&](const Piece &y) -> bool {              // convert into the next buffer
      const uint32_t x = buf % kBufs;
      if (buf >= kBufs && !mbar_wait_warp(kv_empty + 8 * x, ((buf / kBufs) - 1) & 1, abort_flag, A.dev_status))
        return false;
#pragma unroll
      for (int p = 0; p < kPer; ++p) {
        const uint32_t s0 = e4m3_pair_f16x2(__byte_perm(y.scale, 0, p ? 0x4242 : 0x4040));
        const uint32_t s1 = e4m3_pair_f16x2(__byte_perm(y.scale, 0, p ? 0x4343 : 0x4141));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t s = k < 2 ? s0 : s1, c = y.code[4 * p + k];
          const uint4 v = make_uint4(mul_f16x2(e2m1x2_f16x2<0>(c), s), mul_f16x2(e2m1x2_f16x2<1>(c), s),
                                     mul_f16x2(e2m1x2_f16x2<2>(c), s), mul_f16x2(e2m1x2_f16x2<3>(c), s));
          const int pos = (kPer == 2 ? p : p_lane & 1) * 4 + k;
          *reinterpret_cast<uint4 *>(dst + x * L::kTile + ((pos ^ (t & 7)) << 4)) = v;
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(kv_full + 8 * x);
      ++buf;
      return true;
    };
    while (ok && walk.next(P, G)) {
      const int n = G.s1 - G.s0;
      // K of tile 0; then K of tile 1 and V of tile 0 on their way, the page of tile 2
      fetch_page(G.s0);
      row_of(G.s0, tile);
      load(next_k, A.k_q, A.k_sf, row);
      fetch_page(G.s0 + 1);
      if (!put(next_k)) break;
      row_of(G.s0 + 1, tile + 1);
      load(next_k, A.k_q, A.k_sf, row);
      load(next_v, A.v_q, A.v_sf, row_prev);
      fetch_page(G.s0 + 2);
      for (int i = 0; i < n; ++i, ++tile) {
        // K of tile i + 1, V of tile i; each register set is refilled for the next tile at once
        if (i + 1 < n && !put(next_k)) { ok = false; break; }
        row_of(G.s0 + i + 2, tile + 2);
        load(next_k, A.k_q, A.k_sf, row);
        fetch_page(G.s0 + i + 3);
        if (!put(next_v)) { ok = false; break; }
        load(next_v, A.v_q, A.v_sf, row_prev);
      }
    }
  } else {
    // ================================================================ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kSoftRegs));
    Walk walk(P);
    Segment G = {};
    constexpr int kHalf = T / 2;                          // keys of a tile per thread
    const int quad = warp & 3, side = warp >> 2;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const int r = 32 * quad + lane;                       // row of the block
    volatile float *xch = reinterpret_cast<volatile float *>(smem + L::kXch);
    const float kgs = __ldg(A.k_gs), vgs = __ldg(A.v_gs);
    uint32_t tile = 0, item = 0;
    // A wait that gives up (abort) does not end the loop: the two warps of a row
    // stay in step, every later wait returns at once, and nothing more is stored.
    bool ok = true;
    uint32_t qw[D / 4];                                   // this thread's half of its row of Q, bf16
    auto load_q = [&](const Segment &g) {
      const int row = g.block * kRows + r, qi = row / A.group, h = g.head * A.group + row - qi * A.group;
      if (r < g.nrows) {
        const uint16_t *q = A.q + (int64_t)(g.seq.first + qi) * A.ld_q + (int64_t)h * D + side * (D / 2);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint4 v = __ldg(reinterpret_cast<const uint4 *>(q + 8 * i));
          qw[4 * i] = v.x; qw[4 * i + 1] = v.y; qw[4 * i + 2] = v.z; qw[4 * i + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 4; ++i) qw[i] = 0;
      }
    };
    bool more = walk.next(P, G);
    if (more) load_q(G);
    while (more) {
      // ---- Q into tensor memory, each thread half of its row
      const bool live = r < G.nrows;
      const int row = G.block * kRows + r, qi = row / A.group, h = G.head * A.group + row - qi * A.group;
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < D / 4; ++i) top = __vmaxu2(top, qw[i] & 0x7FFF7FFFu);
      top = max(top & 0xFFFFu, top >> 16);
      xch[side * kRows + r] = __uint_as_float(top << 16);
      pair_sync(quad);
      top = max(top, __float_as_uint(xch[(side ^ 1) * kRows + r]) >> 16);
      pair_sync(quad);
      float up, down;
      row_power((int)(top >> 7), up, down);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)
          v[k] = pack_f16x2(__uint_as_float(qw[16 * c + k] << 16) * up, __uint_as_float(qw[16 * c + k] & 0xFFFF0000u) * up);
        tm_st16(tmem + lanes + L::kQ + side * (D / 4) + 16 * c, v);
      }
      tm_wait_st();
      tc_fence_before();
      mbar_arrive(q_ready);
      // never 0, so that a masked score of -inf stays -inf
      const float sc = fmaxf(A.scale_log2 * kgs * kScaleFix * down, 1.17549435e-38f);
      const int limit = live ? (int)kv::visible_keys(G.seq.len, G.seq.queries, qi, A.causal != 0) : 0;
      float m = kFloor, l = 0.0f;
      const int n = G.s1 - G.s0;
      for (int i = 0; i < n; ++i, ++tile) {
        const uint32_t x = tile & 1;
        ok &= mbar_wait_warp(s_full + 8 * x, (tile >> 1) & 1, abort_flag, A.dev_status);
        tc_fence_after();
        const uint32_t st = tmem + lanes + L::kS + x * T + side * kHalf;
        uint32_t s[kHalf];
        tm_ld<kHalf>(st, s);
        const int tok0 = (G.s0 + i) * T + side * kHalf;
        const int left = limit - tok0;                    // columns of this half that the row sees
        const bool bad = bad_tag[tile & 7] == (int)tile + 1;
        if (__any_sync(0xffffffffu, left < kHalf) || bad) {
#pragma unroll
          for (int k = 0; k < kHalf; ++k) s[k] = k < left ? s[k] : 0xFF800000u;
          if (bad) {                                      // leave out the tokens of bad pages
#pragma unroll
            for (int k = 0; k < kHalf; ++k)
              if (tok0 + k < G.seq.len &&
                  !kv::page_ok(__ldg(A.table + (int64_t)G.b * A.max_pages + fast_div((uint32_t)(tok0 + k), A.by_page)),
                               A.num_pages))
                s[k] = 0xFF800000u;
          }
        }
        // ---- the row's largest score, over both halves
        float t0 = __uint_as_float(s[0]), t1 = __uint_as_float(s[1]), t2 = __uint_as_float(s[2]),
              t3 = __uint_as_float(s[3]);
#pragma unroll
        for (int k = 4; k + 4 < kHalf; k += 8) {
          t0 = max3(t0, __uint_as_float(s[k]), __uint_as_float(s[k + 4]));
          t1 = max3(t1, __uint_as_float(s[k + 1]), __uint_as_float(s[k + 5]));
          t2 = max3(t2, __uint_as_float(s[k + 2]), __uint_as_float(s[k + 6]));
          t3 = max3(t3, __uint_as_float(s[k + 3]), __uint_as_float(s[k + 7]));
        }
        t0 = max3(t0, __uint_as_float(s[kHalf - 4]), __uint_as_float(s[kHalf - 3]));
        t1 = max3(t1, __uint_as_float(s[kHalf - 2]), __uint_as_float(s[kHalf - 1]));
        float top_s = fmaxf(max3(t0, t1, t2), t3);
        xch[(x * 2 + side) * kRows + r] = top_s;
        pair_sync(quad);
        top_s = fmaxf(top_s, xch[(x * 2 + (side ^ 1)) * kRows + r]);
        const float top_x = top_s == -INFINITY ? -INFINITY : top_s * sc;
        if (__any_sync(0xffffffffu, top_x > m + kLazy)) { // the same decision in both warps of the rows
          const float to = fmaxf(m, top_x);
          const float f = ex2(m - to);
          m = to;
          l *= f;
          if (i > 0) {
            ok &= mbar_wait_warp(pv_done, (tile - 1) & 1, abort_flag, A.dev_status);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[16];
              tm_ld16(tmem + lanes + L::kO + side * (D / 2) + 16 * c, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tm_st16(tmem + lanes + L::kO + side * (D / 2) + 16 * c, o);
            }
          }
        }
        // ---- P over this half of S
        const uint64_t sc2 = pair_f32(sc, sc), neg_m = pair_f32(-m, -m);
        uint64_t sum0 = 0, sum1 = 0;
        uint32_t p[kHalf / 2];
#pragma unroll
        for (int k = 0; k < kHalf / 2; ++k) {
          const uint64_t v = fma_f32x2(((uint64_t)s[2 * k + 1] << 32) | s[2 * k], sc2, neg_m);
          const float a = ex2(__uint_as_float((uint32_t)v)), b = ex2(__uint_as_float((uint32_t)(v >> 32)));
          if (k & 1) sum1 = add_f32x2(sum1, pair_f32(a, b));
          else sum0 = add_f32x2(sum0, pair_f32(a, b));
          p[k] = pack_f16x2(a, b);
        }
        sum0 = add_f32x2(sum0, sum1);
        l += __uint_as_float((uint32_t)sum0) + __uint_as_float((uint32_t)(sum0 >> 32));
        tm_st<kHalf / 2>(st, p);
        tm_wait_st();
        tc_fence_before();
        mbar_arrive(p_full + 8 * x);
      }
      // ---- the item's last P V, then O out, each thread half of its row; the
      // next item's Q is on its way meanwhile
      const Segment done = G;
      more = walk.next(P, G);
      if (more) load_q(G);
      ok &= mbar_wait_warp(o_done, item & 1, abort_flag, A.dev_status);
      ++item;
      tc_fence_after();
      pair_sync(quad);                                    // the other half's last read of xch is over
      xch[side * kRows + r] = l;
      pair_sync(quad);
      l = xch[r] + xch[kRows + r];                        // both threads in the same order
      pair_sync(quad);
      const bool whole = done.s0 == 0 && done.s1 == done.steps;
      const int64_t slot = 2 * (int64_t)blockIdx.x + kv::part_slot(blockIdx.x, walk.per, done.item_start);
      const int64_t at = (int64_t)(done.seq.first + qi) * A.heads_q + h;
      const float f = whole ? (l == 0.0f ? 0.0f : vgs * kScaleFix / l) : 1.0f;
#pragma unroll 1
      for (int c = side * (D / 64); c < (side + 1) * (D / 64); ++c) {
        uint32_t o[32];
        tm_ld32(tmem + lanes + L::kO + 32 * c, o);
        if (live && ok) {
          if (whole && A.out_bf16) {
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(A.out) + at * D + 32 * c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                    : "=r"(w[j])
                    : "f"(__uint_as_float(o[8 * k + 2 * j + 1]) * f), "f"(__uint_as_float(o[8 * k + 2 * j]) * f));
              dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            float4 *dst = reinterpret_cast<float4 *>(
                whole ? static_cast<float *>(A.out) + at * D + 32 * c : P.ws_o + (slot * kRows + r) * D + 32 * c);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              dst[k] = make_float4(__uint_as_float(o[4 * k]) * f, __uint_as_float(o[4 * k + 1]) * f,
                                   __uint_as_float(o[4 * k + 2]) * f, __uint_as_float(o[4 * k + 3]) * f);
          }
        }
      }
      tc_fence_before();
      if (live && ok && side == 0) {
        if (!whole)
          *reinterpret_cast<float2 *>(P.ws_ml + (slot * kRows + r) * 2) = make_float2(m, l);
        else if (A.lse)
          A.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == W_MMA_P)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(L::kCols) : "memory");
}

// Joins the items that several CTAs shared.  CTA (c, y): the item in which
// CTA c's range of the prefill kernel begins, if c is the second CTA with tiles
// of it; 16 rows of it.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const PlanArgs P) {
  const Args &A = P.a;
  const int per = P.count[1], total = P.count[2];
  const int c = blockIdx.x + 1;
  const int64_t pos = (int64_t)c * per;
  if (pos >= total) return;
  const int e = P.start[c];
  const int2 what = P.entry[e];
  const int base = P.prefix[e], cost = (P.prefix[e + 1] - base) / A.heads_kv, steps = cost - kItemCost;
  const int head = ((int)pos - base) / cost, start = base + head * cost;
  int lo, hi;
  kv::item_part(c, per, start, kItemCost, steps, lo, hi);
  if (lo == 0 || lo >= hi) return;              // c has none of its tiles, or the first of them
  const int c0 = (start + kItemCost) / per, c1 = (start + cost - 1) / per;
  if (c0 != c - 1) return;                      // not the second CTA
  const Seq seq = load_seq(A, what.x);
  const int nrows = min(kRows, seq.queries * A.group - what.y * kRows);
  constexpr int kLanes = D / 4, kPass = 256 / kLanes;
  const int d = (threadIdx.x % kLanes) * 4;
  for (int i = threadIdx.x / kLanes; i < 16; i += kPass) {
    const int r = blockIdx.y * 16 + i;
    if (r >= nrows) return;
    float M = kFloor, sum = 0.0f;
    for (int k = c0; k <= c1; ++k)
      M = fmaxf(M, P.ws_ml[((int64_t)(2 * k + kv::part_slot(k, per, start)) * kRows + r) * 2]);
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int k = c0; k <= c1; ++k) {
      const int64_t at = (int64_t)(2 * k + kv::part_slot(k, per, start)) * kRows + r;
      const float2 ml = *reinterpret_cast<const float2 *>(P.ws_ml + at * 2);
      const float4 x = *reinterpret_cast<const float4 *>(P.ws_o + at * D + d);
      const float f = ex2(ml.x - M);
      sum += f * ml.y;
      acc.x += f * x.x; acc.y += f * x.y; acc.z += f * x.z; acc.w += f * x.w;
    }
    const int row = what.y * kRows + r, qi = row / A.group, h = head * A.group + row - qi * A.group;
    const int64_t at = (int64_t)(seq.first + qi) * A.heads_q + h;
    const float f = sum == 0.0f ? 0.0f : __ldg(A.v_gs) * kScaleFix / sum;
    store_out(A, at, D, d, acc, f);
    if (A.lse && d == 0) A.lse[at] = sum == 0.0f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
  }
}

namespace {

int64_t prefill_entries(int batch, int64_t max_query, int group) {
  return batch * ((max_query * group + kRows - 1) / kRows);
}

template <int D>
nvfp4_status run_prefill(PlanArgs p, uint8_t *ws, cudaStream_t stream) {
  using L = Pre<D>;
  auto kern = prefill_kernel<D>;
  if (!host::set_max_dynamic_smem(reinterpret_cast<const void *>(kern), L::kBytes)) return NVFP4_ERR_CUDA;
  const int64_t entries = prefill_entries(p.a.batch, p.a.max_query, p.a.group);
  p.tile = L::T;
  p.grid = host::sm_count();
  p.count = reinterpret_cast<int32_t *>(ws);
  ws += 256;
  p.prefix = reinterpret_cast<int32_t *>(ws);
  ws += align256(4 * (entries + 1));
  p.entry = reinterpret_cast<int2 *>(ws);
  ws += align256(8 * entries);
  p.start = reinterpret_cast<int32_t *>(ws);
  ws += align256(4 * (int64_t)p.grid);
  p.ws_ml = reinterpret_cast<float *>(ws);
  ws += align256(2 * (int64_t)p.grid * kRows * 8);
  p.ws_o = reinterpret_cast<float *>(ws);
  plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return NVFP4_ERR_CUDA;
  kern<<<(unsigned)p.grid, kPreThreads, L::kBytes, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return NVFP4_ERR_CUDA;
  if (p.grid > 1) join_kernel<D><<<dim3((unsigned)(p.grid - 1), kRows / 16), 256, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // namespace

int64_t prefill_workspace(int batch, int64_t max_query, int group, int D) {
  const int64_t entries = prefill_entries(batch, max_query, group), grid = host::sm_count();
  return 256 + align256(4 * (entries + 1)) + align256(8 * entries) + align256(4 * grid) +
         align256(2 * grid * kRows * 8) + align256(2 * grid * kRows * D * 4);
}

nvfp4_status launch_prefill(const Args &a, int D, int row_floor, uint8_t *ws, cudaStream_t stream) {
  PlanArgs p = {};
  p.a = a;
  p.row_floor = row_floor;
  if (D == 64) return run_prefill<64>(p, ws, stream);
  if (D == 128) return run_prefill<128>(p, ws, stream);
  return run_prefill<256>(p, ws, stream);
}

}  // namespace attn
}  // namespace nvfp4
