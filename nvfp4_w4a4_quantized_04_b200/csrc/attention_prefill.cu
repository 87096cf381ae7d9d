// Attention over the paged NVFP4 cache: prefill form (sm_100a), for sequences
// with many rows (row = query * group + head of the KV group).
//
// Same mathematics as the decode form (attention.cu).  Here 128 rows share
// every key, so the products are what bounds it, and they run on the 5th
// generation tensor cores:
//   S [128 rows, T keys]  = Q K^T    tcgen05.mma kind::f16, A = Q in tensor memory,
//   O [128 rows, D]      += P V      A = P in tensor or shared memory,
// with K and V dequantized to f16 (exactly) once per tile into shared memory.
//
// Roles of a CTA (one per SM):
//  * warps 0-7, softmax: two threads per row, each with 64 keys of a 128-key
//    tile.  They read S into registers at once, which frees it for the next
//    tile's MMAs, turn it into P (f16), keep the running maximum and sum, put Q
//    into tensor memory (f16, a power of two per row) at the start of an item and
//    store O at its end.  A tile's weights are taken by the maximum as it stands,
//    without looking for a larger one first; only when their sum exceeds 2^13 are
//    they taken again and O in tensor memory rescaled.
//  * warps 8-23, converters: cache codes -> f16 tiles in shared memory in a
//    ring of four units of 32 KB (16 KB with D = 64).  A unit of K is 128 tokens x
//    up to 128 elements, a unit of V up to 256 elements of 64 or 128 tokens, both
//    as [64-element chunk][token][128 bytes]: K-major for S (keys are N) and
//    N-major for O (keys are K), so V needs no transposition.
//  * warp 25, loader: codes and scales by bulk copies, several tiles ahead.  (As
//    ordinary loads of 16 bytes a lane from 8 rows they took 1290 of the about
//    1680 wavefronts a 64-key tile that kept the load/store pipe 77 % busy; begun
//    by each converter warp for itself, the copies' issue was half of its time.)
//  * warp 24, one thread issues the MMAs: as soon as S of tile i is read, S of a
//    later tile, and when P of tile i is there, P V, without waiting for any MMA
//    in between.  P lies apart from S, with D = 256 in shared memory (tensor
//    memory is full): where it was written over S, the next S had to wait for
//    P V, and the tensor cores idled through both waits.
// A tile has 128 keys because an S MMA costs about 56 cycles with N = 64 keys
// and little more with N = 128.
// Keeping Q in tensor memory instead of shared memory halves what the first
// product reads from shared memory, whose bandwidth the converters' stores and
// the B operands already fill (256 cycles each for K and V, stored and read,
// of the about 1024 that the MMAs of a tile take).
//
// Split: a plan kernel lists the (sequence, row block) pairs with their key
// tiles; the line of all (pair, head, tile) steps is cut evenly over the CTAs,
// and items that several CTAs share are joined by a third kernel.
//
// Two orders that the barriers have to keep, each of which was once missing:
//  * a warp that raised no maximum may finish the next tile's P while another
//    still rescales O for this one, so p_full alternates between two barriers;
//  * a staging slot goes back to the loader only behind the use of its values and
//    a proxy fence, or the next bulk copy passes reads that are still in flight.
//
// Measured, all three kernels: 4096 queries of 32 heads on 8 of 128 over their own
// keys: 221 us, 621 TFLOP/s (38 % of cuBLAS's bf16 rate), bound by the softmax
// warps: of 2470 cycles a tile they spend 1500 in the weights (the exponentials
// alone take 1024) and the rest waiting for S, loading it, voting and storing P;
// an item costs about 13000 cycles besides.  2048 queries of 32 heads on 4 of 256
// over 32 Ki keys: 2098 us, 1015 TFLOP/s (63 %), bound by shared-memory bandwidth:
// 1500 us without the conversion and its stores.
#include "attention.cuh"
#include "attention_internal.cuh"
#include "encode.cuh"
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
constexpr int kSoft = 8, kConv = 16;          // softmax and converter warps
constexpr int W_CONV = kSoft, W_MMA_P = kSoft + kConv, W_LOAD = W_MMA_P + 1;
constexpr int kPreThreads = (W_MMA_P + 4) * 32;   // seven warpgroups; the last has two working warps
// Registers per thread after the roles part (setmaxnreg moves them between
// warpgroups): 256 x 136 + 512 x 48 + 128 x 40 = 64512, the 896 x 72 that the
// block is launched with.
constexpr int kLaunchRegs = 72, kSoftRegs = 136, kConvRegs = 48, kRestRegs = 40;
static_assert(32 * (kSoft * kSoftRegs + kConv * kConvRegs + 4 * kRestRegs) <= kPreThreads * kLaunchRegs, "registers");
// What an item costs besides its tiles (Q in, the first S, O out), in tiles:
// the line that is cut over the CTAs counts it, so that a CTA with many short
// items takes no longer than the others.
constexpr int kItemCost = 3;
// A tile's weights may add up to this before the maximum is raised: every
// weight then is an f16 (65504 is the largest).
constexpr float kMostSum = 8192.0f;

template <int D> struct Pre {
  static constexpr int T = 128;                         // keys per tile
  static constexpr int kUnits = D == 256 ? 2 : 1;       // ring units of a K or V tile
  static constexpr int kUnit = T * D * 2 / kUnits;      // bytes of one
  static constexpr int kBufs = 4;                       // units in the ring
  static constexpr bool kPShared = D == 256;            // P in shared memory, else in tensor memory
  static constexpr uint32_t kO = 0, kQ = D, kS = D + D / 2;   // tensor memory columns
  static constexpr uint32_t kP = kS + T;                // two P tiles in turn (unless shared)
  static constexpr uint32_t kCols = 512;
  static constexpr int kPAt = kBufs * kUnit;
  static constexpr int kPBytes = kPShared ? kRows * T * 2 : 0;
  // codes and scales of tiles on their way
  static constexpr int kSlots = D == 256 ? 3 : 6;
  static constexpr int kCodeBytes = T * D / 2, kScaleBytes = T * D / 16, kSlotBytes = kCodeBytes + kScaleBytes;
  static constexpr int kStageAt = kPAt + kPBytes;
  static constexpr int kBar = kStageAt + kSlots * kSlotBytes;
  // kv_full[], kv_empty[], s_full, s_free, pv_done, p_full[2], o_done, q_ready, drain, staged[], unstaged[]
  static constexpr int kNumBars = 2 * kBufs + 8 + 2 * kSlots;
  static constexpr int kMisc = kBar + kNumBars * 8;      // tmem base, abort flag, bad-page tags[16]
  static constexpr int kXch = kMisc + 8 + 64;            // [4][128] floats between a row's two threads
  static constexpr int kBytes = kXch + 4 * kRows * 4 + 1024;
  static_assert(kS + T + (kPShared ? 0 : T) <= kCols, "tensor memory");
  static_assert(kBytes <= 232448, "shared memory");
};

struct PlanArgs {
  Args a;
  int32_t row_floor;       // sequences with at most this many rows are left to the decode kernel
  int32_t tile;
  int32_t chunk;           // tokens per bulk copy: a power of two that divides the tile and the page
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
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Args &A = P.a;
  const int t = threadIdx.x;
  if (t == 0 && !scales_ok(A)) report(A.dev_status, NVFP4_ERR_INVALID_ARG);
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
  int item_end = 0, cost = 0;          // of the item before; its entry's last head
  __device__ __forceinline__ Walk(const PlanArgs &P) {
    per = P.count[1];
    const int total = P.count[2];
    pos = (int)min((int64_t)total, (int64_t)blockIdx.x * per);
    end = (int)min((int64_t)total, (int64_t)pos + per);
    entry = P.start[blockIdx.x];
  }
  __device__ __forceinline__ bool next(const PlanArgs &P, Segment &g) {
    while (pos < end) {
      if (cost && pos == item_end && g.head + 1 < P.a.heads_kv) {
        ++g.head;                      // the next head of the same rows: nothing to look up
        g.item_start = pos;
      } else {
        while (P.prefix[entry + 1] <= pos) ++entry;
        const int2 e = P.entry[entry];
        const int base = P.prefix[entry];
        cost = (P.prefix[entry + 1] - base) / P.a.heads_kv;
        g.steps = cost - kItemCost;
        g.head = (pos - base) / cost;
        g.item_start = base + g.head * cost;
        g.b = e.x;
        g.block = e.y;
        g.seq = load_seq(P.a, e.x);
        g.nrows = min(kRows, g.seq.queries * P.a.group - g.block * kRows);
      }
      kv::item_part(blockIdx.x, per, g.item_start, kItemCost, g.steps, g.s0, g.s1);
      item_end = g.item_start + cost;
      pos = min(end, item_end);
      if (g.s0 < g.s1) return true;    // else only the item's fixed cost falls into this range
    }
    return false;
  }
};

// Columns of this warp's lanes.  tm_ld32 and tm_ld16 are complete on return;
// tm_ld_begin only starts the load and tm_ld_end, which names the registers,
// completes it.
__device__ __forceinline__ void tm_ld_begin(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tm_ld_end(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31]) :: "memory");
}
__device__ __forceinline__ void tm_ld_begin(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tm_ld_end(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :: "memory");
}

__device__ __forceinline__ void tm_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  tm_ld_begin(taddr, r);
  tm_ld_end(r);
}
__device__ __forceinline__ void tm_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  tm_ld_begin(taddr, r);
  tm_ld_end(r);
}

__device__ __forceinline__ void tm_st32(uint32_t taddr, const uint32_t *v) {
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

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
      :: "r"(d), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

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

__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Barrier of the two warps that share 32 rows.
__device__ __forceinline__ void pair_sync(int quadrant) {
  asm volatile("bar.sync %0, 64;" :: "r"(1 + quadrant) : "memory");
}
// The same, and whether any of the 64 threads says so.
__device__ __forceinline__ bool pair_any(int quadrant, bool x) {
  uint32_t any;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 q, %2, 0;\nbar.red.or.pred p, %1, 64, q;\nselp.u32 %0, 1, 0, p;\n}"
      : "=r"(any) : "r"(1 + quadrant), "r"((uint32_t)x) : "memory");
  return any != 0;
}

__device__ __forceinline__ void tm_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
         "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// One lane of the (whole) warp.  With elect.sync the compiler keeps the MMA
// operands in uniform registers; behind `lane == 0` every MMA issue cost about
// 110 cycles, more than the MMA itself.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred q;\nelect.sync _|q, 0xFFFFFFFF;\nselp.b32 %0, 1, 0, q;\n}" : "=r"(p));
  return p != 0;
}

// 64 scores from token `tok0` on: those past the row's limit, and with `bad`
// those of tokens on bad pages, to -inf.
__device__ __forceinline__ void mask_scores(const Args &A, const Segment &G, uint32_t (&s)[2][32], int left, int tok0,
                                            bool bad) {
#pragma unroll
  for (int k = 0; k < 64; ++k) s[k >> 5][k & 31] = k < left ? s[k >> 5][k & 31] : 0xFF800000u;
  if (bad) {
#pragma unroll 1
    for (int k = 0; k < 64; ++k)
      if (tok0 + k < G.seq.len &&
          !kv::page_ok(__ldg(A.table + (int64_t)G.b * A.max_pages + fast_div((uint32_t)(tok0 + k), A.by_page)),
                       A.num_pages)) {
#pragma unroll
        for (int j = 0; j < 64; ++j)
          if (j == k) s[j >> 5][j & 31] = 0xFF800000u;
      }
  }
}

// The weights exp2(s sc - m) of 64 scores as packed f16 pairs, and their fp32 sum
// (kRaised as in exponent()).
template <bool kRaised>
__device__ __forceinline__ float weights(const uint32_t (&s)[2][32], float sc, float m, uint32_t (&p)[32]) {
  const uint64_t sc2 = pair_f32(sc, sc), neg_m = pair_f32(-m, -m);
  uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const uint32_t *x = &s[k >> 4][2 * (k & 15)];
    // (the rounded form in scalars: a packed product and sum were fused all the same)
    const uint64_t v = kRaised ? pair_f32(exponent<true>(__uint_as_float(x[0]), sc, m), exponent<true>(__uint_as_float(x[1]), sc, m))
                               : fma_f32x2(((uint64_t)x[1] << 32) | x[0], sc2, neg_m);
    const float a = ex2(__uint_as_float((uint32_t)v)), b = ex2(__uint_as_float((uint32_t)(v >> 32)));
    if (k & 1) sum1 = add_f32x2(sum1, pair_f32(a, b));
    else sum0 = add_f32x2(sum0, pair_f32(a, b));
    p[k] = pack_f16x2(a, b);
  }
  sum0 = add_f32x2(sum0, sum1);
  return __uint_as_float((uint32_t)sum0) + __uint_as_float((uint32_t)(sum0 >> 32));
}

template <int D>
__global__ void __launch_bounds__(kPreThreads, 1) prefill_kernel(const PlanArgs P) {
  using L = Pre<D>;
  constexpr int T = L::T, kBufs = L::kBufs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const Args &A = P.a;
  const uint32_t sbase = smem_addr(smem);
  const uint32_t kv_full = sbase + L::kBar, kv_empty = kv_full + 8 * kBufs, s_full = kv_empty + 8 * kBufs;
  const uint32_t s_free = s_full + 8, pv_done = s_free + 8, p_full = pv_done + 8, o_done = p_full + 16;
  const uint32_t q_ready = o_done + 8, drain = q_ready + 8, staged = drain + 8, unstaged = staged + 8 * L::kSlots;
  volatile uint32_t *tmem_holder = reinterpret_cast<volatile uint32_t *>(smem + L::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);
  volatile int *bad_tag = reinterpret_cast<volatile int *>(smem + L::kMisc + 8);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < 16; ++i) bad_tag[i] = 0;   // the loads are up to 8 tiles ahead of the softmax
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(kv_full + 8 * i, kConv * 32);
      mbar_init(kv_empty + 8 * i, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, kSoft * 32);
    mbar_init(pv_done, 1);
    mbar_init(p_full, kSoft * 32);
    mbar_init(p_full + 8, kSoft * 32);
    mbar_init(o_done, 1);
    mbar_init(q_ready, kSoft * 32);
    mbar_init(drain, 1);
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(staged + 8 * i, 1);
      mbar_init(unstaged + 8 * i, kConv);
    }
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
  asm volatile("griddepcontrol.wait;" ::: "memory");         // the plan is written

  if (warp >= W_MMA_P) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kRestRegs));
    if (warp == W_MMA_P) {
    // ================================================================ MMA issuer
    // Tiles in the order of use: K of the first, then per tile i the K of tile
    // i + 1 (if any) and the V of tile i.
    Walk walk(P);
    Segment G = {};
    uint32_t buf = 0, tile = 0, item = 0;
    bool ok = true;
    auto qk = [&]() -> bool {                       // S of the next tile
#pragma unroll
      for (int u = 0; u < L::kUnits; ++u, ++buf) {
        const uint32_t x = buf % kBufs;
        if (!mbar_wait_warp(kv_full + 8 * x, (buf / kBufs) & 1, abort_flag, A.dev_status)) return false;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t at = sbase + x * L::kUnit;
          constexpr int kSteps = D / 16 / L::kUnits;
#pragma unroll
          for (int k = 0; k < kSteps; ++k)
            mma_ts(tmem + L::kS, tmem + L::kQ + 8 * (u * kSteps + k),
                   gemm::desc_sw128(at + (k >> 2) * (T * 128)) + 2 * (k & 3), idesc(T, false), u > 0 || k > 0);
          tc_commit(kv_empty + 8 * x);
          if (u + 1 == L::kUnits) tc_commit(s_full);
        }
        __syncwarp();
      }
      return true;
    };
    while (ok && walk.next(P, G)) {
      if (!mbar_wait_warp(q_ready, item & 1, abort_flag, A.dev_status)) { ok = false; break; }
      tc_fence_after();
      const int n = G.s1 - G.s0;
      ok = qk();
      for (int i = 0; ok && i < n; ++i, ++tile) {
        if (i + 1 < n && (!mbar_wait_warp(s_free, tile & 1, abort_flag, A.dev_status) || !qk())) {
          ok = false;
          break;
        }
        if (!mbar_wait_warp(p_full + 8 * (tile & 1), (tile >> 1) & 1, abort_flag, A.dev_status)) { ok = false; break; }
#pragma unroll
        for (int u = 0; ok && u < L::kUnits; ++u, ++buf) {
          const uint32_t x = buf % kBufs;
          if (!mbar_wait_warp(kv_full + 8 * x, (buf / kBufs) & 1, abort_flag, A.dev_status)) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t at = sbase + x * L::kUnit;
            constexpr int kKeys = T / L::kUnits;          // keys of a unit of V
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k) {
              if (L::kPShared)
                mma_ss(tmem + L::kO, gemm::desc_sw128(sbase + L::kPAt + u * (kRows * 128)) + 2 * k,
                       desc_n_major(at + k * 2048, kKeys * 128), idesc(D, true), i > 0 || u > 0 || k > 0);
              else
                mma_ts(tmem + L::kO, tmem + L::kP + (tile & 1) * (T / 2) + 8 * k, desc_n_major(at + k * 2048, kKeys * 128), idesc(D, true),
                       i > 0 || k > 0);
            }
            tc_commit(kv_empty + 8 * x);
            if (u + 1 == L::kUnits) {
              tc_commit(pv_done);
              if (i + 1 == n) tc_commit(o_done);
            }
          }
          __syncwarp();
        }
      }
      ++item;
    }
    if (elect_one()) {
      tc_commit(drain);
      const long long t0 = clock64();
      while (!gemm::mbar_try_wait(drain, 0) && clock64() - t0 < gemm::kWaitBudgetCycles) {}
    }
    __syncwarp();
    } else if (warp == W_LOAD) {
    // ================================================================ loader
    // Codes and scales of tiles in the order of use, a slot each.  Lane i copies
    // the i-th `chunk` tokens of the tile, which lie on one page.  Tokens behind
    // the sequence's end and on bad pages are not copied: what the slot holds in
    // their place decodes to finite values, and their scores are masked.
    Walk walk(P);
    Segment G = {};
    uint32_t load = 0, tile = 0;
    bool ok = true;
    const int chunk = P.chunk, chunks = T / chunk;
    auto fetch = [&](int i) -> int32_t {                  // this lane's page of tile i of the segment, -1 none, -2 bad
      const int tok = (G.s0 + i) * T + lane * chunk;
      if (lane >= chunks || G.s0 + i >= G.s1 || tok >= G.seq.len) return -1;
      const int32_t page = __ldg(A.table + (int64_t)G.b * A.max_pages + fast_div((uint32_t)tok, A.by_page));
      return kv::page_ok(page, A.num_pages) ? page : -2;
    };
    auto copy = [&](int32_t page, int i, const uint8_t *q, const uint8_t *sf) -> bool {
      const uint32_t slot = load % L::kSlots, bar = staged + 8 * slot, to = sbase + L::kStageAt + slot * L::kSlotBytes;
      if (load >= L::kSlots &&
          !mbar_wait_warp(unstaged + 8 * slot, ((load / L::kSlots) - 1) & 1, abort_flag, A.dev_status))
        return false;
      const uint32_t mine = __ballot_sync(0xffffffffu, page >= 0);
      if (lane == 0) {
        if (mine) gemm::mbar_arrive_expect_tx(bar, __popc(mine) * chunk * (D / 2 + D / 16));
        else mbar_arrive(bar);
      }
      __syncwarp();
      if (page >= 0) {
        const int tok = (G.s0 + i) * T + lane * chunk;
        const int in_page = tok - (int)fast_div((uint32_t)tok, A.by_page) * A.page_size;
        const int64_t row = kv::pool_row(page, A.heads_kv, A.page_size, G.head, in_page);
        gemm::bulk_load(to + lane * chunk * (D / 2), q + row * (D / 2), chunk * (D / 2), bar);
        gemm::bulk_load(to + L::kCodeBytes + lane * chunk * (D / 16), sf + row * (D / 16), chunk * (D / 16), bar);
      }
      ++load;
      return true;
    };
    while (ok && walk.next(P, G)) {
      const int n = G.s1 - G.s0;
      // K a tile ahead of V; a tile's pages are read a step ahead of its K and
      // kept until V's turn
      int32_t p0 = fetch(0), p1 = fetch(1);
      for (int i = -1; ok && i < n; ++i) {
        const int32_t p2 = i >= 0 ? fetch(i + 2) : -1;
        const int k = i + 1;
        const int32_t pk = i < 0 ? p0 : p1;
        if (k < n) {
          if (__any_sync(0xffffffffu, pk == -2)) {
            if (pk == -2) report(A.dev_status, NVFP4_ERR_INDEX);
            if (lane == 0) bad_tag[(tile + k) & 15] = (int)(tile + k) + 1;
          }
          ok = copy(pk, k, A.k_q, A.k_sf);
        }
        if (i >= 0) {
          if (ok) ok = copy(p0, i, A.v_q, A.v_sf);
          p0 = p1;
          p1 = p2;
        }
      }
      tile += n;
    }
    // no copy is left on its way when the block ends
    for (uint32_t x = load > L::kSlots ? load - L::kSlots : 0; x != load; ++x) {
      const long long t0 = clock64();
      while (!gemm::mbar_try_wait(staged + 8 * (x % L::kSlots), (x / L::kSlots) & 1) &&
             clock64() - t0 < gemm::kWaitBudgetCycles) {}
    }
    }
  } else if (warp >= W_CONV) {
    // ================================================================ converters
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kConvRegs));
    // A lane takes one 16-byte piece (32 codes) of one token of a unit.  Which
    // piece depends on the token, so that 8 lanes read 8 different 16-byte
    // positions of the staged rows (pairs of lanes share one in K with D = 256)
    // and write 8 different ones of the swizzled tile.  With D = 64 a unit has
    // work for half of the warps.
    const int w = warp - W_CONV;
    const bool idle = D == 64 && w >= kConv / 2;
    int at_codes[2], at_scale[2], at_dst[2];              // of a unit of K, of V
    uint32_t flips = 0;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int kTok = D == 64 ? 16 : D == 256 && v ? 4 : 8;
      const int t = (w * kTok + lane % kTok) % T, c = lane / kTok;
      const int p = D == 64 ? ((t >> 2) + c) & 1 : D == 256 && v ? (2 * t + c) & 7 : ((t >> 1) + c) & 3;
      at_codes[v] = t * (D / 2) + p * 16;
      at_scale[v] = L::kCodeBytes + t * (D / 16) + p * 2;
      at_dst[v] = (p >> 1) * (T / (D == 256 && v ? 2 : 1) * 128) + t * 128;
      flips |= (uint32_t)(((p & 1) * 4) ^ (t & 7)) << (8 * v);
    }
    Walk walk(P);
    Segment G = {};
    uint32_t buf = 0, load = 0;
    bool ok = true;
    while (ok && walk.next(P, G)) {
      const int n = G.s1 - G.s0;
      for (int j = 0; ok && j < 2 * n; ++j, ++load) {
        const bool is_v = j > 0 && ((j & 1) == 0 || j == 2 * n - 1);   // K, then K and V in turn, then V
        const uint32_t slot = load % L::kSlots;
        if (!mbar_wait_warp(staged + 8 * slot, (load / L::kSlots) & 1, abort_flag, A.dev_status)) { ok = false; break; }
#pragma unroll
        for (int u = 0; ok && u < L::kUnits; ++u, ++buf) {
          const uint32_t x = buf % kBufs;
          // K: the unit's 128 elements of every token; V: its 64 tokens
          const uint32_t from = sbase + L::kStageAt + slot * L::kSlotBytes;
          const int code_u = u * (is_v ? 64 * (D / 2) : 64), scale_u = u * (is_v ? 64 * (D / 16) : 8);
          const uint4 code = lds_v4(from + code_u + (is_v ? at_codes[1] : at_codes[0]));
          const uint32_t scale = lds_u16(from + scale_u + (is_v ? at_scale[1] : at_scale[0]));
          if (buf >= kBufs && !mbar_wait_warp(kv_empty + 8 * x, ((buf / kBufs) - 1) & 1, abort_flag, A.dev_status)) {
            ok = false;
            break;
          }
          if (!idle) {
            const uint32_t s0 = e4m3_pair_f16x2(__byte_perm(scale, 0, 0x4040));
            const uint32_t s1 = e4m3_pair_f16x2(__byte_perm(scale, 0, 0x4141));
            const uint32_t c[4] = {code.x, code.y, code.z, code.w};
            const uint32_t flip = (is_v ? flips >> 8 : flips) & 7;
            uint8_t *dst = smem + x * L::kUnit + (is_v ? at_dst[1] : at_dst[0]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t s = k < 2 ? s0 : s1;
              const uint4 v = make_uint4(mul_f16x2(e2m1x2_f16x2<0>(c[k]), s), mul_f16x2(e2m1x2_f16x2<1>(c[k]), s),
                                         mul_f16x2(e2m1x2_f16x2<2>(c[k]), s), mul_f16x2(e2m1x2_f16x2<3>(c[k]), s));
              *reinterpret_cast<uint4 *>(dst + ((flip ^ k) << 4)) = v;
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          mbar_arrive(kv_full + 8 * x);
          // Only now is the slot given back: every lane's reads are behind the fence, so
          // that the next bulk copy into it (async proxy) cannot pass them.
          if (u + 1 == L::kUnits) {
            __syncwarp();
            if (lane == 0) mbar_arrive(unstaged + 8 * slot);
          }
        }
      }
    }
  } else {
    // ================================================================ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kSoftRegs));
    Walk walk(P);
    Segment G = {};
    const int quad = warp & 3, side = warp >> 2;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const int r = 32 * quad + lane;                       // row of the block
    volatile float *xch = reinterpret_cast<volatile float *>(smem + L::kXch);
    const float kgs = scales_ok(A) ? __ldg(A.k_gs) : NAN, vgs = __ldg(A.v_gs);
    uint32_t tile = 0, item = 0;
    // A wait that gives up (abort) does not end the loop: the two warps of a row
    // stay in step, every later wait returns at once, and nothing more is stored.
    bool ok = true;
    uint32_t qw[D / 4];                                   // this thread's half of its row of Q, bf16
    auto load_q = [&](const Segment &g) {
      const int row = g.block * kRows + r, qi = (int)fast_div((uint32_t)row, A.by_group), h = g.head * A.group + row - qi * A.group;
      if (r < g.nrows) {
        const uint16_t *q = A.q + (int64_t)(g.seq.first + qi) * A.ld_q + (int64_t)h * D + side * (D / 2);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint4 v, w;
          load_block(q + 16 * i, A.v8_q, v, w);           // a whole sector a lane
          qw[8 * i] = v.x; qw[8 * i + 1] = v.y; qw[8 * i + 2] = v.z; qw[8 * i + 3] = v.w;
          qw[8 * i + 4] = w.x; qw[8 * i + 5] = w.y; qw[8 * i + 6] = w.z; qw[8 * i + 7] = w.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 4; ++i) qw[i] = 0;
      }
    };
    bool more = walk.next(P, G);
    while (more) {
      load_q(G);
      // ---- Q into tensor memory, each thread half of its row
      const bool live = r < G.nrows;
      const int row = G.block * kRows + r, qi = (int)fast_div((uint32_t)row, A.by_group), h = G.head * A.group + row - qi * A.group;
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
      const float sc = score_scale(A, kgs, down);
      const int limit = live ? (int)kv::visible_keys(G.seq.len, G.seq.queries, qi, A.causal != 0) : 0;
      float m = kFloor, l = 0.0f;
      const int n = G.s1 - G.s0;
      for (int i = 0; i < n; ++i, ++tile) {
        ok &= mbar_wait_warp(s_full, tile & 1, abort_flag, A.dev_status);
        tc_fence_after();
        uint32_t s[2][32];                                // this thread's 64 scores
        tm_ld_begin(tmem + lanes + L::kS + side * 64, s[0]);
        tm_ld_begin(tmem + lanes + L::kS + side * 64 + 32, s[1]);
        tm_ld_end(s[0]);
        tm_ld_end(s[1]);
        tc_fence_before();
        mbar_arrive(s_free);
        const int tok0 = (G.s0 + i) * T + side * 64;
        const bool bad = bad_tag[tile & 15] == (int)tile + 1;
        if (__any_sync(0xffffffffu, limit - tok0 < 64) || bad) mask_scores(A, G, s, limit - tok0, tok0, bad);
        uint32_t p[32];
        float sum = 0.0f;
        if (i > 0) sum = weights<false>(s, sc, m, p);
        // Do the weights of any of the 32 rows call for larger maxima?
        if (pair_any(quad, i == 0 || sum > kMostSum)) {
          float top = __uint_as_float(s[0][0]);
#pragma unroll
          for (int k = 1; k < 63; k += 2)
            top = max3(top, __uint_as_float(s[k >> 5][k & 31]), __uint_as_float(s[(k + 1) >> 5][(k + 1) & 31]));
          top = fmaxf(top, __uint_as_float(s[1][31]));
          // (a buffer of xch per tile parity: its last readers have met since)
          volatile float *x = xch + (tile & 1) * 2 * kRows;
          x[side * kRows + r] = top;
          pair_sync(quad);
          top = fmaxf(top, x[(side ^ 1) * kRows + r]);
          const float to = fmaxf(m, top == -INFINITY ? -INFINITY : top * sc);
          const float f = ex2(m - to);
          m = to;
          l *= f;
          if (i > 0) {                                    // O by the new maximum, half of the row each
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
            tm_wait_st();
          }
          sum = weights<true>(s, sc, m, p);
        }
        l += sum;
        // ---- P for the MMA.  The one tile in shared memory is free once P V of the
        // tile before is over.  Of the two in tensor memory this one is free: S of
        // this tile was committed behind the P V that used it last.
        if (L::kPShared) {
          if (tile > 0) ok &= mbar_wait_warp(pv_done, (tile - 1) & 1, abort_flag, A.dev_status);
          uint8_t *at = smem + L::kPAt + side * (kRows * 128) + r * 128;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4 *>(at + ((k ^ (r & 7)) << 4)) = make_uint4(p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        } else {
          tm_st32(tmem + lanes + L::kP + (tile & 1) * (T / 2) + side * 32, p);
          tm_wait_st();
        }
        tc_fence_before();
        // One barrier per tile parity: a warp may be here with the next tile while
        // another still raises its maxima.  It cannot be two tiles ahead, since S of
        // that tile waits for every warp's s_free of the next one.
        mbar_arrive(p_full + 8 * (tile & 1));
      }
      // ---- the item's last P V, then O out, each thread half of its row.
      // (Q of the next item is loaded only behind it: held in registers meanwhile, it
      // made the tile loop spill, 232 against 217 us for a prompt of 4096.)
      const bool whole = G.s0 == 0 && G.s1 == G.steps;
      const int64_t slot = 2 * (int64_t)blockIdx.x + kv::part_slot(blockIdx.x, walk.per, G.item_start);
      const int64_t at = (int64_t)(G.seq.first + qi) * A.heads_q + h;
      more = walk.next(P, G);
      ok &= mbar_wait_warp(o_done, item & 1, abort_flag, A.dev_status);
      ++item;
      tc_fence_after();
      // the row's sum (the maximum is the same in both threads)
      pair_sync(quad);
      xch[side * kRows + r] = l;
      pair_sync(quad);
      l = xch[r] + xch[kRows + r];
      pair_sync(quad);
      const float f = whole ? (l == 0.0f ? 0.0f : vgs * kScaleFix / l) : 1.0f;
#pragma unroll 1
      for (int c = side * (D / 64); c < (side + 1) * (D / 64); ++c) {
        uint32_t o[32];
        tm_ld32(tmem + lanes + L::kO + 32 * c, o);
        if (live && ok) {
          if (whole && A.out_bf16) {
            uint16_t *dst = static_cast<uint16_t *>(A.out) + at * D + 32 * c;
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
              w[j] = bf16x2_of(pair_f32(__uint_as_float(o[2 * j]) * f, __uint_as_float(o[2 * j + 1]) * f));
#pragma unroll
            for (int j = 0; j < 2; ++j)
              store_block(dst + 16 * j, A.v8_out, make_uint4(w[8 * j], w[8 * j + 1], w[8 * j + 2], w[8 * j + 3]),
                          make_uint4(w[8 * j + 4], w[8 * j + 5], w[8 * j + 6], w[8 * j + 7]));
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
// of it; kJoinRows rows of it, one per D/4 threads.
template <int D> constexpr int kJoinRows = 256 / (D / 4);
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const PlanArgs P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
  constexpr int kLanes = D / 4;
  const int d = (threadIdx.x % kLanes) * 4, r = blockIdx.y * kJoinRows<D> + threadIdx.x / kLanes;
  if (r >= nrows) return;
  float M = kFloor, sum = 0.0f;
  for (int k = c0; k <= c1; ++k)
    M = fmaxf(M, P.ws_ml[((int64_t)(2 * k + kv::part_slot(k, per, start)) * kRows + r) * 2]);
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int k = c0; k <= c1; ++k) {
    const int64_t at = (int64_t)(2 * k + kv::part_slot(k, per, start)) * kRows + r;
    const float2 ml = *reinterpret_cast<const float2 *>(P.ws_ml + at * 2);
    const float4 x = *reinterpret_cast<const float4 *>(P.ws_o + at * D + d);
    const float f = ex2(ml.x - M);
    sum += f * ml.y;
    acc.x += f * x.x; acc.y += f * x.y; acc.z += f * x.z; acc.w += f * x.w;
  }
  const int row = what.y * kRows + r, qi = (int)fast_div((uint32_t)row, A.by_group),
            h = head * A.group + row - qi * A.group;
  const int64_t at = (int64_t)(seq.first + qi) * A.heads_q + h;
  const float f = sum == 0.0f ? 0.0f : __ldg(A.v_gs) * kScaleFix / sum;
  store_out(A, at, D, d, acc, f);
  if (A.lse && d == 0) A.lse[at] = sum == 0.0f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
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
  p.chunk = kv::kPageGranule;
  while (p.chunk < L::T && p.a.page_size % (2 * p.chunk) == 0) p.chunk *= 2;
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
  // both may be set up while the kernel before them ends (griddepcontrol.wait)
  if (!launch_behind(kern, dim3((unsigned)p.grid), kPreThreads, L::kBytes, stream, p)) return NVFP4_ERR_CUDA;
  // an item takes at most all of a CTA's rows: rows beyond max_query * group do not exist
  const int64_t rows = (int64_t)p.a.max_query * p.a.group < kRows ? (int64_t)p.a.max_query * p.a.group : kRows;
  if (p.grid > 1 && !launch_behind(join_kernel<D>, dim3((unsigned)(p.grid - 1), (unsigned)((rows + kJoinRows<D> - 1) / kJoinRows<D>)),
                                   256, 0, stream, p))
    return NVFP4_ERR_CUDA;
  return NVFP4_OK;
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
namespace gemm {
nvfp4_status set_wait_budget_prefill(long long cycles) {
  return cudaMemcpyToSymbol(c_wait_budget, &cycles, sizeof(cycles)) == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
}  // namespace gemm

}  // namespace nvfp4
