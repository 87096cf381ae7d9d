// Attention over the paged NVFP4 cache: decode and few-query form (sm_100a).
//
//   O_r = sum_j softmax_j(scale q_r . k_j) v_j,   k_j = k_gs (e2m1 * e4m3),  v_j likewise,
// over the keys that row r sees ("Qwen3.8-2.4T-A95B-NVFP4": the NVFP4 KV cache
// is dequantized when attention reads it).  The cache is read at 4.5 bits an
// element and never written out at 16.
//
// Rows.  The queries of a sequence and the heads of one KV group form rows
// (row = query * group + head); a work item is (sequence, KV head) with its up
// to 8 * NT rows, so the heads of a group share each read of K and V.
// Sequences with more rows go to the prefill form (attention_prefill.cu).
//
// What bounds it.  HBM: 9/16 byte an element of K and V against 4 operations
// per row.  To reach that rate a 32-lane instruction may be spent on every
// ~55 elements, which rules out anything but register dequantization, so:
//  * S^T = K Q^T and O^T = V^T P^T run as mma.sync m16n8k16 with the cache as
//    the A operand and 8 rows as N: a warp dequantizes its A fragments from
//    the codes it reads (E2M1 -> f16 is one conversion per two codes, times
//    the E4M3 scale as one f16x2 multiply; the product is exact in f16), and
//    no dequantized value goes through shared memory.
//  * K codes need no shuffling: a lane takes 16-byte pieces of its token's
//    row, and the head dimension is permuted the same way on both operands.
//    V is contracted over tokens, so pairs of tokens are interleaved at the
//    nibble level (four logic operations per 16 codes) before the conversion.
//  * P^T comes out of the first MMA as an accumulator with tokens as rows and
//    turns into the second one's B operand by an 8x8 transpose (movmatrix).
//  * Every warp has its own ring of cp.async stages (32 tokens of K and V) and
//    its own softmax state; warps meet only at the end of an item.
//  * 32 rows of 256 elements leave no registers for the output in one warp.
//    There a team of two warps shares a step: each takes the scores of one half
//    of its tokens for all rows and the outputs of one half of the head, so
//    every element is still converted once.  They show each other P in shared
//    memory, with one barrier a step, which is also the vote below.
//  * The weights are taken by the running maximum as it stands, which is raised
//    only when a lane's weights of a step add up to more than 2^13 (P stays
//    below f16's range): the usual step has one vote instead of a maximum, a
//    reduction and a rescale.
// Q is brought to f16 by a power of two per row that puts the row's largest
// element at 2^14: exact for every element within 2^29 of it.
//
// Split.  All items' steps (32 tokens each, and kItemSteps for an item's begin
// and end) form one line that is cut evenly over the CTAs, so ragged batches,
// one long sequence and many short ones all fill the GPU; an item that several
// CTAs share is joined by a second kernel from (max, sum, unnormalized O) parts
// in the workspace.
//
// Measured, with the join, in replayed graphs: 64 sequences of up to 16 Ki tokens, 8 KV
// heads of 128 and 4 heads each: 136 us, 4.7 TB/s (72 % of a copy's rate; 140 to 148
// in plain calls on other boxes); one of 256 Ki tokens, 4 KV heads of 256 and 8 heads
// each: 69 us, 4.4 TB/s; 32 of 8 Ki with 4 queries of 8 heads on 4 of 256: 86 us.  No
// pipe is full (at D 128 issue slots 63 %, ALU with the conversions 52 %, DRAM 58 %,
// tensor 26 %): the stalls are fixed latencies and the math pipe, with four warps a
// scheduler at D 128 and two at D 256; more warps a SM with fewer registers each are
// slower.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <type_traits>

#include "attention.cuh"
#include "attention_internal.cuh"
#include "host_util.cuh"

namespace nvfp4 {
namespace attn {

constexpr int kStep = 32;                // tokens per step
// What an item's begin and end (page ids, Q, the first loads' latency, the join
// of the warps) weigh in the even split, in steps.  64 sequences of 982..16384
// tokens with 8 KV heads of 128: 148 us at 0, 140 at 8, 135 at 16, 137 at 32,
// 143 at 64; 32 of 4 queries with 4 KV heads of 256: 104, 94, 86, 91, 104 us.
constexpr int kItemSteps = 16;
// A step's weights of one lane may add up to this before the maximum is raised:
// every weight then is an f16 (65504 is the largest).
constexpr float kMostSum = 8192.0f;

// ws_head: prefix[batch + 1], then steps per CTA.
struct DecodeArgs {
  Args a;
  int32_t row_cap;      // sequences with more rows than this are left to the prefill kernel
  int32_t *ws_head;
  float *ws_ml;         // [2 * grid][R][2]
  float *ws_o;          // [2 * grid][R][D]
  int32_t grid;
};

// Steps of one item (sequence, KV head); false when the prefill form takes the
// sequence or it has no queries.
__device__ __forceinline__ bool seq_steps(const DecodeArgs &P, const Seq &s, int &steps) {
  const bool mine = s.queries > 0 && s.queries * P.a.group <= P.row_cap;
  steps = mine ? (s.len + kStep - 1) / kStep : 0;
  return mine;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Bytes of one half stage (16 tokens): K codes, V codes, K scales, V scales.
template <int D> struct Half {
  static constexpr int kCodes = 8 * D, kScales = D;
  static constexpr int kK = 0, kV = kCodes, kKs = 2 * kCodes, kVs = 2 * kCodes + kScales;
  static constexpr int kBytes = 2 * kCodes + 2 * kScales;
};

// Shared-memory byte offset of 16-byte piece c of token t's codes inside a half
// stage.  K rows of 128 bytes swap halves on odd tokens, V lines of 128 bytes
// rotate by token pair, so that the fragment reads below have no bank conflicts.
template <int D>
__device__ __forceinline__ int k_piece(int t, int c) {
  if (D == 256) c ^= (t & 1) << 2;
  return t * (D / 2) + c * 16;
}
template <int D>
__device__ __forceinline__ int v_piece(int t, int c) {
  const int pos = t * (D / 32) + c;                       // 16-byte position
  const int sw = D == 64 ? ((t >> 2) & 1) << 1 : ((t >> 1) & 3) << 1;
  return (pos ^ sw) * 16;
}

// kTeam warps share a step; a CTA has kWarps / kTeam teams.
template <int D, int NT, int kStages, int kWarps, int kTeam>
struct Layout {
  static constexpr int R = 8 * NT, kTeams = kWarps / kTeam;
  static constexpr int kStageBytes = 2 * Half<D>::kBytes;
  static constexpr int kRing = kTeams * kStages * kStageBytes;
  static constexpr int kRS = D + 20;                      // row stride of the O exchange, in floats
  static constexpr int kO = kTeams * R * kRS * 4;
  static constexpr int kMain = kRing > kO ? kRing : kO;
  static constexpr int kQ = kMain;                        // Q fragments: NT * (D/16) * 32 lanes * 8 bytes
  static constexpr int kRow = kQ + NT * (D / 16) * 256;   // per row: scale, limit
  static constexpr int kMl = kRow + R * 8;                // per warp and row: max, sum
  static constexpr int kTop = kMl + kWarps * R * 8;       // per warp of a team and row: max of a step
  static constexpr int kP = kTop + (kTeam == 2 ? kWarps * R * 4 : 0);       // per warp: its P of two steps
  static constexpr int kScan = kP + (kTeam == 2 ? kWarps * 2 * NT * 256 : 0);   // scan scratch
  static constexpr int kPrefix = kScan + 64;
  static constexpr int bytes(int batch) { return kPrefix + 4 * (batch + 2); }
};

// Barrier of the two warps of team `team`, true when `any` holds in one of them.
__device__ __forceinline__ bool team_any(int team, bool any) {
  uint32_t r;
  asm volatile(
      "{.reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.red.or.pred q, %2, 64, p; selp.u32 %0, 1, 0, q;}"
      : "=r"(r) : "r"((uint32_t)any), "r"(team + 1) : "memory");
  return r != 0;
}

template <int D, int NT, int kStages, int kWarps, int kMinCtas, int kTeam>
__global__ void __launch_bounds__(kWarps * 32, kMinCtas) decode_kernel(const DecodeArgs P) {
  using L = Layout<D, NT, kStages, kWarps, kTeam>;
  static_assert(kTeam == 1 || (kTeam == 2 && D == 256), "the halves of V are cut for D = 256");
  constexpr int kThreads = kWarps * 32, kTeams = L::kTeams;
  constexpr int kH = 2 / kTeam;          // halves of a step whose scores a warp takes
  using H = Half<D>;
  constexpr int R = L::R;
  constexpr int J = D / 16;              // k-steps of S
  constexpr int JO = J / kTeam;          // m-tiles of O: the team's warps share the head dimension
  extern __shared__ __align__(128) uint8_t smem[];
  const Args &A = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int team = warp / kTeam, half = warp % kTeam;
  float2 *s_row = reinterpret_cast<float2 *>(smem + L::kRow);
  float2 *s_ml = reinterpret_cast<float2 *>(smem + L::kMl);
  int32_t *s_scan = reinterpret_cast<int32_t *>(smem + L::kScan);
  int32_t *s_prefix = reinterpret_cast<int32_t *>(smem + L::kPrefix);

  // ---- prefix sums of the sequences' steps
  {
    const int per = (A.batch + kThreads - 1) / kThreads;
    const int b0 = min(A.batch, tid * per), b1 = min(A.batch, b0 + per);
    int local = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) bad |= !offsets_ok(A, b);
    if (__syncthreads_or(bad)) {         // nothing is computed: the combine kernel sees 0 steps per CTA
      if (blockIdx.x == 0 && tid == 0) {
        P.ws_head[A.batch + 1] = 0;
        report(A.dev_status, NVFP4_ERR_INDEX);
      }
      return;
    }
    for (int b = b0; b < b1; ++b) {
      int steps;
      seq_steps(P, load_seq(A, b), steps);
      const int n = steps ? (steps + kItemSteps) * A.heads_kv : 0;
      s_prefix[b] = n;
      local += n;
    }
    int incl = local;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int run = incl - local;
    for (int w = 0; w < warp; ++w) run += s_scan[w];
    for (int b = b0; b < b1; ++b) {
      const int n = s_prefix[b];
      s_prefix[b] = run;
      run += n;
    }
    if (tid == kThreads - 1) s_prefix[A.batch] = run;
    __syncthreads();
  }
  const int total = s_prefix[A.batch];
  const int per_cta = (int)kv::steps_per_cta(total, gridDim.x, kTeams);    // one step per team at least
  if (blockIdx.x == 0) {
    for (int b = tid; b <= A.batch; b += kThreads) P.ws_head[b] = s_prefix[b];
    if (tid == 0) P.ws_head[A.batch + 1] = per_cta;
  }
  // sequences without keys: rows of zeros
  for (int b = blockIdx.x; b < A.batch; b += gridDim.x) {
    const Seq s = load_seq(A, b);
    int steps;
    if (!seq_steps(P, s, steps) || steps) continue;
    for (int i = tid; i < s.queries * A.heads_q * (D / 4); i += kThreads) {
      const int64_t at = (int64_t)s.first * A.heads_q + i / (D / 4);
      store_out(A, at, D, (i % (D / 4)) * 4, make_float4(0.0f, 0.0f, 0.0f, 0.0f), 0.0f);
      if (A.lse && i % (D / 4) == 0) A.lse[at] = -INFINITY;
    }
  }
  const bool scales = scales_ok(A);
  if (!scales && blockIdx.x == 0 && tid == 0) report(A.dev_status, NVFP4_ERR_INVALID_ARG);
  const float kgs = scales ? __ldg(A.k_gs) : NAN, vgs = __ldg(A.v_gs);
  int pos = (int)min((int64_t)total, (int64_t)blockIdx.x * per_cta);
  const int end = (int)min((int64_t)total, (int64_t)pos + per_cta);
  const uint32_t ring = smem_addr(smem) + team * kStages * L::kStageBytes;
  const uint32_t qs = smem_addr(smem + L::kQ) + lane * 8;

  while (pos < end) {
    const int b = upper_group(s_prefix, A.batch, pos);
    const Seq seq = load_seq(A, b);
    int steps;
    seq_steps(P, seq, steps);
    const int local = pos - s_prefix[b];
    const int head = local / (steps + kItemSteps), start = s_prefix[b] + head * (steps + kItemSteps);
    pos = min(end, start + kItemSteps + steps);
    int s0, s1;
    kv::item_part(blockIdx.x, per_cta, start, kItemSteps, steps, s0, s1);
    if (s0 == s1) continue;              // only the item's fixed part lies in this range
    const int nrows = seq.queries * A.group;

    // ---- Q fragments: one warp per row, f16 with a power of two per row
    __syncthreads();
    for (int r = warp; r < R; r += kWarps) {
      constexpr int kPer = D / 32;
      float v[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = 0.0f;
      int limit = 0;
      if (r < nrows) {
        const int qi = r / A.group, h = head * A.group + r - qi * A.group;
        const uint16_t *p = A.q + (int64_t)(seq.first + qi) * A.ld_q + (int64_t)h * D + lane * kPer;
        uint32_t w[kPer / 2];
        if constexpr (kPer == 8) {
          const uint4 x = *reinterpret_cast<const uint4 *>(p);
          w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        } else if constexpr (kPer == 4) {
          const uint2 x = *reinterpret_cast<const uint2 *>(p);
          w[0] = x.x; w[1] = x.y;
        } else {
          w[0] = *reinterpret_cast<const uint32_t *>(p);
        }
#pragma unroll
        for (int i = 0; i < kPer / 2; ++i) {
          v[2 * i] = __uint_as_float(w[i] << 16);
          v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
        limit = (int)kv::visible_keys(seq.len, seq.queries, qi, A.causal != 0);
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
      top = __reduce_max_sync(0xffffffffu, top);
      float up, down;
      row_power((int)(top >> 23), up, down);
#pragma unroll
      for (int i = 0; i < kPer; i += (kPer >= 4 ? 4 : 2)) {
        const int d = lane * kPer + i;
        int tq, j;
        if (D == 64) { tq = d >> 4; j = (d & 15) >> 2; }
        else { const int c = d >> 5; tq = c & 3; j = (c >> 2) * 8 + ((d & 31) >> 2); }
        uint8_t *dst = smem + L::kQ + (((r >> 3) * J + j) * 32 + (r & 7) * 4 + tq) * 8 + (d & 3) * 2;
        if constexpr (kPer >= 4)
          *reinterpret_cast<uint2 *>(dst) =
              make_uint2(pack_f16x2(v[i] * up, v[i + 1] * up), pack_f16x2(v[i + 2] * up, v[i + 3] * up));
        else
          *reinterpret_cast<uint32_t *>(dst) = pack_f16x2(v[i] * up, v[i + 1] * up);
      }
      if (lane == 0) s_row[r] = make_float2(score_scale(A, kgs, down), __int_as_float(limit));
    }
    __syncthreads();
    float sc[NT][2];
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 x = s_row[8 * nt + 2 * t4 + i];
        sc[nt][i] = x.x;
        lim[nt][i] = __float_as_int(x.y);
      }
    // what every row sees (the rows that pad the block see nothing: they count as the first row)
    const int lim_min = (int)kv::visible_keys(seq.len, seq.queries, 0, A.causal != 0);

    float o[JO][NT][4];
#pragma unroll
    for (int i = 0; i < JO; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][nt][k] = 0.0f;
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // rows that pad the block (zeros, never stored) start where they stay
        m[nt][i] = 8 * nt + 2 * t4 + i < nrows ? (float)kFloor : 0.0f;
        l[nt][i] = 0.0f;
      }

    // ---- the team's steps: s0 + team, + kTeams, ...
    const int mine = max(0, (s1 - s0 - team + kTeams - 1) / kTeams);
    int64_t base_reg = -1;               // lane i: pool row of half (i & 1) of iteration (block of 16) + i / 2
    auto fetch_pages = [&](int it0) {
      const int tok = (s0 + team + (it0 + (lane >> 1)) * kTeams) * kStep + (lane & 1) * 16;
      base_reg = -1;
      if (it0 + (lane >> 1) < mine && tok < seq.len) {
        const int e = (int)fast_div((uint32_t)tok, A.by_page);
        const int32_t page = A.table[(int64_t)b * A.max_pages + e];
        if (kv::page_ok(page, A.num_pages))
          base_reg = kv::pool_row(page, A.heads_kv, A.page_size, head, tok - e * A.page_size);
        else
          report(A.dev_status, NVFP4_ERR_INDEX);
      }
    };
    uint32_t valid = 0;                  // bit (2 * stage + half): the half was loaded
    auto load_stage = [&](int it) {
      if (it < mine) {
        if ((it & 15) == 0) fetch_pages(it);
        const int stage = it % kStages;
#pragma unroll
        for (int hh = 0; hh < kH; ++hh) {
          const int h = hh + half;
          const int64_t base = __shfl_sync(0xffffffffu, base_reg, 2 * (it & 15) + h);
          const uint32_t dst = ring + stage * L::kStageBytes + h * H::kBytes;
          valid &= ~(1u << (2 * stage + h));
          if (base >= 0) {
            valid |= 1u << (2 * stage + h);
            const uint8_t *kp = A.k_q + base * (D / 2), *vp = A.v_q + base * (D / 2);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
              const int c = i * 32 + lane, t = c / (D / 32), pc = c % (D / 32);
              cp_async16(dst + H::kK + k_piece<D>(t, pc), kp + c * 16);
              cp_async16(dst + H::kV + v_piece<D>(t, pc), vp + c * 16);
            }
            if ((lane & 15) < D / 16) {
              const bool is_v = lane >= 16;
              cp_async16(dst + (is_v ? H::kVs : H::kKs) + (lane & 15) * 16,
                         (is_v ? A.v_sf : A.k_sf) + base * (D / 16) + (lane & 15) * 16);
            }
          }
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) load_stage(i);

    for (int it = 0; it < mine; ++it) {
      // a team's stages are free for the next load only behind its barrier below
      if constexpr (kTeam == 1) load_stage(it + kStages - 1);
      cp_async_wait<kStages - kTeam>();
      __syncwarp();
      const int stage = it % kStages;
      const uint32_t st = ring + stage * L::kStageBytes;
      const int tok0 = (s0 + team + it * kTeams) * kStep;

      // S^T: tokens g and g + 8 of each half against the rows 2 t4, 2 t4 + 1.
      // A lone warp's halves go side by side: each fragment of Q is read once, and their
      // chains of MMAs are independent.
      float s[kH][NT][4];
#pragma unroll
      for (int h = 0; h < kH; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[h][nt][k] = 0.0f;
      constexpr int kPieces = D == 256 ? 2 : 1, kWords = D == 64 ? 2 : 4;
#pragma unroll
      for (int pc = 0; pc < kPieces; ++pc) {
        uint32_t ka[kH][4], kb[kH][4], sa[kH], sb[kH];
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          const uint32_t hb = st + (h + half) * H::kBytes;
          if constexpr (D == 64) {
            const uint2 x = lds_v2(hb + H::kK + g * 32 + t4 * 8), y = lds_v2(hb + H::kK + (g + 8) * 32 + t4 * 8);
            ka[h][0] = x.x; ka[h][1] = x.y; kb[h][0] = y.x; kb[h][1] = y.y;
            sa[h] = lds_u8(hb + H::kKs + g * 4 + t4);
            sb[h] = lds_u8(hb + H::kKs + (g + 8) * 4 + t4);
          } else {
            const uint4 x = lds_v4(hb + H::kK + k_piece<D>(g, t4 + 4 * pc));
            const uint4 y = lds_v4(hb + H::kK + k_piece<D>(g + 8, t4 + 4 * pc));
            ka[h][0] = x.x; ka[h][1] = x.y; ka[h][2] = x.z; ka[h][3] = x.w;
            kb[h][0] = y.x; kb[h][1] = y.y; kb[h][2] = y.z; kb[h][3] = y.w;
            sa[h] = lds_u16(hb + H::kKs + g * (D / 16) + 2 * (t4 + 4 * pc));
            sb[h] = lds_u16(hb + H::kKs + (g + 8) * (D / 16) + 2 * (t4 + 4 * pc));
          }
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          const int j = pc * 8 + 2 * w;
          uint2 q0[NT], q1[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            q0[nt] = lds_v2(qs + (nt * J + j) * 256);
            q1[nt] = lds_v2(qs + (nt * J + j + 1) * 256);
          }
#pragma unroll
          for (int h = 0; h < kH; ++h) {
            const uint32_t fa = e4m3_pair_f16x2(__byte_perm(sa[h], 0, w < 2 ? 0x2020 : 0x2121));
            const uint32_t fb = e4m3_pair_f16x2(__byte_perm(sb[h], 0, w < 2 ? 0x2020 : 0x2121));
            const uint32_t a = ka[h][w], b = kb[h][w];
            const uint32_t a0 = mul_f16x2(e2m1x2_f16x2<0>(a), fa), a1 = mul_f16x2(e2m1x2_f16x2<0>(b), fb);
            const uint32_t a2 = mul_f16x2(e2m1x2_f16x2<1>(a), fa), a3 = mul_f16x2(e2m1x2_f16x2<1>(b), fb);
            const uint32_t c0 = mul_f16x2(e2m1x2_f16x2<2>(a), fa), c1 = mul_f16x2(e2m1x2_f16x2<2>(b), fb);
            const uint32_t c2 = mul_f16x2(e2m1x2_f16x2<3>(a), fa), c3 = mul_f16x2(e2m1x2_f16x2<3>(b), fb);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16(s[h][nt], a0, a1, a2, a3, q0[nt].x, q0[nt].y);
              mma_f16(s[h][nt], c0, c1, c2, c3, q1[nt].x, q1[nt].y);
            }
          }
        }
      }

      // The weights by the maximum as it stands; only when a lane's weights of
      // this step add up to too much is the maximum raised and all of them taken
      // again.  Steps that every row sees whole need no mask.
      const uint32_t have = valid >> (2 * stage + half);
      const bool all = tok0 + kStep <= lim_min && (have & (kH == 2 ? 3 : 1)) == (kH == 2 ? 3 : 1);
      if (!all) {
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          const bool ok = (have >> h) & 1;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (!ok || tok0 + 16 * (h + half) + g + (k >> 1) * 8 >= lim[nt][k & 1]) s[h][nt][k] = -INFINITY;
        }
      }
      uint32_t pb[2][NT][2];             // of the halves [kH] first
      float sum[NT][2];
      auto take = [&](auto raised) {
        float most = 0.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[kH][4];
#pragma unroll
          for (int h = 0; h < kH; ++h) {
#pragma unroll
            for (int k = 0; k < 4; ++k) p[h][k] = ex2(exponent<raised>(s[h][nt][k], sc[nt][k & 1], m[nt][k & 1]));
            pb[h][nt][0] = pack_f16x2(p[h][0], p[h][1]);
            pb[h][nt][1] = pack_f16x2(p[h][2], p[h][3]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            sum[nt][i] = p[0][i] + p[0][i + 2];
            if constexpr (kH == 2) sum[nt][i] += p[1][i] + p[1][i + 2];
            most = fmaxf(most, sum[nt][i]);
          }
        }
        return most > kMostSum;
      };
      auto turn = [&]() {                // tokens as rows -> the second MMA's B operand
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < kH; ++h) {
            pb[h][nt][0] = transpose8x8(pb[h][nt][0]);
            pb[h][nt][1] = transpose8x8(pb[h][nt][1]);
          }
      };
      // A team's warps show each other their P: two buffers, since the partner may
      // still read the one before.
      const uint32_t p_mine = smem_addr(smem + L::kP) + ((warp * 2 + (it & 1)) * NT * 32 + lane) * 8;
      auto show = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sts_v2(p_mine + nt * 256, pb[0][nt][0], pb[0][nt][1]);
      };
      bool raise = take(std::false_type{});
      if constexpr (kTeam == 1) {
        raise = __any_sync(0xffffffffu, raise);
      } else {
        turn();
        show();
        raise = team_any(team, raise);
        load_stage(it + kStages - 1);
      }
      if (raise) {
        float x[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float y = fmaxf(s[0][nt][i], s[0][nt][i + 2]);
            if constexpr (kH == 2) y = fmaxf(y, fmaxf(s[1][nt][i], s[1][nt][i + 2]));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
            x[nt][i] = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
          }
        if constexpr (kTeam == 2) {
          float *top = reinterpret_cast<float *>(smem + L::kTop) + team * 2 * R;
          if (g == 0)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              *reinterpret_cast<float2 *>(top + half * R + 8 * nt + 2 * t4) = make_float2(x[nt][0], x[nt][1]);
          team_any(team, false);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 y = *reinterpret_cast<const float2 *>(top + (half ^ 1) * R + 8 * nt + 2 * t4);
            x[nt][0] = fmaxf(x[nt][0], y.x);
            x[nt][1] = fmaxf(x[nt][1], y.y);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float y = x[nt][i];
            const float to = fmaxf(y == -INFINITY ? y : y * sc[nt][i], m[nt][i]);
            const float f = ex2(m[nt][i] - to);
            m[nt][i] = to;
            l[nt][i] *= f;
#pragma unroll
            for (int j = 0; j < JO; ++j) {
              o[j][nt][i] *= f;
              o[j][nt][i + 2] *= f;
            }
          }
        take(std::true_type{});
        if constexpr (kTeam == 2) {
          turn();
          show();
          team_any(team, false);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        l[nt][0] += sum[nt][0];
        l[nt][1] += sum[nt][1];
      }
      if constexpr (kTeam == 1) {
        turn();
      } else {
        const uint32_t p_other = p_mine + (half ? -1 : 1) * (2 * NT * 256);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 x = lds_v2(p_other + nt * 256);
          pb[1][nt][0] = x.x;
          pb[1][nt][1] = x.y;
        }
      }

      // O^T += V^T P^T: lane (g, t4) holds head elements [g D/8, (g+1) D/8) of tokens 2 t4, 2 t4 + 1, + 8, + 9;
      // a team's warps take one half of each such run
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t hb = st + (kTeam == 1 ? h : h ^ half) * H::kBytes;
        constexpr int kWords = D / 64 / kTeam;
        uint32_t v[4][kWords], vs[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int t = 2 * t4 + (k & 1) + (k >> 1) * 8;
          if constexpr (kTeam == 2) {
            const uint2 x = lds_v2(hb + H::kV + v_piece<D>(t, g) + half * 8);
            v[k][0] = x.x; v[k][1] = x.y;
            vs[k] = lds_u8(hb + H::kVs + t * 16 + 2 * g + half);
          } else if constexpr (D == 256) {
            const uint4 x = lds_v4(hb + H::kV + v_piece<D>(t, g));
            v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
            vs[k] = lds_u16(hb + H::kVs + t * 16 + 2 * g);
          } else if constexpr (D == 128) {
            const uint2 x = lds_v2(hb + H::kV + v_piece<D>(t, g >> 1) + (g & 1) * 8);
            v[k][0] = x.x; v[k][1] = x.y;
            vs[k] = lds_u8(hb + H::kVs + t * 8 + g);
          } else {
            v[k][0] = lds_u32(hb + H::kV + v_piece<D>(t, g >> 2) + (g & 3) * 4);
            vs[k] = lds_u8(hb + H::kVs + t * 4 + (g >> 1));
          }
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          const int sel = w < 2 ? 0x6420 : 0x6521;
          const uint32_t f01 = e4m3_pair_f16x2(__byte_perm(vs[0], vs[1], sel));
          const uint32_t f23 = e4m3_pair_f16x2(__byte_perm(vs[2], vs[3], sel));
          // bytes of (token, token + 1) nibble pairs: even head elements, odd head elements
          const uint32_t e01 = (v[0][w] & 0x0F0F0F0Fu) | ((v[1][w] << 4) & 0xF0F0F0F0u);
          const uint32_t d01 = ((v[0][w] >> 4) & 0x0F0F0F0Fu) | (v[1][w] & 0xF0F0F0F0u);
          const uint32_t e23 = (v[2][w] & 0x0F0F0F0Fu) | ((v[3][w] << 4) & 0xF0F0F0F0u);
          const uint32_t d23 = ((v[2][w] >> 4) & 0x0F0F0F0Fu) | (v[3][w] & 0xF0F0F0F0u);
#define NVFP4_PV(B)                                                                                            \
  {                                                                                                            \
    const uint32_t a0 = mul_f16x2(e2m1x2_f16x2<B>(e01), f01), a1 = mul_f16x2(e2m1x2_f16x2<B>(d01), f01);       \
    const uint32_t a2 = mul_f16x2(e2m1x2_f16x2<B>(e23), f23), a3 = mul_f16x2(e2m1x2_f16x2<B>(d23), f23);       \
    _Pragma("unroll") for (int nt = 0; nt < NT; ++nt)                                                          \
        mma_f16(o[4 * w + B][nt], a0, a1, a2, a3, pb[h][nt][0], pb[h][nt][1]);                                 \
  }
          NVFP4_PV(0) NVFP4_PV(1) NVFP4_PV(2) NVFP4_PV(3)
#undef NVFP4_PV
        }
      }
      __syncwarp();
    }
    cp_async_wait<0>();

    // ---- the warps' states joined through shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = l[nt][i];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (g == 0) s_ml[warp * R + 8 * nt + 2 * t4 + i] = make_float2(m[nt][i], x);
      }
    __syncthreads();                     // every warp is done with its ring
    float *s_o = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int j = 0; j < JO; ++j)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float *p = s_o + (team * R + 8 * nt + 2 * t4) * L::kRS + g * (D / 8 + 2) + 2 * (j + half * JO);
        *reinterpret_cast<float2 *>(p) = make_float2(o[j][nt][0], o[j][nt][2]);
        *reinterpret_cast<float2 *>(p + L::kRS) = make_float2(o[j][nt][1], o[j][nt][3]);
      }
    __syncthreads();
    const bool whole = s0 == 0 && s1 == steps;
    const int slot = 2 * blockIdx.x + kv::part_slot(blockIdx.x, per_cta, start);
    for (int i = tid; i < nrows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      float2 ml[kTeams];
      float M = kFloor;
#pragma unroll
      for (int w = 0; w < kTeams; ++w) {
        ml[w] = s_ml[w * kTeam * R + r];
        if constexpr (kTeam == 2) ml[w].y += s_ml[(w * kTeam + 1) * R + r].y;
        M = fmaxf(M, ml[w].x);
      }
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kTeams; ++w) {
        const float f = ex2(ml[w].x - M);
        sum += f * ml[w].y;
        const float *p = s_o + (w * R + r) * L::kRS + d + 2 * (d / (D / 8));
        const float2 x = *reinterpret_cast<const float2 *>(p), y = *reinterpret_cast<const float2 *>(p + 2);
        acc.x += f * x.x; acc.y += f * x.y; acc.z += f * y.x; acc.w += f * y.y;
      }
      if (whole) {
        const int qi = r / A.group, h = head * A.group + r - qi * A.group;
        const int64_t at = (int64_t)(seq.first + qi) * A.heads_q + h;
        const float f = sum == 0.0f ? 0.0f : vgs * kScaleFix / sum;
        store_out(A, at, D, d, acc, f);
        if (A.lse && d == 0) A.lse[at] = sum == 0.0f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
      } else {
        *reinterpret_cast<float4 *>(P.ws_o + ((int64_t)slot * R + r) * D + d) = acc;
        if (d == 0) *reinterpret_cast<float2 *>(P.ws_ml + ((int64_t)slot * R + r) * 2) = make_float2(M, sum);
      }
    }
  }
}

// Joins the items that several CTAs shared: CTA (c, y) rows of the item in
// which CTA c's range of the first kernel begins, if it began earlier and c is
// the first to continue it.  D/4 threads take a row.  kWide, for calls of few
// items, each of many parts: a CTA has one row, whose parts its groups of
// threads share.  Otherwise a group takes a row with all its parts.
template <int D, int R, bool kWide>
struct Join {
  static constexpr int kLanes = D / 4;
  static constexpr int kThreads = kWide || R * kLanes > 512 ? 512 : R * kLanes;
  static constexpr int kGroups = kThreads / kLanes;
  static constexpr int kRows = kWide ? 1 : kGroups;      // rows of a CTA
};
template <int D, int R, bool kWide>
__global__ void __launch_bounds__(Join<D, R, kWide>::kThreads) combine_kernel(const DecodeArgs P) {
  using J = Join<D, R, kWide>;
  constexpr int kLanes = J::kLanes, kThreads = J::kThreads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Args &A = P.a;
  const int tid = threadIdx.x, lane = tid % kLanes, part = tid / kLanes;
  const int r = kWide ? blockIdx.y : blockIdx.y * J::kRows + part, c = blockIdx.x + 1;
  const int per = P.ws_head[A.batch + 1], total = P.ws_head[A.batch];
  const int64_t pos = (int64_t)c * per;
  if (per == 0 || pos >= total) return;  // refused offsets; or a CTA without work
  const int b = upper_group(P.ws_head, A.batch, pos);
  const Seq seq = load_seq(A, b);
  int steps;
  if (!seq_steps(P, seq, steps) || r >= seq.queries * A.group) return;
  const int head = ((int)pos - P.ws_head[b]) / (steps + kItemSteps);
  const int start = P.ws_head[b] + head * (steps + kItemSteps);
  if (start == pos || (int64_t)(c - 1) * per > start) return;
  const int c0 = (start + kItemSteps) / per, c1 = (start + kItemSteps + steps - 1) / per;
  if (c0 == c1) return;                  // one CTA had all of its steps
  auto slot = [&](int k) { return (int64_t)(2 * k + kv::part_slot(k, per, start)) * R + r; };
  float M = kFloor, sum = 0.0f;
  if constexpr (kWide) {
    __shared__ float s_max[kThreads / 32];
    for (int k = c0 + tid; k <= c1; k += kThreads) M = fmaxf(M, P.ws_ml[slot(k) * 2]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    if ((tid & 31) == 0) s_max[tid >> 5] = M;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) M = fmaxf(M, s_max[k]);
  } else {
    for (int k = c0; k <= c1; ++k) M = fmaxf(M, P.ws_ml[slot(k) * 2]);
  }
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int k = kWide ? c0 + part : c0; k <= c1; k += kWide ? J::kGroups : 1) {
    const float2 ml = *reinterpret_cast<const float2 *>(P.ws_ml + slot(k) * 2);
    const float4 x = *reinterpret_cast<const float4 *>(P.ws_o + slot(k) * D + lane * 4);
    const float f = ex2(ml.x - M);
    sum += f * ml.y;
    acc.x += f * x.x; acc.y += f * x.y; acc.z += f * x.z; acc.w += f * x.w;
  }
  if constexpr (kWide) {
    __shared__ float4 s_o[kThreads];
    __shared__ float s_sum[J::kGroups];
    s_o[tid] = acc;
    if (lane == 0) s_sum[part] = sum;
    __syncthreads();
    if (part) return;
    sum = 0.0f;
    acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < J::kGroups; ++k) {
      const float4 x = s_o[k * kLanes + lane];
      sum += s_sum[k];
      acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
    }
  }
  const int qi = r / A.group, h = head * A.group + r - qi * A.group;
  const int64_t at = (int64_t)(seq.first + qi) * A.heads_q + h;
  const float f = sum == 0.0f ? 0.0f : __ldg(A.v_gs) * kScaleFix / sum;
  store_out(A, at, D, lane * 4, acc, f);
  if (A.lse && lane == 0) A.lse[at] = sum == 0.0f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
}

template <int D, int R, bool kWide>
bool launch_combine(const DecodeArgs &p, cudaStream_t stream) {
  using J = Join<D, R, kWide>;
  return launch_behind(combine_kernel<D, R, kWide>, dim3((unsigned)(p.grid - 1), (unsigned)(R / J::kRows)), J::kThreads, 0,
                       stream, p);
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

using kv::kRowLimit;
using kv::tiles_for;

// CTAs that the workspace is sized for: at most 4 per SM.
int64_t max_grid() { return (int64_t)host::sm_count() * 4; }

int64_t decode_workspace(int batch, int64_t rows, int D) {
  const int64_t R = 8 * tiles_for(rows);
  return align256(4 * ((int64_t)batch + 2)) + align256(2 * max_grid() * R * 8) + align256(2 * max_grid() * R * D * 4);
}

template <int D, int NT, int kStages, int kWarps, int kMinCtas, int kTeam = 1>
nvfp4_status run(DecodeArgs p, int64_t total_bound, uint8_t *ws, cudaStream_t stream) {
  using L = Layout<D, NT, kStages, kWarps, kTeam>;
  constexpr int kThreads = kWarps * 32;
  auto kern = decode_kernel<D, NT, kStages, kWarps, kMinCtas, kTeam>;
  const int smem = L::bytes(p.a.batch);
  if (!host::set_max_dynamic_smem(reinterpret_cast<const void *>(kern), L::bytes(kMaxBatch))) return NVFP4_ERR_CUDA;
  // as for the largest batch: registers bound the residency at every batch, and the
  // figures are kept per shared-memory size
  int64_t grid =
      (int64_t)host::sm_count() * host::blocks_per_sm(reinterpret_cast<const void *>(kern), kThreads, L::bytes(kMaxBatch));
  if (grid > max_grid()) grid = max_grid();
  const int64_t want = (total_bound + L::kTeams - 1) / L::kTeams;
  if (grid > want) grid = want < 1 ? 1 : want;
  p.grid = (int32_t)grid;
  p.ws_head = reinterpret_cast<int32_t *>(ws);
  ws += align256(4 * ((int64_t)p.a.batch + 2));
  p.ws_ml = reinterpret_cast<float *>(ws);
  ws += align256(2 * max_grid() * L::R * 8);
  p.ws_o = reinterpret_cast<float *>(ws);
  kern<<<(unsigned)grid, kThreads, smem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return NVFP4_ERR_CUDA;
  if (grid == 1) return NVFP4_OK;
  // Few items have many parts each.  The other way round (128 items of 2 to 3 parts
  // in 32 rows each), a CTA of 512 threads to a row takes 24 us instead of 9.
  const bool wide = (int64_t)p.a.batch * p.a.heads_kv * 8 <= grid;
  return (wide ? launch_combine<D, L::R, true>(p, stream) : launch_combine<D, L::R, false>(p, stream))
             ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // namespace attn
}  // namespace nvfp4

extern "C" {

size_t nvfp4_paged_attention_workspace_size(int batch, int64_t max_query, int q_heads, int kv_heads, int head_dim) {
  using namespace nvfp4::attn;
  if (batch < 1 || batch > kMaxBatch || kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads || q_heads > 4096 ||
      max_query < 1 || max_query > 0x7FFFFFFF / q_heads || (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  const int64_t rows = max_query * (q_heads / kv_heads);
  return (size_t)(decode_workspace(batch, rows, head_dim) +
                  (rows > kRowLimit ? prefill_workspace(batch, max_query, q_heads / kv_heads, head_dim) : 0));
}

nvfp4_status nvfp4_paged_attention(const void *q, int64_t ld_q, int64_t tokens, const int32_t *query_offsets,
                                   int64_t max_query, const int32_t *seq_lens, int batch, const int32_t *page_table,
                                   int max_pages, int q_heads, int kv_heads, int head_dim, const uint8_t *k_q,
                                   const uint8_t *k_sf, const float *k_gs, const uint8_t *v_q, const uint8_t *v_sf,
                                   const float *v_gs, int64_t num_pages, int page_size, float softmax_scale,
                                   int causal, void *out, nvfp4_out_dtype out_dtype, float *lse, void *workspace,
                                   int32_t *dev_status, cudaStream_t stream) {
  using namespace nvfp4;
  using namespace nvfp4::attn;
  if (batch < 0 || batch > kMaxBatch || tokens < 0 || tokens > 0x7FFFFFFF) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads != 0 || q_heads > 4096) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (page_size < kv::kPageGranule || page_size % kv::kPageGranule != 0 || page_size > 65536 || max_pages < 0 ||
      (int64_t)max_pages * page_size > 0x7FFFFFFF - 64 || num_pages < 0 || num_pages > 0x7FFFFFFF)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (out_dtype != NVFP4_OUT_F32 && out_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return NVFP4_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.0f) || !(softmax_scale < 1e30f)) return NVFP4_ERR_INVALID_ARG;
  if (ld_q < (int64_t)q_heads * head_dim || ld_q % 8 != 0) return NVFP4_ERR_INVALID_ARG;
  if (max_query < 1 || max_query > 0x7FFFFFFF / q_heads) return NVFP4_ERR_INVALID_ARG;
  if (!query_offsets && (max_query != 1 || tokens != batch)) return NVFP4_ERR_INVALID_ARG;
  if (batch == 0 || tokens == 0) return NVFP4_OK;
  if (!q || !seq_lens || !out || !k_gs || !v_gs || !workspace || !aligned(q, 16) || !aligned(out, 16) ||
      !aligned(workspace, 256) || !aligned(k_q, 16) || !aligned(k_sf, 16) || !aligned(v_q, 16) || !aligned(v_sf, 16) ||
      !aligned(seq_lens, 4) || !aligned(query_offsets, 4) || !aligned(page_table, 4))
    return NVFP4_ERR_INVALID_ARG;
  if (max_pages > 0 && !page_table) return NVFP4_ERR_INVALID_ARG;
  if (num_pages > 0 && (!k_q || !k_sf || !v_q || !v_sf)) return NVFP4_ERR_INVALID_ARG;
  const int group = q_heads / kv_heads;
  const int64_t rows = max_query * group;
  // The lines of both forms fit 32 bits: row blocks are bounded by the queries
  // that there are, and an item takes its steps or tiles and what it costs besides.
  const int64_t keys = (int64_t)max_pages * page_size;
  const int64_t steps_max = (keys + kStep - 1) / kStep;
  const int64_t blocks = tokens * group / 128 + batch;
  if ((int64_t)batch * kv_heads * (steps_max + kItemSteps) > 0x3FFFFFFF || blocks * kv_heads * (keys / 64 + 4) > 0x3FFFFFFF ||
      (int64_t)batch * ((rows + 127) / 128) > 0x3FFFFFFF)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  DecodeArgs p = {};
  p.a.q = static_cast<const uint16_t *>(q);
  p.a.ld_q = ld_q;
  p.a.tokens = (int32_t)tokens;
  p.a.offsets = query_offsets;
  p.a.lens = seq_lens;
  p.a.batch = batch;
  p.a.max_query = (int32_t)max_query;
  p.a.table = page_table;
  p.a.max_pages = max_pages;
  p.a.page_size = page_size;
  p.a.by_page = make_fastdiv((uint32_t)page_size);
  p.a.by_group = make_fastdiv((uint32_t)group);
  p.a.num_pages = num_pages;
  p.a.k_q = k_q; p.a.k_sf = k_sf; p.a.v_q = v_q; p.a.v_sf = v_sf;
  p.a.k_gs = k_gs; p.a.v_gs = v_gs;
  p.a.heads_q = q_heads; p.a.heads_kv = kv_heads; p.a.group = group;
  p.a.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.a.causal = causal;
  p.a.out = out;
  p.a.out_bf16 = out_dtype == NVFP4_OUT_BF16;
  p.a.v8_q = aligned(q, 32) && ld_q % 16 == 0;
  p.a.v8_out = aligned(out, 32);
  p.a.lse = lse;
  p.a.dev_status = dev_status;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const kv::Forms forms =
      kv::choose_forms(batch, tokens, max_query, group, kv_heads, keys, query_offsets != nullptr, host::sm_count());
  p.row_cap = forms.row_cap;
  if (forms.prefill) {
    const nvfp4_status st =
        launch_prefill(p.a, head_dim, forms.row_cap, ws + decode_workspace(batch, rows, head_dim), stream);
    if (st != NVFP4_OK || forms.row_cap == 0) return st;
  }
  const int nt = forms.row_cap / 8;
  const int64_t total_bound = (int64_t)batch * kv_heads * (steps_max + kItemSteps);
  if (head_dim == 64) {
    if (nt == 1) return run<64, 1, 3, 8, 2>(p, total_bound, ws, stream);
    if (nt == 2) return run<64, 2, 3, 4, 3>(p, total_bound, ws, stream);
    return run<64, 4, 3, 4, 2>(p, total_bound, ws, stream);
  }
  if (head_dim == 128) {
    if (nt == 1) return run<128, 1, 2, 8, 2>(p, total_bound, ws, stream);
    if (nt == 2) return run<128, 2, 3, 4, 3>(p, total_bound, ws, stream);
    return run<128, 4, 3, 4, 2>(p, total_bound, ws, stream);
  }
  if (nt == 1) return run<256, 1, 2, 8, 1>(p, total_bound, ws, stream);
  if (nt == 2) return run<256, 2, 2, 8, 1>(p, total_bound, ws, stream);
  return run<256, 4, 4, 8, 1, 2>(p, total_bound, ws, stream);
}

}  // extern "C"
