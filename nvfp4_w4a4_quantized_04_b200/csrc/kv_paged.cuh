// The paged NVFP4 KV cache: its layout and the index arithmetic that every
// kernel over it uses.
//
// A pool holds num_pages pages for K and for V.  A page holds page_size tokens
// of every KV head, head-major, so that the tokens of one head are contiguous:
//   codes   uint8 [num_pages, heads, page_size, D/2]
//   scales  uint8 [num_pages, heads, page_size, D/16]  (E4M3)
// A slot is page * page_size + row.  Plain host functions too, so that the
// arithmetic is tested without a GPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define NVFP4_HD __host__ __device__ __forceinline__
#else
#define NVFP4_HD inline
#endif

namespace nvfp4 {
namespace kv {

constexpr int kPageGranule = 16;    // page_size is a multiple of this

// Row of (page, head, row in page) in a pool, in units of one token of one head.
NVFP4_HD int64_t pool_row(int64_t page, int heads, int page_size, int head, int row) {
  return (page * heads + head) * (int64_t)page_size + row;
}

// Slot -> page and row; false when the slot is not in the pool.
NVFP4_HD bool split_slot(int64_t slot, int64_t num_pages, int page_size, int64_t &page, int &row) {
  if (slot < 0 || slot >= num_pages * page_size) return false;
  page = slot / page_size;
  row = (int)(slot - page * page_size);
  return true;
}

// A page id as a page table holds it; false when it is not in the pool.
NVFP4_HD bool page_ok(int32_t page, int64_t num_pages) { return page >= 0 && (int64_t)page < num_pages; }

// Keys that query j (0-based) of a sequence with `queries` queries and `len`
// cached tokens sees: causal, aligned at the end (the last query sees all).
NVFP4_HD int64_t visible_keys(int64_t len, int64_t queries, int64_t j, bool causal) {
  if (!causal) return len;
  const int64_t n = len - queries + j + 1;
  return n < 0 ? 0 : n;
}

// ---- work split of the attention kernels.  The work of a call is a line of
// `total` steps; CTA c of `grid` takes steps [c * per, (c+1) * per).
NVFP4_HD int64_t steps_per_cta(int64_t total, int64_t grid, int64_t least) {
  const int64_t per = (total + grid - 1) / grid;
  return per < least ? least : per;
}

// The workspace slot in which CTA c keeps its part of an item whose steps are
// [first, end): 0 when the item was begun by an earlier CTA or begins with c's
// own range, 1 when it begins inside the range.  A CTA has at most one part of
// each kind, so two slots a CTA are enough.
NVFP4_HD int part_slot(int64_t c, int64_t per, int64_t first) { return c * per < first ? 1 : 0; }

// Steps [lo, hi) of an item in CTA c's range [c * per, (c+1) * per) of a line
// on which the item takes `fixed` units from `start` and then one per step.
NVFP4_HD void item_part(int64_t c, int64_t per, int64_t start, int fixed, int steps, int &lo, int &hi) {
  const int64_t a = c * per - start - fixed, b = a + per;
  lo = (int)(a < 0 ? 0 : a > steps ? steps : a);
  hi = (int)(b < 0 ? 0 : b > steps ? steps : b);
}

// ---- which form of the attention takes a sequence, by its rows (queries * group)

// Most rows of a sequence that the decode form takes (the accumulators leave room
// for no more).
constexpr int kRowLimit = 32;

// 8-row tiles of a row block that holds `rows` rows, at most kRowLimit.
inline int tiles_for(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

// The decode form takes sequences of up to row_cap rows (0: is not launched), the
// prefill form the others.
struct Forms {
  int row_cap;
  bool prefill;
};

// From what the host knows: the batch, its tokens, the most queries of a sequence
// and the most keys (the lengths are on the device).  A prefill tile costs the
// same with 4 rows in use as with 128: 32 sequences of 16 Ki tokens beside a prompt of
// 2048 take 387 us there (8 KV heads of 128, 4 heads each) against 133 in the decode
// form, so a batch that may hold both is split.  The second pair of launches costs 6 to
// 12 us where it has nothing to do, so one form takes all where few-row sequences can
// waste no more than that: up to 5 tiles an SM, each 1.3 us (D 128) or 2.4 us (D 256).
//
// A split call's decode form has a tile for single queries (or for the mean rows,
// where these fit it): for the sequences above, 8 rows take 133 us and 32 rows 256.
inline Forms choose_forms(int64_t batch, int64_t tokens, int64_t max_query, int group, int heads_kv, int64_t keys,
                          bool offsets, int64_t sms) {
  const int64_t most = (max_query < tokens ? max_query : tokens) * group;
  if (most <= kRowLimit) return Forms{8 * tiles_for(most), false};
  const int64_t few_row_tiles = batch * heads_kv * (keys / 128 + 4);
  if (!offsets || group > kRowLimit || batch == 1 || few_row_tiles <= 5 * sms) return Forms{0, true};
  const int64_t mean = (tokens * group + batch - 1) / batch;
  return Forms{8 * tiles_for(mean <= kRowLimit && mean > group ? mean : group), true};
}

}  // namespace kv
}  // namespace nvfp4
