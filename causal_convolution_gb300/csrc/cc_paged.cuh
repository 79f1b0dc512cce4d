// What the kernels around a paged cache of keys and values share: the plan of a
// step (which rows belong to which sequence, how long each is, where its pages
// are) and its checks.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "cc_host.h"

namespace cc {

// Sequence b owns rows q_offsets[b] .. q_offsets[b + 1] - 1, the last of its
// kv_lens[b] tokens; token p lies in page page_table[b][p / page_size], slot
// p % page_size.
struct KvPlan {
  const int* q_offsets;
  const int* kv_lens;
  const int* page_table;
  int seqs, max_pages, pages, page_size;
};

enum PlaceResult { PLACE_OK, PLACE_NONE, PLACE_BAD };

// The place of row r: position p in its sequence, page and slot. PLACE_NONE: the
// row is no sequence's; PLACE_BAD: the plan gives it no place within the cache.
__device__ __forceinline__ PlaceResult find_place(const KvPlan& plan, int r, long long& p, int& page, int& slot) {
  // the last b with q_offsets[b] <= r, if the offsets do not fall
  int lo = 0;
  for (int hi = plan.seqs; hi - lo > 1;) {
    const int mid = (lo + hi) >> 1;
    (plan.q_offsets[mid] <= r ? lo : hi) = mid;
  }
  const int begin = plan.q_offsets[lo], end = plan.q_offsets[lo + 1], len = plan.kv_lens[lo];
  if (r < begin || r >= end) return PLACE_NONE;
  p = static_cast<long long>(len) - end + r;
  if (p < 0 || len > static_cast<long long>(plan.max_pages) * plan.page_size) return PLACE_BAD;
  const int n = static_cast<int>(p / plan.page_size);
  slot = static_cast<int>(p - static_cast<long long>(n) * plan.page_size);
  page = plan.page_table[static_cast<long long>(lo) * plan.max_pages + n];
  return page >= 0 && page < plan.pages ? PLACE_OK : PLACE_BAD;
}

inline cc_status check_plan(const char* what, const int32_t* q_offsets, const int32_t* kv_lens,
                            const int32_t* page_table, int max_pages, int pages, int page_size) {
  if (!q_offsets || !kv_lens || !page_table) return fail(CC_ERR_INVALID, "%s: null pointer", what);
  if (!aligned16(q_offsets) || !aligned16(kv_lens) || !aligned16(page_table))
    return fail(CC_ERR_INVALID, "%s: pointers must be 16-byte aligned", what);
  if (max_pages <= 0 || pages <= 0 || page_size <= 0)
    return fail(CC_ERR_INVALID, "%s: page counts and sizes must be positive", what);
  if (page_size % 16 != 0)
    return fail(CC_ERR_UNSUPPORTED, "%s: the page size must be a multiple of 16 (got %d)", what, page_size);
  if ((int64_t)pages * page_size > 0x7fffffffLL)
    return fail(CC_ERR_UNSUPPORTED, "%s: at most 2^31 - 1 slots in a cache", what);
  return CC_OK;
}

// A cache's strides in elements. Slots that overlap are the caller's mistake, but
// within its memory as long as the strides are true. A size of one is never
// stepped over: whatever its stride is (0 in an expanded tensor), it becomes D,
// which a tensor map takes.
inline cc_status check_cache_strides(const char* what, int64_t& page, int64_t token, int64_t& head, int pages,
                                     int kv_heads, int d) {
  if (pages == 1) page = d;
  if (kv_heads == 1) head = d;
  if (page < d || token < d || head < d || page % 8 || token % 8 || head % 8)
    return fail(CC_ERR_INVALID, "%s: cache strides must be at least D and multiples of 8", what);
  if (page >= (1ll << 38) || token >= (1ll << 38) || head >= (1ll << 38))
    return fail(CC_ERR_UNSUPPORTED, "%s: cache strides must be below 2^38 elements", what);
  return CC_OK;
}

}  // namespace cc
