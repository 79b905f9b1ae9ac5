// gvr_long_common.h -- what the host code of include/gvr_long.h shares: the checks of a call's rows, and the ways of attend_shared.
#pragma once

#include <cmath>

#include "../csrc_cache/gvr_cache_common.cuh"
#include "gvr_long.h"

namespace gvrc {

// Entries of a row of the block table, and of what cache_evict keeps: loops may count past them by a turn in 32 bits.
constexpr int64_t MAX_ENTRIES = (int64_t(1) << 31) - (1 << 16);

// The arguments that attend_shared and attend_weights have in common, as attend_decode checks them.
inline gvr_status check_rows(const gvr_cache* cache, const void* q, int64_t q_row_stride, int64_t q_head_stride, int32_t dtype,
                             int64_t num_rows, int32_t num_heads, const int32_t* table, int64_t table_stride,
                             int64_t table_width, const int32_t* lens, int32_t next_n, int32_t ratio, float scale) {
  const gvr_status s = check_cache(cache);
  if (s != GVR_OK) return s;
  if ((dtype != GVR_BF16 && dtype != GVR_F16) || num_rows < 0 || num_heads < 1 || num_heads % cache->num_kv_heads != 0 ||
      num_heads > GVR_ATTEND_MAX_HEADS || !std::isfinite(float(double(scale) * cache->k_scale * 1.4426950408889634)) || table_width < 0 ||
      table_width > MAX_ENTRIES / cache->page_size || next_n < 1 || next_n > GVR_ATTEND_MAX_NEXT_N || ratio < 1 ||
      int64_t(next_n) * (num_heads / cache->num_kv_heads) > (1 << 19) || num_rows > int64_t(GVR_LONG_MAX_REQUESTS) * next_n)
    return GVR_ERR_ARG;
  if (q_row_stride < 0 || q_head_stride < 0 || q_row_stride % 8 != 0 || q_head_stride % 8 != 0 || q_row_stride > kIntMax ||
      q_head_stride > kIntMax || table_stride < table_width || table_stride > kIntMax)
    return GVR_ERR_STRIDE;
  if (num_rows == 0) return GVR_OK;
  if (!q || !lens || (table_width > 0 && !table)) return GVR_ERR_NULL;
  if (!aligned(q, 16) || !aligned(table, 4) || !aligned(lens, 4)) return GVR_ERR_ALIGN;
  return GVR_OK;
}

// Which kernels attend_shared takes: those of its rule, its own, or attend_decode's.
enum { WAY_BY_RULE = 0, WAY_TOGETHER = 1, WAY_APART = 2 };

}  // namespace gvrc

// attend_shared with the choice between the kernels made by the caller.  Exported for the tests alone, which run every case
// both ways: the rule goes by the table's width and would send most small cases to attend_decode's kernels.
extern "C" gvr_status attend_shared_way(int32_t way, const gvr_cache* cache, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                                        int32_t dtype, int64_t num_rows, int32_t num_heads, const int32_t* block_table,
                                        int64_t table_stride, int64_t table_width, const int32_t* kv_lens, int32_t next_n,
                                        int32_t compress_ratio, const int32_t* group_starts, const int32_t* prefix_entries,
                                        int64_t num_groups, float scale, void* out, float* lse, void* workspace,
                                        size_t workspace_bytes, void* stream);
