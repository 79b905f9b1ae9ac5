/*
 * gvr_long.h -- C ABI of libgvrtopk for caches that live long, over the 4-bit paged cache of
 * gvr_cache.h: attention of requests that share long prefixes, the attention weight that each cached
 * entry draws, and eviction of the entries that draw least.
 *
 * Entries, cache, block tables, conventions and statuses are those of gvr_cache.h, with three differences.  A call
 * enqueues up to four kernels (attend_weights: one).  A row of the block table has at most 2^31 - 2^16 entries
 * (table_width * page_size).  Workspaces, where there are any, are required; their content is not kept between calls:
 * calls that can overlap on the GPU, or graphs whose replays can, need one each.
 */
#ifndef GVR_LONG_H
#define GVR_LONG_H

#include "gvr_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GVR_LONG_MAX_REQUESTS 8192 /* requests, and groups, of a call */

/*
 * Whole-cache attention of decode rows (attend_decode without indices) whose requests share prefixes:
 * each group's prefix is read once for all rows of the group.
 *   group_starts    int32 [num_groups + 1]: group g is the requests [group_starts[g], group_starts[g + 1]).
 *                   Requests before the first and behind the last are in no group.  A start below one before it
 *                   counts as that one, a negative one as 0, one beyond the requests as their number.
 *   prefix_entries  int32 [num_groups]: the first prefix_entries[g] entries of all requests of the group
 *                   are the same.  The caller vouches for it, and each of their block tables has them: they are read through
 *                   that of one of the requests, or of each.  (Usually full pages are the very same pages.  The page
 *                   in which a prefix ends may be each request's own copy.)  Negative counts as 0.
 * A request whose rows do not all see the whole prefix, and a request alone in its group, is attended as one in no
 * group.  num_groups 0 to GVR_LONG_MAX_REQUESTS (0: the pointers may be NULL), and as many requests.
 * Where the block table is so narrow, or the requests so few, that sharing is not expected to pay, attend_decode's kernels run.  (By the
 * table's width and the groups listed, as lengths are on the device: a table no wider than the longest request needs is the best one.)
 * Result, roundings and everything else are as in attend_decode without indices; next_n times num_heads /
 * num_kv_heads is at most 2^19, and num_rows times that quotient at most 2^26.
 *   workspace       16-byte aligned, attend_shared_workspace's bytes.
 * Every wait inside the kernel is bounded (0.5 s): should one give up, which is not expected on a healthy GPU, all of
 * out and lse are NaN.
 */
gvr_status attend_shared(const gvr_cache* cache, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                         int32_t dtype, int64_t num_rows, int32_t num_heads, const int32_t* block_table,
                         int64_t table_stride, int64_t table_width, const int32_t* kv_lens, int32_t next_n,
                         int32_t compress_ratio, const int32_t* group_starts, const int32_t* prefix_entries,
                         int64_t num_groups, float scale, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Bytes of workspace that attend_shared needs on the current device for a cache of num_kv_heads heads of head_dim.  Of groups beyond half the
 * requests, which cannot all share, only a line of the plan each, 48 bytes. */
gvr_status attend_shared_workspace(int32_t num_kv_heads, int32_t head_dim, int64_t num_rows, int32_t num_heads,
                                   int32_t next_n, int64_t num_groups, size_t* bytes);

/*
 * The attention weight that each entry draws: for every request b and entry e that it sees,
 *   weights[b][e] += sum over its rows j that see e and their heads h of exp(scale * q[j][h] . k_e - lse[j][h]),
 * the softmax weights of attend_decode without indices over the same arguments, whose lse this takes
 * (fp32 [num_rows][num_heads]).  Everything up to next_n and compress_ratio is as there.
 *   weights  fp32 [requests][weights_stride], weights_stride at least table_width * page_size; only the entries that some
 *            row of the request sees are read and written.
 * Sums are fp32 in a fixed order; an entry that lies on no page draws nothing.  At most GVR_LONG_MAX_REQUESTS requests.
 */
gvr_status attend_weights(const gvr_cache* cache, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                          int32_t dtype, int64_t num_rows, int32_t num_heads, const int32_t* block_table,
                          int64_t table_stride, int64_t table_width, const int32_t* kv_lens, int32_t next_n,
                          int32_t compress_ratio, const float* lse, float scale, float* weights,
                          int64_t weights_stride, void* stream);

/*
 * Cut each request's cache to `keep` entries.  A request of n = kv_lens / compress_ratio entries (at most
 * table_width * page_size) with n > keep keeps its last `recent` entries and of the others the keep - recent
 * of largest weight, those of equal weight by lower number, a NaN before all numbers, -0 as 0.  They keep their order
 * and become entries 0 .. keep - 1.  Pages before the first one in which an entry changes stay the request's; from there
 * on entries are copied to pages taken from free_pages (ceil(keep / page_size) minus the staying ones, requests in
 * order), and the request's old pages from there on are released.  No page that a request held is written: another
 * request may hold it too, and releasing it means this request's hold alone.
 *   weights      fp32 [num_requests][weights_stride], weights_stride at least table_width * page_size; of a request that is
 *                cut, the kept entries' weights in their new places, and 0 from `keep` to n.
 *   block_table  updated in place: new pages, and -1 for released ones that none replaces.
 *   kept         int32 [num_requests][keep]: the old numbers of the entries that it has now, ascending, -1 behind them; of a request
 *                with n <= keep all its entries.
 *   new_lens     int32 [num_requests]: keep * compress_ratio + kv_lens % compress_ratio where it was cut, else kv_lens.
 *   released     int32 [max_released]: released pages, requests in order, pages in order; -1 behind the last one.  What
 *                it has no room for is only counted.
 *   counts       int32 [3]: pages taken from free_pages, pages released, requests that were left as they were although n > keep:
 *                those from the first one on that free_pages has no pages for (in order, none later is served), and requests with
 *                an entry on no page.  Their row of kept is -1 alone.
 * 1 <= keep < 2^31 / compress_ratio and at most 2^31 - 2^16, 0 <= recent <= keep; num_requests at most GVR_LONG_MAX_REQUESTS, num_requests * table_width and
 * num_requests * keep below 2^31.  free_pages: distinct page numbers not in use.  workspace: 16-byte aligned, cache_evict_workspace's bytes.
 * What is written overlaps nothing else that the call reads or writes, but for new_lens, which may be kv_lens.
 */
gvr_status cache_evict(const gvr_cache* cache, float* weights, int64_t weights_stride, int32_t* block_table,
                       int64_t table_stride, int64_t table_width, const int32_t* kv_lens, int64_t num_requests,
                       int32_t compress_ratio, const int32_t* free_pages, int64_t num_free, int32_t keep, int32_t recent,
                       int32_t* kept, int32_t* new_lens, int32_t* released, int64_t max_released, int32_t* counts,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace that cache_evict needs. */
gvr_status cache_evict_workspace(int64_t num_requests, int32_t keep, size_t* bytes);

/* Static English text for a status returned by the functions of this header; never NULL. */
const char* gvr_long_status_string(gvr_status status);

#ifdef __cplusplus
}
#endif

#endif /* GVR_LONG_H */
