/*
 * gvr_cache.h -- C ABI of libgvrtopk for what surrounds the top-K selection of gvr_topk.h in a
 * serving step: block tables and slot maps built on the GPU, a paged K/V cache held in 4 bits,
 * and attention that reads that cache at the selected entries (or whole).
 *
 * A step of a model that selects, in call order on one stream:
 *   cache_tables    pages for the step's new entries, and the slot of each of them
 *   cache_append    the new K and V rows, quantised, to those slots
 *   topk_decode / topk_prefill (gvr_topk.h)   each row's K entries from its indexer scores
 *   attend_decode / attend_prefill            attention over those entries
 *
 * Entries.  A request whose (uncompressed) cache length is len holds len / compress_ratio entries
 * (integer division), numbered from 0: the columns of its row of indexer scores.
 *
 * The cache.  num_pages pages of page_size entries each, an entry being one row per KV head:
 *   data[page * page_stride + (offset * num_kv_heads + head) * row_bytes], row_bytes from
 *   cache_row_bytes: head_dim / 2 bytes of K codes, head_dim / 2 of V codes, head_dim / 16 of K
 *   scales, head_dim / 16 of V scales, and zero to eight unused bytes up to a multiple of 16
 *   (80, 144, 288 bytes for head_dim 64, 128, 256).
 * A code is e2m1 (sign, two exponent bits, one mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6); value 2i
 * of the head is the low half of byte i.  A scale is e4m3 and belongs to 16 consecutive values.
 * The value held is code * scale * k_scale (or v_scale), the latter a float of the whole cache.
 * Quantising a block of 16 values x: scale = e4m3(min(max|x| / (6 k_scale), 448)), code =
 * e2m1(x / (scale * k_scale)), both to nearest, ties to even, codes saturating at 6; quotients
 * are IEEE fp32.  A block whose scale rounds to 0 holds zeros; infinities saturate; a NaN makes
 * its block's scale NaN, so every value of the block reads as NaN.
 * A slot is page * page_size + offset.  A slot outside [0, num_pages * page_size) (-1 is the
 * usual one) names no entry: nothing is written for it, and it reads as zeros.
 *
 * Block tables.  int32 [requests][table_stride]: block_table[q][b] is the page of entries
 * [b * page_size, (b + 1) * page_size) of request q.  A page outside [0, num_pages) is no page:
 * its entries are skipped.
 *
 * Conventions.  As in gvr_topk.h: all pointers but the gvr_cache itself are device pointers to
 * memory that the caller owns; every call checks its arguments on the host, allocates nothing,
 * reads no device memory on the host, does not synchronise, and enqueues one kernel (attention
 * with a workspace: one or two) on `stream` of the current device, so it can be captured in a
 * graph; calls share no state, on any streams.  Counts of 0 are no-ops that return GVR_OK.  Statuses are those of
 * gvr_topk.h; gvr_cache_status_string says what each means here.  Strides, counts of slots and of free
 * pages, and k are below 2^31.
 */
#ifndef GVR_CACHE_H
#define GVR_CACHE_H

#include "gvr_topk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of q, k, v and out. */
enum { GVR_BF16 = 0, GVR_F16 = 1 };

#define GVR_CACHE_MAX_REQUESTS 8192   /* cache_tables */
#define GVR_CACHE_MAX_PAGE_SIZE 4096
#define GVR_ATTEND_MAX_NEXT_N 4096
#define GVR_ATTEND_MAX_HEADS (1 << 20)
#define GVR_ATTEND_WORKSPACE (1 << 25) /* bytes */

typedef struct gvr_cache {
  void* data;           /* device, 16-byte aligned */
  int64_t num_pages;    /* num_pages * page_size < 2^31 */
  int64_t page_stride;  /* bytes between pages: a multiple of 16, at least
                           page_size * num_kv_heads * row_bytes; the whole cache may span 2^32
                           rows, or 64 GB where the stride is not a multiple of row_bytes */
  int32_t page_size;    /* entries per page: a power of two, 1 to GVR_CACHE_MAX_PAGE_SIZE */
  int32_t num_kv_heads; /* 1 to 65535 */
  int32_t head_dim;     /* 64, 128 or 256 */
  int32_t reserved;     /* must be 0 */
  float k_scale;        /* finite and > 0 */
  float v_scale;        /* finite and > 0 */
} gvr_cache;

/* Bytes of one row (one entry of one KV head): 80, 144 or 288; GVR_ERR_ARG for other head_dim. */
gvr_status cache_row_bytes(int32_t head_dim, int32_t* bytes);

/*
 * Block tables and slot maps of one step.  Request q grows from cached_lens[q] to kv_lens[q]
 * (uncompressed lengths; negative ones count as 0), so from e0 = cached / compress_ratio entries
 * to e1 = kv / compress_ratio (no growth where e1 <= e0).  It holds ceil(e0 / page_size) pages
 * and needs min(ceil(e1 / page_size), table_width); the new ones are taken from free_pages in
 * order, requests in order.
 *   block_table  updated in place: the new pages' numbers, -1 where free_pages has run out;
 *                every other element is left as it is.
 *   slots        int32 [num_slots]: the slots of all new entries, requests in order, entries in
 *                order; -1 for an entry that has no page, and behind the last one.
 *   counts       int32 [3]: new entries (whether slots has room for them or not), pages taken
 *                from free_pages, pages missing (beyond free_pages or beyond table_width).  Sums
 *                saturate at 2^31 - 1.
 *   cached_lens, kv_lens  int32 [num_requests], num_requests <= GVR_CACHE_MAX_REQUESTS.
 *   free_pages   int32 [num_free], distinct page numbers not in use; may be NULL if num_free is 0.
 * table_width * page_size < 2^31; num_requests * table_width < 2^31; table_stride >= table_width.
 * With no requests counts and slots are still written (0 and -1).
 */
gvr_status cache_tables(const int32_t* cached_lens, const int32_t* kv_lens, int64_t num_requests,
                        int32_t compress_ratio, int32_t page_size, const int32_t* free_pages,
                        int64_t num_free, int32_t* block_table, int64_t table_stride,
                        int64_t table_width, int32_t* slots, int64_t num_slots, int32_t* counts,
                        void* stream);

/*
 * Quantise K and V rows into the cache: k and v are [num_tokens][num_kv_heads][head_dim] of
 * `dtype` with unit inner stride and the given token and head strides (in elements, multiples of
 * 8; bases 16-byte aligned); token t goes to slots[t].  Slots that name an entry must be
 * distinct: what an entry named twice holds is unspecified (nothing else is affected).
 * num_tokens * num_kv_heads < 2^31.
 */
gvr_status cache_append(const gvr_cache* cache, const void* k, int64_t k_token_stride,
                        int64_t k_head_stride, const void* v, int64_t v_token_stride,
                        int64_t v_head_stride, int32_t dtype, const int32_t* slots,
                        int64_t num_tokens, void* stream);

/*
 * The values held at slots[0 .. num_tokens): k and v, packed [num_tokens][num_kv_heads][head_dim]
 * of `dtype`, 16-byte aligned, either may be NULL.  code * scale is exact in both types;
 * k_scale and v_scale are multiplied in fp32 and the product rounded to `dtype`.
 * num_tokens * num_kv_heads < 2^31.
 */
gvr_status cache_read(const gvr_cache* cache, const int32_t* slots, int64_t num_tokens,
                      int32_t dtype, void* k, void* v, void* stream);

/*
 * Attention of decode rows over the cache.  Row r belongs to request r / next_n and sees its
 * entries [0, n_r), n_r exactly as in topk_decode (0 when kv_lens < next_n), clamped to
 * table_width * page_size.  Query head h reads KV head h / (num_heads / num_kv_heads).  next_n is 1 to
 * GVR_ATTEND_MAX_NEXT_N, num_heads a multiple of num_kv_heads up to GVR_ATTEND_MAX_HEADS.  What no grid
 * holds is refused (GVR_ERR_ARG): KV heads times tiles of 8 to 32 of the queries that share one (num_heads /
 * num_kv_heads, times next_n over whole caches) above 65535.
 *   q       [num_rows][num_heads][head_dim] of `dtype`, unit inner stride, row and head strides in
 *           elements (multiples of 8; base 16-byte aligned).
 *   indices int32 [num_rows][k]: the entries that the row attends to, as topk_decode writes them;
 *           NULL: all n_r entries (k is then ignored).  An index outside [0, n_r) (the -1 pad, the
 *           -2 of a failed row) is skipped; one that occurs twice counts twice.
 *   scale   factor of the scores q . k (1 / sqrt(head_dim) is usual); scale * k_scale finite in fp32.
 *   out     [num_rows][num_heads][head_dim] of `dtype`, packed, 16-byte aligned: softmax over the
 *           row's entries times V.  A row without entries gets zeros.
 *   lse     optional fp32 [num_rows][num_heads]: log of the sum of exp(scale * q . k); -infinity
 *           for a row without entries.  (Merges this with attention over other entries.)
 *   workspace  optional device memory, 16-byte aligned, of any content and size: with it, rows of
 *           many entries and of unequal lengths are spread evenly over the device, in two kernels,
 *           where workspace_bytes is enough (GVR_ATTEND_WORKSPACE always is).  How many is judged by k
 *           or, over whole caches, by the table's width; selections of up to 2048 entries are mostly
 *           faster without a workspace (700 rows of 2048: 159 us with, 142 without).  Its content is not
 *           kept: calls that can overlap on the GPU, or graphs whose replays can, need one each.
 * Scores, softmax and sums are fp32; K and V values are exact.  Before they multiply V, softmax weights
 * exp(score) are rounded to 11-bit significands; those below 2^-21 of the largest that is summed with them
 * (part of the row, or all) are off by at most 2^-32 of that largest one instead.
 */
gvr_status attend_decode(const gvr_cache* cache, const void* q, int64_t q_row_stride,
                         int64_t q_head_stride, int32_t dtype, int64_t num_rows, int32_t num_heads,
                         const int32_t* block_table, int64_t table_stride, int64_t table_width,
                         const int32_t* kv_lens, int32_t next_n, int32_t compress_ratio,
                         const int32_t* indices, int64_t k, float scale, void* out, float* lse,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * Attention of prefill rows over their selection.  Row r belongs to request row_requests[r] and
 * sees that request's entries [0, row_ends[r] - row_starts[r]) (clamped as in attend_decode); a
 * row whose request is outside [0, num_requests) sees none.  row_starts and row_ends are the ones
 * given to topk_prefill, so that its local indices are entry numbers.  indices (required) and
 * everything else as in attend_decode.
 *   row_requests, row_starts, row_ends  int32 [num_rows].
 */
gvr_status attend_prefill(const gvr_cache* cache, const void* q, int64_t q_row_stride,
                          int64_t q_head_stride, int32_t dtype, int64_t num_rows, int32_t num_heads,
                          const int32_t* block_table, int64_t table_stride, int64_t table_width,
                          int64_t num_requests, const int32_t* row_requests,
                          const int32_t* row_starts, const int32_t* row_ends,
                          const int32_t* indices, int64_t k, float scale, void* out, float* lse,
                          void* workspace, size_t workspace_bytes, void* stream);

/* Static English text for a status returned by the functions of this header; never NULL. */
const char* gvr_cache_status_string(gvr_status status);

#ifdef __cplusplus
}
#endif

#endif /* GVR_CACHE_H */
