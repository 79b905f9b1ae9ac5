// gvr_cache_index.h -- the index arithmetic of the cache kernels: which entries a row has, and
// where an entry lies.  Plain C++ as well, so that its bounds are tested on the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define GVRC_FN __host__ __device__ __forceinline__
#else
#define GVRC_FN inline
#endif

namespace gvrc {

// Bytes of one row: codes of K and V, scales of K and V, up to a multiple of 16.
GVRC_FN constexpr int row_bytes(int dim) { return (dim + dim / 8 + 15) / 16 * 16; }

// Pages that hold `entries` entries.
GVRC_FN int pages_of(int entries, int page_shift) {
  return int((int64_t(entries) + (int64_t(1) << page_shift) - 1) >> page_shift);
}

// Byte offset of `head`'s row of an entry on `page`, or -1 where that is no page of the cache.
// `entry` is a number from 0 in the request or in the page alike: only its low bits count.
GVRC_FN int64_t row_offset(int page, int num_pages, int entry, int page_shift, int64_t page_stride, int heads, int head,
                           int bytes) {
  if (page < 0 || page >= num_pages) return -1;
  const int64_t in_page = entry & ((1 << page_shift) - 1);
  return int64_t(page) * page_stride + (in_page * heads + head) * bytes;
}

// The same for a slot (page * page_size + offset); -1 where it names no entry.
GVRC_FN int64_t slot_offset(int slot, int num_pages, int page_shift, int64_t page_stride, int heads, int head, int bytes) {
  if (slot < 0) return -1;
  return row_offset(slot >> page_shift, num_pages, slot, page_shift, page_stride, heads, head, bytes);
}

// Number of an entry's row in units of `unit` bytes, given the page stride, the rows of one entry and
// the head's row in the same units; the caller has checked `page`.  Fits 32 bits (units_fit).
GVRC_FN uint32_t row_unit(int page, int entry, int page_shift, uint32_t page_units, uint32_t entry_units, uint32_t head_units) {
  return uint32_t(page) * page_units + uint32_t(entry & ((1 << page_shift) - 1)) * entry_units + head_units;
}

// The unit: a row where the page stride is a multiple of it (caches of up to 2^32 rows, 320 GB and
// more), else 16 bytes (up to 64 GB).
GVRC_FN int unit_bytes(int64_t page_stride, int bytes) { return page_stride % bytes == 0 ? bytes : 16; }
GVRC_FN bool units_fit(int64_t num_pages, int64_t page_stride, int bytes) {
  return num_pages == 0 || page_stride / unit_bytes(page_stride, bytes) <= 4294967295ll / num_pages;
}

// Slot of an entry on `page`; -1 where there is no page or the slot would not fit 31 bits.
GVRC_FN int slot_of(int page, int entry, int page_shift) {
  if (page < 0) return -1;
  const int64_t s = (int64_t(page) << page_shift) + (entry & ((1 << page_shift) - 1));
  return s < 2147483647 ? int(s) : -1;
}

// Entries that row j of a request's next_n decode rows sees.
GVRC_FN int decode_entries(int kv_len, int next_n, int j, int ratio, int capacity) {
  if (kv_len < next_n) return 0;
  const int n = (kv_len - next_n + j + 1) / ratio;
  return n < capacity ? n : capacity;
}

// Entries of a prefill row's window; a start below 0 counts as 0, an end before it as empty.
GVRC_FN int window_entries(int start, int end, int capacity) {
  const int64_t n = int64_t(end) - (start > 0 ? start : 0);
  return n <= 0 ? 0 : n < capacity ? int(n) : capacity;
}

}  // namespace gvrc
