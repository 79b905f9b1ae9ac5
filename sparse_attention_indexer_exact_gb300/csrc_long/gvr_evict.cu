// gvr_evict.cu -- cache_evict of include/gvr_long.h: which entries of each request stay, and their rows in pages of
// their own.
//
// Two kernels.  The first, a cluster of CTAs a request, finds the M = keep - recent heaviest of the n - recent older
// entries: an exact radix selection over order-preserving 32-bit keys, three digits of 11, 11 and 10 bits from the top, each
// from a histogram in shared memory that the cluster adds up, until all of the crossing bin stays; the keys stay in shared memory
// after the first pass.  Then one
// ordered pass writes the chosen entries' numbers, slots and weights: a position is the number of chosen entries
// before it, so the result does not depend on the order of execution.  The second kernel, CTAs over all requests' new
// entries, copies rows into the new pages and rewrites weights, tables and lists.  Nothing is moved in place: old pages
// are only read, so copies need no order among each other, and pages that other requests hold stay what they are.
//
// What bounds them.  64 requests of up to 5200 entries cut to 4096 (8 heads of 128): 90 to 93 us, of which 67 to 70 copy 490 MB in and out
// at 5.7 to 5.8 TB/s under the profiler (0.85 of the copy rate back to back); the selection's 16 are a chain of barriers, cluster
// round trips and scans.  One request of 9000: 24 to 28 us, 15 and 8.  Five of up to 131072 cut to 20000: 55 to 59, 31 and 23
// (eight CTAs a request hold 16384 keys each; 40 us before the cluster's histograms were read at once).
#include <algorithm>
#include <mutex>

#include "../csrc_cache/gvr_cache_common.cuh"
#include "../csrc/gvr_device.cuh"
#include "gvr_long_common.h"

namespace gvrc {
namespace {

constexpr int BINS = 2048;
constexpr int MAX_KEYS = 48 * 1024;  // of a CTA, in shared memory; what is beyond is read from memory in every pass
constexpr int SLICE = 4096;          // entries worth a CTA
constexpr int MOVE_THREADS = 256;
constexpr int MOVE_BYTES = 1 << 16;  // rows that a CTA copies, about

// What the first kernel leaves of each request for the second.
struct Cut {
  int32_t first;    // the first page that is made anew
  int32_t need;     // pages to take
  int32_t release;  // pages to release
  int32_t state;    // WHOLE: n <= keep; CUT; UNPAGED: an entry lies on no page
  int32_t entries;  // n  (new_lens may lie over kv_lens)
};
enum { WHOLE = 0, CUT = 1, UNPAGED = 2 };

struct EvictParams {
  uint8_t* data;
  float* weights;
  int32_t* table;
  const int32_t* lens;
  const int32_t* free_pages;
  int32_t* kept;
  int32_t* new_lens;
  int32_t* released;
  int32_t* counts;
  Cut* cuts;             // [requests]
  int32_t* slots;        // [requests][keep]: of the kept entries, before
  float* few;            // [requests][keep]: their weights
  int64_t weights_stride, table_stride, page_stride, num_free, max_released;
  int32_t requests, ratio, keep, recent, num_pages, page_shift, capacity, entry_bytes, chunk;
};

__device__ __forceinline__ int entries_of(const EvictParams& p, int r) { return min(max(p.lens[r], 0) / p.ratio, p.capacity); }

// Two or four neighbouring words of a CTA's shared memory in the cluster.
__device__ __forceinline__ void dsmem_words(uint32_t at, uint32_t (&w)[2]) {
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
}
__device__ __forceinline__ void dsmem_words(uint32_t at, uint32_t (&w)[4]) {
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
}

// A NaN before all numbers.
__device__ __forceinline__ uint32_t weight_key(float w) { return w != w ? 0xffffffffu : gvr::order_key(w); }

// Sums over the CTA's threads before this one, and over all, of a pair of counts; `sums` is shared, [32].
template <int WARPS>
__device__ __forceinline__ uint2 scan_before(uint2 v, uint2* sums, uint2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint2 x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, x.x, d), b = __shfl_up_sync(0xffffffffu, x.y, d);
    if (lane >= d) x.x += a, x.y += b;
  }
  __syncthreads();  // the sums of a scan before this one are read
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  uint2 s = lane < WARPS ? sums[lane] : make_uint2(0, 0);
#pragma unroll
  for (int d = 1; d < WARPS; d <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, s.x, d), b = __shfl_up_sync(0xffffffffu, s.y, d);
    if (lane >= d) s.x += a, s.y += b;
  }
  total = make_uint2(__shfl_sync(0xffffffffu, s.x, WARPS - 1), __shfl_sync(0xffffffffu, s.y, WARPS - 1));
  const uint32_t bx = __shfl_sync(0xffffffffu, s.x, max(warp - 1, 0)), by = __shfl_sync(0xffffffffu, s.y, max(warp - 1, 0));
  return make_uint2(x.x - v.x + (warp ? bx : 0), x.y - v.y + (warp ? by : 0));
}

template <int SELECT_THREADS>
__global__ void __launch_bounds__(SELECT_THREADS, 1024 / SELECT_THREADS) evict_select_kernel(EvictParams p) {
  constexpr int WARPS = SELECT_THREADS / 32, OWN = BINS / SELECT_THREADS;  // bins of a thread
  extern __shared__ __align__(16) uint32_t keys[];  // [min(slice, MAX_KEYS)]
  __shared__ __align__(16) uint32_t hist[3][BINS];
  __shared__ uint2 sums[32];
  __shared__ uint32_t found[3];    // the crossing bin, what is still wanted of it, and what it holds
  __shared__ uint32_t mine_of[4];  // of this CTA: entries above the threshold, equal to it; first entry that goes; a missing page
  const int tid = threadIdx.x;
  const int rank = int(gvr::cluster_rank()), cs = int(gvr::cluster_size()), r = int(cs == 1 ? blockIdx.x : gvr::cluster_id_x());
  for (int i = tid; i < 3 * BINS; i += SELECT_THREADS) (&hist[0][0])[i] = 0;
  if (tid == 0) mine_of[2] = 0xffffffffu, mine_of[3] = 0;
  begin();
  // the list of released pages, which may be as long as the table; the pages come in with the next kernel
  for (int64_t i = int64_t(blockIdx.x) * SELECT_THREADS + tid; i < p.max_released; i += int64_t(gridDim.x) * SELECT_THREADS) p.released[i] = -1;
  const int n = entries_of(p, r);
  int32_t* kept = p.kept + int64_t(r) * p.keep;
  if (n <= p.keep) {  // by all CTAs of the cluster alike
    for (int i = rank * SELECT_THREADS + tid; i < p.keep; i += cs * SELECT_THREADS) kept[i] = i < n ? i : -1;
    if (rank == 0 && tid == 0) p.cuts[r] = {0, 0, 0, WHOLE, n};
    return;
  }
  const int32_t* table = p.table + r * p.table_stride;
  const float* weights = p.weights + r * p.weights_stride;
  const int older = n - p.recent, pages = pages_of(n, p.page_shift);
  const int slice = (n + cs - 1) / cs, from = min(rank * slice, n), to = min(from + slice, n);
  const int old_to = min(to, older), held = min(slice, MAX_KEYS);  // keys below from + held are in shared memory
  uint32_t want = uint32_t(p.keep - p.recent);
  __syncthreads();

  bool missing = false;
  for (int b = rank * SELECT_THREADS + tid; b < pages; b += cs * SELECT_THREADS) missing |= uint32_t(table[b]) >= uint32_t(p.num_pages);
  if (missing) mine_of[3] = 1;
  auto key_at = [&](int i) -> uint32_t { return i - from < held ? keys[i - from] : weight_key(weights[i]); };

  // ---- the threshold: the want-th largest key, digit by digit
  uint32_t prefix = 0;  // digits found
  int drop = 0;         // bits below them, which do not matter
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t mask = pass == 2 ? 1023 : 2047;
    if (pass == 0) {
#pragma unroll 4
      for (int i = from + tid; i < old_to; i += SELECT_THREADS) {
        const uint32_t k = weight_key(weights[i]);
        if (i - from < held) keys[i - from] = k;
        atomicAdd(&hist[0][k >> 21], 1);
      }
    } else {
      const int below = pass == 1 ? 21 : 10;  // bits below the digits found
      for (int i = from + tid; i < old_to; i += SELECT_THREADS) {
        const uint32_t k = key_at(i);
        if (k >> below == prefix) atomicAdd(&hist[pass][(k >> shift) & mask], 1);
      }
    }
    if (cs > 1) gvr::cluster_sync();
    else __syncthreads();
    // a thread's bins, the highest first: how many keys of the cluster lie in them and above
    const int bin = BINS - OWN - OWN * tid;
    uint32_t own[OWN], sum = 0;
#pragma unroll
    for (int j = 0; j < OWN; ++j) own[j] = cs > 1 ? 0 : hist[pass][bin + j];
    if (cs > 1) {
      uint32_t from_rank[8][OWN];  // all on their way at once
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < cs) dsmem_words(gvr::dsmem_map(gvr::smem_u32(&hist[pass][bin]), c), from_rank[c]);
#pragma unroll
      for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int j = 0; j < OWN; ++j)
          if (c < cs) own[j] += from_rank[c][j];
    }
#pragma unroll
    for (int j = 0; j < OWN; ++j) sum += own[j];
    uint2 total;
    uint32_t above = scan_before<WARPS>(make_uint2(sum, 0), sums, total).x;
#pragma unroll
    for (int j = OWN - 1; j >= 0; --j) {
      if (above < want && want <= above + own[j]) found[0] = bin + j, found[1] = want - above, found[2] = own[j];
      above += own[j];
    }
    if (tid == 0 && want == 0) found[0] = found[1] = found[2] = 0;  // nothing is wanted, whatever the threshold
    __syncthreads();
    prefix = pass == 0 ? found[0] : prefix << (pass == 1 ? 11 : 10) | found[0];
    want = found[1], drop = shift;
    if (want == found[2]) break;  // all of the bin stays
    __syncthreads();  // they are read before the next pass finds its own
  }
  const uint32_t threshold = prefix, ties = want;  // `ties` entries that equal it stay, those with the lowest numbers
  const bool none = p.keep == p.recent;

  // ---- what lies in the CTAs before this one
  uint2 before = make_uint2(0, 0), total;
  {
    uint2 own = make_uint2(0, 0);
    for (int i = from + tid; i < old_to; i += SELECT_THREADS) {
      const uint32_t k = key_at(i) >> drop;
      own.x += k > threshold, own.y += k == threshold;
    }
    scan_before<WARPS>(own, sums, total);
    if (none) total = make_uint2(0, 0);
    if (tid == 0) mine_of[0] = total.x, mine_of[1] = total.y;
    if (cs > 1) {
      gvr::cluster_sync();
      for (int c = 0; c < rank; ++c) {
        const uint32_t at = gvr::dsmem_map(gvr::smem_u32(mine_of), c);
        before.x += gvr::dsmem_ld_u32(at), before.y += gvr::dsmem_ld_u32(at + 4);
      }
    }
  }

  let_next_start();  // 0.4 to 0.7 us
  // ---- the chosen entries, in order
  int32_t* slots = p.slots + int64_t(r) * p.keep;
  float* few = p.few + int64_t(r) * p.keep;
  const int page_mask = (1 << p.page_shift) - 1;
  uint32_t goes = 0xffffffffu;
  for (int i0 = from; i0 < old_to; i0 += 4 * SELECT_THREADS) {
    uint32_t is[4];
    int page[4];
    float weight[4];
    uint2 own = make_uint2(0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 4 * tid + j;
      if (i < old_to) page[j] = table[i >> p.page_shift], weight[j] = weights[i];  // on their way beside the scan
      const uint32_t k = i < old_to && !none ? key_at(i) >> drop : 0;
      is[j] = i >= old_to ? 3 : none ? 2 : k > threshold ? 0 : k == threshold ? 1 : 2;
      own.x += is[j] == 0, own.y += is[j] == 1;
    }
    uint2 at = scan_before<WARPS>(own, sums, total);
    at.x += before.x, at.y += before.y;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 4 * tid + j;
      if (is[j] == 0 || (is[j] == 1 && at.y < ties)) {
        const int to = int(at.x + min(at.y, ties));
        kept[to] = i, slots[to] = int(uint32_t(page[j]) << p.page_shift) + (i & page_mask), few[to] = weight[j];
      } else if (is[j] != 3) {
        goes = min(goes, uint32_t(i));
      }
      at.x += is[j] == 0, at.y += is[j] == 1;
    }
    before.x += total.x, before.y += total.y;
  }
  for (int i = max(from, older) + tid; i < to; i += SELECT_THREADS) {
    const int at = p.keep - p.recent + (i - older);
    kept[at] = i, slots[at] = int(uint32_t(table[i >> p.page_shift]) << p.page_shift) + (i & page_mask), few[at] = weights[i];
  }

  goes = __reduce_min_sync(0xffffffffu, goes);
  if ((tid & 31) == 0 && goes != 0xffffffffu) atomicMin(&mine_of[2], goes);
  if (cs > 1) gvr::cluster_sync();
  else __syncthreads();
  if (rank == 0 && tid == 0) {
    uint32_t lacks = 0;
    goes = 0xffffffffu;
    for (int c = 0; c < cs; ++c) {
      const uint32_t at = gvr::dsmem_map(gvr::smem_u32(mine_of), c);
      goes = min(goes, gvr::dsmem_ld_u32(at + 8)), lacks |= gvr::dsmem_ld_u32(at + 12);
    }
    // (keep, where the first that goes lies behind: the entries added next are not written into a page that
    // another request may hold)
    const int first = min(int(goes), p.keep) >> p.page_shift;
    if (lacks) p.cuts[r] = {0, 0, 0, UNPAGED, n};
    else p.cuts[r] = {first, pages_of(p.keep, p.page_shift) - first, pages - first, CUT, n};
  }
  if (cs > 1) gvr::cluster_sync();  // no CTA leaves while another reads its shared memory
}

// Sum over the CTA; `sums` is shared, [MOVE_THREADS / 32].
__device__ __forceinline__ int64_t sum_all(int64_t x, int64_t* sums) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0;
#pragma unroll
  for (int w = 0; w < MOVE_THREADS / 32; ++w) x += sums[w];
  return x;
}

__global__ void __launch_bounds__(MOVE_THREADS) evict_move_kernel(EvictParams p) {
  extern __shared__ __align__(16) int64_t places[];  // [2][chunk]: where the chunk's entries lie, and go
  __shared__ int64_t sums[MOVE_THREADS / 32];
  const int tid = threadIdx.x, r = blockIdx.y, chunk0 = blockIdx.x * p.chunk, chunk1 = min(chunk0 + p.chunk, p.keep);
  begin();
  const Cut cut = p.cuts[r];
  if (blockIdx.x == 0 && tid == 0 && cut.state == WHOLE) p.new_lens[r] = p.lens[r];
  int64_t before = 0, gone = 0;  // pages that the requests before this one take, and release
  const bool lists = blockIdx.x == 0;
  if (cut.state == CUT || lists) {
    for (int i = tid; i < r; i += MOVE_THREADS) before += p.cuts[i].need, gone += p.cuts[i].release;
    before = sum_all(before, sums), gone = sum_all(gone, sums);
  }
  const bool served = cut.state == CUT && before + cut.need <= p.num_free;
  if (lists && r == 0) {  // the sums over all requests; the requests served are a first part of them, as sums only grow
    int64_t taken = 0, back = 0, left = 0, so_far = 0;
    for (int i0 = 0; i0 < p.requests; i0 += MOVE_THREADS) {
      const int i = i0 + tid;
      const Cut c = i < p.requests ? p.cuts[i] : Cut{0, 0, 0, WHOLE, 0};
      int64_t x = c.need;  // inclusive sum over the threads
      const int lane = tid & 31;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      __syncthreads();
      if (lane == 31) sums[tid >> 5] = x;
      __syncthreads();
      int64_t all = 0;
      for (int w = 0; w < MOVE_THREADS / 32; ++w) {
        if (w == tid >> 5) x += all;
        all += sums[w];
      }
      const bool is = c.state == CUT && so_far + x <= p.num_free;
      if (is) taken += c.need, back += c.release;
      left += c.state != WHOLE && !is;
      so_far += all;
    }
    taken = sum_all(taken, sums), back = sum_all(back, sums), left = sum_all(left, sums);
    if (tid == 0) p.counts[0] = int(taken), p.counts[1] = int(back), p.counts[2] = int(left);
  }
  if (!served) {
    if (cut.state != WHOLE) {
      for (int i = chunk0 + tid; i < chunk1; i += MOVE_THREADS) p.kept[int64_t(r) * p.keep + i] = -1;
      if (lists && tid == 0) p.new_lens[r] = p.lens[r];
    }
    return;
  }

  if (lists) {
    if (tid == 0) p.new_lens[r] = p.keep * p.ratio + p.lens[r] % p.ratio;
    int32_t* table = p.table + r * p.table_stride + cut.first;
    for (int i = tid; i < cut.release; i += MOVE_THREADS) {
      if (gone + i < p.max_released) p.released[gone + i] = table[i];
      table[i] = i < cut.need ? p.free_pages[before + i] : -1;
    }
  }
  // weights: this chunk's kept ones, and its share of the zeros behind them
  float* weights = p.weights + r * p.weights_stride;
  for (int i = chunk0 + tid; i < chunk1; i += MOVE_THREADS) weights[i] = p.few[int64_t(r) * p.keep + i];
  for (int64_t i = p.keep + int64_t(blockIdx.x) * MOVE_THREADS + tid; i < cut.entries; i += int64_t(gridDim.x) * MOVE_THREADS) weights[i] = 0.f;

  // rows: an entry's rows of all heads lie next to each other
  const int start = max(chunk0, cut.first << p.page_shift), count = chunk1 - start, page_mask = (1 << p.page_shift) - 1;
  if (count <= 0) return;
  int64_t *src = places, *dst = places + p.chunk;
  for (int i = tid; i < count; i += MOVE_THREADS) {
    const int at = start + i, slot = p.slots[int64_t(r) * p.keep + at];
    const int page = p.free_pages[before + (at >> p.page_shift) - cut.first];
    src[i] = (slot >> p.page_shift) * p.page_stride + int64_t(slot & page_mask) * p.entry_bytes;
    dst[i] = uint32_t(page) < uint32_t(p.num_pages) ? page * p.page_stride + int64_t(at & page_mask) * p.entry_bytes : -1;
  }
  __syncthreads();
  const int pieces = p.entry_bytes / 16, skip = MOVE_THREADS / pieces, step = MOVE_THREADS % pieces;
  int e = tid / pieces, piece = tid % pieces;
  constexpr int AHEAD = 8;
  while (e < count) {
    uint4 v[AHEAD];
    int64_t to[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      to[j] = -1;
      if (e < count) {
        v[j] = *reinterpret_cast<const uint4*>(p.data + src[e] + piece * 16);
        if (dst[e] >= 0) to[j] = dst[e] + piece * 16;
      }
      e += skip, piece += step;
      if (piece >= pieces) piece -= pieces, ++e;
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      if (to[j] >= 0) *reinterpret_cast<uint4*>(p.data + to[j]) = v[j];
  }
}

struct EvictDevice {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
};
EvictDevice g_evict_devices[kMaxDevices];

int64_t align16(int64_t x) { return (x + 15) / 16 * 16; }

}  // namespace
}  // namespace gvrc

extern "C" {

gvr_status cache_evict_workspace(int64_t num_requests, int32_t keep, size_t* bytes) {
  using namespace gvrc;
  if (!bytes) return GVR_ERR_NULL;
  if (num_requests < 0 || num_requests > GVR_LONG_MAX_REQUESTS || keep < 1 || keep > MAX_ENTRIES || (num_requests > 0 && keep > kIntMax / num_requests)) return GVR_ERR_ARG;
  *bytes = size_t(align16(num_requests * int64_t(sizeof(Cut))) + 2 * align16(num_requests * keep * 4));
  return GVR_OK;
}

gvr_status cache_evict(const gvr_cache* cache, float* weights, int64_t weights_stride, int32_t* block_table,
                       int64_t table_stride, int64_t table_width, const int32_t* kv_lens, int64_t num_requests,
                       int32_t compress_ratio, const int32_t* free_pages, int64_t num_free, int32_t keep, int32_t recent,
                       int32_t* kept, int32_t* new_lens, int32_t* released, int64_t max_released, int32_t* counts,
                       void* workspace, size_t workspace_bytes, void* stream) {
  using namespace gvrc;
  const gvr_status s = check_cache(cache);
  if (s != GVR_OK) return s;
  size_t least = 0;
  const gvr_status w = cache_evict_workspace(num_requests, keep, &least);
  if (w != GVR_OK) return w;
  if (compress_ratio < 1 || keep > kIntMax / compress_ratio || recent < 0 || recent > keep || num_free < 0 || num_free > kIntMax ||
      max_released < 0 || max_released > kIntMax || table_width < 0 || table_width > MAX_ENTRIES / cache->page_size ||
      (num_requests > 0 && table_width > kIntMax / num_requests))
    return GVR_ERR_ARG;
  // the last length is keep * ratio + ratio - 1
  if (int64_t(keep) * compress_ratio + compress_ratio - 1 > kIntMax) return GVR_ERR_ARG;
  if (table_stride < table_width || table_stride > kIntMax || weights_stride < table_width * cache->page_size || weights_stride > kIntMax)
    return GVR_ERR_STRIDE;
  if (!counts || (max_released > 0 && !released) || (num_free > 0 && !free_pages)) return GVR_ERR_NULL;
  if (num_requests > 0 && (!kv_lens || !kept || !new_lens || (table_width > 0 && (!block_table || !weights)))) return GVR_ERR_NULL;
  if (!aligned(weights, 4) || !aligned(block_table, 4) || !aligned(kv_lens, 4) || !aligned(free_pages, 4) || !aligned(kept, 4) ||
      !aligned(new_lens, 4) || !aligned(released, 4) || !aligned(counts, 4))
    return GVR_ERR_ALIGN;
  if (num_requests > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < least)) return GVR_ERR_WORKSPACE;
  if (num_requests == 0) {
    // nothing to cut; the lists are still written, by the copy engine
    if (cudaMemsetAsync(counts, 0, 12, static_cast<cudaStream_t>(stream)) != cudaSuccess) return GVR_ERR_LAUNCH;
    if (max_released > 0 && cudaMemsetAsync(released, 0xff, size_t(max_released) * 4, static_cast<cudaStream_t>(stream)) != cudaSuccess) return GVR_ERR_LAUNCH;
    return GVR_OK;
  }
  int sms = 0, dev = 0;
  if (sm_count(&sms) != cudaSuccess || cudaGetDevice(&dev) != cudaSuccess) return GVR_ERR_LAUNCH;
  EvictDevice& d = g_evict_devices[dev];  // sm_count has checked dev
  std::call_once(d.once, [&d]() {
    d.err = cudaFuncSetAttribute(evict_select_kernel<1024>, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_KEYS * 4);
    if (d.err == cudaSuccess) d.err = cudaFuncSetAttribute(evict_select_kernel<512>, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_KEYS * 4);
  });
  if (d.err != cudaSuccess) return GVR_ERR_LAUNCH;
  EvictParams p = {};
  p.data = static_cast<uint8_t*>(cache->data);
  p.weights = weights;
  p.table = block_table;
  p.lens = kv_lens;
  p.free_pages = free_pages;
  p.kept = kept;
  p.new_lens = new_lens;
  p.released = released;
  p.counts = counts;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.cuts = reinterpret_cast<Cut*>(ws);
  p.slots = reinterpret_cast<int32_t*>(ws + align16(num_requests * int64_t(sizeof(Cut))));
  p.few = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(p.slots) + align16(num_requests * keep * 4));
  p.weights_stride = weights_stride;
  p.table_stride = table_stride;
  p.page_stride = cache->page_stride;
  p.num_free = num_free;
  p.max_released = max_released;
  p.requests = int32_t(num_requests);
  p.ratio = compress_ratio;
  p.keep = keep;
  p.recent = recent;
  p.num_pages = int32_t(cache->num_pages);
  p.page_shift = log2_of(cache->page_size);
  p.capacity = cache->num_pages > 0 ? int32_t(table_width * cache->page_size) : 0;
  const int64_t entry_bytes = int64_t(cache->num_kv_heads) * row_bytes(cache->head_dim);
  p.entry_bytes = int32_t(entry_bytes);
  p.chunk = int32_t(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(keep, 1024), MOVE_BYTES / entry_bytes)));
  // CTAs a request: as many as its entries are worth, and as lie beside the other requests'
  int cs = 1;
  while (cs < 8 && int64_t(cs) * SLICE < p.capacity && (num_requests * cs * 2 <= sms || int64_t(cs) * MAX_KEYS < p.capacity)) cs *= 2;
  const int64_t slice = (int64_t(p.capacity) + cs - 1) / cs;
  const int smem = int(std::min<int64_t>(slice, MAX_KEYS)) * 4;
  void* args[] = {&p};
  // two CTAs an SM where there are that many
  const bool small = num_requests * cs > sms && slice <= SLICE;
  cudaError_t e = launch(small ? reinterpret_cast<const void*>(evict_select_kernel<512>) : reinterpret_cast<const void*>(evict_select_kernel<1024>),
                         dim3(uint32_t(num_requests * cs)), small ? 512 : 1024, smem, cs, args, stream);
  if (e == cudaSuccess) {
    const int64_t chunks = (int64_t(keep) + p.chunk - 1) / p.chunk;
    e = launch(reinterpret_cast<const void*>(evict_move_kernel), dim3(uint32_t(chunks), uint32_t(num_requests)), MOVE_THREADS, 2 * p.chunk * 8, 1, args, stream);
  }
  return e == cudaSuccess ? GVR_OK : GVR_ERR_LAUNCH;
}

const char* gvr_long_status_string(gvr_status status) {
  switch (status) {
    case GVR_ERR_STRIDE:
      return "a stride is out of range: page strides a multiple of 16 bytes that holds a page, q strides multiples of 8 elements, "
             "table strides at least the table's width, weight strides at least the entries of a table's row";
    case GVR_ERR_ARG:
      return "invalid argument (head_dim 64, 128 or 256; page_size a power of two; counts, ratios, scales, heads, dtype, "
             "keep at least 1, recent 0 to keep, at most 8192 requests and groups)";
    case GVR_ERR_WORKSPACE: return "the workspace is NULL, not 16-byte aligned or too small";
    default: return gvr_cache_status_string(status);
  }
}

}  // extern "C"
