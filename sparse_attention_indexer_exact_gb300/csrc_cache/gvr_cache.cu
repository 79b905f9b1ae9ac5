// gvr_cache.cu -- block tables and slot maps, and the 4-bit cache's writes and reads (declared in
// include/gvr_cache.h).
#include <cuda_bf16.h>

#include <mutex>

#include "gvr_cache_common.cuh"

namespace gvrc {

namespace {
struct Device {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
  int sms = 0;
};
Device g_devices[kMaxDevices];
}  // namespace

cudaError_t sm_count(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  Device& d = g_devices[dev];
  std::call_once(d.once, [&d, dev]() {
    d.err = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
  });
  *sms = d.sms;
  return d.err;
}

namespace {

// ------------------------------------------------------------------------------------- tables
constexpr int TABLE_THREADS = 512, TABLE_THREADS_SMALL = 128;

struct TableParams {
  const int32_t* cached;
  const int32_t* lens;
  const int32_t* free_pages;
  int32_t* table;
  int32_t* slots;
  int32_t* counts;
  int64_t table_stride;
  int64_t num_slots;
  int32_t requests, ratio, page_shift, num_free, width;
};

// a + b for 0 <= a, b <= 2^31 - 1, at most 2^31 - 1: associative, so any order of summing gives
// the same result.
__device__ __forceinline__ int sat_add(int a, int b) { return int(min(uint32_t(a) + uint32_t(b), 0x7fffffffu)); }

struct Growth {
  int entries;     // e0: entries held before
  int new_entries; // max(e1 - e0, 0)
  int have;        // pages held before
  int new_pages;
  int missing;     // pages beyond the table's width
};

__device__ __forceinline__ Growth growth(const TableParams& p, int r) {
  const int e0 = max(p.cached[r], 0) / p.ratio, e1 = max(p.lens[r], 0) / p.ratio;
  Growth g;
  g.entries = e0;
  g.new_entries = max(e1 - e0, 0);
  g.have = pages_of(e0, p.page_shift);
  const int want = pages_of(e1, p.page_shift), need = min(want, p.width);
  g.new_pages = max(need - g.have, 0);
  g.missing = want - need;
  return g;
}

// The last r with first[r] <= x (first is non-decreasing, first[0] = 0 <= x): the request that
// element x of the concatenated lists belongs to, x being below their total.
__device__ __forceinline__ int owner(const int* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Every CTA reads all lengths and scans them (8 bytes a request, from L2 after the first), then
// takes its share of the two concatenated lists: new pages and new entries.  One launch, no
// exchange between CTAs.  The smallest call is a chain of two global round trips (lengths, then a
// page number) around the scan; the largest is bound by the 4 bytes written per slot and that scan.
// 64 requests, one new entry each: 2.2 us.  230 prompts of 1 to 8192 tokens: 7.7 us (1.2 at the rate of a copy).
template <int THREADS, int VEC>
__global__ void __launch_bounds__(THREADS) cache_tables_kernel(TableParams p) {
  constexpr int WARPS = THREADS / 32;
  extern __shared__ int table_smem[];
  int* page_first = table_smem;             // exclusive sums of new pages
  int* entry_first = page_first + p.requests;  // exclusive sums of new entries
  int* held = entry_first + p.requests;     // e0
  __shared__ int warp_pages[WARPS], warp_entries[WARPS], warp_missing[WARPS];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  begin();
  const int per = (p.requests + THREADS - 1) / THREADS;
  const int r0 = min(tid * per, p.requests), r1 = min(r0 + per, p.requests);
  int pages = 0, entries = 0, missing = 0;
  for (int r = r0; r < r1; ++r) {
    const Growth g = growth(p, r);
    page_first[r] = pages;
    entry_first[r] = entries;
    held[r] = g.entries;
    pages = sat_add(pages, g.new_pages);
    entries = sat_add(entries, g.new_entries);
    missing = sat_add(missing, g.missing);
  }
  // inclusive scan over the threads' sums
  int in_pages = pages, in_entries = entries;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, in_pages, d), b = __shfl_up_sync(0xffffffffu, in_entries, d);
    if (lane >= d) {
      in_pages = sat_add(in_pages, a);
      in_entries = sat_add(in_entries, b);
    }
    missing = sat_add(missing, __shfl_xor_sync(0xffffffffu, missing, d));
  }
  int before_pages = __shfl_up_sync(0xffffffffu, in_pages, 1), before_entries = __shfl_up_sync(0xffffffffu, in_entries, 1);
  if (lane == 0) before_pages = before_entries = 0;
  if (lane == 31) {
    warp_pages[warp] = in_pages;
    warp_entries[warp] = in_entries;
    warp_missing[warp] = missing;
  }
  __syncthreads();
  int total_pages = 0, total_entries = 0, total_missing = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w == warp) {
      before_pages = sat_add(before_pages, total_pages);
      before_entries = sat_add(before_entries, total_entries);
    }
    total_pages = sat_add(total_pages, warp_pages[w]);
    total_entries = sat_add(total_entries, warp_entries[w]);
    total_missing = sat_add(total_missing, warp_missing[w]);
  }
  for (int r = r0; r < r1; ++r) {
    page_first[r] = sat_add(page_first[r], before_pages);
    entry_first[r] = sat_add(entry_first[r], before_entries);
  }
  __syncthreads();

  if (blockIdx.x == 0 && tid == 0) {
    const int taken = min(total_pages, p.num_free);
    p.counts[0] = total_entries;
    p.counts[1] = taken;
    p.counts[2] = sat_add(total_missing, total_pages - taken);
  }
  const int64_t stride = int64_t(gridDim.x) * THREADS, at = int64_t(blockIdx.x) * THREADS + tid;
  for (int64_t j = at; j < total_pages; j += stride) {
    const int r = owner(page_first, p.requests, int(j));
    const int block = pages_of(held[r], p.page_shift) + (int(j) - page_first[r]);
    p.table[r * p.table_stride + block] = j < p.num_free ? p.free_pages[j] : -1;
  }
  // VEC consecutive slots a thread: of prompts four, for one search and one 16-byte store (where slots is
  // aligned for it); of decode steps one, as neighbours belong to different requests.
  const bool wide = VEC == 4 && (reinterpret_cast<uintptr_t>(p.slots) & 15) == 0;
  for (int64_t t4 = at * VEC; t4 < p.num_slots; t4 += stride * VEC) {
    int slot[4] = {-1, -1, -1, -1};
    if (t4 < total_entries) {
      int r = owner(entry_first, p.requests, int(t4)), page = -1;
      int64_t at_block = -1;  // the block that `page` is of, of request r
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int64_t t = t4 + i;
        if (t >= total_entries) break;
        if (r + 1 < p.requests && entry_first[r + 1] <= t) r = owner(entry_first, p.requests, int(t)), at_block = -1;
        const int64_t entry = int64_t(held[r]) + (t - entry_first[r]), block = entry >> p.page_shift;
        if (block != at_block) {  // mostly once
          const int have = pages_of(held[r], p.page_shift);
          const int64_t j = block - have + page_first[r];  // place among the new pages
          page = block >= p.width ? -1 : block < have ? p.table[r * p.table_stride + block] : j < p.num_free ? p.free_pages[j] : -1;
          at_block = block;
        }
        slot[i] = slot_of(page, int(entry), p.page_shift);
      }
    }
    if (wide && t4 + 4 <= p.num_slots) {
      *reinterpret_cast<int4*>(p.slots + t4) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (t4 + i < p.num_slots) p.slots[t4 + i] = slot[i];
    }
  }
}

// ------------------------------------------------------------------------------ append and read
constexpr int COPY_THREADS = 256;

struct Factor {
  float value, six, sixth;  // the cache's factor f, 6 f and the correctly rounded 1 / (6 f); sixth 0: divide
};

struct CopyParams {
  uint8_t* data;
  const int32_t* slots;
  const void* k;
  const void* v;
  int64_t k_token, k_head, v_token, v_head;  // strides in elements
  int64_t page_stride;
  uint32_t tokens;
  uint32_t heads;
  int32_t num_pages, page_shift;
  Factor k_scale, v_scale;
  int32_t heads_log2;  // -1: no power of two
};

template <bool BF16>
__device__ __forceinline__ float2 to_f32(uint32_t two) {
  if (BF16) return make_float2(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u));
  return f16x2_to_f32(two);
}

template <bool BF16>
__device__ __forceinline__ uint32_t from_f32(float lo, float hi) {
  uint32_t r;
  if (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Largest magnitude of two 16-bit pairs, a NaN winning (maxima of the types' own bits).
template <bool BF16>
__device__ __forceinline__ uint32_t max_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  if (BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two products and two fused multiply-adds in one instruction each.
__device__ __forceinline__ uint64_t f32x2(float2 v) {
  return uint64_t(__float_as_uint(v.x)) | uint64_t(__float_as_uint(v.y)) << 32;
}
__device__ __forceinline__ float2 f32x2(uint64_t v) {
  return make_float2(__uint_as_float(uint32_t(v)), __uint_as_float(uint32_t(v >> 32)));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// x / d as IEEE division gives it, r being the correctly rounded 1 / d: one residual step makes the product
// x r correctly rounded (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990), as long as nothing over- or underflows.
__device__ __forceinline__ float quotient(float x, float d, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, d, x), r, q);
}

// Half of a block of 16 values in each of two neighbouring lanes: the block's scale (8 bits) and this
// lane's codes (8 x 4 bits).
template <bool BF16>
__device__ __forceinline__ uint32_t quantise(const uint4& v, const Factor& f, uint32_t& codes) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = x[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 4; ++i) m = max_nan<BF16>(m, x[i] & 0x7fff7fffu);
  m = max_nan<BF16>(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const float most = to_f32<BF16>(max_nan<BF16>(m, (m >> 16) | (m << 16))).x;
  // the residual step wants normal numbers all the way: not for zeros, infinities and far factors
  const bool plain = f.sixth != 0.f && most > 1e-18f && most < 1e18f;
  const uint32_t scale = f32_to_e4m3(plain ? quotient(most, f.six, f.sixth) : most / f.six);
  const float unit = f16x2_to_f32(e4m3x2_to_f16x2(scale)).x * f.value;
  codes = 0;
  if (unit > 0.f) {  // neither 0 nor NaN
    if (plain) {
      const float r = __frcp_rn(unit);
      const uint64_t rr = f32x2(make_float2(r, r)), minus = f32x2(make_float2(-unit, -unit));
      float2 q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t a = f32x2(to_f32<BF16>(x[i])), y = mul2(a, rr);
        q[i] = f32x2(fma2(fma2(y, minus, a), rr, y));
      }
      codes = f32x8_to_e2m1(q);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = to_f32<BF16>(x[i]);
        codes |= f32x2_to_e2m1(a.x / unit, a.y / unit) << (8 * i);
      }
    }
  }
  return scale;
}

// Address of a slot's row of one head, or nullptr for a slot that names no entry.
__device__ __forceinline__ uint8_t* row_of(const CopyParams& p, int slot, int head, int bytes) {
  const int64_t off = slot_offset(slot, p.num_pages, p.page_shift, p.page_stride, p.heads, head, bytes);
  return off < 0 ? nullptr : p.data + off;
}

// D / 8 neighbouring lanes take the K and V of one token and head, eight values of each a lane: a warp
// reads (or, for cache_read, writes) 512 neighbouring bytes at a time, and writes 128 (64) of codes.
// 16333 tokens x 8 heads of 128 in bf16, 86 MB in and out: append 17.9 us (4.8 TB/s; the conversions,
// about 11 us of issue, are not all hidden), read 14.4 us (6.0 TB/s; bound by bytes).  Two rows a thread: 18.7.
template <int D, bool BF16>
__global__ void __launch_bounds__(COPY_THREADS) cache_append_kernel(CopyParams p) {
  constexpr int LANES = D / 8;
  begin();
  const uint32_t th = blockIdx.x * uint32_t(COPY_THREADS / LANES) + threadIdx.x / LANES, t = p.heads_log2 >= 0 ? th >> p.heads_log2 : th / p.heads;
  const int h = int(th - t * p.heads), b = threadIdx.x % LANES;
  uint8_t* row = nullptr;
  uint4 k = make_uint4(0, 0, 0, 0), v = k;
  if (t < p.tokens) {  // read whether it has a slot or not, beside its slot: 17.9 us, one after the other 19.4
    const int slot = p.slots[t];
    k = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.k) + int64_t(t) * p.k_token + h * p.k_head)[b];
    v = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.v) + int64_t(t) * p.v_token + h * p.v_head)[b];
    row = row_of(p, slot, h, row_bytes(D));
  }
  uint32_t kc, vc;
  const uint32_t ks = quantise<BF16>(k, p.k_scale, kc), vs = quantise<BF16>(v, p.v_scale, vc);  // by all lanes
  if (!row) return;
  *reinterpret_cast<uint32_t*>(row + b * 4) = kc;
  *reinterpret_cast<uint32_t*>(row + D / 2 + b * 4) = vc;
  // even lanes write the scales of K, odd ones those of V
  row[D + (b & 1) * (D / 16) + b / 2] = uint8_t(b & 1 ? vs : ks);
}

template <bool BF16>
__device__ __forceinline__ uint4 dequantise(uint32_t codes, uint32_t scale, float factor) {
  const uint32_t unit = e4m3x2_to_f16x2(scale | scale << 8);
  uint32_t h[4], out[4];
  e2m1_to_f16x2(codes, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = f16x2_to_f32(hmul2(h[i], unit));  // exact
    out[i] = from_f32<BF16>(x.x * factor, x.y * factor);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(COPY_THREADS) cache_read_kernel(CopyParams p) {
  constexpr int LANES = D / 8;
  begin();
  const uint32_t th = blockIdx.x * uint32_t(COPY_THREADS / LANES) + threadIdx.x / LANES, t = p.heads_log2 >= 0 ? th >> p.heads_log2 : th / p.heads;
  if (t >= p.tokens) return;
  const int b = threadIdx.x % LANES;
  const uint8_t* row = row_of(p, p.slots[t], int(th - t * p.heads), row_bytes(D));
  uint32_t kc = 0, vc = 0, ks = 0, vs = 0;
  if (row) {
    if (p.k) kc = *reinterpret_cast<const uint32_t*>(row + b * 4), ks = row[D + b / 2];
    if (p.v) vc = *reinterpret_cast<const uint32_t*>(row + D / 2 + b * 4), vs = row[D + D / 16 + b / 2];
  }
  const int64_t at = int64_t(th) * LANES + b;
  if (p.k) static_cast<uint4*>(const_cast<void*>(p.k))[at] = dequantise<BF16>(kc, ks, p.k_scale.value);
  if (p.v) static_cast<uint4*>(const_cast<void*>(p.v))[at] = dequantise<BF16>(vc, vs, p.v_scale.value);
}

using CopyKernel = void (*)(CopyParams);

template <bool BF16>
CopyKernel copy_kernel(int dim, bool append) {
  if (dim == 64) return append ? cache_append_kernel<64, BF16> : cache_read_kernel<64, BF16>;
  if (dim == 128) return append ? cache_append_kernel<128, BF16> : cache_read_kernel<128, BF16>;
  return append ? cache_append_kernel<256, BF16> : cache_read_kernel<256, BF16>;
}

Factor factor_of(float f) {
  const float six = 6.f * f;
  return {f, six, f > 1e-12f && f < 1e12f ? 1.f / six : 0.f};
}

gvr_status launch_copy(const gvr_cache* c, CopyParams& p, int32_t dtype, int64_t tokens, bool append, void* stream) {
  if (tokens > kIntMax / c->num_kv_heads) return GVR_ERR_ARG;
  p.data = static_cast<uint8_t*>(c->data);
  p.page_stride = c->page_stride;
  p.tokens = uint32_t(tokens);
  p.num_pages = int32_t(c->num_pages);
  p.heads = c->num_kv_heads;
  p.page_shift = log2_of(c->page_size);
  p.k_scale = factor_of(c->k_scale);
  p.v_scale = factor_of(c->v_scale);
  p.heads_log2 = (c->num_kv_heads & (c->num_kv_heads - 1)) == 0 ? log2_of(c->num_kv_heads) : -1;
  const int64_t rows = COPY_THREADS / (c->head_dim / 8), grid = (tokens * c->num_kv_heads + rows - 1) / rows;
  const CopyKernel kernel = dtype == GVR_BF16 ? copy_kernel<true>(c->head_dim, append) : copy_kernel<false>(c->head_dim, append);
  void* args[] = {&p};
  if (launch(reinterpret_cast<const void*>(kernel), dim3(uint32_t(grid)), COPY_THREADS, 0, 1, args, stream) != cudaSuccess)
    return GVR_ERR_LAUNCH;
  return GVR_OK;
}

// Attributes of the tables kernel, set once per device: its largest shared memory.
struct TableDevice {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
};
TableDevice g_table_devices[kMaxDevices];

}  // namespace
}  // namespace gvrc

extern "C" {

gvr_status cache_row_bytes(int32_t head_dim, int32_t* bytes) {
  if (!bytes) return GVR_ERR_NULL;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return GVR_ERR_ARG;
  *bytes = gvrc::row_bytes(head_dim);
  return GVR_OK;
}

gvr_status cache_tables(const int32_t* cached_lens, const int32_t* kv_lens, int64_t num_requests,
                        int32_t compress_ratio, int32_t page_size, const int32_t* free_pages,
                        int64_t num_free, int32_t* block_table, int64_t table_stride,
                        int64_t table_width, int32_t* slots, int64_t num_slots, int32_t* counts,
                        void* stream) {
  using namespace gvrc;
  if (num_requests < 0 || num_requests > GVR_CACHE_MAX_REQUESTS || compress_ratio < 1 || !page_size_ok(page_size) ||
      num_free < 0 || num_free > kIntMax || num_slots < 0 || num_slots > kIntMax || table_width < 0 ||
      table_width > kIntMax / page_size)
    return GVR_ERR_ARG;
  // new pages are numbered in 32 bits: with more, the last ones would not be written
  if (num_requests > 0 && table_width > kIntMax / num_requests) return GVR_ERR_ARG;
  if (table_stride < table_width || table_stride > kIntMax) return GVR_ERR_STRIDE;
  if (!counts || (num_requests > 0 && (!cached_lens || !kv_lens)) || (num_requests > 0 && table_width > 0 && !block_table) ||
      (num_free > 0 && !free_pages) || (num_slots > 0 && !slots))
    return GVR_ERR_NULL;
  if (!aligned(cached_lens, 4) || !aligned(kv_lens, 4) || !aligned(free_pages, 4) || !aligned(block_table, 4) ||
      !aligned(slots, 4) || !aligned(counts, 4))
    return GVR_ERR_ALIGN;
  int sms = 0, dev = 0;
  if (sm_count(&sms) != cudaSuccess || cudaGetDevice(&dev) != cudaSuccess) return GVR_ERR_LAUNCH;
  TableDevice& td = g_table_devices[dev];  // sm_count has checked dev
  std::call_once(td.once, [&td]() {
    for (const void* k : {reinterpret_cast<const void*>(cache_tables_kernel<TABLE_THREADS, 1>),
                          reinterpret_cast<const void*>(cache_tables_kernel<TABLE_THREADS, 4>)})
      if (td.err == cudaSuccess)
        td.err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, GVR_CACHE_MAX_REQUESTS * 3 * int(sizeof(int)));
  });
  if (td.err != cudaSuccess) return GVR_ERR_LAUNCH;
  TableParams p = {};
  p.cached = cached_lens;
  p.lens = kv_lens;
  p.free_pages = free_pages;
  p.table = block_table;
  p.slots = slots;
  p.counts = counts;
  p.table_stride = table_stride;
  p.num_slots = num_slots;
  p.requests = int32_t(num_requests);
  p.ratio = compress_ratio;
  p.page_shift = log2_of(page_size);
  p.num_free = int32_t(num_free);
  p.width = int32_t(table_width);
  // Enough CTAs for one 16-byte store a thread, at most two per SM: the scan is repeated by each.
  // Decode steps (few slots a request) take one slot a thread, and up to 128 requests a small CTA, whose
  // scan and barriers are shorter: 64 requests 4.8 -> 2.5 us.
  const bool step = num_slots <= 8 * num_requests, small = step && num_requests <= TABLE_THREADS_SMALL;
  const int threads = small ? TABLE_THREADS_SMALL : TABLE_THREADS, per_cta = step ? threads : 4 * threads;
  const int64_t want = (num_slots + per_cta - 1) / per_cta;
  const int grid = int(want < 1 ? 1 : want > 2 * sms ? 2 * sms : want);
  const void* kernel = small  ? reinterpret_cast<const void*>(cache_tables_kernel<TABLE_THREADS_SMALL, 1>)
                       : step ? reinterpret_cast<const void*>(cache_tables_kernel<TABLE_THREADS, 1>)
                              : reinterpret_cast<const void*>(cache_tables_kernel<TABLE_THREADS, 4>);
  void* args[] = {&p};
  if (launch(kernel, dim3(grid), threads, int(num_requests * 3 * sizeof(int)), 1, args, stream) != cudaSuccess)
    return GVR_ERR_LAUNCH;
  return GVR_OK;
}

gvr_status cache_append(const gvr_cache* cache, const void* k, int64_t k_token_stride,
                        int64_t k_head_stride, const void* v, int64_t v_token_stride,
                        int64_t v_head_stride, int32_t dtype, const int32_t* slots,
                        int64_t num_tokens, void* stream) {
  using namespace gvrc;
  const gvr_status s = check_cache(cache);
  if (s != GVR_OK) return s;
  if (num_tokens < 0 || (dtype != GVR_BF16 && dtype != GVR_F16)) return GVR_ERR_ARG;
  if (num_tokens == 0) return GVR_OK;
  if (!k || !v || !slots) return GVR_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return GVR_ERR_ALIGN;
  for (int64_t stride : {k_token_stride, k_head_stride, v_token_stride, v_head_stride})
    if (stride < 0 || stride % 8 != 0 || stride > kIntMax) return GVR_ERR_STRIDE;
  CopyParams p = {};
  p.k = k;
  p.v = v;
  p.slots = slots;
  p.k_token = k_token_stride;
  p.k_head = k_head_stride;
  p.v_token = v_token_stride;
  p.v_head = v_head_stride;
  return launch_copy(cache, p, dtype, num_tokens, true, stream);
}

gvr_status cache_read(const gvr_cache* cache, const int32_t* slots, int64_t num_tokens, int32_t dtype, void* k, void* v,
                      void* stream) {
  using namespace gvrc;
  const gvr_status s = check_cache(cache);
  if (s != GVR_OK) return s;
  if (num_tokens < 0 || (dtype != GVR_BF16 && dtype != GVR_F16)) return GVR_ERR_ARG;
  if (num_tokens == 0 || (!k && !v)) return GVR_OK;
  if (!slots) return GVR_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return GVR_ERR_ALIGN;
  CopyParams p = {};
  p.k = k;
  p.v = v;
  p.slots = slots;
  return launch_copy(cache, p, dtype, num_tokens, false, stream);
}

const char* gvr_cache_status_string(gvr_status status) {
  switch (status) {
    case GVR_OK: return "ok";
    case GVR_ERR_NULL: return "a required pointer is NULL";
    case GVR_ERR_ALIGN: return "cache data, q, k, v and out must be 16-byte aligned, int32 and fp32 buffers 4-byte aligned";
    case GVR_ERR_STRIDE:
      return "a stride is out of range: page strides a multiple of 16 bytes that holds a page, q, k and v strides "
             "multiples of 8 elements, table strides at least the table's width";
    case GVR_ERR_ARG: return "invalid argument (head_dim 64, 128 or 256; page_size a power of two; counts, ratios, scales, heads, k or dtype)";
    case GVR_ERR_LAUNCH: return "kernel launch failed";
    default: return "unknown status";
  }
}

}  // extern "C"
