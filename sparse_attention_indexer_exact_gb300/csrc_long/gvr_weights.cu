// gvr_weights.cu -- attend_weights of include/gvr_long.h: the attention weight that each cached entry draws.
//
// w_e += sum over a request's rows j and heads h of exp(scale q_jh . k_e - lse_jh): with the log-sums known, entries need
// nothing of each other, so there is one pass over K (codes and scales, half of the cache) and no join.
//
// Work split.  The steps of 32 entries of all requests, one behind the other, are cut into equal ranges, one a CTA.  A
// CTA brings its request's queries, as f16 matrix operands, into shared memory once (in parts where they are more than
// that holds), and its warps take steps in turn.  A warp fetches its own entries' K rows, KV head by KV head, by
// asynchronous copies two heads ahead, expands them in registers into the 16-row operand of m16n8k16 (as gvr_attend.cuh
// does), and adds up exp2 of the scores of 8 queries at a time.  A lane ends with the sums of one entry, which it alone
// adds to memory: no atomics, every sum in a fixed order.
//
// Matrix products by mma.sync, as in gvr_attend.cuh and for its reason: a KV head's queries are few, the 4-bit operand
// expands in registers straight into that layout.
//
// What bounds it.  64 requests of up to 16384 entries, 64 heads over 8 of 128: 103 us under the profiler, 107 over the same
// inputs again, 109 over other ones each time.  K is half of a row, but its 64
// bytes of codes and 8 of scales, rows being 144 bytes, touch 17 of 18 blocks of 64 bytes, which is what DRAM gives at least:
// 598 MB, at 5.8 TB/s under the profiler (0.87 of the measured copy rate).  16 rows a request of 6 heads over 4 of 64 (19 requests up to 12345
// entries): 34.5 to 35.6 us, no pipe busy (before its last step: issue 47 %, tensor 29 %): a CTA has
// three turns of its warps, each a chain of copy, expansion, products and exponentials, behind its queries' way into shared memory.  One row of 8192 entries: 7.7 us, latency.
// With the copy of its weights that the benchmark's call makes (1 to 12 us), steps of 16 entries for few warps took one row from 14.4 to 11 us; the queries fetched a turn ahead and two chains of products the
// batch from 113 to 106; no limits where all rows see an entry the 16 rows from 51 to 43, requests
// weighed with what they cost beside their steps from 41 to 36.
#include <algorithm>
#include <mutex>

#include "../csrc_cache/gvr_attend.cuh"
#include "gvr_long_common.h"

namespace gvrc {
namespace {

constexpr int WEIGHT_WARPS = 8, WEIGHT_THREADS = 32 * WEIGHT_WARPS;
constexpr int AHEAD = 3;              // stages of a warp's ring
constexpr int QUERY_BYTES = 1 << 16;  // of queries in shared memory, at most
constexpr int MANY = 4;               // steps of 32 entries a warp
constexpr int REQUEST_WORK = 8;       // what a request costs beside its steps, in steps: its queries, and a last turn of some warps (0, 2, 4, 8, 14:
                                      // 118, 113, 111, 112, 112 us for 64 requests of one row, 41, 41, 39, 36, 36 for 19 of 16 rows)

struct WeightParams {
  const uint8_t* data;
  const uint16_t* q;
  const int32_t* table;
  const int32_t* lens;
  const float* lse;
  float* weights;
  int64_t q_row, q_head, table_stride, weights_stride, num_rows;
  uint32_t unit, page_units, entry_units, row_units;  // as in AttendParams
  int32_t num_pages, page_shift, kv_heads, group, capacity, next_n, ratio, bf16, requests;
  int32_t tiles;        // of 8 queries of a KV head
  int32_t part_tiles;   // of them at a time
  int32_t part_heads;   // KV heads at a time
  float scale_log2, q_sign;
};

// Two neighbouring queries in shared memory, beside their operands: the factors of their scores, to log2 units, and their
// log-sums in those (infinite for no query: it adds nothing); the entries that they see.
struct Queries {
  float factor0, off0, factor1, off1;
};

// MT tiles of 16 entries a step: two, or one where steps of two are too few for the device's warps.
template <int D, int MT>
struct WeightShape {
  static constexpr int STEP = 16 * MT;
  static constexpr int PITCH = (D / 2 + D / 16 + 15) / 16 * 16 | 16;  // of a row's K codes and scales: an odd multiple of 16
  static constexpr int STAGE = STEP * PITCH, RING = AHEAD * STAGE;
  static constexpr int TILE = 8 * D * 2;  // bytes of 8 queries
};

template <int D, int MT>
__global__ void __launch_bounds__(WEIGHT_THREADS, 2) weights_kernel(WeightParams p) {
  using S = WeightShape<D, MT>;
  constexpr int STEP = S::STEP;
  constexpr int CODES = D / 32;  // 16-byte pieces of a row's K codes
  constexpr int KW = D / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int part = p.part_heads * p.part_tiles;
  uint8_t* ring = smem + warp * S::RING;
  uint4* operands = reinterpret_cast<uint4*>(smem + WEIGHT_WARPS * S::RING);  // [part][D / 32][32 lanes]
  Queries* queries = reinterpret_cast<Queries*>(smem + WEIGHT_WARPS * S::RING + part * S::TILE);  // [part][4]
  int2* limits = reinterpret_cast<int2*>(queries + part * 4);  // [part][4]
  int* start = reinterpret_cast<int*>(limits + part * 4);  // [requests + 1]: the work before each request, in steps
  __shared__ int sums[WEIGHT_WARPS];

  begin();
  // ---- steps of all requests
  // entries that some row of the request sees (the last request may have fewer rows)
  auto entries = [&](int r) {
    return decode_entries(p.lens[r], p.next_n, int(min(int64_t(p.next_n), p.num_rows - int64_t(r) * p.next_n)) - 1, p.ratio, p.capacity);
  };
  int before = 0;
  for (int r0 = 0; r0 < p.requests; r0 += WEIGHT_THREADS) {
    const int r = r0 + tid;
    int x = r < p.requests ? (entries(r) + STEP - 1) / STEP : 0;
    if (x > 0) x += REQUEST_WORK;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < WEIGHT_WARPS; ++w) {
      if (w == warp) x += all;
      all += sums[w];
    }
    if (r < p.requests) start[r + 1] = before + x;
    before += all;
  }
  if (tid == 0) start[0] = 0;
  __syncthreads();
  // whole turns of the CTA's warps while there are enough for all CTAs
  const int total = before, ctas = min(int(gridDim.x), (total + WEIGHT_WARPS - 1) / WEIGHT_WARPS);
  if (int(blockIdx.x) >= ctas) return;
  int at = int(int64_t(blockIdx.x) * total / ctas);
  const int last = int(int64_t(blockIdx.x + 1) * total / ctas);
  int request = 0;
  for (int hi = p.requests; hi - request > 1;) {  // the last one that starts at or before `at`
    const int mid = (request + hi) >> 1;
    if (start[mid] <= at) request = mid; else hi = mid;
  }

  const int members = p.next_n * p.group;
  const uint32_t ring_at = gvr::smem_u32(ring);
  for (; at < last; ++request) {
    const int begins = start[request] + REQUEST_WORK, to = min(last, start[request + 1]);
    const int first = max(at - begins, 0), segment = to - begins - first;
    at = max(at, to);
    if (segment <= 0) continue;
    const int kv = p.lens[request], n = entries(request), sure = decode_entries(kv, p.next_n, 0, p.ratio, p.capacity);
    const int32_t* table = p.table + request * p.table_stride;
    float* weights = p.weights + request * p.weights_stride;

    for (int head0 = 0; head0 < p.kv_heads; head0 += p.part_heads)
      for (int tile0 = 0; tile0 < p.tiles; tile0 += p.part_tiles) {
        const int heads = min(p.part_heads, p.kv_heads - head0), tiles = min(p.part_tiles, p.tiles - tile0);
        // ---- the queries: lane (g, c) of a tile holds D / 4 values of query g
        __syncthreads();  // the last part is used up
        // (loaded a turn ahead)
        uint32_t raw[D / 8], next[D / 8];
        float sum = 0.f, next_sum = 0.f;
        auto fetch_query = [&](int i, uint32_t(&to)[D / 8], float& log_sum) {
          const int h = head0 + i / tiles, m = (tile0 + i % tiles) * 8 + g;
          const int64_t row = int64_t(request) * p.next_n + m / p.group;
          const int head = h * p.group + m % p.group;
          const bool live = i < heads * tiles && m < members && row < p.num_rows;
          const uint4* src = reinterpret_cast<const uint4*>(p.q + row * p.q_row + head * p.q_head + c * (D / 4));
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            const uint4 v = live ? src[j] : make_uint4(0, 0, 0, 0);
            to[4 * j] = v.x, to[4 * j + 1] = v.y, to[4 * j + 2] = v.z, to[4 * j + 3] = v.w;
          }
          log_sum = live ? p.lse[row * (int64_t(p.kv_heads) * p.group) + head] : 0.f;
        };
        fetch_query(warp, next, next_sum);
        for (int i = warp; i < heads * tiles; i += WEIGHT_WARPS) {
          const int m = (tile0 + i % tiles) * 8 + g;
          const bool live = m < members && int64_t(request) * p.next_n + m / p.group < p.num_rows;
#pragma unroll
          for (int j = 0; j < D / 8; ++j) raw[j] = next[j];
          sum = next_sum;
          fetch_query(i + WEIGHT_WARPS, next, next_sum);
          float back = 1.f;
          if (p.bf16) {  // exactly to f16, by a power of two per query (gvr_attend.cuh)
            uint32_t big = 0;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) big = __vmaxu2(big, raw[j] & 0x7fff7fffu);
            big = max(big & 0xffffu, big >> 16);
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
            const int exponent = int(big >> 7), up = big == 0 || exponent == 255 ? 0 : min(14 - (exponent - 127), 126);
            const float mul = p.q_sign * __uint_as_float(uint32_t(127 + up) << 23);
            back = __uint_as_float(uint32_t(127 - up) << 23);
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
              raw[j] = pack_f16(__uint_as_float(raw[j] << 16) * mul, __uint_as_float(raw[j] & 0xffff0000u) * mul);
          } else {
            const uint32_t sign = pack_f16(p.q_sign, p.q_sign);
#pragma unroll
            for (int j = 0; j < D / 8; ++j) raw[j] = hmul2(raw[j], sign);
          }
#pragma unroll
          for (int j = 0; j < D / 32; ++j)
            operands[(i * (D / 32) + j) * 32 + lane] = make_uint4(raw[4 * j], raw[4 * j + 1], raw[4 * j + 2], raw[4 * j + 3]);
          if (c == 0) {
            float* query = reinterpret_cast<float*>(queries + i * 4) + 2 * g;
            query[0] = fmaxf(back * p.scale_log2, 1.17549435e-38f);
            query[1] = live ? sum * 1.4426950408889634f : INFINITY;
            reinterpret_cast<int*>(limits + i * 4)[g] = live ? decode_entries(kv, p.next_n, m / p.group, p.ratio, p.capacity) : 0;
          }
        }
        __syncthreads();

        // ---- this warp's steps, KV head by KV head
        const int mine = segment > warp ? (segment - warp + WEIGHT_WARPS - 1) / WEIGHT_WARPS : 0, items = mine * heads;
        int ahead_step = 0, ahead_head = 0;  // of the next item to fetch
        auto entry_of = [&](int step) { return (first + warp + step * WEIGHT_WARPS) * STEP + lane % STEP; };
        auto page_of = [&](int step) {
          const int e = entry_of(step);
          return step < mine && e < n ? table[e >> p.page_shift] : -1;
        };
        int page = page_of(0), page_next = page_of(1);
        uint32_t there_ahead = 0, from = 0;
        uint32_t there_of[AHEAD] = {};  // which lanes' entries exist, of the items under way
        auto fetch = [&](int stage) -> uint32_t {
          if (ahead_step < mine) {
            if (ahead_head == 0) {
              const bool is = uint32_t(page) < uint32_t(p.num_pages);
              there_ahead = __ballot_sync(0xffffffffu, is);
              from = is ? row_unit(page, entry_of(ahead_step), p.page_shift, p.page_units, p.entry_units, uint32_t(head0) * p.row_units) : 0;
              if (there_ahead) {  // a missing entry is fetched from where another lies, and not looked at
                const uint32_t some = __shfl_sync(0xffffffffu, from, __ffs(there_ahead) - 1);
                if (!is) from = some;
              }
              page = page_next;
              page_next = page_of(ahead_step + 2);
            }
            if (there_ahead) {
              const uint32_t to = ring_at + stage * S::STAGE;
              const uint32_t here = from + uint32_t(ahead_head) * p.row_units;
#pragma unroll
              for (int j = 0; j < CODES * MT / 2; ++j) {  // CODES neighbouring lanes copy a row's codes
                const int row = j * (32 / CODES) + lane / CODES;
                const uint32_t of = __shfl_sync(0xffffffffu, here, row);
                copy16(to + row * S::PITCH + lane % CODES * 16, p.data + uint64_t(of) * p.unit + lane % CODES * 16);
              }
              const uint8_t* scales = p.data + uint64_t(here) * p.unit + D;
              const uint32_t scales_to = to + lane * S::PITCH + D / 2;
              if (MT == 1 && lane >= STEP) {
              } else if (D == 256) copy16(scales_to, scales);
              else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(scales_to), "l"(scales), "n"(D == 128 ? 8 : 4) : "memory");
            }
            if (++ahead_head == heads) ahead_head = 0, ++ahead_step;
          }
          copy_commit();
          return there_ahead;
        };
#pragma unroll
        for (int i = 0; i < AHEAD - 1; ++i) there_of[i] = fetch(i);

        float acc[MT][2] = {};  // of entries tile_entry(g), tile_entry(g + 8) of both tiles
        int step = 0, h = 0, stage = 0;
        const int k_at = tile_entry(g) * S::PITCH;
        for (int item = 0; item < items; ++item) {
          copy_wait<AHEAD - 2>();
          __syncwarp();  // the item's rows are here, and every lane is done with the stage before it
          there_of[AHEAD - 1] = fetch(stage == 0 ? AHEAD - 1 : stage - 1);
          const uint32_t there = there_of[0];
#pragma unroll
          for (int j = 0; j < AHEAD - 1; ++j) there_of[j] = there_of[j + 1];
          const int e0 = (first + warp + step * WEIGHT_WARPS) * STEP;
          if (there) {
            const bool border = e0 + STEP > sure;
            const uint8_t* st = ring + stage * S::STAGE;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const uint8_t *r0 = st + k_at + 16 * mt * S::PITCH, *r1 = r0 + S::PITCH;
              uint32_t k0[KW], k1[KW], a[2 * KW][4];  // operands of 2 KW 16-wide steps
              load_words<KW>(r0 + c * (D / 8), k0);
              load_words<KW>(r1 + c * (D / 8), k1);
              uint32_t sc0, sc1;
              if (D == 64) sc0 = r0[D / 2 + c], sc1 = r1[D / 2 + c];
              else if (D == 128) sc0 = *reinterpret_cast<const uint16_t*>(r0 + D / 2 + 2 * c), sc1 = *reinterpret_cast<const uint16_t*>(r1 + D / 2 + 2 * c);
              else sc0 = *reinterpret_cast<const uint32_t*>(r0 + D / 2 + 4 * c), sc1 = *reinterpret_cast<const uint32_t*>(r1 + D / 2 + 4 * c);
#pragma unroll
              for (int w = 0; w < KW; ++w) {
                uint32_t x[4], y[4];
                e2m1_to_f16x2(k0[w], x);
                e2m1_to_f16x2(k1[w], y);
                const int block = w / 2;
                const uint32_t x0 = splat(e4m3x2_to_f16x2(sc0 >> (16 * (block / 2))), block & 1);
                const uint32_t y0 = splat(e4m3x2_to_f16x2(sc1 >> (16 * (block / 2))), block & 1);
#pragma unroll
                for (int j = 0; j < 4; ++j) a[2 * w + j / 2][j % 2 * 2] = hmul2(x[j], x0), a[2 * w + j / 2][j % 2 * 2 + 1] = hmul2(y[j], y0);
              }
              auto add_up = [&](auto bordering) {
                constexpr int AT_ONCE = D == 64 ? 2 : 1;
#pragma unroll AT_ONCE
                for (int t = 0; t < tiles; ++t) {
                  const int tile = h * tiles + t;
                  float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                  for (int j = 0; j < D / 32; ++j) {
                    const uint4 b = operands[(tile * (D / 32) + j) * 32 + lane];
                    mma(s, a[2 * j][0], a[2 * j][1], a[2 * j][2], a[2 * j][3], b.x, b.y);
                    mma(D > 64 ? s2 : s, a[2 * j + 1][0], a[2 * j + 1][1], a[2 * j + 1][2], a[2 * j + 1][3], b.z, b.w);
                  }
                  if (D > 64) {  // long chains in two
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[j] += s2[j];
                  }
                  const Queries q = queries[tile * 4 + c];
                  float w0 = exp2_fast(fmaf(s[0], q.factor0, -q.off0)), w1 = exp2_fast(fmaf(s[1], q.factor1, -q.off1));
                  float w2 = exp2_fast(fmaf(s[2], q.factor0, -q.off0)), w3 = exp2_fast(fmaf(s[3], q.factor1, -q.off1));
                  if (decltype(bordering)::value) {
                    const int2 limit = limits[tile * 4 + c];
                    const int e = e0 + 16 * mt + tile_entry(g);  // the tile's other row is e + 1
                    if (e >= limit.x) w0 = 0.f;
                    if (e >= limit.y) w1 = 0.f;
                    if (e + 1 >= limit.x) w2 = 0.f;
                    if (e + 1 >= limit.y) w3 = 0.f;
                  }
                  acc[mt][0] += w0 + w1, acc[mt][1] += w2 + w3;
                }
              };
              if (border) add_up(std::true_type());
              else add_up(std::false_type());
            }
          }
          stage = stage == AHEAD - 1 ? 0 : stage + 1;
          if (++h == heads) {  // the step's last head: lane i's is entry i
            h = 0, ++step;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                acc[mt][j] += __shfl_xor_sync(0xffffffffu, acc[mt][j], 1);
                acc[mt][j] += __shfl_xor_sync(0xffffffffu, acc[mt][j], 2);
              }
            // entry y of a tile is tile_entry(x + 8 (y & 1)) of x = y & ~1 below 8, and of the x that (x + 3) & 7 leads to it above
            const int y = lane & 15, even = y & ~1, x = even < 8 ? even : (even + 5) & 7;
            float v[2 * MT];
#pragma unroll
            for (int j = 0; j < 2 * MT; ++j) v[j] = __shfl_sync(0xffffffffu, acc[j >> 1][j & 1], 4 * x);
            const float w = lane < 16 ? (y & 1 ? v[1] : v[0]) : (y & 1 ? v[2 * MT - 1] : v[2 * MT - 2]);
            if (lane < STEP && (there >> lane & 1)) weights[e0 + lane] += w;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) acc[mt][0] = acc[mt][1] = 0.f;
          }
        }
        copy_wait<0>();
        __syncwarp();
      }
  }
}

struct WeightInfo {
  const void* kernel;
  int ring;  // bytes of all warps
};
template <int D, int MT>
WeightInfo weight_info() {
  return {reinterpret_cast<const void*>(weights_kernel<D, MT>), WEIGHT_WARPS * WeightShape<D, MT>::RING};
}
WeightInfo weights_kernel_of(int dim, int tiles) {
  if (dim == 64) return tiles == 1 ? weight_info<64, 1>() : weight_info<64, 2>();
  if (dim == 128) return tiles == 1 ? weight_info<128, 1>() : weight_info<128, 2>();
  return tiles == 1 ? weight_info<256, 1>() : weight_info<256, 2>();
}

struct WeightDevice {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
};
WeightDevice g_weight_devices[kMaxDevices];

}  // namespace
}  // namespace gvrc

extern "C" {

gvr_status attend_weights(const gvr_cache* cache, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                          int32_t dtype, int64_t num_rows, int32_t num_heads, const int32_t* block_table,
                          int64_t table_stride, int64_t table_width, const int32_t* kv_lens, int32_t next_n,
                          int32_t compress_ratio, const float* lse, float scale, float* weights,
                          int64_t weights_stride, void* stream) {
  using namespace gvrc;
  gvr_status s = check_rows(cache, q, q_row_stride, q_head_stride, dtype, num_rows, num_heads, block_table, table_stride, table_width,
                            kv_lens, next_n, compress_ratio, scale);
  if (s != GVR_OK) return s;
  if (weights_stride < table_width * cache->page_size || weights_stride > kIntMax) return GVR_ERR_STRIDE;
  if (num_rows == 0) return GVR_OK;
  if (!lse || (table_width > 0 && !weights)) return GVR_ERR_NULL;
  if (!aligned(lse, 4) || !aligned(weights, 4)) return GVR_ERR_ALIGN;
  int sms = 0, dev = 0;
  if (sm_count(&sms) != cudaSuccess || cudaGetDevice(&dev) != cudaSuccess) return GVR_ERR_LAUNCH;
  WeightDevice& d = g_weight_devices[dev];  // sm_count has checked dev
  std::call_once(d.once, [&d, dev]() {
    int most = 0;
    d.err = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    for (int dim : {64, 128, 256})
      for (int tiles : {1, 2})
        if (d.err == cudaSuccess) d.err = cudaFuncSetAttribute(weights_kernel_of(dim, tiles).kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most - 1024);
  });
  if (d.err != cudaSuccess) return GVR_ERR_LAUNCH;
  WeightParams p = {};
  const int row = row_bytes(cache->head_dim), dim = cache->head_dim;
  p.data = static_cast<const uint8_t*>(cache->data);
  p.q = static_cast<const uint16_t*>(q);
  p.table = block_table;
  p.lens = kv_lens;
  p.lse = lse;
  p.weights = weights;
  p.q_row = q_row_stride;
  p.q_head = q_head_stride;
  p.table_stride = table_stride;
  p.weights_stride = weights_stride;
  p.num_rows = num_rows;
  p.unit = unit_bytes(cache->page_stride, row);
  p.page_units = uint32_t(cache->page_stride / p.unit);
  p.row_units = row / p.unit;
  p.entry_units = p.row_units * cache->num_kv_heads;
  p.num_pages = int32_t(cache->num_pages);
  p.page_shift = log2_of(cache->page_size);
  p.kv_heads = cache->num_kv_heads;
  p.group = num_heads / cache->num_kv_heads;
  p.capacity = cache->num_pages > 0 ? int32_t(table_width * cache->page_size) : 0;
  p.next_n = next_n;
  p.ratio = compress_ratio;
  p.bf16 = dtype == GVR_BF16;
  p.requests = int32_t((num_rows + next_n - 1) / next_n);
  // steps are counted in 32 bits
  const int64_t halves = (int64_t(p.capacity) + 15) / 16;
  if ((halves + REQUEST_WORK) * p.requests > kIntMax) return GVR_ERR_ARG;
  // steps of 32 entries, or of 16 where a warp has fewer than MANY of those, by the table's width
  const int64_t warps = int64_t(2) * sms * WEIGHT_WARPS;
  const int mt = halves * p.requests < 2 * MANY * warps ? 1 : 2;
  const int64_t steps = (halves + mt - 1) / mt;
  const WeightInfo info = weights_kernel_of(dim, mt);
  p.tiles = (next_n * p.group + 7) / 8;
  const int most = QUERY_BYTES / (16 * dim);  // tiles that shared memory holds
  p.part_tiles = std::min(p.tiles, most);
  p.part_heads = std::max(1, std::min(p.kv_heads, most / p.part_tiles));
  p.scale_log2 = scale == 0.f ? 1.f : float(std::fabs(double(scale)) * cache->k_scale * 1.4426950408889634);
  p.q_sign = scale > 0.f ? 1.f : scale < 0.f ? -1.f : 0.f;
  const int smem = info.ring + p.part_tiles * p.part_heads * (16 * dim + 4 * int(sizeof(Queries) + sizeof(int2))) + (p.requests + 1) * 4;
  const int64_t grid = std::min<int64_t>(2 * sms, (steps * p.requests + WEIGHT_WARPS - 1) / WEIGHT_WARPS);
  if (grid == 0) return GVR_OK;
  void* args[] = {&p};
  return launch(info.kernel, dim3(uint32_t(grid)), WEIGHT_THREADS, smem, 1, args, stream) == cudaSuccess ? GVR_OK : GVR_ERR_LAUNCH;
}

}  // extern "C"
