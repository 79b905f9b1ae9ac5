// gvr_attend.cu -- attention over the 4-bit paged cache, at the selected entries or over all of a
// row's entries (attend_decode and attend_prefill of include/gvr_cache.h).
//
// Mathematics.  For a query vector q of one head and entries e with keys k_e and values v_e,
//   s_e = scale q.k_e,  o = sum_e exp(s_e - m) v_e / sum_e exp(s_e - m),  lse = m + log sum_e ...
// in one pass over the entries with a running maximum m and running sums that are rescaled when m
// grows, in any grouping of the entries: groups join by the same rescaling.
//
// Work split.  A unit is a set of rows that read the same entries: one row, or (whole-cache decode)
// the next_n rows of a request.  Its queries fall into jobs of one KV head and 8 NT query vectors
// each.  A warp works on one job, alone: it fetches its own entries and keeps its own running state,
// without any CTA barrier.  A CTA holds the warps of several jobs, or SPLIT warps a job; a cluster of
// up to eight CTAs (and, given a workspace, several clusters) divide the entries further.  Warps join
// through shared memory, CTAs through distributed shared memory, clusters through the workspace and a
// second kernel.  Every sum has a fixed order.
//
// A step.  32 entries (codes and scales of K and V, 144 bytes at head_dim 128) arrive in the warp's ring
// of STAGES stages by 16-byte asynchronous copies, STAGES - 1 steps ahead; their numbers and pages are
// loaded two and one steps before that.  (Bulk copies of single rows measured slower: 20 to 48 clocks
// each on an SM whatever their size up to 320 bytes.)  The pitch of a row in shared memory is an odd
// multiple of 16 bytes, which with tile_entry's order spreads the operand reads over all banks.
// S^T = K Q^T and O^T += V^T P^T run on m16n8k16 matrix instructions with entries (for S) and head
// dimensions (for O) on the 16-row side: these have the 4-bit operand, expanded in registers straight
// into the instruction's operand layout, so nothing expanded is ever stored.  e2m1 * e4m3 has at most
// 5 significant bits and an exponent within f16's, so K and V are exact in f16.  Queries are brought
// to f16 exactly, too: a power of two per query puts a bf16 query's largest element at 2^14, and what
// f16 cannot hold below that is under 2^-39 of it.  P is rounded to f16 (11 bits): eight times finer
// than bf16 outputs, and averaged over the entries.
#include <algorithm>
#include <mutex>

#include "gvr_cache_common.cuh"
#include "../csrc/gvr_device.cuh"

namespace gvrc {
namespace {

constexpr int STEP = 32;  // entries a warp takes at a time: one per lane
constexpr int STAGES = 3;
constexpr int MAX_CLUSTER = 8;
constexpr float NO_TOP = -3.4028235e38f;  // the maximum of no scores: finite, so that differences are
constexpr int JOIN_THREADS = 512, JOIN_WAYS = 8;

struct AttendParams {
  const uint8_t* data;
  const void* q;
  const int32_t* table;
  const int32_t* lens;      // decode: kv_lens
  const int32_t* requests;  // prefill: row_requests (else nullptr)
  const int32_t* starts;
  const int32_t* ends;
  const int32_t* indices;   // nullptr: all entries
  void* out;
  float* lse;
  float* parts_out;  // parts > 1: [item][part][Q * (D + 2)] partial results
  int64_t q_row, q_head, table_stride, num_rows, k;
  uint32_t unit, page_units, entry_units, row_units;  // bytes of a unit; pages, entries and rows in units
  int32_t num_pages, page_shift, kv_heads, group, fold, capacity, next_n, ratio, num_requests, bf16;
  int32_t tiles;            // query tiles of a KV head in a unit
  int32_t heads_in, tiles_in, split, split_log2;  // a CTA's jobs: heads_in x tiles_in, SPLIT warps each
  int32_t head_groups, tile_groups;   // CTAs side by side for the jobs of a unit
  int32_t items, parts;     // units x head_groups x tile_groups; clusters of CTAs an item
  float scale_log2;  // |scale| * k_scale * log2(e); 1 for a scale of 0
  float q_sign;      // the scale's sign, which the queries take on (0 for a scale of 0)
  float v_scale;
};

// Row r of a 16-entry matrix tile <-> entry of the 16 (a permutation).  Even and odd entries
// separate, and neighbouring rows four apart modulo 8: with an odd pitch (in 16 bytes) the operand
// reads of K (two neighbouring tile rows a phase) and of V (every other tile row) then fall on
// different shared-memory banks.
__device__ __forceinline__ int tile_entry(int r) {
  const int x = r & 7, e = (x & 1) ? 8 + ((x + 3) & 7) : x;
  return e + (r >> 3);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float4 dsmem_ld_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Both halves of an f16x2 from its low or high one.
__device__ __forceinline__ uint32_t splat(uint32_t two, int high) {
  const __half2 v = *reinterpret_cast<const __half2*>(&two);
  const __half2 r = high ? __high2half2(v) : __low2half2(v);
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 16 * i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
}

template <int D, int NT>
struct Shape {
  static constexpr int RB = row_bytes(D);
  static constexpr int PITCH = 16 * (RB / 16 | 1);  // of a row in shared memory
  static constexpr int Q = 8 * NT;  // query vectors of a job
  static constexpr int WARPS = 4, THREADS = 32 * WARPS;  // at most
  // accumulators and queries take 3 D / 8 NT registers: that leaves room for 16, 12 or 8 warps on an SM
  static constexpr int BLOCKS = D * NT <= 128 && NT == 1 ? 4 : D * NT == 128 ? 3 : 2, FOLD_BLOCKS = D * NT == 128 ? 3 : BLOCKS;
  static constexpr int STAGE_BYTES = STEP * PITCH;
  static constexpr int RING = STAGES * STAGE_BYTES;                          // of a warp
  static constexpr int WALK = RING + STEP * 4;                               // and its places
  static constexpr int JOIN = (Q * D + 4 * Q) * int(sizeof(float));
  static constexpr int WARP_SMEM = WALK > JOIN ? WALK : JOIN;                // the join reuses it
};

// Eight finished values of a head: sums over exp2(score - all) v, their sum `sum`.
template <int D>
__device__ __forceinline__ void write_out(const AttendParams& p, int64_t row, int head, int d, float all, float sum,
                                          const float (&acc)[8]) {
  const float norm = sum == 0.f ? 0.f : p.v_scale / sum;
  uint32_t packed[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float lo = acc[2 * j] * norm, hi = acc[2 * j + 1] * norm;
    if (p.bf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(packed[j]) : "f"(hi), "f"(lo));
    else packed[j] = pack_f16(lo, hi);
  }
  const int64_t at = row * (int64_t(p.kv_heads) * p.group) + head;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at * D + d) = make_uint4(packed[0], packed[1], packed[2], packed[3]);
  if (p.lse && d == 0) p.lse[at] = sum == 0.f ? -INFINITY : (all + log2f(sum)) * 0.69314718055994531f;
}

// FOLD: the unit is the next_n rows of a request (whole-cache decode with next_n > 1).
template <int D, int NT, bool FOLD>
__global__ void __launch_bounds__(Shape<D, NT>::THREADS, FOLD ? Shape<D, NT>::FOLD_BLOCKS : Shape<D, NT>::BLOCKS) attend_kernel(AttendParams p) {
  using S = Shape<D, NT>;
  constexpr int KSTEPS = D / 16;       // 16-wide steps of the head dimension
  constexpr int KW = D / 32;           // 32-bit words of K codes per lane and entry
  constexpr int VW = D / 64;           // the same of V codes
  extern __shared__ __align__(128) uint8_t smem[];

  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same in every lane, and known to be
  const int warps = blockDim.x >> 5;
  const uint32_t rank = gvr::cluster_rank(), cs = gvr::cluster_size();
  const int unit = int(cs == 1 ? blockIdx.x : gvr::cluster_id_x()), part = blockIdx.z;
  const int tile_group = p.head_groups == 1 ? blockIdx.y : blockIdx.y / p.head_groups;
  const int head0 = (int(blockIdx.y) - tile_group * p.head_groups) * p.heads_in, tile0 = tile_group * p.tiles_in;
  const int job = warp >> p.split_log2, sub = warp & (p.split - 1);
  const int tile_in = p.tiles_in == 1 ? 0 : job / p.heads_in;
  const int h = head0 + job - tile_in * p.heads_in, tile = tile0 + tile_in;

  begin();

  // ---- the job's queries, on their way: lane (g, c) holds query 8 t + g at D/4 c + [0, D/4)
  const int m0 = tile * S::Q;
  const int members = tile < p.tiles ? (FOLD ? p.fold * p.group : p.group) : 0;
  uint32_t raw[NT][D / 8];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int m = m0 + 8 * t + g;
    const int64_t row = FOLD ? int64_t(unit) * p.fold + m / p.group : unit;
    const bool live = m < members && row < p.num_rows;
    const uint16_t* src = static_cast<const uint16_t*>(p.q) + row * p.q_row + int64_t(h * p.group + (FOLD ? m % p.group : m)) * p.q_head + c * (D / 4);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 v = live ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
      raw[t][4 * i] = v.x, raw[t][4 * i + 1] = v.y, raw[t][4 * i + 2] = v.z, raw[t][4 * i + 3] = v.w;
    }
  }

  // ---- the unit's entries: request and number of valid ones
  int64_t request;
  int n = 0;        // entries that some row of the unit sees
  int kv = 0;
  if (p.requests) {
    request = p.requests[unit];
    if (request >= 0 && request < p.num_requests) {
      n = window_entries(p.starts[unit], p.ends[unit], p.capacity);
    } else {
      request = 0;
    }
  } else {
    request = FOLD || p.next_n == 1 ? unit : unit / p.next_n;
    kv = p.lens[request];
    const int last = FOLD ? p.next_n - 1 : unit - int(request) * p.next_n;
    n = decode_entries(kv, p.next_n, last, p.ratio, p.capacity);
  }
  const int32_t* table = p.table + request * p.table_stride;
  const int32_t* indices = p.indices ? p.indices + int64_t(unit) * p.k : nullptr;
  const int64_t listed = indices ? (n > 0 ? p.k : 0) : n;  // positions to walk over
  const int steps = int((listed + STEP - 1) / STEP);
  const int walkers = p.parts * int(cs) * p.split, me = (part * int(cs) + int(rank)) * p.split + sub;
  const int mine = walkers == 1 ? steps : steps > me ? (steps - me + walkers - 1) / walkers : 0;

  // ---- fetching
  uint8_t* ring = smem + warp * S::RING;
  uint32_t* places = reinterpret_cast<uint32_t*>(smem + warps * S::RING) + warp * STEP;
  constexpr int CODES = D / 16, SCALES = S::RB / 16 - CODES;  // 16-byte pieces of a row: of codes, of scales
  // (listed entries are loaded whatever the row's length, which may still be on its way)
  const uint32_t stride = walkers * STEP, end = indices ? uint32_t(p.k) : uint32_t(n);
  uint32_t pos = me * STEP + lane;  // of the entry that this lane loads next; below 2^32 even behind the last
  auto load_entry = [&]() -> int {  // -1: none
    int e = -1;
    if (pos < end) e = indices ? __ldg(indices + pos) : int(pos);
    pos += stride;
    return e;
  };
  auto load_page = [&](int e) -> int { return uint32_t(e) < uint32_t(n) ? __ldg(table + (e >> p.page_shift)) : -1; };
  // CODES neighbouring lanes copy a row's codes, every lane a row's scales
  const uint8_t* codes_from = p.data + lane % CODES * 16;
  const uint32_t codes_to = lane / CODES * S::PITCH + lane % CODES * 16, scales_to = lane * S::PITCH + D;
  const uint32_t head_units = h * p.row_units;
  // Starts the copies of a step; returns which lanes' entries exist.
  auto fetch = [&](uint32_t to, int e, int page) -> uint32_t {
    const bool is = uint32_t(page) < uint32_t(p.num_pages);
    const uint32_t there = __ballot_sync(0xffffffffu, is);
    if (there) {
      uint32_t from = row_unit(page, e, p.page_shift, p.page_units, p.entry_units, head_units);
      if (there != 0xffffffffu) {  // a missing entry is fetched from where another lies, and not looked at
        const uint32_t some = __shfl_sync(0xffffffffu, from, __ffs(there) - 1);
        if (!is) from = some;
      }
      places[lane] = from;
      __syncwarp();
#pragma unroll
      for (int j = 0; j < CODES; ++j)
        copy16(to + codes_to + j * (32 / CODES) * S::PITCH, codes_from + uint64_t(places[j * (32 / CODES) + lane / CODES]) * p.unit);
#pragma unroll
      for (int j = 0; j < SCALES; ++j) copy16(to + scales_to + j * 16, p.data + uint64_t(from) * p.unit + D + j * 16);
    }
    copy_commit();
    return there;
  };
  const uint32_t ring_at = gvr::smem_u32(ring);
  uint32_t masks[STAGES];  // of the steps under way
  int e_ahead, e_after, page_ahead;
  {
    int e[STAGES + 1], pg[STAGES];
#pragma unroll
    for (int i = 0; i < STAGES + 1; ++i) e[i] = load_entry();
#pragma unroll
    for (int i = 0; i < STAGES; ++i) pg[i] = load_page(e[i]);
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
      masks[i] = fetch(ring_at + i * S::STAGE_BYTES, e[i], pg[i]);
      __syncwarp();
    }
    e_ahead = e[STAGES - 1], page_ahead = pg[STAGES - 1], e_after = e[STAGES];
  }

  // ---- the queries as operands
  uint32_t qb[NT][KSTEPS][2];
  float factor[NT][2];  // of the scores of queries 8 t + 2 c, 8 t + 2 c + 1: to log2 units
  int limit[NT][2];     // entries that these queries see
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float back = 1.f;
    if (p.bf16) {
      // 2^up with up = 14 - exponent of the largest; none of zero or infinite queries
      uint32_t big = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) big = __vmaxu2(big, raw[t][i] & 0x7fff7fffu);
      big = max(big & 0xffffu, big >> 16);
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
      const int exponent = int(big >> 7), up = big == 0 || exponent == 255 ? 0 : min(14 - (exponent - 127), 126);
      const float mul = p.q_sign * __uint_as_float(uint32_t(127 + up) << 23);
      back = __uint_as_float(uint32_t(127 - up) << 23);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        qb[t][i / 2][i % 2] = pack_f16(__uint_as_float(raw[t][i] << 16) * mul, __uint_as_float(raw[t][i] & 0xffff0000u) * mul);
    } else {
      const uint32_t sign = pack_f16(p.q_sign, p.q_sign);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) qb[t][i / 2][i % 2] = hmul2(raw[t][i], sign);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      factor[t][j] = fmaxf(__shfl_sync(0xffffffffu, back, (2 * c + j) * 4) * p.scale_log2, 1.17549435e-38f);  // never 0
      const int mm = m0 + 8 * t + 2 * c + j;
      if (FOLD) limit[t][j] = decode_entries(kv, p.next_n, min(mm / p.group, p.fold - 1), p.ratio, p.capacity);
    }
  }
  // entries below this are seen by every query of the unit
  const int sure = FOLD ? decode_entries(kv, p.next_n, 0, p.ratio, p.capacity) : n;

  const int first_row = FOLD ? m0 / p.group : 0, last_row = FOLD ? min((m0 + S::Q - 1) / p.group, p.fold - 1) : 0;  // of the job
  int row_of_query[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) row_of_query[t] = FOLD ? (m0 + 8 * t + g) / p.group : 0;

  // ---- the walk
  float o[NT][KSTEPS][4];
  float top[NT][2], total[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int i = 0; i < KSTEPS; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[t][i][j] = 0.f;
    top[t][0] = top[t][1] = NO_TOP;
    total[t][0] = total[t][1] = 0.f;
  }
  // where this lane's operand rows start in a stage: of K, tile rows g and g + 8 (the next entry); of V,
  // columns 2 c and 2 c + 1 (and 8 behind them, the next entries)
  const int k_at = tile_entry(g) * S::PITCH;
  const int v_at0 = tile_entry(2 * c) * S::PITCH, v_at1 = tile_entry(2 * c + 1) * S::PITCH;
  int now = 0;  // this step's stage in bytes
  for (int i = 0; i < mine; ++i) {
    {
      copy_wait<STAGES - 2>();
      __syncwarp();  // the step's entries are here, and every lane is done with the stage before it
      masks[STAGES - 1] = fetch(ring_at + (now == 0 ? (STAGES - 1) * S::STAGE_BYTES : now - S::STAGE_BYTES), e_ahead, page_ahead);
      e_ahead = e_after;
      page_ahead = load_page(e_ahead);
      e_after = load_entry();

      const uint8_t* st = ring + now;
      const uint32_t mask = masks[0];
      now = now == (STAGES - 1) * S::STAGE_BYTES ? 0 : now + S::STAGE_BYTES;
#pragma unroll
      for (int j = 0; j < STAGES - 1; ++j) masks[j] = masks[j + 1];
      if (mask == 0) continue;

      // S^T: two tiles of 16 entries
      float s[2][NT][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const uint8_t* r0 = st + k_at + 16 * mt * S::PITCH;
        const uint8_t* r1 = r0 + S::PITCH;
        uint32_t k0[KW], k1[KW];
        load_words<KW>(r0 + c * (D / 8), k0);
        load_words<KW>(r1 + c * (D / 8), k1);
        uint32_t sc0, sc1;  // the lane's D/64 scales of each row
        if (D == 64) sc0 = r0[D + c], sc1 = r1[D + c];
        else if (D == 128) sc0 = *reinterpret_cast<const uint16_t*>(r0 + D + 2 * c), sc1 = *reinterpret_cast<const uint16_t*>(r1 + D + 2 * c);
        else sc0 = *reinterpret_cast<const uint32_t*>(r0 + D + 4 * c), sc1 = *reinterpret_cast<const uint32_t*>(r1 + D + 4 * c);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[mt][t][j] = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {  // 8 values of each row a word: two 16-wide steps
          uint32_t a[4], b[4];
          e2m1_to_f16x2(k0[w], a);
          e2m1_to_f16x2(k1[w], b);
          const int block = w / 2;  // 16 values a scale
          const uint32_t two0 = e4m3x2_to_f16x2(sc0 >> (16 * (block / 2))), two1 = e4m3x2_to_f16x2(sc1 >> (16 * (block / 2)));
          const uint32_t x0 = splat(two0, block & 1), x1 = splat(two1, block & 1);
#pragma unroll
          for (int j = 0; j < 4; ++j) a[j] = hmul2(a[j], x0), b[j] = hmul2(b[j], x1);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma(s[mt][t], a[0], b[0], a[1], b[1], qb[t][2 * w][0], qb[t][2 * w][1]);
            mma(s[mt][t], a[2], b[2], a[3], b[3], qb[t][2 * w + 1][0], qb[t][2 * w + 1][1]);
          }
        }
      }

      // entries that are skipped or beyond a query's limit leave the sums
      // entries that only some rows of the unit see (at most at its end)
      const int64_t first = int64_t(me + i * walkers) * STEP;
      const bool border = FOLD && first + STEP > sure;
      if (mask != 0xffffffffu || border) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = 16 * mt + tile_entry(g + 8 * (j >> 1));
            const bool there = (mask >> at) & 1;
#pragma unroll
            for (int t = 0; t < NT; ++t)
              if (!there || (border && first + at >= limit[t][j & 1])) s[mt][t][j] = -INFINITY;
          }
      }

      // The base that scores are taken against: the maximum when it was last set, kept while no score is
      // more than 2^8 above it (P stays within f16).
      bool grow = false;
      float high[NT][2];  // of this lane's scores, in log2 units; factors are positive
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          high[t][j] = fmaxf(fmaxf(s[0][t][j], s[0][t][j + 2]), fmaxf(s[1][t][j], s[1][t][j + 2])) * factor[t][j];
          grow |= high[t][j] > top[t][j] + 8.f;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float down[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float next = fmaxf(top[t][j], high[t][j]);
            next = fmaxf(next, __shfl_xor_sync(0xffffffffu, next, 4));
            next = fmaxf(next, __shfl_xor_sync(0xffffffffu, next, 8));
            next = fmaxf(next, __shfl_xor_sync(0xffffffffu, next, 16));
            down[j] = exp2_fast(top[t][j] - next);
            top[t][j] = next;
            total[t][j] *= down[j];
          }
#pragma unroll
          for (int x = 0; x < KSTEPS; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[t][x][j] *= down[j & 1];
        }
      }

      uint32_t pb[2][NT][2];  // P^T as operands
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const float e0 = exp2_fast(fmaf(s[mt][t][0], factor[t][0], -top[t][0])), e1 = exp2_fast(fmaf(s[mt][t][1], factor[t][1], -top[t][1]));
          const float e2 = exp2_fast(fmaf(s[mt][t][2], factor[t][0], -top[t][0])), e3 = exp2_fast(fmaf(s[mt][t][3], factor[t][1], -top[t][1]));
          total[t][0] += e0 + e2;
          total[t][1] += e1 + e3;
          pb[mt][t][0] = transpose8x8(pack_f16(e0, e1));
          pb[mt][t][1] = transpose8x8(pack_f16(e2, e3));
        }
      }

      // O^T += V^T P^T: lane (g, c) expands V at D/8 g + [0, D/8) of four entries of each tile.  An
      // entry that is left out has P = 0 and, as 0 x NaN is NaN, a V scale of 0.  At the border that
      // differs from row to row, so each row of the job takes a pass with its own entries.
      auto add_values = [&](uint32_t there, const uint32_t (&pj)[2][NT][2]) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          uint32_t v[4][VW], vs[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint8_t* r = st + (x & 1 ? v_at1 : v_at0) + (16 * mt + (x >> 1)) * S::PITCH;
            load_words<VW>(r + D / 2 + g * (D / 16), v[x]);
            if (D == 64) vs[x] = r[D + D / 16 + (g >> 1)];
            else if (D == 128) vs[x] = r[D + D / 16 + g];
            else vs[x] = *reinterpret_cast<const uint16_t*>(r + D + D / 16 + 2 * g);
          }
          if (there != 0xffffffffu) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (!((there >> (16 * mt + tile_entry(2 * c + (x & 1) + 8 * (x >> 1)))) & 1)) vs[x] = 0;
          }
          uint32_t x01[VW > 2 ? 2 : 1], x23[VW > 2 ? 2 : 1];  // scales of the entry pairs
#pragma unroll
          for (int b = 0; b < (VW > 2 ? 2 : 1); ++b) {
            x01[b] = e4m3x2_to_f16x2(__byte_perm(vs[0], vs[1], b ? 0x0051 : 0x0040));
            x23[b] = e4m3x2_to_f16x2(__byte_perm(vs[2], vs[3], b ? 0x0051 : 0x0040));
          }
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            // bytes of (entry 0, entry 1) codes: of the even values, of the odd values
            uint32_t lo01[4], hi01[4], lo23[4], hi23[4];
            e2m1_to_f16x2((v[0][w] & 0x0f0f0f0fu) | ((v[1][w] << 4) & 0xf0f0f0f0u), lo01);
            e2m1_to_f16x2(((v[0][w] >> 4) & 0x0f0f0f0fu) | (v[1][w] & 0xf0f0f0f0u), hi01);
            e2m1_to_f16x2((v[2][w] & 0x0f0f0f0fu) | ((v[3][w] << 4) & 0xf0f0f0f0u), lo23);
            e2m1_to_f16x2(((v[2][w] >> 4) & 0x0f0f0f0fu) | (v[3][w] & 0xf0f0f0f0u), hi23);
            const uint32_t y01 = x01[w / 2], y23 = x23[w / 2];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const uint32_t a0 = hmul2(lo01[b], y01), a1 = hmul2(hi01[b], y01);
              const uint32_t a2 = hmul2(lo23[b], y23), a3 = hmul2(hi23[b], y23);
#pragma unroll
              for (int t = 0; t < NT; ++t) mma(o[t][4 * w + b], a0, a1, a2, a3, pj[mt][t][0], pj[mt][t][1]);
            }
          }
        }
      };
      if (!border) {
        add_values(mask, pb);
      } else {
        for (int j = first_row; j <= last_row; ++j) {
          const int64_t seen = decode_entries(kv, p.next_n, j, p.ratio, p.capacity) - first;
          uint32_t pj[2][NT][2];
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int x = 0; x < 2; ++x) pj[mt][t][x] = row_of_query[t] == j ? pb[mt][t][x] : 0;
          add_values(mask & (seen <= 0 ? 0u : seen >= 32 ? 0xffffffffu : (1u << int(seen)) - 1), pj);
        }
      }
    }
  }
  copy_wait<0>();
  __syncthreads();  // every copy has landed, every stage is read: the ring becomes the partial results

  // ---- the lanes' sums of each query
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float v = total[t][j];
      v += __shfl_xor_sync(0xffffffffu, v, 4);
      v += __shfl_xor_sync(0xffffffffu, v, 8);
      v += __shfl_xor_sync(0xffffffffu, v, 16);
      total[t][j] = v;
    }
  const int jobs = warps >> p.split_log2;
  if (walkers == 1) {  // the warp has its job's whole sums: lane (g, c) writes D/8 values
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int m = m0 + 8 * t + 2 * c + j;
        const int64_t row = FOLD ? int64_t(unit) * p.fold + m / p.group : unit;
        if (m >= members || row >= p.num_rows) continue;
#pragma unroll
        for (int x = 0; x < KSTEPS; x += 4) {
          float acc[8];
#pragma unroll
          for (int y = 0; y < 4; ++y) acc[2 * y] = o[t][x + y][j], acc[2 * y + 1] = o[t][x + y][j + 2];
          write_out<D>(p, row, h * p.group + (FOLD ? m % p.group : m), g * (D / 8) + 2 * x, top[t][j], total[t][j], acc);
        }
      }
    return;
  }

  // ---- join the warps of a job, then the CTAs
  float* partial = reinterpret_cast<float*>(smem);   // [warps][Q][D]
  float* tops = partial + warps * S::Q * D;          // [warps][Q]
  float* sums = tops + warps * S::Q;                 // [warps][Q]
  float* joined = sums + warps * S::Q;               // [jobs][2][Q]: maximum and sum of a job in this CTA
  if (g == 0) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        tops[warp * S::Q + 8 * t + 2 * c + j] = top[t][j];
        sums[warp * S::Q + 8 * t + 2 * c + j] = total[t][j];
      }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int qi = 8 * t + 2 * c + j;
      float all = NO_TOP;
      for (int w = job * p.split; w < (job + 1) * p.split; ++w) all = fmaxf(all, tops[w * S::Q + qi]);
      const float down = exp2_fast(top[t][j] - all);
      float* dst = partial + (warp * S::Q + qi) * D + g * (D / 8);
#pragma unroll
      for (int x = 0; x < KSTEPS; ++x)
        *reinterpret_cast<float2*>(dst + 2 * x) = make_float2(o[t][x][j] * down, o[t][x][j + 2] * down);
      if (sub == 0 && g == 0) {
        float sum = 0.f;
        for (int w = job * p.split; w < (job + 1) * p.split; ++w) {
          const float tw = tops[w * S::Q + qi];
          sum += sums[w * S::Q + qi] * exp2_fast(tw - all);
        }
        joined[job * 2 * S::Q + qi] = all;
        joined[job * 2 * S::Q + S::Q + qi] = sum;
      }
    }
  __syncthreads();
  constexpr int EIGHTS = D / 8;
  if (p.split > 1) {
    // the job's sum over its warps, in place of its first warp's
    for (int i = tid; i < jobs * S::Q * D / 4; i += blockDim.x) {
      float4* at = reinterpret_cast<float4*>(partial) + i / (S::Q * D / 4) * p.split * (S::Q * D / 4) + i % (S::Q * D / 4);
      float4 sum = *at;
      for (int w = 1; w < p.split; ++w) {
        const float4 v = at[w * S::Q * D / 4];
        sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
      }
      *at = sum;
    }
  }
  if (cs > 1) gvr::cluster_sync();
  else __syncthreads();
  const uint32_t partial_addr = gvr::smem_u32(partial), joined_addr = gvr::smem_u32(joined);
  // each CTA of the cluster finishes its share of jobs x queries x head dimension, eight values a thread
  for (int i = int(rank) * blockDim.x + tid; i < jobs * S::Q * EIGHTS; i += int(cs) * blockDim.x) {
    const int jb = i / (S::Q * EIGHTS), qi = i / EIGHTS % S::Q, d = i % EIGHTS * 8;
    const int m = (tile0 + jb / p.heads_in) * S::Q + qi, hj = head0 + jb % p.heads_in;
    const int64_t row = FOLD ? int64_t(unit) * p.fold + m / p.group : unit;
    if (m >= p.fold * p.group || row >= p.num_rows) continue;
    const uint32_t top_at = joined_addr + (jb * 2 * S::Q + qi) * 4, sum_at = top_at + S::Q * 4;
    const uint32_t at = partial_addr + (jb * p.split * S::Q * D + qi * D + d) * 4;
    float all = NO_TOP, sum = 0.f, acc[8];
#pragma unroll
    for (int y = 0; y < 8; ++y) acc[y] = 0.f;
    for (uint32_t r = 0; r < cs; ++r) all = fmaxf(all, __uint_as_float(gvr::dsmem_ld_u32(gvr::dsmem_map(top_at, r))));
    for (uint32_t r = 0; r < cs; ++r) {
      const float tr = __uint_as_float(gvr::dsmem_ld_u32(gvr::dsmem_map(top_at, r)));
      const float down = exp2_fast(tr - all);
      sum += down * __uint_as_float(gvr::dsmem_ld_u32(gvr::dsmem_map(sum_at, r)));
      const float4 a = dsmem_ld_f32x4(gvr::dsmem_map(at, r)), b = dsmem_ld_f32x4(gvr::dsmem_map(at + 16, r));
      acc[0] += down * a.x, acc[1] += down * a.y, acc[2] += down * a.z, acc[3] += down * a.w;
      acc[4] += down * b.x, acc[5] += down * b.y, acc[6] += down * b.z, acc[7] += down * b.w;
    }
    if (p.parts > 1) {
      float* dst = p.parts_out + (((int64_t(unit) * gridDim.y + blockIdx.y) * jobs + jb) * p.parts + part) * (S::Q * (D + 2));
      *reinterpret_cast<float4*>(dst + qi * D + d) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      *reinterpret_cast<float4*>(dst + qi * D + d + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
      if (d == 0) dst[S::Q * D + qi] = all, dst[S::Q * (D + 1) + qi] = sum;
    } else {
      write_out<D>(p, row, hj * p.group + (FOLD ? m % p.group : m), d, all, sum, acc);
    }
  }
  if (cs > 1) gvr::cluster_sync();  // no CTA leaves while another reads its shared memory
}

// Joins the parts of a job that was split over several clusters: one CTA a job, eight values a
// thread, JOIN_WAYS threads for the same values taking every JOIN_WAYS-th part in order and then
// joining through shared memory.  It is launched while the walk still runs and waits for its end.
template <int D, int NT>
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(AttendParams p) {
  using S = Shape<D, NT>;
  constexpr int EIGHTS = D / 8, TURN = JOIN_THREADS / JOIN_WAYS, PART = S::Q * (D + 2);
  __shared__ float shared[JOIN_WAYS][TURN][10];
  const int jobs = p.heads_in * p.tiles_in, item = blockIdx.x / jobs, jb = blockIdx.x % jobs;
  const int groups = p.head_groups * p.tile_groups, group = item % groups;
  const int h = group % p.head_groups * p.heads_in + jb % p.heads_in;
  const int tile = group / p.head_groups * p.tiles_in + jb / p.heads_in;
  const int64_t unit = item / groups;
  const float* src = p.parts_out + int64_t(blockIdx.x) * p.parts * PART;
  const int way = threadIdx.x / TURN, at = threadIdx.x % TURN;
  begin();
  for (int i0 = 0; i0 < S::Q * EIGHTS; i0 += TURN) {
    const int i = i0 + at, qi = i / EIGHTS, d = (i % EIGHTS) * 8;
    float all = NO_TOP, sum = 0.f, acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
#pragma unroll 4
    for (int r = way; r < p.parts; r += JOIN_WAYS) {
      const float* from = src + int64_t(r) * PART;
      const float tr = from[S::Q * D + qi], sr = from[S::Q * (D + 1) + qi];
      const float4 a = *reinterpret_cast<const float4*>(from + qi * D + d), b = *reinterpret_cast<const float4*>(from + qi * D + d + 4);
      const float next = fmaxf(all, tr), down = exp2_fast(all - next), up = exp2_fast(tr - next);
      all = next, sum = sum * down + sr * up;
      acc[0] = acc[0] * down + a.x * up, acc[1] = acc[1] * down + a.y * up, acc[2] = acc[2] * down + a.z * up;
      acc[3] = acc[3] * down + a.w * up, acc[4] = acc[4] * down + b.x * up, acc[5] = acc[5] * down + b.y * up;
      acc[6] = acc[6] * down + b.z * up, acc[7] = acc[7] * down + b.w * up;
    }
    float* mine = shared[way][at];
    mine[0] = all, mine[1] = sum;
#pragma unroll
    for (int j = 0; j < 8; ++j) mine[2 + j] = acc[j];
    __syncthreads();
    const int m = tile * S::Q + qi;
    const int64_t row = unit * p.fold + m / p.group;
    if (way == 0 && m < p.fold * p.group && row < p.num_rows) {
      for (int w = 1; w < JOIN_WAYS; ++w) {
        const float* other = shared[w][at];
        const float next = fmaxf(all, other[0]), down = exp2_fast(all - next), up = exp2_fast(other[0] - next);
        all = next, sum = sum * down + other[1] * up;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = acc[j] * down + other[2 + j] * up;
      }
      write_out<D>(p, row, h * p.group + m % p.group, d, all, sum, acc);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------------- host
struct KernelInfo {
  const void* kernel[2];  // by FOLD
  const void* join;
  int queries, warps;
  int part_bytes;  // of one job's results
  int warp_smem;   // shared memory of a warp
};

template <int D, int NT>
KernelInfo info() {
  using S = Shape<D, NT>;
  return {{reinterpret_cast<const void*>(attend_kernel<D, NT, false>), reinterpret_cast<const void*>(attend_kernel<D, NT, true>)},
          reinterpret_cast<const void*>(join_kernel<D, NT>), S::Q,
          S::WARPS, S::Q * (D + 2) * int(sizeof(float)), S::WARP_SMEM};
}

constexpr int KERNELS = 6;
const KernelInfo& kernel_info(int i) {
  static const KernelInfo all[KERNELS] = {info<64, 1>(), info<64, 2>(), info<64, 4>(), info<128, 1>(), info<128, 2>(), info<256, 1>()};
  return all[i];
}

// 8, 16 or 32 query vectors a job, as far as the accumulators (head_dim / 16 x 4 registers for each
// 8) leave room.
int choose_kernel(int dim, int64_t members) {
  if (dim == 64) return members <= 8 ? 0 : members <= 16 ? 1 : 2;
  if (dim == 128) return members <= 8 ? 3 : 4;
  return 5;
}

struct Device {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
  int sms = 0, smem_per_sm = 0, smem_reserved = 0;
  int warps[KERNELS][2] = {};  // resident per SM, as far as registers go
};
Device g_devices[kMaxDevices];

cudaError_t device_info(Device** out) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  Device& d = g_devices[dev];  // sm_count has checked dev
  std::call_once(d.once, [&d, sms, dev]() {
    d.sms = sms;
    int most = 0;
    d.err = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (d.err == cudaSuccess) d.err = cudaDeviceGetAttribute(&d.smem_per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
    if (d.err == cudaSuccess) d.err = cudaDeviceGetAttribute(&d.smem_reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev);
    for (int i = 0; i < KERNELS && d.err == cudaSuccess; ++i) {
      const KernelInfo& k = kernel_info(i);
      for (int f = 0; f < 2; ++f) {
        cudaFuncAttributes a;
        if (d.err == cudaSuccess) d.err = cudaFuncGetAttributes(&a, k.kernel[f]);
        if (d.err == cudaSuccess)
          d.err = cudaFuncSetAttribute(k.kernel[f], cudaFuncAttributeMaxDynamicSharedMemorySize, most - int(a.sharedSizeBytes));
        if (d.err == cudaSuccess)
          d.err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&d.warps[i][f], k.kernel[f], 32, 0);
      }
    }
  });
  *out = &d;
  return d.err;
}

// A launch shape: a CTA's jobs are all query tiles of a KV head as far as its warps go, then
// neighbouring KV heads (a divisor of their number), then several warps a job.
struct Geometry {
  int heads_in = 1, tiles_in = 1, head_groups = 1, tile_groups = 1, split_log2 = 0, cluster = 1;
  int64_t groups = 1, parts = 1;  // CTAs side by side for a unit; clusters of CTAs for the entries
  float cost = 1e30f;
};

// Expected time in us of a launch, from what was measured over shapes of 1 to 700 rows and 512 to 131071
// entries: a step of each kernel beside w warps on its SM, what a warp does around its steps, what a
// second join and what many CTAs cost.  (head_dim 128, 8 queries: 0.55 a step alone, 1.16 beside 8 warps,
// 2.03 beside 16, so more than 8 warps an SM gain little, and cost their start.  CTAs of eight warps were
// slower everywhere: their clusters spread less evenly over the SMs.)
struct Expected {
  float least, fixed, per_warp;
};
constexpr Expected STEP_US[KERNELS] = {{0.35f, 0.2f, 0.06f}, {0.5f, 0.4f, 0.07f}, {0.8f, 0.6f, 0.1f},
                                       {0.55f, 0.3f, 0.108f}, {0.8f, 0.8f, 0.1f}, {0.9f, 0.9f, 0.16f}};

struct Call {
  int kernel, kv_heads, tiles;
  int64_t units, steps, part_room;
  bool listed, large;  // entries listed by indices; a cache larger than the TLBs cover
};

Geometry plan(const Device& d, const KernelInfo& info, int warps_by_registers, const Call& call, int warps) {
  Geometry g;
  g.tile_groups = (call.tiles + warps - 1) / warps;
  g.tiles_in = (call.tiles + g.tile_groups - 1) / g.tile_groups;
  g.heads_in = std::min(call.kv_heads, warps / g.tiles_in);
  while (call.kv_heads % g.heads_in) --g.heads_in;
  g.head_groups = call.kv_heads / g.heads_in;
  g.groups = int64_t(g.tile_groups) * g.head_groups;
  while ((g.heads_in * g.tiles_in) << (g.split_log2 + 1) <= warps) ++g.split_log2;
  const int jobs = g.heads_in * g.tiles_in, cta_warps = jobs << g.split_log2;
  const int per_sm = std::max(1, std::min(warps_by_registers / cta_warps, d.smem_per_sm / (cta_warps * info.warp_smem + d.smem_reserved)));
  const int64_t resident = int64_t(d.sms) * per_sm, items = call.units * g.groups;
  const int64_t turns = (call.steps + (1 << g.split_log2) - 1) >> g.split_log2;  // steps of a warp, were there one CTA
  const Expected& x = STEP_US[call.kernel];
  const float missing = call.listed && call.large ? 0.21f / 256.f * std::pow(float(g.head_groups), 0.7f) : 0.f;
  for (int64_t split = 1; split == 1 || split <= turns;) {
    // up to a cluster, then whole clusters (`parts`) joined by a second kernel through the workspace
    const int cs = int(std::min<int64_t>(split, MAX_CLUSTER));
    const int64_t parts = split / cs, ctas = items * split;
    if (parts > 1 && (parts * items * jobs > call.part_room || ctas > resident)) break;
    const float own = float((turns + split - 1) / split);
    auto cta_us = [&](float w) {
      float step = std::max(x.least, x.fixed + x.per_warp * (call.listed ? w : 0.7f * w));  // of whole rows some end early
      // heads of a listed entry that are fetched by CTAs apart: more requests, and in a cache that the TLBs
      // do not cover more misses (5 GB, 8 heads in 4 groups beside 14 warps: 1.4 times)
      if (call.listed) step *= 1.f + 0.015f * float(g.head_groups - 1) + (call.large ? missing * w * w : 0.f);
      return 0.2f * w + 0.4f * float(cta_warps) + own * step;
    };
    float cost;
    if (ctas <= resident) cost = cta_us(float((ctas + d.sms - 1) / d.sms * cta_warps));
    else cost = float(ctas) / float(resident) * cta_us(float(per_sm * cta_warps)) + cta_us(float(cta_warps));
    if (!call.listed) cost *= 1.f + 0.25f / float(split);  // rows shorter than the table: the longest end last
    if (ctas > 1024) cost += 0.011f * float(ctas - 1024);
    if (cta_warps > jobs || split > 1) cost += 0.7f;
    if (parts > 1) cost += 2.5f;
    if (cost < g.cost) g.cost = cost, g.cluster = cs, g.parts = parts;
    split = split < MAX_CLUSTER ? split + 1 : split * 2;
  }
  return g;
}

gvr_status attend(const gvr_cache* cache, AttendParams& p, int64_t q_row_stride, int64_t q_head_stride, int32_t dtype,
                  int64_t num_rows, int32_t num_heads, int64_t table_stride, int64_t table_width, int64_t k, float scale,
                  void* workspace, size_t workspace_bytes, void* stream) {
  const int group = num_heads / cache->num_kv_heads;
  p.data = static_cast<const uint8_t*>(cache->data);
  const int row = row_bytes(cache->head_dim);
  p.unit = unit_bytes(cache->page_stride, row);
  p.page_units = uint32_t(cache->page_stride / p.unit);
  p.row_units = row / p.unit;
  p.entry_units = p.row_units * cache->num_kv_heads;
  p.q_row = q_row_stride;
  p.q_head = q_head_stride;
  p.table_stride = table_stride;
  p.num_rows = num_rows;
  p.k = k;
  p.num_pages = int32_t(cache->num_pages);
  p.page_shift = log2_of(cache->page_size);
  p.kv_heads = cache->num_kv_heads;
  p.group = group;
  p.capacity = cache->num_pages > 0 ? int32_t(table_width * cache->page_size) : 0;  // no pages: no entries
  p.bf16 = dtype == GVR_BF16;
  p.scale_log2 = scale == 0.f ? 1.f : float(std::fabs(double(scale)) * cache->k_scale * 1.4426950408889634);
  p.q_sign = scale > 0.f ? 1.f : scale < 0.f ? -1.f : 0.f;
  p.v_scale = cache->v_scale;
  // whole-cache decode: the rows of a request read the same entries, so they share a unit
  p.fold = p.indices ? 1 : p.next_n;
  const int64_t members = int64_t(p.fold) * group;
  if (members > kIntMax) return GVR_ERR_ARG;
  const int kernel = choose_kernel(cache->head_dim, members);
  const KernelInfo& info = kernel_info(kernel);
  p.tiles = int32_t((members + info.queries - 1) / info.queries);
  const int64_t units = (num_rows + p.fold - 1) / p.fold;
  if (int64_t(p.kv_heads) * p.tiles > 65535 || units > kIntMax / MAX_CLUSTER / (int64_t(p.kv_heads) * p.tiles)) return GVR_ERR_ARG;
  Device* d = nullptr;
  if (device_info(&d) != cudaSuccess) return GVR_ERR_LAUNCH;
  const int64_t steps = ((p.indices ? k : p.capacity) + STEP - 1) / STEP;
  const Call call = {kernel, p.kv_heads, p.tiles, units, steps,
                     workspace ? int64_t(std::min<size_t>(workspace_bytes, size_t(1) << 40)) / info.part_bytes : 0,
                     p.indices != nullptr, cache->num_pages * cache->page_stride > (int64_t(2) << 30)};
  Geometry best;
  for (int warps = info.warps; warps >= 1; warps /= 2) {
    const Geometry g = plan(*d, info, d->warps[kernel][p.fold > 1], call, warps);
    if (g.cost < best.cost) best = g;
  }
  p.heads_in = best.heads_in;
  p.tiles_in = best.tiles_in;
  p.head_groups = best.head_groups;
  p.tile_groups = best.tile_groups;
  p.split_log2 = best.split_log2;
  p.split = 1 << best.split_log2;
  p.items = int32_t(units * best.groups);
  const int jobs = p.heads_in * p.tiles_in, threads = 32 * jobs * p.split, smem = jobs * p.split * info.warp_smem, cs = best.cluster;
  const int64_t groups = best.groups;
  p.parts = int32_t(best.parts);
  p.parts_out = static_cast<float*>(workspace);
  void* args[] = {&p};
  const void* main_kernel = info.kernel[p.fold > 1];
  const dim3 grid(uint32_t(units * cs), uint32_t(groups), uint32_t(p.parts));
  cudaError_t e = launch(main_kernel, grid, threads, smem, cs, args, stream);
  if (e == cudaSuccess && p.parts > 1) e = launch(info.join, dim3(uint32_t(p.items * jobs)), JOIN_THREADS, 0, 1, args, stream);
  return e == cudaSuccess ? GVR_OK : GVR_ERR_LAUNCH;
}

gvr_status check_attend(const gvr_cache* cache, const void* q, int64_t q_row_stride, int64_t q_head_stride, int32_t dtype,
                        int64_t num_rows, int32_t num_heads, const int32_t* table, int64_t table_stride,
                        int64_t table_width, float scale, const void* out, const float* lse) {
  const gvr_status s = check_cache(cache);
  if (s != GVR_OK) return s;
  if ((dtype != GVR_BF16 && dtype != GVR_F16) || num_rows < 0 || num_heads < 1 || num_heads % cache->num_kv_heads != 0 ||
      num_heads > 1 << 20 || !std::isfinite(scale) || table_width < 0 || table_width > kIntMax / cache->page_size)
    return GVR_ERR_ARG;
  if (q_row_stride < 0 || q_head_stride < 0 || q_row_stride % 8 != 0 || q_head_stride % 8 != 0 || q_row_stride > kIntMax ||
      q_head_stride > kIntMax || table_stride < table_width || table_stride > kIntMax)
    return GVR_ERR_STRIDE;
  if (num_rows == 0) return GVR_OK;
  if (!q || !out || (table_width > 0 && !table)) return GVR_ERR_NULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(table, 4) || !aligned(lse, 4)) return GVR_ERR_ALIGN;
  return GVR_OK;
}

}  // namespace
}  // namespace gvrc

extern "C" {

gvr_status attend_decode(const gvr_cache* cache, const void* q, int64_t q_row_stride, int64_t q_head_stride, int32_t dtype,
                         int64_t num_rows, int32_t num_heads, const int32_t* block_table, int64_t table_stride,
                         int64_t table_width, const int32_t* kv_lens, int32_t next_n, int32_t compress_ratio,
                         const int32_t* indices, int64_t k, float scale, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
  using namespace gvrc;
  const gvr_status s = check_attend(cache, q, q_row_stride, q_head_stride, dtype, num_rows, num_heads, block_table,
                                    table_stride, table_width, scale, out, lse);
  if (s != GVR_OK) return s;
  if (next_n < 1 || next_n > 4096 || compress_ratio < 1 || (indices && (k < 1 || k > kIntMax))) return GVR_ERR_ARG;
  if (num_rows == 0) return GVR_OK;
  if (!kv_lens) return GVR_ERR_NULL;
  if (!aligned(kv_lens, 4) || !aligned(indices, 4) || !aligned(workspace, 16)) return GVR_ERR_ALIGN;
  AttendParams p = {};
  p.q = q;
  p.table = block_table;
  p.lens = kv_lens;
  p.indices = indices;
  p.out = out;
  p.lse = lse;
  p.next_n = next_n;
  p.ratio = compress_ratio;
  return attend(cache, p, q_row_stride, q_head_stride, dtype, num_rows, num_heads, table_stride, table_width, k, scale, workspace,
                workspace_bytes, stream);
}

gvr_status attend_prefill(const gvr_cache* cache, const void* q, int64_t q_row_stride, int64_t q_head_stride, int32_t dtype,
                          int64_t num_rows, int32_t num_heads, const int32_t* block_table, int64_t table_stride,
                          int64_t table_width, int64_t num_requests, const int32_t* row_requests, const int32_t* row_starts,
                          const int32_t* row_ends, const int32_t* indices, int64_t k, float scale, void* out, float* lse,
                          void* workspace, size_t workspace_bytes, void* stream) {
  using namespace gvrc;
  const gvr_status s = check_attend(cache, q, q_row_stride, q_head_stride, dtype, num_rows, num_heads, block_table,
                                    table_stride, table_width, scale, out, lse);
  if (s != GVR_OK) return s;
  if (num_requests < 0 || num_requests > kIntMax || k < 1 || k > kIntMax) return GVR_ERR_ARG;
  if (num_rows == 0) return GVR_OK;
  if (!row_requests || !row_starts || !row_ends || !indices) return GVR_ERR_NULL;
  if (!aligned(row_requests, 4) || !aligned(row_starts, 4) || !aligned(row_ends, 4) || !aligned(indices, 4) || !aligned(workspace, 16)) return GVR_ERR_ALIGN;
  AttendParams p = {};
  p.q = q;
  p.table = block_table;
  p.requests = row_requests;
  p.starts = row_starts;
  p.ends = row_ends;
  p.indices = indices;
  p.out = out;
  p.lse = lse;
  p.next_n = 1;
  p.ratio = 1;
  p.num_requests = int32_t(num_requests);
  return attend(cache, p, q_row_stride, q_head_stride, dtype, num_rows, num_heads, table_stride, table_width, k, scale, workspace,
                workspace_bytes, stream);
}

}  // extern "C"
