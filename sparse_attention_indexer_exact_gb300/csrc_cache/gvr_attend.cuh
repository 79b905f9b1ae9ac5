// gvr_attend.cuh -- the kernels of attention over the 4-bit paged cache, at the selected entries or over
// all of a row's entries (attend_decode and attend_prefill of include/gvr_cache.h).
//
// Mathematics.  For a query vector q of one head and entries e with keys k_e and values v_e,
//   s_e = scale q.k_e,  o = sum_e exp(s_e - m) v_e / sum_e exp(s_e - m),  lse = m + log sum_e ...
// in one pass over the entries with a base m that follows their running maximum and running sums that
// are rescaled when m grows, in any grouping of the entries: groups join by the same rescaling.
//
// Work split.  A unit is a set of rows that read the same entries: one row, or (whole-cache decode)
// the next_n rows of a request.  Its queries fall into jobs of one KV head and 8 NT query vectors
// each.  A warp works on one job, alone: it fetches its own entries and keeps its own running state,
// without any CTA barrier.  A CTA holds the warps of several jobs, or SPLIT warps a job; a cluster of
// up to eight CTAs divide the entries further.  Warps join through shared memory, CTAs through distributed
// shared memory.  Or (given a workspace, for long units) CTAs take equal shares of all units' steps, and a
// second kernel joins the pieces.  Every sum has a fixed order.
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
// f16 cannot hold below that is under 2^-39 of it.  P is rounded to f16: eight times finer than bf16
// outputs, and averaged over the entries.  To use f16's range the base lies 2^7 below the maximum, when it
// is set: P is at most 2^7 then, and 2^15 before the base is set again.  So weights down to 2^-21 of the
// largest of their walk have 11 bits, and what lies below is off by at most 2^-32 of it (with the maximum as
// the base it was 2^-14 and 2^-25, and a long tail 18 nats below one entry was lost).
//
// What bounds it.  The work of a step, no one unit: at head_dim 128 and 8 queries it takes a warp 587
// instructions, of them 32 matrix instructions, 128 expansions and 128 scale products, and an SM partition about
// 1100 clocks, whether two warps share it or four, while the matrix, FMA and ALU pipes are busy 23, 31 and 44 %
// of them, 2.1 of 4 instructions are issued a clock and DRAM gives 55 %.  Of 69.4 us (2048 entries a row), leaving out
// the copies takes 10.7, V's scale products 6.3, V's interleaving 4.3, K's scale products 2.9, the exponentials 1.0.  The
// expansion costs the same for 1 to 8 queries, so more query heads a KV head cost little up to there.
// A scale product on the accumulators or on P instead would take fewer, but needs the 16 values of a scale
// in one tile row's lanes, which the cache's order of codes does not give.
// 128 rows x 1024 of up to 131072 entries, 8 KV heads of 128, 64 query heads: 42.8 us, 3.6 TB/s of rows read
// (147 MB; 22.9 us at the rate of a copy).  700 prefill rows x up to 2048 entries, 4 KV heads of 128, 32 query
// heads: 140 us.  One row x 512 entries: 6.8 us.
#pragma once

#include <type_traits>

#include "gvr_cache_common.cuh"
#include "../csrc/gvr_device.cuh"

namespace gvrc {

constexpr int STEP = 32;  // entries a warp takes at a time: one per lane
constexpr int STAGES = 3;
constexpr int MAX_CLUSTER = 8;
constexpr float NO_TOP = -3.4028235e38f;  // the base of no scores: finite, so that differences are
constexpr float BELOW = 7.f;              // of the base to the maximum that it is set from, in log2 units
constexpr float ABOVE = 15.f;             // of a score to the base, at most: P up to 2^15 is within f16
constexpr int JOIN_THREADS = 128;

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
  float* pieces;     // balanced: partial results, Q (D + 2) floats each
  int64_t q_row, q_head, table_stride, num_rows, k;
  uint32_t unit, page_units, entry_units, row_units;  // bytes of a unit; pages, entries and rows in units
  int32_t num_pages, page_shift, kv_heads, group, fold, capacity, next_n, ratio, num_requests, bf16;
  int32_t tiles;            // query tiles of a KV head in a unit
  int32_t heads_in, tiles_in, split, split_log2;  // a CTA's jobs: heads_in x tiles_in, SPLIT warps each
  int32_t head_groups, tile_groups;   // CTAs side by side for the jobs of a unit
  int32_t units, balanced_ctas, ways_log2;  // CTAs of balanced_kernel side by side, a group; lanes of join_kernel for the same values
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
  // accumulators and queries take 3 D / 8 NT registers: that leaves room for 16, 12 or 8 warps on an SM.  (At head_dim
  // 256 shared memory has room for fewer, 29,312 bytes each: 4, 6 or 7 in CTAs of four, two or one.)
  static constexpr int BLOCKS = D * NT <= 128 && NT == 1 ? 4 : D * NT == 128 ? 3 : 2, FOLD_BLOCKS = D * NT == 128 ? 3 : BLOCKS;
  // of balanced_kernel, in CTAs of at most four
  static constexpr int BALANCED_WARPS = D * NT >= 256 ? 8 : 12;
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
  // v_scale last: v_scale / sum would lose bits, or all, of a small factor over many entries
  const float norm = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t packed[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float lo = acc[2 * j] * norm * p.v_scale, hi = acc[2 * j + 1] * norm * p.v_scale;
    if (p.bf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(packed[j]) : "f"(hi), "f"(lo));
    else packed[j] = pack_f16(lo, hi);
  }
  const int64_t at = row * (int64_t(p.kv_heads) * p.group) + head;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at * D + d) = make_uint4(packed[0], packed[1], packed[2], packed[3]);
  if (p.lse && d == 0) p.lse[at] = sum == 0.f ? -INFINITY : (all + log2f(sum)) * 0.69314718055994531f;
}

// The queries of a job, on their way: lane (g, c) holds query 8 t + g at D/4 c + [0, D/4).
// FOLD: the unit is the next_n rows of a request (whole-cache decode with next_n > 1).
template <int D, int NT, bool FOLD>
__device__ __forceinline__ void load_queries(const AttendParams& p, int unit, int h, int m0, int members, uint32_t (&raw)[NT][D / 8]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int m = m0 + 8 * t + g;
    const int64_t row = FOLD ? int64_t(unit) * p.fold + m / p.group : unit;
    const bool live = m < members && row < p.num_rows;
    const uint16_t* src = static_cast<const uint16_t*>(p.q) + row * p.q_row + int64_t(h * p.group + (FOLD ? m % p.group : m)) * p.q_head + c * (D / 4);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 v = live ? reinterpret_cast<const uint4*>(src)[i] : make_uint4(0, 0, 0, 0);
      raw[t][4 * i] = v.x, raw[t][4 * i + 1] = v.y, raw[t][4 * i + 2] = v.z, raw[t][4 * i + 3] = v.w;
    }
  }
}

// A unit's entries.
struct Unit {
  const int32_t* table;
  const int32_t* indices;  // nullptr: all entries
  int n;                   // entries that some row of the unit sees
  int kv;                  // kv_lens of a decode unit
  uint32_t listed;         // positions to walk over: k or n
};

template <bool FOLD>
__device__ __forceinline__ Unit load_unit(const AttendParams& p, int unit) {
  Unit u;
  int64_t request;
  u.n = u.kv = 0;
  if (p.requests) {
    request = p.requests[unit];
    if (request >= 0 && request < p.num_requests) {
      u.n = window_entries(p.starts[unit], p.ends[unit], p.capacity);
    } else {
      request = 0;
    }
  } else {
    request = FOLD || p.next_n == 1 ? unit : unit / p.next_n;
    u.kv = p.lens[request];
    u.n = decode_entries(u.kv, p.next_n, FOLD ? p.next_n - 1 : unit - int(request) * p.next_n, p.ratio, p.capacity);
  }
  u.table = p.table + request * p.table_stride;
  u.indices = p.indices ? p.indices + int64_t(unit) * p.k : nullptr;
  u.listed = u.indices ? (u.n > 0 ? uint32_t(p.k) : 0) : uint32_t(u.n);
  return u;
}

__device__ __forceinline__ int steps_of(uint32_t listed) { return int((listed + (STEP - 1)) / STEP); }

// A warp's walk over `mine` steps of a unit's entries, from step `first` on, every `every`-th; positions
// from `end` on are not looked at.  Leaves sums of exp2(score - top) v, the tops (bases) and the sums of exp2.
template <int D, int NT, bool FOLD>
__device__ __forceinline__ void walk(const AttendParams& p, const Unit& u, int h, int m0, int first_step, int every, int mine,
                                     uint32_t end, uint8_t* ring, uint32_t* places, const uint32_t (&raw)[NT][D / 8],
                                     float (&o)[NT][D / 16][4], float (&top)[NT][2], float (&total)[NT][2]) {
  using S = Shape<D, NT>;
  constexpr int KSTEPS = D / 16;       // 16-wide steps of the head dimension
  constexpr int KW = D / 32;           // 32-bit words of K codes per lane and entry
  constexpr int VW = D / 64;           // the same of V codes
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, n = u.n, kv = u.kv;
  const int32_t *table = u.table, *indices = u.indices;

  // ---- fetching
  constexpr int CODES = D / 16, SCALES = S::RB / 16 - CODES;  // 16-byte pieces of a row: of codes, of scales
  const uint32_t stride = every * STEP;
  uint32_t pos = first_step * STEP + lane;  // of the entry that this lane loads next; below 2^32 even behind the last
  auto load_entry = [&]() -> int {  // -1: none
    int e = -1;
    if (pos < end) e = indices ? indices[pos] : int(pos);
    pos += stride;
    return e;
  };
  auto load_page = [&](int e) -> int { return uint32_t(e) < uint32_t(n) ? table[e >> p.page_shift] : -1; };
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

  // ---- the walk
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
      const int64_t first = int64_t(first_step + i * every) * STEP;
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

      // The base that scores are taken against: 2^7 below the maximum when it was last set, kept while no
      // score is more than 2^15 above it.
      bool grow = false;
      float high[NT][2];  // of this lane's scores, in log2 units; factors are positive
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          high[t][j] = fmaxf(fmaxf(s[0][t][j], s[0][t][j + 2]), fmaxf(s[1][t][j], s[1][t][j + 2])) * factor[t][j];
          grow |= high[t][j] > top[t][j] + ABOVE;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float down[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float next = fmaxf(top[t][j], high[t][j] - BELOW);
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
      // differs from row to row, so rows that see equally many entries, `only`, take a pass with their own
      // entries, which leaves the other rows' sums (a NaN that they do not see reaches them too) as they were.
      auto add_values = [&](uint32_t there, auto bordering, int only) {
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
              for (int t = 0; t < NT; ++t) {
                float(&sum)[4] = o[t][4 * w + b];
                if (!decltype(bordering)::value) {
                  mma(sum, a0, a1, a2, a3, pb[mt][t][0], pb[mt][t][1]);
                } else {
                  float with[4] = {sum[0], sum[1], sum[2], sum[3]};
                  mma(with, a0, a1, a2, a3, pb[mt][t][0], pb[mt][t][1]);
#pragma unroll
                  for (int j = 0; j < 4; ++j) sum[j] = limit[t][j & 1] == only ? with[j] : sum[j];
                }
              }
            }
          }
        }
      };
      if (!border) {
        add_values(mask, std::false_type(), 0);
      } else {
        int before = -1;
        for (int j = first_row; j <= last_row; ++j) {
          const int limit_j = decode_entries(kv, p.next_n, j, p.ratio, p.capacity);
          if (limit_j == before) continue;
          before = limit_j;
          const int64_t seen = limit_j - first;
          add_values(mask & (seen <= 0 ? 0u : seen >= 32 ? 0xffffffffu : (1u << int(seen)) - 1), std::true_type(), limit_j);
        }
      }
    }
  }
  copy_wait<0>();
  __syncwarp();  // every copy has landed, every stage is read

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
}

template <int D, int NT, bool FOLD>
__global__ void __launch_bounds__(Shape<D, NT>::THREADS, FOLD ? Shape<D, NT>::FOLD_BLOCKS : Shape<D, NT>::BLOCKS) attend_kernel(AttendParams p) {
  using S = Shape<D, NT>;
  constexpr int KSTEPS = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];

  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same in every lane, and known to be
  const int warps = blockDim.x >> 5;
  const uint32_t rank = gvr::cluster_rank(), cs = gvr::cluster_size();
  const int unit = int(cs == 1 ? blockIdx.x : gvr::cluster_id_x());
  const int tile_group = p.head_groups == 1 ? blockIdx.y : blockIdx.y / p.head_groups;
  const int head0 = (int(blockIdx.y) - tile_group * p.head_groups) * p.heads_in, tile0 = tile_group * p.tiles_in;
  const int job = warp >> p.split_log2, sub = warp & (p.split - 1);
  const int tile_in = p.tiles_in == 1 ? 0 : job / p.heads_in;
  const int h = head0 + job - tile_in * p.heads_in, tile = tile0 + tile_in;

  begin();
  const int m0 = tile * S::Q;
  const int members = tile < p.tiles ? (FOLD ? p.fold * p.group : p.group) : 0;
  uint32_t raw[NT][D / 8];
  load_queries<D, NT, FOLD>(p, unit, h, m0, members, raw);
  const Unit u = load_unit<FOLD>(p, unit);
  const int steps = steps_of(u.listed), walkers = int(cs) * p.split, me = int(rank) * p.split + sub;
  const int mine = walkers == 1 ? steps : steps > me ? (steps - me + walkers - 1) / walkers : 0;
  float o[NT][KSTEPS][4], top[NT][2], total[NT][2];
  // (listed entries are loaded whatever the row's length, which may still be on its way)
  walk<D, NT, FOLD>(p, u, h, m0, me, walkers, mine, u.indices ? uint32_t(p.k) : uint32_t(u.n), smem + warp * S::RING,
                    reinterpret_cast<uint32_t*>(smem + warps * S::RING) + warp * STEP, raw, o, top, total);
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

  // ---- join the warps of a job, then the CTAs; the rings become the partial results
  __syncthreads();
  float* partial = reinterpret_cast<float*>(smem);   // [warps][Q][D]
  float* tops = partial + warps * S::Q * D;          // [warps][Q]
  float* sums = tops + warps * S::Q;                 // [warps][Q]
  float* joined = sums + warps * S::Q;               // [jobs][2][Q]: base and sum of a job in this CTA
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
    write_out<D>(p, row, hj * p.group + (FOLD ? m % p.group : m), d, all, sum, acc);
  }
  if (cs > 1) gvr::cluster_sync();  // no CTA leaves while another reads its shared memory
}

// Units of unequal lengths in equal shares: the steps of all units, one behind the other, are cut into as
// many equal ranges as there are CTAs (of a group of heads and a query tile, blockIdx.y).  A CTA walks over
// its range, unit by unit, and writes a piece for each: piece c + u of CTA c and unit u, which is unique, as
// both only grow along the steps.  A warp has a head: CTAs of four neighbouring heads, whose rows lie next
// to each other, took 46.2 us where CTAs of two took 53.3 (48 requests of 1 to 16384 entries, 4 KV heads of
// 64) and clusters, one a unit, 73.5; 131071 entries of one request, 8 KV heads of 128: 40.5, 42.7 and 46.9.  The join starts while
// the last pieces are written: 0.3 to 0.5 us (from the start of this kernel on its CTAs would lie unevenly: up to 2 more).
__device__ __forceinline__ int range_start(int c, int ctas, int steps) { return int(int64_t(c) * steps / ctas); }

template <int D, int NT, bool FOLD>
__global__ void __launch_bounds__(128, Shape<D, NT>::BALANCED_WARPS / 4) balanced_kernel(AttendParams p) {
  using S = Shape<D, NT>;
  constexpr int KSTEPS = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0), warps = blockDim.x >> 5;
  int* start = reinterpret_cast<int*>(smem + warps * S::WARP_SMEM);  // [units + 1]: the steps before each unit
  const int tile = blockIdx.y / p.head_groups, h = (int(blockIdx.y) - tile * p.head_groups) * p.heads_in + warp;

  begin();
  for (int i = tid; i < p.units; i += blockDim.x) start[i + 1] = steps_of(load_unit<FOLD>(p, i).listed);
  __syncthreads();
  if (warp == 0) {
    int before = 0;
    for (int i = lane; i - lane < p.units; i += 32) {
      int x = i < p.units ? start[i + 1] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      if (i < p.units) start[i + 1] = before + x;
      before += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) start[0] = 0;
  }
  __syncthreads();
  const int steps = start[p.units], ctas = min(int(gridDim.x), steps);
  if (int(blockIdx.x) >= ctas) return;
  int at = range_start(blockIdx.x, ctas, steps);
  const int last = range_start(blockIdx.x + 1, ctas, steps);
  int unit = 0;
  for (int hi = p.units; hi - unit > 1;) {  // the last unit that starts at or before `at`
    const int mid = (unit + hi) >> 1;
    if (start[mid] <= at) unit = mid; else hi = mid;
  }
  const int m0 = tile * S::Q, members = FOLD ? p.fold * p.group : p.group;
  float* pieces = p.pieces + int64_t(blockIdx.y * p.heads_in + warp) * (gridDim.x + p.units) * (S::Q * (D + 2));
  while (at < last) {
    const int mine = min(last, start[unit + 1]) - at, first = at - start[unit];
    if (mine > 0) {
      uint32_t raw[NT][D / 8];
      load_queries<D, NT, FOLD>(p, unit, h, m0, members, raw);
      const Unit u = load_unit<FOLD>(p, unit);
      float o[NT][KSTEPS][4], top[NT][2], total[NT][2];
      walk<D, NT, FOLD>(p, u, h, m0, first, 1, mine, min(u.listed, uint32_t(first + mine) * STEP), smem + warp * S::RING,
                        reinterpret_cast<uint32_t*>(smem + warps * S::RING) + warp * STEP, raw, o, top, total);
      if (at + mine == last) let_next_start();  // all that is left is this piece
      float* piece = pieces + int64_t(int(blockIdx.x) + unit) * (S::Q * (D + 2));
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int qi = 8 * t + 2 * c + j;
#pragma unroll
          for (int x = 0; x < KSTEPS; x += 2)
            *reinterpret_cast<float4*>(piece + qi * D + g * (D / 8) + 2 * x) =
                make_float4(o[t][x][j], o[t][x][j + 2], o[t][x + 1][j], o[t][x + 1][j + 2]);
          if (g == 0) piece[S::Q * D + qi] = top[t][j], piece[S::Q * (D + 1) + qi] = total[t][j];
        }
      at += mine;
    }
    ++unit;
  }
}

// Joins the pieces of a unit, KV head and query tile (blockIdx.x and y): eight values a thread; 2^ways_log2
// lanes next to each other take every 2^ways_log2-th piece of the same values, in order, and join by shuffles.
// Bound by latency (5 us behind balanced_kernel for 228 pieces of each of 8 heads of 128, 7.6 MB): 8 threads
// a value and CTAs of 512 threads, one a head, took 25 us there, as each thread went through 29 pieces.
template <int D, int NT, bool FOLD>
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(AttendParams p) {
  using S = Shape<D, NT>;
  constexpr int EIGHTS = D / 8, PIECE = S::Q * (D + 2), WARPS = JOIN_THREADS / 32;
  __shared__ int sums[2][WARPS];
  const int unit = blockIdx.x, tid = threadIdx.x;
  const int tile = blockIdx.y / p.kv_heads, h = int(blockIdx.y) - tile * p.kv_heads;
  int before = 0, steps = 0;  // of the units before this one, of all
  for (int i = tid; i < p.units; i += JOIN_THREADS) {
    const int x = steps_of(load_unit<FOLD>(p, i).listed);
    steps += x;
    if (i < unit) before += x;
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, d);
    steps += __shfl_xor_sync(0xffffffffu, steps, d);
  }
  if ((tid & 31) == 0) sums[0][tid >> 5] = before, sums[1][tid >> 5] = steps;
  __syncthreads();
  before = steps = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) before += sums[0][w], steps += sums[1][w];
  const int own = steps_of(load_unit<FOLD>(p, unit).listed), ctas = min(p.balanced_ctas, steps);
  // the last CTA whose range starts at or before step s is ((s + 1) ctas - 1) / steps
  const int first = own ? int((int64_t(before + 1) * ctas - 1) / steps) : 0;
  const int count = own ? int((int64_t(before + own) * ctas - 1) / steps) - first + 1 : 0;
  const int i = (int(blockIdx.z) * JOIN_THREADS + tid) >> p.ways_log2, ways = 1 << p.ways_log2, way = tid & (ways - 1);
  const int qi = i / EIGHTS, d = (i % EIGHTS) * 8;
  const bool is = qi < S::Q;
  const int group = tile * p.head_groups + h / p.heads_in;
  const float* src = p.pieces + (int64_t(group * p.heads_in + h % p.heads_in) * (p.balanced_ctas + p.units) + first + unit) * PIECE;
  begin();  // so far only what balanced_kernel has found written, too
  float all = NO_TOP, sum = 0.f, acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
#pragma unroll 4
  for (int r = is ? way : count; r < count; r += ways) {
    const float* from = src + int64_t(r) * PIECE;
    const float tr = from[S::Q * D + qi], sr = from[S::Q * (D + 1) + qi];
    const float4 a = *reinterpret_cast<const float4*>(from + qi * D + d), b = *reinterpret_cast<const float4*>(from + qi * D + d + 4);
    const float next = fmaxf(all, tr), down = exp2_fast(all - next), up = exp2_fast(tr - next);
    all = next, sum = sum * down + sr * up;
    acc[0] = acc[0] * down + a.x * up, acc[1] = acc[1] * down + a.y * up, acc[2] = acc[2] * down + a.z * up;
    acc[3] = acc[3] * down + a.w * up, acc[4] = acc[4] * down + b.x * up, acc[5] = acc[5] * down + b.y * up;
    acc[6] = acc[6] * down + b.z * up, acc[7] = acc[7] * down + b.w * up;
  }
  for (int x = 1; x < ways; x <<= 1) {
    const float other = __shfl_xor_sync(0xffffffffu, all, x), next = fmaxf(all, other);
    const float scale = exp2_fast(all - next);  // of both sides the same base: every lane ends with the same sums
    all = next, sum *= scale;
    sum += __shfl_xor_sync(0xffffffffu, sum, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      acc[j] *= scale;
      acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], x);
    }
  }
  const int m = tile * S::Q + qi;
  const int64_t row = FOLD ? int64_t(unit) * p.fold + m / p.group : unit;
  if (is && way == 0 && m < p.fold * p.group && row < p.num_rows)
    write_out<D>(p, row, h * p.group + (FOLD ? m % p.group : m), d, all, sum, acc);
}

// What the host needs to know of a kernel.
struct KernelInfo {
  const void* kernel[2];    // by FOLD
  const void* balanced[2];
  const void* join[2];
  int queries;
  int piece_bytes;  // partial results of one job
  int warp_smem;    // shared memory of a warp
  int balanced_warps;
};

template <int D, int NT>
KernelInfo info() {
  using S = Shape<D, NT>;
  return {{reinterpret_cast<const void*>(attend_kernel<D, NT, false>), reinterpret_cast<const void*>(attend_kernel<D, NT, true>)},
          {reinterpret_cast<const void*>(balanced_kernel<D, NT, false>), reinterpret_cast<const void*>(balanced_kernel<D, NT, true>)},
          {reinterpret_cast<const void*>(join_kernel<D, NT, false>), reinterpret_cast<const void*>(join_kernel<D, NT, true>)},
          S::Q, S::Q * (D + 2) * int(sizeof(float)), S::WARP_SMEM, S::BALANCED_WARPS};
}

// One translation unit per head_dim.
constexpr int KERNELS = 6;  // head_dim 64: 8, 16, 32 queries a job; 128: 8, 16; 256: 8
KernelInfo attend_64(int i);
KernelInfo attend_128(int i);
KernelInfo attend_256();

}  // namespace gvrc
