// gvr_shared.cuh -- the kernels of attention whose requests share prefixes (attend_shared of include/gvr_long.h).
//
// Mathematics.  As in gvr_attend.cuh: one pass over the entries, with a base that follows each query's running maximum
// and sums that are rescaled when it grows; partial results of disjoint entries join by the same rescaling.  A query of
// request r in group g is the join of entries [0, P_g), which all of the group's queries see, and [P_g, n_r).
//
// Work split.  A set is a group's prefix or a request's remaining entries: queries that read the same entries.  Per KV
// head it has units of 256 queries (head_dim 256: 128).  The steps of N entries of all units, one behind the other, are cut
// into equal ranges, one a CTA of an SM.  A CTA walks over its range, unit by unit, and leaves a piece for each: sums over
// exp2(score - base) v, base and sum.  A last kernel joins the pieces of every query.  Every sum has a fixed order.
//
// A CTA.  Four warps bring K and four bring V: rows of codes and scales arrive by asynchronous copies, are expanded
// (e2m1 times e4m3 is exact in f16) and laid into shared memory as matrix operands.  One thread issues the products
// S = Q K^T and O += P V on the fifth-generation tensor cores, 128 queries a tile: S and O lie in tensor memory.  Four warps a
// tile take S, a query a thread, so that maximum, base and sum need no exchange, and write P, in f16, over it; P is read
// from there as an operand.  Two tiles take turns: while one's P is made, the other's products run.  Where a unit
// has up to 128 queries both tiles hold them, one taking the even steps, one the odd ones.
#pragma once

#include "../csrc_cache/gvr_attend.cuh"
#include "gvr_long_common.h"
#include "gvr_tcgen05.cuh"

namespace gvrc {

// Queries that read the same entries: rows row0 .. of a group, or of a request.
struct Set {
  int32_t start;    // work before it, in tile steps
  int32_t steps;    // of N entries, of each unit
  int32_t units;    // KV heads x query tiles
  int32_t both;     // each step is taken by both tiles (more than 128 queries)
  int32_t first;    // entries [first, end)
  int32_t end;
  int32_t request;  // whose block table
  int32_t row0;
  int32_t queries;  // of a KV head: rows x group
  int32_t unit0;    // units before it of its kind
  int32_t kv;       // kv_lens of a request; -1: a prefix
  int32_t pad;
};

struct Plan {
  int32_t total;   // work in all sets
  int32_t ctas;    // that take shares of it
  int32_t sets;    // sets that have work, in order
  int32_t failed;  // a wait gave up
};

// What a request's rows join.
struct Joined {
  int32_t suffix;  // its set, -1: none
  int32_t prefix;  // its group's, -1: none
};

struct SharedParams {
  const uint8_t* data;
  const uint16_t* q;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* group_starts;
  const int32_t* prefix_entries;
  void* out;
  float* lse;
  Plan* plan;
  Set* sets;          // [groups + requests]
  Joined* joined;     // [requests]
  int32_t* cta_set;   // [grid]: the set in which a CTA's share begins
  float* prefix_pieces;
  float* suffix_pieces;
  int64_t q_row, q_head, table_stride, num_rows;
  uint32_t unit, page_units, entry_units, row_units;  // as in AttendParams
  int32_t num_pages, page_shift, kv_heads, group, capacity, next_n, ratio, bf16, requests, groups, grid;
  int32_t suffix_rows;  // rows of a tile in a suffix piece (a multiple of 8)
  float scale_log2, q_sign, v_scale;
};

template <int D>
struct SharedShape {
  static constexpr int N = D == 256 ? 64 : 128;      // entries a step
  static constexpr int TILES = D == 256 ? 1 : 2;     // O takes D columns of tensor memory a tile, S two times N
  static constexpr int KBUF = 2, VBUF = D == 64 ? 2 : 1;
  static constexpr int STAGES = 3;                   // of raw rows
  static constexpr int QUERIES = 128 * TILES;        // of a unit
  static constexpr int ROWS = N / 4;                 // rows a warp brings in a step
  static constexpr int PITCH = (D / 2 + D / 16 + 15) / 16 * 16 | 16;  // of a raw row: codes and scales of K or V
  static constexpr int RING = STAGES * ROWS * PITCH;  // of a warp
  static constexpr int Q_BYTES = 128 * D * 2, KV_BYTES = N * D * 2;
  static constexpr int WARPS = 4 * TILES + 9, THREADS = 32 * WARPS;
  static constexpr int PIECE = QUERIES * (D + 2);    // floats of a prefix piece
  static constexpr int S_AT = 0, O_AT = 2 * N;       // columns
  static constexpr int NAN_SLOTS = 4;
  static constexpr int SMEM = TILES * Q_BYTES + (KBUF + VBUF) * KV_BYTES + 8 * RING + 1024;  // 1024 to align
};

// ------------------------------------------------------------------------------------------------ the plan
constexpr int PLAN_THREADS = 1024;
constexpr int LEAST_WORK = 2;  // tile steps worth a CTA

struct Sum2 {
  int work, units;
};

// Inclusive sums over the CTA; `sums` is shared, [32].
__device__ __forceinline__ Sum2 plan_scan(int work, int flag, int units, int2* sums, int* flags, int& flag_sum, int2& total, int& flag_total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, work, d), b = __shfl_up_sync(0xffffffffu, flag, d), c = __shfl_up_sync(0xffffffffu, units, d);
    if (lane >= d) work += a, flag += b, units += c;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = make_int2(work, units), flags[warp] = flag;
  __syncthreads();
  int2 s = sums[lane];
  int f = flags[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, s.x, d), b = __shfl_up_sync(0xffffffffu, f, d), c = __shfl_up_sync(0xffffffffu, s.y, d);
    if (lane >= d) s.x += a, f += b, s.y += c;
  }
  total = make_int2(__shfl_sync(0xffffffffu, s.x, 31), __shfl_sync(0xffffffffu, s.y, 31));
  flag_total = __shfl_sync(0xffffffffu, f, 31);
  const int bw = __shfl_sync(0xffffffffu, s.x, max(warp - 1, 0)), bf = __shfl_sync(0xffffffffu, f, max(warp - 1, 0)),
            bu = __shfl_sync(0xffffffffu, s.y, max(warp - 1, 0));
  flag_sum = flag + (warp ? bf : 0);
  return {work + (warp ? bw : 0), units + (warp ? bu : 0)};
}

// One CTA: groups, what their requests share, the sets that have work, and where each CTA's share begins.
template <int D>
__global__ void __launch_bounds__(PLAN_THREADS, 1) shared_plan_kernel(SharedParams p) {
  using S = SharedShape<D>;
  extern __shared__ __align__(16) int plan_smem[];
  int* from = plan_smem;              // [groups + 1]: first request of each group, non-decreasing
  int* sharing = from + p.groups + 1;  // [groups]: requests that share the prefix; later the group's set
  int* lead = sharing + p.groups;     // [groups]: the first of them
  int* starts = lead + p.groups;      // [groups + requests]: of the sets that have work
  __shared__ int2 sums[32];
  __shared__ int flags[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  begin();
  // groups begin where their start says, but not before the one before them
  int most = 0;
  for (int i0 = 0; i0 <= p.groups && p.groups > 0; i0 += PLAN_THREADS) {
    const int i = i0 + tid;
    int x = i <= p.groups ? min(max(p.group_starts[i], 0), p.requests) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x = max(x, y);
    }
    __syncthreads();
    if (lane == 31) flags[warp] = x;
    __syncthreads();
    for (int w = 0; w < warp; ++w) x = max(x, flags[w]);
    x = max(x, most);
    for (int w = 0; w < 32; ++w) most = max(most, flags[w]);
    if (i <= p.groups) from[i] = x;
    if (i < p.groups) sharing[i] = 0, lead[i] = p.requests;
  }
  __syncthreads();
  auto prefix_of = [&](int g) { return min(max(p.prefix_entries[g], 0), p.capacity); };
  // the group whose prefix all rows of request r see, -1: none
  auto group_of = [&](int r, int kv) {
    if (p.groups == 0 || r < from[0] || r >= from[p.groups]) return -1;
    int lo = 0;
    for (int hi = p.groups; hi - lo > 1;) {
      const int mid = (lo + hi) >> 1;
      if (from[mid] <= r) lo = mid; else hi = mid;
    }
    const int prefix = prefix_of(lo);
    return prefix > 0 && decode_entries(kv, p.next_n, 0, p.ratio, p.capacity) >= prefix ? lo : -1;
  };
  for (int r = tid; r < p.requests; r += PLAN_THREADS) {
    const int g = group_of(r, p.lens[r]);
    if (g >= 0) atomicAdd(&sharing[g], 1), atomicMin(&lead[g], r);
  }
  __syncthreads();

  int2 before = make_int2(0, 0);
  int sets = 0;
  // `set` with all but its sums: takes its place if it has work; returns the place or -1
  auto place = [&](bool is, Set set) -> int {
    const int tiles = (set.queries + S::QUERIES - 1) / S::QUERIES;
    set.both = S::TILES == 2 && set.queries > 128;
    set.units = is ? p.kv_heads * tiles : 0;
    set.steps = is && set.end > set.first ? (set.end - set.first + S::N - 1) / S::N : 0;
    const int work = set.units * set.steps * (1 + set.both);
    int at, flag_total;
    int2 total;
    const Sum2 x = plan_scan(work, work > 0, set.units, sums, flags, at, total, flag_total);
    at += sets - 1;
    set.start = before.x + x.work - work;
    if (set.kv < 0) set.unit0 = before.y + x.units - set.units;
    before.x += total.x, before.y += total.y, sets += flag_total;
    if (work == 0) return -1;
    p.sets[at] = set;
    starts[at] = set.start;
    return at;
  };
  for (int g0 = 0; g0 < p.groups; g0 += PLAN_THREADS) {
    const int g = g0 + tid;
    Set set = {};
    const bool is = g < p.groups && sharing[g] >= 2;
    set.kv = -1;
    if (is) {
      set.end = prefix_of(g);
      set.request = lead[g];
      set.row0 = from[g] * p.next_n;
      set.queries = int(min(int64_t(from[g + 1]) * p.next_n, p.num_rows) - set.row0) * p.group;
    }
    const int at = place(is, set);
    if (g < p.groups) sharing[g] = at;
  }
  __syncthreads();
  for (int r0 = 0; r0 < p.requests; r0 += PLAN_THREADS) {
    const int r = r0 + tid;
    Set set = {};
    Joined join = {-1, -1};
    if (r < p.requests) {
      set.kv = max(p.lens[r], 0);
      const int g = group_of(r, p.lens[r]);
      join.prefix = g < 0 ? -1 : sharing[g];
      set.first = join.prefix < 0 ? 0 : prefix_of(g);
      set.end = decode_entries(p.lens[r], p.next_n, p.next_n - 1, p.ratio, p.capacity);
      set.request = r;
      set.row0 = r * p.next_n;
      set.queries = int(min(int64_t(p.next_n), p.num_rows - set.row0)) * p.group;
      set.unit0 = r * (p.kv_heads * ((p.next_n * p.group + S::QUERIES - 1) / S::QUERIES));
    }
    join.suffix = place(r < p.requests, set);
    if (r < p.requests) p.joined[r] = join;
  }
  __syncthreads();
  const int total = before.x, ctas = max(1, min(p.grid, total / LEAST_WORK));
  if (tid == 0) *p.plan = {total, ctas, sets, 0};
  for (int c = tid; c < ctas; c += PLAN_THREADS) {
    const int at = range_start(c, ctas, total);
    int lo = 0;
    for (int hi = sets; hi - lo > 1;) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= at) lo = mid; else hi = mid;
    }
    p.cta_set[c] = lo;
  }
}

// ------------------------------------------------------------------------------------------------ the walk
// A CTA's part of a unit: steps [lo, hi).
struct Segment {
  Set set;
  int unit, lo, hi;
  int head, tile;  // KV head, and number of the unit among the set's query tiles
};

// The steps of [from, to) of the work of a unit that begins at `start`: a step of work 2 belongs to where its first half lies.
__device__ __forceinline__ int step_of(int at, int start, int both, int steps) {
  const int x = max(at - start, 0);
  return min(both ? (x + 1) >> 1 : x, steps);
}

struct Walker {
  const Set* sets;
  int at, last, next_set, count;
  Set set;

  __device__ __forceinline__ Walker(const SharedParams& p, const Plan& plan) {
    const int c = blockIdx.x;
    sets = p.sets;
    count = plan.sets;
    at = last = 0;
    if (c < plan.ctas && plan.total > 0) {
      at = range_start(c, plan.ctas, plan.total);
      last = range_start(c + 1, plan.ctas, plan.total);
      next_set = p.cta_set[c];
      load();
    }
  }
  __device__ __forceinline__ void load() {
    const int4* from = reinterpret_cast<const int4*>(sets + next_set);
    const int4 a = from[0], b = from[1], c = from[2];
    set = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
    ++next_set;
  }
  __device__ __forceinline__ bool next(Segment& s, int kv_heads) {
    while (at < last) {
      const int work = set.steps << set.both, unit = (at - set.start) / work, start = set.start + unit * work;
      const int to = min(last, start + work);
      s.lo = step_of(at, start, set.both, set.steps), s.hi = step_of(to, start, set.both, set.steps);
      s.set = set;
      s.unit = unit;
      s.tile = unit / kv_heads;
      s.head = unit - s.tile * kv_heads;
      at = to;
      if (at < last && unit + 1 == set.units && to == start + work && next_set < count) load();
      if (s.hi > s.lo) return true;
    }
    return false;
  }
};

// The next bit of a counter of uses of a barrier with `N` phases in turn.
struct Turn {
  uint32_t used = 0;
  __device__ __forceinline__ int slot(int n) const { return n == 1 ? 0 : int(used) & (n - 1); }
  __device__ __forceinline__ uint32_t parity(int n) const { return (n == 1 ? used : used >> 1) & 1; }  // n is 1 or 2
};

constexpr uint64_t GIVE_UP_NS = 500000000;

struct SharedBars {
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2], q_full[2], s_full[2], p_full[2], o_full[2], done;
};

// The next step's rows of K or V, by one warp: fetched STAGES - 1 steps ahead, expanded into the operand tile.
template <int D, bool V>
__device__ __forceinline__ bool bring(const SharedParams& p, const Plan& plan, SharedBars* bars, uint8_t* ring, uint32_t tiles, int w, uint32_t* masks, uint32_t* nans) {
  using S = SharedShape<D>;
  constexpr int R = S::ROWS, LANES = 32 / R;       // lanes that expand a row
  constexpr int CODES = D / 32;                    // 16-byte pieces of a row's codes
  constexpr int BUF = V ? S::VBUF : S::KBUF;
  constexpr int SCALES = D / 16;
  const int lane = threadIdx.x & 31, row = lane % R;  // whose address this lane finds
  const uint32_t ring_at = gvr::smem_u32(ring);
  // ---- fetching
  Walker ahead(p, plan);
  Segment f;
  bool more = ahead.next(f, p.kv_heads);
  int step = more ? f.lo : 0;
  const int32_t* table = p.table + (more ? f.set.request : 0) * p.table_stride;
  auto entry = [&]() { return f.set.first + step * S::N + w * R + row; };
  auto load_page = [&]() { const int e = entry(); return more && e < f.set.end ? table[e >> p.page_shift] : -1; };
  int page = load_page();
  uint32_t there_of[S::STAGES] = {};
  auto fetch = [&](int stage) -> uint32_t {
    uint32_t there = 0;
    if (more) {
      const bool is = uint32_t(page) < uint32_t(p.num_pages);
      there = __ballot_sync(0xffffffffu, is);
      uint32_t from = is ? row_unit(page, entry(), p.page_shift, p.page_units, p.entry_units, uint32_t(f.head) * p.row_units) : 0;
      if (there) {  // a missing entry is fetched from where another lies, and left out
        const uint32_t some = __shfl_sync(0xffffffffu, from, __ffs(there) - 1);
        if (!is) from = some;
        const uint32_t to = ring_at + stage * (R * S::PITCH);
#pragma unroll
        for (int j = 0; j < R * CODES / 32; ++j) {
          const int r = j * (32 / CODES) + lane / CODES;
          const uint32_t of = __shfl_sync(0xffffffffu, from, r);
          copy16(to + r * S::PITCH + lane % CODES * 16, p.data + uint64_t(of) * p.unit + (V ? D / 2 : 0) + lane % CODES * 16);
        }
        if (lane < R) {
          const uint8_t* scales = p.data + uint64_t(from) * p.unit + D + (V ? SCALES : 0);
          const uint32_t scales_to = to + lane * S::PITCH + D / 2;
          if (SCALES == 16) copy16(scales_to, scales);
          else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(scales_to), "l"(scales), "n"(SCALES == 8 ? 8 : 4) : "memory");
        }
      }
      if (++step == f.hi) {
        more = ahead.next(f, p.kv_heads);
        if (more) step = f.lo, table = p.table + f.set.request * p.table_stride;
      }
      page = load_page();
    }
    copy_commit();
    return there;
  };
#pragma unroll
  for (int i = 0; i < S::STAGES - 1; ++i) there_of[i] = fetch(i);

  // ---- expanding
  Walker walk(p, plan);
  Segment s;
  Turn turn;
  int stage = 0;
  uint32_t count = 0;  // steps so far
  uint32_t segments[2] = {0, 0};  // so far with work for each tile
  const int r_own = R == 32 ? lane : lane / LANES, part = R == 32 ? 0 : lane % LANES;  // its row, and which part of it
  const int tile_row = w * R + r_own;
  bool ok = true;
  while (ok && walk.next(s, p.kv_heads)) {
    const bool one = s.hi - s.lo == 1 && !s.set.both;  // only one tile has work, the first
    const int sure = s.set.kv < 0 ? s.set.end : decode_entries(s.set.kv, p.next_n, 0, p.ratio, p.capacity);
    for (int i = s.lo; i < s.hi; ++i, ++count) {
      copy_wait<S::STAGES - 2>();
      __syncwarp();
      there_of[S::STAGES - 1] = fetch(stage == 0 ? S::STAGES - 1 : stage - 1);
      const uint32_t there = there_of[0];
#pragma unroll
      for (int j = 0; j < S::STAGES - 1; ++j) there_of[j] = there_of[j + 1];
      const uint8_t* raw = ring + stage * (R * S::PITCH) + r_own * S::PITCH;
      stage = stage == S::STAGES - 1 ? 0 : stage + 1;
      const int slot = turn.slot(BUF);
      ok = gvr::mbar_wait_bounded(V ? &bars->v_free[slot] : &bars->k_free[slot], turn.parity(BUF) ^ 1, GIVE_UP_NS);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const bool is = there >> r_own & 1;
      constexpr int VALUES = D / LANES;  // of this lane
      uint32_t scales[VALUES / 64 > 0 ? VALUES / 64 : 1];  // four a word
      load_words<VALUES / 64>(raw + D / 2 + part * (VALUES / 16), scales);
      if (V) {
        const int e = s.set.first + i * S::N + tile_row;
        if (!is) {  // P is 0 there, and 0 x NaN is not
#pragma unroll
          for (int j = 0; j < VALUES / 64; ++j) scales[j] = 0;
        } else if (s.set.first + i * S::N + S::N > sure && e >= sure) {
          // A NaN that only some rows see: it is taken out of V, and put into those rows' results (by the block of 16 values)
          uint32_t blocks = 0;
#pragma unroll
          for (int j = 0; j < VALUES / 16; ++j) {
            const uint32_t b = scales[j / 4] >> (8 * (j % 4)) & 0xff;
            if ((b & 0x7f) == 0x7f) blocks |= 1u << (part * (VALUES / 16) + j), scales[j / 4] &= ~(0xffu << (8 * (j % 4)));
          }
          if (blocks)
            for (int t = 0; t < S::TILES; ++t) {
              if (!s.set.both && S::TILES == 2 && t != ((i - s.lo) & 1)) continue;
              for (int r = 0; r < 128; ++r) {
                const int m = s.tile * S::QUERIES + (s.set.both ? 128 * t : 0) + r;
                if (m < s.set.queries && decode_entries(s.set.kv, p.next_n, m / p.group, p.ratio, p.capacity) > e)
                  atomicOr(&nans[(segments[t] % S::NAN_SLOTS * S::TILES + t) * 128 + r], blocks);
              }
            }
        }
      }
      const uint32_t to = tiles + slot * S::KV_BYTES + tile_row * 128;
      uint32_t codes[4];
#pragma unroll
      for (int c16 = 0; c16 < VALUES / 32; ++c16) {  // 32 values: 16 bytes of codes, two blocks
        const uint4 v = *reinterpret_cast<const uint4*>(raw + part * (VALUES / 2) + c16 * 16);
        codes[0] = v.x, codes[1] = v.y, codes[2] = v.z, codes[3] = v.w;
        const uint32_t two = e4m3x2_to_f16x2(scales[c16 / 2] >> (16 * (c16 % 2)));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t h[4];
          e2m1_to_f16x2(codes[j], h);
          const uint32_t x = splat(two, j / 2);
#pragma unroll
          for (int y = 0; y < 4; ++y) h[y] = hmul2(h[y], x);
          const int piece = part * (VALUES / 8) + c16 * 4 + j;  // of 8 values
          const uint32_t dst = to + piece / 8 * (S::N * 128) + ((piece % 8) ^ (tile_row & 7)) * 16;
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
        }
      }
      if (!V && lane == 0) {  // which entries are there, for those who take the scores
        if (R == 32) masks[(count & 3) * 4 + w] = there;
        else reinterpret_cast<uint16_t*>(masks)[(count & 3) * 8 + w] = uint16_t(there);
      }
      gvr::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) gvr::mbar_arrive(V ? &bars->v_full[slot] : &bars->k_full[slot]);
      ++turn.used;
    }
    ++segments[0];
    if (!one) ++segments[1];
  }
  copy_wait<0>();
  return ok;
}

// Issues the products of all of the CTA's steps; by one thread.
template <int D>
__device__ __forceinline__ bool multiply(const SharedParams& p, const Plan& plan, SharedBars* bars, uint32_t tmem, uint32_t q_at, uint32_t k_at, uint32_t v_at) {
  using S = SharedShape<D>;
  constexpr uint32_t QK = product_f16(S::N, false), PV = product_f16(D, true);
  Walker walk(p, plan);
  Segment s;
  Turn k_turn, v_turn;
  uint32_t q_used[2] = {0, 0}, p_used[2] = {0, 0};
  int buffer = 0;  // one tile: of S, in turn
  while (walk.next(s, p.kv_heads)) {
    const bool both = S::TILES == 2 && s.set.both;
    const int tasks = (s.hi - s.lo) << (both ? 1 : 0);
    // task i: step i (both: i / 2), tile i % 2, scores in buffer i % 2 (one tile: in turn)
    auto scores = [&](int i) -> bool {
      const int tile = S::TILES == 2 ? i & 1 : 0, b = S::TILES == 2 ? tile : (buffer + i) & 1;
      if (i < S::TILES) {
        if (!gvr::mbar_wait_bounded(&bars->q_full[tile], q_used[tile] & 1, GIVE_UP_NS)) return false;
        ++q_used[tile];
      }
      const bool last = !both || tile == 1;  // that needs the step's K
      const int slot = k_turn.slot(S::KBUF);
      if (!both || tile == 0)
        if (!gvr::mbar_wait_bounded(&bars->k_full[slot], k_turn.parity(S::KBUF), GIVE_UP_NS)) return false;
      tc_fence_after();
      const uint32_t a = q_at + tile * S::Q_BYTES, k = k_at + slot * S::KV_BYTES;
#pragma unroll
      for (int x = 0; x < D / 16; ++x)
        tc_mma(tmem + S::S_AT + b * S::N, operand_k_major(a + x / 4 * (128 * 128) + x % 4 * 32), operand_k_major(k + x / 4 * (S::N * 128) + x % 4 * 32), QK, x > 0);
      tc_commit(&bars->s_full[b]);
      if (last) {
        tc_commit(&bars->k_free[slot]);
        ++k_turn.used;
      }
      return true;
    };
    auto values = [&](int i) -> bool {
      const int tile = S::TILES == 2 ? i & 1 : 0, b = S::TILES == 2 ? tile : (buffer + i) & 1;
      const int slot = v_turn.slot(S::VBUF);
      if (!both || tile == 0)
        if (!gvr::mbar_wait_bounded(&bars->v_full[slot], v_turn.parity(S::VBUF), GIVE_UP_NS)) return false;
      if (!gvr::mbar_wait_bounded(&bars->p_full[b], p_used[b] & 1, GIVE_UP_NS)) return false;
      ++p_used[b];
      tc_fence_after();
      const uint32_t v = v_at + slot * S::KV_BYTES;
#pragma unroll
      for (int x = 0; x < S::N / 16; ++x)
        tc_mma_tmem(tmem + S::O_AT + tile * D, tmem + S::S_AT + b * S::N + x * 8, operand_mn_major(v + x * (16 * 128), S::N * 128), PV, i >= S::TILES || x > 0);
      tc_commit(&bars->o_full[b]);
      if (!both || tile == 1) {
        tc_commit(&bars->v_free[slot]);
        ++v_turn.used;
      }
      return true;
    };
    if (!scores(0)) return false;
    if (tasks > 1 && !scores(1)) return false;
    for (int i = 0; i < tasks; ++i) {
      if (!values(i)) return false;
      if (i + 2 < tasks && !scores(i + 2)) return false;
    }
    if (S::TILES == 1) buffer = (buffer + tasks) & 1;
  }
  return true;
}

// By a whole warp, all of whose lanes go on, or give up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, gvr::mbar_wait_bounded(bar, parity, GIVE_UP_NS));
}

// Takes the scores of a tile, a query a thread: P, bases and sums, and at the end of each segment its piece.
template <int D>
__device__ __forceinline__ bool soften(const SharedParams& p, const Plan& plan, SharedBars* bars, uint32_t tmem, uint32_t q_at, int tile, const uint32_t* masks, uint32_t* nans) {
  using S = SharedShape<D>;
  constexpr int WORDS = S::N / 32;
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, row = quarter * 32 + lane;  // in the tile, and lane of tensor memory
  const uint32_t lanes = uint32_t(quarter) << 21;  // 32 quarter << 16
  const uint32_t q_row_at = q_at + tile * S::Q_BYTES + row * 128;
  Walker walk(p, plan);
  Segment s, next;
  uint32_t s_used[2] = {0, 0}, o_used[2] = {0, 0};
  uint32_t steps = 0, segments = 0;  // K steps of the segments before, and segments with work for this tile
  int buffer = 0;

  // Segment-wide facts of this thread's query.
  struct Query {
    float factor;
    int limit;    // entries that it sees
    int index;    // among the set's queries; -1: none
    bool warp;    // some thread of the warp has one
    int tasks;
  };
  auto begin_segment = [&](const Segment& g) -> Query {
    Query x;
    const bool both = S::TILES == 2 && g.set.both;
    const int n = g.hi - g.lo;
    x.tasks = S::TILES == 1 || both ? n : (n + 1 - tile) >> 1;
    const int m = g.tile * S::QUERIES + (both ? 128 * tile : 0) + row;
    bool live = m < g.set.queries;
    const int rel = m / p.group;
    const int64_t at = int64_t(g.set.row0) + rel;
    x.limit = g.set.end;
    if (live) {
      if (g.set.kv >= 0) x.limit = decode_entries(g.set.kv, p.next_n, rel, p.ratio, p.capacity);
      else live = p.joined[at / p.next_n].prefix >= 0;
    }
    x.index = live ? m : -1;
    x.factor = 1.f;
    x.warp = __any_sync(0xffffffffu, live);
    if (x.tasks == 0) return x;
    if (x.warp) {
      const uint4* src = reinterpret_cast<const uint4*>(p.q + at * p.q_row + int64_t(g.head * p.group + m - rel * p.group) * p.q_head);
      float mul = p.q_sign, back = 1.f;
      if (p.bf16) {  // exactly to f16 by a power of two per query (gvr_attend.cuh)
        uint32_t big = 0;
#pragma unroll 8
        for (int j = 0; j < D / 8; ++j) {
          const uint4 v = live ? src[j] : make_uint4(0, 0, 0, 0);
          big = __vmaxu2(__vmaxu2(big, v.x & 0x7fff7fffu), v.y & 0x7fff7fffu);
          big = __vmaxu2(__vmaxu2(big, v.z & 0x7fff7fffu), v.w & 0x7fff7fffu);
        }
        big = max(big & 0xffffu, big >> 16);
        const int exponent = int(big >> 7), up = big == 0 || exponent == 255 ? 0 : min(14 - (exponent - 127), 126);
        mul = p.q_sign * __uint_as_float(uint32_t(127 + up) << 23);
        back = __uint_as_float(uint32_t(127 - up) << 23);
      }
      const uint32_t sign = pack_f16(p.q_sign, p.q_sign);
#pragma unroll 8
      for (int j = 0; j < D / 8; ++j) {
        const uint4 v = live ? src[j] : make_uint4(0, 0, 0, 0);
        uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int y = 0; y < 4; ++y)
          h[y] = p.bf16 ? pack_f16(__uint_as_float(h[y] << 16) * mul, __uint_as_float(h[y] & 0xffff0000u) * mul) : hmul2(h[y], sign);
        const uint32_t dst = q_row_at + j / 8 * (128 * 128) + ((j % 8) ^ (row & 7)) * 16;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
      }
      x.factor = fmaxf(back * p.scale_log2, 1.17549435e-38f);
    }
    gvr::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) gvr::mbar_arrive(&bars->q_full[tile]);
    return x;
  };

  bool more = walk.next(s, p.kv_heads);
  Query x, x_next;
  if (more) x = begin_segment(s);
  while (more) {
    const bool both = S::TILES == 2 && s.set.both;
    float top = NO_TOP, total = 0.f;
    for (int i = 0; i < x.tasks; ++i) {
      const int b = S::TILES == 2 ? tile : (buffer + i) & 1;
      if (!warp_wait(&bars->s_full[b], s_used[b] & 1)) return false;
      ++s_used[b];
      tc_fence_after();
      const int step = S::TILES == 1 || both ? i : 2 * i + tile;
      if (x.warp) {
        const uint32_t scores = tmem + lanes + S::S_AT + b * S::N;
        uint32_t there[WORDS];  // entries that this query sees
        bool all = true;
        const int e0 = s.set.first + (s.lo + step) * S::N;
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
          there[w] = reinterpret_cast<const volatile uint32_t*>(masks)[((steps + step) & 3) * 4 + w];
          const int seen = x.limit - (e0 + 32 * w);
          if (seen < 32) there[w] &= seen <= 0 ? 0u : (1u << seen) - 1;
          all &= there[w] == 0xffffffffu;
        }
        const bool whole = __all_sync(0xffffffffu, all || x.index < 0);
        // the largest score
        float high = -INFINITY;
#pragma unroll
        for (int c = 0; c < WORDS; ++c) {
          uint32_t v[32];
          tmem_load(scores + 32 * c, v);
          tmem_load_wait();
          if (!whole) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(there[c] >> j & 1)) v[j] = 0xff800000u;
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) high = fmaxf(high, __uint_as_float(v[j]));
        }
        high *= x.factor;
        if (__any_sync(0xffffffffu, high > top + ABOVE)) {
          const float base = fmaxf(top, high - BELOW), down = exp2_fast(top - base);
          top = base, total *= down;
          if (i > 0) {  // O so far: all products of this tile are complete, as the next one waits for this P
            const int ob = S::TILES == 2 ? tile : b ^ 1;
            if (!warp_wait(&bars->o_full[ob], (o_used[ob] - 1) & 1)) return false;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t v[32];
              tmem_load(tmem + lanes + S::O_AT + tile * D + 32 * c, v);
              tmem_load_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * down);
              tmem_store(tmem + lanes + S::O_AT + tile * D + 32 * c, v);
            }
          }
        }
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < WORDS; ++c) {
          uint32_t v[32], h[16];
          tmem_load(scores + 32 * c, v);
          tmem_load_wait();
          if (!whole) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(there[c] >> j & 1)) v[j] = 0xff800000u;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float e0 = exp2_fast(fmaf(__uint_as_float(v[2 * j]), x.factor, -top)), e1 = exp2_fast(fmaf(__uint_as_float(v[2 * j + 1]), x.factor, -top));
            part[2 * j & 3] += e0, part[(2 * j + 1) & 3] += e1;
            h[j] = pack_f16(e0, e1);
          }
          tmem_store(scores + 16 * c, h);  // over scores that have been read
        }
        total += (part[0] + part[1]) + (part[2] + part[3]);
        tmem_store_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) gvr::mbar_arrive(&bars->p_full[b]);
      ++o_used[b];
    }
    if (S::TILES == 1) buffer = (buffer + x.tasks) & 1;
    steps += s.hi - s.lo;

    more = walk.next(next, p.kv_heads);
    if (more) x_next = begin_segment(next);  // its Q may be laid down: this segment's products with Q are complete

    // ---- the piece
    if (x.warp) {
      const bool prefix = s.set.kv < 0;
      const int rows = prefix ? 128 : p.suffix_rows;  // of a tile
      const int64_t floats = prefix ? S::PIECE : S::TILES * rows * (D + 2);
      float* piece = (prefix ? p.prefix_pieces : p.suffix_pieces) + int64_t(int(blockIdx.x) + s.set.unit0 + s.unit) * floats;
      const int at = tile * rows + row, height = S::TILES * rows;
      float* sums = piece + int64_t(height) * D;
      uint32_t nan = 0;
      if (x.tasks > 0) {
        const int ob = S::TILES == 2 ? tile : buffer ^ 1;
        if (!warp_wait(&bars->o_full[ob], (o_used[ob] - 1) & 1)) return false;
        tc_fence_after();
        uint32_t* mine = nans + (segments % S::NAN_SLOTS * S::TILES + tile) * 128 + row;
        nan = *reinterpret_cast<volatile uint32_t*>(mine);
        if (nan) *mine = 0;
      }
      if (x.index >= 0) sums[at] = top, sums[height + at] = total;
      if (x.tasks > 0) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_load(tmem + lanes + S::O_AT + tile * D + 32 * c, v);
          tmem_load_wait();
          if (nan) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (nan >> (2 * c + j / 16) & 1) v[j] = 0x7fc00000u;
          }
          if (x.index >= 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<uint4*>(piece + (int64_t(8 * c + j) * height + at) * 4) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          }
        }
        tc_fence_before();
      }
    }
    if (x.tasks > 0) ++segments;
    s = next, x = x_next;
  }
  return true;
}

template <int D>
__global__ void __launch_bounds__(SharedShape<D>::THREADS, 1) shared_kernel(SharedParams p) {
  using S = SharedShape<D>;
  extern __shared__ uint8_t dynamic[];
  __shared__ SharedBars bars;
  __shared__ uint32_t tmem_at, masks[4 * 4], nans[S::NAN_SLOTS * S::TILES * 128];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  uint8_t* base = dynamic + ((1024 - (gvr::smem_u32(dynamic) & 1023)) & 1023);
  const uint32_t q_at = gvr::smem_u32(base), k_at = q_at + S::TILES * S::Q_BYTES, v_at = k_at + S::KBUF * S::KV_BYTES;
  uint8_t* rings = base + S::TILES * S::Q_BYTES + (S::KBUF + S::VBUF) * S::KV_BYTES;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      gvr::mbar_init(&bars.k_full[i], 4), gvr::mbar_init(&bars.k_free[i], 1);
      gvr::mbar_init(&bars.v_full[i], 4), gvr::mbar_init(&bars.v_free[i], 1);
      gvr::mbar_init(&bars.q_full[i], 4), gvr::mbar_init(&bars.s_full[i], 1);
      gvr::mbar_init(&bars.p_full[i], 4), gvr::mbar_init(&bars.o_full[i], 1);
    }
    gvr::mbar_init(&bars.done, 1);
    gvr::mbar_init_fence();
  }
  for (int i = tid; i < S::NAN_SLOTS * S::TILES * 128; i += S::THREADS) nans[i] = 0;
  constexpr int FIRST_K = 4 * S::TILES, FIRST_V = FIRST_K + 4, ISSUER = FIRST_V + 4;
  if (warp == ISSUER) tmem_alloc_all(gvr::smem_u32(&tmem_at));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  begin();
  const int4 held = *reinterpret_cast<const int4*>(p.plan);
  const Plan plan = {held.x, held.y, held.z, held.w};
  bool ok;
  if (warp < FIRST_K) {
    ok = soften<D>(p, plan, &bars, tmem, q_at, warp / 4, masks, nans);
  } else if (warp < FIRST_V) {
    ok = bring<D, false>(p, plan, &bars, rings + (warp - FIRST_K) * S::RING, k_at, warp - FIRST_K, masks, nans);
  } else if (warp < ISSUER) {
    ok = bring<D, true>(p, plan, &bars, rings + (warp - FIRST_K) * S::RING, v_at, warp - FIRST_V, masks, nans);
  } else {
    ok = true;
    if (lane == 0) {
      ok = multiply<D>(p, plan, &bars, tmem, q_at, k_at, v_at);
      tc_commit(&bars.done);  // whatever has been issued is complete before its memory is given up
      ok &= gvr::mbar_wait_bounded(&bars.done, 0, GIVE_UP_NS);
    }
    __syncwarp();
  }
  if (!ok) p.plan->failed = 1;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == ISSUER) tmem_free_all(tmem);
}

// ------------------------------------------------------------------------------------------------ the join
constexpr int JOIN_SHARED_THREADS = 128;

// Sums of one query at four neighbouring dimensions.
struct Joining {
  float top = NO_TOP, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};

  __device__ __forceinline__ void add(float t, float s, const float4& v) {
    if (s == 0.f) return;  // saw nothing there (and what it holds may be a NaN of entries that it does not see)
    const float next = fmaxf(top, t), down = exp2_fast(top - next), up = exp2_fast(t - next);
    top = next, sum = sum * down + s * up;
    acc[0] = acc[0] * down + v.x * up, acc[1] = acc[1] * down + v.y * up, acc[2] = acc[2] * down + v.z * up, acc[3] = acc[3] * down + v.w * up;
  }
};

// All pieces of query m of a set's KV head.
template <int D>
__device__ __forceinline__ void join_set(const SharedParams& p, const Plan& plan, int which, int head, int m, int d4, Joining& j) {
  using S = SharedShape<D>;
  const int4* from = reinterpret_cast<const int4*>(p.sets + which);
  const int4 a = from[0], b = from[1], c = from[2];
  const Set set = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
  const bool prefix = set.kv < 0;
  const int tile = m / S::QUERIES, in = m - tile * S::QUERIES, unit = tile * p.kv_heads + head;
  const int work = set.steps << set.both, start = set.start + unit * work;
  // the last CTA whose share begins at or before x is ((x + 1) ctas - 1) / total
  const int c0 = int((int64_t(start + 1) * plan.ctas - 1) / plan.total), c1 = int((int64_t(start + work) * plan.ctas - 1) / plan.total);
  const int rows = prefix ? 128 : p.suffix_rows, height = S::TILES * rows;
  const int64_t floats = prefix ? S::PIECE : height * (D + 2);
  const float* pieces = (prefix ? p.prefix_pieces : p.suffix_pieces) + int64_t(set.unit0 + unit) * floats;
  const int at = set.both ? in / 128 * rows + in % 128 : in;
  const bool twice = S::TILES == 2 && !set.both;  // even steps in one tile, odd ones in the other
  for (int x = c0; x <= c1; ++x) {
    const int lo = step_of(range_start(x, plan.ctas, plan.total), start, set.both, set.steps);
    const int hi = step_of(range_start(x + 1, plan.ctas, plan.total), start, set.both, set.steps);
    if (hi <= lo) continue;
    const float* piece = pieces + int64_t(x) * floats;
    const float* sums = piece + int64_t(height) * D;
    j.add(sums[at], sums[height + at], *reinterpret_cast<const float4*>(piece + (int64_t(d4) * height + at) * 4));
    if (twice && hi - lo > 1)
      j.add(sums[rows + at], sums[height + rows + at], *reinterpret_cast<const float4*>(piece + (int64_t(d4) * height + rows + at) * 4));
  }
}

// blockIdx.x: requests x KV heads; y: parts of the request's queries x dimensions, four dimensions a thread.
template <int D>
__global__ void __launch_bounds__(JOIN_SHARED_THREADS) shared_join_kernel(SharedParams p) {
  const int r = blockIdx.x / p.kv_heads, h = blockIdx.x - r * p.kv_heads, members = p.next_n * p.group;
  begin();
  const int4 held = *reinterpret_cast<const int4*>(p.plan);
  const Plan plan = {held.x, held.y, held.z, held.w};
  const Joined join = p.joined[r];
  const int prefix_row0 = join.prefix >= 0 ? p.sets[join.prefix].row0 : 0;
  for (int i = blockIdx.y * JOIN_SHARED_THREADS + threadIdx.x; i < members * (D / 4); i += gridDim.y * JOIN_SHARED_THREADS) {
    const int d4 = i / members, m = i - d4 * members, rel = m / p.group;
    const int64_t row = int64_t(r) * p.next_n + rel;
    if (row >= p.num_rows) continue;
    Joining j;
    if (join.prefix >= 0) join_set<D>(p, plan, join.prefix, h, int(int64_t(r) * p.next_n - prefix_row0) * p.group + m, d4, j);
    if (join.suffix >= 0) join_set<D>(p, plan, join.suffix, h, m, d4, j);
    if (plan.failed) j.sum = NAN;
    const float norm = j.sum == 0.f ? 0.f : 1.f / j.sum;
    uint32_t packed[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const float lo = j.acc[2 * y] * norm * p.v_scale, hi = j.acc[2 * y + 1] * norm * p.v_scale;
      if (p.bf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(packed[y]) : "f"(hi), "f"(lo));
      else packed[y] = pack_f16(lo, hi);
    }
    const int64_t at = row * (int64_t(p.kv_heads) * p.group) + h * p.group + (m - rel * p.group);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at * D + d4 * 4) = make_uint2(packed[0], packed[1]);
    if (p.lse && d4 == 0) p.lse[at] = j.sum == 0.f ? -INFINITY : (j.top + log2f(j.sum)) * 0.69314718055994531f;
  }
}

// What the host needs to know of a head dimension's kernels.
struct SharedInfo {
  const void *plan, *kernel, *join;
  int threads, smem, queries, tiles, step, piece_floats;
};
template <int D>
SharedInfo shared_info() {
  using S = SharedShape<D>;
  return {reinterpret_cast<const void*>(shared_plan_kernel<D>), reinterpret_cast<const void*>(shared_kernel<D>),
          reinterpret_cast<const void*>(shared_join_kernel<D>), S::THREADS, S::SMEM, S::QUERIES, S::TILES, S::N, S::PIECE};
}
SharedInfo shared_64();
SharedInfo shared_128();
SharedInfo shared_256();

}  // namespace gvrc
