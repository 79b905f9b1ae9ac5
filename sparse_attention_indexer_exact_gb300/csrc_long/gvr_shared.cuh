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
// (Of many requests with few entries behind their prefix, these are no sets: gvr_tails.cuh leaves pieces of them.)
//
// A CTA.  One warp walks over the share: it notes the segments for the others and starts the copies of their rows, a
// page's rows of a head (up to a step's) a bulk tensor copy.  Four warps expand K and four V (e2m1 times e4m3 is exact
// in f16), from there into matrix operands in shared memory.  One lane of a warp issues the products
// S = Q K^T and O += P V on the fifth-generation tensor cores, 128 queries a tile: S and O lie in tensor memory.  Eight warps a
// tile take S, two threads a query, each half of the step's entries, and write P, in f16, over it; P is read from there as an
// operand.  Two tiles take turns: while one's P is made, the other's products run.  Where a unit
// has up to 128 queries both tiles hold them, one taking the even steps, one the odd ones.
//
// What bounds it (64 requests of 2 rows behind 32000 entries, 64 heads over 8 of 128: 165 us, 0.42 of the tensor cores' measured
// rate; the plan takes 5 us of it, the tails 35, the shares 112, the join 12; without tails as much in all).  A step of a unit of 256 queries takes 2.2 us, of 128 queries
// 1.25 (head_dim 64: 1.8 and 1.0; 256, 64 entries and 128 queries: 1.25).  No pipe is busy: the tensor pipe 52 %, issue
// 57 %, DRAM 5 %.  What counts is the way of a tile through
// its step, scores -> maximum -> exponentials -> P -> products -> scores, about 3400 clocks of which the other tile's hide half.
// Tensor memory has no room for more tiles: at head_dim 128 two times O and S take all of its columns.
//
// Tried, with times of that call at their time: a lone thread as issuer instead of a converged warp's elected lane (367 us against 325), loops
// unrolled (260 against 213: code beyond the instruction caches), counters of barriers in arrays (185 against 175: they
// lie in memory), copies by warps instead of tensor copies (+8 us), one thread a query (slower), three of eight exponentials by a
// polynomial (slower), a pass without the maximum of the step (spills), the first scores kept in registers from the
// maximum's pass to the exponentials' (+2.5), queries read twice, for their largest and to convert them (+12), P handed over by halves (+3), V waited for by halves (+4) or quarters (+13), an issuer
// a tile (+32: their products interleave, and each tile's are through later).  Without exponentials, expansions and
// maxima, and with one product for eight, 140 of then 194 us were left.  The joining kernel is not let start early: its CTAs, few of
// which read most, would gather on the SMs that are through first (66 us became 80 where 640 queries of one KV head share
// 131071 entries).
#pragma once

#include <cuda.h>

#include "../csrc_cache/gvr_attend.cuh"
#include "gvr_long_common.h"
#include "gvr_shares.h"
#include "gvr_tails.cuh"
#include "gvr_tcgen05.cuh"

namespace gvrc {

// Queries that read the same entries: rows row0 .. of a group, or of a request.
struct Set {
  int32_t start;    // work before it, in tile steps
  int32_t steps;    // of N entries, of each unit
  int32_t units;    // KV heads x query tiles
  int32_t full;     // of them those of more than 128 queries, the first ones: both tiles take each step
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
  int32_t* cta_start;  // [grid + 1]: where it begins
  float* prefix_pieces;
  float* suffix_pieces;
  float* tail_pieces;
  int64_t q_row, q_head, table_stride, num_rows;
  uint32_t unit, page_units, entry_units, row_units;  // as in AttendParams
  int32_t num_pages, page_shift, kv_heads, group, capacity, next_n, ratio, bf16, requests, groups, grid;
  int32_t suffix_rows;  // rows of a tile in a suffix piece (a multiple of 8)
  int32_t tail_entries, tail_height;  // requests with at most so many entries behind their prefix have a tail in place of a set (0: none)
  float scale_log2, q_sign, v_scale;
};

template <int D>
struct SharedShape {
  static constexpr int N = D == 256 ? 64 : 128;      // entries a step
  static constexpr int TILES = D == 256 ? 1 : 2;     // O takes D columns of tensor memory a tile, S two times N
  static constexpr int QUERIES = 128 * TILES;        // of a unit
  static constexpr int ROWS = N / 4;                 // rows a warp expands in a step
  static constexpr int Q_BYTES = 128 * D * 2, KV_BYTES = N * D * 2;
  static constexpr int RB = row_bytes(D), RAW = N * RB, STAGES = D == 64 ? 6 : 3;  // rows as they are, of the steps under way
  static constexpr int WARPS = 8 * TILES + 12, THREADS = 32 * WARPS;  // S takers, K and V, and the issuer, the walker and two idle ones
  static constexpr int PIECE = QUERIES * (D + 2);    // floats of a prefix piece
  static constexpr int S_AT = 0, O_AT = 2 * N;  // columns; P lies over its scores, the halves' where theirs begin
  static constexpr int NAN_SLOTS = 2;
  static constexpr int SMEM = TILES * Q_BYTES + 3 * KV_BYTES + STAGES * RAW + 1024;  // two of K, one of V; 1024 to align
  // Registers of a thread: those who take S hold half a row of it.  Their sum is what the CTA is launched with (896 threads of
  // 72; head_dim 256: 640 of 96, which need no exchange).
  static constexpr int SOFT_REGS = 88, BRING_REGS = 56, REST_REGS = 40;
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
  int* prefixes = lead + p.groups;    // [groups]
  int* lens = prefixes + p.groups;    // [requests]
  int* starts = lens + p.requests;    // [groups + requests]: of the sets that have work
  __shared__ int2 sums[32];
  __shared__ int flags[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  begin();
  let_next_start();  // its CTAs, one an SM, set up meanwhile
  for (int r = tid; r < p.requests; r += PLAN_THREADS) lens[r] = p.lens[r];  // all reads on their way at once
  // groups begin where their start says, but not before the one before them
  int most = 0;
  for (int i0 = 0; i0 <= p.groups && p.groups > 0; i0 += PLAN_THREADS) {
    const int i = i0 + tid;
    int x = i <= p.groups ? min(max(p.group_starts[i], 0), p.requests) : 0;
    const int prefix = i < p.groups ? min(max(p.prefix_entries[i], 0), p.capacity) & -STEP : 0;  // tails begin where their steps do
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
    if (i < p.groups) sharing[i] = 0, lead[i] = p.requests, prefixes[i] = prefix;
  }
  __syncthreads();
  // the group whose prefix all rows of request r see, -1: none
  auto group_of = [&](int r, int kv) {
    if (p.groups == 0 || r < from[0] || r >= from[p.groups]) return -1;
    int lo = 0;
    for (int hi = p.groups; hi - lo > 1;) {
      const int mid = (lo + hi) >> 1;
      if (from[mid] <= r) lo = mid; else hi = mid;
    }
    const int prefix = prefixes[lo];
    return prefix > 0 && decode_entries(kv, p.next_n, 0, p.ratio, p.capacity) >= prefix ? lo : -1;
  };
  for (int r = tid; r < p.requests; r += PLAN_THREADS) {
    const int g = group_of(r, lens[r]);
    if (g >= 0) atomicAdd(&sharing[g], 1), atomicMin(&lead[g], r);
  }
  __syncthreads();

  int2 before = make_int2(0, 0);
  int sets = 0;
  // `set` with all but its sums: takes its place if it has work; returns the place or -1
  auto place = [&](bool is, Set set) -> int {
    const int tiles = (set.queries + S::QUERIES - 1) / S::QUERIES;
    set.units = is ? p.kv_heads * tiles : 0;
    set.full = S::TILES == 2 && is ? p.kv_heads * ((set.queries + 127) / S::QUERIES) : 0;
    const int first = set.first & -S::N;  // steps begin at multiples of N
    set.steps = is && set.end > set.first ? (set.end - first + S::N - 1) / S::N : 0;
    const int work = set.steps ? unit_start(set.units, set.full, set.steps) : 0;
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
      set.end = prefixes[g];
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
    Joined join = {-1, -1, 0, 0};
    if (r < p.requests) {
      set.kv = max(lens[r], 0);
      const int g = group_of(r, lens[r]);
      join.prefix = g < 0 ? -1 : sharing[g];
      set.first = join.prefix < 0 ? 0 : prefixes[g];
      set.end = decode_entries(lens[r], p.next_n, p.next_n - 1, p.ratio, p.capacity);
      set.request = r;
      set.row0 = r * p.next_n;
      set.queries = int(min(int64_t(p.next_n), p.num_rows - set.row0)) * p.group;
      set.unit0 = r * (p.kv_heads * ((p.next_n * p.group + S::QUERIES - 1) / S::QUERIES));
    }
    const bool tail = set.end > set.first && set.end - set.first <= p.tail_entries;
    if (tail) join.tail_first = set.first / STEP, join.tail_steps = (set.end - set.first + STEP - 1) / STEP;
    join.suffix = place(r < p.requests && !tail, set);
    if (r < p.requests) p.joined[r] = join;
  }
  __syncthreads();
  const int total = before.x, ctas = max(1, min(p.grid, total / LEAST_WORK));
  if (tid == 0) *p.plan = {total, ctas, sets, 0};
  for (int c = tid; c <= ctas; c += PLAN_THREADS) {
    const int at = share_start(c, ctas, total);
    p.cta_start[c] = at;
    if (c == ctas) break;
    int lo = 0;
    for (int hi = sets; hi - lo > 1;) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= at) lo = mid; else hi = mid;
    }
    p.cta_set[c] = lo;
  }
}

// ------------------------------------------------------------------------------------------------ the walk
// A CTA's part of a unit: steps [lo, hi) of its set's; 0 steps: no more.
struct __align__(16) Segment {
  int32_t first, end, kv;       // entry of the first step; the set's last entry, and its length (-1: a prefix)
  int32_t row0, queries, both;  // of the set; whether both tiles take each step
  int32_t lo, hi, head, tile;   // KV head, and number of the unit among the set's query tiles
  float* piece;
};

// Waits for the phase with parity `parity` to complete, giving up after 2^30 clocks, half a second.  (In one piece, so that
// a warp that waits counts as going the same way in all lanes, and what it computes as the same in all of them.)
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u64 t0, t1;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "mov.u64 t0, %%clock64;\n\t"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "@p bra DONE;\n\t"
      "mov.u64 t1, %%clock64;\n\t"
      "sub.u64 t1, t1, t0;\n\t"
      "setp.lt.u64 q, t1, 0x40000000;\n\t"
      "@q bra AGAIN;\n\t"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(gvr::smem_u32(bar)), "r"(parity), "r"(1000000)  // ns that a try may sleep
      : "memory");
  return ok != 0;
}

constexpr int SEGMENTS = 4;  // noted ahead
constexpr int STEP_NOTES = 8, MOST_STAGES = 6;

// Uses of two buffers in turn.
struct Turn {
  uint32_t used = 0;
  __device__ __forceinline__ int slot() const { return int(used & 1); }
  __device__ __forceinline__ uint32_t parity() const { return used >> 1 & 1; }
};

struct SharedBars {
  uint64_t raw_full[MOST_STAGES], raw_free[MOST_STAGES], k_full[2], k_free[2], v_full[2], v_free[2], q_full[2], s_full[2], p_full[2], o_full[2], done;
  uint64_t seg_full[SEGMENTS], seg_free[SEGMENTS];
};

// A step, for those who expand its rows and take its scores.
struct __align__(16) StepNote {
  uint32_t there[4];  // which of its entries exist
  int border;         // its first entry if some rows of its unit do not see all of it, else -1; -2: no more steps
  int set, where;     // of a border step: its set; its query tile << 12 | tiles' numbers of segments << 8, 4 | both tiles take it << 1 | parity in the segment
  int pad;
};

// What the warps of a CTA tell each other beside the operands.
struct SharedNotes {
  Segment segments[SEGMENTS];
  StepNote steps[STEP_NOTES];  // rows are loaded at most STAGES + 1 steps before their scores are through with
};

__device__ __forceinline__ bool next_segment(SharedBars* bars, uint32_t count) { return bar_wait(&bars->seg_full[count % SEGMENTS], count / SEGMENTS & 1); }
__device__ __forceinline__ void leave_segment(SharedBars* bars, uint32_t count) { gvr::mbar_arrive(&bars->seg_free[count % SEGMENTS]); }

// The rows [y, ...) of a page, of one head: as many as the map's box has.
__device__ __forceinline__ void copy_box(uint32_t to, const CUtensorMap* map, int x, int y, int page, uint64_t* bar) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(to), "l"(map), "r"(x),
               "r"(y), "r"(page), "r"(gvr::smem_u32(bar))
               : "memory");
}

// Walks over the CTA's share: notes segments and steps, starts the copies of their rows.  By one warp; lane i finds the pages
// of a step's i-th box (or, where pages are too small for boxes, which begin on multiples of 128 bytes, of entries i, i + 32, ...).
template <int D>
__device__ __forceinline__ bool walk(const SharedParams& p, const CUtensorMap* map, const Plan& plan, SharedNotes* notes, SharedBars* bars, uint32_t raw_at) {
  using S = SharedShape<D>;
  const int lane = threadIdx.x & 31;
  const bool boxes = p.page_shift >= 3;
  const int box_shift = min(p.page_shift, S::N == 128 ? 7 : 6), per_step = S::N >> box_shift;  // rows of a box, boxes of a step
  int at = 0, last = 0, next_set = 0;
  int4 a, b, c;  // the next set, on its way
  a = b = c = make_int4(0, 0, 0, 0);
  auto ask = [&]() {
    const int4* from = reinterpret_cast<const int4*>(p.sets + next_set);
    a = from[0], b = from[1], c = from[2];
  };
  Set set = {};
  if (int(blockIdx.x) < plan.ctas && plan.total > 0) {
    at = p.cta_start[blockIdx.x], last = p.cta_start[blockIdx.x + 1];
    next_set = p.cta_set[blockIdx.x];
    ask();
  }
  bool fresh = true;
  uint32_t steps = 0, stage = 0, turn = 0, first_only = 0;
  for (uint32_t count = 0;; ++count) {
    Segment s = {};
    while (at < last) {
      if (fresh) {
        set = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
        if (++next_set < plan.sets) ask();
      }
      const int unit = unit_at(at - set.start, set.full, set.steps), both = unit < set.full;
      const int start = set.start + unit_start(unit, set.full, set.steps), end = start + unit_work(set.steps, both), to = min(last, end);
      s.lo = step_of(at, start, both, set.steps), s.hi = step_of(to, start, both, set.steps);
      fresh = unit + 1 == set.units && to == end;
      at = to;
      if (s.hi <= s.lo) continue;
      s.end = set.end, s.kv = set.kv;
      s.first = (set.first & -S::N) + s.lo * S::N;
      s.row0 = set.row0, s.queries = set.queries, s.both = both;
      s.tile = unit / p.kv_heads;
      s.head = unit - s.tile * p.kv_heads;
      const int64_t piece = int(blockIdx.x) + set.unit0 + unit;
      s.piece = set.kv < 0 ? p.prefix_pieces + piece * S::PIECE : p.suffix_pieces + piece * (S::TILES * p.suffix_rows * (D + 2));
      break;
    }
    const int slot = count % SEGMENTS;
    if (!__all_sync(0xffffffffu, bar_wait(&bars->seg_free[slot], (count / SEGMENTS & 1) ^ 1))) return false;
    if (lane == 0) {
      notes->segments[slot] = s;
      gvr::mbar_arrive(&bars->seg_full[slot]);
    }
    const int left = s.hi - s.lo;
    const int sure = set.kv < 0 ? set.end : decode_entries(set.kv, p.next_n, 0, p.ratio, p.capacity);
    const int where = s.tile << 12 | int((count - first_only) % S::NAN_SLOTS) << 8 | int(count % S::NAN_SLOTS) << 4 | s.both << 1;
    first_only += left == 1 && !s.both;
    const int32_t* table = p.table + set.request * p.table_stride;
    const int x = s.head * (S::RB / 4);  // in words
    auto page_of = [&](int i) {  // of this lane's box of the segment's i-th step
      const int e = s.first + i * S::N + (lane << box_shift);
      return boxes && lane < per_step && i < left && e < set.end ? table[e >> p.page_shift] : -1;
    };
    int page = page_of(0);
    for (int i = 0; i < left || (left == 0 && i == 0); ++i) {  // without steps: the note that there are no more
      const int next_page = page_of(i + 1);
      if (!__all_sync(0xffffffffu, bar_wait(&bars->raw_free[stage], turn ^ 1))) return false;
      StepNote& note = notes->steps[steps & (STEP_NOTES - 1)];
      const int e0 = s.first + i * S::N;
      const uint32_t to = raw_at + stage * S::RAW;
      uint64_t* full = &bars->raw_full[stage];
      if (lane == 0) {
        note.border = left == 0 ? -2 : e0 + S::N > sure ? e0 : -1;
        note.set = next_set - 1, note.where = where | (i & 1);
      }
      if (boxes) {
        const bool is = uint32_t(page) < uint32_t(p.num_pages);
        const uint32_t got = __ballot_sync(0xffffffffu, is);
#pragma unroll
        for (int w = 0; w < S::N / 32; ++w) {  // entry 32 w + lane
          const int e = e0 + 32 * w + lane;
          const uint32_t there = __ballot_sync(0xffffffffu, got >> ((32 * w + lane) >> box_shift) & 1 && e >= set.first && e < set.end);
          if (lane == 0) note.there[w] = there;
        }
        if (lane == 0) gvr::mbar_arrive_expect_tx(full, uint32_t(__popc(got)) * (S::RB << box_shift));
        __syncwarp();
        if (is) copy_box(to + lane * (S::RB << box_shift), map, x, (e0 + (lane << box_shift)) & ((1 << p.page_shift) - 1), page, full);
      } else {
        int rows = 0, pages[S::N / 32];
#pragma unroll
        for (int w = 0; w < S::N / 32; ++w) {
          const int e = e0 + 32 * w + lane;
          pages[w] = left > 0 && e >= set.first && e < set.end ? table[e >> p.page_shift] : -1;
          const uint32_t there = __ballot_sync(0xffffffffu, uint32_t(pages[w]) < uint32_t(p.num_pages));
          if (lane == 0) note.there[w] = there;
          rows += __popc(there);
        }
        if (lane == 0) gvr::mbar_arrive_expect_tx(full, rows * S::RB);
        __syncwarp();
#pragma unroll
        for (int w = 0; w < S::N / 32; ++w)
          if (uint32_t(pages[w]) < uint32_t(p.num_pages)) {
            const uint32_t of = row_unit(pages[w], e0 + 32 * w + lane, p.page_shift, p.page_units, p.entry_units, uint32_t(s.head) * p.row_units);
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to + (32 * w + lane) * S::RB),
                         "l"(p.data + uint64_t(of) * p.unit), "r"(S::RB), "r"(gvr::smem_u32(full))
                         : "memory");
          }
      }
      page = next_page;
      ++steps;
      if (++stage == S::STAGES) stage = 0, turn ^= 1;
    }
    if (left == 0) return true;
  }
}

// A NaN that only some rows of a unit see is taken out of V, and put into those rows' results: `blocks` of 16 values of
// entry e, which the rows whose limit lies behind it note.  Of a prefix's rows only those of requests that share it: a
// warp that takes scores neither reads nor clears the notes of rows that are all without one.
template <int D>
__device__ __noinline__ void note_nan(const Set* set, const Joined* joined, int next_n, int group, int ratio, int capacity, int where, int e, uint32_t blocks,
                                      uint32_t* nans) {
  using S = SharedShape<D>;
  const Set of = *set;
  for (int t = 0; t < S::TILES; ++t) {
    const bool both = where >> 1 & 1;
    if (!both && S::TILES == 2 && t != (where & 1)) continue;
    const int slot = where >> (t ? 8 : 4) & 15;
    for (int x = 0; x < 128; ++x) {
      const int m = (where >> 12) * S::QUERIES + (both ? 128 * t : 0) + x;
      if (m >= of.queries) break;
      const int rel = m / group;
      const bool sees = of.kv < 0 ? joined[(of.row0 + rel) / next_n].prefix >= 0 && of.end > e : decode_entries(of.kv, next_n, rel, ratio, capacity) > e;
      if (sees) atomicOr(&nans[(slot * S::TILES + t) * 128 + x], blocks);
    }
  }
}

// Expands K or V, a quarter of each step's rows a warp.  A lane has a row (head_dim 256: half of one); 16-byte reads and
// stores of eight lanes fall on different banks.
template <int D>
__device__ __forceinline__ bool bring(const SharedParams& p, SharedBars* bars, const uint8_t* raw, uint32_t tiles, int w, bool is_v, const SharedNotes* notes, uint32_t* nans) {
  using S = SharedShape<D>;
  constexpr int R = S::ROWS, LANES = 32 / R, VALUES = D / LANES;  // of a lane
  const int lane = threadIdx.x & 31, part = R == 32 ? 0 : lane & 1;
  const int row = w * R + (R == 32 ? lane : lane >> 1), half = w / 2;  // V's one buffer goes by halves
  const uint8_t* from = raw + row * S::RB + (is_v ? D / 2 : 0) + part * (VALUES / 2);
  const uint8_t* scales_from = raw + row * S::RB + D + (is_v ? D / 16 : 0) + part * (VALUES / 16);
  const uint32_t to = tiles + row * 128 + part * (VALUES / 64) * (S::N * 128) + ((row & 7) << 4);
  uint32_t stage = 0, turn = 0;
  for (uint32_t step = 0;; ++step) {
    if (!__all_sync(0xffffffffu, bar_wait(&bars->raw_full[stage], turn))) return false;
    const StepNote& note = notes->steps[step & (STEP_NOTES - 1)];
    const int border = note.border;
    if (border == -2) return true;
    uint32_t scales[VALUES / 64];  // four a word
    load_words<VALUES / 64>(scales_from + stage * S::RAW, scales);
    if (!(note.there[row / 32] >> (row % 32) & 1)) {
#pragma unroll
      for (int j = 0; j < VALUES / 64; ++j) scales[j] = 0;  // P is 0 there, and 0 x NaN is not
    }
    const int slot = is_v ? 0 : int(step & 1);
    if (!__all_sync(0xffffffffu, bar_wait(is_v ? &bars->v_free[half] : &bars->k_free[slot], (is_v ? step & 1 : step >> 1 & 1) ^ 1))) return false;
    // Behind the wait: the products of the step before this one are complete, so that each tile's takers have written P of
    // a later segment than the one that had this segment's slot, and that one's notes are read and cleared.
    if (is_v && border >= 0) {
      uint32_t blocks = 0;
#pragma unroll
      for (int j = 0; j < VALUES / 16; ++j)
        if ((scales[j / 4] >> (8 * (j % 4)) & 0x7f) == 0x7f) blocks |= 1u << (part * (VALUES / 16) + j), scales[j / 4] &= ~(0xffu << (8 * (j % 4)));
      if (blocks) note_nan<D>(p.sets + note.set, p.joined, p.next_n, p.group, p.ratio, p.capacity, note.where, border + row, blocks, nans);
    }
    const uint8_t* at = from + stage * S::RAW;
    uint32_t dst = to + slot * S::KV_BYTES;
#pragma unroll 1
    for (int x = 0; x < VALUES / 32; x += 2) {  // 64 values, a panel: 32 bytes of codes, four scales
      const uint4 v0 = *reinterpret_cast<const uint4*>(at + x * 16), v1 = *reinterpret_cast<const uint4*>(at + x * 16 + 16);
      const uint32_t codes[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
      const uint32_t four = VALUES == 64 || x == 0 ? scales[0] : scales[VALUES / 64 - 1];
      const uint32_t two[2] = {e4m3x2_to_f16x2(four), e4m3x2_to_f16x2(four >> 16)};
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        uint32_t h[4];
        e2m1_to_f16x2(codes[y], h);
        const uint32_t f = splat(two[y / 4], y / 2 & 1);
#pragma unroll
        for (int z = 0; z < 4; ++z) h[z] = hmul2(h[z], f);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst ^ (y << 4)), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
      }
      dst += S::N * 128;
    }
    gvr::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      gvr::mbar_arrive(is_v ? &bars->v_full[half] : &bars->k_full[slot]);
      gvr::mbar_arrive(&bars->raw_free[stage]);
    }
    if (++stage == S::STAGES) stage = 0, turn ^= 1;
  }
}

// By a whole warp, all of whose lanes go on, or give up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, bar_wait(bar, parity)); }

// Issues the products of all of the CTA's steps; by one warp, of which one lane does.
template <int D>
__device__ __forceinline__ bool multiply(SharedBars* bars, const SharedNotes* notes, uint32_t tmem, uint32_t q_at, uint32_t k_at, uint32_t v_at) {
  using S = SharedShape<D>;
  constexpr uint32_t QK = product_f16(S::N, false), PV = product_f16(D, true);
  const int lane = threadIdx.x & 31;
  Turn k_turn;
  uint32_t v_used = 0;
  uint32_t q_phase = 0, p_phase = 0;  // a bit a tile, a bit a buffer of S  (arrays would be in memory, between every two products)
  int buffer = 0;                     // one tile: of S, in turn
  for (uint32_t count = 0;; ++count) {
    if (!warp_wait(&bars->seg_full[count % SEGMENTS], count / SEGMENTS & 1)) return false;
    const Segment& s = notes->segments[count % SEGMENTS];
    const bool both = S::TILES == 2 && __shfl_sync(0xffffffffu, s.both, 0);
    const int tasks = __shfl_sync(0xffffffffu, s.hi - s.lo, 0) << (both ? 1 : 0);
    __syncwarp();
    if (lane == 0) leave_segment(bars, count);
    __syncwarp();
    if (tasks == 0) return true;
    // Task i: step i (both: i / 2), tile i % 2, scores in buffer i % 2 (one tile: in turn).  Behind the values of task i
    // come the scores of task i + 2, which take the place of its P.
    bool ok = true;
    for (int i = -2; i < tasks; ++i) {
      const int next = i + 2, tile = S::TILES == 2 ? i & 1 : 0, b = S::TILES == 2 ? tile : (buffer + i) & 1;
      const bool weigh = i >= 0, score = next < tasks;
      const bool first = !both || tile == 0, last = !both || tile == 1;  // that needs a step's K and V
      const int slot = k_turn.slot();
      const uint64_t q = operand_k_major(q_at + tile * S::Q_BYTES), k = operand_k_major(k_at + slot * S::KV_BYTES), v = operand_mn_major(v_at, S::N * 128);
      const uint32_t scores = tmem + S::S_AT + b * S::N, sums = tmem + S::O_AT + tile * D;
      if (weigh) {
        if (first) ok &= bar_wait(&bars->v_full[0], v_used & 1) & bar_wait(&bars->v_full[1], v_used & 1);
        ok &= bar_wait(&bars->p_full[b], p_phase >> b & 1);
        p_phase ^= 1u << b;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < S::N / 16; ++x) {
            tc_mma_tmem(sums, scores + x / (S::N / 32) * (S::N / 2) + x % (S::N / 32) * 8, v + ((x * (16 * 128)) >> 4), PV, i >= S::TILES || x > 0);
            if (x == S::N / 32 - 1 && last) tc_commit(&bars->v_free[0]);
          }
          if (last) tc_commit(&bars->v_free[1]);
          tc_commit(&bars->o_full[b]);
        }
        __syncwarp();
      }
      if (score) {
        if (next < S::TILES) {
          ok &= bar_wait(&bars->q_full[tile], q_phase >> tile & 1);
          q_phase ^= 1u << tile;
        }
        if (first) ok &= bar_wait(&bars->k_full[slot], k_turn.parity());
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
            tc_mma(scores, q + ((x / 4 * (128 * 128) + x % 4 * 32) >> 4), k + ((x / 4 * (S::N * 128) + x % 4 * 32) >> 4), QK, x > 0);
          tc_commit(&bars->s_full[b]);
          if (last) tc_commit(&bars->k_free[slot]);
        }
        __syncwarp();
      }
      if (last && weigh) ++v_used;
      if (last && score) ++k_turn.used;
      if (!__all_sync(0xffffffffu, ok)) return false;
    }
    if (S::TILES == 1) buffer = (buffer + tasks) & 1;
  }
}

__device__ __forceinline__ uint64_t two_f32(uint32_t lo, uint32_t hi) { return uint64_t(lo) | uint64_t(hi) << 32; }
__device__ __forceinline__ uint64_t fma_two(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_two(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint64_t exp2_two(uint64_t x) {
  return two_f32(__float_as_uint(exp2_fast(__uint_as_float(uint32_t(x)))), __float_as_uint(exp2_fast(__uint_as_float(uint32_t(x >> 32)))));
}

__device__ __forceinline__ float max_three(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Meets the warp that has the other half of the same rows; true for both if `is` is for a thread of either.
__device__ __forceinline__ bool meet(int pair, bool is) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.cta.red.or.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(r)
               : "r"(pair + 1), "r"(uint32_t(is))
               : "memory");
  return r != 0;
}

// Takes the scores of a tile, half of a step's entries of a query a thread: P, bases and sums, and at the end of each segment
// its piece, half of the dimensions a thread.
template <int D>
__device__ __forceinline__ bool soften(const SharedParams& p, SharedBars* bars, uint32_t tmem, uint32_t q_at, int warp, SharedNotes* notes, uint32_t* nans, float* exchange) {
  using S = SharedShape<D>;
  constexpr int COLUMNS = S::N / 2, WORDS = COLUMNS / 32;  // of this thread
  const int tile = warp >> 3, half = warp >> 2 & 1, quarter = warp & 3;
  const int lane = threadIdx.x & 31, row = quarter * 32 + lane;  // in the tile, and lane of tensor memory
  const int pair = tile * 4 + quarter;
  float* mine = exchange + (tile * 2 + half) * 128 + row;
  const float* other = exchange + (tile * 2 + (half ^ 1)) * 128 + row;
  float* totals = exchange + S::TILES * 2 * 128;  // of the second halves
  const uint32_t lanes = uint32_t(quarter) << 21;  // 32 quarter << 16
  const uint32_t q_row_at = q_at + tile * S::Q_BYTES + row * 128;
  uint32_t done = 0;                 // tasks of this tile so far: theirs are S and O in turn (one tile: in two buffers)
  uint32_t steps = 0, segments = 0;  // K steps of the segments before, and segments with work for this tile
  uint32_t count = 0;                // segments so far
  // A wait that gave up: this warp goes on without waiting until it meets the other one, and both end.
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) ok = warp_wait(bar, parity);
  };

  auto wait_products = [&]() {  // with V, of the last task
    const uint32_t last = done - 1;
    wait(&bars->o_full[S::TILES == 2 ? tile : int(last & 1)], (S::TILES == 2 ? last : last >> 1) & 1);
  };

  // Segment-wide facts of this thread's query.
  struct Query {
    float factor;
    int limit;    // entries that it sees
    int first;    // this thread's first entry of the segment's first step
    bool live;
    bool warp;    // some thread of the warp has one
    bool both;
    int steps;    // of the segment; 0: no more
    int tasks;    // of them this tile's
    int height;   // rows of the piece
    int at;       // its place among them
    float* piece;  // of that place
  };
  auto begin_segment = [&](Query& x) {
    wait(&bars->seg_full[count % SEGMENTS], count / SEGMENTS & 1);
    if (meet(pair, !ok)) {
      ok = false;
      x.steps = x.tasks = 0;
      return;
    }
    const Segment g = notes->segments[count % SEGMENTS];
    __syncwarp();
    if (lane == 0) leave_segment(bars, count);
    ++count;
    x.both = S::TILES == 2 && g.both;
    x.steps = g.hi - g.lo;
    x.tasks = S::TILES == 1 || x.both ? x.steps : (x.steps + 1 - tile) >> 1;
    x.first = g.first + half * COLUMNS;
    const int m = g.tile * S::QUERIES + (x.both ? 128 * tile : 0) + row;
    bool live = m < g.queries;
    const int rel = m / p.group;
    const int64_t at = int64_t(g.row0) + rel;
    x.limit = g.end;
    if (live) {
      if (g.kv >= 0) x.limit = decode_entries(g.kv, p.next_n, rel, p.ratio, p.capacity);
      else live = p.joined[at / p.next_n].prefix >= 0;
    }
    x.live = live;
    x.factor = 1.f;
    x.warp = __any_sync(0xffffffffu, live);
    const int rows = g.kv < 0 ? 128 : p.suffix_rows;  // of a tile
    x.height = S::TILES * rows;
    x.at = tile * rows + row;
    x.piece = g.piece + x.at;
    if (x.tasks == 0) return;
    if (x.warp) {
      // half of the query's values, in one go as far as registers have room
      constexpr int PARTS = D / 16, HELD = PARTS < 8 ? PARTS : 8;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + at * p.q_row + int64_t(g.head * p.group + m - rel * p.group) * p.q_head) + half * PARTS;
      uint4 v[HELD];
      auto load = [&](int j0) {
#pragma unroll
        for (int j = 0; j < HELD; ++j) v[j] = live ? src[j0 + j] : make_uint4(0, 0, 0, 0);
      };
      float mul = p.q_sign, back = 1.f;
      if (p.bf16) {  // exactly to f16 by a power of two per query (gvr_attend.cuh)
        uint32_t big = 0;
#pragma unroll 1
        for (int j0 = PARTS - HELD; j0 >= 0; j0 -= HELD) {  // the first ones last: they stay
          load(j0);
#pragma unroll
          for (int j = 0; j < HELD; ++j) {
            big = __vmaxu2(__vmaxu2(big, v[j].x & 0x7fff7fffu), v[j].y & 0x7fff7fffu);
            big = __vmaxu2(__vmaxu2(big, v[j].z & 0x7fff7fffu), v[j].w & 0x7fff7fffu);
          }
        }
        big = max(big & 0xffffu, big >> 16);
        *mine = __uint_as_float(big);
        meet(pair, false);
        big = max(big, *reinterpret_cast<const volatile uint32_t*>(other));
        const int exponent = int(big >> 7), up = big == 0 || exponent == 255 ? 0 : min(14 - (exponent - 127), 126);
        mul = p.q_sign * __uint_as_float(uint32_t(127 + up) << 23);
        back = __uint_as_float(uint32_t(127 - up) << 23);
      } else {
        load(0);
      }
      const uint32_t sign = pack_f16(p.q_sign, p.q_sign);
#pragma unroll 1
      for (int j0 = 0; j0 < PARTS; j0 += HELD) {
        if (j0 > 0) load(j0);
#pragma unroll
        for (int j = 0; j < HELD; ++j) {
          uint32_t h[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
          for (int y = 0; y < 4; ++y)
            h[y] = p.bf16 ? pack_f16(__uint_as_float(h[y] << 16) * mul, __uint_as_float(h[y] & 0xffff0000u) * mul) : hmul2(h[y], sign);
          const int part = half * PARTS + j0 + j;
          const uint32_t dst = q_row_at + part / 8 * (128 * 128) + ((part % 8) ^ (row & 7)) * 16;
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
        }
      }
      x.factor = fmaxf(back * p.scale_log2, 1.17549435e-38f);
    }
    gvr::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) gvr::mbar_arrive(&bars->q_full[tile]);
  };

  Query x, x_next;
  begin_segment(x);
  while (x.steps > 0) {
    float top = NO_TOP, total = 0.f;
    for (int i = 0; i < x.tasks; ++i) {
      const int b = S::TILES == 2 ? tile : int(done & 1);
      wait(&bars->s_full[b], (S::TILES == 2 ? done : done >> 1) & 1);
      tc_fence_after();
      const int step = S::TILES == 1 || x.both ? i : 2 * i + tile;
      if (x.warp) {
        const uint32_t scores = tmem + lanes + S::S_AT + b * S::N + half * COLUMNS;
        const uint64_t factor = two_f32(__float_as_uint(x.factor), __float_as_uint(x.factor));
        uint32_t there[WORDS];  // entries that this query sees
        bool all = true;
        const int e0 = x.first + step * S::N;
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
          there[w] = *const_cast<const volatile uint32_t*>(&notes->steps[(steps + step) & (STEP_NOTES - 1)].there[half * WORDS + w]);
          const int seen = x.limit - (e0 + 32 * w);
          if (seen < 32) there[w] &= seen <= 0 ? 0u : (1u << seen) - 1;
          all &= there[w] == 0xffffffffu;
        }
        const bool whole = __all_sync(0xffffffffu, all || !x.live);
        auto mask = [&](int c, uint32_t(&s32)[32]) {
          if (!whole) {
            const uint32_t seen = c == 0 ? there[0] : there[WORDS - 1];
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(seen >> j & 1)) s32[j] = 0xff800000u;
          }
        };
        // (Loops stay loops here and in bring(): unrolled, the warps' code at a time is more than the instruction caches feed
        // four kinds of warps from.)
        float high[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int c = 0; c < WORDS; ++c) {
          uint32_t v[32];
          tmem_load(scores + 32 * c, v);
          tmem_load_wait();
          mask(c, v);
#pragma unroll
          for (int j = 0; j < 32; j += 2) high[j / 2 & 3] = max_three(high[j / 2 & 3], __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
        }
        float most = fmaxf(fmaxf(high[0], high[1]), fmaxf(high[2], high[3])) * x.factor;
        if (meet(pair, most > top + ABOVE)) {
          *mine = most;
          meet(pair, false);
          most = fmaxf(most, *const_cast<const volatile float*>(other));
          const float next_top = fmaxf(top, most - BELOW), down = exp2_fast(top - next_top);
          top = next_top, total *= down;
          if (i > 0) {  // O so far: all products of this tile are complete but for those that wait for this P
            wait_products();
            tc_fence_after();
#pragma unroll 1
            for (int c = half * (D / 32); c < (half + 1) * (D / 32); ++c) {
              uint32_t o[16];
              tmem_load(tmem + lanes + S::O_AT + tile * D + 16 * c, o);
              tmem_load_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * down);
              tmem_store(tmem + lanes + S::O_AT + tile * D + 16 * c, o);
            }
          }
        }
        const uint64_t base = two_f32(__float_as_uint(-top), __float_as_uint(-top));
        uint64_t part[2] = {0, 0};
#pragma unroll 1
        for (int c = 0; c < WORDS; ++c) {
          uint32_t v[32], h[16];
          tmem_load(scores + 32 * c, v);
          tmem_load_wait();
          mask(c, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint64_t e = exp2_two(fma_two(two_f32(v[2 * j], v[2 * j + 1]), factor, base));
            part[j & 1] = add_two(part[j & 1], e);
            h[j] = pack_f16(__uint_as_float(uint32_t(e)), __uint_as_float(uint32_t(e >> 32)));
          }
          tmem_store(scores + 16 * c, h);  // over scores that have been read
        }
        const uint64_t sum = add_two(part[0], part[1]);
        total += __uint_as_float(uint32_t(sum)) + __uint_as_float(uint32_t(sum >> 32));
        tmem_store_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) gvr::mbar_arrive(&bars->p_full[b]);
      ++done;
    }
    steps += x.steps;
    if (x.warp && half == 1) totals[tile * 128 + row] = total;
    begin_segment(x_next);  // meets the other warp; its Q may be laid down: this segment's products with Q are complete

    // ---- the piece
    if (x.warp) {
      uint32_t nan = 0;
      if (x.tasks > 0) {
        wait_products();
        tc_fence_after();
        nan = *const_cast<volatile uint32_t*>(nans + (segments % S::NAN_SLOTS * S::TILES + tile) * 128 + row);
      }
      if (half == 0 && x.live) {
        x.piece[int64_t(x.height) * D] = top;
        x.piece[int64_t(x.height) * (D + 1)] = total + *const_cast<const volatile float*>(totals + tile * 128 + row);
      }
      if (x.tasks > 0) {
        // four values of a query lie together, those of neighbouring queries next to each other
        float* to = x.piece + 3 * x.at;
#pragma unroll
        for (int c = half * (D / 64); c < (half + 1) * (D / 64); ++c) {
          uint32_t v[32];
          tmem_load(tmem + lanes + S::O_AT + tile * D + 32 * c, v);
          tmem_load_wait();
          if (nan) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (nan >> (2 * c + j / 16) & 1) v[j] = 0x7fc00000u;
          }
          if (x.live) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<uint4*>(to + int64_t(8 * c + j) * x.height * 4) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          }
        }
        tc_fence_before();
      }
      // both have read them before they are used again
      meet(pair, false);
      if (nan && half == 0) nans[(segments % S::NAN_SLOTS * S::TILES + tile) * 128 + row] = 0;
    }
    if (x.tasks > 0) ++segments;
    x = x_next;
  }
  return ok;
}

template <int REGS, bool MORE>
__device__ __forceinline__ void registers() {
  if (MORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

template <int D>
__global__ void __launch_bounds__(SharedShape<D>::THREADS, 1) shared_kernel(SharedParams p, const __grid_constant__ CUtensorMap map) {
  using S = SharedShape<D>;
  extern __shared__ uint8_t dynamic[];
  __shared__ SharedBars bars;
  __shared__ SharedNotes notes;
  __shared__ uint32_t tmem_at, nans[S::NAN_SLOTS * S::TILES * 128];
  __shared__ float exchange[S::TILES * 3 * 128];  // of the two threads of a query: maxima, sums
  const int tid = threadIdx.x;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t q_at = (gvr::smem_u32(dynamic) + 1023) & ~1023u, k_at = q_at + S::TILES * S::Q_BYTES, v_at = k_at + 2 * S::KV_BYTES, raw_at = v_at + S::KV_BYTES;
  const uint8_t* raw = dynamic + (raw_at - gvr::smem_u32(dynamic));
  if (tid == 0) {
    for (int i = 0; i < S::STAGES; ++i) gvr::mbar_init(&bars.raw_full[i], 1), gvr::mbar_init(&bars.raw_free[i], 8);
    for (int i = 0; i < 2; ++i) {
      gvr::mbar_init(&bars.k_full[i], 4), gvr::mbar_init(&bars.k_free[i], 1);
      gvr::mbar_init(&bars.v_full[i], 2), gvr::mbar_init(&bars.v_free[i], 1);
      gvr::mbar_init(&bars.q_full[i], 8), gvr::mbar_init(&bars.s_full[i], 1);
      gvr::mbar_init(&bars.p_full[i], 8), gvr::mbar_init(&bars.o_full[i], 1);
    }
    gvr::mbar_init(&bars.done, 1);
    for (int i = 0; i < SEGMENTS; ++i) gvr::mbar_init(&bars.seg_full[i], 1), gvr::mbar_init(&bars.seg_free[i], 8 * S::TILES + 1);
    gvr::mbar_init_fence();
  }
  for (int i = tid; i < S::NAN_SLOTS * S::TILES * 128; i += S::THREADS) nans[i] = 0;
  constexpr int BRINGERS = 8 * S::TILES, ISSUER = BRINGERS + 8, WALKER = ISSUER + 1;
  if (warp == ISSUER) tmem_alloc_all(gvr::smem_u32(&tmem_at));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  begin();
  const int4 held = *reinterpret_cast<const int4*>(p.plan);
  const Plan plan = {held.x, held.y, held.z, held.w};
  constexpr bool EXCHANGE = S::TILES == 2;
  bool ok;
  if (warp < BRINGERS) {
    if (EXCHANGE) registers<S::SOFT_REGS, true>();
    ok = soften<D>(p, &bars, tmem, q_at, warp, &notes, nans, exchange);
  } else if (warp < ISSUER) {
    if (EXCHANGE) registers<S::BRING_REGS, false>();
    const bool is_v = warp >= BRINGERS + 4;
    ok = bring<D>(p, &bars, raw, is_v ? v_at : k_at, (warp - BRINGERS) & 3, is_v, &notes, nans);
  } else {
    if (EXCHANGE) registers<S::REST_REGS, false>();
    ok = true;
    if (warp == ISSUER) {
      ok = multiply<D>(&bars, &notes, __shfl_sync(0xffffffffu, tmem, 0), q_at, k_at, v_at);
      if (elect_one()) tc_commit(&bars.done);  // whatever has been issued is complete before its memory is given up
      __syncwarp();
      ok &= warp_wait(&bars.done, 0);
    } else if (warp == WALKER) {
      ok = walk<D>(p, &map, plan, &notes, &bars, raw_at);
    }
  }
  if (!ok) p.plan->failed = 1;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == ISSUER) tmem_free_all(tmem);
}

// ------------------------------------------------------------------------------------------------ the join
constexpr int JOIN_ROWS = 16, JOIN_SHARED_THREADS = 256;  // queries and threads of a CTA
constexpr int JOIN_AT_ONCE = 8;                           // pieces under way
__host__ __device__ constexpr int join_width(int split) { return JOIN_SHARED_THREADS / JOIN_ROWS / split * 4; }  // dimensions of a CTA

// A piece, for the CTA's queries.
struct Listed {
  const float* piece;  // nullptr: none
  int height, at;      // its rows; that of the CTA's first query
};

// Pieces of a query at most: the units that it is in are cut where CTAs' shares end, and of each CTA it has up to two.
__host__ __device__ constexpr int join_pieces(int grid) { return 2 * (grid + 3) + TAIL_CHUNKS; }
__host__ __device__ constexpr int join_smem(int grid) { return join_pieces(grid) * (JOIN_ROWS * 8 + int(sizeof(Listed))); }

// blockIdx.x: requests x KV heads; y: JOIN_ROWS of the request's queries; z: dimensions, four a thread.  Neighbouring
// threads have neighbouring queries, as they lie in a piece.  The pieces of the CTA's queries are listed first, and each one's
// factor found, once for all dimensions; then a thread adds up its values of every SPLIT-th piece, JOIN_AT_ONCE loads under way.
template <int D, int SPLIT>
__global__ void __launch_bounds__(JOIN_SHARED_THREADS) shared_join_kernel(SharedParams p) {
  using S = SharedShape<D>;
  extern __shared__ __align__(16) uint8_t join_memory[];
  const int most = join_pieces(p.grid);
  float* factors = reinterpret_cast<float*>(join_memory);  // [most][JOIN_ROWS]: bases, then factors; -1: not this query's
  float* sums = factors + most * JOIN_ROWS;                // [most][JOIN_ROWS]
  Listed* list = reinterpret_cast<Listed*>(sums + most * JOIN_ROWS);
  __shared__ float tops[JOIN_ROWS], totals[JOIN_ROWS];
  __shared__ float4 parts[SPLIT == 1 ? 1 : JOIN_SHARED_THREADS];
  const int tid = threadIdx.x, lane = tid & 31, r = blockIdx.x / p.kv_heads, head = blockIdx.x - r * p.kv_heads;
  // queries of the request (the last one may have fewer rows: their units and pieces end with them)
  const int members = int(min(int64_t(p.next_n), p.num_rows - int64_t(r) * p.next_n)) * p.group, m0 = blockIdx.y * JOIN_ROWS;
  begin();
  if (m0 >= members) return;
  const int4 held = *reinterpret_cast<const int4*>(p.plan);
  const Plan plan = {held.x, held.y, held.z, held.w};
  const Joined join = p.joined[r];
  // ---- the list, by part: the prefix's unit of the first query, the unit behind that (the CTA's queries can lie in two),
  // and the request's own
  int count = 0, ends[3], border = members;  // queries from the border on are in the prefix's second unit
#pragma unroll
  for (int part = 0; part < 3; ++part) {
    const int which = part < 2 ? join.prefix : join.suffix;
    if (which >= 0) {
      const int4* from = reinterpret_cast<const int4*>(p.sets + which);
      const int4 a = from[0], b = from[1], c = from[2];
      const Set set = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
      const int offset = part < 2 ? (r * p.next_n - set.row0) * p.group : 0;  // of the request's queries in the set
      const int tile = (offset + m0) / S::QUERIES + (part == 1);
      if (part == 0) border = (tile + 1) * S::QUERIES - offset;
      if (part != 1 || border < min(m0 + JOIN_ROWS, members)) {
        const int unit = tile * p.kv_heads + head, both = unit < set.full;
        const int start = set.start + unit_start(unit, set.full, set.steps), work = unit_work(set.steps, both);
        const int c0 = share_of(start, plan.ctas, plan.total), c1 = share_of(start + work - 1, plan.ctas, plan.total);
        const int rows = part < 2 ? 128 : p.suffix_rows, height = S::TILES * rows;
        const int64_t floats = part < 2 ? S::PIECE : height * (D + 2);
        const int twice = S::TILES == 2 && !both;  // even steps in one tile, odd ones in the other
        const float* pieces = (part < 2 ? p.prefix_pieces : p.suffix_pieces) + int64_t(set.unit0 + unit) * floats;
        const int here = (c1 - c0 + 1) << twice;
        for (int x = tid; x < here; x += JOIN_SHARED_THREADS) {
          const int cta = c0 + (x >> twice), second = twice ? x & 1 : 0;
          const int lo = step_of(share_start(cta, plan.ctas, plan.total), start, both, set.steps);
          const int hi = step_of(share_start(cta + 1, plan.ctas, plan.total), start, both, set.steps);
          list[count + x] = {hi - lo > second ? pieces + int64_t(cta) * floats : nullptr, height, offset + m0 - tile * S::QUERIES + second * rows};
        }
        count += here;
      }
    }
    ends[part] = count;
  }
  const int chunks = (join.tail_steps + TAIL_CHUNK - 1) / TAIL_CHUNK;
  if (tid < chunks) list[count + tid] = {p.tail_pieces + (int64_t(blockIdx.x) * TAIL_CHUNKS + tid) * p.tail_height * (D + 2), p.tail_height, m0};
  count += chunks;
  __syncthreads();
  for (int i0 = tid; i0 < count * JOIN_ROWS; i0 += JOIN_AT_ONCE * JOIN_SHARED_THREADS) {
    float top[JOIN_AT_ONCE], sum[JOIN_AT_ONCE];
#pragma unroll
    for (int j = 0; j < JOIN_AT_ONCE; ++j) {
      const int i = i0 + j * JOIN_SHARED_THREADS, k = i / JOIN_ROWS, row = i % JOIN_ROWS, m = m0 + row;
      top[j] = NO_TOP, sum[j] = 0.f;
      if (k < count && m < members && (k >= ends[1] || (k >= ends[0]) == (m >= border)) && list[k].piece) {
        const float* at = list[k].piece + int64_t(list[k].height) * D + list[k].at + row;
        top[j] = at[0], sum[j] = at[list[k].height];
      }
    }
#pragma unroll
    for (int j = 0; j < JOIN_AT_ONCE; ++j) {
      const int i = i0 + j * JOIN_SHARED_THREADS;
      if (i < count * JOIN_ROWS) factors[i] = top[j], sums[i] = sum[j];
    }
  }
  __syncthreads();
  // ---- each query's base, factors and sum, by a warp, two queries each
  for (int row = tid >> 5; row < JOIN_ROWS; row += JOIN_SHARED_THREADS / 32) {
    float top = NO_TOP, total = 0.f;
    for (int k = lane; k < count; k += 32)
      if (sums[k * JOIN_ROWS + row] != 0.f) top = fmaxf(top, factors[k * JOIN_ROWS + row]);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    for (int k = lane; k < count; k += 32) {
      const float sum = sums[k * JOIN_ROWS + row], factor = exp2_fast(factors[k * JOIN_ROWS + row] - top);
      // a sum of 0 saw nothing there (and what it holds may be a NaN of entries that it does not see)
      factors[k * JOIN_ROWS + row] = sum == 0.f ? -1.f : factor;
      if (sum != 0.f) total += sum * factor;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    if (lane == 0) tops[row] = top, totals[row] = total;
  }
  __syncthreads();
  // ---- the values
  constexpr int WIDTH4 = join_width(SPLIT) / 4;
  const int row = tid % JOIN_ROWS, m = m0 + row, d4 = blockIdx.z * WIDTH4 + tid / JOIN_ROWS % WIDTH4, first = tid / (JOIN_ROWS * WIDTH4);
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k0 = first; k0 < count; k0 += SPLIT * JOIN_AT_ONCE) {
    float4 v[JOIN_AT_ONCE];
    float f[JOIN_AT_ONCE];
#pragma unroll
    for (int i = 0; i < JOIN_AT_ONCE; ++i) {
      const int k = k0 + i * SPLIT;
      f[i] = k < count ? factors[k * JOIN_ROWS + row] : -1.f;  // (a query behind the last one has none)
      if (f[i] >= 0.f) {
        const Listed l = list[k];
        v[i] = *reinterpret_cast<const float4*>(l.piece + (int64_t(d4) * l.height + l.at + row) * 4);
      }
    }
#pragma unroll
    for (int i = 0; i < JOIN_AT_ONCE; ++i)
      if (f[i] >= 0.f) acc[0] += f[i] * v[i].x, acc[1] += f[i] * v[i].y, acc[2] += f[i] * v[i].z, acc[3] += f[i] * v[i].w;
  }
  if (SPLIT > 1) {
    parts[tid] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (first > 0) return;
#pragma unroll
    for (int i = 1; i < SPLIT; ++i) {
      const float4 v = parts[tid + i * (JOIN_ROWS * WIDTH4)];
      acc[0] += v.x, acc[1] += v.y, acc[2] += v.z, acc[3] += v.w;
    }
  }
  if (m >= members) return;
  const int rel = m / p.group;
  const int64_t row_at = int64_t(r) * p.next_n + rel;
  const float total = plan.failed ? NAN : totals[row], norm = total == 0.f ? 0.f : 1.f / total;
  uint32_t packed[2];
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    // v_scale last: v_scale / total would lose bits, or all, of a small factor over many entries
    const float lo = acc[2 * y] * norm * p.v_scale, hi = acc[2 * y + 1] * norm * p.v_scale;
    if (p.bf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(packed[y]) : "f"(hi), "f"(lo));
    else packed[y] = pack_f16(lo, hi);
  }
  const int64_t at = row_at * (int64_t(p.kv_heads) * p.group) + head * p.group + (m - rel * p.group);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at * D + d4 * 4) = make_uint2(packed[0], packed[1]);
  if (p.lse && d4 == 0) p.lse[at] = total == 0.f ? -INFINITY : (tops[row] + log2f(total)) * 0.69314718055994531f;
}

// What the host needs to know of a head dimension's kernels.
struct SharedInfo {
  const void *plan, *kernel, *join[3];  // joins: of split 1, 4 and 16
  int threads, smem, queries, tiles, step, piece_floats;
  TailInfo (*tails)(int64_t members);
};
template <int D>
SharedInfo shared_info() {
  using S = SharedShape<D>;
  return {reinterpret_cast<const void*>(shared_plan_kernel<D>), reinterpret_cast<const void*>(shared_kernel<D>),
          {reinterpret_cast<const void*>(shared_join_kernel<D, 1>), reinterpret_cast<const void*>(shared_join_kernel<D, 4>),
           reinterpret_cast<const void*>(shared_join_kernel<D, 16>)}, S::THREADS, S::SMEM, S::QUERIES, S::TILES, S::N, S::PIECE, tails_of<D>};
}
SharedInfo shared_64();
SharedInfo shared_128();
SharedInfo shared_256();

}  // namespace gvrc
