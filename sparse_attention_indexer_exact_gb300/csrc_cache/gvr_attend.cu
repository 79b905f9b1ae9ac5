// gvr_attend.cu -- attention over the 4-bit paged cache, at the selected entries or over all of a
// row's entries (attend_decode and attend_prefill of include/gvr_cache.h).
//
// Mathematics.  For a query vector q of one head and entries e with keys k_e and values v_e,
//   s_e = scale q.k_e,  o = sum_e exp(s_e - m) v_e / sum_e exp(s_e - m),  lse = m + log sum_e ...
// in one pass over the entries with a running maximum m and running sums that are rescaled when m
// grows, in any grouping of the entries: groups join by the same rescaling.
//
// Work split.  An item is one KV head and up to 8 NT query vectors that read the same entries: the
// query heads of the group (for whole-cache decode, those of all next_n rows of the request).  A
// cluster of CTAs takes an item; each of its warps walks over its own steps of 32 entries with its
// own running state, without any CTA barrier; warps join through shared memory, CTAs through
// distributed shared memory.  So a call is one launch with no workspace and a fixed order of sums.
//
// A step.  32 rows (codes and scales of K and V, 144 bytes at head_dim 128) arrive in the warp's
// ring by 16-byte asynchronous copies, STAGES - 1 steps ahead; rows of skipped entries are filled
// with zeros.  S^T = K Q^T and O^T += V^T P^T run on m16n8k16 matrix instructions with entries
// (for S) and head dimensions (for O) on the 16-row side: these have the 4-bit operand, expanded
// in registers straight into the instruction's operand layout, so nothing expanded is ever stored.
// e2m1 * e4m3 has at most 5 significant bits and an exponent within f16's, so K and V are exact
// in f16.  Queries are brought to f16 exactly, too: a power of two per query puts its largest
// element at 2^14, and what f16 cannot hold below that is under 2^-39 of it.  P is rounded to f16
// (11 bits): eight times finer than the 16-bit outputs' bf16 and averaged over the entries.
#include <mutex>

#include "gvr_cache_common.cuh"
#include "../csrc/gvr_device.cuh"

namespace gvrc {
namespace {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int STEP = 32;  // entries per step: one per lane
constexpr int MAX_CLUSTER = 8;

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
  int64_t page_stride, q_row, q_head, table_stride, num_rows, k;
  int32_t num_pages, page_shift, kv_heads, group, fold, tiles, capacity, next_n, ratio, num_requests, bf16;
  float scale_log2;  // scale * k_scale * log2(e)
  float v_scale;
};

// Row r of a 16-entry matrix tile <-> entry of the 16 (a permutation).  Even and odd entries
// separate, and neighbouring rows four apart modulo 8: with row pitches of 80, 144 and 288 bytes
// the operand reads of K (two neighbouring tile rows a phase) and of V (every other tile row)
// then fall on different shared-memory banks.
__device__ __forceinline__ int tile_entry(int r) {
  const int x = r & 7, e = (x & 1) ? 8 + ((x + 3) & 7) : x;
  return e + (r >> 3);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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
  static constexpr int CHUNKS = RB / 16;  // 16-byte pieces of a row
  static constexpr int STAGES = D == 256 ? 3 : 4;
  static constexpr int STAGE_BYTES = STEP * RB;
  static constexpr int RING = WARPS * STAGES * STAGE_BYTES;
  static constexpr int Q = 8 * NT;  // query vectors of an item
  static constexpr int JOIN = (WARPS * Q * D + 3 * WARPS * Q) * int(sizeof(float));
  static constexpr int OFFSETS = WARPS * STEP * 8;
  static constexpr int SMEM = (RING > JOIN ? RING : JOIN) + OFFSETS;
};

template <int D, int NT>
__global__ void __launch_bounds__(THREADS) attend_kernel(AttendParams p) {
  using S = Shape<D, NT>;
  constexpr int STAGES = S::STAGES;
  constexpr int KSTEPS = D / 16;       // 16-wide steps of the head dimension
  constexpr int KW = D / 32;           // 32-bit words of K codes per lane and entry
  constexpr int VW = D / 64;           // the same of V codes
  extern __shared__ __align__(128) uint8_t smem[];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const uint32_t rank = gvr::cluster_rank(), cs = gvr::cluster_size();
  int64_t item = blockIdx.x / cs;
  const int h = int(item % p.kv_heads);
  item /= p.kv_heads;
  const int tile = int(item % p.tiles);
  const int64_t unit = item / p.tiles;  // a row, or (whole-cache decode) a request's next_n rows

  // ---- the item's entries: request and number of valid ones
  int64_t request;
  int n = 0;        // entries that some row of the item sees
  int kv = 0;
  if (p.requests) {
    request = p.requests[unit];
    if (request >= 0 && request < p.num_requests) {
      n = window_entries(p.starts[unit], p.ends[unit], p.capacity);
    } else {
      request = 0;
    }
  } else {
    request = p.fold > 1 ? unit : unit / p.next_n;
    kv = p.lens[request];
    const int last = p.fold > 1 ? p.next_n - 1 : int(unit % p.next_n);
    n = decode_entries(kv, p.next_n, last, p.ratio, p.capacity);
  }
  const int32_t* table = p.table + request * p.table_stride;
  const int32_t* indices = p.indices ? p.indices + unit * p.k : nullptr;
  const int64_t listed = indices ? (n > 0 ? p.k : 0) : n;  // positions to walk over
  const int steps = int((listed + STEP - 1) / STEP);
  const int walkers = int(cs) * WARPS, me = int(rank) * WARPS + warp;
  const int mine = steps > me ? (steps - me + walkers - 1) / walkers : 0;

  // ---- the item's queries as operands: lane (g, c) holds query 8 t + g at D/4 c + [0, D/4)
  const int m0 = tile * S::Q;
  const int members = p.fold * p.group;
  uint32_t qb[NT][KSTEPS][2];
  float factor[NT][2];  // of the scores of queries 8 t + 2 c, 8 t + 2 c + 1: to log2 units
  int limit[NT][2];     // entries that these queries see
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int m = m0 + 8 * t + g;
    const int64_t row = unit * p.fold + m / p.group;
    const bool live = m < members && row < p.num_rows;
    uint32_t raw[D / 8];
    if (live) {
      const uint16_t* src = static_cast<const uint16_t*>(p.q) + row * p.q_row + int64_t(h * p.group + m % p.group) * p.q_head + c * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i);
        raw[4 * i] = v.x, raw[4 * i + 1] = v.y, raw[4 * i + 2] = v.z, raw[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) raw[i] = 0;
    }
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const float2 v = p.bf16 ? make_float2(__uint_as_float(raw[i] << 16), __uint_as_float(raw[i] & 0xffff0000u))
                              : f16x2_to_f32(raw[i]);
      big = fmaxf(big, fmaxf(fabsf(v.x), fabsf(v.y)));
    }
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    // 2^up with up = 14 - exponent(big); no scaling of zero or infinite queries
    int up = 14 - (int(__float_as_uint(big) >> 23) - 127);
    up = big == 0.f || up < -113 ? 0 : min(up, 126);
    const float mul = __uint_as_float(uint32_t(127 + up) << 23), back = __uint_as_float(uint32_t(127 - up) << 23);
#pragma unroll
    for (int s = 0; s < KSTEPS; ++s)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t w = raw[2 * s + j];
        const float2 v = p.bf16 ? make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)) : f16x2_to_f32(w);
        qb[t][s][j] = pack_f16(v.x * mul, v.y * mul);
      }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      factor[t][j] = __shfl_sync(0xffffffffu, back, (2 * c + j) * 4) * p.scale_log2;
      const int mm = m0 + 8 * t + 2 * c + j;
      limit[t][j] = p.fold > 1 ? decode_entries(kv, p.next_n, min(mm / p.group, p.fold - 1), p.ratio, p.capacity) : n;
    }
  }
  // entries below this are seen by every query of the item
  const int sure = p.fold > 1 ? decode_entries(kv, p.next_n, 0, p.ratio, p.capacity) : n;

  // ---- the walk
  uint8_t* ring = smem + warp * STAGES * S::STAGE_BYTES;
  int64_t* offsets = reinterpret_cast<int64_t*>(smem + S::SMEM - S::OFFSETS) + warp * STEP;

  auto load_entry = [&](int i) -> int {  // this lane's entry in my i-th step (-1: none)
    if (i >= mine) return -1;
    const int64_t pos = int64_t(me + i * walkers) * STEP + lane;
    if (pos >= listed) return -1;
    const int e = indices ? __ldg(indices + pos) : int(pos);
    return e < n ? e : -1;
  };
  auto load_page = [&](int e) -> int { return e >= 0 ? __ldg(table + (e >> p.page_shift)) : -1; };
  // issue the copies of a step; returns which lanes' entries exist
  auto issue = [&](int i, int e, int page) -> uint32_t {
    const int64_t off = row_offset(page, p.num_pages, e, p.page_shift, p.page_stride, p.kv_heads, h, S::RB);
    offsets[lane] = off;
    const uint32_t mask = __ballot_sync(0xffffffffu, off >= 0);
    __syncwarp();
    if (i < mine) {
      const uint32_t dst = gvr::smem_u32(ring + (i % STAGES) * S::STAGE_BYTES);
#pragma unroll
      for (int j = 0; j < S::CHUNKS; ++j) {
        const int id = j * 32 + lane, row = id / S::CHUNKS, part = id % S::CHUNKS;
        const int64_t o = offsets[row];
        copy16(dst + id * 16, p.data + (o < 0 ? 0 : o + part * 16), o < 0 ? 0 : 16);
      }
    }
    copy_commit();
    __syncwarp();
    return mask;
  };

  float o[NT][KSTEPS][4];
  float top[NT][2], total[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int i = 0; i < KSTEPS; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[t][i][j] = 0.f;
    top[t][0] = top[t][1] = -INFINITY;
    total[t][0] = total[t][1] = 0.f;
  }

  uint32_t masks[STAGES];
  {
    int e[STAGES + 1];
#pragma unroll
    for (int i = 0; i < STAGES + 1; ++i) e[i] = load_entry(i);
    int pg[STAGES - 1];
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) pg[i] = load_page(e[i]);
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) masks[i] = issue(i, e[i], pg[i]);
    masks[STAGES - 1] = 0;
    // carried: entry and page of step STAGES - 1, entry of step STAGES
    int e_next = e[STAGES - 1], e_after = e[STAGES];
    int pg_next = load_page(e_next);

    for (int i = 0; i < mine; ++i) {
      copy_wait<STAGES - 2>();
      __syncwarp();
      masks[STAGES - 1] = issue(i + STAGES - 1, e_next, pg_next);
      e_next = e_after;
      pg_next = load_page(e_next);
      e_after = load_entry(i + STAGES + 1);

      const uint8_t* st = ring + (i % STAGES) * S::STAGE_BYTES;
      const uint32_t mask = masks[0];
#pragma unroll
      for (int j = 0; j < STAGES - 1; ++j) masks[j] = masks[j + 1];

      // S^T: two tiles of 16 entries
      float s[2][NT][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const uint8_t* r0 = st + (16 * mt + tile_entry(g)) * S::RB;
        const uint8_t* r1 = st + (16 * mt + tile_entry(g + 8)) * S::RB;
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
          const uint32_t x0 = __byte_perm(two0, two0, block & 1 ? 0x3232 : 0x1010), x1 = __byte_perm(two1, two1, block & 1 ? 0x3232 : 0x1010);
#pragma unroll
          for (int j = 0; j < 4; ++j) a[j] = hmul2(a[j], x0), b[j] = hmul2(b[j], x1);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma(s[mt][t], a[0], b[0], a[1], b[1], qb[t][2 * w][0], qb[t][2 * w][1]);
            mma(s[mt][t], a[2], b[2], a[3], b[3], qb[t][2 * w + 1][0], qb[t][2 * w + 1][1]);
          }
        }
      }

      // to log2 units; entries that are skipped or beyond a query's limit leave the sums
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[mt][t][j] *= factor[t][j & 1];
      const int first = (me + i * walkers) * STEP;
      if (mask != 0xffffffffu || (p.fold > 1 && first > sure - STEP)) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = 16 * mt + tile_entry(g + 8 * (j >> 1));
            const bool there = (mask >> at) & 1;
#pragma unroll
            for (int t = 0; t < NT; ++t)
              if (!there || (p.fold > 1 && first + at >= limit[t][j & 1])) s[mt][t][j] = -INFINITY;
          }
      }

      // running maximum: kept while the step's maximum is at most 2^8 above it (P stays within f16)
      bool grow = false;
      float high[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v = fmaxf(fmaxf(s[0][t][j], s[0][t][j + 2]), fmaxf(s[1][t][j], s[1][t][j + 2]));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
          high[t][j] = v;
          grow |= v > top[t][j] + 8.f;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float down[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float next = fmaxf(top[t][j], high[t][j]);
            down[j] = top[t][j] == -INFINITY ? 0.f : exp2_fast(top[t][j] - next);
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
        const float base0 = top[t][0] == -INFINITY ? 0.f : top[t][0], base1 = top[t][1] == -INFINITY ? 0.f : top[t][1];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const float e0 = exp2_fast(s[mt][t][0] - base0), e1 = exp2_fast(s[mt][t][1] - base1);
          const float e2 = exp2_fast(s[mt][t][2] - base0), e3 = exp2_fast(s[mt][t][3] - base1);
          total[t][0] += e0 + e2;
          total[t][1] += e1 + e3;
          pb[mt][t][0] = transpose8x8(pack_f16(e0, e1));
          pb[mt][t][1] = transpose8x8(pack_f16(e2, e3));
        }
      }

      // O^T += V^T P^T: lane (g, c) expands V at D/8 g + [0, D/8) of four entries of each tile
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t v[4][VW], vs[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint8_t* r = st + (16 * mt + tile_entry(2 * c + (x & 1) + 8 * (x >> 1))) * S::RB;
          load_words<VW>(r + D / 2 + g * (D / 16), v[x]);
          if (D == 64) vs[x] = r[D + D / 16 + (g >> 1)];
          else if (D == 128) vs[x] = r[D + D / 16 + g];
          else vs[x] = *reinterpret_cast<const uint16_t*>(r + D + D / 16 + 2 * g);
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
            for (int t = 0; t < NT; ++t) mma(o[t][4 * w + b], a0, a1, a2, a3, pb[mt][t][0], pb[mt][t][1]);
          }
        }
      }
    }
  }
  copy_wait<0>();
  __syncthreads();  // the ring becomes the warps' partial results

  // ---- join the warps, then the CTAs
  float* part = reinterpret_cast<float*>(smem);           // [WARPS][Q][D]
  float* tops = part + WARPS * S::Q * D;                  // [WARPS][Q]
  float* sums = tops + WARPS * S::Q;                      // [WARPS][Q]
  float* joined = sums + WARPS * S::Q;                    // [2][Q]: the CTA's maximum and sum
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float v = total[t][j];
      v += __shfl_xor_sync(0xffffffffu, v, 4);
      v += __shfl_xor_sync(0xffffffffu, v, 8);
      v += __shfl_xor_sync(0xffffffffu, v, 16);
      if (g == 0) {
        tops[warp * S::Q + 8 * t + 2 * c + j] = top[t][j];
        sums[warp * S::Q + 8 * t + 2 * c + j] = v;
      }
    }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int qi = 8 * t + 2 * c + j;
      float all = -INFINITY;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) all = fmaxf(all, tops[w * S::Q + qi]);
      const float down = top[t][j] == -INFINITY ? 1.f : exp2_fast(top[t][j] - all);
      float* dst = part + (warp * S::Q + qi) * D + g * (D / 8);
#pragma unroll
      for (int x = 0; x < KSTEPS; ++x)
        *reinterpret_cast<float2*>(dst + 2 * x) = make_float2(o[t][x][j] * down, o[t][x][j + 2] * down);
      if (warp == 0 && g == 0) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const float tw = tops[w * S::Q + qi];
          sum += sums[w * S::Q + qi] * (tw == -INFINITY ? 1.f : exp2_fast(tw - all));
        }
        joined[qi] = all;
        joined[S::Q + qi] = sum;
      }
    }
  __syncthreads();
  if (cs > 1) {
    // the CTA's own sum over its warps, in place of warp 0's part, for the other CTAs to read
    for (int i = tid; i < S::Q * D / 4; i += THREADS) {
      float4* at = reinterpret_cast<float4*>(part) + i;
      float4 sum = *at;
#pragma unroll
      for (int w = 1; w < WARPS; ++w) {
        const float4 v = at[w * S::Q * D / 4];
        sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
      }
      *at = sum;
    }
    gvr::cluster_sync();
  }
  const uint32_t part_addr = gvr::smem_u32(part), joined_addr = gvr::smem_u32(joined);
  // each CTA of the cluster finishes its share of the queries x head dimension, eight values a thread
  constexpr int EIGHTS = D / 8;
  for (int i = int(rank) * THREADS + tid; i < S::Q * EIGHTS; i += int(cs) * THREADS) {
    const int qi = i / EIGHTS, d = (i % EIGHTS) * 8;
    const int m = m0 + qi;
    const int64_t row = unit * p.fold + m / p.group;
    if (m >= members || row >= p.num_rows) continue;
    float all, sum = 0.f, acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    if (cs == 1) {
      all = joined[qi], sum = joined[S::Q + qi];
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float4* src = reinterpret_cast<const float4*>(part + (w * S::Q + qi) * D + d);
        const float4 a = src[0], b = src[1];
        acc[0] += a.x, acc[1] += a.y, acc[2] += a.z, acc[3] += a.w, acc[4] += b.x, acc[5] += b.y, acc[6] += b.z, acc[7] += b.w;
      }
    } else {
      all = -INFINITY;
      for (uint32_t r = 0; r < cs; ++r) all = fmaxf(all, __uint_as_float(gvr::dsmem_ld_u32(gvr::dsmem_map(joined_addr + qi * 4, r))));
      for (uint32_t r = 0; r < cs; ++r) {
        const float tr = __uint_as_float(gvr::dsmem_ld_u32(gvr::dsmem_map(joined_addr + qi * 4, r)));
        const float down = tr == -INFINITY ? 1.f : exp2_fast(tr - all);
        sum += down * __uint_as_float(gvr::dsmem_ld_u32(gvr::dsmem_map(joined_addr + (S::Q + qi) * 4, r)));
#pragma unroll
        for (int j = 0; j < 8; ++j)
          acc[j] += down * __uint_as_float(gvr::dsmem_ld_u32(gvr::dsmem_map(part_addr + ((qi * D) + d + j) * 4, r)));
      }
    }
    const float norm = sum == 0.f ? 0.f : p.v_scale / sum;
    uint32_t packed[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float lo = acc[2 * j] * norm, hi = acc[2 * j + 1] * norm;
      if (p.bf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(packed[j]) : "f"(hi), "f"(lo));
      else packed[j] = pack_f16(lo, hi);
    }
    const int64_t head = row * (int64_t(p.kv_heads) * p.group) + h * p.group + m % p.group;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + head * D + d) = make_uint4(packed[0], packed[1], packed[2], packed[3]);
    if (p.lse && d == 0) p.lse[head] = sum == 0.f ? -INFINITY : (all + log2f(sum)) * 0.69314718055994531f;
  }
  if (cs > 1) gvr::cluster_sync();  // no CTA leaves while another reads its shared memory
}

// ------------------------------------------------------------------------------------- host
struct KernelInfo {
  const void* kernel;
  int smem;
  int queries;
};

template <int D, int NT>
KernelInfo info() {
  return {reinterpret_cast<const void*>(attend_kernel<D, NT>), Shape<D, NT>::SMEM, 8 * NT};
}

constexpr int KERNELS = 6;
const KernelInfo& kernel_info(int i) {
  static const KernelInfo all[KERNELS] = {info<64, 1>(), info<64, 2>(), info<64, 4>(), info<128, 1>(), info<128, 2>(), info<256, 1>()};
  return all[i];
}

// Fewest passes over the entries, then fewest query vectors: 8, 16 or 32 of them a pass, as far as
// the accumulators (head_dim / 16 x 4 registers for each 8) leave room.
int choose_kernel(int dim, int members) {
  if (dim == 64) return members <= 8 ? 0 : members <= 16 ? 1 : 2;
  if (dim == 128) return members <= 8 ? 3 : 4;
  return 5;
}

struct Device {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
  int resident[KERNELS] = {};  // CTAs on the whole device
};
Device g_devices[kMaxDevices];

cudaError_t resident_ctas(int kernel, int* ctas) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  Device& d = g_devices[dev];  // sm_count has checked dev
  std::call_once(d.once, [&d, sms]() {
    for (int i = 0; i < KERNELS && d.err == cudaSuccess; ++i) {
      const KernelInfo& k = kernel_info(i);
      d.err = cudaFuncSetAttribute(k.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
      if (d.err == cudaSuccess) d.err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&d.resident[i], k.kernel, THREADS, k.smem);
      d.resident[i] *= sms;
    }
  });
  *ctas = d.resident[kernel];
  return d.err;
}

gvr_status attend(const gvr_cache* cache, AttendParams& p, int64_t q_row_stride, int64_t q_head_stride, int32_t dtype,
                  int64_t num_rows, int32_t num_heads, int64_t table_stride, int64_t table_width, int64_t k, float scale,
                  void* stream) {
  const int group = num_heads / cache->num_kv_heads;
  // with no pages every copy is of 0 bytes: from any valid address
  p.data = static_cast<const uint8_t*>(cache->num_pages > 0 ? cache->data : p.q);
  p.page_stride = cache->page_stride;
  p.q_row = q_row_stride;
  p.q_head = q_head_stride;
  p.table_stride = table_stride;
  p.num_rows = num_rows;
  p.k = k;
  p.num_pages = int32_t(cache->num_pages);
  p.page_shift = log2_of(cache->page_size);
  p.kv_heads = cache->num_kv_heads;
  p.group = group;
  p.capacity = int32_t(table_width * cache->page_size);
  p.bf16 = dtype == GVR_BF16;
  p.scale_log2 = float(double(scale) * cache->k_scale * 1.4426950408889634);
  p.v_scale = cache->v_scale;
  // whole-cache decode: the rows of a request read the same entries, so they share an item
  p.fold = p.indices ? 1 : p.next_n;
  const int64_t members = int64_t(p.fold) * group;
  if (members > kIntMax) return GVR_ERR_ARG;
  const int kernel = choose_kernel(cache->head_dim, int(members > 64 ? 64 : members));
  const KernelInfo& info = kernel_info(kernel);
  p.tiles = int32_t((members + info.queries - 1) / info.queries);
  const int64_t units = (num_rows + p.fold - 1) / p.fold;
  if (units > kIntMax / p.tiles / p.kv_heads / MAX_CLUSTER) return GVR_ERR_ARG;
  const int64_t items = units * p.tiles * p.kv_heads;
  int resident = 0;
  if (resident_ctas(kernel, &resident) != cudaSuccess) return GVR_ERR_LAUNCH;
  // CTAs per item: until the device is full, while each warp keeps a step
  const int64_t most = p.indices ? k : p.capacity;
  int cs = 1;
  while (cs < MAX_CLUSTER && items * cs < resident && int64_t(cs) * 2 * WARPS * STEP <= most) cs *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(uint32_t(items * cs));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = size_t(info.smem);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = uint32_t(cs);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {&p};
  return cudaLaunchKernelExC(&cfg, info.kernel, args) == cudaSuccess ? GVR_OK : GVR_ERR_LAUNCH;
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
                         const int32_t* indices, int64_t k, float scale, void* out, float* lse, void* stream) {
  using namespace gvrc;
  const gvr_status s = check_attend(cache, q, q_row_stride, q_head_stride, dtype, num_rows, num_heads, block_table,
                                    table_stride, table_width, scale, out, lse);
  if (s != GVR_OK) return s;
  if (next_n < 1 || next_n > 4096 || compress_ratio < 1 || (indices && (k < 1 || k > kIntMax))) return GVR_ERR_ARG;
  if (num_rows == 0) return GVR_OK;
  if (!kv_lens) return GVR_ERR_NULL;
  if (!aligned(kv_lens, 4) || !aligned(indices, 4)) return GVR_ERR_ALIGN;
  AttendParams p = {};
  p.q = q;
  p.table = block_table;
  p.lens = kv_lens;
  p.indices = indices;
  p.out = out;
  p.lse = lse;
  p.next_n = next_n;
  p.ratio = compress_ratio;
  return attend(cache, p, q_row_stride, q_head_stride, dtype, num_rows, num_heads, table_stride, table_width, k, scale, stream);
}

gvr_status attend_prefill(const gvr_cache* cache, const void* q, int64_t q_row_stride, int64_t q_head_stride, int32_t dtype,
                          int64_t num_rows, int32_t num_heads, const int32_t* block_table, int64_t table_stride,
                          int64_t table_width, int64_t num_requests, const int32_t* row_requests, const int32_t* row_starts,
                          const int32_t* row_ends, const int32_t* indices, int64_t k, float scale, void* out, float* lse,
                          void* stream) {
  using namespace gvrc;
  const gvr_status s = check_attend(cache, q, q_row_stride, q_head_stride, dtype, num_rows, num_heads, block_table,
                                    table_stride, table_width, scale, out, lse);
  if (s != GVR_OK) return s;
  if (num_requests < 0 || num_requests > kIntMax || k < 1 || k > kIntMax) return GVR_ERR_ARG;
  if (num_rows == 0) return GVR_OK;
  if (!row_requests || !row_starts || !row_ends || !indices) return GVR_ERR_NULL;
  if (!aligned(row_requests, 4) || !aligned(row_starts, 4) || !aligned(row_ends, 4) || !aligned(indices, 4)) return GVR_ERR_ALIGN;
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
  return attend(cache, p, q_row_stride, q_head_stride, dtype, num_rows, num_heads, table_stride, table_width, k, scale, stream);
}

}  // extern "C"
