// gvr_tails.cuh -- the entries behind a prefix, of attend_shared's requests that have few of them and few queries: what
// gvr_attend.cuh's walk does to a request's rows, from an entry on.
//
// A CTA has a request's queries of a KV head (up to Q of them: a tile) and a chunk of its entries; its warps take steps of 32 in
// turn, and their sums join in shared memory to one piece.  Products are mma.sync ones, 8 queries wide, as the queries are few.
#pragma once

#include "../csrc_cache/gvr_attend.cuh"

namespace gvrc {

// What a request's rows join.
struct __align__(16) Joined {
  int32_t suffix;                 // its set, -1: none
  int32_t prefix;                 // its group's, -1: none
  int32_t tail_first, tail_steps;  // its tail, in steps of 32 entries; 0: none
};

// Entries of a chunk, in steps, and chunks of a tail.  (64 requests of 2 rows, 8 KV heads of 128, 10 to 2000 entries each behind a
// prefix: 177 us with two chunks of 32 steps, 179 with one of 64, 185 with four of 16, 200 with eight of 8.)
constexpr int TAIL_CHUNK = 32, TAIL_CHUNKS = 2, TAIL_ENTRIES = TAIL_CHUNKS * TAIL_CHUNK * STEP;

struct TailParams {
  const Joined* joined;
  float* pieces;  // [requests][KV heads][TAIL_CHUNKS][D / 4][height][4], then bases and sums [height]
  int32_t height;  // queries, up to whole tiles
};

template <int D, int NT>
struct TailShape {
  using S = Shape<D, NT>;
  static constexpr int WARPS = D == 256 ? 2 : 4, THREADS = 32 * WARPS;  // (head_dim 256: for more CTAs an SM)
  static constexpr int PITCH = D + 4;                                   // floats of a query in shared memory
  static constexpr int JOIN = S::Q * (PITCH + 2) * 4;                   // of a warp
  static constexpr int SMEM = WARPS * (S::WALK > JOIN ? S::WALK : JOIN);
};

// blockIdx.x: requests x KV heads; y: tiles; z: chunks.
template <int D, int NT>
__global__ void __launch_bounds__(TailShape<D, NT>::THREADS, Shape<D, NT>::FOLD_BLOCKS) tails_kernel(AttendParams p, TailParams t) {
  using S = Shape<D, NT>;
  using T = TailShape<D, NT>;
  constexpr int KSTEPS = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int r = blockIdx.x / p.kv_heads, h = blockIdx.x - r * p.kv_heads, m0 = blockIdx.y * S::Q;
  begin();
  const int4 held = *reinterpret_cast<const int4*>(t.joined + r);
  const int first = held.z + int(blockIdx.z) * TAIL_CHUNK, steps = min(held.w - int(blockIdx.z) * TAIL_CHUNK, TAIL_CHUNK);
  if (steps <= 0) return;
  uint32_t raw[NT][D / 8];
  load_queries<D, NT, true>(p, r, h, m0, p.fold * p.group, raw);
  const Unit u = load_unit<true>(p, r);
  float o[NT][KSTEPS][4], top[NT][2], total[NT][2];
  walk<D, NT, true>(p, u, h, m0, first + warp, T::WARPS, steps > warp ? (steps - warp + T::WARPS - 1) / T::WARPS : 0, uint32_t(u.n), smem + warp * S::RING,
                    reinterpret_cast<uint32_t*>(smem + T::WARPS * S::RING) + warp * STEP, raw, o, top, total);
  copy_wait<0>();
  __syncthreads();  // the rings become the warps' sums
  float* partial = reinterpret_cast<float*>(smem);  // [WARPS][Q][PITCH]
  float* tops = partial + T::WARPS * S::Q * T::PITCH;  // [WARPS][Q]
  float* sums = tops + T::WARPS * S::Q;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int qi = 8 * n + 2 * c + j;
      float* dst = partial + (warp * S::Q + qi) * T::PITCH + g * (D / 8);
#pragma unroll
      for (int x = 0; x < KSTEPS; x += 2)
        *reinterpret_cast<float4*>(dst + 2 * x) = make_float4(o[n][x][j], o[n][x][j + 2], o[n][x + 1][j], o[n][x + 1][j + 2]);
      if (g == 0) tops[warp * S::Q + qi] = top[n][j], sums[warp * S::Q + qi] = total[n][j];
    }
  __syncthreads();
  float* piece = t.pieces + (int64_t(blockIdx.x) * TAIL_CHUNKS + blockIdx.z) * t.height * (D + 2);
  for (int i = tid; i < S::Q * D / 4; i += T::THREADS) {
    const int qi = i % S::Q, d4 = i / S::Q;
    float all = NO_TOP, sum = 0.f;
#pragma unroll
    for (int w = 0; w < T::WARPS; ++w)
      if (sums[w * S::Q + qi] != 0.f) all = fmaxf(all, tops[w * S::Q + qi]);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < T::WARPS; ++w) {
      const float own = sums[w * S::Q + qi];
      if (own == 0.f) continue;  // it saw nothing (and what it holds may be a NaN of entries that it does not see)
      const float down = exp2_fast(tops[w * S::Q + qi] - all);
      const float4 x = *reinterpret_cast<const float4*>(partial + (w * S::Q + qi) * T::PITCH + 4 * d4);
      sum += own * down, v.x += x.x * down, v.y += x.y * down, v.z += x.z * down, v.w += x.w * down;
    }
    *reinterpret_cast<float4*>(piece + (int64_t(d4) * t.height + m0 + qi) * 4) = v;
    if (d4 == 0) piece[int64_t(t.height) * D + m0 + qi] = all, piece[int64_t(t.height) * (D + 1) + m0 + qi] = sum;
  }
}

struct TailInfo {
  const void* kernel;
  int queries, threads, smem;
};
template <int D, int NT>
TailInfo tail_info() {
  using T = TailShape<D, NT>;
  return {reinterpret_cast<const void*>(tails_kernel<D, NT>), Shape<D, NT>::Q, T::THREADS, T::SMEM};
}
// By the queries of a request and KV head.
template <int D>
TailInfo tails_of(int64_t members) {
  if constexpr (D == 64) return members <= 8 ? tail_info<64, 1>() : members <= 16 ? tail_info<64, 2>() : tail_info<64, 4>();
  else if constexpr (D == 128) return members <= 8 ? tail_info<128, 1>() : tail_info<128, 2>();
  else return tail_info<256, 1>();
}

}  // namespace gvrc
