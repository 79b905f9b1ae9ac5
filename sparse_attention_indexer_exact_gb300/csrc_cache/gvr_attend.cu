// gvr_attend.cu -- attend_decode and attend_prefill of include/gvr_cache.h: argument checks, launch shape
// and launch of the kernels of gvr_attend.cuh.
#include <algorithm>
#include <mutex>

#include "gvr_attend.cuh"

namespace gvrc {
namespace {

constexpr int MAX_WARPS = 4;           // of a CTA
// Equal shares (balanced_kernel) take a second kernel, 3 us.  Against clusters, 8 KV heads of 128: one request of
// 1024 entries 10.1 us against 8.2, of 1536 9.9 against 9.8, of 2048 10.2 against 11.4; 8 requests of up to 2048
// 14 against 12, 64 28.5 against 31.5.  400 of up to 2000, two rows each, 4 KV heads of 64: 57 against 73.
constexpr int BALANCED_STEPS = 48;     // of 32 entries, at least: k, or the table's width, as lengths are on the device
constexpr int BALANCED_UNITS = 1024;   // at most

const KernelInfo& kernel_info(int i) {
  static const KernelInfo all[KERNELS] = {attend_64(0), attend_64(1), attend_64(2), attend_128(0), attend_128(1), attend_256()};
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
  int warps[KERNELS][2] = {};     // resident per SM, as far as registers go
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
        for (const void* one : {k.kernel[f], k.balanced[f]}) {
          cudaFuncAttributes a;
          if (d.err == cudaSuccess) d.err = cudaFuncGetAttributes(&a, one);
          if (d.err == cudaSuccess)
            d.err = cudaFuncSetAttribute(one, cudaFuncAttributeMaxDynamicSharedMemorySize, most - int(a.sharedSizeBytes));
        }
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
  int64_t groups = 1;  // CTAs side by side for a unit
  float cost = 1e30f;
};

// Expected time in us of a launch, from what was measured over shapes of 1 to 700 rows and 512 to 131071
// entries: a step of each kernel beside w warps on its SM, what a warp does around its steps, what a join
// and what many CTAs cost.  (head_dim 128, 8 queries: 0.55 a step alone, 1.16 beside 8 warps,
// 2.03 beside 16, so more than 8 warps an SM gain little, and cost their start.  CTAs of eight warps were
// slower everywhere: their clusters spread less evenly over the SMs.)
struct Expected {
  float least, fixed, per_warp;
};
constexpr Expected STEP_US[KERNELS] = {{0.35f, 0.2f, 0.06f}, {0.5f, 0.4f, 0.07f}, {0.8f, 0.6f, 0.1f},
                                       {0.55f, 0.3f, 0.108f}, {0.8f, 0.8f, 0.1f}, {0.9f, 0.9f, 0.16f}};

struct Call {
  int kernel, kv_heads, tiles;
  int64_t units, steps;
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
  for (int cs = 1; cs <= MAX_CLUSTER && cs <= std::max<int64_t>(1, turns); ++cs) {
    const int64_t ctas = items * cs;
    const float own = float((turns + cs - 1) / cs);
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
    if (!call.listed) cost *= 1.f + 0.25f / float(cs);  // rows shorter than the table: the longest end last
    if (ctas > 1024) cost += 0.011f * float(ctas - 1024);
    if (cta_warps > jobs || cs > 1) cost += 0.7f;
    if (cost < g.cost) g.cost = cost, g.cluster = cs;
  }
  return g;
}

// The shape of balanced_kernel, or false where units are too short or many.
bool balanced_shape(const Device& d, const KernelInfo& info, int64_t units, int64_t steps, size_t workspace_bytes, AttendParams& p) {
  if (units > BALANCED_UNITS || steps < BALANCED_STEPS || units * steps > kIntMax / 2) return false;
  p.heads_in = p.kv_heads % 4 == 0 ? 4 : p.kv_heads % 2 == 0 ? 2 : 1;
  p.head_groups = p.kv_heads / p.heads_in;
  const int per_sm = std::min(info.balanced_warps / p.heads_in,
                              int(d.smem_per_sm / (p.heads_in * info.warp_smem + (units + 1) * 4 + d.smem_reserved)));
  const int64_t groups = int64_t(p.head_groups) * p.tiles, least = 3;  // steps worth a CTA
  const int64_t ctas = std::min(int64_t(d.sms) * per_sm / groups, units * steps / least);
  // units that are many against the CTAs fill the device without being cut
  if (ctas < 2 || units > 2 * ctas) return false;
  if ((ctas + units) * groups * p.heads_in * info.piece_bytes > int64_t(std::min<size_t>(workspace_bytes, size_t(1) << 40))) return false;
  p.balanced_ctas = int32_t(ctas);
  p.ways_log2 = 0;
  while (p.ways_log2 < 5 && (units << (p.ways_log2 + 2)) < ctas) ++p.ways_log2;  // up to four pieces a lane where units are equal
  return true;
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
  const bool fold = p.fold > 1;
  p.units = int32_t(units);
  void* args[] = {&p};
  if (workspace && balanced_shape(*d, info, units, steps, workspace_bytes, p)) {
    p.pieces = static_cast<float*>(workspace);
    const dim3 grid(uint32_t(p.balanced_ctas), uint32_t(p.head_groups * p.tiles));
    cudaError_t e = launch(info.balanced[fold], grid, 32 * p.heads_in, p.heads_in * info.warp_smem + int(units + 1) * 4, 1, args, stream);
    const int join_ctas = ((info.queries * cache->head_dim / 8 << p.ways_log2) + JOIN_THREADS - 1) / JOIN_THREADS;
    if (e == cudaSuccess) e = launch(info.join[fold], dim3(uint32_t(units), uint32_t(p.kv_heads * p.tiles), uint32_t(join_ctas)), JOIN_THREADS, 0, 1, args, stream);
    return e == cudaSuccess ? GVR_OK : GVR_ERR_LAUNCH;
  }
  const Call call = {kernel, p.kv_heads, p.tiles, units, steps, p.indices != nullptr,
                     cache->num_pages * cache->page_stride > (int64_t(2) << 30)};
  Geometry best;
  for (int warps = MAX_WARPS; warps >= 1; warps /= 2) {
    const Geometry g = plan(*d, info, d->warps[kernel][fold], call, warps);
    if (g.cost < best.cost) best = g;
  }
  p.heads_in = best.heads_in;
  p.tiles_in = best.tiles_in;
  p.head_groups = best.head_groups;
  p.tile_groups = best.tile_groups;
  p.split_log2 = best.split_log2;
  p.split = 1 << best.split_log2;
  const int jobs = p.heads_in * p.tiles_in, threads = 32 * jobs * p.split, smem = jobs * p.split * info.warp_smem, cs = best.cluster;
  const int64_t groups = best.groups;
  const dim3 grid(uint32_t(units * cs), uint32_t(groups));
  const cudaError_t e = launch(info.kernel[fold], grid, threads, smem, cs, args, stream);
  return e == cudaSuccess ? GVR_OK : GVR_ERR_LAUNCH;
}

gvr_status check_attend(const gvr_cache* cache, const void* q, int64_t q_row_stride, int64_t q_head_stride, int32_t dtype,
                        int64_t num_rows, int32_t num_heads, const int32_t* table, int64_t table_stride,
                        int64_t table_width, float scale, const void* out, const float* lse) {
  const gvr_status s = check_cache(cache);
  if (s != GVR_OK) return s;
  if ((dtype != GVR_BF16 && dtype != GVR_F16) || num_rows < 0 || num_heads < 1 || num_heads % cache->num_kv_heads != 0 ||
      num_heads > GVR_ATTEND_MAX_HEADS || !std::isfinite(float(double(scale) * cache->k_scale * 1.4426950408889634)) || table_width < 0 || table_width > kIntMax / cache->page_size)
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
  if (next_n < 1 || next_n > GVR_ATTEND_MAX_NEXT_N || compress_ratio < 1 || (indices && (k < 1 || k > kIntMax))) return GVR_ERR_ARG;
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
