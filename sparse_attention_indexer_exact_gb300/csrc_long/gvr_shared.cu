// gvr_shared.cu -- attend_shared of include/gvr_long.h: argument checks, workspace and launches of the kernels of
// gvr_shared.cuh.
#include <algorithm>
#include <mutex>

#include "gvr_shared.cuh"

namespace gvrc {
namespace {

const SharedInfo& shared_kernels(int dim) {
  static const SharedInfo all[3] = {shared_64(), shared_128(), shared_256()};
  return all[dim == 64 ? 0 : dim == 128 ? 1 : 2];
}

struct SharedDevice {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
};
SharedDevice g_shared_devices[kMaxDevices];

// Tails: at most so many tiles of queries, as each expands their entries anew; by a kernel of its own, which few requests are
// not worth.  128 requests over 3200 entries, 2880 of them common: 96 -> 69 us with 8 KV heads of 128 and 4 queries each,
// 48 -> 43 with 4 of 64 and 12; 32 requests over 12800: 60 -> 53; 64 of 2 rows behind 32000, 10 to 2000 of their own: 166 -> 165;
// By requests x KV heads, with and without tails: 54 (27 requests, heads of 256) 64 and 43 us, 96 (12, 128) 65 and 56, 100 (25, 64) 35 and 28,
// 192 (24, 128) 86 and 83, 196 (49, 64) 43.7 and 40.5, 256 (32, 128) 99 and 95, 256 (64, 64) 46 and 46, 512 (64, 128) 167 and 174.
constexpr int TAIL_TILES = 4, LEAST_TAILS = 256;
constexpr int64_t MAX_QUERIES = 1 << 26;  // of a KV head: their tiles' numbers share words with flags

// Where everything lies in the workspace.
struct Layout {
  int64_t plan, sets, joined, cta_set, cta_start, prefix, suffix, tails, bytes;
  int32_t suffix_rows, tail_tiles, tail_height;
};

int64_t align16(int64_t x) { return (x + 15) / 16 * 16; }

// The driver's encoder of tensor maps.
using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                            const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
Encode encoder() {
  static const Encode f = []() -> Encode {
    void* at = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &at, 12000, cudaEnableDefault, &found) != cudaSuccess || found != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<Encode>(at);
  }();
  return f;
}

// The cache as words [pages][entries][row words of all heads], copied by a head's rows of up to `step` entries of a page.
bool tensor_map(const gvr_cache* c, int step, CUtensorMap* map) {
  const Encode encode = encoder();
  const cuuint64_t row = row_bytes(c->head_dim), entry = row * c->num_kv_heads;
  const cuuint64_t size[3] = {entry / 4, cuuint64_t(c->page_size), cuuint64_t(c->num_pages)}, stride[2] = {entry, cuuint64_t(c->page_stride)};
  const cuuint32_t box[3] = {cuuint32_t(row / 4), cuuint32_t(std::min(c->page_size, step)), 1}, each[3] = {1, 1, 1};
  return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, c->data, size, stride, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Groups whose prefix is shared, at most: each has two requests.  (Callers may list many more, most of them empty.)
int64_t sharing_groups(int64_t groups, int64_t requests) { return std::min(groups, requests / 2); }

gvr_status layout(const SharedInfo& k, int dim, int64_t kv_heads, int64_t group, int64_t num_rows, int64_t next_n, int64_t groups, int64_t grid, Layout* l) {
  const int64_t requests = (num_rows + next_n - 1) / next_n, members = next_n * group;
  const int64_t tiles = (members + k.queries - 1) / k.queries, sharing = sharing_groups(groups, requests);
  // a group has its queries / k.queries tiles and at most one more
  const int64_t prefix_units = sharing > 0 ? kv_heads * (num_rows * group / k.queries + sharing) : 0;
  const int64_t suffix_units = requests * kv_heads * tiles;
  if (prefix_units > kIntMax / 2 || suffix_units > kIntMax / 2) return GVR_ERR_ARG;
  l->suffix_rows = int32_t(std::min<int64_t>(128, (members + 7) / 8 * 8));
  const int64_t suffix_floats = int64_t(k.tiles) * l->suffix_rows * (dim + 2);
  l->plan = 0;
  l->sets = align16(sizeof(Plan));
  l->joined = l->sets + align16((groups + requests) * int64_t(sizeof(Set)));
  l->cta_set = l->joined + align16(requests * int64_t(sizeof(Joined)));
  l->cta_start = l->cta_set + align16(grid * 4);
  l->prefix = l->cta_start + align16((grid + 1) * 4);
  l->suffix = l->prefix + (sharing > 0 ? (grid + prefix_units) * k.piece_floats * 4 : 0);
  l->tails = l->suffix + (grid + suffix_units) * suffix_floats * 4;
  const int32_t tail_queries = k.tails(members).queries;
  l->tail_tiles = int32_t((members + tail_queries - 1) / tail_queries);
  if (l->tail_tiles > TAIL_TILES || requests * kv_heads < LEAST_TAILS) l->tail_tiles = 0;
  l->tail_height = l->tail_tiles * tail_queries;
  l->bytes = l->tails + align16(requests * kv_heads * TAIL_CHUNKS * l->tail_height * (dim + 2) * 4);
  return GVR_OK;
}

// Whether attend_decode, which reads each request's entries by themselves, is expected to take less time, by the table's width, as the
// lengths are on the device.  Measured apart and together: 2 requests of 800 entries (8 KV heads of 128, 4 queries each) 8.5 and
// 19 us, 32 of 800 14 and 35, 128 of 3200 91 and 69, 32 of 12800 90 and 53; of 2 heads of 256, 32 of 3200 25 and 34, of 12800 64 and 47.
struct Expected {
  float rows[3];  // apart: us a million rows, for jobs of 8, 16 and 32 queries
  float step[2];  // together: us a step of a unit of one tile, of two
};
bool better_apart(const SharedInfo& k, int dim, const SharedParams& p, int64_t members, int64_t groups, bool tails, int sms) {
  const Expected x = dim == 64    ? Expected{{17.f, 24.f, 38.f}, {1.f, 1.85f}}
                     : dim == 128 ? Expected{{25.f, 37.f, 37.f}, {1.25f, 2.2f}}
                                  : Expected{{66.f, 66.f, 66.f}, {1.27f, 1.27f}};
  const int job = members <= 8 || dim == 256 ? 0 : members <= 16 || dim == 128 ? 1 : 2;  // as attend_decode chooses
  const int64_t tiles = (members + (8 << job) - 1) / (8 << job);
  if (p.kv_heads * tiles > 65535) return false;  // attend_decode refuses them
  const double apart = 8. + 1e-6 * x.rows[job] * double(p.requests) * double(p.kv_heads * tiles) * double(p.capacity);
  const int64_t sets = groups > 0 ? std::min<int64_t>(groups, p.requests) : p.requests, queries = (p.num_rows * p.group + sets - 1) / sets;
  const double units = double(sets) * double(p.kv_heads) * double((queries + k.queries - 1) / k.queries);
  const double steps = double((int64_t(p.capacity) + k.step - 1) / k.step);
  const double together = 20. + (tails ? 0.03 : 0.06) * double(p.requests) * double(p.kv_heads) + units * steps * x.step[queries > 128] / sms;
  return apart <= together;
}

}  // namespace
}  // namespace gvrc

extern "C" {

gvr_status attend_shared_workspace(int32_t num_kv_heads, int32_t head_dim, int64_t num_rows, int32_t num_heads,
                                   int32_t next_n, int64_t num_groups, size_t* bytes) {
  using namespace gvrc;
  if (!bytes) return GVR_ERR_NULL;
  if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || num_kv_heads < 1 || num_kv_heads > 65535 || num_rows < 0 || num_heads < 1 ||
      num_heads % num_kv_heads != 0 || num_heads > GVR_ATTEND_MAX_HEADS || next_n < 1 || next_n > GVR_ATTEND_MAX_NEXT_N ||
      int64_t(next_n) * (num_heads / num_kv_heads) > (1 << 19) || num_groups < 0 || num_groups > GVR_LONG_MAX_REQUESTS ||
      num_rows > int64_t(GVR_LONG_MAX_REQUESTS) * next_n || num_rows * (num_heads / num_kv_heads) > MAX_QUERIES)
    return GVR_ERR_ARG;
  int sms = 0;
  if (sm_count(&sms) != cudaSuccess) return GVR_ERR_LAUNCH;
  Layout l = {};
  const gvr_status s = layout(shared_kernels(head_dim), head_dim, num_kv_heads, num_heads / num_kv_heads, num_rows, next_n, num_groups, sms, &l);
  *bytes = size_t(l.bytes);
  return s;
}

gvr_status attend_shared_way(int32_t way, const gvr_cache* cache, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                             int32_t dtype, int64_t num_rows, int32_t num_heads, const int32_t* block_table,
                             int64_t table_stride, int64_t table_width, const int32_t* kv_lens, int32_t next_n,
                             int32_t compress_ratio, const int32_t* group_starts, const int32_t* prefix_entries,
                             int64_t num_groups, float scale, void* out, float* lse, void* workspace,
                             size_t workspace_bytes, void* stream) {
  using namespace gvrc;
  const gvr_status s = check_rows(cache, q, q_row_stride, q_head_stride, dtype, num_rows, num_heads, block_table, table_stride, table_width,
                                  kv_lens, next_n, compress_ratio, scale);
  if (s != GVR_OK) return s;
  if (num_groups < 0 || num_groups > GVR_LONG_MAX_REQUESTS || num_rows * (num_heads / cache->num_kv_heads) > MAX_QUERIES) return GVR_ERR_ARG;
  if (num_rows == 0) return GVR_OK;
  if (!out || (num_groups > 0 && (!group_starts || !prefix_entries))) return GVR_ERR_NULL;
  if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(group_starts, 4) || !aligned(prefix_entries, 4)) return GVR_ERR_ALIGN;
  const int dim = cache->head_dim, row = row_bytes(dim);
  const SharedInfo& k = shared_kernels(dim);
  SharedParams p = {};
  p.kv_heads = cache->num_kv_heads;
  p.group = num_heads / cache->num_kv_heads;
  p.capacity = cache->num_pages > 0 ? int32_t(table_width * cache->page_size) : 0;
  p.requests = int32_t((num_rows + next_n - 1) / next_n);
  // work is counted in 32 bits: each unit's steps, twice where two tiles take them, and what it costs beside
  const int64_t steps = (int64_t(p.capacity) + k.step - 1) / k.step + UNIT_WORK, members = int64_t(next_n) * p.group;
  const int64_t units = int64_t(p.kv_heads) * (num_rows * p.group / k.queries + sharing_groups(num_groups, p.requests) + p.requests * ((members + k.queries - 1) / k.queries));
  if (units > kIntMax / 2 || (steps > 0 && units > kIntMax / 2 / steps)) return GVR_ERR_ARG;
  int sms = 0, dev = 0;
  if (sm_count(&sms) != cudaSuccess || cudaGetDevice(&dev) != cudaSuccess) return GVR_ERR_LAUNCH;
  Layout l = {};
  const gvr_status fits = layout(k, dim, p.kv_heads, p.group, num_rows, next_n, num_groups, sms, &l);
  if (fits != GVR_OK) return fits;
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < size_t(l.bytes)) return GVR_ERR_WORKSPACE;
  p.num_rows = num_rows;
  if (way == WAY_APART || (way == WAY_BY_RULE && better_apart(k, dim, p, members, num_groups, l.tail_tiles > 0, sms)))
    return attend_decode(cache, q, q_row_stride, q_head_stride, dtype, num_rows, num_heads, block_table, table_stride, table_width, kv_lens, next_n,
                         compress_ratio, nullptr, 1, scale, out, lse, workspace, workspace_bytes, stream);
  SharedDevice& d = g_shared_devices[dev];  // sm_count has checked dev
  std::call_once(d.once, [&d, sms]() {
    for (int each : {64, 128, 256}) {
      const SharedInfo& i = shared_kernels(each);
      if (d.err == cudaSuccess) d.err = cudaFuncSetAttribute(i.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, i.smem);
      for (const void* join : i.join)
        if (d.err == cudaSuccess) d.err = cudaFuncSetAttribute(join, cudaFuncAttributeMaxDynamicSharedMemorySize, join_smem(sms));
      for (int64_t members : {8, 16, 32}) {
        const TailInfo t = i.tails(members);
        if (d.err == cudaSuccess) d.err = cudaFuncSetAttribute(t.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, t.smem);
      }
      if (d.err == cudaSuccess)
        d.err = cudaFuncSetAttribute(i.plan, cudaFuncAttributeMaxDynamicSharedMemorySize, (7 * GVR_LONG_MAX_REQUESTS + 1) * 4);
    }
  });
  if (d.err != cudaSuccess) return GVR_ERR_LAUNCH;
  p.data = static_cast<const uint8_t*>(cache->data);
  p.q = static_cast<const uint16_t*>(q);
  p.table = block_table;
  p.lens = kv_lens;
  p.group_starts = group_starts;
  p.prefix_entries = prefix_entries;
  p.out = out;
  p.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.plan = reinterpret_cast<Plan*>(ws + l.plan);
  p.sets = reinterpret_cast<Set*>(ws + l.sets);
  p.joined = reinterpret_cast<Joined*>(ws + l.joined);
  p.cta_set = reinterpret_cast<int32_t*>(ws + l.cta_set);
  p.cta_start = reinterpret_cast<int32_t*>(ws + l.cta_start);
  p.prefix_pieces = reinterpret_cast<float*>(ws + l.prefix);
  p.suffix_pieces = reinterpret_cast<float*>(ws + l.suffix);
  p.tail_pieces = reinterpret_cast<float*>(ws + l.tails);
  p.suffix_rows = l.suffix_rows;
  p.tail_height = l.tail_height;
  p.tail_entries = l.tail_tiles > 0 ? TAIL_ENTRIES : 0;
  p.q_row = q_row_stride;
  p.q_head = q_head_stride;
  p.table_stride = table_stride;
  p.unit = unit_bytes(cache->page_stride, row);
  p.page_units = uint32_t(cache->page_stride / p.unit);
  p.row_units = row / p.unit;
  p.entry_units = p.row_units * cache->num_kv_heads;
  p.num_pages = int32_t(cache->num_pages);
  p.page_shift = log2_of(cache->page_size);
  p.next_n = next_n;
  p.ratio = compress_ratio;
  p.bf16 = dtype == GVR_BF16;
  p.groups = int32_t(num_groups);
  p.grid = sms;
  p.scale_log2 = scale == 0.f ? 1.f : float(std::fabs(double(scale)) * cache->k_scale * 1.4426950408889634);
  p.q_sign = scale > 0.f ? 1.f : scale < 0.f ? -1.f : 0.f;
  p.v_scale = cache->v_scale;
  CUtensorMap map = {};
  if (p.page_shift >= 3 && p.num_pages > 0 && !tensor_map(cache, k.step, &map)) return GVR_ERR_LAUNCH;
  void* args[] = {&p, &map};
  const int plan_smem = int(5 * num_groups + 1 + 2 * p.requests) * 4;
  cudaError_t e = launch(k.plan, dim3(1), PLAN_THREADS, plan_smem, 1, args, stream);
  const int64_t tasks = int64_t(p.requests) * p.kv_heads;
  if (e == cudaSuccess && l.tail_tiles > 0) {
    AttendParams a = {};
    a.data = p.data, a.q = q, a.table = block_table, a.lens = kv_lens;
    a.q_row = p.q_row, a.q_head = p.q_head, a.table_stride = p.table_stride, a.num_rows = p.num_rows;
    a.unit = p.unit, a.page_units = p.page_units, a.entry_units = p.entry_units, a.row_units = p.row_units;
    a.num_pages = p.num_pages, a.page_shift = p.page_shift, a.kv_heads = p.kv_heads, a.group = p.group, a.fold = next_n, a.capacity = p.capacity;
    a.next_n = next_n, a.ratio = p.ratio, a.bf16 = p.bf16, a.scale_log2 = p.scale_log2, a.q_sign = p.q_sign;
    TailParams t = {p.joined, p.tail_pieces, p.tail_height};
    void* tail_args[] = {&a, &t};
    const TailInfo i = k.tails(members);
    e = launch(i.kernel, dim3(uint32_t(tasks), uint32_t(l.tail_tiles), TAIL_CHUNKS), i.threads, i.smem, 1, tail_args, stream);
  }
  if (e == cudaSuccess) e = launch(k.kernel, dim3(uint32_t(sms)), k.threads, k.smem, 1, args, stream);
  if (e == cudaSuccess) {
    const int64_t blocks = (members + JOIN_ROWS - 1) / JOIN_ROWS;
    // A value's pieces are shared out among 4 threads where CTAs are fewer than SMs (640 queries of one KV head behind 131071
    // entries 65.0 -> 61.5 us, two requests of 700 entries 20.0 -> 19.0; 196 and 216 CTAs took 3 us more), among 16 where
    // they are very few and the pieces can be many (8 queries of one KV head over 194560 entries 49 -> 40 us; with few pieces 2 us more).
    const int64_t ctas = tasks * blocks * (dim / join_width(1));
    const int which = ctas >= sms ? 0 : ctas * 8 < sms && p.capacity >= 64 * k.step ? 2 : 1, split = 1 << (2 * which);
    const dim3 grid(uint32_t(tasks), uint32_t(blocks), uint32_t(dim / join_width(split)));
    e = launch(k.join[which], grid, JOIN_SHARED_THREADS, join_smem(sms), 1, args, stream);
  }
  return e == cudaSuccess ? GVR_OK : GVR_ERR_LAUNCH;
}

gvr_status attend_shared(const gvr_cache* cache, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                         int32_t dtype, int64_t num_rows, int32_t num_heads, const int32_t* block_table,
                         int64_t table_stride, int64_t table_width, const int32_t* kv_lens, int32_t next_n,
                         int32_t compress_ratio, const int32_t* group_starts, const int32_t* prefix_entries,
                         int64_t num_groups, float scale, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
  return attend_shared_way(gvrc::WAY_BY_RULE, cache, q, q_row_stride, q_head_stride, dtype, num_rows, num_heads, block_table, table_stride,
                           table_width, kv_lens, next_n, compress_ratio, group_starts, prefix_entries, num_groups, scale, out, lse,
                           workspace, workspace_bytes, stream);
}

}  // extern "C"
