// gvr_cache_common.cuh -- what the cache kernels share: the argument checks of a gvr_cache, its
// row layout, and the conversions between 16-bit values, e2m1 codes and e4m3 scales.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "gvr_cache.h"
#include "gvr_cache_index.h"

namespace gvrc {

constexpr int64_t kIntMax = 2147483647;
constexpr int kMaxDevices = 64;

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int log2_of(int32_t pow2) {
  int s = 0;
  while ((int32_t(1) << s) < pow2) ++s;
  return s;
}

inline bool page_size_ok(int32_t ps) { return ps >= 1 && ps <= GVR_CACHE_MAX_PAGE_SIZE && (ps & (ps - 1)) == 0; }

inline gvr_status check_cache(const gvr_cache* c) {
  if (!c) return GVR_ERR_NULL;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return GVR_ERR_ARG;
  if (!page_size_ok(c->page_size) || c->num_kv_heads < 1 || c->num_kv_heads > 65535 || c->reserved != 0)
    return GVR_ERR_ARG;
  if (c->num_pages < 0 || c->num_pages > kIntMax / c->page_size) return GVR_ERR_ARG;
  if (!std::isfinite(c->k_scale) || !std::isfinite(c->v_scale) || !(c->k_scale > 0) || !(c->v_scale > 0))
    return GVR_ERR_ARG;
  if (c->page_stride % 16 != 0 ||
      c->page_stride < int64_t(c->page_size) * c->num_kv_heads * row_bytes(c->head_dim))
    return GVR_ERR_STRIDE;
  // an address is page * page_stride + ... in 64 bits
  if (c->num_pages > 0 && c->page_stride > INT64_MAX / 2 / c->num_pages) return GVR_ERR_STRIDE;
  if (!units_fit(c->num_pages, c->page_stride, row_bytes(c->head_dim))) return GVR_ERR_STRIDE;
  if (c->num_pages > 0 && !c->data) return GVR_ERR_NULL;
  if (!aligned(c->data, 16)) return GVR_ERR_ALIGN;
  return GVR_OK;
}

// The current device's number of SMs (looked up once per device).
cudaError_t sm_count(int* sms);

// Launches in clusters of `cluster` CTAs, allowed to begin while the kernel before it in the stream ends:
// every kernel here calls begin() before it touches memory.
inline cudaError_t launch(const void* kernel, dim3 grid, int threads, int smem, int cluster, void** args, void* stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(uint32_t(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = uint32_t(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

// Waits until the kernel before this one is complete and its writes are visible.  (No kernel but one
// lets the next one start earlier than at its end: CTAs that wait in the free slots of a running kernel
// lie unevenly over the SMs, and a decode batch took 70 us instead of 43.)
// What a kernel before this one may have written is read with ordinary loads alone: they stay behind this wait
// and see its writes, while loads through the read-only path (ld.global.nc) are for memory that nothing
// writes while the kernel is there, and this kernel may be there while the one before still runs.
__device__ __forceinline__ void begin() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets the next kernel start once every CTA of this one has come here, after begin(), or has ended.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ------------------------------------------------------------------------------- conversions
// Four bytes of two e2m1 codes each -> four f16x2, low half from the low four bits.  Exact.
__device__ __forceinline__ void e2m1_to_f16x2(uint32_t codes, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}

// Two e4m3 in the low 16 bits -> f16x2.  Exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
  return r;
}

// Nearest e4m3 (ties to even, saturating at 448, NaN kept) in the low 8 bits.
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}"
      : "=r"(r)
      : "f"(0.f), "f"(x));
  return r;
}

// Nearest e2m1 codes (ties to even, saturating at 6) of lo and hi in one byte.
__device__ __forceinline__ uint32_t f32x2_to_e2m1(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t, z;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tmov.b32 %0, {t, 0, 0, 0};\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// Four such bytes.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float2 (&v)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
  return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2_rn(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  const __half2 v = *reinterpret_cast<const __half2*>(&h);
  return __half22float2(v);
}

}  // namespace gvrc
