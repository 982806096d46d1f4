// idx_device.h -- what the latent cache's HIP sources share: vector types,
// conversions between bf16 / e4m3fn and float, and the host side's small
// helpers.
#ifndef IDX_DEVICE_H
#define IDX_DEVICE_H

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "latent_cache.h"

namespace {

constexpr int kPage = IDX_PAGE_POSITIONS;   // 64 positions a page
constexpr int kLatent = IDX_LATENT_DIM;     // 512
constexpr int kFp8 = 0;
constexpr int kBf16 = 1;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void bf16x8_to_float(const u32x4& raw, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __builtin_bit_cast(float, raw[k] << 16);
    v[2 * k + 1] = __builtin_bit_cast(float, raw[k] & 0xffff0000u);
  }
}

// Rounds to nearest even.
__device__ __forceinline__ u32x4 float_to_bf16x8(const float (&v)[8]) {
  bf16x8 r;
#pragma unroll
  for (int k = 0; k < 8; ++k) r[k] = (__bf16)v[k];
  return __builtin_bit_cast(u32x4, r);
}

// 8 e4m3fn bytes -> 8 bf16 (exact: every e4m3fn value is a bf16 value).
__device__ __forceinline__ bf16x8 fp8x8_to_bf16x8(uint32_t lo, uint32_t hi) {
  u32x4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
  return __builtin_bit_cast(bf16x8, r);
}

// Compute units of the current device (queried once per device).
inline int device_cu_count() {
  static std::atomic<int> cache[64];  // per device; concurrent callers store the same value
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  int n = cache[dev].load(std::memory_order_relaxed);
  if (n <= 0) {
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
      n = 256;
    cache[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

inline bool aligned(const void* ptr, uintptr_t a) { return ((uintptr_t)ptr & (a - 1)) == 0; }

inline int launch_status() { return hipGetLastError() == hipSuccess ? IDX_OK : IDX_ERR_LAUNCH; }

// Page strides of a pool of `key` pages of head_dim values a position.
inline int validate_pool(int key, int32_t head_dim, int64_t num_pages, int64_t kv_page_stride,
                         int64_t kscale_page_stride) {
  const int64_t min_kv = (int64_t)kPage * head_dim * (key == kFp8 ? 1 : 2);
  const int64_t most = (int64_t)1 << 32;
  if (num_pages < 0 || num_pages > ((int64_t)1 << 40) || kv_page_stride < min_kv || kv_page_stride > most) return IDX_ERR_SHAPE;
  if (key == kFp8 && (kscale_page_stride < kPage * 4 || kscale_page_stride > most)) return IDX_ERR_SHAPE;
  return IDX_OK;
}

inline int validate_pool_pointers(int key, const void* kv_pages, const float* kscale, int64_t kv_page_stride,
                                  int64_t kscale_page_stride) {
  if (!kv_pages || (key == kFp8 ? kscale == nullptr : kscale != nullptr)) return IDX_ERR_NULL;
  if (!aligned(kv_pages, 16) || (kv_page_stride % 16) != 0) return IDX_ERR_ALIGN;
  if (key == kFp8 && (!aligned(kscale, 4) || (kscale_page_stride % 4) != 0)) return IDX_ERR_ALIGN;
  return IDX_OK;
}

}  // namespace

#endif  // IDX_DEVICE_H
