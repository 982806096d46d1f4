// kv_device.h -- what the HIP sources of the cache of keys and values by head
// share: its pools, and the host's checks of them.
#ifndef KV_DEVICE_H
#define KV_DEVICE_H

#include "idx_device.h"
#include "kv_cache.h"

namespace {

constexpr int32_t kMaxWidth = 1 << 24;
constexpr int32_t kMaxGroup = 128;  // query heads of a key head

// Head h of page g: values at kv + g * kv_page + h * kv_head, scales likewise.
struct KvStrides {
  int64_t kv_page, kv_head, ks_page, ks_head;
};

// Where row b's page table is.
struct Tables {
  const int32_t* pt;
  const int32_t* rt;  // table of each row, or NULL: row b's
  int64_t stride;
  int32_t num_tables;
  __device__ __forceinline__ const int32_t* of(int64_t b, bool& ok) const {
    ok = true;
    if (!rt) return pt + b * stride;
    const int32_t t = rt[b];
    ok = t >= 0 && t < num_tables;
    return pt + (int64_t)(ok ? t : 0) * stride;
  }
};

inline bool head_dim_ok(int32_t d) { return d == 64 || d == 128 || d == 256; }

inline uint32_t pages_limit(int64_t num_pages) {
  return (uint32_t)(num_pages < (int64_t)1 << 31 ? num_pages : (int64_t)1 << 31);
}

inline int validate_kv_strides(int key, int32_t kv_heads, int32_t head_dim, int64_t num_pages, const KvStrides& s) {
  const int64_t far = (int64_t)1 << 38, block = (int64_t)kPage * head_dim * (key == kFp8 ? 1 : 2);
  const int st = validate_pool(key, head_dim, num_pages, s.kv_page, s.ks_page);
  if (st != IDX_OK) return st;
  if (kv_heads > 1 && (s.kv_head < block || s.kv_head > far)) return IDX_ERR_SHAPE;
  if (kv_heads > 1 && key == kFp8 && (s.ks_head < kPage * 4 || s.ks_head > far)) return IDX_ERR_SHAPE;
  return IDX_OK;
}

inline int validate_kv_pointers(int key, int32_t kv_heads, const void* pages, const float* scale, const KvStrides& s) {
  const int st = validate_pool_pointers(key, pages, scale, s.kv_page, s.ks_page);
  if (st != IDX_OK || kv_heads <= 1) return st;
  if (s.kv_head % 16 != 0 || (key == kFp8 && s.ks_head % 4 != 0)) return IDX_ERR_ALIGN;
  return IDX_OK;
}

}  // namespace

#endif  // KV_DEVICE_H
