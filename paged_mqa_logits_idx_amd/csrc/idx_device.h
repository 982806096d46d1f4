// idx_device.h -- what the caches' HIP sources share: vector types, conversions
// between bf16 / e4m3fn and float, the quantiser, DMA and waits, a softmax's end,
// and the host side's small helpers.
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
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef int v2i __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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

// Outputs of a call that writes 16 MiB or more pass the caches by: the inputs
// keep their place, and the next kernel would not find them there whole.  65536
// latents stored 23.1 us, 26 by ordinary stores, stored and read back 48.2 and 53.2;
// but 16384 stored 8.7 and 9.5, stored and read back 16.6 and 16.2, and 32768 26.3
// and 25.8.
inline bool is_far(int64_t n, int64_t bytes) { return n >= (((int64_t)1 << 24) + bytes - 1) / bytes; }

template <bool FAR, class T>
__device__ __forceinline__ void put(T v, uint8_t* to) {
  if constexpr (FAR) __builtin_nontemporal_store(v, reinterpret_cast<T*>(to));
  else *reinterpret_cast<T*>(to) = v;
}

// The lane's value of another lane of its row of 16.
template <int CTRL, class T>
__device__ __forceinline__ T row_lane(T v) {
  return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// f over the LPV lanes of a vector, in all of them: neighbours, pairs of a
// quad, mirrored halves of a row and rows as operands of the arithmetic itself
// (shuffles go through LDS), then rows and halves of the wave.
template <int LPV, class T, class F>
__device__ __forceinline__ T vector_fold(T v, F f) {
  v = f(v, row_lane<0xb1>(v));   // quad_perm 1 0 3 2
  v = f(v, row_lane<0x4e>(v));   // quad_perm 2 3 0 1
  v = f(v, row_lane<0x141>(v));  // row_half_mirror
  if constexpr (LPV > 8) v = f(v, row_lane<0x140>(v));  // row_mirror
  if constexpr (LPV > 16) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = f(__builtin_bit_cast(T, (uint32_t)r[0]), __builtin_bit_cast(T, (uint32_t)r[1]));
  }
  if constexpr (LPV > 32) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = f(__builtin_bit_cast(T, (uint32_t)r[0]), __builtin_bit_cast(T, (uint32_t)r[1]));
  }
  return v;
}

// Rounds to the nearest e4m3fn codes, ties to even.
__device__ __forceinline__ u32x2 float_to_fp8x8(const float (&q)[8]) {
  u32x2 codes;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
    codes[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], c, true);
  }
  return codes;
}

// The same values; a signalling NaN, which least and largest would answer with, is a
// quiet one, which they pass over.
__device__ __forceinline__ void quiet(float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = __builtin_canonicalizef(v[e]);  // (one by one in the bounds of four prompts: 40.5 -> 41.2 us)
}

// Scale amax / 448 of the vector v * factor and e4m3fn codes of its values / scale,
// clamped to +-448: both quotients as the float32 division rounds them.  The
// factor is left out of the quotients, which do not depend on it: 8 products and a
// rounding of every value less.  A division
// takes some ten instructions and the kernel is bound by them, so each is a
// product and a correction by its residual (Markstein's), q0 = v*y with y the
// reciprocal and q = q0 - (scale*q0 - v)*y, which is the correctly rounded
// quotient away from underflow and overflow, and keeps the sign of a zero; the
// clamp does nothing then.  Where the scale may leave [2^-60, 2^100], the factor is
// far from 1 (or 0, of squares that overflow), or a value is not a number or all are
// zero, `normed` gives the values with the factor in, from the input (without it they may
// have left float32's range), and the division is taken; a NaN has no part in amax
// and becomes +-448.  The two round differently, so each vector has its own choice:
// that another one of the wave needs the division must not change its bytes.  `used`:
// the lane's vector has a slot, its result matters.
template <int LPV, class F>
__device__ __forceinline__ u32x2 quantise(const float (&v)[8], float factor, bool used, float& scale, F normed) {
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = __builtin_elementwise_maximum(m, fabsf(v[k]));  // NaN if one is
  // (never negative: ordered as its bits are, a NaN above all)
  const auto larger = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  m = __uint_as_float(vector_fold<LPV>(__float_as_uint(m), larger));
  const bool near = m >= 0x1p-51f && m <= 0x1p108f && factor >= 0x1p-60f && factor <= 0x1p60f;
  const float c = 1.0f / 448.0f, s0 = m * c;
  scale = fmaf(fmaf(-448.0f, s0, m), c, s0);
  const float y0 = __builtin_amdgcn_rcpf(scale), y = fmaf(fmaf(-scale, y0, 1.0f), y0, y0);
  float q[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float q0 = v[k] * y;
    q[k] = fmaf(-fmaf(scale, q0, -v[k]), y, q0);
  }
  u32x2 codes = float_to_fp8x8(q);
  scale *= factor;
  if (__ballot(used && !near) != 0) {
    float f[8];
    normed(f);
    quiet(f);  // (a value that neither norm nor rotation touches is as it was stored)
    m = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(f[k]));
    m = __uint_as_float(vector_fold<LPV>(__float_as_uint(m), larger));
    const float far = m > 0.0f ? m / 448.0f : 1.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) q[k] = copysignf(__builtin_amdgcn_fmed3f(f[k] / far, -448.0f, 448.0f), f[k]);
    const u32x2 divided = float_to_fp8x8(q);
    if (!near) scale = far, codes = divided;
  }
  return codes;
}

__device__ __forceinline__ int32_t uniform(int32_t x) { return __builtin_amdgcn_readfirstlane(x); }

// The workgroup's waves meet here; their LDS writes before it are visible
// after it.  Memory operations other than LDS ones stay in flight.
__device__ __forceinline__ void barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// 64 lanes x 16 bytes from `src` (each lane its own) to LDS `dst` + 16 * lane.
// In assembly so that the compiler, which would wait for every DMA before any
// LDS read, leaves the order to the explicit waits; m0, which the instruction takes
// the place from, is an operand, so that the compiler knows what is in it (the
// s_nop: a state between its write and the DMA).
__device__ __forceinline__ void dma16(const uint8_t* src, uint32_t dst) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "{m0}"(dst) : "memory");
}

// The same of what no other workgroup reads: it is the first to leave the caches.
__device__ __forceinline__ void dma16_once(const uint8_t* src, uint32_t dst) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt" ::"v"(src), "{m0}"(dst) : "memory");
}

__device__ __forceinline__ void dma4(const uint8_t* src, uint32_t dst) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "{m0}"(dst) : "memory");
}

// Waits until at most N vector-memory operations are outstanding.
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// The end of a softmax: sums relative to 2^m become outputs (times by * half *
// half) and the log of the denominator, in which a sink's base-2 logit joins.
// 2^(m - ref) is applied in two halves: it may be far below float32's range
// where the sink is far above the scores, and the outputs not yet.
struct Closing {
  float by, half, lse;
};
__device__ __forceinline__ Closing close_sum(float m, float z, float sink) {
  // (finite, so that a sink of infinity leaves nothing but itself, not a NaN)
  const float top = fmaxf(m, sink), ref = top == -INFINITY ? 0.0f : fminf(top, 3.4028234663852886e38f);
  Closing c;
  c.half = __builtin_amdgcn_exp2f(0.5f * (m - ref));
  const float total = z * c.half * c.half + __builtin_amdgcn_exp2f(sink - ref);
  c.by = total == 0.0f ? 0.0f : 1.0f / total;
  c.lse = total == 0.0f ? -INFINITY : (ref + log2f(total)) * kLn2;
  return c;
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
