// norm_rope.hip -- norm, rotation, paged store and read back (gfx950 kernels
// and C-ABI entry points declared in include/latent_cache.h).
//
//   y = x / sqrt(mean(x^2) + eps) * weight,   (a, b) -> (a cos - b sin, a sin + b cos)
//   scale = amax / 448,  code = e4m3(y / scale),   out = bf16(code * scale)
//
// Every kernel gives a vector of D values to D/8 neighbouring lanes, 8 values
// (16 bytes of bf16) each: sums and maxima over a vector stay inside its lanes,
// a wave covers 64*8/D vectors, and a vector is read once and written once.
// Values are float32 between the load and the one rounding of the store.
#include <type_traits>

#include "idx_device.h"

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

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

struct Vectors {
  const uint8_t* x;      // bf16
  const float* weight;   // [D] or NULL
  const int64_t* pos;    // [n]
  const float* freq;     // [rope/2]
  int64_t n;
  int64_t x_stride;      // bytes
  int32_t heads;
  int32_t rope;          // rotated values
  int32_t first;         // first rotated value
  uint32_t per_pair;     // 2^20 / (rope / 2), rounded up: (i * per_pair) >> 20 is i / (rope / 2) for i < 2^10
  uint32_t flags;
  float eps;
};

// cos and sin of position * frequency.  The product and its reduction to
// quarters of a turn are float64: at position 2^20 a float32 angle would already
// be off by 0.03 rad.  (2 / pi as a double and the product's rounding leave
// |angle| 2^-51 rad of error: 10^-6 at 2^31.)  What is left, x in [-1/2, 1/2]
// quarters, is rounded to float32 (2^-26 of a quarter) and goes into polynomials
// fitted here for the least largest error over the interval.  With their float32
// coefficients they are off by 2^-25.0 (sin) and 2^-27.1 (cos), in float32
// arithmetic by 2^-23.4 and 2^-24.0; about half of the instructions of a library's
// pair.
__device__ __forceinline__ f32x2 turn(int64_t position, float freq) {
  const double angle = (double)position * (double)freq;
  const double whole = rint(angle * 0.63661977236758134308);
  // (the bounds hold by themselves, but for a rounding, until little is left of the
  // angle; a NaN, which the angle of an infinite frequency is, passes them)
  const float left = (float)fma(angle, 0.63661977236758134308, -whole);
  const float x = __builtin_elementwise_maximum(__builtin_elementwise_minimum(left, 0.5f), -0.5f), xx = x * x;
  // the quarter: 1.5 * 2^52 has the integers as its last bits
  const uint32_t quarter = (uint32_t)__builtin_bit_cast(uint64_t, whole + 0x1.8p52);
  const float s = x * fmaf(xx, fmaf(xx, fmaf(xx, -4.60166e-3f, 7.968003e-2f), -0.64596346f), 1.57079632f);
  const float c = fmaf(xx, fmaf(xx, fmaf(xx, fmaf(xx, 9.04021671e-4f, -2.08602885e-2f), 0.253669244f), -1.23370054f), 1.0f);
  const float a = quarter & 1 ? c : s, b = quarter & 1 ? s : c;
  return (f32x2){__uint_as_float(__float_as_uint(b) ^ (quarter + 1) << 30 & 0x80000000u),
                 __uint_as_float(__float_as_uint(a) ^ quarter << 30 & 0x80000000u)};
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

// 1 / sqrt(v) to 2^-23 of itself; the instruction takes no denormals.
__device__ __forceinline__ float inverse_root(float v) {
  const bool tiny = v < 0x1p-100f;
  return __builtin_amdgcn_rsqf(tiny ? v * 0x1p64f : v) * (tiny ? 0x1p32f : 1.0f);
}

// How the rotated values pair up: a kernel each (one kernel that asks takes 16
// moves a token more to bring the three ways' values together).
enum { kPlain, kNeighbours, kHalves };

// Norm and rotation of the lane's 8 values; `table` holds its token's turns,
// `w` its 8 weights.  LATE: without the norm's factor, which is returned.  Called by
// whole waves.
template <int LPV, int ROPE, bool LATE>
__device__ __forceinline__ float norm_rotate(const Vectors& p, int sub, const float (&w)[8], const f32x2* table,
                                             float (&v)[8]) {
  float factor = 1.0f;
  if (!(p.flags & IDX_NORM_OFF)) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s = fmaf(v[k], v[k], s);
    s = vector_fold<LPV>(s, [](float a, float b) { return a + b; });
    const float r = inverse_root(s * (1.0f / (8 * LPV)) + p.eps);
    if constexpr (LATE) factor = r;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = LATE ? v[k] * w[k] : v[k] * r * w[k];
  }
  const int at = 8 * sub - p.first;  // the lane's first value within the rotated part
  const bool in = at >= 0 && at < p.rope;
  if constexpr (ROPE == kHalves) {
    const int half = p.rope >> 1;
    const bool low = at < half;
    // the other value of each pair is half/8 lanes away
    const int lane = threadIdx.x & 63, other = in ? (low ? lane + half / 8 : lane - half / 8) : lane;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float o = __shfl(v[k], other);
      if (in) {
        const f32x2 cs = table[(low ? at : at - half) + k];
        v[k] = low ? v[k] * cs.x - o * cs.y : o * cs.y + v[k] * cs.x;
      }
    }
  } else if (ROPE == kNeighbours && in) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const f32x2 cs = table[(at >> 1) + k];
      const float a = v[2 * k], b = v[2 * k + 1];
      v[2 * k] = a * cs.x - b * cs.y;
      v[2 * k + 1] = a * cs.y + b * cs.x;
    }
  }
  return factor;
}

template <int LPV>
__device__ __forceinline__ void load_weight(const Vectors& p, int sub, float (&w)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = p.weight ? p.weight[8 * sub + k] : 1.0f;
}

// Unit = one token x `STEPS` groups of kWaves * 64/LPV heads, which share the
// token's turns.  Bound by memory: 4096 tokens of 64 heads of 512 take 90 to 93 us,
// 537 MB at 5.8 to 6.0 TB/s (of a bare copy as large 97).
template <int LPV, int ROPE, int STEPS>
__global__ __launch_bounds__(kThreads) void norm_rope_kernel(Vectors p, uint8_t* out, int32_t groups) {
  extern __shared__ f32x2 table[];
  constexpr int kDim = 8 * LPV, kVecs = 64 / LPV;
  const int lane = threadIdx.x & 63, sub = lane % LPV;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float w[8];
  load_weight<LPV>(p, sub, w);
  for (int64_t unit = blockIdx.x; unit < p.n * groups; unit += gridDim.x) {
    const int64_t t = unit / groups;
    const int h0 = (int)(unit % groups) * (STEPS * kWaves * kVecs) + wave * kVecs + lane / LPV;
    u32x4 raw[STEPS];
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      const int h = h0 + u * kWaves * kVecs;
      raw[u] = (u32x4){0u, 0u, 0u, 0u};
      if (h < p.heads) raw[u] = *reinterpret_cast<const u32x4*>(p.x + t * p.x_stride + ((int64_t)h * kDim + 8 * sub) * 2);
    }
    if constexpr (ROPE != kPlain) {
      __syncthreads();  // the last unit's turns have been used
      for (int i = threadIdx.x; i < p.rope >> 1; i += kThreads) table[i] = turn(p.pos[t], p.freq[i]);
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      const int h = h0 + u * kWaves * kVecs;
      float v[8];
      bf16x8_to_float(raw[u], v);
      norm_rotate<LPV, ROPE, false>(p, sub, w, table, v);
      if (h < p.heads)
        put<(STEPS > 1)>(float_to_bf16x8(v), out + ((t * p.heads + h) * kDim + 8 * sub) * 2);
    }
  }
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

struct Pool {
  uint8_t* kv;
  uint8_t* ks;
  int64_t slots;  // 64 * pages
  int64_t kv_stride, ks_stride;
};

constexpr int kSteps = 2;  // (65536 latents: 24.2 us, 24.6 with 1 and 23.4 with 4; 16384: 9.5, 9.5 and 10.6)

// Unit = kSteps groups of 64/LPV tokens, a wave's; the next unit's vectors are
// on their way while one is worked on.  A wave has its tokens' turns to itself,
// so no wave waits for another.  65536 latents to e4m3 take 23 us: 102 MB at
// 4.4 TB/s, but bound by the vector instructions (some 170 a token, issuing in nearly
// all of the SIMDs' cycles); to bf16 23 us too, 135 MB at 5.8 TB/s.
template <int KEY, int LPV, int ROPE, bool FAR>
__global__ __launch_bounds__(kThreads) void norm_rope_store_kernel(Vectors p, Pool pool, const int64_t* slots) {
  extern __shared__ f32x2 table[];
  constexpr int kDim = 8 * LPV, kVecs = 64 / LPV, kTokens = kSteps * kVecs;
  const int lane = threadIdx.x & 63, sub = lane % LPV;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pairs = p.rope >> 1;
  f32x2* turns = table + wave * kTokens * pairs;
  struct Unit {
    u32x4 raw[kSteps];
    int64_t slot[kSteps];
  };
  auto load = [&](int64_t t0) {
    Unit unit;
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int64_t t = t0 + u * kVecs + lane / LPV;
      unit.raw[u] = (u32x4){0u, 0u, 0u, 0u};
      unit.slot[u] = -1;
      if (t < p.n) {
        unit.slot[u] = slots[t];
        unit.raw[u] = *reinterpret_cast<const u32x4*>(p.x + t * p.x_stride + 16 * sub);
      }
    }
    return unit;
  };
  const int64_t step = (int64_t)gridDim.x * kWaves * kTokens;
  int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * kTokens;
  Unit next = load(t0);
  float w[8];
  load_weight<LPV>(p, sub, w);
  for (; t0 < p.n; t0 += step) {
    const Unit unit = next;
    next = load(t0 + step);
    if constexpr (ROPE != kPlain) {
#pragma unroll 1
      for (int i = lane; i < kTokens * pairs; i += 64) {
        const int token = (int)((uint32_t)i * p.per_pair >> 20);
        const int64_t t = t0 + token < p.n ? t0 + token : t0;
        turns[i] = turn(p.pos[t], p.freq[i - token * pairs]);
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const f32x2* mine = turns + (u * kVecs + lane / LPV) * pairs;
      float v[8];
      bf16x8_to_float(unit.raw[u], v);
      const float factor = norm_rotate<LPV, ROPE, KEY == kFp8>(p, sub, w, mine, v);
      const int64_t slot = unit.slot[u];
      const bool ok = slot >= 0 && slot < pool.slots;
      const int64_t page = ok ? slot / kPage : 0, i = ok ? slot % kPage : 0;
      if constexpr (KEY == kBf16) {
        if (ok) put<FAR>(float_to_bf16x8(v), pool.kv + page * pool.kv_stride + (i * kDim + 8 * sub) * 2);
      } else {
        float scale;
        const u32x2 codes = quantise<LPV>(v, factor, ok, scale, [&](float (&f)[8]) {
          u32x4 raw = unit.raw[u];
          asm volatile("" : "+v"(raw));  // (or the values of every token are kept for here: 8 moves)
          bf16x8_to_float(raw, f);
          norm_rotate<LPV, ROPE, false>(p, sub, w, mine, f);
        });
        if (ok) {
          put<FAR>(codes, pool.kv + page * pool.kv_stride + i * kDim + 8 * sub);
          if (sub == 0) *reinterpret_cast<float*>(pool.ks + page * pool.ks_stride + 4 * i) = scale;
        }
      }
    }
    __builtin_amdgcn_wave_barrier();  // the turns have been used
  }
}

// Unit = `STEPS` groups of kWaves * 64/LPV slots: their loads are under way at
// once, in two trips (slots, then codes and scales).  Bound by memory: 262208
// latents from e4m3 take 78 us, 404 MB at 5.2 TB/s.
template <int KEY, int LPV, int STEPS, bool FAR>
__global__ __launch_bounds__(kThreads) void load_slots_kernel(Pool pool, const int64_t* slots, int64_t n,
                                                              uint8_t* out, int64_t out_stride) {
  constexpr int kDim = 8 * LPV, kVecs = 64 / LPV, kTokens = STEPS * kWaves * kVecs;
  const int lane = threadIdx.x & 63, sub = lane % LPV, wave = threadIdx.x >> 6;
  for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < n; t0 += (int64_t)gridDim.x * kTokens) {
    int64_t slot[STEPS];
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      const int64_t t = t0 + (u * kWaves + wave) * kVecs + lane / LPV;
      slot[u] = t < n ? slots[t] : -1;
      if (slot[u] >= pool.slots) slot[u] = -1;
    }
    u32x4 raw[STEPS];
    float scale[STEPS];
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      raw[u] = (u32x4){0u, 0u, 0u, 0u};
      scale[u] = 0.0f;
      if (slot[u] < 0) continue;
      const int64_t page = slot[u] / kPage, i = slot[u] % kPage;
      if constexpr (KEY == kBf16) {
        raw[u] = *reinterpret_cast<const u32x4*>(pool.kv + page * pool.kv_stride + (i * kDim + 8 * sub) * 2);
      } else {
        const u32x2 c = *reinterpret_cast<const u32x2*>(pool.kv + page * pool.kv_stride + i * kDim + 8 * sub);
        raw[u].x = c.x;
        raw[u].y = c.y;
        scale[u] = *reinterpret_cast<const float*>(pool.ks + page * pool.ks_stride + 4 * i);
      }
    }
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      if (slot[u] < 0) continue;
      const int64_t t = t0 + (u * kWaves + wave) * kVecs + lane / LPV;
      u32x4 r = raw[u];
      if constexpr (KEY == kFp8) {
        float v[8];
        bf16x8_to_float(__builtin_bit_cast(u32x4, fp8x8_to_bf16x8(raw[u].x, raw[u].y)), v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= scale[u];
        r = float_to_bf16x8(v);
      }
      put<FAR>(r, out + t * out_stride + 16 * sub);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side.

constexpr int64_t kMaxGrid = (int64_t)1 << 20;  // larger problems loop (grid-stride)

inline dim3 grid_of(int64_t units) { return dim3((uint32_t)(units < kMaxGrid ? units : kMaxGrid)); }

// The checks that the norm and rotation's arguments share; `pointers`: there
// is something to do, so the pointers are looked at.
int validate_vectors(const void* x, const float* norm_weight, const int64_t* positions, const float* inv_freq,
                     int64_t n, int32_t num_heads, int32_t head_dim, int32_t rope_dim, uint32_t flags, float eps,
                     int64_t x_row_stride) {
  if (rope_dim < 0 || rope_dim > head_dim || rope_dim % 16 != 0 ||
      (flags & ~(IDX_NORM_OFF | IDX_ROPE_LEADING | IDX_ROPE_HALVES)) != 0)
    return IDX_ERR_UNSUPPORTED;
  if (n < 0 || num_heads < 0 || n > ((int64_t)1 << 40) || !(eps >= 0.0f) || !(eps < INFINITY) ||
      x_row_stride < (int64_t)num_heads * head_dim || x_row_stride > ((int64_t)1 << 32))
    return IDX_ERR_SHAPE;
  if (n == 0 || num_heads == 0) return IDX_OK;
  if (!x || (rope_dim > 0 && (!positions || !inv_freq)) || ((flags & IDX_NORM_OFF) && norm_weight)) return IDX_ERR_NULL;
  if (!aligned(x, 16) || x_row_stride % 8 != 0 || !aligned(norm_weight, 16) || !aligned(positions, 8) ||
      !aligned(inv_freq, 4))
    return IDX_ERR_ALIGN;
  return IDX_OK;
}

Vectors vectors_of(const void* x, const float* norm_weight, const int64_t* positions, const float* inv_freq,
                   int64_t n, int32_t num_heads, int32_t head_dim, int32_t rope_dim, uint32_t flags, float eps,
                   int64_t x_row_stride) {
  Vectors p;
  p.x = static_cast<const uint8_t*>(x);
  p.weight = norm_weight;
  p.pos = positions;
  p.freq = inv_freq;
  p.n = n;
  p.x_stride = 2 * x_row_stride;
  p.heads = num_heads;
  p.rope = rope_dim;
  p.first = (flags & IDX_ROPE_LEADING) ? 0 : head_dim - rope_dim;
  p.per_pair = rope_dim > 0 ? ((1u << 20) + rope_dim / 2 - 1) / (uint32_t)(rope_dim / 2) : 0;
  p.flags = flags;
  p.eps = eps;
  return p;
}

// The kernel for a rotation: f(std::integral_constant<int, ROPE>).
template <class F>
void for_rotation(const Vectors& p, F f) {
  if (p.rope == 0) f(std::integral_constant<int, kPlain>{});
  else if (p.flags & IDX_ROPE_HALVES) f(std::integral_constant<int, kHalves>{});
  else f(std::integral_constant<int, kNeighbours>{});
}

template <int LPV>
void launch_norm_rope(const Vectors& p, void* out, hipStream_t stream) {
  constexpr int kOne = kWaves * (64 / LPV);  // heads of one step
  const size_t lds = (size_t)(p.rope / 2) * sizeof(f32x2);
  const int32_t groups = (p.heads + 4 * kOne - 1) / (4 * kOne), single = (p.heads + kOne - 1) / kOne;
  uint8_t* to = static_cast<uint8_t*>(out);
  for_rotation(p, [&](auto rope) {
    constexpr int kRope = decltype(rope)::value;
    // four steps, and past the caches, where a token's heads are more than one step
    // has places for and the units fill the device (more than 16 MiB then).  128 MiB:
    // 2048 tokens of 64 heads of 512 49 us, 53 in one step, 26214 of 5 65 and 71,
    // 30840 of 17 of 128 68 and 79; but 32768 of 4 of 512 74 and 54, 131072 of one 226
    // and 137, and 4096 of one of 128 10 and 6.4; 1024 of 64 of 128, 1024 units, 11.2
    // and 10.1.  Ordinary stores instead: 4096 of 64 of 512 93 -> 96, 2048 of 40 28 ->
    // 35, 2048 of 64 49 -> 47, but with a kernel that reads all of it next 194 -> 185,
    // 60 -> 59 and 98 -> 87.
    if (p.heads > kOne && p.n * groups >= 16 * device_cu_count())
      norm_rope_kernel<LPV, kRope, 4><<<grid_of(p.n * groups), dim3(kThreads), lds, stream>>>(p, to, groups);
    else
      norm_rope_kernel<LPV, kRope, 1><<<grid_of(p.n * single), dim3(kThreads), lds, stream>>>(p, to, single);
  });
}

template <int KEY, int LPV>
void launch_store(const Vectors& p, const Pool& pool, const int64_t* slots, hipStream_t stream) {
  constexpr int kTokens = kSteps * kWaves * (64 / LPV);
  const size_t lds = (size_t)(p.rope / 2) * sizeof(f32x2) * kTokens;
  // a grid of 16 blocks a CU goes round, with the next loads under way (65536
  // latents to e4m3 and bf16: 24.2 and 23.3 us, 24.0 and 23.7 with 8 a CU)
  const int64_t units = (p.n + kTokens - 1) / kTokens, most = 16 * device_cu_count();
  const dim3 grid((uint32_t)(units < most ? units : most));
  for_rotation(p, [&](auto rope) {
    constexpr int kRope = decltype(rope)::value;
    if (is_far(p.n, LPV * (KEY == kFp8 ? 8 : 16)))
      norm_rope_store_kernel<KEY, LPV, kRope, true><<<grid, dim3(kThreads), lds, stream>>>(p, pool, slots);
    else
      norm_rope_store_kernel<KEY, LPV, kRope, false><<<grid, dim3(kThreads), lds, stream>>>(p, pool, slots);
  });
}

template <int KEY>
int norm_rope_store(const void* x, const float* norm_weight, const int64_t* positions, const float* inv_freq,
                    const int64_t* slots, int64_t n, int32_t head_dim, int32_t rope_dim, uint32_t flags, float eps,
                    int64_t x_row_stride, void* kv_pages, float* kscale, int64_t num_pages, int64_t kv_page_stride,
                    int64_t kscale_page_stride, hipStream_t stream) {
  if (head_dim != IDX_HEAD_DIM && head_dim != kLatent) return IDX_ERR_UNSUPPORTED;
  int st = validate_vectors(x, norm_weight, positions, inv_freq, n, 1, head_dim, rope_dim, flags, eps, x_row_stride);
  if (st != IDX_OK) return st;
  st = validate_pool(KEY, head_dim, num_pages, kv_page_stride, kscale_page_stride);
  if (st != IDX_OK || n == 0) return st;
  if (!slots) return IDX_ERR_NULL;
  st = validate_pool_pointers(KEY, kv_pages, kscale, kv_page_stride, kscale_page_stride);
  if (st != IDX_OK) return st;
  if (!aligned(slots, 8)) return IDX_ERR_ALIGN;
  const Vectors p = vectors_of(x, norm_weight, positions, inv_freq, n, 1, head_dim, rope_dim, flags, eps, x_row_stride);
  const Pool pool = {static_cast<uint8_t*>(kv_pages), reinterpret_cast<uint8_t*>(kscale), num_pages * kPage,
                     kv_page_stride, kscale_page_stride};
  (void)hipGetLastError();  // start from a clean error state
  if (head_dim == kLatent) launch_store<KEY, kLatent / 8>(p, pool, slots, stream);
  else launch_store<KEY, IDX_HEAD_DIM / 8>(p, pool, slots, stream);
  return launch_status();
}

template <int KEY, int LPV>
void launch_load(const Pool& pool, const int64_t* slots, int64_t n, void* out, int64_t out_row_stride,
                 hipStream_t stream) {
  constexpr int kOne = kWaves * (64 / LPV);
  uint8_t* o = static_cast<uint8_t*>(out);
  const dim3 ones = grid_of((n + kOne - 1) / kOne);
  // past the caches: 78 us, 96 with ordinary stores (262208 latents from e4m3);
  // four steps of e4m3 then, 87 us in one, but bf16 moves as much in one: 73 us, 77
  // in four (196608)
  if (!is_far(n, 16 * LPV))
    load_slots_kernel<KEY, LPV, 1, false><<<ones, dim3(kThreads), 0, stream>>>(pool, slots, n, o, 2 * out_row_stride);
  else if constexpr (KEY == kBf16)
    load_slots_kernel<KEY, LPV, 1, true><<<ones, dim3(kThreads), 0, stream>>>(pool, slots, n, o, 2 * out_row_stride);
  else
    load_slots_kernel<KEY, LPV, 4, true><<<grid_of((n + 4 * kOne - 1) / (4 * kOne)), dim3(kThreads), 0, stream>>>(
        pool, slots, n, o, 2 * out_row_stride);
}

template <int KEY>
int load_slots(const void* kv_pages, const float* kscale, const int64_t* slots, int64_t n, int32_t head_dim,
               int64_t num_pages, int64_t kv_page_stride, int64_t kscale_page_stride, void* out,
               int64_t out_row_stride, hipStream_t stream) {
  if (head_dim != IDX_HEAD_DIM && head_dim != kLatent) return IDX_ERR_UNSUPPORTED;
  if (n < 0 || n > ((int64_t)1 << 40) || out_row_stride < head_dim || out_row_stride > ((int64_t)1 << 32))
    return IDX_ERR_SHAPE;
  int st = validate_pool(KEY, head_dim, num_pages, kv_page_stride, kscale_page_stride);
  if (st != IDX_OK || n == 0) return st;
  if (!slots || !out) return IDX_ERR_NULL;
  st = validate_pool_pointers(KEY, kv_pages, kscale, kv_page_stride, kscale_page_stride);
  if (st != IDX_OK) return st;
  if (!aligned(slots, 8) || !aligned(out, 16) || out_row_stride % 8 != 0) return IDX_ERR_ALIGN;
  const Pool pool = {static_cast<uint8_t*>(const_cast<void*>(kv_pages)),
                     reinterpret_cast<uint8_t*>(const_cast<float*>(kscale)), num_pages * kPage, kv_page_stride,
                     kscale_page_stride};
  (void)hipGetLastError();
  if (head_dim == kLatent) launch_load<KEY, kLatent / 8>(pool, slots, n, out, out_row_stride, stream);
  else launch_load<KEY, IDX_HEAD_DIM / 8>(pool, slots, n, out, out_row_stride, stream);
  return launch_status();
}

}  // namespace

extern "C" {

int idx_norm_rope(const void* x, const float* norm_weight, const int64_t* positions, const float* inv_freq,
                  void* out, int64_t n, int32_t num_heads, int32_t head_dim, int32_t rope_dim, uint32_t flags,
                  float eps, int64_t x_row_stride, hipStream_t stream) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 256 && head_dim != 512) return IDX_ERR_UNSUPPORTED;
  const int st = validate_vectors(x, norm_weight, positions, inv_freq, n, num_heads, head_dim, rope_dim, flags, eps,
                                  x_row_stride);
  if (st != IDX_OK || n == 0 || num_heads == 0) return st;
  if (!out) return IDX_ERR_NULL;
  if (!aligned(out, 16)) return IDX_ERR_ALIGN;
  const Vectors p = vectors_of(x, norm_weight, positions, inv_freq, n, num_heads, head_dim, rope_dim, flags, eps,
                               x_row_stride);
  (void)hipGetLastError();
  switch (head_dim) {
    case 64: launch_norm_rope<8>(p, out, stream); break;
    case 128: launch_norm_rope<16>(p, out, stream); break;
    case 256: launch_norm_rope<32>(p, out, stream); break;
    default: launch_norm_rope<64>(p, out, stream); break;
  }
  return launch_status();
}

int idx_norm_rope_store_fp8(const void* x, const float* norm_weight, const int64_t* positions,
                            const float* inv_freq, const int64_t* slots, int64_t n, int32_t head_dim,
                            int32_t rope_dim, uint32_t flags, float eps, int64_t x_row_stride, void* kv_pages,
                            float* kscale, int64_t num_pages, int64_t kv_page_stride, int64_t kscale_page_stride,
                            hipStream_t stream) {
  return norm_rope_store<kFp8>(x, norm_weight, positions, inv_freq, slots, n, head_dim, rope_dim, flags, eps,
                               x_row_stride, kv_pages, kscale, num_pages, kv_page_stride, kscale_page_stride, stream);
}

int idx_norm_rope_store_bf16(const void* x, const float* norm_weight, const int64_t* positions,
                             const float* inv_freq, const int64_t* slots, int64_t n, int32_t head_dim,
                             int32_t rope_dim, uint32_t flags, float eps, int64_t x_row_stride, void* kv_pages,
                             int64_t num_pages, int64_t kv_page_stride, hipStream_t stream) {
  return norm_rope_store<kBf16>(x, norm_weight, positions, inv_freq, slots, n, head_dim, rope_dim, flags, eps,
                                x_row_stride, kv_pages, nullptr, num_pages, kv_page_stride, 0, stream);
}

int idx_load_slots_fp8(const void* kv_pages, const float* kscale, const int64_t* slots, int64_t n, int32_t head_dim,
                       int64_t num_pages, int64_t kv_page_stride, int64_t kscale_page_stride, void* out,
                       int64_t out_row_stride, hipStream_t stream) {
  return load_slots<kFp8>(kv_pages, kscale, slots, n, head_dim, num_pages, kv_page_stride, kscale_page_stride, out,
                          out_row_stride, stream);
}

int idx_load_slots_bf16(const void* kv_pages, const int64_t* slots, int64_t n, int32_t head_dim, int64_t num_pages,
                        int64_t kv_page_stride, void* out, int64_t out_row_stride, hipStream_t stream) {
  return load_slots<kBf16>(kv_pages, nullptr, slots, n, head_dim, num_pages, kv_page_stride, 0, out, out_row_stride,
                           stream);
}

}  // extern "C"
