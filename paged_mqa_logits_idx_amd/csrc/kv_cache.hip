// kv_cache.hip -- page tables and slot maps of a batch, paged store of keys and
// values, bounds of pages' keys and scores of pages by them (gfx950 kernels and
// C-ABI entry points declared in include/kv_cache.h).
#include <type_traits>

#include "kv_device.h"

namespace {

// ---------------------------------------------------------------------------
// Page tables and slot maps.

struct Plan {
  const int32_t* cached;
  const int32_t* added;
  const int32_t* free_pages;
  int32_t* pt;
  int64_t* slots;
  int64_t* positions;
  int32_t* row_table;
  int32_t* seqlens;
  int64_t* starts;
  int64_t* taken;
  int64_t num_free, pt_stride, n;
  int32_t requests, width;
};

// What a request has and gets.
struct Request {
  int64_t cached, added, low, need;  // positions, new ones, its pages so far, new ones
};
__device__ __forceinline__ Request request_of(const Plan& p, int32_t cached, int32_t added) {
  Request q;
  q.cached = max(cached, 0);
  q.added = max(added, 0);
  q.low = (q.cached + kPage - 1) / kPage;
  const int64_t high = min((q.cached + q.added + kPage - 1) / kPage, (int64_t)p.width);
  q.need = max(high - q.low, (int64_t)0);
  return q;
}

// Every workgroup adds up the requests by itself (they are few, and read from the
// caches), so that one launch does it all: its threads have runs of `per` requests,
// whose sums are scanned in LDS.  A token's request is found by halving over
// the runs, then a walk along one; a new page's likewise.  Lengths of up to 4 requests
// a thread are held in LDS for the walks (1024 requests and 65536 tokens 6.4 -> 5.4 us).
// A launch and three trips to memory (lengths, the page, the store) are its time: 64
// requests of one token 2.8 us.  The grid goes by the rows: pages alone (n 0) are one
// workgroup's, the 65536 of 1024 prompts of 4096 tokens 181 us, with their slots 42.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void plan_kernel(Plan p) {
  __shared__ int64_t tokens[THREADS + 1], pages[THREADS + 1];
  __shared__ int64_t sums[2][THREADS / 64];
  constexpr int kHeld = THREADS <= 256 ? 4 * THREADS : 0;
  __shared__ int32_t held[2][kHeld > 0 ? kHeld : 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int32_t per = (p.requests + THREADS - 1) / THREADS;
  const int32_t r0 = min(tid * per, p.requests), r1 = min(r0 + per, p.requests);
  const auto request_at = [&](int32_t r) {
    return kHeld > 0 ? request_of(p, held[0][r], held[1][r]) : request_of(p, p.cached[r], p.added[r]);
  };
  int64_t t = 0, g = 0;
  for (int32_t r = r0; r < r1; ++r) {
    const int32_t cached = p.cached[r], added = p.added[r];
    if (kHeld > 0) held[0][r] = cached, held[1][r] = added;
    const Request q = request_of(p, cached, added);
    t += q.added;
    g += q.need;
  }
  const int64_t own_t = t, own_g = g;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int64_t a = __shfl_up((long long)t, d), b = __shfl_up((long long)g, d);
    if (lane >= d) t += a, g += b;
  }
  if (lane == 63) sums[0][wave] = t, sums[1][wave] = g;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w)
    if (w < wave) t += sums[0][w], g += sums[1][w];
  tokens[tid] = t - own_t;
  pages[tid] = g - own_g;
  if (tid == THREADS - 1) tokens[THREADS] = t, pages[THREADS] = g;
  __syncthreads();
  const int64_t all_tokens = tokens[THREADS], all_pages = pages[THREADS];

  if (blockIdx.x == 0) {
    if (p.starts) {
      int64_t at = tokens[tid];
      for (int32_t r = r0; r < r1; ++r) {
        p.starts[r] = at;
        at += max(kHeld > 0 ? held[1][r] : p.added[r], 0);
      }
      if (tid == 0) p.starts[p.requests] = all_tokens;
    }
    if (p.taken && tid == 0) *p.taken = all_pages;
  }

  const auto run_of = [&](const int64_t* from, int64_t x) {  // the last run that starts at or before x
    int at = 0;
#pragma unroll
    for (int d = THREADS / 2; d > 0; d /= 2)
      if (from[at + d] <= x) at += d;
    return at;
  };
  const auto free_page = [&](int64_t i) { return i < p.num_free ? p.free_pages[i] : -1; };
  const int64_t first = (int64_t)blockIdx.x * THREADS + tid, step = (int64_t)gridDim.x * THREADS;
  for (int64_t row = first; row < p.n; row += step) {
    int64_t slot = -1, position = 0;
    int32_t request = 0, length = 0;
    if (row < all_tokens) {
      const int run = run_of(tokens, row);
      int64_t start = tokens[run], base = pages[run];
      request = run * per;
      Request q = request_at(request);
      while (row >= start + q.added) {
        start += q.added;
        base += q.need;
        q = request_at(++request);
      }
      position = q.cached + (row - start);
      length = (int32_t)min(position + 1, (int64_t)INT32_MAX);
      const int64_t j = position / kPage;
      int32_t page = -1;
      if (j < p.width) page = j < q.low ? p.pt[request * p.pt_stride + j] : free_page(base + j - q.low);
      if (page >= 0) slot = (int64_t)page * kPage + position % kPage;
    }
    if (p.slots) p.slots[row] = slot;
    if (p.positions) p.positions[row] = position;
    if (p.row_table) p.row_table[row] = request;
    if (p.seqlens) p.seqlens[row] = length;
  }
  for (int64_t i = first; i < all_pages; i += step) {
    const int run = run_of(pages, i);
    int64_t base = pages[run];
    int32_t request = run * per;
    Request q = request_at(request);
    while (i >= base + q.need) {
      base += q.need;
      q = request_at(++request);
    }
    p.pt[request * p.pt_stride + q.low + (i - base)] = free_page(i);
  }
}

// ---------------------------------------------------------------------------
// Store of keys and values.

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// 16 bytes; ONCE: not read again soon, the first to leave the caches.
template <bool ONCE>
__device__ __forceinline__ u32x4 get(const uint8_t* from) {
  if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(from));
  return *reinterpret_cast<const u32x4*>(from);
}

struct Store {
  const uint8_t* x[2];  // keys, values (bf16)
  uint8_t* kv[2];
  uint8_t* ks[2];
  const int64_t* slots;
  int64_t x_stride[2];  // bytes
  int64_t vectors;      // tokens * heads, of each
  int64_t pool_slots;   // 64 * pages
  KvStrides s;
  int32_t heads;
};

constexpr int kStoreSteps = 2;

// A vector of D values is D/8 lanes' (16 bytes of bf16 each); a wave takes
// kStoreSteps groups of 64*8/D neighbouring vectors of the keys and the same of
// the values, all loads under way at once.  Bound by memory: 32768 tokens of 8 bf16
// heads of 128, keys and values, 268 MB, take 51.5 us, 5.2 TB/s, to e4m3, 204 MB, 42.6, 4.8
// TB/s (with one step 52.8 and 43.8, with four 51.9 and 43.5; 4096 tokens 6.9 and 7.8, with one
// 7.8 and 7.4, with four 6.6 and 8.3; 64 tokens 2.6 and 3.5, 2.4 and 2.9, 3.2 and 4.6).
template <int KEY, int LPV, bool FAR>
__global__ __launch_bounds__(kThreads) void store_kv_kernel(Store p) {
  constexpr int kDim = 8 * LPV, kVecs = 64 / LPV, kUnit = kStoreSteps * kVecs;
  const int lane = threadIdx.x & 63, sub = lane % LPV, wave = threadIdx.x >> 6;
  const int64_t step = (int64_t)gridDim.x * kWaves * kUnit;
  for (int64_t v0 = ((int64_t)blockIdx.x * kWaves + wave) * kUnit; v0 < p.vectors; v0 += step) {
    u32x4 raw[kStoreSteps][2];
    int64_t slot[kStoreSteps];
    int32_t head[kStoreSteps];
#pragma unroll
    for (int u = 0; u < kStoreSteps; ++u) {
      const int64_t v = v0 + u * kVecs + lane / LPV;
      slot[u] = -1;
      head[u] = 0;
      raw[u][0] = raw[u][1] = (u32x4){0u, 0u, 0u, 0u};
      if (v < p.vectors) {
        const int64_t t = p.vectors <= UINT32_MAX ? (uint32_t)v / (uint32_t)p.heads : v / p.heads;
        head[u] = (int32_t)(v - t * p.heads);
        slot[u] = p.slots[t];
#pragma unroll
        for (int w = 0; w < 2; ++w)
          raw[u][w] = get<FAR>(p.x[w] + t * p.x_stride[w] + ((int64_t)head[u] * kDim + 8 * sub) * 2);
      }
    }
#pragma unroll
    for (int u = 0; u < kStoreSteps; ++u) {
      const bool ok = slot[u] >= 0 && slot[u] < p.pool_slots;
      const int64_t page = ok ? slot[u] / kPage : 0, i = ok ? slot[u] % kPage : 0;
      const int64_t at = page * p.s.kv_page + head[u] * p.s.kv_head;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if constexpr (KEY == kBf16) {
          if (ok) put<FAR>(raw[u][w], p.kv[w] + at + (i * kDim + 8 * sub) * 2);
        } else {
          float v[8], scale;
          bf16x8_to_float(raw[u][w], v);
          const u32x2 codes = quantise<LPV>(v, 1.0f, ok, scale, [&](float (&f)[8]) {
            bf16x8_to_float(raw[u][w], f);
          });
          if (ok) {
            put<FAR>(codes, p.kv[w] + at + i * kDim + 8 * sub);
            if (sub == 0) *reinterpret_cast<float*>(p.ks[w] + page * p.s.ks_page + head[u] * p.s.ks_head + 4 * i) = scale;
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Bounds of pages' keys.

struct Bounds {
  const uint8_t* kv;
  const uint8_t* ks;
  Tables tables;
  const int32_t* first;  // or NULL
  const int32_t* sl;
  uint8_t* out;          // bf16 [pages][heads][2][D]
  KvStrides s;
  uint32_t pages_lim, side;  // side: a row's workgroups that stand together
  int32_t heads, width;
};

constexpr float kBf16Max = 3.3895313892515355e38f;

// The bf16 next to v (finite: clamped) that is no less (UP) or no more.
template <bool UP>
__device__ __forceinline__ uint32_t outwards(float v) {
  const uint32_t bits = __float_as_uint(__builtin_amdgcn_fmed3f(v, -kBf16Max, kBf16Max));
  return ((bits >> 31 != 0) == UP ? bits : bits + 0xffffu) >> 16;
}

// f over the lanes whose number is the same modulo LP, in all of them: turns of a row
// of 16 as operands of the arithmetic itself, then rows and halves of the wave.
template <int LP, class F>
__device__ __forceinline__ float fold_apart(float v, F f) {
  if constexpr (LP <= 4) v = f(v, row_lane<0x124>(v));  // row_ror 4
  if constexpr (LP <= 8) v = f(v, row_lane<0x128>(v));  // row_ror 8
  if constexpr (LP <= 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// A wave takes a page of a head: a lane 16 bytes of a position, 1024 bytes of the
// block a load, all of the block's loads under way at once; then the lanes that
// have the same values of other positions.  Bound by memory: four prompts of up to
// 32768 positions of 8 heads of 128 bf16 values, 199 MB, take 39.5 to 41.5 us, 4.8 to 5.0
// TB/s (41.2 on the card on which columns of 128 bytes, twice the waves, took 42.5, of 64 bytes
// 61.6); in e4m3, 106 MB, 32.2, 3.3 TB/s: twice the vector instructions a byte.
template <int KEY, int DIM>
__global__ __launch_bounds__(kThreads) void page_bounds_kernel(Bounds p) {
  constexpr int kPer = KEY == kFp8 ? 16 : 8;  // values of a lane
  constexpr int LP = DIM / kPer, kLoads = LP, kStep = 64 / LP;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t b = blockIdx.x / p.side, first = ((int64_t)blockIdx.y * p.side + blockIdx.x % p.side) * kWaves + wave;
  bool table_ok;
  const int32_t* tab = p.tables.of(b, table_ok);
  const int64_t L = min((int64_t)max(p.sl[b], 0), (int64_t)p.width * kPage);
  const int64_t j0 = p.first ? max(p.first[b], 0) / kPage : 0, j1 = (L + kPage - 1) / kPage;
  if (!table_ok || j0 >= j1) return;
  const int64_t items = (j1 - j0) * p.heads;
  for (int64_t item = first; item < items; item += (int64_t)gridDim.y * p.side * kWaves) {
    const int64_t over = items <= UINT32_MAX ? (uint32_t)item / (uint32_t)p.heads : item / p.heads;
    const int64_t j = j0 + over, h = item - over * p.heads;
    const int32_t page = tab[j];
    if ((uint32_t)page >= p.pages_lim) continue;
    const int live = (int)min(L - j * kPage, (int64_t)kPage);
    const uint8_t* block = p.kv + (int64_t)page * p.s.kv_page + h * p.s.kv_head;
    const float* scales = reinterpret_cast<const float*>(p.ks + (int64_t)page * p.s.ks_page + h * p.s.ks_head);
    u32x4 raw[kLoads];
    float scale[kLoads];
    if constexpr (KEY == kFp8) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) scale[i] = scales[kStep * i + lane / LP];
    }
    // (past the caches, whatever the sizes: four prompts, 199 MB, 46.9 -> 41.2 us, a decode
    // step of 64 rows, 3.5 MB, 5.15 -> 5.3; asking for the size first cost 4 of the 6)
#pragma unroll
    for (int i = 0; i < kLoads; ++i) raw[i] = get<true>(block + 1024 * i + 16 * lane);
    if (live < kPage) {  // positions past the row's end: no numbers, which have no part
      const uint32_t nan = KEY == kFp8 ? 0x7f7f7f7fu : 0x7fc07fc0u;
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        if (kStep * i + lane / LP >= live) raw[i] = (u32x4){nan, nan, nan, nan};
    }
    float lo[kPer], hi[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) lo[e] = INFINITY, hi[e] = -INFINITY;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      float v[kPer];
      if constexpr (KEY == kFp8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(raw[i][e], false), c = __builtin_amdgcn_cvt_pk_f32_fp8(raw[i][e], true);
          v[4 * e] = a[0] * scale[i], v[4 * e + 1] = a[1] * scale[i];
          v[4 * e + 2] = c[0] * scale[i], v[4 * e + 3] = c[1] * scale[i];
        }
      } else {
        bf16x8_to_float(raw[i], v);
        quiet(v);
      }
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        lo[e] = fminf(lo[e], v[e]);
        hi[e] = fmaxf(hi[e], v[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      lo[e] = fold_apart<LP>(lo[e], [](float a, float b) { return fminf(a, b); });
      hi[e] = fold_apart<LP>(hi[e], [](float a, float b) { return fmaxf(a, b); });
    }
    if (lane >= 2 * LP) continue;
    const bool up = lane >= LP;
    uint32_t word[kPer / 2];
#pragma unroll
    for (int e = 0; e < kPer; e += 2) {
      uint32_t two[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool none = lo[e + k] > hi[e + k];
        two[k] = none ? 0u : up ? outwards<true>(hi[e + k]) : outwards<false>(lo[e + k]);
      }
      word[e / 2] = two[0] | two[1] << 16;
    }
    uint8_t* to = p.out + (((int64_t)page * p.heads + h) * 2 * DIM + lane * kPer) * 2;
#pragma unroll
    for (int e = 0; e < kPer / 8; ++e)
      *reinterpret_cast<u32x4*>(to + 16 * e) = (u32x4){word[4 * e], word[4 * e + 1], word[4 * e + 2], word[4 * e + 3]};
  }
}

// ---------------------------------------------------------------------------
// Scores of pages.

struct Scores {
  const uint8_t* q;
  const uint8_t* bounds;
  Tables tables;
  const int32_t* sl;
  float* out;
  int32_t* counts;  // or NULL
  int64_t out_stride, blocks;
  uint32_t pages_lim;
  int32_t rows, heads, kv_heads, width, first, last;
};

// max(q lo, q hi) is q hi where q is positive and q lo where it is negative, so the
// sum is a product of [min(q, 0), max(q, 0)] with [lo, hi]: bf16 matrix instructions
// with exact products and float32 sums.  A row's tiles are 16 pages of a head, heads
// first, whose bounds stand side by side; a wave takes one: its bounds, whole rows, to
// LDS by DMA, from there as the B operand against 16 query heads at a time; a lane then
// has 4 heads of a page.  64 rows of up to 512 pages, 87 MB, take 18.2 us, 4.8 TB/s (bounds
// as operands straight from memory, 64 bytes of 16 pages a load, 21.1); 4097 pages of one
// row 5.9, a launch and two trips to memory.
__device__ const u32x4 kZeroBounds[4 * 256 / 16] = {};  // of pages that are none

template <int DIM>
__global__ __launch_bounds__(kThreads) void page_scores_kernel(Scores p) {
  constexpr int kSteps = DIM / 32, kRowBytes = 4 * DIM, kChunks = kRowBytes / 16, kRowsPerDma = 1024 / kRowBytes;
  // chunk c (16 bytes) of row r stands at place c ^ r: 16 lanes read one chunk of 16 rows
  __shared__ __attribute__((aligned(1024))) uint8_t rows[kWaves][16 * kRowBytes];
  const int lane = threadIdx.x & 63, n = lane & 15, quad = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t lds = (uint32_t)(uintptr_t)(lds_u8*)&rows[wave][0];
  const int32_t group = p.heads / p.kv_heads;
  const int64_t units = (int64_t)p.rows * p.blocks;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t b = units <= UINT32_MAX ? (uint32_t)unit / (uint32_t)p.blocks : unit / p.blocks;
    const uint32_t tile = (uint32_t)(unit - b * p.blocks) * kWaves + wave, at = tile / (uint32_t)p.kv_heads;
    const int32_t h = (int32_t)(tile - at * (uint32_t)p.kv_heads), j = (int32_t)(16 * at) + n;
    const int32_t L = p.sl[b];
    bool table_ok;
    const int32_t* tab = p.tables.of(b, table_ok);
    const int32_t page = j < p.width && table_ok ? tab[j] : -1;  // (before the length is there)
    const int32_t count = min((max(L, 0) - 1) / kPage + (L > 0), p.width);
    const int64_t row = b * p.kv_heads + h;
    u32x4 q[kSteps];  // of 16 query heads (past the group's last: its last)
    const auto queries = [&](int32_t i) {
      const uint8_t* from = p.q + ((b * p.heads + (int64_t)h * group + min(i + n, group - 1)) * DIM + 8 * quad) * 2;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) q[s] = *reinterpret_cast<const u32x4*>(from + 64 * s);
    };
    float best = -INFINITY;
    if (j - n < count) {
      queries(0);
      const bool ok = (uint32_t)page < p.pages_lim && j < count;
      const uint64_t row_at = (uint64_t)(ok ? p.bounds + ((int64_t)page * p.kv_heads + h) * kRowBytes : reinterpret_cast<const uint8_t*>(kZeroBounds));
#pragma unroll
      for (int i = 0; i < 16 / kRowsPerDma; ++i) {
        const int r = kRowsPerDma * i + lane / kChunks;
        const uint64_t at_r = (uint64_t)(uint32_t)__shfl((int)(row_at >> 32), r) << 32 | (uint32_t)__shfl((int)row_at, r);
        dma16(reinterpret_cast<const uint8_t*>(at_r) + 16 * ((lane % kChunks) ^ r), lds + 1024 * i);
      }
      wait_vm<0>();
      bf16x8 side[2][kSteps];
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
          side[w][s] = *reinterpret_cast<const bf16x8*>(&rows[wave][n * kRowBytes + 16 * ((w * (DIM / 8) + 4 * s + quad) ^ n)]);
      for (int32_t i = 0;;) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          u32x4 neg, pos;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t sign = (q[s][e] >> 15 & 0x00010001u) * 0xffffu;
            neg[e] = q[s][e] & sign;
            pos[e] = q[s][e] & ~sign;
          }
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, neg), side[0][s], acc, 0, 0, 0);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, pos), side[1][s], acc, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) best = __builtin_elementwise_maximum(best, acc[e]);  // (a NaN stays)
        i += 16;
        if (i >= group) break;
        queries(i);
      }
      best = __builtin_elementwise_maximum(best, __shfl_xor(best, 16));
      best = __builtin_elementwise_maximum(best, __shfl_xor(best, 32));
      if (!ok) best = __builtin_nanf("");
    }
    if (j < p.first || j >= (int64_t)count - p.last) best = INFINITY;
    if (j >= count) best = -INFINITY;
    if (quad == 0 && j < p.width) p.out[row * p.out_stride + j] = best;
    if (p.counts && quad == 0 && j == 0) p.counts[row] = count;
  }
}

// ---------------------------------------------------------------------------
// Host side.

template <class F>
int for_dim(int32_t head_dim, F f) {
  switch (head_dim) {
    case 64: f(std::integral_constant<int, 64>{}); break;
    case 128: f(std::integral_constant<int, 128>{}); break;
    default: f(std::integral_constant<int, 256>{});
  }
  return launch_status();
}

template <int KEY>
int store_kv(const void* keys, const void* values, const int64_t* slots, int64_t n, int32_t kv_heads,
             int32_t head_dim, int64_t k_row_stride, int64_t v_row_stride, void* k_pages, void* v_pages,
             float* kscale, float* vscale, int64_t num_pages, const KvStrides& s, hipStream_t stream) {
  if (!head_dim_ok(head_dim)) return IDX_ERR_UNSUPPORTED;
  const int64_t most = (int64_t)1 << 32;
  if (n < 0 || kv_heads < 0 || n > ((int64_t)1 << 32) || k_row_stride < (int64_t)kv_heads * head_dim ||
      v_row_stride < (int64_t)kv_heads * head_dim || k_row_stride > most || v_row_stride > most)
    return IDX_ERR_SHAPE;
  int st = validate_kv_strides(KEY, kv_heads, head_dim, num_pages, s);
  if (st != IDX_OK || n == 0 || kv_heads == 0) return st;
  if (!keys || !values || !slots) return IDX_ERR_NULL;
  st = validate_kv_pointers(KEY, kv_heads, k_pages, kscale, s);
  if (st == IDX_OK) st = validate_kv_pointers(KEY, kv_heads, v_pages, vscale, s);
  if (st != IDX_OK) return st;
  if (!aligned(keys, 16) || !aligned(values, 16) || k_row_stride % 8 != 0 || v_row_stride % 8 != 0 || !aligned(slots, 8))
    return IDX_ERR_ALIGN;
  Store p;
  p.x[0] = static_cast<const uint8_t*>(keys);
  p.x[1] = static_cast<const uint8_t*>(values);
  p.kv[0] = static_cast<uint8_t*>(k_pages);
  p.kv[1] = static_cast<uint8_t*>(v_pages);
  p.ks[0] = reinterpret_cast<uint8_t*>(kscale);
  p.ks[1] = reinterpret_cast<uint8_t*>(vscale);
  p.slots = slots;
  p.x_stride[0] = 2 * k_row_stride;
  p.x_stride[1] = 2 * v_row_stride;
  p.vectors = n * kv_heads;
  p.pool_slots = num_pages * kPage;
  p.s = s;
  p.heads = kv_heads;
  (void)hipGetLastError();  // start from a clean error state
  return for_dim(head_dim, [&](auto dim) {
    constexpr int LPV = decltype(dim)::value / 8, kUnit = kStoreSteps * kWaves * (64 / LPV);
    const int64_t units = (p.vectors + kUnit - 1) / kUnit, cap = 16 * device_cu_count();
    const dim3 grid((uint32_t)(units < cap ? units : cap));
    if (is_far(p.vectors, LPV * (KEY == kFp8 ? 16 : 32)))
      store_kv_kernel<KEY, LPV, true><<<grid, dim3(kThreads), 0, stream>>>(p);
    else
      store_kv_kernel<KEY, LPV, false><<<grid, dim3(kThreads), 0, stream>>>(p);
  });
}

// The checks that bounds and scores share of a row's pages.
int validate_rows(int32_t rows, int32_t kv_heads, int32_t table_width, int32_t num_tables, int64_t page_table_row_stride) {
  return rows < 0 || kv_heads < 0 || table_width < 0 || table_width > kMaxWidth || num_tables < 0 ||
                 page_table_row_stride < 0 || (int64_t)rows * kv_heads > INT32_MAX
             ? IDX_ERR_SHAPE
             : IDX_OK;
}

template <int KEY>
int page_bounds(const void* k_pages, const float* kscale, const int32_t* page_table, const int32_t* row_table,
                int32_t num_tables, const int32_t* first, const int32_t* seqlens, void* bounds, int32_t rows,
                int32_t kv_heads, int32_t head_dim, int32_t table_width, int64_t num_pages, const KvStrides& s,
                int64_t page_table_row_stride, hipStream_t stream) {
  if (!head_dim_ok(head_dim)) return IDX_ERR_UNSUPPORTED;
  int st = validate_rows(rows, kv_heads, table_width, num_tables, page_table_row_stride);
  if (st == IDX_OK) st = validate_kv_strides(KEY, kv_heads, head_dim, num_pages, s);
  const int64_t side = ((int64_t)kv_heads + kWaves - 1) / kWaves;
  if (st == IDX_OK && rows * side >= ((int64_t)1 << 32) / kThreads) st = IDX_ERR_SHAPE;  // (a launch has less than 2^32 threads)
  if (st != IDX_OK || rows == 0 || kv_heads == 0 || table_width == 0) return st;
  if (!page_table || !seqlens || !bounds) return IDX_ERR_NULL;
  st = validate_kv_pointers(KEY, kv_heads, k_pages, kscale, s);
  if (st != IDX_OK) return st;
  if (!aligned(page_table, 4) || !aligned(row_table, 4) || !aligned(first, 4) || !aligned(seqlens, 4) || !aligned(bounds, 16))
    return IDX_ERR_ALIGN;
  Bounds p;
  p.kv = static_cast<const uint8_t*>(k_pages);
  p.ks = reinterpret_cast<const uint8_t*>(kscale);
  p.tables = {page_table, row_table, page_table_row_stride, num_tables};
  p.first = first;
  p.sl = seqlens;
  p.out = static_cast<uint8_t*>(bounds);
  p.s = s;
  p.pages_lim = pages_limit(num_pages);
  p.heads = kv_heads;
  p.width = table_width;
  (void)hipGetLastError();
  // The workgroups of one page of a row, then those of the next row: what the rows have
  // of a decode step so is all dies', and neighbours read neighbouring blocks.
  p.side = (uint32_t)side;
  int64_t y = table_width;
  const int64_t cap = (16 * (int64_t)device_cu_count() + (int64_t)rows * p.side - 1) / ((int64_t)rows * p.side);
  if (y > cap) y = cap;
  return for_dim(head_dim, [&](auto dim) {
    page_bounds_kernel<KEY, decltype(dim)::value><<<dim3((uint32_t)rows * p.side, (uint32_t)y), dim3(kThreads), 0, stream>>>(p);
  });
}

}  // namespace

extern "C" {

int idx_plan_batch(const int32_t* cached, const int32_t* added, int32_t requests, const int32_t* free_pages,
                   int64_t num_free, int32_t* page_table, int32_t table_width, int64_t page_table_row_stride,
                   int64_t n, int64_t* slots, int64_t* positions, int32_t* row_table, int32_t* seqlens,
                   int64_t* starts, int64_t* taken, hipStream_t stream) {
  if (requests < 0 || requests > 65536 || num_free < 0 || table_width < 0 || table_width > kMaxWidth || n < 0 ||
      n > ((int64_t)1 << 40) || page_table_row_stride < 0 || (requests > 1 && page_table_row_stride < table_width))
    return IDX_ERR_SHAPE;
  if (n == 0 && requests == 0 && !starts && !taken) return IDX_OK;
  if ((requests > 0 && (!cached || !added || (table_width > 0 && !page_table))) || (num_free > 0 && !free_pages))
    return IDX_ERR_NULL;
  if (!aligned(cached, 4) || !aligned(added, 4) || !aligned(free_pages, 4) || !aligned(page_table, 4) ||
      !aligned(slots, 8) || !aligned(positions, 8) || !aligned(row_table, 4) || !aligned(seqlens, 4) ||
      !aligned(starts, 8) || !aligned(taken, 8))
    return IDX_ERR_ALIGN;
  const Plan p = {cached, added, free_pages, page_table, slots, positions, row_table, seqlens, starts, taken,
                  num_free, page_table_row_stride, n, requests, table_width};
  (void)hipGetLastError();
  const int threads = requests <= 1024 ? 256 : 1024;
  int64_t grid = (n + threads - 1) / threads;
  if (grid < 1) grid = 1;
  if (grid > 2 * device_cu_count()) grid = 2 * device_cu_count();
  if (threads == 256) plan_kernel<256><<<dim3((uint32_t)grid), dim3(256), 0, stream>>>(p);
  else plan_kernel<1024><<<dim3((uint32_t)grid), dim3(1024), 0, stream>>>(p);
  return launch_status();
}

int idx_store_kv_fp8(const void* keys, const void* values, const int64_t* slots, int64_t n, int32_t kv_heads,
                     int32_t head_dim, int64_t k_row_stride, int64_t v_row_stride, void* k_pages, void* v_pages,
                     float* kscale, float* vscale, int64_t num_pages, int64_t kv_page_stride,
                     int64_t kv_head_stride, int64_t kscale_page_stride, int64_t kscale_head_stride,
                     hipStream_t stream) {
  return store_kv<kFp8>(keys, values, slots, n, kv_heads, head_dim, k_row_stride, v_row_stride, k_pages, v_pages, kscale,
                        vscale, num_pages, {kv_page_stride, kv_head_stride, kscale_page_stride, kscale_head_stride}, stream);
}

int idx_store_kv_bf16(const void* keys, const void* values, const int64_t* slots, int64_t n, int32_t kv_heads,
                      int32_t head_dim, int64_t k_row_stride, int64_t v_row_stride, void* k_pages, void* v_pages,
                      int64_t num_pages, int64_t kv_page_stride, int64_t kv_head_stride, hipStream_t stream) {
  return store_kv<kBf16>(keys, values, slots, n, kv_heads, head_dim, k_row_stride, v_row_stride, k_pages, v_pages, nullptr,
                         nullptr, num_pages, {kv_page_stride, kv_head_stride, 0, 0}, stream);
}

int idx_page_bounds_fp8(const void* k_pages, const float* kscale, const int32_t* page_table,
                        const int32_t* row_table, int32_t num_tables, const int32_t* first,
                        const int32_t* seqlens, void* bounds, int32_t rows, int32_t kv_heads, int32_t head_dim,
                        int32_t table_width, int64_t num_pages, int64_t kv_page_stride, int64_t kv_head_stride,
                        int64_t kscale_page_stride, int64_t kscale_head_stride, int64_t page_table_row_stride,
                        hipStream_t stream) {
  return page_bounds<kFp8>(k_pages, kscale, page_table, row_table, num_tables, first, seqlens, bounds, rows, kv_heads,
                           head_dim, table_width, num_pages,
                           {kv_page_stride, kv_head_stride, kscale_page_stride, kscale_head_stride},
                           page_table_row_stride, stream);
}

int idx_page_bounds_bf16(const void* k_pages, const int32_t* page_table, const int32_t* row_table,
                         int32_t num_tables, const int32_t* first, const int32_t* seqlens, void* bounds,
                         int32_t rows, int32_t kv_heads, int32_t head_dim, int32_t table_width,
                         int64_t num_pages, int64_t kv_page_stride, int64_t kv_head_stride,
                         int64_t page_table_row_stride, hipStream_t stream) {
  return page_bounds<kBf16>(k_pages, nullptr, page_table, row_table, num_tables, first, seqlens, bounds, rows, kv_heads,
                            head_dim, table_width, num_pages, {kv_page_stride, kv_head_stride, 0, 0},
                            page_table_row_stride, stream);
}

int idx_page_scores(const void* q, const void* bounds, const int32_t* page_table, const int32_t* row_table,
                    int32_t num_tables, const int32_t* seqlens, float* scores, int32_t* page_counts,
                    int32_t rows, int32_t num_heads, int32_t kv_heads, int32_t head_dim, int32_t table_width,
                    int64_t num_pages, int64_t page_table_row_stride, int64_t score_stride, int32_t first_pages,
                    int32_t last_pages, hipStream_t stream) {
  if (!head_dim_ok(head_dim) || (int64_t)num_heads > (int64_t)kMaxGroup * kv_heads) return IDX_ERR_UNSUPPORTED;
  const int st = validate_rows(rows, kv_heads, table_width, num_tables, page_table_row_stride);
  if (st != IDX_OK) return st;
  if (num_heads < 0 || (kv_heads > 0 && num_heads % kv_heads != 0) || num_pages < 0 || score_stride < table_width ||
      score_stride > ((int64_t)1 << 32) || first_pages < 0 || last_pages < 0)
    return IDX_ERR_SHAPE;
  if (rows == 0 || kv_heads == 0 || num_heads == 0) return IDX_OK;
  if (!q || !seqlens || (table_width > 0 && (!bounds || !page_table || !scores))) return IDX_ERR_NULL;
  if (!aligned(q, 16) || !aligned(bounds, 16) || !aligned(page_table, 4) || !aligned(row_table, 4) ||
      !aligned(seqlens, 4) || !aligned(scores, 4) || !aligned(page_counts, 4))
    return IDX_ERR_ALIGN;
  Scores p;
  p.q = static_cast<const uint8_t*>(q);
  p.bounds = static_cast<const uint8_t*>(bounds);
  p.tables = {page_table, row_table, page_table_row_stride, num_tables};
  p.sl = seqlens;
  p.out = scores;
  p.counts = page_counts;
  p.out_stride = score_stride;
  // (a table without columns has tiles for the counts)
  p.blocks = ((int64_t)(table_width > 0 ? (table_width + 15) / 16 : 1) * kv_heads + kWaves - 1) / kWaves;
  if (p.blocks > INT32_MAX / kWaves) return IDX_ERR_SHAPE;
  p.pages_lim = pages_limit(num_pages);
  p.rows = rows;
  p.heads = num_heads;
  p.kv_heads = kv_heads;
  p.width = table_width;
  p.first = first_pages;
  p.last = last_pages;
  const int64_t units = (int64_t)rows * p.blocks, cap = (int64_t)1 << 20;
  const dim3 grid((uint32_t)(units < cap ? units : cap));
  (void)hipGetLastError();
  return for_dim(head_dim, [&](auto dim) {
    page_scores_kernel<decltype(dim)::value><<<grid, dim3(kThreads), 0, stream>>>(p);
  });
}

}  // extern "C"
