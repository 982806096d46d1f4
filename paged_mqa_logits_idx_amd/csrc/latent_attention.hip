// latent_attention.hip -- attention over a paged cache of latents (gfx950
// kernels and C-ABI entry points declared in include/latent_cache.h).
//
// Row b attends with H heads of 512 values to the latents c_p of its positions
// p in S_b (a top-k's list, or every position below the row's length); one
// latent is key and value of all heads:
//   x_hp = scale * <q_bh, c_p>
//   z_h  = sum_p exp(x_hp) (+ exp(sink_h)),  out_bh = sum_p exp(x_hp) c_p / z_h
//
// Work decomposition.  A unit is (row, split of its positions, block of HT
// heads), one workgroup of WAVES waves, over tiles of 64 positions.  Each tile
// is gathered once from its pages into LDS by DMA (512 bytes of e4m3 codes or
// 1024 of bf16 a position) while the tile before it is used, and read twice:
//   scores   X^T = C Q^T:  wave w takes position block w % 4 (16 positions) and
//            head group w / 4; the queries stay in registers (B operand), the
//            latents are the A operand, row major in LDS.  A lane then holds 4
//            positions of one head: a softmax maximum is two lane swaps.
//   values   O^T += C^T P^T:  wave w takes 512 / WAVES of the values, of all HT
//            heads; C^T comes out of the same LDS tile through the transposing
//            LDS reads, P^T through a small LDS buffer (64 positions x HT).
// So a latent is moved from memory once a unit and its codes are widened to
// bf16 (exactly) on the way into the matrix units; the position's scale is
// applied to its scores and to its probabilities, in float32.
//
// Running maximum: all waves agree on a reference m_h for each head.  It
// moves, and the sums are rescaled, only when a tile's maximum exceeds it by
// more than 2^8 (of base-2 logits): probabilities then reach 256 instead of 1,
// which costs no precision, and most tiles rescale nothing.
//
// Rounding: scores, exponentials, sums and outputs are float32; the products
// take bf16 operands, which rounds the probability (times the e4m3 scale) once,
// by 2^-9 of itself at most, independently from position to position.  The
// denominator sums the unrounded probabilities.
#include "idx_device.h"

namespace {

constexpr int kTile = 64;           // positions of a tile
constexpr float kLazy = 8.0f;       // base-2 logits that the maximum may exceed its reference by
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef int v2i __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));

// A position that is masked, or whose page id lies outside the pool, is
// gathered from here: it must not bring values of its own into the products.
__device__ const u32x4 kZeroLatent[2 * kLatent / 16] = {};

struct Attend {
  const uint8_t* q;    // bf16 [rows][heads][512]
  const uint8_t* kv;
  const uint8_t* ks;
  const int32_t* pt;
  const int32_t* rt;   // table of each row, or NULL: row b's
  const int32_t* idx;  // [rows][k] (k >= 0)
  const int32_t* sl;
  const float* sinks;  // [heads] or NULL
  uint8_t* out;        // bf16 [rows][heads][512]
  float* lse;          // [rows][heads] or NULL
  float* part;         // splits > 1: [rows][splits][heads][512], then their m and l
  int64_t kv_stride, ks_stride, pt_stride;
  uint32_t pages_lim;  // min(num_pages, 2^31): page ids below it are in the pool
  int32_t rows, heads, width, num_tables;
  int32_t k;           // length of a row's list; -1: every position
  int32_t splits, head_blocks;
  float scale2;        // scale * log2(e)
};

__device__ __forceinline__ int32_t uniform(int32_t x) { return __builtin_amdgcn_readfirstlane(x); }

// The workgroup's waves meet here; their LDS writes before it are visible
// after it.  Memory operations other than LDS ones stay in flight.
__device__ __forceinline__ void barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// 64 lanes x 16 bytes from `src` (each lane its own) to LDS `dst` + 16 * lane.
// In assembly so that the compiler, which would wait for every DMA before any
// LDS read, leaves the order to the explicit waits.
__device__ __forceinline__ void dma16(const uint8_t* src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(dst) : "memory", "m0");
}

__device__ __forceinline__ float max_over_g(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}

// Where chunk c (16 bytes) of position r stands within the position's LDS row:
// rows of a multiple of 256 bytes would put one chunk of all positions into
// the same banks.  16 positions spread over 16 chunks, 8 consecutive ones over
// 8 even offsets (the transposing bf16 reads take pairs of chunks).
__device__ __forceinline__ int swizzle(int c, int r) { return c ^ (((r & 7) << 1) | ((r >> 3) & 1)); }

// The end of a softmax: sums relative to 2^m become outputs (times by * half *
// half) and the log of the denominator, in which a sink's base-2 logit joins.
// 2^(m - ref) is applied in two halves: it may be far below float32's range
// where the sink is far above the scores, and the outputs not yet.
struct Closing {
  float by, half, lse;
};
__device__ __forceinline__ Closing close_sum(float m, float z, float sink) {
  const float top = fmaxf(m, sink), ref = top == -INFINITY ? 0.0f : top;
  Closing c;
  c.half = __builtin_amdgcn_exp2f(0.5f * (m - ref));
  const float total = z * c.half * c.half + __builtin_amdgcn_exp2f(sink - ref);
  c.by = total == 0.0f ? 0.0f : 1.0f / total;
  c.lse = total == 0.0f ? -INFINITY : (ref + log2f(total)) * kLn2;
  return c;
}

template <int KEY, int WAVES, int HT>
struct AttendShared {
  static constexpr int kRowBytes = KEY == kFp8 ? kLatent : 2 * kLatent;
  uint8_t tile[2][kTile * kRowBytes];
  __bf16 p[HT * kTile];      // [head][position], 16-byte chunks swizzled by head
  float mx[HT][4];           // maxima of the tile's position blocks
  float sum[4][HT];
};

template <int KEY, int WAVES, int HT>
__global__ __launch_bounds__(64 * WAVES, 2) void latent_attention_kernel(Attend a) {
  constexpr int kRowBytes = KEY == kFp8 ? kLatent : 2 * kLatent;
  constexpr int kChunks = kRowBytes / 16;           // of a position
  constexpr int NB = HT / 16;                       // head blocks of the unit
  constexpr int NQ = NB / (WAVES / 4);              // head blocks of a wave's scores
  constexpr int kDims = kLatent / WAVES;            // values of a wave's outputs
  constexpr int MB = kDims / 16;
  constexpr int kPerWave = kTile / WAVES;           // positions that a wave gathers
  constexpr int kPerDma = 64 / kChunks;             // positions of one DMA
  __shared__ __attribute__((aligned(16))) AttendShared<KEY, WAVES, HT> sh;

  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);
  const int pb = wave & 3, hg = wave >> 2;

  // Units of one row and split (its head blocks read the same latents) follow
  // each other on one XCD; the last rows, the longest of a causal batch, start
  // first.
  const int32_t at = blockIdx.x >> 3;
  const int32_t hb = at % a.head_blocks;
  const int64_t rs = (int64_t)(at / a.head_blocks) * 8 + (blockIdx.x & 7);
  if (rs >= (int64_t)a.rows * a.splits) return;
  const int32_t b = a.rows - 1 - (int32_t)(rs / a.splits), split = (int32_t)(rs % a.splits);
  const int32_t h0 = hb * HT;

  const int32_t L = min(max(a.sl[b], 0), a.width * kPage);
  const int32_t count = uniform(a.k >= 0 ? min(a.k, L) : L);
  const int32_t tiles = (count + kTile - 1) / kTile;
  const int32_t mine = tiles > split ? (tiles - split + a.splits - 1) / a.splits : 0;
  const int32_t table = a.rt ? a.rt[b] : 0;
  const bool table_ok = !a.rt || (table >= 0 && table < a.num_tables);
  const int32_t* tab = a.pt + (int64_t)(a.rt ? (table_ok ? table : 0) : b) * a.pt_stride;
  const int32_t* idx = a.k >= 0 ? a.idx + (int64_t)b * a.k : nullptr;

  f32x4 acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = (f32x4){0.f, 0.f, 0.f, 0.f};
  float m[NB], sum[NQ];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) m[nb] = -INFINITY;
#pragma unroll
  for (int u = 0; u < NQ; ++u) sum[u] = 0.0f;

  if (mine > 0) {
    // Queries, B operand: lane (n, g) holds head n's values 16*(4s' + g) + 8u .. +8
    // of step s = 2s' + u (e4m3: two steps share a 16-byte chunk of codes), or
    // 8*(4s + g) .. +8 (bf16).  Heads past the last are zero.
    bf16x8 q[NQ][16];
#pragma unroll
    for (int u = 0; u < NQ; ++u) {
      const int32_t h = h0 + 16 * (hg * NQ + u) + n;
      const uint8_t* qh = a.q + ((int64_t)b * a.heads + h) * (2 * kLatent);
#pragma unroll
      for (int s = 0; s < 16; ++s) {
        u32x4 v = {0u, 0u, 0u, 0u};
        const int d = KEY == kFp8 ? 16 * (4 * (s >> 1) + g) + 8 * (s & 1) : 8 * (4 * s + g);
        if (h < a.heads) v = *reinterpret_cast<const u32x4*>(qh + 2 * d);
        q[u][s] = __builtin_bit_cast(bf16x8, v);
      }
    }

    // Lane l follows position 16*pb + l%16 of a tile for the wave's scores
    // (mask and scale), and position kPerWave*wave + l%kPerWave for its DMA.
    // `where`: the position (-1: none).
    auto where = [&](int32_t tile, int at) -> int32_t {
      const int32_t t = tile * kTile + at;
      if (t >= count) return -1;
      if (!idx) return t;
      const int32_t p = idx[t];
      return p >= 0 && p < L ? p : -1;
    };
    // page of a position (-1: none, or its id lies outside the pool)
    auto page_of = [&](int32_t p) -> int32_t {
      if (p < 0 || !table_ok) return -1;
      const int32_t page = tab[p / kPage];
      return page >= 0 && (uint32_t)page < a.pages_lim ? page : -1;
    };
    const uint32_t lds_tile = (uint32_t)(uintptr_t)(lds_u8*)&sh.tile[0][0];
    auto gather = [&](int32_t p, int32_t page, int buf) {
      const uint8_t* src = page >= 0 ? a.kv + (int64_t)page * a.kv_stride + (p % kPage) * kRowBytes
                                     : reinterpret_cast<const uint8_t*>(kZeroLatent);
      const uint32_t lo = (uint32_t)(uintptr_t)src, hi = (uint32_t)((uintptr_t)src >> 32);
#pragma unroll
      for (int d = 0; d < kPerWave / kPerDma; ++d) {
        const int r = d * kPerDma + lane / kChunks;  // of the wave's positions
        const uintptr_t base = ((uintptr_t)__shfl(hi, r) << 32) | __shfl(lo, r);
        const int c = swizzle(lane % kChunks, wave * kPerWave + r);
        dma16(reinterpret_cast<const uint8_t*>(base) + 16 * c,
              lds_tile + (uint32_t)(buf * kTile * kRowBytes + (wave * kPerWave + d * kPerDma) * kRowBytes));
      }
    };

    const int gat = wave * kPerWave + lane % kPerWave, sat = 16 * pb + n;
    int32_t tile = split;
    int32_t gp = where(tile, gat), sp = where(tile, sat);
    int32_t spage = page_of(sp);
    gather(gp, page_of(gp), 0);
    for (int32_t i = 0; i < mine; ++i, tile += a.splits) {
      const int buf = i & 1;
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      barrier();  // the tile is there, and every wave is done with the one before
      // mask and scale of the wave's 16 score positions
      const bool live = sp >= 0, bad = live && spage < 0;
      float ks = 1.0f;
      if (KEY == kFp8 && spage >= 0)
        ks = *reinterpret_cast<const float*>(a.ks + (int64_t)spage * a.ks_stride + 4 * (sp % kPage));
      const uint32_t live_mask = (uint32_t)__ballot(live) & 0xffffu, bad_mask = (uint32_t)__ballot(bad) & 0xffffu;
      if (i + 1 < mine) {
        gp = where(tile + a.splits, gat);
        sp = where(tile + a.splits, sat);
        spage = page_of(sp);
        gather(gp, page_of(gp), buf ^ 1);
      }

      // scores
      const uint8_t* rows = sh.tile[buf];
      f32x4 x[NQ];
#pragma unroll
      for (int u = 0; u < NQ; ++u) x[u] = (f32x4){0.f, 0.f, 0.f, 0.f};
      const int r = 16 * pb + n;
#pragma unroll
      for (int s = 0; s < 16; s += KEY == kFp8 ? 2 : 1) {
        if constexpr (KEY == kFp8) {
          const u32x4 c = *reinterpret_cast<const u32x4*>(rows + r * kRowBytes + 16 * swizzle(4 * (s >> 1) + g, r));
          const bf16x8 c0 = fp8x8_to_bf16x8(c.x, c.y), c1 = fp8x8_to_bf16x8(c.z, c.w);
#pragma unroll
          for (int u = 0; u < NQ; ++u) x[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(c0, q[u][s], x[u], 0, 0, 0);
#pragma unroll
          for (int u = 0; u < NQ; ++u) x[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(c1, q[u][s + 1], x[u], 0, 0, 0);
        } else {
          const bf16x8 c = *reinterpret_cast<const bf16x8*>(rows + r * kRowBytes + 16 * swizzle(4 * s + g, r));
#pragma unroll
          for (int u = 0; u < NQ; ++u) x[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(c, q[u][s], x[u], 0, 0, 0);
        }
      }
      float ksr[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) ksr[e] = KEY == kFp8 ? __shfl(ks, 4 * g + e) : 1.0f;
#pragma unroll
      for (int u = 0; u < NQ; ++u) {
        float top = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = x[u][e] * (a.scale2 * ksr[e]);
          if (bad_mask >> (4 * g + e) & 1) v = __builtin_nanf("");
          if (!(live_mask >> (4 * g + e) & 1)) v = -INFINITY;
          x[u][e] = v;
          top = fmaxf(top, v);
        }
        top = max_over_g(top);
        if (g == 0) sh.mx[16 * (hg * NQ + u) + n][pb] = top;
      }
      barrier();

      // the heads' references; sums follow where one moves
      bool moved = false;
      float to[NB], by[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const f32x4 t = *reinterpret_cast<const f32x4*>(sh.mx[16 * nb + n]);
        const float top = fmaxf(fmaxf(t.x, t.y), fmaxf(t.z, t.w));
        to[nb] = top > m[nb] + kLazy ? top : m[nb];
        by[nb] = to[nb] == m[nb] ? 1.0f : __builtin_amdgcn_exp2f(m[nb] - to[nb]);
        moved |= to[nb] != m[nb];
        m[nb] = to[nb];
      }
      if (__ballot(moved) != 0) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) acc[mb][nb] *= by[nb];
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
          float f = by[u];
#pragma unroll
          for (int nb = NQ; nb < NB; nb += NQ)
            if (hg * NQ == nb) f = by[nb + u];
          sum[u] *= f;
        }
      }
      // probabilities: sums unrounded; times the latent's scale, as bf16, to LDS
#pragma unroll
      for (int u = 0; u < NQ; ++u) {
        float ref = m[u];
#pragma unroll
        for (int nb = NQ; nb < NB; nb += NQ)
          if (hg * NQ == nb) ref = m[nb + u];
        if (ref == -INFINITY) ref = 0.0f;  // nothing live yet: the exponentials are 0
        bf16x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = __builtin_amdgcn_exp2f(x[u][e] - ref);
          sum[u] += p;
          w[e] = (__bf16)(p * ksr[e]);
        }
        const int h = 16 * (hg * NQ + u) + n, c = 2 * pb + (g >> 1);
        *reinterpret_cast<bf16x4*>(&sh.p[h * kTile + 8 * (c ^ (h & 7)) + 4 * (g & 1)]) = w;
      }
      barrier();

      // values
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        bf16x8 w[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int h = 16 * nb + n;
          w[nb] = *reinterpret_cast<const bf16x8*>(&sh.p[h * kTile + 8 * ((4 * s + g) ^ (h & 7))]);
        }
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          bf16x8 v;
          if constexpr (KEY == kFp8) {
            // 16 lanes read 8 positions x 16 values: lanes 2j, 2j+1 the 16
            // codes of position j, lane n gets value n of the 8 positions
            const int r = 32 * s + 8 * g + (n >> 1), c = kDims / 16 * wave + mb;
            const v2i t = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                (__attribute__((address_space(3))) v2i*)(rows + r * kRowBytes + 16 * swizzle(c, r) + 8 * (n & 1)));
            v = fp8x8_to_bf16x8((uint32_t)t.x, (uint32_t)t.y);
          } else {
            // 16 lanes read 4 positions x 16 values: lanes 4j .. 4j+3 the 32
            // bytes of position j
            v4s t[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int r = 32 * s + 8 * g + 4 * j + (n >> 2), c = kDims / 8 * wave + 2 * mb + (n >> 1 & 1);
              t[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                  (__attribute__((address_space(3))) v4s*)(rows + r * kRowBytes + 16 * swizzle(c, r) + 8 * (n & 1)));
            }
            v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(t[0], t[1], 0, 1, 2, 3, 4, 5, 6, 7));
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            acc[mb][nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, w[nb], acc[mb][nb], 0, 0, 0);
        }
      }
    }
  }

  // sums over the position blocks
#pragma unroll
  for (int u = 0; u < NQ; ++u) {
    float s = sum[u];
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (g == 0) sh.sum[pb][16 * (hg * NQ + u) + n] = s;
  }
  barrier();
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int32_t h = h0 + 16 * nb + n;
    if (h >= a.heads) continue;
    float z = (sh.sum[0][16 * nb + n] + sh.sum[1][16 * nb + n]) + (sh.sum[2][16 * nb + n] + sh.sum[3][16 * nb + n]);
    const int64_t head = (int64_t)b * a.heads + h;
    if (a.splits > 1) {
      const int64_t ph = ((int64_t)b * a.splits + split) * a.heads + h;
      float* ml = a.part + (int64_t)a.rows * a.splits * a.heads * kLatent + 2 * ph;
      if (wave == 0 && g == 0) {
        ml[0] = m[nb];
        ml[1] = z;
      }
      if (mine > 0) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
          *reinterpret_cast<f32x4*>(a.part + ph * kLatent + kDims * wave + 16 * mb + 4 * g) = acc[mb][nb];
      }
      continue;
    }
    const Closing c = close_sum(m[nb], z, a.sinks ? a.sinks[h] * kLog2e : -INFINITY);
    if (a.lse && wave == 0 && g == 0) a.lse[head] = c.lse;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      bf16x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = (__bf16)(acc[mb][nb][e] * c.by * c.half * c.half);
      *reinterpret_cast<bf16x4*>(a.out + (head * kLatent + kDims * wave + 16 * mb + 4 * g) * 2) = o;
    }
  }
}

// Joins the splits of a row: one wave a head, 8 values a lane.  The order of
// the splits is fixed, so the result does not depend on their timing.
__global__ __launch_bounds__(256) void latent_combine_kernel(Attend a) {
  const int lane = threadIdx.x & 63;
  const int64_t head = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (head >= (int64_t)a.rows * a.heads) return;
  const int64_t b = head / a.heads;
  const int32_t h = (int32_t)(head % a.heads);
  const float* ml = a.part + (int64_t)a.rows * a.splits * a.heads * kLatent;
  float top = -INFINITY;
  for (int32_t s = 0; s < a.splits; ++s) top = fmaxf(top, ml[2 * ((b * a.splits + s) * a.heads + h)]);
  const float ref = top == -INFINITY ? 0.0f : top;
  float total = 0.0f;
  float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int32_t s = 0; s < a.splits; ++s) {
    const int64_t ph = (b * a.splits + s) * a.heads + h;
    const float m = ml[2 * ph], z = ml[2 * ph + 1];
    if (m == -INFINITY && z == 0.0f) continue;  // nothing live (nothing written, maybe)
    const float f = __builtin_amdgcn_exp2f(m - ref);
    total += z * f;
    const f32x4* src = reinterpret_cast<const f32x4*>(a.part + ph * kLatent + 8 * lane);
    const f32x4 lo = src[0], hi = src[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[e] = fmaf(lo[e], f, o[e]);
      o[4 + e] = fmaf(hi[e], f, o[4 + e]);
    }
  }
  const Closing c = close_sum(top, total, a.sinks ? a.sinks[h] * kLog2e : -INFINITY);
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = o[e] * c.by * c.half * c.half;
  *reinterpret_cast<u32x4*>(a.out + (head * kLatent + 8 * lane) * 2) = float_to_bf16x8(o);
  if (a.lse && lane == 0) a.lse[head] = c.lse;
}

// ---------------------------------------------------------------------------
// Host side.

constexpr int kMaxHeads = 128;
constexpr int kHeadTile = 32;
constexpr int32_t kMaxWidth = 1 << 24;

// Splits of a row's positions: enough units for two workgroups a CU, at least
// two tiles each.  From the scalar arguments alone (the lengths are on the
// device).
int splits_of(int32_t rows, int32_t num_heads, int32_t table_width, int32_t k) {
  const int64_t most = k >= 0 ? (k < (int64_t)table_width * kPage ? k : (int64_t)table_width * kPage)
                                : (int64_t)table_width * kPage;
  const int64_t tiles = (most + kTile - 1) / kTile;
  const int64_t units = (int64_t)rows * ((num_heads + kHeadTile - 1) / kHeadTile);
  int64_t s = 2 * device_cu_count() / (units > 0 ? units : 1);
  if (s > tiles / 2) s = tiles / 2;
  if (s > 64) s = 64;
  return s < 1 ? 1 : (int)s;
}

int64_t workspace_of(int32_t rows, int32_t num_heads, int splits) {
  return splits > 1 ? (int64_t)rows * num_heads * splits * (kLatent + 2) * 4 : 0;
}

bool dims_ok(int32_t rows, int32_t num_heads, int32_t table_width, int32_t k) {
  return rows >= 0 && num_heads >= 0 && num_heads <= kMaxHeads && table_width >= 0 && table_width <= kMaxWidth &&
         k >= -1;
}

template <int KEY>
int latent_attention(const void* q, const void* kv_pages, const float* kscale, const int32_t* page_table,
                     const int32_t* row_table, int32_t num_tables, const int32_t* topk_idx, const int32_t* seqlens,
                     const float* sinks, void* out, float* lse, int32_t rows, int32_t num_heads, int32_t head_dim,
                     int32_t table_width, int64_t num_pages, int64_t kv_page_stride, int64_t kscale_page_stride,
                     int64_t page_table_row_stride, int32_t k, float scale, void* workspace,
                     int64_t workspace_bytes, hipStream_t stream) {
  if (head_dim != kLatent || num_heads > kMaxHeads) return IDX_ERR_UNSUPPORTED;
  if (!dims_ok(rows, num_heads, table_width, k) || page_table_row_stride < 0 || num_tables < 0 ||
      !(scale > -INFINITY && scale < INFINITY) || workspace_bytes < 0)
    return IDX_ERR_SHAPE;
  int st = validate_pool(KEY, kLatent, num_pages, kv_page_stride, kscale_page_stride);
  if (st != IDX_OK || rows == 0 || num_heads == 0) return st;
  if (!q || !seqlens || !out || (table_width > 0 && !page_table) || (k > 0 && !topk_idx) || (k < 0 && topk_idx))
    return IDX_ERR_NULL;
  st = validate_pool_pointers(KEY, kv_pages, kscale, kv_page_stride, kscale_page_stride);
  if (st != IDX_OK) return st;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(page_table, 4) || !aligned(row_table, 4) ||
      !aligned(topk_idx, 4) || !aligned(seqlens, 4) || !aligned(sinks, 4) || !aligned(lse, 4) || !aligned(workspace, 16))
    return IDX_ERR_ALIGN;

  Attend a;
  a.splits = splits_of(rows, num_heads, table_width, k);
  const int64_t need = workspace_of(rows, num_heads, a.splits);
  if (need > 0 && !workspace) return IDX_ERR_NULL;
  if (workspace_bytes < need) return IDX_ERR_SHAPE;
  a.q = static_cast<const uint8_t*>(q);
  a.kv = static_cast<const uint8_t*>(kv_pages);
  a.ks = reinterpret_cast<const uint8_t*>(kscale);
  a.pt = page_table;
  a.rt = row_table;
  a.idx = topk_idx;
  a.sl = seqlens;
  a.sinks = sinks;
  a.out = static_cast<uint8_t*>(out);
  a.lse = lse;
  a.part = static_cast<float*>(workspace);
  a.kv_stride = kv_page_stride;
  a.ks_stride = kscale_page_stride;
  a.pt_stride = page_table_row_stride;
  a.pages_lim = (uint32_t)(num_pages < ((int64_t)1 << 31) ? num_pages : ((int64_t)1 << 31));
  a.rows = rows;
  a.heads = num_heads;
  a.width = table_width;
  a.k = k;
  a.num_tables = num_tables;
  a.head_blocks = (num_heads + kHeadTile - 1) / kHeadTile;
  a.scale2 = scale * kLog2e;
  const int64_t groups = ((int64_t)rows * a.splits + 7) / 8 * a.head_blocks;
  if (groups > (int64_t)1 << 28) return IDX_ERR_SHAPE;
  (void)hipGetLastError();  // start from a clean error state
  if constexpr (KEY == kFp8)
    latent_attention_kernel<KEY, 8, kHeadTile><<<dim3((uint32_t)(8 * groups)), dim3(512), 0, stream>>>(a);
  else
    latent_attention_kernel<KEY, 8, kHeadTile><<<dim3((uint32_t)(8 * groups)), dim3(512), 0, stream>>>(a);
  if (a.splits > 1)
    latent_combine_kernel<<<dim3((uint32_t)(((int64_t)rows * num_heads + 3) / 4)), dim3(256), 0, stream>>>(a);
  return launch_status();
}

}  // namespace

extern "C" {

int64_t idx_latent_attention_workspace(int32_t rows, int32_t num_heads, int32_t table_width, int32_t k) {
  if (!dims_ok(rows, num_heads, table_width, k)) return -1;
  return workspace_of(rows, num_heads, splits_of(rows, num_heads, table_width, k));
}

int idx_latent_attention_fp8(const void* q, const void* kv_pages, const float* kscale, const int32_t* page_table,
                             const int32_t* row_table, int32_t num_tables, const int32_t* topk_idx,
                             const int32_t* seqlens, const float* sinks, void* out, float* lse, int32_t rows,
                             int32_t num_heads, int32_t head_dim, int32_t table_width, int64_t num_pages,
                             int64_t kv_page_stride, int64_t kscale_page_stride, int64_t page_table_row_stride,
                             int32_t k, float scale, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  return latent_attention<kFp8>(q, kv_pages, kscale, page_table, row_table, num_tables, topk_idx, seqlens, sinks, out,
                                lse, rows, num_heads, head_dim, table_width, num_pages, kv_page_stride,
                                kscale_page_stride, page_table_row_stride, k, scale, workspace, workspace_bytes,
                                stream);
}

int idx_latent_attention_bf16(const void* q, const void* kv_pages, const int32_t* page_table,
                              const int32_t* row_table, int32_t num_tables, const int32_t* topk_idx,
                              const int32_t* seqlens, const float* sinks, void* out, float* lse, int32_t rows,
                              int32_t num_heads, int32_t head_dim, int32_t table_width, int64_t num_pages,
                              int64_t kv_page_stride, int64_t page_table_row_stride, int32_t k, float scale,
                              void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  return latent_attention<kBf16>(q, kv_pages, nullptr, page_table, row_table, num_tables, topk_idx, seqlens, sinks,
                                 out, lse, rows, num_heads, head_dim, table_width, num_pages, kv_page_stride, 0,
                                 page_table_row_stride, k, scale, workspace, workspace_bytes, stream);
}

}  // extern "C"
