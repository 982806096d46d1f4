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
#include <type_traits>

#include "idx_device.h"

namespace {

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
  uint32_t pages_lim;  // page ids below it are in the pool
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
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(dst) : "memory");
}

__device__ __forceinline__ void dma4(const uint8_t* src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "s"(dst) : "memory");
}
// Waits until at most N vector-memory operations are outstanding.
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
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

// Tile shapes: 32 KiB of latents either way, and as many waves as it takes for
// each to hold its part of the queries and of the outputs in registers.
template <int KEY>
struct Shape {
  static constexpr int kTile = KEY == kFp8 ? 64 : 32;                     // positions of a tile
  static constexpr int kRowBytes = KEY == kFp8 ? kLatent : 2 * kLatent;   // of a position
  static constexpr int kWaves = 8, HT = 64;
  static constexpr int kChunks = kRowBytes / 16;    // of a position
  static constexpr int NB = HT / 16;                // head blocks
  static constexpr int PB = kTile / 16;             // position blocks
  static constexpr int HG = kWaves / PB;            // head groups: a wave scores one position block x one group
  static constexpr int NQ = NB / HG;                // head blocks of a group
  static constexpr int kDims = kLatent / kWaves;    // values of a wave's outputs
  static constexpr int MB = kDims / 16;
  static constexpr int kGather = kTile / kWaves;    // positions that a wave gathers
  static constexpr int kPerDma = 64 / kChunks;      // positions of one DMA
  static constexpr int kDmaOps = kGather / kPerDma + (KEY == kFp8 ? 1 : 0);  // of a wave and tile, scales included
  static constexpr int kBuffers = 4;
  static constexpr int kRing = 2048 / kTile;        // tiles whose positions are resolved ahead
};

template <int KEY>
struct AttendShared {
  using S = Shape<KEY>;
  uint8_t tile[S::kBuffers][S::kTile * S::kRowBytes];
  float scale[S::kBuffers][S::kTile];   // e4m3 scales of the tiles' positions
  uint32_t ref[S::kRing][S::kTile];     // slots of the positions (64 * page + i), or kMasked, kBad
  __bf16 p[2][S::HT * S::kTile];        // [head][position], 16-byte chunks swizzled by head
  float mx[S::HT][S::PB];               // maxima of the tile's position blocks
  float sum[S::PB][S::HT];
};

constexpr uint32_t kMasked = 0xffffffffu;  // no position
constexpr uint32_t kBad = 0xfffffffeu;     // its page id lies outside the pool
constexpr int64_t kMaxPages = (int64_t)1 << 25;  // 64 * page + i stays below kBad (and 2^25 pages are a TiB)

template <int KEY>
__global__ __launch_bounds__(512, 2) void latent_attention_kernel(Attend a) {
  using S = Shape<KEY>;
  constexpr int kTile = S::kTile, kRowBytes = S::kRowBytes, NB = S::NB, NQ = S::NQ, MB = S::MB, PB = S::PB;
  __shared__ __attribute__((aligned(16))) AttendShared<KEY> sh;

  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);
  const int pb = wave % PB, hg = wave / PB;

  // Units of one row and split (its head blocks read the same latents) follow
  // each other on one XCD; the last rows, the longest of a causal batch, start
  // first.
  const int32_t at = blockIdx.x >> 3;
  const int32_t hb = at % a.head_blocks;
  const int64_t rs = (int64_t)(at / a.head_blocks) * 8 + (blockIdx.x & 7);
  if (rs >= (int64_t)a.rows * a.splits) return;
  const int32_t b = a.rows - 1 - (int32_t)(rs / a.splits), split = (int32_t)(rs % a.splits);
  const int32_t h0 = hb * S::HT;

  const int32_t L = uniform(min(max(a.sl[b], 0), a.width * kPage));
  const int32_t count = a.k >= 0 ? min(a.k, L) : L;
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
    // Slots of the positions of the unit's tiles [j0, j0 + n), `many` a thread
    // at once.
    auto resolve = [&](int32_t j0, int32_t n, auto many) {
      constexpr int kMany = decltype(many)::value;
#pragma unroll 1
      for (int32_t i0 = threadIdx.x; i0 < n * kTile; i0 += kMany * 512) {
        int32_t p[kMany], page[kMany];
#pragma unroll
        for (int e = 0; e < kMany; ++e) {
          const int32_t i = i0 + e * 512, t = (split + (j0 + i / kTile) * a.splits) * kTile + i % kTile;
          p[e] = -1;
          if (i < n * kTile && t < count) p[e] = idx ? idx[t] : t;
        }
#pragma unroll
        for (int e = 0; e < kMany; ++e) {
          page[e] = -1;
          if (p[e] >= 0 && p[e] < L && table_ok) page[e] = tab[p[e] / kPage];
        }
#pragma unroll
        for (int e = 0; e < kMany; ++e) {
          const int32_t i = i0 + e * 512;
          uint32_t r = kMasked;
          if (p[e] >= 0 && p[e] < L)
            r = page[e] >= 0 && (uint32_t)page[e] < a.pages_lim ? (uint32_t)page[e] * kPage + p[e] % kPage : kBad;
          if (i < n * kTile) sh.ref[(j0 + i / kTile) % S::kRing][i % kTile] = r;
        }
      }
    };
    const uint32_t lds_tile = (uint32_t)(uintptr_t)(lds_u8*)&sh.tile[0][0];
    const uint32_t lds_scale = (uint32_t)(uintptr_t)(lds_u8*)&sh.scale[0][0];
    // Tile j into its buffer; every wave issues kDmaOps operations.
    auto gather = [&](int32_t j) {
      int lane = threadIdx.x & 63; asm volatile("" : "+v"(lane)); 
      const int buf = j % S::kBuffers;
      const uint32_t* ref = sh.ref[j % S::kRing];
#pragma unroll
      for (int d = 0; d < S::kGather / S::kPerDma; ++d) {
        const int first = S::kGather * wave + d * S::kPerDma, r = first + lane / S::kChunks;
        const uint32_t slot = ref[r];
        const uint8_t* src = slot < kBad ? a.kv + (int64_t)(slot / kPage) * a.kv_stride + (slot % kPage) * kRowBytes
                                         : reinterpret_cast<const uint8_t*>(kZeroLatent);
        dma16(src + 16 * swizzle(lane % S::kChunks, r), lds_tile + (uint32_t)((buf * kTile + first) * kRowBytes));
      }
      if constexpr (KEY == kFp8) {
        const uint32_t slot = ref[S::kGather * wave + lane % S::kGather];
        const uint8_t* src = slot < kBad ? a.ks + (int64_t)(slot / kPage) * a.ks_stride + 4 * (slot % kPage)
                                         : reinterpret_cast<const uint8_t*>(kZeroLatent);
        if (lane < S::kGather) dma4(src, lds_scale + (uint32_t)((buf * kTile + S::kGather * wave) * 4));
      }
    };

    // Queries: by DMA into the tile buffers, rows of 1 KiB as they stand in
    // memory, while the first slots are resolved; from there to registers as
    // the B operand.  Lane (n, g) holds head n's values 16*(4s' + g) + 8u .. +8
    // of step s = 2s' + u (e4m3: two steps share a 16-byte chunk of codes), or
    // 8*(4s + g) .. +8 (bf16).  Heads past the last are zero.  (Loading the
    // fragments from memory took 16 bytes of 64 lines an instruction: 7 us a
    // unit instead of 2.)
#pragma unroll
    for (int e = 0; e < S::HT / S::kWaves; ++e) {
      const int h = S::kWaves * e + wave;
      const uint8_t* src = h0 + h < a.heads ? a.q + ((int64_t)b * a.heads + h0 + h) * (2 * kLatent)
                                            : reinterpret_cast<const uint8_t*>(kZeroLatent);
      dma16(src + 16 * swizzle(lane, h), lds_tile + (uint32_t)(h * 2 * kLatent));
    }
    resolve(0, min(mine, S::kRing), std::integral_constant<int, 4>{});
    wait_vm<0>();
    barrier();
    bf16x8 q[NQ][16];
#pragma unroll
    for (int u = 0; u < NQ; ++u) {
      const int h = 16 * (hg * NQ + u) + n;
#pragma unroll
      for (int s = 0; s < 16; ++s) {
        const int c = KEY == kFp8 ? 2 * (4 * (s >> 1) + g) + (s & 1) : 4 * s + g;
        q[u][s] = *reinterpret_cast<const bf16x8*>(&sh.tile[0][0] + h * 2 * kLatent + 16 * swizzle(c, h));
      }
    }
    barrier();
    for (int32_t j = 0; j < min(mine, 3); ++j) gather(j);

    f32x4 x[NQ];  // scores of the wave's positions 16*pb + 4*g + e and heads 16*(hg*NQ + u) + n
    auto score = [&](int32_t j) {
      int lane = threadIdx.x & 63; asm volatile("" : "+v"(lane)); const int n = lane & 15, g = lane >> 4; 
      const uint8_t* rows = sh.tile[j % S::kBuffers];
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
      const u32x4 ref = *reinterpret_cast<const u32x4*>(&sh.ref[j % S::kRing][16 * pb + 4 * g]);
      f32x4 by = {a.scale2, a.scale2, a.scale2, a.scale2};
      if constexpr (KEY == kFp8) by *= *reinterpret_cast<const f32x4*>(&sh.scale[j % S::kBuffers][16 * pb + 4 * g]);
#pragma unroll
      for (int u = 0; u < NQ; ++u) {
        float top = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = x[u][e] * by[e];
          if (ref[e] >= kBad) v = ref[e] == kBad ? __builtin_nanf("") : -INFINITY;
          x[u][e] = v;
          top = fmaxf(top, v);
        }
        top = max_over_g(top);
        if (g == 0) sh.mx[16 * (hg * NQ + u) + n][pb] = top;
      }
    };

    // The references that the tile's maxima leave, and its probabilities.  Sums
    // take them unrounded; times the latent's scale, as bf16, they go to LDS.
    auto probabilities = [&](int32_t j) {
      float by[NB];  // what the sums so far are to be multiplied with
      bool moved = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float top = sh.mx[16 * nb + n][0];
#pragma unroll
        for (int k = 1; k < PB; ++k) top = fmaxf(top, sh.mx[16 * nb + n][k]);
        const float to = top > m[nb] + kLazy ? top : m[nb];
        by[nb] = to == m[nb] ? 1.0f : __builtin_amdgcn_exp2f(m[nb] - to);
        moved |= to != m[nb];
        m[nb] = to;
      }
      f32x4 ks = {1.f, 1.f, 1.f, 1.f};
      if constexpr (KEY == kFp8) ks = *reinterpret_cast<const f32x4*>(&sh.scale[j % S::kBuffers][16 * pb + 4 * g]);
#pragma unroll
      for (int u = 0; u < NQ; ++u) {
        float ref = m[u], f = by[u];
#pragma unroll
        for (int nb = NQ; nb < NB; nb += NQ) {
          ref = hg * NQ == nb ? m[nb + u] : ref;
          f = hg * NQ == nb ? by[nb + u] : f;
        }
        if (ref == -INFINITY) ref = 0.0f;  // nothing live yet: the exponentials are 0
        float part = 0.0f;
        bf16x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = __builtin_amdgcn_exp2f(x[u][e] - ref);
          part += p;
          w[e] = (__bf16)(p * ks[e]);
        }
        sum[u] = sum[u] * f + part;
        const int h = 16 * (hg * NQ + u) + n, c = 2 * pb + (g >> 1);
        *reinterpret_cast<bf16x4*>(&sh.p[j & 1][h * kTile + 8 * (c ^ (h & (kTile / 8 - 1))) + 4 * (g & 1)]) = w;
      }
      if (__ballot(moved) != 0) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) acc[mb][nb] *= by[nb];
      }
    };
    auto accumulate = [&](int32_t j) {
      int lane = threadIdx.x & 63; asm volatile("" : "+v"(lane)); const int n = lane & 15, g = lane >> 4; 
      const uint8_t* rows = sh.tile[j % S::kBuffers];
#pragma unroll
      for (int s = 0; s < kTile / 32; ++s) {
        bf16x8 w[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int h = 16 * nb + n;
          w[nb] = *reinterpret_cast<const bf16x8*>(&sh.p[j & 1][h * kTile + 8 * ((4 * s + g) ^ (h & (kTile / 8 - 1)))]);
        }
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          bf16x8 v;
          if constexpr (KEY == kFp8) {
            // 16 lanes read 8 positions x 16 values: lanes 2j, 2j+1 the 16
            // codes of position j, lane n gets value n of the 8 positions
            const int r = 32 * s + 8 * g + (n >> 1), c = MB * wave + mb;
            const v2i t = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                (__attribute__((address_space(3))) v2i*)(rows + r * kRowBytes + 16 * swizzle(c, r) + 8 * (n & 1)));
            v = fp8x8_to_bf16x8((uint32_t)t.x, (uint32_t)t.y);
          } else {
            // 16 lanes read 4 positions x 16 values: lanes 4j .. 4j+3 the 32
            // bytes of position j
            v4s t[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int r = 32 * s + 8 * g + 4 * k + (n >> 2), c = 2 * (MB * wave + mb) + (n >> 1 & 1);
              t[k] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                  (__attribute__((address_space(3))) v4s*)(rows + r * kRowBytes + 16 * swizzle(c, r) + 8 * (n & 1)));
            }
            v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(t[0], t[1], 0, 1, 2, 3, 4, 5, 6, 7));
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            acc[mb][nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, w[nb], acc[mb][nb], 0, 0, 0);
        }
      }
    };

    // A tile has arrived when at most the operations of the tiles issued after
    // it are outstanding (they complete in order).
    // While tile j + 1 is scored, tiles j + 2 and j + 3 are on their way; tile
    // j's latents are added up before its successor's probabilities are taken.
    for (int32_t j = -1; j < mine; ++j) {
      const bool more = j + 1 < mine;
      if (more) {
        if (j + 3 < mine && j < 0) wait_vm<2 * S::kDmaOps>();
        else if (j + 2 < mine) wait_vm<S::kDmaOps>();
        else wait_vm<0>();
      }
      barrier();  // tile j + 1 and tile j's probabilities are there; every wave is done with tile j - 1
      if (j >= 0 && j + 3 < mine) {
        gather(j + 3);
        // half of the ring anew, past the tiles whose slots are still read
        constexpr int kHalf = S::kRing / 2;
        if (j - 1 >= kHalf && (j - 1) % kHalf == 0 && j - 1 + kHalf < mine)
          resolve(j - 1 + kHalf, min(kHalf, mine - (j - 1 + kHalf)), std::integral_constant<int, 1>{});
      }
      if (more) score(j + 1);
      barrier();
      if (j >= 0) accumulate(j);
      if (more) probabilities(j + 1);
    }
    barrier();
  }

  // Sums over the position blocks, and the outputs of all waves as rows of
  // float32 in the tile buffers, so that they leave in whole lines.
#pragma unroll
  for (int u = 0; u < NQ; ++u) {
    float s = sum[u];
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (g == 0) sh.sum[pb][16 * (hg * NQ + u) + n] = s;
  }
  barrier();
  uint8_t* rows = &sh.tile[0][0];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int h = 16 * nb + n;
    float z = sh.sum[0][h];
#pragma unroll
    for (int k = 1; k < PB; ++k) z += sh.sum[k][h];
    float by = 1.0f, half = 1.0f;
    if (a.splits > 1) {
      const int64_t ph = ((int64_t)b * a.splits + split) * a.heads + h0 + h;
      float* ml = a.part + (int64_t)a.rows * a.splits * a.heads * kLatent + 2 * ph;
      if (h0 + h < a.heads && wave == 0 && g == 0) *reinterpret_cast<f32x2*>(ml) = (f32x2){m[nb], z};
    } else {
      const Closing c = close_sum(m[nb], z, a.sinks && h0 + h < a.heads ? a.sinks[h0 + h] * kLog2e : -INFINITY);
      if (a.lse && h0 + h < a.heads && wave == 0 && g == 0) a.lse[(int64_t)b * a.heads + h0 + h] = c.lse;
      by = c.by, half = c.half;
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
      *reinterpret_cast<f32x4*>(rows + h * 4 * kLatent + 16 * swizzle((S::kDims * wave + 16 * mb) / 4 + g, h)) =
          acc[mb][nb] * by * half * half;
  }
  barrier();
  if (a.splits > 1 && mine == 0) return;  // a split with nothing in it leaves m and l only
  for (int h = wave; h < S::HT && h0 + h < a.heads; h += S::kWaves) {
    const f32x4 lo = *reinterpret_cast<const f32x4*>(rows + h * 4 * kLatent + 16 * swizzle(2 * lane, h));
    const f32x4 hi = *reinterpret_cast<const f32x4*>(rows + h * 4 * kLatent + 16 * swizzle(2 * lane + 1, h));
    if (a.splits > 1) {
      f32x4* to = reinterpret_cast<f32x4*>(a.part + (((int64_t)b * a.splits + split) * a.heads + h0 + h) * kLatent + 8 * lane);
      to[0] = lo;
      to[1] = hi;
    } else {
      const float o[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      *reinterpret_cast<u32x4*>(a.out + (((int64_t)b * a.heads + h0 + h) * kLatent + 8 * lane) * 2) = float_to_bf16x8(o);
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
  // lane s holds split s's reference and sum (at most 64 splits)
  f32x2 mz = {-INFINITY, 0.0f};
  if (lane < a.splits) mz = *reinterpret_cast<const f32x2*>(ml + 2 * ((b * a.splits + lane) * a.heads + h));
  float top = mz.x;
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor(top, k));
  const float ref = top == -INFINITY ? 0.0f : top;
  // nothing live: nothing written, maybe
  const bool live = !(mz.x == -INFINITY && mz.y == 0.0f);
  const float f = live ? __builtin_amdgcn_exp2f(mz.x - ref) : 0.0f;
  const uint64_t written = __ballot(live);
  float total = mz.y * f;
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) total += __shfl_xor(total, k);
  float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const float* rows = a.part + (b * a.splits * a.heads + h) * kLatent + 8 * lane;
#pragma unroll 4
  for (int32_t s = 0; s < a.splits; ++s) {
    const float fs = __shfl(f, s);
    f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
    if (written >> s & 1) {
      const f32x4* src = reinterpret_cast<const f32x4*>(rows + (int64_t)s * a.heads * kLatent);
      lo = src[0];
      hi = src[1];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[e] = fmaf(lo[e], fs, o[e]);
      o[4 + e] = fmaf(hi[e], fs, o[4 + e]);
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
constexpr int kMaxSplits = 64;  // (a lane each where they are joined)
constexpr int kHeadTile = 64;
constexpr int kTile = 64;  // positions that a split has at least two of
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
  if (s > kMaxSplits) s = kMaxSplits;
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
  if (!dims_ok(rows, num_heads, table_width, k) || num_pages > kMaxPages || page_table_row_stride < 0 || num_tables < 0 ||
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
  a.pages_lim = (uint32_t)num_pages;
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
  latent_attention_kernel<KEY><<<dim3((uint32_t)(8 * groups)), dim3(512), 0, stream>>>(a);
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
