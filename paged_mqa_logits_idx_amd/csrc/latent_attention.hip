// latent_attention.hip -- attention over a paged cache of latents (gfx950
// kernels and C-ABI entry points declared in include/latent_cache.h).
//
// Row b attends with H heads of 512 values to the latents c_p of its positions
// p in S_b (a top-k's list, or every position below the row's length); one
// latent is key and value of all heads:
//   x_hp = scale * <q_bh, c_p>
//   z_h  = sum_p exp(x_hp) (+ exp(sink_h)),  out_bh = sum_p exp(x_hp) c_p / z_h
//
// Work decomposition.  A unit is (row, split of its positions, block of 64
// heads), one workgroup of eight waves, two on each SIMD, over tiles of 64
// positions.  Each tile is gathered once from its pages into LDS by DMA (512
// bytes of e4m3 codes or 1024 of bf16 a position) while tiles before it are used,
// and read twice by the matrix units (32 x 32 x 16, bf16):
//   scores   X = C Q^T:  four blocks of 32 positions x 32 heads.  Two waves a
//            block take 256 of the 512 values each and trade halves of their sums
//            through LDS, so that each goes on with 16 of the positions.  The
//            queries stay in registers (64 a lane), the latents are read from LDS.
//            A lane then holds 8 positions of one head.
//   outputs  O^T += C^T P^T:  a wave takes 64 of the values, of all 64 heads (64
//            registers a lane); C^T comes out of the same LDS tile through the
//            transposing LDS reads, P^T through a small LDS buffer.
// So a latent is moved from memory once a unit, and its codes are widened to bf16
// (exactly) on the way into the matrix units; the position's scale is applied to
// its scores and to its probabilities, in float32.  The e4m3 products of the
// matrix units themselves would need no widening, but drop what lies 2^-12.5
// below the largest product: 1.7e-5 of the result (bf16 operands: 2e-7), of
// scores whose errors the exponential passes on in full.
//
// A row is split where its units are fewer than the CUs; the splits leave sums
// and outputs in float32, which a second kernel joins.  All rows are split alike,
// by the table's width: a batch of several lengths takes as long as its longest row
// (16 rows of 2432 to 8192 positions: 16 tiles for the longest row's units, 10.4 on
// average), and units that no whole number of splits spreads over the CUs leave
// some idle (64 heads over 2048 positions: 128 rows 64 us, 129 rows 71, 256 rows
// 98, 257 rows 151).
//
// What bounds it.  Many rows: 4096 of 64 heads over 2048 of 5632 positions take
// 0.90 to 0.95 ms (the cards differ), 0.95 to 1.0 PFLOP/s (a library product of
// 8192^3 1.18).  Of the SIMDs' cycles the matrix units have 45 %, vector
// instructions issue in 46 % (173 a wave and tile, 96 of them the widening's, which
// take 7.5 clocks, not 4), the LDS has 26 % of its own; taking away any one part
// shortens a tile by a seventh at most.  A unit's start and end take 10 us of 59:
// lists of 64 positions 86 us for 2048 rows, of 512 180, of 2048 450 to 480.  Heads
// are multiplied in blocks of 64, whatever their number: 8 heads take 0.80 ms, 72
// heads 1.74.  Few rows: 64 of 64 heads over 2048 of 32768 positions take 39 us, of
// which 8 the joining: 107 MB are read and 34 written (the splits' outputs) in 31
// us, then 35 read; one row takes 14.5, three loads in a row (list, page id,
// latent), two tiles and two launches.
//
// Running maximum: all waves agree on a reference m_h for each head.  It
// moves, and the sums are rescaled, only when the probabilities that a lane has of
// a tile add up to more than 256: they reach that instead of 1, which costs no
// precision, and most tiles rescale nothing.
//
// Rounding: scores, exponentials, sums and outputs are float32; the products
// take bf16 operands, which rounds the probability (times the e4m3 scale) once,
// by 2^-8 of itself at most, independently from position to position.  The
// denominator sums the unrounded probabilities.
#include <type_traits>

#include "idx_device.h"

namespace {

constexpr float kLimit = 256.0f;    // what a lane's 8 probabilities may add up to; one is above 2^kLazy then
constexpr float kLazy = 5.0f;       // base-2 logits that a maximum exceeds its reference by where it moves
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxHeads = 128;
constexpr int kHeadTile = 64;       // heads of a unit
constexpr int kTile = 64;           // positions of a tile
constexpr int kPartials = kHeadTile * kLatent;  // float32 outputs of a unit

typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef int v2i __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));

// A position that is masked, or (16 bytes on) whose page id lies outside the pool,
// is gathered from here: it must not bring values of its own into the products.
__device__ const u32x4 kZeroLatent[2 * kLatent / 16 + 1] = {};

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
  float* part;         // splits > 1: [rows][splits][head_blocks] units of outputs, then their heads' m and l
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

// Where chunk c (16 bytes) of position r stands within the position's LDS row:
// rows of a multiple of 256 bytes would put one chunk of all positions into the
// same banks.  Any 16 positions in a row take 16 places.  The transposing reads
// take, of 32 lanes, two chunks of 8 positions whose bit 2 is one (e4m3), or four
// chunks of 4 positions (bf16): also 16 places.
template <int KEY>
__device__ __forceinline__ constexpr int swizzle(int c, int r) {
  return c ^ (KEY == kFp8 ? (r & 3) << 1 | (r & 8) | (r >> 2 & 1) : (r & 3) << 2 | (r >> 2 & 3));
}

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

// A unit's tile: 64 positions x 64 heads, four 32 x 32 blocks of scores.  Eight
// waves, two on each SIMD: the two waves of a block take 256 of the 512 values
// each and add their halves up through LDS (so a wave keeps 64 registers of
// queries and 64 of outputs, and has as many again to read LDS ahead of the
// matrix units).
template <int KEY>
struct Shape {
  static constexpr int HT = kHeadTile;
  static constexpr int kWaves = 8, kThreads = 64 * kWaves;
  static constexpr int kRowBytes = KEY == kFp8 ? kLatent : 2 * kLatent;  // of a position
  static constexpr int kChunks = kRowBytes / 16;    // of a position
  static constexpr int kBuffers = KEY == kFp8 ? 4 : 2;
  static constexpr int kDims = kLatent / kWaves;    // values of a wave's outputs
  static constexpr int MB = kDims / 32, NB = HT / 32;
  static constexpr int kGather = kTile / kWaves;    // positions that a wave gathers
  static constexpr int kPerDma = 64 / kChunks;      // positions of one DMA
  static constexpr int kDmas = kGather / kPerDma;
  static constexpr int kRing = 8;                   // tiles whose positions are resolved, four at a time
};

template <int KEY>
struct AttendShared {
  using S = Shape<KEY>;
  uint8_t tile[S::kBuffers][kTile * S::kRowBytes];
  uint64_t at[S::kRing][kTile];      // where the positions' latents are
  float scale[S::kRing][kTile];      // their e4m3 scales
  bf16x8 p[4][2][S::HT];                // probabilities, by 16 positions, half of a wave and head
  union {
    f32x4 part[4][2][2][64];            // halves of scores on their way: by block, wave and lane
    float mx[S::HT][4];                 // maxima of the tile's blocks of 16 positions
  };
  __attribute__((aligned(4))) uint16_t special[S::kRing][2];  // whether half a tile has a position that is masked or bad
  uint32_t over[4];                     // whether a tile's scores exceed the references, by tile % 4
  float by[S::HT];                      // factors of a moved reference; at the end the references
  float sum[4][S::HT];
};

template <int KEY>
__global__ __launch_bounds__(Shape<KEY>::kThreads, 2) void latent_attention_kernel(Attend a) {
  using S = Shape<KEY>;
  constexpr int kRowBytes = S::kRowBytes, NB = S::NB, MB = S::MB;
  __shared__ __attribute__((aligned(16))) AttendShared<KEY> sh;

  const int lane = threadIdx.x & 63, n = lane & 31, half = lane >> 5;
  const int wave = uniform(threadIdx.x >> 6);
  const int pb = wave & 1, hg = wave >> 1 & 1;  // the wave's block of scores: positions 32*pb, heads 32*hg
  const int kh = wave >> 2;                     // and its half of the values, 256*kh

  // Units of one row and split (its head blocks read the same latents) follow
  // each other on one XCD; the last rows, the longest of a causal batch, start
  // first.
  static_assert(kMaxHeads <= 2 * kHeadTile);  // one block of heads a row or two
  const int hshift = a.head_blocks - 1, hb = (int)(blockIdx.x >> 3) & hshift;
  const uint32_t rs = blockIdx.x >> (3 + hshift) << 3 | (blockIdx.x & 7), splits = (uint32_t)a.splits;
  if (rs >= (uint32_t)a.rows * splits) return;
  const uint32_t row = splits > 1 ? rs / splits : rs;
  const int32_t b = a.rows - 1 - (int32_t)row, split = (int32_t)(rs - row * splits);
  const int32_t h0 = hb * S::HT;

  // What depends on nothing but the arguments goes out first: waves 0 .. 3 load
  // the list's entries of the first kRing tiles, before the length that may cut
  // it short is there, and waves 4 .. 7 the queries (a wave's loads complete in
  // order: queries ahead of a page id would hold it up).
  //
  // Queries: by DMA into the last 64 KiB of the tile buffers, rows of 1 KiB as
  // they stand in memory; from there to registers as the B operand (loading the
  // fragments from memory took 16 bytes of 64 lines an instruction: 7 us a unit
  // instead of 2).  Heads past the last are zero.
  const uint32_t lds_tile = (uint32_t)(uintptr_t)(lds_u8*)&sh.tile[0][0];
  const uint32_t lds_scale = (uint32_t)(uintptr_t)(lds_u8*)&sh.scale[0][0];
  const uint8_t* zero = reinterpret_cast<const uint8_t*>(kZeroLatent);
  constexpr uint32_t kQueryAt = sizeof(sh.tile) - S::HT * 2 * kLatent;
  constexpr int kResolvers = S::kWaves / 2, kMany = S::kRing * kTile / (64 * kResolvers);
  const int32_t whole = a.width * kPage, bound = a.k >= 0 ? min(a.k, whole) : whole;
  const int32_t* idx = a.k >= 0 ? a.idx + (int64_t)b * a.k : nullptr;
  auto entry = [&](int32_t j, int32_t i) -> int32_t {  // entry i of the unit's tile j, or -1
    const int32_t t = (split + j * a.splits) * kTile + i;
    return t >= bound ? -1 : idx ? idx[t] : t;
  };
  int32_t early[kMany];  // lane's entry of tiles kMany * wave ..
  if (wave < kResolvers) {
#pragma unroll
    for (int e = 0; e < kMany; ++e) early[e] = entry(kMany * wave + e, lane);
  } else {
    auto ask = [&](auto dma) {
#pragma unroll
      for (int e = 0; e < S::HT / (S::kWaves - kResolvers); ++e) {
        const int h = (S::kWaves - kResolvers) * e + wave - kResolvers;
        const uint8_t* src = h0 + h < a.heads ? a.q + ((int64_t)b * a.heads + h0 + h) * (2 * kLatent) : zero;
        dma(src + 16 * swizzle<KEY>(lane, h), lds_tile + kQueryAt + (uint32_t)(h * 2 * kLatent));
      }
    };
    // An unsplit row's queries are read once: 1 to 3 % of a prefill; read like that
    // by several splits, 33 rows take 22.5 us, not 21.4.
    if (splits > 1) ask([](const uint8_t* src, uint32_t dst) { dma16(src, dst); });
    else ask([](const uint8_t* src, uint32_t dst) { dma16_once(src, dst); });
  }
  const int32_t L = uniform(min(max(a.sl[b], 0), whole));
  const int32_t count = min(bound, L);
  const int32_t tiles = (count + kTile - 1) / kTile;
  const uint32_t left = tiles > split ? (uint32_t)(tiles - split) : 0u;
  const int32_t mine = (int32_t)(splits > 1 ? (left + splits - 1) / splits : left);
  const int32_t table = a.rt ? a.rt[b] : 0;
  const bool table_ok = !a.rt || (table >= 0 && table < a.num_tables);
  const int32_t* tab = a.pt + (int64_t)(a.rt ? (table_ok ? table : 0) : b) * a.pt_stride;

  f32x16 acc[MB][NB];  // values kDims*wave + 32*mb + 8*(i/4) + 4*half + i%4 of heads 32*nb + n
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = (f32x16)(0.0f);
  // Of head 32*hg + n: reference (0 before the first), what a lane's 8
  // probabilities may add up to by it (nothing, before the first), sum of
  // probabilities.
  float m = 0.0f, limit = -1.0f, sum = 0.0f;

  if (mine > 0) {
    // Where positions are: page ids of the entries, then the ring's places of tile
    // j's, and its scales on their way; lane l has place l (or half + l of a tile).
    auto page_of = [&](int32_t p) -> int32_t { return (uint32_t)p < (uint32_t)whole && table_ok ? tab[p / kPage] : -1; };
    auto keep = [&](int32_t j, int32_t half_, int32_t p, int32_t page) {
      const int at = half_ + lane;
      const uint8_t *src = zero, *scale = zero;
      bool ok = false;
      if ((split + j * a.splits) * kTile + at < count && (uint32_t)p < (uint32_t)L) {
        ok = (uint32_t)page < a.pages_lim;
        src = ok ? a.kv + (uint64_t)page * (uint64_t)a.kv_stride + (p % kPage) * kRowBytes : zero + 16;
        if (ok) scale = a.ks + (uint64_t)page * (uint64_t)a.ks_stride + 4 * (p % kPage);
      }
      sh.at[j % S::kRing][at] = (uintptr_t)src;
      if (KEY == kFp8) dma4(scale, lds_scale + (uint32_t)((j % S::kRing * kTile + half_) * 4));
      const uint64_t odd = __ballot(!ok);
      if (lane % 32 == 0) sh.special[j % S::kRing][at / 32] = (uint32_t)(odd >> lane) != 0;
    };
    // Tile j into its buffer, in kDmas operations of every wave; past the last,
    // whatever the ring has.
    const uint32_t place = 16 * swizzle<KEY>(lane % S::kChunks, S::kGather * wave + lane / S::kChunks);
    auto source_of = [&](int32_t j, int d) -> uint64_t {
      return sh.at[j % S::kRing][S::kGather * wave + d * S::kPerDma + lane / S::kChunks];
    };
    auto gather_part = [&](int32_t j, uint64_t from, int d) {
      dma16(reinterpret_cast<const uint8_t*>(from + (place ^ (16 * swizzle<KEY>(0, S::kPerDma * d)))),
            lds_tile + (uint32_t)((j % S::kBuffers * kTile + S::kGather * wave + d * S::kPerDma) * kRowBytes));
    };
    auto gather = [&](int32_t j) {
#pragma unroll
      for (int d = 0; d < S::kDmas; ++d) gather_part(j, source_of(j, d), d);
    };

    if (threadIdx.x < 4) sh.over[threadIdx.x] = 0;
    if (wave < kResolvers) {
      int32_t page[kMany];
#pragma unroll
      for (int e = 0; e < kMany; ++e) page[e] = page_of(early[e]);
#pragma unroll
      for (int e = 0; e < kMany; ++e) keep(kMany * wave + e, 0, early[e], page[e]);
    }
    barrier();
    constexpr int kEarly = S::kBuffers - S::HT * 2 * kLatent / (kTile * kRowBytes);  // tiles beside the queries
#pragma unroll
    for (int32_t j = 0; j < kEarly; ++j) gather(j);
    wait_vm<kEarly * S::kDmas>();
    barrier();
    // Lane (n, half) holds head n's values of step s: 16*(2*(s/2) + half) +
    // 8*(s%2) .. +8 (e4m3: two steps share a 16-byte chunk of codes) or
    // 8*(2*s + half) .. +8 (bf16).
    bf16x8 q[16];
#pragma unroll
    for (int s = 0; s < 16; ++s) {
      const int h = 32 * hg + n, c = 32 * kh + (KEY == kFp8 ? 2 * (2 * (s >> 1) + half) + (s & 1) : 2 * s + half);
      q[s] = *reinterpret_cast<const bf16x8*>(&sh.tile[0][0] + kQueryAt + h * 2 * kLatent + 16 * swizzle<KEY>(c, h));
    }
    barrier();

    // The rows of scores of a wave's products: the position that its lane reads
    // as A operand is row n, but for kh 1 row n ^ 16, so that products 0..7 are
    // those of the 16 positions 32*pb + 16*kh that the wave goes on with
    // (8*(i/4) + 4*half + i%4 of them) and products 8..15 its partner's.
    const int kr = 32 * pb + (n ^ 16 * kh);
    auto read_k = [&](const uint8_t* rows, int t) {  // fp8: values 16 of step pair t; bf16: 8 of step t
      return *reinterpret_cast<const u32x4*>(rows + kr * kRowBytes + 16 * swizzle<KEY>((KEY == kFp8 ? 16 : 32) * kh + 2 * t + half, kr));
    };
    auto send = [&](const f32x16& x) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        sh.part[wave & 3][kh ^ 1][k][lane] = (f32x4){x[8 + 4 * k], x[9 + 4 * k], x[10 + 4 * k], x[11 + 4 * k]};
    };
    float x[8];  // products of the wave's 16 positions and head 32*hg + n
    auto receive = [&](const f32x16& mine_) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const f32x4 v = sh.part[wave & 3][kh][k][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * k + e] = mine_[4 * k + e] + v[e];
      }
    };
    // Scores of tile j, while tile j + 1 is gathered.
    auto score = [&](int32_t j) -> f32x16 {
      static_assert(KEY == kFp8 || S::kDmas == 8);
      uint64_t from = source_of(j + 1, 0);
      const uint8_t* rows = sh.tile[j % S::kBuffers];
      f32x16 half0 = (f32x16)(0.0f);
#pragma unroll
      for (int s = 0; s < 16; s += 2) {
        bf16x8 c0, c1;
        if constexpr (KEY == kFp8) {
          const u32x4 c = read_k(rows, s / 2);
          c0 = fp8x8_to_bf16x8(c.x, c.y), c1 = fp8x8_to_bf16x8(c.z, c.w);
        } else {
          c0 = __builtin_bit_cast(bf16x8, read_k(rows, s)), c1 = __builtin_bit_cast(bf16x8, read_k(rows, s + 1));
        }
        half0 = __builtin_amdgcn_mfma_f32_32x32x16_bf16(c0, q[s], half0, 0, 0, 0);
        half0 = __builtin_amdgcn_mfma_f32_32x32x16_bf16(c1, q[s + 1], half0, 0, 0, 0);
        gather_part(j + 1, from, s / 2);
        if (s < 14) from = source_of(j + 1, s / 2 + 1);
      }
      send(half0);
      return half0;
    };
    const int own = 32 * pb + 16 * kh + 4 * half;  // the lane's positions: own + 8*k .. +4
    auto read_ks = [&](int32_t j, int k) -> f32x4 {
      if constexpr (KEY == kFp8) return *reinterpret_cast<const f32x4*>(&sh.scale[j % S::kRing][own + 8 * k]);
      return (f32x4){1.f, 1.f, 1.f, 1.f};
    };
    auto special_of = [&](int32_t j) { return *reinterpret_cast<const uint32_t*>(sh.special[j % S::kRing]); };
    float part;  // the sum of the lane's probabilities
    // Base-2 logits of tile j less a reference, masks applied.
    auto logits = [&](int32_t j, float ref, float (&t)[8]) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const f32x4 ks = read_ks(j, k);
#pragma unroll
        for (int e = 0; e < 4; ++e) t[4 * k + e] = fmaf(x[4 * k + e], a.scale2 * ks[e], -ref);
      }
      if (uniform(special_of(j)) != 0) {
        const uint64_t masked = (uintptr_t)zero, bad = masked + 16;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint64_t at = sh.at[j % S::kRing][own + 8 * (e / 4) + e % 4];
          t[e] = at == bad ? __builtin_nanf("") : t[e];
          t[e] = at == masked ? -INFINITY : t[e];
        }
      }
    };
    auto max_of = [&](const float (&t)[8]) {
      return fmaxf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])), fmaxf(fmaxf(t[4], t[5]), fmaxf(t[6], t[7])));
    };
    // Probabilities: their sum unrounded; times the latents' scales, as bf16, to
    // LDS, where a lane's 8 positions are 8 k-values of the B operand of one step
    // of 16 positions.
    auto weigh = [&](int32_t j, const float (&t)[8]) {
      bf16x8 w;
      part = 0.0f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const f32x4 ks = read_ks(j, k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = __builtin_amdgcn_exp2f(t[4 * k + e]);
          part += p;
          w[4 * k + e] = (__bf16)(p * ks[e]);
        }
      }
      sh.p[2 * pb + kh][half][32 * hg + n] = w;
    };
    // Tile j's probabilities by the reference as it is, and whether it will do: it
    // will not where a lane's add up to more than kLimit, or the head has none.
    auto probabilities = [&](int32_t j) {
      float t[8];
      logits(j, m, t);
      weigh(j, t);
      if (__ballot(part > limit) != 0) sh.over[j & 3] = 1;
    };
    // The heads' references anew from tile j's maxima, the sums so far to match,
    // and the tile's probabilities again.
    auto refer = [&](int32_t j) {
      float t[8];
      logits(j, 0.0f, t);
      float top = max_of(t);
      top = fmaxf(top, __shfl_xor(top, 32));
      const int h = 32 * hg + n;
      if (half == 0) sh.mx[h][2 * pb + kh] = top;
      barrier();
      const f32x4 all = *reinterpret_cast<const f32x4*>(sh.mx[h]);
      top = fmaxf(fmaxf(all.x, all.y), fmaxf(all.z, all.w));
      const bool live = limit > 0.0f, moves = live ? top - m > kLazy : top > -INFINITY;
      const float f = moves ? (live ? __builtin_amdgcn_exp2f(m - top) : 0.0f) : 1.0f;
      if (moves) m = top, limit = kLimit;
      sum *= f;
      if (pb == 0 && kh == 0 && half == 0) sh.by[h] = f;
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] -= m;
      weigh(j, t);
      barrier();
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const float by = sh.by[32 * nb + n];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) acc[mb][nb] *= by;
      }
    };
    auto settle = [&](int32_t j) {
      if (j == 0 || uniform(sh.over[j & 3]) != 0) refer(j);
      sum += part;
    };

    // A operand of the outputs: 32 values 32*mb of the wave's, over step s of 16
    // positions (slots as the probabilities': 8*(k/4) + 4*half + k%4).
    const int lane16 = lane & 15, g = lane >> 4;
    struct Codes {
      v2i lo, hi;  // fp8: lo only
    };
    auto read_v = [&](const uint8_t* rows, int s, int mb) -> Codes {
      Codes t;
      if constexpr (KEY == kFp8) {
        // 16 lanes read 8 positions x 16 values: lanes 2k, 2k+1 the 16 codes of
        // position k, lane i gets value i of the 8 positions
        const int k = lane16 >> 1, r = 16 * s + 8 * (k >> 2) + 4 * half + (k & 3), c = 2 * (MB * wave + mb) + (g & 1);
        t.lo = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) v2i*)(rows + r * kRowBytes + 16 * swizzle<KEY>(c, r) + 8 * (lane & 1)));
      } else {
        // 16 lanes read 4 positions x 16 values: lanes 4k .. 4k+3 the 32 bytes of
        // position k
        v4s u[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 16 * s + 8 * e + 4 * half + (lane16 >> 2);
          const int c = 4 * (MB * wave + mb) + 2 * (g & 1) + (lane16 >> 1 & 1);
          u[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) v4s*)(rows + r * kRowBytes + 16 * swizzle<KEY>(c, r) + 8 * (lane & 1)));
        }
        t.lo = __builtin_bit_cast(v2i, u[0]), t.hi = __builtin_bit_cast(v2i, u[1]);
      }
      return t;
    };
    auto widen = [&](const Codes& t) -> bf16x8 {
      if constexpr (KEY == kFp8) return fp8x8_to_bf16x8((uint32_t)t.lo.x, (uint32_t)t.lo.y);
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(t.lo, t.hi, 0, 1, 2, 3));
    };
    auto read_w = [&](int s, int nb) { return sh.p[s][half][32 * nb + n]; };
    auto accumulate = [&](int32_t j, const Codes (&early)[MB]) {
      const uint8_t* rows = sh.tile[j % S::kBuffers];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8 w[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) w[nb] = read_w(s, nb);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          const bf16x8 v = widen(s == 0 ? early[mb] : read_v(rows, s, mb));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            acc[mb][nb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, w[nb], acc[mb][nb], 0, 0, 0);
        }
      }
    };

    // One instruction stream a tile.  Phase j scores tile j + 1, adds up tile j's
    // latents and gathers tile j + 3, as if no position of tile j + 1 were masked
    // (a tile that has some takes its probabilities again).  The 16 products of
    // the scores and the 8 pairs of products of the outputs (pair i: step i / 2 of
    // 16 positions, values i % 2) are laid out so that the matrix units have work
    // whose operands are in registers wherever a wave would wait:
    //   pairs 0, 1       while the first codes of tile j + 1 are read,
    //   pairs 2, 3       among the scores, with the LDS reads three steps ahead,
    //                    the conversion of the next codes and the gather,
    //   pairs 4 .. 7     in the time of the probabilities, before them in one of
    //                    a SIMD's two waves and behind them in the other.
    // The gather's four operations stand apart: the memory path takes one in
    // about 50 cycles, and a wave whose operation has to wait issues nothing else
    // (all in one place they held up every phase by 1500 cycles).
    auto add = [&](const bf16x8& v, const bf16x8 (&w)[NB], int mb) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, w[nb], acc[mb][nb], 0, 0, 0);
    };
    // FIRST: tile 0 is scored, nothing added up; LAST: the other way round.
    auto phase = [&](int32_t j, auto first, auto last) {
      constexpr bool kScore = !decltype(last)::value, kAdd = !decltype(first)::value;
      constexpr int kAhead = 3;
      const uint8_t* kt = sh.tile[(j + 1) % S::kBuffers];
      const uint8_t* vt = sh.tile[j % S::kBuffers];
      uint32_t over = 0, special = 0;
      u32x4 kk[kAhead];
      bf16x8 w[4][NB], c0, c1, v;
      Codes vv[4];
      uint64_t from = 0;
      if constexpr (kAdd) {
        over = sh.over[j & 3];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) w[0][nb] = read_w(0, nb);
        vv[0] = read_v(vt, 0, 0);
        vv[1] = read_v(vt, 0, 1);
      }
      if constexpr (kScore) {
#pragma unroll
        for (int t = 0; t < kAhead; ++t) kk[t] = read_k(kt, t);
        special = special_of(j + 1);
      }
      if constexpr (kAdd) {
        if (j == 0 || uniform(over) != 0) {
          refer(j);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) w[0][nb] = read_w(0, nb);
        }
        sum += part;
        if (threadIdx.x == 0) sh.over[(j + 3) & 3] = 0;  // (read a phase ago, used again two phases on)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) w[1][nb] = read_w(1, nb);
        add(widen(vv[0]), w[0], 0);
        vv[0] = read_v(vt, 1, 0);
        add(widen(vv[1]), w[0], 1);
        vv[1] = read_v(vt, 1, 1);
        if constexpr (kScore) from = source_of(j + 3, 0);
      }
      f32x16 sc = (f32x16)(0.0f);
      if constexpr (kScore) c0 = fp8x8_to_bf16x8(kk[0].x, kk[0].y), c1 = fp8x8_to_bf16x8(kk[0].z, kk[0].w);
      if constexpr (kAdd) v = widen(vv[0]);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        __builtin_amdgcn_sched_barrier(0);
        const int mb = t / 4, nb = t / 2 % 2;  // pairs 2, 3: a product in every other step
        if constexpr (kScore) sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(c0, q[2 * t], sc, 0, 0, 0);
        if (kAdd && t % 2 == 0) acc[mb][nb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, w[1][nb], acc[mb][nb], 0, 0, 0);
        if constexpr (kScore) sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(c1, q[2 * t + 1], sc, 0, 0, 0);
        if (kScore && t + 1 < 8) {
          const u32x4 c = kk[(t + 1) % kAhead];
          c0 = fp8x8_to_bf16x8(c.x, c.y), c1 = fp8x8_to_bf16x8(c.z, c.w);
        }
        if (kScore && t + kAhead < 8) kk[t % kAhead] = read_k(kt, t + kAhead);
        if constexpr (kAdd) {
          if (t == 3) v = widen(vv[1]);
          if (t >= 4) vv[t - 4] = read_v(vt, 2 + (t - 4) / MB, (t - 4) % MB);
          if (t >= 6) w[t - 4][0] = read_w(t - 4, 0), w[t - 4][1] = read_w(t - 4, 1);
        }
        if constexpr (kScore && kAdd) {
          if (t == 1 || t == 4 || t == 7) gather_part(j + 3, from, t / 3), from = source_of(j + 3, t / 3 + 1);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (kScore) {
        send(sc);
        barrier();  // the halves are there; tile j's probabilities have been read
        receive(sc);
      }
      auto outputs = [&]() {
        if constexpr (kAdd) {
#pragma unroll
          for (int i = 0; i < 4; ++i) add(widen(vv[i]), w[2 + i / MB], i % MB);
        }
      };
      auto chances = [&]() {
        const f32x4 ks[2] = {read_ks(j + 1, 0), read_ks(j + 1, 1)};
        part = 0.0f;
        bf16x8 out;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float by = ks[e / 4][e % 4], t = fmaf(x[e], a.scale2 * by, -m);
          const float p = __builtin_amdgcn_exp2f(t);
          part += p;
          out[e] = (__bf16)(p * by);
        }
        sh.p[2 * pb + kh][half][32 * hg + n] = out;
        if (__ballot(part > limit) != 0) sh.over[(j + 1) & 3] = 1;
      };
      if constexpr (kScore && kAdd) {
        gather_part(j + 3, from, 3);
        if (kh == 0) outputs();
        __builtin_amdgcn_sched_barrier(0);
        chances();
        __builtin_amdgcn_sched_barrier(0);
        if (kh != 0) outputs();
      } else if constexpr (kScore) {
        chances();
      } else {
        outputs();
      }
      if (kScore && uniform(special) != 0) probabilities(j + 1);
    };
    // The ring's places of tiles j + 4 .. j + 7, half a tile a wave: of those before
    // tile j.
    auto resolve = [&](int32_t j) {
      const int32_t tile = j + 4 + wave / 2, half_ = kTile / 2 * (wave & 1);
      if (j == 0 || j % 4 != 0 || j + 4 >= mine || lane >= 32) return;
      const int32_t p = entry(tile, half_ + lane);
      keep(tile, half_, p, page_of(p));
    };

    if constexpr (KEY == kFp8) {
      // Of a SIMD's two waves one goes first throughout: they drift apart, and one
      // has matrix instructions where the other has not (1 % of a prefill).
      if (kh != 0) __builtin_amdgcn_s_setprio(1);
      // Tiles j + 2 and j + 3 are on their way during phase j.  A tile has arrived
      // when at most the operations of the tiles issued after it are outstanding
      // (they complete in order).
      gather(2);
      wait_vm<2 * S::kDmas>();
      barrier();
      phase(-1, std::true_type{}, std::false_type{});
      int32_t j = 0;
      for (; j + 1 < mine; ++j) {
        wait_vm<S::kDmas>();
        barrier();  // tile j + 1 and tile j's probabilities are there; every wave is done with tile j - 1
        phase(j, std::false_type{}, std::false_type{});
        resolve(j);
      }
      wait_vm<0>();
      barrier();
      phase(j, std::false_type{}, std::true_type{});
    } else {
      // Two buffers: a tile is scored and added up while the next is on its way.
      // Its gather is spread over the scores, and the first latents of the outputs
      // are read before the probabilities are there (2048 rows of 64 heads over 2048
      // positions, 480 to 510 us now, took 606 us without, 592 with the second, 568
      // with both when these came).
      for (int32_t j = 0; j < mine; ++j) {
        wait_vm<0>();
        barrier();  // tile j is there; every wave is done with tile j - 1
        if (threadIdx.x == 0) sh.over[(j + 3) & 3] = 0;
        resolve(j);
        const f32x16 half0 = score(j);
        barrier();
        receive(half0);
        probabilities(j);
        Codes early[MB];
#pragma unroll
        for (int i = 0; i < MB; ++i) early[i] = read_v(sh.tile[j % S::kBuffers], 0, i);
        barrier();
        settle(j);
        accumulate(j, early);
      }
      wait_vm<0>();
    }
    barrier();
  }

  // Sums over the position blocks.
  {
    const float s = sum + __shfl_xor(sum, 32);
    if (half == 0) sh.sum[2 * pb + kh][32 * hg + n] = s;
    if (half == 0 && pb == 0 && kh == 0) sh.by[32 * hg + n] = limit > 0.0f ? m : -INFINITY;
  }
  wait_vm<0>();  // (nothing in it: the queries are still on their way)
  barrier();
  auto total = [&](int h) { return (sh.sum[0][h] + sh.sum[1][h]) + (sh.sum[2][h] + sh.sum[3][h]); };
  if (a.splits > 1) {
    // The outputs as they stand in the registers; a split with nothing in it
    // leaves references and sums only.
    const int64_t unit = ((int64_t)b * a.splits + split) * a.head_blocks + hb;
    if (threadIdx.x < S::HT)
      *reinterpret_cast<f32x2*>(a.part + (int64_t)a.rows * a.splits * a.head_blocks * kPartials + 2 * (S::HT * unit + threadIdx.x)) =
          (f32x2){sh.by[threadIdx.x], total(threadIdx.x)};
    if (mine == 0) return;
    f32x4* to = reinterpret_cast<f32x4*>(a.part + unit * kPartials) + lane;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if (h0 + 32 * nb + n >= a.heads) continue;
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const f32x16& o = acc[mb][nb];
          to[64 * (4 * (NB * (MB * wave + mb) + nb) + k)] = (f32x4){o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]};
        }
    }
    return;
  }
  // The outputs of all waves as rows in the tile buffers, so that they leave in
  // whole lines; past the caches, where the latents stay (2048 rows of 64 heads over
  // 512 and 2048 positions 180 and 482 us, with ordinary stores 185 and 485; 4096
  // rows 948 and 964).
  uint8_t* rows = &sh.tile[0][0];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int h = 32 * nb + n;
    const Closing c = close_sum(sh.by[h], total(h), a.sinks && h0 + h < a.heads ? a.sinks[h0 + h] * kLog2e : -INFINITY);
    if (a.lse && h0 + h < a.heads && wave == 0 && half == 0) a.lse[(int64_t)b * a.heads + h0 + h] = c.lse;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const f32x16 o = acc[mb][nb] * c.by * c.half * c.half;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<bf16x4*>(rows + h * 2 * kLatent + 16 * swizzle<KEY>(S::kDims / 8 * wave + 4 * mb + k, h) + 8 * half) =
            (bf16x4){(__bf16)o[4 * k], (__bf16)o[4 * k + 1], (__bf16)o[4 * k + 2], (__bf16)o[4 * k + 3]};
    }
  }
  barrier();
#pragma unroll
  for (int e = 0; e < S::HT / S::kWaves; ++e) {
    const int h = S::kWaves * e + wave;
    if (h0 + h < a.heads)
      __builtin_nontemporal_store(*reinterpret_cast<const u32x4*>(rows + h * 2 * kLatent + 16 * swizzle<KEY>(lane, h)),
                                  reinterpret_cast<u32x4*>(a.out + ((int64_t)b * a.heads + h0 + h) * (2 * kLatent) + 16 * lane));
  }
}

// Joins the splits of a row: a wave, a workgroup of its own (of four waves, one
// row took 0.7 us more), has 32 values of 8 heads, 4 a lane, which are 16 bytes
// of a unit's outputs (8 heads of them a line).  16 splits' loads are under way at
// once, outputs and sums together: which splits have written any is known only
// with the sums.  The order of the splits is fixed, so the
// result does not depend on their timing.
template <int kBatch>
__global__ __launch_bounds__(64) void latent_combine_kernel(Attend a) {
  const int lane = threadIdx.x;
  const int block = (int)blockIdx.x, piece = lane >> 3;  // values 32*block + 4*piece .. +4
  const int32_t h = 8 * (int32_t)blockIdx.y + (lane & 7), n = h % kHeadTile;
  const int64_t b = blockIdx.z;
  const int64_t unit0 = b * a.splits * a.head_blocks + h / kHeadTile;
  // the lane's 16 bytes of a unit (accumulator (block, n / 32), chunk piece / 2)
  const f32x4* from = reinterpret_cast<const f32x4*>(a.part + unit0 * kPartials) +
                      64 * (4 * (kHeadTile / 32 * block + n / 32) + piece / 2) + 32 * (piece & 1) + n % 32;
  const f32x2* ml = reinterpret_cast<const f32x2*>(a.part + (int64_t)a.rows * a.splits * a.head_blocks * kPartials) +
                    kHeadTile * unit0 + n;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  float top = -INFINITY, total = 0.0f;
#pragma unroll 1
  for (int32_t s0 = 0; s0 < a.splits; s0 += kBatch) {
    f32x2 mz[kBatch];
    f32x4 v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      mz[i] = (f32x2){-INFINITY, 0.0f};
      if (s0 + i < a.splits) {
        mz[i] = ml[(int64_t)(s0 + i) * a.head_blocks * kHeadTile];
        v[i] = __builtin_nontemporal_load(&from[(int64_t)(s0 + i) * a.head_blocks * (kPartials / 4)]);
      }
    }
    float ref = top;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) ref = fmaxf(ref, mz[i].x);
    const float base = ref == -INFINITY ? 0.0f : ref, by = __builtin_amdgcn_exp2f(top - base);
    top = ref;
    total *= by;
    o *= by;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      // (nothing live in a split: nothing written, maybe)
      if (s0 + i < a.splits && !(mz[i].x == -INFINITY && mz[i].y == 0.0f)) {
        const float f = __builtin_amdgcn_exp2f(mz[i].x - base);
        total = fmaf(mz[i].y, f, total);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = fmaf(v[i][e], f, o[e]);
      }
    }
  }
  if (h >= a.heads) return;
  const int64_t head = b * a.heads + h;
  const Closing c = close_sum(top, total, a.sinks ? a.sinks[h] * kLog2e : -INFINITY);
  bf16x4 w;
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = (__bf16)(o[e] * c.by * c.half * c.half);
  *reinterpret_cast<bf16x4*>(a.out + (head * kLatent + 32 * block + 4 * piece) * 2) = w;
  if (a.lse && block == 0 && piece == 0) a.lse[head] = c.lse;
}

// ---------------------------------------------------------------------------
// Host side.

constexpr int32_t kMaxWidth = 1 << 24;
constexpr int64_t kMaxUnits = 8000000;  // a launch has less than 2^32 threads

// Splits of a row's positions, from the scalar arguments alone (the lengths are
// on the device): a unit takes about 2.2 us a tile, and joining s splits about
// 2.2 * s / 8 more, so up to sqrt(8 * tiles), all of the same number of tiles,
// while every unit has a CU of its own.  One row of 64 heads over 8, 16, 32 and
// 4097 tiles takes 12.1, 13.4, 14.6 and 74 us; with a tile a split, at most 256
// splits, 12.1, 13.1, 15.6 and 75; the first three unsplit 20, 34 and 61.
int splits_of(int32_t rows, int32_t num_heads, int32_t table_width, int32_t k) {
  const int64_t most = k >= 0 ? (k < (int64_t)table_width * kPage ? k : (int64_t)table_width * kPage)
                                : (int64_t)table_width * kPage;
  const int64_t tiles = (most + kTile - 1) / kTile;
  const int64_t units = (int64_t)rows * ((num_heads + kHeadTile - 1) / kHeadTile);
  int64_t s = device_cu_count() / (units > 0 ? units : 1);
  while (s > 1 && s * s > 8 * tiles) --s;
  if (s <= 1) return 1;
  const int64_t each = (tiles + s - 1) / s;
  return (int)((tiles + each - 1) / each);
}

int64_t workspace_of(int32_t rows, int32_t num_heads, int splits) {
  const int64_t blocks = (num_heads + kHeadTile - 1) / kHeadTile;
  return splits > 1 ? rows * splits * blocks * (kPartials + 2 * kHeadTile) * 4 : 0;
}

bool dims_ok(int32_t rows, int32_t num_heads, int32_t table_width, int32_t k) {
  return rows >= 0 && num_heads >= 0 && num_heads <= kMaxHeads && table_width >= 0 && table_width <= kMaxWidth &&
         k >= -1 && (int64_t)rows * ((num_heads + kHeadTile - 1) / kHeadTile) <= kMaxUnits;
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
      !(fabsf(scale * kLog2e) < INFINITY) || workspace_bytes < 0)
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
  a.pages_lim = (uint32_t)(num_pages < (int64_t)1 << 31 ? num_pages : (int64_t)1 << 31);
  a.rows = rows;
  a.heads = num_heads;
  a.width = table_width;
  a.k = k;
  a.num_tables = num_tables;
  a.head_blocks = (num_heads + kHeadTile - 1) / kHeadTile;
  a.scale2 = scale * kLog2e;
  const int64_t groups = ((int64_t)rows * a.splits + 7) / 8 * a.head_blocks;
  (void)hipGetLastError();  // start from a clean error state
  latent_attention_kernel<KEY><<<dim3((uint32_t)(8 * groups)), dim3(Shape<KEY>::kThreads), 0, stream>>>(a);
  if (a.splits > 1) {
    const dim3 grid(kLatent / 32, (uint32_t)((num_heads + 7) / 8), (uint32_t)rows);  // (at most a row a CU)
    // A batch no larger than the splits: the kernel for 16 has registers for fewer
    // waves (64 rows of 64 heads, 4 splits: 40 us with the attention itself, 43 by
    // the kernel for 16), and a kernel for 4 makes more trips (one row of 16 splits
    // 14.5 and 15.2, of 179 splits 74 and 84).
    if (a.splits <= 4)
      latent_combine_kernel<4><<<grid, dim3(64), 0, stream>>>(a);
    else if (a.splits <= 8)
      latent_combine_kernel<8><<<grid, dim3(64), 0, stream>>>(a);
    else
      latent_combine_kernel<16><<<grid, dim3(64), 0, stream>>>(a);
  }
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
