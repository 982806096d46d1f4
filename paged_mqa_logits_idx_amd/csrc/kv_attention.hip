// kv_attention.hip -- attention of one new token per row over the paged keys and
// values by head (gfx950 kernels and C-ABI entry points declared in
// include/kv_cache.h).
//
//   x_ip = scale * <q_i, k_p>,  z_i = sum_p exp(x_ip) (+ exp(sink_i)),
//   out_i = sum_p exp(x_ip) v_p / z_i
//
// for the query heads i of a key head and its positions p.  A unit is (row, key
// head, block of 16 * HW of its query heads): it reads every page of its own once.
//
// Work decomposition.  The pages of all units, one after the other, are cut into
// even shares, one a workgroup, whatever the rows' lengths: a share's pieces are the
// end of a unit, whole units and the start of one.  Whole units are finished by their
// workgroup, the other pieces leave sums and outputs in float32, which a second
// kernel joins.  Where units fill the device evenly by themselves, each is a
// workgroup's and nothing is joined.
//
// A workgroup has four waves: HW of them have 16 query heads each, and 4 / HW groups of
// such take tiles of kTile positions of a piece in turn.  Keys and values arrive by
// DMA, in LDS places of a group's own.  Up to 16 heads (HW 1): a wave by itself, the
// next keys arrive while the values are used and the next values while the keys
// are, and no wave waits for another until the piece ends.  More heads: the waves of
// a group read the same tiles, bring a part of each, and meet once a tile, while
// later ones are on their way.  (Waves with 64 heads of their own had 500 registers
// and 28 KB of code: 64 rows of up to 8192 positions of one key head took them 63 us,
// in e4m3 61, where these take 58 and 43.)  The matrix units (16 x 16 x 32, bf16) take
//   scores   X = K Q^T:  a lane gets 4 positions of a head for each 16 of the tile;
//   outputs  O^T += V^T P^T:  the lane's positions of two such blocks are its 8
//            k-values, so P stays in registers; V^T comes out of LDS through the
//            transposing reads in the same order.
// Rounding: scores, exponentials, sums and outputs are float32, the denominator sums
// unrounded probabilities; the products take bf16 operands.  Up to 16 heads (HW 1),
// which memory bounds, a probability (times the value's e4m3 scale) goes in as bf16
// and again as bf16 of what that leaves: 16 bits of it, for 0 to 4 % of the time (64
// rows of up to 32768 positions bf16 823 -> 822 us, e4m3 453 -> 456; 32 selected pages
// of each 82.2 -> 82.5 and 51.4 -> 52.3; 33 rows of 17 e4m3 pages of heads of 64 13.4 ->
// 14.0; one row of 64 positions 5.1 -> 5.3 and 5.8 -> 6.1).  With more heads the waves' chains of products bound it, and it goes in
// once, off by 2^-8 of itself at most: 64 rows of 64 heads of one key head and up to
// 8192 positions would take 44.5 us for 42.6, in e4m3 42.1 for 37.8.
//
// Running maximum: a head's reference moves, and sums and outputs are rescaled,
// only where a tile's maximum exceeds it by more than kLazy: probabilities reach 2^8
// instead of 1, which costs no precision, and most tiles rescale nothing.
//
// What bounds it.  Long rows: memory.  64 rows of 8 heads of 128 (64 query heads) and
// up to 32768 bf16 positions, 5.4 GB, take 820 to 945 us (the cards differ), 5.7 to 6.6
// TB/s; 32 selected e4m3 pages of each, 279 MB, 48 us, 5.8 TB/s; of the SIMDs' cycles
// the matrix units have 7 and 10 %.  One row of 8192 positions, 34 MB, takes 13.3: 6 of memory,
// the way to the first keys (length, page id, keys one after the other) and a second
// kernel, 2.5 and a launch.  64 heads of one key head, 64 rows of up to 8192 bf16
// positions, 168 MB, 42 to 48 us: the pieces' outputs are a fifth of what is moved, and joining
// them 8 us.  64 positions of one row 5 us, a launch and three trips to memory: code is
// kept short where it runs once, since the first run of each line waits for it (an end
// unrolled by heads, of 10 KB, cost a call of 64 heads 12 us).
#include <type_traits>

#include "kv_device.h"

namespace {

constexpr float kLazy = 8.0f;     // base-2 logits that a tile's maximum exceeds its reference by where that moves
constexpr float kNone = -3.4028234663852886e38f;  // a reference before the first: no logit is less but -infinity
constexpr int kWaves = 4, kThreads = 64 * kWaves;

struct Cut {
  int32_t share, by_unit;
};

struct Attend {
  const uint8_t* q;     // bf16 [rows][heads][D]
  const uint8_t* kv[2];
  const uint8_t* ks[2];
  Tables tables;
  const int32_t* idx;   // [rows][kv_heads][k] (k >= 0)
  const int32_t* sl;
  const float* sinks;   // [heads] or NULL
  uint8_t* out;         // bf16 [rows][heads][D]
  float* lse;           // [rows][heads] or NULL
  Cut* cut;
  int32_t* prefix;      // [rows + 1]: pages (by unit: pieces) of the rows before, of one unit each
  f32x2* ml;            // references and sums of the pieces: [2 * shares][16 * HW]
  f32x4* part;          // their outputs
  KvStrides s;
  uint32_t pages_lim;
  int32_t rows, heads, kv_heads, group, blocks, width, k;
  int32_t shares;       // workgroups with a share; 0: a unit each
  int32_t least, slack, few, most_pieces;  // pages of a share; see cut_of
  int32_t once;         // whether keys and values pass the caches by
  float scale2;         // scale * log2(e)
};

__device__ __forceinline__ int64_t uniform64(int64_t x) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int32_t)(x >> 32)) << 32 | (uint32_t)uniform((int32_t)x));
}

// The same value, of which the compiler knows nothing: what is made of it is made
// here, not kept in registers from before a loop.
__device__ __forceinline__ uint32_t here(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) v2i lds_v2i;
typedef __attribute__((address_space(3))) v4s lds_v4s;

// 64 lanes x 16 bytes from base + off (off each lane's own) to LDS dst + 16 * lane.
// (s_nop: a scalar that a vector instruction has written, as base's halves are, can be
// read by a memory instruction five states on; the compiler counts them for its own
// instructions, not for those in assembly.)
// ONCE: of what is not read again soon, the first to leave the caches.
template <bool ONCE>
__device__ __forceinline__ void dma16_from(int64_t base, uint32_t off, uint32_t dst) {
  if constexpr (ONCE)
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1 nt" ::"v"(off), "s"(base), "{m0}"(dst) : "memory");
  else
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(dst) : "memory");
}

template <int KEY, int DIM, int HW>
struct Form {
  static constexpr int kRowBytes = KEY == kFp8 ? DIM : 2 * DIM;  // of a position
  static constexpr int kGroups = kWaves / HW;
  static constexpr int kTile = 8192 / kRowBytes < 32 ? 32 : 8192 / kRowBytes > 64 ? 64 : 8192 / kRowBytes;
  static constexpr int kBytes = kTile * kRowBytes;  // of a tile's keys, and of its values
  // A CU's LDS is two workgroups', or one's where half of it has too few places.
  static constexpr int kLeast = (HW > 1 ? 2 : 1) * kGroups * 2 * kBytes;
  static constexpr int kPerCu = kLeast > 65536 ? 1 : 2;
  static constexpr int kFit = 131072 / kPerCu / (kGroups * 2 * kBytes);
  static constexpr int kPlaces = HW == 1 ? 1 : kFit > 4 ? 4 : kFit;  // tiles of a group in use or on their way
  static constexpr int kDmas = kBytes / 1024 / HW;  // a wave's, of a tile's keys, and of its values
  static constexpr int kScaleDmas = KEY == kFp8 ? kTile / 32 : 0;
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kRowsPerLine = kRowBytes < 256 ? 256 / kRowBytes : 1;
  static constexpr int kMask = (kChunks < 16 ? kChunks : 16) - 1;
  static constexpr int kSteps = DIM / 32;   // of the scores' sums
  static constexpr int kParts = DIM / 16;   // blocks of 16 values
  static constexpr int kSubs = kTile / 16;  // blocks of 16 positions
  static constexpr bool kFine = HW == 1;    // probabilities of 16 bits

  // Chunk c (16 bytes) of position r stands at place c ^ key(r) of its LDS row, so
  // that what 16 lanes (keys: one chunk of 16 positions) or 32 (values: one or two
  // chunks of 16 or 8 positions) read at once lies in different banks.
  static __device__ __forceinline__ constexpr int key_k(int r) { return (r / kRowsPerLine) & kMask; }
  static __device__ __forceinline__ constexpr int key_v(int r) {
    if (KEY == kBf16) return ((r / kRowsPerLine) << 1) & kMask;
    return ((r / kRowsPerLine) & (kMask >> 1)) | ((r >> 4 & 1) ? (kMask + 1) / 2 : 0);
  }
};

template <int KEY, int DIM, int HW>
struct AttendShared {
  using F = Form<KEY, DIM, HW>;
  uint8_t tile[F::kGroups][F::kPlaces][2][F::kBytes];  // keys, values; at the end outputs
  float scale[kWaves][F::kPlaces][2][KEY == kFp8 ? F::kTile : 4];  // (each wave brings its own)
  f32x2 ml[kWaves][16];
  int32_t sums[kWaves];
  int32_t start[2];
};

// A row's length, and the pages of its units.
__device__ __forceinline__ int32_t length_of(const Attend& a, int64_t b) {
  return min(max(a.sl[b], 0), a.width * kPage);
}
__device__ __forceinline__ int32_t pages_of(const Attend& a, int32_t L) {
  const int32_t c = (int32_t)(((uint32_t)L + kPage - 1) / kPage);
  return a.k >= 0 ? min(a.k, c) : c;
}

// How the units' pages (`total` of all units) are cut: into shares of the same number
// of pages, whatever units they are of, or each unit by itself into pieces of at
// most that many, one a workgroup.  The latter has workgroups to spare for the units'
// last pieces and larger shares for it, but no workgroup with two pieces, which cost
// 3 us each; it is taken where the shares are no more than `slack` larger, and some
// share would end inside a unit (`uneven`).  A unit is
// not cut into more than 32 * HW pieces by far: joining them costs more than a
// larger share (one row of 8 units of 128 pages: 64 pieces each 14.8 us, 32 pieces
// 13.7, 16 pieces 14.1; of 256 pages 19.8, 19.6 and 18.4).  Rows of more than a wave's lanes
// are not cut by units: 64 rows of 2 heads and 1024 bf16 positions take 18.8 us, 65 20.6, in
// e4m3 15.3 and 18.3.  Pieces of 64 heads are about as many
// bytes as a page of their keys and values: shares of up to `few` (6) pages are made
// by half the workgroups (bf16, 8 rows of up to 64 and 128 pages 17.0 and 18.4 us by all, 14.3
// and 17.1 by half; 64 rows of 64 pages in e4m3, shares of 5 and 10 pages, 26.8 and 30.4).
template <class F>
__device__ __forceinline__ Cut cut_of(const Attend& a, int32_t total, F uneven) {
  const auto up = [](uint32_t x, uint32_t by) { return (int32_t)((x + by - 1) / by); };
  const int32_t units = a.rows * a.kv_heads * a.blocks;
  int32_t share = up((uint32_t)total, (uint32_t)a.shares);
  if (a.few > 0) {
    const int32_t twice = up((uint32_t)total, (uint32_t)(a.shares / 2));
    if (twice <= a.few) share = twice;
  }
  Cut c = {max(share, max(a.least, up((uint32_t)total, (uint32_t)(units * a.most_pieces)))), 0};
  if (a.rows <= 64 && 2 * units <= a.shares) {
    const int32_t more = max(c.share, up((uint32_t)total, (uint32_t)(a.shares - units)));
    if (more - c.share <= a.slack && uneven(c.share)) c = {more, 1};
  }
  return c;
}

template <int KEY, int DIM, int HW>
__global__ __launch_bounds__(kThreads, (Form<KEY, DIM, HW>::kPerCu)) void kv_attention_kernel(Attend a) {
  using F = Form<KEY, DIM, HW>;
  constexpr int kTile = F::kTile, kRowBytes = F::kRowBytes, kSteps = F::kSteps, kParts = F::kParts, kSubs = F::kSubs;
  constexpr int kTilesPerPage = kPage / kTile;
  __shared__ __attribute__((aligned(1024))) AttendShared<KEY, DIM, HW> sh;
  const int lane = threadIdx.x & 63, n = lane & 15, quad = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6), hw = wave % HW, group = wave / HW;
  const int32_t per_row = a.kv_heads * a.blocks;

  // The workgroup's pages: of units in order, `end` of them, from page `page0` of unit
  // `unit` of row `b`.
  int64_t b;
  int32_t unit, page0 = 0, count, end, L;
  int32_t early_j = 0, early_page = 0;  // of a unit's first 64 pages, looked up before the row's length is there
  if (a.shares == 0) {
    b = blockIdx.x / (uint32_t)per_row;
    unit = (int32_t)(blockIdx.x - (uint32_t)b * (uint32_t)per_row);
    bool ok;
    const int32_t* tab = a.tables.of(b, ok);
    early_j = lane;
    if (a.k >= 0) early_j = lane < a.k ? a.idx[(b * a.kv_heads + unit / a.blocks) * (int64_t)a.k + lane] : -1;
    early_page = (uint32_t)early_j < (uint32_t)a.width && ok ? tab[early_j] : -1;
    L = length_of(a, b);
    count = end = pages_of(a, L);
  } else if (a.rows <= 64) {  // every wave by itself, a lane a row
    const auto scan = [&](int32_t v) {
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int32_t u = __shfl_up(v, d);
        if (lane >= d) v += u;
      }
      return v;
    };
    const int32_t mine = lane < a.rows ? length_of(a, lane) : 0, own = pages_of(a, mine);
    int32_t each = own, upto = scan(own);  // what a unit of the lane's row counts for, and the rows before it with it
    const Cut cut = cut_of(a, __builtin_amdgcn_readlane(upto, 63) * per_row, [&](int32_t share) {
      return __ballot((uint32_t)own % (uint32_t)share != 0) != 0;
    });
    if (cut.by_unit) {
      each = (own + cut.share - 1) / cut.share;
      upto = scan(each);
    }
    if (blockIdx.x == 0 && wave == 0) {
      if (lane < a.rows) a.prefix[lane] = upto - each;
      if (lane == 63) a.prefix[a.rows] = upto;
      if (lane == 0) *a.cut = cut;
    }
    const int32_t total = __builtin_amdgcn_readlane(upto, 63) * per_row;
    const int64_t first = cut.by_unit ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * cut.share;
    if (first >= total) return;
    const int row = __builtin_ctzll(__ballot(upto * per_row > (int32_t)first));
    b = row;
    L = __builtin_amdgcn_readlane(mine, row);
    count = __builtin_amdgcn_readlane(own, row);
    const int32_t n_each = __builtin_amdgcn_readlane(each, row);
    const int32_t at = (int32_t)first - (__builtin_amdgcn_readlane(upto, row) - n_each) * per_row;
    unit = at / n_each;
    page0 = at - unit * n_each;
    if (cut.by_unit) {
      const int32_t piece = page0;
      page0 = (int32_t)((int64_t)piece * count / n_each);
      end = (int32_t)((int64_t)(piece + 1) * count / n_each) - page0;
    } else {
      end = min(cut.share, total - (int32_t)first);
    }
  } else {
    const int32_t per = (a.rows + kThreads - 1) / kThreads;
    const int32_t r0 = min((int)threadIdx.x * per, a.rows), r1 = min(r0 + per, a.rows);
    int32_t own = 0;
    for (int32_t r = r0; r < r1; ++r) own += pages_of(a, length_of(a, r));
    int32_t upto = own;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int32_t v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    if (lane == 63) sh.sums[wave] = upto;
    __syncthreads();
    int32_t total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) upto += sh.sums[w];
      total += sh.sums[w];
    }
    const Cut cut = cut_of(a, total * per_row, [](int32_t) { return false; });
    if (blockIdx.x == 0) {
      int32_t p = upto - own;
      for (int32_t r = r0; r < r1; ++r) {
        a.prefix[r] = p;
        p += pages_of(a, length_of(a, r));
      }
      if (threadIdx.x == 0) {
        a.prefix[a.rows] = total;
        *a.cut = cut;
      }
    }
    total *= per_row;
    const int64_t first = (int64_t)blockIdx.x * cut.share;
    if (first >= total) return;
    end = min(cut.share, total - (int32_t)first);
    const int32_t at = (int32_t)first;
    if (at < upto * per_row && at >= (upto - own) * per_row) {
      int32_t p = (upto - own) * per_row, r = r0, c = pages_of(a, length_of(a, r));
      while (at >= p + c * per_row) {
        p += c * per_row;
        c = pages_of(a, length_of(a, ++r));
      }
      sh.start[0] = r;
      sh.start[1] = at - p;
    }
    __syncthreads();
    b = uniform(sh.start[0]);
    page0 = uniform(sh.start[1]);
    L = uniform(length_of(a, b));
    count = pages_of(a, L);
    unit = page0 / count;
    page0 -= unit * count;
  }

  const uint32_t lds_tile = (uint32_t)(uintptr_t)(lds_u8*)&sh.tile[group][0][0][0];
  const uint32_t lds_scale = (uint32_t)(uintptr_t)(lds_u8*)&sh.scale[wave][0][0][0];
  // DMA i of a wave brings rows dr + kRowsPerDma * i of a tile; the lane's source
  constexpr int kRowsPerDma = 1024 / kRowBytes;
  const int dr = hw * (kTile / HW) + lane / F::kChunks, dc = lane % F::kChunks;
  const uint32_t from_k = dr * kRowBytes + 16 * (dc ^ F::key_k(dr)), from_v = dr * kRowBytes + 16 * (dc ^ F::key_v(dr));
  // Where the lane reads of a tile: keys, chunk `quad` of position n; values, of its
  // first block of 16, chunks 0 (and 1) of position vr.  Other chunks are this place
  // with bits of the chunk turned over, other positions (16 and 32 on have the same
  // keys) a sum.
  const int vr = KEY == kFp8 ? 16 * (n >> 3) + 4 * quad + (n >> 1 & 3) : 4 * quad + (n >> 2);
  const uint32_t lane_k = lds_tile + n * kRowBytes + 16 * (quad ^ F::key_k(n));
  const uint32_t lane_v = lds_tile + F::kBytes + vr * kRowBytes + 16 * ((KEY == kFp8 ? 0 : n >> 1 & 1) ^ F::key_v(vr)) + 8 * (n & 1);

  int32_t slot = 0;  // of a piece that is not whole: the share's first, or its last
  while (true) {
    const int32_t pages = min(count - page0, end);
    const int32_t h = unit / a.blocks, hb = unit - h * a.blocks;
    const int32_t head0 = h * a.group + 16 * (hb * HW + hw);        // the wave's first, of the row's
    const int32_t heads = min(16, a.group - 16 * (hb * HW + hw));    // (may be less than one)
    const int32_t live = (int32_t)(((uint32_t)L + kPage - 1) / kPage);
    bool table_ok;
    const int32_t* tab = a.tables.of(b, table_ok);
    const int32_t* list = a.k >= 0 ? a.idx + (b * a.kv_heads + h) * (int64_t)a.k : nullptr;

    bf16x8 q[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int d = KEY == kFp8 ? 64 * (s / 2) + 16 * quad + 8 * (s & 1) : 32 * s + 8 * quad;
      q[s] = (bf16x8)((__bf16)0.0f);
      if (n < heads) q[s] = *reinterpret_cast<const bf16x8*>(a.q + ((b * a.heads + head0 + n) * DIM + d) * 2);
    }

    f32x4 acc[kParts];
#pragma unroll
    for (int p = 0; p < kParts; ++p) acc[p] = (f32x4){0.f, 0.f, 0.f, 0.f};
    float ref = kNone, sum = 0.0f;  // of head n: reference, the lane's sum
    bool bad = false;

    // The group's tiles: page `page` of the pool, positions `first` .. of it, `left` of
    // them live (none: nothing to be read).
    struct Tile {
      int32_t page, first, left;
    };
    int32_t ids_from = -64, ids, ids_left;  // lane: page id (-1 outside the pool, -2 to skip) and live positions of page ids_from + lane
    const int32_t tiles = pages * kTilesPerPage;
    auto look = [&](int32_t tile, Tile& t) -> bool {
      t.left = 0;
      if (tile >= tiles) return false;
      const int32_t e = tile / kTilesPerPage;
      if (e >= ids_from + 64) {
        ids_from = e / 64 * 64;
        ids = -2;
        ids_left = 0;
        if (ids_from + lane < pages) {
          const bool early = a.shares == 0 && e < 64;
          const int32_t j = early ? early_j : list ? list[page0 + ids_from + lane] : page0 + ids_from + lane;
          if ((uint32_t)j < (uint32_t)live) {
            const int32_t page = early ? early_page : table_ok ? tab[j] : -1;
            ids = (uint32_t)page < a.pages_lim ? page : -1;
            ids_left = min(L - j * kPage, kPage);
          }
        }
      }
      t.page = __builtin_amdgcn_readlane(ids, e - ids_from);
      t.first = (tile % kTilesPerPage) * kTile;
      if (t.page == -1) bad = true;
      if (t.page >= 0) t.left = max(__builtin_amdgcn_readlane(ids_left, e - ids_from) - t.first, 0);
      return t.left > 0;
    };
    auto fetch = [&](const Tile& t, int place, auto which) {  // keys (with both scales) or values
      constexpr int kWhich = decltype(which)::value;
      const int64_t base = uniform64((int64_t)(uintptr_t)a.kv[kWhich] + t.page * a.s.kv_page + h * a.s.kv_head + t.first * kRowBytes);
      if constexpr (KEY == kFp8 && kWhich == 0) {
        const int64_t at_ = t.page * a.s.ks_page + h * a.s.ks_head + 4 * t.first;
        const uint32_t to = lds_scale + place * 8 * kTile;
        if constexpr (kTile == 64) {
          dma4(a.ks[0] + at_ + 4 * lane, to);
          dma4(a.ks[1] + at_ + 4 * lane, to + 256);
        } else {
          dma4((lane < 32 ? a.ks[0] : a.ks[1]) + at_ + 4 * (lane & 31), to);
        }
      }
      const uint32_t to = lds_tile + (2 * place + kWhich) * F::kBytes + hw * (F::kBytes / HW);
      const uint32_t from = here(kWhich == 0 ? from_k : from_v);
      const auto bring = [&](auto once) {
#pragma unroll
        for (int i = 0; i < F::kDmas; ++i) {
          const int key = kWhich == 0 ? F::key_k(kRowsPerDma * i) : F::key_v(kRowsPerDma * i);
          dma16_from<decltype(once)::value>(base, (from ^ (16 * key)) + 1024 * i, to + 1024 * i);
        }
      };
      if (a.once) bring(std::true_type{});
      else bring(std::false_type{});
    };
    constexpr std::integral_constant<int, 0> kKeys{};
    constexpr std::integral_constant<int, 1> kVals{};

    f32x4 x[kSubs];        // of a tile's positions 16 * s + 4 * quad .. and head n: scores, then base-2 logits
    f32x4 ks[kSubs], vs[kSubs];
    bf16x8 w[kSubs / 2], rest[F::kFine ? kSubs / 2 : 1];  // probabilities, and what bf16 leaves of them
    // (All reads of a tile's keys, or of 32 positions' values, are asked for before the
    // first product: left to itself the compiler waits for each where it is used.)
    auto score = [&](int place) {
      const uint32_t from = here(lane_k + place * 2 * F::kBytes);
      u32x4 raw[F::kChunks / 4][kSubs];
#pragma unroll
      for (int c = 0; c < F::kChunks / 4; ++c)
#pragma unroll
        for (int s = 0; s < kSubs; ++s) raw[c][s] = *(lds_u32x4*)(uintptr_t)((from ^ (64 * c)) + 16 * s * kRowBytes);
      if constexpr (KEY == kFp8) {
#pragma unroll
        for (int s = 0; s < kSubs; ++s) {
          ks[s] = *reinterpret_cast<const f32x4*>(&sh.scale[wave][place][0][16 * s + 4 * quad]);
          vs[s] = *reinterpret_cast<const f32x4*>(&sh.scale[wave][place][1][16 * s + 4 * quad]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < kSubs; ++s) x[s] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < F::kChunks / 4; ++c)
#pragma unroll
        for (int s = 0; s < kSubs; ++s) {
          const u32x4 k = raw[c][s];
          if constexpr (KEY == kFp8) {
            x[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8x8_to_bf16x8(k.x, k.y), q[2 * c], x[s], 0, 0, 0);
            x[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8x8_to_bf16x8(k.z, k.w), q[2 * c + 1], x[s], 0, 0, 0);
          } else {
            x[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k), q[c], x[s], 0, 0, 0);
          }
        }
    };
    auto weigh = [&](int32_t left) {
#pragma unroll
      for (int s = 0; s < kSubs; ++s) x[s] *= KEY == kFp8 ? ks[s] * a.scale2 : (f32x4){a.scale2, a.scale2, a.scale2, a.scale2};
      if (left < kTile) {  // past the row's end: no logit, and values of no weight, whatever is there
#pragma unroll
        for (int s = 0; s < kSubs; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool dead = 16 * s + 4 * quad + e >= left;
            x[s][e] = dead ? -INFINITY : x[s][e];
            if constexpr (KEY == kFp8) vs[s][e] = dead ? 0.0f : vs[s][e];
          }
      }
      float top = x[0][0];
#pragma unroll
      for (int s = 0; s < kSubs; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, x[s][e]);
      if (__ballot(top > ref + kLazy) != 0) {
        float m = fmaxf(top, __shfl_xor(top, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        m = fmaxf(m, ref);
        const float f = __builtin_amdgcn_exp2f(ref - m);
        ref = m;
        sum *= f;
#pragma unroll
        for (int p = 0; p < kParts; ++p) acc[p] *= f;
      }
#pragma unroll
      for (int s = 0; s < kSubs; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = __builtin_amdgcn_exp2f(x[s][e] - ref);
          sum += p;
          const float y = KEY == kFp8 ? p * vs[s][e] : p;
          w[s / 2][4 * (s & 1) + e] = (__bf16)y;
          if constexpr (F::kFine) rest[s / 2][4 * (s & 1) + e] = (__bf16)(y - (float)(__bf16)y);
        }
    };
    auto add = [&](int place, int32_t left) {
      if (left < kTile) {  // (their probability is 0, they may be no numbers)
        for (int i = left * F::kChunks + lane; i < kTile * F::kChunks; i += 64)
          *reinterpret_cast<u32x4*>(sh.tile[group][place][1] + 16 * i) = (u32x4){0u, 0u, 0u, 0u};
      }
      const uint32_t from = here(lane_v + place * 2 * F::kBytes);
#pragma unroll
      for (int i = 0; i < kSubs / 2; ++i) {
        v4s u[kParts][2];  // (e4m3: one of 8 codes)
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
          if constexpr (KEY == kFp8) {
            u[p][0] = __builtin_bit_cast(v4s, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i*)(uintptr_t)((from ^ (16 * p)) + 32 * i * kRowBytes)));
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e)
              u[p][e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(uintptr_t)((from ^ (32 * p)) + (32 * i + 16 * e) * kRowBytes));
          }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
          bf16x8 v;
          if constexpr (KEY == kFp8) {
            const u32x2 c = __builtin_bit_cast(u32x2, u[p][0]);
            v = fp8x8_to_bf16x8(c.x, c.y);
          } else {
            v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(u[p][0], u[p][1], 0, 1, 2, 3, 4, 5, 6, 7));
          }
          acc[p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, w[i], acc[p], 0, 0, 0);
          if constexpr (F::kFine) acc[p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, rest[i], acc[p], 0, 0, 0);
        }
      }
    };
    // The queries have arrived, as far as the compiler knows too: a first use inside the
    // loop made it wait there for everything under way, in every round (64 rows of 64
    // heads of one key head 61 -> 51 us, 32 selected e4m3 pages of 64 rows 49.5 -> 47.8).  They were asked for before the
    // page ids that have been waited for.
    auto queries_there = [&] {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) asm volatile("" : "+v"(q[s]));
    };
    // What a wave has read from LDS is there: DMAs may overwrite it.
    auto reads_done = [] { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); };

    // Operations of a wave complete in order: what it waits for has arrived when no more
    // are outstanding than were issued after it.
    if constexpr (HW == 1) {
      int32_t next = wave;
      auto find = [&](Tile& t) {
        bool found = false;
        for (; next < tiles && !found; next += kWaves) found = look(next, t);
        return found;
      };
      Tile cur, nxt;
      bool more = find(cur);
      queries_there();
      if (more) {
        fetch(cur, 0, kKeys);
        fetch(cur, 0, kVals);
      }
      while (more) {
        const bool ahead = find(nxt);
        wait_vm<F::kDmas>();
        score(0);
        reads_done();
        if (ahead) fetch(nxt, 0, kKeys);
        weigh(cur.left);
        if (ahead) wait_vm<F::kDmas + F::kScaleDmas>();
        else wait_vm<0>();
        add(0, cur.left);
        reads_done();
        if (ahead) fetch(nxt, 0, kVals);
        cur = nxt;
        more = ahead;
      }
    } else {
      // Tile r of a group goes to place r % kPlaces.  When the waves meet for it, their
      // parts have arrived and all are done with tile r - 1, whose place the next takes.
      constexpr int kBehind = F::kPlaces - 1, kOps = 2 * F::kDmas + F::kScaleDmas;  // tiles on their way, operations of each
      static_assert(kBehind >= 1 && kBehind <= 3 && 2 * kOps <= 63);
      const int32_t rounds = (tiles + F::kGroups - 1) / F::kGroups;
      int32_t lefts[kBehind];  // of the tiles on their way, the next one's first
      Tile t;
      const bool first = look(group, t);
      queries_there();
#pragma unroll 1
      for (int r = 0; r < kBehind; ++r) {
        if (r == 0 ? first : look(r * F::kGroups + group, t)) {
          fetch(t, r, kKeys);
          fetch(t, r, kVals);
        }
#pragma unroll
        for (int i = 0; i + 1 < kBehind; ++i) lefts[i] = lefts[i + 1];
        lefts[kBehind - 1] = t.left;
      }
      int place = 0;
#pragma unroll 1
      for (int32_t r = 0; r < rounds; ++r) {
        const int32_t left = lefts[0];
        int after = 0;
#pragma unroll
        for (int i = 1; i < kBehind; ++i) after += lefts[i] > 0 ? 1 : 0;
        if (kBehind > 2 && after == 2) wait_vm<2 * kOps>();
        else if (kBehind > 1 && after == 1) wait_vm<kOps>();
        else wait_vm<0>();
        barrier();
        const int last = place == 0 ? F::kPlaces - 1 : place - 1;
        if (look((r + kBehind) * F::kGroups + group, t)) {
          fetch(t, last, kKeys);
          fetch(t, last, kVals);
        }
        score(place);
        weigh(left);
        add(place, left);
#pragma unroll
        for (int i = 0; i + 1 < kBehind; ++i) lefts[i] = lefts[i + 1];
        lefts[kBehind - 1] = t.left;
        place = place + 1 == F::kPlaces ? 0 : place + 1;
      }
    }

    // The groups' sums and outputs together, blocks of 16 values as they stand in the
    // registers, through the tiles' places.
    const bool whole = a.shares == 0 || pages == count;
    const int64_t head = b * a.heads + head0, piece = 2 * (int64_t)blockIdx.x + slot;
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (bad) sum = __builtin_nanf("");
    float top = sum == 0.0f ? -INFINITY : ref, total = sum;
    if constexpr (F::kGroups > 1) {
      static_assert(kWaves * 64 * DIM <= (int)sizeof(sh.tile));
      if (quad == 0) sh.ml[wave][n] = (f32x2){top, total};
      barrier();
      f32x2 ml[F::kGroups];
      top = -INFINITY;
      total = 0.0f;
#pragma unroll
      for (int g = 0; g < F::kGroups; ++g) {
        ml[g] = sh.ml[g * HW + hw][n];
        top = fmaxf(top, ml[g].x);
      }
      const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int g = 0; g < F::kGroups; ++g) total = fmaf(ml[g].y, __builtin_amdgcn_exp2f(ml[g].x - base), total);
      const float f = __builtin_amdgcn_exp2f(sh.ml[wave][n].x - base);
      f32x4* to = reinterpret_cast<f32x4*>(&sh.tile[0][0][0][0]) + wave * kParts * 64 + lane;
#pragma unroll
      for (int p = 0; p < kParts; ++p) to[64 * p] = acc[p] * f;
    }
    Closing c = {1.0f, 1.0f, 0.0f};
    if (whole) c = close_sum(top, total, a.sinks && n < heads ? a.sinks[head0 + n] * kLog2e : -INFINITY);
    if (group == 0 && quad == 0) {
      if (!whole) a.ml[(piece * HW + hw) * 16 + n] = (f32x2){top, total};
      else if (a.lse && n < heads) a.lse[head + n] = c.lse;
    }
    if constexpr (F::kGroups > 1) barrier();
#pragma unroll
    for (int i = 0; i < kParts / F::kGroups; ++i) {
      const int p = F::kGroups * i + group;
      f32x4 o = acc[i];
      if constexpr (F::kGroups > 1) {
        const f32x4* from = reinterpret_cast<const f32x4*>(&sh.tile[0][0][0][0]) + (hw * kParts + p) * 64 + lane;
        o = from[0];
#pragma unroll
        for (int g = 1; g < F::kGroups; ++g) o += from[g * HW * kParts * 64];
      }
      if (whole) {
        o = o * c.by * c.half * c.half;
        if (n < heads)
          *reinterpret_cast<bf16x4*>(a.out + ((head + n) * DIM + 16 * p + 4 * quad) * 2) =
              (bf16x4){(__bf16)o[0], (__bf16)o[1], (__bf16)o[2], (__bf16)o[3]};
      } else {
        a.part[((piece * HW + hw) * kParts + p) * 64 + lane] = o;
      }
    }
    barrier();  // (LDS is the next piece's)
    if (a.shares == 0) return;
    slot = 1;
    end -= pages;
    if (end <= 0) return;
    page0 = 0;
    if (++unit == per_row) {
      unit = 0;
      do {
        L = uniform(length_of(a, ++b));
        count = pages_of(a, L);
      } while (count == 0);
    }
  }
}

// Joins the pieces of a unit, and writes the units that have no pages: blocks of 16
// values of 16 heads, kParts * HW of them a unit.  The waves of a unit's workgroups take
// the blocks in turn.  FEW units: a workgroup a block, its waves take the pieces in
// turn and join what they have through LDS.  The order is fixed, so the result
// does not depend on the pieces' timing.
template <int DIM, int HW, bool FEW>
__global__ __launch_bounds__(kThreads) void kv_join_kernel(Attend a) {
  constexpr int kParts = DIM / 16, kBatch = FEW ? 16 : 4, kEvery = FEW ? kWaves : 1;
  __shared__ f32x4 outs[FEW ? kWaves : 1][64];
  __shared__ f32x2 mls[FEW ? kWaves : 1][16];
  const int lane = threadIdx.x & 63, n = lane & 15, quad = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);
  const int32_t per_row = a.kv_heads * a.blocks;
  const int32_t b = (int32_t)(blockIdx.x / (uint32_t)per_row), unit = (int32_t)(blockIdx.x - (uint32_t)b * (uint32_t)per_row);
  const int32_t h = unit / a.blocks, hb = unit - h * a.blocks;
  const Cut cut = *a.cut;
  const int32_t before = a.prefix[b], each = a.prefix[b + 1] - before;
  const int32_t s = before * per_row + unit * each;  // the unit's pages or pieces: s .. s + each
  const int32_t share = cut.by_unit ? 1 : cut.share;
  const int32_t w0 = s / share, w1 = each > 0 ? (s + each - 1) / share : w0 - 1;
  if (w0 == w1) return;  // whole
  for (int block = FEW ? (int)blockIdx.y : (int)blockIdx.y * kWaves + wave; block < HW * kParts;
       block += FEW ? HW * kParts : (int)gridDim.y * kWaves) {
    const int t = block / kParts, p = block % kParts;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float top = -INFINITY, total = 0.0f;
#pragma unroll 1
    for (int32_t w = FEW ? w0 + wave : w0; w <= w1; w += kBatch * kEvery) {
      f32x2 ml[kBatch];
      f32x4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int32_t x = w + i * kEvery;
        ml[i] = (f32x2){-INFINITY, 0.0f};
        v[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
        if (x <= w1) {
          const int64_t piece = 2 * (int64_t)x + (x == w0 && s != w0 * share ? 1 : 0);
          ml[i] = a.ml[piece * 16 * HW + 16 * t + n];
          v[i] = a.part[((piece * HW + t) * kParts + p) * 64 + lane];
        }
      }
      float to = top;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) to = fmaxf(to, ml[i].x);
      const float base = to == -INFINITY ? 0.0f : to, by = __builtin_amdgcn_exp2f(top - base);
      top = to;
      total *= by;
      o *= by;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float f = __builtin_amdgcn_exp2f(ml[i].x - base);
        total = fmaf(ml[i].y, f, total);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = fmaf(v[i][e], f, o[e]);
      }
    }
    if constexpr (FEW) {
      outs[wave][lane] = o;
      if (quad == 0) mls[wave][n] = (f32x2){top, total};
      __syncthreads();
      if (wave != 0) return;
      f32x2 ml[kWaves];
      top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        ml[w] = mls[w][n];
        top = fmaxf(top, ml[w].x);
      }
      const float base = top == -INFINITY ? 0.0f : top;
      o = (f32x4){0.f, 0.f, 0.f, 0.f};
      total = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(ml[w].x - base);
        total = fmaf(ml[w].y, f, total);
        const f32x4 v = outs[w][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = fmaf(v[e], f, o[e]);
      }
    }
    const int32_t i = hb * 16 * HW + 16 * t + n;
    if (i >= a.group) continue;
    const int32_t head = h * a.group + i;
    const Closing c = close_sum(top, total, a.sinks ? a.sinks[head] * kLog2e : -INFINITY);
    o = o * c.by * c.half * c.half;
    *reinterpret_cast<bf16x4*>(a.out + (((int64_t)b * a.heads + head) * DIM + 16 * p + 4 * quad) * 2) =
        (bf16x4){(__bf16)o[0], (__bf16)o[1], (__bf16)o[2], (__bf16)o[3]};
    if (a.lse && p == 0 && quad == 0) a.lse[(int64_t)b * a.heads + head] = c.lse;
  }
}

// ---------------------------------------------------------------------------
// Host side.

constexpr int64_t kMaxHeads = 8000000;  // of a call's rows together: a launch has less than 2^32 threads

struct Split {
  int hw, blocks, shares;  // waves of 16 heads of a unit, blocks of them a group, workgroups (0: a unit each)
  int least, slack, few;
  bool once;
  int64_t bytes;
};

inline int64_t padded(int64_t n) { return (n + 255) / 256 * 256; }

bool dims_ok(int32_t rows, int32_t num_heads, int32_t kv_heads, int32_t table_width, int32_t k) {
  return rows >= 0 && num_heads >= 0 && kv_heads >= 0 && (kv_heads == 0 ? num_heads == 0 : num_heads % kv_heads == 0) &&
         table_width >= 0 && table_width <= kMaxWidth && k >= -1 && (int64_t)rows * num_heads <= kMaxHeads;
}

// Workgroups of a form that a CU holds.
int per_cu(int key, int32_t head_dim, int hw) {
  const auto of = [&](auto d, auto n) {
    return key == kFp8 ? Form<kFp8, decltype(d)::value, decltype(n)::value>::kPerCu : Form<kBf16, decltype(d)::value, decltype(n)::value>::kPerCu;
  };
  const auto with = [&](auto d) {
    return hw == 1 ? of(d, std::integral_constant<int, 1>{}) : hw == 2 ? of(d, std::integral_constant<int, 2>{}) : of(d, std::integral_constant<int, 4>{});
  };
  return head_dim == 64 ? with(std::integral_constant<int, 64>{}) : head_dim == 128 ? with(std::integral_constant<int, 128>{})
                                                                                   : with(std::integral_constant<int, 256>{});
}

// From the scalar arguments alone (the lengths are on the device).
Split split_of(int key, int32_t rows, int32_t num_heads, int32_t kv_heads, int32_t head_dim, int32_t table_width, int32_t k) {
  Split s = {1, 1, 0, 0, 0, 0, false, 0};
  if (rows == 0 || num_heads == 0) return s;
  const int32_t group = num_heads / kv_heads;
  while (s.hw < kWaves && 16 * s.hw < group) s.hw *= 2;
  // (Two blocks read keys and values twice: 64 rows of one key head and up to 8192 bf16
  // positions take 43 us with 64 query heads and 68 with 128, in e4m3 38 and 57.)
  s.blocks = (group + 16 * s.hw - 1) / (16 * s.hw);
  const int64_t units = (int64_t)rows * kv_heads * s.blocks;
  const int64_t most = k >= 0 && k < table_width ? k : table_width;  // pages of a unit
  const int64_t workgroups = (int64_t)per_cu(key, head_dim, s.hw) * device_cu_count();
  const int64_t page_bytes = (int64_t)2 * kPage * head_dim * (key == kFp8 ? 1 : 2);
  // Keys and values of a call that may read 256 MiB or more, the size of the last cache,
  // would leave it before they are read again, and pass it by: 64 rows of 8 heads and 32
  // selected pages of e4m3 (279 MB) 59 -> 52 us, all of up to 512 pages of bf16 (5.4 GB)
  // 1025 -> 945, 64 rows of 2 heads with 32 queries each (335 MB) 75 -> 64.  But 33 rows of 8
  // heads of 64 and 17 pages (39 MB, three such in turn) 13.1 -> 14.8, 32 rows of one head
  // with 64 queries (84 MB) 30.5 -> 36.7.  (What the tables may name decides, since the lengths
  // are on the device: 8 rows of 8 heads and 1920 positions in tables of 4097 columns 21.5 ->
  // 21.0 in bf16, 31 MB, but 17.4 -> 18.0 in e4m3, 16 MB.)
  s.once = s.blocks == 1 && units * most * page_bytes >= (int64_t)1 << 28;
  // More units than four rounds of workgroups: whole.  Rows of like lengths gain by it: 300
  // rows of 8 heads and 512 bf16 positions each 103 us, cut 119, of up to 512 and 2048 (a
  // quarter of it the least) 73 and 250, cut 98 and 282.  One row of 32768 among 299 of 512
  // loses: 346, cut 143.
  if (units > 4 * workgroups || units * most > INT32_MAX / 2) return s;
  // A unit of few pages is done by its workgroup before a second kernel could join its
  // pieces: 8 units of 4, 8 and 16 pages of 32 KB take 6.3, 8.4 and 12.3 us whole, 8.1,
  // 8.2 and 8.8 cut; 64 units 6.6, 8.5 and 14.2, and 11.2, 11.8 and 15.4; 8 units of
  // 64 heads and 2, 4 and 8 pages 8.2, 11.8 and 19.2, and 9.5, 12.3 and 12.9.  So are units
  // that fill the device, unless rows may be far longer than others: 512 units of
  // up to 16, 32 and 128 pages (a quarter of it the least) 36, 71 and 257 us, cut 45, 77
  // and 248.  (By the table's width: 64 rows of 8 heads and 256 positions take 17.0 us in tables
  // of 4 columns, whole, and 17.9 in tables of 4097, cut; in e4m3 11.8 and 14.8.)
  if (most * s.hw <= 8 || (2 * units >= workgroups && most <= 32)) return s;
  // Selections are mostly of one size: whole units, where the last round of workgroups
  // is full, nearly half full, or short (43008 bytes are 4 us of a workgroup's).  Rows of 8
  // heads in bf16, on 512 workgroups: 64, 30 and 48 rows of 32 pages 99, 55.5 and 76 us, cut
  // 101, 63 and 81; cut, 4 rows of 32 and 10 of 64 15.4 and 40.5, whole 22.6 and 48.4.  It errs
  // for 20 rows of 32 (cut 46.5, whole 41.5), where the last round is just over half full (33
  // rows of 32 and 128 69 and 241, cut 63 and 190) and for lists of a few long rows among
  // short ones (all of 32768 positions in 4 rows and of 1024 in 60 329, cut 136).
  const int64_t last = units % workgroups;
  if (k >= 0 && (last == 0 || (2 * workgroups - 5 * last) * most * page_bytes < 5 * workgroups * 43008)) return s;
  s.least = s.hw == 4 ? 1 : 2;
  s.slack = (int)(65536 / page_bytes);
  const int64_t want = (units * most + s.least - 1) / s.least + units;  // (a unit's last piece may be short)
  s.shares = (int)(want < workgroups ? want : workgroups);
  if (s.hw == kWaves && s.shares > device_cu_count()) s.few = 6;
  s.bytes = padded(8 + 4 * ((int64_t)rows + 1)) + padded(2 * (int64_t)s.shares * 16 * s.hw * 8) +
            2 * (int64_t)s.shares * s.hw * head_dim * 64;
  return s;
}

template <int KEY, int DIM, int HW>
void launch(const Attend& a, const Split& split, hipStream_t stream) {
  const uint32_t units = (uint32_t)((int64_t)a.rows * a.kv_heads * a.blocks);
  kv_attention_kernel<KEY, DIM, HW><<<dim3(split.shares ? (uint32_t)split.shares : units), dim3(kThreads), 0, stream>>>(a);
  if (split.shares == 0) return;
  // Pieces are shared among waves where a unit may have 16, or 8 and few blocks in all (32
  // units of 32 blocks, 8 pieces each: 14.4 us so, the attention with it, 12.4 otherwise; one
  // unit of them 9.2 and 9.5).
  const int64_t blocks = (int64_t)units * HW * DIM / 16;
  if (split.shares >= (blocks <= 512 ? 8 : 16) * (int64_t)units) kv_join_kernel<DIM, HW, true><<<dim3(units, HW * DIM / 16), dim3(kThreads), 0, stream>>>(a);
  else {
    uint32_t y = 512 / units;
    if (y > HW * DIM / 16 / kWaves) y = HW * DIM / 16 / kWaves;
    kv_join_kernel<DIM, HW, false><<<dim3(units, y < 1 ? 1 : y), dim3(kThreads), 0, stream>>>(a);
  }
}

template <int KEY, int DIM>
void launch_for(const Attend& a, const Split& split, hipStream_t stream) {
  if (split.hw == 1) return launch<KEY, DIM, 1>(a, split, stream);
  if (split.hw == 2) return launch<KEY, DIM, 2>(a, split, stream);
  launch<KEY, DIM, 4>(a, split, stream);
}

template <int KEY>
int kv_attention(const void* q, const void* k_pages, const void* v_pages, const float* kscale, const float* vscale,
                 const int32_t* page_table, const int32_t* row_table, int32_t num_tables, const int32_t* page_idx,
                 const int32_t* seqlens, const float* sinks, void* out, float* lse, int32_t rows, int32_t num_heads,
                 int32_t kv_heads, int32_t head_dim, int32_t table_width, int64_t num_pages, const KvStrides& s,
                 int64_t page_table_row_stride, int32_t k, float scale, void* workspace, int64_t workspace_bytes,
                 hipStream_t stream) {
  if (!head_dim_ok(head_dim) || (int64_t)num_heads > (int64_t)kMaxGroup * kv_heads) return IDX_ERR_UNSUPPORTED;
  if (!dims_ok(rows, num_heads, kv_heads, table_width, k) || page_table_row_stride < 0 || num_tables < 0 ||
      !(fabsf(scale * kLog2e) < INFINITY) || workspace_bytes < 0)
    return IDX_ERR_SHAPE;
  int st = validate_kv_strides(KEY, kv_heads, head_dim, num_pages, s);
  if (st != IDX_OK || rows == 0 || num_heads == 0) return st;
  if (!q || !seqlens || !out || (table_width > 0 && !page_table) || (k > 0 && !page_idx) || (k < 0 && page_idx))
    return IDX_ERR_NULL;
  st = validate_kv_pointers(KEY, kv_heads, k_pages, kscale, s);
  if (st == IDX_OK) st = validate_kv_pointers(KEY, kv_heads, v_pages, vscale, s);
  if (st != IDX_OK) return st;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(page_table, 4) || !aligned(row_table, 4) || !aligned(page_idx, 4) ||
      !aligned(seqlens, 4) || !aligned(sinks, 4) || !aligned(lse, 4) || !aligned(workspace, 16))
    return IDX_ERR_ALIGN;
  const Split split = split_of(KEY, rows, num_heads, kv_heads, head_dim, table_width, k);
  if (split.bytes > 0 && !workspace) return IDX_ERR_NULL;
  if (workspace_bytes < split.bytes) return IDX_ERR_SHAPE;
  Attend a;
  a.q = static_cast<const uint8_t*>(q);
  a.kv[0] = static_cast<const uint8_t*>(k_pages);
  a.kv[1] = static_cast<const uint8_t*>(v_pages);
  a.ks[0] = reinterpret_cast<const uint8_t*>(kscale);
  a.ks[1] = reinterpret_cast<const uint8_t*>(vscale);
  a.tables = {page_table, row_table, page_table_row_stride, num_tables};
  a.idx = page_idx;
  a.sl = seqlens;
  a.sinks = sinks;
  a.out = static_cast<uint8_t*>(out);
  a.lse = lse;
  uint8_t* space = static_cast<uint8_t*>(workspace);
  a.cut = reinterpret_cast<Cut*>(space);
  a.prefix = reinterpret_cast<int32_t*>(space + 8);
  a.ml = reinterpret_cast<f32x2*>(space + padded(8 + 4 * ((int64_t)rows + 1)));
  a.part = reinterpret_cast<f32x4*>(reinterpret_cast<uint8_t*>(a.ml) + padded(2 * (int64_t)split.shares * 16 * split.hw * 8));
  a.s = s;
  a.pages_lim = pages_limit(num_pages);
  a.rows = rows;
  a.heads = num_heads;
  a.kv_heads = kv_heads;
  a.group = num_heads / kv_heads;
  a.blocks = split.blocks;
  a.width = table_width;
  a.k = k;
  a.shares = split.shares;
  a.least = split.least;
  a.slack = split.slack;
  a.few = split.few;
  a.once = split.once;
  a.most_pieces = 32 * split.hw;
  a.scale2 = scale * kLog2e;
  (void)hipGetLastError();  // start from a clean error state
  if (head_dim == 64) launch_for<KEY, 64>(a, split, stream);
  else if (head_dim == 128) launch_for<KEY, 128>(a, split, stream);
  else launch_for<KEY, 256>(a, split, stream);
  return launch_status();
}

}  // namespace

extern "C" {

int64_t idx_kv_attention_workspace(int32_t rows, int32_t num_heads, int32_t kv_heads, int32_t head_dim,
                                   int32_t table_width, int32_t k) {
  if (!head_dim_ok(head_dim) || !dims_ok(rows, num_heads, kv_heads, table_width, k) ||
      (int64_t)num_heads > (int64_t)kMaxGroup * kv_heads)
    return -1;
  // (either key type's call may be made with it)
  const int64_t one = split_of(kFp8, rows, num_heads, kv_heads, head_dim, table_width, k).bytes;
  const int64_t two = split_of(kBf16, rows, num_heads, kv_heads, head_dim, table_width, k).bytes;
  return one > two ? one : two;
}

int idx_kv_attention_fp8(const void* q, const void* k_pages, const void* v_pages, const float* kscale,
                         const float* vscale, const int32_t* page_table, const int32_t* row_table,
                         int32_t num_tables, const int32_t* page_idx, const int32_t* seqlens,
                         const float* sinks, void* out, float* lse, int32_t rows, int32_t num_heads,
                         int32_t kv_heads, int32_t head_dim, int32_t table_width, int64_t num_pages,
                         int64_t kv_page_stride, int64_t kv_head_stride, int64_t kscale_page_stride,
                         int64_t kscale_head_stride, int64_t page_table_row_stride, int32_t k, float scale,
                         void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  return kv_attention<kFp8>(q, k_pages, v_pages, kscale, vscale, page_table, row_table, num_tables, page_idx, seqlens, sinks,
                            out, lse, rows, num_heads, kv_heads, head_dim, table_width, num_pages,
                            {kv_page_stride, kv_head_stride, kscale_page_stride, kscale_head_stride},
                            page_table_row_stride, k, scale, workspace, workspace_bytes, stream);
}

int idx_kv_attention_bf16(const void* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
                          const int32_t* row_table, int32_t num_tables, const int32_t* page_idx,
                          const int32_t* seqlens, const float* sinks, void* out, float* lse, int32_t rows,
                          int32_t num_heads, int32_t kv_heads, int32_t head_dim, int32_t table_width,
                          int64_t num_pages, int64_t kv_page_stride, int64_t kv_head_stride,
                          int64_t page_table_row_stride, int32_t k, float scale, void* workspace,
                          int64_t workspace_bytes, hipStream_t stream) {
  return kv_attention<kBf16>(q, k_pages, v_pages, nullptr, nullptr, page_table, row_table, num_tables, page_idx, seqlens,
                             sinks, out, lse, rows, num_heads, kv_heads, head_dim, table_width, num_pages,
                             {kv_page_stride, kv_head_stride, 0, 0}, page_table_row_stride, k, scale, workspace,
                             workspace_bytes, stream);
}

}  // extern "C"
