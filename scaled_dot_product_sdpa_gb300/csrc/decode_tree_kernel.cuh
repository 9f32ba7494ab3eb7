// decode_tree_kernel.cuh -- attention of several new tokens per sequence over a paged cache (see
// decode_tree.cuh): the kernel, the join of rows that were cut, and their launch for one head_dim.
//
// Both products run on the tensor cores with the rows (a key head's query heads times new tokens) as
// the 128-row operand, so that a softmax thread owns one row and no maximum or sum leaves it:
//     S [128 rows x 128 keys] = Q K^T,   O [128 rows x d] += P V,   P from tensor memory, over its S.
// Weights enter the second product (in fp16 times 2^11, in bf16 times 2^-40, see kShift) of up to 32 rows as two 16-bit parts, P = hi + lo,
// over twice the keys (that keeps 16 bits in bf16, 22 in fp16), of more rows rounded to the cache's type (see
// tree_split_weights).  The tensor cores add to an fp32 accumulator by cutting off what falls below its last bit: so
// a sum leaves its accumulator every `fold` tiles (see tree_fold), for a place in shared memory (up to 32 rows) or the workspace where it is
// added to in fp32, rounded to nearest, and the weights' sum with it.  Each such run of tiles goes by its own maximum, so that a weight's last bit is one of that
// run's, however long the row is (in fp16 weights below 2^-25 of the maximum are subnormal, kept to 2^-36 of it).
//
// d <= 128: two accumulator sets ("streams"), each an S tile, an O tile and a softmax warpgroup of its own,
// so that one's products run while the other's softmax does.  Where a key head's rows fill one row tile
// the streams take its key tiles in turn, each with its own running maximum and sum, and are
// joined at the unit's end; where there are more rows, the streams are two row tiles that share
// every K and V tile.  d >= 256: tensor memory holds one O beside two S tiles; one warpgroup.
//
// Work: the units' key tiles (see TreeShape) in order of sequence, key head, tokens, cut into equal shares, one
// per persistent CTA, whatever the lengths.  A share's first and last units may be parts of longer ones: those partial
// results go to the workspace, and tree_join_kernel joins them in a fixed order.
//
// Warps: an MMA issuer, three TMA producers (keys, values, queries), 4 or 8 of softmax.  K and V tiles pass through one ring of
// slots (128 keys x 64 or 128 columns); pages of fewer than 128 slots make several TMA boxes a slot, one a lane.  The key
// producer tells the issuer what a tile is, the query producer the softmax what a segment is, so that each
// thing is worked out once and in one place: what a role runs through in its turn competes for the instruction caches with
// the seven others (as first written, 147 us where 93 are taken now, a third of all issue slots waited for instructions).
//
// Measured on GB300 (131072 tokens x 8 key heads x 128, bf16, pages of 16; 537 MB, floor 79 us, of which 8 to 11 are launch,
// first tile and join): 16 or 32 rows a key head 92 to 93 us, 64 92, 128 94 (5.7 TB/s; a longer row runs at 7.0 TB/s), 256 121
// (1140 TFLOP/s), 512 222 (1237).  The same bytes at d = 64 117, bound by the issuer's turn of twelve products a tile (with 32 rows
// 133: twenty); at 256 98 to 99; at 512 with up to 64 rows 132 to 134 (K is read for each half of V's columns), with 128 247 (and again
// for each 64 rows).  Pages of 8 109: a producer issues a box of 8 rows in about 94 cycles.  One sequence of 1000 tokens 11 us; 200 of
// 50 to 300 tokens, 32/8 heads x 4 tokens, 106: a unit of two tiles is a chain of two softmaxes, two products and a result, which explains half of it.
#pragma once

#include <atomic>

#include "decode_tree.cuh"
#include "attn_fwd_kernel.cuh"
#include "ptx_paged.cuh"
#include "rope.cuh"
#include "vec16.cuh"

namespace gbattn {
namespace {

constexpr unsigned kTreeSmemAlign = 7;  // GBATTN_DEV_SMEM_ALIGN
constexpr int kProducers = 3;
constexpr int kAhead = 2;       // tiles whose page numbers a producer reads ahead
// Weights are kept times 2^11 in fp16, so that those of a long tail stay normal numbers.  In bf16, whose values reach the end of
// fp32, they enter the second product times 2^-40: 2^31 of them, of up to 2^4, times the largest value stay below 2^128.  (By a
// product of its own, which is exact: off the exponent's argument it would round the weights to 2^-19 of themselves.)
template <bool BF>
constexpr float kShift = BF ? 0.f : 11.f;
template <bool BF>
constexpr float kValueScale = BF ? 0x1p-40f : 1.f;
template <bool BF>
constexpr float kValueBack = BF ? 0x1p40f : 1.f;
constexpr int kTreeSegs = 8;    // segments whose words are kept
constexpr float kSlack = 4.f;   // the running maximum moves when a logit exceeds it by 2^4

// RT: row tiles of a unit.
template <int D, int RT>
struct TreeCfg {
  static constexpr int WG = tree_streams(D);            // softmax warpgroups, accumulators
  static constexpr int SOFTMAX = 128 * WG;
  static constexpr int THREADS = SOFTMAX + 32 + 32 * kProducers;
  static constexpr int CW = D == 64 ? 64 : 128;         // columns of a ring slot
  static constexpr int NBOX = CW / 64;
  static constexpr int BOX_BYTES = kTreeTile * 128;
  static constexpr int SLOT_BYTES = NBOX * BOX_BYTES;
  static constexpr int DV = tree_columns(D);            // columns of O
  static constexpr int NC = D / CW, NV = DV / CW;       // slots of a K tile, of a V tile
  static constexpr int MAX_SLOTS = D == 64 ? 12 : 6;
  // With one slot a tile, the commit that frees K's slot also tells that S is there (a commit costs its thread about 190
  // cycles): the slot's next load but two (of V, or of the K after it) waits for the weights made of that S.
  static constexpr bool ONE = NC == 1;
  static constexpr int PAGE_BYTES = 2 * kAhead * 16 * 4;  // page numbers read ahead, of two producers
  static constexpr int EXCHANGE_BYTES = WG == 2 && RT == 1 ? 2 * 2 * 128 * 4 : 0;  // the streams' maxima and sums
  static constexpr int BAR_BYTES = 768;                 // barriers, the tiles' and the segments' words
  static constexpr int SMEM_MOST = 232448;
  static constexpr int ROOM = SMEM_MOST - PAGE_BYTES - EXCHANGE_BYTES - BAR_BYTES;  // queries, ring and sums
  // barriers
  static constexpr int B_FULL = 0, B_EMPTY = MAX_SLOTS, B_QFULL = 2 * MAX_SLOTS, B_QEMPTY = B_QFULL + 2, B_SFULL = B_QEMPTY + 2, B_PFULL = B_SFULL + 2,
                       B_PDONE = B_PFULL + 2, B_DRAIN = B_PDONE + 2, B_MEET = B_DRAIN + 1, B_SEG = B_MEET + 1, NBAR = B_SEG + kTreeSegs;
  // tensor memory
  static constexpr int T_O = 256;
  static_assert(T_O + WG * DV <= 512, "tensor memory");
  static_assert(RT == 1 || WG == 2, "two row tiles are two streams");
};

__device__ __forceinline__ int tiles_of(int n) { return (n >> 7) + ((n & 127) != 0); }

// a / b of non-negative numbers, by 32-bit division where it serves (it nearly always does).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Tokens of a sequence, and its new ones (none where either is bad).
struct Tokens {
  int len, cnt;
};
// Its numbers as they are (a sequence behind the last one: none), and what they come to.
__device__ __forceinline__ Tokens given_tokens(const TreeParams &p, int b) {
  if (b >= p.B) return {0, 0};
  return {p.lengths[b], p.counts ? p.counts[b] : p.T};
}
__device__ __forceinline__ Tokens sound_tokens(const TreeParams &p, Tokens s, bool report = false) {
  if (s.len >= 0 && s.cnt >= 0 && s.cnt <= p.T && s.cnt <= s.len && s.len <= static_cast<long long>(p.table_w) * p.page) return s;
  if (report) atomicCAS(p.status, 0u, kDevBadLength);
  return {0, 0};
}
__device__ __forceinline__ Tokens tokens_of(const TreeParams &p, int b, bool report = false) { return sound_tokens(p, given_tokens(p, b), report); }
// Key tiles of a sequence's unit of tokens tu * span ..: without a mask its last row sees no key behind itself.
__device__ __forceinline__ int unit_tiles(const TreeParams &p, Tokens s, int tu, int span) {
  return tiles_of(p.mask ? s.len : s.len - s.cnt + static_cast<int>(min(static_cast<long long>(s.cnt), (tu + 1LL) * span)));
}

// What the issuer needs to know of a tile, in a word that comes with its K: groups of 16 keys, whether it is the first and the
// last of its segment, whether O begins anew with it, whether it is its accumulator's last of the segment; the
// queries' buffer and that buffer's phase.
constexpr uint32_t kTileGroups = 15, kTileFirst = 16, kTileLast = 32, kTileFresh = 64, kTileDone = 128;
constexpr int kTileBuffer = 8, kTileTurn = 9;
constexpr uint32_t kTileInfos = 16;  // words kept: more than the ring's tiles and those between their QK and their PV

// A run of one unit's tiles within a CTA's share.
struct Seg {
  int b, kv, tu, x, tile, count, tiles;  // x: block of heads and half of the columns; tiles: of the whole unit
  Tokens s;
};
struct Start {  // a CTA's share: its first unit, the tile in it, its tiles in all
  int b, kv, tu, x, tile;
  Tokens s;
  long long left;
};

// Walks over a CTA's share, with the next sequence's lengths on the way.
struct Walk {
  Start at;
  Tokens ahead;  // as given: nothing waits for them before they are needed
  const TreeParams &p;
  const int span, nx;
  __device__ Walk(const TreeParams &pp, const Start &start)
      : at(start), p(pp), span(pp.s.tokens * pp.s.tiles), nx(pp.s.head_units * pp.s.halves) {
    ahead = given_tokens(p, at.left > 0 ? at.b + 1 : p.B);
  }
  __device__ bool next(Seg &s) {
    if (at.left <= 0 || at.b >= p.B || at.s.cnt == 0) return false;  // (the latter two not unless the lengths change under the kernel)
    s.b = at.b;
    s.kv = at.kv;
    s.tu = at.tu;
    s.x = at.x;
    s.s = at.s;
    s.tile = at.tile;
    s.tiles = unit_tiles(p, at.s, at.tu, span);
    s.count = static_cast<int>(min(at.left, static_cast<long long>(s.tiles - at.tile)));
    at.left -= s.count;
    at.tile += s.count;
    if (at.tile == s.tiles) {
      at.tile = 0;
      if (++at.x == nx) {
        at.x = 0;
        if ((++at.tu) * static_cast<long long>(span) >= at.s.cnt) {
          at.tu = 0;
          if (++at.kv == p.Hkv) {
            at.kv = 0;
            do {
              ++at.b;
              at.s = sound_tokens(p, ahead);
              ahead = given_tokens(p, at.b + 1);
            } while (at.left > 0 && at.b < p.B && at.s.cnt == 0);
          }
        }
      }
    }
    return true;
  }
};

// The same by one thread, tile by tile, with the page and slot of the tile's row `row` (a page's
// slots follow one another through the tiles of a segment, so that only its first tile divides).
struct Cursor {
  Walk w;
  Seg s;
  int i = 0, seg = -1, row;
  int index = 0, slot = 0;   // index: in the sequence's table row
  int keys = 0, behind = 0;  // valid keys in the tile; tokens of the sequence from the tile's first on
  __device__ Cursor(const TreeParams &p, const Start &at, int r) : w(p, at), row(r) { s.count = 0; }
  __device__ bool next() {
    if (i == s.count) {
      if (!w.next(s)) return false;
      i = 0;
      ++seg;
      const int first = s.tile * kTreeTile, pos = first + row;
      index = pos / w.p.page;
      slot = pos - index * w.p.page;
      behind = s.s.len - first;
    } else {
      index += w.p.tile_pages;
      slot += w.p.tile_slots;
      if (slot >= w.p.page) {
        slot -= w.p.page;
        ++index;
      }
      behind -= kTreeTile;
    }
    ++i;
    keys = min(kTreeTile, behind);
    return true;
  }
};

// Where a tile's V begins in the ring's order: K0 K1 V0 K2 V1 ... (T tiles) or, for two row tiles, K0 V0 K1 V1 ...
template <class C, int RT>
__device__ __forceinline__ uint32_t v_pos(uint32_t t, uint32_t T) {
  return RT == 2 ? t * (C::NC + C::NV) + C::NC : min(t + 2, T) * C::NC + t * C::NV;
}

// The first n of 32 bits.
__device__ __forceinline__ uint32_t first_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// 32 of a row's logits (fp32 bits): those whose bits are not set become -inf.
__device__ __forceinline__ void hide(uint32_t (&s)[32], uint32_t seen) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (!(seen >> c & 1u)) s[c] = 0xff800000u;
}
__device__ __forceinline__ float max32(const uint32_t (&r)[32]) {
  const float *const s = reinterpret_cast<const float *>(r);
  float m[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    m[k] = fmaxf(fmax3(fmax3(s[8 * k], s[8 * k + 1], s[8 * k + 2]), s[8 * k + 3], s[8 * k + 4]), fmax3(s[8 * k + 5], s[8 * k + 6], s[8 * k + 7]));
  return fmax3(m[0], m[1], fmaxf(m[2], m[3]));
}
// Two weights as they enter the second product.
template <bool BF>
__device__ __forceinline__ uint64_t scaled(uint64_t w) {
  return BF ? fmul2(w, f32x2(kValueScale<BF>, kValueScale<BF>)) : w;
}
// 16 logits as weights 2^(s c2 - m), rounded once; adds the weights to acc.
template <bool BF>
__device__ __forceinline__ void pack16(const uint32_t (&r)[16], uint32_t *w, uint64_t c2x2, uint64_t negm, uint64_t (&acc)[4], float &top) {
  const float *const s = reinterpret_cast<const float *>(r);
  top = fmaxf(fmax3(top, fmax3(fmax3(s[0], s[1], s[2]), s[3], s[4]), fmax3(fmax3(s[5], s[6], s[7]), s[8], s[9])), fmax3(fmax3(s[10], s[11], s[12]), fmax3(s[13], s[14], s[15]), s[0]));
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    float x0, x1;
    f32x2_split(ffma2(f32x2(s[2 * c], s[2 * c + 1]), c2x2, negm), x0, x1);
    const float w0 = ex2_approx(x0), w1 = ex2_approx(x1);
    acc[c & 3] = fadd2(acc[c & 3], f32x2(w0, w1));
    f32x2_split(scaled<BF>(f32x2(w0, w1)), x0, x1);
    w[c] = pack2<BF>(x0, x1);
  }
}
// 32 logits as weights 2^(s c2 - m): hi parts, then lo parts, 16 columns each, over the logits at `to`.  Adds the weights to acc.
template <bool BF, bool LO>
__device__ __forceinline__ void weights32(const uint32_t (&r)[32], uint32_t to, uint64_t c2x2, uint64_t negm, uint64_t (&acc)[4]) {
  const float *const s = reinterpret_cast<const float *>(r);
  uint32_t w[LO ? 32 : 16];
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    float x0, x1;
    f32x2_split(ffma2(f32x2(s[2 * c], s[2 * c + 1]), c2x2, negm), x0, x1);
    const float w0 = ex2_approx(x0), w1 = ex2_approx(x1);
    acc[c & 3] = fadd2(acc[c & 3], f32x2(w0, w1));
    f32x2_split(scaled<BF>(f32x2(w0, w1)), x0, x1);
    if constexpr (LO)
      split_weights<BF>(x0, x1, w[c], w[16 + c]);
    else
      w[c] = pack2<BF>(x0, x1);
  }
  if constexpr (LO)
    tmem_st32x32_async(to, w);
  else
    tmem_st32x16(to, w);
}

template <int D, int RT, bool BF, bool LO>
__global__ void __launch_bounds__(TreeCfg<D, RT>::THREADS, 1)
    decode_tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TreeParams p) {
  using C = TreeCfg<D, RT>;
  constexpr int kThreads = C::THREADS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  struct Misc {
    uint4 segments[kTreeSegs][2];  // b, kv, tu, x with kSegWhole and kSegBegins; tile, count, len, cnt
    union {
      long long warp_tiles[kThreads / 32];  // until the shares are known
      uint32_t infos[kTileInfos];           // then
    };
    Start start;
    uint32_t tmem_base;
    volatile uint32_t abort_flag;
  };
  constexpr uint32_t kSegWhole = 1u << 31, kSegBegins = 1u << 30;
  const uint32_t base = smem_u32(smem_raw);
  uint8_t *const base_ptr = smem_raw;
  if (base & 1023u) {  // swizzled tiles lie on 1 KB boundaries; so does dynamic shared memory (there is no other here)
    grid_wait_prior();
    if (threadIdx.x == 0) {
      atomicCAS(p.status, 0u, kTreeSmemAlign);
      p.records[blockIdx.x] = {};
    }
    return;
  }
  const uint32_t NSLOT = p.slots;
  const int NQB = p.q_buffers;
  const uint32_t q_tile = static_cast<uint32_t>(p.s.q_rows) * 128u * (D / 64), q_bytes = q_tile * RT;  // of a row tile, of a unit
  // Queries, ring, sums, page numbers, exchange, barriers.  (A product reads 128 rows of queries from each box: behind the last one, the ring.)
  const uint32_t ring = q_bytes * static_cast<uint32_t>(NQB), off_sums = ring + NSLOT * C::SLOT_BYTES;
  const uint32_t off_pages = off_sums + (LO ? static_cast<uint32_t>(C::WG * C::DV * 4 * p.s.q_rows) : 0u);
  const uint32_t off_exchange = off_pages + C::PAGE_BYTES, off_bars = off_exchange + C::EXCHANGE_BYTES;
  float *const exchange = reinterpret_cast<float *>(base_ptr + off_exchange);  // [maximum, sum][stream][row]
  // (Rounded up to 16 bytes for the segments' words.)
  constexpr uint32_t kMiscAt = (8 * C::NBAR + 15) & ~15;
  Misc &misc = *reinterpret_cast<Misc *>(base_ptr + off_bars + kMiscAt);
  static_assert(kMiscAt + sizeof(Misc) <= C::BAR_BYTES, "barrier room");
  const uint32_t info_at = smem_u32(misc.infos), segments_at = smem_u32(misc.segments);
  const uint32_t bars = base + off_bars;
  auto BAR = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kIssuer = 0, kSoftmax = 4;  // the issuer's warp, the first of softmax

  if (tid == 0) {
    for (uint32_t i = 0; i < NSLOT; ++i) {
      mbar_init(BAR(C::B_FULL + i), 1);
      mbar_init(BAR(C::B_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(C::B_QFULL + i), 1);
      mbar_init(BAR(C::B_QEMPTY + i), 1);
      mbar_init(BAR(C::B_SFULL + i), 1);
      mbar_init(BAR(C::B_PFULL + i), 4);
      mbar_init(BAR(C::B_PDONE + i), 1);
    }
    mbar_init(BAR(C::B_DRAIN), 1);
    mbar_init(BAR(C::B_MEET), 8);
    for (int i = 0; i < kTreeSegs; ++i) mbar_init(BAR(C::B_SEG + i), 1);
    misc.abort_flag = 0u;
    misc.start = {};
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kIssuer) {
    tmem_alloc(smem_u32(&misc.tmem_base), 512);
    tmem_relinquish();
    // Only now: a dependent kernel's CTA must not take the tensor memory first and then wait for this kernel's end.
    grid_launch_dependents();
  }
  grid_wait_prior();  // what follows reads the previous kernels' results

  // ------------------------------------------------------------ this CTA's share
  // Thread i counts the tiles of its run of sequences; a scan over the block gives the total
  // and finds the sequence in which this CTA's share begins.
  const int span = p.s.tokens * RT, nx = p.s.head_units * p.s.halves;
  auto head_tiles = [&](Tokens s) -> long long {  // of a key head
    const int units = (s.cnt + span - 1) / span;
    if (p.mask) return static_cast<long long>(units) * nx * tiles_of(s.len);
    long long n = 0;
    for (int tu = 0; tu < units; ++tu) n += unit_tiles(p, s, tu, span);
    return n * nx;
  };
  const int per = (p.B + kThreads - 1) / kThreads;
  const int s0 = static_cast<int>(min(static_cast<long long>(p.B), static_cast<long long>(tid) * per)), s1 = min(p.B, s0 + per);
  long long mine = 0;
  Tokens at_s0 = {0, 0};
  for (int b = s0; b < s1; ++b) {
    const Tokens s = tokens_of(p, b, blockIdx.x == 0);
    if (b == s0) at_s0 = s;
    mine += head_tiles(s) * p.Hkv;
  }
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) misc.warp_tiles[warp] = upto;
  __syncthreads();
  long long total = 0;
#pragma unroll 1
  for (int w = 0; w < min(kThreads, p.B + 31) / 32; ++w) {  // the others have no sequences
    if (w < warp) upto += misc.warp_tiles[w];
    total += misc.warp_tiles[w];
  }
  // The first G CTAs have a tile at least, the others none: a unit's parts lie in CTAs next to one another.
  const long long G = min(static_cast<long long>(gridDim.x), max(total, 1LL)), cta = min(static_cast<long long>(blockIdx.x), G);
  const long long u0 = quotient(total * cta, G), u1 = quotient(total * min(cta + 1, G), G);
  if (u0 < u1 && upto - mine <= u0 && u0 < upto) {
    long long off = u0 - (upto - mine);
    for (int b = s0; b < s1; ++b) {
      const Tokens s = b == s0 ? at_s0 : tokens_of(p, b);
      const long long head = head_tiles(s);
      if (off >= head * p.Hkv) {
        off -= head * p.Hkv;
        continue;
      }
      const int kv = static_cast<int>(quotient(off, head));
      off -= kv * head;
      int tu = 0, tiles = unit_tiles(p, s, 0, span);
      if (p.mask) {
        tu = static_cast<int>(quotient(off, static_cast<long long>(tiles) * nx));
        off -= static_cast<long long>(tu) * tiles * nx;
      } else {
        while (off >= static_cast<long long>(tiles) * nx) {
          off -= static_cast<long long>(tiles) * nx;
          tiles = unit_tiles(p, s, ++tu, span);
        }
      }
      const int x = static_cast<int>(quotient(off, tiles));
      misc.start = {b, kv, tu, x, static_cast<int>(off - static_cast<long long>(x) * tiles), s, u1 - u0};
      break;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc.tmem_base;
  const uint32_t tiles = static_cast<uint32_t>(u1 - u0);
  const Start start = misc.start;
  bool ok = true;

  if (warp < kSoftmax) {
    if (warp > kIssuer) {
      // ---------------------------------------------------------- producers: one of keys, one of values, one of queries
      const int which = warp - kIssuer - 1;
      uint32_t filled = 0, laps = 0;  // bits of the ring slots that this producer filled, and their phases
      if (which < 2) {
        const bool keys = which == 0;
        // A lane copies its box of a slot; lane 0 waits for the slot and announces the bytes.
        const int rows = p.box_rows, shift = 31 - __clz(rows), lanes = (kTreeTile >> shift) * C::NBOX;
        const int row = (lane / C::NBOX) * rows, box = lane % C::NBOX;
        const bool deals = lane < lanes;
        const CUtensorMap *const tm = keys ? &tm_k : &tm_v;
        uint32_t slot = 0, lap = 0;  // the ring slot next in turn, and its phase
        auto step = [&](uint32_t n) {
          slot += n;
          while (slot >= NSLOT) {
            slot -= NSLOT;
            lap ^= 1u;
          }
        };
        if (!keys) step(RT == 2 ? C::NC : min(2u, tiles) * C::NC);
        // Page numbers come through shared memory, asynchronously, kAhead tiles ahead: a producer that
        // waited for each in a register would run at the table's latency.
        const uint32_t mine_p = base + off_pages + (which * kAhead * 16 + lane / C::NBOX) * 4;
        Cursor pre(p, start, row), it(p, start, row);
        uint32_t stage = 0, taken = 0;  // the next page number asked for, and taken
        auto prefetch = [&]() {
          if (deals && pre.next() && row < pre.keys) cp_async_4(mine_p + stage * 64, p.table + pre.s.b * p.table_s + pre.index);
          cp_async_commit();
          stage = stage + 1 == kAhead ? 0 : stage + 1;
        };
        prefetch();  // the first tile's; the others once that one is under way
        for (uint32_t t = 0; t < tiles && it.next(); ++t) {
          const bool deal = deals && row < it.keys;
          int page = 0;
          if (t == 0)
            cp_async_wait<0>();
          else
            cp_async_wait<kAhead - 1>();
          if (deal) {
            page = static_cast<int>(ld_shared_u32(mine_p + taken * 64));
            if (page < 0 || page >= p.pages) atomicCAS(p.status, 0u, kDevBadPage);  // TMA reads zeros there
          }
          taken = taken + 1 == kAhead ? 0 : taken + 1;
          const uint32_t bytes = static_cast<uint32_t>(((it.keys + rows - 1) >> shift) * rows) * 128u * C::NBOX;
          const int column = keys || p.s.halves == 1 ? 0 : (it.s.x & 1) * C::DV;  // the first
          // What the issuer needs to know of the tile.
          const int j = it.i - 1, turn = C::WG == 2 && RT == 1 ? j >> 1 : j;  // turn: of the accumulator
          const int ahead = C::WG == 2 && RT == 1 ? 2 : 1;
          const uint32_t info =
              static_cast<uint32_t>((it.keys + 15) >> 4) | (j == 0 ? kTileFirst : 0u) | (j + 1 == it.s.count ? kTileLast : 0u) |
              ((turn & (p.fold - 1)) == 0 ? kTileFresh : 0u) | (j + ahead >= it.s.count ? kTileDone : 0u) |
              (NQB == 1 ? static_cast<uint32_t>(it.seg & 1) << kTileTurn : static_cast<uint32_t>(it.seg & 1) << kTileBuffer | static_cast<uint32_t>(it.seg >> 1 & 1) << kTileTurn);
          const int n = keys ? C::NC : C::NV;
          for (int c = 0; c < n; ++c) {
            // The first lap passes at once: the phase before a barrier's first counts as complete.  A later one's is never
            // two behind: the slot's load before was behind this producer's own last one but NSLOT, and that is consumed
            // (NSLOT > NC).  Lane 0 waits for all: a lane that tested the barrier by itself could come so late that the slot
            // had been filled and freed once more, and its parity would not come round again.
            if (lane == 0)
              ok = wait_bounded(BAR(C::B_EMPTY + slot), lap ^ 1u, &misc.abort_flag, p.status, kDevTimeoutLoad, p.wait_limit);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            filled |= 1u << slot;
            laps = (laps & ~(1u << slot)) | lap << slot;
            if (lane == 0) {
              if (keys && c == 0) st_shared_u32(info_at + (t % kTileInfos) * 4, info);
              mbar_arrive_expect_tx(BAR(C::B_FULL + slot), bytes);
            }
            if (deal)
              tma_load_4d(base + ring + slot * C::SLOT_BYTES + box * C::BOX_BYTES + row * 128, tm, column + c * C::CW + box * 64, it.slot, it.s.kv, page,
                          BAR(C::B_FULL + slot));
            step(1);
          }
          if (!ok) break;
          if (keys)
            step(RT == 1 && t == 0 ? 0 : C::NV);
          else
            step(RT == 2 || t + 3 <= tiles ? C::NC : 0);
#pragma unroll 1
          for (int i = t == 0 ? 0 : kAhead - 1; i < kAhead; ++i) prefetch();
        }
        cp_async_wait<0>();
      } else if (lane == 0) {
        // A unit's queries, and for the softmax what there is to know of the segment.
        TreeRecord record = {};
        Walk w(p, start);
        Seg q;
        int s = 0, held[2] = {0, 0};  // tiles of the segments whose queries are in the buffers
        for (; ok && w.next(q); ++s) {
          const int buf = NQB == 1 ? 0 : s & 1, turn = NQB == 1 ? s : s >> 1;
          // This wait may last for a whole segment, so that it gets a limit for each of its tiles (the others' waits, of a tile at
          // most, run out first where something is wrong, and end this one too).
          if (turn > 0)
            ok = wait_bounded(BAR(C::B_QEMPTY + buf), (turn - 1) & 1, &misc.abort_flag, p.status, kDevTimeoutLoad, p.wait_limit * (buf ? held[1] : held[0]));
          if (!ok) break;
          if (buf) held[1] = q.count; else held[0] = q.count;
          // The words of the segment kTreeSegs before are past: the QK of the segment NQB before is done, so the PVs of all tiles but
          // its last two are, and both warpgroups have come to those.
          const bool whole = q.count == q.tiles, begins = q.tile == 0;
          const uint32_t words = segments_at + (s % kTreeSegs) * 32;
          st_shared_v4(words, q.b, q.kv, q.tu, q.x | (whole ? kSegWhole : 0u) | (begins ? kSegBegins : 0u));
          st_shared_v4(words + 16, q.tile, q.count, q.s.len, q.s.cnt);
          mbar_arrive(BAR(C::B_SEG + s % kTreeSegs));
          const uint32_t bar = BAR(C::B_QFULL + buf), dst = base + buf * q_bytes;
          mbar_arrive_expect_tx(bar, static_cast<uint32_t>(p.s.heads * p.s.tokens) * 128u * (D / 64) * RT);
          const int head = q.kv * p.G + (p.s.halves == 1 ? q.x : q.x >> 1) * p.s.heads;
#pragma unroll 1
          for (int x = 0; x < RT * (D / 64); ++x) {
            const int tile = RT == 1 ? 0 : x / (D / 64), column = x % (D / 64);
            tma_load_4d(dst + tile * q_tile + column * static_cast<uint32_t>(p.s.q_rows) * 128u, &tm_q, column * 64, (q.tu * RT + tile) * p.s.tokens, head, q.b, bar);
          }
          if (!whole && begins) {
            // The unit goes on in the next CTAs: up to the one whose share holds its last tile `end`, the
            // largest c with floor(total c / G) <= end, that is c < (end + 1) G / total.
            const long long end = u1 + (q.tiles - q.count) - 1;
            record = {q.b, q.kv, q.tu, q.x, q.s.cnt, static_cast<int>(quotient((end + 1) * G - 1, total)) - static_cast<int>(blockIdx.x) + 1, {0, 0}};
          }
        }
        p.records[blockIdx.x] = record;
        if (misc.abort_flag)
          for (int i = max(0, s - NQB); i < s; ++i)
            wait_drain(BAR(C::B_QFULL + (NQB == 1 ? 0 : i & 1)), (NQB == 1 ? i : i >> 1) & 1, p.wait_limit >> 10);
      }
      // After a time-out: copies that nobody waited for land before the CTA ends (a slot that was filled again never comes
      // round, and gets some milliseconds).
      if (lane == 0 && misc.abort_flag)
        for (uint32_t x = 0; x < NSLOT; ++x)
          if (filled >> x & 1u) wait_drain(BAR(C::B_FULL + x), laps >> x & 1u, p.wait_limit >> 10);
      __syncwarp();
    } else {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t idesc_s = BF ? idesc_bf16_f32(128, 128, 0, 0) : idesc_f16_f32(128, 128, 0, 0);
      const uint32_t idesc_o = BF ? idesc_bf16_f32(128, C::CW, 0, 1) : idesc_f16_f32(128, C::CW, 0, 1);
      const SDesc dq = sdesc_split(sdesc_sw128(base, 16, 1024)), dk = sdesc_split(sdesc_sw128(base + ring, 16, 1024));
      const SDesc dv = sdesc_split(sdesc_sw128(base + ring, C::BOX_BYTES, 1024));
      const uint32_t q_box = static_cast<uint32_t>(p.s.q_rows) * 128u;
      // The whole warp walks and waits, one lane of it issues: in code that a single lane runs every operand of a
      // product costs a move of its own to the warp's registers (about 120 cycles a product instead of 64).
      {
        const bool one = elect_one();
        bool got = true;
        auto wait = [&](int bar, uint32_t phase) {
          got = __all_sync(0xffffffffu, wait_bounded(BAR(bar), phase & 1u, &misc.abort_flag, p.status, kDevTimeoutMma, p.wait_limit)) && got;
        };
        auto commit = [&](int bar) {
          if (one) umma_commit(BAR(bar));
        };
        struct Pos {  // the ring slot next in turn, and its phase
          uint32_t slot = 0, lap = 0;
        };
        Pos at, at_v;  // two row tiles: of K and of V, apart
        auto step = [&](Pos &a, int n) {
          a.slot += n;
          if (a.slot >= NSLOT) {
            a.slot -= NSLOT;
            a.lap ^= 1u;
          }
        };
        if (RT == 2) step(at_v, C::NC);
        // S of stream s of the tile that `i` tells of; frees K's slots after the last stream's.  (The first slot is full.)
        auto qk = [&](int s, uint32_t i, bool free) {
          const uint32_t buf = i >> kTileBuffer & 1u;
          if ((i & kTileFirst) && (RT == 1 || s == 0)) wait(C::B_QFULL + buf, i >> kTileTurn);
          Pos a = at;
          SDesc q = {dq.lo + ((buf * q_bytes + (RT == 2 ? s * q_tile : 0)) >> 4), dq.hi};
          for (int c = 0; c < C::NC; ++c, step(a, 1)) {
            if (c > 0) wait(C::B_FULL + a.slot, a.lap);
            if (got) {
              tc_fence_after();
              SDesc k = {dk.lo + a.slot * (C::SLOT_BYTES >> 4), dk.hi};
              if (one)
#pragma unroll
                for (int box = 0; box < C::NBOX; ++box, q.lo += q_box >> 4)
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk) umma_ss_off(tmem + s * 128, q, kk * 32, k, box * C::BOX_BYTES + kk * 32, idesc_s, (c | box | kk) != 0);
              if (free) commit(C::B_EMPTY + a.slot);
            }
          }
          if (free) {
            if (RT == 1) at = a; else step(at, C::NC + C::NV);
          }
          if (got) {
            if (!C::ONE || !free) commit(C::B_SFULL + s);
            if (free && (i & kTileLast)) commit(C::B_QEMPTY + buf);
          }
        };
        auto pv = [&](int s, uint32_t i, bool free, bool ready) {
          Pos a = RT == 1 ? at : at_v;
          const uint32_t o = tmem + C::T_O + (C::WG == 2 ? s * C::DV : 0), w = tmem + s * 128;
          const int groups = i & kTileGroups;
          const uint32_t go_on = i & kTileFresh ? 0u : 1u;  // O adds to what is there
          for (int c = 0; c < C::NV; ++c, step(a, 1)) {
            if (!ready || c > 0) wait(C::B_FULL + a.slot, a.lap);
            if (got) {
              tc_fence_after();
              const SDesc v = {dv.lo + a.slot * (C::SLOT_BYTES >> 4), dv.hi};
              auto group = [&](int kk) {  // hi, then lo, 16 columns on
                const uint32_t part = w + (kk >> 1) * 32 + (kk & 1) * 8;
                umma_ts_off(o + c * C::CW, part, v, kk * 2048, idesc_o, kk > 0 ? 1u : go_on);
                if (LO) umma_ts_off(o + c * C::CW, part + 16, v, kk * 2048, idesc_o, 1);
              };
              if (groups == kTreeTile / 16) {
                if (one)
#pragma unroll
                  for (int kk = 0; kk < kTreeTile / 16; ++kk) group(kk);
              } else {
#pragma unroll 1
                for (int kk = 0; kk < groups; ++kk)
                  if (one) group(kk);
              }
              if (free) commit(C::B_EMPTY + a.slot);
            }
          }
          if (free) {
            if (RT == 1) at = a; else step(at_v, C::NC + C::NV);
          }
          if (got && (C::WG == 1 || (i & kTileDone))) commit(C::B_PDONE + s);
        };
        // Step n: PV of stream n & 1, then that stream's next QK, into the S tile whose weights the PV reads.  One
        // row tile: PV of tile n, QK of tile n + 2; two: PV of tile n / 2, QK of the next.  The tensor core holds two
        // products in its queue, about 130 cycles; a look at a barrier takes that long, so the three are taken together.
        uint32_t info[2] = {0, 0};  // of the tiles in the streams' S
        const int steps = static_cast<int>(tiles) * RT;
#pragma unroll 1
        for (int n = -2; n < steps && got; ++n) {
          const int s = n & 1, next = RT == 1 ? n + 2 : (n >> 1) + 1;
          const bool free = RT == 1 || s == 1, more = next < static_cast<int>(tiles);
          Pos v = RT == 1 ? at : at_v, k = at;
          if (RT == 1 && n >= 0) step(k, C::NV);
          const bool k_there = more && mbar_test(BAR(C::B_FULL + k.slot), k.lap);
          if (n >= 0) {
            const bool v_there = mbar_test(BAR(C::B_FULL + v.slot), v.lap);
            const bool p_there = mbar_test(BAR(C::B_PFULL + s), static_cast<uint32_t>(n) >> 1 & 1u);
            const bool v_ready = __all_sync(0xffffffffu, v_there);
            if (!__all_sync(0xffffffffu, p_there)) wait(C::B_PFULL + s, static_cast<uint32_t>(n) >> 1);
            pv(s, s ? info[1] : info[0], free, v_ready);
          }
          if (more) {
            if (!__all_sync(0xffffffffu, k_there)) wait(C::B_FULL + k.slot, k.lap);
            const uint32_t i = ld_shared_u32(info_at + (next % kTileInfos) * 4);
            if (s) info[1] = i; else info[0] = i;
            qk(s, i, free);
          }
        }
        if (__any_sync(0xffffffffu, misc.abort_flag != 0)) {  // after a time-out: products in flight end before the CTA does
          commit(C::B_DRAIN);
          wait_drain(BAR(C::B_DRAIN), 0, p.wait_limit);
        }
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------- softmax, results
    const int stream = (warp - kSoftmax) >> 2, at_once = tid - 32 * kSoftmax, r = tid & 127;  // r: this thread's row of the row tile
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);  // this warp's 32 TMEM lanes
    for (long long i = blockIdx.x; i < static_cast<long long>(p.B) * p.Hq; i += gridDim.x) {  // rows behind the new tokens
      const int cnt = tokens_of(p, static_cast<int>(i / p.Hq)).cnt;
      if (cnt == p.T) continue;
      uint4 *const o = static_cast<uint4 *>(p.o) + (i * p.T + cnt) * (D / 8);
      for (long long e = at_once; e < static_cast<long long>(p.T - cnt) * (D / 8); e += C::SOFTMAX) o[e] = make_uint4(0u, 0u, 0u, 0u);
      for (int t = cnt + at_once; t < p.T; t += C::SOFTMAX) p.lse[i * p.T + t] = -INFINITY;
    }
    auto wait = [&](int bar, uint32_t phase) {
      ok = __all_sync(0xffffffffu, wait_bounded(BAR(bar), phase & 1u, &misc.abort_flag, p.status, kDevTimeoutSoftmax, p.wait_limit)) && ok;
    };
    // The two warpgroups meet twice a segment, on one barrier (bounded waits, as all others); who has come waits before
    // it comes again.
    uint32_t meetings = 0;
    bool owed = false;  // the last meeting was not waited for
    auto come = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::B_MEET));
    };
    auto met = [&]() { wait(C::B_MEET, meetings++); };
    const int row_tile = RT == 2 ? stream : 0;
    const int heads_row = r / p.s.tokens, token_row = r - heads_row * p.s.tokens;
    // Of this stream, this row: four columns of all rows lie side by side, so that a warp's stores fill whole lines.  Those of up to 32
    // rows are in shared memory: a look at the workspace waits behind the ring's loads for 2 to 3 us.
    const int sums_step = LO ? p.s.q_rows : p.s.rows;
    float4 *const sums = (LO ? reinterpret_cast<float4 *>(base_ptr + off_sums) + stream * (C::DV / 4) * sums_step
                             : reinterpret_cast<float4 *>(p.sums) + (static_cast<long long>(blockIdx.x) * C::WG + stream) * (C::DV / 4) * sums_step) + r;
    uint32_t steps = 0, ends = 0, ends_other = 0;  // S tiles of this stream, ends of segments of this and of the other one
    uint32_t g = 0;                // tiles of the share before the segment
    struct {
      int b, kv, tu, x, tile, count;
      Tokens s;
    } s;
    s.count = 0;
    for (int n_seg = 0; g < tiles; ++n_seg, g += s.count) {
      wait(C::B_SEG + n_seg % kTreeSegs, static_cast<uint32_t>(n_seg) / kTreeSegs);
      if (!ok) break;  // (after a time-out the other warps' waits end, too)
      const uint4 w0 = ld_shared_v4(segments_at + (n_seg % kTreeSegs) * 32), w1 = ld_shared_v4(segments_at + (n_seg % kTreeSegs) * 32 + 16);
      const bool whole = (w0.w & kSegWhole) != 0, begins = (w0.w & kSegBegins) != 0;
      s = {static_cast<int>(w0.x), static_cast<int>(w0.y), static_cast<int>(w0.z), static_cast<int>(w0.w & ~(kSegWhole | kSegBegins)),
           static_cast<int>(w1.x), static_cast<int>(w1.y), {static_cast<int>(w1.z), static_cast<int>(w1.w)}};
      const int half = p.s.halves == 1 ? 0 : s.x & 1, hu = p.s.halves == 1 ? s.x : s.x >> 1;
      const int head = hu * p.s.heads + heads_row, t = (s.tu * RT + row_tile) * p.s.tokens + token_row;
      const bool valid = heads_row < p.s.heads && head < p.G && t < s.s.cnt;
      const bool any = __any_sync(0xffffffffu, valid);  // a warp without rows passes the barriers only
      const int old = s.s.len - s.s.cnt;
      const unsigned *const bits = p.mask + s.b * p.mask_sb + min(t, p.T - 1) * p.mask_sl;  // (not read without a mask)
      float m = -INFINITY, l = 0.f, m_sums = -INFINITY, l_sums = 0.f;
      bool folded = false;
      const int j0 = C::WG == 2 && RT == 1 ? static_cast<int>((stream ^ g) & 1u) : 0, dj = C::WG == 2 && RT == 1 ? 2 : 1;
      const uint32_t o_at = lanes + C::T_O + (C::WG == 2 ? stream * C::DV : 0);
      for (int j = j0; j < s.count; j += dj, ++steps) {
        // After a time-out the remaining tiles run through the barriers only.
        const int buf = C::WG == 2 ? stream : static_cast<int>(steps & 1u);
        const uint32_t phase = C::WG == 2 ? steps : steps >> 1;
        const int k0 = (s.tile + j) * kTreeTile, n = s.s.len - k0;  // n: keys from the tile's first on
        const uint32_t s_at = lanes + buf * 128;
        const int turn = C::WG == 2 && RT == 1 ? j >> 1 : j;
        // ---- which of the tile's keys this row sees
        // (without a mask: any that the row tile's first token does not see; the sums stay within 31 bits at any length)
        const bool edge = k0 - old + kTreeTile > (p.mask ? 0 : min((s.tu * RT + row_tile) * p.s.tokens + 1, s.s.cnt));
        uint32_t seen[4];
        if (edge && any) {
          const int a = old - k0;  // the tile's column of the first new token
          if (p.mask) {
            const int q = (-a) >> 5, sh = (-a) & 31;  // the first column is bit sh of word q
            uint32_t word[5];
#pragma unroll
            for (int i = 0; i < 5; ++i) word[i] = valid && q + i >= 0 && q + i < p.words ? bits[q + i] : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) seen[i] = (__funnelshift_r(word[i], word[i + 1], sh) | first_bits(a - 32 * i)) & first_bits(n - 32 * i);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) seen[i] = first_bits(min(a + t + 1, n) - 32 * i);
          }
        }
        if (C::ONE && (RT == 1 || stream == 1)) {
          const uint32_t at = RT == 1 ? g + static_cast<uint32_t>(j) : steps, pos = RT == 1 ? max(2 * at, 1u) - 1 : 2 * at, lap = pos / NSLOT;
          wait(C::B_EMPTY + static_cast<int>(pos - lap * NSLOT), lap);
        } else {
          wait(C::B_SFULL + buf, phase);
        }
        tc_fence_after();
        if (any) {
          // The tile's logits are read twice, in pieces of 32 and loops that stay rolled (of their own where nothing is hidden):
          // the softmax's and the issuer's code then fit the instruction caches beside each other, and the registers hold
          // a piece.  128 rows, unrolled over 128 logits: 107 us, with 300 to 470 bytes spilled; rolled 101.
          const bool fold = turn > 0 && (turn & (p.fold - 1)) == 0;
          const uint64_t c2x2 = f32x2(p.c2, p.c2);
          bool made = false;
          if constexpr (RT == 2 && D == 64) {
            // Weights by the maximum so far, of logits that are read once; seldom is it left behind, and they are made again.  2048 new
            // tokens behind 6144, 32/8 heads x 64 179 -> 165 us (both before bf16's scale, 172 with it).  Not at 128, where the issuer's turns bound the kernel (4 x 2048 new
            // tokens 503 -> 512), nor for one row tile, where more code costs what it saves (pages of 128 106 -> 96, of 16 51 -> 52).
            if (!edge && turn > 0 && !fold) {
              const float from = m == -INFINITY ? 0.f : m - kShift<BF>;
              const uint64_t negm = f32x2(-from, -from);
              uint64_t acc[4];
              uint32_t w[4][16];
              float top = -INFINITY;
#pragma unroll
              for (int k = 0; k < 4; ++k) acc[k] = f32x2(0.f, 0.f);
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                uint32_t x[16];
                tmem_ld32x16(s_at + 16 * c, x);
                pack16<BF>(x, &w[c >> 1][(c & 1) * 8], c2x2, negm, acc, top);
              }
              if (!__any_sync(0xffffffffu, valid && top * p.c2 > m + kSlack)) {
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_st32x16(s_at + 32 * c, w[c]);
                float la, lb;
                f32x2_split(fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3])), la, lb);
                l += la + lb;
                made = true;
              }
            }
          }
          if (!made) {
            float top = -INFINITY;
            if (!edge) {
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                uint32_t x[32];
                tmem_ld32x32(s_at + 32 * c, x);
                top = fmaxf(top, max32(x));
              }
            } else {
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                const uint32_t here = c < 2 ? c == 0 ? seen[0] : seen[1] : c == 2 ? seen[2] : seen[3];
                uint32_t x[32];
                tmem_ld32x32(s_at + 32 * c, x);
                hide(x, here);
                top = fmaxf(top, max32(x));
              }
            }
            top = valid ? top * p.c2 : -INFINITY;
            // ---- the running maximum, and what it does to the sum and to O.  With two streams PV of the
            // stream's tile before is complete here: it was issued before this S, by the same thread.
            if (turn == 0) {
              m = top;
            } else if (fold || __any_sync(0xffffffffu, top > m + kSlack)) {
              if constexpr (C::WG == 1) {
                wait(C::B_PDONE + (static_cast<int>(steps - 1) & 1), (steps - 1) >> 1);
                tc_fence_after();
              }
              if (fold && ok) {
                // (Two maxima of -inf: sums of nothing, whatever their factors; fminf drops their difference, a NaN.)
                const float keep = ex2_approx(fminf(m_sums - m, 0.f)), add = ex2_approx(fminf(m - m_sums, 0.f));
#pragma unroll 1
                for (int c = 0; c < C::DV; c += 32) {
                  uint32_t o[32];
                  tmem_ld32x32(o_at + c, o);
                  if (valid)
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                      float4 x = make_float4(__uint_as_float(o[e]) * add, __uint_as_float(o[e + 1]) * add, __uint_as_float(o[e + 2]) * add, __uint_as_float(o[e + 3]) * add);
                      if (folded) {
                        const float4 y = sums[(c + e) / 4 * sums_step];
                        x = make_float4(fmaf(y.x, keep, x.x), fmaf(y.y, keep, x.y), fmaf(y.z, keep, x.z), fmaf(y.w, keep, x.w));
                      }
                      sums[(c + e) / 4 * sums_step] = x;
                    }
                }
                l_sums = fmaf(l_sums, keep, l * add);  // (the weights' sum, too: in one number each tile of a row of 2^31 would be rounded to 2^-8)
                l = 0.f;
                m_sums = fmaxf(m_sums, m);
                m = top;  // the next `fold` tiles go by their own maximum
                folded = true;
              }
              const bool up = top > m + kSlack;
              const float keep = up ? ex2_approx(m - top) : 1.f;
              m = up ? top : m;
              l *= keep;
              if (!fold && ok) {
#pragma unroll 1
                for (int c = 0; c < C::DV; c += 32) {
                  uint32_t o[32];
                  tmem_ld32x32(o_at + c, o);
#pragma unroll
                  for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                  tmem_st32x32(o_at + c, o);
                }
              }
            }
            // ---- the row's weights, as hi + lo
            const float from = m == -INFINITY ? 0.f : m - kShift<BF>;
            const uint64_t negm = f32x2(-from, -from);
            uint64_t acc[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[k] = f32x2(0.f, 0.f);
            if (!edge) {
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                uint32_t x[32];
                tmem_ld32x32(s_at + 32 * c, x);
                weights32<BF, LO>(x, s_at + 32 * c, c2x2, negm, acc);
              }
            } else {
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                const uint32_t here = c < 2 ? c == 0 ? seen[0] : seen[1] : c == 2 ? seen[2] : seen[3];
                uint32_t x[32];
                tmem_ld32x32(s_at + 32 * c, x);
                hide(x, here);
                weights32<BF, LO>(x, s_at + 32 * c, c2x2, negm, acc);
              }
            }
            float la, lb;
            f32x2_split(fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3])), la, lb);
            l += la + lb;
            tmem_wait_st();
          }
        }
        if ((n & 15) != 0 && n < kTreeTile && (RT == 1 || stream == 0)) {
          // PV takes keys in groups of 16.  Whatever lies behind the last token in its group (unwritten slots,
          // earlier tiles) times a weight of zero must be zero: clear those rows of V, eight threads to a row.
          const uint32_t at = RT == 1 ? g + static_cast<uint32_t>(j) : steps;
          if constexpr (C::WG == 1) {
            // The slots' earlier loads, of V(at - 1) and K(at + 1), must be past, or a wait for V's load would take
            // the phase before theirs for it.  (Two streams: of K(at) at the latest.)
            if (at >= 1) wait(C::B_PDONE + (static_cast<int>(at - 1) & 1), (at - 1) >> 1);
            if (at + 1 < tiles) wait(C::B_SFULL + (static_cast<int>(at + 1) & 1), (at + 1) >> 1);
          }
          const uint32_t v0 = v_pos<C, RT>(at, tiles);
          for (int c = 0; c < C::NV; ++c) {
            const uint32_t lap = (v0 + c) / NSLOT, slot = v0 + c - lap * NSLOT;
            wait(C::B_FULL + static_cast<int>(slot), lap);
            const int row = n + (r >> 3);
            if (ok && row < ((n + 15) & ~15))
#pragma unroll
              for (int z = 0; z < C::NBOX; ++z)
                st_shared_v4(base + ring + slot * C::SLOT_BYTES + z * C::BOX_BYTES + row * 128 + (r & 7) * 16, 0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (C::WG == 2 && RT == 1 && owed) {  // the other warpgroup has read this stream's O of the segment before
          met();
          owed = false;
          tc_fence_after();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::B_PFULL + buf));
      }
      // ---------------------------------------------------------- the segment's results
      // What left the accumulator, and what is in it, to their common maximum.
      float back = 0.f, own = 1.f;
      if (folded) {
        back = ex2_approx(fminf(m_sums - m, 0.f));
        own = ex2_approx(fminf(m - m_sums, 0.f));
        l = fmaf(l_sums, back, l * own);
        m = fmaxf(m_sums, m);
      }
      const bool has = j0 < s.count, has_other = C::WG == 2 && RT == 1 && (j0 ^ 1) < s.count;  // whether the streams had tiles of it
      if constexpr (C::WG == 2 && RT == 1) {
        // Each row's maxima and sums change hands while the last products run.
        if (owed) met();
        owed = false;
        exchange[stream * 128 + r] = m;
        exchange[256 + stream * 128 + r] = l;
        if (!folded) come();
      }
      if (C::WG == 1) {
        wait(C::B_PDONE + (static_cast<int>(steps - 1) & 1), (steps - 1) >> 1);
      } else if (has) {
        wait(C::B_PDONE + stream, ends);
        ++ends;
      }
      tc_fence_after();
      const long long part = 2LL * blockIdx.x + (begins ? 1 : 0);
      const size_t row_out = (static_cast<size_t>(s.b) * p.Hq + s.kv * p.G + head) * p.T + t;
      if (folded) {  // what left the accumulator comes back (long rows only)
#pragma unroll 1
        for (int c = 0; c < C::DV; c += 32) {
          uint32_t o[32];
          tmem_ld32x32(o_at + c, o);
          if (valid)
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 y = sums[(c + e) / 4 * sums_step];
              o[e] = __float_as_uint(fmaf(y.x, back, __uint_as_float(o[e]) * own));
              o[e + 1] = __float_as_uint(fmaf(y.y, back, __uint_as_float(o[e + 1]) * own));
              o[e + 2] = __float_as_uint(fmaf(y.z, back, __uint_as_float(o[e + 2]) * own));
              o[e + 3] = __float_as_uint(fmaf(y.w, back, __uint_as_float(o[e + 3]) * own));
            }
          tmem_st32x32(o_at + c, o);
        }
        tc_fence_before();
        if constexpr (C::WG == 2 && RT == 1) come();  // not before: the other warpgroup reads this O
      }
      float f_own = 1.f, f_other = 0.f;
      if constexpr (C::WG == 2 && RT == 1) {
        // Join the streams: each warpgroup takes half of the columns.
        met();
        if (has_other) {
          wait(C::B_PDONE + (stream ^ 1), ends_other);
          ++ends_other;
        }
        tc_fence_after();
        const float mo = exchange[(stream ^ 1) * 128 + r], lo = exchange[256 + (stream ^ 1) * 128 + r];
        const float M = fmaxf(m, mo);
        f_own = m == -INFINITY ? 0.f : ex2_approx(m - M);
        f_other = has_other && mo != -INFINITY ? ex2_approx(mo - M) : 0.f;
        // the same order in both warpgroups
        l = stream == 0 ? fmaf(f_own, l, f_other * lo) : fmaf(f_other, lo, f_own * l);
        m = M;
      }
      if (any) {
        const float lse2 = m - kShift<BF> + __log2f(l);
        const float inv = l == 0.f ? 0.f : __fdividef(kValueBack<BF>, l);
        if (valid && ok && half == 0 && (C::WG == 1 || RT == 2 || stream == 0) && whole) p.lse[row_out] = lse2 * 0.69314718055994531f;
        if (valid && ok && (C::WG == 1 || RT == 2 || stream == 0) && !whole) p.part_lse[(part * RT + row_tile) * p.s.rows + r] = lse2;
        const int c0 = C::WG == 2 && RT == 1 ? stream * (C::DV / 2) : 0, c1 = C::WG == 2 && RT == 1 ? c0 + C::DV / 2 : C::DV;
        const uint32_t o_other = lanes + C::T_O + (stream ^ 1) * C::DV;
#pragma unroll 1
        for (int c = c0; c < c1; c += 32) {
          uint32_t o[32];
          if (has) {
            tmem_ld32x32(o_at + c, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(f_own * __uint_as_float(o[e]));
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (C::WG == 2 && RT == 1 && has_other) {
            uint32_t x[32];
            tmem_ld32x32(o_other + c, x);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(fmaf(f_other, __uint_as_float(x[e]), __uint_as_float(o[e])));
          }
          if (!valid || !ok) continue;
          if (whole) {
            uint4 *const to = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.o) + row_out * D + half * C::DV + c);
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t h[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) h[i] = pack2<BF>(__uint_as_float(o[e + 2 * i]) * inv, __uint_as_float(o[e + 2 * i + 1]) * inv);
              to[e / 8] = make_uint4(h[0], h[1], h[2], h[3]);
            }
          } else {
            float4 *const to = reinterpret_cast<float4 *>(p.part_o) + ((part * RT + row_tile) * (C::DV / 4) + c / 4) * p.s.rows + r;
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              to[e / 4 * p.s.rows] = make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv, __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
          }
        }
      }
      tc_fence_before();
      if constexpr (C::WG == 2 && RT == 1) {  // the other stream's O, and the exchange, are free again
        come();
        owed = true;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) tmem_dealloc(tmem, 512);
}

constexpr int kJoinThreads = 256, kJoinAtOnce = 8;
constexpr float kJoinScale = 0x1p-8f;  // up to kTreeMaxCtas values of the largest size add up to one within fp32
static_assert(kTreeMaxCtas * kJoinScale < 1.f, "sums of a join");

// Joins the units that were cut: block (c, y, z) takes 64 columns and 32 rows (row tiles one after the other) of the unit that CTA
// c's share ends in, a warp eight of the columns, a lane a row; the loads of kJoinAtOnce parts are under way together.
// M = max lse, o = sum 2^(lse - M) o / sum.
template <int D, int RT, bool BF>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const __grid_constant__ TreeParams p) {
  constexpr int DV = TreeCfg<D, RT>::DV;
  grid_launch_dependents();
  grid_wait_prior();
  const int cta = blockIdx.x, lane = threadIdx.x & 31;
  const TreeRecord rec = p.records[cta];
  if (rec.parts == 0) return;
  const int row = blockIdx.z * 32 + lane, row_tile = RT == 1 ? 0 : blockIdx.z * 32 / p.s.rows, r = row - row_tile * p.s.rows;
  const int half = p.s.halves == 1 ? 0 : rec.x & 1, hu = p.s.halves == 1 ? rec.x : rec.x >> 1;
  const int g = r / p.s.tokens, head = hu * p.s.heads + g, t = (rec.tu * RT + row_tile) * p.s.tokens + r - g * p.s.tokens;
  if (g >= p.s.heads || head >= p.G || t >= rec.cnt) return;
  const size_t out = (static_cast<size_t>(rec.b) * p.Hq + rec.kv * p.G + head) * p.T + t;
  const int c = blockIdx.y * 64 + (threadIdx.x >> 5) * 8;
  float M = -INFINITY, sum = 0.f, o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = 0.f;
  for (int first = 0; first < rec.parts; first += kJoinAtOnce) {
    float lse[kJoinAtOnce];
    float4 x[kJoinAtOnce][2];
#pragma unroll
    for (int u = 0; u < kJoinAtOnce; ++u) {
      const int i = min(first + u, rec.parts - 1);
      const long long part = (i == 0 ? 2LL * cta + 1 : 2LL * (cta + i)) * RT + row_tile;
      const float4 *const from = reinterpret_cast<const float4 *>(p.part_o) + (part * (DV / 4) + c / 4) * p.s.rows + r;
      lse[u] = p.part_lse[part * p.s.rows + r];
      x[u][0] = from[0];
      x[u][1] = from[p.s.rows];
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < kJoinAtOnce; ++u) {
      if (first + u >= rec.parts) lse[u] = -INFINITY;
      top = fmaxf(top, lse[u]);
    }
    const float from = top == -INFINITY ? 0.f : top, keep = ex2_approx(M - from);
    M = top;
    sum *= keep;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= keep;
#pragma unroll
    for (int u = 0; u < kJoinAtOnce; ++u) {
      const float w = ex2_approx(lse[u] - from);
      sum += w;
      if (first + u < rec.parts) {
        const float v[8] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w, x[u][1].x, x[u][1].y, x[u][1].z, x[u][1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(w * kJoinScale, v[e], o[e]);
      }
    }
  }
  if (c == 0 && half == 0) p.lse[out] = (M + __log2f(sum)) * 0.69314718055994531f;
  const float inv = sum == 0.f ? 0.f : 1.f / (sum * kJoinScale);
  uint32_t h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = pack2<BF>(o[2 * e] * inv, o[2 * e + 1] * inv);
  *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.o) + out * D + half * DV + c) = make_uint4(h[0], h[1], h[2], h[3]);
}

template <int D, int RT, bool BF, bool LO>
cudaError_t launch_tree_as(const TreeLaunch &a) {
  using C = TreeCfg<D, RT>;
  auto *kern = decode_tree_kernel<D, RT, BF, LO>;
  static std::atomic<unsigned long long> configured{0};  // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(configured >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_MOST);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured |= 1ull << dev;
  }
  TreeParams p = a.p;
  // Queries of two units where the ring keeps five slots of 32 KB beside them and the sums.
  const int q_bytes = p.s.q_rows * 2 * D * RT, sums_bytes = LO ? C::WG * C::DV * 4 * p.s.q_rows : 0, room = C::ROOM - sums_bytes;
  p.q_buffers = (room - 2 * q_bytes) / C::SLOT_BYTES >= (D == 64 ? 10 : 5) ? 2 : 1;
  p.slots = std::min(C::MAX_SLOTS, (room - p.q_buffers * q_bytes) / C::SLOT_BYTES);
  const int smem = p.q_buffers * q_bytes + p.slots * C::SLOT_BYTES + sums_bytes + C::PAGE_BYTES + C::EXCHANGE_BYTES + C::BAR_BYTES;
  // At most one CTA per tile that the tables have room for (and lengths, of 31 bits, can name).
  const long long row_tiles =
      std::min((static_cast<long long>(p.table_w) * p.page + kTreeTile - 1) / kTreeTile, (1LL << 31) / kTreeTile);
  const long long units = static_cast<long long>(p.B) * p.Hkv * p.s.token_units * p.s.head_units * p.s.halves;
  const unsigned grid = static_cast<unsigned>(std::min<long long>(units > kTreeMaxCtas ? units : units * row_tiles, std::min(a.sm_count, kTreeMaxCtas)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, a.tm_q, a.tm_k, a.tm_v, p);
  if (e != cudaSuccess || row_tiles == 1) return e;  // a unit of one tile is never cut
  cfg.gridDim = dim3(grid, C::DV / 64, static_cast<unsigned>(RT * p.s.rows / 32));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, tree_join_kernel<D, RT, BF>, p);
}

template <int D, int RT>
cudaError_t launch_tree(const TreeLaunch &a) {
  if constexpr (RT == 1)
    if (tree_split_weights(a.p.G, a.p.T)) return a.p.bf16 ? launch_tree_as<D, 1, true, true>(a) : launch_tree_as<D, 1, false, true>(a);
  return a.p.bf16 ? launch_tree_as<D, RT, true, false>(a) : launch_tree_as<D, RT, false, false>(a);
}

}  // namespace
}  // namespace gbattn
