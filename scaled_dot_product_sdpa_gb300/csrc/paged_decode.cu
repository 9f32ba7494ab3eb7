// paged_decode.cu -- decoding over a paged cache (see paged_decode.cuh).
//
// Bound by the HBM reads of K and V: a key head's rows are used by G query heads, 2 G FLOPs per
// byte, more than the CUDA cores can do at HBM speed from G = 4 on.  So both products run on
// the tensor cores, in the orientation that makes the keys the 128-row operand:
//     S^T [128 keys x N heads]  = K [128 x d] Q^T           (K as TMA wrote it, K-major)
//     O^T [128 columns x 2N]   += V^T [128 x 128 keys] P^T  (V as TMA wrote it, MN-major)
// No byte of K or V passes through a register, and a softmax thread owns one key with all its
// heads.  The weights P enter the second product as two 16-bit parts, P = hi + lo, in separate
// columns (N heads are padded to 8 while a product of 128 rows has at least 16 columns, so with
// up to 8 heads the second part is free); that keeps 16 bits (bf16) or 22 (fp16) of a weight,
// and they are scaled by 2^13 so that fp16 keeps those of a long tail (2^-38 of the largest).  Sums over many tiles leave
// the tensor cores' accumulators every few tiles (kFold).
//
// Work: the (sequence, key head, block of query heads, 128-key tile) units in that order, cut
// into equal shares, one per persistent CTA, whatever the sequences' lengths.  A share's first
// and last rows may be parts of longer ones: those partial results go to the workspace, and
// paged_merge_kernel joins them in a fixed order (M = max lse, o = sum 2^(lse - M) o / sum).
//
// A CTA is eight warps: four of softmax (warp w reads TMEM lanes 32 w ..: keys, or columns of O),
// an MMA issuer (one thread) and three TMA producers.  K and V tiles pass through one ring of
// slots (128 keys x 64 or 128 columns) in the order K0 K1 V0 K2 V1 ...; QK runs a tile ahead of PV,
// and a row's results are taken after the next row's first tile.  Pages of fewer than 128 slots
// make several TMA boxes per slot; a producer issues one in about 53 cycles, so the boxes are dealt
// over three of them (one: pages of 8 tokens 645 us, of 16 454, of 128 302; three: 305, 301, 298).
//
// Measured on GB300 (64 sequences x 8 key heads x 8000 tokens, d = 128, bf16; 2.1 GB): 294 to 303 us for
// pages of 8 to 128 tokens and up to 8 query heads to a key head, 7.0 TB/s (103% of the copy
// bandwidth: a read-only stream); 16 query heads 307 to 315.  The same bytes at d = 64 310 to 317 (16
// heads 382: softmax and both products of 16 columns take longer than a tile of 64 columns does
// to arrive), d = 256 298 to 308, d = 512 317 to 320.  More heads to a key head: 17 to 32 of 128 take 482 to 541,
// 32 of 64 934, of 256 449 (a tile's softmax of 32 columns); blocks beyond 32 heads (16 at d = 512) read the cache again: 64 heads
// 1052 (d = 512: 1235), 128 2072 (2431).  One sequence of 1000 tokens: 9.2 us, the chain of launch, lengths, table, load, two products
// and the join.  No instance spills but 16 heads at d = 64 (68 bytes, two CTAs of 128 registers a thread).
#include <atomic>

#include "paged_decode.cuh"
#include "attn_fwd_kernel.cuh"
#include "ptx_paged.cuh"
#include "rope.cuh"
#include "vec16.cuh"

namespace gbattn {
namespace {

constexpr int kProducers = 3;  // producer warps
constexpr int kAhead = 4;      // tiles whose page numbers a producer reads ahead
constexpr int kThreads = 160 + 32 * kProducers;
constexpr float kShift = 13.f;  // weights are kept times 2^13
constexpr float kSlack = 2.f;   // the running maximum moves when a logit exceeds it by 2^2
// The tensor cores add to an fp32 accumulator by cutting off what falls below its last bit, so that a sum over n products
// of 16 keys comes out too small by about n 2^-24 (512 tiles of values of 1 in fp16: 3837 x 2^-24).  So O is begun anew
// every kFold tiles, and whenever the running maximum moves; what the tiles before add up to is kept, rounded to nearest
// and scaled to the maximum, in columns of its own.  With 8 that error stays at 2^-18 however long a row is.  GB300, 64 x 8
// key heads x 8000 keys x 128, and the same bytes at d = 64: with up to 8 query heads all choices 311 us and 322; 16 heads
// at d = 64: every 4 tiles 398, 8 386, 16 379, never 377; 32 heads at 128: 576, 541, 530, 527.
constexpr int kFold = 8;

template <int D, int NH>
struct PagedCfg {
  static constexpr int RES = paged_resident(D, NH);      // CTAs on an SM
  static constexpr int CW = D == 64 || RES == 2 ? 64 : 128;  // columns of a ring slot
  static constexpr int NC = D / CW;                     // slots of a K or V tile
  static constexpr int NBOX = CW / 64;                  // 64-column boxes of a slot
  static constexpr int BOX_BYTES = kPagedTile * 128;
  static constexpr int SLOT_BYTES = NBOX * BOX_BYTES;
  static constexpr int VS = D >= 128 && CW == 64 ? 2 : 1;  // slots of a PV product (128 columns of V)
  static constexpr int NQ = NH < 16 ? 16 : NH;          // rows of the Q operand (a product of 128 rows has N % 16 = 0)
  static constexpr int Q_BYTES = NH * D * 2;            // the operand's rows from NH on are whatever follows: their columns of S are not read
  static constexpr int NP = 2 * NH;                     // columns of P^T: hi parts, then lo parts
  static constexpr int P_BYTES = NP * kPagedTile * 2;
  static constexpr int NQB = NH == 8 && D <= 128 && RES == 1 ? 4 : NH == 32 && D == 256 ? 1 : 2;  // query buffers: segments looked ahead
  // floats: warps' maxima of two tiles, their sums of two segments, the maxima of two segments
  static constexpr int RED_SUMS = 8 * NH, RED_TOPS = 16 * NH, RED_BYTES = 18 * NH * 4;
  static constexpr int PAGE_BYTES = kProducers * kAhead * 32 * 4;  // page numbers read ahead, per producer lane
  static constexpr int BAR_BYTES = 512;                 // barriers and a few words
  static constexpr int SMEM_MOST = RES == 2 ? 115712 : 232448;  // 228 KB an SM, 1 KB a CTA kept by the system
  static constexpr int ROOM = SMEM_MOST - 1024 - NQB * Q_BYTES - 2 * P_BYTES - RED_BYTES - PAGE_BYTES - BAR_BYTES;
  static constexpr int FIT = ROOM / SLOT_BYTES, MOST = 196608 / SLOT_BYTES;
  static constexpr int NSLOT = (FIT < MOST ? FIT : MOST) / VS * VS;  // a PV product's slots lie side by side
  // With one slot a tile, the commit that frees K's slot also tells that S is there, and the one that
  // frees V's that PV is done (a commit costs its thread about 190 cycles); nothing else is
  // committed to that slot before the softmax has looked, as the ring holds more than four tiles' slots.
  static constexpr bool ONE = NC == 1;
  static_assert(!ONE || NSLOT >= 5, "slots that the softmax waits on");
  static_assert(NC % VS == 0, "PV products of whole slots");
  static_assert(NSLOT > NC, "a tile's V slots are resident together while the next K slots pass");
  static constexpr int OFF_Q = NSLOT * SLOT_BYTES;
  static constexpr int OFF_P = OFF_Q + NQB * Q_BYTES;
  static constexpr int OFF_RED = OFF_P + 2 * P_BYTES;
  static constexpr int OFF_PAGES = OFF_RED + RED_BYTES;
  static constexpr int OFF_BAR = OFF_PAGES + PAGE_BYTES;
  // barriers
  static constexpr int B_FULL = 0, B_EMPTY = NSLOT, B_QFULL = 2 * NSLOT, B_QEMPTY = B_QFULL + NQB, B_SFULL = B_QEMPTY + NQB,
                       B_PFULL = B_SFULL + 2, B_PDONE = B_PFULL + 2, B_DRAIN = B_PDONE + 2, NBAR = B_DRAIN + 1;
  static constexpr int SMEM_BYTES = 1024 + OFF_BAR + BAR_BYTES;
  static_assert(SMEM_BYTES <= SMEM_MOST, "shared memory budget");
  static constexpr int NO = D <= 128 ? 1 : D / 128;     // 128-column blocks of O
  static constexpr int T_O = 2 * NQ;                    // TMEM columns: S twice, then O twice
  static constexpr int T_SUM = T_O + 2 * NO * NP;        // O of two segments, then the sums of the tiles before O was last begun
  static constexpr int T_USED = T_SUM + NO * NH;
  static constexpr int T_COLS = T_USED <= 64 ? 64 : T_USED <= 128 ? 128 : T_USED <= 256 ? 256 : 512;
  static_assert(T_USED <= 512, "tensor memory");
};

// P^T is the B operand, MN-major: a row per key of 2 NH values (hi parts, then lo parts), 32, 64
// or 128 bytes long, swizzled over that span (16-byte chunk index ^= (address >> 7) & 1, 3, 7),
// so that a softmax thread stores its key's weights as whole vectors without bank conflicts.
template <int NH>
__device__ __forceinline__ uint64_t p_desc(uint32_t addr) {
  const uint64_t d = sdesc_sw128(addr, 16, 8 * 4 * NH);  // 8 keys to the next group along K
  constexpr uint64_t mode = NH == 8 ? 6 : NH == 16 ? 4 : 2;  // 32-, 64-, 128-byte swizzle
  return (d & ~(7ull << 61)) | (mode << 61);
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t a, uint32_t (&r)[N]) {
  if constexpr (N == 8) tmem_ld32x8(a, r);
  else if constexpr (N == 16) tmem_ld32x16(a, r);
  else if constexpr (N == 32) tmem_ld32x32(a, r);
  else tmem_ld32x64(a, r);
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t a, const uint32_t (&r)[N]) {
  if constexpr (N == 8) tmem_st32x8(a, r);
  else if constexpr (N == 16) tmem_st32x16(a, r);
  else if constexpr (N == 32) tmem_st32x32(a, r);
  else tmem_st32x64(a, r);
}

// Two weights as packed hi parts and packed lo parts, hi + lo = w up to the second rounding.
template <bool BF>
__device__ __forceinline__ void split_weights(float a, float b, uint32_t &hi, uint32_t &lo) {
  hi = pack2<BF>(a, b);
  float x, y;
  if constexpr (BF) {
    x = __uint_as_float(hi << 16);
    y = __uint_as_float(hi & 0xffff0000u);
  } else {
    const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    x = t.x;
    y = t.y;
  }
  lo = pack2<BF>(a - x, b - y);
}

// out[h] = the sum of l[h] over the warp: lanes halve the heads that they hold as they exchange.
template <int NH>
__device__ __forceinline__ void warp_sums(const float (&l)[NH], float *out) {
  const int lane = threadIdx.x & 31;
  float v[NH];
#pragma unroll
  for (int h = 0; h < NH; ++h) v[h] = l[h];
  int off = 16;
#pragma unroll
  for (int n = NH / 2; n >= 1; n >>= 1, off >>= 1) {
    const bool up = (lane & off) != 0;
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const float give = up ? v[k] : v[k + n], keep = up ? v[k + n] : v[k];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, give, off);
    }
  }
#pragma unroll
  for (; off >= 1; off >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
  constexpr int per = 32 / NH;  // lanes that hold the same head
  if ((lane & (per - 1)) == 0) out[lane / per] = v[0];
}

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Tokens of sequence b, a bad length clamped into [0, table's end].
__device__ __forceinline__ int clamp_length(int n, const PagedParams &p) {
  const long long most = static_cast<long long>(p.table_w) * p.page;
  return n < 0 ? 0 : n > most ? static_cast<int>(most) : n;
}
__device__ __forceinline__ int tiles_of(int n) { return (n >> 7) + ((n & 127) != 0); }

// A run of one key head's (and block of query heads') tiles within a CTA's share.
struct Seg {
  int b, hv, len, tile, count, tiles;  // tiles: of the whole row
};

// A CTA's share: its first unit's sequence (and that one's length), key head and tile, and its units.
struct Start {
  int b, len, hv, tile;
  long long units;
};

// Walks over a CTA's share.  By a warp, whose lanes hold 32 lengths at a time, or by one thread,
// which has the next sequence's length on the way.
template <bool WARP>
struct Walk {
  int b, hv = 0, tile = 0, hvs, len = 0, ahead = 0, base;
  long long left;
  const PagedParams &p;
  __device__ Walk(const PagedParams &pp, const Start &at) : p(pp) {
    hvs = pp.Hkv * pp.blocks;
    b = base = at.b;
    left = at.units;
    hv = at.hv;
    tile = at.tile;
    if (left <= 0) return;
    if constexpr (WARP) {
      fetch();
    } else {
      len = at.len;
      ahead = load(b + 1);
    }
  }
  __device__ int load(int i) const { return i < p.B ? clamp_length(p.lengths[i], p) : 0; }
  __device__ void fetch() {
    base = b;
    len = load(b + static_cast<int>(threadIdx.x & 31));
  }
  __device__ int length() const {
    if constexpr (WARP) return __shfl_sync(0xffffffffu, len, b - base);
    return len;
  }
  __device__ void advance() {  // to sequence b + 1
    ++b;
    if constexpr (WARP) {
      if (b - base == 32 && b < p.B) fetch();
    } else {
      len = ahead;
      ahead = load(b + 1);
    }
  }
  __device__ bool next(Seg &s) {
    if (left <= 0 || b >= p.B) return false;  // (b ends in time unless the lengths change under the kernel)
    s.b = b;
    s.hv = hv;
    s.len = length();
    s.tile = tile;
    s.tiles = tiles_of(s.len);
    s.count = static_cast<int>(min(left, static_cast<long long>(s.tiles - tile)));
    left -= s.count;
    tile += s.count;
    if (tile == s.tiles) {
      tile = 0;
      if (++hv == hvs) {
        hv = 0;
        do advance();
        while (left > 0 && b < p.B && length() == 0);
      }
    }
    return true;
  }
};

// The same by one thread, tile by tile, with the page and slot of the tile's row `row` (a page's
// slots follow one another through the tiles of a segment, so that only its first tile divides).
struct Cursor {
  Walk<false> w;
  Seg s;
  int i = 0, seg = -1, row;
  int index = 0, slot = 0;   // index: in the sequence's table row
  int keys = 0, behind = 0;  // valid keys in the tile; tokens of the sequence from the tile's first on
  int head = 0;
  __device__ Cursor(const PagedParams &p, const Start &at, int r) : w(p, at), row(r) { s.count = 0; }
  __device__ bool next() {
    if (i == s.count) {
      if (!w.next(s)) return false;
      i = 0;
      ++seg;
      const int first = s.tile * kPagedTile, pos = first + row;
      index = pos / w.p.page;
      slot = pos - index * w.p.page;
      behind = s.len - first;
      head = w.p.blocks == 1 ? s.hv : s.hv / w.p.blocks;
    } else {
      index += w.p.tile_pages;
      slot += w.p.tile_slots;
      if (slot >= w.p.page) {
        slot -= w.p.page;
        ++index;
      }
      behind -= kPagedTile;
    }
    ++i;
    keys = min(kPagedTile, behind);
    return true;
  }
  __device__ bool first() const { return i == 1; }
};

// Where a tile's K and V begin in the ring's order K0 K1 V0 K2 V1 ... (T tiles, nc slots each).
__device__ __forceinline__ uint32_t k_pos(uint32_t t, int nc) { return t == 0 ? 0 : (2 * t - 1) * nc; }
__device__ __forceinline__ uint32_t v_pos(uint32_t t, uint32_t T, int nc) { return (min(t + 2, T) + t) * nc; }

template <int D, int NH>
__global__ void __launch_bounds__(kThreads, PagedCfg<D, NH>::RES)
    decode_paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const PagedParams p) {
  using C = PagedCfg<D, NH>;
  extern __shared__ uint8_t smem_raw[];
  struct Misc {
    long long warp_tiles[kThreads / 32];
    Start start;
    uint32_t tmem_base;
    volatile uint32_t abort_flag;
    volatile uint32_t fresh[2];  // whether a tile's PV begins O anew, by the buffer of its weights
  };
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *const base_ptr = smem_raw + (base - raw);
  float *const red = reinterpret_cast<float *>(base_ptr + C::OFF_RED);
  Misc &misc = *reinterpret_cast<Misc *>(base_ptr + C::OFF_BAR + 8 * C::NBAR);
  static_assert(8 * C::NBAR + sizeof(Misc) <= C::BAR_BYTES, "barrier room");
  const uint32_t bars = base + C::OFF_BAR;
  auto BAR = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < C::NSLOT; ++i) {
      mbar_init(BAR(C::B_FULL + i), kProducers);
      mbar_init(BAR(C::B_EMPTY + i), 1);
    }
    for (int i = 0; i < C::NQB; ++i) {
      mbar_init(BAR(C::B_QFULL + i), 1);
      mbar_init(BAR(C::B_QEMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(C::B_SFULL + i), 1);
      mbar_init(BAR(C::B_PFULL + i), 4);
      mbar_init(BAR(C::B_PDONE + i), 1);
    }
    mbar_init(BAR(C::B_DRAIN), 1);
    misc.abort_flag = 0u;
    misc.start = {0, 0, 0, 0, 0};
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 4) {
    tmem_alloc(smem_u32(&misc.tmem_base), C::T_COLS);
    tmem_relinquish();
    // Only now: a dependent kernel's CTA beside this one must not take the tensor memory first and
    // then wait for this kernel's end.
    grid_launch_dependents();
  }
  grid_wait_prior();  // what follows reads the previous kernels' results

  // ------------------------------------------------------------ this CTA's share
  // Thread i counts the units of its run of sequences; a scan over the block gives the total
  // and finds the sequence in which this CTA's share begins.
  const int hvs = p.Hkv * p.blocks;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int s0 = min(p.B, tid * per), s1 = min(p.B, s0 + per);
  long long mine = 0;
  int len0 = 0;  // of its first sequence
  for (int b = s0; b < s1; ++b) {
    const int n = p.lengths[b], m = clamp_length(n, p);
    if (b == s0) len0 = m;
    if (n != m && blockIdx.x == 0) atomicCAS(p.status, 0u, kDevBadLength);
    mine += static_cast<long long>(tiles_of(m)) * hvs;
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
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) upto += misc.warp_tiles[w];
    total += misc.warp_tiles[w];
  }
  // The first G CTAs have a unit at least, the others none: a row's parts lie in CTAs next to one another.
  const long long G = min(static_cast<long long>(gridDim.x), max(total, 1LL)), cta = min(static_cast<long long>(blockIdx.x), G);
  const long long u0 = total * cta / G, u1 = total * min(cta + 1, G) / G;
  if (u0 < u1 && upto - mine <= u0 && u0 < upto) {
    long long off = u0 - (upto - mine);
    int n = len0;
    for (int b = s0; b < s1; ++b) {
      if (b > s0) n = clamp_length(p.lengths[b], p);
      const long long units = static_cast<long long>(tiles_of(n)) * hvs;
      if (off >= units) {
        off -= units;
        continue;
      }
      const unsigned long long nt = static_cast<unsigned long long>(tiles_of(n)), o = static_cast<unsigned long long>(off);
      // 32-bit division where it serves (it nearly always does)
      const unsigned long long hv = (o >> 32) == 0 ? static_cast<uint32_t>(o) / static_cast<uint32_t>(nt) : o / nt;
      misc.start = {b, n, static_cast<int>(hv), static_cast<int>(o - hv * nt), u1 - u0};
      break;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc.tmem_base;
  const long long T = u1 - u0;
  const Start start = misc.start;
  bool ok = true;

  if (warp >= 5) {
    // ---------------------------------------------------------- producers
    const int which = warp - 5;
    // A lane copies its box of a slot, if it has one in the tile (boxes of K and V are dealt out over
    // the producers); lane 0 waits for the slot and announces the producer's bytes.
    const int rows = p.box_rows, lanes = kPagedTile / rows * C::NBOX;
    const int row = (lane / C::NBOX) * rows, box = lane % C::NBOX;  // this lane's box of a slot
    const bool deals_k = lane < lanes && lane % kProducers == which;
    const bool deals_v = lane < lanes && (lanes + lane) % kProducers == which;
    const bool deals = deals_k || deals_v;
    uint32_t slot = 0, lap = 0, filled = 0;  // the ring slot next in turn, its phase, slots filled (up to NSLOT)
    int queries = 0;                         // query tiles loaded
    // Page numbers come through shared memory, asynchronously, kAhead tiles ahead: a producer that
    // waited for each in a register would run at the table's latency.
    const uint32_t mine_p = base + C::OFF_PAGES + (which * kAhead * 32 + lane) * 4;
    Cursor pre(p, start, row), it(p, start, row);
    uint32_t stage = 0;
    auto prefetch = [&]() {
      if (deals && pre.next() && row < pre.keys) cp_async_4(mine_p + stage * 128, p.table + pre.s.b * p.table_s + pre.index);
      cp_async_commit();
      stage = stage + 1 == kAhead ? 0 : stage + 1;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) prefetch();
    struct Load {
      int keys, head, page, slot;
    };
    auto look = [&](Load &l) -> bool {  // the next tile, and this lane's page of it
      if (!it.next()) return false;
      l.keys = it.keys;
      l.head = it.head;
      l.slot = it.slot;
      l.page = 0;
      cp_async_wait<kAhead - 1>();
      if (deals && row < l.keys) {
        l.page = static_cast<int>(ld_shared_u32(mine_p + stage * 128));
        if (l.page < 0 || l.page >= p.pages) atomicCAS(p.status, 0u, kDevBadPage);  // TMA reads zeros there
      }
      prefetch();
      return true;
    };
    // Bytes of this producer in a tile of `keys`: boxes first, first + kProducers, ... of the used ones.
    const int shift = 31 - __clz(rows);
    auto bytes_of = [&](int keys, int first) -> uint32_t {
      const int used = ((keys + rows - 1) >> shift) * C::NBOX;
      return used > first ? static_cast<uint32_t>((used - first + kProducers - 1) / kProducers * rows) * 128u : 0u;
    };
    const int first_k = which, first_v = (which + kProducers - lanes % kProducers) % kProducers;
    const uint32_t full_k = bytes_of(kPagedTile, first_k), full_v = bytes_of(kPagedTile, first_v);
    auto fill = [&](const Load &l, const CUtensorMap *tm, bool deal, int first, uint32_t full) {
      const uint32_t bytes = l.keys == kPagedTile ? full : bytes_of(l.keys, first);
      deal = deal && row < l.keys;
      for (int c = 0; c < C::NC; ++c) {
        // The first lap passes at once: the phase before a barrier's first counts as complete.  Lane 0
        // waits for all: a lane that tested the barrier by itself could come so late that the slot
        // had been filled and freed once more, and its parity would not come round again.
        if (lane == 0)
          ok = wait_bounded(BAR(C::B_EMPTY + slot), lap ^ 1u, &misc.abort_flag, p.status, kDevTimeoutLoad, p.wait_limit);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (filled < C::NSLOT) ++filled;
        if (lane == 0) mbar_arrive_expect_tx(BAR(C::B_FULL + slot), bytes);
        if (deal)
          tma_load_4d(base + slot * C::SLOT_BYTES + box * C::BOX_BYTES + row * 128, tm, c * C::CW + box * 64, l.slot, l.head, l.page,
                      BAR(C::B_FULL + slot));
        if (++slot == C::NSLOT) {
          slot = 0;
          lap ^= 1u;
        }
      }
    };
    auto query = [&]() {  // Q of a segment, before its first K
      const int s = it.seg;
      if (s >= C::NQB) ok = wait_bounded(BAR(C::B_QEMPTY + s % C::NQB), (s / C::NQB - 1) & 1, &misc.abort_flag, p.status, kDevTimeoutLoad, p.wait_limit);
      if (!ok) return;
      queries = s + 1;
      const uint32_t bar = BAR(C::B_QFULL + s % C::NQB), dst = base + C::OFF_Q + (s % C::NQB) * C::Q_BYTES;
      mbar_arrive_expect_tx(bar, static_cast<uint32_t>(p.q_rows) * 128u * (D / 64));
      const int head = it.head * p.G + (it.s.hv - it.head * p.blocks) * NH;
      for (int x = 0; x < D / 64; ++x) tma_load_3d(dst + x * NH * 128, &tm_q, x * 64, head, it.s.b, bar);
    };
    Load v, k;
    bool have_v = false, have_k = look(k);
    while (ok && (have_k || have_v)) {
      if (have_k) {
        if (it.first()) {
          if (which == kProducers - 1 && lane == 0) query();
          ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        if (ok) fill(k, &tm_k, deals_k, first_k, full_k);
      }
      if (ok && have_v) fill(v, &tm_v, deals_v, first_v, full_v);
      v = k;
      have_v = have_k;
      have_k = have_k && look(k);
    }
    cp_async_wait<0>();
    // After a time-out: copies that nobody waited for land before the CTA ends (a slot before the
    // next in turn was last filled in this lap; one that not every producer filled never completes,
    // and gets some milliseconds).
    if (lane == 0 && misc.abort_flag) {
      for (uint32_t x = 0; x < filled; ++x) wait_drain(BAR(C::B_FULL + x), x < slot ? lap : lap ^ 1u, p.wait_limit >> 10);
      for (int x = max(0, queries - C::NQB); x < queries; ++x)
        wait_drain(BAR(C::B_QFULL + x % C::NQB), (x / C::NQB) & 1, p.wait_limit >> 10);
    }
    __syncwarp();
  } else if (warp == 4) {
    // ---------------------------------------------------------- MMA issuer
    const uint32_t idesc_s = p.bf16 ? idesc_bf16_f32(128, C::NQ, 0, 0) : idesc_f16_f32(128, C::NQ, 0, 0);
    const uint32_t idesc_o = p.bf16 ? idesc_bf16_f32(128, C::NP, 1, 1) : idesc_f16_f32(128, C::NP, 1, 1);
    const SDesc dk = sdesc_split(sdesc_sw128(base, 16, 1024));
    // V^T: 64-column boxes BOX_BYTES apart; at d = 64 there is one, read twice (rows 64 .. of O are not used)
    const SDesc dv = sdesc_split(sdesc_sw128(base, D == 64 ? 0 : C::BOX_BYTES, 1024));
    const SDesc dq = sdesc_split(sdesc_sw128(base + C::OFF_Q, 16, 1024));
    const SDesc dp = sdesc_split(p_desc<NH>(base + C::OFF_P));
    if (lane == 0) {
      // One thread waits and issues: no lane has to agree on anything, and a product's set-up is not
      // paid for in votes (about 500 of 2100 cycles a tile, d = 64).
      bool got = true;
      auto wait = [&](int bar, uint32_t phase) {
        got = got && wait_bounded(BAR(bar), phase & 1u, &misc.abort_flag, p.status, kDevTimeoutMma, p.wait_limit);
      };
      uint32_t slot = 0, lap = 0;  // the ring slot next in turn, and its phase
      auto step = [&]() {
        if (++slot == C::NSLOT) {
          slot = 0;
          lap ^= 1u;
        }
      };
      auto qk = [&](uint32_t i, uint32_t seg, bool first, bool last) {
        const uint32_t buf = i & 1u, qb = seg % C::NQB;
        if (first) wait(C::B_QFULL + qb, seg / C::NQB);
        // S(i - 2) has been read: PV(i - 2), issued before, waited for the weights made of it.
        for (int c = 0; c < C::NC; ++c, step()) {
          wait(C::B_FULL + slot, lap);
          if (got) {
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < C::CW / 16; ++kk)
              umma_ss_off(tmem + buf * C::NQ, dk, slot * C::SLOT_BYTES + (kk >> 2) * C::BOX_BYTES + (kk & 3) * 32, dq,
                          qb * C::Q_BYTES + (c * C::NBOX + (kk >> 2)) * NH * 128 + (kk & 3) * 32, idesc_s, (c | kk) != 0);
            umma_commit(BAR(C::B_EMPTY + slot));
          }
        }
        if (got) {
          if (!C::ONE) umma_commit(BAR(C::B_SFULL + buf));
          if (last) umma_commit(BAR(C::B_QEMPTY + qb));
        }
      };
      auto pv = [&](uint32_t i, uint32_t seg, int groups) {  // groups of 16 keys
        const uint32_t buf = i & 1u, o = tmem + C::T_O + (seg & 1u) * (C::NO * C::NP);
        wait(C::B_PFULL + buf, i >> 1);
        const bool first = misc.fresh[buf] != 0;
        for (int c = 0; c < C::NC / C::VS; ++c) {
          wait(C::B_FULL + slot, lap);
          if (C::VS == 2) wait(C::B_FULL + slot + 1, lap);
          if (got) {
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kPagedTile / 16; ++kk)
              if (kk < groups)
                umma_ss_off(o + c * C::NP, dv, slot * C::SLOT_BYTES + kk * 2048, dp, buf * C::P_BYTES + kk * (16 * 4 * NH), idesc_o,
                            !first || kk > 0);
            umma_commit(BAR(C::B_EMPTY + slot));
            if (C::VS == 2) umma_commit(BAR(C::B_EMPTY + slot + 1));
          }
          step();
          if (C::VS == 2) step();
        }
        if (!C::ONE && got) umma_commit(BAR(C::B_PDONE + buf));
      };
      // QK a tile ahead of PV; a segment is looked up when its first QK is due.
      Walk<false> w(p, start);
      Seg s;
      uint32_t i = 0, seg = 0;
      bool pending = false;  // PV(i - 1) is due
      uint32_t pending_seg = 0;
      int pending_groups = 0;
      while (got && w.next(s)) {
        for (int j = 0; got && j < s.count; ++j, ++i) {
          qk(i, seg, j == 0, j == s.count - 1);
          if (got && pending) pv(i - 1, pending_seg, pending_groups);
          pending = true;
          pending_seg = seg;
          pending_groups = (min(kPagedTile, s.len - (s.tile + j) * kPagedTile) + 15) >> 4;
        }
        ++seg;
      }
      if (got && pending) pv(i - 1, pending_seg, pending_groups);
      if (misc.abort_flag) {  // after a time-out: products in flight end before the CTA does
        umma_commit(BAR(C::B_DRAIN));
        wait_drain(BAR(C::B_DRAIN), 0, p.wait_limit);
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- softmax (and empty sequences)
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp) << 21);  // this warp's 32 TMEM lanes
    for (int b = blockIdx.x; b < p.B; b += gridDim.x)
      if (clamp_length(p.lengths[b], p) == 0) {
        uint32_t *const o = static_cast<uint32_t *>(p.o) + static_cast<size_t>(b) * p.Hq * (D / 2);
        for (int i = tid; i < p.Hq * (D / 2); i += 128) o[i] = 0u;
        for (int i = tid; i < p.Hq; i += 128) p.lse[static_cast<size_t>(b) * p.Hq + i] = -INFINITY;
      }
    PagedRecord record = {0, 0, 0, 0};
    auto wait = [&](int bar, uint32_t phase) {
      ok = __all_sync(0xffffffffu, wait_bounded(BAR(bar), static_cast<uint32_t>(phase & 1), &misc.abort_flag, p.status, kDevTimeoutSoftmax,
                                                p.wait_limit)) && ok;
    };
    auto wait_s = [&](uint32_t t) {  // S of tile t is there
      const uint32_t x = k_pos(t, 1);
      if (C::ONE)
        wait(C::B_EMPTY + static_cast<int>(x % C::NSLOT), x / C::NSLOT);
      else
        wait(C::B_SFULL + static_cast<int>(t & 1), t >> 1);
    };
    const uint32_t tiles = static_cast<uint32_t>(T);
    auto wait_pv = [&](uint32_t t) {  // PV of tile t is done
      const uint32_t x = v_pos(t, tiles, 1);
      if (C::ONE)
        wait(C::B_EMPTY + static_cast<int>(x % C::NSLOT), x / C::NSLOT);
      else
        wait(C::B_PDONE + static_cast<int>(t & 1), t >> 1);
    };
    constexpr int W = NH < 32 ? 8 : 16;  // columns at once (8 and 16: 16 heads at d = 64 387 and 395 us, 32 at 128 572 and 541)
    const uint32_t sum_at = lanes + C::T_SUM;
    // A segment's results wait for its last PV; they are taken after the next segment's first tile (and so before
    // sum_at holds sums of that one).
    struct {
      int heads = 0;  // 0: none due
      bool whole, begins, sums;  // sums: there are some in sum_at
      uint32_t last, seg;
      size_t row0;
    } due;
    auto results = [&]() {
      wait_pv(due.last);
      tc_fence_after();
      const size_t part = 2 * static_cast<size_t>(blockIdx.x) + (due.begins ? 1 : 0);
      const float *const sums = red + C::RED_SUMS + (due.seg & 1) * 4 * NH, *const tops = red + C::RED_TOPS + (due.seg & 1) * NH;
      const uint32_t from = lanes + C::T_O + (due.seg & 1) * (C::NO * C::NP);
      float inv[NH];
#pragma unroll
      for (int g = 0; g < NH; g += 4) {
        inv[g] = inv[g + 1] = inv[g + 2] = inv[g + 3] = 0.f;
        if (g < due.heads) {
          const float4 *const r = reinterpret_cast<const float4 *>(sums + g);
          const float4 a = r[0], b = r[NH / 4], c = r[2 * NH / 4], d = r[3 * NH / 4];
          const float t[4] = {(a.x + b.x) + (c.x + d.x), (a.y + b.y) + (c.y + d.y), (a.z + b.z) + (c.z + d.z), (a.w + b.w) + (c.w + d.w)};
#pragma unroll
          for (int e = 0; e < 4; ++e) inv[g + e] = t[e] == 0.f ? 0.f : __fdividef(1.f, t[e]);  // t < 2^126: 2 ulp
        }
      }
      if (ok && tid < due.heads) {
        const float lse2 = tops[tid] - kShift + __log2f((sums[tid] + sums[NH + tid]) + (sums[2 * NH + tid] + sums[3 * NH + tid]));
        if (due.whole)
          p.lse[due.row0 + tid] = lse2 * 0.69314718055994531f;
        else
          p.part_lse[part * NH + tid] = lse2;
      }
#pragma unroll
      for (int ob = 0; ob < C::NO; ++ob) {
        uint32_t o[C::NP];
        tmem_ld<C::NP>(from + ob * C::NP, o);
        const int col = ob * 128 + tid;
        if (!ok || (D < 128 && tid >= D)) continue;
#pragma unroll
        for (int h = 0; h < NH; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) + __uint_as_float(o[NH + h]));
        if (due.sums) {
#pragma unroll
          for (int g = 0; g < NH; g += W) {
            uint32_t t[W];
            tmem_ld<W>(sum_at + ob * NH + g, t);
#pragma unroll
            for (int h = 0; h < W; ++h) o[g + h] = __float_as_uint(__uint_as_float(t[h]) + __uint_as_float(o[g + h]));
          }
        }
#pragma unroll
        for (int h = 0; h < NH; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * inv[h]);
        if (!due.whole) {
          float *to = p.part_o + part * NH * D + col;
#pragma unroll
          for (int h = 0; h < NH; ++h, to += D)
            if (h < due.heads) *to = __uint_as_float(o[h]);
        } else {
          uint16_t *to = static_cast<uint16_t *>(p.o) + due.row0 * D + col;
#pragma unroll
          for (int h = 0; h < NH; h += 2, to += 2 * D) {
            const uint32_t two = p.bf16 ? pack2<true>(__uint_as_float(o[h]), __uint_as_float(o[h + 1]))
                                        : pack2<false>(__uint_as_float(o[h]), __uint_as_float(o[h + 1]));
            if (h < due.heads) to[0] = static_cast<uint16_t>(two);
            if (h + 1 < due.heads) to[D] = static_cast<uint16_t>(two >> 16);
          }
        }
      }
      tc_fence_before();
      due.heads = 0;
    };
    Walk<true> w(p, start);
    Seg s;
    uint32_t i = 0;  // tiles done
    for (uint32_t seg = 0; w.next(s); ++seg) {
      const int kv = p.blocks == 1 ? s.hv : s.hv / p.blocks, block = s.hv - kv * p.blocks, heads = min(NH, p.G - block * NH);
      const uint32_t o_at = lanes + C::T_O + (seg & 1) * (C::NO * C::NP);
      float m[NH], l[NH];
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
      }
      int since = 0;      // tiles in O
      bool sums = false;  // whether sum_at holds those before them
      for (int j = 0; j < s.count; ++j, ++i, ++since) {
        // After a time-out the remaining tiles run through the barriers only.
        const int buf = static_cast<int>(i & 1), n = s.len - (s.tile + j) * kPagedTile;
        uint32_t x[NH];
        wait_s(i);
        tc_fence_after();
        tmem_ld<NH>(lanes + buf * C::NQ, x);
        float top[NH];
#pragma unroll
        for (int g = 0; g < NH; g += 8)
          if (g < heads) {  // eight at a time, without branches between them
#pragma unroll
            for (int h = g; h < g + 8; ++h) {
              const float v = tid < n ? __uint_as_float(x[h]) * p.c2 : -INFINITY;
              x[h] = __float_as_uint(v);
              top[h] = warp_max(v);
            }
          } else {
#pragma unroll
            for (int h = g; h < g + 8; ++h) top[h] = 0.f;
          }
        float *const mine_r = red + (buf * 4 + warp) * NH;
        if (lane == 0) {
#pragma unroll
          for (int h = 0; h < NH; h += 4) *reinterpret_cast<float4 *>(mine_r + h) = make_float4(top[h], top[h + 1], top[h + 2], top[h + 3]);
        }
        softmax_sync();
        // ---- the running maximum, and what it does to the sums and to O
        int moved = 0;  // the same in every thread
#pragma unroll
        for (int g = 0; g < NH; g += 4)
          if (g < heads) {
            const float4 *const r = reinterpret_cast<const float4 *>(red + buf * 4 * NH + g);
            const float4 r0 = r[0], r1 = r[NH / 4], r2 = r[2 * NH / 4], r3 = r[3 * NH / 4];
            top[g] = fmaxf(fmaxf(r0.x, r1.x), fmaxf(r2.x, r3.x));
            top[g + 1] = fmaxf(fmaxf(r0.y, r1.y), fmaxf(r2.y, r3.y));
            top[g + 2] = fmaxf(fmaxf(r0.z, r1.z), fmaxf(r2.z, r3.z));
            top[g + 3] = fmaxf(fmaxf(r0.w, r1.w), fmaxf(r2.w, r3.w));
#pragma unroll
            for (int h = g; h < g + 4; ++h) moved |= static_cast<int>(h < heads) & static_cast<int>(top[h] > m[h] + kSlack);
          }
        if (j == 0) {
          moved = 0;
#pragma unroll
          for (int h = 0; h < NH; ++h) m[h] = top[h];
        }
        if (i >= 2) wait_pv(i - 2);  // the weights' buffer, and fresh, are free again
        const bool begins = j == 0 || moved || since == kFold;  // O anew
        if (begins && j > 0) {
          // Before the weights, not after: the factors need not live beside them (16 heads at d = 64 387 us, after them 458;
          // 32 at 128 541 and 605).
          float keep[NH];
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const bool up = top[h] > m[h] + kSlack;
            keep[h] = up ? ex2_approx(m[h] - top[h]) : 1.f;
            l[h] *= keep[h];
            m[h] = up ? top[h] : m[h];
          }
          wait_pv(i - 1);
          if (ok) {
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < C::NO * NH; c += W) {
              const uint32_t from = o_at + c / NH * C::NP + c % NH;
              uint32_t t[W], o[W];
              tmem_ld<W>(from, t);
              tmem_ld<W>(from + NH, o);
#pragma unroll
              for (int h = 0; h < W; ++h) t[h] = __float_as_uint(__uint_as_float(t[h]) + __uint_as_float(o[h]));
              if (sums) {
                tmem_ld<W>(sum_at + c, o);
#pragma unroll
                for (int h = 0; h < W; ++h) t[h] = __float_as_uint(__uint_as_float(t[h]) + __uint_as_float(o[h]));
              }
#pragma unroll
              for (int h = 0; h < W; ++h) t[h] = __float_as_uint(__uint_as_float(t[h]) * keep[c % NH + h]);
              tmem_st<W>(sum_at + c, t);
            }
          }
          sums = true;
          since = 0;
        }
        if (tid == 0) misc.fresh[buf] = begins;
        // ---- the weights of this thread's key, as hi + lo
        const uint32_t prow = base + C::OFF_P + buf * C::P_BYTES + tid * (4 * NH);
        const uint32_t swz = NH == 8 ? (tid >> 2) & 1 : NH == 16 ? (tid >> 1) & 3 : tid & 7;
#pragma unroll
        for (int g = 0; g < NH; g += 8)
          if (g < heads) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int h = g; h < g + 8; ++h) {
              const float w = ex2_approx(__uint_as_float(x[h]) - (m[h] == -INFINITY ? 0.f : m[h] - kShift));
              l[h] += w;
              x[h] = __float_as_uint(w);
            }
            if (p.bf16) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                split_weights<true>(__uint_as_float(x[g + 2 * e]), __uint_as_float(x[g + 2 * e + 1]), hi[e], lo[e]);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                split_weights<false>(__uint_as_float(x[g + 2 * e]), __uint_as_float(x[g + 2 * e + 1]), hi[e], lo[e]);
            }
            st_shared_v4(prow + (((g >> 3) ^ swz) << 4), hi[0], hi[1], hi[2], hi[3]);
            st_shared_v4(prow + ((((NH + g) >> 3) ^ swz) << 4), lo[0], lo[1], lo[2], lo[3]);
          }
        if ((n & 15) != 0 && n < kPagedTile) {
          // PV takes keys in groups of 16 (all 128, and every row behind the last token cleared by its own
          // thread: 154 x 32 heads of 4 tokens x 128 82.8 us, now 52).  Whatever lies behind the last token in its group (unwritten
          // slots, earlier tiles) times a weight of zero must be zero: clear those rows of V, eight
          // threads to a row.
          if constexpr (C::NSLOT < 3 * C::NC) {
            // The slots' earlier loads, of V(i - 1) and K(i + 1), must be past, or a wait for V's load
            // would take the phase before theirs for it.  (In a longer ring they were of K(i) at the latest.)
            if (i >= 1) wait_pv(i - 1);
            if (i + 1 < tiles) wait_s(i + 1);
          }
          const uint32_t v0 = v_pos(i, tiles, C::NC);
          for (int c = 0; c < C::NC; ++c) {
            const uint32_t slot = (v0 + c) % C::NSLOT;
            wait(C::B_FULL + static_cast<int>(slot), (v0 + c) / C::NSLOT);
            const int row = n + (tid >> 3);
            if (ok && row < ((n + 15) & ~15))
#pragma unroll
              for (int z = 0; z < C::NBOX; ++z) st_shared_v4(base + slot * C::SLOT_BYTES + z * C::BOX_BYTES + row * 128 + (tid & 7) * 16, 0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::B_PFULL + buf));
        if (due.heads) results();  // of the segment before
      }
      // ---------------------------------------------------------- the segment's sums
      // (the next barrier, of the next tile or the last one, makes them visible)
      warp_sums<NH>(l, red + C::RED_SUMS + ((seg & 1) * 4 + warp) * NH);
      if (tid == 0) {
        float *const tops = red + C::RED_TOPS + (seg & 1) * NH;
#pragma unroll
        for (int h = 0; h < NH; h += 4) *reinterpret_cast<float4 *>(tops + h) = make_float4(m[h], m[h + 1], m[h + 2], m[h + 3]);
      }
      due.heads = heads;
      due.whole = s.count == s.tiles;
      due.begins = s.tile == 0;
      due.sums = sums;
      due.last = i - 1;
      due.seg = seg;
      due.row0 = static_cast<size_t>(s.b) * p.Hq + kv * p.G + block * NH;
      if (!due.whole && due.begins) {
        // The row goes on in the next CTAs: up to the one whose share holds its last unit `end`, the
        // largest c with floor(total c / G) <= end, that is c < (end + 1) G / total.
        const long long end = u1 + (s.tiles - s.count) - 1;
        record.head = static_cast<int>(due.row0);
        record.heads = heads;
        record.parts = static_cast<int>(((end + 1) * G - 1) / total) - static_cast<int>(blockIdx.x) + 1;
      }
    }
    softmax_sync();
    if (due.heads) results();
    if (tid == 0 && p.records) p.records[blockIdx.x] = record;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) tmem_dealloc(tmem, C::T_COLS);
}

// Joins the rows that were cut: block (c, h) the h-th head of the row that CTA c's share ends in, or
// (W > 1: few rows) block (r, h) that of row r, whose CTA it looks up.  W groups of 128 threads, a thread
// to a column, take every W-th part each.
template <int D, int NH, int W>
__global__ void __launch_bounds__(128 * W) paged_merge_kernel(const PagedParams p, const int ctas) {
  __shared__ float weight[kPagedMaxCtas];
  __shared__ float sums[W > 1 ? W - 1 : 1][128];
  __shared__ float shared_sum;
  grid_launch_dependents();
  grid_wait_prior();
  const int h = blockIdx.y, tid = threadIdx.x;
  int cta = blockIdx.x;
  if constexpr (W > 1) {
    __shared__ int found;
    static_assert(128 * W >= kPagedMaxCtas, "a thread to a record");
    if (tid == 0) found = -1;
    __syncthreads();
    const int hvs = p.Hkv * p.blocks, b = blockIdx.x / hvs, hv = blockIdx.x - b * hvs, kv = hv / p.blocks;
    const int head = b * p.Hq + kv * p.G + (hv - kv * p.blocks) * NH;
    if (tid < ctas) {
      const PagedRecord r = p.records[tid];
      if (r.parts > 0 && r.head == head) found = tid;
    }
    __syncthreads();
    cta = found;
    if (cta < 0) return;
  }
  const PagedRecord r = p.records[cta];
  if (h >= r.heads) return;
  auto part = [&](int i) -> size_t { return i == 0 ? 2 * static_cast<size_t>(cta) + 1 : 2 * (static_cast<size_t>(cta) + i); };
  for (int i = tid; i < r.parts; i += 128 * W) weight[i] = p.part_lse[part(i) * NH + h];
  __syncthreads();
  if (tid < 32) {
    float M = -INFINITY, sum = 0.f;
    bool nan = false;
    for (int i = tid; i < r.parts; i += 32) {
      M = fmaxf(M, weight[i]);
      nan = nan || weight[i] != weight[i];
    }
    M = warp_max(M);
    const float from = M == -INFINITY ? 0.f : M;
    for (int i = tid; i < r.parts; i += 32) {
      const float w = ex2_approx(weight[i] - from);
      weight[i] = w;
      sum += w;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (__any_sync(0xffffffffu, nan)) sum = NAN;
    if (tid == 0) {
      shared_sum = sum;
      p.lse[r.head + h] = (M + __log2f(sum)) * 0.69314718055994531f;
    }
  }
  __syncthreads();
  const float sum = shared_sum, inv = sum == 0.f ? 0.f : 1.f / sum;
  const int group = tid >> 7, col = tid & 127;
  for (int c = col; c < (D < 128 ? 128 : D); c += 128) {
    float o = 0.f;
    if (D >= 128 || c < D)
#pragma unroll 8
      for (int i = group; i < r.parts; i += W) o = fmaf(weight[i], p.part_o[(part(i) * NH + h) * D + c], o);
    if constexpr (W > 1) {
      if (group > 0) sums[group - 1][col] = o;
      __syncthreads();
      if (group == 0)
#pragma unroll
        for (int w = 0; w < W - 1; ++w) o += sums[w][col];
      __syncthreads();
    }
    if (group > 0 || (D < 128 && c >= D)) continue;
    o *= inv;
    const size_t at = static_cast<size_t>(r.head + h) * D + c;
    if (p.bf16)
      static_cast<__nv_bfloat16 *>(p.o)[at] = __float2bfloat16_rn(o);
    else
      static_cast<__half *>(p.o)[at] = __float2half_rn(o);
  }
}

template <int D, int NH>
cudaError_t launch_paged(const PagedLaunch &a) {
  using C = PagedCfg<D, NH>;
  auto *kern = decode_paged_kernel<D, NH>;
  static std::atomic<unsigned long long> configured{0};  // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(configured >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured |= 1ull << dev;
  }
  // At most one CTA per unit of work that the tables have room for (and lengths, of 31 bits, can name).
  const long long row_tiles =
      std::min((static_cast<long long>(a.p.table_w) * a.p.page + kPagedTile - 1) / kPagedTile, (1LL << 31) / kPagedTile);
  const long long units = static_cast<long long>(a.p.B) * a.p.Hkv * a.p.blocks * row_tiles;
  const unsigned grid = static_cast<unsigned>(std::min<long long>(units, std::min(C::RES * a.sm_count, kPagedMaxCtas)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  PagedParams p = a.p;
  const bool cut = row_tiles > 1;  // a row of one tile is never cut
  if (!cut) p.records = nullptr;
  e = cudaLaunchKernelEx(&cfg, kern, a.tm_q, a.tm_k, a.tm_v, p);
  if (e != cudaSuccess || !cut) return e;
  // Rows of eight parts and more are joined by eight groups, in blocks for the rows only: one key head of
  // a sequence of 34346 tokens, 269 parts, 26.0 us with one group, 13.6 with eight (16 query heads to each of 8
  // key heads, 20000 tokens: 21.8; with a block for every CTA and head, most of them with nothing to do, 24.3).
  const long long rows = static_cast<long long>(a.p.B) * a.p.Hkv * a.p.blocks;
  const bool wide = 8 * rows <= grid;
  cfg.gridDim = dim3(wide ? static_cast<unsigned>(rows) : grid, static_cast<unsigned>(std::min(NH, a.p.G)));
  cfg.blockDim = dim3(wide ? 1024 : 128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, wide ? paged_merge_kernel<D, NH, 8> : paged_merge_kernel<D, NH, 1>, p, static_cast<int>(grid));
}

template <int D>
cudaError_t launch_paged_d(const PagedLaunch &a) {
  switch (paged_heads(a.p.G, D)) {
    case 8: return launch_paged<D, 8>(a);
    case 16: return launch_paged<D, 16>(a);
    default:
      if constexpr (D <= 256) return launch_paged<D, 32>(a);
      return cudaErrorInvalidValue;  // paged_heads gives at most 16 there
  }
}

}  // namespace

cudaError_t launch_decode_paged(const PagedLaunch &a) {
  switch (a.p.d) {
    case 64: return launch_paged_d<64>(a);
    case 128: return launch_paged_d<128>(a);
    case 256: return launch_paged_d<256>(a);
    default: return launch_paged_d<512>(a);
  }
}

}  // namespace gbattn
