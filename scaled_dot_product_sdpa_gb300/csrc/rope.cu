// rope.cu -- rotary positions, per-head norms and the paged append: kernels and launches.
//
// Every kernel is one pass over its rows and bound by their reads and writes.  A row of d
// elements belongs to consecutive lanes of one warp, E elements each: 8 (8, 16, 32 lanes for
// d = 64, 128, 256), or 16 at d = 512.  A lane holds two vectors of E / 2 elements that contain both
// halves of every pair it turns, so that neither layout needs an exchange between lanes:
//     half layout, lane j < rotary / E:  elements E/2 j .. and rotary/2 + E/2 j ..
//     otherwise (interleaved, and the elements behind `rotary`):  E j .. E j + E - 1
// and in both layouts lane j turns its pairs by the angles E/2 j .. E/2 j + E/2 - 1.  The norm's
// sum of squares is a shuffle reduction over the row's lanes.
//
// The work is cut into units, a few rows for each thread: a tile of `tokens` consecutive (batch,
// row) positions times a step, a run of heads of one tensor (q, k or, for the append, v).  As many
// blocks as fit the GPU at once take equal runs of consecutive units, so that none is left with a
// thin last wave; a block goes through its tiles, their tensors and their steps, and works out
// addresses once per tensor.  A unit's loads are all issued before its first row is worked on; a new
// tile's cosines and sines are computed once, into shared memory, behind them, and each thread keeps
// those of its token in registers.  Arithmetic runs on fp32 pairs (two elements an instruction).
//
// Measured on GB300: rotation of 8 x 64 x 512 x 128 in fp16 25.3 us (5.3 TB/s), of half of each head of
// 100003 x 32 x 64 134 us (6.1 TB/s); norm and rotation of 4 x 40 x 2048 x 128 in bf16 34.9 us (4.8 TB/s), its
// backward pass 57.5 (4.4 TB/s); the append of 8 x 48 x 1024 x 128 37.9, with norms 41.2 (5.3, 4.9 TB/s).
// With norms neither HBM (44% of its peak rate; 50% backward) nor issue (57% and 54% of the slots) is at its
// limit: a unit is a chain of loads, a reduction and stores, and 24 (16) warps an SM are what the registers leave to
// overlap them.  Few heads leave a thread's rows empty and share a tile's angles among few rows: one head each
// of queries and keys x 40495 x 512 84.2 us (29% of the copy bandwidth; backward 113, 32%), the backward pass of two
// heads each x 25 x 8169 x 64 105 (44%).  Tried and slower or flat: 16 elements a lane without the fp32 pairs
// (44.5 and 92 us; with them only at d = 512), addresses worked out per unit (36.6, 62.3), the
// next unit's loads ahead in registers (39 to 60) or through shared memory by asynchronous copies, two to
// four units deep (38.4, 62 to 72), smaller shares in two or four waves (36.9 and more).
//
// Angles: position x inv_freq is reduced in integers.  inv_freq / 2 pi becomes a 64-bit
// binary fraction of a turn; its product with the position, taken modulo 2^64, is the angle
// modulo one turn, wrong by at most (1 + inv_freq / 4) |position| 2^-64 turns (so a position
// of 10^6 costs no accuracy, where an fp32 product would be off by 0.06 radians).
#include <algorithm>
#include <type_traits>

#include "ptx_paged.cuh"
#include "rope.cuh"
#include "vec16.cuh"

namespace gbattn {
namespace {

// Rows that a thread loads before it works on the first, and blocks that share an SM (the
// kernels' launch bounds).  Measured on GB300 with 4 rows and 3 blocks against 2 rows and 4 blocks:
// rotation of 8 x 64 x 512 x 128 25.3 us, 33.0; with norms of 4 x 40 x 2048 x 128 34.9, 48.5.  The
// backward pass reads twice as much a row: 4 rows and 2 blocks 57.5 us, 3 and 2 61.1, 2 and 3 77.7.
// With 16 elements a lane (8 x 32 x 106 x 512, and one head of 40495 rows): 2 rows and 2 blocks 32.8 and
// 113 us, 2 and 1 32.2 and 143, 1 and 2 33.5 and 99.5.  Those instances of the backward pass are the only ones that
// spill (64 to 76 bytes a thread, at 128 registers); 8 x 40 x 304 x 512 turned as a whole 72.0 us (61%).
template <int E>
constexpr int kAtOnce = E == 8 ? 4 : 2;
template <int E>
constexpr int kResident = E == 8 ? 3 : 2;
template <int E>
constexpr int kBwdAtOnce = E == 8 ? 4 : 2;
constexpr int kBwdResident = 2;

// frac(x / 2 pi) 2^64 of a finite double x = m 2^e (m an integer of at most 53 bits):
// m C 2^(e - 2) with C = 2^66 / 2 pi, as a 128-bit integer, modulo 2^64.
__device__ __forceinline__ uint64_t turns_fixed(double x) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(x));
  const int ef = static_cast<int>((bits >> 52) & 0x7ff);
  if (ef == 0) return 0;  // zero, or below 2^-1022
  const uint64_t m = (bits & 0xfffffffffffffull) | (1ull << 52);
  const uint64_t C = 0xa2f9836e4e441529ull;  // 2^66 / 2 pi = 2^65 / pi
  const uint64_t hi = __umul64hi(m, C), lo = m * C;
  const int s = 2 - (ef - 1075);  // shift right by s
  uint64_t f;
  if (s >= 128)
    f = 0;
  else if (s >= 64)
    f = hi >> (s - 64);
  else if (s > 0)
    f = (hi << (64 - s)) | (lo >> s);
  else
    f = s > -64 ? lo << (-s) : 0;
  return (bits >> 63) ? 0ull - f : f;
}

// factor * (cos, sin) of position * freq, freq as turns_fixed gave it.  The upper 32 bits of the
// angle are enough: an error of 2^-32 turns is far below the fp32 sine's own.
__device__ __forceinline__ float2 turn_of(int position, uint64_t freq, float factor, float sign) {
  const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(position)) * freq;
  float s, c;
  sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f, &s, &c);
  return make_float2(factor * c, sign * factor * s);
}

struct Place {       // where a thread works
  int c0, c1;        // first elements of its two vectors
  bool turns;        // whether its pairs are turned
  int lane;          // lane j within the row
};

template <bool INTER, int E>
__device__ __forceinline__ Place place_of(const RopeParams &p, int lpr) {
  Place r;
  r.lane = threadIdx.x & (lpr - 1);
  r.turns = r.lane < p.rotary / E;
  const bool split = !INTER && r.turns;
  r.c0 = split ? E / 2 * r.lane : E * r.lane;
  r.c1 = split ? E / 2 * r.lane + (p.rotary >> 1) : E * r.lane + E / 2;
  return r;
}

// E / 2 16-bit values as they lie in memory.
template <int E>
struct Vec {
  uint32_t w[E / 4];
};
template <int E>
__device__ __forceinline__ Vec<E> load_vec(const uint16_t *p) {
  Vec<E> v;
  if constexpr (E == 8) {
    const uint2 t = __ldg(reinterpret_cast<const uint2 *>(p));
    v.w[0] = t.x;
    v.w[1] = t.y;
  } else {
    const uint4 t = __ldg(reinterpret_cast<const uint4 *>(p));
    v.w[0] = t.x;
    v.w[1] = t.y;
    v.w[2] = t.z;
    v.w[3] = t.w;
  }
  return v;
}
template <int E>
__device__ __forceinline__ void store_vec(uint16_t *p, const Vec<E> &v) {
  if constexpr (E == 8)
    *reinterpret_cast<uint2 *>(p) = make_uint2(v.w[0], v.w[1]);
  else
    *reinterpret_cast<uint4 *>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}
template <int E>
__device__ __forceinline__ Vec<E> zero_vec() {
  Vec<E> v;
#pragma unroll
  for (int i = 0; i < E / 4; ++i) v.w[i] = 0u;
  return v;
}
// A lane's elements as fp32 pairs: A the first elements of its rotary pairs, B the second, two
// rotary pairs to an fp32x2 register, so that all arithmetic runs two elements an instruction.
// Half layout: word i of the first vector is A[i], of the second B[i].  Interleaved: words 2i
// and 2i + 1 (of the lane's E / 2) hold A[i], B[i] as their low and high halves.
template <int E>
struct Pairs {
  uint64_t A[E / 4], B[E / 4];
};
template <bool BF, bool INTER, int E>
__device__ __forceinline__ void unpack(const Vec<E> &a, const Vec<E> &b, Pairs<E> &x) {
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    const uint32_t u = INTER ? (2 * i < E / 4 ? a.w[2 * i] : b.w[2 * i - E / 4]) : a.w[i];
    const uint32_t v = INTER ? (2 * i < E / 4 ? a.w[2 * i + 1] : b.w[2 * i + 1 - E / 4]) : b.w[i];
    float u0, u1, v0, v1;
    unpack2<BF>(u, u0, u1);
    unpack2<BF>(v, v0, v1);
    x.A[i] = INTER ? f32x2(u0, v0) : f32x2(u0, u1);
    x.B[i] = INTER ? f32x2(u1, v1) : f32x2(v0, v1);
  }
}
template <bool BF, bool INTER, int E>
__device__ __forceinline__ void store_row(uint16_t *row, int over, const Pairs<E> &x) {
  Vec<E> a, b;
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    float p0, p1, q0, q1;
    f32x2_split(x.A[i], p0, p1);
    f32x2_split(x.B[i], q0, q1);
    const uint32_t u = INTER ? pack2<BF>(p0, q0) : pack2<BF>(p0, p1), v = INTER ? pack2<BF>(p1, q1) : pack2<BF>(q0, q1);
    if constexpr (INTER) {
      (2 * i < E / 4 ? a.w[2 * i] : b.w[2 * i - E / 4]) = u;
      (2 * i < E / 4 ? a.w[2 * i + 1] : b.w[2 * i + 1 - E / 4]) = v;
    } else {
      a.w[i] = u;
      b.w[i] = v;
    }
  }
  store_vec<E>(row, a);
  store_vec<E>(row + over, b);
}

// Cosines, sines and negated sines of a lane's pairs (1, 0 where it does not turn).
template <int E>
struct Turn {
  uint64_t c[E / 4], s[E / 4], n[E / 4];
};
template <int E>
__device__ __forceinline__ void turn_pairs(Pairs<E> &x, const Turn<E> &t) {
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    const uint64_t a = x.A[i], b = x.B[i];
    x.A[i] = ffma2(b, t.n[i], fmul2(a, t.c[i]));
    x.B[i] = ffma2(a, t.s[i], fmul2(b, t.c[i]));
  }
}

// The norms' weights as fp32 in shared memory, q's, then k's, each in the order in which a lane's
// pairs want them: lane j's A and B at E j and E j + E / 2.
template <bool BF, bool INTER, int E>
__device__ __forceinline__ void fill_weights(float *weights, const RopeParams &p) {
  for (int i = threadIdx.x; i < 2 * p.d; i += kRopeThreads) {
    const bool is_q = i < p.d;
    const uint16_t *const w = static_cast<const uint16_t *>(is_q ? p.q_w : p.k_w);
    if (!w) continue;
    const int k = is_q ? i : i - p.d, j = k / E, e = k % E, half = e / (E / 2), r = e % (E / 2);  // lane, A or B, place there
    const bool split = !INTER && j < p.rotary / E;
    // unpack's order: interleaved pairs where INTER; else the lane's first and second vector
    const int from = split ? half * (p.rotary >> 1) + E / 2 * j + r : INTER ? E * j + 2 * r + half : E * j + half * (E / 2) + r;
    float lo, hi;
    unpack2<BF>(w[from], lo, hi);
    weights[i] = lo;
  }
}
template <int E>
__device__ __forceinline__ void weight_pairs(const float *w, int lane, Pairs<E> &out) {
#pragma unroll
  for (int i = 0; i < E / 4; i += 2) {
    const float4 a = *reinterpret_cast<const float4 *>(w + E * lane + 2 * i);
    const float4 b = *reinterpret_cast<const float4 *>(w + E * lane + E / 2 + 2 * i);
    out.A[i] = f32x2(a.x, a.y);
    out.A[i + 1] = f32x2(a.z, a.w);
    out.B[i] = f32x2(b.x, b.y);
    out.B[i + 1] = f32x2(b.z, b.w);
  }
}

// sum of x y over a row's lanes
template <int E>
__device__ __forceinline__ float lane_dot(const Pairs<E> &x, const Pairs<E> &y) {
  uint64_t t = fmul2(x.A[0], y.A[0]);
  t = ffma2(x.B[0], y.B[0], t);
#pragma unroll
  for (int i = 1; i < E / 4; ++i) {
    t = ffma2(x.A[i], y.A[i], t);
    t = ffma2(x.B[i], y.B[i], t);
  }
  float lo, hi;
  f32x2_split(t, lo, hi);
  return lo + hi;
}

// The block's frequencies as fixed-point turns, and the factor of each pair (NaN where the
// frequency is not finite).
struct Frequencies {
  uint64_t turns[256];
  float factor[256];
};
__device__ __forceinline__ void fill_frequencies(Frequencies &f, const RopeParams &p) {
  for (int i = threadIdx.x; i < (p.rotary >> 1); i += kRopeThreads) {
    const double x = p.inv_freq[i];
    f.turns[i] = turns_fixed(x);
    f.factor[i] = isfinite(x) ? p.factor : NAN;
  }
}
// The tile's cosines and sines: a row of a token's pairs after the other, 16 bytes apart so that
// neither the threads of fill_turns (neighbouring tokens) nor a row's lanes (neighbouring pairs)
// meet in few banks.
__host__ __device__ constexpr int turns_row(int rotary) { return (rotary >> 1) + 2; }
__device__ __forceinline__ void fill_turns(float2 *table, const int *pos, const Frequencies &f, const RopeParams &p) {
  const int shift = 31 - __clz(p.tokens);
  for (int i = threadIdx.x; i < (p.rotary >> 1) << shift; i += kRopeThreads) {
    const int r = i >> shift;
    const int token = i & (p.tokens - 1);
    table[token * turns_row(p.rotary) + r] = turn_of(pos[token], f.turns[r], f.factor[r], p.sign);
  }
}
template <int E>
__device__ __forceinline__ void load_turns(const float2 *table, int token, int rotary, const Place &at, Turn<E> &t) {
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    float4 x = make_float4(1.f, 0.f, 1.f, 0.f);  // two pairs
    if (at.turns) x = *reinterpret_cast<const float4 *>(table + token * turns_row(rotary) + E / 2 * at.lane + 2 * i);
    t.c[i] = f32x2(x.x, x.z);
    t.s[i] = f32x2(x.y, x.w);
    t.n[i] = f32x2(-x.y, -x.w);
  }
}

// The units of this block, as a run over tiles and steps; a step is a run of heads of one tensor.
struct Units {
  int tile, step, left;  // B L fits 31 bits, and so do a block's units (2^40 rows in all at most)
};
__device__ __forceinline__ Units units_of(const RopeParams &p) {
  const long long u0 = p.units * blockIdx.x / gridDim.x, u1 = p.units * (blockIdx.x + 1) / gridDim.x;
  Units u;
  u.tile = static_cast<int>(u0 / p.steps);
  u.step = static_cast<int>(u0 - static_cast<long long>(u.tile) * p.steps);
  u.left = static_cast<int>(u1 - u0);
  return u;
}

// f of a constant number of rows, the least of U, U / 2 and 1 that is not below n (the same in every
// thread): a step of few heads is not worked on as if it had all its rows (backward pass of 2 heads of 25 x
// 8169 x 64 132.9 us, now 105.1; the forward pass has less to save and pays in registers: 4 x 40 x 2048 x
// 128 34.9, 36.2).
template <int U, typename F>
__device__ __forceinline__ void on_rows(int n, const F &f) {
  if constexpr (U > 2) {
    if (n <= 1) return f(std::integral_constant<int, 1>());
  }
  if constexpr (U > 1) {
    if (n <= U / 2) return f(std::integral_constant<int, U / 2>());
  }
  f(std::integral_constant<int, U>());
}

// A thread's token in the current tile.
struct Token {
  int b, l;
  bool in;  // whether there is one
};
__device__ __forceinline__ Token token_of(const RopeParams &p, int n) {
  Token t;
  t.in = n < p.B * p.L;
  t.b = t.in ? n / p.L : 0;
  t.l = t.in ? n - t.b * p.L : 0;
  return t;
}
__device__ __forceinline__ const uint16_t *row_at(const void *p, const Token &t, long long batch, long long row) {
  return static_cast<const uint16_t *>(p) + t.b * batch + t.l * row;
}

// attn_rope and (APPEND) attn_cache_append.  The append's new tokens of sequence b are counts[b]
// rows (all L without counts) at positions lengths[b] - counts[b] .. lengths[b] - 1; their keys
// and values go to the pages that the table names, their queries to q_out (zeros behind the
// last token).
template <bool BF, bool NORM, bool INTER, int E, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads, kResident<E>) rope_kernel(const RopeParams p) {
  constexpr int U = kAtOnce<E>;
  extern __shared__ __align__(16) float2 turns[];
  __shared__ int pos[kRopeMaxTokens];
  __shared__ long long cell[APPEND ? kRopeMaxTokens : 1];  // element offset of the page slot, -1: none, -2: behind the last token
  __shared__ Frequencies freq;
  __shared__ __align__(16) float weights[NORM ? 1024 : 4];
  grid_launch_dependents();
  grid_wait_prior();
  const int lpr = p.d / E, groups = kRopeThreads / lpr / p.tokens;
  const Place at = place_of<INTER, E>(p, lpr);
  const int row = threadIdx.x / lpr, token = row / groups, group = row - token * groups;
  const uint32_t out_h = static_cast<uint32_t>(p.L) * static_cast<uint32_t>(p.d);  // below 2^32
  const bool plain = APPEND && !NORM && p.rotary == 0;
  const float inv_d = 1.f / static_cast<float>(p.d);  // exact: a power of two
  if constexpr (NORM) fill_weights<BF, INTER, E>(weights, p);
  fill_frequencies(freq, p);
  const int per = groups * p.at_once;
  for (Units u = units_of(p); u.left > 0; u.step = 0, ++u.tile) {  // a tile
    const int n0 = u.tile * p.tokens, stop = min(p.steps, u.step + u.left);
    u.left -= stop - u.step;
    const Token tok = token_of(p, n0 + token);
    bool reads = tok.in, fresh = true;
    if constexpr (APPEND)
      if (p.counts && tok.in) reads = tok.l < p.counts[tok.b];  // rows behind the last token are not read
    long long to = 0;
    Turn<E> turn;
    for (int s = u.step; s < stop;) {  // its steps of one tensor
      const int kind = s < p.steps_q ? 0 : s < p.steps_q + p.steps_k ? 1 : 2;
      const int heads = kind == 0 ? p.Hq : p.Hkv, first = kind == 0 ? 0 : kind == 1 ? p.steps_q : p.steps_q + p.steps_k;
      const int end = min(stop, first + (kind == 0 ? p.steps_q : p.steps_k));
      int h0 = (s - first) * per + group;
      const uint32_t src_h = static_cast<uint32_t>(kind == 0 ? p.qs[1] : kind == 1 ? p.ks[1] : p.vs[1]);
      const uint16_t *src = row_at(kind == 0 ? p.q : kind == 1 ? p.k : p.v, tok, kind == 0 ? p.qs[0] : kind == 1 ? p.ks[0] : p.vs[0],
                                   kind == 0 ? p.qs[2] : kind == 1 ? p.ks[2] : p.vs[2]) +
                            static_cast<uint64_t>(h0) * src_h + at.c0;
      const int over = at.c1 - at.c0;
      const uint64_t src_step = static_cast<uint64_t>(groups) * src_h;
      const bool paged = APPEND && kind != 0, copies = APPEND && (plain || kind == 2);
      const uint32_t dst_h = paged ? static_cast<uint32_t>(p.head_s) : out_h;
      const uint64_t dst_step = static_cast<uint64_t>(groups) * dst_h;
      uint16_t *dst = static_cast<uint16_t *>(paged ? (kind == 1 ? p.k_pages : p.v_pages) : kind == 0 ? p.q_out : p.k_out) +
                      static_cast<uint64_t>(h0) * dst_h + at.c0;
      if (!paged) dst += static_cast<long long>(tok.b) * heads * out_h + static_cast<long long>(tok.l) * p.d;
      bool placed = !paged;
      for (; s < end; ++s, h0 += per) {
        const int rows_here = tok.in && h0 < heads ? min(p.at_once, (heads - h0 + groups - 1) / groups) : 0;  // of this thread
        Vec<E> a[U], b[U];
        if (__all_sync(0xffffffffu, reads && rows_here == U)) {
#pragma unroll
          for (int i = 0; i < U; ++i, src += src_step) {
            a[i] = load_vec<E>(src);
            b[i] = load_vec<E>(src + over);
          }
        } else {
#pragma unroll
          for (int i = 0; i < U; ++i) {
            a[i] = b[i] = zero_vec<E>();
            if (reads && i < rows_here) {
              a[i] = load_vec<E>(src + i * src_step);
              b[i] = load_vec<E>(src + i * src_step + over);
            }
          }
          src += p.at_once * src_step;
        }
        if (fresh) {  // the same in every thread
          fresh = false;
          __syncthreads();  // the tile before is done with the tables
          if (threadIdx.x < p.tokens) {
            const Token t = token_of(p, n0 + threadIdx.x);
            int x = 0;
            if constexpr (!APPEND) {
              if (t.in) x = p.positions ? p.positions[t.b * p.pos_s + t.l] : t.l;
            } else {
              long long cl = -2;
              if (t.in) {
                const int len = p.lengths[t.b], count = p.counts ? p.counts[t.b] : p.L;
                if (count < 0 || count > p.L || len < count || len > static_cast<long long>(p.table_w) * p.page) {
                  atomicCAS(p.status, 0u, kDevBadLength);
                } else if (t.l < count) {
                  x = len - count + t.l;
                  const int index = x / p.page, page = p.table[t.b * p.table_s + index];
                  cl = -1;
                  if (page < 0 || page >= p.pages)
                    atomicCAS(p.status, 0u, kDevBadPage);
                  else
                    cl = page * p.page_s + static_cast<long long>(x - index * p.page) * p.slot_s;
                }
              }
              cell[threadIdx.x] = cl;
            }
            pos[threadIdx.x] = x;
          }
          __syncthreads();
          if (p.rotary > 0) {
            fill_turns(turns, pos, freq, p);
            __syncthreads();
          }
          load_turns<E>(turns, token, p.rotary, at, turn);
          if constexpr (APPEND) to = cell[token];
        }
        if (!placed) {
          placed = true;
          dst += max(to, 0LL);
        }
        const bool clears = APPEND && kind == 0 && to == -2;
        const int stored = paged && to < 0 ? 0 : rows_here;
        if (copies || clears) {
#pragma unroll
          for (int i = 0; i < U; ++i)
            if (i < stored) {
              store_vec<E>(dst + i * dst_step, clears ? zero_vec<E>() : a[i]);
              store_vec<E>(dst + i * dst_step + over, clears ? zero_vec<E>() : b[i]);
            }
        }
        if constexpr (NORM) {
          if (!copies) {  // the same in every thread: the shuffles need whole rows
            Pairs<E> x[U];
#pragma unroll
            for (int i = 0; i < U; ++i) unpack<BF, INTER, E>(a[i], b[i], x[i]);
            Pairs<E> w;
            weight_pairs<E>(weights + (kind == 0 ? 0 : p.d), at.lane, w);
            float ss[U];
#pragma unroll
            for (int i = 0; i < U; ++i) ss[i] = lane_dot<E>(x[i], x[i]);
            for (int o = 1; o < lpr; o <<= 1)
#pragma unroll
              for (int i = 0; i < U; ++i) ss[i] += __shfl_xor_sync(0xffffffffu, ss[i], o);
#pragma unroll
            for (int i = 0; i < U; ++i) {
              const float rstd = rsqrtf(ss[i] * inv_d + p.eps);
              const uint64_t r = f32x2(rstd, rstd);
#pragma unroll
              for (int e = 0; e < E / 4; ++e) {
                x[i].A[e] = fmul2(fmul2(x[i].A[e], r), w.A[e]);
                x[i].B[e] = fmul2(fmul2(x[i].B[e], r), w.B[e]);
              }
            }
            if (at.turns)
#pragma unroll
              for (int i = 0; i < U; ++i) turn_pairs<E>(x[i], turn);
            const int out = clears ? 0 : stored;
            uint16_t *row = dst;
#pragma unroll
            for (int i = 0; i < U; ++i, row += dst_step)
              if (i < out) store_row<BF, INTER, E>(row, over, x[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < U; ++i)
            if (i < (clears || copies ? 0 : stored)) {
              Pairs<E> x;
              unpack<BF, INTER, E>(a[i], b[i], x);
              if (at.turns) turn_pairs<E>(x, turn);
              store_row<BF, INTER, E>(dst + i * dst_step, over, x);
            }
        }
        dst += p.at_once * dst_step;
      }
    }
  }
}

// The backward pass with norms.  With dy the upstream gradient turned back, xh = x rstd and
// g = dy w:   dx = rstd (g - xh mean(g xh)),   dw += dy xh.  Each block leaves its part of the
// weights' gradients in parts[block][q, k][d], which rope_dw_kernel adds up in a fixed order.
template <bool BF, bool INTER, int E>
__global__ void __launch_bounds__(kRopeThreads, kBwdResident) rope_bwd_kernel(const RopeParams p) {
  constexpr int U = kBwdAtOnce<E>;
  extern __shared__ __align__(16) float2 turns[];
  __shared__ int pos[kRopeMaxTokens];
  __shared__ Frequencies freq;
  __shared__ __align__(16) float weights[1024];
  __shared__ float sums[2][E][kRopeThreads];  // each thread's part of q's and k's weight gradients
  grid_launch_dependents();
  grid_wait_prior();
  const int lpr = p.d / E, groups = kRopeThreads / lpr / p.tokens;
  const Place at = place_of<INTER, E>(p, lpr);
  const int row = threadIdx.x / lpr, token = row / groups, group = row - token * groups;
  const uint32_t out_h = static_cast<uint32_t>(p.L) * static_cast<uint32_t>(p.d);
  const float inv_d = 1.f / static_cast<float>(p.d);
  fill_weights<BF, INTER, E>(weights, p);
  fill_frequencies(freq, p);
  Pairs<E> dw;  // of the tensor that the steps are in
  auto add_up = [&](int which) {
#pragma unroll
    for (int e = 0; e < E / 4; ++e) {
      float f[4];
      f32x2_split(dw.A[e], f[0], f[1]);
      f32x2_split(dw.B[e], f[2], f[3]);
      sums[which][2 * e][threadIdx.x] += f[0];
      sums[which][2 * e + 1][threadIdx.x] += f[1];
      sums[which][E / 2 + 2 * e][threadIdx.x] += f[2];
      sums[which][E / 2 + 2 * e + 1][threadIdx.x] += f[3];
      dw.A[e] = dw.B[e] = 0ull;  // pairs of 0.0f
    }
  };
#pragma unroll
  for (int e = 0; e < E; ++e) sums[0][e][threadIdx.x] = sums[1][e][threadIdx.x] = 0.f;
#pragma unroll
  for (int e = 0; e < E / 4; ++e) dw.A[e] = dw.B[e] = 0ull;
  const int per = groups * p.at_once, over = at.c1 - at.c0;
  auto rows_of_step = [&](int heads, int i) { return min(p.at_once, (heads - i * per + groups - 1) / groups); };  // of group 0, the most
  const uint64_t out_step = static_cast<uint64_t>(groups) * out_h;
  for (Units u = units_of(p); u.left > 0; u.step = 0, ++u.tile) {  // a tile
    const int n0 = u.tile * p.tokens, stop = min(p.steps, u.step + u.left);
    u.left -= stop - u.step;
    const Token tok = token_of(p, n0 + token);
    bool fresh = true;
    Turn<E> turn;
    for (int s = u.step; s < stop;) {  // its steps of one tensor
      const bool is_q = s < p.steps_q;
      const int heads = is_q ? p.Hq : p.Hkv, first = is_q ? 0 : p.steps_q, end = min(stop, first + (is_q ? p.steps_q : p.steps_k));
      int h0 = (s - first) * per + group;
      const uint32_t x_h = static_cast<uint32_t>(is_q ? p.qs[1] : p.ks[1]), up_h = static_cast<uint32_t>(is_q ? p.dqs[1] : p.dks[1]);
      const uint16_t *src = row_at(is_q ? p.q : p.k, tok, is_q ? p.qs[0] : p.ks[0], is_q ? p.qs[2] : p.ks[2]) +
                            static_cast<uint64_t>(h0) * x_h + at.c0;
      const uint16_t *up = row_at(is_q ? p.dq : p.dk, tok, is_q ? p.dqs[0] : p.dks[0], is_q ? p.dqs[2] : p.dks[2]) +
                           static_cast<uint64_t>(h0) * up_h + at.c0;
      const uint64_t step = static_cast<uint64_t>(groups) * x_h, up_step = static_cast<uint64_t>(groups) * up_h;
      uint16_t *dst = static_cast<uint16_t *>(is_q ? p.q_out : p.k_out) + static_cast<long long>(tok.b) * heads * out_h +
                      static_cast<long long>(tok.l) * p.d + static_cast<uint64_t>(h0) * out_h + at.c0;
      for (; s < end; ++s, h0 += per, dst += p.at_once * out_step) {
        const int rows_here = tok.in && h0 < heads ? min(p.at_once, (heads - h0 + groups - 1) / groups) : 0;  // of this thread
        Vec<E> a[U], b[U], da[U], db[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          a[i] = b[i] = da[i] = db[i] = zero_vec<E>();
          if (i < rows_here) {
            a[i] = load_vec<E>(src + i * step);
            b[i] = load_vec<E>(src + i * step + over);
            da[i] = load_vec<E>(up + i * up_step);
            db[i] = load_vec<E>(up + i * up_step + over);
          }
        }
        src += p.at_once * step;
        up += p.at_once * up_step;
        if (fresh) {
          fresh = false;
          __syncthreads();
          if (threadIdx.x < p.tokens) {
            const Token t = token_of(p, n0 + threadIdx.x);
            pos[threadIdx.x] = !t.in ? 0 : p.positions ? p.positions[t.b * p.pos_s + t.l] : t.l;
          }
          __syncthreads();
          if (p.rotary > 0) {
            fill_turns(turns, pos, freq, p);
            __syncthreads();
          }
          load_turns<E>(turns, token, p.rotary, at, turn);
        }
        on_rows<U>(rows_of_step(heads, s - first), [&](auto rows) {
          constexpr int R = rows.value;
          Pairs<E> w;
          weight_pairs<E>(weights + (is_q ? 0 : p.d), at.lane, w);
          uint16_t *row = dst;
          Pairs<E> g[R];
          float ss[R], gx[R];
#pragma unroll
          for (int i = 0; i < R; ++i) unpack<BF, INTER, E>(da[i], db[i], g[i]);
          if (at.turns)
#pragma unroll
            for (int i = 0; i < R; ++i) turn_pairs<E>(g[i], turn);
#pragma unroll
          for (int i = 0; i < R; ++i) {
            Pairs<E> x, gw;
            unpack<BF, INTER, E>(a[i], b[i], x);
#pragma unroll
            for (int e = 0; e < E / 4; ++e) {
              gw.A[e] = fmul2(g[i].A[e], w.A[e]);
              gw.B[e] = fmul2(g[i].B[e], w.B[e]);
            }
            ss[i] = lane_dot<E>(x, x);
            gx[i] = lane_dot<E>(gw, x);
          }
          for (int o = 1; o < lpr; o <<= 1)
#pragma unroll
            for (int i = 0; i < R; ++i) {
              ss[i] += __shfl_xor_sync(0xffffffffu, ss[i], o);
              gx[i] += __shfl_xor_sync(0xffffffffu, gx[i], o);
            }
#pragma unroll
          for (int i = 0; i < R; ++i, row += out_step) {
            const float rstd = i < rows_here ? rsqrtf(ss[i] * inv_d + p.eps) : 0.f;  // (infinite for a row of zeros without eps)
            const float mean = gx[i] * rstd * inv_d;  // mean(g xh)
            const uint64_t r = f32x2(rstd, rstd), m = f32x2(-mean, -mean);
            Pairs<E> x;  // unpacked again: a register for a word rather than two
#pragma unroll
            for (int e = 0; e < E / 4; ++e) asm volatile("" : "+r"(a[i].w[e]), "+r"(b[i].w[e]));
            unpack<BF, INTER, E>(a[i], b[i], x);
#pragma unroll
            for (int e = 0; e < E / 4; ++e) {
              const uint64_t ha = fmul2(x.A[e], r), hb = fmul2(x.B[e], r);
              dw.A[e] = ffma2(g[i].A[e], ha, dw.A[e]);
              dw.B[e] = ffma2(g[i].B[e], hb, dw.B[e]);
              x.A[e] = fmul2(r, ffma2(ha, m, fmul2(g[i].A[e], w.A[e])));
              x.B[e] = fmul2(r, ffma2(hb, m, fmul2(g[i].B[e], w.B[e])));
            }
            if (i < rows_here) store_row<BF, INTER, E>(row, over, x);
          }
        });
      }
      add_up(is_q ? 0 : 1);
    }
  }
  __syncthreads();
  // Lane j's element e (A's, then B's) of every row of threads.
  float *const part = p.parts + static_cast<size_t>(blockIdx.x) * 2 * p.d;
  for (int i = threadIdx.x; i < 2 * p.d; i += kRopeThreads) {
    const int which = i >= p.d, k = i - which * p.d, j = k / E, e = k % E, r = e % (E / 2), half = e / (E / 2);
    float t = 0.f;
    for (int row_of = 0; row_of < kRopeThreads; row_of += lpr) t += sums[which][e][row_of + j];
    const bool split = !INTER && j < p.rotary / E;
    part[which * p.d + (split ? half * (p.rotary >> 1) + E / 2 * j + r : INTER ? E * j + 2 * r + half : E * j + e)] = t;
  }
}

// dw[which][i] = sum over parts; one block per (which, 16 columns), 16 x 64 threads.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float *parts, int n, int d, float *dq_w, float *dk_w) {
  __shared__ float red[64][17];
  grid_launch_dependents();
  grid_wait_prior();
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4, which = blockIdx.y, col = blockIdx.x * 16 + x;
  float t = 0.f;
#pragma unroll 8
  for (int r = y; r < n; r += 64) t += parts[(static_cast<size_t>(r) * 2 + which) * d + col];
  red[y][x] = t;
  __syncthreads();
  if (threadIdx.x < 512) {  // a warp to a column
    const int lane = threadIdx.x & 31, c = threadIdx.x >> 5;
    t = red[lane][c] + red[lane + 32][c];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0) (which ? dk_w : dq_w)[blockIdx.x * 16 + c] = t;
  }
}

template <typename... A>
cudaError_t launch(void (*kern)(A...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// The units.  A tile's angles are computed by every block that has a unit of it, so a tile gets
// as many tokens (a power of two) as leave each of `blocks` blocks about one tile (one token a
// tile took 19.4 us for norm and rotation of 1 x 40 x 2048 x 128 on GB300, four 16.6), but no fewer
// than four, whose angles one pass of the block's threads computes anyway, and no more than
// kRopeMaxTokens (a head's rows of neighbouring tokens are written together: 32 rows of d = 64
// are 4 KB; 100003 x 32 x 64 136.6 us, with 16 tokens 142.2).  Fewer rows a thread where that
// leaves blocks without a unit.  Returns the blocks to launch.
int plan(RopeParams &p, bool append, int blocks, int at_once) {
  const long long N = static_cast<long long>(p.B) * p.L;
  const int rows = kRopeThreads / (p.d > 256 ? p.d / 16 : p.d / 8);
  const int most = std::min(kRopeMaxTokens, rows);
  p.tokens = 1;
  while (2 * p.tokens <= most && (2LL * p.tokens * blocks <= N || (p.tokens < 4 && p.tokens < N))) p.tokens *= 2;
  for (p.at_once = at_once;; p.at_once >>= 1) {
    const int per = rows / p.tokens * p.at_once;
    p.steps_q = (p.Hq + per - 1) / per;
    p.steps_k = (p.Hkv + per - 1) / per;
    p.steps = p.steps_q + (append ? 2 : 1) * p.steps_k;
    p.units = (N + p.tokens - 1) / p.tokens * p.steps;
    if (p.at_once == 1 || p.units >= blocks) break;
  }
  return static_cast<int>(std::min<long long>(p.units, blocks));
}

size_t turns_bytes(const RopeParams &p) { return p.rotary ? static_cast<size_t>(p.tokens) * turns_row(p.rotary) * sizeof(float2) : 0; }

// Shared memory of a block: the kernels' own arrays (backward: by the elements a lane), and the longest table that
// plan() can ask for at head_dim d.  Up to 48 KB of both together need no asking.
constexpr int kOwnBytes = kRopeMaxTokens * (4 + 8) + static_cast<int>(sizeof(Frequencies)) + 1024 * 4;  // rope_kernel, at most
template <int E>
constexpr int kBwdOwnBytes = kRopeMaxTokens * 4 + static_cast<int>(sizeof(Frequencies)) + 1024 * 4 + 2 * E * kRopeThreads * 4;
constexpr int most_turns(int d) {
  const int rows = kRopeThreads / (d > 256 ? d / 16 : d / 8);
  return (rows < kRopeMaxTokens ? rows : kRopeMaxTokens) * turns_row(d) * static_cast<int>(sizeof(float2));
}
constexpr int kSmemUnasked = 48 * 1024, kSmemSm = 228 * 1024;  // of an SM, 1 KB a block kept by the system
template <int E>
constexpr bool fits_unasked(int d) {
  return kOwnBytes + most_turns(d) <= kSmemUnasked && (E == 16 || kBwdOwnBytes<E> + most_turns(d) <= kSmemUnasked);
}
static_assert(fits_unasked<8>(64) && fits_unasked<8>(128) && fits_unasked<8>(256) && fits_unasked<16>(512), "launches without asking");
static_assert(kBwdResident * (kBwdOwnBytes<16> + most_turns(512) + 1024) <= kSmemSm, "the backward pass at 512");

// The instance for a call's type, norm, layout and head_dim.
template <bool APPEND>
auto pick(bool bf, bool norm, bool inter, int d) {
#define ROPE_PICK(E)                                                                                                         \
  (bf ? (norm ? (inter ? rope_kernel<true, true, true, E, APPEND> : rope_kernel<true, true, false, E, APPEND>)               \
              : (inter ? rope_kernel<true, false, true, E, APPEND> : rope_kernel<true, false, false, E, APPEND>))            \
      : (norm ? (inter ? rope_kernel<false, true, true, E, APPEND> : rope_kernel<false, true, false, E, APPEND>)             \
              : (inter ? rope_kernel<false, false, true, E, APPEND> : rope_kernel<false, false, false, E, APPEND>)))
  return d > 256 ? ROPE_PICK(16) : ROPE_PICK(8);
#undef ROPE_PICK
}
auto pick_bwd(bool bf, bool inter, int d) {
#define ROPE_PICK(E)                                                                   \
  (bf ? (inter ? rope_bwd_kernel<true, true, E> : rope_bwd_kernel<true, false, E>)     \
      : (inter ? rope_bwd_kernel<false, true, E> : rope_bwd_kernel<false, false, E>))
  return d > 256 ? ROPE_PICK(16) : ROPE_PICK(8);
#undef ROPE_PICK
}

template <bool APPEND>
cudaError_t launch_rows(RopeLaunch &a) {
  const bool norm = a.p.q_w != nullptr || a.p.k_w != nullptr, wide = a.p.d > 256;
  const int grid = plan(a.p, APPEND, a.sm_count * (wide ? kResident<16> : kResident<8>), wide ? kAtOnce<16> : kAtOnce<8>);
  return launch(pick<APPEND>(a.bf16, norm, a.interleaved, a.p.d), dim3(grid), kRopeThreads, turns_bytes(a.p), a.stream, RopeParams(a.p));
}

}  // namespace

cudaError_t launch_rope(RopeLaunch &a) { return launch_rows<false>(a); }
cudaError_t launch_append(RopeLaunch &a) { return launch_rows<true>(a); }

cudaError_t launch_rope_bwd(RopeLaunch &a) {
  const bool wide = a.p.d > 256;
  const int blocks = a.sm_count * kBwdResident;
  const int grid = plan(a.p, false, std::min(kRopeMaxParts, blocks), wide ? kBwdAtOnce<16> : kBwdAtOnce<8>);
  auto *const kern = pick_bwd(a.bf16, a.interleaved, a.p.d);
  cudaError_t e = cudaSuccess;
  // Eight tokens of 288 rotated elements and more at 512: up to 55 KB with the kernel's own.  Always asked for as the
  // most, so that calls of two host threads do not take it from one another.
  if (wide && kBwdOwnBytes<16> + turns_bytes(a.p) > kSmemUnasked)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most_turns(512));
  if (e != cudaSuccess) return e;
  e = launch(kern, dim3(grid), kRopeThreads, turns_bytes(a.p), a.stream, RopeParams(a.p));
  if (e != cudaSuccess) return e;
  return launch(rope_dw_kernel, dim3(a.p.d / 16, a.p.k_w ? 2 : 1), 1024, 0, a.stream, static_cast<const float *>(a.p.parts), grid, a.p.d,
                a.p.dq_w, a.p.dk_w);
}

}  // namespace gbattn
