// rope.cu -- rotary positions, per-head norms and the paged append: kernels and launches.
//
// Every kernel is one pass over its rows and bound by their reads and writes.  A row of d
// elements belongs to d / 16 consecutive lanes (4, 8, 16, 32 for d = 64, 128, 256, 512); a
// lane holds two 16-byte vectors that contain both halves of every pair it turns, so that
// neither layout needs an exchange between lanes:
//     half layout, lane j < rotary / 16:  elements 8j .. 8j+7 and rotary/2 + 8j .. +7
//     otherwise (interleaved, and the elements behind `rotary`):  16j .. 16j+15
// and in both layouts lane j turns its pairs by the angles 8j .. 8j+7.  The norm's sum of
// squares is a shuffle reduction over the row's lanes.
// A block takes `tokens` consecutive (batch, row) positions; their cosines and sines are
// computed once, into shared memory, and each thread keeps the eight that it needs in
// registers while it walks over the heads of its token.
//
// Angles: position x inv_freq is reduced in integers.  inv_freq / 2 pi becomes a 64-bit
// binary fraction of a turn; its product with the position, taken modulo 2^64, is the angle
// modulo one turn, wrong by at most (1 + inv_freq / 4) |position| 2^-64 turns (so a position
// of 10^6 costs no accuracy, where an fp32 product would be off by 0.06 radians).
#include <algorithm>

#include "ptx.cuh"
#include "rope.cuh"
#include "vec16.cuh"

namespace gbattn {
namespace {

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

// factor * (cos, sin) of position * freq
__device__ __forceinline__ float2 turn_of(int position, double freq, float factor, float sign) {
  const int64_t turn = static_cast<int64_t>(static_cast<uint64_t>(static_cast<int64_t>(position)) * turns_fixed(freq));
  float s, c;
  sincospif(static_cast<float>(turn) * 0x1p-63f, &s, &c);
  const bool bad = (static_cast<uint64_t>(__double_as_longlong(freq)) & 0x7ff0000000000000ull) == 0x7ff0000000000000ull;
  return bad ? make_float2(NAN, NAN) : make_float2(factor * c, sign * factor * s);
}

struct Place {       // where a thread works
  int c0, c1;        // first elements of its two vectors
  bool turns;        // whether its pairs are turned
  int lane;          // lane j within the row
};

template <bool INTER>
__device__ __forceinline__ Place place_of(const RopeParams &p, int lpr) {
  Place r;
  r.lane = threadIdx.x & (lpr - 1);
  r.turns = r.lane < (p.rotary >> 4);
  const bool split = !INTER && r.turns;
  r.c0 = split ? 8 * r.lane : 16 * r.lane;
  r.c1 = split ? 8 * r.lane + (p.rotary >> 1) : 16 * r.lane + 8;
  return r;
}

__device__ __forceinline__ float row_sum(float x, int lpr) {
  for (int o = 1; o < lpr; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Turn the pairs of (x0, x1) in place; e-th pair by (c[e], s[e]).
template <bool INTER>
__device__ __forceinline__ void turn_pairs(float *x, const float *c, const float *s) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = INTER ? 2 * e : e, j = INTER ? 2 * e + 1 : e + 8;
    const float a = x[i], b = x[j];
    x[i] = a * c[e] - b * s[e];
    x[j] = b * c[e] + a * s[e];
  }
}

__device__ __forceinline__ uint4 load16(const uint16_t *p) { return __ldg(reinterpret_cast<const uint4 *>(p)); }
__device__ __forceinline__ void store16(uint16_t *p, uint4 v) { *reinterpret_cast<uint4 *>(p) = v; }

constexpr int kHeadsAtOnce = 4;  // rows a thread loads before it works on the first

// Rows of heads [h0, h1) of one tensor at one token: norm, turn, store.  Every thread of the
// block runs the same number of steps (the shuffles need whole rows).
template <bool BF, bool NORM, bool INTER>
__device__ __forceinline__ void rope_heads(const uint16_t *src, long long src_h, uint16_t *dst, long long dst_h, int h0,
                                           int h1, int group, int groups, bool valid, const Place &at, int lpr,
                                           const float *c, const float *s, const uint16_t *weight, float eps, float inv_d) {
  if (h0 >= h1) return;
  float w[16];
  if constexpr (NORM) {
    vec_unpack<BF>(load16(weight + at.c0), w);
    vec_unpack<BF>(load16(weight + at.c1), w + 8);
  }
  for (int base = h0; base < h1; base += groups * kHeadsAtOnce) {
    uint4 a[kHeadsAtOnce], b[kHeadsAtOnce];
#pragma unroll
    for (int u = 0; u < kHeadsAtOnce; ++u) {
      const int h = base + u * groups + group;
      a[u] = b[u] = make_uint4(0, 0, 0, 0);
      if (valid && h < h1) {
        a[u] = load16(src + h * src_h + at.c0);
        b[u] = load16(src + h * src_h + at.c1);
      }
    }
#pragma unroll
    for (int u = 0; u < kHeadsAtOnce; ++u) {
      const int h = base + u * groups + group;
      float x[16];
      vec_unpack<BF>(a[u], x);
      vec_unpack<BF>(b[u], x + 8);
      if constexpr (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
        const float rstd = rsqrtf(row_sum(ss, lpr) * inv_d + eps);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = x[e] * rstd * w[e];
      }
      if (at.turns) turn_pairs<INTER>(x, c, s);
      if (valid && h < h1) {
        store16(dst + h * dst_h + at.c0, vec_pack<BF>(x));
        store16(dst + h * dst_h + at.c1, vec_pack<BF>(x + 8));
      }
    }
  }
}

// Fill the block's table of cosines and sines: entry [token][r].
__device__ __forceinline__ void fill_turns(float2 *table, const int *pos, const RopeParams &p) {
  const int half = p.rotary >> 1;
  for (int i = threadIdx.x; i < p.tokens * half; i += kRopeThreads)
    table[i] = turn_of(pos[i / half], __ldg(p.inv_freq + i % half), p.factor, p.sign);
}
__device__ __forceinline__ void load_turns(const float2 *table, int token, const Place &at, const RopeParams &p, float *c,
                                           float *s) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 t = at.turns ? table[token * (p.rotary >> 1) + 8 * at.lane + e] : make_float2(1.f, 0.f);
    c[e] = t.x;
    s[e] = t.y;
  }
}

template <bool BF, bool NORM, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  extern __shared__ float2 turns[];
  __shared__ int pos[kRopeMaxTokens];
  grid_launch_dependents();
  grid_wait_prior();
  const int lpr = p.d >> 4, rows = kRopeThreads / lpr, groups = rows / p.tokens;
  const long long n0 = static_cast<long long>(blockIdx.x) * p.tokens, N = static_cast<long long>(p.B) * p.L;
  if (threadIdx.x < p.tokens) {
    const long long n = n0 + threadIdx.x;
    int x = 0;
    if (n < N) x = p.positions ? p.positions[(n / p.L) * p.pos_s + n % p.L] : static_cast<int>(n % p.L);
    pos[threadIdx.x] = x;
  }
  __syncthreads();
  fill_turns(turns, pos, p);
  __syncthreads();
  const Place at = place_of<INTER>(p, lpr);
  const int row = threadIdx.x / lpr, token = row / groups, group = row - token * groups;
  float c[8], s[8];
  load_turns(turns, token, at, p, c, s);
  const long long n = n0 + token;
  const bool valid = n < N;
  const long long b = valid ? n / p.L : 0, l = valid ? n % p.L : 0;
  const int h0 = blockIdx.y * p.heads_per_block, h1 = min(p.Hq + p.Hkv, h0 + p.heads_per_block);
  const float inv_d = 1.f / static_cast<float>(p.d);
  const long long out_h = static_cast<long long>(p.L) * p.d;
  rope_heads<BF, NORM, INTER>(static_cast<const uint16_t *>(p.q) + b * p.qs[0] + l * p.qs[2], p.qs[1],
                              static_cast<uint16_t *>(p.q_out) + b * p.Hq * out_h + l * p.d, out_h, h0, min(h1, p.Hq), group,
                              groups, valid, at, lpr, c, s, static_cast<const uint16_t *>(p.q_w), p.eps, inv_d);
  rope_heads<BF, NORM, INTER>(static_cast<const uint16_t *>(p.k) + b * p.ks[0] + l * p.ks[2], p.ks[1],
                              static_cast<uint16_t *>(p.k_out) + b * p.Hkv * out_h + l * p.d, out_h, max(h0 - p.Hq, 0),
                              h1 - p.Hq, group, groups, valid, at, lpr, c, s, static_cast<const uint16_t *>(p.k_w), p.eps, inv_d);
}

// The append: sequence b's new tokens are counts[b] rows (all L without counts) at positions
// lengths[b] - counts[b] .. lengths[b] - 1; their keys (turned when rotary > 0) and values go
// to the pages that the table names, their queries to q_out (zeros behind the last token).
template <bool BF, bool NORM, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) append_kernel(const RopeParams p) {
  extern __shared__ float2 turns[];
  __shared__ int pos[kRopeMaxTokens];
  __shared__ long long cell[kRopeMaxTokens];  // element offset of the token's page slot, -1: none, -2: behind the last token
  grid_launch_dependents();
  grid_wait_prior();
  const int lpr = p.d >> 4, rows = kRopeThreads / lpr, groups = rows / p.tokens;
  const long long n0 = static_cast<long long>(blockIdx.x) * p.tokens, N = static_cast<long long>(p.B) * p.L;
  if (threadIdx.x < p.tokens) {
    const long long n = n0 + threadIdx.x;
    int x = 0;
    long long at = -2;
    if (n < N) {
      const long long b = n / p.L;
      const int t = static_cast<int>(n % p.L);
      const int len = p.lengths[b], count = p.counts ? p.counts[b] : p.L;
      if (count < 0 || count > p.L || len < count || len > static_cast<long long>(p.table_w) * p.page) {
        atomicCAS(p.status, 0u, kDevBadLength);
      } else if (t < count) {
        x = len - count + t;
        const int page = p.table[b * p.table_s + x / p.page];
        at = -1;
        if (page < 0 || page >= p.pages)
          atomicCAS(p.status, 0u, kDevBadPage);
        else
          at = page * p.page_s + static_cast<long long>(x % p.page) * p.slot_s;
      }
    }
    pos[threadIdx.x] = x;
    cell[threadIdx.x] = at;
  }
  __syncthreads();
  fill_turns(turns, pos, p);
  __syncthreads();
  const Place at = place_of<INTER>(p, lpr);
  const int row = threadIdx.x / lpr, token = row / groups, group = row - token * groups;
  float c[8], s[8];
  load_turns(turns, token, at, p, c, s);
  const long long n = n0 + token, to = cell[token];
  const bool in = n < N;
  const long long b = in ? n / p.L : 0, l = in ? n % p.L : 0;
  const int h0 = blockIdx.y * p.heads_per_block, h1 = min(p.Hq + 2 * p.Hkv, h0 + p.heads_per_block);
  const float inv_d = 1.f / static_cast<float>(p.d);
  if (p.Hq) {
    const long long out_h = static_cast<long long>(p.L) * p.d;
    uint16_t *const out = static_cast<uint16_t *>(p.q_out) + b * p.Hq * out_h + l * p.d;
    const int e1 = min(h1, p.Hq);
    if (in && to == -2)
      for (int h = h0 + group; h < e1; h += groups) {
        store16(out + h * out_h + at.c0, make_uint4(0, 0, 0, 0));
        store16(out + h * out_h + at.c1, make_uint4(0, 0, 0, 0));
      }
    rope_heads<BF, NORM, INTER>(static_cast<const uint16_t *>(p.q) + b * p.qs[0] + l * p.qs[2], p.qs[1], out, out_h, h0, e1,
                                group, groups, in && to != -2, at, lpr, c, s, static_cast<const uint16_t *>(p.q_w), p.eps, inv_d);
  }
  const bool valid = in && to >= 0;
  const int k0 = max(h0 - p.Hq, 0), k1 = min(h1 - p.Hq, p.Hkv);
  const int v0 = max(h0 - p.Hq - p.Hkv, 0), v1 = h1 - p.Hq - p.Hkv;
  const uint16_t *const ksrc = static_cast<const uint16_t *>(p.k) + b * p.ks[0] + l * p.ks[2];
  const uint16_t *const vsrc = static_cast<const uint16_t *>(p.v) + b * p.vs[0] + l * p.vs[2];
  uint16_t *const kdst = static_cast<uint16_t *>(p.k_pages) + (valid ? to : 0);
  uint16_t *const vdst = static_cast<uint16_t *>(p.v_pages) + (valid ? to : 0);
  if (NORM || p.rotary) {
    rope_heads<BF, NORM, INTER>(ksrc, p.ks[1], kdst, p.head_s, k0, k1, group, groups, valid, at, lpr, c, s,
                                static_cast<const uint16_t *>(p.k_w), p.eps, inv_d);
  } else if (valid) {
    for (int h = k0 + group; h < k1; h += groups) {
      store16(kdst + h * p.head_s + at.c0, load16(ksrc + h * p.ks[1] + at.c0));
      store16(kdst + h * p.head_s + at.c1, load16(ksrc + h * p.ks[1] + at.c1));
    }
  }
  if (valid)
    for (int h = v0 + group; h < v1; h += groups) {
      store16(vdst + h * p.head_s + at.c0, load16(vsrc + h * p.vs[1] + at.c0));
      store16(vdst + h * p.head_s + at.c1, load16(vsrc + h * p.vs[1] + at.c1));
    }
}

// Backward rows of heads [h0, h1): with dy the upstream gradient turned back, xh = x rstd and
// g = dy w,   dx = rstd (g - xh mean(g xh)),   dw += dy xh  (this thread's 16 columns).
template <bool BF, bool INTER>
__device__ __forceinline__ void rope_heads_bwd(const uint16_t *dz, long long dz_h, const uint16_t *src, long long src_h,
                                               uint16_t *dst, long long dst_h, int h0, int h1, int group, int groups,
                                               bool valid, const Place &at, int lpr, const float *c, const float *s,
                                               const uint16_t *weight, float eps, float inv_d, float *dw) {
  if (h0 >= h1) return;
  float w[16];
  vec_unpack<BF>(load16(weight + at.c0), w);
  vec_unpack<BF>(load16(weight + at.c1), w + 8);
  constexpr int U = 2;
  for (int base = h0; base < h1; base += groups * U) {
    uint4 a[U], b[U], da[U], db[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = base + u * groups + group;
      a[u] = b[u] = da[u] = db[u] = make_uint4(0, 0, 0, 0);
      if (valid && h < h1) {
        a[u] = load16(src + h * src_h + at.c0);
        b[u] = load16(src + h * src_h + at.c1);
        da[u] = load16(dz + h * dz_h + at.c0);
        db[u] = load16(dz + h * dz_h + at.c1);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = base + u * groups + group;
      float x[16], g[16];
      vec_unpack<BF>(a[u], x);
      vec_unpack<BF>(b[u], x + 8);
      vec_unpack<BF>(da[u], g);
      vec_unpack<BF>(db[u], g + 8);
      if (at.turns) turn_pairs<INTER>(g, c, s);
      float ss = 0.f, gx = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        ss = fmaf(x[e], x[e], ss);
        gx = fmaf(g[e] * w[e], x[e], gx);
      }
      ss = row_sum(ss, lpr);
      gx = row_sum(gx, lpr);
      const float rstd = rsqrtf(ss * inv_d + eps);
      const float mean = gx * rstd * inv_d;  // mean(g xh)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float xh = x[e] * rstd;
        dw[e] = fmaf(g[e], xh, dw[e]);
        x[e] = rstd * (g[e] * w[e] - xh * mean);
      }
      if (valid && h < h1) {
        store16(dst + h * dst_h + at.c0, vec_pack<BF>(x));
        store16(dst + h * dst_h + at.c1, vec_pack<BF>(x + 8));
      }
    }
  }
}

// Blocks walk over token tiles; each leaves its part of the weights' gradients in
// parts[block][q, k][d], which rope_dw_kernel adds up in a fixed order.
template <bool BF, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_bwd_kernel(const RopeParams p) {
  extern __shared__ float2 turns[];
  __shared__ int pos[kRopeMaxTokens];
  __shared__ float red[8][512];
  grid_launch_dependents();
  grid_wait_prior();
  const int lpr = p.d >> 4, rows = kRopeThreads / lpr, groups = rows / p.tokens;
  const long long N = static_cast<long long>(p.B) * p.L;
  const Place at = place_of<INTER>(p, lpr);
  const int row = threadIdx.x / lpr, token = row / groups, group = row - token * groups;
  const int h0 = blockIdx.y * p.heads_per_block, h1 = min(p.Hq + p.Hkv, h0 + p.heads_per_block);
  const float inv_d = 1.f / static_cast<float>(p.d);
  const long long out_h = static_cast<long long>(p.L) * p.d;
  float dwq[16], dwk[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) dwq[e] = dwk[e] = 0.f;
  for (long long n0 = static_cast<long long>(blockIdx.x) * p.tokens; n0 < N; n0 += static_cast<long long>(gridDim.x) * p.tokens) {
    __syncthreads();
    if (threadIdx.x < p.tokens) {
      const long long n = n0 + threadIdx.x;
      int x = 0;
      if (n < N) x = p.positions ? p.positions[(n / p.L) * p.pos_s + n % p.L] : static_cast<int>(n % p.L);
      pos[threadIdx.x] = x;
    }
    __syncthreads();
    fill_turns(turns, pos, p);
    __syncthreads();
    float c[8], s[8];
    load_turns(turns, token, at, p, c, s);
    const long long n = n0 + token;
    const bool valid = n < N;
    const long long b = valid ? n / p.L : 0, l = valid ? n % p.L : 0;
    rope_heads_bwd<BF, INTER>(static_cast<const uint16_t *>(p.dq) + b * p.dqs[0] + l * p.dqs[2], p.dqs[1],
                              static_cast<const uint16_t *>(p.q) + b * p.qs[0] + l * p.qs[2], p.qs[1],
                              static_cast<uint16_t *>(p.q_out) + b * p.Hq * out_h + l * p.d, out_h, h0, min(h1, p.Hq), group,
                              groups, valid, at, lpr, c, s, static_cast<const uint16_t *>(p.q_w), p.eps, inv_d, dwq);
    rope_heads_bwd<BF, INTER>(static_cast<const uint16_t *>(p.dk) + b * p.dks[0] + l * p.dks[2], p.dks[1],
                              static_cast<const uint16_t *>(p.k) + b * p.ks[0] + l * p.ks[2], p.ks[1],
                              static_cast<uint16_t *>(p.k_out) + b * p.Hkv * out_h + l * p.d, out_h, max(h0 - p.Hq, 0), h1 - p.Hq,
                              group, groups, valid, at, lpr, c, s, static_cast<const uint16_t *>(p.k_w), p.eps, inv_d, dwk);
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float *const part = p.parts + (static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 2 * p.d;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float *const dw = which ? dwk : dwq;
#pragma unroll
    for (int e = 0; e < 16; ++e)
      for (int o = lpr; o < 32; o <<= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], o);
    __syncthreads();
    if (lane < lpr) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        red[warp][at.c0 + e] = dw[e];
        red[warp][at.c1 + e] = dw[8 + e];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.d; i += kRopeThreads) {
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < kRopeThreads / 32; ++k) t += red[k][i];
      part[which * p.d + i] = t;
    }
  }
}

// dw[which][i] = sum over parts; one block per (which, 32 columns), 32 x 32 threads.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float *parts, int n, int d, float *dq_w, float *dk_w) {
  __shared__ float red[32][33];
  grid_launch_dependents();
  grid_wait_prior();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, which = blockIdx.y, col = blockIdx.x * 32 + x;
  float t = 0.f;
#pragma unroll 4
  for (int r = y; r < n; r += 32) t += parts[(static_cast<size_t>(r) * 2 + which) * d + col];
  red[y][x] = t;
  __syncthreads();
  t = red[x][y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (x == 0) (which ? dk_w : dq_w)[blockIdx.x * 32 + y] = t;
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

// Tokens and heads of a block.  As many tokens (a power of two up to 8, so that a head's rows
// of neighbouring tokens are written together) as still leave two blocks per SM; with fewer
// tokens than that the heads are split over blocks too.
dim3 plan(RopeParams &p, int heads, int sm_count, long long max_blocks) {
  const long long N = static_cast<long long>(p.B) * p.L, want = 2LL * sm_count;
  p.tokens = kRopeMaxTokens;
  while (p.tokens > 1 && (N + p.tokens - 1) / p.tokens < want) p.tokens >>= 1;
  const long long tiles = (N + p.tokens - 1) / p.tokens;
  const int groups = kRopeThreads / (p.d >> 4) / p.tokens;
  long long split = std::max(1LL, std::min<long long>(want / tiles, (heads + groups - 1) / groups));
  p.heads_per_block = static_cast<int>((heads + split - 1) / split);
  split = (heads + p.heads_per_block - 1) / p.heads_per_block;
  return dim3(static_cast<unsigned>(std::min(tiles, std::max(1LL, max_blocks / split))), static_cast<unsigned>(split));
}

size_t turns_bytes(const RopeParams &p) { return static_cast<size_t>(p.tokens) * (p.rotary / 2) * sizeof(float2); }

constexpr long long kNoCap = 1LL << 40;

}  // namespace

cudaError_t launch_rope(RopeLaunch &a) {
  const dim3 grid = plan(a.p, a.p.Hq + a.p.Hkv, a.sm_count, kNoCap);
  const bool norm = a.p.q_w != nullptr;
  auto *kern = a.bf16 ? (norm ? (a.interleaved ? rope_kernel<true, true, true> : rope_kernel<true, true, false>)
                              : (a.interleaved ? rope_kernel<true, false, true> : rope_kernel<true, false, false>))
                      : (norm ? (a.interleaved ? rope_kernel<false, true, true> : rope_kernel<false, true, false>)
                              : (a.interleaved ? rope_kernel<false, false, true> : rope_kernel<false, false, false>));
  return launch(kern, grid, kRopeThreads, turns_bytes(a.p), a.stream, RopeParams(a.p));
}

cudaError_t launch_append(RopeLaunch &a) {
  const dim3 grid = plan(a.p, a.p.Hq + 2 * a.p.Hkv, a.sm_count, kNoCap);
  const bool norm = a.p.q_w != nullptr || a.p.k_w != nullptr;
  auto *kern = a.bf16 ? (norm ? (a.interleaved ? append_kernel<true, true, true> : append_kernel<true, true, false>)
                              : (a.interleaved ? append_kernel<true, false, true> : append_kernel<true, false, false>))
                      : (norm ? (a.interleaved ? append_kernel<false, true, true> : append_kernel<false, true, false>)
                              : (a.interleaved ? append_kernel<false, false, true> : append_kernel<false, false, false>));
  return launch(kern, grid, kRopeThreads, turns_bytes(a.p), a.stream, RopeParams(a.p));
}

cudaError_t launch_rope_bwd(RopeLaunch &a) {
  const dim3 grid = plan(a.p, a.p.Hq + a.p.Hkv, a.sm_count, std::min<long long>(kRopeMaxParts, 4LL * a.sm_count));
  auto *kern = a.bf16 ? (a.interleaved ? rope_bwd_kernel<true, true> : rope_bwd_kernel<true, false>)
                      : (a.interleaved ? rope_bwd_kernel<false, true> : rope_bwd_kernel<false, false>);
  const cudaError_t e = launch(kern, grid, kRopeThreads, turns_bytes(a.p), a.stream, RopeParams(a.p));
  if (e != cudaSuccess) return e;
  return launch(rope_dw_kernel, dim3(a.p.d / 32, a.p.k_w ? 2 : 1), 1024, 0, a.stream, static_cast<const float *>(a.p.parts),
                static_cast<int>(grid.x * grid.y), a.p.d, a.p.dq_w, a.p.dk_w);
}

}  // namespace gbattn
