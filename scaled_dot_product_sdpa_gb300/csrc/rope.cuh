// rope.cuh -- rotary positions with optional per-head RMS norms of queries and keys, and the
// paged cache's append, which shares their row code: parameters and launch entry points.
//
// For a row x of one head at position p (w: the norm's weight, when there is one)
//     y = x * rsqrt(mean(x^2) + eps) * w                  (or y = x without a norm)
//     z_i = f (y_i cos a - y_j sin a),  z_j = f (y_j cos a + y_i sin a),  a = p inv_freq[r]
// for the r-th pair (i, j) of the first `rotary` elements -- (r, r + rotary / 2) or, when
// interleaved, (2r, 2r + 1) -- and z = y for the other elements.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace gbattn {

constexpr unsigned kDevBadPage = 8;    // a page number outside the cache within a sequence's length
constexpr unsigned kDevBadLength = 9;  // a length that is negative or beyond the page table
constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTokens = 32;     // tokens a block works on at once
constexpr int kRopeMaxParts = 320;     // partial weight gradients (blocks) of the backward pass

struct RopeParams {
  const void *q, *k, *v;             // rows [B, H, L, d] by strides; v: append only
  long long qs[3], ks[3], vs[3];     // element strides of batch, head, row
  const void *dq, *dk;               // backward: upstream gradients, by strides dqs, dks
  long long dqs[3], dks[3];
  void *q_out, *k_out;               // contiguous [B, H, L, d]
  float *parts;                      // backward with norms: [blocks, 2, d] partial weight gradients
  float *dq_w, *dk_w;                // backward with norms: [d] weight gradients
  const double *inv_freq;            // [rotary / 2]
  const int *positions;              // [B, L] with row stride pos_s, or null: the row's own index
  long long pos_s;
  const void *q_w, *k_w;             // [d] norm weights, or null
  float eps, factor, sign;           // sign -1 turns backwards
  int B, Hq, Hkv, L, d, rotary;
  int tokens;                        // per block: a power of two up to kRopeMaxTokens
  int at_once;                       // rows of a unit that each thread works on
  int steps, steps_q, steps_k;       // units of a tile: all, of q, of k (and of v)
  long long units;                   // in all
  // append
  void *k_pages, *v_pages;           // [pages, Hkv, page, d] by strides
  long long page_s, head_s, slot_s;
  const int *table, *lengths, *counts;
  long long table_s;
  int table_w, page, pages;
  unsigned *status;
};

struct RopeLaunch {
  RopeParams p;
  bool bf16, interleaved;
  int sm_count;
  cudaStream_t stream;
};

cudaError_t launch_rope(RopeLaunch &a);      // q, k -> q_out, k_out (sign -1: gradients without norms)
cudaError_t launch_rope_bwd(RopeLaunch &a);  // dq, dk, q, k -> q_out, k_out, dq_w, dk_w (with norms)
cudaError_t launch_append(RopeLaunch &a);    // k, v (and q) -> pages (and q_out)

}  // namespace gbattn
