// paged_decode.cuh -- attention of one new token per sequence over a paged key/value
// cache: parameters and launch entry point.
//
// For sequence b with n = lengths[b] cached tokens and query head h, which shares the keys
// and values of head h / (Hq / Hkv):
//     o[b, h]   = sum_{j < n} softmax_j(scale q[b, h] . k_j) v_j,    lse[b, h] = log sum_{j < n} exp(scale q[b, h] . k_j)
// (o = 0, lse = -inf when n = 0), key j being slot j % page of page table[b, j / page].
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

namespace gbattn {

// Persistent CTAs on an SM.  Two where registers and shared memory hold them (up to 8 heads at once
// and d <= 128, or 16 and d = 64): one CTA's tile is a chain of a softmax and two products, and at
// d = 64 or with short sequences the second fills its gaps.  GB300, one and two CTAs: 128 x 8 heads x
// 8000 keys x 64 394 and 319 us, 64 of them with 16 query heads a key head 251 and 201; 256 sequences
// of 100 keys x 128, 32/8 heads, 33.9 and 30.2; 154 x 32 heads of 4 keys 70.4 and 52.0; long rows at
// d = 128 315 and 309; one sequence of 1000 keys 9.5 and 9.5, of 20000 x 64, 128/8 heads, 21.1 and 19.7.
constexpr int paged_resident(int d, int heads) { return (heads == 8 && d <= 128) || (heads == 16 && d == 64) ? 2 : 1; }
constexpr int kPagedMaxCtas = 304;  // CTAs at most (two on each SM); sizes the workspace
constexpr int kPagedTile = 128;     // keys per tile

// Query heads of one key head that a CTA works on at once, and how many such blocks of heads
// a key head's G query heads make (each reads the keys again).
constexpr int paged_heads(int G, int d) { return G <= 8 ? 8 : G <= 16 || d > 256 ? 16 : 32; }
constexpr int paged_blocks(int G, int d) { return (G + paged_heads(G, d) - 1) / paged_heads(G, d); }

// Workspace: a record per CTA, then two partial results per CTA, each of paged_heads rows of
// o[d] (normalised), then the base-2 log-sum-exps of all rows.
struct PagedRecord {
  int head;   // b * Hq + first query head of the rows that this CTA's last partial begins; unused when parts = 0
  int heads;
  int parts;  // partial results to join: this CTA's second, then the first of each of the following parts - 1 CTAs
  int pad;
};
constexpr long long paged_workspace_bytes(int G, int d) {
  return kPagedMaxCtas * (16LL + 2LL * paged_heads(G, d) * (d + 1) * 4);
}

struct PagedParams {
  PagedRecord *records;                // workspace
  float *part_o, *part_lse;            // [2 kPagedMaxCtas][heads][d], [2 kPagedMaxCtas][heads]
  const int *table, *lengths;
  long long table_s;
  int table_w, page, pages;
  int B, Hq, Hkv, d;
  int G, blocks;                       // query heads per key head; blocks of them
  int box_rows;                        // rows of a TMA box: a power of two <= 128 that divides the page
  int q_rows;                          // rows of a query box
  int tile_pages, tile_slots;          // kPagedTile / page, kPagedTile % page
  bool bf16;
  float c2;                            // scale log2(e)
  void *o;                             // [B, Hq, d]
  float *lse;                          // [B, Hq]
  unsigned *status;
  long long wait_limit;
};

struct PagedLaunch {
  CUtensorMap tm_q, tm_k, tm_v;
  PagedParams p;
  int sm_count;
  cudaStream_t stream;
};

cudaError_t launch_decode_paged(const PagedLaunch &a);

}  // namespace gbattn
