// attn_decode_paged.cuh -- attention of one new token per sequence over a paged key/value
// cache: parameters and launch entry point.
//
// For sequence b with n = lengths[b] cached tokens and query head h, which shares the keys
// and values of head h / (Hq / Hkv):
//     o[b, h]   = sum_{j < n} softmax_j(scale q[b, h] . k_j) v_j,    lse[b, h] = log sum_{j < n} exp(scale q[b, h] . k_j)
// (o = 0, lse = -inf when n = 0), key j being slot j % page of page table[b, j / page].
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace gbattn {

struct PagedParams {
  const void *q;                       // [B, Hq, d] by strides
  long long q_b, q_h;
  const void *k_pages, *v_pages;       // [pages, Hkv, page, d] by strides
  long long page_s, head_s, slot_s;
  const int *table, *lengths;
  long long table_s;
  int table_w, page, pages;
  int B, Hq, Hkv, d;
  float c2;                            // scale log2(e)
  void *o;                             // [B, Hq, d]
  float *lse;                          // [B, Hq]
  unsigned *status;
};

struct PagedLaunch {
  PagedParams p;
  bool bf16;
  int sm_count;
  cudaStream_t stream;
};

cudaError_t launch_decode_paged(const PagedLaunch &a);

}  // namespace gbattn
