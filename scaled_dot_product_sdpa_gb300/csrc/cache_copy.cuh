// cache_copy.cuh -- copying pages of a paged key/value cache: parameters and launch.
#pragma once

#include <cuda_runtime.h>

namespace gbattn {

// Pages of one launch.  The pairs travel as kernel arguments (host lists, no copy to the
// device), whose room is 32,764 bytes in all: the larger list is the round number below
// (32,764 - sizeof(CopyShape) - 4) / 8, the smaller one keeps short calls' arguments to 0.5 KB.
constexpr int kCopyPairsSmall = 60;
constexpr int kCopyPairsLarge = 4000;

struct CopyShape {
  char *k, *v;
  long long page_b;            // bytes from page to page
  long long head_b, slot_b;    // bytes between the pieces of a page (pieces > 1)
  int piece_vecs;              // 16-byte vectors of a contiguous piece
  int pieces, slots;           // pieces of a page; pieces (slots) to a head
};

struct CopyLaunch {
  CopyShape s;
  const int *src, *dst;        // host
  int n;                       // at most kCopyPairsLarge
  cudaStream_t stream;
};

cudaError_t launch_cache_copy(const CopyLaunch &a);

}  // namespace gbattn
