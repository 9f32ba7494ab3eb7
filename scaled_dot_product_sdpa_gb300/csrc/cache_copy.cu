// cache_copy.cu -- copying pages of a paged cache, keys and values in one launch.
//
// Bound by the reads and writes of the pages.  A block moves up to 1024 16-byte vectors of
// one page of keys or of values, each thread four, all four loads issued before the first
// store.  GB300: 4000 pages of 16 x 8 x 128 (0.5 GB read and written) 77.6 us, the copy bandwidth; seven
// pages 7 to 8 us, the call.
#include <algorithm>
#include <cstring>

#include "cache_copy.cuh"
#include "ptx.cuh"

namespace gbattn {
namespace {

constexpr int kThreads = 256, kVecs = 4;

template <int N>
struct CopyParams {
  CopyShape s;
  int blocks;  // per page
  int src[N], dst[N];  // read as far as the grid's pairs go
};

template <int N>
__global__ void __launch_bounds__(kThreads) cache_copy_kernel(const __grid_constant__ CopyParams<N> p) {
  grid_launch_dependents();
  grid_wait_prior();
  const int page = blockIdx.x / p.blocks, part = blockIdx.x - page * p.blocks;
  const int pair = page >> 1;
  char *const base = (page & 1) ? p.s.v : p.s.k;
  const char *const from = base + p.src[pair] * p.s.page_b;
  char *const to = base + p.dst[pair] * p.s.page_b;
  const int vecs = p.s.pieces * p.s.piece_vecs;
  uint4 x[kVecs];
  long long at[kVecs];
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const int i = (part * kVecs + u) * kThreads + threadIdx.x;
    at[u] = -1;
    if (i < vecs) {
      if (p.s.pieces == 1) {
        at[u] = 16LL * i;
      } else {
        const int piece = i / p.s.piece_vecs, in = i - piece * p.s.piece_vecs;
        const int head = piece / p.s.slots, slot = piece - head * p.s.slots;
        at[u] = head * p.s.head_b + slot * p.s.slot_b + 16LL * in;
      }
      x[u] = *reinterpret_cast<const uint4 *>(from + at[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < kVecs; ++u)
    if (at[u] >= 0) *reinterpret_cast<uint4 *>(to + at[u]) = x[u];
}

template <int N>
cudaError_t launch_n(const CopyLaunch &a) {
  CopyParams<N> p;
  p.s = a.s;
  p.blocks = (a.s.pieces * a.s.piece_vecs + kThreads * kVecs - 1) / (kThreads * kVecs);
  std::memcpy(p.src, a.src, sizeof(int) * a.n);
  std::memcpy(p.dst, a.dst, sizeof(int) * a.n);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * a.n) * static_cast<unsigned>(p.blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_copy_kernel<N>, p);
}

}  // namespace

cudaError_t launch_cache_copy(const CopyLaunch &a) {
  return a.n <= kCopyPairsSmall ? launch_n<kCopyPairsSmall>(a) : launch_n<kCopyPairsLarge>(a);
}

}  // namespace gbattn
