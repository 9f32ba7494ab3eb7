// abi_host.cuh -- what the files of C entry points share: per-device setup, the driver's
// tensor-map encoder (both in gbattn_abi.cu) and argument checks.
#pragma once

#include <cuda.h>

#include <cstdint>

namespace gbattn {

// SM count and status word of the current device (GBATTN_OK, or an error code when it is
// not usable).
int abi_device(int *sm_count, unsigned **status);
// A tiled tensor map of 16-bit elements with 128-byte swizzle; GBATTN_OK or
// GBATTN_ERR_TENSORMAP.  After abi_device.
int abi_encode(CUtensorMap *tm, bool bf16, int rank, const void *ptr, const cuuint64_t *dims, const cuuint64_t *strides,
               const cuuint32_t *box);

inline bool abi_overlaps(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}
inline bool abi_aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

}  // namespace gbattn
