// attn_decode_paged.cu -- decoding over a paged cache: one block per sequence and query head,
// whose eight warps take the keys in turn, each with its own running maximum and sum, and
// join them at the end.
#include "attn_decode_paged.cuh"
#include "ptx.cuh"
#include "rope.cuh"
#include "vec16.cuh"

namespace gbattn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

template <bool BF, int D>
__global__ void __launch_bounds__(kThreads) decode_paged_kernel(const PagedParams p) {
  __shared__ float part[kWarps][D + 2];
  grid_launch_dependents();
  grid_wait_prior();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / p.Hq, h = blockIdx.x - b * p.Hq, hk = h / (p.Hq / p.Hkv);
  constexpr int E = D / 32;  // elements 2 lane + 64 i + {0, 1} of a row
  float q[E], acc[E], m = -INFINITY, l = 0.f;
  const uint16_t *const qrow = static_cast<const uint16_t *>(p.q) + b * p.q_b + h * p.q_h;
  auto load = [&](const uint16_t *row, float *x) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const uint32_t w = *reinterpret_cast<const uint32_t *>(row + 64 * i + 2 * lane);
      if constexpr (BF) {
        x[2 * i] = __uint_as_float(w << 16);
        x[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
      } else {
        const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        x[2 * i] = t.x;
        x[2 * i + 1] = t.y;
      }
    }
  };
  load(qrow, q);
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  long long n = p.lengths[b];
  const long long most = static_cast<long long>(p.table_w) * p.page;
  if (n < 0 || n > most) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0u, kDevBadLength);
    n = n < 0 ? 0 : most;
  }
  for (long long j = warp; j < n; j += kWarps) {
    const int page = p.table[b * p.table_s + j / p.page];
    float k[E], v[E];
    if (page < 0 || page >= p.pages) {
      if (lane == 0) atomicCAS(p.status, 0u, kDevBadPage);
#pragma unroll
      for (int e = 0; e < E; ++e) k[e] = v[e] = 0.f;
    } else {
      const long long at = page * p.page_s + hk * p.head_s + (j % p.page) * p.slot_s;
      load(static_cast<const uint16_t *>(p.k_pages) + at, k);
      load(static_cast<const uint16_t *>(p.v_pages) + at, v);
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= p.c2;
    const float top = fmaxf(m, s);
    const float base = top == -INFINITY ? 0.f : top;
    const float keep = ex2_approx(m - base), w = ex2_approx(s - base);
    m = top;
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * keep + w * v[e];
  }
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    part[warp][64 * i + 2 * lane] = acc[2 * i];
    part[warp][64 * i + 2 * lane + 1] = acc[2 * i + 1];
  }
  if (lane == 0) {
    part[warp][D] = m;
    part[warp][D + 1] = l;
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part[w][D]);
  const float base = top == -INFINITY ? 0.f : top;
  for (int w = 0; w < kWarps; ++w) sum += part[w][D + 1] * ex2_approx(part[w][D] - base);
  for (int c = threadIdx.x; c < D; c += kThreads) {
    float o = 0.f;
    for (int w = 0; w < kWarps; ++w) o += part[w][c] * ex2_approx(part[w][D] - base);
    o = sum > 0.f ? o / sum : (sum == 0.f ? 0.f : sum);
    const size_t at = static_cast<size_t>(blockIdx.x) * D + c;
    if constexpr (BF)
      static_cast<__nv_bfloat16 *>(p.o)[at] = __float2bfloat16_rn(o);
    else
      static_cast<__half *>(p.o)[at] = __float2half_rn(o);
  }
  if (threadIdx.x == 0) p.lse[blockIdx.x] = (top + log2f(sum)) * 0.69314718055994531f;
}

}  // namespace

cudaError_t launch_decode_paged(const PagedLaunch &a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.p.B) * static_cast<unsigned>(a.p.Hq));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (a.p.d) {
    case 64: return cudaLaunchKernelEx(&cfg, a.bf16 ? decode_paged_kernel<true, 64> : decode_paged_kernel<false, 64>, a.p);
    case 128: return cudaLaunchKernelEx(&cfg, a.bf16 ? decode_paged_kernel<true, 128> : decode_paged_kernel<false, 128>, a.p);
    case 256: return cudaLaunchKernelEx(&cfg, a.bf16 ? decode_paged_kernel<true, 256> : decode_paged_kernel<false, 256>, a.p);
    default: return cudaLaunchKernelEx(&cfg, a.bf16 ? decode_paged_kernel<true, 512> : decode_paged_kernel<false, 512>, a.p);
  }
}

}  // namespace gbattn
