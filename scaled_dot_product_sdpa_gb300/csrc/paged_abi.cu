// paged_abi.cu -- the C entry points of the operators beside the attention kernels
// (include/gbattn.h): argument checks and launches of attn_rope, attn_rope_bwd,
// attn_cache_append, attn_cache_copy and attn_decode_paged.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdlib>

#include "abi_host.cuh"
#include "paged_decode.cuh"
#include "cache_copy.cuh"
#include "gbattn.h"
#include "rope.cuh"

namespace gbattn {
namespace {

struct Rows {
  const void *p;
  long long sb, sh, sl;
};

struct Span {  // bytes [p, p + n)
  const void *p;
  size_t n;
};

bool finite_nonneg(float x) { return std::isfinite(x) && x >= 0.f; }
bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256 || d == 512; }
// n > 0 steps of a stride stay within 2^40 elements, more than any memory, so that no sum of them overflows.
bool reach_ok(long long s, long long n) { return s >= 0 && s <= (1LL << 40) / n; }
bool stride_ok(long long s, long long n) { return s % 8 == 0 && s < (1LL << 39) && reach_ok(s, n); }
bool rows_ok(const Rows &r, int B, int H, int L) {
  return stride_ok(r.sb, B) && stride_ok(r.sh, H) && r.sh < (1LL << 32) && stride_ok(r.sl, L);
}

Span rows_span(const Rows &r, int B, int H, int L, int d) {
  if (!r.p) return {nullptr, 0};
  const long long last = (B - 1LL) * r.sb + (H - 1LL) * r.sh + (L - 1LL) * r.sl + d;
  return {r.p, static_cast<size_t>(last) * 2u};
}
Span dense_span(const void *p, long long n, int bytes) { return {p, p ? static_cast<size_t>(n) * bytes : 0}; }

// No output overlaps an input or another output.
bool disjoint(const Span *out, int n_out, const Span *in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    if (!out[i].n) continue;
    for (int j = 0; j < n_in; ++j)
      if (in[j].n && abi_overlaps(out[i].p, out[i].n, in[j].p, in[j].n)) return false;
    for (int j = i + 1; j < n_out; ++j)
      if (out[j].n && abi_overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return false;
  }
  return true;
}

int check_dims(int dtype, int B, int Hq, int Hkv, int L, int d) {
  if (dtype != GBATTN_F16 && dtype != GBATTN_BF16) return GBATTN_ERR_DTYPE;
  if (B <= 0 || Hq < 0 || Hkv < 0 || Hq + static_cast<long long>(Hkv) <= 0 || L <= 0) return GBATTN_ERR_DIMS;
  const long long heads = Hq + 2LL * Hkv;
  if (heads > INT_MAX / 4 || static_cast<long long>(B) * L > INT_MAX / 4 ||
      heads > (1LL << 40) / (static_cast<long long>(B) * L))
    return GBATTN_ERR_DIMS;
  if (!head_dim_ok(d)) return GBATTN_ERR_HEAD_DIM;
  return static_cast<long long>(L) * d < (1LL << 32) ? GBATTN_OK : GBATTN_ERR_DIMS;
}

int check_rope(const double *inv_freq, int rotary, float factor, float eps, const int *positions, long long positions_stride,
               const void *q_weight, const void *k_weight, int B, int Hq, int Hkv, int d) {
  if (rotary < 0 || rotary > d || rotary % 16 || (rotary > 0 && !inv_freq)) return GBATTN_ERR_ROTARY;
  // Norms: a weight for each tensor that is there, or none.
  const bool norm = q_weight || k_weight;
  if (norm && ((Hq > 0) != (q_weight != nullptr) || (Hkv > 0) != (k_weight != nullptr))) return GBATTN_ERR_ROTARY;
  if (!abi_aligned(inv_freq, 8) || !abi_aligned(positions, 4) || !abi_aligned(q_weight, 16) || !abi_aligned(k_weight, 16))
    return GBATTN_ERR_ALIGN;
  if (!std::isfinite(factor) || !(factor > 0.f) || !finite_nonneg(eps)) return GBATTN_ERR_SCALE;
  if (positions && !reach_ok(positions_stride, B)) return GBATTN_ERR_STRIDE;
  return GBATTN_OK;
}

// Whether two equal sets of rows of d elements at sum_i n_i strides[i], 0 <= n_i < counts[i], one
// moved by `gap`, meet: whether gap is within d of some sum_i m_i strides[i], |m_i| < counts[i].
// Each stride is at least the extent of what is inside it, so that only the two multiples
// next to the gap can come near it.
bool rows_meet(long long gap, const long long *strides, const long long *counts, int n, int d) {
  if (n == 0) return gap < d && gap > -d;
  if (counts[0] == 1 || strides[0] == 0) return rows_meet(gap, strides + 1, counts + 1, n - 1, d);
  long long m = gap / strides[0];
  if (gap % strides[0] < 0) --m;
  for (int i = 0; i < 2; ++i, ++m)
    if (m < counts[0] && -m < counts[0] && rows_meet(gap - m * strides[0], strides + 1, counts + 1, n - 1, d)) return true;
  return false;
}

// A cache's shape and strides; `extent`: elements from a page's first to behind its last.
int check_pages(const void *k, const void *v, long long sp, long long sh, long long ss, int pages, int page, int Hkv, int d,
                long long *extent) {
  if (pages <= 0 || Hkv <= 0) return GBATTN_ERR_DIMS;
  if (page <= 0 || page % 8) return GBATTN_ERR_PAGES;
  if (!stride_ok(sp, pages) || !stride_ok(sh, Hkv) || sh >= (1LL << 32) || !stride_ok(ss, page)) return GBATTN_ERR_STRIDE;
  const long long slots = (page - 1LL) * ss + d, heads = (Hkv - 1LL) * sh + d;
  const bool head_outer = ss >= d && (Hkv == 1 || sh >= slots), slot_outer = (Hkv == 1 || sh >= d) && ss >= heads;
  if (!head_outer && !slot_outer) return GBATTN_ERR_STRIDE;
  *extent = (page - 1LL) * ss + (Hkv - 1LL) * sh + d;
  if (pages > 1 && sp < *extent) return GBATTN_ERR_STRIDE;
  if (!abi_aligned(k, 16) || !abi_aligned(v, 16)) return GBATTN_ERR_ALIGN;
  // Keys and values may interleave (the two halves of one array) but share no element.
  const uintptr_t x = reinterpret_cast<uintptr_t>(k), y = reinterpret_cast<uintptr_t>(v);
  const uintptr_t gap = (x < y ? y - x : x - y) / 2;
  const long long strides[3] = {sp, head_outer ? sh : ss, head_outer ? ss : sh};
  const long long counts[3] = {pages, head_outer ? Hkv : page, head_outer ? page : Hkv};
  if (gap < static_cast<uintptr_t>(1) << 62 && rows_meet(static_cast<long long>(gap), strides, counts, 3, d)) return GBATTN_ERR_ALIAS;
  return GBATTN_OK;
}

Span pages_span(const void *p, long long sp, long long extent, int pages) {
  return {p, static_cast<size_t>((pages - 1LL) * sp + extent) * 2u};
}

void fill_rope(RopeParams &p, const double *inv_freq, int rotary, float factor, const int *positions, long long positions_stride,
               const void *q_weight, const void *k_weight, float eps, int B, int Hq, int Hkv, int L, int d) {
  p.inv_freq = inv_freq;
  p.rotary = rotary;
  p.factor = factor;
  p.sign = 1.f;
  p.positions = positions;
  p.pos_s = positions_stride;
  p.q_w = q_weight;
  p.k_w = k_weight;
  p.eps = eps;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.L = L;
  p.d = d;
}
void fill_rows(long long *s, const Rows &r) {
  s[0] = r.sb;
  s[1] = r.sh;
  s[2] = r.sl;
}

long long positions_count(const int *positions, long long stride, int B, int L) {
  return positions ? (B - 1LL) * stride + L : 0;
}

int done(cudaError_t e) { return e == cudaSuccess ? GBATTN_OK : GBATTN_ERR_LAUNCH; }

}  // namespace
}  // namespace gbattn

using namespace gbattn;

extern "C" int attn_rope(const void *q, long long q_sb, long long q_sh, long long q_sl, const void *k, long long k_sb,
                         long long k_sh, long long k_sl, void *q_out, void *k_out, const double *inv_freq, int rotary,
                         int interleaved, float factor, const int *positions, long long positions_stride,
                         const void *q_weight, const void *k_weight, float eps, int dtype, int B, int Hq, int Hkv, int L,
                         int d, void *stream) {
  if (!q || !q_out || (Hkv > 0 && (!k || !k_out))) return GBATTN_ERR_NULL;
  int rc = check_dims(dtype, B, Hq, Hkv, L, d);
  if (rc != GBATTN_OK) return rc;
  if (Hq <= 0) return GBATTN_ERR_DIMS;
  if (!abi_aligned(q, 16) || !abi_aligned(k, 16) || !abi_aligned(q_out, 16) || !abi_aligned(k_out, 16)) return GBATTN_ERR_ALIGN;
  if ((rc = check_rope(inv_freq, rotary, factor, eps, positions, positions_stride, q_weight, k_weight, B, Hq, Hkv, d)) != GBATTN_OK)
    return rc;
  const Rows rq{q, q_sb, q_sh, q_sl}, rk{Hkv > 0 ? k : nullptr, k_sb, k_sh, k_sl};
  if (!rows_ok(rq, B, Hq, L) || (rk.p && !rows_ok(rk, B, Hkv, L))) return GBATTN_ERR_STRIDE;
  const long long rows = static_cast<long long>(B) * L;
  const Span out[2] = {dense_span(q_out, rows * Hq * d, 2), dense_span(rk.p ? k_out : nullptr, rows * Hkv * d, 2)};
  const Span in[6] = {rows_span(rq, B, Hq, L, d), rows_span(rk, B, Hkv, L, d), dense_span(inv_freq, rotary / 2, 8),
                      dense_span(positions, positions_count(positions, positions_stride, B, L), 4), dense_span(q_weight, d, 2),
                      dense_span(k_weight, d, 2)};
  if (!disjoint(out, 2, in, 6)) return GBATTN_ERR_ALIAS;
  RopeLaunch a = {};
  unsigned *status = nullptr;
  if ((rc = abi_device(&a.sm_count, &status)) != GBATTN_OK) return rc;
  fill_rope(a.p, inv_freq, rotary, factor, positions, positions_stride, q_weight, k_weight, eps, B, Hq, Hkv, L, d);
  a.p.q = q;
  a.p.k = rk.p;
  fill_rows(a.p.qs, rq);
  fill_rows(a.p.ks, rk);
  a.p.q_out = q_out;
  a.p.k_out = k_out;
  a.bf16 = dtype == GBATTN_BF16;
  a.interleaved = interleaved != 0;
  a.stream = static_cast<cudaStream_t>(stream);
  return done(launch_rope(a));
}

extern "C" long long attn_rope_bwd_workspace_bytes(int d) {
  if (!head_dim_ok(d)) return GBATTN_ERR_HEAD_DIM;
  return static_cast<long long>(kRopeMaxParts) * 2 * d * 4;
}

extern "C" int attn_rope_bwd(const void *dq_up, long long dq_sb, long long dq_sh, long long dq_sl, const void *dk_up,
                             long long dk_sb, long long dk_sh, long long dk_sl, const void *q, long long q_sb,
                             long long q_sh, long long q_sl, const void *k, long long k_sb, long long k_sh, long long k_sl,
                             void *dq, void *dk, float *dq_weight, float *dk_weight, const double *inv_freq, int rotary,
                             int interleaved, float factor, const int *positions, long long positions_stride,
                             const void *q_weight, const void *k_weight, float eps, void *workspace, int dtype, int B, int Hq,
                             int Hkv, int L, int d, void *stream) {
  const bool norm = q_weight || k_weight;
  if (!dq_up || !dq || (Hkv > 0 && (!dk_up || !dk))) return GBATTN_ERR_NULL;
  if (norm && (!q || !dq_weight || !workspace || (Hkv > 0 && (!k || !dk_weight)))) return GBATTN_ERR_NULL;
  int rc = check_dims(dtype, B, Hq, Hkv, L, d);
  if (rc != GBATTN_OK) return rc;
  if (Hq <= 0) return GBATTN_ERR_DIMS;
  const void *const ptrs[10] = {dq_up, dk_up, dq, dk, norm ? q : nullptr, norm ? k : nullptr, norm ? dq_weight : nullptr,
                                norm ? dk_weight : nullptr, norm ? workspace : nullptr, nullptr};
  for (const void *p : ptrs)
    if (!abi_aligned(p, 16)) return GBATTN_ERR_ALIGN;
  if ((rc = check_rope(inv_freq, rotary, factor, eps, positions, positions_stride, q_weight, k_weight, B, Hq, Hkv, d)) != GBATTN_OK)
    return rc;
  const bool keys = Hkv > 0;
  const Rows gq{dq_up, dq_sb, dq_sh, dq_sl}, gk{keys ? dk_up : nullptr, dk_sb, dk_sh, dk_sl};
  const Rows rq{norm ? q : nullptr, q_sb, q_sh, q_sl}, rk{norm && keys ? k : nullptr, k_sb, k_sh, k_sl};
  if (!rows_ok(gq, B, Hq, L) || (gk.p && !rows_ok(gk, B, Hkv, L)) || (rq.p && !rows_ok(rq, B, Hq, L)) ||
      (rk.p && !rows_ok(rk, B, Hkv, L)))
    return GBATTN_ERR_STRIDE;
  const long long rows = static_cast<long long>(B) * L;
  const Span out[5] = {dense_span(dq, rows * Hq * d, 2), dense_span(keys ? dk : nullptr, rows * Hkv * d, 2),
                       dense_span(norm ? dq_weight : nullptr, d, 4), dense_span(norm && keys ? dk_weight : nullptr, d, 4),
                       dense_span(norm ? workspace : nullptr, attn_rope_bwd_workspace_bytes(d), 1)};
  const Span in[8] = {rows_span(gq, B, Hq, L, d), rows_span(gk, B, Hkv, L, d), rows_span(rq, B, Hq, L, d),
                      rows_span(rk, B, Hkv, L, d), dense_span(inv_freq, rotary / 2, 8),
                      dense_span(positions, positions_count(positions, positions_stride, B, L), 4), dense_span(q_weight, d, 2),
                      dense_span(k_weight, d, 2)};
  if (!disjoint(out, 5, in, 8)) return GBATTN_ERR_ALIAS;
  RopeLaunch a = {};
  unsigned *status = nullptr;
  if ((rc = abi_device(&a.sm_count, &status)) != GBATTN_OK) return rc;
  fill_rope(a.p, inv_freq, rotary, factor, positions, positions_stride, q_weight, k_weight, eps, B, Hq, Hkv, L, d);
  a.p.sign = -1.f;
  a.p.q_out = dq;
  a.p.k_out = dk;
  a.bf16 = dtype == GBATTN_BF16;
  a.interleaved = interleaved != 0;
  a.stream = static_cast<cudaStream_t>(stream);
  if (!norm) {  // the rotation turned back
    a.p.q = gq.p;
    a.p.k = gk.p;
    fill_rows(a.p.qs, gq);
    fill_rows(a.p.ks, gk);
    return done(launch_rope(a));
  }
  a.p.dq = gq.p;
  a.p.dk = gk.p;
  fill_rows(a.p.dqs, gq);
  fill_rows(a.p.dks, gk);
  a.p.q = rq.p;
  a.p.k = rk.p;
  fill_rows(a.p.qs, rq);
  fill_rows(a.p.ks, rk);
  a.p.parts = static_cast<float *>(workspace);
  a.p.dq_w = dq_weight;
  a.p.dk_w = dk_weight;
  return done(launch_rope_bwd(a));
}

extern "C" int attn_cache_append(const void *k, long long k_sb, long long k_sh, long long k_sl, const void *v, long long v_sb,
                                 long long v_sh, long long v_sl, const void *q, long long q_sb, long long q_sh,
                                 long long q_sl, void *q_out, void *k_pages, void *v_pages, long long page_stride,
                                 long long head_stride, long long slot_stride, int pages, int page, const int *table,
                                 long long table_stride, int table_width, const int *lengths, const int *counts,
                                 const double *inv_freq, int rotary, int interleaved, float factor, const void *q_weight,
                                 const void *k_weight, float eps, int dtype, int B, int Hq, int Hkv, int L, int d,
                                 void *stream) {
  if (!k || !v || !k_pages || !v_pages || !table || !lengths || (Hq > 0 && (!q || !q_out))) return GBATTN_ERR_NULL;
  int rc = check_dims(dtype, B, Hq, Hkv, L, d);
  if (rc != GBATTN_OK) return rc;
  if (Hkv <= 0 || table_width <= 0) return GBATTN_ERR_DIMS;
  if (!abi_aligned(k, 16) || !abi_aligned(v, 16) || (Hq > 0 && (!abi_aligned(q, 16) || !abi_aligned(q_out, 16))) ||
      !abi_aligned(table, 4) || !abi_aligned(lengths, 4) || !abi_aligned(counts, 4))
    return GBATTN_ERR_ALIGN;
  if ((rc = check_rope(inv_freq, rotary, factor, eps, nullptr, 0, q_weight, k_weight, B, Hq, Hkv, d)) != GBATTN_OK) return rc;
  const Rows rk{k, k_sb, k_sh, k_sl}, rv{v, v_sb, v_sh, v_sl}, rq{Hq > 0 ? q : nullptr, q_sb, q_sh, q_sl};
  if (!rows_ok(rk, B, Hkv, L) || !rows_ok(rv, B, Hkv, L) || (rq.p && !rows_ok(rq, B, Hq, L)) || !reach_ok(table_stride, B))
    return GBATTN_ERR_STRIDE;
  long long extent = 0;
  if ((rc = check_pages(k_pages, v_pages, page_stride, head_stride, slot_stride, pages, page, Hkv, d, &extent)) != GBATTN_OK)
    return rc;
  const Span q_to[1] = {dense_span(rq.p ? q_out : nullptr, static_cast<long long>(B) * L * Hq * d, 2)};
  const Span caches[2] = {pages_span(k_pages, page_stride, extent, pages), pages_span(v_pages, page_stride, extent, pages)};
  const Span in[9] = {rows_span(rk, B, Hkv, L, d), rows_span(rv, B, Hkv, L, d), rows_span(rq, B, Hq, L, d),
                      dense_span(inv_freq, rotary / 2, 8), dense_span(q_weight, d, 2), dense_span(k_weight, d, 2),
                      dense_span(table, (B - 1LL) * table_stride + table_width, 4), dense_span(lengths, B, 4),
                      dense_span(counts, B, 4)};
  if (!disjoint(q_to, 1, in, 9) || !disjoint(q_to, 1, caches, 2) || !disjoint(caches, 1, in, 9) || !disjoint(caches + 1, 1, in, 9))
    return GBATTN_ERR_ALIAS;
  RopeLaunch a = {};
  unsigned *status = nullptr;
  if ((rc = abi_device(&a.sm_count, &status)) != GBATTN_OK) return rc;
  fill_rope(a.p, inv_freq, rotary, factor, nullptr, 0, q_weight, k_weight, eps, B, Hq, Hkv, L, d);
  a.p.q = rq.p;
  a.p.k = k;
  a.p.v = v;
  fill_rows(a.p.qs, rq);
  fill_rows(a.p.ks, rk);
  fill_rows(a.p.vs, rv);
  a.p.q_out = q_out;
  a.p.k_pages = k_pages;
  a.p.v_pages = v_pages;
  a.p.page_s = page_stride;
  a.p.head_s = head_stride;
  a.p.slot_s = slot_stride;
  a.p.table = table;
  a.p.table_s = table_stride;
  a.p.table_w = table_width;
  a.p.lengths = lengths;
  a.p.counts = counts;
  a.p.page = page;
  a.p.pages = pages;
  a.p.status = status;
  a.bf16 = dtype == GBATTN_BF16;
  a.interleaved = interleaved != 0;
  a.stream = static_cast<cudaStream_t>(stream);
  return done(launch_append(a));
}

extern "C" int attn_cache_copy(void *k_pages, void *v_pages, long long page_stride, long long head_stride, long long slot_stride,
                               int pages, int page, int Hkv, int d, const int *src, const int *dst, int n, void *stream) {
  if (!k_pages || !v_pages || (n > 0 && (!src || !dst))) return GBATTN_ERR_NULL;
  if (n < 0) return GBATTN_ERR_DIMS;
  if (!head_dim_ok(d)) return GBATTN_ERR_HEAD_DIM;
  long long extent = 0;
  int rc = check_pages(k_pages, v_pages, page_stride, head_stride, slot_stride, pages, page, Hkv, d, &extent);
  if (rc != GBATTN_OK) return rc;
  const long long vecs = static_cast<long long>(Hkv) * page * (d / 8);
  if (vecs > (1 << 24)) return GBATTN_ERR_DIMS;  // 256 MB of keys in a page
  for (int i = 0; i < n; ++i)
    if (src[i] < 0 || src[i] >= pages || dst[i] < 0 || dst[i] >= pages) return GBATTN_ERR_PAGES;
  CopyLaunch a = {};
  int sm_count = 0;
  unsigned *status = nullptr;
  if ((rc = abi_device(&sm_count, &status)) != GBATTN_OK) return rc;
  if (n == 0) return GBATTN_OK;
  a.s.k = static_cast<char *>(k_pages);
  a.s.v = static_cast<char *>(v_pages);
  a.s.page_b = page_stride * 2;
  const bool dense = extent == static_cast<long long>(Hkv) * page * d;  // no gaps: one piece whatever the order
  a.s.pieces = dense ? 1 : Hkv * page;
  a.s.piece_vecs = dense ? static_cast<int>(vecs) : d / 8;
  a.s.slots = page;
  a.s.head_b = head_stride * 2;
  a.s.slot_b = slot_stride * 2;
  a.stream = static_cast<cudaStream_t>(stream);
  // Cut the list where a pair depends on an earlier one of its launch: it reads or writes a
  // page that one writes, or writes a page that one reads.  `mark` holds for each page the
  // last launch that read it (even entries) and wrote it (odd ones).
  unsigned *const mark = static_cast<unsigned *>(std::calloc(static_cast<size_t>(pages) * 2, sizeof(unsigned)));
  int *const list = static_cast<int *>(std::malloc(sizeof(int) * 2 * kCopyPairsLarge));
  rc = mark && list ? GBATTN_OK : GBATTN_ERR_MEMORY;
  unsigned launch = 1;
  a.src = list;
  a.dst = list + kCopyPairsLarge;
  int held = 0;
  for (int i = 0; rc == GBATTN_OK && i <= n; ++i) {
    const bool cut = i == n || held == kCopyPairsLarge || mark[2 * src[i] + 1] == launch || mark[2 * dst[i]] == launch ||
                     mark[2 * dst[i] + 1] == launch;
    if (cut && held) {
      a.n = held;
      rc = done(launch_cache_copy(a));
      held = 0;
      ++launch;
    }
    if (i == n || rc != GBATTN_OK || src[i] == dst[i]) continue;
    list[held] = src[i];
    list[kCopyPairsLarge + held++] = dst[i];
    mark[2 * src[i]] = launch;
    mark[2 * dst[i] + 1] = launch;
  }
  std::free(mark);
  std::free(list);
  return rc;
}

extern "C" long long attn_decode_paged_workspace_bytes(int Hq, int Hkv, int d) {
  if (Hq <= 0 || Hkv <= 0) return GBATTN_ERR_DIMS;
  if (Hq % Hkv) return GBATTN_ERR_HEADS;
  if (!head_dim_ok(d)) return GBATTN_ERR_HEAD_DIM;
  return paged_workspace_bytes(Hq / Hkv, d);
}

extern "C" int attn_decode_paged(const void *q, long long q_sb, long long q_sh, const void *k_pages, const void *v_pages,
                                 long long page_stride, long long head_stride, long long slot_stride, int pages, int page,
                                 const int *table, long long table_stride, int table_width, const int *lengths, void *o,
                                 float *lse, void *workspace, int dtype, int B, int Hq, int Hkv, int d, float scale,
                                 void *stream) {
  if (!q || !k_pages || !v_pages || !table || !lengths || !o || !lse || !workspace) return GBATTN_ERR_NULL;
  int rc = check_dims(dtype, B, Hq, Hkv, 1, d);
  if (rc != GBATTN_OK) return rc;
  if (Hq <= 0 || Hkv <= 0 || table_width <= 0 || static_cast<long long>(B) * Hq > INT_MAX / 2) return GBATTN_ERR_DIMS;
  if (Hq % Hkv) return GBATTN_ERR_HEADS;
  if (!abi_aligned(q, 16) || !abi_aligned(o, 16) || !abi_aligned(lse, 16) || !abi_aligned(workspace, 16) || !abi_aligned(table, 4) ||
      !abi_aligned(lengths, 4))
    return GBATTN_ERR_ALIGN;
  if (!std::isfinite(scale) || !(scale > 0.f)) return GBATTN_ERR_SCALE;
  const Rows rq{q, q_sb, q_sh, 0};
  if (!rows_ok(rq, B, Hq, 1) || !reach_ok(table_stride, B)) return GBATTN_ERR_STRIDE;
  long long extent = 0;
  if ((rc = check_pages(k_pages, v_pages, page_stride, head_stride, slot_stride, pages, page, Hkv, d, &extent)) != GBATTN_OK)
    return rc;
  const long long heads = static_cast<long long>(B) * Hq;
  const Span out[3] = {dense_span(o, heads * d, 2), dense_span(lse, heads, 4),
                       dense_span(workspace, attn_decode_paged_workspace_bytes(Hq, Hkv, d), 1)};
  const Span in[5] = {rows_span(rq, B, Hq, 1, d), pages_span(k_pages, page_stride, extent, pages),
                      pages_span(v_pages, page_stride, extent, pages),
                      dense_span(table, (B - 1LL) * table_stride + table_width, 4), dense_span(lengths, B, 4)};
  if (!disjoint(out, 3, in, 5)) return GBATTN_ERR_ALIAS;
  PagedLaunch a;
  PagedParams &p = a.p;
  p = {};
  if ((rc = abi_device(&a.sm_count, &p.status)) != GBATTN_OK) return rc;
  p.table = table;
  p.table_s = table_stride;
  p.table_w = table_width;
  p.lengths = lengths;
  p.page = page;
  p.pages = pages;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.d = d;
  p.G = Hq / Hkv;
  p.blocks = paged_blocks(p.G, d);
  p.box_rows = std::min(page & -page, kPagedTile);
  const int rows_at_once = paged_heads(p.G, d);
  p.q_rows = std::min(rows_at_once, p.G);
  p.tile_pages = kPagedTile / page;
  p.tile_slots = kPagedTile % page;
  p.bf16 = dtype == GBATTN_BF16;
  p.c2 = scale * 1.4426950408889634f;
  p.o = o;
  p.lse = lse;
  p.wait_limit = 1LL << 32;  // about two seconds of SM clock
  p.records = static_cast<PagedRecord *>(workspace);
  p.part_o = reinterpret_cast<float *>(p.records + kPagedMaxCtas);
  p.part_lse = p.part_o + 2LL * kPagedMaxCtas * rows_at_once * d;
  // [pages, Hkv, page, d] by strides; a dimension of one element may have any stride
  auto bytes = [](long long stride, long long count, int d) { return static_cast<cuuint64_t>(count > 1 ? stride : d) * 2u; };
  const cuuint64_t kv_dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(page), static_cast<cuuint64_t>(Hkv),
                                 static_cast<cuuint64_t>(pages)};
  const cuuint64_t kv_strides[3] = {bytes(slot_stride, page, d), bytes(head_stride, Hkv, d), bytes(page_stride, pages, d)};
  const cuuint32_t kv_box[4] = {64, static_cast<cuuint32_t>(p.box_rows), 1, 1};
  const cuuint64_t q_dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(B)};
  const cuuint64_t q_strides[2] = {bytes(q_sh, Hq, d), bytes(q_sb, B, d)};
  const cuuint32_t q_box[3] = {64, static_cast<cuuint32_t>(p.q_rows), 1};
  if (abi_encode(&a.tm_q, p.bf16, 3, q, q_dims, q_strides, q_box) || abi_encode(&a.tm_k, p.bf16, 4, k_pages, kv_dims, kv_strides, kv_box) ||
      abi_encode(&a.tm_v, p.bf16, 4, v_pages, kv_dims, kv_strides, kv_box))
    return GBATTN_ERR_TENSORMAP;
  a.stream = static_cast<cudaStream_t>(stream);
  return done(launch_decode_paged(a));
}
