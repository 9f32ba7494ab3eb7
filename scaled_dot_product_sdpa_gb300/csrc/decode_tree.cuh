// decode_tree.cuh -- attention of several new tokens per sequence over a paged key/value cache:
// parameters, how rows are dealt out, and the launch entry point.
//
// Sequence b has n = lengths[b] cached tokens, the last c = counts[b] of them new; row t < c of its
// queries, the new token n - c + t, sees the n - c older ones and, of the new ones, those of its
// mask (bit j % 32 of word j / 32 of mask[b, t]), or without a mask those up to itself.  Over what it sees,
//     o[b, h, t] = sum_j softmax_j(scale q[b, h, t] . k_j) v_j,    lse[b, h, t] = log sum_j exp(scale q[b, h, t] . k_j)
// with keys and values of head h / (Hq / Hkv); o = 0, lse = -inf where it sees nothing and for t >= c.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace gbattn {

constexpr int kTreeMaxCtas = 160;  // persistent CTAs at most, one an SM; sizes the workspace
constexpr int kTreeTile = 128;     // keys per tile, and rows per row tile

// How the rows of a key head, its G query heads' T tokens, are dealt to row tiles of up to 128 (d = 512: 64):
// `heads` query heads x `tokens` tokens each, row g * tokens + t.  A unit of work is `tiles` row tiles
// (one, or two that share every key they read) of one sequence and key head.
struct TreeShape {
  int heads, tokens;        // of a row tile
  int tiles;                // of a unit: 1 or 2
  int token_units, head_units;
  int halves;               // of the value columns (d = 512: tensor memory holds 256 of them beside two S tiles)
  int rows;                 // stride of a row tile's rows in the workspace
  int q_rows;               // rows of a row tile's queries in shared memory (a multiple of 8)
};
constexpr int tree_div_up(int a, int b) { return (a + b - 1) / b; }
constexpr TreeShape tree_shape(int G, int T, int d) {
  TreeShape s{};
  const int tile = d > 256 ? kTreeTile / 2 : kTreeTile;  // 128 queries of 512 would leave no room for keys
  s.head_units = tree_div_up(G, G < tile ? G : tile);
  s.heads = tree_div_up(G, s.head_units);
  const int most = tile / s.heads;
  s.tiles = d <= 128 && T > most ? 2 : 1;
  s.token_units = tree_div_up(T, most * s.tiles);
  s.tokens = tree_div_up(T, s.token_units * s.tiles);
  s.halves = d > 256 ? 2 : 1;
  s.rows = tree_div_up(s.heads * s.tokens, 32) * 32;
  s.q_rows = tree_div_up(s.heads * s.tokens, 8) * 8;
  return s;
}

// Whether weights enter the second product as two 16-bit parts, or rounded to 16 bits.  With few rows of a key head (a few
// drafts) a verified token's row keeps the bits that attn_decode_paged gives it, and mostly at a small price: GB300, both parts (with sums
// in shared memory) and one, 16 rows, 8 x 32 x 8192 keys 175 and 171 us, 32 rows, 131072 x 8 x 128 96 and 91, 65536 x 8 x 256 98 and 92, but
// 262144 x 8 x 64 134 and 106.  With many the products bound the kernel, by their time and, in a long run, by their power (clocks of
// 1.4 GHz instead of 2.07): 128 rows, 1,048,576 x 8 keys x 128 728 and 609 us, 2048 new tokens of 4 prompts 764 and 656 (with sums in
// the workspace every 64 or 512 tiles; those of 128 rows would not fit shared memory).
constexpr bool tree_split_weights(int G, int T) { return static_cast<long long>(G) * T <= 32; }

// Tiles after which an accumulator's sums leave it.  The tensor cores add to it by cutting off what falls below its last bit, up to
// 2^-23 of a sum a product (half of that where the sum grows evenly): every 8 tiles where the weights have two parts, as in
// attn_decode_paged, so that the sums keep about what those parts hold (16 products a tile, 2^-17 to 2^-16); where they are
// rounded to 16 bits every 64 in fp16 (2^-15 to 2^-14) and 128 in bf16 (2^-14 to 2^-13), an eighth to a quarter and a 32nd to a 16th of a half
// step.  GB300, with two parts every 8, 16 and 32 tiles: 8 x 32 x 8192 keys x 16 rows 171, 170 and 168 us, 131072 x 8 x 128 with 32 rows 94,
// 92 and 91, 262144 x 8 x 64 134, 131 and 130, 65536 x 8 x 256 98, 95 and 92; with one, in bf16, every 64, 128 and 512: 1,048,576 x 128 rows
// 650, 598 and 588, 2048 new tokens behind 65536 1940, 1838 and 1792.
constexpr int tree_fold(int G, int T, bool bf16) { return tree_split_weights(G, T) ? 8 : bf16 ? 128 : 64; }

// Workspace: a record per CTA, then two partial results per CTA, each of `tiles` row tiles' log-sum-exps (base 2) and o
// (normalised, fp32), then the sums that leave the tensor cores' accumulators in long rows (of up to 32 rows: in shared memory).
struct TreeRecord {
  int b, kv, tu, x, cnt;  // the unit whose row tiles this CTA's last partial begins, and its sequence's new tokens
  int parts;              // partial results to join: this CTA's second, then the first of each of the following parts - 1 CTAs
  int pad[2];
};
constexpr int tree_columns(int d) { return d > 256 ? 256 : d; }          // of o in a unit
constexpr int tree_streams(int d) { return d <= 128 ? 2 : 1; }           // accumulators of a CTA
constexpr long long tree_part_floats(const TreeShape &s, int d) { return static_cast<long long>(s.tiles) * s.rows * tree_columns(d); }
constexpr long long tree_workspace_bytes(int G, int T, int d) {
  const TreeShape s = tree_shape(G, T, d);
  const long long sums = tree_split_weights(G, T) ? 0 : static_cast<long long>(tree_streams(d)) * s.rows * tree_columns(d);
  return kTreeMaxCtas * (static_cast<long long>(sizeof(TreeRecord)) + 4LL * (2 * s.tiles * s.rows + 2 * tree_part_floats(s, d) + sums));
}

struct TreeParams {
  TreeShape s;
  TreeRecord *records;                 // workspace
  float *part_lse, *part_o, *sums;     // [2 ctas][tiles][rows], [2 ctas][tiles][columns / 4][rows][4], [ctas][streams][columns / 4][rows][4]
  const int *table, *lengths, *counts; // counts null: T
  long long table_s;
  int table_w, page, pages;
  const unsigned *mask;                // null: a chain
  long long mask_sb, mask_sl;          // words from a sequence's (0: one mask for all), from a row's to the next
  int words;                           // of a row
  int B, Hq, Hkv, G, T, d;
  int box_rows;                        // rows of a TMA box: a power of two <= 128 that divides the page
  int tile_pages, tile_slots;          // kTreeTile / page, kTreeTile % page
  int fold;                            // tiles after which the sums leave an accumulator: a power of two
  int q_buffers, slots;                // of shared memory: units whose queries it holds, pieces of keys and values
  bool bf16;
  float c2;                            // scale log2(e)
  void *o;                             // [B, Hq, T, d]
  float *lse;                          // [B, Hq, T]
  unsigned *status;
  long long wait_limit;
};

struct TreeLaunch {
  CUtensorMap tm_q, tm_k, tm_v;
  TreeParams p;
  int sm_count;
  cudaStream_t stream;
};

cudaError_t launch_decode_tree_64(const TreeLaunch &a);
cudaError_t launch_decode_tree_128(const TreeLaunch &a);
cudaError_t launch_decode_tree_256(const TreeLaunch &a);
cudaError_t launch_decode_tree_512(const TreeLaunch &a);
inline cudaError_t launch_decode_tree(const TreeLaunch &a) {
  switch (a.p.d) {
    case 64: return launch_decode_tree_64(a);
    case 128: return launch_decode_tree_128(a);
    case 256: return launch_decode_tree_256(a);
    default: return launch_decode_tree_512(a);
  }
}

}  // namespace gbattn
