// Structures and launch interface of the backward pass and of the learned
// relative position bias.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <vector>

#include "fa_internal.h"
#include "fa_kernel.h"

namespace fa {

// Work item of a backward kernel: one (sequence, head, 128-row tile). In the
// query list the tile is 128 query rows and [lo, hi) are its key tiles; in
// the key list it is 128 keys and [lo, hi) are its query tiles. Tiles in
// [full_lo, full_hi) need no element mask.
struct BwdItem {
  int32_t b, h, tile;
  int32_t stat;  // row-statistics block: the tile's own (query list), or that
                 // of the (sequence, head)'s query tile 0 (key list)
  int32_t lo, hi, full_lo, full_hi;
  int32_t span;  // key list: this key tile's KeySpan; dQ list: that of key tile 0
  int32_t pad[3];
};
static_assert(sizeof(BwdItem) == 48, "BwdItem layout");

// Where the key walk writes the dS of a key tile: the tile of dS of query tile
// t in [lo, hi) is first + t. One per key tile, [h][key tiles of all
// sequences].
struct KeySpan {
  int32_t first, lo, hi, pad;
};
static_assert(sizeof(KeySpan) == 16, "KeySpan layout");

// Query tiles that see keys [c0, c0 + 128) of sequence s: [lo, hi) holds
// every tile with a visible pair; in [full_lo, full_hi) every stored row sees
// every stored key of the tile (keys past the sequence's end are not stored
// and rows past its end have zero weight, so neither needs a mask).
FA_HD TileRange key_tile_rows(const SeqRec& s, int64_t c0) {
  TileRange t{0, 0, 0, 0};
  if (c0 >= s.skv || s.sq <= 0) return t;
  const int64_t c1 = imin64(c0 + kTileN, s.skv) - 1;  // last stored key
  // Row i sees key j when i >= j - hi_off (any i for j < prefix) and
  // i <= j - lo_off.
  const int64_t i_first = s.prefix > c0 ? 0 : imax64(0, c0 - s.hi_off);
  const int64_t i_last = imin64(int64_t(s.sq) - 1, c1 - s.lo_off);
  if (i_first > i_last) return t;
  t.lo = int32_t(i_first / kTileM);
  t.hi = int32_t(i_last / kTileM + 1);
  t.full_lo = t.full_hi = t.lo;
  if (s.flags & kSeqDenseMask) return t;
  const int64_t a = s.prefix > c1 ? 0 : imax64(0, c1 - s.hi_off);
  const int64_t z = imin64(int64_t(s.sq) - 1, c0 - s.lo_off);  // last row that sees key c0
  if (a > z) return t;
  int64_t f_lo = (a + kTileM - 1) / kTileM;
  int64_t f_hi = z == int64_t(s.sq) - 1 ? z / kTileM + 1 : (z + 1) / kTileM;
  f_lo = imax64(f_lo, t.lo);
  f_hi = imin64(f_hi, t.hi);
  if (f_hi > f_lo) {
    t.full_lo = int32_t(f_lo);
    t.full_hi = int32_t(f_hi);
  }
  return t;
}

// Sums of the bias's gradient by distance that a key tile writes: entry e
// stands for the distance e - reach - kRelPad (a tile that holds a distance
// inside (-reach, reach) reaches up to 254 past either end).
FA_HD int32_t rel_width(int32_t reach) { return 2 * reach + 1 + 2 * kRelPad; }

// A bias table and its copy by distance (see RelBias).
struct RelTable {
  const float* table;        // [num_buckets][N]
  const int32_t* bucket_of;  // device, [2 reach + 1]
  float* ext;                // out: [N][4][rel_row(reach)]
  int32_t N, reach;
};
// Lays the table out by distance, and sets n_zero words at `zero` to 0.
cudaError_t launch_rel_expand(const RelTable& t, unsigned int* zero, int64_t n_zero,
                              cudaStream_t stream);

// ------------------------------------------------------------- the backward
struct __align__(64) BwdParams {
  CUtensorMap tm_q, tm_k, tm_v, tm_do;
  const SeqRec* seqs;
  const BwdItem* q_items;
  const BwdItem* k_items;
  const BwdItem* g_items;    // two query tiles each, for the dQ kernel
  const KeySpan* spans;
  // dS in bf16 (see launch_bwd), or null: tiles of [16][128 keys][8 queries].
  __nv_bfloat16* ds;
  // Row statistics, one block of 2 x 128 floats per query tile: the negated
  // lse in log2 units (-inf for rows that see no key or are not stored, so
  // that their weights are 0 without a mask), then dlse - delta.
  float* stats;
  // Dense attenMask, else null: one bit per pair, 1 = hidden, 32 keys of a
  // query row or 32 query rows of a key to a word (see BwdMaskParams).
  const uint32_t* bits_q;
  const uint32_t* bits_k;
  unsigned int* err_word;
  const void* q;             // bf16 operands and gradients, one layout
  const void* k;
  const void* v;
  const void* o;
  const void* d_o;
  const float* lse;
  const float* d_lse;        // or null
  void* dq;
  void* dk;
  void* dv;
  const float* slopes;       // ALiBi, else null
  RelBias rel;
  RelTable rel_table;        // source of rel.ext, laid out with the row statistics
  // Gradient of the bias by distance: one row of rel_width sums per key tile
  // (indexed by its span), else null.
  float* rel_part;
  unsigned int* rel_done;    // [N] counters of launch_rel_reduce, set to 0 with the statistics
  int64_t q_sb, q_sh, q_st;  // element strides of Q, O and their gradients
  int64_t k_sb, k_sh, k_st;  // of K, V and their gradients
  int64_t l_sb, l_sh;        // of lse
  int32_t m_sb, m_sh;        // mask plane = b * m_sb + h * m_sh
  int32_t m_rows, m_keys;    // query rows and keys, rounded up to whole tiles
  int32_t alibi;             // fa_alibi_t
  unsigned int* claims;      // claimed items of the three lists, 0 at the start
  int32_t n_claims;          // words to set to 0 with the statistics
  int32_t n_q, n_k, n_g;     // items
  int32_t tnd;
  float scale, scale_log2;
  uint64_t timeout_ns;
};

// Head dims at which dS may be written out (the host's rule and what it
// measured: refresh_lists); the kernels of the others have no code for it.
constexpr bool bwd_may_write_ds(int64_t D) { return D == 128; }

// dQ, dK, dV and rel_part.
//
// Without p.ds by two walks that need nothing of each other: dQ by query tiles
// (S, dP, dQ), dK and dV by key tiles (S, dP, dV, dK): seven products a pair
// of tiles. With p.ds the key walk also writes dS to memory, 32 KB a pair of
// tiles, and a third kernel multiplies it by K: five products. The matrix
// products run into the card's power limit, so at head dim 128 two products
// less are worth the memory traffic once there is enough work (the host's rule
// and what it measured: refresh_lists).
cudaError_t launch_bwd(int D, const BwdParams& p, int num_sms, cudaStream_t stream,
                       const char** why);

// Dense masks, one pass over the bytes: classifies every 128 x 128 tile of
// every plane and packs it both ways,
//     bits_q[plane][key / 32][row],   bits_k[plane][row / 32][key]
// (rows and keys rounded up to whole tiles, pairs past the end hidden), so that
// a thread of either walk reads one word per 32 pairs, next to its neighbours'.
// Then gives the query, key and dQ items and the spans their ranges from the
// classes: [lo, hi) from the first to the last tile with a visible pair, the
// longest run of fully visible ones.
struct BwdMaskParams {
  const uint8_t* mask;   // [planes][Sq][Skv], nonzero = masked
  uint32_t* bits_q;
  uint32_t* bits_k;
  uint8_t* cls;          // [plane][n_qt][n_kt], fa_tile_class_t
  SeqRec geo;            // the geometry every sequence shares
  BwdItem* q_items;
  BwdItem* k_items;
  BwdItem* g_items;
  KeySpan* spans;
  int64_t planes;
  int32_t m_sb, m_sh;    // plane = b * m_sb + h * m_sh
  int32_t n_q, n_k, n_g, n_qt, n_kt;
};

// Row statistics of every query tile (see BwdParams::stats), with a bias its
// layout by distance, with a mask (planes > 0) the above.
cudaError_t launch_bwd_stats(int D, const BwdParams& p, const BwdMaskParams& mask,
                             cudaStream_t stream);

// dtable[c][h] = the sum of rel_part over head h's key tiles (rows
// [h * tiles, (h + 1) * tiles) of rel_part) and the distances of bucket c, in
// a fixed order. dist: scratch, fp64 [N][rel_width]; done: [N], 0.
cudaError_t launch_rel_reduce(const float* rel_part, double* dist, unsigned int* done,
                              const int32_t* bucket_of, float* dtable, int32_t N, int32_t tiles,
                              int32_t num_buckets, int32_t reach, cudaStream_t stream);

}  // namespace fa
