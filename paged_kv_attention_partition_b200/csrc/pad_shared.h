// Shared-prefix decode: launch parameters and the work schedule that the main
// kernel and the merge both derive from the lengths.
//
// Work is laid on one line.  An item is a set of query rows of one KV head
// against a token range: a prefix item is a block of sequences (their heads of
// the group, up to kSharedRows rows) against the shared pages; a rest item is
// one sequence against its own tokens behind the prefix.  An item costs w_item
// + chunks * (weight of a chunk), a chunk being `chunk` tokens.  CTA i of G takes
// the line's part [i q, (i+1) q), q = ceil(total / G): it may start and end
// inside an item, and a cut falls on the chunk whose cost contains it.  So every
// CTA gets the same work whatever the lengths, no unit is empty, and long
// sequences are split as far as the GPU needs.
//
// A unit is (item, CTA).  Items and CTAs both only grow along the line, so
// item + CTA numbers the units without a table, and that number places a unit's
// partial results.  (The walk itself: pad_shared_walk.cuh.)
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "pad_internal.h"

namespace pad {

constexpr int kTileRows = 128;  // query rows of one tensor-core tile
constexpr float kTinyScale = 1.4e-45f;  // the smallest positive fp32: stands in for a score scale of 0

// Query rows of a unit: two tiles, one at D = 256 (whose fp32 accumulator takes
// half of the tensor memory).
__host__ __device__ constexpr int shared_rows(int D) { return D == 256 ? kTileRows : 2 * kTileRows; }
// Tokens of a chunk.
constexpr int kSharedChunk = 64;
// Chunks that one accumulator takes at most (even: a piece starts on the accumulator that
// the unit started on).  The tensor core cuts off what an addition to its fp32 sums
// carries beyond them, so a sum of n products loses up to n 2^-23 of itself: measured,
// 2^-13 over 85000 tokens, 0.3 % over 1.4 million, 1.3 % over 5.4 million.  Longer units go
// through in pieces, added up in fp32 with rounding; that also keeps every role's wait for
// another's unit at a few milliseconds.
constexpr int kSharedPiece = 1024;
// Accumulators: two tiles of rows, or one tile's even and odd chunks.
__host__ __device__ constexpr int shared_accs(int D) { return D == 256 ? 1 : 2; }

// What one copy of K or V brings: rows of 128-byte column blocks, laid out in groups
// of 8 rows x all column blocks.
enum SharedBox : int32_t {
  kBoxPage = 0,   // a page's rows (at most a chunk's): (128 bytes, 8 rows, column blocks, row groups, block and head)
  kBoxGroup = 1,  // 8 rows: (128 bytes, 8 rows, column blocks, head, block), for caches whose block stride is not
                  // a multiple of the head stride
  // (an E4M3 cache: a page's rows, at most a chunk's, as they are: (head_dim, slot, head, block))
  kBoxRows = 2,   // pages below 8 slots: one column block of a page: (128 bytes, rows, column block, head, block)
};

struct SharedParams {
  CUtensorMap tmk, tmv;    // caches, boxes as box_kind says
  CUtensorMap tmqp, tmqr;  // q: boxes of 64 head_dim x gt heads x nseq sequences (prefix), x 1 (rest)
  const int32_t *shared_table;
  const int32_t *tables;
  int64_t table_stride;
  const int32_t *seq_lens;
  int32_t n_shared;    // pages of the prefix
  int32_t max_blocks;  // table width, >= n_shared
  int32_t num_blocks;
  int32_t B, Hq, Hkv, g;
  int32_t HT, gt;      // head tiles of a group, heads of one (the last may have fewer)
  int32_t nseq, nrb;   // sequences of a prefix row block, row blocks
  int32_t bs_log2;
  int32_t box_kind, box_log2;  // SharedBox, rows of a box
  int32_t box_pitch;           // E4M3: bytes from box to box, at least 128
  int32_t blk_heads;           // kBoxPage: block stride / head stride
  int32_t ctas;
  int32_t w_item, w_pre1, w_pre2, w_rest;  // cost of an item; of a prefix chunk of one and two tiles, of a rest chunk
  float scale_log2, v_scale;
  const float *sinks;
  uint16_t *out;
  int64_t o_sb, o_sh;
  float *lse;
  int64_t lse_sb, lse_sh;
  float *o_part;     // [part rows, D], normalised by the unit's own sum
  float *lse_part;   // [part rows], log2 units
  int64_t rest_row0; // first part row of the rest units
  int32_t pre_rows, rest_rows;  // part rows of a prefix and a rest unit
  uint32_t *err;
};

// Part rows: an accumulator each for one-tile units.
__host__ __device__ inline int shared_part_rows(int rows, int D) {
  return shared_accs(D) == 2 && rows <= kTileRows ? 2 * rows : rows;
}

cudaError_t launch_shared(const SharedParams &p, int D, bool kv_fp8, cudaStream_t s);

}  // namespace pad
