// What the kernels of the linear cross entropy share: the workspace, the
// pieces of the vocabulary, and the launches of one piece.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {

// Columns of the logits that leave one (maximum, sum) a row.
constexpr int CE_PART = 64;
// Row tiles are CE_ROWS high: the compacted rows are padded to that with zeros.
constexpr int CE_ROWS = 256;
// Chunks of the vocabulary over which dhidden is summed: a chunk's sum stays in
// one accumulator, the chunks are added in FP32 in order.  Set by the type
// alone, so that a row's sums do not depend on the batch.
constexpr int CE_CHUNK_BF16 = 8192, CE_CHUNK_F32 = 512;

// Of a row that counts, in compacted order.  In bfloat16 a row of g is kept
// times a factor within 2^-8 of 1, chosen so that the target's entry, the
// largest by far in most rows, is a bfloat16 number: rounding it would put one
// and the same relative error of up to 2^-8 on nearly all of the row's dhidden
// and of its part of dweight.  The factor is taken back out in FP32 from dhidden, and
// from the row of h that meets the row of g in dweight's product (rounded
// element by element, errors that have nothing to do with one another).
struct CeRow {
  float lse2;  // lse * log2(e)
  float c;     // scale * dloss * (1 + 2 z lse), times the factor
  float b;     // the target's entry of g, times the factor
  int target;  // -1: a row of padding
};

struct CeLayout {
  int tpad, nchunks, chunk, per_piece, npieces, nparts;
  int64_t dp;       // row length of the compacted rows, elements
  int64_t ldw;      // row length of the weights' copy (0: the caller's weights are read)
  int64_t ldg;      // row length of a piece of g
  size_t count, row_of, place, rows, inv, hc, hc2, wc, part, xt, g, acc, bytes;
};

inline CeLayout ce_layout(const CeArgs &a, int mode) {
  CeLayout l = {};
  const int64_t e = a.f32 ? 4 : 2;
  l.tpad = (int)round_up(std::max(a.T, 1), CE_ROWS);
  l.chunk = a.f32 ? CE_CHUNK_F32 : CE_CHUNK_BF16;
  l.nchunks = (int)ceil_div(a.V, l.chunk);
  l.nparts = (int)ceil_div(a.V, CE_PART);
  l.dp = round_up(a.D, 64);
  // Tensor maps want rows on 16-byte boundaries; other weights are copied first.
  l.ldw = !a.f32 && (a.ld_w % 8 || ((uintptr_t)a.weight & 15)) ? round_up(a.D, 8) : 0;
  // A piece: as many chunks as keep g and dhidden's sums within twice the size
  // of L2, one at least; all pieces about equally long.  With only a few chunks a
  // piece its sums would be written and read once more for little, so
  // then it is one chunk, added to the sums before it in the product's epilogue.
  const int64_t budget = (int64_t)256 << 20;
  int64_t per = std::min(budget / (l.tpad * (int64_t)l.chunk * e), budget / (l.tpad * l.dp * 4));
  if (per < 3 && per < l.nchunks) per = 1;
  l.per_piece = (int)std::min<int64_t>(std::max<int64_t>(per, 1), l.nchunks);
  l.per_piece = (int)ceil_div(l.nchunks, ceil_div(l.nchunks, l.per_piece));
  l.npieces = (int)ceil_div(l.nchunks, l.per_piece);
  l.ldg = std::min((int64_t)l.per_piece * l.chunk, round_up(a.V, CE_ROWS));
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t r = at;
    at += (size_t)round_up(bytes, 1024);
    return r;
  };
  l.count = take(256);
  l.row_of = take((int64_t)l.tpad * 4);
  l.place = take((int64_t)l.tpad * 4);
  l.rows = take((int64_t)l.tpad * sizeof(CeRow));
  l.inv = take((int64_t)l.tpad * 4);
  l.hc = take(l.tpad * l.dp * e);
  l.hc2 = take(!a.f32 && (mode & CE_GRAD) ? l.tpad * l.dp * e : 0);
  l.wc = take(l.ldw ? a.V * l.ldw * e : 0);
  l.part = take(mode & CE_LOSS ? (int64_t)l.nparts * l.tpad * 8 : 0);
  l.xt = take(mode & CE_LOSS ? (int64_t)l.tpad * 4 : 0);
  l.g = take(mode & CE_GRAD ? l.tpad * l.ldg * e : 0);
  // One plane for each chunk of a piece, where a piece has several, and the
  // sum over the pieces, where there are several.
  const int64_t planes = (l.per_piece > 1 ? l.per_piece : 0) + (l.npieces > 1 ? 1 : 0);
  l.acc = take(mode & CE_GRAD ? planes * l.tpad * l.dp * 4 : 0);
  l.bytes = at;
  return l;
}

// What the matrix products of one call see.
struct CeMats {
  int V, D, tpad;
  int64_t ldh, ldw, ldg;
  const int *count;     // rows that count
  const int *row_of;    // their places among the caller's rows
  const CeRow *rows;
  const float *inv;     // 1 / the rows' factors
  const void *h, *h2, *w;  // compacted rows; over their factors; weights
  void *g;              // [tpad, ldg]
  float scale;
  float2 *part;         // [nparts, tpad]
  float *xt;            // [tpad]: the targets' logits, in units of log 2
  // gradients
  bool gf32, accumulate;
  void *dh, *dw;
  int64_t ld_dh;
  float *acc, *planes;  // [tpad, ldh] each
  int *status;
};

// One piece of the vocabulary: columns [v0, v0 + n), chunk columns a chunk.
struct CePiece {
  int v0, n, chunk, nchunks;
  bool first, last;
};

// The logits' (maximum, sum) of every 64 columns without the targets', and the targets' logits.
cudaError_t ce_tc_stats(const CeMats &m, cudaStream_t stream);
cudaError_t ce_simt_stats(const CeMats &m, cudaStream_t stream);
// g of a piece.
cudaError_t ce_tc_logits_grad(const CeMats &m, const CePiece &p, cudaStream_t stream);
cudaError_t ce_simt_logits_grad(const CeMats &m, const CePiece &p, cudaStream_t stream);
// Its two products: dweight's rows of the piece; dhidden's sums, into a plane
// for each chunk where a piece has several, else added to what the pieces
// before have left in acc, and written out by the last.
cudaError_t ce_tc_grads(const CeMats &m, const CePiece &p, cudaStream_t stream);
cudaError_t ce_simt_grads(const CeMats &m, const CePiece &p, cudaStream_t stream);

}  // namespace moe
