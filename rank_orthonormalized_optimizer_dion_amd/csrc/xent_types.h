// Types and launchers of the output head's cross entropy (k_xent.hip,
// xent_api.hip).
#pragma once
#include "linear_types.h"

namespace dion {

// What becomes of the logits z = x W^T of a piece of the vocabulary, columns
// j0 .. j0 + n - 1 of `vocab`.
struct XentEpi {
  const int64_t* target;   // t
  int64_t ignore;          // target of rows without loss
  int64_t vocab;
  int32_t j0;
  // forward: per row and partial column (a wavefront's or a workgroup's share
  // of the vocabulary, `part` columns of t values) the largest logit, the sum
  // of exp(z - largest) and, with label smoothing, the sum of z; and the
  // target's logit
  int32_t col0;            // first partial column of the piece
  float* top;
  float* sum;
  float* total;            // or null
  float* hit;              // t
  // backward: dz in bfloat16 planes, zero past the piece's columns and (with
  // `prows` > t) rows
  const float* lse;        // t
  const float* dloss;      // t
  float keep, share;       // 1 - smoothing, smoothing / vocab
  float slope;             // 2 z-loss
  uint16_t* dz;
  int64_t pitch;           // columns, padded
  int64_t ld, plane;       // elements from row to row, from plane to plane
  int32_t prows, planes;
};

struct XentJoin {
  const float* top;
  const float* sum;
  const float* total;
  const float* hit;
  const int64_t* target;
  int64_t ignore, vocab;
  float* loss;             // or null
  float* lse;              // or null
  int32_t t, cols;
  float keep, smoothing, z_loss;
};

// Partial columns of a piece of n columns.
constexpr int kXentGroup = 16;   // columns of a workgroup with few tokens
inline int64_t xent_tile_cols(int64_t ty) { return 2 * ty; }   // two wavefronts across a tile
inline int64_t xent_group_cols(int64_t n) { return (n + kXentGroup - 1) / kXentGroup; }

// z by tiles, by the matrix cores for up to 64 tokens, by rows for up to 8
// (s.out: dtype of x and W only); grad: backward.
hipError_t launch_xent_product(const LinProduct& p, const XentEpi& e, bool grad, int tile, hipStream_t st);
hipError_t launch_xent_skinny(const LinSkinny& s, const XentEpi& e, bool grad, hipStream_t st);
hipError_t launch_xent_rows(const LinSkinny& s, const XentEpi& e, bool grad, bool vec, hipStream_t st);
hipError_t launch_xent_join(const XentJoin& j, hipStream_t st);

}  // namespace dion
