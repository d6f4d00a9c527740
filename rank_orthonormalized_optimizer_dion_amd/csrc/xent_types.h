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
  float* dz32;             // float32 tiles: dz as it is
  int64_t pitch, plane;    // elements from row to row, from plane to plane
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

// Partial columns of a launch of tiles: one per wavefront across a tile.
inline int64_t xent_tile_cols(int64_t ty) { return 2 * ty; }
inline int64_t xent_tile_cols32(int64_t ty) { return 4 * ty; }

// float32 tiles (mm32.h): C (M x N) = sum of A B^T over K.
constexpr int kXentM32 = 128, kXentN32 = 256;
struct XentProduct32 {
  const float* a;
  const float* b;
  int64_t lda, ldb;
  int32_t M, N, K;
  int32_t tx, ty, items;   // workgroups
  int32_t full, slices;    // mm16.h, Work16
  float* part;
  uint32_t* count;
  float* out;              // dx, dW
  int64_t ldo;
  int32_t accumulate;
  int32_t apart;           // dx, dW: cut tiles are added up by a launch of their own
};
// Cut tiles of at least this many slices, which one workgroup per tile would
// read one after the other.
constexpr int kXentApart = 6;
enum XentKind32 { kXentStats32 = 0, kXentDz32, kXentDx32, kXentDw32 };
hipError_t launch_xent_f32(const XentProduct32& p, const XentEpi& e, XentKind32 kind, hipStream_t st);

// Few tokens (k_xent_few.hip).
// Tokens: in bfloat16 up to 64 for gradients, whose dz these kernels hold in two
// planes (as the linear layer's, kLinFewTokens; the tiles hold it in one: 64 tokens,
// 2048 -> 32000 133 us, as tiles 130; 40 tokens 120 and 129; 64 tokens, 4096 -> 32000
// 234 and 265, 768 -> 50257 129 and 99), and for the forward where the tiles would
// need copies of x or W (2048 -> 32000 at an odd pitch, 64 tokens 71 us, 65 as tiles
// 110); up to 32 in the forward where they read them in place and in float32 (32
// tokens: 82 us forward, 65 as tiles 94, 64 of them 159).
constexpr int kXentFew16 = 64, kXentFew = 32;
constexpr int kFewDwRows = 64;     // rows of dW of a wavefront
// Bytes of W from which it is read past the caches, which it would only sweep.
// Forward and backward in turn, through and past them: 24 tokens in float32, 2048
// -> 26000 (203 MiB) 237 and 252 us, -> 32000 (250 MiB) 295 and 284; 8 tokens in
// bfloat16, 4096 -> 32000 (250 MiB) 257 and 223, -> 128000 945 and 914.
constexpr int64_t kFewFar = int64_t{224} << 20;
struct XentFew {
  const void* w;           // n rows of k
  int64_t ldw;
  int32_t n, k, t;
  const void* x;           // t rows: planes in bfloat16, 16-byte aligned, or x itself
  int64_t ldx, xplane;
  int32_t kx;              // columns that are there (and zero from k on)
  int32_t tp;              // tokens of the transposed operands: 32 or 64
  int32_t far;             // W past the caches
  const uint16_t* xt;      // planes of k x tp
  int64_t xtplane;
  uint16_t* dzt;           // planes of pitch x tp
  int64_t dztplane;
};
struct XentPrep {
  const void* x;
  int64_t ldx;
  int32_t t, k, tp;
  uint16_t* xp;            // planes of t x ldp, zero past k; or null
  int64_t ldp, xplane;
  uint16_t* xt;            // or null
  int64_t xtplane;
  int32_t first;           // workgroups of dz's launch before those that make xt
};
struct XentDw {
  void* dw;
  int64_t ld;
  int32_t cols;            // of a workgroup
  int32_t accumulate;
  int32_t down, tiles;     // workgroups down the rows, and in all (set at the launch)
};
struct XentDxSum {
  const float* part;       // `parts` times t x k
  int32_t parts, t, k;
  void* dx;                // or null: nothing to do
  int64_t ld;
  int32_t dtype;
};
// Blocks of 16 rows of W that a workgroup turns into z at a time.
int few_rows(int t, int64_t n, bool f32, bool grad, bool far);
// raw: x as it is (at most 16 tokens, no grad); groups: forward's workgroups,
// each of which leaves one partial column; prep (grad): first, and xt or null
hipError_t launch_few_z(const XentFew& f, const XentEpi& e, const XentPrep& prep, bool f32, bool grad, bool raw, int rt,
                        int groups, hipStream_t st);
hipError_t launch_few_prep(const XentPrep& a, bool f32, hipStream_t st);
hipError_t launch_few_dx(const XentFew& f, const XentEpi& e, bool f32, int parts, float* part, hipStream_t st);
hipError_t launch_few_dxsum(const XentDxSum& s, hipStream_t st);
hipError_t launch_few_dw(const XentFew& f, const XentDw& d, const XentDxSum& sum, bool f32, hipStream_t st);

// bfloat16 operands in a layout that the tiles read (rows x cols of pitch ld, to
// prows x pitch), and the cut tiles' arrival counters cleared.
struct XentCopy {
  const uint16_t* src;
  int64_t ld;
  int64_t rows, prows;
  int32_t cols;
  uint16_t* dst;
  int64_t pitch;
  int32_t blocks;          // set at the launch
};
struct XentCopies {
  XentCopy c[2];
  uint32_t* count;         // or null
};
hipError_t launch_xent_copies(XentCopies a, hipStream_t st);

// z by tiles; grad: backward.
hipError_t launch_xent_product(const LinProduct& p, const XentEpi& e, bool grad, int tile, hipStream_t st);
hipError_t launch_xent_join(const XentJoin& j, hipStream_t st);

}  // namespace dion
