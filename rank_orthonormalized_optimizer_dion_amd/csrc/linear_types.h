// Types and launchers of the linear layer (k_linear.hip, linear_api.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dion {

// The output side of a product: y = act(acc + bias) + residual with z =
// acc + bias kept on request, or out (+)= acc.
struct LinOut {
  void* y;
  int64_t ldy;
  const float* bias;       // or null
  const void* residual;    // or null
  int64_t ldr;
  void* z;                 // or null
  int64_t ldz;
  int32_t act;             // DION_ACT_*
  int32_t dtype;           // of y, residual and z: 0 float32, 1 bfloat16
  int32_t accumulate;      // out += acc (y only, no bias / act / residual)
  int32_t wide;            // the residual is float32 whatever dtype is
};

// C (M x N) = sum over `nseg` plane pairs of A B^T, reduction length K.
struct LinProduct {
  const uint16_t* a;
  const uint16_t* b;
  int64_t lda, ldb, sa, sb;   // pitches; elements from plane to plane
  int32_t M, N, K;
  int32_t nseg;               // 1; 2: A in two planes; 6: both operands in three
  int32_t tx, ty;
  int32_t items;              // workgroups
  int32_t full, slices;       // mm16.h, Work16
  float* part;
  uint32_t* count;
  LinOut out;
};

// Operand layouts of the three products (see mm16.h: K-major or x-major).
enum LinKind : int32_t {
  kLinForward = 0,   // x W^T:   both K-major
  kLinDx,            // dz W:    K-major, x-major
  kLinDw,            // dz^T x:  both x-major
};

struct LinPack {
  const void* src;      // rows x cols, pitch ld; float32 or bfloat16
  int64_t ld;
  const void* z;        // pre-activation (dz = src act'(z)), or null
  int64_t ldz;
  uint16_t* dst;        // planes, pitch `pitch` >= cols, zero past cols and rows; or null
  int64_t pitch, plane;
  float* sums;          // partial column sums, one row per chunk; or null
  int64_t rows;
  int64_t prows;        // rows of the planes: `rows` up to a whole reduction stage
  int32_t cols, chunk;  // rows per workgroup
  int32_t act, dtype, planes;
  int32_t gx, blocks;   // workgroups across the columns, and in all
};

// Up to three copies in one launch, which also clears the arrival counters
// of the products that follow.
constexpr int kLinPacks = 3;
struct LinPacks {
  LinPack p[kLinPacks];
  uint32_t* count;
  int32_t n, counts;
};

struct LinSkinny {
  const void* x;
  const void* w;
  int64_t ldx, ldw;
  int32_t t, n, k;
  LinOut out;
};

// k_lin_skinny up to this many tokens, tiles beyond.  Timed both ways: 17 and 33
// tokens, 3072 -> 8192 14.7 and 21.3 us against 23.7 and 24.6; 64 tokens 768 -> 768
// 8.3 us against 9.4, but 8192 -> 3072 37.8 us against 25.9.
constexpr int kSkinnyTokens = 64;
// k_lin_rows (float32, or rows not 16-byte aligned) up to this many: 8 tokens
// of float32 3072 -> 8192 52 us, as split planes on tiles 100 us.
constexpr int kRowTokens = 8;

hipError_t launch_lin_product(const LinProduct& p, LinKind kind, int tile, hipStream_t st);
hipError_t launch_lin_packs(const LinPacks& p, hipStream_t st);
hipError_t launch_lin_colsum(const float* part, int chunks, int n, float* out, int accumulate,
                             hipStream_t st);
hipError_t launch_lin_skinny(const LinSkinny& p, hipStream_t st);
hipError_t launch_lin_rows(const LinSkinny& p, bool vec, hipStream_t st);

}  // namespace dion
