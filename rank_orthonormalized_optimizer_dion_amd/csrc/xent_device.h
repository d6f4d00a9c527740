// Device helpers of the cross entropy (k_xent.hip, k_xent_few.hip).
#pragma once
#include "mm16.h"
#include "xent_types.h"

namespace dion {

namespace {

constexpr float kLog2E = 1.44269504088896341f;

// exp(x), one ulp of exp2 and x's rounding; x - y is formed first, so that the
// largest term is exactly 1.
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * kLog2E); }

// Lanes 16 r .. 16 r + 15 together (one DPP row).
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, true);
}
// quad_perm lane ^ 1, lane ^ 2, row_half_mirror, row_mirror
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp<0xb1>(v));
  v = fmaxf(v, dpp<0x4e>(v));
  v = fmaxf(v, dpp<0x141>(v));
  return fmaxf(v, dpp<0x140>(v));
}
__device__ __forceinline__ float row_sum(float v) {
  v += dpp<0xb1>(v);
  v += dpp<0x4e>(v);
  v += dpp<0x141>(v);
  return v + dpp<0x140>(v);
}

// A largest value as what is subtracted: nothing where there is no value.
__device__ __forceinline__ float base_of(float top) { return top == -INFINITY ? 0.0f : top; }

// (top, sum) of two sets of logits together.
__device__ __forceinline__ void merge(float& top, float& sum, float t2, float s2) {
  const float t = fmaxf(top, t2), b = base_of(t);
  sum = sum * exp_fast(top - b) + s2 * exp_fast(t2 - b);
  top = t;
}

// What dz needs of a row.  Rows without loss, and rows past the last, have
// `mask` zero: their dz is zero whatever their logits are.  A target outside
// the vocabulary makes its row NaN.
struct XentRow {
  float lse, a, b, c;
  int mask;
};
__device__ __forceinline__ XentRow xent_row(const XentEpi& e, int row, int t, int64_t& y) {
  XentRow r{0.0f, 0.0f, 0.0f, 0.0f, 0};
  y = -1;
  if (row < t) {
    const int64_t target = e.target[row];
    if (target != e.ignore) {
      const bool in = target >= 0 && target < e.vocab;
      const float d = in ? e.dloss[row] : NAN;
      y = in ? target : -1;
      r.lse = e.lse[row];
      r.a = d * (1.0f + e.slope * r.lse);
      r.b = d * e.share;
      r.c = d * e.keep;
      r.mask = -1;
    }
  }
  return r;
}
__device__ __forceinline__ float dz_of(float z, float lse, float a, float b, int mask) {
  const float d = a * exp_fast(z - lse) - b;
  return __uint_as_float(__float_as_uint(d) & mask);
}

}  // namespace

}  // namespace dion
