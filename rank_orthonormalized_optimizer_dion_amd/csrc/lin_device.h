// Device helpers shared by the linear layer and the cross entropy
// (k_linear.hip, k_xent.hip, k_xent_few.hip): element access and plane pairs.
#pragma once
#include "linear_types.h"
#include "mm16.h"

namespace dion {

namespace {

__device__ __forceinline__ float load_value(const void* p, int64_t o, int dtype) {
  return dtype ? bf16_to_f32(static_cast<const uint16_t*>(p)[o]) : static_cast<const float*>(p)[o];
}
__device__ __forceinline__ void store_value(void* p, int64_t o, int dtype, float v) {
  if (dtype) static_cast<uint16_t*>(p)[o] = to_bf16(v);
  else static_cast<float*>(p)[o] = v;
}

// Eight consecutive values, `left` of which exist, as vectors where all do:
// global memory takes vector accesses at any address.
__device__ __forceinline__ void load8(const void* p, int64_t o, int dtype, int left, float (&v)[8]) {
  if (left >= 8) {
    if (dtype) {
      u32x4 u;
      __builtin_memcpy(&u, static_cast<const uint16_t*>(p) + o, 16);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(u[k] << 16);
        v[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
      }
    } else {
      f32x4 a, b;
      __builtin_memcpy(&a, static_cast<const float*>(p) + o, 16);
      __builtin_memcpy(&b, static_cast<const float*>(p) + o + 4, 16);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = a[k];
        v[4 + k] = b[k];
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < left ? load_value(p, o + k, dtype) : 0.0f;
  }
}
__device__ __forceinline__ void store8(void* p, int64_t o, int dtype, int left, const float (&v)[8]) {
  if (left >= 8) {
    if (dtype) {
      uint16_t h[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) h[k] = to_bf16(v[k]);
      const u32x4 u = pack8(h);
      __builtin_memcpy(static_cast<uint16_t*>(p) + o, &u, 16);
    } else {
      const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
      __builtin_memcpy(static_cast<float*>(p) + o, &a, 16);
      __builtin_memcpy(static_cast<float*>(p) + o + 4, &b, 16);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) store_value(p, o + k, dtype, v[k]);
  }
}

// Plane pairs of the reduction's segments, one hexadecimal digit per segment:
// looked up without a branch, which would cut the product's loop into pieces
// that the scheduler cannot fill (float32 backward, 1021 tokens, 2051 x 773: 144 to 133 us).
struct Pairs {
  uint32_t a, b;
};
__device__ __forceinline__ Pairs plane_pairs(int nseg) {
  // six: x = hi + mid + lo; (mid mid) (lo hi) (hi lo) (mid hi) (hi mid)
  // (hi hi), smallest first; the dropped pairs are below 3 2^-24 of the
  // product.  two: lo, then hi of A.  one: plane 0.
  return nseg == 6 ? Pairs{0x001021u, 0x010201u} : nseg == 2 ? Pairs{0x01u, 0u} : Pairs{0u, 0u};
}

// The sum over a product's plane pairs.  One pair has a loop of its own: half
// of the scalar instructions between its matrix instructions.
template <class S>
__device__ __forceinline__ void lin_product_tile(const LinProduct& p, const typename S::A& ta, const typename S::B& tb,
                                                 int kbeg, int kend, u32x4* smem, typename S::Acc (&acc)[S::FM][S::FN]) {
  const Planes16 planes{p.a, p.b, p.sa, p.sb};
  if (p.nseg == 1) {
    tile_product<S>(ta, tb, planes, 1, [](int, int& a, int& b) { a = b = 0; }, kbeg, kend, smem, acc);
    return;
  }
  const Pairs pairs = plane_pairs(p.nseg);
  tile_product<S>(ta, tb, planes, p.nseg,
                  [pairs](int i, int& a, int& b) {
                    a = (pairs.a >> (4 * i)) & 15;
                    b = (pairs.b >> (4 * i)) & 15;
                  },
                  kbeg, kend, smem, acc);
}

template <int TILE, LinKind KIND>
using LinShape = Shape16<B16, TILE, TILE, TILE / 64, 2, 1, KIND == kLinDw, KIND != kLinForward>;

// The first of several planes of x.  A finite x above bfloat16's largest
// number would round to infinity and leave -infinity for the next plane; it
// is cut off instead (float32's largest and bfloat16's share the exponent),
// which leaves a remainder of 16 bits that two planes hold exactly.
__device__ __forceinline__ uint16_t first_plane(float x) {
  const uint16_t h = to_bf16(x);
  const uint32_t b = __float_as_uint(x);
  return (h & 0x7fff) == 0x7f80 && (b & 0x7fffffffu) < 0x7f800000u ? static_cast<uint16_t>(b >> 16) : h;
}

}  // namespace

}  // namespace dion
