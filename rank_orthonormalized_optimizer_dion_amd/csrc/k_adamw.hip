// AdamW over a list of tensors in one pass: the kernel behind
// dion_adamw_step.
//
//   g = c G;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   X = (1 - lr wd) X - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Every element is read and written once, in pieces of four per lane (16
// bytes of float32).  With states in 8 bits, 16 lanes hold a block of 64
// elements, whose largest magnitude they find among themselves.
//
// Bound by memory (a 4 GiB copy: 4.72 TB/s).  50257 x 768 with bfloat16 gradients:
// 164 us, 6.1 TB/s; two of 32000 x 4096 with 8-bit states 660 us, 5.6 TB/s.
#include <cstddef>
#include <type_traits>

#include "adamw_types.h"
#include "device_common.h"

namespace dion {

namespace {

// The magnitude of a block in the leading lanes' bits: the largest of 16
// lanes (one DPP row), in every one of them.  Magnitudes order like their
// bits, infinity and NaN on top.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  const auto step = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
  v = step(v, __builtin_amdgcn_update_dpp(0, v, 0xb1, 0xf, 0xf, true));    // quad_perm: lane ^ 1
  v = step(v, __builtin_amdgcn_update_dpp(0, v, 0x4e, 0xf, 0xf, true));    // quad_perm: lane ^ 2
  v = step(v, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, true));   // row_half_mirror
  v = step(v, __builtin_amdgcn_update_dpp(0, v, 0x140, 0xf, 0xf, true));   // row_mirror
  return v;
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// A block's scale 2^(byte - 127) as a float (255: NaN).
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte == 255 ? 0x7fc00000u : byte == 0 ? 0x00400000u : byte << 23);
}

// The byte of a block's scale from its largest magnitude's bits: that one
// comes to lie in [128, 256), an eighth of e4m3's range below its end, so
// that rounding up stays inside.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const int e = static_cast<int>(top >> 23);
  return e == 255 ? 255u : static_cast<uint32_t>(max(e - 7, 1));
}

// a >= 0, scaled, to e4m3 with the dither u in [0, 1): floor(a / ulp + u) ulp,
// a value that e4m3 holds exactly.  The mean over u is a, which is what lets
// a state move by less than an ulp per step: nearest rounding would lose
// every change of v below 6% (a step changes v by 1 - beta2 of the
// difference).  LEAST: ulps that a nonzero value keeps at least.
template <int LEAST>
__device__ __forceinline__ float dithered(float a, float u) {
  const uint32_t e = max(__float_as_uint(a) >> 23, 121u);   // subnormal below 2^-6
  float q = floorf(a * __uint_as_float((257u - e) << 23) + u);
  if constexpr (LEAST > 0) q = a > 0.0f ? fmaxf(q, static_cast<float>(LEAST)) : 0.0f;
  return q * __uint_as_float((e - 3u) << 23);
}

// Four values' codes: magnitudes q, signs of x.
__device__ __forceinline__ uint32_t codes(const float (&q)[4], const float (&x)[4]) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(copysignf(q[0], x[0]), copysignf(q[1], x[1]), w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(copysignf(q[2], x[2]), copysignf(q[3], x[3]), w, true);
  return static_cast<uint32_t>(w);
}
__device__ __forceinline__ void values(uint32_t w, float (&x)[4]) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
  x[0] = lo[0];
  x[1] = lo[1];
  x[2] = hi[0];
  x[3] = hi[1];
}

// The 32 bits of element i's dither: the index, shifted by the seed, times a
// multiplier near 2^32 over the golden ratio, its upper bits folded into the lower
// ones before and after a second multiplication.  Both multipliers and both
// shifts are those of the published xxHash32 algorithm (its first two primes and
// the first two steps of its final mix), whose distribution is known to be good.
__device__ __forceinline__ uint32_t dither(uint32_t i, uint32_t seed) {
  uint32_t h = (i + seed) * 0x9e3779b1u;
  h = (h ^ (h >> 15)) * 0x85ebca77u;
  return h ^ (h >> 13);
}

// The root of float32 states' v, within an ulp.  The instruction takes numbers
// below the normal ones for zero, and a step would then be m / eps, so small v
// are scaled for it (eps may be far below their roots).
__device__ __forceinline__ float root_of(float v) {
  const bool low = v < 0x1p-96f;
  const float r = __builtin_amdgcn_sqrtf(low ? v * 0x1p32f : v);
  return low ? r * 0x1p-16f : r;
}

// Four consecutive elements from i; `left` of them exist.  VEC: as one access
// where all four exist.  NT: past the caches, which a large step's tensors would
// only sweep.
template <class V, bool VEC, bool NT, class T>
__device__ __forceinline__ void load4(const T* p, int64_t i, int64_t left, T (&v)[4]) {
  static_assert(sizeof(V) == 4 * sizeof(T), "one access of four");
  if (VEC && left >= 4) {
    const gptr<const V> at = (gptr<const V>)(p + i);
    const V u = NT ? __builtin_nontemporal_load(at) : *at;
    __builtin_memcpy(v, &u, sizeof(V));
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = k < left ? p[i + k] : T(0);
  }
}
template <class V, bool VEC, bool NT, class T>
__device__ __forceinline__ void store4(T* p, int64_t i, int64_t left, const T (&v)[4]) {
  if (VEC && left >= 4) {
    V u;
    __builtin_memcpy(&u, v, sizeof(V));
    if constexpr (NT) __builtin_nontemporal_store(u, (gptr<V>)(p + i));
    else *(gptr<V>)(p + i) = u;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < left) p[i + k] = v[k];
  }
}

template <bool BF>
struct GradBits {
  using T = typename std::conditional<BF, uint16_t, float>::type;
  using V = typename std::conditional<BF, u32x2, f32x4>::type;
};

// One workgroup's chunk.  The moments take one rounding per operation, as the
// formulas read (no fused multiply-adds): a code then depends on nothing but
// the formulas.
template <bool BF, int BITS, int QUADS, bool VEC, bool NT>
__device__ __forceinline__ void adamw_chunk_of(const AdamwTensor& t, int64_t base, float b1, float c1, float b2,
                                               float c2, float rate, float root, float eps, uint32_t seed, float scale) {
#pragma clang fp contract(off)
  using GT = typename GradBits<BF>::T;
  using GV = typename GradBits<BF>::V;
  using ST = typename std::conditional<BITS == 8, uint8_t, float>::type;
  using SV = typename std::conditional<BITS == 8, uint32_t, f32x4>::type;
  float x[QUADS][4];
  GT gr[QUADS][4];
  ST ms[QUADS][4], vs[QUADS][4];
  uint32_t sm[QUADS], sv[QUADS];
  const int64_t blocks = (t.count() + kAdamwBlock - 1) / kAdamwBlock;
  const int64_t i0 = base + 4 * static_cast<int64_t>(threadIdx.x);
#pragma unroll
  for (int q = 0; q < QUADS; ++q) {
    const int64_t i = i0 + 1024 * q, left = t.count() - i;
    load4<f32x4, VEC, NT>(t.X, i, left, x[q]);
    load4<GV, VEC, NT>(static_cast<const GT*>(t.G), i, left, gr[q]);
    load4<SV, VEC, NT>(static_cast<const ST*>(t.M), i, left, ms[q]);
    load4<SV, VEC, NT>(static_cast<const ST*>(t.V), i, left, vs[q]);
    if constexpr (BITS == 8) {
      sm[q] = left > 0 ? t.S[i / kAdamwBlock] : 0;
      sv[q] = left > 0 ? t.S[blocks + i / kAdamwBlock] : 0;
    }
  }
#pragma unroll
  for (int q = 0; q < QUADS; ++q) {
    const int64_t i = i0 + 1024 * q, left = t.count() - i;
    float m[4], v[4], r[4];
    if constexpr (BITS == 8) {
      uint32_t cm, cr;
      __builtin_memcpy(&cm, ms[q], 4);
      __builtin_memcpy(&cr, vs[q], 4);
      values(cm, m);
      values(cr, r);
      const float a = scale_of(sm[q]), b = scale_of(sv[q]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        m[k] = m[k] * a;
        r[k] = r[k] * b;
        v[k] = r[k] * r[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        m[k] = ms[q][k];
        v[k] = vs[q][k];
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float g;
      if constexpr (BF) g = bf16_to_f32(gr[q][k]);
      else g = gr[q][k];
      g = g * scale;
      m[k] = m[k] * b1 + g * c1;
      v[k] = v[k] * b2 + g * g * c2;
      r[k] = BITS == 8 ? sqrtf(v[k]) : root_of(v[k]);
      // a relative error of 2^-22 in the step is far below X's own rounding; the
      // reciprocal's argument is at least eps, which is a normal number
      x[q][k] = x[q][k] * t.decay - m[k] * rate * __builtin_amdgcn_rcpf(r[k] * root + eps);
    }
    if (left > 0) store4<f32x4, VEC, NT>(t.X, i, left, x[q]);
    if constexpr (BITS == 8) {
      uint32_t tm = 0, tr = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k >= left) m[k] = r[k] = 0.0f;
        tm = max(tm, magnitude(m[k]));
        tr = max(tr, magnitude(r[k]));
      }
      const uint32_t bm = scale_byte(row_max(tm)), br = scale_byte(row_max(tr));
      // 255, NaN: the block's values do not matter
      const float a = __uint_as_float((254u - min(bm, 253u)) << 23), b = __uint_as_float((254u - min(br, 253u)) << 23);
      float qm[4], qr[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t h = dither(static_cast<uint32_t>(i) + k, seed);
        qm[k] = dithered<0>(fabsf(m[k]) * a, static_cast<float>(h & 0xffffu) * 0x1p-16f);
        qr[k] = dithered<1>(r[k] * b, static_cast<float>(h >> 16) * 0x1p-16f);
      }
      if (left > 0) {
        const uint32_t cm = codes(qm, m), cr = codes(qr, r);
        __builtin_memcpy(ms[q], &cm, 4);
        __builtin_memcpy(vs[q], &cr, 4);
        store4<SV, VEC, NT>(static_cast<ST*>(t.M), i, left, ms[q]);
        store4<SV, VEC, NT>(static_cast<ST*>(t.V), i, left, vs[q]);
        if ((threadIdx.x & 15) == 0) {
          t.S[i / kAdamwBlock] = static_cast<uint8_t>(bm);
          t.S[blocks + i / kAdamwBlock] = static_cast<uint8_t>(br);
        }
      }
    } else if (left > 0) {
      store4<SV, VEC, NT>(static_cast<ST*>(t.M), i, left, m);
      store4<SV, VEC, NT>(static_cast<ST*>(t.V), i, left, v);
    }
  }
}

// The launch's arguments are read where they stand: a tensor's index is known
// at run time only, and the arguments as a value indexed with it would be
// copied to private memory first.
template <bool BF, int BITS, int QUADS, bool NT, int CAP>
__global__ __launch_bounds__(256) void k_adamw(AdamwLaunch<CAP> arg) {
  typedef __attribute__((address_space(4))) const AdamwLaunch<CAP>* kptr;
  const kptr L = (kptr)__builtin_amdgcn_kernarg_segment_ptr();
  (void)arg;
  const int item = blockIdx.x, count = L->count;
  int which = 0;
  if constexpr (CAP > 4) {   // a lane looks at one tensor's first workgroup, or two
    static_assert(CAP <= 128, "two tensors per lane");
    const int lane = threadIdx.x & 63;
    which = __popcll(__ballot(lane < count && L->first[min(lane, CAP - 1)] <= item)) +
            __popcll(__ballot(lane + 64 < count && L->first[min(lane + 64, CAP - 1)] <= item)) - 1;
  } else {
#pragma unroll
    for (int i = 1; i < CAP; ++i) which += i < count && L->first[i] <= item;
  }
  which = __builtin_amdgcn_readfirstlane(which);
  struct { uint32_t w[kAdamwWords]; } u;
#pragma unroll
  for (int k = 0; k < kAdamwWords; ++k) u.w[k] = L->t[which][k];
  AdamwTensor t;
  __builtin_memcpy(&t, &u, sizeof(u));
  const int64_t base = static_cast<int64_t>(item - L->first[which]) * (1024 * QUADS);
  float scale = 1.0f;
  if (L->grad_scale) {
    scale = *L->grad_scale;
    // not finite: the whole step leaves everything as it was
    if ((__float_as_uint(scale) & 0x7f800000u) == 0x7f800000u) return;
  }
  if (t.vec())
    adamw_chunk_of<BF, BITS, QUADS, true, NT>(t, base, L->b1, L->c1, L->b2, L->c2, L->rate, L->root, L->eps, L->seed, scale);
  else
    adamw_chunk_of<BF, BITS, QUADS, false, NT>(t, base, L->b1, L->c1, L->b2, L->c2, L->rate, L->root, L->eps, L->seed, scale);
}

template <bool BF, int BITS, int CAP>
hipError_t go(const AdamwLaunch<CAP>& L, bool large, hipStream_t st) {
  if (large) k_adamw<BF, BITS, adamw_quads(BITS, true), true, CAP><<<dim3(L.total), dim3(256), 0, st>>>(L);
  else k_adamw<BF, BITS, adamw_quads(BITS, false), false, CAP><<<dim3(L.total), dim3(256), 0, st>>>(L);
  return hipGetLastError();
}
template <int CAP>
hipError_t go(const AdamwLaunch<CAP>& L, int gdtype, int state_bits, bool large, hipStream_t st) {
  if (gdtype) return state_bits == 8 ? go<true, 8>(L, large, st) : go<true, 32>(L, large, st);
  return state_bits == 8 ? go<false, 8>(L, large, st) : go<false, 32>(L, large, st);
}

}  // namespace

hipError_t launch_adamw(const AdamwLaunch<kAdamwTensors>& L, int gdtype, int state_bits, bool large, hipStream_t st) {
  if (L.count > kAdamwFew) return go(L, gdtype, state_bits, large, st);
  AdamwLaunch<kAdamwFew> few;
  __builtin_memcpy(&few, &L, offsetof(AdamwLaunch<kAdamwFew>, first));
  for (int i = 0; i < kAdamwFew; ++i) {
    few.first[i] = L.first[i];
    __builtin_memcpy(few.t[i], L.t[i], sizeof(few.t[i]));
  }
  return go(few, gdtype, state_bits, large, st);
}

}  // namespace dion
