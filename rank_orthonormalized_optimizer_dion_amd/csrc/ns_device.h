// Device helpers shared by the Newton-Schulz kernels.
#pragma once
#include "device_common.h"
#include "ns_types.h"

namespace dion {

__device__ __forceinline__ int uniform_index(int i) { return __builtin_amdgcn_readfirstlane(i); }

// The matrix and the local work item of item t.  Launch arguments and the
// table are read through the scalar cache, and every read here that misses
// it costs about a microsecond before the first tile can be asked for: the
// classes are all loaded at once and chosen among in registers (unused ones
// start past every item), and the descriptor is one block of scalar loads.
__device__ __forceinline__ void ns_locate(const NsLaunch& L, int t, NsDesc& d, NsClass& c, int& local) {
  c = L.cls[0];
#pragma unroll
  for (int i = 1; i < kNsMaxClasses; ++i) {
    const NsClass k = L.cls[i];
    const bool in = t >= k.base;
    c.first = in ? k.first : c.first;
    c.tiles = in ? k.tiles : c.tiles;
    c.base = in ? k.base : c.base;
    c.tx = in ? k.tx : c.tx;
    c.ty = in ? k.ty : c.ty;
  }
  const int rel = t - c.base;
  const int mi = rel / c.tiles;
  local = rel - mi * c.tiles;
  if (L.table) {
    typedef __attribute__((address_space(4))) const uint32_t* cptr;   // constant memory: scalar loads
    const cptr src = (cptr)(reinterpret_cast<const uint32_t*>(L.table + uniform_index(c.first + mi)));
    struct { uint32_t w[sizeof(NsDesc) / 4]; } u;
#pragma unroll
    for (size_t i = 0; i < sizeof(NsDesc) / 4; ++i) u.w[i] = src[i];
    d = __builtin_bit_cast(NsDesc, u);
  } else {
    d = L.inl;
  }
}

template <typename GT>
__device__ __forceinline__ float load_g(const void* G, int64_t o) {
  if constexpr (sizeof(GT) == 2) return bf16_to_f32(static_cast<const uint16_t*>(G)[o]);
  else return static_cast<const float*>(G)[o];
}

// The new momentum and the matrix to orthogonalize, each one rounding per
// operation, the same in both kernels that form them.
__device__ __forceinline__ float ns_moment(const NsLaunch& L, float g, float m) { return fmaf(L.mu, m, g); }
__device__ __forceinline__ float ns_dir(const NsLaunch& L, float g, float m1) {
  return L.nesterov ? fmaf(L.mu, m1, g) : m1;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
  return v;
}

// ||D||_F from k_ns_norm's partial sums, by all of a workgroup of W wavefronts.
template <int W>
__device__ __forceinline__ double ns_norm(const NsLaunch& L, const NsDesc& d, double (&part)[W]) {
  const double* parts = reinterpret_cast<const double*>(L.ws + d.oS);
  double sum = 0.0;
  for (int i = threadIdx.x; i < d.parts; i += 64 * W) sum += parts[i];
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  double v[W];
#pragma unroll
  for (int w = 0; w < W; ++w) v[w] = part[w];
#pragma unroll
  for (int h = 1; h < W; h *= 2)
#pragma unroll
    for (int w = 0; w < W; w += 2 * h) v[w] += v[w + h];
  return sqrt(v[0]);
}

}  // namespace dion
