// Device helpers shared by the Newton-Schulz kernels.
#pragma once
#include "device_common.h"
#include "ns_types.h"

namespace dion {

// The matrix and the local work item of item t.
__device__ __forceinline__ void ns_locate(const NsLaunch& L, int t, NsDesc& d, NsClass& c, int& local) {
  c = L.cls[0];
#pragma unroll
  for (int i = 1; i < kNsMaxClasses; ++i)
    if (i < L.nclass && t >= L.cls[i].base) c = L.cls[i];
  const int rel = t - c.base;
  const int mi = rel / c.tiles;
  local = rel - mi * c.tiles;
  d = L.table ? L.table[c.first + mi] : L.inl;
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

}  // namespace dion
