// Types and launcher of the AdamW step (k_adamw.hip, adamw_api.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dion {

// Elements that share the two scales of an 8-bit state.
constexpr int kAdamwBlock = 64;

// 52 bytes: as 32-bit words, so that as many as possible fit a launch's
// arguments.
constexpr int kAdamwWords = 13;
struct AdamwTensor {
  float* X;
  const void* G;
  void* M;
  void* V;
  uint8_t* S;       // 8-bit states: scales of M's blocks, then of V's
  int64_t n;        // elements, doubled, plus 1 where every pointer admits the accesses of four elements
  float decay;      // 1 - lr * weight decay
  __host__ __device__ int64_t count() const { return n >> 1; }
  __host__ __device__ bool vec() const { return n & 1; }
};

// One launch's tensors travel in its arguments: no table has to be uploaded
// or kept.  72 fill the 4 KB that arguments may take (144 vectors of 768: 9.5 us, three launches of 64 15);
// 4 make a launch with few tensors cheaper for the host.
template <int CAP>
struct AdamwLaunch {
  const float* grad_scale;        // or null
  int32_t count, total;           // tensors, workgroups
  float b1, c1, b2, c2;           // beta1, 1 - beta1, beta2, 1 - beta2
  float rate, root, eps;          // lr / (1 - beta1^t), (1 - beta2^t)^-1/2
  uint32_t seed;                  // of the 8-bit states' rounding, mixed
  int32_t first[CAP];             // first workgroup of each tensor
  uint32_t t[CAP][kAdamwWords];   // AdamwTensor
};
constexpr int kAdamwTensors = 72, kAdamwFew = 4;
static_assert(sizeof(AdamwLaunch<kAdamwTensors>) <= 4096, "kernel arguments");

// Steps that move more than the memory-side cache holds go past the caches: 40
// million elements 176 us, through them 192; 10 million 43 and 40.
constexpr int64_t kAdamwLarge = int64_t{256} << 20;
// Pieces of four elements per thread, 256 threads per workgroup: two in large
// steps with 8-bit states (40 million elements 109 us, 114 with one), else one
// (float32: 176, with two 176, with four 180).
constexpr __host__ __device__ int adamw_quads(int state_bits, bool large) { return state_bits == 8 && large ? 2 : 1; }
hipError_t launch_adamw(const AdamwLaunch<kAdamwTensors>& L, int gdtype, int state_bits, bool large, hipStream_t st);

}  // namespace dion
