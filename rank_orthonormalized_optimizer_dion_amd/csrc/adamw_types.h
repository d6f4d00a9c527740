// Types and launcher of the AdamW step (k_adamw.hip, adamw_api.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dion {

// Elements that share the two scales of an 8-bit state.
constexpr int kAdamwBlock = 64;

struct AdamwTensor {
  float* X;
  const void* G;
  void* M;
  void* V;
  uint8_t* S;       // 8-bit states: scales of M's blocks, then of V's
  int64_t n;
  float decay;      // 1 - lr * weight decay
  int32_t vec;      // every pointer admits the accesses of four elements
};

// One launch's tensors travel in its arguments: no table has to be uploaded
// or kept.  As many as a wavefront has lanes, each of which looks at one
// tensor's first work item.
constexpr int kAdamwTensors = 64;
struct AdamwLaunch {
  int32_t first[kAdamwTensors];   // first workgroup of each tensor
  AdamwTensor t[kAdamwTensors];
  const float* grad_scale;        // or null
  int32_t count, total;           // tensors, workgroups
  float b1, c1, b2, c2;           // beta1, 1 - beta1, beta2, 1 - beta2
  float rate, root, eps;          // lr / (1 - beta1^t), (1 - beta2^t)^-1/2
  uint32_t seed;                  // of the 8-bit states' rounding, mixed
};
static_assert(sizeof(AdamwLaunch) <= 4096, "kernel arguments");

// Elements of a workgroup of 256 threads: `quads` times four per thread.
inline int64_t adamw_chunk(int quads) { return 1024 * static_cast<int64_t>(quads); }
// quads: 1 or 4
hipError_t launch_adamw(const AdamwLaunch& L, int gdtype, int state_bits, int quads, hipStream_t st);

}  // namespace dion
