// Host side of dion_adamw_step: argument validation and the launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "adamw_types.h"
#include "dion.h"

#define DION_API extern "C" __attribute__((visibility("default")))

static_assert(dion::kAdamwBlock == DION_ADAMW_BLOCK, "block of the 8-bit states");

namespace dion {
namespace {

constexpr int64_t kAdamwMaxElements = int64_t{1} << 33;
constexpr int32_t kAdamwMaxItems = (1 << 24) - 1;   // of a launch: fewer than 2^32 threads
static_assert(kAdamwMaxElements / 1024 <= kAdamwMaxItems, "a tensor fits a launch");

struct Bytes {
  uintptr_t p;
  uint64_t n;
};
bool bytes_overlap(const Bytes& a, const Bytes& b) { return a.p < b.p + b.n && b.p < a.p + a.n; }

bool adamw_ok(const dion_adamw_tensor& t, int gdtype, int state_bits, const float* grad_scale) {
  if (t.n < 0 || t.n > kAdamwMaxElements || !std::isfinite(t.weight_decay)) return false;
  if (t.n == 0) return true;
  const bool eight = state_bits == DION_STATE_8BIT;
  if (!t.X || !t.G || !t.M || !t.V || (eight && !t.S)) return false;
  const uint64_t n = static_cast<uint64_t>(t.n), ge = gdtype == DION_DTYPE_BF16 ? 2 : 4, se = eight ? 1 : 4;
  const Bytes all[] = {{reinterpret_cast<uintptr_t>(t.X), 4 * n},
                       {reinterpret_cast<uintptr_t>(t.M), se * n},
                       {reinterpret_cast<uintptr_t>(t.V), se * n},
                       {reinterpret_cast<uintptr_t>(eight ? t.S : nullptr), eight ? 2 * ((n + kAdamwBlock - 1) / kAdamwBlock) : 0},
                       {reinterpret_cast<uintptr_t>(t.G), ge * n}};
  if (all[0].p % 4 != 0 || all[1].p % se != 0 || all[2].p % se != 0 || all[4].p % ge != 0) return false;
  const Bytes scale = {reinterpret_cast<uintptr_t>(grad_scale), 4};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < i; ++j)
      if (all[i].n && all[j].n && bytes_overlap(all[i], all[j])) return false;
    if (i < 4 && grad_scale && all[i].n && bytes_overlap(all[i], scale)) return false;   // G may hold it
  }
  return true;
}

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

int adamw_run(const dion_adamw_tensor* list, int count, double lr, double beta1, double beta2, double eps,
              int64_t step, const float* grad_scale, int state_bits, uint32_t seed, int gdtype, void* stream) {
  if (!list || count < 1 || count > DION_MAX_LIST) return DION_ERR_INVALID_ARG;
  if (gdtype != DION_DTYPE_F32 && gdtype != DION_DTYPE_BF16) return DION_ERR_INVALID_ARG;
  if (state_bits != DION_STATE_F32 && state_bits != DION_STATE_8BIT) return DION_ERR_INVALID_ARG;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || step < 1) return DION_ERR_INVALID_ARG;
  if (!std::isfinite(lr) || !(eps >= 1.17549435e-38 && eps <= 1e30)) return DION_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(grad_scale) % 4 != 0) return DION_ERR_INVALID_ARG;
  AdamwLaunch<kAdamwTensors> L{};
  // 1 - beta and the bias corrections are formed before they are rounded
  L.b1 = static_cast<float>(beta1);
  L.c1 = static_cast<float>(1.0 - beta1);
  L.b2 = static_cast<float>(beta2);
  L.c2 = static_cast<float>(1.0 - beta2);
  L.rate = static_cast<float>(lr / (1.0 - std::pow(beta1, static_cast<double>(step))));
  L.root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, static_cast<double>(step))));
  L.eps = static_cast<float>(eps);
  L.seed = seed * 0x632be5abu;
  L.grad_scale = grad_scale;
  if (!std::isfinite(L.rate) || !std::isfinite(L.root)) return DION_ERR_INVALID_ARG;
  int64_t elements = 0;
  for (int i = 0; i < count; ++i) {
    if (!adamw_ok(list[i], gdtype, state_bits, grad_scale)) return DION_ERR_INVALID_ARG;
    if (!std::isfinite(static_cast<float>(1.0 - lr * list[i].weight_decay))) return DION_ERR_INVALID_ARG;
    elements += list[i].n;
  }
  const hipStream_t st = static_cast<hipStream_t>(stream);
  // bytes read and written per element
  const int64_t each = 8 + (gdtype == DION_DTYPE_BF16 ? 2 : 4) + (state_bits == DION_STATE_8BIT ? 4 : 16);
  const bool large = elements > kAdamwLarge / each;
  const int64_t chunk = 1024 * adamw_quads(state_bits, large);
  const auto flush = [&] {
    if (L.count == 0) return hipSuccess;
    const hipError_t e = launch_adamw(L, gdtype, state_bits, large, st);
    L.count = L.total = 0;
    return e;
  };
  for (int i = 0; i < count; ++i) {
    const dion_adamw_tensor& a = list[i];
    if (a.n == 0) continue;
    const int64_t items = (a.n + chunk - 1) / chunk;
    if (L.count == kAdamwTensors || items > kAdamwMaxItems - L.total)
      if (flush() != hipSuccess) return DION_ERR_HIP;
    const int se = state_bits == DION_STATE_8BIT ? 4 : 16;   // bytes of four elements' states
    const bool vec = aligned(a.X, 16) && aligned(a.G, gdtype == DION_DTYPE_BF16 ? 8 : 16) && aligned(a.M, se) && aligned(a.V, se);
    const AdamwTensor t = {a.X, a.G, a.M, a.V, a.S, 2 * a.n + vec, static_cast<float>(1.0 - lr * a.weight_decay)};
    std::memcpy(L.t[L.count], &t, sizeof(L.t[0]));
    L.first[L.count++] = L.total;
    L.total += static_cast<int32_t>(items);
  }
  return flush() == hipSuccess ? DION_OK : DION_ERR_HIP;
}

}  // namespace
}  // namespace dion

using namespace dion;

DION_API int dion_adamw_step_batched(const dion_adamw_tensor* tensors, int count, double lr, double beta1,
                                     double beta2, double eps, int64_t step, const float* grad_scale,
                                     int state_bits, uint32_t seed, int g_dtype, void* stream) {
  return adamw_run(tensors, count, lr, beta1, beta2, eps, step, grad_scale, state_bits, seed, g_dtype, stream);
}

DION_API int dion_adamw_step(float* X, const void* G, void* M, void* V, uint8_t* S, int64_t n, double lr,
                             double beta1, double beta2, double eps, double weight_decay, int64_t step,
                             const float* grad_scale, int state_bits, uint32_t seed, int g_dtype, void* stream) {
  const dion_adamw_tensor t = {X, G, M, V, S, n, weight_decay};
  return adamw_run(&t, 1, lr, beta1, beta2, eps, step, grad_scale, state_bits, seed, g_dtype, stream);
}
