// What the cross entropy makes of a tile of logits (k_xent.hip, k_xent_f32.hip).
#pragma once
#include <utility>

#include "xent_device.h"

namespace dion {

namespace {

// f(integral_constant 0), f(1), ...: DPP controls have to be constants.
template <class F, int... I>
__device__ __forceinline__ void each(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F f) {
  each(f, std::make_integer_sequence<int, N>{});
}

// The accumulators of a wavefront hold 64 rows; lane l keeps the data of row
// 16 (l % 16 / 4) + 4 (l / 16) + l % 4, which accumulator row (m, v) of its 16
// lanes asks lane 4 m + v of them for (row_newbcast).
__device__ __forceinline__ int own_row(int lane) { return 16 * ((lane & 15) >> 2) + 4 * (lane >> 4) + (lane & 3); }
constexpr int kBcast = 0x150;   // DPP row_newbcast: of lane 0

template <class S>
__device__ __forceinline__ void stats_tile(typename S::Acc (&acc)[S::FM][S::FN], const XentEpi& e, int t, int n,
                                           int row0, int col0, int part) {
  const int lane = threadIdx.x & 63, l15 = lane & 15;
  const int own = row0 + own_row(lane);
  // the target's column, counted from this wavefront's first
  int local = -1;
  if (own < t) {
    const int64_t y = e.target[own] - e.j0 - col0;
    if (y >= 0 && y < S::TN && col0 + y < n) local = static_cast<int>(y);
  }
  const bool any = __ballot(local >= 0) != 0;
  if (any)
    each<4 * S::FM>([&](auto i) {
      constexpr int m = i / 4, v = i % 4;
      const int want = dpp<kBcast + i>(local);
#pragma unroll
      for (int q = 0; q < S::FN; ++q)
        if (want == S::F * q + l15) e.hit[row0 + S::F * m + 4 * (lane >> 4) + v] = acc[m][q][v];
    });
  const bool edge = col0 + S::TN > n;
  float top = 0.0f, sum = 0.0f, total = 0.0f;
  each<4 * S::FM>([&](auto i) {
    constexpr int m = i / 4, v = i % 4;
    float z[S::FN];
#pragma unroll
    for (int q = 0; q < S::FN; ++q) z[q] = acc[m][q][v];
    if (e.total) {
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < S::FN; ++q) s += !edge || col0 + S::F * q + l15 < n ? z[q] : 0.0f;
      s = row_sum(s);
      total = l15 == i ? s : total;
    }
    if (edge) {
#pragma unroll
      for (int q = 0; q < S::FN; ++q) z[q] = col0 + S::F * q + l15 < n ? z[q] : -INFINITY;
    }
    float hi = z[0];
#pragma unroll
    for (int q = 1; q < S::FN; ++q) hi = fmaxf(hi, z[q]);
    hi = row_max(hi);
    const float b = base_of(hi);
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < S::FN; ++q) s += exp_fast(z[q] - b);
    s = row_sum(s);
    top = l15 == i ? hi : top;
    sum = l15 == i ? s : sum;
  });
  if (own < t) {
    const int64_t at = static_cast<int64_t>(part) * t + own;
    e.top[at] = top;
    e.sum[at] = sum;
    if (e.total) e.total[at] = total;
  }
}

template <class S>
__device__ __forceinline__ void dz_tile(typename S::Acc (&acc)[S::FM][S::FN], const XentEpi& e, int t, int n,
                                        int row0, int col0) {
  const int lane = threadIdx.x & 63, l15 = lane & 15;
  int64_t y;
  const XentRow r = xent_row(e, row0 + own_row(lane), t, y);
  y -= e.j0 + col0;
  const int local = y >= 0 && y < S::TN ? static_cast<int>(y) : -1;
  const bool any = __ballot(local >= 0) != 0, edge = col0 + S::TN > n;
  each<4 * S::FM>([&](auto i) {
    constexpr int m = i / 4, v = i % 4;
    const float lse = dpp<kBcast + i>(r.lse), a = dpp<kBcast + i>(r.a), b = dpp<kBcast + i>(r.b);
    const int mask = dpp<kBcast + i>(r.mask);
#pragma unroll
    for (int q = 0; q < S::FN; ++q) acc[m][q][v] = dz_of(acc[m][q][v], lse, a, b, mask);
    if (any) {
      const int want = dpp<kBcast + i>(local);
      const float c = dpp<kBcast + i>(r.c);
#pragma unroll
      for (int q = 0; q < S::FN; ++q) acc[m][q][v] -= want == S::F * q + l15 ? c : 0.0f;
    }
    if (edge) {
#pragma unroll
      for (int q = 0; q < S::FN; ++q) acc[m][q][v] = col0 + S::F * q + l15 < n ? acc[m][q][v] : 0.0f;
    }
  });
}

}  // namespace

}  // namespace dion
