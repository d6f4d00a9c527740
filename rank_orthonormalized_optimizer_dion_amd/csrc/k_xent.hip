// Softmax cross entropy of an output head without its logits: the kernels
// behind dion_cross_entropy_forward and dion_cross_entropy_backward.
//
//   z = x W^T;  lse = log sum_j exp z_j
//   loss = lse - (1 - e) z_y - e mean_j z_j + zc lse^2
//   dz_j = dloss ((1 + 2 zc lse) exp(z_j - lse) - (1 - e) [j = y] - e / n)
//   dx = dz W;  dW = dz^T x
//
// z comes out of the linear layer's products (mm16.h, lin_device.h) and stays
// in the accumulators.  Forward: every wavefront reduces its columns of a row
// to their largest and their sum of exponentials, k_xent_join puts the pieces
// of the vocabulary together.  Backward: z once more, turned into dz in the
// accumulators and written in bfloat16, a piece of the vocabulary at a time,
// for the two products that follow (k_lin_mm).
#include <utility>

#include "dion.h"
#include "lin_device.h"
#include "work16.h"
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

// Eight values of dz as bfloat16 planes.
__device__ __forceinline__ void store_dz(const XentEpi& e, int64_t row, int col, const float (&v)[8]) {
  uint16_t* at = e.dz + row * e.pitch + col;
  float rest[8];
  uint16_t h[8];
  for (int pl = 0; pl < e.planes; ++pl) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = pinned(pl == 0 ? v[k] : rest[k]);
      h[k] = pl == 0 && e.planes > 1 ? first_plane(x) : to_bf16(x);
      rest[k] = x - bf16_to_f32(h[k]);
    }
    *reinterpret_cast<u32x4*>(at + pl * e.plane) = pack8(h);
  }
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

template <int TILE, bool GRAD>
__global__ __launch_bounds__(2 * TILE, 2) void k_xent_mm(LinProduct p, XentEpi e) {
  using S = LinShape<TILE, kLinForward>;
  static_assert(S::TM == 64 && S::F == 16, "rows of a wavefront");
  __shared__ u32x4 smem[S::LDS_CELLS];
  const Work16 work{p.full, p.tx * p.ty - p.full, p.slices, p.part, p.count};
  const Item16 it = item16(work, xcd_item(blockIdx.x, gridDim.x));
  int ti, tj;
  tile_order(it.tile, p.tx, p.ty, ti, tj);
  const int r0 = ti * TILE, c0 = tj * TILE;
  int kbeg, kend;
  slice16<S>(it, p.K, kbeg, kend);
  typename S::Acc acc[S::FM][S::FN];
  typename S::A ta;
  typename S::B tb;
  ta.init(p.lda, r0, p.M);
  tb.init(p.ldb, c0, p.N);
  lin_product_tile<S>(p, ta, tb, kbeg, kend, smem, acc);
  if (!join16<S>(work, it, smem, acc)) return;
  const int wave = wave16();
  const int row0 = r0 + (wave / S::WN) * S::TM, col0 = c0 + (wave % S::WN) * S::TN;
  if constexpr (GRAD) {
    dz_tile<S>(acc, e, p.M, p.N, row0, col0);
    tile_runs<S, false>(
        acc, smem, [](int, int) { return NoPre{}; },
        [&](int r, int q, const float (&v)[8], const NoPre&) {
          const int row = r0 + r, col = c0 + q;
          if (row < e.prows && col < e.pitch) store_dz(e, row, col, v);
        });
  } else {
    stats_tile<S>(acc, e, p.M, p.N, row0, col0, e.col0 + 2 * tj + wave % S::WN);
  }
}

// lse and loss from the partial columns: TOK tokens by 256 / TOK lanes of
// columns per workgroup.  The loss is formed from differences to the largest
// logit, not from lse, so that a confident prediction's small loss keeps its
// digits.
template <int TOK>
__global__ __launch_bounds__(256) void k_xent_join(XentJoin j) {
  constexpr int LANES = 256 / TOK;
  __shared__ float red[3][LANES][TOK];
  const int tok = threadIdx.x % TOK, lane = threadIdx.x / TOK;
  const int row = blockIdx.x * TOK + tok;
  float top = -INFINITY, sum = 0.0f, total = 0.0f;
  if (row < j.t) {
#pragma unroll 4
    for (int c = lane; c < j.cols; c += LANES) {
      const int64_t at = static_cast<int64_t>(c) * j.t + row;
      merge(top, sum, j.top[at], j.sum[at]);
      if (j.total) total += j.total[at];
    }
  }
  red[0][lane][tok] = top;
  red[1][lane][tok] = sum;
  red[2][lane][tok] = total;
  __syncthreads();
#pragma unroll
  for (int h = LANES / 2; h > 0; h /= 2) {
    if (lane < h) {
      merge(top, sum, red[0][lane + h][tok], red[1][lane + h][tok]);
      total += red[2][lane + h][tok];
      red[0][lane][tok] = top;
      red[1][lane][tok] = sum;
      red[2][lane][tok] = total;
    }
    __syncthreads();
  }
  if (lane != 0 || row >= j.t) return;
  const float rest = logf(sum), lse = top + rest;
  if (j.lse) j.lse[row] = lse;
  if (!j.loss) return;
  const int64_t y = j.target[row];
  float loss = 0.0f;
  if (y != j.ignore) {
    loss = NAN;   // a target outside the vocabulary
    if (y >= 0 && y < j.vocab) {
      loss = rest + j.keep * (top - j.hit[row]) + j.z_loss * lse * lse;
      if (j.total) loss += j.smoothing * (top - total / static_cast<float>(j.vocab));
    }
  }
  j.loss[row] = loss;
}

template <int TILE>
hipError_t product(const LinProduct& p, const XentEpi& e, bool grad, hipStream_t st) {
  if (grad) k_xent_mm<TILE, true><<<dim3(p.items), dim3(2 * TILE), 0, st>>>(p, e);
  else k_xent_mm<TILE, false><<<dim3(p.items), dim3(2 * TILE), 0, st>>>(p, e);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_xent_product(const LinProduct& p, const XentEpi& e, bool grad, int tile, hipStream_t st) {
  if (tile == 256) return product<256>(p, e, grad, st);
  return product<128>(p, e, grad, st);
}

hipError_t launch_xent_join(const XentJoin& j, hipStream_t st) {
  // few tokens: a workgroup each
  if (j.t <= 256) k_xent_join<1><<<dim3(j.t), dim3(256), 0, st>>>(j);
  else k_xent_join<16><<<dim3((j.t + 15) / 16), dim3(256), 0, st>>>(j);
  return hipGetLastError();
}

}  // namespace dion
