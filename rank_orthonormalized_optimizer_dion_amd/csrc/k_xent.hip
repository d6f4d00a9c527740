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

// f(integral_constant 0), f(1), ...: DPP controls have to be constants.
template <class F, int... I>
__device__ __forceinline__ void each(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F f) {
  each(f, std::make_integer_sequence<int, N>{});
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

// Eight values of dz (COUNT of them) as bfloat16 planes.
template <int COUNT>
__device__ __forceinline__ void store_dz(const XentEpi& e, int64_t row, int col, const float (&v)[COUNT]) {
  uint16_t* at = e.dz + row * e.ld + col;
  float rest[COUNT];
  uint16_t h[COUNT];
  for (int pl = 0; pl < e.planes; ++pl) {
#pragma unroll
    for (int k = 0; k < COUNT; ++k) {
      const float x = pinned(pl == 0 ? v[k] : rest[k]);
      h[k] = pl == 0 && e.planes > 1 ? first_plane(x) : to_bf16(x);
      rest[k] = x - bf16_to_f32(h[k]);
    }
    if constexpr (COUNT == 8) *reinterpret_cast<u32x4*>(at + pl * e.plane) = pack8(h);
    else at[pl * e.plane] = h[0];
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
          if (row < e.prows && col < e.pitch) store_dz<8>(e, row, col, v);
        });
  } else {
    stats_tile<S>(acc, e, p.M, p.N, row0, col0, e.col0 + 2 * tj + wave % S::WN);
  }
}

// Few tokens, bfloat16: 16 columns per workgroup, 16 lanes per token.  What
// the rows need is loaded before the products, not after them.
template <int TB, bool GRAD>
__global__ __launch_bounds__(512) void k_xent_skinny(LinSkinny p, XentEpi e) {
  __shared__ float red[8][TB][16][17];
  constexpr int B = (TB + 1) / 2;   // 512 threads hold 32 tokens
  const int n0 = blockIdx.x * kXentGroup;
  const int c = threadIdx.x & 15, col = n0 + c;
  XentRow r[B];
  int64_t y[B];
#pragma unroll
  for (int b = 0; b < B; ++b) {
    const int token = 32 * b + (threadIdx.x >> 4);
    if constexpr (GRAD) r[b] = xent_row(e, token, p.t, y[b]);
    else y[b] = token < p.t ? e.target[token] : -1;
  }
  skinny_sums<TB>(p, n0, red);
  __syncthreads();
#pragma unroll
  for (int b = 0; b < B; ++b) {
    const int token = 32 * b + (threadIdx.x >> 4);
    if (token >= 16 * TB) continue;
    float z = 0.0f;
#pragma unroll
    for (int s = 0; s < 8; ++s) z += red[s][token >> 4][token & 15][c];
    if constexpr (GRAD) {
      float v[1] = {dz_of(z, r[b].lse, r[b].a, r[b].b, r[b].mask)};
      if (y[b] == e.j0 + col) v[0] -= r[b].c;
      if (col >= p.n) v[0] = 0.0f;
      if (token < p.t && col < e.pitch) store_dz<1>(e, token, col, v);
    } else {
      const bool in = col < p.n;
      const float hi = row_max(in ? z : -INFINITY), base = base_of(hi);
      const float s = row_sum(in ? exp_fast(z - base) : 0.0f), total = e.total ? row_sum(in ? z : 0.0f) : 0.0f;
      if (token < p.t) {
        if (in && y[b] == e.j0 + col) e.hit[token] = z;
        if (c == 0) {
          const int64_t at = static_cast<int64_t>(e.col0 + blockIdx.x) * p.t + token;
          e.top[at] = hi;
          e.sum[at] = s;
          if (e.total) e.total[at] = total;
        }
      }
    }
  }
}

// Few tokens in float32 or of any alignment: 4 columns per wavefront.
template <int T, bool BF, bool VEC, bool GRAD>
__global__ __launch_bounds__(256) void k_xent_rows(LinSkinny p, XentEpi e) {
  __shared__ float part[3][4][T];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = blockIdx.x * kXentGroup + 4 * wave;
  float z[4][T];
#pragma unroll
  for (int c = 0; c < 4; ++c) row_sums<T, BF, VEC>(p, min(n0 + c, p.n - 1), z[c]);
  if constexpr (GRAD) {
#pragma unroll
    for (int i = 0; i < T; ++i)
      if (lane == i && i < p.t) {
        int64_t y;
        const XentRow r = xent_row(e, i, p.t, y);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int col = n0 + c;
          float v[1] = {dz_of(z[c][i], r.lse, r.a, r.b, r.mask)};
          if (y == e.j0 + col) v[0] -= r.c;
          if (col >= p.n) v[0] = 0.0f;
          if (col < e.pitch) store_dz<1>(e, i, col, v);
        }
      }
  } else {
#pragma unroll
    for (int i = 0; i < T; ++i) {
      float hi = -INFINITY, s = 0.0f, total = 0.0f;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (n0 + c < p.n) hi = fmaxf(hi, z[c][i]);
      const float base = base_of(hi);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (n0 + c < p.n) {
          s += exp_fast(z[c][i] - base);
          total += z[c][i];
        }
      if (lane == i && i < p.t) {
        part[0][wave][i] = hi;
        part[1][wave][i] = s;
        part[2][wave][i] = total;
        const int64_t y = e.target[i] - e.j0 - n0;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (y == c && n0 + c < p.n) e.hit[i] = z[c][i];
      }
    }
    __syncthreads();
    const int i = threadIdx.x;
    if (i < T && i < p.t) {
      float hi = part[0][0][i], s = part[1][0][i], total = part[2][0][i];
#pragma unroll
      for (int w = 1; w < 4; ++w) {
        merge(hi, s, part[0][w][i], part[1][w][i]);
        total += part[2][w][i];
      }
      const int64_t at = static_cast<int64_t>(e.col0 + blockIdx.x) * p.t + i;
      e.top[at] = hi;
      e.sum[at] = s;
      if (e.total) e.total[at] = total;
    }
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

template <int T, bool BF, bool GRAD>
hipError_t rows(const LinSkinny& s, const XentEpi& e, bool vec, int groups, hipStream_t st) {
  if (vec) k_xent_rows<T, BF, true, GRAD><<<dim3(groups), dim3(256), 0, st>>>(s, e);
  else k_xent_rows<T, BF, false, GRAD><<<dim3(groups), dim3(256), 0, st>>>(s, e);
  return hipGetLastError();
}
template <int T>
hipError_t rows(const LinSkinny& s, const XentEpi& e, bool grad, bool vec, int groups, hipStream_t st) {
  if (s.out.dtype) return grad ? rows<T, true, true>(s, e, vec, groups, st) : rows<T, true, false>(s, e, vec, groups, st);
  return grad ? rows<T, false, true>(s, e, vec, groups, st) : rows<T, false, false>(s, e, vec, groups, st);
}

// Workgroups of 16 columns: those of the piece, or of dz's padded rows.
int groups_of(const LinSkinny& s, const XentEpi& e, bool grad) {
  return grad ? static_cast<int>(e.pitch / kXentGroup) : (s.n + kXentGroup - 1) / kXentGroup;
}

template <int TB>
hipError_t skinny(const LinSkinny& s, const XentEpi& e, bool grad, hipStream_t st) {
  const dim3 grid(groups_of(s, e, grad)), block(512);
  if (grad) k_xent_skinny<TB, true><<<grid, block, 0, st>>>(s, e);
  else k_xent_skinny<TB, false><<<grid, block, 0, st>>>(s, e);
  return hipGetLastError();
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

hipError_t launch_xent_skinny(const LinSkinny& s, const XentEpi& e, bool grad, hipStream_t st) {
  if (s.t <= 16) return skinny<1>(s, e, grad, st);
  return s.t <= 32 ? skinny<2>(s, e, grad, st) : skinny<4>(s, e, grad, st);
}

hipError_t launch_xent_rows(const LinSkinny& s, const XentEpi& e, bool grad, bool vec, hipStream_t st) {
  const int groups = groups_of(s, e, grad);
  if (s.t == 1) return rows<1>(s, e, grad, vec, groups, st);
  return s.t <= 4 ? rows<4>(s, e, grad, vec, groups, st) : rows<8>(s, e, grad, vec, groups, st);
}

hipError_t launch_xent_join(const XentJoin& j, hipStream_t st) {
  // few tokens: a workgroup each
  if (j.t <= 256) k_xent_join<1><<<dim3(j.t), dim3(256), 0, st>>>(j);
  else k_xent_join<16><<<dim3((j.t + 15) / 16), dim3(256), 0, st>>>(j);
  return hipGetLastError();
}

}  // namespace dion
