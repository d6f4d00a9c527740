// Softmax cross entropy of an output head without its logits: the kernels
// behind dion_cross_entropy_forward and dion_cross_entropy_backward.
//
//   z = x W^T;  lse = log sum_j exp z_j
//   loss = lse - (1 - e) z_y - e mean_j z_j + zc lse^2
//   dz_j = dloss ((1 + 2 zc lse) exp(z_j - lse) - (1 - e) [j = y] - e / n)
//   dx = dz W;  dW = dz^T x
//
// This file: bfloat16, more than a few tokens (k_xent_few.hip; float32:
// k_xent_f32.hip).  z comes out of the linear layer's tiles (mm16.h,
// lin_device.h) and stays in the accumulators.  Forward: every wavefront reduces
// its columns of a row to their largest and their sum of exponentials,
// k_xent_join puts them together.  Backward: z once more, turned into dz in the
// accumulators and written in bfloat16, a piece of the vocabulary at a time, for
// the two products that follow (k_lin_mm).
//
// Bound by the matrix cores where the reduction is long: 8192 tokens, 4096 ->
// 32000 forward 1.68 to 1.72 ms (1.27 PFLOP/s; the library's product alone 1.53 to
// 1.6 ms), of which the epilogues, which nothing hides, are 4%; gradients 4.9 to
// 5.1 ms for three such products.  Of 768, a tile's 24 stages are followed by an
// epilogue of half their time: gradients of 4096 tokens, 768 -> 50257, 1.03 ms, 0.40
// of it for dz, whose products would take 0.22.
#include <algorithm>

#include "dion.h"
#include "lin_device.h"
#include "work16.h"
#include "xent_tile.h"

namespace dion {

namespace {

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
          if (row < e.prows && col < e.pitch) {   // zero past the piece's columns and rows
            uint16_t h[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) h[k] = to_bf16(v[k]);
            *reinterpret_cast<u32x4*>(e.dz + row * e.pitch + col) = pack8(h);
          }
        });
  } else {
    stats_tile<S>(acc, e, p.M, p.N, row0, col0, e.col0 + 2 * tj + wave % S::WN);
  }
}

// lse and loss from the partial columns: a workgroup's TOK tokens by lanes of
// columns.  1021 tokens of 788 columns: 21 us with 256 threads per 16 tokens, 8
// with 1024.  The loss is formed from differences to the largest logit, not from
// lse, so that a confident prediction's small loss keeps its digits.
template <int TOK>
constexpr int kJoinThreads = TOK == 1 ? 256 : 1024;
template <int TOK>
__global__ __launch_bounds__(kJoinThreads<TOK>) void k_xent_join(XentJoin j) {
  constexpr int LANES = kJoinThreads<TOK> / TOK;
  static_assert(TOK == 1 || TOK == 16, "the last step has 16 lanes per token");
  __shared__ float red[3][16][TOK + 1];
  const int first = blockIdx.x * TOK;
  float top = -INFINITY, sum = 0.0f, total = 0.0f;
  if (first + static_cast<int>(threadIdx.x) % TOK < j.t) {
    const int row = first + threadIdx.x % TOK;
#pragma unroll 4
    for (int c = threadIdx.x / TOK; c < j.cols; c += LANES) {
      const int64_t at = static_cast<int64_t>(c) * j.t + row;
      merge(top, sum, j.top[at], j.sum[at]);
      if (j.total) total += j.total[at];
    }
  }
  // to 16 per token, then the 16 lanes of a DPP row
  const auto of_row = [&] {
    const float hi = row_max(top);
    sum = row_sum(sum * exp_fast(top - base_of(hi)));
    total = row_sum(total);
    top = hi;
  };
  if constexpr (TOK == 1) {
    of_row();
  } else {
#pragma unroll
    for (int h = 16; h < 64; h *= 2) {
      merge(top, sum, __shfl_xor(top, h), __shfl_xor(sum, h));
      total += __shfl_xor(total, h);
    }
  }
  const int part = TOK == 1 ? threadIdx.x / 16 : threadIdx.x / 64, tok = threadIdx.x % TOK;
  if (TOK == 1 ? threadIdx.x % 16 == 0 : threadIdx.x % 64 < 16) {
    red[0][part][tok] = top;
    red[1][part][tok] = sum;
    red[2][part][tok] = total;
  }
  __syncthreads();
  if (threadIdx.x >= 16 * TOK) return;
  top = red[0][threadIdx.x % 16][threadIdx.x / 16];
  sum = red[1][threadIdx.x % 16][threadIdx.x / 16];
  total = red[2][threadIdx.x % 16][threadIdx.x / 16];
  of_row();
  const int row = first + threadIdx.x / 16;
  if (threadIdx.x % 16 != 0 || row >= j.t) return;
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

// Copies of bfloat16 operands whose rows the tiles cannot read in place: 16
// bytes per thread and step, zero past the columns and (to the last whole
// stage) past the rows.  65 tokens, 1999 -> 32000, forward: 168 us with the
// linear layer's copies, 2 bytes per access, 92 with these.
__global__ __launch_bounds__(256) void k_xent_copy(XentCopies a) {
  const int which = static_cast<int>(blockIdx.x) >= a.c[0].blocks;
  const XentCopy c = a.c[which];
  if (blockIdx.x == 0 && a.count)
    for (int i = threadIdx.x; i < kTileSlots128; i += 256) a.count[i] = 0;
  const int64_t cells = c.pitch / 8, total = c.prows * cells, step = static_cast<int64_t>(c.blocks) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x - (which ? a.c[0].blocks : 0)) * 256 + threadIdx.x; i < total; i += 4 * step) {
    u32x4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t at = i + u * step, row = at / cells;
      const int col = static_cast<int>(at - row * cells) * 8, left = at < total && row < c.rows ? c.cols - col : 0;
      const uint16_t* p = c.src + row * c.ld + col;
      if (left >= 8) {
        __builtin_memcpy(&v[u], p, 16);
      } else {
        uint16_t h[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) h[k] = k < left ? p[k] : 0;
        v[u] = pack8(h);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * step < total) *reinterpret_cast<u32x4*>(c.dst + (i + u * step) * 8) = v[u];
  }
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

hipError_t launch_xent_copies(XentCopies a, hipStream_t st) {
  int blocks = 0;
  for (XentCopy& c : a.c) {
    c.blocks = static_cast<int32_t>(std::min<int64_t>((c.prows * (c.pitch / 8) + 1023) / 1024, 4096));
    blocks += c.blocks;
  }
  k_xent_copy<<<dim3(blocks > 0 ? blocks : 1), dim3(256), 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_xent_join(const XentJoin& j, hipStream_t st) {
  // few tokens: a workgroup each
  if (j.t <= 256) k_xent_join<1><<<dim3(j.t), dim3(256), 0, st>>>(j);
  else k_xent_join<16><<<dim3((j.t + 15) / 16), dim3(kJoinThreads<16>), 0, st>>>(j);
  return hipGetLastError();
}

}  // namespace dion
