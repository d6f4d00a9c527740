// The cross entropy's products in float32 (mm32.h): z with the epilogues of
// k_xent.hip, dz kept in float32, dx = dz W and dW = dz^T x.  Bound by the matrix
// cores and by splitting values for them: 1021 tokens, 773 -> 50257 forward 0.44 ms,
// 177 TFLOP/s of float32 products, six times that of plane products (matrix cores
// busy 60%).  The gradients of 515 tokens, 517 -> 10007, 52 + 62 + 57 us, are one
// round of tiles each, of which 20% to 46% are padding.
#include "dion.h"
#include "mm32.h"
#include "work16.h"
#include "xent_tile.h"

namespace dion {

namespace {

enum Kind32 { kZ = 0, kDx, kDw };   // K-major both; K-major, x-major; x-major both

template <Kind32 KIND, bool GRAD>
__global__ __launch_bounds__(512, 2) void k_f32_mm(XentProduct32 p, XentEpi e) {
  using S = Shape32<KIND == kDw, KIND != kZ>;
  static_assert(S::TM == 64 && S::F == 16, "rows of a wavefront");
  __shared__ u32x4 smem[S::LDS_CELLS];
  const Work16 work{p.full, p.tx * p.ty - p.full, p.slices, p.part, p.count};
  const Item16 it = item16(work, xcd_item(blockIdx.x, gridDim.x));
  int ti, tj;
  tile_order(it.tile, p.tx, p.ty, ti, tj);
  const int r0 = ti * S::BM, c0 = tj * S::BN;
  int kbeg, kend;
  slice16<S>(it, p.K, kbeg, kend);
  typename S::Acc acc[S::FM][S::FN];
  typename S::TA ta;
  typename S::TB tb;
  ta.init(p.a, p.lda, r0, p.M);
  tb.init(p.b, p.ldb, c0, p.N);
  tile_product32<S>(ta, tb, S::TA::whole(r0, p.M) && S::TB::whole(c0, p.N), kbeg, kend, smem, acc);
  if constexpr (KIND != kZ) {
    if (p.apart && it.slices > 1) {   // k_f32_join's
      f32x4* at = reinterpret_cast<f32x4*>(p.part) + (static_cast<int64_t>(it.cut) * it.slices + it.slice) * (S::BM * S::BN / 4) + threadIdx.x;
#pragma unroll
      for (int m = 0; m < S::FM; ++m)
#pragma unroll
        for (int n = 0; n < S::FN; ++n) at[(m * S::FN + n) * S::NT] = acc[m][n];
      return;
    }
  }
  if (!join16<S>(work, it, smem, acc)) return;
  if constexpr (KIND == kZ) {
    const int wave = wave16();
    const int row0 = r0 + (wave / S::WN) * S::TM, col0 = c0 + (wave % S::WN) * S::TN;
    if constexpr (GRAD) {
      dz_tile<S>(acc, e, p.M, p.N, row0, col0);
      tile_runs<S, false>(
          acc, smem, [](int, int) { return NoPre{}; },
          [&](int r, int q, const float (&v)[8], const NoPre&) {
            const int row = r0 + r, col = c0 + q;
            if (row < p.M && col < e.pitch) {   // zero past the piece's columns
              float* at = e.dz32 + row * e.pitch + col;
              *reinterpret_cast<f32x4*>(at) = f32x4{v[0], v[1], v[2], v[3]};
              *reinterpret_cast<f32x4*>(at + 4) = f32x4{v[4], v[5], v[6], v[7]};
            }
          });
    } else {
      stats_tile<S>(acc, e, p.M, p.N, row0, col0, e.col0 + S::WN * tj + wave % S::WN);
    }
  } else {
    struct Pre {
      float v[8];
    };
    tile_runs<S, false>(
        acc, smem,
        [&](int r, int q) {
          Pre o{};
          const int row = r0 + r, col = c0 + q;
          if (p.accumulate && row < p.M && col < p.N) {
            const float* at = p.out + row * p.ldo + col;
            if (col + 8 <= p.N) {
              __builtin_memcpy(o.v, at, 32);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) o.v[i] = col + i < p.N ? at[i] : 0.0f;
            }
          }
          return o;
        },
        [&](int r, int q, const float (&v)[8], const Pre& old) {
          const int row = r0 + r, col = c0 + q;
          if (row >= p.M || col >= p.N) return;
          float* at = p.out + row * p.ldo + col;
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = v[i] + old.v[i];
          if (col + 8 <= p.N) {
            __builtin_memcpy(at, o, 32);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (col + i < p.N) at[i] = o[i];
          }
        });
  }
}

// The slices of cut tiles, in order: a workgroup per 1/8 of a tile (two pieces
// of each thread's accumulators).  z and dx of 515 tokens, 10007 -> 517, 17
// slices: 124 us with one workgroup per tile adding, 107 so.
__global__ __launch_bounds__(512) void k_f32_join(XentProduct32 p) {
  using S = Shape32<false, true>;   // the accumulators' layout is the same in both kinds
  constexpr int PARTS = S::FM * S::FN / 2;
  const int cut = blockIdx.x / PARTS, part = blockIdx.x % PARTS;
  const f32x4* at = reinterpret_cast<const f32x4*>(p.part) + static_cast<int64_t>(cut) * p.slices * (S::BM * S::BN / 4) + threadIdx.x;
  f32x4 sum[2] = {};
#pragma unroll 4
  for (int s = 0; s < p.slices; ++s)
#pragma unroll
    for (int i = 0; i < 2; ++i) sum[i] += at[s * (S::BM * S::BN / 4) + (2 * part + i) * S::NT];
  int ti, tj;
  tile_order(p.full + cut, p.tx, p.ty, ti, tj);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = (2 * part + i) / S::FN, n = (2 * part + i) % S::FN;
    const int row = ti * S::BM + (wave / S::WN) * S::TM + 16 * m + 4 * (lane >> 4);
    const int col = tj * S::BN + (wave % S::WN) * S::TN + 16 * n + (lane & 15);
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (row + v < p.M && col < p.N) {
        float* o = p.out + (row + v) * p.ldo + col;
        *o = p.accumulate ? *o + sum[i][v] : sum[i][v];
      }
  }
}

}  // namespace

hipError_t launch_xent_f32(const XentProduct32& p, const XentEpi& e, XentKind32 kind, hipStream_t st) {
  const dim3 grid(p.items), block(512);
  switch (kind) {
    case kXentStats32: k_f32_mm<kZ, false><<<grid, block, 0, st>>>(p, e); break;
    case kXentDz32: k_f32_mm<kZ, true><<<grid, block, 0, st>>>(p, e); break;
    case kXentDx32: k_f32_mm<kDx, false><<<grid, block, 0, st>>>(p, e); break;
    default: k_f32_mm<kDw, false><<<grid, block, 0, st>>>(p, e); break;
  }
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || !p.apart) return err;
  k_f32_join<<<dim3(8 * (p.tx * p.ty - p.full)), block, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace dion
