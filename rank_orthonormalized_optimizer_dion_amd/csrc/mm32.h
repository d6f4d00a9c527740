// Dense products of float32 operands C = A B^T on the bfloat16 matrix cores,
// the operands as they lie in memory: K-major or x-major (mm16.h), any pitch,
// 4-byte aligned.
//
// A float32 value is the sum of three bfloat16 planes: hi, its upper 16 bits;
// mid, the rest rounded to bfloat16; lo, what is left, exact.  A product is six
// plane products, (mid mid) (lo hi) (hi lo) (mid hi) (hi mid) (hi hi); the dropped
// ones are below 2^-22 of it, of either sign.  Unlike copies in planes, which a
// plain product then sweeps six times (k_lin_pack, k_lin_mm), a value is read
// once, split once on its way from registers into LDS (seven instructions), and
// a stage of LDS feeds all six (1021 tokens, 773 -> 50257: 410 us, by copies
// 530; 2048 tokens, 4096 -> 16000: 228 TFLOP/s, 1.37 PFLOP/s of plane products,
// where a plain bfloat16 product of the library reaches 1.40 to 1.45).
//
// Tiles of 128 x 256 by 8 wavefronts of 64 x 64, two LDS stages of 32 k and
// three planes: while a stage is multiplied, the next one's values, already in
// registers, are split and written, and the one after it is loaded.  Two
// wavefronts per SIMD let splitting and matrix instructions overlap.  (Meeting
// halfway through a stage instead, the next stage's first operands read during
// the second half: 2% to 5% slower.)
#pragma once
#include "mm16.h"

namespace dion {

// Eight values' planes, packed by pairs.
struct Split8 {
  u32x4 p[3];
};
__device__ __forceinline__ Split8 split_planes(const float (&v)[8]) {
  Split8 o;
  uint32_t hi[8], mid[8], lo[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi[i] = __float_as_uint(v[i]);
    const float rest = v[i] - __uint_as_float(hi[i] & 0xffff0000u);
    mid[i] = __float_as_uint(rest) + 0x8000u;
    lo[i] = __float_as_uint(rest - __uint_as_float(mid[i] & 0xffff0000u));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {   // upper halves of two registers
    o.p[0][i] = __builtin_amdgcn_perm(hi[2 * i + 1], hi[2 * i], 0x07060302u);
    o.p[1][i] = __builtin_amdgcn_perm(mid[2 * i + 1], mid[2 * i], 0x07060302u);
    o.p[2][i] = __builtin_amdgcn_perm(lo[2 * i + 1], lo[2 * i], 0x07060302u);
  }
  return o;
}

// One operand of a tile: BX x by 32 k per stage, in chunks of 8 consecutive
// floats, which become one 16-byte cell of each plane (mm16.h's layouts).  x past
// the last re-reads the last (K-major) or is zero (x-major), k past the last is
// zero.
template <int BX, int NT, bool MC>
struct Tile32 {
  using Cells = Tile16<BX, NT, MC, 1>;
  static constexpr int CH = BX * 4 / NT;
  static_assert(BX * 4 % NT == 0, "chunks do not split over the threads");
  static constexpr int PLANE = BX * 4;   // cells
  const float* p[CH];   // this lane's chunks at k = 0
  int64_t ld;
  int32_t at[CH];       // their cells
  int32_t left[CH];     // x from the chunk's first to the last (x-major)

  __device__ __forceinline__ void init(const float* base, int64_t ld_, int x0, int xn) {
    ld = ld_;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = j * NT + static_cast<int>(threadIdx.x), row = c / Cells::CPR, cell = c % Cells::CPR;
      at[j] = row * Cells::CPR + (cell ^ Cells::swz(row));
      if constexpr (MC) {
        left[j] = xn - x0 - 8 * cell;
        p[j] = base + row * ld_ + x0 + 8 * cell;
      } else {
        left[j] = 8;
        p[j] = base + min(x0 + row, xn - 1) * ld_ + 8 * cell;
      }
    }
  }
  // Whether every chunk of a whole stage exists.
  static __device__ __forceinline__ bool whole(int x0, int xn) { return !MC || x0 + BX <= xn; }
  // The chunks of the stage at k0 of a reduction that ends at K.  WHOLE: all of
  // them exist.
  template <bool WHOLE>
  __device__ __forceinline__ void load(int k0, int K, float (&v)[CH][8]) const {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = j * NT + static_cast<int>(threadIdx.x);
      const int count = WHOLE ? 8 : MC ? (k0 + c / Cells::CPR < K ? left[j] : 0) : K - k0 - 8 * (c % Cells::CPR);
      const float* q = p[j] + (MC ? k0 * ld : k0);
      if (WHOLE || count >= 8) {
        f32x4 a, b;
        __builtin_memcpy(&a, q, 16);
        __builtin_memcpy(&b, q + 4, 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[j][i] = a[i];
          v[j][4 + i] = b[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = i < count ? q[i] : 0.0f;
      }
    }
  }
  __device__ __forceinline__ void store(const float (&v)[CH][8], u32x4* lds) const {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const Split8 s = split_planes(v[j]);
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) lds[pl * PLANE + at[j]] = s.p[pl];
    }
  }
};

template <bool AMC, bool BMC>
struct Shape32 : Shape16<B16, 128, 256, 2, 4, 1, AMC, BMC> {
  using Base = Shape16<B16, 128, 256, 2, 4, 1, AMC, BMC>;
  using TA = Tile32<128, Base::NT, AMC>;
  using TB = Tile32<256, Base::NT, BMC>;
  static constexpr int STAGE = 3 * (TA::PLANE + TB::PLANE);   // cells
  static constexpr int LDS_CELLS = 2 * STAGE > Base::ECELLS ? 2 * STAGE : Base::ECELLS;
};

// acc = sum over k in [kbeg, kend).  whole: both tiles lie inside their
// operands.
template <class S>
__device__ __forceinline__ void tile_product32(const typename S::TA& ta, const typename S::TB& tb, bool whole, int kbeg,
                                               int kend, u32x4* smem, typename S::Acc (&acc)[S::FM][S::FN]) {
#pragma unroll
  for (int m = 0; m < S::FM; ++m)
#pragma unroll
    for (int n = 0; n < S::FN; ++n) acc[m][n] = typename S::Acc{};
  if (kend <= kbeg) return;
  const int xm = (wave16() / S::WN) * S::TM, xn = (wave16() % S::WN) * S::TN;
  float va[S::TA::CH][8], vb[S::TB::CH][8];
  const auto load = [&](auto all, int k) {
    ta.template load<decltype(all)::value>(k, kend, va);
    tb.template load<decltype(all)::value>(k, kend, vb);
  };
  const auto store = [&](int stage) {
    u32x4* st = smem + stage * S::STAGE;
    ta.store(va, st);
    tb.store(vb, st + 3 * S::TA::PLANE);
  };
  // one stage; FAST: two more follow, all of whose chunks exist
  const auto step = [&](auto fast, int k, int stage) {
    constexpr bool FAST = decltype(fast)::value;
    const u32x4* st = smem + stage * S::STAGE;
    Vec16<S> a[3][S::FM], b[3][S::FN];
    const auto get_a = [&](int pl) {
#pragma unroll
      for (int m = 0; m < S::FM; ++m) a[pl][m] = S::A::template frag<Vec16<S>>(st + pl * S::TA::PLANE, xm + 16 * m, 0);
    };
    const auto get_b = [&](int pl) {
#pragma unroll
      for (int n = 0; n < S::FN; ++n)
        b[pl][n] = S::B::template frag<Vec16<S>>(st + 3 * S::TA::PLANE + pl * S::TB::PLANE, xn + 16 * n, 0);
    };
    const auto mul = [&](int pa, int pb) {
#pragma unroll
      for (int m = 0; m < S::FM; ++m)
#pragma unroll
        for (int n = 0; n < S::FN; ++n) acc[m][n] = S::E::mfma(a[pa][m], b[pb][n], acc[m][n]);
    };
    get_a(1);
    get_b(1);
    get_a(2);
    get_b(0);
    mul(1, 1);
    get_a(0);
    get_b(2);
    mul(2, 0);
    if (FAST || k + kStep16 < kend) store(stage ^ 1);
    mul(0, 2);
    if constexpr (FAST) load(std::true_type{}, k + 2 * kStep16);
    else if (k + 2 * kStep16 < kend) load(std::false_type{}, k + 2 * kStep16);
    mul(1, 0);
    mul(0, 1);
    mul(0, 0);
    __syncthreads();
  };
  load(std::false_type{}, kbeg);
  store(0);
  if (kbeg + kStep16 < kend) load(std::false_type{}, kbeg + kStep16);
  __syncthreads();
  int k = kbeg, stage = 0;
  if (whole)
    for (; k + 3 * kStep16 <= kend; k += kStep16, stage ^= 1) step(std::true_type{}, k, stage);
  for (; k < kend; k += kStep16, stage ^= 1) step(std::false_type{}, k, stage);
}

}  // namespace dion
