// Dense products C = A B^T on the 16-bit matrix cores of gfx950, shared by
// the Newton-Schulz orthogonalization (k_ns.hip) and the linear layer
// (k_linear.hip).
//
// Operands are planes of 16-bit values (float16 or bfloat16) in global
// memory, row pitch a multiple of 8 elements and 16-byte aligned:
//   K-major   (MC = false): element (x, k) at p[x ld + k]
//   x-major   (MC = true):  element (x, k) at p[k ld + x]
// x is the output dimension the operand feeds (a row of C for A, a column
// of C for B).  A value of more than 16 bits is a sum of PL planes (value =
// hi + lo); the product is then hi hi + hi lo + lo hi, three matrix
// instructions per product into the same float32 accumulator.
//
// Tiles go from global memory straight to LDS (global_load_lds, 16 bytes per
// lane), no registers and no conversion.  A wavefront's 64 lanes write 64
// consecutive 16-byte cells, so a swizzle can only permute which cell of the
// source each lane fetches:
//   K-major: cell (x, c), c = k / 8, sits at x (BK / 8) + (c ^ s(x)), so the
//     ds_read_b128 of an MFMA operand (32 rows x, one c per half wavefront)
//     touches all bank groups evenly;
//   x-major: cell (k, c), c = x / 8, sits at k (BX / 8) + (c ^ 4 (k & 3));
//     ds_read_b64_tr_b16 transposes 4 k by 16 x blocks on the way out.
#pragma once
#include "device_common.h"

namespace dion {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
template <class T> using lptr = __attribute__((address_space(3))) T*;

struct F16 {
  using Vec = f16x8;
  static __device__ __forceinline__ f32x16 mfma(Vec a, Vec b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};
struct B16 {
  using Vec = bf16x8;
  static __device__ __forceinline__ f32x16 mfma(Vec a, Vec b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};

// 16 zero bytes in global memory: the source of tile cells past the
// reduction's end.
static __device__ u32x4 g_zero_cell;

// One operand of a tile: `p` the plane (uniform), its pitch, the tile's
// first x, the number of x and the reduction length K (K-major operands: the
// columns from K to the next multiple of 8 exist and are zero).  Cells past
// K are zero; x past the last re-reads the last
// x (K-major) or the last 8 x (x-major), which only feeds outputs that are
// never stored.
template <int BX, int BK, int NT, bool MC>
struct Tile16 {
  static constexpr int CELLS = BX * BK / 8;
  static constexpr int PER = CELLS / NT;   // loads per thread and tile
  static_assert(CELLS % NT == 0 && (BK == 32 || BK == 64), "tile does not split over the threads");
  static constexpr int CPR = MC ? BX / 8 : BK / 8;   // cells per LDS row
  uint32_t off[PER];   // byte offset of this lane's source cell at k0 = 0
  int64_t xoff, ld;

  static __device__ __forceinline__ int swz(int row) {
    if constexpr (MC) return 4 * (row & 3);
    else if constexpr (BK == 64) return row & 7;
    else return (row >> 1) & 3;
  }

  __device__ __forceinline__ void init(int64_t ld_, int x0, int xn) {
    ld = ld_;
    xoff = MC ? x0 : x0 * ld_;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int c = j * NT + static_cast<int>(threadIdx.x);
      const int row = c / CPR, cell = (c % CPR) ^ swz(row);
      if constexpr (MC) {
        const int x = min(cell * 8, (xn - x0 - 1) & ~7);
        off[j] = static_cast<uint32_t>(row * ld_ * 2 + x * 2);
      } else {
        off[j] = static_cast<uint32_t>(min(row, xn - x0 - 1) * ld_ * 2 + cell * 16);
      }
    }
  }

  __device__ __forceinline__ void issue(const uint16_t* plane, int k0, int K, u32x4* lds) const {
    const char* base = reinterpret_cast<const char*>(plane + xoff + (MC ? k0 * ld : static_cast<int64_t>(k0)));
    const int wave = threadIdx.x >> 6;
    const bool whole = k0 + BK <= K;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const char* src = base + off[j];
      if (!whole) {
        const int c = j * NT + static_cast<int>(threadIdx.x);
        const int row = c / CPR;
        const int k = k0 + (MC ? row : ((c % CPR) ^ swz(row)) * 8);
        if (k >= K) src = reinterpret_cast<const char*>(&g_zero_cell);
      }
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src),
                                       (lptr<void>)(lds + j * NT + wave * 64), 16, 0, 0);
    }
  }

  // The MFMA operand of 32 x from x0 (a multiple of 32) and 16 k from 16 q:
  // lane l holds x = x0 + l % 32, k = 16 q + 8 (l / 32) + 0..7.
  template <class V>
  static __device__ __forceinline__ V frag(const u32x4* lds, int x0, int q) {
    const int lane = threadIdx.x & 63;
    if constexpr (!MC) {
      const int row = x0 + (lane & 31), c = 2 * q + (lane >> 5);
      return __builtin_bit_cast(V, lds[row * CPR + (c ^ swz(row))]);
    } else {
      const int i = lane & 15;
      const int k = 16 * q + 8 * (lane >> 5) + (i >> 2);
      const int cell = (x0 >> 3) + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
      const char* at = reinterpret_cast<const char*>(lds + k * CPR + (cell ^ swz(i >> 2))) + 8 * (i & 1);
      struct { s16x4 a, b; } v;
      v.a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lptr<s16x4>)(const_cast<char*>(at)));
      v.b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lptr<s16x4>)(const_cast<char*>(at + 4 * CPR * 16)));
      return __builtin_bit_cast(V, v);
    }
  }
};

// Shape of one tile product: BM x BN outputs, BK reduction steps per LDS
// stage, WM x WN wavefronts, PL planes per operand.
template <class E_, int BM_, int BN_, int BK_, int WM_, int WN_, int PL_, bool AMC_, bool BMC_>
struct Shape16 {
  using E = E_;
  static constexpr int BM = BM_, BN = BN_, BK = BK_, WM = WM_, WN = WN_, PL = PL_;
  static constexpr int NT = 64 * WM * WN;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
  using A = Tile16<BM, BK, NT, AMC_>;
  using B = Tile16<BN, BK, NT, BMC_>;
  static constexpr int STAGE = PL * (A::CELLS + B::CELLS);   // 16-byte cells
  // epilogue staging: one 32 x TN block of floats per wavefront, rows padded
  // by 4, or its transpose (TN = 64: two 32 x 32 blocks, 32 rows of 64)
  static constexpr int EPITCH = 68;
  static constexpr int ECELLS = WM * WN * 32 * EPITCH / 4;
  static constexpr int LDS_CELLS = 2 * STAGE > ECELLS ? 2 * STAGE : ECELLS;
  static_assert(TN == 64 && TM % 64 == 0, "the epilogue stages 64-wide blocks");
};

// A sum over reduction segments: segment s multiplies plane as[s] of A by
// plane bs[s] of B over the same K.  One segment for plain products, six for
// three-way split operands.
struct Planes16 {
  const uint16_t* a;
  const uint16_t* b;
  int64_t sa, sb;   // elements from one plane to the next
};

template <class S>
__device__ __forceinline__ void tile_mma(const u32x4* st, f32x16 (&acc)[S::FM][S::FN]) {
  using V = typename S::E::Vec;
  const int wave = threadIdx.x >> 6;
  const int xm = (wave / S::WN) * S::TM, xn = (wave % S::WN) * S::TN;
  const u32x4* a = st;
  const u32x4* b = st + S::PL * S::A::CELLS;
#pragma unroll
  for (int q = 0; q < S::BK / 16; ++q) {
    V fa[S::PL][S::FM], fb[S::PL][S::FN];
#pragma unroll
    for (int p = 0; p < S::PL; ++p) {
#pragma unroll
      for (int n = 0; n < S::FN; ++n) fb[p][n] = S::B::template frag<V>(b + p * S::B::CELLS, xn + 32 * n, q);
#pragma unroll
      for (int m = 0; m < S::FM; ++m) fa[p][m] = S::A::template frag<V>(a + p * S::A::CELLS, xm + 32 * m, q);
    }
#pragma unroll
    for (int m = 0; m < S::FM; ++m)
#pragma unroll
      for (int n = 0; n < S::FN; ++n) {
        if constexpr (S::PL == 2) {
          acc[m][n] = S::E::mfma(fa[1][m], fb[0][n], acc[m][n]);
          acc[m][n] = S::E::mfma(fa[0][m], fb[1][n], acc[m][n]);
        }
        acc[m][n] = S::E::mfma(fa[0][m], fb[0][n], acc[m][n]);
      }
  }
}

// acc = sum over nseg segments and k in [kbeg, kend) (kbeg a multiple of
// BK).  Two LDS stages: the loads of step t + 1 are in flight during the
// matrix instructions of step t, and one barrier per step both publishes
// the stage just loaded and frees the one just read.
template <class S, class Seg>
__device__ __forceinline__ void tile_product(const typename S::A& ta, const typename S::B& tb,
                                             const Planes16& pl, int nseg, Seg seg, int kbeg,
                                             int kend, u32x4* smem,
                                             f32x16 (&acc)[S::FM][S::FN]) {
#pragma unroll
  for (int m = 0; m < S::FM; ++m)
#pragma unroll
    for (int n = 0; n < S::FN; ++n)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[m][n][v] = 0.0f;
  const int nk = (kend - kbeg + S::BK - 1) / S::BK;
  const int total = nk * nseg;
  if (total <= 0) return;
  int is = 0, ik = kbeg;   // segment and reduction offset of the next issue
  auto issue = [&](u32x4* st) {
    int ia, ib;
    seg(is, ia, ib);
    const uint16_t* a = pl.a + ia * pl.sa;
    const uint16_t* b = pl.b + ib * pl.sb;
#pragma unroll
    for (int p = 0; p < S::PL; ++p) {
      ta.issue(a + p * pl.sa, ik, kend, st + p * S::A::CELLS);
      tb.issue(b + p * pl.sb, ik, kend, st + S::PL * S::A::CELLS + p * S::B::CELLS);
    }
    ik += S::BK;
    if (ik >= kend) {
      ik = kbeg;
      ++is;
    }
  };
  issue(smem);
  for (int t = 0; t < total; ++t) {
    __syncthreads();
    if (t + 1 < total) issue(smem + ((t + 1) & 1) * S::STAGE);
    tile_mma<S>(smem + (t & 1) * S::STAGE, acc);
  }
  __syncthreads();   // the stages become the epilogue's staging area
}

// Hands the tile's values to out(row, col, v) in runs of 8 along a row,
// row and col relative to the tile, through LDS (each wavefront its own
// 32 x 64 floats): the accumulators hold 4 consecutive rows of one column
// per lane, and every consumer wants whole row segments.
template <class S, class Out>
__device__ __forceinline__ void tile_rows(const f32x16 (&acc)[S::FM][S::FN], u32x4* smem, Out out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int xm = (wave / S::WN) * S::TM, xn = (wave % S::WN) * S::TN;
  float* buf = reinterpret_cast<float*>(smem) + wave * 32 * S::EPITCH;
#pragma unroll
  for (int m = 0; m < S::FM; ++m) {
#pragma unroll
    for (int n = 0; n < S::FN; ++n)
#pragma unroll
      for (int v = 0; v < 16; ++v)
        buf[(8 * (v >> 2) + 4 * (lane >> 5) + (v & 3)) * S::EPITCH + 32 * n + (lane & 31)] = acc[m][n][v];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 3), c = 8 * (lane & 7);
      const f32x4 lo = *reinterpret_cast<const f32x4*>(buf + r * S::EPITCH + c);
      const f32x4 hi = *reinterpret_cast<const f32x4*>(buf + r * S::EPITCH + c + 4);
      const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      out(xm + 32 * m + r, xn + c, v);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// The same for the transposed tile: out(col, row, v) with v the 8 rows
// row .. row + 7 of one column.
template <class S, class Out>
__device__ __forceinline__ void tile_cols(const f32x16 (&acc)[S::FM][S::FN], u32x4* smem, Out out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int xm = (wave / S::WN) * S::TM, xn = (wave % S::WN) * S::TN;
  float* buf = reinterpret_cast<float*>(smem) + wave * 32 * S::EPITCH;
#pragma unroll
  for (int n = 0; n < S::FN; ++n)
#pragma unroll
    for (int m = 0; m < S::FM; m += 2) {
#pragma unroll
      for (int mm = 0; mm < 2; ++mm)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16& a = acc[m + mm][n];
          *reinterpret_cast<f32x4*>(buf + (lane & 31) * S::EPITCH + 32 * mm + 8 * q + 4 * (lane >> 5)) =
              f32x4{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 3), c = 8 * (lane & 7);
        const f32x4 lo = *reinterpret_cast<const f32x4*>(buf + r * S::EPITCH + c);
        const f32x4 hi = *reinterpret_cast<const f32x4*>(buf + r * S::EPITCH + c + 4);
        const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        out(xn + 32 * n + r, xm + 32 * m + c, v);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
}

// Round to nearest even.
__device__ __forceinline__ uint16_t to_f16(float x) { return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x)); }
__device__ __forceinline__ float f16_to_f32(uint16_t u) { return static_cast<float>(__builtin_bit_cast(_Float16, u)); }
__device__ __forceinline__ uint16_t to_bf16(float x) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x)); }

// x as it is in a register.  A split into hi = round(x) and lo = x - hi needs
// the same x on both sides: left to itself the compiler may fold the
// multiplication that made x into one of the two conversions (one rounding
// where the other has two), and hi then differs from the hi that lo was
// taken from by a whole unit wherever x lies next to a tie.
__device__ __forceinline__ float pinned(float x) {
  asm volatile("" : "+v"(x));
  return x;
}

__device__ __forceinline__ u32x4 pack8(const uint16_t (&h)[8]) {
  return u32x4{h[0] | (static_cast<uint32_t>(h[1]) << 16), h[2] | (static_cast<uint32_t>(h[3]) << 16),
               h[4] | (static_cast<uint32_t>(h[5]) << 16), h[6] | (static_cast<uint32_t>(h[7]) << 16)};
}

}  // namespace dion
