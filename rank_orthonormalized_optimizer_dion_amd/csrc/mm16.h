// Dense products C = A B^T on the 16-bit matrix cores of gfx950, shared by
// the Newton-Schulz orthogonalization (k_ns.hip) and the linear layer
// (k_linear.hip).
//
// Operands are 16-bit values (float16 or bfloat16) in global memory, row
// pitch a multiple of 8 elements and 16-byte aligned:
//   K-major   (MC = false): element (x, k) at p[x ld + k]
//   x-major   (MC = true):  element (x, k) at p[k ld + x]
// x is the output dimension the operand feeds (a row of C for A, a column
// of C for B).  A value of more than 16 bits is a pair hi + lo (PL = 2): rows
// then hold 16 hi, the 16 lo of the same columns, the next 16 hi, ... (pitch
// 2 ld), and the product is hi hi + hi lo + lo hi, three matrix instructions
// per product into the same float32 accumulator.
//
// Tiles go from global memory straight to LDS (global_load_lds, 16 bytes per
// lane), no registers and no conversion.  A wavefront's 64 lanes write 64
// consecutive 16-byte cells, so a swizzle can only permute which cell of the
// source each lane fetches.  64 banks serve 16 cells at a time; the
// permutations let 16 consecutive lanes cover 16 different cells modulo 16:
//   K-major: cell (x, c) of a row of 4 cells sits at 4 x + (c ^ (x / 4) % 4);
//   x-major: cell (k, c), c = x / 8, sits at k CPR + (c ^ (4 (k % 4) + 2
//     (k / 8 % 2))); ds_read_b64_tr_b16 transposes 4 k by 16 x blocks on the
//     way out.
// Counted (share of the LDS's working cycles lost to conflicts): x-major tiles
// of one plane 1%, K-major tiles of two planes 2%; K-major tiles of one plane
// 50% (a read takes four cells of 16 rows there, two of 32 rows with two
// planes), and products with an x-major tile of two planes 33%.
#pragma once
#include <type_traits>

#include "device_common.h"

namespace dion {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
template <class T> using lptr = __attribute__((address_space(3))) T*;

// A wavefront-uniform value as a scalar: what came from memory or from the
// thread index stays in vector registers otherwise, and so do the loop
// counters and addresses made from it.
__device__ __forceinline__ int uniform32(int v) { return __builtin_amdgcn_readfirstlane(v); }
template <class T>
__device__ __forceinline__ T* uniform_at(T* p) {
  return reinterpret_cast<T*>(uniform64(reinterpret_cast<int64_t>(p)));
}
__device__ __forceinline__ int wave16() { return uniform32(static_cast<int>(threadIdx.x >> 6)); }

// Plain products use the 16 x 16 x 32 matrix instruction, pairs of planes the
// 32 x 32 x 16 one (a stage holds 16 k of a pair).  Both run at the same
// peak, but the card's power limit sets the clock: on random data an 8192^3
// float16 product ran at 1120 TFLOP/s with 32 x 32 x 16 and at 1220 with
// 16 x 16 x 32 (all-zero data: 1740 and 1820).
struct F16 {
  using Vec = f16x8;
  static __device__ __forceinline__ f32x16 mfma(Vec a, Vec b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mfma(Vec a, Vec b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
struct B16 {
  using Vec = bf16x8;
  static __device__ __forceinline__ f32x4 mfma(Vec a, Vec b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};

// 16 zero bytes in global memory: the source of tile cells past the
// reduction's end.
static __device__ u32x4 g_zero_cell;

// One LDS stage holds kStep16 16-bit values of the reduction per x: 32 k, or
// 16 k as hi and lo.
constexpr int kStep16 = 32;

// One operand of a tile: its pitch (2 ld when PL = 2), the tile's first x,
// the number of x and the reduction length K (K-major operands: the columns
// from K to the next multiple of 8 exist and are zero).  Cells past K are
// zero; x past the last re-reads the last x (K-major) or the last 8 x
// (x-major), which only feeds outputs that are never stored.
template <int BX, int NT, bool MC, int PL>
struct Tile16 {
  static constexpr int CELLS = BX * kStep16 / 8;
  static constexpr int PER = CELLS / NT;   // loads per thread and stage
  static constexpr int CPR = MC ? PL * BX / 8 : kStep16 / 8;   // cells per LDS row
  static constexpr int KS = kStep16 / PL;  // k per stage
  static constexpr int READS = MC ? 2 : 1; // LDS reads per MFMA operand
  static_assert(CELLS % NT == 0, "tile does not split over the threads");
  uint32_t off[PER];   // byte offset of this lane's source cell at k0 = 0
  int64_t xoff, ld;

  static __device__ __forceinline__ int swz(int row) { return MC ? 4 * (row & 3) + 2 * ((row >> 3) & 1) : (row >> 2) & 3; }

  __device__ __forceinline__ void init(int64_t ld_, int x0, int xn) {
    ld = ld_;
    xoff = MC ? static_cast<int64_t>(PL) * x0 : x0 * ld_;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int c = j * NT + static_cast<int>(threadIdx.x);
      const int row = c / CPR, cell = (c % CPR) ^ swz(row);
      if constexpr (MC) {
        const int x = min(cell * 8, (PL * (xn - x0) - 1) & ~7);
        off[j] = static_cast<uint32_t>(row * ld_ * 2 + x * 2);
      } else {
        off[j] = static_cast<uint32_t>(min(row, xn - x0 - 1) * ld_ * 2 + cell * 16);
      }
    }
  }

  // WHOLE: the stage lies inside the reduction.
  template <bool WHOLE>
  __device__ __forceinline__ void issue(const uint16_t* p, int k0, int K, u32x4* lds) const {
    const char* base = reinterpret_cast<const char*>(p + xoff + (MC ? k0 * ld : static_cast<int64_t>(PL) * k0));
    const int wave = wave16();
    if constexpr (WHOLE) {
#if defined(__HIP_DEVICE_COMPILE__)   // the host pass does not know the builtins' types
      // scalar base, 32-bit lane offsets: no address arithmetic per lane
      const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(uniform_at(base)), 0, 0xffffffffu, 0x00020000);
#pragma unroll
      for (int j = 0; j < PER; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lptr<void>)(lds + j * NT + wave * 64), 16, off[j], 0, 0, 0);
#endif
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int c = j * NT + static_cast<int>(threadIdx.x);
        const int row = c / CPR;
        const bool in = MC ? k0 + row < K : PL * k0 + ((c % CPR) ^ swz(row)) * 8 < PL * K;
        const char* src = in ? base + off[j] : reinterpret_cast<const char*>(&g_zero_cell);
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src),
                                         (lptr<void>)(lds + j * NT + wave * 64), 16, 0, 0);
      }
    }
  }

  // PL = 1: the 16 x 16 x 32 operand of the 16 x from x0 (a multiple of 16):
  // lane l holds x = x0 + l % 16, k = 8 (l / 16) + 0..7.
  // PL = 2: the 32 x 32 x 16 operand of the 32 x from x0 (a multiple of 32):
  // lane l holds x = x0 + l % 32 and the hi (f = 0) or lo (f = 1) of k =
  // 8 (l / 32) + 0..7.
  template <class V>
  static __device__ __forceinline__ V frag(const u32x4* lds, int x0, int f) {
    const int lane = threadIdx.x & 63;
    if constexpr (!MC) {
      const int row = x0 + (PL == 1 ? lane & 15 : lane & 31), c = PL == 1 ? lane >> 4 : 2 * f + (lane >> 5);
      return __builtin_bit_cast(V, lds[row * CPR + (c ^ swz(row))]);
    } else {
      const int i = lane & 15;
      const int k = 8 * (PL == 1 ? lane >> 4 : lane >> 5) + (i >> 2);
      const int block = (x0 >> 4) + (PL == 1 ? 0 : (lane >> 4) & 1);   // 16 x
      const int cell = (PL == 1 ? 2 * block : 4 * block + 2 * f) + ((i & 3) >> 1);
      const char* at = reinterpret_cast<const char*>(lds + k * CPR + (cell ^ swz(k))) + 8 * (i & 1);
      struct { s16x4 a, b; } v;
      v.a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lptr<s16x4>)(const_cast<char*>(at)));
      v.b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lptr<s16x4>)(const_cast<char*>(at + 4 * CPR * 16)));
      return __builtin_bit_cast(V, v);
    }
  }
};

// Shape of one tile product: BM x BN outputs, WM x WN wavefronts, ST LDS
// stages (a power of two).
template <class E_, int BM_, int BN_, int WM_, int WN_, int ST_, int PL_, bool AMC_, bool BMC_>
struct Shape16 {
  using E = E_;
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, ST = ST_, PL = PL_;
  static constexpr int NT = 64 * WM * WN;
  static constexpr int TM = BM / WM, TN = BN / WN;
  static constexpr int F = PL == 1 ? 16 : 32;            // side of a matrix instruction's output
  static constexpr int FM = TM / F, FN = TN / F;
  using Acc = typename std::conditional<PL == 1, f32x4, f32x16>::type;
  using A = Tile16<BM, NT, AMC_, PL>;
  using B = Tile16<BN, NT, BMC_, PL>;
  static constexpr int STAGE = A::CELLS + B::CELLS;   // 16-byte cells
  static constexpr int PER = A::PER + B::PER;         // loads per thread and stage
  // epilogue staging: one 64 x 64 block of floats per wavefront, rows padded by 4
  static constexpr int EPITCH = 68;
  static constexpr int ECELLS = WM * WN * 64 * EPITCH / 4;
  static constexpr int LDS_CELLS = ST * STAGE > ECELLS ? ST * STAGE : ECELLS;
  static_assert(TN % 64 == 0 && TM % 64 == 0, "the epilogue stages 64-wide blocks");
};

// A sum over reduction segments: segment s multiplies plane `a` of A by
// plane `b` of B over the same K (three-way split operands: planes apart by
// sa, sb elements).
struct Planes16 {
  const uint16_t* a;
  const uint16_t* b;
  int64_t sa, sb;
};

template <class S>
using Vec16 = typename S::E::Vec;

// The operands of wavefront rows m0 .. m0 + M - 1 of A, and of all its
// columns of B.
template <class S, int M>
__device__ __forceinline__ void load_a(Vec16<S> (&a)[M], const u32x4* st, int m0, int f) {
  const int xm = (wave16() / S::WN) * S::TM;
#pragma unroll
  for (int m = 0; m < M; ++m) a[m] = S::A::template frag<Vec16<S>>(st, xm + S::F * (m0 + m), f);
}
template <class S>
__device__ __forceinline__ void load_b(Vec16<S> (&b)[S::FN], const u32x4* st, int f) {
  const int xn = (wave16() % S::WN) * S::TN;
#pragma unroll
  for (int n = 0; n < S::FN; ++n) b[n] = S::B::template frag<Vec16<S>>(st + S::A::CELLS, xn + S::F * n, f);
}
template <class S, int M>
__device__ __forceinline__ void mma16(const Vec16<S> (&a)[M], const Vec16<S> (&b)[S::FN], int m0,
                                      typename S::Acc (&acc)[S::FM][S::FN]) {
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int n = 0; n < S::FN; ++n) acc[m0 + m][n] = S::E::mfma(a[m], b[n], acc[m0 + m][n]);
}

// Waits until at most N of this wavefront's loads are outstanding, then for
// the other wavefronts: what they loaded before is in LDS for everybody.
template <int N>
__device__ __forceinline__ void arrive16() {
  static_assert(N < 64, "vmcnt holds 6 bits");
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"i"(N) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The instruction mix of one cluster of M matrix instructions: R LDS reads
// spread over the first half of them, then G direct loads over the rest, so
// that they issue in the matrix pipe's shadow instead of before it.  (The
// loads write LDS, so the compiler keeps them behind the reads.)
template <int M, int R, int G, int I = 0>
__device__ __forceinline__ void interleave16() {
  if constexpr (I < M) {
    constexpr int H = M / 2;
    constexpr int r = I < H ? (I + 1) * R / H - I * R / H : 0;
    constexpr int g = I >= H ? (I + 1 - H) * G / (M - H) - (I - H) * G / (M - H) : 0;
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (r > 0) __builtin_amdgcn_sched_group_barrier(0x100, r, 0);
    if constexpr (g > 0) __builtin_amdgcn_sched_group_barrier(0x010, g, 0);
    interleave16<M, R, G, I + 1>();
  }
}

// acc = sum over nseg segments and k in [kbeg, kend).
//
// A step t runs two clusters of matrix instructions.  During the first it
// reads the rest of stage t's operands; then it meets the other wavefronts
// (stage t + 1 has arrived; everybody is done with stage t - 1); during the
// second it reads the first operands of stage t + 1 and starts the loads of
// stage t + ST - 1.  So loads have ST - 2 steps to arrive, and a wavefront
// always has a cluster whose operands are in registers when it reaches the
// barrier.  Two wavefronts per SIMD (256 x 256 tiles, 4 stages) or two
// workgroups per CU (128 x 128, 4 stages) fill each other's gaps; a launch
// of too few 128 x 128 tiles for that takes 8 stages (against 4: the linear
// layer from 3% faster to 2% slower, Newton-Schulz lists 1% to 3% slower).
// kend - kbeg is a multiple of a stage's k.
template <class S, class Seg>
__device__ __forceinline__ void tile_loop(const typename S::A& ta, const typename S::B& tb,
                                          const Planes16& pl, int total, Seg seg, int kbeg,
                                          int kend, u32x4* smem, typename S::Acc (&acc)[S::FM][S::FN]) {
  int is = 0, ik = kbeg;   // segment and reduction offset of the next issue
  auto stage = [&](int t) { return smem + (t & (S::ST - 1)) * S::STAGE; };
  auto issue = [&](int t) {
    int ia, ib;
    seg(is, ia, ib);
    u32x4* st = stage(t);
    ta.template issue<true>(pl.a + ia * pl.sa, ik, kend, st);
    tb.template issue<true>(pl.b + ib * pl.sb, ik, kend, st + S::A::CELLS);
    ik += S::A::KS;
    const bool wrap = ik >= kend;
    ik = wrap ? kbeg : ik;
    is += wrap;
  };
  constexpr int D = S::ST - 1;   // stages in flight
#pragma unroll
  for (int i = 0; i < D; ++i)
    if (i < total) issue(i);
  if (total >= D) arrive16<(D - 1) * S::PER>();
  else arrive16<0>();
  constexpr int RA = S::A::READS, RB = S::B::READS;
  int t = 0;
  if constexpr (S::PL == 1) {
    // clusters: the upper and the lower half of the wavefront's rows
    constexpr int H = S::FM / 2;
    Vec16<S> a0[H], a1[H], b0[S::FN], b1[S::FN];
    auto step = [&](int t, Vec16<S> (&b)[S::FN], Vec16<S> (&next)[S::FN]) {
      load_a<S>(a1, stage(t), H, 0);
      mma16<S>(a0, b, 0, acc);
      interleave16<H * S::FN, H * RA, 0>();
      arrive16<(D - 2) * S::PER>();
      load_a<S>(a0, stage(t + 1), 0, 0);
      load_b<S>(next, stage(t + 1), 0);
      issue(t + D);
      mma16<S>(a1, b, H, acc);
      interleave16<H * S::FN, H * RA + S::FN * RB, S::PER>();
    };
    load_a<S>(a0, smem, 0, 0);
    load_b<S>(b0, smem, 0);
    for (; t < total - D - 1; t += 2) {
      step(t, b0, b1);
      step(t + 1, b1, b0);
    }
    if (t < total - D) {
      step(t, b0, b1);
#pragma unroll
      for (int n = 0; n < S::FN; ++n) b0[n] = b1[n];
      ++t;
    }
    // every load has been started: one more meeting, then no barriers
    for (bool met = false; t < total; ++t) {
      load_a<S>(a1, stage(t), H, 0);
      mma16<S>(a0, b0, 0, acc);
      mma16<S>(a1, b0, H, acc);
      if (t + 1 < total) {
        if (!met) arrive16<0>();
        met = true;
        load_a<S>(a0, stage(t + 1), 0, 0);
        load_b<S>(b0, stage(t + 1), 0);
      }
    }
  } else {
    // clusters: hi hi and hi lo, then lo hi
    constexpr int MM = S::FM * S::FN, RR = S::FM * RA + S::FN * RB;
    Vec16<S> ah[S::FM], bh[S::FN], al[S::FM], bl[S::FN];
    load_a<S>(ah, smem, 0, 0);
    load_b<S>(bh, smem, 0);
    for (; t < total - D; ++t) {
      load_b<S>(bl, stage(t), 1);
      load_a<S>(al, stage(t), 0, 1);
      mma16<S>(ah, bh, 0, acc);
      mma16<S>(ah, bl, 0, acc);
      interleave16<2 * MM, RR, 0>();
      arrive16<(D - 2) * S::PER>();
      Vec16<S> next[S::FN];
      load_a<S>(ah, stage(t + 1), 0, 0);
      load_b<S>(next, stage(t + 1), 0);
      issue(t + D);
      mma16<S>(al, bh, 0, acc);
      interleave16<MM, RR, S::PER>();
#pragma unroll
      for (int n = 0; n < S::FN; ++n) bh[n] = next[n];
    }
    for (bool met = false; t < total; ++t) {
      load_b<S>(bl, stage(t), 1);
      load_a<S>(al, stage(t), 0, 1);
      mma16<S>(ah, bh, 0, acc);
      mma16<S>(ah, bl, 0, acc);
      mma16<S>(al, bh, 0, acc);
      if (t + 1 < total) {
        if (!met) arrive16<0>();
        met = true;
        load_a<S>(ah, stage(t + 1), 0, 0);
        load_b<S>(bh, stage(t + 1), 0);
      }
    }
  }
}

template <class S, class Seg>
__device__ __forceinline__ void tile_product(const typename S::A& ta, const typename S::B& tb,
                                             const Planes16& pl, int nseg, Seg seg, int kbeg,
                                             int kend, u32x4* smem,
                                             typename S::Acc (&acc)[S::FM][S::FN]) {
#pragma unroll
  for (int m = 0; m < S::FM; ++m)
#pragma unroll
    for (int n = 0; n < S::FN; ++n) acc[m][n] = typename S::Acc{};
  const int len = kend - kbeg;
  if (len <= 0) return;
  const int kfull = kend - len % S::A::KS;
  const int total = (kfull - kbeg) / S::A::KS * nseg;
  if (total > 0) {
    tile_loop<S>(ta, tb, pl, total, seg, kbeg, kfull, smem, acc);
    __syncthreads();   // the stages become the tail's, or the epilogue's staging area
  }
  // the ragged end of the reduction: one stage per segment
  for (int s = 0; kfull < kend && s < nseg; ++s) {
    int ia, ib;
    seg(s, ia, ib);
    ta.template issue<false>(pl.a + ia * pl.sa, kfull, kend, smem);
    tb.template issue<false>(pl.b + ib * pl.sb, kfull, kend, smem + S::A::CELLS);
    arrive16<0>();
    Vec16<S> a[S::FM], b[S::FN];
    load_a<S>(a, smem, 0, 0);
    load_b<S>(b, smem, 0);
    mma16<S>(a, b, 0, acc);
    if constexpr (S::PL == 2) {
      Vec16<S> al[S::FM], bl[S::FN];
      load_a<S>(al, smem, 0, 1);
      load_b<S>(bl, smem, 1);
      mma16<S>(a, bl, 0, acc);
      mma16<S>(al, b, 0, acc);
    }
    __syncthreads();
  }
}

// xcd_remap's chunks for the whole rounds of a launch; its last, partial round
// (all of a small launch) in one run of consecutive items per XCD, so that
// the tiles of one matrix meet in one or two L2s there too.
__device__ __forceinline__ int xcd_item(int b, int nb) {
  constexpr int ROUND = 8 * kXcdChunk;
  const int whole = nb / ROUND * ROUND;
  if (b < whole) return xcd_remap(b, nb);
  const int rest = nb - whole, x = (b - whole) & 7, each = rest >> 3, more = rest & 7;
  return whole + x * each + min(x, more) + ((b - whole) >> 3);
}

// How a launch's tiles share the chip.  Tiles 0 .. full - 1 are one
// workgroup's each.  The rest, less than a round of the chip's workgroup
// slots, would leave most of it idle for a whole tile's time: each of them is
// cut along the reduction into `slices` workgroups.
// Items go slice by slice: neighbours are then tiles that share panels of the
// same piece of the reduction.
struct Work16 {
  int32_t full, cut, slices;
  float* part;       // a tile of float32 per slice of the cut tiles
  uint32_t* count;   // one per cut tile, zero between launches
};
struct Item16 {
  int tile, slice, slices, cut;   // cut: index among the cut tiles
};
__device__ __forceinline__ Item16 item16(const Work16& w, int t) {
  if (t < w.full) return {t, 0, 1, 0};
  const int u = t - w.full, slice = u / w.cut, cut = u - slice * w.cut;
  return {w.full + cut, slice, w.slices, cut};
}

// The slice of [0, K) that an item works on, in whole stages.
template <class S>
__device__ __forceinline__ void slice16(const Item16& it, int K, int& kbeg, int& kend) {
  const int stages = (K + S::A::KS - 1) / S::A::KS, per = (stages + it.slices - 1) / it.slices * S::A::KS;
  kbeg = min(K, it.slice * per);
  kend = min(K, kbeg + per);
}

// Joins the slices of a cut tile: each leaves its sums in global memory; the
// workgroup that comes last (no one waits) adds all of them up in the order
// of the slices, whoever it is, so the result does not depend on the order of
// arrival.  Returns whether this workgroup goes on to the epilogue.
//
// The slices run on different XCDs, whose L2s do not see each other's lines.
// The sums are written and read with device-scope accesses, which go past
// them, so that waiting for one's own stores is enough: a device-scope fence
// would write back and invalidate the XCD's whole L2, once per wavefront (the
// 2048 x 2048 float32 case took 2.36 ms with it, 0.98 ms uncut, 0.80 ms so).
template <class S>
__device__ __forceinline__ bool join16(const Work16& w, const Item16& it, u32x4* smem,
                                       typename S::Acc (&acc)[S::FM][S::FN]) {
  if (it.slices == 1) return true;
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int Q = sizeof(typename S::Acc) / 16, V = S::FM * S::FN * Q;   // 16-byte pieces per thread
  constexpr int TILE = S::BM * S::BN * 4;
  constexpr int DEVICE = 0x10;   // cache policy: device scope
  constexpr int G = 8;           // pieces of a group: what is in flight has to leave registers to the sums
  static_assert(V % G == 0, "pieces come in groups");
  const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
      uniform_at(reinterpret_cast<char*>(w.part) + static_cast<int64_t>(it.cut) * it.slices * TILE), 0,
      it.slices * TILE, 0x00020000);
  const int lane = threadIdx.x * 16;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const typename S::Acc& a = acc[i / Q / S::FN][i / Q % S::FN];
    const int q = 4 * (i % Q);
    const f32x4 v = {a[q], a[q + 1], a[q + 2], a[q + 3]};
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rsrc, lane + i * (S::NT * 16),
                                           it.slice * TILE, DEVICE);
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wavefront's sums have arrived
  __syncthreads();
  uint32_t* flag = reinterpret_cast<uint32_t*>(smem);
  if (threadIdx.x == 0)
    *flag = __hip_atomic_fetch_add(w.count + it.cut, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  const bool last = *flag == static_cast<uint32_t>(it.slices - 1);
  __syncthreads();   // the flag's cell becomes staging area
  if (!last) return false;
  if (threadIdx.x == 0) __hip_atomic_store(w.count + it.cut, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
  for (int m = 0; m < S::FM; ++m)
#pragma unroll
    for (int n = 0; n < S::FN; ++n) acc[m][n] = typename S::Acc{};
  // two slices' pieces are loaded before the first is added
#pragma unroll
  for (int g = 0; g < V; g += G)
#pragma unroll 1
    for (int s = 0; s < it.slices; s += 2) {
      f32x4 v[2][G];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < G; ++i) {
          v[k][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          if (s + k < it.slices)
            v[k][i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                    rsrc, lane + (g + i) * (S::NT * 16), (s + k) * TILE, DEVICE));
        }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < G; ++i) {
          typename S::Acc& a = acc[(g + i) / Q / S::FN][(g + i) / Q % S::FN];
#pragma unroll
          for (int e = 0; e < 4; ++e) a[4 * ((g + i) % Q) + e] += v[k][i][e];
        }
    }
#endif
  return true;
}

// Hands the tile's values to out(row, col, v, pre) in runs of 8 along a row,
// row and col relative to the tile, through LDS (each wavefront its own
// 64 x 64 floats): the accumulators hold 4 consecutive rows of one column
// per lane, and every consumer wants whole row segments.  pre = fetch(row,
// col) is what the run needs from global memory; a batch of four runs is
// fetched before the first of them is written, because the compiler cannot
// move a load over a store to memory it may alias.
// TRANS: the tile's transpose instead: out(col, row, v, pre) with v the 8
// rows row .. row + 7 of one column.
template <class S, bool TRANS, class Fetch, class Out>
__device__ __forceinline__ void tile_runs(const typename S::Acc (&acc)[S::FM][S::FN], u32x4* smem, Fetch fetch, Out out) {
  const int lane = threadIdx.x & 63, wave = wave16();
  const int xm = (wave / S::WN) * S::TM, xn = (wave % S::WN) * S::TN;
  float* buf = reinterpret_cast<float*>(smem) + wave * 64 * S::EPITCH;
  constexpr int B = 64 / S::F;   // blocks per side of the staged piece
  // lane l holds column l % F of a block and, from row 4 (l / F), 4 rows
  // (16 x 16) or 4 groups of 4 rows, 8 rows apart (32 x 32)
  const int col = lane & (S::F - 1), row = 4 * (lane / S::F);
#pragma unroll
  for (int m = 0; m < S::FM; m += B)
#pragma unroll
    for (int n = 0; n < S::FN; n += B) {
#pragma unroll
      for (int mm = 0; mm < B; ++mm)
#pragma unroll
        for (int nn = 0; nn < B; ++nn) {
          const typename S::Acc& a = acc[m + mm][n + nn];
#pragma unroll
          for (int q = 0; q < (S::PL == 1 ? 1 : 4); ++q) {
            const int r = S::F * mm + 8 * q + row, c = S::F * nn + col;
            if constexpr (TRANS) {
              *reinterpret_cast<f32x4*>(buf + c * S::EPITCH + r) =
                  f32x4{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
            } else {
#pragma unroll
              for (int v = 0; v < 4; ++v) buf[(r + v) * S::EPITCH + c] = a[4 * q + v];
            }
          }
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const int r0 = (TRANS ? xn + S::F * n : xm + S::F * m) + (lane >> 3);
      const int c0 = (TRANS ? xm + S::F * m : xn + S::F * n) + 8 * (lane & 7);
      const float* at = buf + (lane >> 3) * S::EPITCH + 8 * (lane & 7);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        decltype(fetch(0, 0)) pre[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) pre[i] = fetch(r0 + 32 * h + 8 * i, c0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float* p = at + (32 * h + 8 * i) * S::EPITCH;
          const f32x4 lo = *reinterpret_cast<const f32x4*>(p), hi = *reinterpret_cast<const f32x4*>(p + 4);
          const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          out(r0 + 32 * h + 8 * i, c0, v, pre[i]);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
}
struct NoPre {};

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
