// The whole orthogonalization (or Muon step) of a small matrix in one
// workgroup: dion_orthogonalize and dion_muon_step on matrices whose smaller
// side is at most 128 and whose planes fit the LDS.
//
// X (p x q, p <= q) stays in LDS as float16 hi + lo planes through all
// iterations; the p x p matrices A and B live in registers and pass through
// one LDS plane (hi, then lo) to become matrix operands.  Products are hi hi
// + hi lo + lo hi on v_mfma_f32_16x16x32_f16 in both arithmetic modes: such a
// matrix has few singular values for its rounding errors to average over, and
// no second product would be saved that costs as much as a launch.
//
// Per iteration and 8 wavefronts:
//   A = X X^T           K-major operands, each wavefront a block of A
//   A^2                 A through the LDS plane; B = a I + b A + c A^2
//   X <- B X            each wavefront its own columns of X, which it alone
//                       reads and overwrites
//
// One compute unit's matrix cores bound it: at 128 x 256 an iteration has
// 15,400 cycles of matrix instructions per SIMD and takes 28,900 (12 us; the
// rest is barriers around the one p x p plane).  Five quintic iterations of
// 256 x 128: 74 us, where the grouped launches took 165; 64 x 64: 22 us; 200
// matrices of 256 x 128 in one call: 0.42 ms.
#include "dion.h"
#include "mm16.h"
#include "ns_types.h"
#include "ns_device.h"

namespace dion {

namespace {

constexpr int kWaves = 8;

// X plane: PP rows of QP values, 16-byte cells.  The cell's low 4 bits are
// permuted by the row so that 16 rows of one column cell (K-major operands),
// and rows 0-3 and 8-11 of one pair of cells (transposed reads), fall on
// different banks.
__device__ __forceinline__ int x_swz(int row) {
  return 2 * ((row & 3) + 4 * ((row >> 3) & 1)) + ((row >> 2) & 1);
}
template <int QP>
__device__ __forceinline__ int x_cell(int row, int cell) {
  return row * (QP / 8) + (cell ^ x_swz(row));
}
// The p x p plane: rows of PP values; cells permuted by the row.
template <int PP>
__device__ __forceinline__ int a_cell(int row, int cell) {
  return row * (PP / 8) + (cell ^ (PP == 128 ? row & 15 : (row >> 1) & 7));
}

template <int PP, int QP>
struct Small {
  static constexpr int XCELLS = PP * QP / 8, ACELLS = PP * PP / 8;
  static constexpr int LDS_CELLS = 2 * XCELLS + ACELLS;
  static constexpr int NB = PP / 16;               // 16-blocks per side of A
  static constexpr int FM = NB / 4, FN = NB / 2;   // blocks per wavefront (4 x 2 wavefronts)
  static constexpr int FC = QP / 16 / kWaves;      // column blocks of X per wavefront
  static constexpr int KS = PP / 32;               // reduction steps over p
  static_assert(FM >= 1 && FC >= 1, "too small for 8 wavefronts");

  // K-major operand of 16 rows from r0, k from 32 ks, of an X plane
  static __device__ __forceinline__ f16x8 x_row(const u32x4* x, int r0, int ks, int lane) {
    return __builtin_bit_cast(f16x8, x[x_cell<QP>(r0 + (lane & 15), 4 * ks + (lane >> 4))]);
  }
  // operand of the 16 columns from c0 (x = column), k = rows from 32 ks
  static __device__ __forceinline__ f16x8 x_col(const u32x4* x, int c0, int ks, int lane) {
    const int i = lane & 15;
    const int row = 32 * ks + 8 * (lane >> 4) + (i >> 2), cell = (c0 >> 3) + ((i & 3) >> 1);
    struct { s16x4 a, b; } v;
    v.a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lptr<s16x4>)(reinterpret_cast<char*>(const_cast<u32x4*>(x) + x_cell<QP>(row, cell)) + 8 * (i & 1)));
    v.b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lptr<s16x4>)(reinterpret_cast<char*>(const_cast<u32x4*>(x) + x_cell<QP>(row + 4, cell)) + 8 * (i & 1)));
    return __builtin_bit_cast(f16x8, v);
  }
  static __device__ __forceinline__ f16x8 a_row(const u32x4* a, int r0, int ks, int lane) {
    return __builtin_bit_cast(f16x8, a[a_cell<PP>(r0 + (lane & 15), 4 * ks + (lane >> 4))]);
  }
  // Writes one plane (hi or lo parts) of this wavefront's blocks of a
  // symmetric p x p matrix: lane l holds 4 rows of column l % 16, stored as 4
  // columns of that row.
  static __device__ __forceinline__ void a_store(u32x4* a, const f32x4 (&v)[FM][FN], bool lo, int lane) {
    const int wave = wave16();
    const int r0 = 16 * FM * (wave >> 1) + 4 * (lane >> 4), c0 = 16 * FN * (wave & 1) + (lane & 15);
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        const int r = r0 + 16 * m, c = c0 + 16 * n;
        uint16_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = v[m][n][e];
          h[e] = to_f16(x);
          if (lo) h[e] = to_f16(x - f16_to_f32(h[e]));
        }
        u32x2* at = reinterpret_cast<u32x2*>(a + a_cell<PP>(c, r >> 3)) + ((r >> 2) & 1);
        *at = u32x2{h[0] | (static_cast<uint32_t>(h[1]) << 16), h[2] | (static_cast<uint32_t>(h[3]) << 16)};
      }
  }
};

template <typename GT, int PP, int QP>
__global__ __launch_bounds__(64 * kWaves) void k_ns_small(NsSmall L) {
  using T = Small<PP, QP>;
  constexpr int FM = T::FM, FN = T::FN, FC = T::FC, KS = T::KS;
  __shared__ u32x4 smem[T::LDS_CELLS];
  u32x4* xh = smem;
  u32x4* xl = smem + T::XCELLS;
  u32x4* ab = smem + 2 * T::XCELLS;
  NsDesc d;
  NsClass c;
  int local;
  ns_locate(L.common, blockIdx.x, d, c, local);
  const int wave = wave16();
  const int p = uniform32(d.p), q = uniform32(d.q), tall = uniform32(d.tall);

  // D, in groups of 4 consecutive columns of X (row i, columns j .. j + 3): a
  // 16-byte piece of the caller's row when wide; 4 rows of the caller's when
  // tall, neighbouring lanes then reading neighbouring columns.  Every load
  // is in flight before the first use.
  constexpr int NG = PP * QP / 4 / (64 * kWaves);
  const bool vec = !tall && q % 4 == 0 && d.ldg % 4 == 0 &&
                   (reinterpret_cast<uint64_t>(d.G) & (4 * sizeof(GT) - 1)) == 0 &&
                   (reinterpret_cast<uint64_t>(d.M) & 15) == 0;
  const int64_t gi = tall ? 1 : d.ldg, gj = tall ? d.ldg : 1;   // strides of G by X's row and column
  const int mi = tall ? 1 : q, mj = tall ? p : 1;               // and of M
  auto group = [&](int u, int& i, int& j) {
    const int g = threadIdx.x + 64 * kWaves * u;
    if (tall) {
      i = g % PP;
      j = 4 * (g / PP);
    } else {
      i = g / (QP / 4);
      j = 4 * (g % (QP / 4));
    }
    return i < p && j < q;
  };
  float x[NG][4], m1[NG][4];
  double sum = 0.0;
#pragma unroll
  for (int u = 0; u < NG; ++u) {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[u][k] = m1[u][k] = 0.0f;
    int i, j;
    if (!group(u, i, j)) continue;
    const int64_t o = i * gi + j * gj;
    const float* mp = d.M + (i * mi + j * mj);
    if (vec) {
      if constexpr (sizeof(GT) == 2) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(d.G) + o);
        x[u][0] = __uint_as_float(w.x << 16);
        x[u][1] = __uint_as_float(w.x & 0xffff0000u);
        x[u][2] = __uint_as_float(w.y << 16);
        x[u][3] = __uint_as_float(w.y & 0xffff0000u);
      } else {
        const f32x4 w = *reinterpret_cast<const f32x4*>(static_cast<const float*>(d.G) + o);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[u][k] = w[k];
      }
      if (d.M) {
        const f32x4 w = *reinterpret_cast<const f32x4*>(mp);
#pragma unroll
        for (int k = 0; k < 4; ++k) m1[u][k] = w[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j + k < q) {
          x[u][k] = load_g<GT>(d.G, o + k * gj);
          if (d.M) m1[u][k] = mp[k * mj];
        }
    }
  }
#pragma unroll
  for (int u = 0; u < NG; ++u)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (d.M) {
        m1[u][k] = ns_moment(L.common, x[u][k], m1[u][k]);
        x[u][k] = ns_dir(L.common, x[u][k], m1[u][k]);
      }
      sum += static_cast<double>(x[u][k]) * x[u][k];
    }
  sum = wave_sum(sum);
  double* part = reinterpret_cast<double*>(ab);
  if ((threadIdx.x & 63) == 0) part[wave] = sum;
  __syncthreads();
  sum = 0.0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) sum += part[w];
  const double norm = sqrt(sum);
  const bool finite = norm < 1.7e308;   // false for NaN too
  if (threadIdx.x == 0) L.common.status[d.slot] = finite ? 0 : kNsNonFinite;
  if (!finite) return;
  int e2 = 0;
  const double f = norm > 0.0 ? frexp(norm, &e2) : 0.0;
  const float tau = f > 0.0 ? static_cast<float>(1.0 / f) : 0.0f;

  // X planes, zero past p and q
  for (int i = threadIdx.x; i < 2 * T::XCELLS; i += 64 * kWaves) smem[i] = u32x4{0, 0, 0, 0};
  __syncthreads();
#pragma unroll
  for (int u = 0; u < NG; ++u) {
    int i, j;
    if (!group(u, i, j)) continue;
    // the step's momentum, now that D is known to be finite
    if (d.M) {
      float* mp = d.M + (i * mi + j * mj);
      if (vec) {
        *reinterpret_cast<f32x4*>(mp) = f32x4{m1[u][0], m1[u][1], m1[u][2], m1[u][3]};
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (j + k < q) mp[k * mj] = m1[u][k];
      }
    }
    uint16_t hi[4], lo[4];   // the columns past q are zero
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float v = pinned(ldexpf(x[u][k], -e2) * L.common.x0);
      hi[k] = to_f16(v);
      lo[k] = to_f16(v - f16_to_f32(hi[k]));
    }
    const int at = 2 * x_cell<QP>(i, j >> 3) + ((j >> 2) & 1);
    reinterpret_cast<u32x2*>(xh)[at] = u32x2{hi[0] | (static_cast<uint32_t>(hi[1]) << 16), hi[2] | (static_cast<uint32_t>(hi[3]) << 16)};
    reinterpret_cast<u32x2*>(xl)[at] = u32x2{lo[0] | (static_cast<uint32_t>(lo[1]) << 16), lo[2] | (static_cast<uint32_t>(lo[3]) << 16)};
  }
  __syncthreads();

  const int r0 = 16 * FM * (wave >> 1), c0 = 16 * FN * (wave & 1);   // this wavefront's block of A
  const int col0 = 16 * FC * wave;                                    // and its columns of X
  const int qsteps = (q + 31) / 32;
  f32x4 y[FC][T::NB];   // (B X)^T on those columns
  float fy = 0.0f;
  for (int it = 0; it < L.steps; ++it) {
    // a lane number that is new in every iteration: the hundreds of LDS and
    // output addresses made from it would otherwise be computed once, before
    // the loop, and spilled (the 64 x 512 and 128 x 256 forms still spill six to
    // ten registers)
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const NsSmall::Iter s = L.it[it];
    const bool last = it == L.steps - 1;
    // A = X X^T
    f32x4 a[FM][FN];
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int n = 0; n < FN; ++n) a[m][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int ks = 0; ks < qsteps; ++ks) {
      f16x8 ah[FM], al[FM], bh[FN], bl[FN];
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        ah[m] = T::x_row(xh, r0 + 16 * m, ks, lane);
        al[m] = T::x_row(xl, r0 + 16 * m, ks, lane);
      }
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        bh[n] = T::x_row(xh, c0 + 16 * n, ks, lane);
        bl[n] = T::x_row(xl, c0 + 16 * n, ks, lane);
      }
#pragma unroll
      for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int n = 0; n < FN; ++n) {
          a[m][n] = F16::mfma(al[m], bh[n], a[m][n]);
          a[m][n] = F16::mfma(ah[m], bl[n], a[m][n]);
          a[m][n] = F16::mfma(ah[m], bh[n], a[m][n]);
        }
    }
    const float t1 = it == 0 ? tau : 1.0f;
    const float fg = s.f_gram * t1 * t1;
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int v = 0; v < 4; ++v) a[m][n][v] = pinned(fg * a[m][n][v]);
    // B = f_i I + f_a A + f_acc A A^T
    if (s.f_acc != 0.0f) {
      f32x4 b[FM][FN];
#pragma unroll
      for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int n = 0; n < FN; ++n) b[m][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      T::a_store(ab, a, false, lane);
      __syncthreads();
      f16x8 ah[KS][FM], bh[KS][FN];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
        for (int m = 0; m < FM; ++m) ah[ks][m] = T::a_row(ab, r0 + 16 * m, ks, lane);
#pragma unroll
        for (int n = 0; n < FN; ++n) bh[ks][n] = T::a_row(ab, c0 + 16 * n, ks, lane);
#pragma unroll
        for (int m = 0; m < FM; ++m)
#pragma unroll
          for (int n = 0; n < FN; ++n) b[m][n] = F16::mfma(ah[ks][m], bh[ks][n], b[m][n]);
      }
      __syncthreads();
      T::a_store(ab, a, true, lane);
      __syncthreads();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        f16x8 al[FM], bl[FN];
#pragma unroll
        for (int m = 0; m < FM; ++m) al[m] = T::a_row(ab, r0 + 16 * m, ks, lane);
#pragma unroll
        for (int n = 0; n < FN; ++n) bl[n] = T::a_row(ab, c0 + 16 * n, ks, lane);
#pragma unroll
        for (int m = 0; m < FM; ++m)
#pragma unroll
          for (int n = 0; n < FN; ++n) {
            b[m][n] = F16::mfma(al[m], bh[ks][n], b[m][n]);
            b[m][n] = F16::mfma(ah[ks][m], bl[n], b[m][n]);
          }
        __builtin_amdgcn_sched_barrier(0);
      }
      __syncthreads();
#pragma unroll
      for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int n = 0; n < FN; ++n)
#pragma unroll
          for (int v = 0; v < 4; ++v) a[m][n][v] = fmaf(s.f_acc, b[m][n][v], s.f_a * a[m][n][v]);
    } else {
#pragma unroll
      for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int n = 0; n < FN; ++n)
#pragma unroll
          for (int v = 0; v < 4; ++v) a[m][n][v] = s.f_a * a[m][n][v];
    }
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int row = r0 + 16 * m + 4 * (lane >> 4) + v;
          if (row == c0 + 16 * n + (lane & 15) && row < p) a[m][n][v] += s.f_i;
          a[m][n][v] = pinned(a[m][n][v]);
        }
    // X <- B X on this wavefront's columns, as (X^T B)^T: a lane then holds 4
    // consecutive columns of one row
    T::a_store(ab, a, false, lane);
    f16x8 yh[KS][FC], yl[KS][FC];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int n = 0; n < FC; ++n) {
        yh[ks][n] = T::x_col(xh, col0 + 16 * n, ks, lane);
        yl[ks][n] = T::x_col(xl, col0 + 16 * n, ks, lane);
      }
#pragma unroll
    for (int n = 0; n < FC; ++n)
#pragma unroll
      for (int m = 0; m < T::NB; ++m) y[n][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    __syncthreads();
#pragma unroll
    for (int m = 0; m < T::NB; ++m)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const f16x8 b = T::a_row(ab, 16 * m, ks, lane);
#pragma unroll
        for (int n = 0; n < FC; ++n) {
          y[n][m] = F16::mfma(yl[ks][n], b, y[n][m]);
          y[n][m] = F16::mfma(yh[ks][n], b, y[n][m]);
        }
        if (ks == KS - 1) __builtin_amdgcn_sched_barrier(0);   // no hoarding of operands in registers
      }
    __syncthreads();
    T::a_store(ab, a, true, lane);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < T::NB; ++m)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const f16x8 b = T::a_row(ab, 16 * m, ks, lane);
#pragma unroll
        for (int n = 0; n < FC; ++n) y[n][m] = F16::mfma(yh[ks][n], b, y[n][m]);
        if (ks == KS - 1) __builtin_amdgcn_sched_barrier(0);
      }
    fy = s.f_apply * t1;
    if (!last) {
#pragma unroll
      for (int n = 0; n < FC; ++n)
#pragma unroll
        for (int m = 0; m < T::NB; ++m) {
          const int row = 16 * m + (lane & 15), j = col0 + 16 * n + 4 * (lane >> 4);
          uint16_t hi[4], lo[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float x = pinned(fy * y[n][m][v]);
            hi[v] = to_f16(x);
            lo[v] = to_f16(x - f16_to_f32(hi[v]));
          }
          const int at = 2 * x_cell<QP>(row, j >> 3) + ((j >> 2) & 1);
          reinterpret_cast<u32x2*>(xh)[at] = u32x2{hi[0] | (static_cast<uint32_t>(hi[1]) << 16), hi[2] | (static_cast<uint32_t>(hi[3]) << 16)};
          reinterpret_cast<u32x2*>(xl)[at] = u32x2{lo[0] | (static_cast<uint32_t>(lo[1]) << 16), lo[2] | (static_cast<uint32_t>(lo[3]) << 16)};
        }
      __syncthreads();
    }
  }
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  // the old weights of a step are loaded before the first new one is
  // stored: a load cannot be moved over a store that may alias it
  const int es = L.common.odtype ? 2 : 4;
  const bool ovec = !tall && d.ldo % 4 == 0 && (reinterpret_cast<uint64_t>(d.O) & (4 * es - 1)) == 0;
  const int64_t oi = tall ? 1 : d.ldo, oj = tall ? d.ldo : 1;
  float* w32 = static_cast<float*>(d.O);
  uint16_t* w16 = static_cast<uint16_t*>(d.O);
#pragma unroll
  for (int n = 0; n < FC; ++n) {
    const int j = col0 + 16 * n + 4 * (lane >> 4);
    if (j >= q) continue;
    const bool four = ovec && j + 4 <= q;
    if (L.step) {
      float w[T::NB][4];
#pragma unroll
      for (int m = 0; m < T::NB; ++m) {
        const int i = 16 * m + (lane & 15);
        if (i >= p) continue;
        if (four) {
          const f32x4 v = *reinterpret_cast<const f32x4*>(w32 + i * oi + j);
#pragma unroll
          for (int k = 0; k < 4; ++k) w[m][k] = v[k];
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) w[m][k] = j + k < q ? w32[i * oi + (j + k) * oj] : 0.0f;
        }
      }
#pragma unroll
      for (int m = 0; m < T::NB; ++m)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          y[n][m][k] = fmaf(-d.scale, fy * y[n][m][k], L.common.decay * w[m][k]);
    } else {
#pragma unroll
      for (int m = 0; m < T::NB; ++m)
#pragma unroll
        for (int k = 0; k < 4; ++k) y[n][m][k] = fy * y[n][m][k];
    }
#pragma unroll
    for (int m = 0; m < T::NB; ++m) {
      const int i = 16 * m + (lane & 15);
      if (i >= p) continue;
      const f32x4 v = y[n][m];
      const int64_t o = i * oi + j * oj;
      if (L.common.odtype) {
        const uint16_t h[4] = {to_bf16(v[0]), to_bf16(v[1]), to_bf16(v[2]), to_bf16(v[3])};
        if (four) {
          *reinterpret_cast<u32x2*>(w16 + o) = u32x2{h[0] | (static_cast<uint32_t>(h[1]) << 16), h[2] | (static_cast<uint32_t>(h[3]) << 16)};
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (j + k < q) w16[o + k * oj] = h[k];
        }
      } else if (four) {
        *reinterpret_cast<f32x4*>(w32 + o) = v;
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (j + k < q) w32[o + k * oj] = v[k];
      }
    }
  }
}

template <typename GT>
hipError_t small(const NsSmall& L, int pp, int qp, hipStream_t st) {
  const dim3 grid(L.common.total), block(64 * kWaves);
  if (pp == 64 && qp == 128) k_ns_small<GT, 64, 128><<<grid, block, 0, st>>>(L);
  else if (pp == 64 && qp == 256) k_ns_small<GT, 64, 256><<<grid, block, 0, st>>>(L);
  else if (pp == 64 && qp == 512) k_ns_small<GT, 64, 512><<<grid, block, 0, st>>>(L);
  else if (pp == 128 && qp == 128) k_ns_small<GT, 128, 128><<<grid, block, 0, st>>>(L);
  else if (pp == 128 && qp == 256) k_ns_small<GT, 128, 256><<<grid, block, 0, st>>>(L);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ns_small(const NsSmall& L, int pp, int qp, hipStream_t st) {
  return L.common.gdtype ? small<uint16_t>(L, pp, qp, st) : small<float>(L, pp, qp, st);
}

}  // namespace dion
