// Newton-Schulz orthogonalization on the 16-bit matrix cores: the kernels
// behind dion_orthogonalize and dion_muon_step.
//
//   X <- D / ||D||_F, then per iteration  X <- (a I + b A + c A^2) X,
//   A = X X^T, on the smaller side of the matrix (p <= q):
//
//   k_ns_norm   partial sums of squares of D (float64)
//   k_ns_load   momentum update, X planes (transposed when tall)
//   k_ns_mm     A = X X^T;  B = a I + b A + c A A^T;  X <- B X
//
// The planes are float16 with power-of-two scales, not bfloat16: the
// singular values stay bounded by the polynomial, so the range is known in
// advance, and float16's 11 bits leave an error of about 1.2e-3 in the
// result of five quintic iterations where bfloat16's 8 bits leave 1.1e-2
// (N(0, 1) matrices), at the same matrix rate.  Two planes (hi + lo, 22
// bits) give float32's accuracy at a third of the rate.
//
// Bound and measured (MI355X): large matrices by the matrix cores at the
// clock the power limit leaves (8192 x 28672, float16, five quintic
// iterations: 27.7 ms, 1.14 PFLOP/s of algorithmic work; one layer of the 3B
// stack, float32: 15.4 ms, 1.01 PFLOP/s of matrix-core products); 768-row
// stacks by each tile's prologue and epilogue (six layers, float16: 0.98 to 1.05 ms);
// a few matrices by launch latency (five of about 1500 x 500: 0.26 ms in 18
// launches).
#include "mm16.h"
#include "ns_device.h"
#include "ns_types.h"
#include "work16.h"

namespace dion {

namespace {

__global__ __launch_bounds__(256) void k_ns_table(NsUpload u) {
  const int words = u.count * static_cast<int>(sizeof(NsDesc) / 4);
  const uint32_t* src = reinterpret_cast<const uint32_t*>(u.d);
  uint32_t* dst = reinterpret_cast<uint32_t*>(u.dst);
  for (int i = threadIdx.x; i < words; i += 256) dst[i] = src[i];
}

// Partial sums of squares of D over `chunk` elements each, in float64 (a
// float32 gradient's squares leave float32's range).  Read-only: a matrix
// whose norm turns out not finite keeps its momentum.
template <typename GT>
__global__ __launch_bounds__(256) void k_ns_norm(NsLaunch L) {
  __shared__ double part[4];
  NsDesc d;
  NsClass c;
  int local;
  ns_locate(L, blockIdx.x, d, c, local);
  if (local == 0 && threadIdx.x == 0) L.status[d.slot] = 0;
  if (blockIdx.x == 0 && L.count)
    for (int i = threadIdx.x; i < kNsCounts; i += 256) L.count[i] = 0;
  const int n = d.tall ? d.p : d.q;   // columns as the caller stores them
  const int64_t total = static_cast<int64_t>(d.p) * d.q;
  const int64_t beg = local * d.chunk;
  const int64_t end = min(total, beg + d.chunk);
  double sum = 0.0;
  auto add = [&](float g, float m) {
    const float v = d.M ? ns_dir(L, g, ns_moment(L, g, m)) : g;
    sum += static_cast<double>(v) * v;
  };
  if (d.ldg == n && n % 4 == 0 && (reinterpret_cast<uint64_t>(d.G) & (4 * sizeof(GT) - 1)) == 0 &&
      (reinterpret_cast<uint64_t>(d.M) & 15) == 0) {
    for (int64_t e = beg + 4 * threadIdx.x; e < end; e += 1024) {
      float g[4];
      if constexpr (sizeof(GT) == 2) {
        const u32x2 u = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(d.G) + e);
        g[0] = __uint_as_float(u.x << 16);
        g[1] = __uint_as_float(u.x & 0xffff0000u);
        g[2] = __uint_as_float(u.y << 16);
        g[3] = __uint_as_float(u.y & 0xffff0000u);
      } else {
        const f32x4 u = *reinterpret_cast<const f32x4*>(static_cast<const float*>(d.G) + e);
        for (int i = 0; i < 4; ++i) g[i] = u[i];
      }
      f32x4 m = {0.0f, 0.0f, 0.0f, 0.0f};
      if (d.M) m = *reinterpret_cast<const f32x4*>(d.M + e);
#pragma unroll
      for (int i = 0; i < 4; ++i) add(g[i], m[i]);
    }
  } else {
    for (int64_t e = beg + threadIdx.x; e < end; e += 256) {
      const int64_t r = e / n, j = e - r * n;
      add(load_g<GT>(d.G, r * d.ldg + j), d.M ? d.M[e] : 0.0f);
    }
  }
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0)
    reinterpret_cast<double*>(L.ws + d.oS)[local] = (part[0] + part[1]) + (part[2] + part[3]);
}

// Where the eight values from (row, col), col a multiple of 8, of a matrix
// of `pitch` columns sit: their hi parts, and kLoOffset further their lo.
constexpr int kLoOffset = 16;
template <int PL>
__device__ __forceinline__ int64_t plane_at(int64_t row, int col, int64_t pitch) {
  return PL == 2 ? row * 2 * pitch + (col >> 4) * 32 + (col & 15) : row * pitch + col;
}
template <int PL>
__device__ __forceinline__ void store_planes(uint16_t* at, const float (&v)[8]) {
  uint16_t hi[8], lo[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float x = PL == 2 ? pinned(v[k]) : v[k];
    hi[k] = to_f16(x);
    if constexpr (PL == 2) lo[k] = to_f16(x - f16_to_f32(hi[k]));
  }
  *reinterpret_cast<u32x4*>(at) = pack8(hi);
  if constexpr (PL == 2) *reinterpret_cast<u32x4*>(at + kLoOffset) = pack8(lo);
}

// X = D 2^-e as planes (times the planes' scale), 2^-e the power of two that
// brings ||D|| into [0.5, 1): exact for a bfloat16 D, so the rest of the normalization, tau
// in (1, 2], goes into the first iteration's products.  One 64 x 64 tile of
// the planes per workgroup; the step's momentum is updated on the way.
template <typename GT, int PL>
__global__ __launch_bounds__(256) void k_ns_load(NsLaunch L) {
  __shared__ float tile[64][65];
  __shared__ double part[4];
  NsDesc d;
  NsClass c;
  int local;
  ns_locate(L, blockIdx.x, d, c, local);
  const double norm = ns_norm<4>(L, d, part);
  const bool finite = norm < 1.7e308;   // false for NaN too
  if (local == 0 && threadIdx.x == 0) {
    if (!finite) L.status[d.slot] = kNsNonFinite;
  }
  if (!finite) return;
  int e = 0;
  const double f = norm > 0.0 ? frexp(norm, &e) : 0.0;   // norm = f 2^e, f in [0.5, 1)
  if (local == 0 && threadIdx.x == 0)
    *reinterpret_cast<float*>(L.ws + d.oS + kNsParts * 8) = f > 0.0 ? static_cast<float>(1.0 / f) : 0.0f;

  const int ti = local / c.ty, tj = local % c.ty;
  const int i0 = 64 * ti, j0 = 64 * tj;   // planes' coordinates
  const int rows = d.tall ? d.q : d.p, cols = d.tall ? d.p : d.q;   // the caller's
  const int r0 = d.tall ? j0 : i0, c0 = d.tall ? i0 : j0;
#pragma unroll 4
  for (int s = 0; s < 16; ++s) {
    const int r = r0 + 4 * s + (threadIdx.x >> 6), col = c0 + (threadIdx.x & 63);
    float v = 0.0f;
    if (r < rows && col < cols) {
      v = load_g<GT>(d.G, r * d.ldg + col);
      if (d.M) {
        const int64_t o = static_cast<int64_t>(r) * cols + col;
        const float m1 = ns_moment(L, v, d.M[o]);
        d.M[o] = m1;
        v = ns_dir(L, v, m1);
      }
      v = ldexpf(v, -e) * L.x0;
    }
    tile[4 * s + (threadIdx.x >> 6)][threadIdx.x & 63] = v;
  }
  __syncthreads();
  const int64_t pitch = ns_pitch(d.q, PL);
  uint16_t* X = reinterpret_cast<uint16_t*>(L.ws + d.oX);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int i = 32 * s + (threadIdx.x >> 3), j = 8 * (threadIdx.x & 7);
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = d.tall ? tile[j + k][i] : tile[i][j + k];
    store_planes<PL>(X + plane_at<PL>(i0 + i, j0 + j, pitch), v);
  }
}

// Upper-triangle tiles of an nt x nt grid in groups of 4 tile rows, each
// walked down its rows first, so that concurrent tiles share row and column
// panels: a group starting at row f has the triangle of its first 4 columns,
// then whole columns of 4.
constexpr int kSymRows = 4;
__device__ __forceinline__ void sym_tile(int t, int nt, int& ti, int& tj) {
  constexpr int TRI = kSymRows * (kSymRows + 1) / 2;
  int first = 0;
  while (nt - first > kSymRows && t >= TRI + kSymRows * (nt - first - kSymRows)) {
    t -= TRI + kSymRows * (nt - first - kSymRows);
    first += kSymRows;
  }
  if (t < TRI) {
    const int j = (t >= 1) + (t >= 3) + (t >= 6);
    ti = first + t - j * (j + 1) / 2;
    tj = first + j;
  } else {
    ti = first + (t - TRI) % kSymRows;
    tj = first + kSymRows + (t - TRI) / kSymRows;
  }
}

// Eight stored values: as loaded, and as numbers.
template <int PL>
struct NsRun {
  u32x4 hi, lo;
  __device__ __forceinline__ void load(const uint16_t* at) {
    hi = *reinterpret_cast<const u32x4*>(at);
    if constexpr (PL == 2) lo = *reinterpret_cast<const u32x4*>(at + kLoOffset);
  }
  __device__ __forceinline__ float value(int k) const {
    const float h = static_cast<float>(__builtin_bit_cast(f16x8, hi)[k]);
    if constexpr (PL == 2) return h + static_cast<float>(__builtin_bit_cast(f16x8, lo)[k]);
    else return h;
  }
};

template <int PL, int TILE, int ST, bool BMC>
using NsShape = Shape16<F16, TILE, TILE, TILE / 64, 2, ST, PL, false, BMC>;

// One tile of one of the three products.  Products that are symmetric
// compute the tiles on and above the diagonal and write each one's
// transpose too.
template <int PL, int TILE, int ST, NsEpi EPI>
__global__ __launch_bounds__(2 * TILE) void k_ns_mm(NsLaunch L) {
  constexpr bool SYM = EPI == kNsGram || EPI == kNsGramPoly || EPI == kNsPoly;
  using S = NsShape<PL, TILE, ST, !SYM>;
  __shared__ u32x4 smem[S::LDS_CELLS];
  NsDesc d;
  NsClass c;
  int local;
  const Work16 work{L.full, L.total - L.full, L.slices, L.part, L.count};
  const Item16 it = item16(work, xcd_item(blockIdx.x, gridDim.x));
  ns_locate(L, it.tile, d, c, local);
  int ti, tj;
  if constexpr (SYM) {
    sym_tile(local, c.tx, ti, tj);
  } else {
    tile_order(local, c.tx, c.ty, ti, tj);
  }
  if (uniform32(L.status[d.slot]) & kNsNonFinite) return;

  ti = uniform32(ti);
  tj = uniform32(tj);
  const int pp = uniform32(static_cast<int>(ns_pad(d.p))), qp = uniform32(static_cast<int>(ns_pad(d.q)));
  const int pitchA = uniform32(static_cast<int>(ns_pitch(d.p, PL))), pitchX = uniform32(static_cast<int>(ns_pitch(d.q, PL)));
  const int64_t planeX = static_cast<int64_t>(pp) * pitchX;
  uint16_t* X = uniform_at(reinterpret_cast<uint16_t*>(L.ws + d.oX) + L.src * PL * planeX);
  uint16_t* A = uniform_at(reinterpret_cast<uint16_t*>(L.ws + d.oA));
  uint16_t* B = uniform_at(reinterpret_cast<uint16_t*>(L.ws + d.oB));
  const int r0 = ti * TILE, c0 = tj * TILE;

  typename S::Acc acc[S::FM][S::FN];
  typename S::A ta;
  typename S::B tb;
  auto one = [](int, int& a, int& b) { a = b = 0; };
  int kbeg, kend;
  slice16<S>(it, EPI == kNsGram || EPI == kNsGramPoly ? qp : pp, kbeg, kend);
  if constexpr (EPI == kNsGram || EPI == kNsGramPoly) {
    ta.init(PL * pitchX, r0, pp);
    tb.init(PL * pitchX, c0, pp);
    tile_product<S>(ta, tb, Planes16{X, X, 0, 0}, 1, one, kbeg, kend, smem, acc);
  } else if constexpr (EPI == kNsPoly) {
    ta.init(PL * pitchA, r0, pp);
    tb.init(PL * pitchA, c0, pp);
    tile_product<S>(ta, tb, Planes16{A, A, 0, 0}, 1, one, kbeg, kend, smem, acc);
  } else {
    ta.init(PL * pitchA, r0, pp);
    tb.init(PL * pitchX, c0, qp);
    tile_product<S>(ta, tb, Planes16{B, X, 0, 0}, 1, one, kbeg, kend, smem, acc);
  }

  if (!join16<S>(work, it, smem, acc)) return;

  float f = L.f_acc;
  if (L.tau) {
    const float tau = *reinterpret_cast<const float*>(L.ws + d.oS + kNsParts * 8);
    f *= L.tau == 2 ? tau * tau : tau;
  }
  auto none = [](int, int) { return NoPre{}; };
  if constexpr (SYM) {
    uint16_t* dst = EPI == kNsGram ? A : B;
    auto fetch = [&](int row, int col) {
      NsRun<PL> w{};
      if (EPI == kNsPoly && row < pp && col < pp) w.load(A + plane_at<PL>(row, col, pitchA));
      return w;
    };
    auto put = [&](int row, int col, const float (&v)[8], const NsRun<PL>& a) {
      if (row >= pp || col >= pp) return;
      float w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (EPI == kNsPoly) w[k] = fmaf(f, v[k], L.f_a * a.value(k));
        else w[k] = f * v[k];
        if constexpr (EPI != kNsGram) {
          if (row == col + k && row < d.p) w[k] += L.f_i;
        }
      }
      store_planes<PL>(dst + plane_at<PL>(row, col, pitchA), w);
    };
    tile_runs<S, false>(acc, smem, [&](int r, int q) { return fetch(r0 + r, c0 + q); },
                        [&](int r, int q, const float (&v)[8], const NsRun<PL>& a) { put(r0 + r, c0 + q, v, a); });
    if (ti != tj)
      tile_runs<S, true>(acc, smem, [&](int r, int q) { return fetch(c0 + r, r0 + q); },
                         [&](int r, int q, const float (&v)[8], const NsRun<PL>& a) { put(c0 + r, r0 + q, v, a); });
  } else if constexpr (EPI == kNsApply) {
    uint16_t* next = reinterpret_cast<uint16_t*>(L.ws + d.oX) + (1 - L.src) * PL * planeX;
    tile_runs<S, false>(acc, smem, none, [&](int r, int q, const float (&v)[8], NoPre) {
      const int row = r0 + r, col = c0 + q;
      if (row >= pp || col >= qp) return;
      float w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = f * v[k];
      store_planes<PL>(next + plane_at<PL>(row, col, pitchX), w);
    });
  } else {
    const int rows = d.tall ? d.q : d.p, cols = d.tall ? d.p : d.q;
    const bool vec = (reinterpret_cast<uint64_t>(d.O) & 15) == 0 && d.ldo % (L.odtype ? 8 : 4) == 0;
    auto fetch = [&](int row, int col) {
      f32x8 x{};
      if constexpr (EPI == kNsStep) {
        const float* at = static_cast<const float*>(d.O) + row * d.ldo + col;
        if (row < rows && vec && col + 8 <= cols) {
          const f32x4 a = *reinterpret_cast<const f32x4*>(at), b = *reinterpret_cast<const f32x4*>(at + 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[k] = a[k];
            x[4 + k] = b[k];
          }
        } else if (row < rows) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (col + k < cols) x[k] = at[k];
        }
      }
      return x;
    };
    const float step = d.scale * f;
    auto put = [&](int row, int col, const float (&v)[8], const f32x8& x) {
      if (row >= rows || col >= cols) return;
      const int64_t o = row * d.ldo + col;
      const int left = cols - col;
      float w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = EPI == kNsStep ? fmaf(-step, v[k], L.decay * x[k]) : f * v[k];
      if (EPI == kNsOut && L.odtype) {
        uint16_t* at = static_cast<uint16_t*>(d.O) + o;
        uint16_t h[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) h[k] = to_bf16(w[k]);
        if (vec && left >= 8) {
          *reinterpret_cast<u32x4*>(at) = pack8(h);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < left) at[k] = h[k];
        }
      } else {
        float* at = static_cast<float*>(d.O) + o;
        if (vec && left >= 8) {
          *reinterpret_cast<f32x4*>(at) = f32x4{w[0], w[1], w[2], w[3]};
          *reinterpret_cast<f32x4*>(at + 4) = f32x4{w[4], w[5], w[6], w[7]};
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < left) at[k] = w[k];
        }
      }
    };
    if (d.tall)
      tile_runs<S, true>(acc, smem, [&](int r, int q) { return fetch(c0 + r, r0 + q); },
                         [&](int r, int q, const float (&v)[8], const f32x8& x) { put(c0 + r, r0 + q, v, x); });
    else
      tile_runs<S, false>(acc, smem, [&](int r, int q) { return fetch(r0 + r, c0 + q); },
                          [&](int r, int q, const float (&v)[8], const f32x8& x) { put(r0 + r, c0 + q, v, x); });
  }
}

template <int PL, int TILE, int ST>
hipError_t product(const NsLaunch& L, int items, NsEpi epi, hipStream_t st) {
  const dim3 grid(items), block(2 * TILE);
  switch (epi) {
    case kNsGram: k_ns_mm<PL, TILE, ST, kNsGram><<<grid, block, 0, st>>>(L); break;
    case kNsGramPoly: k_ns_mm<PL, TILE, ST, kNsGramPoly><<<grid, block, 0, st>>>(L); break;
    case kNsPoly: k_ns_mm<PL, TILE, ST, kNsPoly><<<grid, block, 0, st>>>(L); break;
    case kNsApply: k_ns_mm<PL, TILE, ST, kNsApply><<<grid, block, 0, st>>>(L); break;
    case kNsOut: k_ns_mm<PL, TILE, ST, kNsOut><<<grid, block, 0, st>>>(L); break;
    case kNsStep: k_ns_mm<PL, TILE, ST, kNsStep><<<grid, block, 0, st>>>(L); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ns_table(const NsUpload& u, hipStream_t st) {
  k_ns_table<<<dim3(1), dim3(256), 0, st>>>(u);
  return hipGetLastError();
}

hipError_t launch_ns_norm(const NsLaunch& L, hipStream_t st) {
  const dim3 grid(L.total), block(256);
  if (L.gdtype) k_ns_norm<uint16_t><<<grid, block, 0, st>>>(L);
  else k_ns_norm<float><<<grid, block, 0, st>>>(L);
  return hipGetLastError();
}

hipError_t launch_ns_load(const NsLaunch& L, int planes, hipStream_t st) {
  const dim3 grid(L.total), block(256);
  if (planes == 2) {
    if (L.gdtype) k_ns_load<uint16_t, 2><<<grid, block, 0, st>>>(L);
    else k_ns_load<float, 2><<<grid, block, 0, st>>>(L);
  } else {
    if (L.gdtype) k_ns_load<uint16_t, 1><<<grid, block, 0, st>>>(L);
    else k_ns_load<float, 1><<<grid, block, 0, st>>>(L);
  }
  return hipGetLastError();
}

hipError_t launch_ns_product(const NsLaunch& L, int items, NsEpi epi, int planes, int tile, hipStream_t st) {
  if (tile == 256) return planes == 2 ? product<2, 256, 4>(L, items, epi, st) : product<1, 256, 4>(L, items, epi, st);
  if (items <= kTileSlots256) return planes == 2 ? product<2, 128, 8>(L, items, epi, st) : product<1, 128, 8>(L, items, epi, st);
  return planes == 2 ? product<2, 128, 4>(L, items, epi, st) : product<1, 128, 4>(L, items, epi, st);
}

}  // namespace dion
