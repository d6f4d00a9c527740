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
#include "mm16.h"
#include "ns_types.h"

namespace dion {

namespace {

__device__ __forceinline__ void ns_locate(const NsLaunch& L, int t, NsDesc& d, NsClass& c, int& local) {
  c = L.cls[0];
#pragma unroll
  for (int i = 1; i < kNsMaxClasses; ++i)
    if (i < L.nclass && t >= L.cls[i].base) c = L.cls[i];
  const int rel = t - c.base;
  const int mi = rel / c.tiles;
  local = rel - mi * c.tiles;
  d = L.table ? L.table[c.first + mi] : L.inl;
}

__global__ __launch_bounds__(256) void k_ns_table(NsUpload u) {
  const int words = u.count * static_cast<int>(sizeof(NsDesc) / 4);
  const uint32_t* src = reinterpret_cast<const uint32_t*>(u.d);
  uint32_t* dst = reinterpret_cast<uint32_t*>(u.dst);
  for (int i = threadIdx.x; i < words; i += 256) dst[i] = src[i];
}

template <typename GT>
__device__ __forceinline__ float load_g(const void* G, int64_t o) {
  if constexpr (sizeof(GT) == 2) return bf16_to_f32(static_cast<const uint16_t*>(G)[o]);
  else return static_cast<const float*>(G)[o];
}

// The new momentum and the matrix to orthogonalize, each one rounding per
// operation, the same in both kernels that form them.
__device__ __forceinline__ float ns_moment(const NsLaunch& L, float g, float m) { return fmaf(L.mu, m, g); }
__device__ __forceinline__ float ns_dir(const NsLaunch& L, float g, float m1) {
  return L.nesterov ? fmaf(L.mu, m1, g) : m1;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
  return v;
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

// Eight values as planes.
template <int PL>
__device__ __forceinline__ void store_planes(uint16_t* at, int64_t plane, const float (&v)[8]) {
  uint16_t hi[8], lo[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float x = PL == 2 ? pinned(v[k]) : v[k];
    hi[k] = to_f16(x);
    if constexpr (PL == 2) lo[k] = to_f16(x - f16_to_f32(hi[k]));
  }
  *reinterpret_cast<u32x4*>(at) = pack8(hi);
  if constexpr (PL == 2) *reinterpret_cast<u32x4*>(at + plane) = pack8(lo);
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
  double sum = 0.0;
  const double* parts = reinterpret_cast<const double*>(L.ws + d.oS);
  for (int i = threadIdx.x; i < d.parts; i += 256) sum += parts[i];
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  sum = (part[0] + part[1]) + (part[2] + part[3]);
  const double norm = sqrt(sum);
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
  const int64_t pitch = ns_pad(d.q), plane = ns_pad(d.p) * pitch;
  uint16_t* X = reinterpret_cast<uint16_t*>(L.ws + d.oX);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int i = 32 * s + (threadIdx.x >> 3), j = 8 * (threadIdx.x & 7);
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = d.tall ? tile[j + k][i] : tile[i][j + k];
    store_planes<PL>(X + (i0 + i) * pitch + j0 + j, plane, v);
  }
}

// Upper-triangle tiles of an nt x nt grid in groups of 4 tile rows: group g
// holds columns 4 g .. nt - 1, four rows each, walked down the rows first,
// so that concurrent tiles share row and column panels.  The few items of a
// group that fall below the diagonal return at once.
constexpr int kSymRows = 4;
__device__ __forceinline__ bool sym_tile(int t, int nt, int& ti, int& tj) {
  int first = 0;
  while (t >= kSymRows * (nt - first)) {
    t -= kSymRows * (nt - first);
    first += kSymRows;
  }
  ti = first + t % kSymRows;
  tj = first + t / kSymRows;
  return ti <= tj && ti < nt;
}

template <int PL>
__device__ __forceinline__ void load_planes(const uint16_t* at, int64_t plane, float (&v)[8]) {
  const f16x8 hi = __builtin_bit_cast(f16x8, *reinterpret_cast<const u32x4*>(at));
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = static_cast<float>(hi[k]);
  if constexpr (PL == 2) {
    const f16x8 lo = __builtin_bit_cast(f16x8, *reinterpret_cast<const u32x4*>(at + plane));
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += static_cast<float>(lo[k]);
  }
}

template <int PL, int TILE, bool BMC>
using NsShape = Shape16<F16, TILE, TILE, PL == 2 ? 32 : 64, 2, TILE / 64, PL, false, BMC>;

// One tile of one of the three products.  Products that are symmetric
// compute the tiles on and above the diagonal and write each one's
// transpose too.
template <int PL, int TILE, NsEpi EPI>
__global__ __launch_bounds__(64 * 2 * TILE / 64) void k_ns_mm(NsLaunch L) {
  constexpr bool SYM = EPI == kNsGram || EPI == kNsGramPoly || EPI == kNsPoly;
  using S = NsShape<PL, TILE, !SYM>;
  __shared__ u32x4 smem[S::LDS_CELLS];
  NsDesc d;
  NsClass c;
  int local;
  ns_locate(L, xcd_remap(blockIdx.x, gridDim.x), d, c, local);
  int ti, tj;
  if constexpr (SYM) {
    if (!sym_tile(local, c.tx, ti, tj)) return;
  } else {
    tile_order(local, c.tx, c.ty, ti, tj);
  }
  if (L.status[d.slot] & kNsNonFinite) return;

  const int pp = static_cast<int>(ns_pad(d.p)), qp = static_cast<int>(ns_pad(d.q));
  const int64_t planeX = static_cast<int64_t>(pp) * qp, planeA = static_cast<int64_t>(pp) * pp;
  uint16_t* X = reinterpret_cast<uint16_t*>(L.ws + d.oX) + L.src * PL * planeX;
  uint16_t* A = reinterpret_cast<uint16_t*>(L.ws + d.oA);
  uint16_t* B = reinterpret_cast<uint16_t*>(L.ws + d.oB);
  const int r0 = ti * TILE, c0 = tj * TILE;

  f32x16 acc[S::FM][S::FN];
  typename S::A ta;
  typename S::B tb;
  auto one = [](int, int& a, int& b) { a = b = 0; };
  if constexpr (EPI == kNsGram || EPI == kNsGramPoly) {
    ta.init(qp, r0, pp);
    tb.init(qp, c0, pp);
    tile_product<S>(ta, tb, Planes16{X, X, planeX, planeX}, 1, one, 0, qp, smem, acc);
  } else if constexpr (EPI == kNsPoly) {
    ta.init(pp, r0, pp);
    tb.init(pp, c0, pp);
    tile_product<S>(ta, tb, Planes16{A, A, planeA, planeA}, 1, one, 0, pp, smem, acc);
  } else {
    ta.init(pp, r0, pp);
    tb.init(qp, c0, qp);
    tile_product<S>(ta, tb, Planes16{B, X, planeA, planeX}, 1, one, 0, pp, smem, acc);
  }

  float f = L.f_acc;
  if (L.tau) {
    const float tau = *reinterpret_cast<const float*>(L.ws + d.oS + kNsParts * 8);
    f *= L.tau == 2 ? tau * tau : tau;
  }
  if constexpr (SYM) {
    uint16_t* dst = EPI == kNsGram ? A : B;
    auto put = [&](int row, int col, const float (&v)[8]) {
      if (row >= pp || col >= pp) return;
      const int64_t o = static_cast<int64_t>(row) * pp + col;
      float w[8];
      if constexpr (EPI == kNsPoly) {
        load_planes<PL>(A + o, planeA, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = fmaf(f, v[k], L.f_a * w[k]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = f * v[k];
      }
      if constexpr (EPI != kNsGram) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (row == col + k && row < d.p) w[k] += L.f_i;
      }
      store_planes<PL>(dst + o, planeA, w);
    };
    tile_rows<S>(acc, smem, [&](int r, int q, const float (&v)[8]) { put(r0 + r, c0 + q, v); });
    if (ti != tj) tile_cols<S>(acc, smem, [&](int r, int q, const float (&v)[8]) { put(c0 + r, r0 + q, v); });
  } else if constexpr (EPI == kNsApply) {
    uint16_t* next = reinterpret_cast<uint16_t*>(L.ws + d.oX) + (1 - L.src) * PL * planeX;
    tile_rows<S>(acc, smem, [&](int r, int q, const float (&v)[8]) {
      const int row = r0 + r, col = c0 + q;
      if (row >= pp || col >= qp) return;
      float w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = f * v[k];
      store_planes<PL>(next + static_cast<int64_t>(row) * qp + col, planeX, w);
    });
  } else {
    const int rows = d.tall ? d.q : d.p, cols = d.tall ? d.p : d.q;
    const bool vec = (reinterpret_cast<uint64_t>(d.O) & 15) == 0 && d.ldo % (L.odtype ? 8 : 4) == 0;
    auto put = [&](int row, int col, const float (&v)[8]) {
      if (row >= rows || col >= cols) return;
      const int64_t o = row * d.ldo + col;
      const int left = cols - col;
      if constexpr (EPI == kNsStep) {
        float* x = static_cast<float*>(d.O) + o;
        const float step = d.scale * f;
        if (vec && left >= 8) {
          f32x4 a = *reinterpret_cast<f32x4*>(x), b = *reinterpret_cast<f32x4*>(x + 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            a[k] = fmaf(-step, v[k], L.decay * a[k]);
            b[k] = fmaf(-step, v[4 + k], L.decay * b[k]);
          }
          *reinterpret_cast<f32x4*>(x) = a;
          *reinterpret_cast<f32x4*>(x + 4) = b;
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < left) x[k] = fmaf(-step, v[k], L.decay * x[k]);
        }
      } else if (L.odtype) {
        uint16_t* x = static_cast<uint16_t*>(d.O) + o;
        uint16_t h[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) h[k] = to_bf16(f * v[k]);
        if (vec && left >= 8) {
          *reinterpret_cast<u32x4*>(x) = pack8(h);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < left) x[k] = h[k];
        }
      } else {
        float* x = static_cast<float*>(d.O) + o;
        if (vec && left >= 8) {
          *reinterpret_cast<f32x4*>(x) = f32x4{f * v[0], f * v[1], f * v[2], f * v[3]};
          *reinterpret_cast<f32x4*>(x + 4) = f32x4{f * v[4], f * v[5], f * v[6], f * v[7]};
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < left) x[k] = f * v[k];
        }
      }
    };
    if (d.tall) tile_cols<S>(acc, smem, [&](int r, int q, const float (&v)[8]) { put(c0 + r, r0 + q, v); });
    else tile_rows<S>(acc, smem, [&](int r, int q, const float (&v)[8]) { put(r0 + r, c0 + q, v); });
  }
}

template <int PL, int TILE>
hipError_t product(const NsLaunch& L, NsEpi epi, hipStream_t st) {
  const dim3 grid(L.total), block(64 * 2 * TILE / 64);
  switch (epi) {
    case kNsGram: k_ns_mm<PL, TILE, kNsGram><<<grid, block, 0, st>>>(L); break;
    case kNsGramPoly: k_ns_mm<PL, TILE, kNsGramPoly><<<grid, block, 0, st>>>(L); break;
    case kNsPoly: k_ns_mm<PL, TILE, kNsPoly><<<grid, block, 0, st>>>(L); break;
    case kNsApply: k_ns_mm<PL, TILE, kNsApply><<<grid, block, 0, st>>>(L); break;
    case kNsOut: k_ns_mm<PL, TILE, kNsOut><<<grid, block, 0, st>>>(L); break;
    case kNsStep: k_ns_mm<PL, TILE, kNsStep><<<grid, block, 0, st>>>(L); break;
  }
  return hipGetLastError();
}

}  // namespace

int ns_sym_items(int nt) {
  int items = 0;
  for (int first = 0; first < nt; first += kSymRows) items += kSymRows * (nt - first);
  return items;
}

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

hipError_t launch_ns_product(const NsLaunch& L, NsEpi epi, int planes, int tile, hipStream_t st) {
  if (planes == 2) return tile == 256 ? product<2, 256>(L, epi, st) : product<2, 128>(L, epi, st);
  return tile == 256 ? product<1, 256>(L, epi, st) : product<1, 128>(L, epi, st);
}

}  // namespace dion
