// The orthogonalization (or Muon step) of a matrix with at most 16 rows or
// columns in one workgroup, in plain float32 arithmetic.
//
// X (p x q) stays in LDS as float32.  A matrix with so few singular values
// does not average its roundings: hi + lo planes of 22 bits left such results
// up to ten times further from the exact ones than float32, and the matrix
// cores would be fed with padding anyway.  A = X X^T is taken in blocks of
// 2 x 2 or 4 x 4 rows, the columns dealt to a block's threads, which sets its
// time (LDS reads: 2 per S multiply-adds of an S x S block; 16 x 2048, five
// quintic iterations: 253 us with a pair of rows per thread, 123 us in 4 x 4
// blocks; 4 x 3000: 32 us; 8 x 8: 22 us); B X takes a thread per column.
#include "dion.h"
#include "mm16.h"
#include "ns_types.h"
#include "ns_device.h"

namespace dion {

namespace {

constexpr int kTinyThreads = 1024;

template <typename GT, int P>
__global__ __launch_bounds__(kTinyThreads) void k_ns_tiny(NsSmall L) {
  constexpr int S = P == 16 ? 4 : P == 1 ? 1 : 2, SIDE = P / S;   // A in SIDE x SIDE blocks of S x S
  constexpr int T = kTinyThreads / (SIDE * SIDE), PARTS = T / 64;   // threads per block, wavefronts
  __shared__ float X[kNsTinyFloats + 16];
  __shared__ float A[P][P + 1], B[P][P + 1], part[kTinyThreads / 64][S * S];
  __shared__ double dpart[kTinyThreads / 64];
  NsDesc d;
  NsClass c;
  int local;
  ns_locate(L.common, blockIdx.x, d, c, local);
  const int p = uniform32(d.p), q = uniform32(d.q), tall = uniform32(d.tall);
  const int pitch = q | 1;   // odd: rows start on different banks
  const int total = p * q;
  // element e in the caller's order (rows of q when wide, of p when tall)
  auto row_col = [&](int e, int& i, int& j, int64_t& g) {
    if (tall) {
      j = e / p;
      i = e - j * p;
      g = j * d.ldg + i;
    } else {
      i = e / q;
      j = e - i * q;
      g = i * d.ldg + j;
    }
  };
  double sum = 0.0;
#pragma unroll 4
  for (int e = threadIdx.x; e < total; e += kTinyThreads) {
    int i, j;
    int64_t g;
    row_col(e, i, j, g);
    float v = load_g<GT>(d.G, g);
    if (d.M) v = ns_dir(L.common, v, ns_moment(L.common, v, d.M[e]));
    X[i * pitch + j] = v;
    sum += static_cast<double>(v) * v;
  }
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) dpart[threadIdx.x >> 6] = sum;
  __syncthreads();
  sum = 0.0;
#pragma unroll
  for (int w = 0; w < kTinyThreads / 64; ++w) sum += dpart[w];
  const double norm = sqrt(sum);
  const bool finite = norm < 1.7e308;   // false for NaN too
  if (threadIdx.x == 0) L.common.status[d.slot] = finite ? 0 : kNsNonFinite;
  if (!finite) return;
  int e2 = 0;
  const double f = norm > 0.0 ? frexp(norm, &e2) : 0.0;
  const float inv = f > 0.0 ? static_cast<float>(1.0 / f) : 0.0f;
#pragma unroll 4
  for (int e = threadIdx.x; e < total; e += kTinyThreads) {
    int i, j;
    int64_t g;
    row_col(e, i, j, g);
    X[i * pitch + j] = ldexpf(X[i * pitch + j], -e2) * inv;
    if (d.M) d.M[e] = ns_moment(L.common, load_g<GT>(d.G, g), d.M[e]);
  }
  __syncthreads();

  const int block = threadIdx.x / T, t = threadIdx.x % T;
  const int bi = S * (block / SIDE), bk = S * (block % SIDE);
  for (int it = 0; it < L.steps; ++it) {
    const float ca = L.coef[it][0], cb = L.coef[it][1], cc = L.coef[it][2];
    float a[S][S];
#pragma unroll
    for (int r = 0; r < S; ++r)
#pragma unroll
      for (int k = 0; k < S; ++k) a[r][k] = 0.0f;
    // rows past p re-read the last one; their sums are set to zero below
#pragma unroll 2
    for (int j = t; j < q; j += T) {
      float u[S], v[S];
#pragma unroll
      for (int r = 0; r < S; ++r) {
        u[r] = X[min(bi + r, p - 1) * pitch + j];
        v[r] = X[min(bk + r, p - 1) * pitch + j];
      }
#pragma unroll
      for (int r = 0; r < S; ++r)
#pragma unroll
        for (int k = 0; k < S; ++k) a[r][k] = fmaf(u[r], v[k], a[r][k]);
    }
#pragma unroll
    for (int r = 0; r < S; ++r)
#pragma unroll
      for (int k = 0; k < S; ++k) {
#pragma unroll
        for (int s = 32; s > 0; s >>= 1) a[r][k] += __shfl_xor(a[r][k], s);
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][r * S + k] = a[r][k];
      }
    __syncthreads();
    const int pi = threadIdx.x / P, pk = threadIdx.x % P;
    if (threadIdx.x < P * P) {
      const int from = ((pi / S) * SIDE + pk / S) * PARTS, at = (pi % S) * S + pk % S;
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < PARTS; ++w) s += part[from + w][at];
      A[pi][pk] = pi < p && pk < p ? s : 0.0f;
    }
    __syncthreads();
    if (threadIdx.x < P * P) {
      float s = 0.0f;
#pragma unroll
      for (int l = 0; l < P; ++l) s = fmaf(A[pi][l], A[l][pk], s);
      // with the diagonal apart: X <- a X + (b A + c A^2) X
      B[pi][pk] = fmaf(cc, s, cb * A[pi][pk]);
    }
    __syncthreads();
    for (int j = threadIdx.x; j < q; j += kTinyThreads) {
      float x[P];
#pragma unroll
      for (int k = 0; k < P; ++k) x[k] = k < p ? X[k * pitch + j] : 0.0f;
#pragma unroll 1   // one row of B in registers at a time
      for (int i = 0; i < p; ++i) {
        float y = 0.0f;
#pragma unroll
        for (int k = 0; k < P; ++k) y = fmaf(B[i][k], x[k], y);
        X[i * pitch + j] = fmaf(ca, X[i * pitch + j], y);
      }
    }
    __syncthreads();
  }
#pragma unroll 4
  for (int e = threadIdx.x; e < total; e += kTinyThreads) {
    int i, j;
    int64_t g;
    row_col(e, i, j, g);
    const int r = tall ? j : i, col = tall ? i : j;
    const int64_t o = r * d.ldo + col;
    const float v = X[i * pitch + j];
    if (L.step) {
      float* w = static_cast<float*>(d.O) + o;
      *w = fmaf(-d.scale, v, L.common.decay * *w);
    } else if (L.common.odtype) {
      static_cast<uint16_t*>(d.O)[o] = to_bf16(v);
    } else {
      static_cast<float*>(d.O)[o] = v;
    }
  }
}

template <typename GT>
hipError_t tiny(const NsSmall& L, int p, hipStream_t st) {
  const dim3 grid(L.common.total), block(kTinyThreads);
  switch (p) {
    case 1: k_ns_tiny<GT, 1><<<grid, block, 0, st>>>(L); break;
    case 2: k_ns_tiny<GT, 2><<<grid, block, 0, st>>>(L); break;
    case 4: k_ns_tiny<GT, 4><<<grid, block, 0, st>>>(L); break;
    case 8: k_ns_tiny<GT, 8><<<grid, block, 0, st>>>(L); break;
    case 16: k_ns_tiny<GT, 16><<<grid, block, 0, st>>>(L); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ns_tiny(const NsSmall& L, int p, hipStream_t st) {
  return L.common.gdtype ? tiny<uint16_t>(L, p, st) : tiny<float>(L, p, st);
}

}  // namespace dion
