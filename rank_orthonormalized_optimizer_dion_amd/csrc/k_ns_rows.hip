// The orthogonalization (or Muon step) of a matrix with at most 16 rows or
// columns that does not fit one compute unit's LDS (k_ns_tiny), in plain
// float32 arithmetic as there: such a matrix has few singular values for the
// roundings of 16-bit planes to average over, and padding to the matrix cores'
// tiles would multiply its memory and products by up to 64.
//
// X (p x q, p <= 16) lies in the workspace as float32 rows; a workgroup owns
// a chunk of columns, a thread one column at a time in registers:
//   stage 0           X = D / ||D||_F (the momentum is updated on the way)
//   stage 1 .. steps  X <- a X + (b A + c A^2) X, the last one to the output
// and every stage but the last leaves its chunk's part of A = X X^T (float32
// sums, entries on and below the diagonal), which every workgroup of the next
// stage adds up in the chunks' order, in float64.  A stage reads and writes X
// once.
//
// Measured (MI355X, five quintic iterations: seven launches, which bound the
// small ones): 5 x 7000 45 us, 1 x 1048576 53 us, 16 x 65536 94 us, 16 x
// 131071 115 us; as two padded float16 planes on the matrix cores these took
// 233, 2315, 486 and 680 us, with errors of up to 4e-6 (here 1.6e-6) and 130
// times the workspace (1 x 1048576).  At the limit of the one-workgroup form:
// 16 x 2048 127 us there, 16 x 2049 82 us here; 1 x 32768 52 us and 1 x 32769
// 49 us; 4 x 8192 68 us and 4 x 10000 47 us.
#include "dion.h"
#include "mm16.h"
#include "ns_device.h"
#include "ns_types.h"

namespace dion {

namespace {

constexpr int kThreads = kNsRowThreads, kRowWaves = kThreads / 64;

// Sums over a wavefront's lanes of N values per lane.  Each step halves the
// values a lane keeps, sending the other half to the lane across: N exchanges
// instead of 6 N.
template <int N, int M, int T>
__device__ __forceinline__ void fold_lanes(float (&v)[T], int lane) {
  if constexpr (M > 0) {
    constexpr int H = (N + 1) / 2;
    const bool up = lane & M;
#pragma unroll
    for (int e = 0; e < H; ++e) {
      const float a = v[e], b = e + H < N ? v[e + H] : 0.0f;
      v[e] = (up ? b : a) + __shfl_xor(up ? a : b, M);
    }
    fold_lanes<H, M / 2>(v, lane);
  }
}
// Which of the N values a lane's e-th sum is; -1: none.
template <int N, int M>
__device__ __forceinline__ int fold_index(int e, int lane) {
  if constexpr (M == 0) {
    return e;
  } else {
    constexpr int H = (N + 1) / 2;
    int i = fold_index<H, M / 2>(e, lane);
    if (i >= 0 && (lane & M)) i += H;
    return i < N ? i : -1;
  }
}
constexpr int fold_count(int n) {
  for (int m = 32; m > 0; m /= 2) n = (n + 1) / 2;
  return n;
}

enum Stage { kLoad, kIterate, kOutput };

// GT: G's type (kLoad), else float.
template <Stage STAGE, int P, typename GT>
__global__ __launch_bounds__(kThreads) void k_ns_rows(NsRows L) {
  constexpr int T = P * (P + 1) / 2;   // entry (i, k), k <= i, of A at i (i + 1) / 2 + k
  // lanes that share an entry's sum over the chunks
  constexpr int R = P == 16 ? 2 : P == 8 ? 8 : P == 4 ? 32 : 64;
  static_assert(T * R <= kThreads, "every entry has its lanes");
  __shared__ float A[P][P], B[P][P], part[kRowWaves][T];
  __shared__ double dpart[kRowWaves];
  NsDesc d;
  NsClass c;
  int local;
  ns_locate(L.common, blockIdx.x, d, c, local);
  const int p = uniform32(d.p), q = uniform32(d.q), tall = uniform32(d.tall);
  const int tiles = uniform32(c.tiles);
  const int64_t pitch = ns_row_pitch(q);
  const int cols = ns_row_cols(q), beg = uniform32(local) * cols, end = min(q, beg + cols);
  const int lane = threadIdx.x & 63, wave = wave16();
  float* X = uniform_at(reinterpret_cast<float*>(L.common.ws + d.oX));
  float* sums = reinterpret_cast<float*>(L.common.ws + (L.stage & 1 ? d.oB : d.oA));

  int e2 = 0;
  float inv = 0.0f;
  if constexpr (STAGE == kLoad) {
    const double norm = ns_norm<kRowWaves>(L.common, d, dpart);
    const bool finite = norm < 1.7e308;   // false for NaN too
    if (!finite) {
      if (local == 0 && threadIdx.x == 0) L.common.status[d.slot] = kNsNonFinite;
      return;
    }
    const double f = norm > 0.0 ? frexp(norm, &e2) : 0.0;
    inv = f > 0.0 ? static_cast<float>(1.0 / f) : 0.0f;
  } else {
    if (uniform32(L.common.status[d.slot]) & kNsNonFinite) return;
    const float* from = reinterpret_cast<const float*>(L.common.ws + (L.stage & 1 ? d.oA : d.oB));
    const int e = threadIdx.x / R, r = threadIdx.x % R;
    double s = 0.0;
    if (e < T) {
#pragma unroll 16
      for (int k = r; k < tiles; k += R) s += from[static_cast<int64_t>(k) * T + e];
    }
#pragma unroll
    for (int m = R / 2; m > 0; m >>= 1) s += __shfl_xor(s, m);
    if (e < T && r == 0) {
      int i = 0;
      while ((i + 1) * (i + 2) / 2 <= e) ++i;
      const int k = e - i * (i + 1) / 2;
      A[i][k] = A[k][i] = static_cast<float>(s);
    }
    __syncthreads();
    if (threadIdx.x < P * P) {
      const int i = threadIdx.x / P, k = threadIdx.x % P;
      float t = 0.0f;
#pragma unroll
      for (int l = 0; l < P; ++l) t = fmaf(A[i][l], A[l][k], t);
      // with the diagonal apart: X <- a X + (b A + c A^2) X
      B[i][k] = fmaf(L.c, t, L.b * A[i][k]);
    }
    __syncthreads();
  }

  // strides by X's row and column: of G, of the step's momentum, of the output
  const int64_t gi = tall ? 1 : d.ldg, gj = tall ? d.ldg : 1;
  const int64_t mi = tall ? 1 : q, mj = tall ? p : 1;
  const int64_t oi = tall ? 1 : d.ldo, oj = tall ? d.ldo : 1;
  float acc[T];
#pragma unroll
  for (int e = 0; e < T; ++e) acc[e] = 0.0f;
  for (int j = beg + threadIdx.x; j < end; j += kThreads) {
    float x[P], y[P];
    if constexpr (STAGE == kLoad) {
      // every load before the first store: one may not move over the other
#pragma unroll
      for (int i = 0; i < P; ++i) {
        y[i] = i < p ? load_g<GT>(d.G, j * gj + i * gi) : 0.0f;
        x[i] = i < p && d.M ? d.M[j * mj + i * mi] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (i < p && d.M) {
          x[i] = ns_moment(L.common, y[i], x[i]);
          d.M[j * mj + i * mi] = x[i];
          y[i] = ns_dir(L.common, y[i], x[i]);
        }
        y[i] = ldexpf(y[i], -e2) * inv;
      }
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) x[i] = i < p ? X[i * pitch + j] : 0.0f;
      // B is read anew for every column and, with 16 rows, row by row: its 256
      // values at once would be spilled
      int zero = 0;
      asm volatile("" : "+v"(zero));
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < P; ++k) s = fmaf((&B[i][k])[zero], x[k], s);
        y[i] = fmaf(L.a, x[i], s);
        if (P == 16) asm volatile("" : "+v"(zero), "+v"(y[i]));
      }
    }
    if constexpr (STAGE == kOutput) {
      float* w32 = static_cast<float*>(d.O) + j * oj;
      uint16_t* w16 = static_cast<uint16_t*>(d.O) + j * oj;
      if (L.step) {
#pragma unroll
        for (int i = 0; i < P; ++i) x[i] = i < p ? w32[i * oi] : 0.0f;
#pragma unroll
        for (int i = 0; i < P; ++i) y[i] = fmaf(-d.scale, y[i], L.common.decay * x[i]);
      }
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (i >= p) continue;
        if (L.common.odtype) w16[i * oi] = to_bf16(y[i]);
        else w32[i * oi] = y[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (i < p) X[i * pitch + j] = y[i];
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int k = 0; k <= i; ++k) acc[i * (i + 1) / 2 + k] = fmaf(y[i], y[k], acc[i * (i + 1) / 2 + k]);
    }
  }
  if constexpr (STAGE == kOutput) return;
  fold_lanes<T, 32>(acc, lane);
#pragma unroll
  for (int e = 0; e < fold_count(T); ++e) {
    const int i = fold_index<T, 32>(e, lane);
    if (i >= 0) part[wave][i] = acc[e];
  }
  __syncthreads();
  if (threadIdx.x < T) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowWaves; ++w) s += part[w][threadIdx.x];
    sums[static_cast<int64_t>(local) * T + threadIdx.x] = s;
  }
}

template <int P>
hipError_t rows(const NsRows& L, hipStream_t st) {
  const dim3 grid(L.common.total), block(kThreads);
  if (L.stage == L.steps) k_ns_rows<kOutput, P, float><<<grid, block, 0, st>>>(L);
  else if (L.stage > 0) k_ns_rows<kIterate, P, float><<<grid, block, 0, st>>>(L);
  else if (L.common.gdtype) k_ns_rows<kLoad, P, uint16_t><<<grid, block, 0, st>>>(L);
  else k_ns_rows<kLoad, P, float><<<grid, block, 0, st>>>(L);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ns_rows(const NsRows& L, int p, hipStream_t st) {
  switch (p) {
    case 1: return rows<1>(L, st);
    case 2: return rows<2>(L, st);
    case 4: return rows<4>(L, st);
    case 8: return rows<8>(L, st);
    case 16: return rows<16>(L, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace dion
