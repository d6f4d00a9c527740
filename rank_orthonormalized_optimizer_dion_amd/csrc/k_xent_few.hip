// Cross entropy of few tokens (at most 64): reading W once per product, and
// writing dW, is what it costs, in any type and at any alignment (24 tokens, 2048
// -> 32000: z 36 us, dx 30, dW 31, 3.7 to 4.4 TB/s; one token, 768 -> 32000
// forward 13.2 us, 11.5 of it k_few_z, 4.3 TB/s).  All products run on the
// bfloat16 matrix cores with operands that come straight from global memory into
// registers:
//
//   z  = x W^T      k_few_z     a lane's 16 consecutive elements of a row of W
//                               are two operands; the 8 wavefronts of a
//                               workgroup share the reduction
//   dx = dz W       k_few_dx    the reduction runs down W's columns: a lane
//                               loads 16 bytes of each of 8 rows, which are
//                               the operands of as many products as it has
//                               columns (which column of the output is whose
//                               is free); no transposition through LDS
//   dW = dz^T x     k_few_dw    x transposed once (k_few_prep); a lane's 16
//                               outputs are consecutive
//
// float32 values are split into three bfloat16 planes in registers and take
// six products, as in the tiles (lin_device.h); dz comes in two planes with
// bfloat16 tensors (their roundings would average over too few tokens), three
// with float32.
#include "dion.h"
#include "lin_device.h"
#include "mm32.h"
#include "xent_device.h"
#include "xent_types.h"

namespace dion {

namespace {

// 16 bytes at any alignment of the element type (global memory takes vector
// accesses at any address).  FAR: past the caches.
template <class V, bool FAR = false, class T>
__device__ __forceinline__ V load_any(const T* p) {
  V v;
  if constexpr (FAR) {
    typedef V Any __attribute__((aligned(2)));
    v = __builtin_nontemporal_load(reinterpret_cast<const Any*>(p));
  } else {
    __builtin_memcpy(&v, p, sizeof(V));
  }
  return v;
}

// Eight values as the operands of their planes.
template <int PL>
struct Planes8 {
  u32x4 p[PL];
};
__device__ __forceinline__ Planes8<3> split8(const float (&v)[8]) {
  const Split8 s = split_planes(v);
  return {{s.p[0], s.p[1], s.p[2]}};
}

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// The product of two operands' planes, smallest first: three by three as in
// plane_pairs, else every plane of one with the single plane of the other.
template <int PA, int PB>
__device__ __forceinline__ f32x4 mfma_planes(const Planes8<PA>& a, const Planes8<PB>& b, f32x4 c) {
  if constexpr (PA == 3) {
    c = mfma(a.p[1], b.p[1], c);
    c = mfma(a.p[2], b.p[0], c);
    c = mfma(a.p[0], b.p[2], c);
    c = mfma(a.p[1], b.p[0], c);
    c = mfma(a.p[0], b.p[1], c);
    return mfma(a.p[0], b.p[0], c);
  } else {
    static_assert(PB == 1 || PA == 1, "one operand in planes");
#pragma unroll
    for (int k = PA * PB - 1; k >= 0; --k) c = mfma(a.p[PA == 1 ? 0 : k], b.p[PB == 1 ? 0 : k], c);
    return c;
  }
}

// What a lane reads of 64 consecutive elements of a row of k, from column c
// (a multiple of 64): two operands of eight, elements 32 h + 8 g .. of the
// lane's group g = lane / 16, so that every load takes 64 consecutive bytes of
// a row.  In float32 an operand takes two loads, elements 32 h + 4 g .. and 32 h +
// 16 + 4 g ..: x's planes are stored in that order (k_few_prep).  Elements past
// the row are zero.  TAIL: the row may end inside.
template <bool F32>
struct Raw16 {
  u32x4 v[F32 ? 4 : 2];
};
template <bool F32, bool TAIL, bool FAR = false>
__device__ __forceinline__ Raw16<F32> load16(const void* row, int c, int k) {
  constexpr int N = F32 ? 4 : 8;   // elements of a load
  using T = typename std::conditional<F32, float, uint16_t>::type;
  const int g = (threadIdx.x & 63) >> 4;
  Raw16<F32> o;
#pragma unroll
  for (int i = 0; i < (F32 ? 4 : 2); ++i) {
    const int c0 = c + (F32 ? 16 : 32) * i + N * g;
    const T* p = static_cast<const T*>(row) + c0;
    if (!TAIL || c0 + N <= k) {
      o.v[i] = load_any<u32x4, FAR>(p);
    } else {
      T v[N];
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = c0 + j < k ? p[j] : T(0);
      __builtin_memcpy(&o.v[i], v, 16);
    }
  }
  return o;
}
template <bool F32>
__device__ __forceinline__ Planes8<F32 ? 3 : 1> planes16(const Raw16<F32>& r, int h) {
  if constexpr (F32) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(r.v[2 * h][i]);
      v[4 + i] = __uint_as_float(r.v[2 * h + 1][i]);
    }
    return split8(v);
  } else {
    return {{r.v[h]}};
  }
}

// Pieces of z's reduction that a wavefront loads at a time.
template <int TB, int RT, bool F32>
constexpr int kFewZPieces = F32 ? (TB * RT == 1 ? 2 : 1) : TB == 2 && RT == 1 ? 4 : TB * RT <= 8 ? 2 : 1;

// Planes of x (zero past its columns) and of its transpose (tokens padded by
// zeros to a.tp), 64 columns per block.
template <bool F32>
__device__ __forceinline__ void prep_block(const XentPrep& a, int block, float* tile) {
  constexpr int P = F32 ? 3 : 1;
  const int c0 = block * 64, pitch = a.tp + 1;
#pragma unroll 4
  for (int i = threadIdx.x; i < a.tp * 64; i += 512) {
    const int token = i >> 6, c = i & 63;
    const bool in = token < a.t && c0 + c < a.k;
    float v = in ? load_value(a.x, token * a.ldx + c0 + c, !F32) : 0.0f;
    tile[c * pitch + token] = v;
    if (a.xp && token < a.t) {
      // float32: the order of load16
      const int at = F32 ? (c & ~31) + 8 * ((c & 15) >> 2) + (c & 3) + 4 * ((c >> 4) & 1) : c;
      for (int pl = 0; pl < P; ++pl) {
        const float u = pinned(v);
        const uint16_t h = pl == 0 && P > 1 ? first_plane(u) : to_bf16(u);
        v = u - bf16_to_f32(h);
        a.xp[pl * a.xplane + token * a.ldp + c0 + at] = h;
      }
    }
  }
  if (!a.xt) return;
  __syncthreads();
#pragma unroll 4
  for (int i = threadIdx.x; i < a.tp * 64; i += 512) {
    const int token = i & (a.tp - 1), c = i / a.tp;
    if (c0 + c >= a.k) continue;
    float v = tile[c * pitch + token];
    for (int pl = 0; pl < P; ++pl) {
      const float u = pinned(v);
      const uint16_t h = pl == 0 && P > 1 ? first_plane(u) : to_bf16(u);
      v = u - bf16_to_f32(h);
      a.xt[pl * a.xtplane + static_cast<int64_t>(c0 + c) * a.tp + token] = h;
    }
  }
}

template <bool F32>
__global__ __launch_bounds__(512) void k_few_prep(XentPrep a) {
  __shared__ float tile[64 * (kXentFew16 + 1)];
  prep_block<F32>(a, blockIdx.x, tile);
}

// z for 16 RT rows of W at a time, its statistics or dz; the 8 wavefronts of a
// workgroup take turns at 64-element pieces of the reduction.  What is read
// again and again is x: RT blocks of rows share its operands.  RAW: x is read as it is, like W (one block of 16
// tokens), else from planes whose rows are readable, and zero past k, up to f.kx
// columns.  With dz, workgroups past the first `prep.first` transpose x for dW.
template <int TB, int RT, bool F32, bool RAW, bool GRAD, bool FAR>
__global__ __launch_bounds__(512, RT == 2 ? 4 : 2) void k_few_z(XentFew f, XentEpi e, XentPrep prep) {
  constexpr int P = F32 ? 3 : 1, ES = F32 ? 4 : 2;
  constexpr int B = (TB + 1) / 2;                       // 512 threads hold 32 tokens by 16 rows of W
  constexpr int RR = RT * TB <= 8 ? RT : 8 / TB;   // blocks of rows that meet in LDS at a time
  static_assert(RT % RR == 0, "whole rounds");
  struct Sums {
    float v[8][RR][TB][16][17];   // wavefront, block of rows, token / 16, token % 16, row
  };
  constexpr int kPrep = 64 * (16 * TB < 32 ? 33 : 16 * TB + 1);
  __shared__ union {
    Sums red;
    float tile[GRAD ? kPrep : 1];
  } lds;
  if constexpr (GRAD) {
    if (static_cast<int>(blockIdx.x) >= prep.first) {
      prep_block<F32>(prep, blockIdx.x - prep.first, lds.tile);
      return;
    }
  }
  const int workers = GRAD ? prep.first : static_cast<int>(gridDim.x);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = threadIdx.x & 15;
  XentRow r[B];
  int64_t y[B];
  float top[B], sum[B], total[B];
#pragma unroll
  for (int b = 0; b < B; ++b) {
    const int token = 32 * b + (threadIdx.x >> 4);
    top[b] = -INFINITY;
    sum[b] = total[b] = 0.0f;
    if constexpr (GRAD) r[b] = xent_row(e, token, f.t, y[b]);
    else y[b] = token < f.t ? e.target[token] : -1;
  }
  const char* xr[TB];
#pragma unroll
  for (int b = 0; b < TB; ++b)
    xr[b] = static_cast<const char*>(f.x) + min(16 * b + (lane & 15), f.t - 1) * f.ldx * (RAW ? ES : 2);
  const int rows = GRAD ? static_cast<int>(e.pitch) : f.n;
  for (int n0 = blockIdx.x * 16 * RT; n0 < rows; n0 += workers * 16 * RT) {
    const char* wr[RT];
#pragma unroll
    for (int q = 0; q < RT; ++q)
      wr[q] = static_cast<const char*>(f.w) + min(n0 + 16 * q + (lane & 15), f.n - 1) * f.ldw * ES;
    f32x4 acc[RT][TB];
#pragma unroll
    for (int q = 0; q < RT; ++q)
#pragma unroll
      for (int b = 0; b < TB; ++b) acc[q][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // U pieces of 64 elements of the reduction: W's loads, then the products
    const auto pieces = [&](auto tail, auto count, int k0) {
      constexpr bool TAIL = decltype(tail)::value;
      constexpr int N = decltype(count)::value;
      Raw16<F32> w[N][RT], xw[N][RAW ? TB : 1];
      Planes8<P> x[N][RAW ? 1 : TB][2];
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const int k = k0 + 512 * u;
#pragma unroll
        for (int q = 0; q < RT; ++q) w[u][q] = load16<F32, TAIL, FAR>(wr[q], k, f.k);
#pragma unroll
        for (int b = 0; b < TB; ++b) {
          if constexpr (RAW) {
            xw[u][b] = load16<F32, TAIL>(xr[b], k, f.k);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int pl = 0; pl < P; ++pl) {
                const int c8 = k + 32 * h + 8 * (lane >> 4);
                x[u][b][h].p[pl] = !TAIL || c8 < f.kx
                                       ? *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(xr[b]) + pl * f.xplane + c8)
                                       : u32x4{0, 0, 0, 0};
              }
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < N; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int q = 0; q < RT; ++q) {
            const Planes8<P> a = planes16<F32>(w[u][q], h);
#pragma unroll
            for (int b = 0; b < TB; ++b) {
              if constexpr (RAW) acc[q][b] = mfma_planes(a, planes16<F32>(xw[u][b], h), acc[q][b]);
              else acc[q][b] = mfma_planes(a, x[u][b][h], acc[q][b]);
            }
          }
    };
    constexpr int U = kFewZPieces<TB, RT, F32>;
    using std::integral_constant;
    int k0 = 64 * wave;
    if constexpr (U > 1)
      for (; k0 + 512 * (U - 1) + 64 <= f.k; k0 += 512 * U) pieces(std::false_type{}, integral_constant<int, U>{}, k0);
    for (; k0 + 64 <= f.k; k0 += 512) pieces(std::false_type{}, integral_constant<int, 1>{}, k0);
    if (k0 < f.k) pieces(std::true_type{}, integral_constant<int, 1>{}, k0);
#pragma unroll
    for (int q0 = 0; q0 < RT; q0 += RR) {
      // lane l, register i: row 4 (l / 16) + i of W, token l % 16
#pragma unroll
      for (int q = 0; q < RR; ++q)
#pragma unroll
        for (int b = 0; b < TB; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) lds.red.v[wave][q][b][lane & 15][4 * (lane >> 4) + i] = acc[q0 + q][b][i];
      __syncthreads();
#pragma unroll
      for (int b = 0; b < B; ++b)
#pragma unroll
        for (int q = 0; q < RR; ++q) {
          const int token = 32 * b + (threadIdx.x >> 4), col = n0 + 16 * (q0 + q) + c;
          float z = 0.0f;
          if (token < 16 * TB) {
#pragma unroll
            for (int s = 0; s < 8; ++s) z += lds.red.v[s][q][token >> 4][token & 15][c];
          }
          if constexpr (GRAD) {
            float v = dz_of(z, r[b].lse, r[b].a, r[b].b, r[b].mask);
            if (y[b] == e.j0 + col) v -= r[b].c;
            if (col >= f.n || token >= f.t) v = 0.0f;
            if (token < f.tp && col < e.pitch) {   // dz by rows, and transposed with its tokens padded by zeros
              for (int pl = 0; pl < e.planes; ++pl) {
                const float u = pinned(v);
                const uint16_t h = pl == 0 ? first_plane(u) : to_bf16(u);
                v = u - bf16_to_f32(h);
                if (token < f.t) e.dz[pl * e.plane + token * e.pitch + col] = h;
                f.dzt[pl * f.dztplane + static_cast<int64_t>(col) * f.tp + token] = h;
              }
            }
          } else {
            const bool in = col < f.n && token < f.t;
            const float hi = row_max(in ? z : -INFINITY), base = base_of(hi);
            const float s = row_sum(in ? exp_fast(z - base) : 0.0f);
            merge(top[b], sum[b], hi, s);
            if (e.total) total[b] += row_sum(in ? z : 0.0f);
            if (in && y[b] == e.j0 + col) e.hit[token] = z;
          }
        }
      __syncthreads();
    }
  }
  if constexpr (!GRAD) {
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int token = 32 * b + (threadIdx.x >> 4);
      if (token < f.t && c == 0) {
        const int64_t at = static_cast<int64_t>(blockIdx.x) * f.t + token;
        e.top[at] = top[b];
        e.sum[at] = sum[b];
        if (e.total) e.total[at] = total[b];
      }
    }
  }
}

// dx's sums over every `gridDim.y`-th block of 4 x 32 rows of W, for 16
// times CW columns.
template <int TB, bool F32, bool FAR>
__global__ __launch_bounds__(256, 2) void k_few_dx(XentFew f, const uint16_t* dz, int64_t pitch, int64_t plane, float* part) {
  constexpr int CW = F32 ? 4 : 8, PW = F32 ? 3 : 1, PZ = F32 ? 3 : 2;
  using T = typename std::conditional<F32, float, uint16_t>::type;
  __shared__ float red[2][CW * TB * 4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // lanes past the last whole group of columns take that one again
  const int c = min((static_cast<int>(blockIdx.x) * 16 + (lane & 15)) * CW, max(f.k - CW, 0));
  const int steps = (f.n + 31) / 32;
  f32x4 acc[CW][TB];
#pragma unroll
  for (int m = 0; m < CW; ++m)
#pragma unroll
    for (int b = 0; b < TB; ++b) acc[m][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const uint16_t* zr[TB];
#pragma unroll
  for (int b = 0; b < TB; ++b) zr[b] = dz + min(16 * b + (lane & 15), f.t - 1) * pitch + 8 * (lane >> 4);
  const bool whole = CW <= f.k;
#pragma unroll 2
  for (int s = blockIdx.y * 4 + wave; s < steps; s += 4 * gridDim.y) {
    const int j0 = 32 * s + 8 * (lane >> 4);
    u32x4 w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const T* p = static_cast<const T*>(f.w) + min(j0 + i, f.n - 1) * f.ldw + c;
      if (whole) {
        w[i] = load_any<u32x4, FAR>(p);
      } else {
        T v[CW];
#pragma unroll
        for (int m = 0; m < CW; ++m) v[m] = c + m < f.k ? p[m] : T(0);
        __builtin_memcpy(&w[i], v, 16);
      }
    }
    Planes8<PZ> a[TB];
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int pl = 0; pl < PZ; ++pl) a[b].p[pl] = *reinterpret_cast<const u32x4*>(zr[b] + pl * plane + 32 * s);
    if (32 * s + 32 > f.n) {   // rows past the last, whatever the clamped row holds
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j0 + i >= f.n) w[i] = u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int m = 0; m < CW; ++m) {
      Planes8<PW> b;
      if constexpr (F32) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i][m]);
        b = split8(v);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)   // column m of rows 2 i and 2 i + 1
          b.p[0][i] = __builtin_amdgcn_perm(w[2 * i + 1][m / 2], w[2 * i][m / 2], m % 2 ? 0x07060302u : 0x05040100u);
      }
#pragma unroll
      for (int q = 0; q < TB; ++q) acc[m][q] = mfma_planes(a[q], b, acc[m][q]);
    }
  }
  // the four wavefronts' sums, in a fixed order
#pragma unroll
  for (int h = 2; h > 0; h /= 2) {
    if (wave >= h && wave < 2 * h) {
#pragma unroll
      for (int m = 0; m < CW; ++m)
#pragma unroll
        for (int b = 0; b < TB; ++b)
#pragma unroll
          for (int v = 0; v < 4; ++v) red[wave - h][(m * TB + b) * 4 + v][lane] = acc[m][b][v];
    }
    __syncthreads();
    if (wave < h) {
#pragma unroll
      for (int m = 0; m < CW; ++m)
#pragma unroll
        for (int b = 0; b < TB; ++b)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[m][b][v] += red[wave][(m * TB + b) * 4 + v][lane];
    }
    __syncthreads();
  }
  if (wave != 0) return;
  // lane l, register v: token 4 (l / 16) + v, this lane's columns
#pragma unroll
  for (int b = 0; b < TB; ++b)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int token = 16 * b + 4 * (lane >> 4) + v;
      if (token >= f.t) continue;
      float* out = part + (static_cast<int64_t>(blockIdx.y) * f.t + token) * f.k + c;
#pragma unroll
      for (int m = 0; m < CW; ++m)
        if (c + m < f.k) out[m] = acc[m][b][v];
    }
}

// 256 elements of dx from the partial sums, in order.
__device__ __forceinline__ void dxsum_block(const XentDxSum& a, int64_t block) {
  const int64_t size = static_cast<int64_t>(a.t) * a.k, i = block * 256 + threadIdx.x;
  if (i >= size) return;
  float s = 0.0f;
#pragma unroll 8
  for (int p = 0; p < a.parts; ++p) s += a.part[p * size + i];
  const int64_t row = i / a.k;
  store_value(a.dx, row * a.ld + (i - row * a.k), a.dtype, s);
}
__global__ __launch_bounds__(256) void k_few_dxsum(XentDxSum a) { dxsum_block(a, blockIdx.x); }

// dW: a wavefront's 16 RJ rows by the columns of its part, 64 at a time.
// Workgroups past the first d.tiles sum up dx.
template <int TT, bool F32>
__global__ __launch_bounds__(256, 2) void k_few_dw(XentFew f, XentDw d, XentDxSum sum) {
  constexpr int PX = F32 ? 3 : 1, PZ = F32 ? 3 : 2, RJ = kFewDwRows / 16;
  if (static_cast<int>(blockIdx.x) >= d.tiles) {
    dxsum_block(sum, blockIdx.x - d.tiles);
    return;
  }
  const int down = blockIdx.x % d.down, across = blockIdx.x / d.down;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int j0 = (down * 4 + wave) * 16 * RJ;
  if (j0 >= f.n) return;
  Planes8<PZ> z[RJ][TT];
#pragma unroll
  for (int q = 0; q < RJ; ++q)
#pragma unroll
    for (int s = 0; s < TT; ++s)
#pragma unroll
      for (int pl = 0; pl < PZ; ++pl)
        z[q][s].p[pl] = *reinterpret_cast<const u32x4*>(
            f.dzt + pl * f.dztplane + static_cast<int64_t>(min(j0 + 16 * q + (lane & 15), f.n - 1)) * f.tp + 32 * s + 8 * (lane >> 4));
  const int r = lane & 15;
  for (int c0 = across * d.cols; c0 < min(f.k, (across + 1) * d.cols); c0 += 64) {
    f32x4 acc[4][RJ];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      // which column the operand's row r is is free: four lanes' stores of 16
      // bytes are made 64 consecutive bytes
      const int64_t c = min(c0 + (F32 ? 16 * m + r : 32 * (m >> 1) + 8 * (r >> 2) + 4 * (m & 1) + (r & 3)), f.k - 1);
#pragma unroll
      for (int q = 0; q < RJ; ++q) acc[m][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < TT; ++s) {
        Planes8<PX> x;
#pragma unroll
        for (int pl = 0; pl < PX; ++pl)
          x.p[pl] = *reinterpret_cast<const u32x4*>(f.xt + pl * f.xtplane + c * f.tp + 32 * s + 8 * (lane >> 4));
#pragma unroll
        for (int q = 0; q < RJ; ++q) acc[m][q] = mfma_planes(x, z[q][s], acc[m][q]);
      }
    }
    constexpr int N = F32 ? 4 : 8;   // outputs of a store
#pragma unroll
    for (int q = 0; q < RJ; ++q) {
      const int j = j0 + 16 * q + r;
      if (j >= f.n) continue;
#pragma unroll
      for (int i = 0; i < 16 / N; ++i) {
        const int c = c0 + 4 * N * i + N * (lane >> 4);
        const int64_t at = j * d.ld + c;
        float v[N];
#pragma unroll
        for (int u = 0; u < N; ++u) v[u] = acc[i * (N / 4) + u / 4][q][u % 4];
        if (c + N <= f.k) {
          if constexpr (F32) {
            float* p = static_cast<float*>(d.dw) + at;
            f32x4 u = {v[0], v[1], v[2], v[3]};
            if (d.accumulate) u += load_any<f32x4>(p);
            __builtin_memcpy(p, &u, 16);
          } else {
            uint16_t* p = static_cast<uint16_t*>(d.dw) + at;
            uint16_t h[8], old[8];
            if (d.accumulate) __builtin_memcpy(old, p, 16);
#pragma unroll
            for (int u = 0; u < 8; ++u) h[u] = to_bf16(d.accumulate ? v[u] + bf16_to_f32(old[u]) : v[u]);
            const u32x4 u = pack8(h);
            __builtin_memcpy(p, &u, 16);
          }
        } else {
#pragma unroll
          for (int u = 0; u < N; ++u)
            if (c + u < f.k) store_value(d.dw, at + u, !F32, d.accumulate ? v[u] + load_value(d.dw, at + u, !F32) : v[u]);
        }
      }
    }
  }
}

template <int TB, int RT, bool F32, bool FAR>
hipError_t few_z(const XentFew& f, const XentEpi& e, const XentPrep& prep, bool grad, bool raw, int groups, hipStream_t st) {
  const dim3 grid(grad ? prep.first + (prep.xt ? (f.k + 63) / 64 : 0) : groups), block(512);
  if (grad) {
    k_few_z<TB, RT, F32, false, true, FAR><<<grid, block, 0, st>>>(f, e, prep);
  } else if constexpr (TB == 1) {
    if (raw) k_few_z<TB, RT, F32, true, false, FAR><<<grid, block, 0, st>>>(f, e, prep);
    else k_few_z<TB, RT, F32, false, false, FAR><<<grid, block, 0, st>>>(f, e, prep);
  } else {
    k_few_z<TB, RT, F32, false, false, FAR><<<grid, block, 0, st>>>(f, e, prep);
  }
  return hipGetLastError();
}
template <int TB, bool F32>
hipError_t few_z(const XentFew& f, const XentEpi& e, const XentPrep& prep, bool grad, bool raw, int rt, int groups, hipStream_t st) {
  if constexpr (TB == 1 || (TB == 2 && !F32))
    if (rt == 2) return few_z<TB, 2, F32, false>(f, e, prep, grad, raw, groups, st);
  if (rt == 1)
    return f.far ? few_z<TB, 1, F32, true>(f, e, prep, grad, raw, groups, st) : few_z<TB, 1, F32, false>(f, e, prep, grad, raw, groups, st);
  return f.far ? few_z<TB, 4, F32, true>(f, e, prep, grad, raw, groups, st) : few_z<TB, 4, F32, false>(f, e, prep, grad, raw, groups, st);
}

template <int TB, bool F32>
hipError_t few_dx(const XentFew& f, const XentEpi& e, int parts, float* part, hipStream_t st) {
  constexpr int cols = 16 * (F32 ? 4 : 8);
  const dim3 grid((f.k + cols - 1) / cols, parts), block(256);
  if (f.far) k_few_dx<TB, F32, true><<<grid, block, 0, st>>>(f, e.dz, e.pitch, e.plane, part);
  else k_few_dx<TB, F32, false><<<grid, block, 0, st>>>(f, e.dz, e.pitch, e.plane, part);
  return hipGetLastError();
}

unsigned dxsum_blocks(const XentDxSum& s) { return s.dx ? static_cast<unsigned>((static_cast<int64_t>(s.t) * s.k + 255) / 256) : 0; }

template <int TT, bool F32>
hipError_t few_dw(const XentFew& f, XentDw d, const XentDxSum& sum, hipStream_t st) {
  constexpr int rows = 4 * kFewDwRows;
  d.down = (f.n + rows - 1) / rows;
  d.tiles = d.down * ((f.k + d.cols - 1) / d.cols);
  k_few_dw<TT, F32><<<dim3(d.tiles + dxsum_blocks(sum)), dim3(256), 0, st>>>(f, d, sum);
  return hipGetLastError();
}

}  // namespace

int few_rows(int t, int64_t n, bool f32, bool grad, bool far) {
  // 16 rows of W per workgroup where 64 would not make one per CU, or for a few
  // tokens, whose lanes read the same rows of x (one token, 2048 -> 32000: 30 us, 34
  // with 64).
  if (t <= 4 || n < 256 * 64) return 1;
  // 64 rows: x is read a quarter as often (24 tokens, 2048 -> 32000: 36 us, 55 with
  // 16), by one workgroup per CU.  32 rows, by two that fill each other's gaps,
  // where the registers allow it: dz in bfloat16 up to 32 tokens (24 tokens, 2048
  // -> 32000: gradients 114 us, 117 with 64; -> 17000 70 and 73; 8 tokens, 768 -> 50257
  // 68 and 74), but not past the caches (24 tokens, 4096 -> 32000: 220 and 215); the
  // rest where 64 rows would leave an eighth of the rounds empty (24 tokens, 768 ->
  // 50257: 26.1 and 29.9; 2048 -> 17000 25.8 and 29.4, but -> 32000 34.7 and 31.4; 8
  // tokens in float32, 1024 -> 17000 23.3 and 28.4, but 16 tokens, 2048 -> 32000 74 and
  // 62).
  const int64_t blocks = (n + 63) / 64, slots = (blocks + 255) / 256 * 256;
  const bool whole = 8 * blocks >= 7 * slots;
  if (far || t > (f32 ? 16 : 32)) return 4;
  return (grad && !f32) || !whole ? 2 : 4;
}

hipError_t launch_few_prep(const XentPrep& a, bool f32, hipStream_t st) {
  const dim3 grid((a.k + 63) / 64), block(512);
  if (f32) k_few_prep<true><<<grid, block, 0, st>>>(a);
  else k_few_prep<false><<<grid, block, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_few_z(const XentFew& f, const XentEpi& e, const XentPrep& prep, bool f32, bool grad, bool raw, int rt,
                        int groups, hipStream_t st) {
  if (f32) {
    if (f.t <= 16) return few_z<1, true>(f, e, prep, grad, raw, rt, groups, st);
    return few_z<2, true>(f, e, prep, grad, raw, rt, groups, st);
  }
  if (f.t <= 16) return few_z<1, false>(f, e, prep, grad, raw, rt, groups, st);
  return f.t <= 32 ? few_z<2, false>(f, e, prep, grad, raw, rt, groups, st)
                   : few_z<4, false>(f, e, prep, grad, raw, rt, groups, st);
}

hipError_t launch_few_dx(const XentFew& f, const XentEpi& e, bool f32, int parts, float* part, hipStream_t st) {
  if (f32) {
    if (f.t <= 16) return few_dx<1, true>(f, e, parts, part, st);
    return few_dx<2, true>(f, e, parts, part, st);
  }
  if (f.t <= 16) return few_dx<1, false>(f, e, parts, part, st);
  return f.t <= 32 ? few_dx<2, false>(f, e, parts, part, st) : few_dx<4, false>(f, e, parts, part, st);
}

hipError_t launch_few_dxsum(const XentDxSum& s, hipStream_t st) {
  k_few_dxsum<<<dim3(dxsum_blocks(s)), dim3(256), 0, st>>>(s);
  return hipGetLastError();
}

hipError_t launch_few_dw(const XentFew& f, const XentDw& d, const XentDxSum& sum, bool f32, hipStream_t st) {
  if (f32) return few_dw<1, true>(f, d, sum, st);
  return f.tp <= 32 ? few_dw<1, false>(f, d, sum, st) : few_dw<2, false>(f, d, sum, st);
}

}  // namespace dion
