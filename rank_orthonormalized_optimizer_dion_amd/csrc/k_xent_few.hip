// Cross entropy of few tokens (up to 64 in bfloat16, 128 in float32): reading
// W once per product, and writing dW, is what it costs, in any type and at any
// alignment.  All products run on the bfloat16 matrix cores with operands that
// come straight from global memory into registers:
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
#include "xent_device.h"
#include "xent_types.h"

namespace dion {

namespace {

// 16 bytes at any alignment of the element type (global memory takes vector
// accesses at any address).
template <class V, class T>
__device__ __forceinline__ V load_any(const T* p) {
  V v;
  __builtin_memcpy(&v, p, sizeof(V));
  return v;
}

// Eight values as the operands of their planes.
template <int PL>
struct Planes8 {
  u32x4 p[PL];
};
__device__ __forceinline__ Planes8<3> split8(const float (&v)[8]) {
  Planes8<3> o;
  float rest[8];
  uint16_t h[8];
#pragma unroll
  for (int pl = 0; pl < 3; ++pl) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = pinned(pl == 0 ? v[k] : rest[k]);
      h[k] = pl == 0 ? first_plane(x) : to_bf16(x);
      rest[k] = x - bf16_to_f32(h[k]);
    }
    o.p[pl] = pack8(h);
  }
  return o;
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

// Sixteen consecutive elements from column c of a row of k, as two operands;
// elements past the row are zero.  TAIL: the row may end inside.
template <bool F32, bool TAIL>
__device__ __forceinline__ void load16(const void* row, int c, int k, Planes8<F32 ? 3 : 1> (&o)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c0 = c + 8 * h;
    if constexpr (F32) {
      const float* p = static_cast<const float*>(row) + c0;
      float v[8];
      if (!TAIL || c0 + 8 <= k) {
        const f32x4 lo = load_any<f32x4>(p), hi = load_any<f32x4>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = lo[i];
          v[4 + i] = hi[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c0 + i < k ? p[i] : 0.0f;
      }
      o[h] = split8(v);
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(row) + c0;
      if (!TAIL || c0 + 8 <= k) {
        o[h].p[0] = load_any<u32x4>(p);
      } else {
        uint16_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c0 + i < k ? p[i] : 0;
        o[h].p[0] = pack8(v);
      }
    }
  }
}

// z for 16 rows of W at a time, its statistics or dz.  RAW: x is read as it
// is, like W (one block of 16 tokens), else from planes whose rows are
// readable, and zero past k, up to f.kx columns.
template <int TB, bool F32, bool RAW, bool GRAD>
__global__ __launch_bounds__(512) void k_few_z(XentFew f, XentEpi e) {
  constexpr int P = F32 ? 3 : 1, ES = F32 ? 4 : 2;
  constexpr int B = (TB + 1) / 2;   // 512 threads hold 32 tokens by 16 columns
  __shared__ float red[8][TB][16][17];
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
  const int groups = GRAD ? static_cast<int>(e.pitch / kXentGroup) : (f.n + kXentGroup - 1) / kXentGroup;
  for (int g = blockIdx.x; g < groups; g += gridDim.x) {
    const int n0 = g * kXentGroup, col = n0 + c;
    const char* wr = static_cast<const char*>(f.w) + min(n0 + (lane & 15), f.n - 1) * f.ldw * ES;
    f32x4 acc[TB];
#pragma unroll
    for (int b = 0; b < TB; ++b) acc[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // 64 elements of the reduction: 16 per lane
    const auto piece = [&](auto tail, int k0) {
      constexpr bool TAIL = decltype(tail)::value;
      const int k = k0 + 16 * (lane >> 4);
      Planes8<P> w[2], x[TB][2];
      load16<F32, TAIL>(wr, k, f.k, w);
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        if constexpr (RAW) {
          load16<F32, TAIL>(xr[b], k, f.k, x[b]);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int pl = 0; pl < P; ++pl)
              x[b][h].p[pl] = !TAIL || k + 8 * h < f.kx
                                  ? *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(xr[b]) + pl * f.xplane + k + 8 * h)
                                  : u32x4{0, 0, 0, 0};
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < TB; ++b) acc[b] = mfma_planes(w[h], x[b][h], acc[b]);
    };
    int k0 = 64 * wave;
    constexpr int U = F32 || TB > 2 ? 2 : 4;   // pieces in flight
#pragma unroll U
    for (; k0 + 64 <= f.k; k0 += 64 * 8) piece(std::false_type{}, k0);
    if (k0 < f.k) piece(std::true_type{}, k0);
    // lane l, register i: row 4 (l / 16) + i of W, token l % 16
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[wave][b][lane & 15][4 * (lane >> 4) + i] = acc[b][i];
    __syncthreads();
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int token = 32 * b + (threadIdx.x >> 4);
      float z = 0.0f;
      if (token < 16 * TB) {
#pragma unroll
        for (int s = 0; s < 8; ++s) z += red[s][token >> 4][token & 15][c];
      }
      if constexpr (GRAD) {
        float v[1] = {dz_of(z, r[b].lse, r[b].a, r[b].b, r[b].mask)};
        if (y[b] == e.j0 + col) v[0] -= r[b].c;
        if (col >= f.n || token >= f.t) v[0] = 0.0f;
        if (token < f.tp) {   // dz by rows, and transposed with its tokens padded by zeros
          float rest = v[0];
          for (int pl = 0; pl < e.planes; ++pl) {
            const float u = pinned(rest);
            const uint16_t h = pl == 0 ? first_plane(u) : to_bf16(u);
            rest = u - bf16_to_f32(h);
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

// Planes of x (zero past its columns) and of its transpose (tokens padded by
// zeros to f.tp), 64 columns per workgroup.
template <bool F32>
__global__ __launch_bounds__(256) void k_few_prep(XentPrep a) {
  constexpr int P = F32 ? 3 : 1;
  __shared__ float tile[64][129];
  const int c0 = blockIdx.x * 64;
  for (int i = threadIdx.x; i < a.tp * 64; i += 256) {
    const int token = i >> 6, c = i & 63;
    const bool in = token < a.t && c0 + c < a.k;
    float v = in ? load_value(a.x, token * a.ldx + c0 + c, !F32) : 0.0f;
    tile[c][token] = v;
    if (a.xp && token < a.t) {
      for (int pl = 0; pl < P; ++pl) {
        const float u = pinned(v);
        const uint16_t h = pl == 0 && P > 1 ? first_plane(u) : to_bf16(u);
        v = u - bf16_to_f32(h);
        a.xp[pl * a.xplane + token * a.ldp + c0 + c] = h;
      }
    }
  }
  if (!a.xt) return;
  __syncthreads();
  for (int i = threadIdx.x; i < a.tp * 64; i += 256) {
    const int token = i % a.tp, c = i / a.tp;
    if (c0 + c >= a.k) continue;
    float v = tile[c][token];
    for (int pl = 0; pl < P; ++pl) {
      const float u = pinned(v);
      const uint16_t h = pl == 0 && P > 1 ? first_plane(u) : to_bf16(u);
      v = u - bf16_to_f32(h);
      a.xt[pl * a.xtplane + static_cast<int64_t>(c0 + c) * a.tp + token] = h;
    }
  }
}

// dx's sums over every `gridDim.y`-th block of 4 x 32 rows of W, for 16
// times CW columns.
template <int TB, bool F32>
__global__ __launch_bounds__(256) void k_few_dx(XentFew f, const uint16_t* dz, int64_t pitch, int64_t plane, float* part) {
  constexpr int CW = F32 ? 4 : 8, PW = F32 ? 3 : 1, PZ = F32 ? 3 : 2;
  using T = typename std::conditional<F32, float, uint16_t>::type;
  __shared__ float red[2][CW * TB * 4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = (blockIdx.x * 16 + (lane & 15)) * CW;
  const int steps = (f.n + 31) / 32;
  f32x4 acc[CW][TB];
#pragma unroll
  for (int m = 0; m < CW; ++m)
#pragma unroll
    for (int b = 0; b < TB; ++b) acc[m][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const uint16_t* zr[TB];
#pragma unroll
  for (int b = 0; b < TB; ++b) zr[b] = dz + min(16 * b + (lane & 15), f.t - 1) * pitch + 8 * (lane >> 4);
  const bool whole = c + CW <= f.k;
#pragma unroll 2
  for (int s = blockIdx.y * 4 + wave; s < steps; s += 4 * gridDim.y) {
    const int j0 = 32 * s + 8 * (lane >> 4);
    u32x4 w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const T* p = static_cast<const T*>(f.w) + min(j0 + i, f.n - 1) * f.ldw + c;
      if (whole) {
        w[i] = load_any<u32x4>(p);
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

// dx from the partial sums, in order.
__global__ __launch_bounds__(256) void k_few_dxsum(const float* part, int parts, int t, int k, void* dx, int64_t lddx,
                                                   int dtype) {
  const int64_t size = static_cast<int64_t>(t) * k, i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= size) return;
  float s = 0.0f;
#pragma unroll 8
  for (int p = 0; p < parts; ++p) s += part[p * size + i];
  const int64_t row = i / k;
  store_value(dx, row * lddx + (i - row * k), dtype, s);
}

// dW: a wavefront's 16 RJ rows by the columns of its part, 64 at a time.
template <int TT, bool F32>
__global__ __launch_bounds__(256) void k_few_dw(XentFew f, XentDw d) {
  constexpr int PX = F32 ? 3 : 1, PZ = F32 ? 3 : 2, RJ = kFewDwRows / 16 / (TT == 4 ? 2 : 1);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int j0 = (blockIdx.x * 4 + wave) * 16 * RJ;
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
  for (int c0 = blockIdx.y * d.cols; c0 < min(f.k, (static_cast<int>(blockIdx.y) + 1) * d.cols); c0 += 64) {
    f32x4 acc[4][RJ];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      // the operand's row r is column 16 (r / 4) + 4 m + r % 4: a lane's outputs
      // are then 16 consecutive columns
      const int64_t c = min(c0 + 16 * (r >> 2) + 4 * m + (r & 3), f.k - 1);
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
    const int c = c0 + 16 * (lane >> 4);
#pragma unroll
    for (int q = 0; q < RJ; ++q) {
      const int j = j0 + 16 * q + r;
      if (j >= f.n) continue;
      const int64_t at = j * d.ld + c;
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = acc[i / 4][q][i % 4];
      if (c + 16 <= f.k) {
        if constexpr (F32) {
          float* p = static_cast<float*>(d.dw) + at;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f32x4 u = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
            if (d.accumulate) u += load_any<f32x4>(p + 4 * i);
            __builtin_memcpy(p + 4 * i, &u, 16);
          }
        } else {
          uint16_t* p = static_cast<uint16_t*>(d.dw) + at;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint16_t h[8], old[8];
            if (d.accumulate) __builtin_memcpy(old, p + 8 * i, 16);
#pragma unroll
            for (int k = 0; k < 8; ++k) h[k] = to_bf16(d.accumulate ? v[8 * i + k] + bf16_to_f32(old[k]) : v[8 * i + k]);
            const u32x4 u = pack8(h);
            __builtin_memcpy(p + 8 * i, &u, 16);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (c + i < f.k) store_value(d.dw, at + i, !F32, d.accumulate ? v[i] + load_value(d.dw, at + i, !F32) : v[i]);
      }
    }
  }
}

template <int TB, bool F32>
hipError_t few_z(const XentFew& f, const XentEpi& e, bool grad, bool raw, int groups, hipStream_t st) {
  const dim3 grid(groups), block(512);
  if (grad) {
    k_few_z<TB, F32, false, true><<<grid, block, 0, st>>>(f, e);
  } else if constexpr (TB == 1) {
    if (raw) k_few_z<TB, F32, true, false><<<grid, block, 0, st>>>(f, e);
    else k_few_z<TB, F32, false, false><<<grid, block, 0, st>>>(f, e);
  } else {
    k_few_z<TB, F32, false, false><<<grid, block, 0, st>>>(f, e);
  }
  return hipGetLastError();
}

template <int TB, bool F32>
hipError_t few_dx(const XentFew& f, const XentEpi& e, int parts, float* part, hipStream_t st) {
  constexpr int cols = 16 * (F32 ? 4 : 8);
  k_few_dx<TB, F32><<<dim3((f.k + cols - 1) / cols, parts), dim3(256), 0, st>>>(f, e.dz, e.pitch, e.plane, part);
  return hipGetLastError();
}

template <int TT, bool F32>
hipError_t few_dw(const XentFew& f, const XentDw& d, hipStream_t st) {
  constexpr int rows = 4 * kFewDwRows / (TT == 4 ? 2 : 1);
  k_few_dw<TT, F32><<<dim3((f.n + rows - 1) / rows, (f.k + d.cols - 1) / d.cols), dim3(256), 0, st>>>(f, d);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_few_prep(const XentPrep& a, bool f32, hipStream_t st) {
  const dim3 grid((a.k + 63) / 64), block(256);
  if (f32) k_few_prep<true><<<grid, block, 0, st>>>(a);
  else k_few_prep<false><<<grid, block, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_few_z(const XentFew& f, const XentEpi& e, bool f32, bool grad, bool raw, int groups, hipStream_t st) {
  if (f32) {
    if (f.t <= 16) return few_z<1, true>(f, e, grad, raw, groups, st);
    if (f.t <= 32) return few_z<2, true>(f, e, grad, raw, groups, st);
    return f.t <= 64 ? few_z<4, true>(f, e, grad, raw, groups, st) : few_z<8, true>(f, e, grad, raw, groups, st);
  }
  if (f.t <= 16) return few_z<1, false>(f, e, grad, raw, groups, st);
  return f.t <= 32 ? few_z<2, false>(f, e, grad, raw, groups, st) : few_z<4, false>(f, e, grad, raw, groups, st);
}

hipError_t launch_few_dx(const XentFew& f, const XentEpi& e, bool f32, int parts, float* part, hipStream_t st) {
  if (f32) {
    if (f.t <= 16) return few_dx<1, true>(f, e, parts, part, st);
    if (f.t <= 32) return few_dx<2, true>(f, e, parts, part, st);
    return f.t <= 64 ? few_dx<4, true>(f, e, parts, part, st) : few_dx<8, true>(f, e, parts, part, st);
  }
  if (f.t <= 16) return few_dx<1, false>(f, e, parts, part, st);
  return f.t <= 32 ? few_dx<2, false>(f, e, parts, part, st) : few_dx<4, false>(f, e, parts, part, st);
}

hipError_t launch_few_dxsum(const XentFew& f, const float* part, int parts, void* dx, int64_t lddx, int dtype,
                            hipStream_t st) {
  const int64_t size = static_cast<int64_t>(f.t) * f.k;
  k_few_dxsum<<<dim3(static_cast<unsigned>((size + 255) / 256)), dim3(256), 0, st>>>(part, parts, f.t, f.k, dx, lddx, dtype);
  return hipGetLastError();
}

hipError_t launch_few_dw(const XentFew& f, const XentDw& d, bool f32, hipStream_t st) {
  if (f32) {
    if (f.tp <= 32) return few_dw<1, true>(f, d, st);
    return f.tp <= 64 ? few_dw<2, true>(f, d, st) : few_dw<4, true>(f, d, st);
  }
  return f.tp <= 32 ? few_dw<1, false>(f, d, st) : few_dw<2, false>(f, d, st);
}

}  // namespace dion
