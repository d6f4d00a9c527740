// The linear layer on the bfloat16 matrix cores: the kernels behind
// dion_linear_forward and dion_linear_backward.
//
//   z = x W^T + b,  y = act(z) + residual           k_lin_mm (forward)
//   dz = dy act'(z),  db = sum over tokens of dz    k_lin_pack, k_lin_colsum
//   dx = dz W,  dW = dz^T x                         k_lin_mm
//
// bfloat16 tensors are read as they are: forward, dx and dW differ in which
// side of each operand the reduction runs along, and the x-major tiles are
// transposed on their way out of LDS (mm16.h), so no transposed copy of an
// activation or a weight is ever written.  float32 tensors are first split
// three ways into bfloat16 planes (24 bits) and multiplied as six plane
// products: float32's accuracy for values from 2^-110 up to the largest
// (below, the planes end at 2^-133).
//
// Bound and measured (MI355X): large batches by the matrix cores (8192
// tokens, 8192 -> 3072 with GELU, bias and residual: 432 us, 0.95 PFLOP/s; the
// backward of 3072 -> 8192: 0.93 ms, 0.89 PFLOP/s), one token by streaming W
// (3072 -> 8192: 11.9 us, 4.2 TB/s), float32 by the six products of its split
// planes (1021 tokens, 773 -> 2051, backward: 133 us) and, with few tokens, by
// writing and sweeping the weight's planes (9 tokens, 3072 -> 8192: 101 us; 8
// tokens without them: 52 us).
#include "dion.h"
#include "linear_types.h"
#include "mm16.h"
#include "work16.h"

namespace dion {

namespace {

// Phi(z), the normal distribution function, without the cancellation of
// (1 + erf) / 2: that form is 4% off at z = -5 and zero from z = -5.5 on.
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(-0.70710678118654752f * z); }

__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case DION_ACT_RELU: return z > 0.0f || z != z ? z : 0.0f;
    case DION_ACT_RELU2: return z > 0.0f || z != z ? z * z : 0.0f;
    case DION_ACT_GELU: return z * normal_cdf(z);
    case DION_ACT_SILU: return z / (1.0f + expf(-z));
    default: return z;
  }
}

__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case DION_ACT_RELU: return z > 0.0f ? 1.0f : z != z ? z : 0.0f;
    case DION_ACT_RELU2: return z > 0.0f || z != z ? 2.0f * z : 0.0f;
    case DION_ACT_GELU:
      return normal_cdf(z) + z * 0.39894228040143268f * expf(-0.5f * z * z);
    case DION_ACT_SILU: {
      const float s = 1.0f / (1.0f + expf(-z));
      return s * (1.0f + z * (1.0f - s));
    }
    default: return 1.0f;
  }
}

__device__ __forceinline__ float load_value(const void* p, int64_t o, int dtype) {
  return dtype ? bf16_to_f32(static_cast<const uint16_t*>(p)[o]) : static_cast<const float*>(p)[o];
}
__device__ __forceinline__ void store_value(void* p, int64_t o, int dtype, float v) {
  if (dtype) static_cast<uint16_t*>(p)[o] = to_bf16(v);
  else static_cast<float*>(p)[o] = v;
}

// Eight consecutive values, as vectors where the address allows.
__device__ __forceinline__ bool aligned16(const void* p, int64_t ld, int dtype) {
  return (reinterpret_cast<uint64_t>(p) & 15) == 0 && ld % (dtype ? 8 : 4) == 0;
}
__device__ __forceinline__ void load8(const void* p, int64_t o, int dtype, bool vec, int left, float (&v)[8]) {
  if (vec && left >= 8) {
    if (dtype) {
      const u32x4 u = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + o);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(u[k] << 16);
        v[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
      }
    } else {
      const float* q = static_cast<const float*>(p) + o;
      const f32x4 a = *reinterpret_cast<const f32x4*>(q), b = *reinterpret_cast<const f32x4*>(q + 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = a[k];
        v[4 + k] = b[k];
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < left ? load_value(p, o + k, dtype) : 0.0f;
  }
}
__device__ __forceinline__ void store8(void* p, int64_t o, int dtype, bool vec, int left, const float (&v)[8]) {
  if (vec && left >= 8) {
    if (dtype) {
      uint16_t h[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) h[k] = to_bf16(v[k]);
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + o) = pack8(h);
    } else {
      float* q = static_cast<float*>(p) + o;
      *reinterpret_cast<f32x4*>(q) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(q + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) store_value(p, o + k, dtype, v[k]);
  }
}

// What a run of 8 outputs (row, col .. col + 7) adds to the activation or
// to the product: the residual, or the old output when accumulating.
struct LinPre {
  float w[8];
};
__device__ __forceinline__ LinPre lin_fetch(const LinOut& o, int row, int col, int left) {
  LinPre p{};
  const void* src = o.accumulate ? o.y : o.residual;
  const int64_t ld = o.accumulate ? o.ldy : o.ldr;
  if (src) load8(src, row * ld + col, o.dtype, aligned16(src, ld, o.dtype), left, p.w);
  return p;
}

// The epilogue of such a run.  ACT: the activation, or -1 for o.act.
template <int ACT>
__device__ __forceinline__ void lin_out(const LinOut& o, int row, int col, int left, const float (&acc)[8],
                                        const LinPre& pre) {
  const int act = ACT < 0 ? o.act : ACT;
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = acc[k];
  if (o.bias) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) v[k] += o.bias[col + k];
  }
  if (o.z) store8(o.z, row * o.ldz + col, o.dtype, aligned16(o.z, o.ldz, o.dtype), left, v);
  if (act != DION_ACT_NONE) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = act_value(v[k], act);
  }
  if (o.residual || o.accumulate) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += pre.w[k];
  }
  store8(o.y, row * o.ldy + col, o.dtype, aligned16(o.y, o.ldy, o.dtype), left, v);
}

// Plane pairs of the reduction's segments, one hexadecimal digit per segment:
// looked up without a branch, which would cut the product's loop into pieces
// that the scheduler cannot fill (float32 backward, 1021 tokens, 2051 x 773: 144 to 133 us).
struct Pairs {
  uint32_t a, b;
};
__device__ __forceinline__ Pairs plane_pairs(int nseg) {
  // six: x = hi + mid + lo; (mid mid) (lo hi) (hi lo) (mid hi) (hi mid)
  // (hi hi), smallest first; the dropped pairs are below 3 2^-24 of the
  // product.  two: lo, then hi of A.  one: plane 0.
  return nseg == 6 ? Pairs{0x001021u, 0x010201u} : nseg == 2 ? Pairs{0x01u, 0u} : Pairs{0u, 0u};
}

template <int TILE, int ST, LinKind KIND>
using LinShape = Shape16<B16, TILE, TILE, TILE / 64, 2, ST, 1, KIND == kLinDw, KIND != kLinForward>;

template <int TILE, int ST, LinKind KIND, int ACT>
__global__ __launch_bounds__(2 * TILE) void k_lin_mm(LinProduct p) {
  using S = LinShape<TILE, ST, KIND>;
  __shared__ u32x4 smem[S::LDS_CELLS];
  const Work16 work{p.full, p.tx * p.ty - p.full, p.slices, p.part, p.count};
  const Item16 it = item16(work, xcd_item(blockIdx.x, gridDim.x));
  int ti, tj;
  tile_order(it.tile, p.tx, p.ty, ti, tj);
  const int r0 = ti * TILE, c0 = tj * TILE;
  int kbeg, kend;
  slice16<S>(it, p.K, kbeg, kend);
  typename S::Acc acc[S::FM][S::FN];
  typename S::A ta;
  typename S::B tb;
  ta.init(p.lda, r0, p.M);
  tb.init(p.ldb, c0, p.N);
  const Pairs pairs = plane_pairs(p.nseg);
  tile_product<S>(ta, tb, Planes16{p.a, p.b, p.sa, p.sb}, p.nseg,
                  [pairs](int i, int& a, int& b) {
                    a = (pairs.a >> (4 * i)) & 15;
                    b = (pairs.b >> (4 * i)) & 15;
                  },
                  kbeg, kend, smem, acc);
  if (!join16<S>(work, it, smem, acc)) return;
  tile_runs<S, false>(
      acc, smem,
      [&](int r, int q) {
        const int row = r0 + r, col = c0 + q;
        return row < p.M && col < p.N ? lin_fetch(p.out, row, col, p.N - col) : LinPre{};
      },
      [&](int r, int q, const float (&v)[8], const LinPre& pre) {
        const int row = r0 + r, col = c0 + q;
        if (row < p.M && col < p.N) lin_out<ACT>(p.out, row, col, p.N - col, v, pre);
      });
}

// The first of several planes of x.  A finite x above bfloat16's largest
// number would round to infinity and leave -infinity for the next plane; it
// is cut off instead (float32's largest and bfloat16's share the exponent),
// which leaves a remainder of 16 bits that two planes hold exactly.
__device__ __forceinline__ uint16_t first_plane(float x) {
  const uint16_t h = to_bf16(x);
  const uint32_t b = __float_as_uint(x);
  return (h & 0x7fff) == 0x7f80 && (b & 0x7fffffffu) < 0x7f800000u ? static_cast<uint16_t>(b >> 16) : h;
}

// dz = src act'(z) (or src itself) as planes, zero past its columns and rows,
// and its column sums over this workgroup's `chunk` rows.  256 columns by 8
// row lanes per workgroup.
__device__ __forceinline__ void pack_block(const LinPack& p, int block, float (&red)[8][256 + 8]) {
  const int bx = block % p.gx, by = block / p.gx;
  const int col = (bx * 32 + (threadIdx.x & 31)) * 8;
  const int lane = threadIdx.x >> 5;
  const int64_t r0 = static_cast<int64_t>(by) * p.chunk;
  const int64_t r1 = min(p.prows, r0 + p.chunk);
  const bool vs = aligned16(p.src, p.ld, p.dtype), vz = aligned16(p.z, p.ldz, p.dtype);
  const int left = p.cols - col;
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (col < (p.dst ? p.pitch : p.cols)) {
    for (int64_t r = r0 + lane; r < r1; r += 8) {
      const int in = r < p.rows ? left : 0;   // rows past the last are zero
      float v[8];
      load8(p.src, r * p.ld + col, p.dtype, vs, in, v);
      if (p.z) {
        float z[8];
        load8(p.z, r * p.ldz + col, p.dtype, vz, in, z);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= k < in ? act_slope(z[k], p.act) : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] += v[k];
      if (p.dst) {
        uint16_t* at = p.dst + r * p.pitch + col;
        uint16_t h[8];
        float rest[8];
        for (int pl = 0; pl < p.planes; ++pl) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float x = pinned(pl == 0 ? v[k] : rest[k]);
            h[k] = pl == 0 && p.planes > 1 ? first_plane(x) : to_bf16(x);
            rest[k] = x - bf16_to_f32(h[k]);
          }
          *reinterpret_cast<u32x4*>(at + pl * p.plane) = pack8(h);
        }
      }
    }
  }
  if (!p.sums) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) red[lane][(threadIdx.x & 31) * 8 + k] = sum[k];
  __syncthreads();
  const int c = bx * 256 + threadIdx.x;
  if (c < p.cols) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i][threadIdx.x];
    p.sums[static_cast<int64_t>(by) * p.cols + c] = s;
  }
}

__global__ __launch_bounds__(256) void k_lin_pack(LinPacks a) {
  __shared__ float red[8][256 + 8];
  int b = blockIdx.x;
  if (b == 0)
    for (int i = threadIdx.x; i < a.counts; i += 256) a.count[i] = 0;
#pragma unroll
  for (int i = 0; i < kLinPacks; ++i) {
    if (i < a.n && b >= 0 && b < a.p[i].blocks) pack_block(a.p[i], b, red);
    b -= i < a.n ? a.p[i].blocks : 0;
  }
}

// The sum of the chunks' column sums: 32 columns by 8 lanes of chunks.
__global__ __launch_bounds__(256) void k_lin_colsum(const float* part, int chunks, int n, float* out,
                                                    int accumulate) {
  __shared__ float red[8][32];
  const int col = threadIdx.x & 31, lane = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + col;
  float s = 0.0f;
  if (c < n) {
#pragma unroll 8
    for (int i = lane; i < chunks; i += 8) s += part[static_cast<int64_t>(i) * n + c];
  }
  red[lane][col] = s;
  __syncthreads();
  if (lane != 0 || c >= n) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += red[i][col];
  out[c] = accumulate ? out[c] + s : s;
}

// Few tokens (t <= 16 TB), bfloat16: the weight is read once and that is
// the cost.  A workgroup owns 16 rows of W, its 8 wavefronts take turns at
// 64-element pieces of the reduction (a lane reads 32 consecutive bytes of
// its row, the two halves feeding two matrix instructions in the same k
// order for x), and their sums meet in LDS.
template <int TB>
__global__ __launch_bounds__(512) void k_lin_skinny(LinSkinny p) {
  __shared__ float red[8][TB][16][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = blockIdx.x * 16;
  const int row = min(n0 + (lane & 15), p.n - 1);
  const uint16_t* w = static_cast<const uint16_t*>(p.w) + row * p.ldw + 16 * (lane >> 4);
  const uint16_t* x[TB];
#pragma unroll
  for (int b = 0; b < TB; ++b)
    x[b] = static_cast<const uint16_t*>(p.x) + min(16 * b + (lane & 15), p.t - 1) * p.ldx + 16 * (lane >> 4);
  f32x4 acc[TB];
#pragma unroll
  for (int b = 0; b < TB; ++b) acc[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto step = [&](const u32x4 (&a)[2], const u32x4 (&v)[TB][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = 0; b < TB; ++b)
        acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[h]),
                                                         __builtin_bit_cast(bf16x8, v[b][h]), acc[b], 0, 0, 0);
  };
  constexpr int U = TB <= 2 ? 4 : 2;   // pieces in flight
  int k = 64 * wave;
  for (; k + 64 * 8 * (U - 1) + 64 <= p.k; k += 64 * 8 * U) {
    u32x4 a[U][2], v[U][TB][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        a[u][h] = *reinterpret_cast<const u32x4*>(w + k + 512 * u + 8 * h);
#pragma unroll
        for (int b = 0; b < TB; ++b) v[u][b][h] = *reinterpret_cast<const u32x4*>(x[b] + k + 512 * u + 8 * h);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) step(a[u], v[u]);
  }
  for (; k < p.k; k += 64 * 8) {
    u32x4 a[2], v[TB][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = k + 16 * (lane >> 4) + 8 * h < p.k;
      a[h] = in ? *reinterpret_cast<const u32x4*>(w + k + 8 * h) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int b = 0; b < TB; ++b) v[b][h] = in ? *reinterpret_cast<const u32x4*>(x[b] + k + 8 * h) : u32x4{0, 0, 0, 0};
    }
    step(a, v);
  }
  // 16 x 16 output: lane l, register i holds row 4 (l / 16) + i (of W),
  // column l % 16 (token)
#pragma unroll
  for (int b = 0; b < TB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][b][lane & 15][4 * (lane >> 4) + i] = acc[b][i];
  __syncthreads();
  // 16 TB tokens x 2 runs of 8 outputs
  for (int e = threadIdx.x; e < TB * 32; e += 512) {
    const int token = e >> 1, c = 8 * (e & 1);
    if (token >= p.t || n0 + c >= p.n) continue;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.0f;
#pragma unroll
      for (int s = 0; s < 8; ++s) v[i] += red[s][token >> 4][token & 15][c + i];
    }
    lin_out<-1>(p.out, token, n0 + c, p.n - n0 - c, v, lin_fetch(p.out, token, n0 + c, p.n - n0 - c));
  }
}

// Few tokens in float32, or bfloat16 rows that are not 16-byte aligned: a
// wavefront per output row, float32 multiply-adds over the lanes.
template <int T, bool BF, bool VEC>
__global__ __launch_bounds__(256) void k_lin_rows(LinSkinny p) {
  constexpr int V = VEC ? (BF ? 8 : 4) : 1;
  const int lane = threadIdx.x & 63;
  const int n = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (n >= p.n) return;
  float acc[T];
#pragma unroll
  for (int i = 0; i < T; ++i) acc[i] = 0.0f;
  auto get = [&](const void* base, int64_t o, float (&v)[8]) {
    if constexpr (VEC && BF) {
      const u32x4 u = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + o);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(u[k] << 16);
        v[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
      }
    } else if constexpr (VEC) {
      const f32x4 u = *reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + o);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = u[k];
    } else {
      v[0] = load_value(base, o, BF);
    }
  };
#pragma unroll 4
  for (int k = V * lane; k < p.k; k += 64 * V) {
    float a[8], v[8];
    get(p.w, n * p.ldw + k, a);
#pragma unroll
    for (int i = 0; i < T; ++i) {
      get(p.x, min(i, p.t - 1) * p.ldx + k, v);
#pragma unroll
      for (int j = 0; j < V; ++j) acc[i] = fmaf(a[j], v[j], acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < T; ++i) {
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) acc[i] += __shfl_xor(acc[i], s);
  }
#pragma unroll
  for (int i = 0; i < T; ++i)
    if (lane == i && i < p.t) {
      const float v[8] = {acc[i], 0, 0, 0, 0, 0, 0, 0};
      lin_out<-1>(p.out, i, n, 1, v, lin_fetch(p.out, i, n, 1));
    }
}

template <int TILE, int ST, LinKind KIND, int ACT>
hipError_t product(const LinProduct& p, hipStream_t st) {
  k_lin_mm<TILE, ST, KIND, ACT><<<dim3(p.items), dim3(2 * TILE), 0, st>>>(p);
  return hipGetLastError();
}

template <int TILE, int ST>
hipError_t product(const LinProduct& p, LinKind kind, hipStream_t st) {
  if (kind == kLinDx) return product<TILE, ST, kLinDx, DION_ACT_NONE>(p, st);
  if (kind == kLinDw) return product<TILE, ST, kLinDw, DION_ACT_NONE>(p, st);
  switch (p.out.act) {
    case DION_ACT_RELU: return product<TILE, ST, kLinForward, DION_ACT_RELU>(p, st);
    case DION_ACT_RELU2: return product<TILE, ST, kLinForward, DION_ACT_RELU2>(p, st);
    case DION_ACT_GELU: return product<TILE, ST, kLinForward, DION_ACT_GELU>(p, st);
    case DION_ACT_SILU: return product<TILE, ST, kLinForward, DION_ACT_SILU>(p, st);
    default: return product<TILE, ST, kLinForward, DION_ACT_NONE>(p, st);
  }
}

template <int T>
hipError_t rows(const LinSkinny& p, bool vec, hipStream_t st) {
  const dim3 grid((p.n + 3) / 4), block(256);
  if (p.out.dtype) {
    if (vec) k_lin_rows<T, true, true><<<grid, block, 0, st>>>(p);
    else k_lin_rows<T, true, false><<<grid, block, 0, st>>>(p);
  } else {
    if (vec) k_lin_rows<T, false, true><<<grid, block, 0, st>>>(p);
    else k_lin_rows<T, false, false><<<grid, block, 0, st>>>(p);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lin_product(const LinProduct& p, LinKind kind, int tile, hipStream_t st) {
  if (tile == 256) return product<256, 4>(p, kind, st);
  return p.items <= kTileSlots256 ? product<128, 8>(p, kind, st) : product<128, 4>(p, kind, st);
}

hipError_t launch_lin_packs(const LinPacks& p, hipStream_t st) {
  int blocks = 0;
  for (int i = 0; i < p.n; ++i) blocks += p.p[i].blocks;
  k_lin_pack<<<dim3(blocks > 0 ? blocks : 1), dim3(256), 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_lin_colsum(const float* part, int chunks, int n, float* out, int accumulate, hipStream_t st) {
  k_lin_colsum<<<dim3((n + 31) / 32), dim3(256), 0, st>>>(part, chunks, n, out, accumulate);
  return hipGetLastError();
}

hipError_t launch_lin_skinny(const LinSkinny& p, hipStream_t st) {
  const dim3 grid((p.n + 15) / 16), block(512);
  if (p.t <= 16) k_lin_skinny<1><<<grid, block, 0, st>>>(p);
  else if (p.t <= 32) k_lin_skinny<2><<<grid, block, 0, st>>>(p);
  else k_lin_skinny<4><<<grid, block, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_lin_rows(const LinSkinny& p, bool vec, hipStream_t st) {
  if (p.t == 1) return rows<1>(p, vec, st);
  if (p.t <= 4) return rows<4>(p, vec, st);
  return rows<8>(p, vec, st);
}

}  // namespace dion
