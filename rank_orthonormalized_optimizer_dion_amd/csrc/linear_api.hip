// Host side of dion_linear_forward and dion_linear_backward: argument
// validation, workspace layout and schedule.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "dion.h"
#include "linear_types.h"
#include "work16.h"

#define DION_API extern "C" __attribute__((visibility("default")))

namespace dion {
namespace {

size_t lin_align(size_t x) { return (x + 255) / 256 * 256; }
int64_t lin_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
constexpr int64_t kLinMaxTokens = int64_t{1} << 24;
constexpr int64_t kLinMaxPitch = int64_t{1} << 30;
// Operands are read in place up to this pitch: the offsets inside a tile
// (256 rows) are 32-bit byte offsets.
constexpr int64_t kLinDirectPitch = int64_t{1} << 22;
// The dz of an activation is rounded to bfloat16 for the products; with few
// tokens it takes two planes (hi + lo) instead: its roundings average over
// too few terms there, and the products' time is the weights' traffic.
constexpr int kLinFewTokens = 64;
constexpr int64_t kLinBigTiles = 256;   // 256 x 256 tiles in a product of at least this many

struct Span {
  const void* p;
  int64_t rows, cols, ld;
  int64_t esize;
  bool misplaced() const { return reinterpret_cast<uintptr_t>(p) % esize != 0; }
  size_t bytes() const { return rows > 0 ? static_cast<size_t>(((rows - 1) * ld + cols) * esize) : 0; }
};

bool lin_overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes() && y < x + a.bytes();
}

bool span_ok(const Span& s, bool required) {
  if (!s.p) return !required || s.rows == 0;
  return s.ld >= s.cols && s.ld <= kLinMaxPitch && !s.misplaced();
}

struct LinCall {
  dion_linear a;
  int64_t e;   // element size
  Span x, w, bias, res, y, z, dy, dx, dw, db;
};

bool lin_common(const dion_linear* l, LinCall& c) {
  if (!l) return false;
  c.a = *l;
  if (l->t < 0 || l->t > kLinMaxTokens || l->n < 1 || l->k < 1 || l->n > DION_MAX_DIM || l->k > DION_MAX_DIM)
    return false;
  if (l->dtype != DION_DTYPE_F32 && l->dtype != DION_DTYPE_BF16) return false;
  if (l->act < DION_ACT_NONE || l->act > DION_ACT_SILU) return false;
  c.e = l->dtype == DION_DTYPE_BF16 ? 2 : 4;
  c.x = {l->x, l->t, l->k, l->ldx, c.e};
  c.w = {l->w, l->n, l->k, l->ldw, c.e};
  c.bias = {l->bias, 1, l->n, l->n, 4};
  c.res = {l->residual, l->t, l->n, l->ldr, c.e};
  c.y = {l->y, l->t, l->n, l->ldy, c.e};
  c.z = {l->z, l->t, l->n, l->ldz, c.e};
  c.dy = {l->dy, l->t, l->n, l->lddy, c.e};
  c.dx = {l->dx, l->t, l->k, l->lddx, c.e};
  c.dw = {l->dw, l->n, l->k, l->lddw, c.e};
  c.db = {l->db, 1, l->n, l->n, 4};
  return true;
}

bool lin_forward_ok(const dion_linear* l, LinCall& c) {
  if (!lin_common(l, c)) return false;
  if (!span_ok(c.x, true) || !span_ok(c.w, true) || !span_ok(c.y, true) || !span_ok(c.res, false) ||
      !span_ok(c.z, false) || !span_ok(c.bias, false))
    return false;
  for (const Span* in : {&c.x, &c.w, &c.bias})
    if (lin_overlap(*in, c.y) || lin_overlap(*in, c.z)) return false;
  if (lin_overlap(c.y, c.z) || lin_overlap(c.res, c.z)) return false;
  // y may be the residual itself (added in place), not a shifted view of it
  if (lin_overlap(c.res, c.y) && !(c.res.p == c.y.p && c.res.ld == c.y.ld)) return false;
  return true;
}

bool lin_backward_ok(const dion_linear* l, LinCall& c) {
  if (!lin_common(l, c)) return false;
  if (!span_ok(c.dy, true) || !span_ok(c.dx, false) || !span_ok(c.dw, false) || !span_ok(c.db, false)) return false;
  if (!span_ok(c.x, c.dw.p != nullptr) || !span_ok(c.w, c.dx.p != nullptr)) return false;
  if (!span_ok(c.z, l->act != DION_ACT_NONE)) return false;
  const Span* outs[] = {&c.dx, &c.dw, &c.db};
  for (int i = 0; i < 3; ++i) {
    for (const Span* in : {&c.dy, &c.z, &c.x, &c.w})
      if (lin_overlap(*in, *outs[i])) return false;
    for (int j = 0; j < i; ++j)
      if (lin_overlap(*outs[i], *outs[j])) return false;
  }
  return true;
}

// Whether a bfloat16 operand can feed the tiles in place: whole 16-byte
// cells in every row.
bool lin_direct(const Span& s) {
  return s.esize == 2 && reinterpret_cast<uintptr_t>(s.p) % 16 == 0 && s.ld % 8 == 0 && s.cols % 8 == 0 &&
         s.ld <= kLinDirectPitch;
}

// A bump allocator over the workspace; with a null base it only counts.
struct Arena {
  char* base;
  size_t used = 0;
  template <class T>
  T* take(size_t count) {
    T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
    used += lin_align(count * sizeof(T));
    return p;
  }
};

#define LIN_TRY(expr)             \
  do {                            \
    const hipError_t e_ = (expr); \
    if (e_ != hipSuccess) return e_; \
  } while (0)

// Operand planes: the caller's tensor itself, or a padded copy.
struct Operand {
  const uint16_t* p;
  int64_t ld, plane;
};

struct Run {
  Arena ws;
  bool go;   // false: only size the workspace
  hipStream_t st;
};

// A padded copy of `s` (times act'(z) when z is given) in `planes` planes,
// and on request its column sums.
hipError_t lin_pack(Run& r, const Span& s, int planes, const Span* z, int act, bool copy, float* db, int accumulate,
                    Operand& out) {
  LinPack p{};
  p.src = s.p;
  p.ld = s.ld;
  p.rows = s.rows;
  p.cols = static_cast<int32_t>(s.cols);
  p.dtype = s.esize == 2;
  p.planes = planes;
  p.act = act;
  if (z) {
    p.z = z->p;
    p.ldz = z->ld;
  }
  // at most 256 rows of partial sums
  p.chunk = static_cast<int32_t>(std::max<int64_t>(32, lin_cdiv(lin_cdiv(s.rows, 256), 8) * 8));
  const int chunks = static_cast<int>(lin_cdiv(s.rows, p.chunk));
  if (copy) {
    p.pitch = lin_cdiv(s.cols, 64) * 64;
    p.plane = s.rows * p.pitch;
    p.dst = r.ws.take<uint16_t>(static_cast<size_t>(p.planes) * p.plane);
    out = {p.dst, p.pitch, p.plane};
  }
  if (db) p.sums = r.ws.take<float>(static_cast<size_t>(chunks) * s.cols);
  if (!r.go) return hipSuccess;
  if (s.rows > 0) LIN_TRY(launch_lin_pack(p, r.st));
  if (db) LIN_TRY(launch_lin_colsum(p.sums, chunks, p.cols, db, accumulate, r.st));
  return hipSuccess;
}

hipError_t lin_operand(Run& r, const Span& s, Operand& out) {
  if (lin_direct(s)) {
    out = {static_cast<const uint16_t*>(s.p), s.ld, 0};
    return hipSuccess;
  }
  return lin_pack(r, s, s.esize == 2 ? 1 : 3, nullptr, DION_ACT_NONE, true, nullptr, 0, out);
}

// A K-major operand's columns from K to the next multiple of 8 are zero (K
// is one already for a tensor read in place, and a copy is padded); an
// x-major operand's rows past K are not read.
hipError_t lin_product(Run& r, const Operand& a, const Operand& b, int64_t M, int64_t N, int64_t K,
                       int nseg, LinKind kind, const LinOut& out) {
  LinProduct p{};
  p.a = a.p;
  p.b = b.p;
  p.lda = a.ld;
  p.ldb = b.ld;
  p.sa = a.plane;
  p.sb = b.plane;
  p.M = static_cast<int32_t>(M);
  p.N = static_cast<int32_t>(N);
  p.K = static_cast<int32_t>(K);
  p.nseg = nseg;
  p.out = out;
  // 256 x 256 tiles where they fill the chip
  const int tile = lin_cdiv(M, 256) * lin_cdiv(N, 256) >= kLinBigTiles ? 256 : 128;
  p.tx = static_cast<int32_t>(lin_cdiv(M, tile));
  p.ty = static_cast<int32_t>(lin_cdiv(N, tile));
  const Cut16 c = cut_tiles(static_cast<int64_t>(p.tx) * p.ty, tile, lin_cdiv(K, 32) * nseg);
  p.items = static_cast<int32_t>(c.items());
  p.full = static_cast<int32_t>(c.full);
  p.slices = static_cast<int32_t>(c.slices);
  if (c.cut) {
    p.part = r.ws.take<float>(cut_bytes(c, tile) / 4);
    p.count = r.ws.take<uint32_t>(c.cut);
  }
  if (!r.go) return hipSuccess;
  if (c.cut) LIN_TRY(launch_lin_zero(p.count, static_cast<int>(c.cut), r.st));
  return launch_lin_product(p, kind, tile, r.st);
}

hipError_t lin_forward(Run& r, const LinCall& c) {
  const dion_linear& l = c.a;
  if (l.t == 0) return hipSuccess;
  LinOut out{};
  out.y = l.y;
  out.ldy = l.ldy;
  out.bias = l.bias;
  out.residual = l.residual;
  out.ldr = l.ldr;
  out.z = l.z;
  out.ldz = l.ldz;
  out.act = l.act;
  out.dtype = l.dtype == DION_DTYPE_BF16;
  const bool f32 = !out.dtype;
  const bool direct = lin_direct(c.x) && lin_direct(c.w);
  LinSkinny s{l.x, l.w, l.ldx, l.ldw, static_cast<int32_t>(l.t), static_cast<int32_t>(l.n),
              static_cast<int32_t>(l.k), out};
  if (direct && l.t <= kSkinnyTokens) return r.go ? launch_lin_skinny(s, r.st) : hipSuccess;
  if (l.t <= kRowTokens) {
    const int64_t v = 16 / c.e;
    const bool vec = reinterpret_cast<uintptr_t>(l.x) % 16 == 0 && reinterpret_cast<uintptr_t>(l.w) % 16 == 0 &&
                     l.ldx % v == 0 && l.ldw % v == 0 && l.k % v == 0;
    return r.go ? launch_lin_rows(s, vec, r.st) : hipSuccess;
  }
  Operand x, w;
  LIN_TRY(lin_operand(r, c.x, x));
  LIN_TRY(lin_operand(r, c.w, w));
  return lin_product(r, x, w, l.t, l.n, l.k, f32 ? 6 : 1, kLinForward, out);
}

hipError_t lin_backward(Run& r, const LinCall& c) {
  const dion_linear& l = c.a;
  const bool f32 = l.dtype == DION_DTYPE_F32, act = l.act != DION_ACT_NONE;
  const bool products = l.dx || l.dw;
  Operand dz{}, x{}, w{};
  const bool copy = products && (act || !lin_direct(c.dy));
  const int planes = f32 ? 3 : act && l.t <= kLinFewTokens ? 2 : 1;
  const int nseg = f32 ? 6 : planes;
  if (copy || l.db)
    LIN_TRY(lin_pack(r, c.dy, planes, act ? &c.z : nullptr, l.act, copy, l.db, l.accumulate, dz));
  if (products && !copy) dz = {static_cast<const uint16_t*>(l.dy), l.lddy, 0};
  LinOut out{};
  out.dtype = !f32;
  if (l.dx && l.t > 0) {
    LIN_TRY(lin_operand(r, c.w, w));
    out.y = l.dx;
    out.ldy = l.lddx;
    LIN_TRY(lin_product(r, dz, w, l.t, l.k, l.n, nseg, kLinDx, out));
  }
  if (l.dw) {
    if (l.t > 0) LIN_TRY(lin_operand(r, c.x, x));
    out.y = l.dw;
    out.ldy = l.lddw;
    out.accumulate = l.accumulate != 0;
    LIN_TRY(lin_product(r, dz, x, l.n, l.k, l.t, nseg, kLinDw, out));
  }
  return hipSuccess;
}

template <class Check, class Go>
size_t lin_size(const dion_linear* l, Check check, Go go) {
  LinCall c;
  if (!check(l, c)) return 0;
  Run r{{nullptr}, false, nullptr};
  (void)go(r, c);
  return r.ws.used + 256;   // a valid query is never 0
}

template <class Check, class Go>
int lin_run(const dion_linear* l, void* workspace, size_t bytes, void* stream, Check check, Go go) {
  LinCall c;
  if (!check(l, c)) return DION_ERR_INVALID_ARG;
  Run size{{nullptr}, false, nullptr};
  (void)go(size, c);
  if (size.ws.used > 0 &&
      (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 != 0 || bytes < size.ws.used))
    return DION_ERR_WORKSPACE;
  Run r{{static_cast<char*>(workspace)}, true, static_cast<hipStream_t>(stream)};
  return go(r, c) == hipSuccess ? DION_OK : DION_ERR_HIP;
}

}  // namespace
}  // namespace dion

using namespace dion;

DION_API size_t dion_linear_forward_workspace_size(const dion_linear* l) {
  return lin_size(l, lin_forward_ok, lin_forward);
}

DION_API int dion_linear_forward(const dion_linear* l, void* workspace, size_t workspace_bytes, void* stream) {
  return lin_run(l, workspace, workspace_bytes, stream, lin_forward_ok, lin_forward);
}

DION_API size_t dion_linear_backward_workspace_size(const dion_linear* l) {
  return lin_size(l, lin_backward_ok, lin_backward);
}

DION_API int dion_linear_backward(const dion_linear* l, void* workspace, size_t workspace_bytes, void* stream) {
  return lin_run(l, workspace, workspace_bytes, stream, lin_backward_ok, lin_backward);
}
