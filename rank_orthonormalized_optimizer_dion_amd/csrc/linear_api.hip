// Host side of dion_linear_forward and dion_linear_backward: argument
// validation, workspace layout and schedule.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include "dion.h"
#include "linear_types.h"
#include "span.h"
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
// 256 x 256 tiles in a product of at least this many (one per CU), else 128 x
// 128.  Timed in bfloat16: 4096 tokens, 4096 -> 4096 110 us, with 128 x 128 163
// us; backward, 4096 tokens, 3072 -> 3072 (144 and 192 tiles) 257 us, with 256 x 256 227
// us.  The count is of padded tiles: 100 tokens, 768 -> 66000 take 46 us, with
// 128 x 128 31 us.
constexpr int64_t kLinBigTiles = 256;

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
    if (spans_overlap(*in, c.y) || spans_overlap(*in, c.z)) return false;
  if (spans_overlap(c.y, c.z) || spans_overlap(c.res, c.z)) return false;
  // y may be the residual itself (added in place), not a shifted view of it
  if (spans_overlap(c.res, c.y) && !(c.res.p == c.y.p && c.res.ld == c.y.ld)) return false;
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
      if (spans_overlap(*in, *outs[i])) return false;
    for (int j = 0; j < i; ++j)
      if (spans_overlap(*outs[i], *outs[j])) return false;
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
  LinPacks packs;
};

constexpr int kLinStage = 32;   // k of a reduction stage (mm16.h)

// Adds a padded copy of `s` (times act'(z) when z is given) in `planes`
// planes to the call's copies, and on request its column sums.
void lin_pack(Run& r, const Span& s, int planes, const Span* z, int act, bool copy, bool sums, Operand& out) {
  LinPack p{};
  p.src = s.p;
  p.ld = s.ld;
  p.rows = s.rows;
  p.prows = copy ? lin_cdiv(s.rows, kLinStage) * kLinStage : s.rows;
  p.cols = static_cast<int32_t>(s.cols);
  p.dtype = s.esize == 2;
  p.planes = planes;
  p.act = act;
  if (z) {
    p.z = z->p;
    p.ldz = z->ld;
  }
  // at most 256 rows of partial sums
  p.chunk = static_cast<int32_t>(std::max<int64_t>(16, lin_cdiv(lin_cdiv(p.prows, 256), 8) * 8));
  const int64_t chunks = lin_cdiv(p.prows, p.chunk);
  if (copy) {
    p.pitch = lin_cdiv(s.cols, 64) * 64;
    p.plane = p.prows * p.pitch;
    p.dst = r.ws.take<uint16_t>(static_cast<size_t>(planes) * p.plane);
    out = {p.dst, p.pitch, p.plane};
  }
  if (sums) p.sums = r.ws.take<float>(static_cast<size_t>(chunks) * s.cols);
  p.gx = static_cast<int32_t>(lin_cdiv(copy ? p.pitch : s.cols, 256));
  p.blocks = static_cast<int32_t>(p.gx * chunks);
  r.packs.p[r.packs.n++] = p;
}

void lin_operand(Run& r, const Span& s, Operand& out) {
  if (lin_direct(s)) out = {static_cast<const uint16_t*>(s.p), s.ld, 0};
  else lin_pack(r, s, s.esize == 2 ? 1 : 3, nullptr, DION_ACT_NONE, true, false, out);
}

// One product's launch.  A K-major operand's columns from K to the next
// multiple of 8 are zero (K is one already for a tensor read in place, and a
// copy is padded); an x-major operand's rows past K are not read.  padded:
// both operands are copies, zero to the end of K's last stage.
struct Product {
  LinProduct p;
  LinKind kind;
  int tile;
};
Product lin_product(Run& r, const Operand& a, const Operand& b, int64_t M, int64_t N, int64_t K, bool padded,
                    int nseg, LinKind kind, const LinOut& out) {
  Product f{};
  LinProduct& p = f.p;
  f.kind = kind;
  if (padded) K = lin_cdiv(K, kLinStage) * kLinStage;
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
  f.tile = lin_cdiv(M, 256) * lin_cdiv(N, 256) >= kLinBigTiles ? 256 : 128;
  p.tx = static_cast<int32_t>(lin_cdiv(M, f.tile));
  p.ty = static_cast<int32_t>(lin_cdiv(N, f.tile));
  const Cut16 c = cut_tiles(static_cast<int64_t>(p.tx) * p.ty, f.tile, lin_cdiv(K, kLinStage) * nseg);
  p.items = static_cast<int32_t>(c.items());
  p.full = static_cast<int32_t>(c.full);
  p.slices = static_cast<int32_t>(c.slices);
  if (c.cut) {
    p.part = r.ws.take<float>(cut_bytes(c, f.tile) / 4);
    p.count = r.packs.count;   // shared by the call's products: all zero between launches
    r.packs.counts = kTileSlots128;
  }
  return f;
}

// The copies (and counters) a call's products need, then the products.
hipError_t lin_enqueue(Run& r, std::initializer_list<const Product*> products) {
  if (r.packs.n > 0 || r.packs.counts > 0) LIN_TRY(launch_lin_packs(r.packs, r.st));
  for (const Product* f : products)
    if (f->p.items > 0) LIN_TRY(launch_lin_product(f->p, f->kind, f->tile, r.st));
  return hipSuccess;
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
  lin_operand(r, c.x, x);
  lin_operand(r, c.w, w);
  const bool padded = !lin_direct(c.x) && !lin_direct(c.w);
  const Product y = lin_product(r, x, w, l.t, l.n, l.k, padded, f32 ? 6 : 1, kLinForward, out);
  return r.go ? lin_enqueue(r, {&y}) : hipSuccess;
}

hipError_t lin_backward(Run& r, const LinCall& c) {
  const dion_linear& l = c.a;
  const bool f32 = l.dtype == DION_DTYPE_F32, act = l.act != DION_ACT_NONE;
  const bool products = l.dx || l.dw;
  Operand dz{}, x{}, w{};
  const bool copy = products && (act || !lin_direct(c.dy));
  const int planes = f32 ? 3 : act && l.t <= kLinFewTokens ? 2 : 1;
  const int nseg = f32 ? 6 : planes;
  if (copy || l.db) lin_pack(r, c.dy, planes, act ? &c.z : nullptr, l.act, copy, l.db != nullptr, dz);
  const LinPack sums = r.packs.p[0];
  if (products && !copy) dz = {static_cast<const uint16_t*>(l.dy), l.lddy, 0};
  LinOut out{};
  out.dtype = !f32;
  Product dx{}, dw{};
  if (l.dx && l.t > 0) {
    lin_operand(r, c.w, w);
    out.y = l.dx;
    out.ldy = l.lddx;
    dx = lin_product(r, dz, w, l.t, l.k, l.n, copy && !lin_direct(c.w), nseg, kLinDx, out);
  }
  if (l.dw) {
    if (l.t > 0) lin_operand(r, c.x, x);
    out.y = l.dw;
    out.ldy = l.lddw;
    out.accumulate = l.accumulate != 0;
    dw = lin_product(r, dz, x, l.n, l.k, l.t, copy && !lin_direct(c.x), nseg, kLinDw, out);
  }
  if (!r.go) return hipSuccess;
  LIN_TRY(lin_enqueue(r, {&dx, &dw}));
  if (l.db)
    LIN_TRY(launch_lin_colsum(sums.sums, sums.blocks / sums.gx, sums.cols, l.db, l.accumulate, r.st));
  return hipSuccess;
}

template <class Check, class Go>
size_t lin_size(const dion_linear* l, Check check, Go go) {
  LinCall c;
  if (!check(l, c)) return 0;
  Run r{{nullptr}, false, nullptr, {}};
  r.packs.count = r.ws.take<uint32_t>(kTileSlots128);
  (void)go(r, c);
  return r.ws.used;
}

template <class Check, class Go>
int lin_run(const dion_linear* l, void* workspace, size_t bytes, void* stream, Check check, Go go) {
  LinCall c;
  if (!check(l, c)) return DION_ERR_INVALID_ARG;
  Run size{{nullptr}, false, nullptr, {}};
  size.packs.count = size.ws.take<uint32_t>(kTileSlots128);
  const size_t counters = size.ws.used;
  (void)go(size, c);
  const bool needed = size.packs.counts > 0 || size.ws.used > counters;
  if (needed && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 != 0 || bytes < size.ws.used))
    return DION_ERR_WORKSPACE;
  Run r{{static_cast<char*>(workspace)}, true, static_cast<hipStream_t>(stream), {}};
  r.packs.count = r.ws.take<uint32_t>(kTileSlots128);
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
