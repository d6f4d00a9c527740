// Host side shared by the linear layer and the cross entropy: workspace
// layout, operand copies and product launches (linear_api.hip, xent_api.hip).
#pragma once
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include "dion.h"
#include "linear_types.h"
#include "span.h"
#include "work16.h"

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
// 128.  Timed in bfloat16: 4096 tokens, 4096 -> 4096 105 us, with 128 x 128 148
// us; backward, 4096 tokens, 3072 -> 3072 (144 and 192 tiles) 184 us, with 256 x 256 169
// us.  The count is of padded tiles: 100 tokens, 768 -> 66000 take 42 us, with
// 128 x 128 28 us.
constexpr int64_t kLinBigTiles = 256;

bool span_ok(const Span& s, bool required) {
  if (!s.p) return !required || s.rows == 0;
  return s.ld >= s.cols && s.ld <= kLinMaxPitch && !s.misplaced();
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
// tile: 128 or 256, or 0 for the linear layer's rule.
Product lin_product(Run& r, const Operand& a, const Operand& b, int64_t M, int64_t N, int64_t K, bool padded,
                    int nseg, LinKind kind, const LinOut& out, int tile = 0) {
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
  f.tile = tile ? tile : lin_cdiv(M, 256) * lin_cdiv(N, 256) >= kLinBigTiles ? 256 : 128;
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

}  // namespace
}  // namespace dion
