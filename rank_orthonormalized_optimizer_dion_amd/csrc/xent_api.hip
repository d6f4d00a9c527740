// Host side of dion_cross_entropy_forward and dion_cross_entropy_backward:
// argument validation, workspace layout and schedule.
#include <hip/hip_runtime.h>

#include <cmath>

#include "linear_host.h"
#include "xent_types.h"

#define DION_API extern "C" __attribute__((visibility("default")))

namespace dion {
namespace {

// Bytes of dz, and of a copied piece of W, that a call holds at a time.
constexpr int64_t kXentPiece = int64_t{256} << 20;
constexpr int64_t kXentStep = 256;   // pieces are whole tiles wide

struct XentCall {
  dion_cross_entropy a;
  int64_t e;   // element size
  Span x, w, target, loss, lse, dloss, dx, dw;
};

bool xent_common(const dion_cross_entropy* a, XentCall& c) {
  if (!a) return false;
  c.a = *a;
  if (a->t < 0 || a->t > kLinMaxTokens || a->n < 1 || a->k < 1 || a->n > DION_MAX_DIM || a->k > DION_MAX_DIM)
    return false;
  if (a->dtype != DION_DTYPE_F32 && a->dtype != DION_DTYPE_BF16) return false;
  if (!(a->label_smoothing >= 0.0f && a->label_smoothing <= 1.0f) || !std::isfinite(a->z_loss)) return false;
  c.e = a->dtype == DION_DTYPE_BF16 ? 2 : 4;
  c.x = {a->x, a->t, a->k, a->ldx, c.e};
  c.w = {a->w, a->n, a->k, a->ldw, c.e};
  c.target = {a->target, 1, a->t, a->t, 8};
  c.loss = {a->loss, 1, a->t, a->t, 4};
  c.lse = {a->lse, 1, a->t, a->t, 4};
  c.dloss = {a->dloss, 1, a->t, a->t, 4};
  c.dx = {a->dx, a->t, a->k, a->lddx, c.e};
  c.dw = {a->dw, a->n, a->k, a->lddw, c.e};
  return span_ok(c.x, true) && (a->t == 0 || (c.target.p && !c.target.misplaced()));
}

bool row_ok(const Span& s, bool required) { return !s.p ? !required || s.cols == 0 : !s.misplaced(); }

// Whether an output shares memory with an input or another output.
template <size_t I, size_t O>
bool apart(const Span* const (&in)[I], const Span* const (&out)[O]) {
  for (size_t i = 0; i < O; ++i) {
    for (const Span* s : in)
      if (s->cols > 0 && out[i]->cols > 0 && spans_overlap(*s, *out[i])) return false;
    for (size_t j = 0; j < i; ++j)
      if (out[j]->cols > 0 && out[i]->cols > 0 && spans_overlap(*out[j], *out[i])) return false;
  }
  return true;
}

bool xent_forward_ok(const dion_cross_entropy* a, XentCall& c) {
  if (!xent_common(a, c) || !span_ok(c.w, true)) return false;
  if (!row_ok(c.loss, false) || !row_ok(c.lse, false) || (a->t > 0 && !a->loss && !a->lse)) return false;
  const Span* const in[] = {&c.x, &c.w, &c.target};
  const Span* const out[] = {&c.loss, &c.lse};
  return apart(in, out);
}

bool xent_backward_ok(const dion_cross_entropy* a, XentCall& c) {
  if (!xent_common(a, c) || !span_ok(c.w, a->t > 0) || !span_ok(c.dx, false) || !span_ok(c.dw, false)) return false;
  if (!row_ok(c.lse, true) || !row_ok(c.dloss, true)) return false;
  const Span* const in[] = {&c.x, &c.w, &c.target, &c.lse, &c.dloss};
  const Span* const out[] = {&c.dx, &c.dw};
  return apart(in, out);
}

// Rows [j0, j0 + rows) of W.
Span xent_rows(const Span& w, int64_t j0, int64_t rows) {
  const char* p = static_cast<const char*>(w.p);
  return {p ? p + j0 * w.ld * w.esize : nullptr, rows, w.cols, w.ld, w.esize};
}

// Columns of the vocabulary per piece: `row` bytes each.
int64_t xent_piece(int64_t n, int64_t row) {
  return std::min(n, std::max(kXentStep, kXentPiece / row / kXentStep * kXentStep));
}

// How z is computed: rows and skinny products of few tokens, or tiles.
enum XentPath { kXentRows, kXentSkinny, kXentTiles };
XentPath xent_path(const XentCall& c, bool& vec) {
  const dion_cross_entropy& a = c.a;
  const int64_t v = 16 / c.e;
  vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && reinterpret_cast<uintptr_t>(a.w) % 16 == 0 && a.ldx % v == 0 &&
        a.ldw % v == 0 && a.k % v == 0;
  if (lin_direct(c.x) && lin_direct(c.w) && a.t <= kSkinnyTokens) return kXentSkinny;
  return a.t <= kRowTokens ? kXentRows : kXentTiles;
}

LinSkinny xent_skinny(const XentCall& c, const Span& w) {
  LinSkinny s{c.a.x, w.p, c.a.ldx, w.ld, static_cast<int32_t>(c.a.t), static_cast<int32_t>(w.rows),
              static_cast<int32_t>(c.a.k), {}};
  s.out.dtype = c.e == 2;
  return s;
}

// The products of one piece or call, after the copies that they need; the
// copies and counters of the launch are then done.
struct XentRun : Run {
  size_t peak = 0;
  hipError_t packs() {
    if (!this->go || (this->Run::packs.n == 0 && this->Run::packs.counts == 0)) return hipSuccess;
    return launch_lin_packs(this->Run::packs, st);
  }
  void done() {
    peak = std::max(peak, ws.used);
    Run::packs.n = 0;
    Run::packs.counts = 0;
  }
};

hipError_t xent_forward(XentRun& r, const XentCall& c) {
  const dion_cross_entropy& a = c.a;
  if (a.t == 0) return hipSuccess;
  bool vec;
  const XentPath path = xent_path(c, vec);
  const int planes = c.e == 2 ? 1 : 3;
  // a piece at a time only where W has to be copied
  const bool copy = path == kXentTiles && !lin_direct(c.w);
  const int64_t piece = copy ? xent_piece(a.n, 2 * planes * lin_cdiv(a.k, 64) * 64) : a.n;
  // one partial column per 64 columns at least
  const int64_t most = path == kXentTiles ? lin_cdiv(a.n, 64) + 2 * lin_cdiv(a.n, piece) : xent_group_cols(a.n);
  XentEpi e{};
  e.target = a.target;
  e.ignore = a.ignore_index;
  e.vocab = a.n;
  e.top = r.ws.take<float>(most * a.t);
  e.sum = r.ws.take<float>(most * a.t);
  if (a.label_smoothing > 0.0f) e.total = r.ws.take<float>(most * a.t);
  e.hit = r.ws.take<float>(a.t);
  int64_t cols = 0;
  if (path != kXentTiles) {
    cols = xent_group_cols(a.n);
    if (r.go) {
      const LinSkinny s = xent_skinny(c, c.w);
      LIN_TRY(path == kXentSkinny ? launch_xent_skinny(s, e, false, r.st) : launch_xent_rows(s, e, false, vec, r.st));
    }
  } else {
    Operand x;
    lin_operand(r, c.x, x);
    const size_t mark = r.ws.used;
    for (int64_t j0 = 0; j0 < a.n; j0 += piece) {
      r.ws.used = mark;
      const Span wj = xent_rows(c.w, j0, std::min(piece, a.n - j0));
      Operand w;
      lin_operand(r, wj, w);
      const Product z = lin_product(r, x, w, a.t, wj.rows, a.k, !lin_direct(c.x) && !lin_direct(c.w), planes == 3 ? 6 : 1,
                                    kLinForward, LinOut{});
      e.j0 = static_cast<int32_t>(j0);
      e.col0 = static_cast<int32_t>(cols);
      cols += xent_tile_cols(z.p.ty);
      LIN_TRY(r.packs());
      if (r.go) LIN_TRY(launch_xent_product(z.p, e, false, z.tile, r.st));
      r.done();
    }
  }
  if (!r.go) return hipSuccess;
  XentJoin j{e.top, e.sum, e.total, e.hit, a.target, a.ignore_index, a.n, a.loss, a.lse, static_cast<int32_t>(a.t),
             static_cast<int32_t>(cols), 1.0f - a.label_smoothing, a.label_smoothing, a.z_loss};
  return launch_xent_join(j, r.st);
}

hipError_t xent_backward(XentRun& r, const XentCall& c) {
  const dion_cross_entropy& a = c.a;
  if (!a.dx && !a.dw) return hipSuccess;
  bool vec;
  const XentPath path = xent_path(c, vec);
  const bool f32 = c.e == 4;
  const int planes = f32 ? 3 : a.t <= kLinFewTokens ? 2 : 1;
  const int nseg = f32 ? 6 : planes;
  LinOut out{};
  out.dtype = !f32;
  if (a.t == 0) {   // no tokens: dW is zero
    if (!a.dw || a.accumulate) return hipSuccess;
    out.y = a.dw;
    out.ldy = a.lddw;
    const Product dw = lin_product(r, Operand{}, Operand{}, a.n, a.k, 0, false, 1, kLinDw, out);
    LIN_TRY(r.packs());
    return r.go ? launch_lin_product(dw.p, kLinDw, dw.tile, r.st) : hipSuccess;
  }
  const int64_t prows = lin_cdiv(a.t, kLinStage) * kLinStage;
  const int64_t wcopy = lin_direct(c.w) ? 0 : 2 * (f32 ? 3 : 1) * lin_cdiv(a.k, 64) * 64;
  const int64_t piece = xent_piece(a.n, std::max(2 * planes * prows, wcopy));
  XentEpi e{};
  e.target = a.target;
  e.ignore = a.ignore_index;
  e.vocab = a.n;
  e.lse = a.lse;
  e.dloss = a.dloss;
  e.keep = 1.0f - a.label_smoothing;
  e.share = static_cast<float>(static_cast<double>(a.label_smoothing) / static_cast<double>(a.n));
  e.slope = 2.0f * a.z_loss;
  e.pitch = lin_cdiv(piece, 64) * 64;
  e.planes = planes;
  e.prows = static_cast<int32_t>(path == kXentTiles ? prows : a.t);
  // two planes lie row by row beside each other: dx then takes them as twice
  // the rows, in one sweep over W, and adds each pair (24 tokens, 2048 -> 32000:
  // dx 49 us, as two sweeps 77)
  const bool fold = planes == 2;
  e.ld = fold ? 2 * e.pitch : e.pitch;
  e.plane = fold ? e.pitch : prows * e.pitch;
  e.dz = r.ws.take<uint16_t>(planes * prows * e.pitch);
  const Operand dz{e.dz, e.ld, e.plane}, dzrows{e.dz, e.pitch, 0};
  // dx over several pieces is summed in float32
  const bool sum = a.dx && piece < a.n && !f32;
  float* dxsum = sum ? r.ws.take<float>(a.t * a.k) : nullptr;
  Operand x{};
  if (path == kXentTiles || a.dw) lin_operand(r, c.x, x);
  const size_t mark = r.ws.used;
  for (int64_t j0 = 0; j0 < a.n; j0 += piece) {
    r.ws.used = mark;
    const Span wj = xent_rows(c.w, j0, std::min(piece, a.n - j0));
    const bool last = j0 + piece >= a.n;
    Operand w{};
    if (path == kXentTiles || a.dx) lin_operand(r, wj, w);
    Product z{}, dx{}, dw{};
    if (path == kXentTiles)
      z = lin_product(r, x, w, a.t, wj.rows, a.k, !lin_direct(c.x) && !lin_direct(c.w), f32 ? 6 : 1, kLinForward, LinOut{});
    if (a.dx) {
      LinOut o = out;
      o.y = a.dx;
      o.ldy = a.lddx;
      if (sum && !last) {
        o.y = dxsum;
        o.ldy = a.k;
        o.dtype = 0;
      }
      o.accumulate = j0 > 0 && !(sum && last);
      if (sum && last) {   // the last piece's product is added and rounded
        o.residual = dxsum;
        o.ldr = a.k;
        o.wide = 1;
      }
      dx = fold ? lin_product(r, dzrows, w, 2 * a.t, a.k, wj.rows, !lin_direct(c.w), 1, kLinDx, o)
                : lin_product(r, dz, w, a.t, a.k, wj.rows, !lin_direct(c.w), nseg, kLinDx, o);
      dx.p.fold = fold;
    }
    if (a.dw) {
      LinOut o = out;
      const Span dj = xent_rows(c.dw, j0, wj.rows);
      o.y = const_cast<void*>(dj.p);
      o.ldy = a.lddw;
      o.accumulate = a.accumulate != 0;
      dw = lin_product(r, dz, x, wj.rows, a.k, a.t, path == kXentTiles && !lin_direct(c.x), nseg, kLinDw, o);
    }
    e.j0 = static_cast<int32_t>(j0);
    LIN_TRY(r.packs());
    if (r.go) {
      if (path == kXentTiles) {
        LIN_TRY(launch_xent_product(z.p, e, true, z.tile, r.st));
      } else {
        const LinSkinny s = xent_skinny(c, wj);
        LIN_TRY(path == kXentSkinny ? launch_xent_skinny(s, e, true, r.st) : launch_xent_rows(s, e, true, vec, r.st));
      }
      if (a.dx) LIN_TRY(launch_lin_product(dx.p, kLinDx, dx.tile, r.st));
      if (a.dw) LIN_TRY(launch_lin_product(dw.p, kLinDw, dw.tile, r.st));
    }
    r.done();
  }
  return hipSuccess;
}

template <class Go>
hipError_t xent_go(XentRun& r, const XentCall& c, Go go) {
  r.Run::packs.count = r.ws.take<uint32_t>(kTileSlots128);
  const hipError_t e = go(r, c);
  r.done();
  return e;
}

template <class Check, class Go>
size_t xent_size(const dion_cross_entropy* a, Check check, Go go) {
  XentCall c;
  if (!check(a, c)) return 0;
  XentRun r{};
  (void)xent_go(r, c, go);
  return r.peak;
}

template <class Check, class Go>
int xent_run(const dion_cross_entropy* a, void* workspace, size_t bytes, void* stream, Check check, Go go) {
  XentCall c;
  if (!check(a, c)) return DION_ERR_INVALID_ARG;
  XentRun size{};
  (void)xent_go(size, c, go);
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 != 0 || bytes < size.peak) return DION_ERR_WORKSPACE;
  XentRun r{};
  r.ws.base = static_cast<char*>(workspace);
  r.go = true;
  r.st = static_cast<hipStream_t>(stream);
  return xent_go(r, c, go) == hipSuccess ? DION_OK : DION_ERR_HIP;
}

}  // namespace
}  // namespace dion

using namespace dion;

DION_API size_t dion_cross_entropy_forward_workspace_size(const dion_cross_entropy* a) {
  return xent_size(a, xent_forward_ok, xent_forward);
}

DION_API int dion_cross_entropy_forward(const dion_cross_entropy* a, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  return xent_run(a, workspace, workspace_bytes, stream, xent_forward_ok, xent_forward);
}

DION_API size_t dion_cross_entropy_backward_workspace_size(const dion_cross_entropy* a) {
  return xent_size(a, xent_backward_ok, xent_backward);
}

DION_API int dion_cross_entropy_backward(const dion_cross_entropy* a, void* workspace, size_t workspace_bytes,
                                         void* stream) {
  return xent_run(a, workspace, workspace_bytes, stream, xent_backward_ok, xent_backward);
}
