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

// Few tokens: their own kernels (k_xent_few.hip).
bool xent_few(const XentCall& c, bool grad) {
  const bool copied = !(lin_direct(c.x) && lin_direct(c.w));
  return c.a.t <= (c.e == 2 && (grad || copied) ? kXentFew16 : kXentFew);
}

// A call's copies, counters and workspace.
struct XentRun : Run {
  size_t peak = 0;
  XentCopies copies{};
  int copied = 0;
  // A bfloat16 operand, in place or as a copy in the next launch of copies.
  void operand(const Span& s, Operand& out) {
    if (lin_direct(s)) {
      out = {static_cast<const uint16_t*>(s.p), s.ld, 0};
      return;
    }
    XentCopy& c = copies.c[copied++];
    c.src = static_cast<const uint16_t*>(s.p);
    c.ld = s.ld;
    c.rows = s.rows;
    c.prows = lin_cdiv(s.rows, kLinStage) * kLinStage;
    c.cols = static_cast<int32_t>(s.cols);
    c.pitch = lin_cdiv(s.cols, 64) * 64;
    c.dst = ws.take<uint16_t>(c.prows * c.pitch);
    out = {c.dst, c.pitch, 0};
  }
  // The copies (and counters) that the products to come need.
  hipError_t prepare() {
    copies.count = packs.counts > 0 ? packs.count : nullptr;
    const hipError_t e = go && (copied > 0 || copies.count) ? launch_xent_copies(copies, st) : hipSuccess;
    peak = std::max(peak, ws.used);
    copies = {};
    copied = 0;
    packs.counts = 0;
    return e;
  }
};

bool few_far(const XentCall& c) { return c.a.n * c.a.k * c.e > kFewFar; }

XentFew few_args(const XentCall& c, const Span& w) {
  XentFew f{};
  f.w = w.p;
  f.ldw = w.ld;
  f.n = static_cast<int32_t>(w.rows);
  f.k = static_cast<int32_t>(c.a.k);
  f.t = static_cast<int32_t>(c.a.t);
  f.tp = c.a.t <= 32 ? 32 : 64;
  f.far = few_far(c);
  return f;
}

// x's planes for the kernels of few tokens (a bfloat16 x of whole 16-byte
// pieces is used as it is), and where its transpose's go.
XentPrep few_prep(XentRun& r, const XentCall& c, bool planes, bool transposed, XentFew& f) {
  const int64_t P = c.e == 2 ? 1 : 3;
  XentPrep a{c.a.x, c.a.ldx, f.t, f.k, f.tp, nullptr, 0, 0, nullptr, 0, 0};
  f.x = c.a.x;
  f.ldx = c.a.ldx;
  f.kx = f.k;
  if (planes && !lin_direct(c.x)) {
    a.ldp = lin_cdiv(f.k, 64) * 64;
    a.xplane = f.t * a.ldp;
    a.xp = r.ws.take<uint16_t>(P * a.xplane);
    f.x = a.xp;
    f.ldx = a.ldp;
    f.xplane = a.xplane;
    f.kx = static_cast<int32_t>(a.ldp);
  }
  if (transposed) {
    a.xtplane = static_cast<int64_t>(f.k) * f.tp;
    a.xt = r.ws.take<uint16_t>(P * a.xtplane);
    f.xt = a.xt;
    f.xtplane = a.xtplane;
  }
  return a;
}

// Workgroups of z's kernel: up to four per CU, which then take several blocks
// of rows in turn.
int64_t few_groups(int64_t n, int rt) { return std::min<int64_t>(lin_cdiv(n, 16 * rt), 1024); }

// The size of a bfloat16 product's tiles by its estimated time, in stages of a
// 256 x 256 tile (0.9 us): rounds of whole tiles, a cut round, a tile's first
// loads and epilogue (6 or 4), and the join of a cut round, whose sums all go
// through memory (18 or 9) before one workgroup per tile reads its slices (2.2
// or 0.6 each).  A stage of a 128 x 128 tile, two of which share a CU, takes
// 0.65.  Against both sizes timed over 30 products (65 to 8192 tokens, widths of
// 512 to 4096, 5000 to 128000 words) it takes the faster one, or one within 3% of
// it; the linear layer's rule (256 tiles of 256 x 256) took the other one in
// four: dx of 2048 tokens, 4096 -> 32000, 616 us against 453.
double xent_estimate(int64_t M, int64_t N, int64_t K, int tile) {
  const int64_t stages = lin_cdiv(K, kLinStage);
  const Cut16 c = cut_tiles(lin_cdiv(M, tile) * lin_cdiv(N, tile), tile, stages);
  const bool big = tile == 256;
  // tiles that cut_tiles leaves whole in the last round are counted as a round
  const int64_t rounds = lin_cdiv(c.full, tile_slots(tile)), last = c.cut > 0;
  const double step = big ? 1.0 : 0.65, start = big ? 6.0 : 4.0;
  double t = (rounds + last) * start + (rounds + (last ? 1.0 / c.slices : 0.0)) * stages * step;
  if (last && c.slices > 1) t += big ? 18.0 + 2.2 * c.slices : 9.0 + 0.6 * c.slices;
  return t;
}
int xent_tile(int64_t M, int64_t N, int64_t K) {
  return xent_estimate(M, N, K, 256) <= xent_estimate(M, N, K, 128) ? 256 : 128;
}

// One float32 product, cut along long reductions as the other tiles are: a
// stage is six products of half a 256 x 256 tile.
XentProduct32 xent_product32(XentRun& r, const float* A, int64_t lda, const float* B, int64_t ldb, int64_t M, int64_t N,
                             int64_t K, bool gradient) {
  XentProduct32 p{};
  p.a = A;
  p.b = B;
  p.lda = lda;
  p.ldb = ldb;
  p.M = static_cast<int32_t>(M);
  p.N = static_cast<int32_t>(N);
  p.K = static_cast<int32_t>(K);
  p.tx = static_cast<int32_t>(lin_cdiv(M, kXentM32));
  p.ty = static_cast<int32_t>(lin_cdiv(N, kXentN32));
  const Cut16 c = cut_tiles(static_cast<int64_t>(p.tx) * p.ty, 256, lin_cdiv(K, kLinStage) * 3);
  p.items = static_cast<int32_t>(c.items());
  p.full = static_cast<int32_t>(c.full);
  p.slices = static_cast<int32_t>(c.slices);
  if (c.cut) {
    p.part = r.ws.take<float>(c.cut * c.slices * kXentM32 * kXentN32);
    p.count = r.packs.count;
    r.packs.counts = 1;
  }
  p.apart = gradient && c.cut && c.slices >= kXentApart;
  return p;
}

hipError_t xent_forward(XentRun& r, const XentCall& c) {
  const dion_cross_entropy& a = c.a;
  if (a.t == 0) return hipSuccess;
  const bool few = xent_few(c, false);
  const bool f32 = !few && c.e == 4;
  // a piece at a time where W has to be copied, and where one launch would have
  // more threads than a grid can (2^32: 2^22 tiles of 128 x 128, far fewer of others)
  const bool copy = !few && !f32 && !lin_direct(c.w);
  const int64_t most_cols = few ? a.n : std::max(kXentStep, (int64_t{1} << 22) / lin_cdiv(a.t, 128) * 128 / kXentStep * kXentStep);
  const int64_t piece = std::min(most_cols, copy ? xent_piece(a.n, 2 * lin_cdiv(a.k, 64) * 64) : a.n);
  // one partial column per 64 columns at least: whole pieces end with a tile
  const int rt = few_rows(static_cast<int>(a.t), a.n, c.e == 4, false, few_far(c));
  const int64_t most = few ? few_groups(a.n, rt) : lin_cdiv(a.n, 64) + 4;
  XentEpi e{};
  e.target = a.target;
  e.ignore = a.ignore_index;
  e.vocab = a.n;
  e.top = r.ws.take<float>(most * a.t);
  e.sum = r.ws.take<float>(most * a.t);
  if (a.label_smoothing > 0.0f) e.total = r.ws.take<float>(most * a.t);
  e.hit = r.ws.take<float>(a.t);
  int64_t cols = 0;
  if (few) {
    cols = most;
    XentFew f = few_args(c, c.w);
    const bool raw = a.t <= 16 && !lin_direct(c.x);
    const XentPrep prep = few_prep(r, c, !raw, false, f);
    if (r.go && prep.xp) LIN_TRY(launch_few_prep(prep, c.e == 4, r.st));
    if (r.go) LIN_TRY(launch_few_z(f, e, prep, c.e == 4, false, raw, rt, static_cast<int>(cols), r.st));
  } else if (f32) {
    const size_t mark = r.ws.used;
    for (int64_t j0 = 0; j0 < a.n; j0 += piece) {
      r.ws.used = mark;
      const Span wj = xent_rows(c.w, j0, std::min(piece, a.n - j0));
      const XentProduct32 z = xent_product32(r, static_cast<const float*>(a.x), a.ldx, static_cast<const float*>(wj.p), a.ldw,
                                             a.t, wj.rows, a.k, false);
      e.j0 = static_cast<int32_t>(j0);
      e.col0 = static_cast<int32_t>(cols);
      cols += xent_tile_cols32(z.ty);
      LIN_TRY(r.prepare());
      if (r.go) LIN_TRY(launch_xent_f32(z, e, kXentStats32, r.st));
    }
  } else {
    Operand x;
    r.operand(c.x, x);
    const size_t mark = r.ws.used;
    for (int64_t j0 = 0; j0 < a.n; j0 += piece) {
      r.ws.used = mark;
      const Span wj = xent_rows(c.w, j0, std::min(piece, a.n - j0));
      Operand w;
      r.operand(wj, w);
      const Product z = lin_product(r, x, w, a.t, wj.rows, a.k, !lin_direct(c.x) && !lin_direct(c.w), 1, kLinForward,
                                    LinOut{}, xent_tile(a.t, wj.rows, a.k));
      e.j0 = static_cast<int32_t>(j0);
      e.col0 = static_cast<int32_t>(cols);
      cols += xent_tile_cols(z.p.ty);
      LIN_TRY(r.prepare());
      if (r.go) LIN_TRY(launch_xent_product(z.p, e, false, z.tile, r.st));
    }
  }
  if (!r.go) return hipSuccess;
  XentJoin j{e.top, e.sum, e.total, e.hit, a.target, a.ignore_index, a.n, a.loss, a.lse, static_cast<int32_t>(a.t),
             static_cast<int32_t>(cols), 1.0f - a.label_smoothing, a.label_smoothing, a.z_loss};
  return launch_xent_join(j, r.st);
}

XentEpi xent_grad(const XentCall& c, int planes, int64_t rows, int64_t piece) {
  const dion_cross_entropy& a = c.a;
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
  e.plane = rows * e.pitch;
  e.planes = planes;
  e.prows = static_cast<int32_t>(rows);
  return e;
}

hipError_t xent_backward_few(XentRun& r, const XentCall& c) {
  const dion_cross_entropy& a = c.a;
  const bool f32 = c.e == 4;
  const int planes = f32 ? 3 : 2;
  XentFew f = few_args(c, c.w);
  const int64_t piece = xent_piece(a.n, 2 * planes * (a.t + f.tp));
  XentEpi e = xent_grad(c, planes, a.t, piece);
  XentPrep prep = few_prep(r, c, true, a.dw != nullptr, f);
  e.dz = r.ws.take<uint16_t>(planes * e.plane);
  f.dztplane = e.pitch * f.tp;
  f.dzt = r.ws.take<uint16_t>(planes * f.dztplane);
  // dx and dW: as many workgroups as the chip holds at a time, by their registers
  // (24 tokens, gradients: 768 -> 50257 76 us, with 1024 of either 82; 4096 -> 32000
  // 198 and 215; 2048 -> 32000 111 and 114)
  const int64_t dx_slots = f32 ? 1024 : a.t <= 32 ? 768 : 512, dw_slots = 768;
  const int64_t pieces = lin_cdiv(a.n, piece), across = lin_cdiv(a.k, f32 ? 64 : 128);
  const int64_t parts = std::max<int64_t>(1, std::min(lin_cdiv(dx_slots, across), lin_cdiv(piece, 128)));
  float* part = a.dx ? r.ws.take<float>(pieces * parts * a.t * a.k) : nullptr;
  if (!r.go) return hipSuccess;
  if (prep.xp) {   // both forms of x before z; else the transpose beside it
    LIN_TRY(launch_few_prep(prep, f32, r.st));
    prep.xt = nullptr;
  }
  XentDxSum sum{part, static_cast<int32_t>(pieces * parts), f.t, f.k, a.dx, a.lddx, !f32};
  for (int64_t p = 0; p < pieces; ++p) {
    const int64_t j0 = p * piece;
    const Span wj = xent_rows(c.w, j0, std::min(piece, a.n - j0));
    f.w = wj.p;
    f.n = static_cast<int32_t>(wj.rows);
    e.j0 = static_cast<int32_t>(j0);
    const int rt = few_rows(f.t, e.pitch, f32, true, f.far);
    prep.first = static_cast<int32_t>(few_groups(e.pitch, rt));
    LIN_TRY(launch_few_z(f, e, prep, f32, true, false, rt, 0, r.st));
    prep.xt = nullptr;
    if (a.dx) LIN_TRY(launch_few_dx(f, e, f32, static_cast<int>(parts), part + p * parts * a.t * a.k, r.st));
    const bool last = p + 1 == pieces;
    if (a.dw) {
      const Span dj = xent_rows(c.dw, j0, wj.rows);
      // in whole steps of 64 columns
      const int64_t down = lin_cdiv(wj.rows, 4 * kFewDwRows);
      const int64_t split = std::min(lin_cdiv(a.k, 64), lin_cdiv(dw_slots, down));
      const XentDw d{const_cast<void*>(dj.p), a.lddw, static_cast<int32_t>(lin_cdiv(lin_cdiv(a.k, split), 64) * 64), a.accumulate, 0, 0};
      LIN_TRY(launch_few_dw(f, d, last ? sum : XentDxSum{}, f32, r.st));
    } else if (last) {
      LIN_TRY(launch_few_dxsum(sum, r.st));
    }
  }
  return hipSuccess;
}

hipError_t xent_backward_f32(XentRun& r, const XentCall& c) {
  const dion_cross_entropy& a = c.a;
  const int64_t piece = xent_piece(a.n, 4 * a.t);
  XentEpi e = xent_grad(c, 1, a.t, piece);
  e.dz32 = r.ws.take<float>(a.t * e.pitch);
  const float* x = static_cast<const float*>(a.x);
  const size_t mark = r.ws.used;
  for (int64_t j0 = 0; j0 < a.n; j0 += piece) {
    r.ws.used = mark;
    const int64_t n = std::min(piece, a.n - j0);
    const float* w = static_cast<const float*>(xent_rows(c.w, j0, n).p);
    const XentProduct32 z = xent_product32(r, x, a.ldx, w, a.ldw, a.t, n, a.k, false);
    XentProduct32 dx{}, dw{};
    if (a.dx) {
      dx = xent_product32(r, e.dz32, e.pitch, w, a.ldw, a.t, a.k, n, true);
      dx.out = static_cast<float*>(a.dx);
      dx.ldo = a.lddx;
      dx.accumulate = j0 > 0;
    }
    if (a.dw) {
      dw = xent_product32(r, e.dz32, e.pitch, x, a.ldx, n, a.k, a.t, true);
      dw.out = static_cast<float*>(const_cast<void*>(xent_rows(c.dw, j0, n).p));
      dw.ldo = a.lddw;
      dw.accumulate = a.accumulate != 0;
    }
    e.j0 = static_cast<int32_t>(j0);
    LIN_TRY(r.prepare());
    if (r.go) {
      LIN_TRY(launch_xent_f32(z, e, kXentDz32, r.st));
      if (a.dx) LIN_TRY(launch_xent_f32(dx, e, kXentDx32, r.st));
      if (a.dw) LIN_TRY(launch_xent_f32(dw, e, kXentDw32, r.st));
    }
  }
  return hipSuccess;
}

hipError_t xent_backward_bf16(XentRun& r, const XentCall& c) {
  const dion_cross_entropy& a = c.a;
  LinOut out{};
  out.dtype = 1;
  const int64_t prows = lin_cdiv(a.t, kLinStage) * kLinStage;
  const int64_t wcopy = lin_direct(c.w) ? 0 : 2 * lin_cdiv(a.k, 64) * 64;
  const int64_t piece = xent_piece(a.n, std::max(2 * prows, wcopy));
  XentEpi e = xent_grad(c, 1, prows, piece);
  e.dz = r.ws.take<uint16_t>(e.plane);
  const Operand dz{e.dz, e.pitch, 0};
  // dx over several pieces is summed in float32
  const bool sum = a.dx && piece < a.n;
  float* dxsum = sum ? r.ws.take<float>(a.t * a.k) : nullptr;
  Operand x{};
  r.operand(c.x, x);
  const bool padded = !lin_direct(c.w), xpadded = !lin_direct(c.x);
  const size_t mark = r.ws.used;
  for (int64_t j0 = 0; j0 < a.n; j0 += piece) {
    r.ws.used = mark;
    const Span wj = xent_rows(c.w, j0, std::min(piece, a.n - j0));
    const bool last = j0 + piece >= a.n;
    Operand w{};
    r.operand(wj, w);
    Product dx{}, dw{};
    const Product z = lin_product(r, x, w, a.t, wj.rows, a.k, padded && xpadded, 1, kLinForward, LinOut{},
                                  xent_tile(a.t, wj.rows, a.k));
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
      dx = lin_product(r, dz, w, a.t, a.k, wj.rows, padded, 1, kLinDx, o, xent_tile(a.t, a.k, wj.rows));
    }
    if (a.dw) {
      LinOut o = out;
      const Span dj = xent_rows(c.dw, j0, wj.rows);
      o.y = const_cast<void*>(dj.p);
      o.ldy = a.lddw;
      o.accumulate = a.accumulate != 0;
      dw = lin_product(r, dz, x, wj.rows, a.k, a.t, xpadded, 1, kLinDw, o, xent_tile(wj.rows, a.k, a.t));
    }
    e.j0 = static_cast<int32_t>(j0);
    LIN_TRY(r.prepare());
    if (r.go) {
      LIN_TRY(launch_xent_product(z.p, e, true, z.tile, r.st));
      if (a.dx) LIN_TRY(launch_lin_product(dx.p, kLinDx, dx.tile, r.st));
      if (a.dw) LIN_TRY(launch_lin_product(dw.p, kLinDw, dw.tile, r.st));
    }
  }
  return hipSuccess;
}

hipError_t xent_backward(XentRun& r, const XentCall& c) {
  const dion_cross_entropy& a = c.a;
  if (!a.dx && !a.dw) return hipSuccess;
  const bool f32 = c.e == 4;
  LinOut out{};
  out.dtype = !f32;
  if (a.t == 0) {   // no tokens: dW is zero
    if (!a.dw || a.accumulate) return hipSuccess;
    out.y = a.dw;
    out.ldy = a.lddw;
    const Product dw = lin_product(r, Operand{}, Operand{}, a.n, a.k, 0, false, 1, kLinDw, out);
    LIN_TRY(r.prepare());
    return r.go ? launch_lin_product(dw.p, kLinDw, dw.tile, r.st) : hipSuccess;
  }
  if (xent_few(c, true)) return xent_backward_few(r, c);
  return f32 ? xent_backward_f32(r, c) : xent_backward_bf16(r, c);
}

template <class Go>
hipError_t xent_go(XentRun& r, const XentCall& c, Go go) {
  r.packs.count = r.ws.take<uint32_t>(kTileSlots128);
  const hipError_t e = go(r, c);
  r.peak = std::max(r.peak, r.ws.used);
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
