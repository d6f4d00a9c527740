// Host side of dion_orthogonalize and dion_muon_step: argument validation,
// workspace layout, plane scales and the launch schedule.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <vector>

#include "dion.h"
#include "ns_types.h"
#include "span.h"
#include "work16.h"

#define DION_API extern "C" __attribute__((visibility("default")))

static_assert(dion::kNsNonFinite == DION_STATUS_NONFINITE, "status bit");

namespace dion {
namespace {

// With DION_MATH_F16 a matrix whose smaller side is at most this still takes
// two planes: its few singular values share each rounding (a 3 x 383 matrix
// came out 4.6e-3 off with one plane, where large ones are 1.2e-3 off), and
// launches, not products, are its cost.
constexpr int kNsSmallSide = 128;
// 256 x 256 tiles in a launch of at least this many (one per CU), else 128 x
// 128.  Timed, float16 unless said: always 128: 4096 x 4096 1.84 ms (1.60),
// 3072 x 8192 1.94 ms (1.86), twelve of 1543 x 1543 1.73 ms (1.83); from 64 tiles
// on: 3072 x 8192 1.70 ms, but 2048 x 2048 float32 0.91 ms (0.80).  The count is
// of padded tiles: matrices of few rows, which fill a fraction of theirs, lose
// by it (300 of 64 x 768: 0.94 ms, 0.71 with 128 x 128).
constexpr int64_t kNsBigTiles = 256;
static_assert(kNsCounts >= kTileSlots128 && kNsCounts >= kTileSlots256, "arrival counters");
constexpr size_t kNsAlign = 256;
size_t ns_align(size_t x) { return (x + kNsAlign - 1) / kNsAlign * kNsAlign; }
int64_t ns_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A call's matrices, the two entry points in one form.
struct NsMatrix {
  const void* G;
  void* O;
  float* M;
  int64_t m, n, ldg, ldo;
  float scale;
};

struct NsPlan {
  std::vector<NsDesc> table;      // grouped by shape
  std::vector<NsClass> shapes;    // first, count of each shape
  size_t status_off = 0, table_off = 0, count_off = 0, part_off = 0, bytes = 0;
};

bool ns_math(int math, int& planes) {
  if (math != DION_MATH_F32 && math != DION_MATH_F16) return false;
  planes = math == DION_MATH_F32 ? 2 : 1;
  return true;
}

bool ns_shape_ok(const NsMatrix& a) {
  return a.m >= 1 && a.n >= 1 && a.m <= DION_MAX_DIM && a.n <= DION_MAX_DIM && a.m * a.n <= INT32_MAX;
}

int ns_validate(const NsMatrix& a, int gdtype, int odtype, bool step) {
  if (!ns_shape_ok(a)) return DION_ERR_INVALID_ARG;
  if (!a.G || !a.O || (step && !a.M)) return DION_ERR_INVALID_ARG;
  if (a.ldg < a.n || a.ldo < a.n || a.ldg > INT32_MAX || a.ldo > INT32_MAX) return DION_ERR_INVALID_ARG;
  const Span g{a.G, a.m, a.n, a.ldg, gdtype == DION_DTYPE_BF16 ? 2 : 4};
  const Span o{a.O, a.m, a.n, a.ldo, odtype == DION_DTYPE_BF16 ? 2 : 4};
  const Span m{a.M, a.m, a.n, a.n, 4};   // the step's
  if (g.misplaced() || o.misplaced() || m.misplaced()) return DION_ERR_INVALID_ARG;
  if (spans_overlap(g, o) || spans_overlap(g, m) || spans_overlap(o, m)) return DION_ERR_INVALID_ARG;
  if (step && !std::isfinite(a.scale)) return DION_ERR_INVALID_ARG;
  return DION_OK;
}

// Whether a p x q matrix (p <= q) takes a one-workgroup form, and the padded
// sides it takes it with: plain float32 for at most 16 rows (sqp = 0; those
// that do not fit take k_ns_rows), else the matrix cores, where X's planes and
// one p x p plane fit 160 KB of LDS.
bool ns_small(int p, int q, int& spp, int& sqp) {
  if (p <= kNsTinySide) {
    spp = p <= 1 ? 1 : p <= 2 ? 2 : p <= 4 ? 4 : p <= 8 ? 8 : 16;
    sqp = 0;
    return static_cast<int64_t>(p) * q <= kNsTinyFloats;
  }
  spp = p <= 64 ? 64 : 128;
  sqp = q <= 128 ? 128 : q <= 256 ? 256 : 512;
  return p <= 128 && q <= (p <= 64 ? 512 : 256);
}

int ns_row_chunks(int q) { return static_cast<int>(ns_cdiv(q, ns_row_cols(q))); }

// One grouped launch per kNsMaxClasses shapes; the shapes are those that
// `pick` accepts.
template <class Pick, class Fill, class Go>
hipError_t ns_grouped(const NsPlan& p, const NsLaunch& base, Pick pick, Fill fill, Go go) {
  NsLaunch L = base;
  auto empty = [&] {
    L.nclass = 0;
    L.total = 0;
    for (NsClass& c : L.cls) {
      c = NsClass{};
      c.base = INT32_MAX;   // no item is past it
      c.tiles = 1;
    }
  };
  empty();
  for (const NsClass& s : p.shapes) {
    if (!pick(s)) continue;
    NsClass c = s;
    fill(p.table[s.first], c);
    c.base = L.total;
    L.cls[L.nclass++] = c;
    L.total += c.count * c.tiles;
    if (L.nclass == kNsMaxClasses) {
      const hipError_t e = go(L);
      if (e != hipSuccess) return e;
      empty();
    }
  }
  return L.nclass > 0 ? go(L) : hipSuccess;
}

#define NS_TRY(expr)              \
  do {                            \
    const hipError_t e_ = (expr); \
    if (e_ != hipSuccess) return e_; \
  } while (0)

// The launches of one product over all matrices of a plan with `planes`
// planes: go(L, items, tile) with L's classes and work split filled in.
// 256 x 256 tiles where they fill the chip, else 128 x 128; the largest
// matrices come first, so that the cut tiles of the last round are the
// smallest matrices'.
template <class Go>
hipError_t ns_launches(const NsPlan& p, const NsLaunch& base, NsEpi epi, int planes, Go go) {
  const bool sym = epi == kNsGram || epi == kNsGramPoly || epi == kNsPoly;
  auto shape = [&](int tile) {
    return [=](const NsDesc& d, NsClass& c) {
      c.tx = static_cast<int32_t>(ns_cdiv(ns_pad(d.p), tile));
      c.ty = sym ? c.tx : static_cast<int32_t>(ns_cdiv(ns_pad(d.q), tile));
      c.tiles = sym ? ns_sym_tiles(c.tx) : c.tx * c.ty;
    };
  };
  int64_t big = 0;
  for (const NsClass& s : p.shapes) {
    if (s.planes != planes) continue;
    NsClass c = s;
    shape(256)(p.table[s.first], c);
    big += static_cast<int64_t>(c.tiles) * c.count;
  }
  if (big == 0) return hipSuccess;
  const int tile = big >= kNsBigTiles ? 256 : 128;
  return ns_grouped(p, base, [=](const NsClass& s) { return s.planes == planes; }, shape(tile), [&](NsLaunch L) {
    const NsDesc& d = p.table[L.cls[L.nclass - 1].first];
    const int64_t k = ns_pad(epi == kNsGram || epi == kNsGramPoly ? d.q : d.p);
    const Cut16 c = cut_tiles(L.total, tile, k * planes / 32);
    L.full = static_cast<int32_t>(c.full);
    L.slices = static_cast<int32_t>(c.slices);
    return go(L, c, tile);
  });
}

hipError_t ns_product(const NsPlan& p, const NsLaunch& base, NsEpi epi, hipStream_t st) {
  for (int planes = 1; planes <= 2; ++planes)
    NS_TRY(ns_launches(p, base, epi, planes, [&](const NsLaunch& L, const Cut16& c, int tile) {
      return launch_ns_product(L, static_cast<int>(c.items()), epi, planes, tile, st);
    }));
  return hipSuccess;
}

// Descriptors grouped by shape, and the workspace: status words, table,
// then each matrix's planes.
void ns_layout(const std::vector<NsMatrix>& mats, int planes, NsPlan& p) {
  const int count = static_cast<int>(mats.size());
  std::vector<int> order(count);
  for (int i = 0; i < count; ++i) order[i] = i;
  std::stable_sort(order.begin(), order.end(), [&](int x, int y) {
    const int64_t a = mats[x].m * mats[x].n, b = mats[y].m * mats[y].n;
    return a != b ? a > b : mats[x].m > mats[y].m;
  });
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += ns_align(bytes);
    return static_cast<int64_t>(at);
  };
  p.status_off = take(sizeof(int32_t) * count);
  p.table_off = take(sizeof(NsDesc) * count);
  p.table.resize(count);
  for (int g = 0; g < count; ++g) {
    const NsMatrix& a = mats[order[g]];
    NsDesc d{};
    d.G = a.G;
    d.O = a.O;
    d.M = a.M;
    d.ldg = a.ldg;
    d.ldo = a.ldo;
    d.tall = a.m > a.n;
    d.p = static_cast<int32_t>(std::min(a.m, a.n));
    d.q = static_cast<int32_t>(std::max(a.m, a.n));
    d.slot = order[g];
    d.scale = a.scale;
    // partial sums of at least 2048 elements, at most kNsParts of them
    const int64_t total = a.m * a.n;
    d.chunk = std::max<int64_t>(2048, ns_cdiv(ns_cdiv(total, kNsParts), 1024) * 1024);
    d.parts = static_cast<int32_t>(ns_cdiv(total, d.chunk));
    int spp, sqp;
    const bool small = ns_small(d.p, d.q, spp, sqp);
    d.planes = small ? 0 : d.p <= kNsTinySide ? kNsFewRows : d.p <= kNsSmallSide ? 2 : planes;
    const size_t row = 2 * d.planes * ns_pad(d.p);
    if (d.planes == kNsFewRows) {
      const size_t sums = sizeof(float) * ns_row_chunks(d.q) * (spp * (spp + 1) / 2);
      d.oX = take(sizeof(float) * d.p * ns_row_pitch(d.q));
      d.oA = take(sums);
      d.oB = take(sums);
      d.oS = take(kNsParts * 8);
    } else if (!small) {
      d.oX = take(2 * row * ns_pitch(d.q, d.planes));
      d.oA = take(row * ns_pitch(d.p, d.planes));
      d.oB = take(row * ns_pitch(d.p, d.planes));
      d.oS = take(kNsParts * 8 + 16);
    }
    p.table[g] = d;
    if (g == 0 || mats[order[g]].m != mats[order[g - 1]].m || mats[order[g]].n != mats[order[g - 1]].n) {
      NsClass c{};
      c.first = g;
      c.planes = d.planes;
      c.spp = spp;
      c.sqp = sqp;
      p.shapes.push_back(c);
    }
    ++p.shapes.back().count;
  }
  p.count_off = take(sizeof(uint32_t) * kNsCounts);
  size_t part = 0;
  for (NsEpi epi : {kNsGram, kNsPoly, kNsApply})
    for (int n = 1; n <= 2; ++n)
      (void)ns_launches(p, NsLaunch{}, epi, n, [&](const NsLaunch&, const Cut16& c, int tile) {
        part = std::max(part, cut_bytes(c, tile));
        return hipSuccess;
      });
  p.part_off = take(part);
  p.bytes = off;
}

// Scales of one iteration's planes (powers of two) and the polynomial.
struct NsIter {
  double a, b, c;
  double sx, sa, sb;
};

// Bounds of the largest singular value before each iteration give the
// planes' scales: float16 holds up to 65504, and a plane's largest value is
// kept at 2^15 at most.  Returns false when the coefficients let singular
// values grow past kNsMaxGrowth.
constexpr double kNsMaxGrowth = 64.0;
bool ns_scales(const float* coeffs, int steps, std::vector<NsIter>& it) {
  auto pow2_below = [](double bound) {   // the power of two that brings `bound` to 2^14..2^15
    return std::ldexp(1.0, 15 - static_cast<int>(std::ceil(std::log2(std::max(bound * 1.01, 1e-3)))));
  };
  double u = 1.0;
  for (int k = 0; k < steps; ++k) {
    NsIter s;
    s.a = coeffs[3 * k];
    s.b = coeffs[3 * k + 1];
    s.c = coeffs[3 * k + 2];
    double poly = 0.0, next = 0.0;
    for (int i = 0; i <= 2048; ++i) {
      const double x = u * i / 2048, w = s.a + x * x * (s.b + x * x * s.c);
      poly = std::max(poly, std::fabs(w));
      next = std::max(next, std::fabs(x * w));
    }
    s.sx = pow2_below(u);
    s.sa = pow2_below(u * u);
    // B = a I + ... : its entries on an all-zero matrix are a itself
    s.sb = pow2_below(std::max(poly, std::fabs(s.a)));
    it.push_back(s);
    u = std::max(1.0, next * 1.01);
    if (!(u <= kNsMaxGrowth)) return false;
  }
  return true;
}

NsSmall ns_small_args(const NsLaunch& L, const std::vector<NsIter>& it, bool step) {
  NsSmall a{};
  a.common = L;
  a.common.x0 = static_cast<float>(it[0].sx);
  a.steps = static_cast<int32_t>(it.size());
  a.step = step;
  for (size_t k = 0; k < it.size(); ++k) {
    const NsIter& s = it[k];
    const double next = k + 1 < it.size() ? it[k + 1].sx : 1.0;
    a.it[k] = {static_cast<float>(s.sa / (s.sx * s.sx)), static_cast<float>(s.c * s.sb / (s.sa * s.sa)),
               static_cast<float>(s.b * s.sb / s.sa), static_cast<float>(s.a * s.sb),
               static_cast<float>(next / (s.sb * s.sx))};
    a.coef[k][0] = static_cast<float>(s.a);
    a.coef[k][1] = static_cast<float>(s.b);
    a.coef[k][2] = static_cast<float>(s.c);
  }
  return a;
}

// The stages of k_ns_rows, over the matrices of each number of rows.
hipError_t ns_rows(const NsPlan& p, const NsLaunch& base, const std::vector<NsIter>& it, bool step, hipStream_t st) {
  const auto few = [](const NsClass& c) { return c.planes == kNsFewRows; };
  if (std::none_of(p.shapes.begin(), p.shapes.end(), few)) return hipSuccess;
  const int steps = static_cast<int>(it.size());
  for (int stage = 0; stage <= steps; ++stage)
    for (const int rows : {1, 2, 4, 8, 16})
      NS_TRY(ns_grouped(p, base, [=](const NsClass& c) { return few(c) && c.spp == rows; },
                        [](const NsDesc& d, NsClass& c) { c.tiles = ns_row_chunks(d.q); },
                        [&](const NsLaunch& K) {
                          const NsIter s = stage > 0 ? it[stage - 1] : NsIter{};
                          return launch_ns_rows({K, stage, steps, step, static_cast<float>(s.a),
                                                 static_cast<float>(s.b), static_cast<float>(s.c)},
                                                rows, st);
                        }));
  return hipSuccess;
}

hipError_t ns_enqueue(NsPlan& p, NsLaunch L, const std::vector<NsIter>& it, bool step,
                      char* ws, hipStream_t st) {
  L.ws = ws;
  L.status = reinterpret_cast<int32_t*>(ws + p.status_off);
  L.count = reinterpret_cast<uint32_t*>(ws + p.count_off);
  L.part = reinterpret_cast<float*>(ws + p.part_off);
  const int count = static_cast<int>(p.table.size());
  if (count == 1) {
    L.inl = p.table[0];
  } else {
    // the table travels in kernel arguments: no host buffer has to outlive
    // the call, and a captured graph holds it
    NsDesc* dst = reinterpret_cast<NsDesc*>(ws + p.table_off);
    for (int g = 0; g < count; g += kNsUpload) {
      NsUpload u{};
      u.count = std::min(kNsUpload, count - g);
      std::copy_n(p.table.begin() + g, u.count, u.d);
      u.dst = dst + g;
      NS_TRY(launch_ns_table(u, st));
    }
    L.table = dst;
  }
  constexpr int kForms[][2] = {{64, 128}, {64, 256}, {64, 512}, {128, 128}, {128, 256},
                               {1, 0}, {2, 0}, {4, 0}, {8, 0}, {16, 0}};
  for (const auto& form : kForms) {   // the one-workgroup forms
    const int spp = form[0], sqp = form[1];
    NS_TRY(ns_grouped(p, L, [=](const NsClass& c) { return c.planes == 0 && c.spp == spp && c.sqp == sqp; },
                      [](const NsDesc&, NsClass& c) { c.tiles = 1; },
                      [&](const NsLaunch& K) {
                        const NsSmall a = ns_small_args(K, it, step);
                        return sqp == 0 ? launch_ns_tiny(a, spp, st) : launch_ns_small(a, spp, sqp, st);
                      }));
  }
  NS_TRY(ns_grouped(p, L, [](const NsClass& c) { return c.planes != 0; },
                    [](const NsDesc& d, NsClass& c) { c.tiles = d.parts; },
                    [&](const NsLaunch& K) { return launch_ns_norm(K, st); }));
  NS_TRY(ns_rows(p, L, it, step, st));
  L.x0 = static_cast<float>(it[0].sx);
  for (int planes = 1; planes <= 2; ++planes)
    NS_TRY(ns_grouped(p, L, [=](const NsClass& c) { return c.planes == planes; }, [](const NsDesc& d, NsClass& c) {
      c.tx = static_cast<int32_t>(ns_pad(d.p) / 64);
      c.ty = static_cast<int32_t>(ns_pad(d.q) / 64);
      c.tiles = c.tx * c.ty;
    }, [&](const NsLaunch& K) { return launch_ns_load(K, planes, st); }));
  const int steps = static_cast<int>(it.size());
  for (int k = 0; k < steps; ++k) {
    const NsIter& s = it[k];
    L.src = k & 1;
    L.tau = k == 0 ? 2 : 0;
    L.f_a = 0.0f;
    if (s.c == 0.0) {
      L.f_acc = static_cast<float>(s.b * s.sb / (s.sx * s.sx));
      L.f_i = static_cast<float>(s.a * s.sb);
      NS_TRY(ns_product(p, L, kNsGramPoly, st));
    } else {
      L.f_acc = static_cast<float>(s.sa / (s.sx * s.sx));
      L.f_i = 0.0f;
      NS_TRY(ns_product(p, L, kNsGram, st));
      L.tau = 0;
      L.f_acc = static_cast<float>(s.c * s.sb / (s.sa * s.sa));
      L.f_a = static_cast<float>(s.b * s.sb / s.sa);
      L.f_i = static_cast<float>(s.a * s.sb);
      NS_TRY(ns_product(p, L, kNsPoly, st));
    }
    L.tau = k == 0 ? 1 : 0;
    const bool last = k == steps - 1;
    L.f_acc = static_cast<float>((last ? 1.0 : it[k + 1].sx) / (s.sb * s.sx));
    NS_TRY(ns_product(p, L, !last ? kNsApply : step ? kNsStep : kNsOut, st));
  }
  return hipSuccess;
}

int ns_run(const std::vector<NsMatrix>& mats, const NsLaunch& base, const float* coeffs, int steps,
           int math, bool step, void* workspace, size_t workspace_bytes, void* stream) {
  int planes;
  if (!ns_math(math, planes) || !coeffs || steps < 1 || steps > kNsMaxSteps) return DION_ERR_INVALID_ARG;
  for (int i = 0; i < 3 * steps; ++i)
    if (!std::isfinite(coeffs[i])) return DION_ERR_INVALID_ARG;
  if (base.gdtype != DION_DTYPE_F32 && base.gdtype != DION_DTYPE_BF16) return DION_ERR_INVALID_ARG;
  if (base.odtype != DION_DTYPE_F32 && base.odtype != DION_DTYPE_BF16) return DION_ERR_INVALID_ARG;
  for (const NsMatrix& a : mats) {
    const int rc = ns_validate(a, base.gdtype, base.odtype, step);
    if (rc != DION_OK) return rc;
  }
  std::vector<NsIter> it;
  if (!ns_scales(coeffs, steps, it)) return DION_ERR_INVALID_ARG;
  NsPlan p;
  ns_layout(mats, planes, p);
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 != 0 || workspace_bytes < p.bytes)
    return DION_ERR_WORKSPACE;
  return ns_enqueue(p, base, it, step, static_cast<char*>(workspace),
                    static_cast<hipStream_t>(stream)) == hipSuccess
             ? DION_OK
             : DION_ERR_HIP;
}

size_t ns_size(const std::vector<NsMatrix>& mats, int math) {
  int planes;
  if (!ns_math(math, planes)) return 0;
  for (const NsMatrix& a : mats)
    if (!ns_shape_ok(a)) return 0;
  NsPlan p;
  ns_layout(mats, planes, p);
  return p.bytes;
}

std::vector<NsMatrix> ns_list(const dion_ns_matrix* mats, int count) {
  std::vector<NsMatrix> v(count);
  for (int i = 0; i < count; ++i)
    v[i] = {mats[i].G, mats[i].O, nullptr, mats[i].m, mats[i].n, mats[i].ldg, mats[i].ldo, 0.0f};
  return v;
}

std::vector<NsMatrix> ns_list(const dion_muon_matrix* mats, int count, float lr) {
  std::vector<NsMatrix> v(count);
  for (int i = 0; i < count; ++i)
    v[i] = {mats[i].G, mats[i].X, mats[i].M, mats[i].m, mats[i].n, mats[i].n, mats[i].n, lr * mats[i].scale};
  return v;
}

// No exception crosses the C boundary: the host side allocates vectors.
template <class F>
int ns_guard(F&& f) {
  try {
    return f();
  } catch (...) {
    return DION_ERR_HIP;
  }
}

}  // namespace
}  // namespace dion

using namespace dion;

DION_API size_t dion_orthogonalize_workspace_size(const dion_ns_matrix* mats, int count, int math) {
  if (!mats || count < 1 || count > DION_MAX_LIST) return 0;
  try {
    return ns_size(ns_list(mats, count), math);
  } catch (...) {
    return 0;
  }
}

DION_API int dion_orthogonalize_batched(const dion_ns_matrix* mats, int count, const float* coeffs,
                                        int steps, int math, int g_dtype, int o_dtype,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  if (!mats || count < 1 || count > DION_MAX_LIST) return DION_ERR_INVALID_ARG;
  return ns_guard([&] {
    NsLaunch L{};
    L.gdtype = g_dtype;
    L.odtype = o_dtype;
    return ns_run(ns_list(mats, count), L, coeffs, steps, math, false, workspace, workspace_bytes, stream);
  });
}

DION_API int dion_orthogonalize(const void* G, int64_t ldg, void* O, int64_t ldo, int64_t m, int64_t n,
                                const float* coeffs, int steps, int math, int g_dtype, int o_dtype,
                                void* workspace, size_t workspace_bytes, void* stream) {
  const dion_ns_matrix a = {G, O, m, n, ldg, ldo};
  return dion_orthogonalize_batched(&a, 1, coeffs, steps, math, g_dtype, o_dtype, workspace,
                                    workspace_bytes, stream);
}

DION_API size_t dion_muon_workspace_size(const dion_muon_matrix* mats, int count, int math) {
  if (!mats || count < 1 || count > DION_MAX_LIST) return 0;
  try {
    return ns_size(ns_list(mats, count, 0.0f), math);
  } catch (...) {
    return 0;
  }
}

DION_API int dion_muon_step_batched(const dion_muon_matrix* mats, int count, float lr, float momentum,
                                    int nesterov, float weight_decay, const float* coeffs, int steps,
                                    int math, int g_dtype, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  if (!mats || count < 1 || count > DION_MAX_LIST) return DION_ERR_INVALID_ARG;
  const float decay = 1.0f - lr * weight_decay;
  if (!std::isfinite(lr) || !std::isfinite(momentum) || !std::isfinite(weight_decay) || !std::isfinite(decay))
    return DION_ERR_INVALID_ARG;
  return ns_guard([&] {
    NsLaunch L{};
    L.gdtype = g_dtype;
    L.odtype = DION_DTYPE_F32;
    L.mu = momentum;
    L.nesterov = nesterov != 0;
    L.decay = decay;
    return ns_run(ns_list(mats, count, lr), L, coeffs, steps, math, true, workspace, workspace_bytes, stream);
  });
}

DION_API int dion_muon_step(float* X, const void* G, float* M, int64_t m, int64_t n, float scale,
                            float lr, float momentum, int nesterov, float weight_decay,
                            const float* coeffs, int steps, int math, int g_dtype, void* workspace,
                            size_t workspace_bytes, void* stream) {
  const dion_muon_matrix a = {X, G, M, m, n, scale};
  return dion_muon_step_batched(&a, 1, lr, momentum, nesterov, weight_decay, coeffs, steps, math,
                                g_dtype, workspace, workspace_bytes, stream);
}
