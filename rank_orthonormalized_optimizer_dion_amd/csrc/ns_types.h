// Types and launchers of the Newton-Schulz orthogonalization (k_ns.hip,
// ns_api.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dion {

constexpr int kNsPad = 64;        // rows and columns of every plane are padded to this, with zeros
constexpr int kNsParts = 512;     // most partial sums of squares per matrix
constexpr int kNsMaxClasses = 8;
constexpr int kNsCounts = 512;    // arrival counters of cut tiles (at most the chip's workgroup slots)
constexpr int kNsUpload = 24;     // descriptors per table upload (kernel arguments: under 4 KB)
constexpr int32_t kNsNonFinite = 8;   // status bit: DION_STATUS_NONFINITE
inline __host__ __device__ int64_t ns_pad(int64_t x) { return (x + kNsPad - 1) / kNsPad * kNsPad; }
// Row pitch (values) of a plane of x columns: an odd number of 256-byte
// units, the granularity at which addresses go round the L2 channels.  A
// tile reads a piece of the same columns of many rows at once; at a pitch of
// a power of two all of them come from one channel.
inline __host__ __device__ int64_t ns_pitch(int64_t x, int planes) {
  const int64_t unit = 128 / planes;
  return ((ns_pad(x) + unit - 1) / unit | 1) * unit;
}

// One matrix, seen from its smaller side: the planes hold the p x q matrix
// (p <= q) that is G or, when G has more rows than columns (tall), its
// transpose.  Offsets are bytes from the workspace base.
struct NsDesc {
  const void* G;    // m x n, pitch ldg
  void* O;          // orthogonalize: the output (pitch ldo); step: the weights X (float32)
  float* M;         // step: the momentum; else null
  int64_t ldg, ldo;
  int32_t p, q;
  int32_t tall;
  int32_t slot;     // index in the caller's list = status word index
  int32_t parts;    // partial sums of squares
  int32_t planes;   // as NsClass
  float scale;      // step: the update's factor lr * s
  int64_t chunk;    // elements of G per partial sum
  // pp = ns_pad(p), qp = ns_pad(q), 16-bit, `planes` per value (mm16.h),
  // pitches ns_pitch (kNsFewRows: X in float32, pitch ns_row_pitch; oA, oB
  // the chunks' sums of A in turn):
  int64_t oX;       // two buffers of pp x qp (X and the next X)
  int64_t oA, oB;   // pp x pp each: A = X X^T, B = a I + b A + c A^2
  int64_t oS;       // parts float64, then the normalization tau (float32)
};

struct NsClass {
  int32_t planes;         // 16-bit planes per value: 1 or 2; 0: the one-workgroup form; kNsFewRows
  int32_t spp, sqp;       // its padded sides; sqp = 0: k_ns_tiny or k_ns_rows with spp >= p rows
  int32_t first, count;   // matrices of this shape in the table
  int32_t tiles, base;    // work items per matrix, first item
  int32_t tx, ty;         // tile grid
};

// What a product's epilogue does.
enum NsEpi : int32_t {
  kNsGram = 0,    // A = X X^T
  kNsGramPoly,    // B = a I + b X X^T (cubic iterations: no A^2)
  kNsPoly,        // B = a I + b A + c A A^T
  kNsApply,       // next X = B X
  kNsOut,         // output = B X
  kNsStep,        // X <- decay X - scale (B X)
};

struct NsLaunch {
  const NsDesc* table;    // device table, or null to use `inl`
  NsDesc inl;
  char* ws;
  int32_t* status;
  int32_t nclass, total;
  NsClass cls[kNsMaxClasses];
  float mu;               // step: momentum; nesterov: D = G + mu M, else D = M
  int32_t nesterov;
  float decay;            // step: 1 - lr * weight decay
  float x0;               // power-of-two scale of the first X's planes
  float f_acc, f_a, f_i;  // epilogue: f_acc * product + f_a * A + f_i * I
  int32_t tau;            // f_acc is multiplied by tau^this (first iteration)
  int32_t src;            // which of the two X buffers is read
  int32_t gdtype, odtype; // 0 float32, 1 bfloat16
  int32_t full, slices;   // mm16.h, Work16 (total counts tiles)
  float* part;
  uint32_t* count;
};

// The one-workgroup form (k_ns_small): every iteration's factors at once.
constexpr int kNsMaxSteps = 32;
struct NsSmall {
  struct Iter {
    float f_gram, f_acc, f_a, f_i, f_apply;   // f_acc = 0: no A^2 (cubic)
  };
  NsLaunch common;        // classes (tiles = 1), status, momentum, types
  int32_t steps, step;    // step: Muon step, else the output is written
  Iter it[kNsMaxSteps];
  float coef[kNsMaxSteps][3];   // a, b, c (k_ns_tiny)
};
// k_ns_tiny: p <= 16 and p q <= kNsTinyFloats, X in LDS as float32
constexpr int kNsTinySide = 16;
constexpr int kNsTinyFloats = 32768;

// k_ns_rows: p <= 16 beyond that.  Columns of a workgroup, at most 256
// workgroups.
constexpr int32_t kNsFewRows = 3;
constexpr int kNsRowThreads = 512;
constexpr int kNsRowChunks = 256;
inline __host__ __device__ int ns_row_cols(int q) {
  constexpr int unit = kNsRowThreads * kNsRowChunks;
  return (q + unit - 1) / unit * kNsRowThreads;
}
inline __host__ __device__ int64_t ns_row_pitch(int q) { return (static_cast<int64_t>(q) + 63) / 64 * 64; }
struct NsRows {
  NsLaunch common;        // classes (tiles: chunks of columns), status, momentum, types
  int32_t stage;          // 0: load; then iteration `stage` with a, b, c
  int32_t steps, step;    // step: Muon step, else the output is written
  float a, b, c;
};

struct NsUpload {
  NsDesc d[kNsUpload];
  NsDesc* dst;
  int32_t count;
};

hipError_t launch_ns_table(const NsUpload& u, hipStream_t st);
// pp, qp: (64, 128), (64, 256), (64, 512), (128, 128) or (128, 256)
hipError_t launch_ns_small(const NsSmall& L, int pp, int qp, hipStream_t st);
// p: 1, 2, 4, 8 or 16
hipError_t launch_ns_tiny(const NsSmall& L, int p, hipStream_t st);
hipError_t launch_ns_rows(const NsRows& L, int p, hipStream_t st);
hipError_t launch_ns_norm(const NsLaunch& L, hipStream_t st);
hipError_t launch_ns_load(const NsLaunch& L, int planes, hipStream_t st);
// tile: 128 or 256
hipError_t launch_ns_product(const NsLaunch& L, int items, NsEpi epi, int planes, int tile, hipStream_t st);
// tiles of a symmetric product over an nt x nt tile grid
inline int ns_sym_tiles(int nt) { return nt * (nt + 1) / 2; }

}  // namespace dion
