// How many workgroups a product's tiles take (host side of mm16.h's Work16).
#pragma once
#include <algorithm>
#include <cmath>
#include <cstdint>

namespace dion {

constexpr int kTileSlots256 = 256;   // one workgroup of 256 x 256 tiles per CU
constexpr int kTileSlots128 = 512;   // two of 128 x 128 tiles
inline int tile_slots(int tile) { return tile == 256 ? kTileSlots256 : kTileSlots128; }

// Reductions shorter than this are not cut.  Timed over 17 cases of 10 to 100
// stages: cutting from 10 stages on 8% to 42% slower in eleven (36 matrices of
// 768 rows 11%; linear, 1000 tokens, 768 -> 768 42%), 2% and 11% faster in two
// (130 x 1000; linear backward, 1000 tokens, 768 -> 768); from 80 on the same or
// slower (1000 x 1000 float32 26%).
constexpr int64_t kMinCutStages = 40;

struct Cut16 {
  int64_t full;    // tiles of one workgroup each
  int64_t cut;     // tiles cut into `slices`
  int64_t slices;
  int64_t items() const { return full + cut * slices; }
};

// `stages`: reduction stages (mm16.h) per tile.  The last round of tiles is
// cut until it fills the chip's slots, but not beyond sqrt(0.4 stages) slices,
// where adding up the slices' sums (each a tile of float32 through one
// workgroup, estimated at 2.5 stages) takes as long as a slice's products.
// Timed once each over seven cases in place of 0.4: 0.1 and 0.2 between 0.6%
// faster and 2.3% slower, 0.8 between 0.2% faster and 5.1% slower (the odd-sized
// list, 260 -> 273 us).
inline Cut16 cut_tiles(int64_t tiles, int tile, int64_t stages) {
  if (stages < kMinCutStages) return {tiles, 0, 1};
  const int64_t slots = tile_slots(tile);
  const int64_t full = tiles / slots * slots, rest = tiles - full;
  if (rest == 0) return {tiles, 0, 1};
  const int64_t most = static_cast<int64_t>(std::sqrt(0.4 * static_cast<double>(stages)));
  const int64_t slices = std::max<int64_t>(1, std::min(slots / rest, most));
  if (slices == 1) return {tiles, 0, 1};
  return {full, rest, slices};
}
inline size_t cut_bytes(const Cut16& c, int tile) {
  return static_cast<size_t>(c.cut * c.slices) * tile * tile * 4;
}

}  // namespace dion
