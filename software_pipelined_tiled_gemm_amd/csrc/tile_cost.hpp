// What a tile class costs: the host's choice of tile is made from these.
#pragma once

#include "product_launch.hpp"

namespace spg {

// Microseconds of a tile class: a k-tile, and a workgroup's start and store, with direct
// copies and register-staged (which has no 256x256 and no pair tile): fitted to the products of
// product.hip (see choose() there); grouped.hip has its own and takes the slots from here
constexpr double kTileUs[kTiles] = {1.27, 0.76, 0.51, 0.32, 0.26, 0.70};
constexpr double kStartUs[kTiles] = {5.3, 5.6, 2.5, 2.75, 2.75, 2.9};
constexpr double kStagedUs[kTiles] = {0.0, 1.30, 0.65, 0.48, 0.42, 0.0};
constexpr double kStagedStartUs[kTiles] = {0.0, 5.3, 3.8, 2.9, 3.3, 0.0};
// direct copies of rows that are not whole 128-byte lines: each 128-byte chunk of a k-tile is
// two lines' halves
constexpr double kCrooked[kTiles] = {1.08, 1.10, 1.05, 1.20, 1.14, 1.18};
// two workgroups on a CU: the pair tile, and the register-staged 64x128 one; alone on their
// CUs the first starts faster and both multiply faster, and a single round in pairs has
// nothing to overlap the starts and stores with
inline bool paired(int t, bool reg) { return t == (reg ? (int)kTileSmall : (int)kTilePair); }
inline double slots(int t, bool reg) { return paired(t, reg) ? 512.0 : 256.0; }
inline double tile_us(int t, bool reg, bool crooked, int64_t wgs) {
    const bool two = paired(t, reg) && wgs > 256;
    if (reg) return two ? 0.84 : kStagedUs[t];
    return (two ? (wgs > 512 ? 0.81 : 1.30) : kTileUs[t]) * (crooked ? kCrooked[t] : 1.0);
}
inline double start_us(int t, bool reg, int64_t wgs) {
    if (!reg && paired(t, reg) && wgs <= 256) return 1.0;
    return reg ? kStagedStartUs[t] : kStartUs[t];
}
constexpr double kLaunchUs = 1.5;

}  // namespace spg
