// Launchers of the tiled products by group: declared for the host unit, defined and explicitly
// instantiated by grouped_unit.hip, which is compiled once per (element type, product, copy mode).
#pragma once

#include "grouped_kernels.hpp"
#include "product_launch.hpp"

namespace spg {

// The products, by how their operands are stored.
enum {
    kRowsGatedNK = 0,    // two matrices [N,K], gated epilogue
    kRowsGatedKN = 1,    // two matrices [K,N]
    kRowsSumNK = 2,      // [dG dU] with matrices [N,K]: one sum over both, B reduction-major
    kRowsSumKN = 3,      // [dG dU] with matrices [K,N]
    kRowsNK = 4,         // one matrix, stored along the reduction
    kRowsKN = 5,         // one matrix, stored across it
    kGroupWeights = 6,   // gradients of the matrices
    kGroupProducts = 7
};

// Tile classes: those of product_launch.hpp, and Thin for groups of few rows, whose time is the
// reading of their matrices: 32 rows (one row of waves), so that nearly all of the ring's LDS
// holds parts of the matrices, and two workgroups a CU.
enum { kTileThin = kTiles, kGroupTiles = kTiles + 1 };
constexpr int kGroupTileM[kGroupTiles] = {256, 256, 128, 64, 64, 128, 32};
constexpr int group_tile_n(int tile, int mats) { return kTileN[tile == kTileThin ? (int)kTileMid : tile] / mats; }   // of one result

// `per`: workgroups of a group (kGroupWeights);
// GATHER: rows of X by their source (kRowsGated*, kRowsNK and kRowsKN only)
template <int ET, int P, bool REG, bool GATHER>
void launch_grouped(int tile, const ProductArgs& a, const GroupArgs& g, int per, dim3 grid, hipStream_t st);

// The sums of the last round's parts
constexpr int64_t part_bytes(int tile) { return (int64_t)kRound * kGroupTileM[tile] * group_tile_n(tile, 1) * 4; }

// dX and dW in one launch (tiles Mid and Small); P: kRowsSumNK, kRowsSumKN, kRowsNK or kRowsKN
template <int ET, int P, bool REG>
void launch_group_gradients(int tile, const ProductArgs& x, const ProductArgs& w, const GroupArgs& g, int nx, int per, dim3 grid,
                            hipStream_t st);

#ifdef SPG_DEFINE_GROUPED
template <int ET, int P, bool REG, bool GATHER, int BM, int BN, int WM, int WN, int S, bool DEEP, int KG, bool TAIL, int WPS>
void launch_group_kernel(const ProductArgs& a, const GroupArgs& g, int per, dim3 grid, hipStream_t st) {
    constexpr bool DUAL = P == kRowsGatedNK || P == kRowsGatedKN, SEG = P == kRowsSumNK || P == kRowsSumKN;
    constexpr bool BN_ = P == kRowsGatedKN || P == kRowsSumNK || P == kRowsKN;
    const dim3 wg(ProductGeom<DUAL, BM, BN, WM, WN, S, DEEP, KG>::NT);
    if constexpr (P == kGroupWeights)
        hipLaunchKernelGGL((grouped_weights<ET, REG, BM, BN, WM, WN, S, DEEP, KG, WPS>), grid, wg, 0, st, a, g, per);
    else
        hipLaunchKernelGGL((grouped_rows<ET, BN_, DUAL, SEG, REG, BM, BN, WM, WN, S, DEEP, KG, TAIL, WPS, GATHER>), grid, wg, 0, st, a, g);
}

// Tails as in launch_tile (product_launch.hpp)
template <int ET, int P, bool REG, bool GATHER, int BM, int BN, int WM, int WN, int S, bool DEEP, int KG, int WPS = 1>
void launch_group_tile(const ProductArgs& a, const GroupArgs& g, int per, dim3 grid, hipStream_t st) {
    if constexpr (P == kGroupWeights || P == kRowsSumNK) {
        launch_group_kernel<ET, P, REG, GATHER, BM, BN, WM, WN, S, DEEP, KG, false, WPS>(a, g, per, grid, st);
    } else if constexpr (BM == 256 && !REG) {
        if (a.K % 8 == 0) launch_group_kernel<ET, P, REG, GATHER, BM, BN, WM, WN, S, DEEP, KG, false, WPS>(a, g, per, grid, st);
        else launch_group_kernel<ET, P, REG, GATHER, BM, BN, WM, WN, S, BN == 256, KG, true, WPS>(a, g, per, grid, st);
    } else {
        launch_group_kernel<ET, P, REG, GATHER, BM, BN, WM, WN, S, DEEP, KG, true, WPS>(a, g, per, grid, st);
    }
}

template <int ET, int P, bool REG, bool GATHER>
void launch_grouped(int tile, const ProductArgs& a, const GroupArgs& g, int per, dim3 grid, hipStream_t st) {
    constexpr bool DUAL = P == kRowsGatedNK || P == kRowsGatedKN;
    // the ping-pong schedule as in launch_product
    constexpr bool DEEP = P != kRowsGatedKN && P != kGroupWeights;
    if constexpr (!REG) {
        if (tile == kTileBig) {
            if constexpr (DUAL) launch_group_tile<ET, P, REG, GATHER, 256, 256, 64, 128, 2, DEEP, 1>(a, g, per, grid, st);
            else launch_group_tile<ET, P, REG, GATHER, 256, 256, 128, 64, 2, DEEP, 1>(a, g, per, grid, st);
        } else if (tile == kTileTall) {   // the matrices' gradients only
            if constexpr (P == kGroupWeights) launch_group_tile<ET, P, REG, GATHER, 256, 128, 64, 64, 3, false, 1>(a, g, per, grid, st);
        } else if (tile == kTileMid) {    // rows only
            if constexpr (P != kGroupWeights) launch_group_tile<ET, P, REG, GATHER, 128, 128, 32, 64, 4, false, 1>(a, g, per, grid, st);
        } else if (tile == kTilePair) {
            launch_group_tile<ET, P, REG, GATHER, 128, 128, 32, 64, 2, false, 1, 4>(a, g, per, grid, st);
        } else if (tile == kTileThin) {
            if constexpr (DUAL) launch_group_tile<ET, P, REG, GATHER, 32, 128, 32, 64, 4, false, 1>(a, g, per, grid, st);
            else if constexpr (P != kGroupWeights) launch_group_tile<ET, P, REG, GATHER, 32, 128, 32, 32, 4, false, 1, 2>(a, g, per, grid, st);
        } else if (tile == kTileSmall) {
            launch_group_tile<ET, P, REG, GATHER, 64, 128, 32, 64, 3, false, 2>(a, g, per, grid, st);
        } else {
            launch_group_tile<ET, P, REG, GATHER, 64, 64, 32, 64, 2, false, 4>(a, g, per, grid, st);
        }
    } else {
        if (tile == kTileTall) {
            if constexpr (P == kGroupWeights) launch_group_tile<ET, P, REG, GATHER, 256, 128, 64, 64, 2, false, 1>(a, g, per, grid, st);
        } else if (tile == kTileMid) {
            if constexpr (P != kGroupWeights) launch_group_tile<ET, P, REG, GATHER, 128, 128, 32, 64, 2, false, 1>(a, g, per, grid, st);
        } else if (tile == kTileThin) {
            if constexpr (DUAL) launch_group_tile<ET, P, REG, GATHER, 32, 128, 32, 64, 2, false, 1>(a, g, per, grid, st);
            else if constexpr (P != kGroupWeights) launch_group_tile<ET, P, REG, GATHER, 32, 128, 32, 32, 2, false, 1, 2>(a, g, per, grid, st);
        } else if (tile == kTileSmall) launch_group_tile<ET, P, REG, GATHER, 64, 128, 32, 64, 2, false, 1>(a, g, per, grid, st);
        else launch_group_tile<ET, P, REG, GATHER, 64, 64, 32, 64, 2, false, 4>(a, g, per, grid, st);
    }
}
template <int ET, int P, bool REG, int BM, int BN, int WM, int WN, int S, int KG>
void launch_both(const ProductArgs& x, const ProductArgs& w, const GroupArgs& g, int nx, int per, dim3 grid, hipStream_t st) {
    constexpr bool SEG = P == kRowsSumNK || P == kRowsSumKN, BN_ = P == kRowsSumNK || P == kRowsKN;
    hipLaunchKernelGGL((grouped_gradients<ET, BN_, SEG, REG, BM, BN, WM, WN, S, KG>), grid,
                       dim3(ProductGeom<false, BM, BN, WM, WN, S, false, KG>::NT), 0, st, x, w, g, nx, per);
}

template <int ET, int P, bool REG>
void launch_group_gradients(int tile, const ProductArgs& x, const ProductArgs& w, const GroupArgs& g, int nx, int per, dim3 grid,
                            hipStream_t st) {
    if constexpr (!REG) {
        if (tile == kTileMid) launch_both<ET, P, REG, 128, 128, 32, 64, 4, 1>(x, w, g, nx, per, grid, st);
        else launch_both<ET, P, REG, 64, 128, 32, 64, 3, 2>(x, w, g, nx, per, grid, st);
    } else {
        if (tile == kTileMid) launch_both<ET, P, REG, 128, 128, 32, 64, 2, 1>(x, w, g, nx, per, grid, st);
        else launch_both<ET, P, REG, 64, 128, 32, 64, 2, 1>(x, w, g, nx, per, grid, st);
    }
}
#endif

}  // namespace spg
