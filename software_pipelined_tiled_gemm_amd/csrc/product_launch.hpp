// Launchers of the feed-forward operators' kernels: declared for the host unit, defined and
// explicitly instantiated by product_unit.hip, which is compiled once per (element type,
// product, copy mode) so that the units build in parallel.
#pragma once

#include <hip/hip_runtime.h>

#include "product_kernels.hpp"

namespace spg {

// The products, by how their operands are stored.
enum {
    kGatedNK = 0,     // X [M,K] with two weights [N,K]
    kGatedKN = 1,     // X [M,K] with two weights [K,N]
    kGradXNK = 2,     // [dG dU] with weights [N,K]: B is stored reduction-major
    kGradXKN = 3,     // [dG dU] with weights [K,N]
    kGradW = 4,       // both operands reduction-major
    kInt8 = 5,        // int8, one B
    kInt8Gated = 6,   // int8, two B
    kProducts = 7
};

// Tile classes: rows x columns of a workgroup's tile (DUAL: columns of both matrices)
// Pair: two workgroups share a CU (64 KiB of LDS and at most 128 registers each), so that
// one's start and store overlap the other's k-tiles: for short reductions
enum { kTileBig = 0, kTileTall = 1, kTileMid = 2, kTileSmall = 3, kTileNarrow = 4, kTilePair = 5, kTiles = 6 };
constexpr int kTileM[kTiles] = {256, 256, 128, 64, 64, 128};
constexpr int kTileN[kTiles] = {256, 128, 128, 128, 64, 128};

template <int ET, int P, bool REG>
void launch_product(int tile, const ProductArgs& a, dim3 grid, hipStream_t st);

// dX, then dWg and dWu, in one launch of nx + nw workgroups (tiles Mid and Small); P says
// how the weights are stored (kGradXNK, kGradXKN)
template <int ET, int P, bool REG>
void launch_gradients(int tile, const ProductArgs& x, const ProductArgs& w, int nx, dim3 grid, hipStream_t st);

#ifdef SPG_DEFINE_PRODUCT
template <int ET, int P, bool REG, int BM, int BN, int WM, int WN, int S, bool DEEP, int KG, bool TAIL, int WPS>
void launch_kernel(const ProductArgs& a, dim3 grid, hipStream_t st) {
    constexpr bool AT = P == kGradW, BNC = P == kGatedKN || P == kGradXNK || P == kGradW;
    constexpr bool DUAL = P == kGatedNK || P == kGatedKN || P == kInt8Gated;
    constexpr bool SEG = P == kGradXNK || P == kGradXKN;
    hipLaunchKernelGGL((product_kernel<ET, AT, BNC, DUAL, SEG, REG, BM, BN, WM, WN, S, DEEP, KG, TAIL, WPS>), grid,
                       dim3(ProductGeom<DUAL, BM, BN, WM, WN, S, DEEP, KG>::NT), 0, st, a);
}

// The 256-row tiles of direct copies are compiled with and without the tails of rows (sums
// that end inside a 16-byte chunk).  Clearing them cuts the blocks of the compiler-placed
// schedule (gated, 4096 x 4096 of 2046, weights [K,N]: 188 us against 102 of 2048): with
// them every 256x256 tile runs the ping-pong.
template <int ET, int P, bool REG, int BM, int BN, int WM, int WN, int S, bool DEEP, int KG, int WPS = 1>
void launch_tile(const ProductArgs& a, dim3 grid, hipStream_t st) {
    constexpr int ES = ET == kElI8 ? 1 : 2;
    if constexpr (P == kGradW || P == kGradXNK) {
        // no operand's rows end inside a chunk: both across the reduction, or dG and dU padded
        launch_kernel<ET, P, REG, BM, BN, WM, WN, S, DEEP, KG, false, WPS>(a, grid, st);
    } else if constexpr (BM == 256 && !REG) {
        if (a.K * ES % 16 == 0) launch_kernel<ET, P, REG, BM, BN, WM, WN, S, DEEP, KG, false, WPS>(a, grid, st);
        else launch_kernel<ET, P, REG, BM, BN, WM, WN, S, BN == 256, KG, true, WPS>(a, grid, st);
    } else {
        launch_kernel<ET, P, REG, BM, BN, WM, WN, S, DEEP, KG, true, WPS>(a, grid, st);
    }
}

template <int ET, int P, bool REG>
void launch_product(int tile, const ProductArgs& a, dim3 grid, hipStream_t st) {
    constexpr bool DUAL = P == kGatedNK || P == kGatedKN || P == kInt8Gated;
    // The ping-pong schedule and its deeper ring (DEEP) where B is K-contiguous and for the
    // long sum of the input gradient; the compiler-placed one on two slots where the
    // reduction-major reads need more addresses (training step of 2048 rows: forward 35 us
    // against 39, weight gradients of 12288 x 4096 593 against 672).
    constexpr bool DEEP = P != kGatedKN && P != kGradW;
    if constexpr (!REG) {
        if (tile == kTileBig) {
            // DUAL: 64 x 128 per wave, so that a wave's output rows are whole 128-byte lines
            if constexpr (DUAL) launch_tile<ET, P, REG, 256, 256, 64, 128, 2, DEEP, 1>(a, grid, st);
            else launch_tile<ET, P, REG, 256, 256, 128, 64, 2, DEEP, 1>(a, grid, st);
        } else if (tile == kTileTall) {
            launch_tile<ET, P, REG, 256, 128, 64, 64, 3, false, 1>(a, grid, st);
        } else if (tile == kTileMid) {
            launch_tile<ET, P, REG, 128, 128, 32, 64, 4, false, 1>(a, grid, st);
        } else if (tile == kTilePair) {
            launch_tile<ET, P, REG, 128, 128, 32, 64, 2, false, 1, 4>(a, grid, st);
        } else if (tile == kTileSmall) {
            launch_tile<ET, P, REG, 64, 128, 32, 64, 3, false, 2>(a, grid, st);
        } else {
            launch_tile<ET, P, REG, 64, 64, 32, 64, 2, false, 4>(a, grid, st);
        }
    } else {
        if (tile == kTileTall) launch_tile<ET, P, REG, 256, 128, 64, 64, 2, false, 1>(a, grid, st);
        else if (tile == kTileMid) launch_tile<ET, P, REG, 128, 128, 32, 64, 2, false, 1>(a, grid, st);
        else if (tile == kTileSmall) launch_tile<ET, P, REG, 64, 128, 32, 64, 2, false, 1>(a, grid, st);
        else launch_tile<ET, P, REG, 64, 64, 32, 64, 2, false, 4>(a, grid, st);
    }
}

template <int ET, int P, bool REG, int BM, int BN, int WM, int WN, int S, int KG>
void launch_gradient_tile(const ProductArgs& x, const ProductArgs& w, int nx, dim3 grid, hipStream_t st) {
    hipLaunchKernelGGL((gradients_kernel<ET, P == kGradXNK, REG, BM, BN, WM, WN, S, KG>), grid,
                       dim3(ProductGeom<false, BM, BN, WM, WN, S, false, KG>::NT), 0, st, x, w, nx);
}

template <int ET, int P, bool REG>
void launch_gradients(int tile, const ProductArgs& x, const ProductArgs& w, int nx, dim3 grid, hipStream_t st) {
    if constexpr (!REG) {
        if (tile == kTileMid) launch_gradient_tile<ET, P, REG, 128, 128, 32, 64, 4, 1>(x, w, nx, grid, st);
        else launch_gradient_tile<ET, P, REG, 64, 128, 32, 64, 3, 2>(x, w, nx, grid, st);
    } else {
        if (tile == kTileMid) launch_gradient_tile<ET, P, REG, 128, 128, 32, 64, 2, 1>(x, w, nx, grid, st);
        else launch_gradient_tile<ET, P, REG, 64, 128, 32, 64, 2, 1>(x, w, nx, grid, st);
    }
}
#endif

}  // namespace spg
