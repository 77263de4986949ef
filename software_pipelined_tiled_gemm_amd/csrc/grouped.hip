// C ABI of the products by group (gemm_grouped_* and gemm_experts_* in include/spgemm.h).
//
// Host side: argument validation (before any HIP call), the choice of kernel from the sizes,
// the workspace layout and the launches.  Nothing here knows how many rows a group has: the
// grids cover what the plan's rows can come to, and the kernels read the offsets.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "errors.hpp"
#include "grouped_launch.hpp"
#include "spgemm.h"
#include "tile_cost.hpp"

using spg::GroupArgs;
using spg::ProductArgs;

namespace {

constexpr int64_t kAlign = 256;   // sections of a workspace
int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// direct copies read from 4-byte aligned addresses
bool words(const void* p) { return (uintptr_t)p % 4 == 0; }

gemm_status launched() {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? GEMM_OK : spg::hip_fail(e);
}

// a launch has less than 2^32 threads along one axis, and one workgroup at least
dim3 spread(int64_t wgs) {
    const int64_t x = std::min<int64_t>(std::max<int64_t>(wgs, 1), 1 << 21);
    return dim3((unsigned)x, (unsigned)std::max<int64_t>(ceil_div(wgs, x), 1));
}

// Rows of operands are addressed by 32-bit offsets below 2^31: 256 of them fit up to here.
constexpr int64_t kMaxRowBytes = ((int64_t)1 << 23) - 128;
constexpr int64_t kMaxBytes = (int64_t)1 << 31;

// Sizes and layouts that the plain and the gated products share.
struct Common {
    int64_t rows, N, K, groups, tokens;   // tokens -1: no source
    bool bf, nk;
    int64_t matrix() const { return N * K * 2; }
    int64_t live() const { return std::max<int64_t>(1, std::min(groups, rows)); }   // groups that may have rows
    // the copy of X in the groups' order
    int64_t pitch() const { return up(K * 2, 128); }
    int64_t gathered() const { return tokens < 0 ? 0 : up(rows * pitch(), kAlign); }
};

gemm_status check(const void* out, int64_t rows, int64_t N, int64_t K, int64_t groups, int64_t tokens, gemm_dtype dtype,
                  gemm_b_layout layout) {
    if (!out || rows < 0 || N < 0 || K < 0 || groups < 1 || tokens < -1) return GEMM_ERR_INVALID_ARG;
    if (dtype != GEMM_F16 && dtype != GEMM_BF16) return GEMM_ERR_INVALID_ARG;
    if (layout != GEMM_B_KN && layout != GEMM_B_NK) return GEMM_ERR_INVALID_ARG;
    const int64_t lim = INT32_MAX / 2 - 512;
    if (rows > lim || N > lim || K > lim || tokens > lim || groups > 65535) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

bool wrong_source(const Common& c, const void* source) { return c.rows > 0 && (c.tokens < 0) != (source == nullptr); }

bool small_workspace(const void* workspace, int64_t bytes, int64_t need) {
    return need > 0 && (!workspace || (uintptr_t)workspace % 16 != 0 || bytes < need);
}

GroupArgs group_args(const Common& c, const int32_t* offsets, const int32_t* source) {
    return GroupArgs{offsets, source, nullptr, c.matrix(), (int32_t)c.groups, (int32_t)c.rows, (int32_t)std::max<int64_t>(c.tokens, 0)};
}

// ---- the choice of kernel --------------------------------------------------------------

// Products of all groups' rows with their matrices: `mats` B side by side in a tile, `kt` k-tiles.
struct RowsShape {
    int64_t rows, live, N, kt;
    int mats;
    double bytes;
};

// Row tiles of BM rows: the last tile of a group is half full on average.
double row_tiles(const RowsShape& s, int BM) {
    return std::max((double)s.live, (double)s.rows / BM + 0.5 * (double)s.live);
}

// What a tile class costs, in microseconds: a call takes
//     base + max(k-tiles * alone, rounds * (k-tiles * busy + tile), bytes / bw)
// with rounds the workgroups over the slots of the CUs: `alone` bounds a grid that leaves CUs
// idle (a k-tile's copies have to come in), `busy` and `tile` (a workgroup's start and store) one
// that fills them, and the matrices' reading (writing, for their gradients) at bw bytes a
// microsecond the rest.  Fitted to every class at 2500 drawn shapes (1 to 256 groups, 1 to 8192
// rows, matrices of 48 to 12288 x 40 to 4096).  Against the best of all classes, parts and the
// streaming kernel at 2500 other shapes, three in ten of them with few tiles and long reductions,
// the choice takes 4.2% more on average and 22% more at 5% of the shapes; for the gradients, 1.9% and 10%.
struct Cost {
    double alone, busy, tile, base, bw;   // bw 0: the class is not chosen
};
// 256x128 is nowhere more than 2% ahead of the others for rows, nor 128x128 for the gradients
constexpr Cost kNone{0, 0, 0, 0, 0};
constexpr Cost kRows[2][2][spg::kGroupTiles] = {   // [register-staged][two matrices]
    {{{0.93, 0.84, 2.5, 6.8, 5.8e6}, kNone, {0.36, 0.41, 2.0, 5.1, 7.4e6}, {0.27, 0.38, 2.4, 5.4, 8.3e6},
      {0.18, 0.26, 2.6, 5.5, 6.0e6}, {0.43, 0.88, 1.8, 4.8, 7.2e6}, {0.24, 0.57, 1.9, 4.3, 10.0e6}},
     {{0.86, 1.10, 2.8, 7.5, 5.9e6}, kNone, {0.37, 0.50, 2.1, 5.2, 7.1e6}, {0.29, 0.43, 2.6, 5.3, 7.3e6},
      {0.19, 0.29, 3.1, 5.6, 5.4e6}, {0.48, 1.05, 1.9, 4.8, 6.9e6}, {0.34, 1.31, 4.6, 4.5, 8.0e6}}},
    {{kNone, kNone, {0.64, 0.51, 2.1, 5.6, 6.6e6}, {0.61, 1.33, 1.5, 5.3, 8.3e6}, {0.32, 0.29, 3.2, 6.3, 6.0e6}, kNone,
      {0.53, 0.77, 1.3, 4.9, 8.8e6}},
     {kNone, kNone, {0.64, 0.56, 2.5, 5.6, 6.2e6}, {0.62, 1.46, 1.8, 5.1, 7.7e6}, {0.37, 0.31, 3.6, 6.4, 5.5e6}, kNone,
      {0.77, 1.84, 2.9, 4.9, 8.3e6}}}};
constexpr Cost kWeights[2][spg::kGroupTiles] = {
    {{0.91, 1.91, 4.4, 7.8, 6.3e6}, {0.49, 1.14, 2.8, 6.1, 5.0e6}, kNone, {0.19, 0.45, 2.4, 5.4, 5.0e6},
     {0.14, 0.37, 2.6, 5.5, 5.0e6}, {0.31, 1.22, 2.6, 4.9, 5.4e6}, kNone},
    {kNone, {0.88, 1.51, 3.4, 7.4, 3.4e6}, kNone, {0.62, 1.58, 3.4, 5.3, 5.0e6}, {0.34, 0.47, 3.2, 6.5, 5.0e6}, kNone, kNone}};
// ... of the tiles that both gradients may share a launch with
constexpr Cost kWeightsMid[2] = {{0.32, 0.67, 2.1, 5.1, 5.0e6}, {0.62, 0.92, 2.4, 6.0, 5.0e6}};

// Workgroups that the CUs hold at once
double slots(int t, bool reg) { return t == spg::kTileThin ? 512.0 : reg && t == spg::kTileSmall ? 768.0 : spg::slots(t, reg); }

double cost_us(const Cost& c, double rounds, double kt, double bytes) {
    return c.base + std::max(std::max(kt * c.alone, rounds * (kt * c.busy + c.tile)), bytes / c.bw);
}

struct Choice {
    int tile;     // -1: no class has few enough workgroups for a launch
    double us;    // estimated
    bool split;   // the last round's tiles (a grid of less than a round: all of them) in parts
    int parts;    // of the rows, for the matrices' gradients
};

// A launch has less than 2^32 threads, a workgroup up to 512.
constexpr int64_t kMostWgs = ((int64_t)1 << 23) - 2 * spg::kRound;

// The most workgroups that the rows can come to: every group with rows has at most one tile that is
// not full.
int64_t most_wgs(int64_t rows, int64_t live, int64_t N, int t, int mats) {
    const int64_t BM = spg::kGroupTileM[t];
    return ((rows - live) / BM + live) * ceil_div(N, spg::group_tile_n(t, mats));
}

double rows_wgs(const RowsShape& s, int t) {
    return row_tiles(s, spg::kGroupTileM[t]) * (double)ceil_div(s.N, spg::group_tile_n(t, s.mats));
}

// Long reductions of few tiles are split over the CUs that have none.  256x256 tiles are in their
// last round, too: past 12 rounds one is less than 8% of the call.  At 400 drawn shapes (1 to 32
// groups, 1 to 2048 rows, matrices of 32 to 2048 columns and reductions of 1024 to 12288) the best
// class with parts takes 0.27 to 1 of the time of the best without (5 columns of 736, 9728:
// 13 and 37 us).
// The matrices' gradients likewise (12432 rows of one group, 144 x 776, both gradients: 33 us, 77
// in one piece).
constexpr double kJoinUs[spg::kGroupTiles] = {0, 0, 0, 4.5, 4.0, 0, 3.5};   // the parts' launch, write and read; 0: not split
double split_us(const Cost& c, int t, double wgs, double all, double bytes, double& parts) {
    const int bm = spg::kGroupTileM[t], bn = spg::group_tile_n(t, 1);
    parts = std::min((double)spg::most_parts(bm, bn), std::floor(spg::kRound / wgs));
    if (kJoinUs[t] == 0 || parts < 2.0) return 1e30;
    const double kt = std::ceil(all / parts);
    if (all - kt < spg::split_gain(bm, bn)) return 1e30;
    return kJoinUs[t] + cost_us(c, std::min(1.0, wgs * parts / spg::kRound), kt, bytes);
}

Choice choose_rows(const RowsShape& s, bool reg) {
    Choice best{-1, 1e30, false, 1};
    for (int t = 0; t < spg::kGroupTiles; ++t) {
        const Cost& c = kRows[reg][s.mats == 2][t];
        if (c.bw == 0 || most_wgs(s.rows, s.live, s.N, t, s.mats) > kMostWgs) continue;
        double n;
        const double wgs = rows_wgs(s, t), us = cost_us(c, wgs / slots(t, reg), (double)s.kt, s.bytes);
        const double parts = split_us(c, t, wgs, (double)s.kt, s.bytes, n);
        const bool last = t == spg::kTileBig && s.kt >= 2 * spg::split_gain(256, 256) && wgs <= 12.0 * spg::kRound;
        if (us < best.us) best = Choice{t, us, last, 1};
        if (parts < best.us) best = Choice{t, parts, true, 1};
    }
    return best;
}

// Gradients of the matrices: `mats` results of every group, a reduction over its rows.
struct WeightsShape {
    int64_t groups, M, N;
    int mats;
    double kt, bytes;
};
WeightsShape weights_shape(const Common& c, int mats) {
    return WeightsShape{c.groups, c.nk ? c.N : c.K, c.nk ? c.K : c.N, mats, (double)c.rows / (double)c.groups / 64.0 + 0.5,
                        (double)mats * c.matrix() * c.groups};
}
double weights_wgs(const WeightsShape& s, int t) {
    return (double)s.groups * s.mats * (double)(ceil_div(s.M, spg::kTileM[t]) * ceil_div(s.N, spg::kTileN[t]));
}
// ... as launched: whole eights of them a group
bool too_many(const WeightsShape& s, int t) { return weights_wgs(s, t) + 8.0 * s.groups > (double)kMostWgs; }

Choice choose_weights(const WeightsShape& s, bool reg) {
    Choice best{-1, 1e30, false, 1};
    for (int t = 0; t < spg::kTiles; ++t) {
        const Cost& c = kWeights[reg][t];
        if (c.bw == 0 || too_many(s, t)) continue;
        double n;
        const double wgs = weights_wgs(s, t), us = cost_us(c, wgs / slots(t, reg), s.kt, s.bytes);
        const double parts = split_us(c, t, wgs, s.kt, s.bytes, n);
        if (us < best.us) best = Choice{t, us, false, 1};
        if (parts < best.us) best = Choice{t, parts, false, (int)n};
    }
    return best;
}

// One launch for both gradients if its estimate is below that of two (as merge() in
// product.hip): the tile, or -1.
int choose_both(const RowsShape& x, const WeightsShape& w, bool reg, double apart) {
    int best = -1;
    for (int t : {(int)spg::kTileMid, (int)spg::kTileSmall}) {
        const Cost& cx = kRows[reg][0][t];
        const Cost& cw = t == spg::kTileMid ? kWeightsMid[reg] : kWeights[reg][t];
        if ((double)most_wgs(x.rows, x.live, x.N, t, 1) + weights_wgs(w, t) + 8.0 * w.groups > (double)kMostWgs) continue;
        const double nx = rows_wgs(x, t) / slots(t, reg), nw = weights_wgs(w, t) / slots(t, reg);
        const double full = nx * ((double)x.kt * cx.busy + cx.tile) + nw * (w.kt * cw.busy + cw.tile);
        const double us = cx.base + std::max(std::max(std::max((double)x.kt * cx.alone, w.kt * cw.alone), full),
                                             x.bytes / cx.bw + w.bytes / cw.bw);
        if (us < apart) {
            apart = us;
            best = t;
        }
    }
    return best;
}

// ---- launches --------------------------------------------------------------------------

template <int ET, int P>
void launch_type(bool reg, int tile, const ProductArgs& a, const GroupArgs& g, int per, dim3 grid, hipStream_t st) {
    constexpr bool ROWS_OF_X = P == spg::kRowsGatedNK || P == spg::kRowsGatedKN || P == spg::kRowsNK || P == spg::kRowsKN;
    if constexpr (ROWS_OF_X) {
        if (g.source) {
            if (reg) spg::launch_grouped<ET, P, true, true>(tile, a, g, per, grid, st);
            else spg::launch_grouped<ET, P, false, true>(tile, a, g, per, grid, st);
            return;
        }
    }
    if (reg) spg::launch_grouped<ET, P, true, false>(tile, a, g, per, grid, st);
    else spg::launch_grouped<ET, P, false, false>(tile, a, g, per, grid, st);
}

template <int P>
void launch_product(bool bf, bool reg, int tile, const ProductArgs& a, const GroupArgs& g, int per, dim3 grid, hipStream_t st) {
    if (bf) launch_type<spg::kElBF16, P>(reg, tile, a, g, per, grid, st);
    else launch_type<spg::kElF16, P>(reg, tile, a, g, per, grid, st);
}

template <int P>
void launch_both(bool bf, bool reg, int tile, const ProductArgs& x, const ProductArgs& w, const GroupArgs& g, int nx, int per,
                 dim3 grid, hipStream_t st) {
    if (bf) {
        if (reg) spg::launch_group_gradients<spg::kElBF16, P, true>(tile, x, w, g, nx, per, grid, st);
        else spg::launch_group_gradients<spg::kElBF16, P, false>(tile, x, w, g, nx, per, grid, st);
    } else {
        if (reg) spg::launch_group_gradients<spg::kElF16, P, true>(tile, x, w, g, nx, per, grid, st);
        else spg::launch_group_gradients<spg::kElF16, P, false>(tile, x, w, g, nx, per, grid, st);
    }
}

void launch_any(int product, bool bf, bool reg, int tile, const ProductArgs& a, const GroupArgs& g, int per, dim3 grid,
                hipStream_t st) {
    switch (product) {
        case spg::kRowsGatedNK: return launch_product<spg::kRowsGatedNK>(bf, reg, tile, a, g, per, grid, st);
        case spg::kRowsGatedKN: return launch_product<spg::kRowsGatedKN>(bf, reg, tile, a, g, per, grid, st);
        case spg::kRowsSumNK: return launch_product<spg::kRowsSumNK>(bf, reg, tile, a, g, per, grid, st);
        case spg::kRowsSumKN: return launch_product<spg::kRowsSumKN>(bf, reg, tile, a, g, per, grid, st);
        case spg::kRowsNK: return launch_product<spg::kRowsNK>(bf, reg, tile, a, g, per, grid, st);
        case spg::kRowsKN: return launch_product<spg::kRowsKN>(bf, reg, tile, a, g, per, grid, st);
        default: return launch_product<spg::kGroupWeights>(bf, reg, tile, a, g, per, grid, st);
    }
}

constexpr int32_t kWhole = 1 << 28;   // k-tiles of a part: the reduction is not split

constexpr uint8_t kGroupRows = 6;     // row tiles of a group rastered together

// rows of tiles rastered together, as set_grid in product.hip
uint8_t raster_rows(int64_t rows) { return (uint8_t)(rows <= 8 ? std::max<int64_t>(rows, 1) : 4); }

// The parts of either choice
int64_t most_part_bytes(const Choice* c) {
    int64_t most = 0;
    for (int r = 0; r < 2; ++r)
        if (c[r].split || c[r].parts > 1) most = std::max(most, spg::part_bytes(c[r].tile));
    return most;
}

// A section of `bytes` at the end of a workspace of `size` bytes so far, -1 if it is not wanted.
int64_t section(bool wanted, int64_t bytes, int64_t& size) {
    if (!wanted || bytes == 0) return -1;
    const int64_t at = size;
    size += up(bytes, kAlign);
    return at;
}
void* at(void* workspace, int64_t offset) { return offset < 0 ? nullptr : (char*)workspace + offset; }

// The rest of a rows product's arguments; returns its workgroups.
int64_t rows_grid(const Common& c, int tile, int mats, ProductArgs& a) {
    a.zm = a.zn = a.split = 1;
    a.kt_part = kWhole;
    a.tiles_m = 0;   // found on the device
    a.tiles_n = (int32_t)ceil_div(a.N, spg::group_tile_n(tile, mats));
    a.group_m = kGroupRows;
    return up(most_wgs(c.rows, c.live(), a.N, tile, mats), 8);
}

// tiles and wave tiles as in launch_grouped
template <int ET, bool DUAL, bool SEG>
void launch_join(int tile, const ProductArgs& a, const GroupArgs& g, hipStream_t st) {
    auto go = [&](auto bm, auto bn, auto wm, auto wn) {
        constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value;
        hipLaunchKernelGGL((spg::grouped_join<ET, DUAL, SEG, BM, BN, decltype(wm)::value, decltype(wn)::value>),
                           dim3(spg::kRound / 2 * (BM * BN / 4096)), dim3(256), 0, st, a, g);
    };
    using std::integral_constant;
    constexpr integral_constant<int, 32> i32{};
    constexpr integral_constant<int, 64> i64{};
    constexpr integral_constant<int, 128> i128{};
    constexpr integral_constant<int, 256> i256{};
    if (tile == spg::kTileBig) {
        if constexpr (DUAL) go(i256, i256, i64, i128);
        else go(i256, i256, i128, i64);
    } else if (tile == spg::kTileThin) {
        if constexpr (DUAL) go(i32, i128, i32, i64);
        else go(i32, i128, i32, i32);
    } else if (tile == spg::kTileSmall) go(i64, i128, i32, i64);
    else go(i64, i64, i32, i64);
}
template <bool DUAL, bool SEG>
void launch_join(bool bf, int tile, const ProductArgs& a, const GroupArgs& g, hipStream_t st) {
    if (bf) launch_join<spg::kElBF16, DUAL, SEG>(tile, a, g, st);
    else launch_join<spg::kElF16, DUAL, SEG>(tile, a, g, st);
}

// parts: their place, used where the choice splits tiles
gemm_status run_rows(int product, const Common& c, bool reg, const Choice& choice, int mats, ProductArgs a, const int32_t* offsets,
                     const int32_t* source, void* parts, hipStream_t st) {
    const int tile = choice.tile;
    int64_t wgs = rows_grid(c, tile, mats, a);
    GroupArgs g = group_args(c, offsets, source);
    if (choice.split) {
        g.part = (float*)parts;
        wgs += spg::kRound;    // a whole round of parts in the place of a part of one
    }
    launch_any(product, c.bf, reg, tile, a, g, 0, dim3((unsigned)wgs), st);
    const gemm_status e = launched();
    if (e != GEMM_OK || !g.part) return e;
    if (mats == 2) launch_join<true, false>(c.bf, tile, a, g, st);
    else if (a.segments == 2) launch_join<false, true>(c.bf, tile, a, g, st);
    else launch_join<false, false>(c.bf, tile, a, g, st);
    return launched();
}

// dW's operands (and with two results dWg's and dWu's): D rows of `ldd` bytes, two matrices
// `second` bytes apart
ProductArgs weights_args(const Common& c, int mats, const char* D, int64_t ldd, int64_t d_cols, int64_t second, const char* X,
                         int64_t ldx, int64_t x_cols, void* dW, void* dW1) {
    ProductArgs w{};
    w.A = c.nk ? D : X;
    if (mats == 2) {
        w.A1 = c.nk ? D + second : X;
        w.C1 = dW1;
    }
    w.B[0] = c.nk ? X : D;
    w.B[1] = c.nk ? X : D + second;
    w.C = dW;
    w.M = (int32_t)(c.nk ? c.N : c.K);
    w.N = (int32_t)(c.nk ? c.K : c.N);
    w.lda = (uint32_t)(c.nk ? ldd : ldx);
    w.ldb = (uint32_t)(c.nk ? ldx : ldd);
    w.a_cols = (int32_t)(c.nk ? d_cols : x_cols);
    w.b_cols = (int32_t)(c.nk ? x_cols : d_cols);
    w.segments = w.split = 1;
    w.zm = (uint8_t)(c.nk ? mats : 1);
    w.zn = (uint8_t)(c.nk ? 1 : mats);
    w.kt_part = kWhole;
    return w;
}

// Its tiles; returns the workgroups of a group.
int64_t weights_grid(int tile, ProductArgs& w) {
    w.tiles_m = (int32_t)ceil_div(w.M, spg::kTileM[tile]);
    w.tiles_n = (int32_t)ceil_div(w.N, spg::kTileN[tile]);
    w.group_m = raster_rows((int64_t)w.tiles_m * w.zm);
    return up((int64_t)w.tiles_m * w.zm * w.tiles_n * w.zn * w.split, 8);
}

template <int BM, int BN, int WM, int WN>
void launch_weights_join(bool bf, const ProductArgs& w, const GroupArgs& g, hipStream_t st) {
    const dim3 grid((unsigned)(g.groups * w.tiles_m * w.zm * w.tiles_n * w.zn * (BM * BN / 4096)));
    if (bf) hipLaunchKernelGGL((spg::weights_join<spg::kElBF16, BM, BN, WM, WN>), grid, dim3(256), 0, st, w, g);
    else hipLaunchKernelGGL((spg::weights_join<spg::kElF16, BM, BN, WM, WN>), grid, dim3(256), 0, st, w, g);
}

gemm_status run_weights(const Common& c, bool reg, const Choice& choice, ProductArgs w, const int32_t* offsets, void* parts,
                        hipStream_t st) {
    w.split = choice.parts;
    const int64_t per = weights_grid(choice.tile, w);
    GroupArgs g = group_args(c, offsets, nullptr);
    g.part = (float*)parts;
    launch_any(spg::kGroupWeights, c.bf, reg, choice.tile, w, g, (int)per, dim3((unsigned)(per * c.groups)), st);
    const gemm_status e = launched();
    if (e != GEMM_OK || choice.parts == 1) return e;
    if (choice.tile == spg::kTileSmall) launch_weights_join<64, 128, 32, 64>(c.bf, w, g, st);
    else launch_weights_join<64, 64, 32, 64>(c.bf, w, g, st);
    return launched();
}

// Both gradients, in one launch where `both` names a tile for it.
gemm_status run_gradients(int product, const Common& c, bool regx, bool regw, const Choice* dx, const Choice* dw, const int* both,
                          ProductArgs x, ProductArgs w, const int32_t* offsets, void* parts, hipStream_t st) {
    const bool reg = regx || regw;
    if (both[reg] >= 0) {
        const int t = both[reg];
        const int64_t nx = rows_grid(c, t, 1, x), per = weights_grid(t, w);
        const GroupArgs g = group_args(c, offsets, nullptr);
        const dim3 grid((unsigned)(nx + per * c.groups));
        switch (product) {
            case spg::kRowsSumNK: launch_both<spg::kRowsSumNK>(c.bf, reg, t, x, w, g, (int)nx, (int)per, grid, st); break;
            case spg::kRowsSumKN: launch_both<spg::kRowsSumKN>(c.bf, reg, t, x, w, g, (int)nx, (int)per, grid, st); break;
            case spg::kRowsNK: launch_both<spg::kRowsNK>(c.bf, reg, t, x, w, g, (int)nx, (int)per, grid, st); break;
            default: launch_both<spg::kRowsKN>(c.bf, reg, t, x, w, g, (int)nx, (int)per, grid, st); break;
        }
        return launched();
    }
    const gemm_status e = run_rows(product, c, regx, dx[regx], 1, x, offsets, nullptr, parts, st);
    return e != GEMM_OK ? e : run_weights(c, regw, dw[regw], w, offsets, parts, st);
}

template <bool BF16, bool DUAL>
void launch_stream(const Common& c, const ProductArgs& a, const GroupArgs& g, hipStream_t st) {
    const dim3 grid((unsigned)ceil_div(a.N, 16), (unsigned)c.live()), wg(512);
    const uintptr_t all = (uintptr_t)a.A | (uintptr_t)a.B[0] | (DUAL ? (uintptr_t)a.B[1] : 0) | (uintptr_t)a.lda | (uintptr_t)a.ldb;
    if (all % 4 == 0) hipLaunchKernelGGL((spg::grouped_stream<BF16, DUAL, true, 8, 4>), grid, wg, 0, st, a, g);
    else hipLaunchKernelGGL((spg::grouped_stream<BF16, DUAL, false, 8, 4>), grid, wg, 0, st, a, g);
}

gemm_status run_stream(const Common& c, bool dual, const ProductArgs& a, const int32_t* offsets, const int32_t* source,
                       hipStream_t st) {
    const GroupArgs g = group_args(c, offsets, source);
    if (c.bf) dual ? launch_stream<true, true>(c, a, g, st) : launch_stream<true, false>(c, a, g, st);
    else dual ? launch_stream<false, true>(c, a, g, st) : launch_stream<false, false>(c, a, g, st);
    return launched();
}

spg::GatherArgs gather_args(const Common& c, const void* X, const int32_t* source, void* to) {
    return spg::GatherArgs{(const char*)X, (char*)to, source, c.rows, c.K * 2, (int32_t)(c.pitch() / 16), (int32_t)c.tokens};
}
int64_t gather_wgs(const Common& c) { return ceil_div(c.rows * (c.pitch() / 16), 256); }

gemm_status run_gather(const Common& c, const void* X, const int32_t* source, void* to, hipStream_t st) {
    hipLaunchKernelGGL((spg::gather_rows<>), spread(gather_wgs(c)), dim3(256), 0, st, gather_args(c, X, source, to));
    return launched();
}

dim3 simple_grid(int64_t outputs, int64_t groups) {
    return dim3((unsigned)std::min<int64_t>(ceil_div(std::max<int64_t>(outputs, 1), 256), 4096), (unsigned)groups);
}

// Any sizes: B as [N,K] (nk) or [K,N] of the product at hand.
gemm_status simple_rows(const Common& c, const ProductArgs& p, bool nk, int64_t lda, int64_t seg_a, bool dual,
                        const int32_t* offsets, const int32_t* source, hipStream_t st) {
    const spg::SimpleGroupArgs a{p, group_args(c, offsets, source), lda, 1, nk ? p.K : 1, nk ? 1 : p.N, seg_a};
    const dim3 grid = simple_grid(ceil_div(c.rows * p.N, c.groups), c.groups);
    if (c.bf) {
        if (dual) hipLaunchKernelGGL((spg::simple_group_rows<true, true>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((spg::simple_group_rows<true, false>), grid, dim3(256), 0, st, a);
    } else {
        if (dual) hipLaunchKernelGGL((spg::simple_group_rows<false, true>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((spg::simple_group_rows<false, false>), grid, dim3(256), 0, st, a);
    }
    return launched();
}

gemm_status simple_weights(const Common& c, const void* D, int64_t ldd, const void* X, void* C, const int32_t* offsets,
                           const int32_t* source, hipStream_t st) {
    const spg::SimpleWeightArgs a{group_args(c, offsets, source), (const char*)D, (const char*)X, (char*)C,
                                  ldd, c.N, c.K, c.nk ? c.K : 1, c.nk ? 1 : c.N};
    const dim3 grid = simple_grid(c.N * c.K, c.groups);
    if (c.bf) hipLaunchKernelGGL((spg::simple_group_weights<true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((spg::simple_group_weights<false>), grid, dim3(256), 0, st, a);
    return launched();
}

// The streaming kernel: matrices along the reduction, few rows a group and few workgroups in
// all.  Against the best tile at 800 drawn shapes it takes 0.5 to 0.8 of the time up to 256
// workgroups (16 columns of one group each), the same at 1024 and up to three times as long
// beyond; a group of more than 16 rows reads its matrix again for every 16 of them.  Two long
// matrices keep its workgroups busy enough to go on up to 4096 (single rows, 12288 x 4096: 70 us
// against 81; of 2000 to 3500 reductions the same time).  A workgroup reads its columns one
// chunk after the other, and where there are few of them and much to read, tiles in parts are
// faster (72 rows of 5 groups, two matrices 96 x 12024: 86 us against 16).
bool streams(const Common& c, int64_t N, int64_t K, int mats, bool along) {
    if (!along || c.rows > 16 * c.live()) return false;
    const int64_t columns = ceil_div(N, 16);
    if (columns * std::max(c.live(), c.rows / 2) > (mats == 2 && K >= 2048 ? 4096 : 1024)) return false;
    const double reads = (1.0 + (double)c.rows / (16.0 * (double)c.live())) * (double)K * mats;
    return reads <= 14000.0 || columns * c.live() >= 512;
}

// Operands' first row and last byte within 32-bit offsets of the stream
bool fits(int64_t rows, int64_t row_bytes) { return rows * row_bytes + 2048 < kMaxBytes; }

}  // namespace

struct gemm_grouped_plan {
    Common c;
    bool simple, simple_back, stream, stream_back, gather;   // gather: X's rows copied into their groups' order
    Choice fwd[2], dx[2], dw[2];         // [register-staged]
    int both[2];                         // a tile class, -1 for two launches
    int64_t ws_run, ws_back;
    int64_t part_run, part_back;         // where the last round's parts go in the workspace, -1: nothing is split
};

struct gemm_experts_plan {
    Common c;
    int act;
    bool simple, simple_back, stream, gather;
    Choice fwd[2], dx[2], dw[2];
    int both[2];
    int64_t np;                    // columns of dG and of dU in the workspace
    int64_t ws_run, ws_back, off_x;
    int64_t part_run, part_back;
};

extern "C" {

gemm_status gemm_grouped_create(gemm_grouped_handle* out, int64_t rows, int64_t N, int64_t K, int64_t groups,
                                int64_t tokens, gemm_dtype dtype, gemm_b_layout layout) {
    if (out) *out = nullptr;
    const gemm_status e = check(out, rows, N, K, groups, tokens, dtype, layout);
    if (e != GEMM_OK) return e;
    gemm_grouped_plan* p = new (std::nothrow) gemm_grouped_plan{};
    if (!p) return GEMM_ERR_OUT_OF_MEMORY;
    const Common c = p->c = Common{rows, N, K, groups, tokens, dtype == GEMM_BF16, layout == GEMM_B_NK};
    // the tiled kernels need 16 bytes of every row they copy, 32-bit offsets, and a grid that can be launched
    p->simple = K < 8 || (!c.nk && N < 8) || K * 2 > kMaxRowBytes || N * 2 > kMaxRowBytes;
    p->simple_back = p->simple || N < 8;
    p->stream = !p->simple && streams(c, N, K, 1, c.nk) && fits(std::max(rows, tokens), K * 2);
    p->stream_back = !p->simple_back && streams(c, K, N, 1, !c.nk) && fits(rows, N * 2);
    const double live = (double)c.live(), io = 2.0 * rows * (N + K) + live * c.matrix();
    const RowsShape fwd{rows, c.live(), N, ceil_div(K, 64), 1, io}, dx{rows, c.live(), K, ceil_div(N, 64), 1, io};
    const WeightsShape dw = weights_shape(c, 1);
    for (int r = 0; r < 2; ++r) {
        p->fwd[r] = choose_rows(fwd, r == 1);
        p->dx[r] = choose_rows(dx, r == 1);
        p->dw[r] = choose_weights(dw, r == 1);
        // rows in parts need a launch of their own (12785 rows of 7 groups, 113 x 137: 25 us, 52 in one launch)
        p->both[r] = p->dw[r].parts > 1 ? -1 : choose_both(dx, dw, r == 1, p->dx[r].us + p->dw[r].us);
        p->simple |= p->fwd[r].tile < 0;
        p->simple_back |= p->dx[r].tile < 0 || p->dw[r].tile < 0;
    }
    p->simple_back |= p->simple;
    p->stream &= !p->simple;
    p->stream_back &= !p->simple_back;
    p->gather = tokens >= 0 && !fits(tokens, K * 2);
    p->ws_run = p->simple || p->stream || !p->gather ? 0 : c.gathered();
    p->part_run = section(!p->simple && !p->stream, most_part_bytes(p->fwd), p->ws_run);
    p->ws_back = p->simple_back ? 0 : c.gathered();
    // dX's and dW's one after the other
    p->part_back = section(!p->simple_back, std::max(p->stream_back ? 0 : most_part_bytes(p->dx), most_part_bytes(p->dw)), p->ws_back);
    *out = p;
    return GEMM_OK;
}

int64_t gemm_grouped_workspace(gemm_grouped_handle h) { return h ? std::max(h->ws_run, h->ws_back) : -1; }
int64_t gemm_grouped_run_workspace(gemm_grouped_handle h) { return h ? h->ws_run : -1; }

gemm_status gemm_grouped_run(gemm_grouped_handle h, const void* X, const void* W, const int32_t* offsets,
                             const int32_t* source, void* Y, void* workspace, int64_t workspace_bytes,
                             hipStream_t stream) {
    if (!h) return GEMM_ERR_INVALID_ARG;
    const Common& c = h->c;
    if (wrong_source(c, source)) return GEMM_ERR_INVALID_ARG;
    if (c.rows == 0 || c.N == 0) return GEMM_OK;
    if (!offsets || !Y || (c.K > 0 && (!W || (!X && c.tokens != 0)))) return GEMM_ERR_INVALID_ARG;
    ProductArgs a{};
    a.A = (const char*)X;
    a.B[0] = (const char*)W;
    a.C = Y;
    a.M = (int32_t)c.rows;
    a.N = (int32_t)c.N;
    a.K = (int32_t)c.K;
    a.lda = (uint32_t)(c.K * 2);
    a.ldb = (uint32_t)((c.nk ? c.K : c.N) * 2);
    a.b_cols = (int32_t)c.N;
    a.segments = 1;
    if (h->simple) return simple_rows(c, a, c.nk, c.K, 0, false, offsets, source, stream);
    if (h->stream) return run_stream(c, false, a, offsets, source, stream);
    if (small_workspace(workspace, workspace_bytes, h->ws_run)) return GEMM_ERR_INVALID_ARG;
    if (h->gather) {
        const gemm_status e = run_gather(c, X, source, workspace, stream);
        if (e != GEMM_OK) return e;
        a.A = (const char*)workspace;
        a.lda = (uint32_t)c.pitch();
        source = nullptr;
    }
    const bool reg = a.lda % 4 != 0 || !words(a.A) || a.ldb % 4 != 0 || !words(W);
    return run_rows(c.nk ? spg::kRowsNK : spg::kRowsKN, c, reg, h->fwd[reg], 1, a, offsets, source, at(workspace, h->part_run), stream);
}

gemm_status gemm_grouped_backward(gemm_grouped_handle h, const void* dY, const void* X, const void* W,
                                  const int32_t* offsets, const int32_t* source, void* dX, void* dW, void* workspace,
                                  int64_t workspace_bytes, hipStream_t stream) {
    if (!h) return GEMM_ERR_INVALID_ARG;
    const Common& c = h->c;
    if (wrong_source(c, source)) return GEMM_ERR_INVALID_ARG;
    if (c.K == 0 || (!dX && !dW) || (c.rows == 0 && c.N == 0)) return GEMM_OK;
    if (!offsets) return GEMM_ERR_INVALID_ARG;
    if (c.rows > 0 && c.N > 0 && (!dY || (dX && !W) || (dW && !X && c.tokens != 0))) return GEMM_ERR_INVALID_ARG;
    if (small_workspace(workspace, workspace_bytes, c.N > 0 ? h->ws_back : 0)) return GEMM_ERR_INVALID_ARG;
    const bool rows = dX && c.rows > 0, weights = dW && c.N > 0;
    ProductArgs a{};
    a.A = (const char*)dY;
    a.B[0] = (const char*)W;
    a.C = dX;
    a.M = (int32_t)c.rows;
    a.N = (int32_t)c.K;
    a.K = (int32_t)c.N;
    a.lda = (uint32_t)(c.N * 2);
    a.ldb = (uint32_t)((c.nk ? c.K : c.N) * 2);
    a.b_cols = (int32_t)c.K;
    a.segments = 1;
    if (h->simple_back) {
        gemm_status e = GEMM_OK;
        if (rows) e = simple_rows(c, a, !c.nk, c.N, 0, false, offsets, nullptr, stream);
        return e != GEMM_OK || !weights ? e : simple_weights(c, dY, c.N, X, dW, offsets, source, stream);
    }
    const char* x = (const char*)X;
    int64_t ldx = c.K * 2, cols = c.K;
    if (weights && source && c.rows > 0) {   // without rows a source may be given, and nothing is read
        const gemm_status e = run_gather(c, X, source, workspace, stream);
        if (e != GEMM_OK) return e;
        x = (const char*)workspace;
        ldx = c.pitch();
        cols = up(c.K, 8);
    }
    const ProductArgs w = weights_args(c, 1, (const char*)dY, c.N * 2, c.N, 0, x, ldx, cols, dW, nullptr);
    const bool regd = a.lda % 4 != 0 || !words(dY);
    const bool regx = regd || a.ldb % 4 != 0 || !words(W), regw = regd || ldx % 4 != 0 || !words(x);
    const int product = c.nk ? spg::kRowsKN : spg::kRowsNK;
    if (rows && weights && !h->stream_back)
        return run_gradients(product, c, regx, regw, h->dx, h->dw, h->both, a, w, offsets, at(workspace, h->part_back), stream);
    gemm_status e = GEMM_OK;
    if (rows)
        e = h->stream_back ? run_stream(c, false, a, offsets, nullptr, stream)
                           : run_rows(product, c, regx, h->dx[regx], 1, a, offsets, nullptr, at(workspace, h->part_back), stream);
    return e != GEMM_OK || !weights ? e : run_weights(c, regw, h->dw[regw], w, offsets, at(workspace, h->part_back), stream);
}

gemm_status gemm_grouped_destroy(gemm_grouped_handle h) {
    delete h;
    return GEMM_OK;
}

gemm_status gemm_experts_create(gemm_experts_handle* out, int64_t rows, int64_t N, int64_t K, int64_t groups,
                                int64_t tokens, gemm_dtype dtype, gemm_b_layout layout, gemm_activation act) {
    if (out) *out = nullptr;
    if (act != GEMM_ACT_SILU && act != GEMM_ACT_GELU_TANH && act != GEMM_ACT_RELU) return GEMM_ERR_INVALID_ARG;
    const gemm_status e = check(out, rows, N, K, groups, tokens, dtype, layout);
    if (e != GEMM_OK) return e;
    gemm_experts_plan* p = new (std::nothrow) gemm_experts_plan{};
    if (!p) return GEMM_ERR_OUT_OF_MEMORY;
    const Common c = p->c = Common{rows, N, K, groups, tokens, dtype == GEMM_BF16, layout == GEMM_B_NK};
    p->act = (int)act;
    p->np = up(N, 64);
    p->simple = K < 8 || (!c.nk && N < 8) || K * 2 > kMaxRowBytes || N * 2 > kMaxRowBytes;
    p->simple_back = p->simple || p->np * 4 > kMaxRowBytes;
    p->stream = !p->simple && streams(c, N, K, 2, c.nk) && fits(std::max(rows, tokens), K * 2);
    const double live = (double)c.live(), io = 2.0 * rows * (N + K) + 2.0 * live * c.matrix();
    const RowsShape fwd{rows, c.live(), N, ceil_div(K, 64), 2, io}, dx{rows, c.live(), K, 2 * ceil_div(N, 64), 1, io};
    const WeightsShape dw = weights_shape(c, 2);
    for (int r = 0; r < 2; ++r) {
        p->fwd[r] = choose_rows(fwd, r == 1);
        p->dx[r] = choose_rows(dx, r == 1);
        p->dw[r] = choose_weights(dw, r == 1);
        // rows in parts need a launch of their own (12785 rows of 7 groups, 113 x 137: 25 us, 52 in one launch)
        p->both[r] = p->dw[r].parts > 1 ? -1 : choose_both(dx, dw, r == 1, p->dx[r].us + p->dw[r].us);
        p->simple |= p->fwd[r].tile < 0;
        p->simple_back |= p->dx[r].tile < 0 || p->dw[r].tile < 0;
    }
    p->simple_back |= p->simple;
    p->stream &= !p->simple;
    p->gather = tokens >= 0 && !fits(tokens, K * 2);
    p->ws_run = p->simple || p->stream || !p->gather ? 0 : c.gathered();
    p->part_run = section(!p->simple && !p->stream, most_part_bytes(p->fwd), p->ws_run);
    p->off_x = up(rows * p->np * 4, kAlign);
    p->ws_back = p->off_x + (p->simple_back ? 0 : c.gathered());
    p->part_back = section(!p->simple_back, std::max(most_part_bytes(p->dx), most_part_bytes(p->dw)), p->ws_back);
    *out = p;
    return GEMM_OK;
}

int64_t gemm_experts_workspace(gemm_experts_handle h) { return h ? std::max(h->ws_run, h->ws_back) : -1; }
int64_t gemm_experts_run_workspace(gemm_experts_handle h) { return h ? h->ws_run : -1; }

gemm_status gemm_experts_run(gemm_experts_handle h, const void* X, const void* Wg, const void* Wu,
                             const int32_t* offsets, const int32_t* source, void* H, void* G, void* U, void* workspace,
                             int64_t workspace_bytes, hipStream_t stream) {
    if (!h || (G == nullptr) != (U == nullptr)) return GEMM_ERR_INVALID_ARG;
    const Common& c = h->c;
    if (wrong_source(c, source)) return GEMM_ERR_INVALID_ARG;
    if (c.rows == 0 || c.N == 0) return GEMM_OK;
    if (!offsets || !H || (c.K > 0 && (!Wg || !Wu || (!X && c.tokens != 0)))) return GEMM_ERR_INVALID_ARG;
    ProductArgs a{};
    a.A = (const char*)X;
    a.B[0] = (const char*)Wg;
    a.B[1] = (const char*)Wu;
    a.C = H;
    a.G = G;
    a.U = U;
    a.M = (int32_t)c.rows;
    a.N = (int32_t)c.N;
    a.K = (int32_t)c.K;
    a.lda = (uint32_t)(c.K * 2);
    a.ldb = (uint32_t)((c.nk ? c.K : c.N) * 2);
    a.b_cols = (int32_t)c.N;
    a.segments = 1;
    a.act = (uint8_t)h->act;
    if (h->simple) return simple_rows(c, a, c.nk, c.K, 0, true, offsets, source, stream);
    if (h->stream) return run_stream(c, true, a, offsets, source, stream);
    if (small_workspace(workspace, workspace_bytes, h->ws_run)) return GEMM_ERR_INVALID_ARG;
    if (h->gather) {
        const gemm_status e = run_gather(c, X, source, workspace, stream);
        if (e != GEMM_OK) return e;
        a.A = (const char*)workspace;
        a.lda = (uint32_t)c.pitch();
        source = nullptr;
    }
    const bool reg = a.lda % 4 != 0 || !words(a.A) || a.ldb % 4 != 0 || !words(Wg) || !words(Wu);
    return run_rows(c.nk ? spg::kRowsGatedNK : spg::kRowsGatedKN, c, reg, h->fwd[reg], 2, a, offsets, source, at(workspace, h->part_run), stream);
}

gemm_status gemm_experts_backward(gemm_experts_handle h, const void* dH, const void* X, const void* Wg, const void* Wu,
                                  const void* G, const void* U, const int32_t* offsets, const int32_t* source, void* dX,
                                  void* dWg, void* dWu, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (!h) return GEMM_ERR_INVALID_ARG;
    const Common& c = h->c;
    if (wrong_source(c, source)) return GEMM_ERR_INVALID_ARG;
    if (c.K == 0 || (c.rows == 0 && c.N == 0)) return GEMM_OK;
    if (!offsets || (c.rows > 0 && !dX) || (c.N > 0 && (!dWg || !dWu))) return GEMM_ERR_INVALID_ARG;
    if (c.rows > 0 && c.N > 0) {
        if (!dH || (!X && c.tokens != 0) || !Wg || !Wu || !G || !U) return GEMM_ERR_INVALID_ARG;
        if (small_workspace(workspace, workspace_bytes, h->ws_back)) return GEMM_ERR_INVALID_ARG;
    }
    const bool simple = h->simple_back || c.rows == 0 || c.N == 0;
    uint16_t* D = (uint16_t*)workspace;
    const char* x = (const char*)X;
    int64_t ldx = c.K * 2, cols = c.K;
    if (c.rows > 0 && c.N > 0) {
        spg::SlopeArgs d{(const uint16_t*)dH, (const uint16_t*)G, (const uint16_t*)U, D, (int32_t)c.rows, (int32_t)c.N,
                         (int32_t)h->np, h->act, ceil_div(c.rows * (h->np / 8), 256)};
        spg::GatherArgs xs{};
        int64_t wgs = d.slopes;
        if (source && !simple) {
            x = (const char*)workspace + h->off_x;
            xs = gather_args(c, X, source, (void*)x);
            wgs += gather_wgs(c);
            ldx = c.pitch();
            cols = up(c.K, 8);
        }
        if (c.bf) hipLaunchKernelGGL((spg::grouped_slopes<true>), spread(wgs), dim3(256), 0, stream, d, xs);
        else hipLaunchKernelGGL((spg::grouped_slopes<false>), spread(wgs), dim3(256), 0, stream, d, xs);
        const gemm_status e = launched();
        if (e != GEMM_OK) return e;
    }
    // dX = [dG dU] . [Wg; Wu]: one sum over both segments
    ProductArgs a{};
    a.A = (const char*)D;
    a.B[0] = (const char*)Wg;
    a.B[1] = (const char*)Wu;
    a.C = dX;
    a.M = (int32_t)c.rows;
    a.N = (int32_t)c.K;
    a.K = (int32_t)c.N;
    a.lda = (uint32_t)(h->np * 4);
    a.ldb = (uint32_t)((c.nk ? c.K : c.N) * 2);
    a.b_cols = (int32_t)c.K;
    a.segments = 2;
    if (simple) {
        gemm_status e = GEMM_OK;
        if (c.rows > 0) e = simple_rows(c, a, !c.nk, 2 * h->np, h->np, false, offsets, nullptr, stream);
        for (int z = 0; z < 2 && c.N > 0 && e == GEMM_OK; ++z)
            e = simple_weights(c, D + z * h->np, 2 * h->np, X, z ? dWu : dWg, offsets, source, stream);
        return e;
    }
    const ProductArgs w = weights_args(c, 2, (const char*)D, h->np * 4, h->np, h->np * 2, x, ldx, cols, dWg, dWu);
    const bool regx = a.ldb % 4 != 0 || !words(Wg) || !words(Wu), regw = ldx % 4 != 0 || !words(x);
    return run_gradients(c.nk ? spg::kRowsSumNK : spg::kRowsSumKN, c, regx, regw, h->dx, h->dw, h->both, a, w, offsets, at(workspace, h->part_back), stream);
}

gemm_status gemm_experts_destroy(gemm_experts_handle h) {
    delete h;
    return GEMM_OK;
}

}  // extern "C"
