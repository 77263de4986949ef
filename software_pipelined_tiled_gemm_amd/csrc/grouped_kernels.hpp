// Device code of the products by group for gfx950 (gemm_grouped_* and gemm_experts_* in
// include/spgemm.h): the rows of group e times matrix e, plain or gated, and their backward
// passes.  Where a group's rows lie is read on the device from its offsets.
#pragma once

#include "product_kernels.hpp"
#include "wave_scan.hpp"

namespace spg {

struct GroupArgs {
    const int32_t* offsets;   // [groups + 1]
    const int32_t* source;    // row -> row of X, or null
    float* part;              // sums of the last tiles' parts, or null: no tile is split (rows)
    int64_t b_step;           // bytes from one group's B matrix to the next (rows), or of C (weights)
    int32_t groups, rows;
    int32_t tokens;           // rows of X where there is a source
};

// First row and rows of a group, whatever the offsets hold.
struct Group {
    int32_t first, n;
};
__device__ __forceinline__ Group group_of(const GroupArgs& g, int e) {
    auto inside = [&](int v) { return v < 0 ? 0 : v > g.rows ? g.rows : v; };
    const int a = inside(g.offsets[e]), b = inside(g.offsets[e + 1]);
    return Group{a, b > a ? b - a : 0};
}

// Group e of 64 from `first` on in lane e - first, and how many units of U rows it has.
template <int U>
__device__ __forceinline__ int units_of(const GroupArgs& g, int e, Group& gr) {
    gr = e < g.groups ? group_of(g, e) : Group{0, 0};
    return (gr.n + U - 1) / U;
}

// All groups' units of U rows.
template <int U>
__device__ __forceinline__ int all_units(const GroupArgs& g, int lane) {
    int total = 0;
    Group gr;
    for (int e = 0; e < g.groups; e += 64) total += __builtin_amdgcn_readlane(wave_scan(units_of<U>(g, e + lane, gr)), 63);
    return total;
}

// Where unit `u` of all groups' units lies: its group, that group, and the unit within it.
struct Found {
    int e, unit;
    Group g;
};
template <int U>
__device__ __forceinline__ Found find_unit(const GroupArgs& g, int u, int lane) {
    for (int e = 0;; e += 64) {
        Group gr;
        const int own = units_of<U>(g, e + lane, gr), upto = wave_scan(own);
        const uint64_t m = __ballot(upto > u);
        if (m != 0 || e + 64 >= g.groups) {
            const int l = m ? __builtin_ctzll(m) : 63;   // m is not 0 for u < all_units()
            return Found{e + l, u - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(own, l)),
                         Group{__builtin_amdgcn_readlane(gr.first, l), __builtin_amdgcn_readlane(gr.n, l)}};
        }
        u -= __builtin_amdgcn_readlane(upto, 63);
    }
}

// Workgroup -> one of T places, a contiguous range of them for each XCD (workgroup id mod 8);
// -1: there are fewer places than workgroups.
__device__ __forceinline__ int xcd_place(int wg, int T) {
    const int x = wg & 7, i = wg >> 3, q = T >> 3, r = T & 7;
    return i < q + (x < r ? 1 : 0) ? x * q + (x < r ? x : r) + i : -1;
}

// Place -> tile, `group_m` rows of tiles rastered together.
__device__ __forceinline__ void raster(int at, int rows, int cols, int group_m, int& tm, int& tn) {
    const int gsz = group_m * cols, g = at / gsz, first = g * group_m;
    const int gm = rows - first < group_m ? rows - first : group_m;
    const int in = at - g * gsz;
    tm = first + in % gm;
    tn = in / gm;
}

// Tiles come in rounds of one per CU, and the last round leaves CUs idle: 592 tiles of 256
// k-tiles are 2.3 rounds and take 3.  Where it is worth it the last round's tiles are split along
// the reduction, a part to each workgroup, and a second launch (grouped_join) adds the parts in
// order: 8192 rows in 8 groups, 4096 x 8192, both passes 3340 us without, 3120 with.  So are the
// tiles of a grid of less than half a round: 12 groups' single row, 840 x 6472 stored [K,N], 26.5
// and 16.5 us.  How many tiles there are is only known here, so both kernels work it out.
struct LastRound {
    int full;      // tiles that stay whole
    int parts;     // of each of the others; 1: none is split
    int kt_part;
};
constexpr int kRound = 256;
// Parts cost a write, a read and a launch: as many k-tiles have to be saved as take that long
// (tile rows by tile columns).
__host__ __device__ constexpr int split_gain(int bm, int bn) { return bm * bn == 256 * 256 ? 24 : 16; }
__host__ __device__ constexpr int most_parts(int bm, int bn) { return bm * bn == 256 * 256 ? 8 : 16; }
template <int BM, int BN>
__device__ __forceinline__ LastRound last_round(int tiles, int kt) {
    const int full = tiles / kRound * kRound, rest = tiles - full;
    int parts = rest > 0 ? kRound / rest : 1;
    parts = parts < most_parts(BM, BN) ? parts : most_parts(BM, BN);
    const int kt_part = (kt + parts - 1) / parts;
    parts = (kt + kt_part - 1) / kt_part;
    if (parts < 2 || kt - kt_part < split_gain(BM, BN)) return LastRound{tiles, 1, kt};
    return LastRound{full, parts, kt_part};
}

// The rows of every group times its matrix on the tiled kernel (product_tile_of): a workgroup
// finds its tile among all groups' row tiles and takes its group for the whole problem.  The
// grid covers the most row tiles that `rows` rows in `groups` groups can come to; what is left
// over ends at once, and comes last.  GATHER: rows of X by their source, read where they lie
// (gathered into a copy first they cost a pass of their own: 23 us of 24576 rows of 4 KiB).
template <int ET, bool B_N, bool DUAL, bool SEG, bool REG, int BM, int BN, int WM, int WN, int S, bool DEEP, int KG, bool TAIL,
          bool GATHER>
__device__ __forceinline__ void rows_tile(ProductArgs args, const GroupArgs& g, int wg, SPG_LDS char* lds) {
    const int lane = threadIdx.x & 63;
    const int tiles = all_units<BM>(g, lane) * args.tiles_n;
    int at = -1, sp = 0;
    args.part = nullptr;
    LastRound last{tiles, 1, 0};
    constexpr bool SPLIT = BM == 256 || BM <= 64;   // the classes that the host splits
    if constexpr (SPLIT)
        if (g.part) last = last_round<BM, BN>(tiles, (args.K + 63) / 64 * (SEG ? 2 : 1));
    if (!SPLIT || wg < last.full) {
        at = xcd_place(wg, last.full);
    } else if (last.parts > 1) {
        at = xcd_place(wg - last.full, (tiles - last.full) * last.parts);
        if (at >= 0) {
            args.part = g.part + (size_t)at * BM * BN;
            args.kt_part = last.kt_part;
            sp = at % last.parts;
            at = last.full + at / last.parts;
        }
    }
    if (at < 0) return;
    // a group's tiles one after the other, so that its matrix is read once for all its rows: up to
    // group_m row tiles go through the columns together, more in even parts
    const int u = at / args.tiles_n;
    const Found f = find_unit<BM>(g, u, lane);
    const int mine = (f.g.n + BM - 1) / BM, parts = (mine + args.group_m - 1) / args.group_m;
    int tm, tn;
    raster(at - (u - f.unit) * args.tiles_n, mine, args.tiles_n, (mine + parts - 1) / parts, tm, tn);
    const size_t out = (size_t)f.g.first * args.N * 2;
    if (!GATHER) args.A += (size_t)f.g.first * args.lda;
    args.B[0] += (size_t)f.e * g.b_step;
    if (DUAL || SEG) args.B[1] += (size_t)f.e * g.b_step;
    args.C = (char*)args.C + out;
    if (DUAL && args.G) {
        args.G = (char*)args.G + out;
        args.U = (char*)args.U + out;
    }
    args.M = f.g.n;
    product_tile_of<ET, false, B_N, DUAL, SEG, REG, BM, BN, WM, WN, S, DEEP, KG, TAIL, GATHER, true, SPLIT>(
        args, tm, tn, sp, lds, SourceRows{GATHER ? g.source + f.g.first : nullptr, g.tokens});
}

template <int ET, bool B_N, bool DUAL, bool SEG, bool REG, int BM, int BN, int WM, int WN, int S, bool DEEP, int KG, bool TAIL,
          int WPS, bool GATHER>
__global__ void __launch_bounds__((ProductGeom<DUAL, BM, BN, WM, WN, S, DEEP, KG>::NT), WPS)
grouped_rows(ProductArgs args, GroupArgs g) {
    __shared__ __attribute__((aligned(1024))) char lds[ProductGeom<DUAL, BM, BN, WM, WN, S, DEEP, KG>::LDS];
    rows_tile<ET, B_N, DUAL, SEG, REG, BM, BN, WM, WN, S, DEEP, KG, TAIL, GATHER>(args, g, blockIdx.x, (SPG_LDS char*)lds);
}

// The parts of a tile added: 4096 of its elements by each workgroup (`blk` of the tile's), each of
// whose waves adds some of the accumulators of the tile's waves, 16 rows x 16 columns a time;
// put(row, column, sums of four columns from there).
template <bool DUAL, int BM, int BN, int WM, int WN, typename F>
__device__ __forceinline__ void join_parts(const float* part, int parts, int blk, F&& put) {
    using G = ProductGeom<DUAL, BM, BN, WM, WN, 2, false, 1>;
    constexpr int UNITS = (DUAL ? G::TN / 2 : G::TN) * G::TM, EACH = G::NW * UNITS / (BM * BN / 4096 * 4);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // four parts' loads of all of a wave's accumulators under way at once: one by one their latencies
    // are most of the time
    constexpr int NM = DUAL ? 2 : 1, UP = UNITS * 256;              // UP: to the up projection's accumulators
    auto own = [&](int i) { return (blk * 4 + wave) * EACH + i; };
    auto load = [&](int k, int i, int h) __attribute__((always_inline)) {
        const int q = own(i), w = q / UNITS, j = q % UNITS;
        return *(const floatx4*)(part + (size_t)k * BM * BN + ((w * G::TN * G::TM + j) * 64 + lane) * 4 + h * UP);
    };
    floatx4 s[EACH][NM];
#pragma unroll
    for (int i = 0; i < EACH; ++i)
#pragma unroll
        for (int h = 0; h < NM; ++h) s[i][h] = load(0, i, h);
    for (int k0 = 1; k0 < parts; k0 += 4) {
        floatx4 v[4][EACH][NM];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < EACH; ++i)
#pragma unroll
                for (int h = 0; h < NM; ++h) v[u][i][h] = load(k0 + u < parts ? k0 + u : parts - 1, i, h);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (k0 + u < parts)
#pragma unroll
                for (int i = 0; i < EACH; ++i)
#pragma unroll
                    for (int h = 0; h < NM; ++h) s[i][h] += v[u][i][h];
    }
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int q = own(i), w = q / UNITS, j = q % UNITS;
        put(w / G::WAVES_N * WM + j % G::TM * 16 + (lane & 15), w % G::WAVES_N * G::WNS + j / G::TM * 16 + 4 * (lane >> 4), s[i][0],
            s[i][NM - 1]);
    }
}

// The parts of the last round's tiles added, and the epilogue.
template <int ET, bool DUAL, bool SEG, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(256) grouped_join(ProductArgs args, GroupArgs g) {
    using G = ProductGeom<DUAL, BM, BN, WM, WN, 2, false, 1>;
    constexpr int JOIN = BM * BN / 4096;
    const int lane = threadIdx.x & 63;
    const int tiles = all_units<BM>(g, lane) * args.tiles_n;
    const LastRound last = last_round<BM, BN>(tiles, (args.K + 63) / 64 * (SEG ? 2 : 1));
    const int t = blockIdx.x / JOIN;
    if (last.parts == 1 || t >= tiles - last.full) return;
    const int at = last.full + t, u = at / args.tiles_n;
    const Found f = find_unit<BM>(g, u, lane);
    const int mine = (f.g.n + BM - 1) / BM, in = (mine + args.group_m - 1) / args.group_m;
    int tm, tn;
    raster(at - (u - f.unit) * args.tiles_n, mine, args.tiles_n, (mine + in - 1) / in, tm, tn);
    join_parts<DUAL, BM, BN, WM, WN>(
        g.part + (size_t)t * last.parts * BM * BN, last.parts, blockIdx.x % JOIN,
        [&](int row, int col, const floatx4& s0, const floatx4& s1) __attribute__((always_inline)) {
            const int m = tm * BM + row, n = tn * G::BNS + col;
            if (m < f.g.n && n < args.N)
                finish4<ET, DUAL>(s0, s1, 0, n, args.N - n < 4 ? args.N - n : 4, (size_t)(f.g.first + m) * args.N + n, args);
        });
}

// The weights' gradients of every group: the reduction runs over the group's rows.  `per`
// workgroups a group (a multiple of 8), so that every group's tiles are spread over all XCDs
// whatever its rows.  A group without rows writes zeros.  args.split: parts that a group's rows are
// taken in, as far as it has k-tiles for them, joined by weights_join; few small matrices and
// many rows leave CUs idle otherwise.
struct RowParts {
    int parts, kt_part;
};
__device__ __forceinline__ RowParts row_parts(int n, int split) {
    const int kt = (n + 63) / 64, kt_part = (kt + split - 1) / split;
    return RowParts{kt_part > 0 ? (kt + kt_part - 1) / kt_part : 1, kt_part};
}

template <int ET, bool REG, int BM, int BN, int WM, int WN, int S, bool DEEP, int KG>
__device__ __forceinline__ void weights_tile(ProductArgs args, const GroupArgs& g, int per, int wg, SPG_LDS char* lds) {
    using G = ProductGeom<false, BM, BN, WM, WN, S, DEEP, KG>;
    const int e = wg / per;
    const int rows = args.tiles_m * args.zm, cols = args.tiles_n * args.zn;
    constexpr bool SPLIT = BM == 64;                  // the classes that the host splits
    int at = xcd_place(wg - e * per, rows * cols * (SPLIT ? args.split : 1)), sp = 0;
    if (at < 0) return;
    const Group gr = group_of(g, e);
    args.part = nullptr;
    if constexpr (SPLIT) {
        sp = at / (rows * cols);
        at -= sp * rows * cols;
        const RowParts p = row_parts(gr.n, args.split);
        if (sp >= p.parts) return;
        if (p.parts > 1) {
            args.part = g.part + (((size_t)e * rows * cols + at) * args.split + sp) * BM * BN;
            args.kt_part = p.kt_part;
        }
    }
    int tm, tn;
    raster(at, rows, cols, args.group_m, tm, tn);
    args.C = (char*)args.C + (size_t)e * g.b_step;
    if (args.zm == 2 || args.zn == 2) args.C1 = (char*)args.C1 + (size_t)e * g.b_step;
    if (gr.n == 0) {
        const bool second = tm >= args.tiles_m || tn >= args.tiles_n;
        const int m0 = (tm >= args.tiles_m ? tm - args.tiles_m : tm) * BM, n0 = (tn >= args.tiles_n ? tn - args.tiles_n : tn) * BN;
        // 16 bytes a thread at any alignment, a row's last elements one by one
        uint16_t* c = (uint16_t*)(second ? args.C1 : args.C) + (size_t)m0 * args.N + n0;
        const int w = args.N - n0 < BN ? args.N - n0 : BN, h = args.M - m0 < BM ? args.M - m0 : BM;
        for (int i = threadIdx.x; i < h * (BN / 8); i += G::NT) {
            const int col = i % (BN / 8) * 8;
            uint16_t* d = c + (size_t)(i / (BN / 8)) * args.N + col;
            if (col + 8 <= w) ((Bytes16*)d)->v = u32x4{};
            else
                for (int e = col; e < w; ++e) *d++ = 0;
        }
        return;
    }
    args.A += (size_t)gr.first * args.lda;
    if (args.zm == 2) args.A1 += (size_t)gr.first * args.lda;
    args.B[0] += (size_t)gr.first * args.ldb;
    if (args.zn == 2) args.B[1] += (size_t)gr.first * args.ldb;
    args.K = gr.n;
    product_tile_of<ET, true, true, false, false, REG, BM, BN, WM, WN, S, DEEP, KG, false, false, false, SPLIT>(args, tm, tn, sp, lds);
}

// The parts of the gradients' tiles added: a workgroup for every 4096 elements of every group's tiles.
template <int ET, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(256) weights_join(ProductArgs args, GroupArgs g) {
    constexpr int JOIN = BM * BN / 4096;
    const int rows = args.tiles_m * args.zm, cols = args.tiles_n * args.zn;
    const int t = blockIdx.x / JOIN, e = t / (rows * cols);
    const RowParts p = row_parts(group_of(g, e).n, args.split);
    if (p.parts == 1) return;
    int tm, tn, z = 0;
    raster(t - e * rows * cols, rows, cols, args.group_m, tm, tn);
    if (tm >= args.tiles_m) { tm -= args.tiles_m; z = 1; }
    if (tn >= args.tiles_n) { tn -= args.tiles_n; z = 1; }
    args.C = (char*)args.C + (size_t)e * g.b_step;
    if (z) args.C1 = (char*)args.C1 + (size_t)e * g.b_step;
    join_parts<false, BM, BN, WM, WN>(
        g.part + (size_t)t * args.split * BM * BN, p.parts, blockIdx.x % JOIN,
        [&](int row, int col, const floatx4& s, const floatx4&) __attribute__((always_inline)) {
            const int m = tm * BM + row, n = tn * BN + col;
            if (m < args.M && n < args.N)
                finish4<ET, false>(s, s, 0, n, args.N - n < 4 ? args.N - n : 4, (size_t)m * args.N + n, args, z);
        });
}

template <int ET, bool REG, int BM, int BN, int WM, int WN, int S, bool DEEP, int KG, int WPS>
__global__ void __launch_bounds__((ProductGeom<false, BM, BN, WM, WN, S, DEEP, KG>::NT), WPS)
grouped_weights(ProductArgs args, GroupArgs g, int per) {
    __shared__ __attribute__((aligned(1024))) char lds[ProductGeom<false, BM, BN, WM, WN, S, DEEP, KG>::LDS];
    weights_tile<ET, REG, BM, BN, WM, WN, S, DEEP, KG>(args, g, per, blockIdx.x, (SPG_LDS char*)lds);
}

// Both gradients in one launch, as gradients_kernel: workgroups 0 .. nx-1 (a multiple of 8) the
// rows', the others the matrices'.
template <int ET, bool B_N, bool SEG, bool REG, int BM, int BN, int WM, int WN, int S, int KG>
__global__ void __launch_bounds__((ProductGeom<false, BM, BN, WM, WN, S, false, KG>::NT))
grouped_gradients(ProductArgs x, ProductArgs w, GroupArgs g, int nx, int per) {
    __shared__ __attribute__((aligned(1024))) char lds[ProductGeom<false, BM, BN, WM, WN, S, false, KG>::LDS];
    const int wg = blockIdx.x;
    if (wg < nx) rows_tile<ET, B_N, false, SEG, REG, BM, BN, WM, WN, S, false, KG, !(SEG && B_N), false>(x, g, wg, (SPG_LDS char*)lds);
    else weights_tile<ET, REG, BM, BN, WM, WN, S, false, KG>(w, g, per, wg - nx, (SPG_LDS char*)lds);
}

// Few rows a group, matrices [N,K]: the product is the reading of the matrices, as in
// stream_kernel.  A workgroup takes 16 columns of one group that has rows (blockIdx.y-th of
// them); its NW waves share K (wave w the chunks w, w + NW, ... of U * 64 bytes a row), every
// lane loads its 16-byte MFMA operands straight from memory, and the waves' sums meet in LDS,
// added in wave order.  Groups of more than 16 rows: 16 at a time.  Rows are read where
// `source` says, by the row's own lanes.
template <bool BF16, bool DUAL, bool WORDS, int NW, int U>
__global__ void __launch_bounds__(NW * 64) grouped_stream(ProductArgs args, GroupArgs g) {
    constexpr int ET = BF16 ? kElBF16 : kElF16;
    constexpr int NM = DUAL ? 2 : 1;
    __shared__ __attribute__((aligned(16))) floatx4 sums[NW][NM][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // the blockIdx.y-th group with rows: a unit of all rows is such a group
    const int live = all_units<(1 << 30)>(g, lane);
    if ((int)blockIdx.y >= live) return;
    const Found f = find_unit<(1 << 30)>(g, blockIdx.y, lane);
    const int M = f.g.n, N = args.N;
    const int kb = args.K * 2;                        // bytes of a row
    const int n0 = blockIdx.x * 16;
    const int cols = N - n0 < 16 ? N - n0 : 16;
    const uint32_t ldb = args.ldb, lda = args.lda;
    struct Rows {
        __amdgpu_buffer_rsrc_t r;
        uint32_t row, shift;
    };
    // this lane's row of a matrix: its resource from the word the matrix starts in, the row from
    // there, and how many bytes past a word it starts
    auto rows_of = [&](const char* p, uint32_t ld, uint32_t n, uint32_t row) __attribute__((always_inline)) -> Rows {
        const uint32_t skip = WORDS ? 0u : (uint32_t)(uintptr_t)p & 3u;
        const uint32_t bytes = skip + (n - 1) * ld + (uint32_t)kb;
        const uint32_t at = skip + row * ld;
        return Rows{make_rsrc_b(p - skip, WORDS ? bytes : (bytes + 3u) & ~3u), WORDS ? at : at & ~3u, WORDS ? 0u : at & 3u};
    };
    const size_t matrix = (size_t)f.e * g.b_step + (size_t)n0 * ldb;
    const uint32_t col = (uint32_t)((lane & 15) < cols ? lane & 15 : cols - 1);
    const Rows b0 = rows_of(args.B[0] + matrix, ldb, (uint32_t)cols, col);
    const Rows b1 = rows_of((DUAL ? args.B[1] : args.B[0]) + matrix, ldb, (uint32_t)cols, col);
    const bool ragged = (kb & 15) != 0;
    const int next = ((lane + 16) & 63) * 4;          // the lane with the row's next 16 bytes
    struct Chunks { u32x4 v[U]; uint32_t end; };

    for (int m0 = 0; m0 < M; m0 += 16) {
        const int m = m0 + (lane & 15);
        int row = m < M ? m : -1;
        if (g.source) {
            if (row >= 0) row = g.source[f.g.first + m];
            if (row >= g.tokens) row = -1;
        }
        const bool some = row >= 0;                   // else a row of zeros
        const Rows x = g.source ? rows_of(args.A, lda, (uint32_t)g.tokens, some ? (uint32_t)row : 0u)
                                : rows_of(args.A + (size_t)f.g.first * lda, lda, (uint32_t)M, some ? (uint32_t)row : 0u);
        floatx4 acc[NM];
#pragma unroll
        for (int q = 0; q < NM; ++q) acc[q] = floatx4{0, 0, 0, 0};
        for (int base = wave * (U * 64); base < kb; base += NW * U * 64) {
            auto load = [&](const Rows& t, bool valid) __attribute__((always_inline)) -> Chunks {
                Chunks c;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int k = base + u * 64 + 16 * (lane >> 4);
                    // as in stream_kernel: the 16 bytes that straddle K are the 16 ending at K, or
                    // the words up to the row's last byte
                    const uint32_t kw = (uint32_t)(WORDS && k + 16 > kb ? kb - 16 : k);
                    const bool in = valid && k < kb + (int)t.shift;
                    c.v[u] = __builtin_amdgcn_raw_buffer_load_b128(t.r, (int)(in ? t.row + kw : kOOB), 0, 0);
                }
                if constexpr (!WORDS)
                    c.end = __builtin_amdgcn_raw_buffer_load_b32(t.r, (int)(valid ? t.row + (uint32_t)(base + U * 64) : kOOB), 0, 0);
                return c;
            };
            auto align = [&](const Rows& t, Chunks& c) __attribute__((always_inline)) {
                if constexpr (!WORDS) {
                    const bool last = lane >= 48;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const uint32_t here = (uint32_t)__builtin_amdgcn_ds_bpermute(next, (int)c.v[u].x);
                        const uint32_t further = u + 1 < U ? (uint32_t)__builtin_amdgcn_ds_bpermute(next, (int)c.v[u + 1 < U ? u + 1 : u].x) : c.end;
                        const uint32_t w[5] = {c.v[u].x, c.v[u].y, c.v[u].z, c.v[u].w, last ? further : here};
#pragma unroll
                        for (int e = 0; e < 4; ++e) c.v[u][e] = __builtin_amdgcn_alignbyte(w[e + 1], w[e], t.shift);
                    }
                }
                if ((ragged || !WORDS) && base + U * 64 > kb) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int k = base + u * 64 + 16 * (lane >> 4);
                        const int gone = k + 16 - kb;
                        const uint32_t sh = gone > 0 && gone < 16 ? 8u * (uint32_t)gone : 0u;
                        if constexpr (WORDS) {
                            c.v[u] = shr128(c.v[u], sh);
                        } else {
                            const u32x4 kept = clear_top(c.v[u], sh);
                            c.v[u] = gone >= 16 ? u32x4{} : kept;
                        }
                    }
                }
            };
            Chunks cx = load(x, some), c0 = load(b0, true), c1;
            if constexpr (DUAL) c1 = load(b1, true);
            align(x, cx);
            align(b0, c0);
            if constexpr (DUAL) align(b1, c1);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                acc[0] = mma<ET>(c0.v[u], cx.v[u], acc[0]);
                if constexpr (DUAL) acc[NM - 1] = mma<ET>(c1.v[u], cx.v[u], acc[NM - 1]);
            }
        }
        if (m0 > 0) __syncthreads();                  // the last 16 rows' sums have been read
#pragma unroll
        for (int q = 0; q < NM; ++q) sums[wave][q][lane] = acc[q];
        __syncthreads();
        // output: 4 consecutive columns of one row a lane of the first wave
        const int n = n0 + 4 * (lane >> 4);
        if (wave == 0 && m < M && n < N) {
            floatx4 s[NM];
#pragma unroll
            for (int q = 0; q < NM; ++q) {
                s[q] = sums[0][q][lane];
#pragma unroll
                for (int w = 1; w < NW; ++w) s[q] += sums[w][q][lane];
            }
            finish4<ET, DUAL>(s[0], s[NM - 1], 0, n, N - n < 4 ? N - n : 4, (size_t)(f.g.first + m) * N + n, args);
        }
    }
}

// Rows brought into their groups' order, on 128-byte lines and padded with zeros (the copies of
// the tiled kernels want rows of one pitch).  A thread moves 16 bytes.
struct GatherArgs {
    const char* src;
    char* dst;
    const int32_t* source;
    int64_t rows, row_bytes;
    int32_t per, tokens;      // 16-byte chunks of a destination row; rows of src
};

__device__ __forceinline__ void gather_at(int64_t i, const GatherArgs& a) {
    const int64_t r = i / a.per;
    if (r >= a.rows) return;
    const int64_t c = (i - r * a.per) * 16, left = a.row_bytes - c;
    const int64_t from = a.source[r];
    u32x4 v = {};
    if (from >= 0 && from < a.tokens && left > 0) {
        const char* s = a.src + from * a.row_bytes + c;
        if (left >= 16) v = ((const Bytes16*)s)->v;
        else
#pragma unroll
            for (int e = 0; e < 16; e += 2)
                if (e < left) v[e >> 2] |= (uint32_t)*(const uint16_t*)(s + e) << ((e & 3) * 8);
    }
    *(u32x4*)(a.dst + i * 16) = v;
}

template <typename = void>   // a template, so that every unit may hold it
__global__ void __launch_bounds__(256) gather_rows(GatherArgs a) {
    gather_at(((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x, a);
}

// The elementwise part of the gated backward pass (gated_slopes), and in the same launch the
// rows of X that the matrices' gradients read: workgroups 0 .. slopes-1 the one, the rest the other.
struct SlopeArgs {
    const uint16_t *dH, *G, *U;
    uint16_t* D;
    int32_t M, N, np, act;
    int64_t slopes;
};

template <bool BF16>
__global__ void __launch_bounds__(256) grouped_slopes(SlopeArgs a, GatherArgs x) {
    const int64_t wg = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (wg < a.slopes) slopes_of<BF16>(wg * 256 + threadIdx.x, a.dH, a.G, a.U, a.D, a.M, a.N, a.np, a.act);
    else if (x.dst) gather_at((wg - a.slopes) * 256 + threadIdx.x, x);
}

// Any strides, one thread per output, a group's outputs in blockIdx.y: for reductions and rows
// that the MFMA kernels do not take.
struct SimpleGroupArgs {
    ProductArgs p;
    GroupArgs g;
    int64_t sam, sak, sbn, sbk;   // element strides, as in SimpleArgs
    int64_t seg_a;
};

template <bool BF16, bool DUAL>
__global__ void __launch_bounds__(256) simple_group_rows(SimpleGroupArgs a) {
    const ProductArgs& p = a.p;
    for (int e = blockIdx.y; e < a.g.groups; e += gridDim.y) {
        const Group gr = group_of(a.g, e);
        const int64_t total = (int64_t)gr.n * p.N;
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
            const int64_t m = i / p.N, n = i - m * p.N, r = gr.first + m;
            int64_t row = r;
            if (a.g.source) {
                row = a.g.source[r];
                if (row < 0 || row >= a.g.tokens) row = -1;   // a row of zeros
            }
            auto at = [&](const char* q, int64_t j) { return bits_to_f32(((const uint16_t*)q)[j], BF16); };
            float s0 = 0, s1 = 0;
            for (int seg = 0; seg < p.segments; ++seg)
                for (int64_t k = 0; k < p.K; ++k) {
                    const float x = row < 0 ? 0.0f : at(p.A, row * a.sam + k * a.sak + seg * a.seg_a);
                    s0 += x * at(p.B[seg] + e * a.g.b_step, n * a.sbn + k * a.sbk);
                    if constexpr (DUAL) s1 += x * at(p.B[1] + e * a.g.b_step, n * a.sbn + k * a.sbk);
                }
            floatx4 v0{s0, s0, s0, s0}, v1{s1, s1, s1, s1};
            finish4<BF16 ? kElBF16 : kElF16, DUAL>(v0, v1, 0, 0, 1, (size_t)(r * p.N + n), p);
        }
    }
}

// dW: D [rows, .] (dY, or dG / dU in a row of ldd elements) against X [., K].
struct SimpleWeightArgs {
    GroupArgs g;
    const char *D, *X;
    char* C;
    int64_t ldd, N, K, sn, sk;    // element strides of C
};

template <bool BF16>
__global__ void __launch_bounds__(256) simple_group_weights(SimpleWeightArgs a) {
    for (int e = blockIdx.y; e < a.g.groups; e += gridDim.y) {
        const Group gr = group_of(a.g, e);
        uint16_t* c = (uint16_t*)(a.C + e * a.g.b_step);
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.N * a.K; i += (int64_t)gridDim.x * 256) {
            const int64_t n = i / a.K, k = i - n * a.K;
            float s = 0;
            for (int64_t r = gr.first; r < gr.first + gr.n; ++r) {
                int64_t row = r;
                if (a.g.source) {
                    row = a.g.source[r];
                    if (row < 0 || row >= a.g.tokens) row = -1;   // a row of zeros
                }
                s += bits_to_f32(((const uint16_t*)a.D)[r * a.ldd + n], BF16) *
                     (row < 0 ? 0.0f : bits_to_f32(((const uint16_t*)a.X)[row * a.K + k], BF16));
            }
            c[n * a.sn + k * a.sk] = f32_to_bits(s, BF16);
        }
    }
}

}  // namespace spg
