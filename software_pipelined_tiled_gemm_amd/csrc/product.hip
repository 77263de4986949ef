// C ABI of the feed-forward operators (declared in include/spgemm.h): the gated projection
// and its backward pass, products of int8 operands, quantisation of rows.
//
// Host side: argument validation (before any HIP call), the choice of kernel, tile and
// parts of the reduction from the shape, the workspace layout and the launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <new>

#include "errors.hpp"
#include "product_launch.hpp"
#include "spgemm.h"

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

// One product of a plan: tile class and parts of the reduction.
struct Shape {
    int64_t M, N;      // of one result
    int64_t kt;        // k-tiles of the whole sum
    int zm, zn;        // results stacked along rows / columns
    int mats;          // B matrices side by side in a tile (2: gated)
    double bytes;      // operands and results, read or written once
    bool crooked;      // rows that are not whole 128-byte lines
};
struct Tiling {
    int tile, split;
    int64_t kt_part;
    double us;         // estimated
};

// Microseconds of a tile class: a k-tile, and a workgroup's start and store, with direct
// copies and register-staged (which has no 256x256 and no pair tile); see choose()
constexpr double kTileUs[spg::kTiles] = {1.27, 0.76, 0.51, 0.32, 0.26, 0.70};
constexpr double kStartUs[spg::kTiles] = {5.3, 5.6, 2.5, 2.75, 2.75, 2.9};
constexpr double kStagedUs[spg::kTiles] = {0.0, 1.30, 0.65, 0.48, 0.42, 0.0};
constexpr double kStagedStartUs[spg::kTiles] = {0.0, 5.3, 3.8, 2.9, 3.3, 0.0};
// direct copies of rows that are not whole 128-byte lines: each 128-byte chunk of a k-tile is
// two lines' halves
constexpr double kCrooked[spg::kTiles] = {1.08, 1.10, 1.05, 1.20, 1.14, 1.18};
// two workgroups on a CU: the pair tile, and the register-staged 64x128 one; alone on their
// CUs the first starts faster and both multiply faster, and a single round in pairs has
// nothing to overlap the starts and stores with
bool paired(int t, bool reg) { return t == (reg ? (int)spg::kTileSmall : (int)spg::kTilePair); }
double slots(int t, bool reg) { return paired(t, reg) ? 512.0 : 256.0; }
double tile_us(int t, bool reg, bool crooked, int64_t wgs) {
    const bool two = paired(t, reg) && wgs > 256;
    if (reg) return two ? 0.84 : kStagedUs[t];
    return (two ? (wgs > 512 ? 0.81 : 1.30) : kTileUs[t]) * (crooked ? kCrooked[t] : 1.0);
}
double start_us(int t, bool reg, int64_t wgs) {
    if (!reg && paired(t, reg) && wgs <= 256) return 1.0;
    return reg ? kStagedStartUs[t] : kStartUs[t];
}
constexpr double kLaunchUs = 1.5;

double sum_us(const Shape& s, int64_t split) {
    return split > 1 ? 4.5 + 2.0 * 4.0 * (double)split * s.M * s.zm * s.N * s.zn * s.mats / 5.5e6 : 0.0;
}
int64_t tiles_of(const Shape& s, int t) {
    return ceil_div(s.M, spg::kTileM[t]) * s.zm * ceil_div(s.N, spg::kTileN[t] / s.mats) * s.zn;
}

// Estimated microseconds of a tile class and a number of parts.  A workgroup fills a CU's LDS
// (half of it for a paired tile): rounds of the CUs times a part's k-tiles and a start and
// store, plus a launch; never less than the operands take to read.  Parts add a kernel and
// their sums' traffic.  The constants are fitted to the measured times of every tile class
// and up to 16 parts at 360 shapes of the seven products, 1 to 12288 rows, columns and
// reductions.  Of whole calls, the sums among them and up to 32 parts, the choice takes 1.6%
// longer than the fastest on average, 40% at worst, more than 10% at 17 of 357 shapes (nine
// of them of at most 64 rows, most of which want more parts).  What
// bounds the small tiles is that a CU copies about 105 bytes a nanosecond into its LDS; what
// bounds short reductions, the start and the store.  Pairs: 4096 x 8192 outputs of 64, 256
// and 1024 reductions take 36, 55 and 140 us against 54, 73 and 164 with one 128x128 tile a
// CU, and 32, 49 and 121 with the 256x256 tile, which needs a large grid.
Tiling choose(const Shape& s, bool reg) {
    Tiling best{spg::kTileSmall, 1, s.kt, 0.0};
    double best_t = -1.0;
    for (int t = 0; t < spg::kTiles; ++t) {
        if (reg && (t == spg::kTileBig || t == spg::kTilePair)) continue;   // not staged through registers
        const int64_t tiles = tiles_of(s, t);
        for (int64_t split = 1; split <= 32 && split <= s.kt; ++split) {
            const int64_t part = ceil_div(s.kt, split);
            if (split > 1 && (part < 4 || ceil_div(s.kt, part) != split)) continue;
            const double rounds = std::ceil((double)(tiles * split) / slots(t, reg));
            double us = kLaunchUs + rounds * (tile_us(t, reg, s.crooked, tiles * split) * (double)part + start_us(t, reg, tiles * split));
            us = std::max(us, 3.0 + s.bytes / 5.0e6) + sum_us(s, split);
            if (best_t < 0 || us < best_t) {
                best_t = us;
                best = Tiling{t, (int)split, part, us};
            }
        }
    }
    return best;
}

// A matrix of a product as its caller stores it, and its copy with 128-byte rows.
struct Stored {
    int64_t rows, row_bytes;
    int64_t pitch() const { return up(row_bytes, 128); }
    int64_t bytes() const { return rows * pitch(); }
    bool aligned() const { return row_bytes % 4 == 0; }
};

// A product of a plan: its tilings with direct copies and register-staged, and whether
// misaligned operands are laid out again first.
struct Planned {
    Shape s;
    Tiling t[2];        // [register-staged]
    bool pack;
    int64_t parts;      // bytes of partial sums
    int64_t packed;     // bytes of the copies
    int64_t bytes() const { return parts + packed; }
};

// The copy reads and writes the misaligned matrices once (about 4.5 TB/s, and a launch).
// M = 2048, N = 4096, K = 1001, two weights: register-staged 51.2 us, direct 30.3 and the
// copy of 20 MB about 12; at M = 300, N = 2731 13.4 against 11.5 and 8.
Planned plan_product(Shape s, std::initializer_list<Stored> mats);

int64_t part_ld(const Shape& s) { return up(s.N, 4) * s.mats * s.zn; }
int64_t part_bytes(const Shape& s, const Tiling& t) {
    return t.split > 1 ? up((int64_t)t.split * s.M * s.zm * part_ld(s) * 4, kAlign) : 0;
}

Planned plan_product(Shape s, std::initializer_list<Stored> mats) {
    int64_t all = 0, bad = 0;
    for (const Stored& m : mats) {
        all += up(m.bytes(), kAlign);
        if (!m.aligned()) bad += m.bytes();
        s.crooked |= m.row_bytes % 128 != 0;
    }
    // rows on odd bytes only reach the direct copies laid out again
    if (bad > 0) s.crooked = false;
    Planned p{s, {choose(s, false), choose(s, true)}, false, 0, 0};
    p.pack = bad > 0 && p.t[0].us + 3.0 + 2.0 * (double)bad / 4.5e6 < p.t[1].us;
    p.parts = std::max(part_bytes(s, p.t[0]), part_bytes(s, p.t[1]));
    p.packed = p.pack ? all : 0;
    return p;
}

// Operands of one product on their way to a launch: pointers and pitches, replaced by those
// of the copies where a plan lays misaligned ones out again.
struct Operands {
    spg::PackArgs pk{};
    int n = 0;
    int64_t total = 0;
    char* at;           // where the next copy goes
    explicit Operands(void* ws) : at((char*)ws) {}
    void copy(const Stored& m, const char*& p, uint32_t& pitch) {
        pk.src[n] = p;
        pk.dst[n] = at;
        pk.row[n] = m.row_bytes;
        pk.per[n] = (int32_t)(m.pitch() / 16);
        pk.chunks[n] = m.bytes() / 16;
        total += pk.chunks[n];
        p = at;
        pitch = (uint32_t)m.pitch();
        at += up(m.bytes(), kAlign);
        ++n;
    }
    gemm_status launch(int es, hipStream_t st) const {
        if (!n) return GEMM_OK;
        const dim3 grid((unsigned)ceil_div(total, 256));
        if (es == 1) hipLaunchKernelGGL(spg::pack_rows<1>, grid, dim3(256), 0, st, pk);
        else hipLaunchKernelGGL(spg::pack_rows<2>, grid, dim3(256), 0, st, pk);
        return launched();
    }
};

// Both gradients in one launch: tile class and parts of dX.
struct Merged {
    bool on;
    int tile, split;
    int64_t kt_part;
};

// One launch if its estimate is below that of two: the longest workgroup, or the work of all
// of them over the CUs.  M = 511, N = 1365, K = 500: 10.0 + 3.9 (dX in 8 parts and their sum)
// and 10.2 us apart.
Merged merge(const Planned& x, const Planned& w, bool reg) {
    Merged best{false, 0, 1, 0};
    if (x.pack || w.pack) return best;
    double best_us = x.t[reg].us + w.t[reg].us;
    for (int t : {(int)spg::kTileMid, (int)spg::kTileSmall})
        for (int64_t split = 1; split <= 16 && split <= x.s.kt; ++split) {
            const int64_t part = ceil_div(x.s.kt, split);
            if (split > 1 && (part < 4 || ceil_div(x.s.kt, part) != split)) continue;
            const int64_t nx = tiles_of(x.s, t) * split, nw = tiles_of(w.s, t);
            const double k = tile_us(t, reg, x.s.crooked || w.s.crooked, nx + nw);
            const double s0 = start_us(t, reg, nx + nw), cx = k * (double)part + s0, cw = k * (double)w.s.kt + s0;
            const double all = ((double)nx * cx + (double)nw * cw) / slots(t, reg);
            // past one round the last workgroups leave CUs idle: half of one's time
            double us = std::max(std::max(cx, cw), nx + nw > slots(t, reg) ? all + 0.5 * std::max(cx, cw) : 0.0);
            us = kLaunchUs + std::max(us, 3.0 + x.s.bytes / 5.0e6) + sum_us(x.s, split);
            if (us < best_us) {
                best_us = us;
                best = Merged{true, t, (int)split, part};
            }
        }
    return best;
}

template <int P, bool REG>
void launch_type(int et, int tile, const ProductArgs& a, dim3 grid, hipStream_t st) {
    if constexpr (P == spg::kInt8 || P == spg::kInt8Gated) spg::launch_product<spg::kElI8, P, REG>(tile, a, grid, st);
    else if (et == spg::kElBF16) spg::launch_product<spg::kElBF16, P, REG>(tile, a, grid, st);
    else spg::launch_product<spg::kElF16, P, REG>(tile, a, grid, st);
}

template <int P>
void launch_mode(int et, bool reg, int tile, const ProductArgs& a, dim3 grid, hipStream_t st) {
    if (reg) launch_type<P, true>(et, tile, a, grid, st);
    else launch_type<P, false>(et, tile, a, grid, st);
}

void launch_tiled(int product, int et, bool reg, int tile, const ProductArgs& a, dim3 grid, hipStream_t st) {
    switch (product) {
        case spg::kGatedNK: return launch_mode<spg::kGatedNK>(et, reg, tile, a, grid, st);
        case spg::kGatedKN: return launch_mode<spg::kGatedKN>(et, reg, tile, a, grid, st);
        case spg::kGradXNK: return launch_mode<spg::kGradXNK>(et, reg, tile, a, grid, st);
        case spg::kGradXKN: return launch_mode<spg::kGradXKN>(et, reg, tile, a, grid, st);
        case spg::kGradW: return launch_mode<spg::kGradW>(et, reg, tile, a, grid, st);
        case spg::kInt8: return launch_mode<spg::kInt8>(et, reg, tile, a, grid, st);
        default: return launch_mode<spg::kInt8Gated>(et, reg, tile, a, grid, st);
    }
}

// Fill in the tile grid of a product; returns its workgroups.
int64_t set_grid(ProductArgs& a, const Shape& s, int tile, int split, int64_t kt_part, void* parts) {
    a.zm = (uint8_t)s.zm;
    a.zn = (uint8_t)s.zn;
    a.tiles_m = (int32_t)ceil_div(s.M, spg::kTileM[tile]);
    a.tiles_n = (int32_t)ceil_div(s.N, spg::kTileN[tile] / s.mats);
    // rows of tiles rastered together: 4 (measured at M = 8192, N = 12288: 2, 4, 8 and 16
    // take 1198, 1186, 1200 and 1215 us), all of them when there are few, else even groups,
    // so that no short last group reads every weight again
    const int64_t rows = (int64_t)a.tiles_m * a.zm;
    a.group_m = (uint8_t)(rows <= 8 ? rows : ceil_div(rows, ceil_div(rows, 4)));
    a.split = (uint8_t)split;
    a.kt_part = (int32_t)kt_part;
    a.part = split > 1 ? (float*)parts : nullptr;
    return rows * a.tiles_n * a.zn * split;
}

// The sum of a split reduction's parts.  More of them than a thread has loads in flight for
// are shared by four waves where one wave for all leaves the CUs idle: 64 x 512 sums of 28
// parts 2.8 us against 3.9 (two matrices 3.8 and 6.7), but 1024 x 1024 of 12 parts 13.3
// against 11.0.
template <int ET, bool DUAL>
void launch_sum(int64_t quads, const ProductArgs& a, hipStream_t st) {
    if (a.split > 8 && quads < 1 << 16) hipLaunchKernelGGL((spg::sum_parts<ET, DUAL, 4>), dim3((unsigned)ceil_div(quads, 64)), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((spg::sum_parts<ET, DUAL, 1>), dim3((unsigned)ceil_div(quads, 256)), dim3(256), 0, st, a);
}

gemm_status run_sum(int et, const Shape& s, const ProductArgs& a, hipStream_t st) {
    const int64_t quads = s.M * s.zm * (up(s.N, 4) / 4) * s.zn;
    const bool dual = s.mats == 2;
    if (et == spg::kElI8) dual ? launch_sum<spg::kElI8, true>(quads, a, st) : launch_sum<spg::kElI8, false>(quads, a, st);
    else if (et == spg::kElBF16) dual ? launch_sum<spg::kElBF16, true>(quads, a, st) : launch_sum<spg::kElBF16, false>(quads, a, st);
    else dual ? launch_sum<spg::kElF16, true>(quads, a, st) : launch_sum<spg::kElF16, false>(quads, a, st);
    return launched();
}

gemm_status run_tiled(int product, int et, bool reg, const Planned& p, ProductArgs a, void* parts, hipStream_t st) {
    const Tiling& t = p.t[reg];
    const int64_t wgs = set_grid(a, p.s, t.tile, t.split, t.kt_part, parts);
    launch_tiled(product, et, reg, t.tile, a, dim3((unsigned)wgs), st);
    const gemm_status e = launched();
    return e != GEMM_OK || t.split == 1 ? e : run_sum(et, p.s, a, st);
}

template <int P>
void launch_merged(int et, bool reg, int tile, const ProductArgs& x, const ProductArgs& w, int nx, dim3 grid, hipStream_t st) {
    if (et == spg::kElBF16) {
        if (reg) spg::launch_gradients<spg::kElBF16, P, true>(tile, x, w, nx, grid, st);
        else spg::launch_gradients<spg::kElBF16, P, false>(tile, x, w, nx, grid, st);
    } else {
        if (reg) spg::launch_gradients<spg::kElF16, P, true>(tile, x, w, nx, grid, st);
        else spg::launch_gradients<spg::kElF16, P, false>(tile, x, w, nx, grid, st);
    }
}

gemm_status run_merged(bool nk, int et, bool reg, const Merged& m, const Shape& sx, const Shape& sw, ProductArgs x,
                       ProductArgs w, void* parts, hipStream_t st) {
    const int64_t nx = set_grid(x, sx, m.tile, m.split, m.kt_part, parts);
    const int64_t nw = set_grid(w, sw, m.tile, 1, sw.kt, nullptr);
    const dim3 grid((unsigned)(nx + nw));
    if (nk) launch_merged<spg::kGradXNK>(et, reg, m.tile, x, w, (int)nx, grid, st);
    else launch_merged<spg::kGradXKN>(et, reg, m.tile, x, w, (int)nx, grid, st);
    const gemm_status e = launched();
    return e != GEMM_OK || m.split == 1 ? e : run_sum(et, sx, x, st);
}

template <int ET, bool DUAL>
void stream_rows(const ProductArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)ceil_div(a.N, 16)), wg(512);
    const uintptr_t all = (uintptr_t)a.A | (uintptr_t)a.B[0] | (DUAL ? (uintptr_t)a.B[1] : 0) | (uintptr_t)a.lda | (uintptr_t)a.ldb;
    if (all % 4 == 0) hipLaunchKernelGGL((spg::stream_kernel<ET, DUAL, true, 8, 4>), grid, wg, 0, st, a);
    else hipLaunchKernelGGL((spg::stream_kernel<ET, DUAL, false, 8, 4>), grid, wg, 0, st, a);
}

template <int ET, bool DUAL>
gemm_status run_simple(const spg::SimpleArgs& a, hipStream_t st) {
    const int64_t n = std::min<int64_t>(ceil_div((int64_t)a.p.M * a.p.N, 256), 1 << 16);
    hipLaunchKernelGGL((spg::simple_product<ET, DUAL>), dim3((unsigned)n), dim3(256), 0, st, a);
    return launched();
}

constexpr int64_t kStreamRows = 16;   // one MFMA tile of rows
// Rows of operands are addressed by 32-bit offsets below 2^31: 256 of them fit up to here.
constexpr int64_t kMaxRowBytes = ((int64_t)1 << 23) - 128;

}  // namespace

struct gemm_gated_plan {
    int64_t M, N, K;
    int et;
    bool nk;
    int act;
    bool simple, simple_back;
    int64_t np;              // columns of dG and of dU in the workspace
    Stored x, w;
    Planned fwd, dx, dw;
    Merged both[2];          // [register-staged]
    int64_t ws_fwd, ws_back, off_part;
};

struct gemm_quantized_plan {
    int64_t M, N, K;
    int out, act;
    bool simple;
    Stored a, b;
    Planned p;
    int64_t ws;
};

namespace {
// few rows with K-contiguous weights: the streaming kernel
bool streams(const gemm_gated_plan* p) { return p->nk && p->M <= kStreamRows; }
}  // namespace

extern "C" {

gemm_status gemm_gated_create(gemm_gated_handle* out, int64_t M, int64_t N, int64_t K, gemm_dtype dtype,
                              gemm_b_layout layout, gemm_activation act) {
    if (!out) return GEMM_ERR_INVALID_ARG;
    *out = nullptr;
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
    if (dtype != GEMM_F16 && dtype != GEMM_BF16) return GEMM_ERR_INVALID_ARG;
    if (layout != GEMM_B_KN && layout != GEMM_B_NK) return GEMM_ERR_INVALID_ARG;
    if (act != GEMM_ACT_SILU && act != GEMM_ACT_GELU_TANH && act != GEMM_ACT_RELU) return GEMM_ERR_INVALID_ARG;
    const int64_t lim = INT32_MAX / 2 - 512;
    if (M > lim || N > lim || K > lim) return GEMM_ERR_UNSUPPORTED;
    gemm_gated_plan* p = new (std::nothrow) gemm_gated_plan;
    if (!p) return GEMM_ERR_OUT_OF_MEMORY;
    p->M = M;
    p->N = N;
    p->K = K;
    p->et = dtype == GEMM_BF16 ? spg::kElBF16 : spg::kElF16;
    p->nk = layout == GEMM_B_NK;
    p->act = (int)act;
    const double m = (double)M, n = (double)N, k = (double)K;
    const bool empty = M == 0 || N == 0;
    // the tiled kernel needs 16 bytes of every row it copies, and 32-bit offsets
    p->simple = empty || K < 8 || (!p->nk && N < 8) || K * 2 > kMaxRowBytes || (!p->nk && N * 2 > kMaxRowBytes);
    p->np = up(N, 64);
    p->simple_back = p->simple || p->np * 4 > kMaxRowBytes || K == 0;
    p->x = Stored{M, K * 2};
    p->w = p->nk ? Stored{N, K * 2} : Stored{K, N * 2};
    const double grad_bytes = 2 * (2 * m * n + 2 * n * k + m * k);
    p->fwd = p->dx = p->dw = Planned{};
    if (!p->simple && !streams(p))
        p->fwd = plan_product(Shape{M, N, ceil_div(K, 64), 1, 1, 2, 2 * (m * k + 2 * n * k + m * n), false}, {p->x, p->w, p->w});
    if (!p->simple_back) {
        p->dx = plan_product(Shape{M, K, 2 * ceil_div(N, 64), 1, 1, 1, grad_bytes, false}, {p->w, p->w});
        p->dw = plan_product(p->nk ? Shape{N, K, ceil_div(M, 64), 2, 1, 1, grad_bytes, false}
                                   : Shape{K, N, ceil_div(M, 64), 1, 2, 1, grad_bytes, false}, {p->x});
    }
    int64_t merged = 0;
    for (int r = 0; r < 2; ++r) {
        p->both[r] = p->simple_back ? Merged{} : merge(p->dx, p->dw, r == 1);
        if (p->both[r].on) merged = std::max(merged, part_bytes(p->dx.s, Tiling{0, p->both[r].split, 0, 0.0}));
    }
    p->ws_fwd = p->fwd.bytes();
    p->off_part = up(M * p->np * 4, kAlign);
    p->ws_back = p->off_part + std::max(merged, std::max(p->dx.parts, p->dw.parts) + p->dx.packed + p->dw.packed);
    *out = p;
    return GEMM_OK;
}

int64_t gemm_gated_workspace(gemm_gated_handle h) { return h ? std::max(h->ws_fwd, h->ws_back) : -1; }
int64_t gemm_gated_run_workspace(gemm_gated_handle h) { return h ? h->ws_fwd : -1; }

gemm_status gemm_gated_run(gemm_gated_handle h, const void* X, const void* Wg, const void* Wu, void* H, void* G,
                           void* U, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (!h || (G == nullptr) != (U == nullptr)) return GEMM_ERR_INVALID_ARG;
    if (h->M == 0 || h->N == 0) return GEMM_OK;
    if (!H || (h->K > 0 && (!X || !Wg || !Wu))) return GEMM_ERR_INVALID_ARG;
    ProductArgs a{};
    a.A = (const char*)X;
    a.B[0] = (const char*)Wg;
    a.B[1] = (const char*)Wu;
    a.C = H;
    a.G = G;
    a.U = U;
    a.M = (int32_t)h->M;
    a.N = (int32_t)h->N;
    a.K = (int32_t)h->K;
    a.lda = (uint32_t)(h->K * 2);
    a.ldb = (uint32_t)((h->nk ? h->K : h->N) * 2);
    a.b_cols = (int32_t)h->N;
    a.segments = 1;
    a.act = (uint8_t)h->act;
    if (h->simple) {
        spg::SimpleArgs s{a, h->K, 1, h->nk ? h->K : 1, h->nk ? 1 : h->N, 0};
        return h->et == spg::kElBF16 ? run_simple<spg::kElBF16, true>(s, stream) : run_simple<spg::kElF16, true>(s, stream);
    }
    if (streams(h)) {
        if (h->et == spg::kElBF16) stream_rows<spg::kElBF16, true>(a, stream);
        else stream_rows<spg::kElF16, true>(a, stream);
        return launched();
    }
    const bool xa = a.lda % 4 == 0 && words(X), wa = a.ldb % 4 == 0 && words(Wg) && words(Wu);
    const bool pack = h->fwd.pack && !(xa && wa);
    const bool reg = !pack && !(xa && wa);
    const int64_t need = (pack ? h->fwd.packed : 0) + part_bytes(h->fwd.s, h->fwd.t[reg]);
    if (need > 0 && (!workspace || (uintptr_t)workspace % 16 != 0 || workspace_bytes < h->ws_fwd)) return GEMM_ERR_INVALID_ARG;
    if (pack) {
        Operands o((char*)workspace + h->fwd.parts);
        if (!xa) o.copy(h->x, a.A, a.lda);
        if (!wa) {
            o.copy(h->w, a.B[0], a.ldb);
            o.copy(h->w, a.B[1], a.ldb);
            a.b_cols = (int32_t)up(h->N, 8);
        }
        const gemm_status e = o.launch(2, stream);
        if (e != GEMM_OK) return e;
    }
    return run_tiled(h->nk ? spg::kGatedNK : spg::kGatedKN, h->et, reg, h->fwd, a, workspace, stream);
}

gemm_status gemm_gated_backward(gemm_gated_handle h, const void* dH, const void* X, const void* Wg, const void* Wu,
                                const void* G, const void* U, void* dX, void* dWg, void* dWu, void* workspace,
                                int64_t workspace_bytes, hipStream_t stream) {
    if (!h) return GEMM_ERR_INVALID_ARG;
    const int64_t M = h->M, N = h->N, K = h->K;
    if (K == 0 || (M == 0 && N == 0)) return GEMM_OK;      // every gradient is empty
    if ((M > 0 && !dX) || (N > 0 && (!dWg || !dWu))) return GEMM_ERR_INVALID_ARG;
    if (M > 0 && N > 0) {
        if (!dH || !X || !Wg || !Wu || !G || !U) return GEMM_ERR_INVALID_ARG;
        if (!workspace || (uintptr_t)workspace % 16 != 0 || workspace_bytes < h->ws_back) return GEMM_ERR_INVALID_ARG;
    }
    const bool bf = h->et == spg::kElBF16;
    uint16_t* D = (uint16_t*)workspace;
    void* parts = (char*)workspace + h->off_part;
    if (M > 0 && N > 0) {
        const int64_t items = M * (h->np / 8);
        const dim3 grid((unsigned)ceil_div(items, 256));
        if (bf) hipLaunchKernelGGL((spg::gated_slopes<true>), grid, dim3(256), 0, stream, (const uint16_t*)dH,
                                   (const uint16_t*)G, (const uint16_t*)U, D, (int)M, (int)N, (int)h->np, h->act);
        else hipLaunchKernelGGL((spg::gated_slopes<false>), grid, dim3(256), 0, stream, (const uint16_t*)dH,
                                (const uint16_t*)G, (const uint16_t*)U, D, (int)M, (int)N, (int)h->np, h->act);
        const gemm_status e = launched();
        if (e != GEMM_OK) return e;
    }
    // dX = [dG dU] . [Wg; Wu]: one sum over both segments
    ProductArgs x{};
    x.A = (const char*)D;
    x.B[0] = (const char*)Wg;
    x.B[1] = (const char*)Wu;
    x.C = dX;
    x.M = (int32_t)M;
    x.N = (int32_t)K;
    x.K = (int32_t)N;
    x.lda = (uint32_t)(h->np * 4);
    x.ldb = (uint32_t)((h->nk ? K : N) * 2);
    x.b_cols = (int32_t)K;
    x.segments = 2;
    // dWg, dWu: [N,K] weights dG^T X and dU^T X, [K,N] weights X^T dG and X^T dU
    ProductArgs w{};
    const char* const d[2] = {(const char*)D, (const char*)(D + h->np)};
    w.A = h->nk ? d[0] : (const char*)X;
    w.A1 = h->nk ? d[1] : (const char*)X;
    for (int z = 0; z < 2; ++z) w.B[z] = h->nk ? (const char*)X : d[z];
    w.C = dWg;
    w.C1 = dWu;
    w.M = (int32_t)(h->nk ? N : K);
    w.N = (int32_t)(h->nk ? K : N);
    w.K = (int32_t)M;
    const int64_t lda = h->nk ? h->np * 4 : K * 2, ldb = h->nk ? K * 2 : h->np * 4;
    w.lda = (uint32_t)lda;
    w.ldb = (uint32_t)ldb;
    w.a_cols = (int32_t)(h->nk ? h->np : K);
    w.b_cols = (int32_t)(h->nk ? K : h->np);
    w.segments = 1;
    if (h->simple_back) {
        if (M > 0) {
            spg::SimpleArgs s{x, 2 * h->np, 1, h->nk ? 1 : N, h->nk ? K : 1, h->np};
            const gemm_status e = bf ? run_simple<spg::kElBF16, false>(s, stream) : run_simple<spg::kElF16, false>(s, stream);
            if (e != GEMM_OK) return e;
        }
        for (int z = 0; z < 2 && N > 0; ++z) {
            ProductArgs one = w;
            one.A = z ? w.A1 : w.A;
            one.B[0] = w.B[z];
            one.C = z ? w.C1 : w.C;
            spg::SimpleArgs s{one, 1, lda / 2, 1, ldb / 2, 0};
            const gemm_status e = bf ? run_simple<spg::kElBF16, false>(s, stream) : run_simple<spg::kElF16, false>(s, stream);
            if (e != GEMM_OK) return e;
        }
        return GEMM_OK;
    }
    const bool wa = x.ldb % 4 == 0 && words(Wg) && words(Wu);
    const bool xa = K % 2 == 0 && words(X);
    const Merged& both = h->both[!(wa && xa)];
    if (both.on)
        return run_merged(h->nk, h->et, !(wa && xa), both, h->dx.s, h->dw.s, x, w, parts, stream);
    Operands o((char*)parts + std::max(h->dx.parts, h->dw.parts));
    if (!wa && h->dx.pack) {
        o.copy(h->w, x.B[0], x.ldb);
        o.copy(h->w, x.B[1], x.ldb);
        x.b_cols = (int32_t)up(K, 8);
    }
    if (!xa && h->dw.pack) {
        const char* p = (const char*)X;
        o.copy(h->x, p, h->nk ? w.ldb : w.lda);
        if (h->nk) w.B[0] = w.B[1] = p;
        else w.A = w.A1 = p;
        (h->nk ? w.b_cols : w.a_cols) = (int32_t)up(K, 8);
    }
    gemm_status e = o.launch(2, stream);
    if (e != GEMM_OK) return e;
    e = run_tiled(h->nk ? spg::kGradXNK : spg::kGradXKN, h->et, !wa && !h->dx.pack, h->dx, x, parts, stream);
    if (e != GEMM_OK) return e;
    return run_tiled(spg::kGradW, h->et, !xa && !h->dw.pack, h->dw, w, parts, stream);
}

gemm_status gemm_gated_destroy(gemm_gated_handle h) {
    delete h;
    return GEMM_OK;
}

gemm_status gemm_quantized_create(gemm_quantized_handle* out, int64_t M, int64_t N, int64_t K, gemm_dtype out_dtype,
                                  gemm_activation act) {
    if (!out) return GEMM_ERR_INVALID_ARG;
    *out = nullptr;
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
    if (out_dtype != GEMM_F16 && out_dtype != GEMM_BF16 && out_dtype != GEMM_F32) return GEMM_ERR_INVALID_ARG;
    if (act != GEMM_ACT_NONE && act != GEMM_ACT_SILU && act != GEMM_ACT_GELU_TANH && act != GEMM_ACT_RELU)
        return GEMM_ERR_INVALID_ARG;
    const int64_t lim = INT32_MAX / 2 - 512;
    // 128 * 128 * K stays below 2^31 up to here: the int32 sums cannot overflow
    if (M > lim || N > lim || K > 131071) return GEMM_ERR_UNSUPPORTED;
    gemm_quantized_plan* p = new (std::nothrow) gemm_quantized_plan;
    if (!p) return GEMM_ERR_OUT_OF_MEMORY;
    p->M = M;
    p->N = N;
    p->K = K;
    p->out = (int)out_dtype;
    p->act = (int)act;
    p->simple = M == 0 || N == 0 || K < 16;
    const double m = (double)M, n = (double)N, k = (double)K;
    const int mats = act == GEMM_ACT_NONE ? 1 : 2;
    p->a = Stored{M, K};
    p->b = Stored{N, K};
    p->p = Planned{};
    if (!p->simple && M > kStreamRows) {
        const Shape s{M, N, ceil_div(K, 128), 1, 1, mats, m * k + mats * n * k + m * n * (out_dtype == GEMM_F32 ? 4 : 2), false};
        p->p = mats == 2 ? plan_product(s, {p->a, p->b, p->b}) : plan_product(s, {p->a, p->b});
    }
    p->ws = p->p.bytes();
    *out = p;
    return GEMM_OK;
}

int64_t gemm_quantized_workspace(gemm_quantized_handle h) { return h ? h->ws : -1; }

gemm_status gemm_quantized_run(gemm_quantized_handle h, const int8_t* A, const float* scale_a, const int8_t* B,
                               const float* scale_b, const int8_t* B2, const float* scale_b2, void* C,
                               void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (!h) return GEMM_ERR_INVALID_ARG;
    const bool dual = h->act != GEMM_ACT_NONE;
    if (!dual && (B2 || scale_b2)) return GEMM_ERR_INVALID_ARG;
    if (h->M == 0 || h->N == 0) return GEMM_OK;
    if (!C || !scale_a || !scale_b || (dual && !scale_b2)) return GEMM_ERR_INVALID_ARG;
    if (h->K > 0 && (!A || !B || (dual && !B2))) return GEMM_ERR_INVALID_ARG;
    ProductArgs a{};
    a.A = (const char*)A;
    a.B[0] = (const char*)B;
    a.B[1] = (const char*)B2;
    a.C = C;
    a.sa = scale_a;
    a.sb[0] = scale_b;
    a.sb[1] = scale_b2;
    a.M = (int32_t)h->M;
    a.N = (int32_t)h->N;
    a.K = (int32_t)h->K;
    a.lda = a.ldb = (uint32_t)h->K;
    a.segments = 1;
    a.out_dtype = (uint8_t)h->out;
    a.act = (uint8_t)h->act;
    if (h->simple) {
        spg::SimpleArgs s{a, h->K, 1, h->K, 1, 0};
        return dual ? run_simple<spg::kElI8, true>(s, stream) : run_simple<spg::kElI8, false>(s, stream);
    }
    if (h->M <= kStreamRows) {
        if (dual) stream_rows<spg::kElI8, true>(a, stream);
        else stream_rows<spg::kElI8, false>(a, stream);
        return launched();
    }
    const bool aa = h->K % 4 == 0 && words(A), ba = h->K % 4 == 0 && words(B) && (!dual || words(B2));
    const bool pack = h->p.pack && !(aa && ba);
    const bool reg = !pack && !(aa && ba);
    const int64_t need = (pack ? h->p.packed : 0) + part_bytes(h->p.s, h->p.t[reg]);
    if (need > 0 && (!workspace || (uintptr_t)workspace % 16 != 0 || workspace_bytes < h->ws)) return GEMM_ERR_INVALID_ARG;
    if (pack) {
        Operands o((char*)workspace + h->p.parts);
        if (!aa) o.copy(h->a, a.A, a.lda);
        if (!ba) {
            o.copy(h->b, a.B[0], a.ldb);
            if (dual) o.copy(h->b, a.B[1], a.ldb);
        }
        const gemm_status e = o.launch(1, stream);
        if (e != GEMM_OK) return e;
    }
    return run_tiled(dual ? spg::kInt8Gated : spg::kInt8, spg::kElI8, reg, h->p, a, workspace, stream);
}

gemm_status gemm_quantized_destroy(gemm_quantized_handle h) {
    delete h;
    return GEMM_OK;
}

gemm_status gemm_quantize_rows(const void* X, gemm_dtype dtype, int64_t rows, int64_t K, int8_t* A, float* scale,
                               hipStream_t stream) {
    if (rows < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
    if (dtype != GEMM_F16 && dtype != GEMM_BF16 && dtype != GEMM_F32) return GEMM_ERR_INVALID_ARG;
    if (rows == 0) return GEMM_OK;
    if (!scale || (K > 0 && (!X || !A))) return GEMM_ERR_INVALID_ARG;
    if (rows > INT32_MAX) return GEMM_ERR_UNSUPPORTED;
    // Vectors of a thread just enough for the row: every further one that it does not need costs
    // (8192 bf16 rows of 4096: 20.8, 21.6, 26.3 and 42.6 us with 2, 4, 8 and 16).  Rows of more
    // than 64 KiB are read twice (8192 fp32 rows of 12288: 138 us, from registers 94).  A wave a
    // row where there are many short ones (8192 bf16 rows of 512: 4.9 us, a workgroup a row 9.0;
    // of 1024: 7.9 and 11.4; but 1024 rows of 1024: 3.4 and 3.3).
    auto go = [&](auto dt) {
        constexpr int D = decltype(dt)::value;
        const int64_t vecs = ceil_div(K, spg::RowVec<D>::E);
        const char* x = (const char*)X;
        auto launch = [&](auto v, auto w) {
            constexpr int V = decltype(v)::value, W = decltype(w)::value;
            const int64_t wgs = ceil_div(rows * W, 4), gx = std::min<int64_t>(wgs, 1 << 23);
            const dim3 grid((unsigned)gx, (unsigned)ceil_div(wgs, gx));
            hipLaunchKernelGGL((spg::quantize_rows<D, V, W>), grid, dim3(256), 0, stream, x, A, scale, K, rows);
        };
        constexpr std::integral_constant<int, 1> wave{};
        constexpr std::integral_constant<int, 4> group{};
        if (vecs <= 2 * 64 && rows >= 2048) launch(std::integral_constant<int, 2>{}, wave);
        else if (vecs <= 2 * 256) launch(std::integral_constant<int, 2>{}, group);
        else if (vecs <= 4 * 256) launch(std::integral_constant<int, 4>{}, group);
        else if (vecs <= 8 * 256) launch(std::integral_constant<int, 8>{}, group);
        else if (vecs <= 16 * 256) launch(std::integral_constant<int, 16>{}, group);
        else launch(std::integral_constant<int, 0>{}, group);
    };
    if (dtype == GEMM_F16) go(std::integral_constant<int, spg::kOutF16>{});
    else if (dtype == GEMM_BF16) go(std::integral_constant<int, spg::kOutBF16>{});
    else go(std::integral_constant<int, spg::kOutF32>{});
    return launched();
}

}  // extern "C"
