// Device code of the feed-forward operators for gfx950 (MI355X): the gated projection, its
// backward pass and the int8 products (declared in include/spgemm.h).
//
// Everything here is a matrix product with something around it:
//   gated      H = act(X Wg) * (X Wu)                    two B matrices, one A
//   dX         dG Wg^T + dU Wu^T                          one sum over two segments
//   dW         X^T dG and X^T dU                          A stored reduction-major, two results
//   quantized  (Aq Bq^T) sa sb, or gated from two of them int8 operands, int32 sums
// so one tiled kernel computes all of them; its template parameters say how the operands
// are stored and what the epilogue does.  Beside it: a kernel for few rows that streams
// the weights through registers, the sum over the parts of a split reduction, the
// elementwise part of the backward pass, and the quantisation of rows.
//
// Operands are addressed in bytes.  A k-tile is 128 bytes of a K-contiguous row: 64
// elements of fp16/bf16 or 128 of int8.  v_mfma_f32_16x16x32_{f16,bf16} and
// v_mfma_i32_16x16x64_i8 take the same 16 bytes per lane at the same places, so the LDS
// layout, the copies and the fragment reads do not depend on the element type.
#pragma once

#include "gemm_kernels.hpp"
#include "tile_copy.hpp"

namespace spg {

enum { kElF16 = 0, kElBF16 = 1, kElI8 = 2 };
enum { kActNone = 0, kActSilu = 1, kActGelu = 2, kActRelu = 3 };

typedef int32_t intx4 __attribute__((ext_vector_type(4)));

// Kept small: the host writes a launch's arguments through PCIe, about 4 ns a byte (an empty
// kernel with 40 bytes of them launches in 2.8 us, with 232 in 3.6).
struct ProductArgs {
    const char* A;
    const char* B[2];   // B[1]: the up projection; the second segment; the second result's B
    void* C;
    union {
        struct {        // int8: row scales of A, column scales of B[0] and B[1]
            const float* sa;
            const float* sb[2];
        };
        struct {        // gated: the pre-activations, or null
            void* G;
            void* U;
        };
        struct {        // weight gradients: the second result and (for [N,K] weights) its A
            const char* A1;
            void* C1;
        };
    };
    float* part;        // split reduction: fp32 (int8: int32) partial sums, or null
    uint32_t lda, ldb;  // bytes between the stored rows of A and of B
    int32_t M, N, K;    // rows and columns of one result, length of one segment of the sum
    int32_t a_cols, b_cols;   // operands stored reduction-major: columns that may be read
    int32_t tiles_m, tiles_n; // of one result
    int32_t kt_part;    // k-tiles of one part
    uint8_t zm, zn;     // results stacked along the rows or columns of the tile grid (1 or 2)
    uint8_t group_m;
    uint8_t split;      // parts of the reduction (the grid is split times the tiles)
    uint8_t segments;   // 1, or 2: B[1] continues the sum where B[0] ends
    uint8_t out_dtype, act;
};

// elements between the rows of partial sums
__device__ __forceinline__ int64_t part_pitch(const ProductArgs& a, bool dual) {
    return (int64_t)((a.N + 3) & ~3) * (dual ? 2 : 1) * a.zn;
}

__device__ __forceinline__ float silu(float x) {
    // x / (1 + exp(-x)), exp as 2^(x log2 e); saturates to -0 and to x.  The hardware's exp2 and
    // reciprocal are within 1 ulp: with the argument's rounding the sigmoid is within 2^-20,
    // a sixteenth of an fp16 result's rounding (2^-11), for 5 instructions
    const float e = __builtin_amdgcn_exp2f(-1.4426950408889634f * x);
    return x * __builtin_amdgcn_rcpf(1.0f + e);
}

template <int ACT>
__device__ __forceinline__ float act_t(float x) {
    if constexpr (ACT == kActSilu) return silu(x);
    else if constexpr (ACT == kActGelu) return gelu_tanh(x);
    else if constexpr (ACT == kActRelu) return x <= 0.0f ? 0.0f : x;   // NaN stays NaN
    else return x;
}

// f(integral_constant<ACT>) for the run-time activation: one uniform branch
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    if (act == kActSilu) f(std::integral_constant<int, kActSilu>{});
    else if (act == kActGelu) f(std::integral_constant<int, kActGelu>{});
    else f(std::integral_constant<int, kActRelu>{});
}

template <typename F>
__device__ __forceinline__ void with_out(int od, F&& f) {
    if (od == kOutF32) f(std::integral_constant<int, kOutF32>{});
    else if (od == kOutBF16) f(std::integral_constant<int, kOutBF16>{});
    else f(std::integral_constant<int, kOutF16>{});
}

template <int OD>
__device__ __forceinline__ uint32_t out_bits(float x) {
    if constexpr (OD == kOutF32) return __builtin_bit_cast(uint32_t, x);
    else return f32_to_bits(x, OD == kOutBF16);
}

// Workgroup id -> tile of the grid and part of the reduction.  Each XCD (workgroup id mod
// 8) gets a contiguous range of (part, tile); tiles are rastered in groups of group_m rows.
__device__ __forceinline__ void product_tile(int wg, const ProductArgs& a, int& tm, int& tn, int& sp) {
    const int rows = a.tiles_m * a.zm, cols = a.tiles_n * a.zn;
    const int T = rows * cols, W = T * a.split;
    const int x = wg & 7, i = wg >> 3, q = W >> 3, r = W & 7;
    wg = x * q + (x < r ? x : r) + i;
    sp = wg / T;
    wg -= sp * T;
    const int gsz = a.group_m * cols;
    const int g = wg / gsz;
    const int first = g * a.group_m;
    const int rem = rows - first;
    const int gm = rem < a.group_m ? rem : a.group_m;
    const int in = wg - g * gsz;
    tm = first + in % gm;
    tn = in / gm;
}

// Swizzle of a reduction-major tile row of CPR 16-byte chunks (the transposing reads).  16
// chunks or more: nswz.  A transposing read takes 32 bytes of rows k .. k+3, and of rows
// k+8 .. k+11 with it; with 128-byte rows two of them share each half of the banks' 256
// bytes, so bits 1 and 3 of the row pick the 32-byte window; with 64-byte rows four
// consecutive rows fill the banks and bit 3 alone separates the two groups.
template <int CPR>
__device__ __forceinline__ int nswz_t(int k) {
    if constexpr (CPR >= 16) return nswz(k);
    else if constexpr (CPR == 8) return 2 * (((k >> 1) & 1) | ((k >> 2) & 2));
    else return 2 * ((k >> 3) & 1);
}

// One 16x16 MFMA: x the B fragment (columns), y the A fragment (rows); the accumulator of
// lane l holds row l%16, columns 4(l/16) .. +3.
template <int ET>
using AccOf = std::conditional_t<ET == kElI8, intx4, floatx4>;

template <int ET>
__device__ __forceinline__ AccOf<ET> mma(const u32x4& x, const u32x4& y, const AccOf<ET>& c) {
    if constexpr (ET == kElI8)
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(intx4, x),
                                                     __builtin_bit_cast(intx4, y), c, 0, 0, 0);
    else
        return mfma16<ET == kElBF16>(x, y, c);
}

// The top `bits` (a multiple of 8, 0 .. 120) of 128 cleared.
__device__ __forceinline__ u32x4 clear_top(u32x4 v, uint32_t bits) {
    u32x4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int keep = 128 - (int)bits - 32 * e;        // bits of this word that stay
        r[e] = keep >= 32 ? v[e] : keep <= 0 ? 0u : v[e] & ((1u << keep) - 1u);
    }
    return r;
}

// A store of 16 bytes to an address that is only element-aligned: compute queues run in
// unaligned-access mode, so it is one instruction.
struct __attribute__((packed, aligned(2))) Bytes16 { u32x4 v; };

// The epilogue of 4 consecutive columns of row m held by one thread, `left` of them inside
// the row; o is their place in the result.  s1 is the up projection's sums when DUAL.
template <int OD>
__device__ __forceinline__ void store4(void* C, size_t o, const float (&v)[4], int left) {
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = out_bits<OD>(v[e]);
    if constexpr (OD == kOutF32) {
        uint32_t* d = (uint32_t*)C + o;
        struct __attribute__((packed, aligned(4))) B16 { u32x4 v; };
        if (left == 4) ((B16*)d)->v = u32x4{b[0], b[1], b[2], b[3]};
        else
            for (int e = 0; e < left; ++e) d[e] = b[e];
    } else {
        uint16_t* d = (uint16_t*)C + o;
        struct __attribute__((packed, aligned(2))) B8 { u32x2 v; };
        if (left == 4) ((B8*)d)->v = u32x2{b[0] | (b[1] << 16), b[2] | (b[3] << 16)};
        else
            for (int e = 0; e < left; ++e) d[e] = (uint16_t)b[e];
    }
}

template <int ET, bool DUAL>
__device__ __forceinline__ void finish4(const AccOf<ET>& s0, const AccOf<ET>& s1, int m, int n, int left, size_t o,
                                        const ProductArgs& args, int z = 0) {
    float v[4], w[4];
    if constexpr (ET == kElI8) {
        // fp32 from here: sums beyond 2^24 are rounded, as is the product with each scale, 2^-24
        // each (16-bit results round by 2^-11 or 2^-8).  Scaled in 64 bits and rounded once:
        // 10.7 -> 11.0 us at 333 x 2050 x 1531, 350 -> 362 at 8192 x 4096 x 12288
        const float rs = args.sa[m];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = e < left ? n + e : n;
            v[e] = (float)s0[e] * rs * args.sb[0][c];
            if constexpr (DUAL) w[e] = (float)s1[e] * rs * args.sb[1][c];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) { v[e] = s0[e]; w[e] = s1[e]; }
    }
    auto put = [&](void* C, const float (&x)[4]) {
        if constexpr (ET == kElBF16) store4<kOutBF16>(C, o, x, left);
        else if constexpr (ET == kElF16) store4<kOutF16>(C, o, x, left);
        else with_out(args.out_dtype, [&](auto od) { store4<decltype(od)::value>(C, o, x, left); });
    };
    if constexpr (DUAL) {
        // G and U in 16 bits, as training keeps them; H from the fp32 sums
        if (ET != kElI8 && args.G) {
            put(args.G, v);
            put(args.U, w);
        }
        float h[4];
        with_act(args.act, [&](auto ac) {
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = act_t<decltype(ac)::value>(v[e]) * w[e];
        });
        put(args.C, h);
    } else {
        put(z ? args.C1 : args.C, v);
    }
}

// One wave's output block through LDS: 32 rows at a time are written to the wave's own
// staging area (4 consecutive columns per lane and accumulator) and read back as 16-byte
// row segments.  val(bn, bm, e) is the output of accumulator (bn, bm), element e.
template <int OD, int TM, int TNO, int WNO, typename F>
__device__ __forceinline__ void store_block(F&& val, SPG_LDS char* stg, void* C, int M, int N, int m_base,
                                            int n_base, int lane) {
    constexpr int OB = OD == kOutF32 ? 4 : 2;
    constexpr int ROWB = WNO * OB;
    constexpr int CPR = ROWB / 16;
    constexpr int E16 = 16 / OB;
    static_assert(CPR == 4 || CPR == 8 || CPR == 16 || CPR == 32, "staging swizzle");
    static_assert(TM % 2 == 0, "32-row blocks");
    auto swz = [](int row) { return CPR >= 16 ? (row & 15) : CPR == 8 ? ((row >> 1) & 7) : ((row >> 2) & 3); };
    // 16-byte stores where rows and base allow, whole-line rows past the caches' allocation
    // (C is not read here), as in store_tile
    const bool vec_ok = ((size_t)N * OB) % 16 == 0 && (uintptr_t)C % 16 == 0;
    const bool nt_rows = vec_ok && ((size_t)N * OB) % 128 == 0 && ROWB >= 128;
    const int lrow = lane & 15;
#pragma unroll
    for (int g = 0; g < TM / 2; ++g) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int bm = 2 * g + h, row = h * 16 + lrow;
#pragma unroll
            for (int bn = 0; bn < TNO; ++bn) {
                uint32_t b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) b[e] = out_bits<OD>(val(bn, bm, e));
                const int byte = (bn * 16 + 4 * (lane >> 4)) * OB;
                SPG_LDS char* dst = stg + row * ROWB + (((byte >> 4) ^ swz(row)) << 4) + (byte & 15);
                if constexpr (OD == kOutF32) *(SPG_LDS u32x4*)dst = u32x4{b[0], b[1], b[2], b[3]};
                else *(SPG_LDS u32x2*)dst = u32x2{b[0] | (b[1] << 16), b[2] | (b[3] << 16)};
            }
        }
#pragma unroll 1
        for (int it = 0; it < (32 * CPR) / 64; ++it) {
            const int idx = it * 64 + lane;
            const int row = idx / CPR, ch = idx % CPR;
            const u32x4 v = *(const SPG_LDS u32x4*)(stg + row * ROWB + ((ch ^ swz(row)) << 4));
            const int gm = m_base + g * 32 + row, gn = n_base + ch * E16;
            if (gm < M && gn < N) {
                char* d = (char*)C + ((size_t)gm * N + gn) * OB;
                if (gn + E16 <= N) {
                    if (nt_rows) __builtin_nontemporal_store(v, (u32x4*)d);
                    else if (vec_ok) *(u32x4*)d = v;
                    else ((Bytes16*)d)->v = v;
                } else {
#pragma unroll
                    for (int e = 0; e < E16; ++e) {
                        if (gn + e >= N) break;
                        if constexpr (OB == 4) ((uint32_t*)d)[e] = v[e];
                        else ((uint16_t*)d)[e] = (uint16_t)(v[e >> 1] >> ((e & 1) * 16));
                    }
                }
            }
        }
    }
}

// Geometry of the tiled kernel: BM x BN tile, WM x WN per wave, S ring slots (DEEP: one
// more of B).  DUAL: the BN columns are BN/2 of each B matrix, and every wave holds WN/2
// of each for the same output columns.  KG groups of NW waves each: group g multiplies the
// k-tiles g, g + KG, ... of the whole tile, with a ring of its own, and their sums meet in
// LDS at the end.
template <bool DUAL, int BM, int BN, int WM, int WN, int S, bool DEEP, int KG>
struct ProductGeom {
    static constexpr int WAVES_N = BN / WN;
    static constexpr int NW = (BM / WM) * WAVES_N;
    static constexpr int NT = NW * KG * 64;
    static constexpr int TM = WM / 16, TN = WN / 16;
    static constexpr int BNS = DUAL ? BN / 2 : BN;      // columns of one B subtile
    static constexpr int WNS = DUAL ? WN / 2 : WN;      // a wave's columns of one B matrix
    static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
    static constexpr int A_OPS = A_BYTES / 1024 / NW, B_OPS = B_BYTES / 1024 / NW;
    static constexpr int L = A_OPS + B_OPS;
    static constexpr int NA = S, NB = S + (DEEP ? 1 : 0);
    static constexpr int RING = NA * A_BYTES + NB * B_BYTES;
    static constexpr int LDS = RING * KG;
    static constexpr int STG = 32 * WNS * 4;            // staging of one wave
    static constexpr int SUMS = (KG - 1) * NW * TM * TN * 1024;   // accumulators of the other groups
    static_assert(BM % WM == 0 && BN % WN == 0 && WM % 32 == 0 && WNS % 32 == 0, "wave tile");
    static_assert(A_OPS * 1024 * NW == A_BYTES && B_OPS * 1024 * NW == B_BYTES, "copy split");
    static_assert(!DUAL || NW % 2 == 0, "half of the waves copy each B matrix");
    static_assert(LDS <= 160 * 1024 && SUMS + NW * STG <= LDS, "LDS budget");
    static_assert(!DEEP || KG == 1, "ping-pong: one group of k-tiles");
    static_assert((S - 1) * L < 64, "vmcnt range");
    static_assert(!DEEP || S == 2, "the B-deep ring has two A and three B slots");
};

// The tiled kernel.  One workgroup owns a BM x BN tile (tm, tn) and one part (sp) of the reduction,
// keeps the sums in registers and streams k-tiles through a ring of LDS slots.
//   A_T   A is stored [K,M] (the weight gradients), read through the transposing LDS read
//   B_N   B is stored [K,N], else [N,K]
//   DUAL  two B matrices side by side in the tile and the gated epilogue: a lane holds the
//         gate's and the up projection's sums of the same outputs, so their product needs
//         no exchange
//   SEG   the sum may run over two segments with a B matrix each
//   REG   operands whose rows or base do not start on 4 bytes: k-tiles go through VGPRs
//         (two slots), loaded at any alignment; else they are copied straight into LDS
//   DEEP  a ring of two A and three B slots under the ping-pong schedule (the K loop)
//   TAIL  the sum may end inside a 16-byte chunk of a K-contiguous row (direct copies);
//         without it the large tiles save the registers and the code: int8 8192 x 4096 x
//         12288 takes 296 us without and 302 to 318 with it
//   KG    the waves form KG groups that take the k-tiles in turn: more waves to hide the
//         latencies of LDS reads, copies and barrier around the few MFMAs of a small tile
//         (64 x 128, 256 workgroups, 128 k-tiles: 44.2 us with one group of four waves and
//         six slots, 40.4 with two groups and three slots each)
// Otherwise a k-tile's barrier sits after the last LDS read of its slot; it publishes the
// next k-tile and releases the slot, which is refilled (k-tile t+S) behind it.
// Reads past an operand: rows past the end fall outside the buffer resource and read zero.
// A K-contiguous row's last k-tile masks the chunks past K by an offset outside every
// resource and clears the part of one that straddles K, so nothing of the next row is
// multiplied: a 0 * inf could not be undone.
//   GATHER  row r of A is row from.index[r] of a matrix of from.rows rows (outside them: zeros)
//   SKIP    waves whose rows all lie past the last one neither read fragments nor multiply, which
//           leaves their SIMDs' matrix cores to the others: for row tiles that are often cut
//   LOCAL   a part of the sum (args.part) goes to a buffer of this tile and part alone, in the
//           accumulators' order
struct SourceRows {
    const int32_t* index;
    int32_t rows;
};
template <int ET, bool A_T, bool B_N, bool DUAL, bool SEG, bool REG, int BM, int BN, int WM, int WN,
          int S, bool DEEP, int KG, bool TAIL, bool GATHER = false, bool SKIP = false, bool LOCAL = false>
__device__ __forceinline__ void product_tile_of(ProductArgs args, int tm, int tn, int sp, SPG_LDS char* lds,
                                                SourceRows from = SourceRows{}) {
    using G = ProductGeom<DUAL, BM, BN, WM, WN, S, DEEP, KG>;
    constexpr int TM = G::TM, TN = G::TN, BNS = G::BNS, WNS = G::WNS, NW = G::NW;
    constexpr int A_OPS = G::A_OPS, B_OPS = G::B_OPS, L = G::L;
    constexpr int ES = ET == kElI8 ? 1 : 2;           // bytes of an element
    constexpr int KT = 128 / ES;                      // elements of a k-tile
    static_assert(ET != kElI8 || (!A_T && !B_N), "int8 operands are K-contiguous");
    static_assert(!REG || (S == 2 && !DEEP), "register staging: two slots");
    static_assert(!SEG || (!A_T && !DUAL), "two segments: the input gradient");
    static_assert(!DUAL || !A_T, "gated: A is [M,K]");
    static_assert(!GATHER || (!A_T && !SEG), "gathered rows lie along the reduction");

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave_id = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kg = KG > 1 ? wave_id / NW : 0;         // group of k-tiles, wave within it
    const int wave = KG > 1 ? wave_id - kg * NW : wave_id;
    SPG_LDS char* ring = lds + kg * G::RING;
    struct Slot { SPG_LDS char* a; SPG_LDS char* b; };
    constexpr int NS = DEEP ? 6 : REG ? 4 : S;        // period of the slot (and register) pattern
    auto slot_of = [&](auto ic) -> Slot {
        constexpr int i = decltype(ic)::value % NS;
        return Slot{ring + (i % G::NA) * G::A_BYTES, ring + G::NA * G::A_BYTES + (i % G::NB) * G::B_BYTES};
    };

    const int wm = wave / G::WAVES_N, wn = wave % G::WAVES_N;

    if constexpr (kPoison) {
        for (int o = tid * 16; o < G::LDS; o += G::NT * 16) *(SPG_LDS u32x4*)(lds + o) = u32x4{~0u, ~0u, ~0u, ~0u};
        __syncthreads();
    }

    int z = 0;
    if (tm >= args.tiles_m) { tm -= args.tiles_m; z = 1; }
    if (tn >= args.tiles_n) { tn -= args.tiles_n; z = 1; }
    const int M = args.M, N = args.N, K = args.K;
    const int m0 = tm * BM, n0 = tn * BNS;
    const int seg_kt = (K + KT - 1) / KT;             // k-tiles of one segment
    const int nkt = SEG ? seg_kt * args.segments : seg_kt;
    const int kt0 = sp * args.kt_part;
    const int kt1 = kt0 + args.kt_part < nkt ? kt0 + args.kt_part : nkt;
    const int nk = (kt1 - kt0 + KG - 1) / KG;         // k-tiles of this part a group takes (>= 1)
    auto kt_of = [&](int t) { return kt0 + t * KG + kg; };
    const int tail = K * ES - (seg_kt - 1) * 128;     // bytes of a segment's last k-tile
    // SEG: A is dG and dU, padded to whole k-tiles
    using RowsA = RowCopy<REG, SEG>;
    using RowsB = RowCopy<REG, false>;
    using Columns = ColumnCopy<REG>;
    // bytes of a K-contiguous row that may be read: whole words for direct copies (rows of
    // whole words, or laid out again and padded with zeros)
    const uint32_t row_bytes = REG ? (uint32_t)(K * ES) : ((uint32_t)(K * ES) + 3u) & ~3u;

    // ---- copy sources ----
    const char* a_ptr = A_T && args.zm == 2 && z ? args.A1 : args.A;
    const char* b_ptr0 = args.B[!DUAL && args.zn == 2 ? z : 0];
    const char* b_ptr1 = args.B[1];
    // DUAL: waves of the lower half copy B[0], the others B[1]
    const bool up = DUAL && wave >= NW / 2;
    const char* b_mine = up ? b_ptr1 : b_ptr0;
    const int a_rows = M - m0 < BM ? M - m0 : BM;
    const int b_rows = N - n0 < BNS ? N - n0 : BNS;
    // Start and size of an operand's resource for a k-tile (0 past this part's last one: reads
    // zero).  K-contiguous rows: 128 bytes further per k-tile, up to the end of the tile's
    // last row.  Reduction-major: 64 rows further, as many of them as exist; columns past the
    // last are masked by offset.
    const uint32_t lda = args.lda, ldb = args.ldb;
    const uint64_t a_at = (uint64_t)(uintptr_t)a_ptr + (A_T ? 0 : (GATHER ? 0 : (uint64_t)m0 * lda) - RowsA::kBack);
    const uint64_t b_at[2] = {(uint64_t)(uintptr_t)b_mine + (B_N ? 0 : (uint64_t)n0 * ldb - RowsB::kBack),
                              (uint64_t)(uintptr_t)(SEG ? b_ptr1 : b_mine) + (B_N ? 0 : (uint64_t)n0 * ldb - RowsB::kBack)};
    const uint32_t a_all = (uint32_t)((GATHER ? (from.rows > 0 ? from.rows : 1) : a_rows) - 1) * lda + (SEG ? lda : row_bytes) + RowsA::kBack;
    const uint32_t b_all = (uint32_t)(b_rows - 1) * ldb + row_bytes + RowsB::kBack;
    auto a_win = [&](int kt) __attribute__((always_inline)) -> Win {
        if constexpr (A_T) return Columns::window(a_at, lda, K, kt, kt < kt1);
        else return RowsA::window(a_at, a_all, kt, kt < kt1);
    };
    auto b_win = [&](int kt) __attribute__((always_inline)) -> Win {
        const bool second = SEG && kt >= seg_kt;
        const int k = second ? kt - seg_kt : kt;
        const uint64_t p = second ? b_at[1] : b_at[0];
        if constexpr (B_N) return Columns::window(p, ldb, K, k, kt < kt1);
        else return RowsB::window(p, b_all, k, kt < kt1);
    };
    // bytes of a K-contiguous row's part of k-tile kt that exist
    auto lim_a = [&](int kt) __attribute__((always_inline)) -> int { return RowsA::limit(kt, seg_kt, tail); };
    auto lim_b = [&](int kt) __attribute__((always_inline)) -> int {
        int k = kt;
        if constexpr (SEG) k = kt >= seg_kt ? kt - seg_kt : kt;
        return RowsB::limit(k, seg_kt, tail);
    };

    // ---- per-lane copy offsets: op j writes 1 KiB of the slot, lane i 16 bytes at 16 i ----
    // K-contiguous: op d holds rows 8d .. 8d+7; the swizzle of a row differs between even
    // and odd d only, so two offsets and a multiple of 16 rows give every op's.  Kept in
    // two registers instead of one per op: with 128 accumulators and two fragment sets the
    // large tiles have about 30 left.  pos: the chunk's first byte within the k-tile (for
    // the mask of the last one).
    const int kc_lo = (lane & 7) ^ (lane >> 4);       // chunk of this lane in an even op
    auto kc_pos = [&](int d) { return (kc_lo ^ ((d & 1) * 4)) * 16; };
    uint32_t kcA[2], kcB[2];                          // K-contiguous: offset of op `first` + 0, 1
    const int firstA = wave * A_OPS;
    int firstB = wave * B_OPS;
    if (DUAL && firstB >= BNS / 8) firstB -= BNS / 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        kcA[h] = (uint32_t)((firstA + h) * 8 + lane / 8) * args.lda + (uint32_t)kc_pos(firstA + h) + RowsA::kBack;
        kcB[h] = (uint32_t)((firstB + h) * 8 + lane / 8) * args.ldb + (uint32_t)kc_pos(firstB + h) + RowsB::kBack;
    }
    const int posA = kc_pos(firstA), posB = kc_pos(firstB);
    // gathered: every op's own row; kMasked - 15 and above lie past the resource, too
    uint32_t gaA[GATHER ? A_OPS : 1];
    if constexpr (GATHER) {
#pragma unroll
        for (int j = 0; j < A_OPS; ++j) {
            const int r = m0 + (firstA + j) * 8 + lane / 8;
            const int row = r < M ? from.index[r] : -1;
            gaA[j] = row >= 0 && row < from.rows ? (uint32_t)row * args.lda + (uint32_t)kc_pos(firstA + j) + RowsA::kBack : kMasked;
        }
    }
    // reduction-major: op d holds 64 / CPR rows; over: columns of the chunk past the last
    uint32_t trA[A_T ? A_OPS : 1], trB[B_N ? B_OPS : 1];
    int overA[A_T ? A_OPS : 1], overB[B_N ? B_OPS : 1];
    auto tr_off = [&](auto cpr_c, int d, int col0, int64_t ld, int cols, uint32_t& off, int& over)
                      __attribute__((always_inline)) {
        constexpr int CPR = decltype(cpr_c)::value, RP = 64 / CPR;
        const int r = d * RP + lane / CPR, c = (lane % CPR) ^ nswz_t<CPR>(r);
        over = Columns::over(col0 + c * 8, cols);
        off = Columns::offset(r, (uint32_t)ld, col0 + c * 8, over);
    };
    if constexpr (A_T) {
#pragma unroll
        for (int j = 0; j < A_OPS; ++j)
            tr_off(std::integral_constant<int, BM / 8>{}, firstA + j, m0, args.lda, args.a_cols, trA[j], overA[j]);
    }
    if constexpr (B_N) {
#pragma unroll
        for (int j = 0; j < B_OPS; ++j)
            tr_off(std::integral_constant<int, BNS / 8>{}, firstB + j, n0, args.ldb, args.b_cols, trB[j], overB[j]);
    }
    // offset of op j for a k-tile of which `lim` bytes exist along a K-contiguous row
    auto src_off = [&](auto jc, int lim) __attribute__((always_inline)) -> uint32_t {
        constexpr int j = decltype(jc)::value;
        if constexpr (j < A_OPS) {
            if constexpr (A_T) return trA[j];
            else if constexpr (GATHER) return RowsA::offset(gaA[j], posA ^ ((j & 1) * 64), lim);
            else return RowsA::offset(kcA[j & 1] + (uint32_t)(j >> 1) * 16u * args.lda, posA ^ ((j & 1) * 64), lim);
        } else {
            constexpr int i = j - A_OPS;
            if constexpr (B_N) return trB[i];
            else return RowsB::offset(kcB[i & 1] + (uint32_t)(i >> 1) * 16u * args.ldb, posB ^ ((i & 1) * 64), lim);
        }
    };
    // REG: bits to shift the loaded chunk down by
    auto src_shift = [&](auto jc, int lim) __attribute__((always_inline)) -> uint32_t {
        constexpr int j = decltype(jc)::value;
        if constexpr (j < A_OPS) {
            if constexpr (A_T) return Columns::shift(overA[j]);
            else return RowsA::shift(posA ^ ((j & 1) * 64), lim);
        } else {
            constexpr int i = j - A_OPS;
            if constexpr (B_N) return Columns::shift(overB[i]);
            else return RowsB::shift(posB ^ ((i & 1) * 64), lim);
        }
    };
    auto lds_dst = [&](const Slot& s, auto jc) __attribute__((always_inline)) -> SPG_LDS char* {
        constexpr int j = decltype(jc)::value;
        if constexpr (j < A_OPS) return s.a + (wave * A_OPS + j) * 1024;
        else return s.b + (wave * B_OPS + (j - A_OPS)) * 1024;
    };
    struct Src { i32x4 a, b; int lim_a, lim_b; };
    auto src_ab = [&](int kta, int ktb) __attribute__((always_inline)) -> Src {
        const Win a = a_win(kta), b = b_win(ktb);
        return Src{make_rsrc((const void*)(uintptr_t)a.p, a.n), make_rsrc((const void*)(uintptr_t)b.p, b.n),
                   lim_a(kta), lim_b(ktb)};
    };
    auto dma_op = [&](const Slot& s, const Src& src, auto jc) __attribute__((always_inline)) {
        constexpr bool ISA = decltype(jc)::value < A_OPS;
        dma16(ISA ? src.a : src.b, lds_dst(s, jc), src_off(jc, ISA ? src.lim_a : src.lim_b));
    };
    // A K-contiguous row's last chunk of a segment that ends inside it (dG and dU end in zeros): what follows K there
    // is the next row's and is cleared in LDS, by the lane that copied it, once this wave's
    // copies of the k-tile have landed and before the barrier that publishes it.
    auto clear_tail = [&](const Slot& s, int kt) __attribute__((always_inline)) {
        if constexpr (TAIL && !REG && ((!A_T && !SEG) || !B_N)) {
            const int lim = lim_b(kt);
            if ((lim & 15) == 0) return;
            // loops, not unrolled: the code stands behind every k-tile of the unrolled pattern
            auto clear = [&](SPG_LDS char* at, int ops, int pos) __attribute__((always_inline)) {
#pragma unroll 1
                for (int j = 0; j < ops; ++j) {
                    if ((pos ^ ((j & 1) * 64)) == (lim & ~15)) {
                        SPG_LDS u32x4* p = (SPG_LDS u32x4*)(at + j * 1024 + lane * 16);
                        *p = clear_top(*p, 8u * (uint32_t)(16 - (lim & 15)));
                    }
                }
            };
            if constexpr (!A_T && !SEG) clear(s.a + firstA * 1024, A_OPS, posA);
            if constexpr (!B_N) clear(s.b + wave * B_OPS * 1024, B_OPS, posB);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
    };
    auto issue = [&](const Slot& s, int kt) __attribute__((always_inline)) {
        const Src src = src_ab(kt, kt);
        static_for<0, L>([&](auto jc) { dma_op(s, src, jc); });
    };
    auto poison_slot = [&](const Slot& s) __attribute__((always_inline)) {
        if constexpr (kPoison) {
            static_for<0, L>([&](auto jc) {
                *(SPG_LDS u32x4*)(lds_dst(s, jc) + lane * 16) = u32x4{~0u, ~0u, ~0u, ~0u};
            });
            if constexpr (!REG) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
    };
    // register staging: PD k-tiles of loads in flight (a k-tile of a small tile is multiplied
    // in a fraction of the memory's latency)
    constexpr int PD = L >= 6 ? 2 : 4;
    u32x4 staged[REG ? PD : 1][REG ? L : 1];
    auto gload = [&](auto pc, int kt) __attribute__((always_inline)) {
        constexpr int p = decltype(pc)::value % PD;
        const Win a = a_win(kt), b = b_win(kt);
        const auto ra = make_rsrc_b((const void*)(uintptr_t)a.p, a.n), rb = make_rsrc_b((const void*)(uintptr_t)b.p, b.n);
        const int lb = lim_b(kt), la = SEG ? lim_a(kt) : lb;
        static_for<0, L>([&](auto jc) {
            constexpr int j = decltype(jc)::value;
            staged[p][j] = __builtin_amdgcn_raw_buffer_load_b128(j < A_OPS ? ra : rb, (int)src_off(jc, j < A_OPS ? la : lb), 0, 0);
        });
    };
    // columns past the last reach into this workgroup's tile
    const bool cut = (A_T && m0 + BM > args.a_cols) || (B_N && n0 + BNS > args.b_cols);
    auto lwrite = [&](const Slot& s, auto pc, int kt) __attribute__((always_inline)) {
        constexpr int p = decltype(pc)::value % PD;
        const int lb = lim_b(kt), la = SEG ? lim_a(kt) : lb;
        // only the last k-tile and the last column tile have chunks to realign: a 128-bit
        // shift by a lane's own amount is about 20 instructions, and doing it for every
        // chunk took longer than the multiplications of the small tiles
        auto put = [&](auto jc, const u32x4& v) __attribute__((always_inline)) { *(SPG_LDS u32x4*)(lds_dst(s, jc) + lane * 16) = v; };
        // realigned where they are staged, so that every chunk is stored as it comes in: with stores of
        // their own on both ways the compiler waits for all of them first (300 x 2731 x 1001, gated:
        // 12.6 us, 12.3 so).  Not for rows by group (1620 in 64 groups, 10560 columns of 49, gated: 119 us
        // so, 94 with both ways): of short reductions the k-tile that is realigned is all there is
        if constexpr (!SKIP) {
            if (lb != 128 || cut)
                static_for<0, L>([&](auto jc) {
                    constexpr int j = decltype(jc)::value;
                    staged[p][j] = shr128(staged[p][j], src_shift(jc, j < A_OPS ? la : lb));
                });
            static_for<0, L>([&](auto jc) { put(jc, staged[p][decltype(jc)::value]); });
            return;
        }
        if (lb == 128 && !cut) {
            static_for<0, L>([&](auto jc) { put(jc, staged[p][decltype(jc)::value]); });
            return;
        }
        static_for<0, L>([&](auto jc) {
            constexpr int j = decltype(jc)::value;
            put(jc, shr128(staged[p][j], src_shift(jc, j < A_OPS ? la : lb)));
        });
    };

    // ---- fragment reads ----
    // K-contiguous: lane l reads row l%16, chunk 4kk + l/16.  Reduction-major: the
    // transposing read, lane i of a 16-lane group supplies 8 bytes of row k0 + i/4 and gets
    // column i of rows k0 .. k0+3; two reads make the lane's 8 elements.
    int aoff[A_T ? TM : 2], boff[B_N ? TN : 2];
    auto frag_k = [&](int row0, int kk) { return (row0 + (lane & 15)) * 128 + (((kk * 4 + (lane >> 4)) ^ kswz(lane & 15)) * 16); };
    auto frag_n = [&](auto cpr_c, int col0) {
        constexpr int CPR = decltype(cpr_c)::value;
        const int kl = (lane >> 4) * 8 + ((lane & 15) >> 2);
        const int chunk = col0 / 8 + ((lane >> 1) & 1);
        return kl * CPR * 16 + (chunk ^ nswz_t<CPR>(kl)) * 16 + (lane & 1) * 8;
    };
    // column (within its B subtile) of a wave's fragment bn
    auto bcol = [&](int bn) { return wn * WNS + (DUAL && bn >= TN / 2 ? bn - TN / 2 : bn) * 16; };
    if constexpr (A_T) {
#pragma unroll
        for (int bm = 0; bm < TM; ++bm) aoff[bm] = frag_n(std::integral_constant<int, BM / 8>{}, wm * WM + bm * 16);
    } else {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) aoff[kk] = frag_k(wm * WM, kk);
    }
    if constexpr (B_N) {
#pragma unroll
        for (int bn = 0; bn < TN; ++bn)
            boff[bn] = frag_n(std::integral_constant<int, BNS / 8>{}, bcol(bn)) + (DUAL && bn >= TN / 2 ? BNS * 128 : 0);
    } else {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) boff[kk] = frag_k(wn * WNS, kk);
    }
    struct Frags { u32x4 a[TM]; u32x4 b[TN]; };
    const bool idle = SKIP && m0 + wm * WM >= M;
    constexpr int RA = A_T ? 2 * TM : TM, RB = B_N ? 2 * TN : TN, NRD = RA + RB;
    auto tr_read = [&](SPG_LDS char* p, u32x4& f, auto hc) __attribute__((always_inline)) {
        constexpr int h = decltype(hc)::value;
        const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((SPG_LDS shortx4*)p));
        f[2 * h] = v[0];
        f[2 * h + 1] = v[1];
    };
    auto read_op = [&](const Slot& s, int kk, Frags& f, auto rc) __attribute__((always_inline)) {
        constexpr int r = decltype(rc)::value;
        if constexpr (r < RA) {
            if constexpr (A_T) {
                constexpr int bm = r / 2, h = r % 2;
                tr_read(s.a + aoff[bm] + (kk * 32 + h * 4) * (BM * 2), f.a[bm], std::integral_constant<int, h>{});
            } else {
                f.a[r] = *(const SPG_LDS u32x4*)(s.a + aoff[kk] + r * 16 * 128);
            }
        } else if constexpr (B_N) {
            constexpr int bn = (r - RA) / 2, h = (r - RA) % 2;
            tr_read(s.b + boff[bn] + (kk * 32 + h * 4) * (BNS * 2), f.b[bn], std::integral_constant<int, h>{});
        } else {
            constexpr int bn = r - RA;
            constexpr int row = DUAL && bn >= TN / 2 ? BNS + (bn - TN / 2) * 16 : bn * 16;
            f.b[bn] = *(const SPG_LDS u32x4*)(s.b + boff[kk] + row * 128);
        }
    };

    AccOf<ET> acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = 0;

    // One k-step: the MFMAs of `now`, with the reads of the next step and (COPY) the copies
    // of a k-tile spread among them; the compiler places them, asked to interleave the LDS
    // reads with the MFMAs (as in the two-round configurations of pipelined_gemm).
    constexpr int NMMA = TN * TM;
    auto stage = [&](const Frags& now, const Slot& rslot, int rkk, Frags& nx, const Slot& cslot, const Src& src,
                     auto copy) __attribute__((always_inline)) {
        __builtin_amdgcn_iglp_opt(2);
        constexpr bool COPY = decltype(copy)::value;
        constexpr int NCP = COPY ? L : 0;
        constexpr int CSP = COPY && NMMA >= 2 * NCP ? 2 : 1;
        constexpr int NRS = (NRD + 1) / 2;
        constexpr int STEPS = NMMA > NRS ? (NMMA > NCP ? NMMA : NCP) : (NRS > NCP ? NRS : NCP);
        static_for<0, STEPS>([&](auto ic) {
            constexpr int i = decltype(ic)::value;
            if constexpr (i < NMMA) {
                constexpr int bn = i / TM, bm = i % TM;
                acc[bn][bm] = mma<ET>(now.b[bn], now.a[bm], acc[bn][bm]);
            }
            if constexpr (COPY && i % CSP == 0 && i / CSP < NCP) dma_op(cslot, src, std::integral_constant<int, i / CSP>{});
            static_for<0, 2>([&](auto rc) {
                constexpr int r = 2 * i + decltype(rc)::value;
                if constexpr (r < NRD) read_op(rslot, rkk, nx, std::integral_constant<int, r>{});
            });
        });
    };

    using C0 = std::integral_constant<int, 0>;
    using C1 = std::integral_constant<int, 1>;
    using C2 = std::integral_constant<int, 2>;
    if constexpr (REG) {
        static_for<0, PD>([&](auto pc) { gload(pc, kt_of(decltype(pc)::value)); });
        lwrite(slot_of(C0{}), C0{}, kt_of(0));
        gload(C0{}, kt_of(PD));
    } else if constexpr (DEEP) {
        issue(slot_of(C0{}), kt0);
        issue(slot_of(C1{}), kt0 + 1);
        const Src src = src_ab(kt0 + 2, kt0 + 2);
        static_for<A_OPS, L>([&](auto jc) { dma_op(slot_of(C2{}), src, jc); });
        wait_vmcnt<L + B_OPS>();
        clear_tail(slot_of(C0{}), kt0);
    } else {
        static_for<0, S>([&](auto sc) { issue(slot_of(sc), kt_of(decltype(sc)::value)); });
        wait_vmcnt<(S - 1) * L>();
        clear_tail(slot_of(C0{}), kt_of(0));
    }
    lds_barrier();
    auto over_ktiles = [&](auto&& ktile) __attribute__((always_inline)) {
        int t = 0;
        for (; t + NS <= nk; t += NS) static_for<0, NS>([&](auto sc) { ktile(sc, t + decltype(sc)::value); });
        const int rem = nk - t;
        static_for<0, NS - 1>([&](auto sc) {
            if (decltype(sc)::value < rem) ktile(sc, t + decltype(sc)::value);
        });
    };
    if constexpr (DEEP) {
        // The large tile runs the ping-pong schedule of pipelined_gemm (schedule 2 there): the
        // two waves of a SIMD (w and w + 4) take turns, one issuing a k-step's MFMAs while
        // the other reads the next fragments and copies, a workgroup barrier between turns.
        // Group 1 runs one phase behind group 0.  K-tile u is read in phases 4u .. 4u+3; its
        // slots are refilled (A of u+2, B of u+3) in the first memory phase of k-tile u+1;
        // before the barrier that opens k-tile u+1's first read every wave has waited for
        // its copies of A(u+1) and B(u+1), leaving B(u+2) in flight.  One fragment set is
        // enough, which leaves the registers that the masks and addresses need: with two
        // sets (the schedule of the smaller tiles) this tile spills up to 60 registers.
        static_assert(!DEEP || NW == 8, "two groups of four waves");
        const int grp = wave >> 2;
        auto phase_barrier = []() __attribute__((always_inline)) {
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        };
        Frags f;
        auto matrix_phase = [&]() __attribute__((always_inline)) {
            if (SKIP && idle) return;
            static_for<0, NMMA>([&](auto ic) {
                constexpr int i = decltype(ic)::value, bn = i / TM, bm = i % TM;
                acc[bn][bm] = mma<ET>(f.b[bn], f.a[bm], acc[bn][bm]);
            });
        };
        if (grp == 1) phase_barrier();
        over_ktiles([&](auto sc, int u) __attribute__((always_inline)) {
            constexpr int i = decltype(sc)::value;
            const Slot cur = slot_of(sc);
            const Slot prev = slot_of(std::integral_constant<int, i + 5>{});
            if (!SKIP || !idle) static_for<0, NRD>([&](auto rc) { read_op(cur, 0, f, rc); });
            if (u >= 1) {
                poison_slot(prev);
                const Src src = src_ab(kt0 + u + 1, kt0 + u + 2);
                static_for<0, L>([&](auto jc) { dma_op(prev, src, jc); });
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            phase_barrier();
            matrix_phase();
            phase_barrier();
            if (!SKIP || !idle) static_for<0, NRD>([&](auto rc) { read_op(cur, 1, f, rc); });
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            const Slot nxt = slot_of(std::integral_constant<int, i + 1>{});
            if (grp == 1) {
                wait_vmcnt<B_OPS>();
                clear_tail(nxt, kt0 + u + 1);
            }
            phase_barrier();
            matrix_phase();
            if (grp == 0) {
                wait_vmcnt<B_OPS>();
                clear_tail(nxt, kt0 + u + 1);
            }
            phase_barrier();
        });
        if (grp == 0) phase_barrier();
    } else {
        Frags fr[2];
        if (!SKIP || !idle) static_for<0, NRD>([&](auto rc) { read_op(slot_of(C0{}), 0, fr[0], rc); });
        const Src none{};
        over_ktiles([&](auto sc, int t) __attribute__((always_inline)) {
            constexpr int s = decltype(sc)::value;
            using Next = std::integral_constant<int, s + 1>;
            const Slot cur = slot_of(sc);
            const Slot nxt = slot_of(Next{});
            if constexpr (REG) {
                // nxt was released by the previous barrier; its writes go first, so that they
                // drain behind the MFMAs of this stage
                poison_slot(nxt);
                lwrite(nxt, Next{}, kt_of(t + 1));
                gload(Next{}, kt_of(t + 1 + PD));
            }
            if (!SKIP || !idle) stage(fr[0], cur, 1, fr[1], cur, none, std::false_type{});
            if constexpr (!REG) {
                wait_vmcnt<(S - 2) * L>();
                clear_tail(nxt, kt_of(t + 1));
            }
            __builtin_amdgcn_sched_barrier(0);
            lds_barrier();
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_setprio(1);
            if constexpr (REG) {
                if (!SKIP || !idle) stage(fr[1], nxt, 0, fr[0], cur, none, std::false_type{});
            } else {
                poison_slot(cur);
                const Src src = src_ab(kt_of(t + S), kt_of(t + S));
                if (!SKIP || !idle) stage(fr[1], nxt, 0, fr[0], cur, src, std::true_type{});
                else static_for<0, L>([&](auto jc) { dma_op(cur, src, jc); });
            }
            __builtin_amdgcn_s_setprio(0);
        });
    }

    // ---- the groups' sums meet, added in group order ----
    if constexpr (KG > 1) {
        wait_vmcnt<0>();
        __syncthreads();
        SPG_LDS AccOf<ET>* sums = (SPG_LDS AccOf<ET>*)lds;
        if (kg > 0) {
#pragma unroll
            for (int i = 0; i < TN * TM; ++i)
                sums[(((kg - 1) * NW + wave) * TN * TM + i) * 64 + lane] = acc[i / TM][i % TM];
        }
        __syncthreads();
        if (kg > 0) return;
#pragma unroll
        for (int g = 1; g < KG; ++g)
#pragma unroll
            for (int i = 0; i < TN * TM; ++i)
                acc[i / TM][i % TM] += sums[(((g - 1) * NW + wave) * TN * TM + i) * 64 + lane];
    }

    // ---- epilogue ----
    const int m_base = m0 + wm * WM, n_base = n0 + wn * WNS;
    if constexpr (LOCAL) {
        if (args.part) {
            float* to = args.part + (size_t)wave * TN * TM * 256 + lane * 4;
            if (!(SKIP && idle))
#pragma unroll
                for (int i = 0; i < TN * TM; ++i) *(AccOf<ET>*)(to + i * 256) = acc[i / TM][i % TM];
            wait_vmcnt<0>();   // as below
            return;
        }
    } else if (args.part) {
        // a part of the sum: raw accumulators, row-major, 16 bytes per lane
        const int np4 = (N + 3) & ~3;
        const int zrow = args.zm == 2 ? z * M : 0, zcol = args.zn == 2 ? z * np4 : 0;
        const int64_t ldp = part_pitch(args, DUAL);
        float* base = args.part + ((size_t)sp * M * args.zm + zrow) * ldp + zcol;
#pragma unroll
        for (int bm = 0; bm < TM; ++bm) {
            const int m = m_base + bm * 16 + (lane & 15);
#pragma unroll
            for (int bn = 0; bn < TN; ++bn) {
                const bool second = DUAL && bn >= TN / 2;
                const int n = n_base + (second ? bn - TN / 2 : bn) * 16 + 4 * (lane >> 4);
                if (m < M && n < N)
                    *(AccOf<ET>*)(base + (size_t)m * ldp + (second ? np4 : 0) + n) = acc[bn][bm];
            }
        }
        wait_vmcnt<0>();   // the zero-fill copies past the last k-tile land before the LDS is given up
        return;
    }
    if constexpr (KG == 1) {
        wait_vmcnt<0>();
        __syncthreads();
    }
    SPG_LDS char* stg = lds + G::SUMS + wave * G::STG;
    if constexpr (ET == kElI8) {
        float rs[TM];
#pragma unroll
        for (int bm = 0; bm < TM; ++bm) {
            const int m = m_base + bm * 16 + (lane & 15);
            rs[bm] = args.sa[m < M ? m : M - 1];
        }
        float cs[TN][4];
#pragma unroll
        for (int bn = 0; bn < TN; ++bn) {
            const bool second = DUAL && bn >= TN / 2;
            const float* sb = args.sb[second ? 1 : 0];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int n = n_base + (second ? bn - TN / 2 : bn) * 16 + 4 * (lane >> 4) + e;
                cs[bn][e] = sb[n < N ? n : N - 1];
            }
        }
        auto scaled = [&](int bn, int bm, int e) __attribute__((always_inline)) {
            // in this order: the product of two small scales may leave fp32's range where the result does not
            return (float)acc[bn][bm][e] * rs[bm] * cs[bn][e];
        };
        with_out(args.out_dtype, [&](auto od) __attribute__((always_inline)) {
            constexpr int OD = decltype(od)::value;
            if constexpr (DUAL)
                with_act(args.act, [&](auto ac) __attribute__((always_inline)) {
                    store_block<OD, TM, TN / 2, WNS>(
                        [&](int bn, int bm, int e) __attribute__((always_inline)) {
                            return act_t<decltype(ac)::value>(scaled(bn, bm, e)) * scaled(bn + TN / 2, bm, e);
                        }, stg, args.C, M, N, m_base, n_base, lane);
                });
            else
                store_block<OD, TM, TN, WNS>(scaled, stg, args.C, M, N, m_base, n_base, lane);
        });
    } else {
        constexpr int OD = ET == kElBF16 ? kOutBF16 : kOutF16;
        if constexpr (DUAL) {
            if (args.G) {
                store_block<OD, TM, TN / 2, WNS>([&](int bn, int bm, int e) __attribute__((always_inline)) { return acc[bn][bm][e]; },
                                                 stg, args.G, M, N, m_base, n_base, lane);
                store_block<OD, TM, TN / 2, WNS>([&](int bn, int bm, int e) __attribute__((always_inline)) { return acc[bn + TN / 2][bm][e]; },
                                                 stg, args.U, M, N, m_base, n_base, lane);
            }
            with_act(args.act, [&](auto ac) __attribute__((always_inline)) {
                store_block<OD, TM, TN / 2, WNS>(
                    [&](int bn, int bm, int e) __attribute__((always_inline)) {
                        return act_t<decltype(ac)::value>(acc[bn][bm][e]) * acc[bn + TN / 2][bm][e];
                    }, stg, args.C, M, N, m_base, n_base, lane);
            });
        } else {
            store_block<OD, TM, TN, WNS>([&](int bn, int bm, int e) __attribute__((always_inline)) { return acc[bn][bm][e]; },
                                         stg, A_T && z ? args.C1 : args.C, M, N, m_base, n_base, lane);
        }
    }
}

template <int ET, bool A_T, bool B_N, bool DUAL, bool SEG, bool REG, int BM, int BN, int WM, int WN,
          int S, bool DEEP, int KG, bool TAIL, int WPS>
__global__ void __launch_bounds__((ProductGeom<DUAL, BM, BN, WM, WN, S, DEEP, KG>::NT), WPS)
product_kernel(ProductArgs args) {
    __shared__ __attribute__((aligned(1024))) char lds[ProductGeom<DUAL, BM, BN, WM, WN, S, DEEP, KG>::LDS];
    int tm, tn, sp;
    product_tile(blockIdx.x, args, tm, tn, sp);
    product_tile_of<ET, A_T, B_N, DUAL, SEG, REG, BM, BN, WM, WN, S, DEEP, KG, TAIL>(args, tm, tn, sp, (SPG_LDS char*)lds);
}

// The input gradient and the weights' gradients of a small training step in one launch:
// workgroups 0 .. nx-1 the tiles of dX, the rest those of dWg and dWu.  Neither fills the
// device, and each launch has its own start, last store and gap (about 4 us of 11).
template <int ET, bool NK, bool REG, int BM, int BN, int WM, int WN, int S, int KG>
__global__ void __launch_bounds__((ProductGeom<false, BM, BN, WM, WN, S, false, KG>::NT))
gradients_kernel(ProductArgs x, ProductArgs w, int nx) {
    __shared__ __attribute__((aligned(1024))) char lds[ProductGeom<false, BM, BN, WM, WN, S, false, KG>::LDS];
    const int wg = blockIdx.x;
    int tm, tn, sp;
    if (wg < nx) {
        product_tile(wg, x, tm, tn, sp);
        product_tile_of<ET, false, NK, false, true, REG, BM, BN, WM, WN, S, false, KG, true>(x, tm, tn, sp, (SPG_LDS char*)lds);
    } else {
        product_tile(wg - nx, w, tm, tn, sp);
        product_tile_of<ET, true, true, false, false, REG, BM, BN, WM, WN, S, false, KG, true>(w, tm, tn, sp, (SPG_LDS char*)lds);
    }
}

// ---------------------------------------------------------------------------
// up to 16 rows: the weights stream through registers
// ---------------------------------------------------------------------------
//
// For M <= 16 and K-contiguous weights the product is the reading of the weights: every
// weight is used once, so nothing is gained by LDS tiles.  A workgroup takes 16 columns of
// each B matrix; its NW waves share K (wave w the chunks w, w + NW, ... of U * 64 bytes a
// row), each lane loads its 16-byte MFMA operands straight from memory at any alignment
// (row l%16, bytes 16 (l/16) of every 64), and the waves' sums meet in LDS, added in wave
// order.  Each load touches 16 rows, half a cache line each: about 20 bytes a cycle and CU,
// twice what HBM delivers, so for more rows, whose X is loaded the same way by every
// workgroup, LDS tiles are faster (M = 64, N = 4096, K = 12288 int8: 28.5 us this way, 13
// with a tile).  Measured at M = 1, N = 12288, K = 4096 bf16, two weights: 38.3 us, 5.25
// TB/s; a second chunk in flight a wave 41.0, 16 waves 37.6 to 42.6, 4 waves 40.3,
// loads marked nontemporal 39.6 (int8, M = 4: 10.7 against 14.6).
//
// WORDS: all rows start on 4 bytes.  Otherwise (odd K in 16 bits, most K in 8) a lane loads
// the 16 bytes from the 4-byte word its chunk starts in, takes the word after them from the
// lane that holds the row's next 16 bytes, and shifts by its row's 1 to 3 bytes: loads that
// are not word-aligned run at half the rate (K = 4095 against 4094: 54.6 and 31.5 us, int8
// 20.4 and 8.3).  Only whole words that hold a byte of the operand are read.
template <int ET, bool DUAL, bool WORDS, int NW, int U>
__global__ void __launch_bounds__(NW * 64) stream_kernel(ProductArgs args) {
    constexpr int ES = ET == kElI8 ? 1 : 2;
    constexpr int NM = DUAL ? 2 : 1;
    __shared__ __attribute__((aligned(16))) AccOf<ET> sums[NW][NM][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int M = args.M, N = args.N;
    const int kb = args.K * ES;                       // bytes of a row
    const int n0 = blockIdx.x * 16;
    const int rows = N - n0 < 16 ? N - n0 : 16;
    const uint32_t ldb = args.ldb, lda = args.lda;
    // a matrix: its resource from the word its first row starts in, this lane's row from
    // there, and how many bytes past a word the row starts
    struct Rows {
        __amdgpu_buffer_rsrc_t r;
        uint32_t row, shift;
    };
    auto rows_of = [&](const char* p, uint32_t ld, int n) __attribute__((always_inline)) -> Rows {
        const uint32_t skip = WORDS ? 0u : (uint32_t)(uintptr_t)p & 3u;
        const uint32_t bytes = skip + (uint32_t)(n - 1) * ld + (uint32_t)kb;
        const uint32_t at = skip + (uint32_t)(lane & 15) * ld;
        return Rows{make_rsrc_b(p - skip, WORDS ? bytes : (bytes + 3u) & ~3u), WORDS ? at : at & ~3u, WORDS ? 0u : at & 3u};
    };
    const Rows x = rows_of(args.A, lda, M);
    const Rows b0 = rows_of(args.B[0] + (size_t)n0 * ldb, ldb, rows);
    const Rows b1 = rows_of((DUAL ? args.B[1] : args.B[0]) + (size_t)n0 * ldb, ldb, rows);
    const bool ragged = (kb & 15) != 0;

    AccOf<ET> acc[NM];
#pragma unroll
    for (int q = 0; q < NM; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[q][e] = 0;

    const int next = ((lane + 16) & 63) * 4;          // the lane with the row's next 16 bytes
    struct Chunks { u32x4 v[U]; uint32_t end; };
    for (int base = wave * (U * 64); base < kb; base += NW * U * 64) {
        auto load = [&](const Rows& m) __attribute__((always_inline)) -> Chunks {
            Chunks c;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = base + u * 64 + 16 * (lane >> 4);
                // WORDS: bytes past K read zero, the 16 that straddle it are the 16 ending at K.
                // Otherwise the words up to the one that holds the row's last byte are read:
                // the chunk before may need the first of these
                const uint32_t kw = (uint32_t)(WORDS && k + 16 > kb ? kb - 16 : k);
                const bool in = k < kb + (int)m.shift;
                c.v[u] = __builtin_amdgcn_raw_buffer_load_b128(m.r, (int)(in ? m.row + kw : kOOB), 0, 0);
            }
            // the word after the last chunk, for the lanes with the row's last 16 bytes of it
            if constexpr (!WORDS)
                c.end = __builtin_amdgcn_raw_buffer_load_b32(m.r, (int)(m.row + (uint32_t)(base + U * 64)), 0, 0);
            return c;
        };
        auto align = [&](const Rows& m, Chunks& c) __attribute__((always_inline)) {
            if constexpr (!WORDS) {
                const bool last = lane >= 48;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    // lanes 48 .. 63 need the first word of lanes 0 .. 15 one chunk further
                    const uint32_t here = (uint32_t)__builtin_amdgcn_ds_bpermute(next, (int)c.v[u].x);
                    const uint32_t further = u + 1 < U ? (uint32_t)__builtin_amdgcn_ds_bpermute(next, (int)c.v[u + 1 < U ? u + 1 : u].x) : c.end;
                    const uint32_t w[5] = {c.v[u].x, c.v[u].y, c.v[u].z, c.v[u].w, last ? further : here};
#pragma unroll
                    for (int e = 0; e < 4; ++e) c.v[u][e] = __builtin_amdgcn_alignbyte(w[e + 1], w[e], m.shift);
                }
            }
            if ((ragged || !WORDS) && base + U * 64 > kb) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int k = base + u * 64 + 16 * (lane >> 4);
                    if constexpr (WORDS) {
                        const uint32_t sh = k < kb && k + 16 > kb ? 8u * (uint32_t)(k + 16 - kb) : 0u;
                        c.v[u] = shr128(c.v[u], sh);
                    } else {
                        // what follows the row's end is the next row's
                        const int gone = k + 16 - kb;
                        const uint32_t sh = gone > 0 && gone < 16 ? 8u * (uint32_t)gone : 0u;
                        const u32x4 kept = clear_top(c.v[u], sh);
                        c.v[u] = gone >= 16 ? u32x4{} : kept;
                    }
                }
            }
        };
        Chunks cx = load(x), c0 = load(b0), c1;
        if constexpr (DUAL) c1 = load(b1);
        align(x, cx);
        align(b0, c0);
        if constexpr (DUAL) align(b1, c1);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            acc[0] = mma<ET>(c0.v[u], cx.v[u], acc[0]);
            if constexpr (DUAL) acc[NM - 1] = mma<ET>(c1.v[u], cx.v[u], acc[NM - 1]);
        }
    }
#pragma unroll
    for (int q = 0; q < NM; ++q) sums[wave][q][lane] = acc[q];
    __syncthreads();

    // output: 4 consecutive columns of one row a lane of the first wave
    if (wave > 0) return;
    const int m = lane & 15, n = n0 + 4 * (lane >> 4);
    if (m >= M || n >= N) return;
    AccOf<ET> s[NM];
#pragma unroll
    for (int q = 0; q < NM; ++q) {
        s[q] = sums[0][q][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) s[q] += sums[w][q][lane];
    }
    finish4<ET, DUAL>(s[0], s[NM - 1], m, n, N - n < 4 ? N - n : 4, (size_t)m * N + n, args);
}

// ---------------------------------------------------------------------------
// operands laid out again
// ---------------------------------------------------------------------------
//
// Rows that do not start on 16 bytes, copied to rows that start on 128, zero past their end:
// for large products the copy costs less than register-staged tiles lose.  One launch for
// the matrices of a product; a thread moves 16 bytes.
struct PackArgs {
    const char* src[3];
    char* dst[3];
    int64_t chunks[3];    // 16-byte chunks of each destination (0: none)
    int64_t row[3];       // bytes of a source row
    int32_t per[3];       // chunks of a destination row
};

template <int ES>
__global__ void __launch_bounds__(256) pack_rows(PackArgs a) {
    int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    int q = 0;
    while (q < 3 && i >= a.chunks[q]) i -= a.chunks[q++];
    if (q == 3) return;
    const int64_t r = i / a.per[q];
    const int64_t c = (i - r * a.per[q]) * 16, left = a.row[q] - c;
    const char* s = a.src[q] + r * a.row[q] + c;
    u32x4 v = {};
    if (left >= 16) {
        struct __attribute__((packed, aligned(ES))) B { u32x4 v; };
        v = ((const B*)s)->v;
    } else {
#pragma unroll
        for (int e = 0; e < 16; e += ES)
            if (e < left) {
                const uint32_t x = ES == 1 ? *(const uint8_t*)(s + e) : *(const uint16_t*)(s + e);
                v[e >> 2] |= x << ((e & 3) * 8);
            }
    }
    *(u32x4*)(a.dst[q] + i * 16) = v;
}

// ---------------------------------------------------------------------------
// the sum over the parts of a split reduction
// ---------------------------------------------------------------------------
//
// Part sums are row-major [split][zm M][ldp]; a thread adds 4 consecutive columns over every
// W-th part, and the W waves' sums meet in LDS, in an order that does not depend on timing;
// then the epilogue.  Bound by the loads' latency, other XCDs having written the parts: eight
// are in flight, and with more parts than that four waves share them.
template <int ET, bool DUAL, int W>
__global__ void __launch_bounds__(256) sum_parts(ProductArgs args) {
    const int np4 = (args.N + 3) & ~3;
    const int quads = np4 / 4 * args.zn;
    const int64_t rows = (int64_t)args.M * args.zm;
    const int lane = W == 1 ? threadIdx.x : threadIdx.x & 63;
    const int first = W == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t i = (int64_t)blockIdx.x * (256 / W) + lane;
    const bool in = i < rows * quads;
    int64_t m = in ? i / quads : 0;
    int n = in ? (int)(i - m * quads) * 4 : 0;
    const int64_t ldp = part_pitch(args, DUAL);
    const size_t step = (size_t)rows * ldp / 4;
    const AccOf<ET>* p = (const AccOf<ET>*)(args.part + (size_t)m * ldp + n);
    AccOf<ET> s0 = p[first * step], s1 = s0;
    if constexpr (DUAL) s1 = p[first * step + np4 / 4];
    for (int k = first + W; k < args.split; k += 8 * W) {
        AccOf<ET> v[8], w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int q = k + j * W < args.split ? k + j * W : k;
            v[j] = p[q * step];
            if constexpr (DUAL) w[j] = p[q * step + np4 / 4];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k + j * W < args.split) {
                s0 += v[j];
                if constexpr (DUAL) s1 += w[j];
            }
    }
    if constexpr (W > 1) {
        __shared__ AccOf<ET> sums[W - 1][DUAL ? 2 : 1][64];
        if (first > 0) {
            sums[first - 1][0][lane] = s0;
            if constexpr (DUAL) sums[first - 1][1][lane] = s1;
        }
        __syncthreads();
        if (first > 0) return;
#pragma unroll
        for (int w = 0; w < W - 1; ++w) {
            s0 += sums[w][0][lane];
            if constexpr (DUAL) s1 += sums[w][1][lane];
        }
    }
    if (!in) return;
    int z = 0;
    if (m >= args.M) { m -= args.M; z = 1; }
    if (n >= np4) { n -= np4; z = 1; }
    const int left = args.N - n < 4 ? args.N - n : 4;
    if (left <= 0) return;
    finish4<ET, DUAL>(s0, s1, (int)m, n, left, (size_t)m * args.N + n, args, z);
}

// ---------------------------------------------------------------------------
// sizes the MFMA kernels do not take (a reduction shorter than one 16-byte chunk, rows
// beyond 32-bit offsets): one thread per output, any strides
// ---------------------------------------------------------------------------
struct SimpleArgs {
    ProductArgs p;
    int64_t sam, sak, sbn, sbk;   // element strides
    int64_t seg_a;                // elements from one segment of A to the next
};

template <int ET, bool DUAL>
__global__ void __launch_bounds__(256) simple_product(SimpleArgs a) {
    const ProductArgs& args = a.p;
    const int64_t total = (int64_t)args.M * args.N;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / args.N, n = i - m * args.N;
        using V = std::conditional_t<ET == kElI8, int32_t, float>;
        V s0 = 0, s1 = 0;
        auto at = [&](const char* p, int64_t j) -> V {
            if constexpr (ET == kElI8) return ((const int8_t*)p)[j];
            else return bits_to_f32(((const uint16_t*)p)[j], ET == kElBF16);
        };
        for (int seg = 0; seg < args.segments; ++seg)
            for (int64_t k = 0; k < args.K; ++k) {
                const V x = at(args.A, m * a.sam + k * a.sak + seg * a.seg_a);
                s0 += x * at(args.B[seg], n * a.sbn + k * a.sbk);
                if constexpr (DUAL) s1 += x * at(args.B[1], n * a.sbn + k * a.sbk);
            }
        AccOf<ET> v0, v1;
        for (int e = 0; e < 4; ++e) { v0[e] = s0; v1[e] = s1; }
        finish4<ET, DUAL>(v0, v1, (int)m, (int)n, 1, (size_t)i, args);
    }
}

// ---------------------------------------------------------------------------
// elementwise part of the backward pass
// ---------------------------------------------------------------------------
//
//   dU = dH act(G),  dG = dH U act'(G)     with s the sigmoid of z (silu: z = G, gelu: z =
//   2c(G + aG^3)): act = G s, act' = s + G s (1 - s) z'
//
// Written side by side in one [M, 2 np] matrix, np = N rounded up to a whole k-tile and the
// columns past N zero: rows are 128-byte aligned whatever N is, and both gradients of the
// weights and the one sum over both segments (dX) read it without masks.  dG and dU are
// rounded to the operands' type, as the products need them (a relative 2^-8 of each term
// in bf16 at most, 2^-11 in fp16, averaged down by the sums; the fp16 ones below 2^-14 lose
// bits and below 2^-25 vanish: the loss's scale has to keep them above).  Bound by memory: 3 reads, 2 writes of M N values.
//
// An infinite G or U is read as the largest finite value of its type: the forward pass made it
// of a finite sum when it rounded it for storage (fp16 ends at 65504), and zero slopes and zero
// dH times infinity would be NaN in a whole row of dX and a whole column of dWg or dWu.
template <bool BF16>
__device__ __forceinline__ void slopes_of(int64_t i, const uint16_t* dH, const uint16_t* G, const uint16_t* U,
                                          uint16_t* D, int M, int N, int np, int act) {
    const int per = np / 8;
    if (i >= (int64_t)M * per) return;
    const int64_t m = i / per;
    const int n = (int)(i - m * per) * 8;
    const size_t o = (size_t)m * N + n;
    u32x4 h = {}, g = {}, u = {};
    if (n + 8 <= N) {
        h = ((const Bytes16*)(dH + o))->v;
        g = ((const Bytes16*)(G + o))->v;
        u = ((const Bytes16*)(U + o))->v;
    } else if (n < N) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (n + e < N) {
                h[e >> 1] |= (uint32_t)dH[o + e] << ((e & 1) * 16);
                g[e >> 1] |= (uint32_t)G[o + e] << ((e & 1) * 16);
                u[e >> 1] |= (uint32_t)U[o + e] << ((e & 1) * 16);
            }
    }
    constexpr float kLargest = BF16 ? 0x1.fep127f : 65504.0f;
    auto finite = [](float v) {   // NaN stays NaN
        return __builtin_elementwise_minimum(__builtin_elementwise_maximum(v, -kLargest), kLargest);
    };
    u32x4 dg = {}, du = {};
    // the activation chosen once, not for every value: with the two limits above, 511 x 1365 took
    // 4.5 us with a branch a value, 4.3 so (and 4.3 without the limits, with the branches)
    with_act(act, [&](auto ac) {
        constexpr int ACT = decltype(ac)::value;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int sh = (e & 1) * 16;
            const float hv = bits_to_f32((uint16_t)(h[e >> 1] >> sh), BF16);
            const float gv = finite(bits_to_f32((uint16_t)(g[e >> 1] >> sh), BF16));
            const float uv = finite(bits_to_f32((uint16_t)(u[e >> 1] >> sh), BF16));
            float a, sl;
            if constexpr (ACT == kActRelu) {
                sl = gv <= 0.0f ? 0.0f : 1.0f;
                a = gv <= 0.0f ? 0.0f : gv;
            } else {
                float z = gv, dz = 1.0f;
                if constexpr (ACT == kActGelu) {
                    // past |G| = 1e15 s is 0 or 1 and its slope's zero must not meet an infinity
                    const float g2 = __builtin_fminf(gv * gv, 1e30f);
                    z = 1.5957691216f * gv * __builtin_fmaf(0.044715f, g2, 1.0f);
                    dz = 1.5957691216f * __builtin_fmaf(0.134145f, g2, 1.0f);
                }
                const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
                a = gv * s;
                sl = __builtin_fmaf(a * (1.0f - s), dz, s);
            }
            // dH U may pass fp32's range (bf16's is as wide) where the slope brings it back
            float d = hv * uv;
            d = BF16 && __builtin_fabsf(d) > 0x1.fffffep127f ? hv * sl * uv : d * sl;
            if (n + e < N) {
                dg[e >> 1] |= (uint32_t)f32_to_bits(d, BF16) << sh;
                du[e >> 1] |= (uint32_t)f32_to_bits(hv * a, BF16) << sh;
            }
        }
    });
    uint16_t* d = D + (size_t)m * 2 * np + n;
    *(u32x4*)d = dg;
    *(u32x4*)(d + np) = du;
}

template <bool BF16>
__global__ void __launch_bounds__(256) gated_slopes(const uint16_t* dH, const uint16_t* G, const uint16_t* U,
                                                    uint16_t* D, int M, int N, int np, int act) {
    slopes_of<BF16>((int64_t)blockIdx.x * 256 + threadIdx.x, dH, G, U, D, M, N, np, act);
}

// ---------------------------------------------------------------------------
// quantisation of rows
// ---------------------------------------------------------------------------
//
// amax = max |x|, scale = amax / 127, a = round to nearest even of 127 x / amax, exactly:
// the rounded fp32 product x (127 / amax) is off by less than 2^-15, so it can only end on
// the wrong side of a half next to one.  There the sign of 254 x - (2r+1) amax decides,
// computed without rounding from the two products' fp32 halves.  Rows whose amax is tiny
// or huge are scaled by a power of two first.  A row of zeros gives zeros and scale 0; a
// row with an infinity or a NaN gives zeros and that as the scale, so that its products
// come out NaN.
__device__ __forceinline__ int quantize1(float x, float inv, float amax) {
#pragma clang fp contract(off)
    const float q = x * inv;
    float r = __builtin_rintf(q);
    const float d = q - r;                            // exact; |d| <= 1/2
    if (__builtin_fabsf(d) > 0.4999f) {
        // the half between floor and floor + 1 of q
        const float lo = __builtin_floorf(q), t = 2.0f * lo + 1.0f;
        const float p = 254.0f * x, pe = __builtin_fmaf(254.0f, x, -p);
        const float c = t * amax, ce = __builtin_fmaf(t, amax, -c);
        const float s = (p - c) + (pe - ce);
        const float even = 2.0f * __builtin_rintf(0.5f * lo);   // the even one of lo and lo + 1 ...
        r = s > 0.0f ? lo + 1.0f : s < 0.0f ? lo : (even == lo ? lo : lo + 1.0f);
    }
    return (int)r;
}

template <int DT>
struct RowVec {
    static constexpr int E = DT == kOutF32 ? 4 : 8;
};

// W waves per row (a workgroup has four: one row or four), the row held in registers between
// the maximum and the rounding (V vectors of 16 bytes a thread); V = 0 reads it twice, for
// any K.
template <int DT, int V, int W>
__global__ void __launch_bounds__(256) quantize_rows(const char* X, int8_t* A, float* scale, int64_t K, int64_t rows) {
    constexpr int L = W * 64;
    const int tid = threadIdx.x & (L - 1);
    constexpr int E = RowVec<DT>::E, XB = DT == kOutF32 ? 4 : 2;
    const int64_t wg = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int64_t row = W == 1 ? wg * 4 + (threadIdx.x >> 6) : wg;
    if (row >= rows) return;                          // whole waves, with W = 4 whole workgroups
    const char* x = X + row * K * XB;
    int8_t* a = A + row * K;
    auto load = [&](int64_t v) -> u32x4 {
        const int64_t k = v * E;
        if (k + E <= K) return ((const Bytes16*)(x + k * XB))->v;
        u32x4 r = {};
        for (int e = 0; e < E; ++e)
            if (k + e < K) {
                if constexpr (XB == 4) r[e] = ((const uint32_t*)x)[k + e];
                else r[e >> 1] |= (uint32_t)((const uint16_t*)x)[k + e] << ((e & 1) * 16);
            }
        return r;
    };
    auto elem = [&](const u32x4& r, int e) -> float {
        if constexpr (XB == 4) { const uint32_t b = r[e]; return __builtin_bit_cast(float, b); }
        else return bits_to_f32((uint16_t)(r[e >> 1] >> ((e & 1) * 16)), DT == kOutBF16);
    };
    const int64_t nv = (K + E - 1) / E;
    u32x4 keep[V > 0 ? V : 1];
    // the largest magnitude as an integer: the order of non-negative floats is that of
    // their bits, with infinity and the NaNs above every finite value
    uint32_t top = 0;
    auto take = [&](const u32x4& r) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t b = __builtin_bit_cast(uint32_t, elem(r, e)) & 0x7fffffffu;
            top = b > top ? b : top;
        }
    };
    if constexpr (V > 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t v = tid + j * L;
            keep[j] = v < nv ? load(v) : u32x4{};
        }
#pragma unroll
        for (int j = 0; j < V; ++j) take(keep[j]);
    } else {
        for (int64_t v = tid; v < nv; v += L) take(load(v));
    }
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)top, s);
        top = o > top ? o : top;
    }
    if constexpr (W > 1) {
        __shared__ uint32_t wmax[W];
        if ((tid & 63) == 0) wmax[tid >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) top = wmax[w] > top ? wmax[w] : top;
    }
    float amax = __builtin_bit_cast(float, top);
    const bool finite = top < 0x7f800000u;
    if (tid == 0) scale[row] = amax / 127.0f;
    // amax near the ends of the range: scaled so that 127 / amax and 254 x stay inside it
    const float pow = amax < 0x1p-80f ? 0x1p80f : amax > 0x1p80f ? 0x1p-80f : 1.0f;
    amax *= pow;
    const float inv = finite && amax > 0.0f ? 127.0f / amax : 0.0f;
    auto put = [&](int64_t v, const u32x4& r) {
        const int64_t k = v * E;
        uint32_t b[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int q = inv != 0.0f ? quantize1(elem(r, e) * pow, inv, amax) : 0;
            b[e >> 2] |= (uint32_t)(q & 255) << ((e & 3) * 8);
        }
        if (k + E <= K) {
            struct __attribute__((packed, aligned(1))) B8 { u32x2 v; };
            struct __attribute__((packed, aligned(1))) B4 { uint32_t v; };
            if constexpr (E == 8) ((B8*)(a + k))->v = u32x2{b[0], b[1]};
            else ((B4*)(a + k))->v = b[0];
        } else {
            for (int e = 0; e < E; ++e)
                if (k + e < K) a[k + e] = (int8_t)(b[e >> 2] >> ((e & 3) * 8));
        }
    };
    if constexpr (V > 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t v = tid + j * L;
            if (v < nv) put(v, keep[j]);
        }
    } else {
        for (int64_t v = tid; v < nv; v += L) put(v, load(v));
    }
}

}  // namespace spg
