// Layer norm and its backward pass (gemm_norm_* in include/spgemm.h).
//
//   n = (x - mean) rstd,  y = n w + b
//   g = dy w,  dx = rstd (g - sum g / K - n sum(g n) / K),  dw = sum_rows dy n,  db = sum_rows dy
//
// The mean is taken off before the squares are summed: the variance of a row far from zero
// keeps its bits, which sum x^2 - mean^2 would lose.
//
// Rows of very large finite values (a deviation of 2^64, a sum of 2^128; not in fp16) take these sums
// past fp32's range.  Their variance shows it, and they are taken once more as x / 2^80.  As a branch
// of its own that costs the other rows one comparison (forward, 8192 x 4096: 27.5 us, 27.3 without;
// 16384 x 1536: 23.4 and 23.3, against 24.8 with a factor in every row's arithmetic).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "errors.hpp"
#include "row_vec.hpp"
#include "spgemm.h"

namespace spg {
namespace {

constexpr int kThreads = 256;

// Sum over a workgroup, in every thread, waves in order.
__device__ __forceinline__ float group_sum(float v, float* lds) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < kThreads / 64; ++w) s += lds[w];
    return s;
}

struct NormArgs {
    const char *X, *dY, *weight, *bias;
    char *Y, *dX, *dweight, *dbias;
    float *mean, *rstd, *part;
    int64_t rows, K, pitch;    // pitch: floats between the parts' rows
    float eps;
};

constexpr float kShrink = 0x1p-80f, kGrow = 0x1p80f, kMost = 3.4028234663852886e38f;

// A row's mean and variance (of x * scale) are what they should be, or no other scale would help.
template <int DT>
__device__ __forceinline__ bool settled(float var, float scale) { return DT == kOutF16 || var <= kMost || scale != 1.0f; }

// What (x * scale - mean) is multiplied by.  Of a scaled row eps is far below the variance's last
// bit, except where there is none.
__device__ __forceinline__ float rstd_of(float var, float eps, float scale) {
    return scale == 1.0f ? 1.0f / sqrtf(var + eps) : var == 0.0f ? kGrow / sqrtf(eps) : 1.0f / sqrtf(var);
}

__device__ __forceinline__ void keep(const NormArgs& a, int64_t row, float mean, float rstd, float scale) {
    if (scale != 1.0f) {
        // a mean is below the largest value, its rounding may not be
        const float m = mean * kGrow;
        mean = __builtin_isinf(m) && !__builtin_isinf(mean) ? __builtin_copysignf(kMost, m) : m;
        rstd *= scale;
    }
    a.mean[row] = mean;
    a.rstd[row] = rstd;
}

// n of a kept row.  x - mean alone may pass fp32's range where both are near its end: such rows are
// taken by halves.
template <int DT>
struct Kept {
    float mean, rstd;
    bool halves;
    __device__ __forceinline__ Kept(float m, float r) : mean(m), rstd(r), halves(DT != kOutF16 && r < 0x1p-100f) {
        if (halves) {
            mean *= 0.5f;
            rstd *= 2.0f;
        }
        // -mean rstd, n of the zeros past a row's end, has to be finite; where it is not, the row is
        // one value throughout (any other deviation is 2^-24 of the mean at least): n is 0
        if (DT != kOutF16 && rstd <= kMost && __builtin_fabsf(mean) * rstd > kMost) rstd = 0.0f;
    }
    // x, or its half
    __device__ __forceinline__ float n(float x) const { return (x - mean) * rstd; }
};

// Rows of up to 64 * W * EPT values: a team of W waves takes a row, EPT values a thread, all of it
// in registers between the sums; a workgroup of four teams (W = 1) or one takes every
// gridDim.x-th row and has the next one's loads in flight while it sums.  weight and bias are
// read once per workgroup.  TAIL: rows that end inside a vector; its shifts and masks take up to 60
// registers, which the other rows save.
template <int DT, int W, int EPT, bool TAIL>
struct Team {
    static constexpr int E = Vec<DT>::E, V = EPT / E, TEAMS = W == 1 ? 4 : 1, NT = W * TEAMS * 64;
    static constexpr int64_t kMost = 64 * W * EPT;
    u32x4 v[V];
    // element of vector i that this thread starts at
    static __device__ __forceinline__ int at(int i) { return (i * W * 64 + (int)(threadIdx.x & (W * 64 - 1))) * E; }
    __device__ __forceinline__ void load(const char* row, int K, bool in) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = in && at(i) < K ? vec<DT>(row, at(i), K) : u32x4{};
    }
    template <int D>
    static __device__ __forceinline__ u32x4 vec(const char* row, int k, int K) {
        struct __attribute__((packed, aligned(Vec<D>::EB))) B { u32x4 v; };
        if constexpr (TAIL) return load_vec<D>(row, k, K);
        else return ((const B*)(row + (uint32_t)(k * Vec<D>::EB)))->v;
    }
    static __device__ __forceinline__ void store(char* row, int k, int K, const float (&x)[E]) {
        struct __attribute__((packed, aligned(Vec<DT>::EB))) B { u32x4 v; };
        if constexpr (TAIL) store_vec<DT>(row, k, K, x);
        else ((B*)(row + (uint32_t)(k * Vec<DT>::EB)))->v = pack_vec<DT>(x);
    }
    __device__ __forceinline__ float operator[](int j) const { return elem<DT>(v[j / E], j % E); }
    __device__ __forceinline__ void halve() {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float h[E];
#pragma unroll
            for (int e = 0; e < E; ++e) h[e] = 0.5f * elem<DT>(v[i], e);
            v[i] = pack_vec<DT>(h);
        }
    }
};

template <int PT, typename T>
__device__ __forceinline__ void load_params(const char* p, int K, float fill, float (&x)[T::V * T::E]) {
#pragma unroll
    for (int i = 0; i < T::V; ++i)
#pragma unroll
        for (int h = 0; h < T::E; h += Vec<PT>::E) {
            const u32x4 v = p && T::at(i) + h < K ? T::template vec<PT>(p, T::at(i) + h, K) : u32x4{};
#pragma unroll
            for (int e = 0; e < Vec<PT>::E && h + e < T::E; ++e) x[i * T::E + h + e] = p ? elem<PT>(v, e) : fill;
        }
}

// Sums of NS values over a team, in every thread; `turn` alternates between two places in LDS, so
// that one barrier a sum is enough: when a place is written again, every wave has passed the
// barrier behind its last reading.
template <int W, int NS>
__device__ __forceinline__ void team_sums(float (&s)[NS], float (*lds)[W][NS], int& turn) {
#pragma unroll
    for (int i = 0; i < NS; ++i) s[i] = wave_sum(s[i]);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < NS; ++i) lds[turn][threadIdx.x >> 6][i] = s[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            if constexpr (W == 16) {
                const int lane = threadIdx.x & 63;
                s[i] = wave_sum(lane < W ? lds[turn][lane & (W - 1)][i] : 0.0f);
            } else {
                s[i] = lds[turn][0][i];
#pragma unroll
                for (int w = 1; w < W; ++w) s[i] += lds[turn][w][i];
            }
        }
        turn ^= 1;
    }
}

template <int DT, int PT, int W, int EPT, bool TAIL>
__global__ void __launch_bounds__((Team<DT, W, EPT, TAIL>::NT)) norm_run(NormArgs a) {
    using T = Team<DT, W, EPT, TAIL>;
    __shared__ float lds[2][W][1];
    const int K = (int)a.K, team = W == 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
    const int64_t step = (int64_t)gridDim.x * T::TEAMS, pitch = a.K * Vec<DT>::EB;
    int64_t row = (int64_t)blockIdx.x * T::TEAMS + team;
    int turn = 0;
    T x, next;
    next.load(a.X + row * pitch, K, row < a.rows);
    float w[EPT], b[EPT];
    load_params<PT, T>(a.weight, K, 1.0f, w);
    load_params<PT, T>(a.bias, K, 0.0f, b);
    for (; row < a.rows; row += step) {
        x = next;
        next.load(a.X + (row + step) * pitch, K, row + step < a.rows);
        // one row of x, or of x / 2^80; false: its sums pass fp32's range
        auto pass = [&](auto scaled) __attribute__((always_inline)) {
            constexpr float F = decltype(scaled)::value ? kShrink : 1.0f;
            float s[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < EPT; ++j) s[0] += x[j] * F;
            team_sums<W, 1>(s, lds, turn);
            const float mean = s[0] / (float)K;
            s[0] = 0.0f;
#pragma unroll
            for (int j = 0; j < EPT; ++j) {
                const float c = x[j] * F - mean;
                s[0] += T::at(j / T::E) + j % T::E < K ? c * c : 0.0f;
            }
            team_sums<W, 1>(s, lds, turn);
            const float var = s[0] / (float)K;
            if (!settled<DT>(var, F)) return false;
            const float rstd = rstd_of(var, a.eps, F);
            if (a.mean && (threadIdx.x & (W * 64 - 1)) == 0) keep(a, row, mean, rstd, F);
#pragma unroll
            for (int i = 0; i < T::V; ++i) {
                float y[T::E];
#pragma unroll
                for (int e = 0; e < T::E; ++e)
                    y[e] = __builtin_fmaf((x[i * T::E + e] * F - mean) * rstd, w[i * T::E + e], b[i * T::E + e]);
                if (T::at(i) < K) T::store(a.Y + row * pitch, T::at(i), K, y);
            }
            return true;
        };
        if (__builtin_expect(!pass(std::false_type{}), 0)) pass(std::true_type{});
    }
}

// dX, and each workgroup's share of the parameters' gradients, summed in registers over its
// rows: part [gridDim.x][2][pitch] fp32.  (x and dy past the row's end are zero, and what they
// give is zero or not stored.)
template <int DT, int PT, int W, int EPT, bool TAIL>
__global__ void __launch_bounds__((Team<DT, W, EPT, TAIL>::NT)) norm_back(NormArgs a) {
    using T = Team<DT, W, EPT, TAIL>;
    __shared__ float lds[2][W][2];
    const int K = (int)a.K, team = W == 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
    const int64_t step = (int64_t)gridDim.x * T::TEAMS, pitch = a.K * Vec<DT>::EB;
    int64_t row = (int64_t)blockIdx.x * T::TEAMS + team;
    int turn = 0;
    // the widest teams have no registers left for the next row's loads, and with rows that end inside
    // a vector not for all of their own: of fp16 and fp32 they keep 28 to 56 bytes a lane in scratch
    // (2048 x 16383 fp16: 70 us, bf16, which keeps none, 67; 16384 columns 55)
    constexpr bool AHEAD = W < 16 || EPT < 16;
    T x, dy, nx, ndy;
    // a row's statistics are under way before its values: waiting for a load waits for those before it
    // (8192 x 4096, both launches: 44.6 us, 46.4 with the next row's values in front of them)
    float nm = 0.0f, nr = 0.0f;
    auto statistics = [&](int64_t r, bool in) __attribute__((always_inline)) {
        nm = in ? a.mean[r] : 0.0f;
        nr = in ? a.rstd[r] : 0.0f;
    };
    if constexpr (AHEAD) {
        statistics(row, row < a.rows);
        nx.load(a.X + row * pitch, K, row < a.rows);
        ndy.load(a.dY + row * pitch, K, row < a.rows);
    }
    float w[EPT], dw[EPT], db[EPT];
    load_params<PT, T>(a.weight, K, 1.0f, w);
#pragma unroll
    for (int j = 0; j < EPT; ++j) dw[j] = db[j] = 0.0f;
    for (; row < a.rows; row += step) {
        if constexpr (!AHEAD) statistics(row, true);
        const float mean = nm, rstd = nr;
        if constexpr (AHEAD) {
            const bool more = row + step < a.rows;
            statistics(row + step, more);
            x = nx;
            dy = ndy;
            nx.load(a.X + (row + step) * pitch, K, more);
            ndy.load(a.dY + (row + step) * pitch, K, more);
        } else {
            x.load(a.X + row * pitch, K, true);
            dy.load(a.dY + row * pitch, K, true);
        }
        const Kept<DT> of(mean, rstd);
        if (__builtin_expect(of.halves, 0)) x.halve();
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            const float d = dy[j], n = of.n(x[j]), g = d * w[j];
            dw[j] = __builtin_fmaf(d, n, dw[j]);
            db[j] += d;
            s[0] += g;
            s[1] = __builtin_fmaf(g, n, s[1]);
        }
        team_sums<W, 2>(s, lds, turn);
        const float ms = s[0] / (float)K, mt = s[1] / (float)K;
#pragma unroll
        for (int i = 0; i < T::V; ++i) {
            float o[T::E];
#pragma unroll
            for (int e = 0; e < T::E; ++e) {
                const int j = i * T::E + e;
                o[e] = rstd * (dy[j] * w[j] - ms - of.n(x[j]) * mt);
            }
            if (T::at(i) < K) T::store(a.dX + row * pitch, T::at(i), K, o);
        }
    }
    if (!a.part) return;
    if constexpr (T::TEAMS > 1) {
        // the four waves' sums meet, in order
        __shared__ __attribute__((aligned(16))) float sums[T::TEAMS - 1][2][EPT][64];
        const int lane = threadIdx.x & 63;
        if (team > 0)
#pragma unroll
            for (int j = 0; j < EPT; ++j) {
                sums[team - 1][0][j][lane] = dw[j];
                sums[team - 1][1][j][lane] = db[j];
            }
        __syncthreads();
        if (team > 0) return;
        for (int t = 0; t < T::TEAMS - 1; ++t)
#pragma unroll
            for (int j = 0; j < EPT; ++j) {
                dw[j] += sums[t][0][j][lane];
                db[j] += sums[t][1][j][lane];
            }
    }
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.pitch;
#pragma unroll
    for (int i = 0; i < T::V; ++i)
        if (T::at(i) < K)
#pragma unroll
            for (int e = 0; e < T::E; e += 4) {
                const int j = i * T::E + e;
                *(floatx4*)(part + T::at(i) + e) = floatx4{dw[j], dw[j + 1], dw[j + 2], dw[j + 3]};
                *(floatx4*)(part + a.pitch + T::at(i) + e) = floatx4{db[j], db[j + 1], db[j + 2], db[j + 3]};
            }
}

// The workgroups' shares added: 64 columns a workgroup, 16 waves share the parts, in order.
constexpr int kParamWaves = 16;
template <int PT>
__global__ void __launch_bounds__(kParamWaves * 64) norm_params(NormArgs a, int parts) {
    __shared__ float lds[kParamWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per = (int)(a.pitch + 63) / 64;              // workgroups of one gradient
    const int which = blockIdx.x >= per;
    const int64_t k = (int64_t)(blockIdx.x - which * per) * 64 + lane;
    char* out = which ? a.dbias : a.dweight;
    if (!out) return;
    float s = 0.0f;
    if (k < a.pitch) {
        const float* p = a.part + which * a.pitch + k;
        constexpr int U = 8;
        for (int i = wave; i < parts; i += U * kParamWaves) {
            float v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = i + u * kParamWaves < parts ? p[(int64_t)(i + u * kParamWaves) * 2 * a.pitch] : 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) s += v[u];
        }
    }
    lds[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || k >= a.K) return;
    for (int i = 1; i < kParamWaves; ++i) s += lds[i][lane];
    store1<PT>(out, k, s);
}

// ---- rows of any length: read again for each sum -------------------------------------------

template <int DT, int PT>
__global__ void __launch_bounds__(kThreads) norm_rows(NormArgs a) {
    __shared__ float lds[kThreads / 64];
    constexpr int E = Vec<DT>::E;
    const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x, K = a.K;
    if (row >= a.rows) return;
    const char* x = a.X + row * K * Vec<DT>::EB;
    auto pass = [&](auto scaled) __attribute__((always_inline)) {   // as in norm_run
        constexpr float F = decltype(scaled)::value ? kShrink : 1.0f;
        float s = 0.0f;
        for (int64_t k = threadIdx.x * E; k < K; k += kThreads * E) {
            const u32x4 v = load_short<DT>(x, k, K);
            for (int e = 0; e < E; ++e) s += elem<DT>(v, e) * F;
        }
        const float mean = group_sum(s, lds) / (float)K;
        s = 0.0f;
        for (int64_t k = threadIdx.x * E; k < K; k += kThreads * E) {
            const u32x4 v = load_short<DT>(x, k, K);
            for (int e = 0; e < E; ++e) {
                const float c = elem<DT>(v, e) * F - mean;
                if (k + e < K) s += c * c;
            }
        }
        const float var = group_sum(s, lds) / (float)K;
        if (!settled<DT>(var, F)) return false;
        const float rstd = rstd_of(var, a.eps, F);
        if (a.mean && threadIdx.x == 0) keep(a, row, mean, rstd, F);
        for (int64_t k = threadIdx.x; k < K; k += kThreads) {
            const float n = (load1<DT>(x, k) * F - mean) * rstd;
            const float w = a.weight ? load1<PT>(a.weight, k) : 1.0f, b = a.bias ? load1<PT>(a.bias, k) : 0.0f;
            store1<DT>(a.Y + row * K * Vec<DT>::EB, k, __builtin_fmaf(n, w, b));
        }
        return true;
    };
    if (__builtin_expect(!pass(std::false_type{}), 0)) pass(std::true_type{});
}

template <int DT, int PT>
__global__ void __launch_bounds__(kThreads) norm_rows_back(NormArgs a) {
    __shared__ float lds[kThreads / 64];
    const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x, K = a.K, o = row * K * Vec<DT>::EB;
    if (row >= a.rows) return;
    const float rstd = a.rstd[row];
    const Kept<DT> of(a.mean[row], rstd);
    const float part = of.halves ? 0.5f : 1.0f;
    float s = 0.0f, t = 0.0f;
    for (int64_t k = threadIdx.x; k < K; k += kThreads) {
        const float n = of.n(load1<DT>(a.X + o, k) * part);
        const float g = load1<DT>(a.dY + o, k) * (a.weight ? load1<PT>(a.weight, k) : 1.0f);
        s += g;
        t += g * n;
    }
    s = group_sum(s, lds) / (float)K;
    t = group_sum(t, lds) / (float)K;
    for (int64_t k = threadIdx.x; k < K; k += kThreads) {
        const float n = of.n(load1<DT>(a.X + o, k) * part);
        const float g = load1<DT>(a.dY + o, k) * (a.weight ? load1<PT>(a.weight, k) : 1.0f);
        store1<DT>(a.dX + o, k, rstd * (g - s - n * t));
    }
}

// The parameters' gradients of `per` rows (blockIdx.y-th): C columns a workgroup, its other threads
// share the rows, which meet in LDS in order.  Several parts go through the workspace and
// norm_params, so that no thread has a long chain of rows to add by itself: four of them for all rows
// end a sum of 10^8 ones at 2^26.  The backward pass of 32768 x 4 takes 26 us (899 with those four), of
// 8192 x 20000 590 (1344).
template <int DT, int PT, int C>
__global__ void __launch_bounds__(kThreads) norm_columns(NormArgs a, int64_t per) {
    constexpr int R = kThreads / C;
    __shared__ float lds[2][R][C];
    const int col = threadIdx.x % C, own = threadIdx.x / C;
    const int64_t k = (int64_t)blockIdx.x * C + col, first = blockIdx.y * per;
    const int64_t last = first + per < a.rows ? first + per : a.rows;
    float w = 0.0f, b = 0.0f;
    if (k < a.K)
#pragma unroll 4
        for (int64_t r = first + own; r < last; r += R) {
            const float dy = load1<DT>(a.dY, r * a.K + k);
            const Kept<DT> of(a.mean[r], a.rstd[r]);
            w += dy * of.n(load1<DT>(a.X, r * a.K + k) * (of.halves ? 0.5f : 1.0f));
            b += dy;
        }
    lds[0][own][col] = w;
    lds[1][own][col] = b;
    __syncthreads();
    if (own > 0 || k >= a.K) return;
    for (int i = 1; i < R; ++i) {
        w += lds[0][i][col];
        b += lds[1][i][col];
    }
    if (a.part) {
        float* part = a.part + (int64_t)blockIdx.y * 2 * a.pitch + k;
        part[0] = w;
        part[a.pitch] = b;
    } else {
        if (a.dweight) store1<PT>(a.dweight, k, w);
        if (a.dbias) store1<PT>(a.dbias, k, b);
    }
}

// a workgroup a row: a launch has less than 2^32 threads along one axis
dim3 row_grid(int64_t rows) {
    const int64_t x = std::min<int64_t>(rows, 1 << 23);
    return dim3((unsigned)x, (unsigned)((rows + x - 1) / x));
}

gemm_status launched() {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? GEMM_OK : hip_fail(e);
}

}  // namespace
}  // namespace spg

struct gemm_norm_plan {
    int64_t rows, K;
    int dt, pt;
    float eps;
    int waves, ept;            // of a team; 0: rows of any length
    int64_t wgs, back_wgs;     // workgroups; of rows of any length, the parts of the parameters' gradients
    int64_t pitch() const { return (K + 7) / 8 * 8; }
};

namespace {

// f(type, type of the parameters) for a plan
template <typename F>
void with_types(const gemm_norm_plan* h, F&& f) {
    using std::integral_constant;
    constexpr integral_constant<int, spg::kOutF32> f32{};
    auto go = [&](auto dt) {
        if (h->pt == GEMM_F32) f(dt, f32);
        else f(dt, dt);
    };
    if (h->dt == GEMM_F16) go(integral_constant<int, spg::kOutF16>{});
    else if (h->dt == GEMM_BF16) go(integral_constant<int, spg::kOutBF16>{});
    else f(f32, f32);
}

// f(waves of a team, values a thread, rows end inside a vector) for a plan whose rows stay in registers
template <typename F>
void with_team(const gemm_norm_plan* h, F&& f) {
    using std::integral_constant;
    auto tail = [&](auto w, auto ept) {
        if (h->K % 8 == 0) f(w, ept, std::false_type{});
        else f(w, ept, std::true_type{});
    };
    auto go = [&](auto w) {
        if (h->ept == 8) tail(w, integral_constant<int, 8>{});
        else tail(w, integral_constant<int, 16>{});
    };
    if (h->waves == 1) go(integral_constant<int, 1>{});
    else if (h->waves == 4) go(integral_constant<int, 4>{});
    else go(integral_constant<int, 16>{});
}

}  // namespace

extern "C" {

gemm_status gemm_norm_create(gemm_norm_handle* out, int64_t rows, int64_t K, gemm_dtype dtype, gemm_dtype param_dtype,
                             float eps) {
    if (!out) return GEMM_ERR_INVALID_ARG;
    *out = nullptr;
    if (rows < 0 || K < 0 || !(eps >= 0.0f) || !std::isfinite(eps)) return GEMM_ERR_INVALID_ARG;
    if (dtype != GEMM_F16 && dtype != GEMM_BF16 && dtype != GEMM_F32) return GEMM_ERR_INVALID_ARG;
    if (param_dtype != dtype && param_dtype != GEMM_F32) return GEMM_ERR_INVALID_ARG;
    const int64_t lim = INT32_MAX / 2 - 512;
    if (rows > lim || K > lim) return GEMM_ERR_UNSUPPORTED;
    gemm_norm_plan* p = new (std::nothrow) gemm_norm_plan{rows, K, (int)dtype, (int)param_dtype, eps, 0, 0, 0, 0};
    if (!p) return GEMM_ERR_OUT_OF_MEMORY;
    // rows shorter than a vector: as rows of any length
    if (K < 8) p->waves = 0;
    else if (K <= 1024 && rows >= 2048) p->waves = 1;
    else if (K <= 4096) p->waves = 4;
    else if (K <= 16384) p->waves = 16;
    if (p->waves) {
        p->ept = K <= 64 * 8 * p->waves ? 8 : 16;
        const int64_t teams = p->waves == 1 ? (rows + 3) / 4 : rows;
        // about as many as the CUs hold at once: each takes the next row as it ends one (8192 x 4096,
        // forward: 27.0 us with 1024, 29.7 with 2048, 38.6 with a workgroup a row; 2048 x 16384: 29.7
        // with 256, 33.5 with 512; 16384 x 1536, 8 values a thread: 22.7 with 2048, 26.7 with 1024)
        p->wgs = std::min<int64_t>(teams, (p->waves == 16 ? 512 : 2048) / (p->ept == 16 ? 2 : 1));
        // each writes its sums of the parameters' gradients; up to 1024 of short rows, if it has eight of
        // them or more (both passes of 16384 x 1536: 60.2 us with 1024, 70.4 with 512; of 8192 x 4096,
        // 16 values a thread, 77.5 and 73.9)
        const int64_t most = p->ept == 16 ? 512 : std::max<int64_t>(512, std::min<int64_t>(1024, teams / 8));
        p->back_wgs = std::min<int64_t>(teams, p->waves == 16 ? 256 : most);
    } else if (rows > 0 && K > 0) {
        // about as many workgroups as the CUs hold at once, 256 rows or more in each
        const int64_t columns = K < 8 ? 1 : (K + 63) / 64;
        p->back_wgs = std::max<int64_t>(1, std::min((rows + 255) / 256, 2048 / columns));
    }
    *out = p;
    return GEMM_OK;
}

int64_t gemm_norm_workspace(gemm_norm_handle h) {
    if (!h) return -1;
    return !h->waves && h->back_wgs == 1 ? 0 : h->back_wgs * 2 * h->pitch() * 4;   // one part is stored at once
}

gemm_status gemm_norm_run(gemm_norm_handle h, const void* X, const void* weight, const void* bias, void* Y, float* mean,
                          float* rstd, hipStream_t stream) {
    if (!h || (mean == nullptr) != (rstd == nullptr)) return GEMM_ERR_INVALID_ARG;
    if (h->rows == 0 || h->K == 0) return GEMM_OK;
    if (!X || !Y) return GEMM_ERR_INVALID_ARG;
    spg::NormArgs a{};
    a.X = (const char*)X;
    a.weight = (const char*)weight;
    a.bias = (const char*)bias;
    a.Y = (char*)Y;
    a.mean = mean;
    a.rstd = rstd;
    a.rows = h->rows;
    a.K = h->K;
    a.eps = h->eps;
    with_types(h, [&](auto dt, auto pt) {
        constexpr int D = decltype(dt)::value, P = decltype(pt)::value;
        if (h->waves)
            return with_team(h, [&](auto w, auto ept, auto tail) {
                constexpr int W = decltype(w)::value, N = decltype(ept)::value;
                constexpr bool T = decltype(tail)::value;
                hipLaunchKernelGGL((spg::norm_run<D, P, W, N, T>), dim3((unsigned)h->wgs), dim3(spg::Team<D, W, N, T>::NT), 0, stream, a);
            });
        hipLaunchKernelGGL((spg::norm_rows<D, P>), spg::row_grid(h->rows),
                           dim3(spg::kThreads), 0, stream, a);
    });
    return spg::launched();
}

gemm_status gemm_norm_backward(gemm_norm_handle h, const void* dY, const void* X, const void* weight, const float* mean,
                               const float* rstd, void* dX, void* dweight, void* dbias, void* workspace,
                               int64_t workspace_bytes, hipStream_t stream) {
    if (!h) return GEMM_ERR_INVALID_ARG;
    if (h->K == 0) return GEMM_OK;
    if (h->rows > 0 && (!dY || !X || !mean || !rstd || !dX)) return GEMM_ERR_INVALID_ARG;
    const int64_t need = gemm_norm_workspace(h);
    if (need > 0 && (dweight || dbias) && (!workspace || (uintptr_t)workspace % 16 != 0 || workspace_bytes < need))
        return GEMM_ERR_INVALID_ARG;
    spg::NormArgs a{};
    a.X = (const char*)X;
    a.dY = (const char*)dY;
    a.weight = (const char*)weight;
    a.dX = (char*)dX;
    a.dweight = (char*)dweight;
    a.dbias = (char*)dbias;
    a.mean = (float*)mean;
    a.rstd = (float*)rstd;
    a.rows = h->rows;
    a.K = h->K;
    a.part = need > 0 && (dweight || dbias) ? (float*)workspace : nullptr;
    a.pitch = h->pitch();
    with_types(h, [&](auto dt, auto pt) {
        constexpr int D = decltype(dt)::value, P = decltype(pt)::value;
        auto join = [&] {
            hipLaunchKernelGGL((spg::norm_params<P>), dim3((unsigned)(2 * ((h->pitch() + 63) / 64))), dim3(spg::kParamWaves * 64), 0,
                               stream, a, (int)h->back_wgs);
        };
        if (h->waves && h->rows > 0) {
            with_team(h, [&](auto w, auto ept, auto tail) {
                constexpr int W = decltype(w)::value, N = decltype(ept)::value;
                constexpr bool T = decltype(tail)::value;
                hipLaunchKernelGGL((spg::norm_back<D, P, W, N, T>), dim3((unsigned)h->back_wgs), dim3(spg::Team<D, W, N, T>::NT), 0, stream, a);
            });
            if (a.part) join();
            return;
        }
        if (h->rows > 0) hipLaunchKernelGGL((spg::norm_rows_back<D, P>), spg::row_grid(h->rows), dim3(spg::kThreads), 0, stream, a);
        if (!dweight && !dbias) return;
        const int64_t parts = std::max<int64_t>(h->back_wgs, 1), per = (h->rows + parts - 1) / parts;   // of no rows: zeros
        if (h->K < 8)
            hipLaunchKernelGGL((spg::norm_columns<D, P, 8>), dim3(1, (unsigned)parts), dim3(spg::kThreads), 0, stream, a, per);
        else
            hipLaunchKernelGGL((spg::norm_columns<D, P, 64>), dim3((unsigned)((h->K + 63) / 64), (unsigned)parts),
                               dim3(spg::kThreads), 0, stream, a, per);
        if (a.part) join();
    });
    return spg::launched();
}

gemm_status gemm_norm_destroy(gemm_norm_handle h) {
    delete h;
    return GEMM_OK;
}

}  // extern "C"
