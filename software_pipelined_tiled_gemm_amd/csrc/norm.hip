// Layer norm and its backward pass (gemm_norm_* in include/spgemm.h).
//
//   n = (x - mean) rstd,  y = n w + b
//   g = dy w,  dx = rstd (g - sum g / K - n sum(g n) / K),  dw = sum_rows dy n,  db = sum_rows dy
//
// The mean is taken off before the squares are summed: the variance of a row far from zero
// keeps its bits, which sum x^2 - mean^2 would lose.
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
    int64_t rows, K;
    float eps;
};

template <int DT, int PT>
__global__ void __launch_bounds__(kThreads) norm_rows(NormArgs a) {
    __shared__ float lds[kThreads / 64];
    constexpr int E = Vec<DT>::E;
    const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x, K = a.K;
    if (row >= a.rows) return;
    const char* x = a.X + row * K * Vec<DT>::EB;
    float s = 0.0f;
    for (int64_t k = threadIdx.x * E; k < K; k += kThreads * E) {
        const u32x4 v = load_vec<DT>(x, k, K);
        for (int e = 0; e < E; ++e) s += elem<DT>(v, e);
    }
    const float mean = group_sum(s, lds) / (float)K;
    s = 0.0f;
    for (int64_t k = threadIdx.x * E; k < K; k += kThreads * E) {
        const u32x4 v = load_vec<DT>(x, k, K);
        for (int e = 0; e < E; ++e) {
            const float c = elem<DT>(v, e) - mean;
            if (k + e < K) s += c * c;
        }
    }
    const float rstd = 1.0f / sqrtf(group_sum(s, lds) / (float)K + a.eps);
    if (a.mean && threadIdx.x == 0) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
    for (int64_t k = threadIdx.x; k < K; k += kThreads) {
        const float n = (load1<DT>(x, k) - mean) * rstd;
        const float w = a.weight ? load1<PT>(a.weight, k) : 1.0f, b = a.bias ? load1<PT>(a.bias, k) : 0.0f;
        store1<DT>(a.Y + row * K * Vec<DT>::EB, k, __builtin_fmaf(n, w, b));
    }
}

template <int DT, int PT>
__global__ void __launch_bounds__(kThreads) norm_rows_back(NormArgs a) {
    __shared__ float lds[kThreads / 64];
    const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x, K = a.K, o = row * K * Vec<DT>::EB;
    if (row >= a.rows) return;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s = 0.0f, t = 0.0f;
    for (int64_t k = threadIdx.x; k < K; k += kThreads) {
        const float n = (load1<DT>(a.X + o, k) - mean) * rstd;
        const float g = load1<DT>(a.dY + o, k) * (a.weight ? load1<PT>(a.weight, k) : 1.0f);
        s += g;
        t += g * n;
    }
    s = group_sum(s, lds) / (float)K;
    t = group_sum(t, lds) / (float)K;
    for (int64_t k = threadIdx.x; k < K; k += kThreads) {
        const float n = (load1<DT>(a.X + o, k) - mean) * rstd;
        const float g = load1<DT>(a.dY + o, k) * (a.weight ? load1<PT>(a.weight, k) : 1.0f);
        store1<DT>(a.dX + o, k, rstd * (g - s - n * t));
    }
}

// One thread a column, four waves sharing the rows.
template <int DT, int PT>
__global__ void __launch_bounds__(kThreads) norm_columns(NormArgs a) {
    __shared__ float lds[kThreads / 64][2][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t k = (int64_t)blockIdx.x * 64 + lane;
    float w = 0.0f, b = 0.0f;
    if (k < a.K)
        for (int64_t r = wave; r < a.rows; r += kThreads / 64) {
            const float dy = load1<DT>(a.dY, r * a.K + k);
            w += dy * ((load1<DT>(a.X, r * a.K + k) - a.mean[r]) * a.rstd[r]);
            b += dy;
        }
    lds[wave][0][lane] = w;
    lds[wave][1][lane] = b;
    __syncthreads();
    if (wave > 0 || k >= a.K) return;
    for (int i = 1; i < kThreads / 64; ++i) {
        w += lds[i][0][lane];
        b += lds[i][1][lane];
    }
    if (a.dweight) store1<PT>(a.dweight, k, w);
    if (a.dbias) store1<PT>(a.dbias, k, b);
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
    gemm_norm_plan* p = new (std::nothrow) gemm_norm_plan{rows, K, (int)dtype, (int)param_dtype, eps};
    if (!p) return GEMM_ERR_OUT_OF_MEMORY;
    *out = p;
    return GEMM_OK;
}

int64_t gemm_norm_workspace(gemm_norm_handle h) { return h ? 0 : -1; }

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
        hipLaunchKernelGGL((spg::norm_rows<decltype(dt)::value, decltype(pt)::value>), spg::row_grid(h->rows),
                           dim3(spg::kThreads), 0, stream, a);
    });
    return spg::launched();
}

gemm_status gemm_norm_backward(gemm_norm_handle h, const void* dY, const void* X, const void* weight, const float* mean,
                               const float* rstd, void* dX, void* dweight, void* dbias, void* workspace,
                               int64_t workspace_bytes, hipStream_t stream) {
    (void)workspace;
    (void)workspace_bytes;
    if (!h) return GEMM_ERR_INVALID_ARG;
    if (h->K == 0) return GEMM_OK;
    if (h->rows > 0 && (!dY || !X || !mean || !rstd || !dX)) return GEMM_ERR_INVALID_ARG;
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
    with_types(h, [&](auto dt, auto pt) {
        constexpr int D = decltype(dt)::value, P = decltype(pt)::value;
        if (h->rows > 0)
            hipLaunchKernelGGL((spg::norm_rows_back<D, P>), spg::row_grid(h->rows), dim3(spg::kThreads), 0, stream, a);
        if (dweight || dbias)
            hipLaunchKernelGGL((spg::norm_columns<D, P>), dim3((unsigned)((h->K + 63) / 64)), dim3(spg::kThreads), 0, stream, a);
    });
    return spg::launched();
}

gemm_status gemm_norm_destroy(gemm_norm_handle h) {
    delete h;
    return GEMM_OK;
}

}  // extern "C"
