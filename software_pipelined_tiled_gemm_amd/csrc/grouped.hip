// C ABI of the products by group (gemm_grouped_* and gemm_experts_* in include/spgemm.h).
//
// Host side: argument validation (before any HIP call), the choice of kernel from the sizes,
// the workspace layout and the launches.  Nothing here knows how many rows a group has: the
// grids cover what the plan's rows can come to, and the kernels read the offsets.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <new>

#include "errors.hpp"
#include "grouped_kernels.hpp"
#include "spgemm.h"

namespace {

constexpr int64_t kAlign = 256;   // sections of a workspace
int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

gemm_status launched() {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? GEMM_OK : spg::hip_fail(e);
}

// Sizes, layouts and workspaces that the plain and the gated products share.
struct Common {
    int64_t rows, N, K, groups, tokens;   // tokens -1: no source
    bool bf, nk;
    int64_t matrix() const { return N * K * 2; }
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

spg::GroupArgs group_args(const Common& c, const int32_t* offsets, const int32_t* source, int64_t b_step) {
    return spg::GroupArgs{offsets, source, b_step, (int32_t)c.groups, (int32_t)c.rows, (int32_t)std::max<int64_t>(c.tokens, 0)};
}

dim3 simple_grid(int64_t outputs, int64_t groups) {
    return dim3((unsigned)std::min<int64_t>(ceil_div(std::max<int64_t>(outputs, 1), 256), 4096), (unsigned)groups);
}

// Rows of every group times its matrix, B as [N,K] (nk) or [K,N]; A's rows through `source`
// where that is not null.  Two B: gated, or (segments 2) one sum over both.
gemm_status simple_rows(const Common& c, const spg::ProductArgs& p, bool nk, int64_t lda, int64_t seg_a, bool dual,
                        const int32_t* offsets, const int32_t* source, hipStream_t st) {
    const spg::SimpleGroupArgs a{p, group_args(c, offsets, source, c.matrix()), lda, 1, nk ? p.K : 1, nk ? 1 : p.N, seg_a};
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
    const spg::SimpleWeightArgs a{group_args(c, offsets, source, c.matrix()), (const char*)D, (const char*)X, (char*)C,
                                  ldd, c.N, c.K, c.nk ? c.K : 1, c.nk ? 1 : c.N};
    const dim3 grid = simple_grid(c.N * c.K, c.groups);
    if (c.bf) hipLaunchKernelGGL((spg::simple_group_weights<true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((spg::simple_group_weights<false>), grid, dim3(256), 0, st, a);
    return launched();
}

bool small_workspace(const void* workspace, int64_t bytes, int64_t need) {
    return need > 0 && (!workspace || (uintptr_t)workspace % 16 != 0 || bytes < need);
}

}  // namespace

struct gemm_grouped_plan {
    Common c;
};

struct gemm_experts_plan {
    Common c;
    int act;
    int64_t np;        // columns of dG and of dU in the workspace
    int64_t ws_back;
};

extern "C" {

gemm_status gemm_grouped_create(gemm_grouped_handle* out, int64_t rows, int64_t N, int64_t K, int64_t groups,
                                int64_t tokens, gemm_dtype dtype, gemm_b_layout layout) {
    if (out) *out = nullptr;
    const gemm_status e = check(out, rows, N, K, groups, tokens, dtype, layout);
    if (e != GEMM_OK) return e;
    gemm_grouped_plan* p = new (std::nothrow) gemm_grouped_plan{
        Common{rows, N, K, groups, tokens, dtype == GEMM_BF16, layout == GEMM_B_NK}};
    if (!p) return GEMM_ERR_OUT_OF_MEMORY;
    *out = p;
    return GEMM_OK;
}

int64_t gemm_grouped_workspace(gemm_grouped_handle h) { return h ? 0 : -1; }
int64_t gemm_grouped_run_workspace(gemm_grouped_handle h) { return h ? 0 : -1; }

gemm_status gemm_grouped_run(gemm_grouped_handle h, const void* X, const void* W, const int32_t* offsets,
                             const int32_t* source, void* Y, void* workspace, int64_t workspace_bytes,
                             hipStream_t stream) {
    (void)workspace;
    (void)workspace_bytes;
    if (!h) return GEMM_ERR_INVALID_ARG;
    const Common& c = h->c;
    if ((c.tokens < 0) != (source == nullptr) && c.rows > 0) return GEMM_ERR_INVALID_ARG;
    if (c.rows == 0 || c.N == 0) return GEMM_OK;
    if (!offsets || !Y || (c.K > 0 && (!W || (!X && c.tokens != 0)))) return GEMM_ERR_INVALID_ARG;
    spg::ProductArgs a{};
    a.A = (const char*)X;
    a.B[0] = (const char*)W;
    a.C = Y;
    a.M = (int32_t)c.rows;
    a.N = (int32_t)c.N;
    a.K = (int32_t)c.K;
    a.segments = 1;
    return simple_rows(c, a, c.nk, c.K, 0, false, offsets, source, stream);
}

gemm_status gemm_grouped_backward(gemm_grouped_handle h, const void* dY, const void* X, const void* W,
                                  const int32_t* offsets, const int32_t* source, void* dX, void* dW, void* workspace,
                                  int64_t workspace_bytes, hipStream_t stream) {
    (void)workspace;
    (void)workspace_bytes;
    if (!h) return GEMM_ERR_INVALID_ARG;
    const Common& c = h->c;
    if ((c.tokens < 0) != (source == nullptr) && c.rows > 0) return GEMM_ERR_INVALID_ARG;
    if (c.K == 0 || (!dX && !dW) || (c.rows == 0 && c.N == 0)) return GEMM_OK;
    if (!offsets) return GEMM_ERR_INVALID_ARG;
    if (c.rows > 0 && c.N > 0 && (!dY || (dX && !W) || (dW && !X && c.tokens != 0))) return GEMM_ERR_INVALID_ARG;
    if (dX && c.rows > 0) {
        spg::ProductArgs a{};
        a.A = (const char*)dY;
        a.B[0] = (const char*)W;
        a.C = dX;
        a.M = (int32_t)c.rows;
        a.N = (int32_t)c.K;
        a.K = (int32_t)c.N;
        a.segments = 1;
        const gemm_status e = simple_rows(c, a, !c.nk, c.N, 0, false, offsets, nullptr, stream);
        if (e != GEMM_OK) return e;
    }
    if (dW && c.N > 0) return simple_weights(c, dY, c.N, X, dW, offsets, source, stream);
    return GEMM_OK;
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
    gemm_experts_plan* p = new (std::nothrow) gemm_experts_plan{
        Common{rows, N, K, groups, tokens, dtype == GEMM_BF16, layout == GEMM_B_NK}, (int)act, up(N, 64), 0};
    if (!p) return GEMM_ERR_OUT_OF_MEMORY;
    p->ws_back = up(rows * p->np * 4, kAlign);
    *out = p;
    return GEMM_OK;
}

int64_t gemm_experts_workspace(gemm_experts_handle h) { return h ? h->ws_back : -1; }
int64_t gemm_experts_run_workspace(gemm_experts_handle h) { return h ? 0 : -1; }

gemm_status gemm_experts_run(gemm_experts_handle h, const void* X, const void* Wg, const void* Wu,
                             const int32_t* offsets, const int32_t* source, void* H, void* G, void* U, void* workspace,
                             int64_t workspace_bytes, hipStream_t stream) {
    (void)workspace;
    (void)workspace_bytes;
    if (!h || (G == nullptr) != (U == nullptr)) return GEMM_ERR_INVALID_ARG;
    const Common& c = h->c;
    if ((c.tokens < 0) != (source == nullptr) && c.rows > 0) return GEMM_ERR_INVALID_ARG;
    if (c.rows == 0 || c.N == 0) return GEMM_OK;
    if (!offsets || !H || (c.K > 0 && (!Wg || !Wu || (!X && c.tokens != 0)))) return GEMM_ERR_INVALID_ARG;
    spg::ProductArgs a{};
    a.A = (const char*)X;
    a.B[0] = (const char*)Wg;
    a.B[1] = (const char*)Wu;
    a.C = H;
    a.G = G;
    a.U = U;
    a.M = (int32_t)c.rows;
    a.N = (int32_t)c.N;
    a.K = (int32_t)c.K;
    a.segments = 1;
    a.act = (uint8_t)h->act;
    return simple_rows(c, a, c.nk, c.K, 0, true, offsets, source, stream);
}

gemm_status gemm_experts_backward(gemm_experts_handle h, const void* dH, const void* X, const void* Wg, const void* Wu,
                                  const void* G, const void* U, const int32_t* offsets, const int32_t* source, void* dX,
                                  void* dWg, void* dWu, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (!h) return GEMM_ERR_INVALID_ARG;
    const Common& c = h->c;
    if ((c.tokens < 0) != (source == nullptr) && c.rows > 0) return GEMM_ERR_INVALID_ARG;
    if (c.K == 0 || (c.rows == 0 && c.N == 0)) return GEMM_OK;
    if (!offsets || (c.rows > 0 && !dX) || (c.N > 0 && (!dWg || !dWu))) return GEMM_ERR_INVALID_ARG;
    if (c.rows > 0 && c.N > 0) {
        if (!dH || (!X && c.tokens != 0) || !Wg || !Wu || !G || !U) return GEMM_ERR_INVALID_ARG;
        if (small_workspace(workspace, workspace_bytes, h->ws_back)) return GEMM_ERR_INVALID_ARG;
    }
    uint16_t* D = (uint16_t*)workspace;
    if (c.rows > 0 && c.N > 0) {
        const dim3 grid((unsigned)ceil_div(c.rows * (h->np / 8), 256));
        if (c.bf) hipLaunchKernelGGL((spg::gated_slopes<true>), grid, dim3(256), 0, stream, (const uint16_t*)dH,
                                     (const uint16_t*)G, (const uint16_t*)U, D, (int)c.rows, (int)c.N, (int)h->np, h->act);
        else hipLaunchKernelGGL((spg::gated_slopes<false>), grid, dim3(256), 0, stream, (const uint16_t*)dH,
                                (const uint16_t*)G, (const uint16_t*)U, D, (int)c.rows, (int)c.N, (int)h->np, h->act);
        const gemm_status e = launched();
        if (e != GEMM_OK) return e;
    }
    if (c.rows > 0) {
        spg::ProductArgs a{};
        a.A = (const char*)D;
        a.B[0] = (const char*)Wg;
        a.B[1] = (const char*)Wu;
        a.C = dX;
        a.M = (int32_t)c.rows;
        a.N = (int32_t)c.K;
        a.K = (int32_t)c.N;
        a.segments = 2;
        const gemm_status e = simple_rows(c, a, !c.nk, 2 * h->np, h->np, false, offsets, nullptr, stream);
        if (e != GEMM_OK) return e;
    }
    for (int z = 0; z < 2 && c.N > 0; ++z) {
        const gemm_status e = simple_weights(c, D + z * h->np, 2 * h->np, X, z ? dWu : dWg, offsets, source, stream);
        if (e != GEMM_OK) return e;
    }
    return GEMM_OK;
}

gemm_status gemm_experts_destroy(gemm_experts_handle h) {
    delete h;
    return GEMM_OK;
}

}  // extern "C"
