// The routing of tokens to experts and the combination of the experts' rows (gemm_route_* and
// gemm_combine_* in include/spgemm.h).
//
// Routing is a top-k per token and a counting sort of the (token, choice) pairs by expert that
// keeps the tokens' order.  A pair's place is
//     offsets[e] + (pairs of e in earlier blocks of tokens) + (earlier tokens of its block with e)
// A token has an expert at most once, so 64 tokens' choices are a 64-bit mask per expert: the
// mask's bits below a token's own are the last term, all its bits the block's count.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <new>

#include "errors.hpp"
#include "row_vec.hpp"
#include "spgemm.h"

namespace spg {
namespace {

constexpr int kMaxExperts = 1024, kMaxChoices = 64;
constexpr int kRouteThreads = 1024;
constexpr int kBlock = 64;          // tokens of a mask
constexpr int kMaxBlocks = 256;     // workgroups of a routing; more tokens: more masks each

struct RouteArgs {
    const char* logits;
    float* gate;
    int32_t *expert, *slot, *source, *offsets, *count;   // count [blocks][experts]
    int32_t T, E, k, per, blocks;                        // per: tokens of a workgroup
    int32_t renorm;
};

// A float's bits in an unsigned order: NaN lowest (0), then -inf, ... , +inf.
__device__ __forceinline__ uint32_t order_of(float x) {
    if (x != x) return 0u;
    // -0 and +0 are equal: one key
    const uint32_t b = x == 0.0f ? 0u : __builtin_bit_cast(uint32_t, x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
constexpr uint32_t kNothing = 0x007fffffu;   // order_of(-inf): it and NaN are never chosen

// The largest key of a wave, as a scalar; by shifts within rows of lanes and the rows' ends, a
// dependent instruction each instead of a trip through LDS (16384 tokens, 8 of 64 experts: the
// choices take %CHOOSE%).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    auto most = [&](auto ctrl, auto rows) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, decltype(rows)::value, 0xf, false);
        v = o > v ? o : v;
    };
    using std::integral_constant;
    constexpr integral_constant<int, 0xf> all{};
    most(integral_constant<int, 0x111>{}, all);   // row_shr:1
    most(integral_constant<int, 0x112>{}, all);
    most(integral_constant<int, 0x114>{}, all);
    most(integral_constant<int, 0x118>{}, all);
    most(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});   // row_bcast:15
    most(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});   // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ float value_of(uint32_t key) {
    return __builtin_bit_cast(float, key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// One wave, one token: C * 64 logits in registers, the k largest one by one.  Lane j ends with
// choice j (expert -1: none) and its gate.
template <int DT, int C>
__device__ __forceinline__ void choose(const RouteArgs& a, int64_t t, int lane, int& expert, float& gate) {
    float x[C];
    uint32_t key[C];
    bool nan = false;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = c * 64 + lane;
        x[c] = e < a.E ? load1<DT>(a.logits, t * a.E + e) : -__builtin_inff();
        key[c] = order_of(x[c]);
        nan |= x[c] != x[c];
    }
    nan = __ballot(nan) != 0;
    expert = -1;
    float value = -__builtin_inff(), top = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int c = 1; c < C; ++c) best = key[c] > best ? key[c] : best;
        best = wave_max(best);
        if (best <= kNothing) break;
        // the lowest index among equals: the first register, then the first lane
        int e = -1;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const uint64_t m = __ballot(key[c] == best);
            if (e < 0 && m) {
                const int l = __builtin_ctzll(m);
                e = c * 64 + l;
                if (lane == l) key[c] = 0u;
            }
        }
        const float v = value_of(best);
        if (j == 0) top = v;
        if (lane == j) {
            expert = e;
            value = v;
        }
    }
    // softmax over the chosen, or over all; expf to the last bit or two: gates are fp32
    const float p = expert >= 0 ? expf(value - top) : 0.0f;
    float all = 0.0f;
    if (a.renorm) {
        all = p;
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) all += x[c] == -__builtin_inff() ? 0.0f : expf(x[c] - top);
    }
    all = wave_sum(all);
    gate = expert < 0 ? 0.0f : nan ? __builtin_nanf("") : p / all;
}

template <int DT>
__device__ __forceinline__ void choose_any(const RouteArgs& a, int64_t t, int lane, int& expert, float& gate) {
    if (a.E <= 64) choose<DT, 1>(a, t, lane, expert, gate);
    else if (a.E <= 128) choose<DT, 2>(a, t, lane, expert, gate);
    else if (a.E <= 256) choose<DT, 4>(a, t, lane, expert, gate);
    else choose<DT, kMaxExperts / 64>(a, t, lane, expert, gate);
}

// The places of the pairs of 64 tokens from t0: base[e] is where expert e's go on.
__device__ __forceinline__ void place_block(const RouteArgs& a, int64_t t0, uint64_t* mask, int* base) {
    const int tid = threadIdx.x;
    const int64_t left = (int64_t)a.T - t0;
    const int n = (int)(left < kBlock ? left : kBlock) * a.k;
    const int32_t* ex = a.expert + t0 * a.k;
    for (int e = tid; e < a.E; e += kRouteThreads) mask[e] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kRouteThreads)
        if (ex[i] >= 0) atomicOr((unsigned long long*)&mask[ex[i]], 1ull << (i / a.k));
    __syncthreads();
    for (int i = tid; i < n; i += kRouteThreads) {
        const int e = ex[i], t = i / a.k;
        int s = -1;
        if (e >= 0) {
            s = base[e] + __builtin_popcountll(mask[e] & ((1ull << t) - 1));
            a.source[s] = (int32_t)(t0 + t);
        }
        a.slot[t0 * a.k + i] = s;
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += kRouteThreads) base[e] += __builtin_popcountll(mask[e]);
    __syncthreads();
}

// Exclusive sum of n <= 1024 values in LDS, by the first wave; returns the total in every lane
// of it.
__device__ __forceinline__ int exclusive(int* v, int n, int lane) {
    int run = 0;
    for (int b = 0; b < n; b += 64) {
        const int own = b + lane < n ? v[b + lane] : 0;
        int s = own;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(s, d);
            if (lane >= d) s += o;
        }
        if (b + lane < n) v[b + lane] = run + s - own;
        run += __shfl(s, 63);
    }
    return run;
}

// Choices and gates of a workgroup's tokens, and how many of them each expert got.  ONE: there
// is one workgroup, which places them too.
template <int DT, bool ONE>
__global__ void __launch_bounds__(kRouteThreads) route_choose(RouteArgs a) {
    __shared__ uint64_t mask[ONE ? kMaxExperts : 1];
    __shared__ int count[kMaxExperts];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < a.E; e += kRouteThreads) count[e] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * a.per, t1 = t0 + a.per < a.T ? t0 + a.per : a.T;
    for (int64_t t = t0 + wave; t < t1; t += kRouteThreads / 64) {
        int expert;
        float gate;
        choose_any<DT>(a, t, lane, expert, gate);
        if (lane < a.k) {
            a.expert[t * a.k + lane] = expert;
            a.gate[t * a.k + lane] = gate;
            if (expert >= 0) atomicAdd(&count[expert], 1);
        }
    }
    __syncthreads();   // orders this workgroup's writes of expert before its reads, too
    if constexpr (ONE) {
        if (wave == 0) {
            const int total = exclusive(count, a.E, lane);
            if (lane == 0) a.offsets[a.E] = total;
        }
        __syncthreads();
        for (int e = tid; e < a.E; e += kRouteThreads) a.offsets[e] = count[e];
        for (int64_t t = t0; t < t1; t += kBlock) place_block(a, t, mask, count);
    } else {
        for (int e = tid; e < a.E; e += kRouteThreads) a.count[(int64_t)blockIdx.x * a.E + e] = count[e];
    }
}

// Places: the groups' starts from all workgroups' counts, then a workgroup's own tokens.
__global__ void __launch_bounds__(kRouteThreads) route_place(RouteArgs a) {
    __shared__ uint64_t mask[kMaxExperts];
    __shared__ int all[kMaxExperts], base[kMaxExperts];
    const int tid = threadIdx.x, lane = tid & 63;
    for (int e = tid; e < a.E; e += kRouteThreads) all[e] = base[e] = 0;
    __syncthreads();
    // threads share the workgroups' counts of an expert; whole numbers, so in any order
    const int per = kRouteThreads / a.E > 0 ? kRouteThreads / a.E : 1;
    const int part = tid / a.E;
    if (part < per)
        for (int e = tid - part * a.E; e < a.E; e += kRouteThreads) {
            int s = 0, before = 0;
            for (int b = part; b < a.blocks; b += per) {
                const int c = a.count[(int64_t)b * a.E + e];
                s += c;
                if (b < (int)blockIdx.x) before += c;
            }
            if (s) atomicAdd(&all[e], s);
            if (before) atomicAdd(&base[e], before);
        }
    __syncthreads();
    if (tid < 64) {
        const int total = exclusive(all, a.E, lane);
        if (blockIdx.x == 0 && lane == 0) a.offsets[a.E] = total;
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += kRouteThreads) {
        if (blockIdx.x == 0) a.offsets[e] = all[e];
        base[e] += all[e];
    }
    const int64_t t0 = (int64_t)blockIdx.x * a.per, t1 = t0 + a.per < a.T ? t0 + a.per : a.T;
    for (int64_t t = t0; t < t1; t += kBlock) place_block(a, t, mask, base);
}

struct RouteBack {
    const char* logits;
    const int32_t* expert;
    const float* dgate;
    char* dlogits;
    int32_t T, E, k, renorm;
};

// One wave, one token: p again from the logits, d by expert.
template <int DT, int C>
__global__ void __launch_bounds__(256) route_back(RouteBack a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (t >= a.T) return;
    int e = lane < a.k ? a.expert[t * a.k + lane] : -1;
    if (e >= a.E) e = -1;
    const float d = e >= 0 ? a.dgate[t * a.k + lane] : 0.0f;
    float x[C], g[C];
    bool mine[C], nan = false;
    uint32_t top_key = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = c * 64 + lane;
        x[c] = i < a.E ? load1<DT>(a.logits, t * a.E + i) : -__builtin_inff();
        g[c] = 0.0f;
        mine[c] = false;
        nan |= x[c] != x[c];
        const uint32_t key = order_of(x[c]);
        top_key = key > top_key ? key : top_key;
    }
    for (int j = 0; j < a.k; ++j) {
        const int ej = __builtin_amdgcn_readlane(e, j);
        const float dj = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, d), j));
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (ej == c * 64 + lane) {
                g[c] = dj;
                mine[c] = true;
            }
    }
    const float top = value_of(wave_max(top_key));
    const bool some = __ballot(e >= 0) != 0;
    float all = 0.0f, inner = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const bool in = a.renorm ? mine[c] : x[c] != -__builtin_inff();
        x[c] = in ? expf(x[c] - top) : 0.0f;
        all += x[c];
        // not 0 * inf: a logit that was not chosen has no gradient of its own
        inner += mine[c] ? x[c] * g[c] : 0.0f;
    }
    all = __ballot(nan) ? __builtin_nanf("") : wave_sum(all);   // as the gates were
    inner = wave_sum(inner) / all;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = c * 64 + lane;
        if (i >= a.E) continue;
        const bool in = some && (a.renorm ? mine[c] : true);
        store1<DT>(a.dlogits, t * a.E + i, in ? x[c] / all * (g[c] - inner) : 0.0f);
    }
}

struct CombineArgs {
    const char *Y, *dout;
    const int32_t* slot;
    const float* gate;
    char *out, *dY;
    float* dgate;
    int64_t tokens, rows, N;
    int32_t k;
};

// One thread, 16 bytes of one token's row.
template <int DT>
__global__ void __launch_bounds__(256) combine_rows(CombineArgs a) {
    constexpr int E = Vec<DT>::E, EB = Vec<DT>::EB;
    const int64_t per = (a.N + E - 1) / E;
    const int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    const int64_t t = i / per, n = (i - t * per) * E;
    if (t >= a.tokens) return;
    float s[E] = {};
    // four rows' loads in flight; what a slot out of range would add is left out, not multiplied
    for (int j0 = 0; j0 < a.k; j0 += 4) {
        int64_t r[4];
        float g[4];
        u32x4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r[i] = j0 + i < a.k ? a.slot[t * a.k + j0 + i] : -1;
            g[i] = a.gate && j0 + i < a.k ? a.gate[t * a.k + j0 + i] : 1.0f;
            if (r[i] >= a.rows) r[i] = -1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (r[i] >= 0) v[i] = load_short<DT>(a.Y + r[i] * a.N * EB, n, a.N);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (r[i] >= 0)
#pragma unroll
                for (int e = 0; e < E; ++e) s[e] = __builtin_fmaf(g[i], elem<DT>(v[i], e), s[e]);
    }
    store_vec<DT>(a.out + t * a.N * EB, n, a.N, s);
}

// One workgroup, one token: its rows of dY, then the dot products.
template <int DT>
__global__ void __launch_bounds__(256) combine_back(CombineArgs a) {
    constexpr int E = Vec<DT>::E, EB = Vec<DT>::EB;
    __shared__ float lds[4];
    const int64_t t = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (t >= a.tokens) return;
    const char* d = a.dout + t * a.N * EB;
    for (int j = 0; j < a.k; ++j) {
        const int64_t r = a.slot[t * a.k + j];
        const bool in = r >= 0 && r < a.rows;
        const float g = a.gate && in ? a.gate[t * a.k + j] : 1.0f;
        float dot = 0.0f;
        if (in)
            for (int64_t n = threadIdx.x * E; n < a.N; n += 256 * E) {
                const u32x4 v = load_short<DT>(d, n, a.N);
                float o[E];
                if (a.dgate) {
                    const u32x4 y = load_short<DT>(a.Y + r * a.N * EB, n, a.N);
#pragma unroll
                    for (int e = 0; e < E; ++e) dot = __builtin_fmaf(elem<DT>(v, e), elem<DT>(y, e), dot);
                }
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = g * elem<DT>(v, e);
                store_vec<DT>(a.dY + r * a.N * EB, n, a.N, o);
            }
        if (a.dgate) {
            dot = wave_sum(dot);
            if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = dot;
            __syncthreads();
            if (threadIdx.x == 0) a.dgate[t * a.k + j] = lds[0] + lds[1] + lds[2] + lds[3];
            __syncthreads();
        }
    }
}

gemm_status launched() {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? GEMM_OK : hip_fail(e);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// a launch has less than 2^32 threads along one axis
dim3 spread(int64_t wgs) {
    const int64_t x = std::min<int64_t>(wgs, 1 << 21);
    return dim3((unsigned)x, (unsigned)ceil_div(wgs, x));
}

// f(element type as a constant)
template <typename F>
void with_type(int dt, F&& f) {
    if (dt == GEMM_F16) f(std::integral_constant<int, kOutF16>{});
    else if (dt == GEMM_BF16) f(std::integral_constant<int, kOutBF16>{});
    else f(std::integral_constant<int, kOutF32>{});
}

bool known(gemm_dtype t) { return t == GEMM_F16 || t == GEMM_BF16 || t == GEMM_F32; }

}  // namespace
}  // namespace spg

struct gemm_route_plan {
    int64_t T, E, k;
    int dt, renorm;
    int64_t per, blocks;
};

struct gemm_combine_plan {
    int64_t tokens, k, rows, N;
    int dt;
};

extern "C" {

gemm_status gemm_route_create(gemm_route_handle* out, int64_t tokens, int64_t experts, int64_t k, gemm_dtype dtype,
                              int32_t renormalise) {
    if (!out) return GEMM_ERR_INVALID_ARG;
    *out = nullptr;
    if (tokens < 0 || experts < 1 || k < 1 || k > experts || k > spg::kMaxChoices || !spg::known(dtype) ||
        (renormalise != 0 && renormalise != 1))
        return GEMM_ERR_INVALID_ARG;
    const int64_t lim = (int64_t)1 << 30;
    if (experts > spg::kMaxExperts || tokens > lim / experts || tokens > lim / k) return GEMM_ERR_UNSUPPORTED;
    gemm_route_plan* p = new (std::nothrow) gemm_route_plan{tokens, experts, k, (int)dtype, renormalise, 0, 0};
    if (!p) return GEMM_ERR_OUT_OF_MEMORY;
    const int64_t masks = spg::ceil_div(tokens, spg::kBlock);
    p->per = spg::kBlock * std::max<int64_t>(1, spg::ceil_div(masks, spg::kMaxBlocks));
    p->blocks = spg::ceil_div(tokens, p->per);
    *out = p;
    return GEMM_OK;
}

int64_t gemm_route_workspace(gemm_route_handle h) { return !h ? -1 : h->blocks > 1 ? h->blocks * h->E * 4 : 0; }

gemm_status gemm_route_run(gemm_route_handle h, const void* logits, float* gate, int32_t* expert, int32_t* slot,
                           int32_t* source, int32_t* offsets, void* workspace, int64_t workspace_bytes,
                           hipStream_t stream) {
    if (!h || !offsets) return GEMM_ERR_INVALID_ARG;
    if (h->T > 0 && (!logits || !gate || !expert || !slot || !source)) return GEMM_ERR_INVALID_ARG;
    const int64_t need = gemm_route_workspace(h);
    if (need > 0 && (!workspace || (uintptr_t)workspace % 16 != 0 || workspace_bytes < need)) return GEMM_ERR_INVALID_ARG;
    const spg::RouteArgs a{(const char*)logits, gate, expert, slot, source, offsets, (int32_t*)workspace,
                           (int32_t)h->T, (int32_t)h->E, (int32_t)h->k, (int32_t)h->per, (int32_t)h->blocks, h->renorm};
    const dim3 wg(spg::kRouteThreads);
    spg::with_type(h->dt, [&](auto dt) {
        constexpr int D = decltype(dt)::value;
        if (h->blocks <= 1) {   // no tokens: the offsets of empty groups
            hipLaunchKernelGGL((spg::route_choose<D, true>), dim3(1), wg, 0, stream, a);
        } else {
            hipLaunchKernelGGL((spg::route_choose<D, false>), dim3((unsigned)h->blocks), wg, 0, stream, a);
            hipLaunchKernelGGL(spg::route_place, dim3((unsigned)h->blocks), wg, 0, stream, a);
        }
    });
    return spg::launched();
}

gemm_status gemm_route_backward(gemm_route_handle h, const void* logits, const int32_t* expert, const float* dgate,
                                void* dlogits, hipStream_t stream) {
    if (!h) return GEMM_ERR_INVALID_ARG;
    if (h->T == 0) return GEMM_OK;
    if (!logits || !expert || !dgate || !dlogits) return GEMM_ERR_INVALID_ARG;
    const spg::RouteBack a{(const char*)logits, expert, dgate, (char*)dlogits, (int32_t)h->T, (int32_t)h->E, (int32_t)h->k, h->renorm};
    const dim3 grid = spg::spread(spg::ceil_div(h->T, 4)), wg(256);
    spg::with_type(h->dt, [&](auto dt) {
        constexpr int D = decltype(dt)::value;
        if (h->E <= 64) hipLaunchKernelGGL((spg::route_back<D, 1>), grid, wg, 0, stream, a);
        else if (h->E <= 128) hipLaunchKernelGGL((spg::route_back<D, 2>), grid, wg, 0, stream, a);
        else if (h->E <= 256) hipLaunchKernelGGL((spg::route_back<D, 4>), grid, wg, 0, stream, a);
        else hipLaunchKernelGGL((spg::route_back<D, spg::kMaxExperts / 64>), grid, wg, 0, stream, a);
    });
    return spg::launched();
}

gemm_status gemm_route_destroy(gemm_route_handle h) {
    delete h;
    return GEMM_OK;
}

gemm_status gemm_combine_create(gemm_combine_handle* out, int64_t tokens, int64_t k, int64_t rows, int64_t N,
                                gemm_dtype dtype) {
    if (!out) return GEMM_ERR_INVALID_ARG;
    *out = nullptr;
    if (tokens < 0 || rows < 0 || N < 0 || k < 1 || k > spg::kMaxChoices || !spg::known(dtype)) return GEMM_ERR_INVALID_ARG;
    const int64_t lim = INT32_MAX / 2 - 512;
    if (tokens > lim / k || rows > lim || N > lim) return GEMM_ERR_UNSUPPORTED;
    gemm_combine_plan* p = new (std::nothrow) gemm_combine_plan{tokens, k, rows, N, (int)dtype};
    if (!p) return GEMM_ERR_OUT_OF_MEMORY;
    *out = p;
    return GEMM_OK;
}

gemm_status gemm_combine_run(gemm_combine_handle h, const void* Y, const int32_t* slot, const float* gate, void* out,
                             hipStream_t stream) {
    if (!h) return GEMM_ERR_INVALID_ARG;
    if (h->tokens == 0 || h->N == 0) return GEMM_OK;
    if (!slot || !out || (h->rows > 0 && !Y)) return GEMM_ERR_INVALID_ARG;
    spg::CombineArgs a{};
    a.Y = (const char*)Y;
    a.slot = slot;
    a.gate = gate;
    a.out = (char*)out;
    a.tokens = h->tokens;
    a.rows = h->rows;
    a.N = h->N;
    a.k = (int32_t)h->k;
    spg::with_type(h->dt, [&](auto dt) {
        constexpr int D = decltype(dt)::value;
        const int64_t items = h->tokens * spg::ceil_div(h->N, spg::Vec<D>::E);
        hipLaunchKernelGGL((spg::combine_rows<D>), spg::spread(spg::ceil_div(items, 256)), dim3(256), 0, stream, a);
    });
    return spg::launched();
}

gemm_status gemm_combine_backward(gemm_combine_handle h, const void* dout, const void* Y, const int32_t* slot,
                                  const float* gate, void* dY, float* dgate, hipStream_t stream) {
    if (!h) return GEMM_ERR_INVALID_ARG;
    if (h->tokens == 0 || (h->N == 0 && !dgate)) return GEMM_OK;
    if (!slot || (h->N > 0 && (!dout || (h->rows > 0 && (!dY || (dgate && !Y)))))) return GEMM_ERR_INVALID_ARG;
    spg::CombineArgs a{};
    a.Y = (const char*)Y;
    a.dout = (const char*)dout;
    a.slot = slot;
    a.gate = gate;
    a.dY = (char*)dY;
    a.dgate = dgate;
    a.tokens = h->tokens;
    a.rows = h->rows;
    a.N = h->N;
    a.k = (int32_t)h->k;
    spg::with_type(h->dt, [&](auto dt) {
        hipLaunchKernelGGL((spg::combine_back<decltype(dt)::value>), spg::spread(h->tokens), dim3(256), 0, stream, a);
    });
    return spg::launched();
}

gemm_status gemm_combine_destroy(gemm_combine_handle h) {
    delete h;
    return GEMM_OK;
}

}  // extern "C"
