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
#include "wave_scan.hpp"

namespace spg {
namespace {

constexpr int kMaxExperts = 1024, kMaxChoices = 64;
constexpr int kRouteThreads = 1024;
constexpr int kBlock = 64;          // tokens of a mask
constexpr int kSimds = 1024;        // 256 CUs of 4
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

__device__ __forceinline__ float value_of(uint32_t key) {
    return __builtin_bit_cast(float, key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// A token's logits lie in L lanes, C one after the other in each: 16 lanes up to 256 experts, so
// that a wave takes four tokens at once, else all 64.  What the lanes of a token share goes through
// DPP, a dependent instruction a step instead of a trip through LDS.  16384 tokens, 8 of 64 experts:
// the choices take 6.5 us, 11.9 with a wave a token and a logit a lane, 16.2 with that
// through LDS; their number of instructions is what takes the time.
template <int L, typename F>
__device__ __forceinline__ int over_lanes(int v, F&& join) {
    static_assert(L == 16 || L == 64, "lanes of a token");
    auto step = [&](auto ctrl, auto rows) {
        v = join(v, __builtin_amdgcn_update_dpp(0, v, decltype(ctrl)::value, decltype(rows)::value, 0xf, false));
    };
    using std::integral_constant;
    constexpr integral_constant<int, 0xf> all{};
    step(integral_constant<int, 0x128>{}, all);   // row_ror:8
    step(integral_constant<int, 0x124>{}, all);
    step(integral_constant<int, 0x122>{}, all);
    step(integral_constant<int, 0x121>{}, all);
    if constexpr (L == 64) {
        const int a = join(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16));
        v = join(a, join(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
    }
    return v;
}
template <int L>
__device__ __forceinline__ uint32_t most_of(uint32_t v) {
    return (uint32_t)over_lanes<L>((int)v, [](int a, int b) { return (int)((uint32_t)a > (uint32_t)b ? a : b); });
}
// in a fixed order, the same in every lane
template <int L>
__device__ __forceinline__ float sum_of(float v) {
    return __builtin_bit_cast(float, over_lanes<L>(__builtin_bit_cast(int, v), [](int a, int b) {
        return __builtin_bit_cast(int, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
    }));
}
// the token's lanes in which `b` holds, as bits
template <int L>
__device__ __forceinline__ uint64_t lanes_of(bool b, int lane) {
    const uint64_t m = __ballot(b);
    if constexpr (L == 64) return m;
    return ((lane & 32 ? (uint32_t)(m >> 32) : (uint32_t)m) >> (lane & 16)) & 0xffffu;
}

// The largest and the sum of a lane's own, in pairs.
template <int C>
__device__ __forceinline__ uint32_t most_own(const uint32_t (&v)[C]) {
    uint32_t r[C];
#pragma unroll
    for (int c = 0; c < C; ++c) r[c] = v[c];
#pragma unroll
    for (int d = C / 2; d; d /= 2)
#pragma unroll
        for (int c = 0; c < d; ++c) r[c] = r[c + d] > r[c] ? r[c + d] : r[c];
    return r[0];
}
template <int C>
__device__ __forceinline__ float sum_own(const float (&v)[C]) {
    float r[C];
#pragma unroll
    for (int c = 0; c < C; ++c) r[c] = v[c];
#pragma unroll
    for (int d = C / 2; d; d /= 2)
#pragma unroll
        for (int c = 0; c < d; ++c) r[c] += r[c + d];
    return r[0];
}

// Logits e0 .. e0 + C - 1 of a row of E; -inf past its end.
template <int DT, int C>
__device__ __forceinline__ void load_own(const char* row, int e0, int E, float (&x)[C]) {
    constexpr int EB = Vec<DT>::EB;
    if constexpr (C * EB >= 8) {
        if (e0 + C <= E) {
            struct __attribute__((packed, aligned(EB))) W { uint32_t w[C * EB / 4]; };
            const W r = *(const W*)(row + e0 * EB);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if constexpr (EB == 4) x[c] = __builtin_bit_cast(float, r.w[c]);
                else x[c] = bits_to_f32((uint16_t)(r.w[c >> 1] >> ((c & 1) * 16)), DT == kOutBF16);
            }
            return;
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = e0 + c < E ? load1<DT>(row, e0 + c) : -__builtin_inff();
}
template <int DT, int C>
__device__ __forceinline__ void store_own(char* row, int e0, int E, const float (&x)[C]) {
    constexpr int EB = Vec<DT>::EB;
    if constexpr (C * EB >= 8) {
        if (e0 + C <= E) {
            struct __attribute__((packed, aligned(EB))) W { uint32_t w[C * EB / 4]; };
            W r = {};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if constexpr (EB == 4) r.w[c] = __builtin_bit_cast(uint32_t, x[c]);
                else r.w[c >> 1] |= (uint32_t)f32_to_bits(x[c], DT == kOutBF16) << ((c & 1) * 16);
            }
            *(W*)(row + e0 * EB) = r;
            return;
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (e0 + c < E) store1<DT>(row, e0 + c, x[c]);
}

// f(lanes of a token, logits of a lane), as constants; wide: so few tokens that each has a wave of
// its own at once, and fewer logits a lane are what is faster
template <typename F>
__host__ __device__ __forceinline__ void with_lanes(int E, bool wide, F&& f) {
    using std::integral_constant;
    constexpr integral_constant<int, 16> row{};
    constexpr integral_constant<int, 64> wave{};
    if (E > 512) f(wave, integral_constant<int, kMaxExperts / 64>{});
    else if (E > 256) f(wave, integral_constant<int, 8>{});
    else if (wide && E <= 64) f(wave, integral_constant<int, 1>{});
    else if (wide) f(wave, integral_constant<int, 4>{});
    else if (E <= 16) f(row, integral_constant<int, 1>{});
    else if (E <= 64) f(row, integral_constant<int, 4>{});
    else if (E <= 128) f(row, integral_constant<int, 8>{});
    else f(row, integral_constant<int, 16>{});
}

// Token t (in: there is one) of L lanes: its k largest logits one by one, their gates, and one
// more for each of their experts in `count`.
template <int DT, int L, int C>
__device__ __forceinline__ void choose(const RouteArgs& a, int64_t t, bool in, int lane, int* count) {
    const int own = lane & (L - 1), e0 = own * C;
    float x[C];
    uint32_t key[C];
    int rank[C];
    load_own<DT, C>(a.logits + t * a.E * Vec<DT>::EB, e0, in ? a.E : 0, x);
    bool nan = false;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        key[c] = order_of(x[c]);
        rank[c] = -1;
        nan |= x[c] != x[c];
    }
    nan = lanes_of<L>(nan, lane) != 0;
    int chosen = 0;
    float top = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        const uint32_t mine = most_own(key), best = most_of<L>(mine);
        const bool live = best > kNothing;
        if (!__ballot(live)) break;
        // the lowest index among equals: the first lane, then its first logit
        const uint64_t at = lanes_of<L>(mine == best, lane);
        bool take = live && own == (L == 64 ? __builtin_ctzll(at) : __builtin_ctz((uint32_t)at));
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const bool it = take && key[c] == best;
            key[c] = it ? 0u : key[c];
            rank[c] = it ? j : rank[c];
            take = take && !it;
        }
        if (j == 0 && live) top = value_of(best);
        chosen += live;
    }
    // softmax over the chosen, or over all; expf to the last bit or two: gates are fp32
    float p[C];
#pragma unroll
    for (int c = 0; c < C; ++c) p[c] = (a.renorm ? rank[c] >= 0 : x[c] != -__builtin_inff()) ? expf(x[c] - top) : 0.0f;
    const float all = sum_of<L>(sum_own(p));
    if (!in) return;
    int32_t* expert = a.expert + t * a.k;
    float* gate = a.gate + t * a.k;
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (rank[c] >= 0) {
            expert[rank[c]] = e0 + c;
            gate[rank[c]] = nan ? __builtin_nanf("") : p[c] / all;
            atomicAdd(&count[e0 + c], 1);
        }
    for (int j = chosen + own; j < a.k; j += L) {
        expert[j] = -1;
        gate[j] = 0.0f;
    }
}

// This thread's first expert of the 64 tokens from t0.
__device__ __forceinline__ int first_pair(const RouteArgs& a, int64_t t0) {
    const int64_t left = (int64_t)a.T - t0;
    return (int)threadIdx.x < (int)(left < kBlock ? left : kBlock) * a.k ? a.expert[t0 * a.k + threadIdx.x] : -1;
}

// The places of the pairs of 64 tokens from t0: base[e] is where expert e's go on; first: as above.
__device__ __forceinline__ void place_block(const RouteArgs& a, int64_t t0, int first, uint64_t* mask, int* base) {
    const int tid = threadIdx.x;
    const int64_t left = (int64_t)a.T - t0;
    const int n = (int)(left < kBlock ? left : kBlock) * a.k;
    const int32_t* ex = a.expert + t0 * a.k;
    for (int e = tid; e < a.E; e += kRouteThreads) mask[e] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kRouteThreads) {
        const int e = i == tid ? first : ex[i];
        if (e >= 0) atomicOr((unsigned long long*)&mask[e], 1ull << (i / a.k));
    }
    __syncthreads();
    for (int i = tid; i < n; i += kRouteThreads) {
        const int e = i == tid ? first : ex[i], t = i / a.k;
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
        const int own = b + lane < n ? v[b + lane] : 0, upto = wave_scan(own);
        if (b + lane < n) v[b + lane] = run + upto - own;
        run += __builtin_amdgcn_readlane(upto, 63);
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
    with_lanes(a.E, ONE && a.T <= kRouteThreads / 64, [&](auto l, auto c) {
        constexpr int L = decltype(l)::value, TW = 64 / L;   // tokens of a wave
        for (int64_t t = t0 + wave * TW; t < t1; t += kRouteThreads / L) {
            const int64_t own = t + lane / L;
            choose<DT, L, decltype(c)::value>(a, own < t1 ? own : t, own < t1, lane, count);
        }
    });
    __syncthreads();   // orders this workgroup's writes of expert before its reads, too
    if constexpr (ONE) {
        if (wave == 0) {
            const int total = exclusive(count, a.E, lane);
            if (lane == 0) a.offsets[a.E] = total;
        }
        __syncthreads();
        for (int e = tid; e < a.E; e += kRouteThreads) a.offsets[e] = count[e];
        for (int64_t t = t0; t < t1; t += kBlock) place_block(a, t, first_pair(a, t), mask, count);
    } else {
        for (int e = tid; e < a.E; e += kRouteThreads) a.count[(int64_t)blockIdx.x * a.E + e] = count[e];
    }
}

// Places: the groups' starts from all workgroups' counts, then a workgroup's own tokens.
__global__ void __launch_bounds__(kRouteThreads) route_place(RouteArgs a) {
    __shared__ uint64_t mask[kMaxExperts];
    __shared__ int all[kMaxExperts], base[kMaxExperts];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t t0 = (int64_t)blockIdx.x * a.per, t1 = t0 + a.per < a.T ? t0 + a.per : a.T;
    const int first = first_pair(a, t0);   // under way while the counts are summed
    for (int e = tid; e < a.E; e += kRouteThreads) all[e] = base[e] = 0;
    __syncthreads();
    // threads share the workgroups' counts of an expert; whole numbers, so in any order
    const int per = kRouteThreads / a.E > 0 ? kRouteThreads / a.E : 1;
    const int part = tid / a.E;
    if (part < per)
        for (int e = tid - part * a.E; e < a.E; e += kRouteThreads) {
            int s = 0, before = 0;
            // eight loads under way at once: one by one their latencies are most of this kernel
            // (16384 tokens, 64 experts: 5.2 us, 7.9 one by one)
            for (int b0 = part; b0 < a.blocks; b0 += 8 * per) {
                int c[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int b = b0 + u * per;
                    c[u] = a.count[(int64_t)(b < a.blocks ? b : a.blocks - 1) * a.E + e];
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int b = b0 + u * per;
                    s += b < a.blocks ? c[u] : 0;
                    before += b < (int)blockIdx.x ? c[u] : 0;
                }
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
    for (int64_t t = t0; t < t1; t += kBlock) place_block(a, t, t == t0 ? first : first_pair(a, t), mask, base);
}

struct RouteBack {
    const char* logits;
    const int32_t* expert;
    const float* dgate;
    char* dlogits;
    int32_t T, E, k, renorm;
};

// p again from the logits, d by expert; lanes as in choose().
template <int DT, int L, int C>
__global__ void __launch_bounds__(256) route_back(RouteBack a) {
    const int lane = threadIdx.x & 63, e0 = (lane & (L - 1)) * C;
    const int64_t own = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (256 / L) + threadIdx.x / L;
    const int64_t t = own < a.T ? own : a.T - 1;   // nothing is stored for it
    float x[C], g[C], s[C];
    uint32_t key[C];
    uint32_t mine = 0;   // a bit a logit: chosen
    bool nan = false, some = false;
    load_own<DT, C>(a.logits + t * a.E * Vec<DT>::EB, e0, a.E, x);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        g[c] = 0.0f;
        nan |= x[c] != x[c];
        key[c] = order_of(x[c]);
    }
#pragma unroll 4
    for (int j = 0; j < a.k; ++j) {
        const int e = a.expert[t * a.k + j];
        const float d = a.dgate[t * a.k + j];
        const bool is = e >= 0 && e < a.E;
        some |= is;
        const int at = is ? e - e0 : -1;
        if (at >= 0 && at < C) mine |= 1u << at;
#pragma unroll
        for (int c = 0; c < C; ++c) g[c] = at == c ? d : g[c];
    }
    const float top = value_of(most_of<L>(most_own(key)));
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const bool in = a.renorm ? mine >> c & 1 : x[c] != -__builtin_inff();
        x[c] = in ? expf(x[c] - top) : 0.0f;
        // not 0 * inf: a logit that was not chosen has no gradient of its own
        s[c] = mine >> c & 1 ? x[c] * g[c] : 0.0f;
    }
    const float sum = sum_of<L>(sum_own(x));
    const float all = lanes_of<L>(nan, lane) ? __builtin_nanf("") : sum;   // as the gates were
    const float inner = sum_of<L>(sum_own(s)) / all;
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] = some && (!a.renorm || (mine >> c & 1)) ? x[c] / all * (g[c] - inner) : 0.0f;
    if (own < a.T) store_own<DT, C>(a.dlogits + t * a.E * Vec<DT>::EB, e0, a.E, s);
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

// a launch has less than 2^32 threads along one axis, and one workgroup at least
dim3 spread(int64_t wgs) {
    const int64_t x = std::min<int64_t>(std::max<int64_t>(wgs, 1), 1 << 21);
    return dim3((unsigned)x, (unsigned)std::max<int64_t>(ceil_div(wgs, x), 1));
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
    spg::with_type(h->dt, [&](auto dt) {
        spg::with_lanes((int)h->E, h->T <= spg::kSimds, [&](auto l, auto c) {
            constexpr int L = decltype(l)::value;
            hipLaunchKernelGGL((spg::route_back<decltype(dt)::value, L, decltype(c)::value>),
                               spg::spread(spg::ceil_div(h->T, 256 / L)), dim3(256), 0, stream, a);
        });
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
