// 16-byte vectors of a row at any element alignment, widened to fp32: what the row operators
// (layer norm, combination, routing) read and write.
#pragma once

#include "gemm_kernels.hpp"

namespace spg {

// An element type's vector: E elements of EB bytes.
template <int DT>
struct Vec {
    static constexpr int EB = DT == kOutF32 ? 4 : 2, E = 16 / EB;
};

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    if constexpr (DT == kOutF32) return ((const float*)p)[i];
    else return bits_to_f32(((const uint16_t*)p)[i], DT == kOutBF16);
}

template <int DT>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
    if constexpr (DT == kOutF32) ((float*)p)[i] = v;
    else ((uint16_t*)p)[i] = f32_to_bits(v, DT == kOutBF16);
}

// Element e of a loaded vector.
template <int DT>
__device__ __forceinline__ float elem(const u32x4& v, int e) {
    if constexpr (DT == kOutF32) {
        const uint32_t b = v[e];
        return __builtin_bit_cast(float, b);
    } else {
        return bits_to_f32((uint16_t)(v[e >> 1] >> ((e & 1) * 16)), DT == kOutBF16);
    }
}

// Vector `at` (elements, below n) of a row of n >= E: what lies past the row's end is not read,
// and zero (the 16 bytes that end there, shifted down).
template <int DT>
__device__ __forceinline__ u32x4 load_vec(const void* row, int64_t at, int64_t n) {
    constexpr int E = Vec<DT>::E, EB = Vec<DT>::EB;
    struct __attribute__((packed, aligned(EB))) B { u32x4 v; };
    const int64_t over = at + E - n;
    u32x4 v = ((const B*)((const char*)row + (over > 0 ? n - E : at) * EB))->v;
    if (over > 0) v = shr128(v, 8u * EB * (uint32_t)over);
    return v;
}

// ... of a row of any length
template <int DT>
__device__ __forceinline__ u32x4 load_short(const void* row, int64_t at, int64_t n) {
    constexpr int E = Vec<DT>::E, EB = Vec<DT>::EB;
    if (n >= E) return load_vec<DT>(row, at, n);
    const char* p = (const char*)row + at * EB;
    u32x4 r = {};
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (at + e < n) {
            if constexpr (EB == 4) r[e] = ((const uint32_t*)p)[e];
            else r[e >> 1] |= (uint32_t)((const uint16_t*)p)[e] << ((e & 1) * 16);
        }
    return r;
}

template <int DT>
__device__ __forceinline__ u32x4 pack_vec(const float (&x)[Vec<DT>::E]) {
    u32x4 r = {};
#pragma unroll
    for (int e = 0; e < Vec<DT>::E; ++e) {
        if constexpr (DT == kOutF32) r[e] = __builtin_bit_cast(uint32_t, x[e]);
        else r[e >> 1] |= (uint32_t)f32_to_bits(x[e], DT == kOutBF16) << ((e & 1) * 16);
    }
    return r;
}

// The inverse of load_vec: nothing past the row's end is written.
template <int DT>
__device__ __forceinline__ void store_vec(void* row, int64_t at, int64_t n, const float (&x)[Vec<DT>::E]) {
    constexpr int E = Vec<DT>::E, EB = Vec<DT>::EB;
    char* p = (char*)row + at * EB;
    const u32x4 v = pack_vec<DT>(x);
    struct __attribute__((packed, aligned(EB))) B { u32x4 v; };
    if (at + E <= n) {
        ((B*)p)->v = v;
        return;
    }
    // the last 1 to E - 1 elements in up to three stores
    const int left = (int)(n - at);
    struct __attribute__((packed, aligned(EB))) B8 { u32x2 v; };
    struct __attribute__((packed, aligned(EB))) B4 { uint32_t v; };
    u32x4 t = v;
    if (left * EB & 8) {
        ((B8*)p)->v = u32x2{t.x, t.y};
        t = u32x4{t.z, t.w, 0u, 0u};
        p += 8;
    }
    if (left * EB & 4) {
        ((B4*)p)->v = t.x;
        t.x = t.y;
        p += 4;
    }
    if (left * EB & 2) *(uint16_t*)p = (uint16_t)t.x;
}

// Sum over the 64 lanes of a wave, in every lane (a scalar), in a fixed order: shifts within rows
// of 16 lanes, then the rows' ends, without a trip through LDS.
__device__ __forceinline__ float wave_sum(float v) {
    auto add = [&](auto ctrl, auto rows) {
        v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value,
                                                                   decltype(rows)::value, 0xf, false));
    };
    using std::integral_constant;
    constexpr integral_constant<int, 0xf> all{};
    add(integral_constant<int, 0x111>{}, all);   // row_shr:1
    add(integral_constant<int, 0x112>{}, all);   // row_shr:2
    add(integral_constant<int, 0x114>{}, all);   // row_shr:4
    add(integral_constant<int, 0x118>{}, all);   // row_shr:8
    add(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});   // row_bcast:15
    add(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});   // row_bcast:31
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

}  // namespace spg
