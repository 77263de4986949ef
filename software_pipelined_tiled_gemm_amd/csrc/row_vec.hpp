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

// Vector `at` (elements) of a row of `n`: what lies past the row's end is not read, and zero.
template <int DT>
__device__ __forceinline__ u32x4 load_vec(const void* row, int64_t at, int64_t n) {
    constexpr int E = Vec<DT>::E, EB = Vec<DT>::EB;
    const char* p = (const char*)row + at * EB;
    struct __attribute__((packed, aligned(EB))) B { u32x4 v; };
    if (at + E <= n) return ((const B*)p)->v;
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
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (at + e < n) {
            if constexpr (EB == 4) ((uint32_t*)p)[e] = v[e];
            else ((uint16_t*)p)[e] = (uint16_t)(v[e >> 1] >> ((e & 1) * 16));
        }
}

// Sum over the 64 lanes of a wave, in every lane, in a fixed order.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
    return v;
}

}  // namespace spg
