// Element types of the operators around the expert layer: fp32, fp16 and bf16
// rows, loaded as fp32 and rounded to the nearest (even) when stored.
#pragma once

#include "moeq8_device.hpp"

namespace moeq8 {

struct bf16_t { uint16_t bits; };
struct f16_t { uint16_t bits; };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(f16_t v) { return half_bits_to_float(v.bits); }
__device__ __forceinline__ float to_f32(bf16_t v) { return __uint_as_float((uint32_t)v.bits << 16); }

__device__ __forceinline__ void from_f32(float& o, float v) { o = v; }
__device__ __forceinline__ void from_f32(f16_t& o, float v) {
    // the pin keeps the fp32 rounding of v's own operation apart from this one
    o.bits = (uint16_t)float_to_half_bits(materialize_f32(v));
}
__device__ __forceinline__ void from_f32(bf16_t& o, float v) {
    o.bits = __builtin_bit_cast(unsigned short, (__bf16)v);
}

// N consecutive elements at any address their type allows, as dword vectors.
// Rows of an odd length start off 16 bytes; gfx950 global memory takes such
// vectors whole, so one instruction serves every row.
typedef uint32_t u32x4b __attribute__((ext_vector_type(4), aligned(1), may_alias));
typedef uint32_t u32x2b __attribute__((ext_vector_type(2), aligned(1), may_alias));

template <typename T, int N>
__device__ __forceinline__ void load_vec(T (&v)[N], const T* p) {
    static_assert(sizeof(T) * N % 16 == 0, "whole 16-byte vectors");
    union { u32x4b u[sizeof(T) * N / 16]; T e[N]; } t;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) * N / 16); ++i) t.u[i] = reinterpret_cast<const u32x4b*>(p)[i];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = t.e[i];
}

// LATER: nontemporal, for what is not read again soon.
template <bool LATER = false, typename T, int N>
__device__ __forceinline__ void store_vec(T* p, const T (&v)[N]) {
    static_assert(sizeof(T) * N % 16 == 0, "whole 16-byte vectors");
    union { u32x4b u[sizeof(T) * N / 16]; T e[N]; } t;
#pragma unroll
    for (int i = 0; i < N; ++i) t.e[i] = v[i];
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) * N / 16); ++i) {
        if constexpr (LATER) __builtin_nontemporal_store(t.u[i], reinterpret_cast<u32x4b*>(p) + i);
        else reinterpret_cast<u32x4b*>(p)[i] = t.u[i];
    }
}

}  // namespace moeq8
