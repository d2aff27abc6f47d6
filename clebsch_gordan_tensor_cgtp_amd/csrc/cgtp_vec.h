// cgtp_vec.h -- vectors of fp32 or bf16 elements in memory, fp32 in registers
// (device code of the node-side operators).
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace cgtp {

struct bf16_t {
    uint16_t bits;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return __uint_as_float((uint32_t)v.bits << 16); }

template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v)
{
    return v;
}
// round to nearest even (the hardware conversion)
template <>
__device__ __forceinline__ bf16_t from_f32<bf16_t>(float v)
{
    return bf16_t{__builtin_bit_cast(uint16_t, (__bf16)v)};
}

// from fp64 in one rounding (through fp32 a bf16 could be off by the second)
template <class T>
__device__ __forceinline__ T from_f64(double v);
template <>
__device__ __forceinline__ float from_f64<float>(double v)
{
    return (float)v;
}
template <>
__device__ __forceinline__ bf16_t from_f64<bf16_t>(double v)
{
    return bf16_t{__builtin_bit_cast(uint16_t, (__bf16)v)};
}

// elements of one 16-byte access
template <class T>
constexpr int kWide = 16 / (int)sizeof(T);

// VEC consecutive elements in one access, aligned to its size
template <class T, int VEC>
__device__ __forceinline__ void load_vec(float (&v)[VEC], const T* __restrict__ p)
{
    if constexpr (VEC == 1) {
        v[0] = to_f32(p[0]);
    } else {
        struct alignas(VEC * sizeof(T)) Pack {
            T e[VEC];
        };
        const Pack q = *reinterpret_cast<const Pack*>(p);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = to_f32(q.e[j]);
    }
}

// V: float, or double for sums that are rounded here
template <class T, int VEC, class V>
__device__ __forceinline__ void store_vec(T* __restrict__ p, const V (&v)[VEC])
{
    auto round = [](V x) {
        if constexpr (sizeof(V) == 8) return from_f64<T>(x);
        else return from_f32<T>(x);
    };
    if constexpr (VEC == 1) {
        p[0] = round(v[0]);
    } else {
        struct alignas(VEC * sizeof(T)) Pack {
            T e[VEC];
        } q;
#pragma unroll
        for (int j = 0; j < VEC; ++j) q.e[j] = round(v[j]);
        *reinterpret_cast<Pack*>(p) = q;
    }
}

// the same as bits, converted where used: half the registers for bf16
template <class T, int VEC>
struct alignas(VEC * sizeof(T)) Raw {
    T e[VEC];
    __device__ __forceinline__ void load(const T* __restrict__ p) { *this = *reinterpret_cast<const Raw*>(p); }
    __device__ __forceinline__ float operator[](int j) const { return to_f32(e[j]); }
};

// whether rows of `elem`-byte elements, ld apart, all begin on `bytes` bytes
inline bool aligned_rows(const void* p, int64_t ld, int64_t elem, int64_t bytes = 16)
{
    return (uintptr_t)p % (uintptr_t)bytes == 0 && ld * elem % bytes == 0;
}

}  // namespace cgtp
