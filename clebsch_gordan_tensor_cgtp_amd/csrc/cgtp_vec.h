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

// sixteen bytes at any address that an element may have (the hardware takes 16-byte accesses anywhere)
template <class T>
struct __attribute__((packed, aligned(sizeof(T)))) Any16 {
    uint32_t w[4];
};

template <class T>
__device__ __forceinline__ uint4 load16(const T* p)
{
    return __builtin_bit_cast(uint4, *reinterpret_cast<const Any16<T>*>(p));
}

template <class T>
__device__ __forceinline__ void store16(T* p, uint4 v)
{
    *reinterpret_cast<Any16<T>*>(p) = __builtin_bit_cast(Any16<T>, v);
}

// the same as bits, converted where used: half the registers for bf16
template <class T, int VEC>
struct alignas(VEC * sizeof(T)) Raw {
    T e[VEC];
    __device__ __forceinline__ void load(const T* __restrict__ p) { *this = *reinterpret_cast<const Raw*>(p); }
    __device__ __forceinline__ float operator[](int j) const { return to_f32(e[j]); }
};

// eight elements of a row as they lie in memory
template <class T>
struct Raw8 {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ float operator[](int j) const
    {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
        return __uint_as_float(j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = uint4{0, 0, 0, 0};
    }
    __device__ __forceinline__ void load(const T* p)
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = load16(p + i * kWide<T>);
    }
    // the first n elements
    __device__ __forceinline__ void load_some(const T* p, int n)
    {
        if (n == 8) {
            load(p);
            return;
        }
        clear();
        T* e = reinterpret_cast<T*>(v);
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < n) e[j] = p[j];
    }
};

// eight elements of a row, of which w are inside
template <class T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8], int w)
{
    if (w == 8) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            constexpr int V = kWide<T>;
            struct alignas(16) Pack {
                T e[V];
            } q;
#pragma unroll
            for (int e = 0; e < V; ++e) q.e[e] = from_f32<T>(v[i * V + e]);
            store16(p + i * V, __builtin_bit_cast(uint4, q));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < w) p[j] = from_f32<T>(v[j]);
    }
}

// whether rows of `elem`-byte elements, ld apart, all begin on `bytes` bytes
inline bool aligned_rows(const void* p, int64_t ld, int64_t elem, int64_t bytes = 16)
{
    return (uintptr_t)p % (uintptr_t)bytes == 0 && ld * elem % bytes == 0;
}

}  // namespace cgtp
