// Eight adjacent values of float32 or bfloat16 memory, as one lane moves them: 16 bytes, or twice 16.
#pragma once

#include <stdint.h>

#include "common.h"

namespace moe {

// Vectors in memory of any element's alignment: the copies become unaligned vector loads and stores, which take as long
// as aligned ones where they do not cross a cache line.
typedef u32x4_t __attribute__((aligned(2))) u32x4_any_t;
typedef f32x4_t __attribute__((aligned(4))) f32x4_any_t;

// As loaded.
template <class T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
    u32x4_t w;
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};
template <>
struct Raw8<float> {
    f32x4_t a, b;
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    }
};

// The first n of eight values at p; the others are zero and not read.  kWhole: n is at least 8, or 0 or less.
template <bool kWhole>
__device__ __forceinline__ Raw8<uint16_t> load_raw(const uint16_t* p, int n)
{
    Raw8<uint16_t> r;
    r.w = u32x4_t{0, 0, 0, 0};
    if (n >= 8) {
        r.w = *reinterpret_cast<const u32x4_any_t*>(p);
    } else if (!kWhole && n > 0) {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n)
                r.w[i / 2] |= static_cast<uint32_t>(p[i]) << (16 * (i % 2));
    }
    return r;
}
template <bool kWhole>
__device__ __forceinline__ Raw8<float> load_raw(const float* p, int n)
{
    Raw8<float> r;
    r.a = r.b = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (n >= 8) {
        r.a = reinterpret_cast<const f32x4_any_t*>(p)[0];
        r.b = reinterpret_cast<const f32x4_any_t*>(p)[1];
    } else if (!kWhole && n > 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < n)
                r.a[i] = p[i];
            if (4 + i < n)
                r.b[i] = p[4 + i];
        }
    }
    return r;
}

__device__ __forceinline__ bool any_nan(const float (&v)[8])
{
    return __builtin_isunordered(v[0], v[1]) || __builtin_isunordered(v[2], v[3]) || __builtin_isunordered(v[4], v[5]) ||
           __builtin_isunordered(v[6], v[7]);
}

template <class T>
__device__ __forceinline__ void load8(float (&v)[8], const T* p, int n)
{
    load_raw<false>(p, n).values(v);
}

__device__ __forceinline__ u32x4_t pack8_bf16(const float (&v)[8])
{
    return u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

// Writes the first n of eight values, rounded to T.  kWhole: n is at least 8.
template <class T, bool kWhole = false>
__device__ __forceinline__ void store8(T* p, const float (&v)[8], int n)
{
    if constexpr (sizeof(T) == 2) {
        if (kWhole || n >= 8) {
            *reinterpret_cast<u32x4_any_t*>(p) = pack8_bf16(v);
            return;
        }
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n)
                p[i] = f32_to_bf16(v[i]);
    } else {
        if (kWhole || n >= 8) {
            reinterpret_cast<f32x4_any_t*>(p)[0] = f32x4_t{v[0], v[1], v[2], v[3]};
            reinterpret_cast<f32x4_any_t*>(p)[1] = f32x4_t{v[4], v[5], v[6], v[7]};
            return;
        }
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n)
                p[i] = v[i];
    }
}

}  // namespace moe
