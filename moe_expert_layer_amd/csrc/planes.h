// Float32 operands on the bfloat16 matrix cores: a value as the sum of bfloat16 planes.
//
// Three planes hold a float32 value exactly (x = x0 + x1 + x2, each the nearest to what is left, so |x1| <= 2^-8 |x| and
// |x2| <= 2^-16 |x|).  Six of the nine products of two values' planes make their product; the three left out are together
// at most 2^-23 of |a| |b|, the size of one float32 rounding.  (Below 2^-110 a value's last bits lie under bfloat16's smallest
// number, 2^-133, which the matrix cores do not flush: they are rounded there.)  Six bfloat16 MFMAs have about 2.6 times the rate of one
// float32 MFMA.
#pragma once

#include "vec8.h"

namespace moe {

// The planes' products, small ones first.
constexpr int kPlanePairs[6][2] = {{2, 0}, {0, 2}, {1, 1}, {1, 0}, {0, 1}, {0, 0}};

// x as the sum of its first P planes (x0 rounds towards zero where the nearest would be infinite).  P = 2 keeps 16 bits
// (what is left out is at most 2^-16 |x|).  An infinity becomes infinity and (three planes) NaN, so that sums it takes
// part in are NaN; kSum: infinity and zeros, whose sum it is.
template <int P, bool kSum = P == 2>
__device__ __forceinline__ void split(float x, uint16_t (&p)[P])
{
#pragma unroll
    for (int i = 0; i < P; ++i) {
        uint16_t b = f32_to_bf16(x);
        const bool finite = (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u;
        if ((b & 0x7FFFu) == 0x7F80u && finite)
            b = static_cast<uint16_t>(__float_as_uint(x) >> 16);
        p[i] = b;
        x = kSum && !finite ? 0.0f : x - bf16_to_f32(b);
    }
}

// Eight values as P planes of eight.
template <int P, bool kSum = P == 2>
__device__ __forceinline__ void split8(const float (&v)[8], u32x4_t (&out)[P])
{
    uint16_t s[8][P];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        split<P, kSum>(v[i], s[i]);
#pragma unroll
    for (int q = 0; q < P; ++q)
        out[q] = u32x4_t{s[0][q] | static_cast<uint32_t>(s[1][q]) << 16, s[2][q] | static_cast<uint32_t>(s[3][q]) << 16,
                         s[4][q] | static_cast<uint32_t>(s[5][q]) << 16, s[6][q] | static_cast<uint32_t>(s[7][q]) << 16};
}

// The planes of an MFMA operand: bfloat16 values are one, float32 values three.
template <class T>
constexpr int kPlanesOf = sizeof(T) == 2 ? 1 : 3;
__device__ __forceinline__ void planes8(const Raw8<uint16_t>& r, u32x4_t (&p)[1]) { p[0] = r.w; }
__device__ __forceinline__ void planes8(const Raw8<float>& r, u32x4_t (&p)[3])
{
    float v[8];
    r.values(v);
    split8<3>(v, p);
}

// Columns 16 p + 8 (lane / 32) .. + 7 of row lane % 32 of a transposed 32 x 32 accumulator block.  A lane holds columns 8 q
// + 4 (lane / 32) + e in register 4 q + e: exchanging halves of the registers of q = 2 p and 2 p + 1 between lanes i and
// i + 32 makes runs of eight.
__device__ __forceinline__ void run8(const f32x16_t& acc, int p, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[8 * p + e]), __float_as_uint(acc[8 * p + 4 + e]),
                                                        false, false);
        v[e] = __uint_as_float(r[0]);
        v[4 + e] = __uint_as_float(r[1]);
    }
}

// One MFMA operand of 16 k x 32 columns read from LDS rows over k (N-contiguous) with the transposing reads: `base` is
// this lane's address (tr_offset) in the block's first k row; row: bytes between k rows.
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;
__device__ __forceinline__ uint32_t tr_offset(int lane, int row)
{
    const int g = lane >> 4, e = (lane >> 2) & 3, q = lane & 3;
    return (8 * (g >> 1) + e) * row + 2 * (16 * (g & 1) + 4 * q);
}
__device__ __forceinline__ bf16x8_t read_tr(uint32_t base, int row)
{
    const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_i16x4_t*>(base));
    const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_i16x4_t*>(base + 4 * row));
    return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

}  // namespace moe
