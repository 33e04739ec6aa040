// What the gated block's kernels do with their sums: the activation and its slope, h, the gradients of g and u, and the
// joining of sums that several workgroups took over parts of K.
#pragma once

#include <type_traits>

#include "dropout.h"
#include "planes.h"

namespace moe {

enum Epi {
    kEpiGated,       // h, and g and u where they are kept
    kEpiGatedBwd,    // dg and du
    kEpiOut          // the product itself
};

struct EpiArgs {
    int M, N;                                   // rows, columns (of one matrix)
    void *o0, *o1;                              // outputs [M, N] of matrix 0 and 1 (kEpiOut), h (kEpiGated)
    void *save_g, *save_u;                      // kEpiGated: g and u, laid out as h (or null)
    const void* dh;                             // kEpiGatedBwd: [M, N]
    uint16_t *dg, *du;                          // kEpiGatedBwd: rows of ld_d values, the planes of one d_plane apart;
    int d_plane, ld_d;                          // the columns from N up to the next multiple of 8 are zero
    int act;
    Dropout drop;
    float* partial;                             // not null: sums of one part of K each, [part, matrix, M, ld_part]
    int ld_part, parts, mats;                   // N rounded up to 8; parts of K; matrices (two in the gated ones)
};

// An argument of 2^-y, y >= 0, and (kF32) what it lacks of the exact value.
struct Exponent {
    float y, rest;
};

// x log2 e (lo: what x >= 0 lacks itself).
template <bool kF32>
__device__ __forceinline__ Exponent exponent(float x, float lo = 0.0f)
{
    constexpr float kL = 1.44269502162933349609375f, kLow = 1.92596299112661746887e-8f;   // log2 e and what it lacks
    const float y = x * kL;
    return {y, kF32 ? fmaf(lo, kL, fmaf(x, kLow, fmaf(x, kL, -y))) : 0.0f};
}

// 2 sqrt(2 / pi) log2 e (x + 0.044715 x^3) for x >= 0, every product's and sum's rest taken along: rounded alone, 95 at x = 9
// would put 1.4e-5 into 2^-y.
template <bool kF32>
__device__ __forceinline__ Exponent tanh_exponent(float x)
{
    constexpr float kA = 2.302208185195923f, kALow = 1.29484020e-8f;                // 2 sqrt(2 / pi) log2 e and what it lacks
    constexpr float kB = 0.0447149984538555145263671875f, kBLow = 1.54614449e-9f;   // 0.044715 and what it lacks
    const float s = x * x, p = fmaf(kB, s, 1.0f), v = x * p, y = kA * v;
    if constexpr (!kF32)
        return {y, 0.0f};
    const float p_rest = fmaf(kB, s, 1.0f - p) + fmaf(kB, fmaf(x, x, -s), kBLow * s);   // p - 1 is exact
    const float v_rest = fmaf(x, p_rest, fmaf(x, p, -v));
    return {y, fmaf(kA, v_rest, fmaf(kALow, v, fmaf(kA, v, -y)))};
}

// 2^-y.  kF32: the rest is put back, which leaves the hardware's 2^y (1 ulp) as the error; else the error is that of the
// argument, about 2^-23 of it.
template <bool kF32>
__device__ __forceinline__ float exp2_minus(const Exponent& x)
{
    const float e = __builtin_amdgcn_exp2f(-x.y);
    if constexpr (!kF32)
        return e;
    return x.y < 150.0f ? fmaf(e, -0.6931471805599453f * x.rest, e) : e;
}

// 1 / x for x >= 1, to 1 ulp.
__device__ __forceinline__ float reciprocal(float x)
{
    const float r = __builtin_amdgcn_rcpf(x);
    return fmaf(r, fmaf(-x, r, 1.0f), r);
}

// act(g) and its slope.  silu and gelu's tanh form are g s(z) with the logistic function s: z = g, and
// z = 2 sqrt(2 / pi) (g + 0.044715 g^3) since (1 + tanh y) / 2 = s(2 y).  gelu takes the normal distribution function from exp(-g^2 / 2) erfcx(x) / 2 with
// x = |g| / sqrt 2, erfcx(x) / 2 = t P(t), t = 1 / (1 + 0.54 x): P of degree 9 was fitted to float64 values of erfcx on
// [0, 14.5] by weighted least squares, relative error 3e-7 in float32.  The exponent is taken from g, whose half is exact,
// not from the rounded x (1.2e-5 at g = -13).  Values are right to 2^-20 in float32 calls.
template <bool kF32>
__device__ __forceinline__ void activation(int act, float g, float& value, float& slope)
{
    if (act == MOE_ACT_GELU) {
        const float x = 0.70710678118654752f * fabsf(g), half = 0.5f * g, x2 = half * g;
        const float e = exp2_minus<kF32>(exponent<kF32>(x2, fmaf(half, g, -x2)));
        // the reciprocal of infinity would come out NaN; e is zero from far below 1e18 on
        const float t = reciprocal(fmaf(0.54f, fminf(x, 1e18f), 1.0f));
        float p = 0.022005289793014526f;
        p = fmaf(p, t, -0.13662242889404297f);
        p = fmaf(p, t, 0.3370496928691864f);
        p = fmaf(p, t, -0.3885047733783722f);
        p = fmaf(p, t, 0.170466348528862f);
        p = fmaf(p, t, -0.03764384239912033f);
        p = fmaf(p, t, 0.1002800464630127f);
        p = fmaf(p, t, 0.12816691398620605f);
        p = fmaf(p, t, 0.15247608721256256f);
        p = fmaf(p, t, 0.15232667326927185f);
        const float q = p * t * e;                             // the distribution function at -|g|
        const float c = g < 0.0f ? q : 1.0f - q;
        value = g * c;
        slope = c + (e == 0.0f ? 0.0f : g * e * 0.39894228040143268f);
        return;
    }
    constexpr float kA = 1.5957691216057308f, kB = 0.044715f;
    const Exponent z = act == MOE_ACT_SILU ? exponent<kF32>(fabsf(g)) : tanh_exponent<kF32>(fabsf(g));
    const float dz = act == MOE_ACT_SILU ? 1.0f : kA * (1.0f + 3.0f * kB * g * g);
    const float e = exp2_minus<kF32>(z), r = reciprocal(1.0f + e);
    const float s = g < 0.0f ? e * r : r, t = g < 0.0f ? r : e * r;    // s(z) and 1 - s(z)
    value = g * s;
    const float st = s * t;
    slope = s + (st == 0.0f ? 0.0f : g * st * dz);
}

// Eight values to the planes at p (one bfloat16 plane, rounded, or three); p aligned to 16 bytes.
template <bool kF32>
__device__ __forceinline__ void store_planes(uint16_t* p, int64_t plane, const float (&v)[8])
{
    if constexpr (kF32) {
        u32x4_t q[3];
        split8<3>(v, q);
#pragma unroll
        for (int i = 0; i < 3; ++i)
            *reinterpret_cast<u32x4_t*>(p + i * plane) = q[i];
    } else {
        *reinterpret_cast<u32x4_t*>(p) = pack8_bf16(v);
    }
}

template <bool kF32>
using Value = std::conditional_t<kF32, float, uint16_t>;

// h of eight columns from col on in one row (col < F), and g and u where they are kept.
template <bool kF32>
__device__ __forceinline__ void finish_gated(const EpiArgs& e, const DropKey& key, float (&g)[8], const float (&u)[8],
                                             int64_t row, int col)
{
    using T = Value<kF32>;
    const int n = e.N - col;
    const int64_t at = row * e.N + col;
    if (e.save_g != nullptr) {
        store8(static_cast<T*>(e.save_g) + at, g, n);
        store8(static_cast<T*>(e.save_u) + at, u, n);
    }
    float h[8], slope;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        activation<kF32>(e.act, g[i], h[i], slope);
        h[i] *= u[i];
    }
    if (e.drop.threshold != 0)
        drop8(h, e.drop, key, static_cast<uint32_t>(col >> 3), static_cast<uint32_t>(row));
    store8(static_cast<T*>(e.o0) + at, h, n);
}

// dg and du of eight columns.  bfloat16: rounded once, so that a plane each enters the products, as the operands do; the
// gradients' error is 0.0023 of their norm, 0.0017 (the rounding of the results) with dg and du in float32, whose two planes
// would double the products' work (4096 x 4096 x 14336: 1560 us of 1670).  Columns from N on are written as zero, they pad the products' K.
template <bool kF32>
__device__ __forceinline__ void finish_gated_bwd(const EpiArgs& e, const DropKey& key, float (&g)[8], float (&u)[8],
                                                 int64_t row, int col)
{
    using T = Value<kF32>;
    const int n = e.N - col;
    float d[8];
    load8(d, static_cast<const T*>(e.dh) + row * e.N + col, n);
    if (e.drop.threshold != 0)
        drop8(d, e.drop, key, static_cast<uint32_t>(col >> 3), static_cast<uint32_t>(row));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float value, slope;
        activation<kF32>(e.act, g[i], value, slope);
        // a dropped place has no gradient whatever its g and u
        g[i] = d[i] == 0.0f || i >= n ? 0.0f : d[i] * u[i] * slope;
        u[i] = d[i] == 0.0f || i >= n ? 0.0f : d[i] * value;
    }
    const int64_t at = row * e.ld_d + col;
    store_planes<kF32>(e.dg + at, e.d_plane, g);
    store_planes<kF32>(e.du + at, e.d_plane, u);
}

// One run of eight columns to where the epilogue puts it: v (and, gated, w: u where v is g), of matrix mat.
template <int kEpi, bool kF32>
__device__ __forceinline__ void finish8(const EpiArgs& e, const DropKey& key, float (&v)[8], float (&w)[8], int mat,
                                        int64_t row, int col)
{
    if constexpr (kEpi == kEpiGated)
        finish_gated<kF32>(e, key, v, w, row, col);
    else if constexpr (kEpi == kEpiGatedBwd)
        finish_gated_bwd<kF32>(e, key, v, w, row, col);
    else
        store8(static_cast<Value<kF32>*>(mat ? e.o1 : e.o0) + row * e.N + col, v, e.N - col);
}

// Where a part's sums of one matrix row lie.
__device__ __forceinline__ float* partial_at(const EpiArgs& e, int part, int mat, int64_t row, int col)
{
    return e.partial + ((static_cast<int64_t>(part) * e.mats + mat) * e.M + row) * e.ld_part + col;
}

// gated_rows.hip: the gated product of few rows, weights straight from memory to the matrix cores.
struct RowsArgs {
    const void *x, *wg, *wu;                    // [M, K], [K, N] of the call's type, any alignment
    int K;
    EpiArgs e;
};
constexpr int kMaxRows = 64, kMinCols = 4;   // at most, at least
// Parts of K that the kernel takes (1: it writes the results itself; otherwise partial sums).
int gated_rows_parts(int dtype, int64_t M, int64_t K, int64_t N);
hipError_t launch_gated_rows(Epi epi, int dtype, const RowsArgs& g, hipStream_t s);
// The results from partial sums (EpiArgs.partial).
hipError_t launch_gated_finish(Epi epi, int dtype, const EpiArgs& e, hipStream_t s);

}  // namespace moe
