// The gate with scores, a balance bias, expert groups and renormalised weights, and its gradient.
//
//   s = softmax(l) over the E experts, or sigmoid(l);   c = s + bias (c = -inf where l = -inf)
//   group score = sum of the group_top largest finite c of its E / G neighbouring experts
//   the topk_groups best groups stay; of their experts the k largest c, lower id first among equals
//   w_j = scale * s_j / (renormalize ? sum_i s_i : 1)
//
// Which experts are chosen is decided as in real arithmetic: without a bias the scores rise with the
// logits, so within the groups the logits themselves are compared; with a bias, and between groups,
// the scores are float64 (float32 scores of neighbouring experts often round to one value).  Almost no
// token needs that: L lanes per token first work in float32 with 32-bit keys, keep a bound on every
// error, and only the tokens in which two values that matter lie within it (about one in a thousand of
// random logits over 256 experts, and every token with a NaN) are done again in float64, one at a time
// by the whole wave.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "moe_expert_layer.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWavesPerBlock = kThreads / 64;

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) { *p = f32_to_bf16(v); }
__device__ __forceinline__ void load_logits4(const float* p, float (&v)[4])
{
    const f32x4_t w = *reinterpret_cast<const f32x4_t*>(p);
#pragma unroll
    for (int c = 0; c < 4; ++c)
        v[c] = w[c];
}
__device__ __forceinline__ void load_logits4(const uint16_t* p, float (&v)[4])
{
    const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        v[2 * c] = __uint_as_float(w[c] << 16);
        v[2 * c + 1] = __uint_as_float(w[c] & 0xffff0000u);
    }
}

// Exchange step S (partner distance 1 << S) of a reduction over a token's lanes inside a row of 16, by
// data-parallel-primitive moves: the mirrors pair each quad, then each half row, with the other one,
// which serves once the lanes of a quad / half row agree.
template <int S>
__device__ __forceinline__ int exchange(int v)
{
    if constexpr (S == 0)
        return __builtin_amdgcn_update_dpp(v, v, 0xB1, 0xf, 0xf, false);       // quad_perm 1 0 3 2
    else if constexpr (S == 1)
        return __builtin_amdgcn_update_dpp(v, v, 0x4E, 0xf, 0xf, false);       // quad_perm 2 3 0 1
    else if constexpr (S == 2)
        return __builtin_amdgcn_update_dpp(v, v, 0x141, 0xf, 0xf, false);      // row_half_mirror
    else
        return __builtin_amdgcn_update_dpp(v, v, 0x140, 0xf, 0xf, false);      // row_mirror
}
template <int S>
__device__ __forceinline__ float exchange(float v)
{
    return __int_as_float(exchange<S>(__float_as_int(v)));
}
template <int S>
__device__ __forceinline__ uint32_t exchange(uint32_t v)
{
    return static_cast<uint32_t>(exchange<S>(static_cast<int>(v)));
}

// Steps 4 and 5: v of the lower and of the upper one of two neighbouring rows / halves, on both.
template <int S>
__device__ __forceinline__ void pair(int v, int& lower, int& upper)
{
    if constexpr (S == 4) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        lower = r[0];
        upper = r[1];
    } else {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        lower = r[0];
        upper = r[1];
    }
}

// v combined by the commutative f over aligned runs of L lanes, on every lane.
template <int L, int S = 0, class V, class F>
__device__ __forceinline__ V reduce(V v, F f)
{
    if constexpr ((1 << S) >= L) {
        return v;
    } else if constexpr (S < 4) {
        return reduce<L, S + 1>(f(v, exchange<S>(v)), f);
    } else {
        int lower, upper;
        pair<S>(__builtin_bit_cast(int, v), lower, upper);
        return reduce<L, S + 1>(f(__builtin_bit_cast(V, lower), __builtin_bit_cast(V, upper)), f);
    }
}
struct Add {
    template <class V>
    __device__ __forceinline__ V operator()(V a, V b) const { return a + b; }
};
struct Max {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct MinU {
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return min(a, b); }
};

// exp2 on the hardware unit (1 ulp) of x log2 e; the product's rounding makes it |x| 2^-24 relative.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }

struct GateArgs {
    const float* bias;       // may be null
    int64_t T;
    int E, k, groups, topk_groups, group_top, sigmoid, renormalize;
    float scale;
    int32_t* ids;
    float* probs;
    int group_shift;         // log2 of the lanes a group's experts cover in one vector; -1: no such layout
    int scratch;             // doubles of LDS per wave for the groups (0 without)
};

// Unsigned integers of the order of the floats (no NaN).
__device__ __forceinline__ uint32_t ordered(float f)
{
    const uint32_t b = __float_as_uint(f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o)
{
    return __uint_as_float((o & 0x80000000u) != 0 ? o & 0x7fffffffu : ~o);
}
// 64-bit keys: 1 for -inf (so that 0 is free for "not a candidate"), the largest for NaN; -0 as +0.
__device__ __forceinline__ uint64_t key64(double c)
{
    if (c != c)
        return ~uint64_t{0};
    const uint64_t b = __builtin_bit_cast(uint64_t, c + 0.0);
    const uint64_t k = (b >> 63) != 0 ? ~b : b | (uint64_t{1} << 63);
    return c == -__builtin_inf() ? 1 : k;
}

// One token in float64 by the whole wave: lane l holds experts l, l + 64, ...  lds: E + groups doubles
// of this wave (with groups alone).
template <class In, int kPer>
__device__ __forceinline__ void gate_token_exact(const In* __restrict__ row, int64_t t, const GateArgs& a,
                                              double* lds)
{
    const int lane = threadIdx.x & 63;
    const auto sum = [](double v) {
        for (int off = 32; off >= 1; off >>= 1)
            v += __shfl_xor(v, off);
        return v;
    };
    float l[kPer];
    float lmax = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + 64 * i;
        l[i] = e < a.E ? load_logit(row + e) : -__builtin_inff();
        lmax = fmaxf(lmax, l[i]);
    }
    double num[kPer];                                         // score = num / den
    double den = 1.0;
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            num[i] = 1.0 / (1.0 + exp(-static_cast<double>(l[i])));
    } else {
        for (int off = 32; off >= 1; off >>= 1)
            lmax = fmaxf(lmax, __shfl_xor(lmax, off));
        den = 0.0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            num[i] = l[i] == -__builtin_inff() ? 0.0 : exp(static_cast<double>(l[i]) - static_cast<double>(lmax));
            den += num[i];
        }
        den = sum(den);
        if (den == 0.0)
            den = 1.0;                                        // every logit is -inf: scores 0
    }
    uint64_t key[kPer];                                       // 0: taken, or no candidate
    double c[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + 64 * i;
        c[i] = num[i] / den + (a.bias != nullptr && e < a.E ? static_cast<double>(a.bias[e]) : 0.0);
        if (l[i] == -__builtin_inff())
            c[i] = -__builtin_inf();
        // a NaN logit makes every softmax score NaN: the logits decide then (NaN first)
        key[i] = e < a.E ? key64(a.bias != nullptr && c[i] == c[i] ? c[i] : static_cast<double>(l[i])) : 0;
    }
    if (a.groups > 1) {
        double* const score = lds + a.E;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 64 * i < a.E)
                lds[lane + 64 * i] = c[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int per = a.E / a.groups;
        for (int q = lane; q < a.groups; q += 64) {
            double b1 = -__builtin_inf(), b2 = -__builtin_inf();
            for (int i = 0; i < per; ++i) {
                const double v = lds[q * per + i];
                b2 = fmax(b2, fmin(b1, v));
                b1 = fmax(b1, v);
            }
            score[q] = a.group_top == 2 && b2 > -__builtin_inf() ? b1 + b2 : b1;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int q = min(lane + 64 * i, a.E - 1) / per;
            const double mine = score[q];
            int rank = 0;
            for (int o = 0; o < a.groups; ++o)
                rank += score[o] > mine || (score[o] == mine && o < q) ? 1 : 0;
            if (rank >= a.topk_groups)
                key[i] = 0;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();                      // read before the wave's next token writes
    }
    int my_id = 0;
    double my_num = 0.0;
    for (int j = 0; j < a.k; ++j) {
        uint64_t best = 0;
        int id = 0;
        double n = 0.0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (key[i] > best) {                              // lower ids first: i ascends
                best = key[i];
                id = lane + 64 * i;
                n = num[i];
            }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            const uint64_t ob = __shfl_xor(static_cast<unsigned long long>(best), off);
            const int oi = __shfl_xor(id, off);
            const double on = __shfl_xor(n, off);
            if (ob > best || (ob == best && oi < id)) {
                best = ob;
                id = oi;
                n = on;
            }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 64 * i == id)
                key[i] = 0;
        if (lane == j) {
            my_id = id;
            my_num = n;
        }
    }
    if (a.renormalize) {
        den = sum(my_num);
        if (den == 0.0)
            den = 1.0;                                        // nothing but zero scores: weights 0
    }
    if (lane < a.k) {
        a.ids[t * a.k + lane] = my_id;
        a.probs[t * a.k + lane] = static_cast<float>(my_num / den * static_cast<double>(a.scale));
    }
}

// L lanes per token; lane g holds the vectors of four experts 4 (L i + g), i < I.
//
// Each candidate is one 32-bit key: the ordered bits of what it is compared by, the lowest four replaced
// by its place in the lane (bfloat16 logits without a bias: the lower 16 bits are free, and the
// complement of the expert's id makes the keys unique and exact).  The next key below M is
// M - 1 - min over the keys v of (M - 1 - v), unsigned: keys at or above M wrap to large values, so
// nothing is taken out of the registers from round to round.
//
// Errors, with u = 2^-24 and x = max - l.  softmax: exp(-x) is off by (2.5 x + 2) u relative (the
// subtraction, the product with log2 e and that constant, a 1-ulp exp2), at most 3 u of the largest
// score since x exp(-x) < 0.37, and the two products add 2 u; the sum's error (an average of x, at most
// ln 1024, and 22 additions: 42 u) is one factor common to the token's scores.  The difference of two is
// thus off by at most 42 + 2 * 5 = 52 u of the largest score.  sigmoid: 10 u each, with scores <= 1.
// Adding the bias rounds by |c| u each and cutting a key drops less than 16 ulp = 32 u |c|.  So two
// values more than 64 u = 2^-18 (largest score + |c|) apart are in the right order, and two group
// scores (sums of two) more than 2^-17 (largest score + |c| + |c'|).  Keys of logits differ only as the
// logits do.
template <class In, int L, int I, bool kVec>
__global__ __launch_bounds__(kThreads) void gate_kernel(const In* __restrict__ logits, const GateArgs a)
{
    constexpr int kPer = 4 * I;
    constexpr int kTokens = 64 / L;                           // per wave
    extern __shared__ __attribute__((aligned(16))) double lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int g = lane & (L - 1), base = lane & ~(L - 1);
    // LDS: each wave's scratch for the groups, then the winners of its tokens
    double* const wide = lds + static_cast<size_t>(wave) * a.scratch;
    int* const won = reinterpret_cast<int*>(lds + static_cast<size_t>(kWavesPerBlock) * a.scratch) +
                        (static_cast<size_t>(wave) * kTokens + lane / L) * a.k;
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / L;
    const bool live = t < a.T;
    const In* row = logits + (live ? t : a.T - 1) * a.E;
    bool unsure = a.groups > 1 && a.group_shift < 0;         // this token needs float64
    if (!__all(unsure)) {
        float l[kPer];
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int e = 4 * (L * i + g);
            float v[4];                                       // past the row's end: its last values, replaced below
            if (kVec) {
                load_logits4(row + min(e, a.E - 4), v);
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    v[c] = load_logit(row + min(e + c, a.E - 1));
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
                l[4 * i + c] = e + c < a.E ? v[c] + 0.0f : -__builtin_inff();   // -0 becomes +0: equal logits tie
        }
        const bool by_logit = a.bias == nullptr;
        float num[kPer];                                      // score = num * inv
        float inv = 1.0f, check = 0.0f;                       // check: NaN if a logit (or bias) is
        float m = 0.0f;
        if (a.sigmoid) {
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                num[q] = __builtin_amdgcn_rcpf(1.0f + fast_exp(-l[q]));
                check += num[q];
            }
        } else {
            m = l[0];
#pragma unroll
            for (int q = 1; q < kPer; ++q)
                m = fmaxf(m, l[q]);
            m = reduce<L>(m, Max{});
            float total = 0.0f;
            m = m == -__builtin_inff() ? 0.0f : m;            // every logit is -inf: scores 0
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                num[q] = fast_exp(l[q] - m);
                total += num[q];
            }
            check = total;
            total = reduce<L>(total, Add{});
            inv = total == 0.0f ? 1.0f : 1.0f / total;
        }
        const float top_score = a.sigmoid ? 1.0f : inv;
        float c[kPer];                                        // what the experts are compared by
        if (by_logit && a.groups == 1) {
#pragma unroll
            for (int q = 0; q < kPer; ++q)
                c[q] = l[q];
        } else {
#pragma unroll
            for (int i = 0; i < I; ++i) {
                const int e = 4 * (L * i + g);
                float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (!by_logit) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        b[q] = a.bias[kVec ? min(e, a.E - 4) + q : min(e + q, a.E - 1)];
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float v = num[4 * i + q] * inv + b[q];
                    check += e + q < a.E ? v : 0.0f;
                    c[4 * i + q] = l[4 * i + q] == -__builtin_inff() ? -__builtin_inff() : v;
                }
            }
        }
        check = reduce<L>(check, Add{});
        unsure = check != check;
        uint32_t dropped = 0;                                 // bit i: the group of vector i is out
        if (a.groups > 1) {
            // a group is an aligned run of 1 << group_shift lanes of one vector
            float* const score = reinterpret_cast<float*>(wide) + (lane / L) * a.groups;
            float mine[I], size = 0.0f;
#pragma unroll
            for (int i = 0; i < I; ++i) {
                const float h1 = fmaxf(c[4 * i], c[4 * i + 1]), l1 = fminf(c[4 * i], c[4 * i + 1]);
                const float h2 = fmaxf(c[4 * i + 2], c[4 * i + 3]), l2 = fminf(c[4 * i + 2], c[4 * i + 3]);
                float b1 = fmaxf(h1, h2), b2 = fmaxf(fminf(h1, h2), h1 >= h2 ? l1 : l2);
                const auto join = [&](float o1, float o2) {
                    b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
                    b1 = fmaxf(b1, o1);
                };
                if (a.group_shift > 0)
                    join(exchange<0>(b1), exchange<0>(b2));
                if (a.group_shift > 1)
                    join(exchange<1>(b1), exchange<1>(b2));
                if (a.group_shift > 2)
                    join(exchange<2>(b1), exchange<2>(b2));
                if (a.group_shift > 3)
                    join(exchange<3>(b1), exchange<3>(b2));
                const bool two = a.group_top == 2 && b2 > -__builtin_inff();
                mine[i] = two ? b1 + b2 : b1;
                size = fmaxf(size, b1 > -__builtin_inff() ? fabsf(b1) + (two ? fabsf(b2) : 0.0f) : 0.0f);
                const int q = (L * i + g) >> a.group_shift;
                if (q < a.groups && (g & ((1 << a.group_shift) - 1)) == 0)
                    score[q] = mine[i];
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            int rank[I] = {};
            for (int o = 0; o < a.groups; ++o) {
                const float other = score[o];
#pragma unroll
                for (int i = 0; i < I; ++i)
                    rank[i] += other > mine[i] || (other == mine[i] && o < ((L * i + g) >> a.group_shift)) ? 1 : 0;
            }
            // the last group kept must lie clearly above the first one dropped
            float in = __builtin_inff(), out = -__builtin_inff();
#pragma unroll
            for (int i = 0; i < I; ++i) {
                if ((L * i + g) >> a.group_shift >= a.groups)
                    continue;
                if (rank[i] >= a.topk_groups) {
                    dropped |= 1u << i;
                    out = fmaxf(out, mine[i]);
                } else {
                    in = fminf(in, mine[i]);
                }
            }
            in = -reduce<L>(-in, Max{});
            out = reduce<L>(out, Max{});
            size = reduce<L>(size, Max{});
            unsure |= a.topk_groups < a.groups && !(in - out > 0x1p-17f * (top_score + size));
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        constexpr bool kIdKey = std::is_same_v<In, uint16_t>;
        const bool id_key = kIdKey && by_logit;
        uint32_t key[kPer];                                   // 0: no candidate
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            const int e = 4 * (L * (q / 4) + g) + q % 4;
            const uint32_t o = ordered(by_logit ? l[q] : c[q]);
            key[q] = id_key ? (o & 0xffff0000u) | (0xffffu - static_cast<uint32_t>(e)) : (o & ~15u) | static_cast<uint32_t>(q);
            if (e >= a.E || (dropped >> (q / 4) & 1) != 0)
                key[q] = 0;
        }
        uint32_t last = 0;                                    // below every key: M - 1 wraps to the top
        float before = 0.0f;
        for (int j = 0; j <= a.k; ++j) {
            const uint32_t from = last - 1;
            uint32_t d = from - key[0];
#pragma unroll
            for (int q = 1; q < kPer; ++q)
                d = min(d, from - key[q]);
            const uint32_t all = reduce<L>(d, MinU{});
            const uint32_t now = from - all;                  // 0, or wrapped above `last`: none left
            const bool none = now == 0 || (j > 0 && now >= last);
            if (!id_key) {
                // the one before must lie clearly above, and one lane alone may hold this one
                const float v = now < 0x00800000u ? -__builtin_inff() : unordered(now & ~15u);
                const float eps = by_logit || v == -__builtin_inff() ? 0.0f : 0x1p-18f * (top_score + fabsf(v));
                const uint64_t holders = __ballot(d == all) >> base;
                const bool sole = __popcll(L == 64 ? holders : holders & ((uint64_t{1} << (L & 63)) - 1)) == 1;
                unsure |= !none && ((j > 0 && !(before - v > eps)) || (j < a.k && !sole));
                before = v;
            }
            unsure |= none && j < a.k;
            if (j < a.k && d == all)
                won[j] = id_key ? 0xffff - static_cast<int>(now & 0xffffu)
                                : 4 * (L * static_cast<int>(now >> 2 & 3) + g) + static_cast<int>(now & 3);
            last = now;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (!__all(unsure)) {
            // the winners' scores again, one a lane
            float total = 0.0f, least = __builtin_inff();
            const auto score = [&](int id) {
                const float x = load_logit(row + id);
                return a.sigmoid ? __builtin_amdgcn_rcpf(1.0f + fast_exp(-x)) : fast_exp(x - m);
            };
            int id = 0;
            float n = 0.0f;
            for (int j = g; j < a.k && !unsure; j += L) {
                id = won[j];
                n = score(id);
                total += n;
                least = fminf(least, n);
            }
            // scores near float32's smallest: their ratios need float64's range
            unsure |= -reduce<L>(-least, Max{}) < 0x1p-100f;
            const float factor = (a.renormalize ? 1.0f / reduce<L>(total, Add{}) : inv) * a.scale;
            for (int j = g; j < a.k && live && !unsure; j += L) {
                if (a.k > L) {
                    id = won[j];
                    n = score(id);
                }
                a.ids[t * a.k + j] = id;
                a.probs[t * a.k + j] = n * factor;
            }
        }
    }
    // the tokens left, one after the other
    uint64_t todo = __ballot(live && unsure && g == 0);
    while (todo != 0) {
        const int first = __ffsll(static_cast<unsigned long long>(todo)) - 1;
        todo &= todo - 1;
        const int64_t tt = static_cast<int64_t>(blockIdx.x) * (kThreads / L) + wave * kTokens + first / L;
        gate_token_exact<In, (4 * L * I + 63) / 64>(logits + tt * a.E, tt, a, wide);
    }
}

template <class V>
__device__ __forceinline__ V group_sum(V v, int L)
{
    for (int off = L / 2; off >= 1; off >>= 1)
        v += __shfl_xor(v, off);
    return v;
}
__device__ __forceinline__ float group_max(float v, int L)
{
    for (int off = L / 2; off >= 1; off >>= 1)
        v = fmaxf(v, __shfl_xor(v, off));
    return v;
}

struct GateBackwardArgs {
    int64_t T;
    int E, k, sigmoid, renormalize;
    float scale;
    const int32_t* ids;
    const float* dprobs;
};

// dl of one token.  With w_j the unscaled weights and d_j = scale dprobs_j:
//   renormalised: q_j = w_j (d_j - sum_i d_i w_i), sigmoid times 1 - s_j; dl_e = the q_j with id e
//   otherwise: sigmoid dl_e = d_j s_j (1 - s_j); softmax dl_e = s_e (d_j [id_j = e] - sum_i d_i s_i)
// An id that occurs twice gets both; ids outside [0, E) are no slots.
template <class In, int L, int kPer>
__global__ __launch_bounds__(kThreads) void gate_backward_kernel(const In* __restrict__ logits,
                                                                 In* __restrict__ dlogits,
                                                                 const GateBackwardArgs a)
{
    const int lane = threadIdx.x & 63;
    const int g = lane & (L - 1), base = lane & ~(L - 1);
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / L;
    const bool live = t < a.T;
    const In* row = logits + (live ? t : 0) * a.E;
    int id = -1;
    float d = 0.0f, lj = -__builtin_inff();
    if (live && g < a.k) {
        id = a.ids[t * a.k + g];
        if (id < 0 || id >= a.E)
            id = -1;
        else {
            d = a.scale * a.dprobs[t * a.k + g];
            lj = load_logit(row + id);
        }
    }
    float dense[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        dense[i] = 0.0f;
    float q;                                                  // this slot's part of its expert's gradient
    if (a.sigmoid) {
        const float s = id >= 0 ? 1.0f / (1.0f + expf(-lj)) : 0.0f;
        const float rest = 1.0f / (1.0f + expf(lj));          // 1 - s
        if (a.renormalize) {
            const float total = group_sum(s, L);
            const float w = total > 0.0f || total != total ? s / total : 0.0f;
            q = w * rest * (d - group_sum(d * w, L));
        } else {
            q = d * s * rest;
        }
    } else if (a.renormalize) {
        const float m = group_max(lj, L);
        const float ex = lj == -__builtin_inff() ? 0.0f : expf(lj - m);
        const float total = group_sum(ex, L);
        const float w = total > 0.0f || total != total ? ex / total : 0.0f;
        q = w * (d - group_sum(d * w, L));
    } else {
        float m = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            dense[i] = g + L * i < a.E ? load_logit(row + g + L * i) : -__builtin_inff();
            m = fmaxf(m, dense[i]);
        }
        m = group_max(m, L);
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            dense[i] = dense[i] == -__builtin_inff() ? 0.0f : expf(dense[i] - m);
            total += dense[i];
        }
        total = group_sum(total, L);
        const float inv = total > 0.0f || total != total ? 1.0f / total : 0.0f;
        const float s = lj == -__builtin_inff() ? 0.0f : expf(lj - m) * inv;
        q = d * s;
        const float dot = group_sum(q, L);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            dense[i] = -dense[i] * inv * dot;
    }
    for (int j = 0; j < a.k; ++j) {
        const int oi = __shfl(id, base + j);
        const float oq = __shfl(q, base + j);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (oi == g + L * i)
                dense[i] += oq;
    }
    if (live) {
        In* out = dlogits + t * a.E;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (g + L * i < a.E)
                store_logit(out + g + L * i, dense[i]);
    }
}

template <class In, int L, int I>
hipError_t launch_gate_n(const In* logits, GateArgs a, hipStream_t s)
{
    const int64_t blocks = ceil_div(a.T * L, kThreads);
    if (blocks >= (int64_t{1} << 31))
        return hipErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(blocks));
    // groups that are whole vectors of a power of two of neighbouring lanes (at most a row of 16)
    const int per = a.E / a.groups;
    a.group_shift = -1;
    for (int b = 0; b <= 4; ++b)
        if (a.groups > 1 && per == 4 << b && (1 << b) <= L)
            a.group_shift = b;
    // a token's experts and groups in float64, or the float32 group scores of the wave's tokens
    a.scratch = a.groups > 1 ? std::max(a.E + a.groups, (64 / L) * a.groups / 2 + 1) : 0;
    const size_t lds = sizeof(double) * kWavesPerBlock * static_cast<size_t>(a.scratch) +
                       sizeof(int) * (kThreads / L) * static_cast<size_t>(a.k);
    const bool vec = a.E % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % (4 * sizeof(In)) == 0;
    if (vec)
        gate_kernel<In, L, I, true><<<grid, dim3(kThreads), lds, s>>>(logits, a);
    else
        gate_kernel<In, L, I, false><<<grid, dim3(kThreads), lds, s>>>(logits, a);
    return hipGetLastError();
}

// The gate's lanes per token: four experts a lane up to 64 (so that small gates fill the wave with
// tokens), then vectors of four over 16 lanes, and the whole wave beyond 256 or for few tokens (a lane's
// work is then a quarter, and no wave waits for another).
template <class In>
hipError_t launch_gate_t(const In* logits, const GateArgs& a, hipStream_t s)
{
    if (a.E > 64 && a.E <= 256 && a.T <= 4 * device_info().cu_count)
        return launch_gate_n<In, 64, 1>(logits, a, s);
    if (a.E <= 8)
        return launch_gate_n<In, 2, 1>(logits, a, s);
    if (a.E <= 16)
        return launch_gate_n<In, 4, 1>(logits, a, s);
    if (a.E <= 32)
        return launch_gate_n<In, 8, 1>(logits, a, s);
    if (a.E <= 64)
        return launch_gate_n<In, 16, 1>(logits, a, s);
    if (a.E <= 128)
        return launch_gate_n<In, 16, 2>(logits, a, s);
    if (a.E <= 256)
        return launch_gate_n<In, 16, 4>(logits, a, s);
    if (a.E <= 512)
        return launch_gate_n<In, 64, 2>(logits, a, s);
    return launch_gate_n<In, 64, 4>(logits, a, s);
}

template <class In, int L, int kPer>
hipError_t launch_backward_n(const In* logits, In* dlogits, const GateBackwardArgs& a, hipStream_t s)
{
    const int64_t blocks = ceil_div(a.T * L, kThreads);
    if (blocks >= (int64_t{1} << 31))
        return hipErrorInvalidValue;
    gate_backward_kernel<In, L, kPer><<<dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s>>>(logits, dlogits, a);
    return hipGetLastError();
}

// Calls f with (lanes per token, experts per lane) for E experts.
template <class F>
hipError_t with_lanes(int E, F f)
{
    using std::integral_constant;
    if (E <= 8)
        return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
    if (E <= 16)
        return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    if (E <= 32)
        return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
    if (E <= 64)
        return f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    if (E <= 128)
        return f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    if (E <= 256)
        return f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
    if (E <= 512)
        return f(integral_constant<int, 64>{}, integral_constant<int, 8>{});
    return f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_gate(const moe_gate& o, const void* logits, int dtype, const float* bias, int64_t T,
                       int64_t E, int64_t k, int32_t* ids, float* probs, hipStream_t s)
{
    if (T <= 0)
        return hipSuccess;
    GateArgs a{};
    a.bias = bias;
    a.T = T;
    a.E = static_cast<int>(E);
    a.k = static_cast<int>(k);
    a.groups = o.groups;
    a.topk_groups = o.topk_groups;
    a.group_top = o.group_top;
    a.sigmoid = o.score == MOE_SCORE_SIGMOID;
    a.renormalize = o.renormalize;
    a.scale = o.scale;
    a.ids = ids;
    a.probs = probs;
    return dtype == MOE_F32 ? launch_gate_t(static_cast<const float*>(logits), a, s)
                            : launch_gate_t(static_cast<const uint16_t*>(logits), a, s);
}

hipError_t launch_gate_backward(const moe_gate& o, const void* logits, int dtype, int64_t T, int64_t E,
                                int64_t k, const int32_t* ids, const float* dprobs, void* dlogits, hipStream_t s)
{
    if (T <= 0)
        return hipSuccess;
    GateBackwardArgs a{};
    a.T = T;
    a.E = static_cast<int>(E);
    a.k = static_cast<int>(k);
    a.sigmoid = o.score == MOE_SCORE_SIGMOID;
    a.renormalize = o.renormalize;
    a.scale = o.scale;
    a.ids = ids;
    a.dprobs = dprobs;
    return with_lanes(a.E, [&](auto L, auto per) {
        return dtype == MOE_F32
                   ? launch_backward_n<float, L(), per()>(static_cast<const float*>(logits), static_cast<float*>(dlogits), a, s)
                   : launch_backward_n<uint16_t, L(), per()>(static_cast<const uint16_t*>(logits),
                                                             static_cast<uint16_t*>(dlogits), a, s);
    });
}

}  // namespace moe
