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
//
// Bound by vector arithmetic, not by its bytes: 65536 tokens of 256 experts in 8 groups, float32, take 39-41 us
// a call (a copy of the bytes would take 15), 68 vector instructions an expert that issue in 88% of the busy
// cycles; in float64 throughout, a wave per token, it took 247 us.  One token takes 4.3 us, a launch and a
// chain of reductions.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "int8_gate.h"

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
        return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xf, 0xf, true);       // quad_perm 1 0 3 2
    else if constexpr (S == 1)
        return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xf, 0xf, true);       // quad_perm 2 3 0 1
    else if constexpr (S == 2)
        return __builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, true);      // row_half_mirror
    else
        return __builtin_amdgcn_mov_dpp(v, 0x140, 0xf, 0xf, true);      // row_mirror
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
struct MaxU {
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return max(a, b); }
};

// exp2 on the hardware unit (1 ulp) of x log2 e; the product's rounding makes it |x| 2^-24 relative.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }

// exp(x - m), m finite, within 4 2^-24: the rounding of the difference is put back as a factor.
__device__ __forceinline__ float exp_difference(float x, float m)
{
    const float d = x - m, part = d - x;
    const float rounding = (x - (d - part)) - (m + part);     // of d, exact
    const float e = expf(d);
    return d > -100.0f ? fmaf(e, rounding, e) : e;
}

struct GateArgs {
    const float* bias;       // may be null
    int64_t T;
    int E, k, groups, topk_groups, group_top, sigmoid, renormalize;
    float scale;
    int32_t* ids;
    float* probs;
    int group_shift;         // log2 of the lanes a group's experts cover in one vector; -1: no such layout
    int part_shift;          // otherwise log2 of the lanes that share a group
    int per, per_inverse;    // experts per group; e / per = e * per_inverse >> 20 for e < 1024
    int scratch;             // doubles of LDS per wave for the groups (0 without): values of its experts and groups
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
    // a NaN or +inf logit makes every softmax score NaN: the logits decide then, NaN first
    const bool lost = !a.sigmoid && den != den;
    uint64_t key[kPer];                                       // 0: taken, or no candidate
    double c[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + 64 * i;
        c[i] = num[i] / den + (a.bias != nullptr && e < a.E ? static_cast<double>(a.bias[e]) : 0.0);
        if (lost || l[i] == -__builtin_inff())
            c[i] = static_cast<double>(l[i]);
        key[i] = e < a.E ? key64(a.bias != nullptr ? c[i] : static_cast<double>(l[i])) : 0;
    }
    if (a.groups > 1) {
        uint64_t* const score = reinterpret_cast<uint64_t*>(lds + a.E);   // keys: a NaN in a group makes it the largest
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 64 * i < a.E)
                lds[lane + 64 * i] = c[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int per = a.E / a.groups;
        for (int q = lane; q < a.groups; q += 64) {
            double b1 = -__builtin_inf(), b2 = -__builtin_inf();
            bool nan = false;
            for (int i = 0; i < per; ++i) {
                const double v = lds[q * per + i];
                nan |= v != v;
                b2 = fmax(b2, fmin(b1, v));
                b1 = fmax(b1, v);
            }
            score[q] = nan ? ~uint64_t{0} : key64(a.group_top == 2 && b2 > -__builtin_inf() ? b1 + b2 : b1);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int q = min(lane + 64 * i, a.E - 1) / per;
            const uint64_t mine = score[q];
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
        uint32_t id = 0;
        double n = 0.0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (key[i] > best) {                              // lower ids first: i ascends
                best = key[i];
                id = lane + 64 * i;
                n = num[i];
            }
        // the largest key by halves, then the lowest id that has it
        const uint32_t hi = reduce<64>(static_cast<uint32_t>(best >> 32), MaxU{});
        const uint32_t low = static_cast<uint32_t>(best >> 32) == hi ? static_cast<uint32_t>(best) : 0;
        const uint32_t lo = reduce<64>(low, MaxU{});
        const bool tops = best == (static_cast<uint64_t>(hi) << 32 | lo);
        const uint32_t first = reduce<64>(tops ? id : ~0u, MinU{});
        const double won = __shfl(n, __ffsll(static_cast<unsigned long long>(__ballot(tops && id == first))) - 1);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (static_cast<uint32_t>(lane + 64 * i) == first)
                key[i] = 0;
        if (lane == j) {
            my_id = static_cast<int>(first);
            my_num = won;
        }
    }
    if (a.renormalize && !lost) {
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
// Each candidate is one 32-bit key: the ordered bits of what it is compared by, the lowest ones replaced
// by its place in the lane (bfloat16 logits without a bias: the lower 16 bits are free, and the
// complement of the expert's id makes the keys unique and exact).  The next key below M is
// M - 1 - min over the keys v of (M - 1 - v), unsigned: keys at or above M wrap to large values, so
// nothing is taken out of the registers from round to round.  The lane that holds a round's key leaves
// it with its number in LDS, where the token's lanes check them and make the weights, one winner a lane,
// from scores computed again to float32's accuracy: with the selection's exponentials a weight was up to 87 u
// off (softmax, logits 60 apart; sigmoid 64 u at -60), now at most 8 u where tested (65536 x 256: 39.0 -> 39.8 us).
//
// Errors, with u = 2^-24 and x = max - l.  softmax: exp(-x) is off by (2.5 x + 2) u relative (the
// subtraction, the product with log2 e and that constant, a 1-ulp exp2), at most 3 u of the largest
// score since x exp(-x) < 0.37, and the two products add 2 u; the sum's error (an average of x, at most
// ln 1024, and 22 additions: 42 u) is one factor common to the token's scores.  The difference of two is
// thus off by at most 42 + 2 * 5 = 52 u of the largest score.  sigmoid: the exponential is off by
// (1.5 |l| + 2) u, which s (1 - s) makes 0.9 u, and the sum and a 1-ulp reciprocal add 3 u: 8 u for two.
// Adding the bias rounds by |c| u each, and cutting a key drops less than kPer ulp = 2 kPer u |c|.  For
// group scores (sums of two) it is twice the scores' part, u for each |c| and for the sum.  Values that
// lie further apart are in the right order.  Keys of logits differ only as the logits do.
template <class In, int L, int I, bool kVec>
__global__ __launch_bounds__(kThreads) void gate_kernel(const In* __restrict__ logits, const GateArgs a)
{
    constexpr int kPer = 4 * I;
    constexpr int kTokens = 64 / L;                           // per wave
    constexpr uint32_t kPlace = kPer - 1;                     // key bits of the place in the lane
    constexpr uint32_t kMasked = 0x00800000u;                 // keys of -inf lie below, all others above
    constexpr float u = 0x1p-24f;
    static_assert((kPer & (kPer - 1)) == 0, "place bits");
    extern __shared__ __attribute__((aligned(16))) double lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int g = lane & (L - 1);
    // LDS: with groups each wave's float64 scratch, then k + 1 places (key, lane) for each token
    double* const wide = lds + static_cast<size_t>(wave) * a.scratch;
    uint2* const won = reinterpret_cast<uint2*>(lds + static_cast<size_t>(kWavesPerBlock) * a.scratch) +
                       (static_cast<size_t>(wave) * kTokens + lane / L) * (a.k + 1);
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / L;
    const bool live = t < a.T;
    const In* row = logits + (live ? t : a.T - 1) * a.E;
    const bool picked = a.topk_groups < a.groups;
    // this token needs float64: all do with more groups than lanes (65536 tokens of 64 experts 81 us in 8 groups,
    // 13 us in 4; of 256 experts 206 us in 32, 38 us in 16)
    bool unsure = picked && a.groups > L;
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
                l[4 * i + c] = v[c];
        }
        // As unsigned integers -inf and the negative NaNs are the largest floats, as signed ones the
        // positive NaNs.  Most tokens hold neither, and most gates fill their lanes.
        uint32_t largest = __float_as_uint(l[0]);
        int positive = __float_as_int(l[0]);
#pragma unroll
        for (int q = 1; q < kPer; ++q) {
            largest = max(largest, __float_as_uint(l[q]));
            positive = max(positive, __float_as_int(l[q]));
        }
        const bool full = a.E == 4 * L * I;
        const bool masks = !full || __any(largest >= 0xff800000u);
        const bool nan = largest > 0xff800000u || positive > 0x7f800000;
        if (!full) {
#pragma unroll
            for (int q = 0; q < kPer; ++q)
                if (4 * (L * (q / 4) + g) + (kVec ? 0 : q % 4) >= a.E)
                    l[q] = -__builtin_inff();
        }
        const bool by_logit = a.bias == nullptr;
        float inv = 1.0f, m = 0.0f;                           // score = numerator * inv
        float c[kPer];                                        // numerators, then what the experts are compared by
        if (a.sigmoid) {
            if (!by_logit || picked) {
#pragma unroll
                for (int q = 0; q < kPer; ++q)
                    c[q] = __builtin_amdgcn_rcpf(1.0f + fast_exp(-l[q]));
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
                c[q] = fast_exp(l[q] - m);
                total += c[q];
            }
            total = reduce<L>(total, Add{});
            unsure |= !(total <= 2048.0f);                    // a +inf logit
            inv = total == 0.0f ? 1.0f : 1.0f / total;
        }
        const float score_err = a.sigmoid ? 8 * u : 52 * u * inv;    // of the difference of two scores
        if (!by_logit || picked) {
#pragma unroll
            for (int i = 0; i < I; ++i) {
                const int e = 4 * (L * i + g);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float b = by_logit ? 0.0f : a.bias[kVec ? min(e, a.E - 4) + q : min(e + q, a.E - 1)];
                    c[4 * i + q] = c[4 * i + q] * inv + b;
                }
            }
            if (masks) {
#pragma unroll
                for (int q = 0; q < kPer; ++q)
                    c[q] = l[q] == -__builtin_inff() ? -__builtin_inff() : c[q];
            }
        }
        unsure |= reduce<L>(nan ? 1 : 0, Add{}) != 0;
        uint32_t keep[I];                                     // per vector: all ones, or 0 if its group is out
        uint32_t dropped = 0;                                 // bit q: the group of c[q] alone is out
#pragma unroll
        for (int i = 0; i < I; ++i)
            keep[i] = ~0u;
        // the n-th largest of the lanes' keys (V of them each); equal keys count once
        const auto nth = [](const auto& keys, int V, int n) {
            uint32_t last = 0;
            for (int j = 0; j < n; ++j) {
                uint32_t d = last - 1 - keys[0];
#pragma unroll
                for (int i = 1; i < V; ++i)
                    d = min(d, last - 1 - keys[i]);
                last = last - 1 - reduce<L>(d, MinU{});
            }
            return last;
        };
        // the two largest over 1 << shift neighbouring lanes
        const auto join = [](int shift, float& b1, float& b2) {
            const auto with = [&](float o1, float o2) {
                b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
                b1 = fmaxf(b1, o1);
            };
            if (L > 1 && shift > 0)
                with(exchange<0>(b1), exchange<0>(b2));
            if (L > 2 && shift > 1)
                with(exchange<1>(b1), exchange<1>(b2));
            if (L > 4 && shift > 2)
                with(exchange<2>(b1), exchange<2>(b2));
            if (L > 8 && shift > 3)
                with(exchange<3>(b1), exchange<3>(b2));
        };
        // equal scores among the kept groups, or the first one dropped not clearly below the last kept
        const auto open = [&](uint32_t last, int kept, int lanes, float out, float size) {
            return reduce<L>(kept, Add{}) != lanes ||
                   !(unordered(last) - reduce<L>(out, Max{}) > 2 * score_err + 8 * u * reduce<L>(size, Max{}));
        };
        const auto group_score = [&](float b1, float b2, float& size) {
            const bool two = a.group_top == 2 && b2 > -__builtin_inff();
            size = fmaxf(size, b1 > -__builtin_inff() ? fabsf(b1) + (two ? fabsf(b2) : 0.0f) : 0.0f);
            return two ? b1 + b2 : b1;
        };
        if (picked && a.group_shift < 0 && !__all(unsure)) {
            // groups of any size: the values go to LDS, 1 << part_shift lanes read a group's
            float* const cs = reinterpret_cast<float*>(wide) + (lane / L) * (a.E + a.groups);
            float* const gs = cs + a.E;
#pragma unroll
            for (int q = 0; q < kPer; ++q)
                if (4 * (L * (q / 4) + g) + q % 4 < a.E)
                    cs[4 * (L * (q / 4) + g) + q % 4] = c[q];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            const int grp = g >> a.part_shift, parts = 1 << a.part_shift;
            float b1 = -__builtin_inff(), b2 = -__builtin_inff(), size = 0.0f, out = -__builtin_inff();
            if (grp < a.groups)
                for (int i = g & (parts - 1); i < a.per; i += parts) {
                    const float v = cs[grp * a.per + i];
                    b2 = fmaxf(b2, fminf(b1, v));
                    b1 = fmaxf(b1, v);
                }
            join(a.part_shift, b1, b2);
            const float mine = group_score(b1, b2, size);
            const uint32_t gkey[1] = {grp < a.groups ? ordered(mine) : 0};
            if (grp < a.groups)
                gs[grp] = mine;
            const uint32_t last = nth(gkey, 1, a.topk_groups);
            const bool in = gkey[0] >= last;
            if (!in && grp < a.groups)
                out = mine;
            unsure |= open(last, in ? 1 : 0, a.topk_groups << a.part_shift, out, size);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            const float least = unordered(last);
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                const int e = min(4 * (L * (q / 4) + g) + q % 4, a.E - 1);
                dropped |= gs[e * a.per_inverse >> 20] >= least ? 0u : 1u << q;
            }
        } else if (picked) {
            // a group is an aligned run of 1 << group_shift lanes of one vector
            float mine[I], size = 0.0f;
            uint32_t gkey[I];
#pragma unroll
            for (int i = 0; i < I; ++i) {
                const float h1 = fmaxf(c[4 * i], c[4 * i + 1]), l1 = fminf(c[4 * i], c[4 * i + 1]);
                const float h2 = fmaxf(c[4 * i + 2], c[4 * i + 3]), l2 = fminf(c[4 * i + 2], c[4 * i + 3]);
                float b1 = fmaxf(h1, h2), b2 = fmaxf(fminf(h1, h2), h1 >= h2 ? l1 : l2);
                join(a.group_shift, b1, b2);
                mine[i] = group_score(b1, b2, size);
                gkey[i] = (L * i + g) >> a.group_shift < a.groups ? ordered(mine[i]) : 0;
            }
            const uint32_t last = nth(gkey, I, a.topk_groups);
            float out = -__builtin_inff();
            int kept = 0;
#pragma unroll
            for (int i = 0; i < I; ++i) {
                if (gkey[i] >= last) {
                    ++kept;
                } else {
                    keep[i] = 0;
                    out = fmaxf(out, gkey[i] != 0 ? mine[i] : -__builtin_inff());
                }
            }
            unsure |= open(last, kept, a.topk_groups << a.group_shift, out, size);
        }
        const bool id_key = std::is_same_v<In, uint16_t> && by_logit;
        uint32_t key[kPer];                                   // 0: no candidate
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            const uint32_t o = ordered(by_logit ? l[q] + 0.0f : c[q]);   // -0 becomes +0: equal logits tie
            key[q] = id_key ? (o & 0xffff0000u) | static_cast<uint32_t>(0xffff - (4 * (L * (q / 4) + g) + q % 4))
                            : (o & ~kPlace) | static_cast<uint32_t>(q);
        }
        if (picked) {
#pragma unroll
            for (int q = 0; q < kPer; ++q)
                key[q] &= keep[q / 4];
            if (a.group_shift < 0) {
#pragma unroll
                for (int q = 0; q < kPer; ++q)
                    key[q] &= (dropped >> q & 1) - 1;
            }
        }
        uint32_t last = 0;                                    // below every key: M - 1 wraps to the top
        int wins = 0;
        for (int j = 0; j <= a.k; ++j) {
            const uint32_t from = last - 1;
            uint32_t d = from - key[0];
#pragma unroll
            for (int q = 1; q < kPer; ++q)
                d = min(d, from - key[q]);
            const uint32_t all = reduce<L>(d, MinU{});
            last = from - all;                                // nothing left: 0, or wrapped above the one before
            if (d == all) {
                won[j] = uint2{last, static_cast<uint32_t>(g)};
                ++wins;
            }
            if (j == a.k - 1)
                unsure |= reduce<L>(wins, Add{}) != a.k;      // two lanes with one key
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        // winner j on lane j % L: in order if clearly above the next one (which may not exist after the last)
        float total = 0.0f, least = __builtin_inff(), n = 0.0f;
        int id = 0, bad = 0;
        const auto winner = [&](int j) {
            const uint2 w = won[j];
            id = id_key ? 0xffff - static_cast<int>(w.x & 0xffffu)
                        : 4 * (L * static_cast<int>((w.x & kPlace) >> 2) + static_cast<int>(w.y)) + static_cast<int>(w.x & 3);
            id = min(id, a.E - 1);
            const float x = load_logit(row + id);
            n = a.sigmoid ? 1.0f / (1.0f + expf(-x)) : exp_difference(x, m);
        };
        for (int j = g; j < a.k; j += L) {
            const uint32_t here = won[j].x, next = won[j + 1].x;
            const bool none = next == 0 || next >= here;
            if (here < kMasked || (none && j + 1 < a.k))
                bad = 1;
            if (!id_key && !none) {
                const float v = unordered(here & ~kPlace), w = unordered(next & ~kPlace);
                const float err = by_logit ? 0.0f : score_err + (2 * kPer + 4) * u * fmaxf(fabsf(v), fabsf(w));
                if (next >= kMasked && !(v - w > err))
                    bad = 1;
            }
            winner(j);
            total += n;
            least = fminf(least, n);
        }
        // scores near float32's smallest: their ratios need float64's range
        unsure |= reduce<L>(bad, Add{}) != 0 || -reduce<L>(-least, Max{}) < 0x1p-100f;
        const float factor = a.renormalize ? 1.0f / reduce<L>(total, Add{}) : inv;   // scale comes last: it may be of any size
        for (int j = g; j < a.k && live && !unsure; j += L) {
            if (a.k > L)
                winner(j);
            a.ids[t * a.k + j] = id;
            a.probs[t * a.k + j] = n * factor * a.scale;
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

// 1 + exp(-l) is infinite in float64 from here down: the largest float32 that is (-709.78271 of -709.782713).
constexpr float kZeroSigmoid = -0x1.62e430p9f;

struct GateBackwardArgs {
    int64_t T;
    int E, k, sigmoid, renormalize;
    float scale;
    const int32_t* ids;
    const float* dprobs;
};

__device__ __forceinline__ void store_logits4(float* p, const f32x4_t& v) { *reinterpret_cast<f32x4_t*>(p) = v; }
__device__ __forceinline__ void store_logits4(uint16_t* p, const f32x4_t& v)
{
    *reinterpret_cast<u32x2_t*>(p) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// dl of one token, scale times the following.  With w_j the unscaled weights and d_j = dprobs_j:
//   renormalised: q_j = w_j (d_j - sum_i d_i w_i), sigmoid times 1 - s_j; dl_e = the q_j with id e
//   otherwise: sigmoid dl_e = d_j s_j (1 - s_j); softmax dl_e = s_e (d_j [id_j = e] - sum_i d_i s_i)
// An id that occurs twice gets both; ids outside [0, E) are no slots.
//
// L lanes per token (at least k: lane j holds slot j).  The token's row of dl is put together in LDS -
// zeros (dense softmax: its exponentials), then the slots' values at their ids - and goes out in vectors
// of four; writing it is what the kernel costs.  An id held by two lanes is found by writing the lanes'
// numbers into the row and reading them back, and only then the lanes look at each other.  Bound by
// memory: 65536 x 256 bfloat16 in 11.3 us a call (30.4 us where every lane stored its own experts) moves 68
// MB at 6 TB/s, half of them stores; a token's 8 chosen logits lie in 3.6 of its row's 4 lines of 128 bytes.
// 8192 x 128 float32 of a dense softmax 5.8 us.
template <class In, int L, bool kVec>
__global__ __launch_bounds__(kThreads) void gate_backward_kernel(const In* __restrict__ logits,
                                                                 In* __restrict__ dlogits,
                                                                 const GateBackwardArgs a)
{
    extern __shared__ __attribute__((aligned(16))) float rows[];
    const int lane = threadIdx.x & 63;
    const int g = lane & (L - 1), base = lane & ~(L - 1);
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / L;
    const bool live = t < a.T;
    const int64_t at = (live ? t : a.T - 1) * a.E;
    const In* row = logits + at;
    float* const dl = rows + static_cast<size_t>(threadIdx.x / L) * ((a.E + 3) & ~3);
    int id = -1;
    float d = 0.0f, lj = -__builtin_inff();
    if (live && g < a.k) {
        id = a.ids[t * a.k + g];
        if (id < 0 || id >= a.E)
            id = -1;
        else {
            d = a.dprobs[t * a.k + g];
            lj = load_logit(row + id);
        }
    }
    const bool dense = !a.sigmoid && !a.renormalize;
    float q, spread = 0.0f;                                   // this slot's value; dense: the factor of the exponentials
    if (a.sigmoid) {
        // s = exp(min(l, 0)) / (1 + exp(-|l|)), 1 - s the other part of 1.  Renormalised, only the ratios of the s count:
        // all are divided by exp(min(largest l, 0)), which keeps them in float32's range however small they are.
        // Scores that float64 does not hold are zero, as in the gate.
        const float e = expf(-fabsf(lj)), part = 1.0f / (1.0f + e);
        const float rest = lj >= 0.0f ? e * part : part;
        if (a.renormalize) {
            const float m = fminf(reduce<L>(lj > kZeroSigmoid ? lj : -__builtin_inff(), Max{}), 0.0f);
            const float s = lj <= kZeroSigmoid ? 0.0f : (lj < 0.0f ? expf(lj - m) : 1.0f) * part;
            const float total = reduce<L>(s, Add{});
            const float w = total > 0.0f || total != total ? s / total : 0.0f;
            q = w * rest * (d - reduce<L>(d * w, Add{}));
        } else {
            q = d * (lj < 0.0f ? e : 1.0f) * part * rest;
        }
    } else if (a.renormalize) {
        const float m = reduce<L>(lj, Max{});
        const float ex = lj == -__builtin_inff() ? 0.0f : expf(lj - m);
        const float total = reduce<L>(ex, Add{});
        const float w = total > 0.0f || total != total ? ex / total : 0.0f;
        q = w * (d - reduce<L>(d * w, Add{}));
    } else {
        float m = -__builtin_inff(), total = 0.0f;
        if (kVec) {
            for (int e = 4 * g; e < a.E; e += 4 * L) {
                float v[4];
                load_logits4(row + e, v);
                m = fmaxf(fmaxf(m, fmaxf(v[0], v[1])), fmaxf(v[2], v[3]));
                *reinterpret_cast<f32x4_t*>(dl + e) = f32x4_t{v[0], v[1], v[2], v[3]};
            }
        } else {
            for (int e = g; e < a.E; e += L) {
                dl[e] = load_logit(row + e);
                m = fmaxf(m, dl[e]);
            }
        }
        m = reduce<L>(m, Max{});
        const auto weight = [&](float v) { return v == -__builtin_inff() ? 0.0f : expf(v - m); };
        if (kVec) {
            for (int e = 4 * g; e < a.E; e += 4 * L) {
                f32x4_t v = *reinterpret_cast<f32x4_t*>(dl + e);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    v[c] = weight(v[c]);
                    total += v[c];
                }
                *reinterpret_cast<f32x4_t*>(dl + e) = v;
            }
        } else {
            for (int e = g; e < a.E; e += L) {
                dl[e] = weight(dl[e]);
                total += dl[e];
            }
        }
        total = reduce<L>(total, Add{});
        const float inv = total > 0.0f || total != total ? 1.0f / total : 0.0f;
        q = d * weight(lj) * inv;
        spread = -inv * reduce<L>(q, Add{}) * a.scale;
    }
    q *= a.scale;
    // ids that several slots name: each such lane takes the sum of theirs, in slot order
    int* const mark = reinterpret_cast<int*>(dl);
    float under = 0.0f;                                       // dense: the exponential at this slot's id
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (dense && id >= 0)
        under = dl[id];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (id >= 0)
        mark[id] = g;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const bool shared = id >= 0 && mark[id] != g;
    if (__any(shared)) {
        float sum = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const int oi = __shfl(id, base + j);
            const float oq = __shfl(q, base + j);
            sum += oi == id ? oq : 0.0f;
        }
        q = sum;
    }
    if (!dense) {
        for (int e = 4 * g; e < a.E; e += 4 * L)              // the row has room for whole vectors
            *reinterpret_cast<f32x4_t*>(dl + e) = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (dense) {
        for (int e = g; e < a.E; e += L)                      // the marked places are written next
            dl[e] *= spread;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    if (id >= 0)
        dl[id] = dense ? under * spread + q : q;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (live) {
        In* out = dlogits + at;
        if (kVec) {
            for (int e = 4 * g; e < a.E; e += 4 * L)
                store_logits4(out + e, *reinterpret_cast<f32x4_t*>(dl + e));
        } else {
            for (int e = g; e < a.E; e += L)
                store_logit(out + e, dl[e]);
        }
    }
}

// Groups of `per` experts as whole vectors of 1 << b neighbouring lanes (at most a row of 16, and at most
// a token's L): b, or -1.
int group_shift(int per, int L)
{
    for (int b = 0; b <= 4; ++b)
        if (per == 4 << b && (1 << b) <= L)
            return b;
    return -1;
}

// Tokens of one launch: at most 2^30 threads.
template <int L>
constexpr int64_t kLaunchTokens = (int64_t{1} << 30) / L;

template <class In, int L, int I>
hipError_t launch_gate_n(const In* logits, GateArgs a, hipStream_t s)
{
    a.group_shift = group_shift(a.E / a.groups, L);
    a.per = a.E / a.groups;
    a.per_inverse = ((1 << 20) + a.per - 1) / a.per;      // 1023 * 2^-20 < 1 / per: exact
    a.part_shift = 0;
    while (a.part_shift < 4 && (a.groups << (a.part_shift + 1)) <= L)
        ++a.part_shift;
    // one token in float64, or the wave's tokens in float32
    const bool wave = a.group_shift < 0 && a.groups <= L;
    a.scratch = a.groups > 1 ? (wave ? std::max(1, 32 / L) : 1) * (a.E + a.groups) : 0;
    const size_t lds = sizeof(double) * kWavesPerBlock * static_cast<size_t>(a.scratch) +
                       sizeof(uint2) * (kThreads / L) * static_cast<size_t>(a.k + 1);
    const bool vec = a.E % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % (4 * sizeof(In)) == 0;
    const int64_t T = a.T;
    for (int64_t t = 0; t < T; t += kLaunchTokens<L>) {
        a.T = std::min(kLaunchTokens<L>, T - t);
        const dim3 grid(static_cast<unsigned>(ceil_div(a.T * L, kThreads)));
        if (vec)
            gate_kernel<In, L, I, true><<<grid, dim3(kThreads), lds, s>>>(logits + t * a.E, a);
        else
            gate_kernel<In, L, I, false><<<grid, dim3(kThreads), lds, s>>>(logits + t * a.E, a);
        if (hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
        a.ids += a.T * a.k;
        a.probs += a.T * a.k;
    }
    return hipSuccess;
}

// The gate's lanes per token.  Four experts a lane where possible: shortest rounds.  With many tokens of more
// than 32 experts, up to 16 experts a lane: what a round costs beside the keys themselves (the exchanges,
// the winner) is then shared by more tokens of the wave.  Measured (us, four experts a lane / 16): 65536
// tokens of 32 experts 10 / 12, of 64 14.7 / 12.4, of 256 53 / 22; 8192 tokens of 64 experts 5.8 / 6.9, of 256
// 8.9 / 5.1; 4096 tokens of 256 6.5 / 7.2: taken from 32 waves a CU on.
template <class In>
hipError_t launch_gate_t(const In* logits, const GateArgs& a, hipStream_t s)
{
    if (a.E <= 8)
        return launch_gate_n<In, 2, 1>(logits, a, s);
    if (a.E <= 16)
        return launch_gate_n<In, 4, 1>(logits, a, s);
    if (a.E <= 32)
        return launch_gate_n<In, 8, 1>(logits, a, s);
    const int few = a.E <= 64 ? 16 : a.E <= 128 ? 32 : 64;
    const int lanes = a.E <= 64 ? 4 : a.E <= 128 ? 8 : a.E <= 256 ? 16 : 32;
    // groups as vectors, or at least no more groups than lanes, if the wider layout can have that
    const int per = a.E / a.groups;
    const bool fits = a.topk_groups == a.groups || group_shift(per, lanes) >= 0 ||
                      (group_shift(per, few) < 0 && (a.groups <= lanes || a.groups > few));
    const bool many = fits && ceil_div(a.T * few, 64) >= 32 * device_info().cu_count;
    if (a.E <= 64)
        return many ? launch_gate_n<In, 4, 4>(logits, a, s) : launch_gate_n<In, 16, 1>(logits, a, s);
    if (a.E <= 128)
        return many ? launch_gate_n<In, 8, 4>(logits, a, s) : launch_gate_n<In, 32, 1>(logits, a, s);
    if (a.E <= 256)
        return many ? launch_gate_n<In, 16, 4>(logits, a, s) : launch_gate_n<In, 64, 1>(logits, a, s);
    if (a.E <= 512)
        return many ? launch_gate_n<In, 32, 4>(logits, a, s) : launch_gate_n<In, 64, 2>(logits, a, s);
    return launch_gate_n<In, 64, 4>(logits, a, s);
}

template <class In, int L>
hipError_t launch_backward_n(const In* logits, In* dlogits, GateBackwardArgs a, hipStream_t s)
{
    const size_t lds = sizeof(float) * (kThreads / L) * static_cast<size_t>((a.E + 3) & ~3);
    const bool vec = a.E % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(dlogits)) % (4 * sizeof(In)) == 0;
    const int64_t T = a.T;
    for (int64_t t = 0; t < T; t += kLaunchTokens<L>) {
        a.T = std::min(kLaunchTokens<L>, T - t);
        const dim3 grid(static_cast<unsigned>(ceil_div(a.T * L, kThreads)));
        if (vec)
            gate_backward_kernel<In, L, true><<<grid, dim3(kThreads), lds, s>>>(logits + t * a.E, dlogits + t * a.E, a);
        else
            gate_backward_kernel<In, L, false><<<grid, dim3(kThreads), lds, s>>>(logits + t * a.E, dlogits + t * a.E, a);
        if (hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
        a.ids += a.T * a.k;
        a.dprobs += a.T * a.k;
    }
    return hipSuccess;
}

// Lanes per token: one per slot, and one per 16 experts.
template <class In>
hipError_t launch_backward_t(const In* logits, In* dlogits, const GateBackwardArgs& a, hipStream_t s)
{
    const int need = std::max(a.k, (a.E + 15) / 16);
    if (need <= 2)
        return launch_backward_n<In, 2>(logits, dlogits, a, s);
    if (need <= 4)
        return launch_backward_n<In, 4>(logits, dlogits, a, s);
    if (need <= 8)
        return launch_backward_n<In, 8>(logits, dlogits, a, s);
    if (need <= 16)
        return launch_backward_n<In, 16>(logits, dlogits, a, s);
    if (need <= 32)
        return launch_backward_n<In, 32>(logits, dlogits, a, s);
    return launch_backward_n<In, 64>(logits, dlogits, a, s);
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
    // groups of one expert each choose nothing that the k largest do not
    const bool alone = o.groups == E;
    a.groups = alone ? 1 : o.groups;
    a.topk_groups = alone ? 1 : o.topk_groups;
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
    return dtype == MOE_F32 ? launch_backward_t(static_cast<const float*>(logits), static_cast<float*>(dlogits), a, s)
                            : launch_backward_t(static_cast<const uint16_t*>(logits), static_cast<uint16_t*>(dlogits), a, s);
}

}  // namespace moe
