// The gate with scores, a balance bias, expert groups and renormalised weights, and its gradient.
//
//   s = softmax(l) over the E experts, or sigmoid(l);   c = s + bias (c = -inf where l = -inf)
//   group score = sum of the group_top largest finite c of its E / G neighbouring experts
//   the topk_groups best groups stay; of their experts the k largest c, lower id first among equals
//   w_j = scale * s_j / (renormalize ? sum_i s_i : 1)
//
// Which experts are chosen is decided as in real arithmetic: without a bias the scores rise with the
// logits, so within the groups the logits themselves are compared; with a bias, and between groups,
// the scores are float64 (float32 scores of neighbouring experts often round to one value).
//
// A group of L lanes serves one token, as in the plain router: lane l holds experts l, l + L, ...
#include "common.h"
#include "internal.h"
#include "moe_expert_layer.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) { *p = f32_to_bf16(v); }

// Keys of the same order as the values: 1 for -inf (so that 0 is free for "not a candidate"), the
// largest for NaN.  -0 is made +0.
__device__ __forceinline__ uint64_t key_of(double c)
{
    if (c != c)
        return ~uint64_t{0};
    const uint64_t b = __builtin_bit_cast(uint64_t, c + 0.0);
    const uint64_t k = (b >> 63) != 0 ? ~b : b | (uint64_t{1} << 63);
    return c == -__builtin_inf() ? 1 : k;
}
__device__ __forceinline__ uint64_t key_of(float c)
{
    if (c != c)
        return ~uint64_t{0};
    const uint32_t b = __float_as_uint(c + 0.0f);
    const uint32_t k = (b >> 31) != 0 ? ~b : b | 0x80000000u;
    return c == -__builtin_inff() ? 1 : static_cast<uint64_t>(k) << 32;
}

__device__ __forceinline__ double exp_of(double v) { return exp(v); }
__device__ __forceinline__ float exp_of(float v) { return expf(v); }

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

struct GateArgs {
    const float* bias;       // may be null
    int64_t T;
    int E, k, groups, topk_groups, group_top, sigmoid, renormalize;
    float scale;
    int32_t* ids;
    float* probs;
};

// kWide: float64 scores, with bias and groups; otherwise float32 scores and selection by logits.
template <class In, int L, int kPer, bool kWide>
__global__ __launch_bounds__(kThreads) void gate_kernel(const In* __restrict__ logits, const GateArgs a)
{
    using V = std::conditional_t<kWide, double, float>;
    const int lane = threadIdx.x & 63;
    const int g = lane & (L - 1), base = lane & ~(L - 1);
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / L;
    const bool live = t < a.T;
    const In* row = logits + (live ? t : 0) * a.E;
    float l[kPer];
    float lmax = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = g + L * i;
        l[i] = e < a.E ? load_logit(row + e) : -__builtin_inff();
        lmax = fmaxf(lmax, l[i]);
    }
    // scores: s = num / den, den shared by the token
    V num[kPer];
    V den = V(1);
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            num[i] = V(1) / (V(1) + exp_of(-static_cast<V>(l[i])));
    } else {
        lmax = group_max(lmax, L);
        den = V(0);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            num[i] = l[i] == -__builtin_inff() ? V(0) : exp_of(static_cast<V>(l[i]) - static_cast<V>(lmax));
            den += num[i];
        }
        den = group_sum(den, L);
        if (den == V(0))
            den = V(1);                                       // every logit is -inf: scores 0
    }
    uint64_t key[kPer];                                       // 0: taken, or no candidate
    if constexpr (kWide) {
        double c[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = g + L * i;
            c[i] = num[i] / den + (a.bias != nullptr && e < a.E ? static_cast<double>(a.bias[e]) : 0.0);
            if (l[i] == -__builtin_inff())
                c[i] = -__builtin_inf();
            // a NaN logit makes every softmax score NaN: the logits decide then (NaN first)
            key[i] = e < a.E ? key_of(a.bias != nullptr && c[i] == c[i] ? c[i] : static_cast<double>(l[i])) : 0;
        }
        if (a.groups > 1) {
            // c of the token's experts, then the groups' scores, in LDS
            extern __shared__ __attribute__((aligned(16))) double lds[];
            double* const tc = lds + static_cast<size_t>(threadIdx.x / L) * (a.E + a.groups);
            double* const score = tc + a.E;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (g + L * i < a.E)
                    tc[g + L * i] = c[i];
            __syncthreads();
            const int per = a.E / a.groups;
            for (int q = g; q < a.groups; q += L) {
                double b1 = -__builtin_inf(), b2 = -__builtin_inf();
                for (int i = 0; i < per; ++i) {
                    const double v = tc[q * per + i];
                    b2 = fmax(b2, fmin(b1, v));
                    b1 = fmax(b1, v);
                }
                score[q] = a.group_top == 2 && b2 > -__builtin_inf() ? b1 + b2 : b1;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int q = min(g + L * i, a.E - 1) / per;
                const double mine = score[q];
                int rank = 0;
                for (int o = 0; o < a.groups; ++o)
                    rank += score[o] > mine || (score[o] == mine && o < q) ? 1 : 0;
                if (rank >= a.topk_groups)
                    key[i] = 0;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            key[i] = g + L * i < a.E ? key_of(l[i]) : 0;
    }
    int my_id = 0;
    V my_num = V(0);
    for (int j = 0; j < a.k; ++j) {
        uint64_t best = 0;
        int id = 0;
        V n = V(0);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (key[i] > best) {                              // lower ids first: i ascends
                best = key[i];
                id = g + L * i;
                n = num[i];
            }
#pragma unroll
        for (int off = L / 2; off >= 1; off >>= 1) {
            const uint64_t ob = __shfl_xor(static_cast<unsigned long long>(best), off);
            const int oi = __shfl_xor(id, off);
            const V on = __shfl_xor(n, off);
            if (ob > best || (ob == best && oi < id)) {
                best = ob;
                id = oi;
                n = on;
            }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (g + L * i == id)
                key[i] = 0;
        if (g == j) {
            my_id = id;
            my_num = n;
        }
    }
    (void)base;
    if (g >= a.k)
        my_num = V(0);
    if (a.renormalize) {
        den = group_sum(my_num, L);
        if (den == V(0))
            den = V(1);                                       // nothing but zero scores: weights 0
    }
    if (live && g < a.k) {
        a.ids[t * a.k + g] = my_id;
        a.probs[t * a.k + g] = static_cast<float>(my_num / den * static_cast<V>(a.scale));
    }
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

template <class In, int L, int kPer>
hipError_t launch_gate_n(const In* logits, const GateArgs& a, bool wide, hipStream_t s)
{
    const int64_t blocks = ceil_div(a.T * L, kThreads);
    if (blocks >= (int64_t{1} << 31))
        return hipErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(blocks));
    const size_t lds = a.groups > 1 ? sizeof(double) * (kThreads / L) * static_cast<size_t>(a.E + a.groups) : 0;
    if (wide)
        gate_kernel<In, L, kPer, true><<<grid, dim3(kThreads), lds, s>>>(logits, a);
    else
        gate_kernel<In, L, kPer, false><<<grid, dim3(kThreads), 0, s>>>(logits, a);
    return hipGetLastError();
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
    const bool wide = bias != nullptr || o.groups > 1;
    return with_lanes(a.E, [&](auto L, auto per) {
        return dtype == MOE_F32 ? launch_gate_n<float, L(), per()>(static_cast<const float*>(logits), a, wide, s)
                                : launch_gate_n<uint16_t, L(), per()>(static_cast<const uint16_t*>(logits), a, wide, s);
    });
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
