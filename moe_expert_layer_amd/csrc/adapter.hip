// Low-rank adapters of many requests beside a shared projection (moe_adapter_add):
//   v[t] = scale[a] x[t] A[a],  out[t] = base[t] + v[t] B[a],  a = ids[t].
#include "dropout.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <class T>
__device__ __forceinline__ float to_float(T v)
{
    if constexpr (sizeof(T) == 2)
        return bf16_to_f32(v);
    else
        return v;
}

__device__ __forceinline__ int rank_of(const int32_t* ranks, int a, int R)
{
    return ranks == nullptr ? R : min(max(ranks[a], 0), R);
}

template <class T>
__global__ __launch_bounds__(kThreads) void adapter_shrink(const T* __restrict__ x, const T* __restrict__ A,
                                                           const int32_t* __restrict__ ids, const float* __restrict__ scale,
                                                           const int32_t* __restrict__ ranks, float* __restrict__ v, int K,
                                                           int L, int R)
{
    const int64_t t = blockIdx.x;
    const int a = ids[t];
    if (a < 0 || a >= L)
        return;
    const int rank = rank_of(ranks, a, R);
    for (int r = threadIdx.x; r < rank; r += kThreads) {
        float sum = 0.0f;
        for (int k = 0; k < K; ++k)
            sum += to_float(x[t * K + k]) * to_float(A[(static_cast<int64_t>(a) * K + k) * R + r]);
        v[t * R + r] = scale == nullptr ? sum : sum * scale[a];
    }
}

template <class T>
__global__ __launch_bounds__(kThreads) void adapter_expand(const T* base, const T* __restrict__ B,
                                                           const int32_t* __restrict__ ids, const int32_t* __restrict__ ranks,
                                                           const float* __restrict__ v, T* out, int N, int L, int R)
{
    const int64_t t = blockIdx.x;
    const int a = ids[t];
    const int rank = a < 0 || a >= L ? 0 : rank_of(ranks, a, R);
    for (int n = threadIdx.x; n < N; n += kThreads) {
        float sum = 0.0f;
        for (int r = 0; r < rank; ++r)
            sum += v[t * R + r] * to_float(B[(static_cast<int64_t>(a) * R + r) * N + n]);
        sum += to_float(base[t * N + n]);
        if constexpr (sizeof(T) == 2)
            out[t * N + n] = f32_to_bf16(sum);
        else
            out[t * N + n] = sum;
    }
}

template <class T>
hipError_t launch(const moe_adapter& p, const void* base, const void* x, const void* a, const void* b, const int32_t* ids,
                  const float* scale, const int32_t* ranks, void* out, float* v, hipStream_t s)
{
    const dim3 grid(static_cast<unsigned>(p.T));
    adapter_shrink<T><<<grid, kThreads, 0, s>>>(static_cast<const T*>(x), static_cast<const T*>(a), ids, scale, ranks, v,
                                                static_cast<int>(p.K), static_cast<int>(p.L), static_cast<int>(p.R));
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    adapter_expand<T><<<grid, kThreads, 0, s>>>(static_cast<const T*>(base), static_cast<const T*>(b), ids, ranks, v,
                                                static_cast<T*>(out), static_cast<int>(p.N), static_cast<int>(p.L),
                                                static_cast<int>(p.R));
    return hipGetLastError();
}

}  // namespace

AdapterLayout adapter_layout(const moe_adapter& p)
{
    AdapterLayout L;
    L.total = align_up(static_cast<size_t>(p.T) * p.R * 4);
    return L;
}

hipError_t launch_adapter(const moe_adapter& p, const void* base, const void* x, const void* a, const void* b,
                          const int32_t* ids, const float* scale, const int32_t* ranks, void* out, void* workspace,
                          hipStream_t s)
{
    if (p.T == 0)
        return hipSuccess;
    float* const v = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + adapter_layout(p).v);
    return p.dtype == MOE_F32 ? launch<float>(p, base, x, a, b, ids, scale, ranks, out, v, s)
                              : launch<uint16_t>(p, base, x, a, b, ids, scale, ranks, out, v, s);
}

}  // namespace moe
