// Dropout of whole rows, with the residual it is added to: out = [residual +] D(x) (moe_dropout), one pass over the
// memory, the mask drawn in registers (dropout.h).
#include <algorithm>

#include "dropout.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;            // groups of 8 columns per thread, loaded together

// n groups of 8 columns (below 2^31), rows of `groups` of them; the first row is row0 of the call.
template <class T, bool kResidual>
__global__ __launch_bounds__(kThreads) void dropout_kernel(const T* x, const T* residual, T* out, int n, Divisor groups,
                                                           int cols, int64_t row0, bool vec, Dropout d)
{
    const DropKey key = drop_key(d);
    float v[kPer][8], r[kPer][8];
    int row[kPer], group[kPer];
    const int first = blockIdx.x * (kThreads * kPer) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int at = first + i * kThreads;
        row[i] = static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(at)) * groups.m) >> groups.shift);
        group[i] = at - row[i] * groups.d;
        if (at >= n || at < 0)
            group[i] = -1;
        if (group[i] >= 0) {
            const int64_t p = (row0 + row[i]) * cols + 8 * group[i];
            load8(v[i], x + p, cols - 8 * group[i], vec);
            if constexpr (kResidual)
                load8(r[i], residual + p, cols - 8 * group[i], vec);
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (group[i] < 0)
            continue;
        drop8(v[i], d, key, static_cast<uint32_t>(group[i]), static_cast<uint32_t>(row0 + row[i]));
        if constexpr (kResidual) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[i][e] += r[i][e];
        }
        store8(out + (row0 + row[i]) * cols + 8 * group[i], v[i], cols - 8 * group[i], vec);
    }
}

template <class T>
hipError_t launch(const void* x, const void* residual, int64_t rows, int64_t cols, const Dropout& d, void* out,
                  hipStream_t s)
{
    const auto aligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    const bool vec = cols * sizeof(T) % 16 == 0 && aligned(x) && aligned(out) && (residual == nullptr || aligned(residual));
    const int64_t groups = ceil_div(cols, 8);
    const Divisor div = divisor(static_cast<int>(groups));
    // the group numbers of one launch stay below 2^31 - 1024, whatever the workgroup
    const int64_t step = ((int64_t{1} << 31) - kThreads * kPer) / groups;
    for (int64_t r = 0; r < rows; r += step) {
        const int n = static_cast<int>(std::min(step, rows - r) * groups);
        const dim3 grid(static_cast<unsigned>(ceil_div(n, kThreads * kPer)));
        if (residual != nullptr)
            dropout_kernel<T, true><<<grid, kThreads, 0, s>>>(static_cast<const T*>(x), static_cast<const T*>(residual),
                                                              static_cast<T*>(out), n, div, static_cast<int>(cols), r, vec, d);
        else
            dropout_kernel<T, false><<<grid, kThreads, 0, s>>>(static_cast<const T*>(x), nullptr, static_cast<T*>(out), n,
                                                               div, static_cast<int>(cols), r, vec, d);
        if (hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_dropout(const void* x, const void* residual, int dtype, int64_t rows, int64_t cols, const Dropout& d,
                          void* out, hipStream_t s)
{
    return dtype == MOE_F32 ? launch<float>(x, residual, rows, cols, d, out, s)
                            : launch<uint16_t>(x, residual, rows, cols, d, out, s);
}

}  // namespace moe
