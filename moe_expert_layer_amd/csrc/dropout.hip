// Dropout of whole rows, with the residual it is added to: out = [residual +] D(x) (moe_dropout), one pass over the
// memory, the mask drawn in registers (dropout.h).  Memory bounds it: 16384 x 7168 bfloat16 with the residual 126 us, 5.6
// TB/s.
#include <algorithm>

#include "dropout.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;            // groups of 8 columns per thread, loaded together

// n groups of 8 columns (below 2^31), rows of `groups` of them; the first row is row0 of the call.
template <class T, bool kResidual>
__global__ __launch_bounds__(kThreads) void dropout_kernel(const T* x, const T* residual, T* out, int n, Divisor groups,
                                                           int cols, int64_t row0, Dropout d)
{
    const DropKey key = drop_key(d);
    Raw8<T> v[kPer], r[kPer];
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
            v[i] = load_raw<false>(x + p, cols - 8 * group[i]);
            if constexpr (kResidual)
                r[i] = load_raw<false>(residual + p, cols - 8 * group[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (group[i] < 0)
            continue;
        float y[8], w[8];
        v[i].values(y);
        drop8(y, d, key, static_cast<uint32_t>(group[i]), static_cast<uint32_t>(row0 + row[i]));
        if constexpr (kResidual) {
            r[i].values(w);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                y[e] += w[e];
        }
        store8(out + (row0 + row[i]) * cols + 8 * group[i], y, cols - 8 * group[i]);
    }
}

template <class T>
hipError_t launch(const void* x, const void* residual, int64_t rows, int64_t cols, const Dropout& d, void* out,
                  hipStream_t s)
{
    const int64_t groups = ceil_div(cols, 8);
    const Divisor div = divisor(static_cast<int>(groups));
    // the group numbers of one launch stay below 2^31 - 1024, whatever the workgroup
    const int64_t step = ((int64_t{1} << 31) - kThreads * kPer) / groups;
    for (int64_t r = 0; r < rows; r += step) {
        const int n = static_cast<int>(std::min(step, rows - r) * groups);
        const dim3 grid(static_cast<unsigned>(ceil_div(n, kThreads * kPer)));
        if (residual != nullptr)
            dropout_kernel<T, true><<<grid, kThreads, 0, s>>>(static_cast<const T*>(x), static_cast<const T*>(residual),
                                                              static_cast<T*>(out), n, div, static_cast<int>(cols), r, d);
        else
            dropout_kernel<T, false><<<grid, kThreads, 0, s>>>(static_cast<const T*>(x), nullptr, static_cast<T*>(out), n,
                                                               div, static_cast<int>(cols), r, d);
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
