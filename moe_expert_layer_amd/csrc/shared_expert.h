// Host-side internals of the shared expert's operators: the gated block with its gradient, dropout and the low-rank
// adapters; launchers shared by api.cpp and the kernels.
#pragma once

#include <atomic>

#include "internal.h"
#include "moe_expert_layer.h"

namespace moe {

// Dropout as the kernels take it: a value is dropped where its 16 random bits are below threshold (0: no dropout, rng
// unread; 65536: everything), kept values are multiplied by scale.  rng: seed and offset on the device.
struct Dropout {
    const int64_t* rng;
    uint32_t threshold;
    float scale;
};

// n / d for 0 <= n < 2^31 as a product (Granlund and Montgomery, "Division by invariant integers using
// multiplication", PLDI 1994): with l = ceil(log2 d), m = floor(2^(31 + l) / d) + 1 < 2^32 + 1 gives
// n / d = floor(n m / 2^(31 + l)).
struct Divisor {
    uint64_t m;
    int shift;
    int d;
};
inline Divisor divisor(int d)
{
    int l = 0;
    while ((int64_t{1} << l) < d)
        ++l;
    return Divisor{(uint64_t{1} << (31 + l)) / static_cast<uint64_t>(d) + 1, 31 + l, d};
}

// Runs launch(first row, threads, workgroups of 256) over rows of `groups` groups of 8 columns, a thread each, with fewer
// than 2^31 threads a launch.
template <class F>
hipError_t for_groups(int64_t rows, int64_t groups, F launch)
{
    const int64_t step = ((int64_t{1} << 31) - 256) / groups;
    for (int64_t r = 0; r < rows; r += step) {
        const int n = static_cast<int>((rows - r < step ? rows - r : step) * groups);
        launch(r, n, static_cast<unsigned>(ceil_div(n, 256)));
        if (hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

// Raises one kernel's limit of dynamic LDS to `bytes` (more than 64 KiB), once per device.
struct LdsLimit {
    std::atomic<bool> done[64];
    hipError_t ensure(const void* kernel, int bytes)
    {
        int dev = 0;
        if (bytes <= 65536)
            return hipSuccess;
        if (hipError_t e = hipGetDevice(&dev); e != hipSuccess)
            return e;
        if (dev < 64 && done[dev])
            return hipSuccess;
        const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == hipSuccess && dev < 64)
            done[dev] = true;
        return e;
    }
};

// dropout.hip: out = [residual +] D(x), rows x cols values of MOE_F32 or MOE_BF16 (moe_dropout).
hipError_t launch_dropout(const void* x, const void* residual, int dtype, int64_t rows, int64_t cols, const Dropout& d,
                          void* out, hipStream_t s);

// Rows of a gated block or an adapter call: their number and 32-bit counters of tiles and steps of K stay far apart.
constexpr int64_t kMaxSharedRows = int64_t{1} << 28;

// gated.hip: the gated block and its gradient (moe_gated_projection, moe_gated_projection_backward).
struct GatedLayout {
    size_t x = 0, wg = 0, wu = 0;      // operands laid out for the products, where the caller's are not already
    size_t dgu = 0;                    // backward: the gradients of g and u
    size_t partial = 0;                // sums over parts of K
    int64_t dx_partial = 0;            // backward: bytes of dx's own, before those of the weights' gradients
    size_t total = 0;
};
GatedLayout gated_layout(const moe_gated& g, bool backward);
hipError_t launch_gated(const moe_gated& g, const Dropout& d, const void* x, const void* wg, const void* wu, void* h,
                        void* saved_gu, void* workspace, hipStream_t s);
hipError_t launch_gated_backward(const moe_gated& g, const Dropout& d, const void* x, const void* wg, const void* wu,
                                 const void* dh, const void* saved_gu, void* dx, void* dwg, void* dwu, void* workspace,
                                 hipStream_t s);

constexpr int kMaxAdapters = 1023;
constexpr int kMaxRank = 128;

// adapter.hip: out = base + each row's adapter (moe_adapter_add).
struct AdapterLayout {
    size_t count = 0, perm = 0, tiles = 0;   // the rows sorted by adapter
    size_t v = 0, part = 0;                  // x A, and its sums over parts of K
    size_t total = 0;
};
AdapterLayout adapter_layout(const moe_adapter& p);
hipError_t launch_adapter(const moe_adapter& p, const void* base, const void* x, const void* a, const void* b,
                          const int32_t* ids, const float* scale, const int32_t* ranks, void* out, void* workspace,
                          hipStream_t s);

}  // namespace moe
