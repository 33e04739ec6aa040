// The gated product of few rows (up to 64) on gfx950: g = x Wg and u = x Wu with the epilogues of the gated block, and the
// joining of sums over parts of K.
//
// What bounds it is the weights' way from memory, so they take the shortest: a lane loads 4 adjacent columns of 8
// consecutive k rows (of one matrix) straight into registers.  bfloat16: v_perm_b32 turns the 8 x 4 block into four MFMA
// operands of 8 k each (v_mfma_f32_16x16x32_bf16, the weights as the first operand); lane l of operand j holds column
// 4 (l % 16) + j, which leaves every lane of the result with 16 adjacent columns of one row.  float32: the words are
// v_mfma_f32_16x16x4_f32 operands as they are, eight of one k per lane group, exact products.  Nothing of the weights goes
// through LDS, and rows of any width and alignment are read the same way.
// A workgroup takes 64 columns of both matrices; its waves take K in turn, 32 rows at a time with the next 32 in flight,
// and join their sums through LDS in a fixed order.  With few columns K is cut over workgroups too.
#include <algorithm>

#include "gated_epilogue.h"

namespace moe {
namespace {

constexpr int kCols = 64;                 // columns per workgroup and matrix
constexpr int kBatch = 32;                // k rows per wave and step

// Four adjacent values as loaded.
template <class T>
struct Raw4;
template <>
struct Raw4<uint16_t> {
    u32x2_t w;
};
template <>
struct Raw4<float> {
    f32x4_t w;
};
typedef u32x2_t __attribute__((aligned(2))) u32x2_any_t;

// The first n of four values at p, the others zero and not read.
__device__ __forceinline__ Raw4<uint16_t> load4(const uint16_t* p, int n)
{
    Raw4<uint16_t> r{u32x2_t{0, 0}};
    if (n >= 4) {
        r.w = *reinterpret_cast<const u32x2_any_t*>(p);
    } else if (n > 0) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < n)
                r.w[i / 2] |= static_cast<uint32_t>(p[i]) << (16 * (i % 2));
    }
    return r;
}
__device__ __forceinline__ Raw4<float> load4(const float* p, int n)
{
    Raw4<float> r{f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}};
    if (n >= 4) {
        r.w = *reinterpret_cast<const f32x4_any_t*>(p);
    } else if (n > 0) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < n)
                r.w[i] = p[i];
    }
    return r;
}

// One step of a wave: 32 k of 64 columns of both matrices, and of kRB blocks of 16 rows of x.
template <class T, int kRB>
struct Step {
    Raw4<T> w[2][8];
    Raw8<T> x[kRB];
};

template <class T, int kRB>
__device__ __forceinline__ void multiply(f32x4_t (&acc)[2][4][kRB], const Step<T, kRB>& s)
{
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u32x4_t f;
                const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    f[i] = __builtin_amdgcn_perm(s.w[m][2 * i + 1].w[j >> 1], s.w[m][2 * i].w[j >> 1], sel);
#pragma unroll
                for (int b = 0; b < kRB; ++b)
                    acc[m][j][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, f),
                                                                           __builtin_bit_cast(bf16x8_t, s.x[b].w),
                                                                           acc[m][j][b], 0, 0, 0);
            }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int b = 0; b < kRB; ++b)
                        acc[m][j][b] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                            s.w[m][i].w[j], i < 4 ? s.x[b].a[i & 3] : s.x[b].b[i & 3], acc[m][j][b], 0, 0, 0);
    }
}

template <class T, int kRB, int kWaves, int kEpi>
__global__ __launch_bounds__(64 * kWaves, sizeof(T) == 2 && kRB == 1 ? 2 : 1) void gated_rows_kernel(RowsArgs g)
{
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    f32x4_t* const join = reinterpret_cast<f32x4_t*>(smem);            // [wave][matrix][j][row block][lane]
    const EpiArgs& e = g.e;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = blockIdx.x * kCols, part = blockIdx.y;
    const int batches = (g.K + kBatch - 1) / kBatch;
    const int b0 = static_cast<int>(static_cast<int64_t>(batches) * part / e.parts);
    const int b1 = static_cast<int>(static_cast<int64_t>(batches) * (part + 1) / e.parts);
    const int kg = 8 * (lane >> 4), col = n0 + 4 * (lane & 15), left = e.N - col;
    const T* const w0 = static_cast<const T*>(g.wg) + col;
    const T* const w1 = static_cast<const T*>(g.wu) + col;
    const T* x[kRB];
#pragma unroll
    for (int b = 0; b < kRB; ++b)                          // rows past the last repeat it and are not written
        x[b] = static_cast<const T*>(g.x) + static_cast<int64_t>(min(16 * b + (lane & 15), e.M - 1)) * g.K;

    const auto load = [&](Step<T, kRB>& s, int batch) {
        const int k = kBatch * batch + kg, n = batch < b1 ? left : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t at = static_cast<int64_t>(k + i) * e.N;
            s.w[0][i] = load4(w0 + at, k + i < g.K ? n : 0);
            s.w[1][i] = load4(w1 + at, k + i < g.K ? n : 0);
        }
#pragma unroll
        for (int b = 0; b < kRB; ++b)
            s.x[b] = load_raw<false>(x[b] + k, batch < b1 ? g.K - k : 0);
    };
    f32x4_t acc[2][4][kRB];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int b = 0; b < kRB; ++b)
                acc[m][j][b] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    Step<T, kRB> s0, s1;
    load(s0, b0 + wave);
    for (int b = b0 + wave; b < b1; b += 2 * kWaves) {
        load(s1, b + kWaves);
        multiply<T, kRB>(acc, s0);
        load(s0, b + 2 * kWaves);
        multiply<T, kRB>(acc, s1);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int b = 0; b < kRB; ++b)
                join[(((wave * 2 + m) * 4 + j) * kRB + b) * 64 + lane] = acc[m][j][b];
    __syncthreads();
    const DropKey key = drop_key(e.drop);
    // a lane's 16 columns of a row (register r, operand j: column 4 r + j) in two runs of 8
    for (int u = tid; u < 128 * kRB; u += 64 * kWaves) {
        const int h = u & 1, l = (u >> 1) & 63, b = u >> 7;
        const int row = 16 * b + (l & 15), c = n0 + 16 * (l >> 4) + 8 * h;
        if (row >= e.M || c >= e.N)
            continue;
        float v[2][8] = {};
        for (int w = 0; w < kWaves; ++w)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float* p = reinterpret_cast<const float*>(&join[(((w * 2 + m) * 4 + j) * kRB + b) * 64 + l]) + 2 * h;
                    v[m][j] += p[0];
                    v[m][4 + j] += p[1];
                }
        if (e.partial != nullptr) {
            store8(partial_at(e, part, 0, row, c), v[0], 8);
            store8(partial_at(e, part, 1, row, c), v[1], 8);
        } else {
            finish8<kEpi, sizeof(T) == 4>(e, key, v[0], v[1], 0, row, c);
        }
    }
}

// The results from the sums of all parts: a thread takes 8 columns of a row (of both matrices where they are gated).
template <int kEpi, bool kF32>
__global__ __launch_bounds__(256) void gated_finish_kernel(EpiArgs e, Divisor groups, int n, int64_t row0)
{
    const int at = blockIdx.x * 256 + threadIdx.x;
    if (at >= n)
        return;
    const int r = static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(at)) * groups.m) >> groups.shift);
    const int col = 8 * (at - r * groups.d);
    const int64_t row = row0 + r;
    const int mat = kEpi == kEpiOut ? blockIdx.y : 0;
    const DropKey key = kEpi == kEpiOut ? DropKey{} : drop_key(e.drop);
    constexpr int kMats = kEpi == kEpiOut ? 1 : 2, kAhead = 8;             // the parts' loads go out eight at a time
    float v[2][8] = {};
    for (int p0 = 0; p0 < e.parts; p0 += kAhead) {
        Raw8<float> a[kAhead][kMats];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int m = 0; m < kMats; ++m)
                a[i][m] = load_raw<true>(partial_at(e, p0 + i, mat + m, row, col), p0 + i < e.parts ? 8 : 0);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int m = 0; m < kMats; ++m) {
                float f[8];
                a[i][m].values(f);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    v[m][c] += f[c];
            }
    }
    finish8<kEpi, kF32>(e, key, v[0], v[1], mat, row, col);
}

template <class T, int kRB, int kWaves, int kEpi>
hipError_t launch_rows(const RowsArgs& g, hipStream_t s)
{
    constexpr int kLds = kWaves * kRB * 8 * 64 * 16;
    static LdsLimit limit;
    if (hipError_t e = limit.ensure(reinterpret_cast<const void*>(&gated_rows_kernel<T, kRB, kWaves, kEpi>), kLds);
        e != hipSuccess)
        return e;
    const dim3 grid(static_cast<unsigned>(ceil_div(g.e.N, kCols)), g.e.parts);
    gated_rows_kernel<T, kRB, kWaves, kEpi><<<grid, 64 * kWaves, kLds, s>>>(g);
    return hipGetLastError();
}

template <class T, int kEpi>
hipError_t launch_blocks(const RowsArgs& g, hipStream_t s)
{
    return g.e.M <= 16 ? launch_rows<T, 1, 8, kEpi>(g, s) : g.e.M <= 32 ? launch_rows<T, 2, 8, kEpi>(g, s)
                                                                     : launch_rows<T, 4, 4, kEpi>(g, s);
}

}  // namespace

int gated_rows_parts(int64_t M, int64_t K, int64_t N)
{
    const int64_t tiles = ceil_div(N, kCols), waves = M <= 32 ? 8 : 4;
    return tiles >= 128 ? 1 : static_cast<int>(std::clamp<int64_t>(256 / tiles, 1, std::max<int64_t>(1, ceil_div(K, kBatch) / waves)));
}

hipError_t launch_gated_rows(Epi epi, int dtype, const RowsArgs& g, hipStream_t s)
{
    if (dtype == MOE_F32)
        return epi == kEpiGated ? launch_blocks<float, kEpiGated>(g, s) : launch_blocks<float, kEpiGatedBwd>(g, s);
    return epi == kEpiGated ? launch_blocks<uint16_t, kEpiGated>(g, s) : launch_blocks<uint16_t, kEpiGatedBwd>(g, s);
}

hipError_t launch_gated_finish(Epi epi, int dtype, const EpiArgs& e, hipStream_t s)
{
    const int64_t groups = ceil_div(e.N, 8);
    const Divisor div = divisor(static_cast<int>(groups));
    return for_groups(e.M, groups, [&](int64_t r, int n, unsigned blocks) {
        const dim3 grid(blocks, epi == kEpiOut ? e.mats : 1);
        if (dtype == MOE_F32) {
            if (epi == kEpiGated)
                gated_finish_kernel<kEpiGated, true><<<grid, 256, 0, s>>>(e, div, n, r);
            else if (epi == kEpiGatedBwd)
                gated_finish_kernel<kEpiGatedBwd, true><<<grid, 256, 0, s>>>(e, div, n, r);
            else
                gated_finish_kernel<kEpiOut, true><<<grid, 256, 0, s>>>(e, div, n, r);
        } else {
            if (epi == kEpiGated)
                gated_finish_kernel<kEpiGated, false><<<grid, 256, 0, s>>>(e, div, n, r);
            else if (epi == kEpiGatedBwd)
                gated_finish_kernel<kEpiGatedBwd, false><<<grid, 256, 0, s>>>(e, div, n, r);
            else
                gated_finish_kernel<kEpiOut, false><<<grid, 256, 0, s>>>(e, div, n, r);
        }
    });
}

}  // namespace moe
