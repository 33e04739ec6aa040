// int8 rows: one float32 scale per row, codes -127 .. 127.
//
//   scale = max|x| / 127,   code = round_to_nearest_even(127 x / max|x|)
//
// The code is that of the real quotient: x and the maximum are brought to the maximum's binade by an
// exact power of two, and for bfloat16 the product 127 x is exact, a quotient that is not a half lies
// at least 2^-9 away from one, and one residual step makes the quotient right to less than an ulp (and
// exact where it is a half), so the rounding cannot go to the wrong side.  For float32 values a
// quotient within 2^-12 of a half is decided again in float64, where 127 x is exact.
//
// Bound by memory: every value is read once and kept in registers between the two steps (16384 x 8192
// float32 rows in 127 us, 5.3 TB/s of reads and writes; 16384 x 7168 bfloat16 in 71 us).
#include <algorithm>

#include "common.h"
#include "int8_gate.h"
#include "int8_tiles.h"

namespace moe {
namespace {

constexpr int kThreads = 256;       // of most kernels; one row's quantisation takes kWideThreads where rows are few
constexpr int kWideThreads = 1024;
constexpr int kVec = 8;
constexpr uint32_t kInfBits = 0x7f800000u;

// Rows (workgroups) along the grid's first axis: a launch takes less than 2^32 threads along one.  More
// rows continue along the third axis.
constexpr int64_t kGridRows = int64_t{1} << 21;

dim3 row_grid(int64_t rows, int64_t columns = 1)
{
    const int64_t x = std::min(rows, kGridRows);
    return dim3(static_cast<unsigned>(x), static_cast<unsigned>(columns), static_cast<unsigned>(ceil_div(rows, x)));
}
__device__ __forceinline__ int64_t grid_row()
{
    return static_cast<int64_t>(blockIdx.z) * gridDim.x + blockIdx.x;
}

// A row's constants: y = x * 2^-e lies in (-2, 2).
struct RowCode {
    float amax;      // maximum in [1, 2)
    float inv;       // 1 / amax
    int shift;       // -e
    bool finite;     // false: the row holds an infinity or NaN
    float scale;
};

__device__ __forceinline__ RowCode row_code(uint32_t amax_bits)
{
    RowCode c;
    c.finite = amax_bits < kInfBits;
    const float amax = __uint_as_float(amax_bits);
    const int e = amax_bits == 0 || !c.finite ? 0 : floor_log2_pos(amax_bits);
    c.shift = -e;
    c.amax = amax_bits == 0 || !c.finite ? 1.0f : ldexpf(amax, -e);
    c.inv = 1.0f / c.amax;
    c.scale = c.finite ? amax / 127.0f : __uint_as_float(0x7fc00000u);
    return c;
}

template <bool kExactProduct>
__device__ __forceinline__ int code_of(float x, const RowCode& c)
{
    const float v = ldexpf(x, c.shift);
    const float y = 127.0f * v;
    const float q0 = y * c.inv;
    const float q1 = fmaf(fmaf(-q0, c.amax, y), c.inv, q0);
    float r = rintf(q1);
    if constexpr (!kExactProduct) {
        // |q1 - r| near a half: the float32 product may have moved the quotient over it
        if (fabsf(fabsf(q1 - r) - 0.5f) < 0x1p-12f)
            r = static_cast<float>(rint(127.0 * static_cast<double>(v) / static_cast<double>(c.amax)));
    }
    return static_cast<int>(r);
}

// The largest value over the kT threads of a row, on each of them: lanes of one wave, or the workgroup.
template <int kT>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* buf)
{
#pragma unroll
    for (int off = (kT < 64 ? kT : 64) / 2; off >= 1; off >>= 1)
        v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), off)));
    if constexpr (kT > 64) {
        if ((threadIdx.x & 63) == 0)
            buf[threadIdx.x >> 6] = v;
        __syncthreads();
        v = buf[0];
#pragma unroll
        for (int w = 1; w < kT / 64; ++w)
            v = max(v, buf[w]);
    }
    return v;
}

// The expert of the group that holds `row`, or -1 where no group does or its expert is outside [0, E); a group
// begins no earlier than any offset before it, as in the tile table (scan_groups).  That leaves the first
// group g whose end lies past the row, and only if the row is not before the first offset: every later group
// has that end before it, and offsets 1 .. g are ends that do not lie past the row.  All threads call it.
__device__ __forceinline__ int row_expert(const int32_t* __restrict__ offsets,
                                          const int32_t* __restrict__ group_expert, int G, int E, int64_t M,
                                          int64_t row, int* found)
{
    if (threadIdx.x == 0)
        *found = INT32_MAX;
    __syncthreads();
    for (int g = threadIdx.x; g < G; g += blockDim.x) {
        const int64_t rb = min(max(static_cast<int64_t>(offsets[g]), int64_t{0}), M);
        const int64_t re = min(static_cast<int64_t>(offsets[g + 1]), M);
        if (row >= rb && row < re)
            atomicMin(found, g);
    }
    __syncthreads();
    const int g = *found;
    if (g == INT32_MAX || row < offsets[0])
        return -1;
    const int e = group_expert != nullptr ? group_expert[g] : g;
    return e >= 0 && e < E ? e : -1;
}

// A row by kT threads (`me` among them; a part of a wave, or the workgroup).  The row's values come from
// Src::load (the thread's vector i < kPer, or kPer: the one at a column), eight neighbouring ones at a time (fewer
// at the row's end); the first kPer vectors of a thread
// stay in registers between the maximum and the codes, as loaded (bfloat16 rows need half the registers
// that way: 56 for 96, eight waves a SIMD for five), later ones are made again.  kWhole: cols is a multiple
// of eight.
template <class Src, int kPer, bool kExactProduct, int kT, bool kWhole = true>
__device__ __forceinline__ void quantize_row(const Src& src, int64_t cols, int8_t* __restrict__ codes,
                                             float* __restrict__ scale, uint32_t* buf, int me)
{
    typename Src::Raw keep[kPer];
    uint32_t amax = 0;
    const auto count = [&](int64_t c) { return kWhole ? kVec : static_cast<int>(min(cols - c, static_cast<int64_t>(kVec))); };
    const auto take = [&](const typename Src::Raw& raw) {
        float x[kVec];
        src.values(raw, x);
#pragma unroll
        for (int v = 0; v < kVec; ++v)
            amax = max(amax, __float_as_uint(x[v]) & 0x7fffffffu);
    };
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int64_t c = (static_cast<int64_t>(i) * kT + me) * kVec;
        if (c < cols) {
            keep[i] = src.load(i, c, count(c));
            take(keep[i]);
        }
    }
    for (int64_t c = (static_cast<int64_t>(kPer) * kT + me) * kVec; c < cols; c += kT * kVec) {
        take(src.load(kPer, c, count(c)));
    }
    const RowCode rc = row_code(row_max<kT>(amax, buf));
    const auto store = [&](int64_t c, const typename Src::Raw& raw) {
        float x[kVec];
        src.values(raw, x);
        u32x2_t w = {0, 0};
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            const int code = rc.finite ? code_of<kExactProduct>(x[v], rc) : 0;
            w[v / 4] |= (static_cast<uint32_t>(code) & 0xffu) << (8 * (v % 4));
        }
        if (kWhole || c + kVec <= cols) {
            __builtin_memcpy(codes + c, &w, kVec);
        } else {
            for (int v = 0; v < cols - c; ++v)
                codes[c + v] = static_cast<int8_t>(w[v / 4] >> (8 * (v % 4)));
        }
    };
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int64_t c = (static_cast<int64_t>(i) * kT + me) * kVec;
        if (c < cols)
            store(c, keep[i]);
    }
    for (int64_t c = (static_cast<int64_t>(kPer) * kT + me) * kVec; c < cols; c += kT * kVec) {
        store(c, src.load(kPer, c, count(c)));
    }
    if (me == 0)
        *scale = rc.scale;
}

// Rows in memory, of any alignment: the copies become unaligned vector loads.
struct Bf16Row {
    using Raw = u32x4_t;
    const uint16_t* x;
    __device__ __forceinline__ Raw load(int, int64_t c, int n) const
    {
        Raw w = {0, 0, 0, 0};
        if (n == kVec)
            __builtin_memcpy(&w, x + c, 16);
        else
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                w[i / 2] |= i < n ? static_cast<uint32_t>(x[c + i]) << (16 * (i % 2)) : 0u;
        return w;
    }
    __device__ __forceinline__ void values(const Raw& w, float (&v)[kVec]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

struct Floats {
    f32x4_t half[2];
};
__device__ __forceinline__ void floats_of(const Floats& w, float (&v)[kVec])
{
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        v[i] = w.half[i / 4][i % 4];
}

struct F32Row {
    using Raw = Floats;
    const float* x;
    __device__ __forceinline__ Raw load(int, int64_t c, int n) const
    {
        Raw w = {};
        if (n == kVec) {
            __builtin_memcpy(&w, x + c, 32);
        } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                w.half[i / 4][i % 4] = i < n ? x[c + i] : 0.0f;
        }
        return w;
    }
    __device__ __forceinline__ void values(const Raw& w, float (&v)[kVec]) const { floats_of(w, v); }
};

// kT threads per row (kThreads / kT rows per workgroup).
template <class T, class Row, int kT, int kPer, bool kExactProduct, bool kWhole>
__global__ __launch_bounds__(kThreads) void int8_quantize_kernel(const T* __restrict__ x, int64_t rows,
                                                                 int64_t cols, int8_t* __restrict__ codes,
                                                                 float* __restrict__ scales)
{
    constexpr int kRows = kThreads / kT;
    __shared__ uint32_t buf[2][kThreads / 64];
    int slot = 0;                                        // two slots: a row's maxima are read while the next row's are written
    const int me = threadIdx.x % kT;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kT; r < rows;
         r += static_cast<int64_t>(gridDim.x) * kRows, slot ^= 1)
        quantize_row<Row, kPer, kExactProduct, kT, kWhole>(Row{x + r * cols}, cols, codes + r * cols, scales + r, buf[slot], me);
}

// The SwiGLU of a row's gate and up sums, quantised; one workgroup per row, whose sums stay in registers
// (kPer vectors a thread; longer rows are summed again for the codes).  The sums are asked for before the
// row's expert is looked up: row_expert where the caller has it, else the group that holds the row.
template <int kT, int kPer>
__global__ __launch_bounds__(kT) void int8_swiglu_partial_kernel(
    const int32_t* __restrict__ partial, int splits, const float* __restrict__ a_scale,
    const int32_t* __restrict__ gather, int gather_k, const float* __restrict__ sg, const float* __restrict__ su,
    const int32_t* __restrict__ row_experts, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ group_expert, int G, int E, int64_t M, int64_t F, int8_t* __restrict__ codes,
    float* __restrict__ scales)
{
    __shared__ uint32_t buf[kT / 64];
    __shared__ int found;
    const int64_t r = grid_row();
    if (r >= M)
        return;
    const int32_t* p = partial + r * 2 * F;
    const int64_t cut = M * 2 * F;
    const auto sums = [&](int64_t c, i32x4_t (&g)[2], i32x4_t (&u)[2]) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            g[q] = *reinterpret_cast<const i32x4_t*>(p + c + 4 * q);
            u[q] = *reinterpret_cast<const i32x4_t*>(p + F + c + 4 * q);
        }
        for (int s = 1; s < splits; ++s)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                g[q] += *reinterpret_cast<const i32x4_t*>(p + s * cut + c + 4 * q);
                u[q] += *reinterpret_cast<const i32x4_t*>(p + s * cut + F + c + 4 * q);
            }
    };
    const int64_t source = gather != nullptr ? gather[r] : r;
    i32x4_t g[kPer][2], u[kPer][2];
    for (int s = 0; s < splits; ++s)                          // the loads of a cut go out together
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int64_t c = (static_cast<int64_t>(i) * kT + threadIdx.x) * kVec;
            if (c < F)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const i32x4_t mine = *reinterpret_cast<const i32x4_t*>(p + s * cut + c + 4 * q);
                    const i32x4_t other = *reinterpret_cast<const i32x4_t*>(p + s * cut + F + c + 4 * q);
                    g[i][q] = s == 0 ? mine : g[i][q] + mine;
                    u[i][q] = s == 0 ? other : u[i][q] + other;
                }
        }
    const int e = row_experts != nullptr ? row_experts[r] : row_expert(offsets, group_expert, G, E, M, r, &found);
    if (e < 0)
        return;
    struct Values {
        using Raw = Floats;
        const decltype(sums)* again;
        const i32x4_t (*g)[2];
        const i32x4_t (*u)[2];
        float a_scale;
        const float* sg;
        const float* su;
        __device__ __forceinline__ void values(const Raw& w, float (&v)[kVec]) const { floats_of(w, v); }
        __device__ __forceinline__ Raw load(int i, int64_t c, int) const   // F is whole vectors
        {
            Raw w;
            i32x4_t gg[2], uu[2];
            if (i < kPer) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    gg[q] = g[i][q];
                    uu[q] = u[i][q];
                }
            } else {
                (*again)(c, gg, uu);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const f32x4_t wg = *reinterpret_cast<const f32x4_t*>(sg + c + 4 * q);
                const f32x4_t wu = *reinterpret_cast<const f32x4_t*>(su + c + 4 * q);
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    w.half[q][n] = swiglu(static_cast<float>(gg[q][n]) * a_scale * wg[n],
                                          static_cast<float>(uu[q][n]) * a_scale * wu[n]);
            }
            return w;
        }
    };
    const Values src{&sums, g, u, a_scale[gather != nullptr ? source / gather_k : r], sg + static_cast<int64_t>(e) * F,
                     su + static_cast<int64_t>(e) * F};
    quantize_row<Values, kPer, false, kT>(src, F, codes + r * F, scales + r, buf, threadIdx.x);
}

// Four columns' partial sums of all cuts (from part[i], cut apart) added up, for kRows rows.  A cut past the last
// is read as the last one and not added, so that the loads go out together, not one after the other.
template <int kRows, int kTogether>
__device__ __forceinline__ void add_cuts(const int32_t* const (&part)[kRows], int splits, int64_t cut, i32x4_t (&a)[kRows])
{
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        a[i] = *reinterpret_cast<const i32x4_t*>(part[i]);
    for (int s = 1; s < splits; s += kTogether) {
        i32x4_t v[kRows][kTogether];
#pragma unroll
        for (int q = 0; q < kTogether; ++q)
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                v[i][q] = *reinterpret_cast<const i32x4_t*>(part[i] + min(s + q, splits - 1) * cut);
#pragma unroll
        for (int q = 0; q < kTogether; ++q)
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                a[i] += s + q < splits ? v[i][q] : i32x4_t{0, 0, 0, 0};
    }
}

__device__ __forceinline__ f32x4_t scaled(const i32x4_t& a, float a_scale, const f32x4_t& w)
{
    f32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = static_cast<float>(a[i]) * a_scale * w[i];
    return v;
}

// A cut product's output: the cuts' int32 sums added (exact, so in any order), scaled, rounded once.  Rows
// across the grid, a row's columns over up to 16 workgroups (8 rows of 14336: 4.8 us, the chain group -> expert
// -> scales).
template <bool kBf16>
__global__ __launch_bounds__(kThreads) void int8_finish_kernel(
    const int32_t* __restrict__ partial, int splits, const float* __restrict__ a_scale,
    const float* __restrict__ w_scale, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ group_expert, int G, int E, int64_t M, int64_t N, void* __restrict__ out)
{
    __shared__ int found;
    const int64_t r = grid_row();
    if (r >= M)
        return;
    // the first columns' sums are asked for before the row's group is looked up
    const int64_t begin = 4 * (static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x);
    const int32_t* sums = partial + r * N;
    const auto total = [&](int64_t c) {
        const int32_t* const part[1] = {sums + c};
        i32x4_t a[1];
        if (splits <= 4)
            add_cuts<1, 3>(part, splits, M * N, a);
        else
            add_cuts<1, 7>(part, splits, M * N, a);
        return a[0];
    };
    i32x4_t sum = {0, 0, 0, 0};
    if (begin < N)
        sum = total(begin);
    const float as = a_scale[r];
    const int e = row_expert(offsets, group_expert, G, E, M, r, &found);
    if (e < 0)
        return;
    const float* ws = w_scale + static_cast<int64_t>(e) * N;
    for (int64_t c = begin; c < N; c += 4 * static_cast<int64_t>(gridDim.y) * kThreads) {
        if (c != begin)
            sum = total(c);
        const f32x4_t v = scaled(sum, as, *reinterpret_cast<const f32x4_t*>(ws + c));
        if constexpr (kBf16)
            *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(out) + r * N + c) =
                u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        else
            *reinterpret_cast<f32x4_t*>(static_cast<float*>(out) + r * N + c) = v;
    }
}

// What the combine uses of a token's slots j .. j + kTogether - 1: no branch on a dropped slot or one past the last, so
// that the loads of several slots go out together.
template <int kTogether>
struct Slots {
    int64_t row[kTogether];                                   // of the sums (0 where not held)
    const float* w[kTogether];                                // the expert's column scales
    float scale[kTogether], p[kTogether];
    bool held[kTogether];
    __device__ __forceinline__ Slots(const int32_t* __restrict__ expert_ids, const int32_t* __restrict__ pos,
                                     const float* __restrict__ probs, const float* __restrict__ a_scale,
                                     const float* __restrict__ w_scale, int64_t t, int j, int k, int64_t M, int64_t N)
    {
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
            const int64_t slot = t * k + min(j + i, k - 1);
            const int64_t at = pos[slot];
            const int id = expert_ids[slot];
            held[i] = j + i < k && at >= 0 && at < M;
            row[i] = held[i] ? at : 0;
            w[i] = w_scale + static_cast<int64_t>(held[i] ? id : 0) * N;
            scale[i] = a_scale[row[i]];
            p[i] = probs[slot];
        }
    }
};

// The combine of the layer from the down projection's partial sums.  Each slot's sum is rounded to float16 as
// the stored rows of the other path are (int8_combine_rows_kernel), scaled in float32, and the k of a token are
// added in slot order by fused multiply-adds from 0: bitwise the same output.  A chain of three loads
// bounds it at few tokens (one token of 4096, 8 cuts: 6.3 us slot by slot and four cuts at a time, 4.6 us so).
template <int kTogether>
__global__ __launch_bounds__(kThreads) void int8_combine_kernel(
    const int32_t* __restrict__ partial, int splits, float unit, const float* __restrict__ a_scale,
    const float* __restrict__ w_scale, const int32_t* __restrict__ expert_ids, const int32_t* __restrict__ pos,
    const float* __restrict__ probs, int64_t T, int k, int64_t M, int64_t N, uint16_t* __restrict__ out)
{
    const int64_t t = grid_row();
    const int64_t c = 4 * (static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x);
    if (t >= T || c >= N)
        return;
    const float back = 1.0f / unit;
    f32x4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = 0; j < k; j += kTogether) {
        const Slots<kTogether> s(expert_ids, pos, probs, a_scale, w_scale, t, j, k, M, N);
        const int32_t* part[kTogether];
        i32x4_t a[kTogether];
        f32x4_t w[kTogether];
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
            part[i] = partial + s.row[i] * N + c;
            w[i] = *reinterpret_cast<const f32x4_t*>(s.w[i] + c);
        }
        add_cuts<kTogether, 14 / kTogether>(part, splits, M * N, a);
#pragma unroll
        for (int i = 0; i < kTogether; ++i)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float v = half_to_f32(static_cast<uint16_t>(pack_half2(static_cast<float>(a[i][n]) * unit, 0.0f)));
                sum[n] = s.held[i] ? fmaf(s.p[i], v * back * s.scale[i] * w[i][n], sum[n]) : sum[n];
            }
    }
    *reinterpret_cast<u32x2_t*>(out + t * N + c) = u32x2_t{pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3])};
}

// The same from stored float16 rows, a thread per eight columns of a token (16384 tokens of 7168, 4 slots each: 231 us
// where the sum of scaled bfloat16 rows took 187; the product that writes the rows unscaled takes 80 us less).
template <int kTogether>
__global__ __launch_bounds__(kThreads) void int8_combine_rows_kernel(
    const uint16_t* __restrict__ rows, float unit, const float* __restrict__ a_scale, const float* __restrict__ w_scale,
    const int32_t* __restrict__ expert_ids, const int32_t* __restrict__ pos, const float* __restrict__ probs, int64_t T,
    int k, int64_t M, int64_t N, uint16_t* __restrict__ out)
{
    const int64_t t = grid_row();
    const int64_t c = 8 * (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x);
    if (t >= T || c >= N)
        return;
    const float back = 1.0f / unit;
    float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = 0; j < k; j += kTogether) {
        const Slots<kTogether> s(expert_ids, pos, probs, a_scale, w_scale, t, j, k, M, N);
        u32x4_t v[kTogether];
        f32x4_t w[kTogether][2];
#pragma unroll
        for (int i = 0; i < kTogether; ++i)
            v[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(rows + s.row[i] * N + c));
#pragma unroll
        for (int i = 0; i < kTogether; ++i)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                w[i][q] = *reinterpret_cast<const f32x4_t*>(s.w[i] + c + 4 * q);
#pragma unroll
        for (int i = 0; i < kTogether; ++i)
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                const float h = half_to_f32(static_cast<uint16_t>(v[i][n / 2] >> (16 * (n % 2))));
                sum[n] = s.held[i] ? fmaf(s.p[i], h * back * s.scale[i] * w[i][n / 4][n % 4], sum[n]) : sum[n];
            }
    }
    *reinterpret_cast<u32x4_t*>(out + t * N + c) =
        u32x4_t{pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3]), pack_bf16x2(sum[4], sum[5]), pack_bf16x2(sum[6], sum[7])};
}

// The table of balanced tiles alone: a thread per group (kWideThreads of them at a time), a scan, then a
// thread per tile, which finds its group by bisection.  One workgroup, few barriers (8 groups 4.8 us, 128
// groups 5.6 us, where the general builder with its two tables takes 5.5 and 9.4).
__global__ __launch_bounds__(kWideThreads) void int8_tiles_kernel(
    const int32_t* __restrict__ offsets, const int32_t* __restrict__ group_expert, int G, int E, int64_t M, int bm,
    MTile* __restrict__ tiles, int32_t* __restrict__ tile_count, int32_t* __restrict__ task_ctr,
    int32_t* __restrict__ status, int write_status)
{
    __shared__ int first[kWideThreads + 1], begin[kWideThreads], rows[kWideThreads], expert[kWideThreads];
    __shared__ int wave_max[kWideThreads / 64], wave_sum[kWideThreads / 64];
    const int me = threadIdx.x;
    int done = 0, reached = 0;                                // tiles and largest offset of the groups so far
    bool bad = false;
    if (me < 2 * kXcdCount)
        task_ctr[me] = 0;
    for (int base = 0; base < G; base += kWideThreads) {
        const int held = min(G - base, kWideThreads);
        const GroupRows r = scan_groups<kWideThreads / 64>(offsets, group_expert, base, G, E, M, bm, reached, wave_max, wave_sum);
        bad |= r.bad;
        first[me] = r.first;
        if (me == 0)
            first[kWideThreads] = r.total;
        begin[me] = r.begin;
        rows[me] = r.rows;
        expert[me] = r.expert;
        __syncthreads();
        const int total = r.total;
        for (int t = me; t < total; t += kWideThreads) {
            int lo = 0, hi = held - 1;                        // the last group whose first tile is at most t
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (first[mid] <= t)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            tiles[done + t] = balanced_tile(expert[lo], begin[lo], rows[lo], first[lo + 1] - first[lo], t - first[lo], done + first[lo]);
        }
        done += total;
        __syncthreads();                                      // read before the next groups are written
    }
    const int any_bad = __syncthreads_or(bad ? 1 : 0);
    if (me == 0) {
        *tile_count = done;
        if (write_status)
            *status = any_bad ? MOE_ERR_EXPERT_ID_OUT_OF_RANGE : MOE_OK;
        else if (any_bad)
            *status = MOE_ERR_EXPERT_ID_OUT_OF_RANGE;
    }
}

// What a small layer call needs before its first product, in one launch: workgroup 0 routes (counts,
// offsets, perm and pos of at most kInt8SmallSlots slots: a slot's rank among equal ids is counted
// directly) and writes the table of balanced row tiles, the others quantise a token row each.  One token of
// 4096 on 8 experts: 4.6 us, in place of five launches of 3 to 6 us each.
__global__ __launch_bounds__(kThreads) void int8_prologue_kernel(
    const int32_t* __restrict__ ids, int T, int k, int E, int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
    int32_t* __restrict__ perm, int32_t* __restrict__ pos, int32_t* __restrict__ row_experts,
    int32_t* __restrict__ status, int bm,
    MTile* __restrict__ tiles, int32_t* __restrict__ tile_count, const uint16_t* __restrict__ x, int64_t H,
    int8_t* __restrict__ codes, float* __restrict__ scales)
{
    __shared__ uint32_t buf[kThreads / 64];
    if (blockIdx.x > 0) {
        const int64_t r = blockIdx.x - 1;
        quantize_row<Bf16Row, 4, true, kThreads>(Bf16Row{x + r * H}, H, codes + r * H, scales + r, buf, threadIdx.x);
        return;
    }
    static_assert(kInt8SmallSlots <= kThreads && kMaxExperts <= 4 * kThreads, "one slot and four experts a thread");
    __shared__ int id[kThreads];
    __shared__ int begin[kMaxExperts + 1], tile_begin[kMaxExperts + 1];
    __shared__ int hist[kMaxExperts];
    __shared__ int wave_sum[2][kThreads / 64];
    const int M = T * k, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int mine = tid < M ? ids[tid] : -1;
    const bool valid = mine >= 0 && mine < E;
    id[tid] = valid ? mine : -1;
    for (int e = tid; e < E; e += kThreads)
        hist[e] = 0;
    __syncthreads();
    if (valid)
        atomicAdd(&hist[mine], 1);
    int rank = 0;
    for (int s = 0; s < M; ++s)
        rank += s < tid && id[s] == mine ? 1 : 0;
    __syncthreads();
    // rows and row tiles before each expert: thread i scans experts 4 i .. 4 i + 3
    int rows = 0, nt = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int n = 4 * tid + q < E ? hist[4 * tid + q] : 0;
        rows += n;
        nt += (n + bm - 1) / bm;
    }
    int rows_in = rows, nt_in = nt;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int a = __shfl_up(rows_in, off), b = __shfl_up(nt_in, off);
        rows_in += lane >= off ? a : 0;
        nt_in += lane >= off ? b : 0;
    }
    if (lane == 63) {
        wave_sum[0][wave] = rows_in;
        wave_sum[1][wave] = nt_in;
    }
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        rows_in += wave_sum[0][w];
        nt_in += wave_sum[1][w];
    }
    rows_in -= rows;
    nt_in -= nt;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int e = 4 * tid + q;
        if (e < E) {
            begin[e] = rows_in;
            tile_begin[e] = nt_in;
            counts[e] = hist[e];
            offsets[e] = rows_in;
            rows_in += hist[e];
            nt_in += (hist[e] + bm - 1) / bm;
            if (e == E - 1) {
                begin[E] = rows_in;
                offsets[E] = rows_in;
                if (tiles != nullptr)
                    *tile_count = nt_in;
                *status = rows_in == M ? MOE_OK : MOE_ERR_EXPERT_ID_OUT_OF_RANGE;
            }
        }
    }
    __syncthreads();
    if (tid < M) {
        const int row = valid ? begin[mine] + rank : -1;
        pos[tid] = row;
        if (valid) {
            perm[row] = tid;
            row_experts[row] = mine;
        }
        if (tid >= begin[E]) {
            perm[tid] = -1;
            row_experts[tid] = -1;
        }
    }
    for (int e = tid; e < E; e += kThreads) {
        const int n = hist[e], R = (n + bm - 1) / bm;
        for (int i = 0; i < R && tiles != nullptr; ++i)
            tiles[tile_begin[e] + i] = balanced_tile(e, begin[e], n, R, i, tile_begin[e]);
    }
}

// Threads per row: 16 up to 256 columns, a wave up to 2048 (no barrier, and more lanes have values), then
// the workgroup.  Measured where a workgroup took each row and where a wave does (16384 bfloat16 rows, us):
// 128 columns 13.8 -> 8.6 (16 threads), 1024 17.1 -> 11.6, 1031 33.4 -> 17.9, 1951 (13918 rows) 34.7 ->
// 23.6, 2048 21.5 -> 20.5; float32 2048 32.3 -> 32.9; float32 8192: 260 by a wave, 127 by the workgroup.
template <class T, class Row, bool kExactProduct, bool kWhole>
hipError_t launch_quantize(const T* x, int64_t rows, int64_t cols, int8_t* codes, float* scales, hipStream_t s)
{
    const auto grid = [&](int per_block) { return dim3(static_cast<unsigned>(std::min(ceil_div(rows, per_block), kGridRows))); };
    if (cols <= 256)
        int8_quantize_kernel<T, Row, 16, 2, kExactProduct, kWhole><<<grid(16), dim3(kThreads), 0, s>>>(x, rows, cols, codes, scales);
    else if (cols <= 2048)
        int8_quantize_kernel<T, Row, 64, 4, kExactProduct, kWhole><<<grid(4), dim3(kThreads), 0, s>>>(x, rows, cols, codes, scales);
    else
        int8_quantize_kernel<T, Row, kThreads, 4, kExactProduct, kWhole><<<grid(1), dim3(kThreads), 0, s>>>(x, rows, cols, codes, scales);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_quantize(int dtype, const void* x, int64_t rows, int64_t cols, int8_t* codes,
                                float* scales, hipStream_t s)
{
    if (rows <= 0)
        return hipSuccess;
    if (dtype == MOE_F32) {
        const auto* v = static_cast<const float*>(x);
        return cols % kVec == 0 ? launch_quantize<float, F32Row, false, true>(v, rows, cols, codes, scales, s)
                                : launch_quantize<float, F32Row, false, false>(v, rows, cols, codes, scales, s);
    }
    const auto* v = static_cast<const uint16_t*>(x);
    return cols % kVec == 0 ? launch_quantize<uint16_t, Bf16Row, true, true>(v, rows, cols, codes, scales, s)
                            : launch_quantize<uint16_t, Bf16Row, true, false>(v, rows, cols, codes, scales, s);
}

hipError_t launch_int8_swiglu_partial(const int32_t* partial, int splits, const float* a_scale,
                                      const int32_t* gather, int gather_k, const float* sg, const float* su,
                                      const int32_t* row_experts, const int32_t* offsets,
                                      const int32_t* group_expert, int64_t G, int64_t E, int64_t M, int64_t F, int8_t* codes, float* scales,
                                      hipStream_t s)
{
    if (M <= 0)
        return hipSuccess;
    const dim3 grid = row_grid(M);
    const int g = static_cast<int>(G), e = static_cast<int>(E);
    // few rows: a whole CU's threads for each (2 rows of 14336: 16.8 -> 7.5 us)
    if (M <= 2 * device_info().cu_count)
        int8_swiglu_partial_kernel<kWideThreads, 2><<<grid, dim3(kWideThreads), 0, s>>>(
            partial, splits, a_scale, gather, gather_k, sg, su, row_experts, offsets, group_expert, g, e, M, F, codes, scales);
    else
        int8_swiglu_partial_kernel<kThreads, 4><<<grid, dim3(kThreads), 0, s>>>(
            partial, splits, a_scale, gather, gather_k, sg, su, row_experts, offsets, group_expert, g, e, M, F, codes, scales);
    return hipGetLastError();
}

hipError_t launch_int8_tiles(const int32_t* offsets, const int32_t* group_expert, int64_t G, int64_t E, int64_t M,
                             int bm, MTile* tiles, int32_t* tile_count, int32_t* task_ctr, int32_t* status,
                             bool write_status, hipStream_t s)
{
    int8_tiles_kernel<<<dim3(1), dim3(kWideThreads), 0, s>>>(offsets, group_expert, static_cast<int>(G),
                                                             static_cast<int>(E), M, bm, tiles, tile_count, task_ctr,
                                                             status, write_status ? 1 : 0);
    return hipGetLastError();
}

hipError_t launch_int8_prologue(const int32_t* ids, int64_t T, int64_t k, int64_t E, int32_t* counts, int32_t* offsets,
                                int32_t* perm, int32_t* pos, int32_t* row_experts, int32_t* status, int bm,
                                MTile* tiles, int32_t* tile_count, const uint16_t* x, int64_t H, int8_t* codes, float* scales,
                                hipStream_t s)
{
    if (T <= 0 || T * k > kInt8SmallSlots || E >= kMaxExperts)
        return hipErrorInvalidValue;
    int8_prologue_kernel<<<dim3(static_cast<unsigned>(x != nullptr ? T + 1 : 1)), dim3(kThreads), 0, s>>>(
        ids, static_cast<int>(T), static_cast<int>(k), static_cast<int>(E), counts, offsets, perm, pos, row_experts, status, bm, tiles,
        tile_count, x, H, codes, scales);
    return hipGetLastError();
}

hipError_t launch_int8_combine(const void* sums, int splits, int64_t K, const float* a_scale, const float* w_scale,
                               const int32_t* expert_ids, const int32_t* pos, const float* probs, int64_t T, int64_t k,
                               int64_t N, uint16_t* out, hipStream_t s)
{
    if (T <= 0)
        return hipSuccess;
    const float unit = int8_half_unit(K);
    const int n = static_cast<int>(k);
    // kTogether: slots whose loads go out together
    if (splits == 0) {
        const unsigned threads = static_cast<unsigned>(std::min<int64_t>(kThreads, ceil_div(N / 8, 64) * 64));
        const dim3 grid = row_grid(T, ceil_div(N / 8, threads));
        const auto* rows = static_cast<const uint16_t*>(sums);
        if (k <= 2)
            int8_combine_rows_kernel<2><<<grid, dim3(threads), 0, s>>>(rows, unit, a_scale, w_scale, expert_ids, pos, probs, T,
                                                                       n, T * k, N, out);
        else
            int8_combine_rows_kernel<4><<<grid, dim3(threads), 0, s>>>(rows, unit, a_scale, w_scale, expert_ids, pos, probs, T,
                                                                       n, T * k, N, out);
        return hipGetLastError();
    }
    const dim3 grid = row_grid(T, ceil_div(N, 4 * kThreads));
    const auto* partial = static_cast<const int32_t*>(sums);
    if (k <= 2)
        int8_combine_kernel<2><<<grid, dim3(kThreads), 0, s>>>(partial, splits, unit, a_scale, w_scale, expert_ids, pos, probs,
                                                               T, n, T * k, N, out);
    else
        int8_combine_kernel<4><<<grid, dim3(kThreads), 0, s>>>(partial, splits, unit, a_scale, w_scale, expert_ids, pos, probs,
                                                               T, n, T * k, N, out);
    return hipGetLastError();
}

hipError_t launch_int8_finish(const int32_t* partial, int splits, const float* a_scale, const float* w_scale,
                              const int32_t* offsets, const int32_t* group_expert, int64_t G, int64_t E,
                              int64_t M, int64_t N, void* out, int out_dtype, hipStream_t s)
{
    if (M <= 0)
        return hipSuccess;
    const dim3 grid = row_grid(M, std::min<int64_t>(ceil_div(N, 4 * kThreads), 16));
    if (out_dtype == MOE_F32)
        int8_finish_kernel<false><<<grid, dim3(kThreads), 0, s>>>(partial, splits, a_scale, w_scale, offsets, group_expert,
                                                                  static_cast<int>(G), static_cast<int>(E), M, N, out);
    else
        int8_finish_kernel<true><<<grid, dim3(kThreads), 0, s>>>(partial, splits, a_scale, w_scale, offsets, group_expert,
                                                                 static_cast<int>(G), static_cast<int>(E), M, N, out);
    return hipGetLastError();
}

}  // namespace moe
