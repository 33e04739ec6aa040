// The gated product of few rows (up to 64) on gfx950: g = x Wg and u = x Wu with the epilogues of the gated block; and the
// results from sums that the products of many rows took over parts of K.
//
// What bounds it is the weights' way from memory, so they take the shortest: a lane loads 4 adjacent columns of 8
// consecutive k rows (of one matrix) straight into registers.  bfloat16: v_perm_b32 turns the 8 x 4 block into four MFMA
// operands of 8 k each (v_mfma_f32_16x16x32_bf16, the weights as the first operand); lane l of operand j holds column
// 4 (l % 16) + j, which leaves every lane of the result with 16 adjacent columns of one row (with 32 columns: 2 adjacent
// columns a lane, two operands, 8 columns).  float32: the words are
// v_mfma_f32_16x16x4_f32 operands as they are, eight of one k per lane group, exact products.  Nothing of the weights goes
// through LDS, and rows of any width and alignment are read the same way.
// A workgroup takes 64 or 32 columns of both matrices; its waves take K in turn, 32 rows at a time with more of them in
// flight, and join their sums through LDS in a fixed order.  One CU moves 70 GB/s with 128-byte rows, 35 with 64-byte ones:
// where the columns give few workgroups, K is cut over workgroups too, which costs a second launch (plan).
// 1 x 4096 x 14336: 50 us, 4.7 TB/s (through LDS tiles 73); 33 x 2048 x 768, 24 x 8 workgroups of 32 columns, 7.4 and 4.2-5.2
// to join the eight parts.
#include <algorithm>

#include "gated_epilogue.h"

namespace moe {
namespace {

constexpr int kBatch = 32;                // k rows per wave and step

// kN (4 or 2) adjacent values as loaded.
template <class T, int kN>
struct RawN {
    static constexpr int kWords = kN * sizeof(T) / 4;
    uint32_t w[kWords];
};

// kN values at p.
template <class T, int kN>
__device__ __forceinline__ RawN<T, kN> load_n(const T* p)
{
    RawN<T, kN> r;
    if constexpr (RawN<T, kN>::kWords == 4) {
        const u32x4_t v = *reinterpret_cast<const u32x4_any_t*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.w[i] = v[i];
    } else if constexpr (RawN<T, kN>::kWords == 2) {
        typedef u32x2_t __attribute__((aligned(2))) u32x2_any_t;
        const u32x2_t v = *reinterpret_cast<const u32x2_any_t*>(p);
        r.w[0] = v[0];
        r.w[1] = v[1];
    } else {
        typedef uint32_t __attribute__((aligned(2))) u32_any_t;
        r.w[0] = *reinterpret_cast<const u32_any_t*>(p);
    }
    return r;
}

// The last kN - skip of the values first, zeros after them.
template <class T, int kN>
__device__ __forceinline__ void shift_down(RawN<T, kN>& r, int skip)
{
    if constexpr (RawN<T, kN>::kWords == 1) {
        r.w[0] = skip >= 2 ? 0u : r.w[0] >> (16 * skip);
    } else if constexpr (RawN<T, kN>::kWords == 2) {
        const uint64_t v = (static_cast<uint64_t>(r.w[1]) << 32 | r.w[0]) >> min(8 * static_cast<int>(sizeof(T)) * skip, 63);
        r.w[0] = skip >= kN ? 0u : static_cast<uint32_t>(v);
        r.w[1] = skip >= kN ? 0u : static_cast<uint32_t>(v >> 32);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t v = 0;
#pragma unroll
            for (int s = 0; s + i < 4; ++s)
                v = skip == s ? r.w[i + s] : v;
            r.w[i] = v;
        }
    }
}

// One step of a wave: 32 k of 16 kN columns of both matrices, and of kRB blocks of 16 rows of x.
template <class T, int kN, int kRB>
struct Step {
    RawN<T, kN> w[2][8];
    Raw8<T> x[kRB];
};

template <class T, int kN, int kRB>
__device__ __forceinline__ void multiply(f32x4_t (&acc)[2][kN][kRB], const Step<T, kN, kRB>& s)
{
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < kN; ++j) {
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
                for (int j = 0; j < kN; ++j)
#pragma unroll
                    for (int b = 0; b < kRB; ++b)
                        acc[m][j][b] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                            __uint_as_float(s.w[m][i].w[j]), i < 4 ? s.x[b].a[i & 3] : s.x[b].b[i & 3], acc[m][j][b], 0, 0, 0);
    }
}

template <class T, int kN, int kRB, int kWaves, int kDepth, int kEpi>
__global__ __launch_bounds__(64 * kWaves) void gated_rows_kernel(RowsArgs g)
{
    constexpr int kRuns = kN / 2;                          // runs of 8 columns of a lane's result
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    f32x4_t* const join = reinterpret_cast<f32x4_t*>(smem);            // [wave][matrix][j][row block][lane]
    const EpiArgs& e = g.e;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = blockIdx.x * 16 * kN, part = blockIdx.y;
    // A lane whose kN columns pass the row's end reads the row's last kN (skip > 0: the first of them belong to lanes
    // before it); in the last workgroup alone, whose lanes shift them into place.
    const int kg = 8 * (lane >> 4), col = n0 + kN * (lane & 15), from = min(col, e.N - kN), skip = col - from;
    const bool ragged = n0 + 16 * kN > e.N;
    const T* const w0 = static_cast<const T*>(g.wg) + from;
    const T* const w1 = static_cast<const T*>(g.wu) + from;
    const T* x[kRB];
#pragma unroll
    for (int b = 0; b < kRB; ++b)                          // rows past the last repeat it and are not written
        x[b] = static_cast<const T*>(g.x) + static_cast<int64_t>(min(16 * b + (lane & 15), e.M - 1)) * g.K;

    // whole: all 32 k exist, and nothing stands between the loads
    const auto load = [&](auto whole, Step<T, kN, kRB>& s, int batch) {
        constexpr bool kWhole = decltype(whole)::value;
        const int k = kBatch * batch + kg;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t at = static_cast<int64_t>(kWhole ? k + i : min(k + i, g.K - 1)) * e.N;
            s.w[0][i] = load_n<T, kN>(w0 + at);
            s.w[1][i] = load_n<T, kN>(w1 + at);
        }
#pragma unroll
        for (int b = 0; b < kRB; ++b)
            s.x[b] = load_raw<kWhole>(x[b] + k, kWhole ? 8 : g.K - k);
        if constexpr (!kWhole) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (k + i >= g.K)
                    s.w[0][i] = s.w[1][i] = RawN<T, kN>{};
        }
    };
    f32x4_t acc[2][kN][kRB];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < kN; ++j)
#pragma unroll
            for (int b = 0; b < kRB; ++b)
                acc[m][j][b] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const auto add = [&](Step<T, kN, kRB>& s) {
        if (ragged)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                shift_down<T, kN>(s.w[0][i], skip);
                shift_down<T, kN>(s.w[1][i], skip);
            }
        multiply<T, kN, kRB>(acc, s);
        __builtin_amdgcn_sched_barrier(0);                 // the next loads go out when these registers are free
    };
    // this wave's whole steps of the workgroup's part of K: first, first + kWaves, ..; kDepth of them in flight
    const int whole = g.K / kBatch;
    const int step0 = static_cast<int>(static_cast<int64_t>(whole) * part / e.parts);
    const int step1 = static_cast<int>(static_cast<int64_t>(whole) * (part + 1) / e.parts);
    const int first = step0 + wave, mine = step1 > first ? (step1 - first + kWaves - 1) / kWaves : 0;
    Step<T, kN, kRB> s[kDepth];
    if (mine > 0) {
#pragma unroll
        for (int u = 0; u < kDepth; ++u)
            load(std::true_type{}, s[u], first + kWaves * min(u, mine - 1));
        int i = 0;
        for (; i + kDepth <= mine; i += kDepth)
#pragma unroll
            for (int u = 0; u < kDepth; ++u) {
                add(s[u]);
                load(std::true_type{}, s[u], first + kWaves * min(i + u + kDepth, mine - 1));
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
        for (int u = 0; u < kDepth - 1; ++u)
            if (i + u < mine)
                add(s[u]);
    }
    if (kBatch * whole < g.K && part == e.parts - 1 && wave == (step1 - step0) % kWaves) {   // the last k, fewer than 32
        load(std::false_type{}, s[0], whole);
        add(s[0]);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < kN; ++j)
#pragma unroll
            for (int b = 0; b < kRB; ++b)
                join[(((wave * 2 + m) * kN + j) * kRB + b) * 64 + lane] = acc[m][j][b];
    __syncthreads();
    const DropKey key = drop_key(e.drop);
    // a lane's columns of a row: operand j, register r is column kN r + j
    for (int u = tid; u < 64 * kRuns * kRB; u += 64 * kWaves) {
        const int h = u % kRuns, l = u / kRuns % 64, b = u / (64 * kRuns);
        const int row = 16 * b + (l & 15), c = n0 + 4 * kN * (l >> 4) + 8 * h;
        if (row >= e.M || c >= e.N)
            continue;
        float v[2][8] = {};
        for (int w = 0; w < kWaves; ++w)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    const float* p = reinterpret_cast<const float*>(&join[(((w * 2 + m) * kN + j) * kRB + b) * 64 + l]);
#pragma unroll
                    for (int r = 0; r < 8 / kN; ++r)
                        v[m][kN * r + j] += p[8 / kN * h + r];
                }
        if (e.partial != nullptr) {
            store8<float, true>(partial_at(e, part, 0, row, c), v[0], 8);
            store8<float, true>(partial_at(e, part, 1, row, c), v[1], 8);
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

template <class T, int kN, int kRB, int kWaves, int kDepth, int kEpi>
hipError_t launch_rows(const RowsArgs& g, hipStream_t s)
{
    constexpr int kLds = kWaves * kRB * 2 * kN * 64 * 16;
    static LdsLimit limit;
    if (hipError_t e = limit.ensure(reinterpret_cast<const void*>(&gated_rows_kernel<T, kN, kRB, kWaves, kDepth, kEpi>), kLds);
        e != hipSuccess)
        return e;
    const dim3 grid(static_cast<unsigned>(ceil_div(g.e.N, 16 * kN)), g.e.parts);
    gated_rows_kernel<T, kN, kRB, kWaves, kDepth, kEpi><<<grid, 64 * kWaves, kLds, s>>>(g);
    return hipGetLastError();
}

struct Plan {
    int n, parts;                                          // columns per lane (4 or 2), parts of K
};

// The shortest time of the ways there are, in us, from measured rates: a workgroup moves 70 KB (n = 4) or 35 KB (n = 2) a
// us, 35 KB or 26 KB with more than 32 rows, and, float32, adds 0.45 TFLOP/s in blocks of 16 rows, the chip moves 5.1 MB a
// us; a launch takes 4, a second one with its passes over the parts' sums 6 and 3 MB a us.  (16 x 8192 x 128 in one part 30
// us, 63 x 5578 x 512 in float32 94; 33 x 2048 x 768 with n = 4 20 us, with n = 2 14 us.)
Plan plan(int64_t M, int64_t K, int64_t N, int64_t size)
{
    Plan best{};
    double time = 1e30;
    const double rows = M <= 16 ? 16.0 : M <= 32 ? 32.0 : 64.0;
    for (int n : {4, 2})
        for (int p = 1; p <= 16 && (p == 1 || K / p >= 256); ++p) {
            const double groups = static_cast<double>(ceil_div(N, 16 * n) * p), k = static_cast<double>(K) / p;
            const double rate = M <= 32 ? (n == 4 ? 70e3 : 35e3) : (n == 4 ? 35e3 : 26e3);
            double one = k * 32.0 * n * static_cast<double>(size) / rate;
            if (size == 4)
                one = std::max(one, rows * k * 64.0 * n / 0.45e6);
            const double rounds = std::max(1.0, groups / 256.0);
            double t = 4.0 + std::max(one * rounds, 2.0 * static_cast<double>(K * N * size) / 5.1e6);
            if (p > 1)
                t += 6.0 + 8.0 * p * static_cast<double>(M * N) / 3e6;
            if (t < time) {
                time = t;
                best = Plan{n, p};
            }
        }
    return best;
}

// Waves per workgroup and steps in flight: what registers (sums 8 kN kRB, a step 4 kN sizeof(T) + 4 kRB or 8 kRB) and
// LDS (2 kN kRB KiB a wave) leave.
template <class T, int kEpi>
hipError_t launch_blocks(const RowsArgs& g, hipStream_t s)
{
    constexpr bool kShort = sizeof(T) == 2;
    if (plan(g.e.M, g.K, g.e.N, sizeof(T)).n == 4)
        return g.e.M <= 16 ? launch_rows<T, 4, 1, 8, 2, kEpi>(g, s) : g.e.M <= 32 ? launch_rows<T, 4, 2, 8, 2, kEpi>(g, s)
                                                                             : launch_rows<T, 4, 4, 4, 2, kEpi>(g, s);
    return g.e.M <= 16   ? launch_rows<T, 2, 1, 8, kShort ? 6 : 3, kEpi>(g, s)
           : g.e.M <= 32 ? launch_rows<T, 2, 2, 8, kShort ? 4 : 2, kEpi>(g, s)
                         : launch_rows<T, 2, 4, kShort ? 8 : 4, 3, kEpi>(g, s);
}

}  // namespace

int gated_rows_parts(int dtype, int64_t M, int64_t K, int64_t N) { return plan(M, K, N, dtype == MOE_F32 ? 4 : 2).parts; }

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
