// Grouped GEMMs on 8-bit integers with one scale per row and one per (expert, output column):
//
//   out[r, n] = a_scale[r] * w_scale[e, n] * sum_k a[r, k] w[e, k, n]        r in a group of expert e
//
// The sum is an exact int32 (|a|, |w| <= 128 and K < 2^17), so the result does not depend on how K
// is cut; one conversion to float32 and two products follow, and the output is rounded once.
//
// Products run on v_mfma_i32_32x32x32_i8 with the weights as the first operand, so a lane holds
// one output row (lane % 32) and four runs of four adjacent columns (8 g + 4 (lane / 32) .. + 3) of
// each 32 x 32 block.  A operand: lane l covers row / column l % 32 and the 16 k of half l / 32 of a
// 32-wide K block.
//
// A workgroup of 8 waves computes BM rows x 256 weight columns (256 outputs, or 128 of the gate and
// 128 of the up matrix): global -> LDS copies into a ring of stages of BK values of K, one barrier
// a step.  A rows lie in LDS as in memory, 16-byte chunks XOR-swizzled by row; the weights lie as in
// memory ([K, N], N contiguous), and the transposing LDS read (ds_read_b64_tr_b8) hands each lane 8
// consecutive k of its column.
#include <algorithm>
#include <atomic>

#include "gemm_common.h"
#include "moe_expert_layer.h"

namespace moe {
namespace {
namespace i8 {

typedef int i32x16_t __attribute__((ext_vector_type(16)));
typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2_t lds_i32x2_t;

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
constexpr int BNB = 256;                       // weight columns per task (both matrices of a gated task)

enum Out { kOutBf16, kOutF32, kOutPartial };

struct Args {
    const uint8_t* A;                          // int8 rows
    const float* a_scale;
    const uint8_t* B0;                         // int8 [E, K, N]; B1: the up matrix of a gated task
    const uint8_t* B1;
    const float* s0;                           // [E, N]
    const float* s1;
    void* out;                                 // [M, N], or int32 partial sums [splits, M, N or 2N]
    const MTile* tiles;
    const int32_t* tile_count;
    const int32_t* gather;                     // may be null: row p of the product is row gather[p] / gather_k of A
    int gather_k;
    int K, N, splits;
    int64_t M;
};

// WM x WN waves of TM x TN blocks of 32 x 32, S stages of BK values of K.
template <int kWM_, int kWN_, int kTM_, int kTN_, int kBK_, int kStages_>
struct Config {
    static constexpr int kWM = kWM_, kWN = kWN_, kTM = kTM_, kTN = kTN_, BK = kBK_, kStages = kStages_;
    static constexpr int BM = kWM * kTM * 32;
    static constexpr int kABytes = BM * BK, kBBytes = BK * BNB;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kSmemBytes = kStages * kStageBytes;
    static constexpr int kACopies = kABytes / 1024 / kWaves;     // 1 KiB copies per wave and step
    static constexpr int kBCopies = kBBytes / 1024 / kWaves;
    static constexpr int kCopies = kACopies + kBCopies;
    static_assert(kWM * kWN == kWaves && kWN * kTN * 32 == BNB, "wave grid");
    static_assert(kABytes % (1024 * kWaves) == 0 && kBBytes % (1024 * kWaves) == 0, "copies per wave");
    static_assert(kSmemBytes <= 160 * 1024, "LDS");
    static_assert(BK == 64 || BK == 128, "A swizzle");
};

// LDS chunk position of 16-byte chunk c of A row r: fragment reads take one chunk of 16 consecutive
// rows at a time, which the XOR spreads over the 256-byte bank window.
template <int BK>
__device__ __forceinline__ int aswz(int c, int r)
{
    return BK == 128 ? c ^ ((r >> 1) & 7) : c ^ ((r >> 2) & 3);
}

// The same for chunk c of weight k row kr, in rows of 256 bytes (one matrix) or 128 (two): the
// transposing reads take 8 consecutive k rows x 2 neighbouring chunks per 32 lanes.
template <bool kGated>
__device__ __forceinline__ int bswz(int c, int kr)
{
    return kGated ? c ^ (((kr >> 1) & 3) << 1) : c ^ ((kr & 7) << 1);
}

template <int N>
__device__ __forceinline__ void step_barrier()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(N) : "memory");
}

__device__ __forceinline__ u32x4_t read16(uint32_t p)
{
    return *reinterpret_cast<const __attribute__((address_space(3))) u32x4_t*>(p);
}

// 16 consecutive k (rows kr .. + 15 from the lane's address) of the lane's column.
template <int kRowBytes>
__device__ __forceinline__ i32x4_t read_tr16(uint32_t p)
{
    const i32x2_t r0 = __builtin_amdgcn_ds_read_tr8_b64_v2i32(reinterpret_cast<lds_i32x2_t*>(p));
    const i32x2_t r1 = __builtin_amdgcn_ds_read_tr8_b64_v2i32(reinterpret_cast<lds_i32x2_t*>(p + 8 * kRowBytes));
    return i32x4_t{r0[0], r0[1], r1[0], r1[1]};
}

// (XCD, place in it) -> a task order in which an XCD's workgroups hold neighbouring tasks, which
// share weight strips and A rows in its L2.
__device__ __forceinline__ int first_task()
{
    const int b = static_cast<int>(blockIdx.x), per = static_cast<int>(gridDim.x) / kXcdCount;
    return (b % kXcdCount) * per + b / kXcdCount;
}

// Column block j of wave column wn: its matrix (gated: 0 gate, 1 up; blocks alternate, in one wave or
// from wave to wave) and its first column among the task's outputs.
template <class C, bool kGated>
__device__ __forceinline__ constexpr int block_mat(int wn, int j)
{
    return !kGated ? 0 : C::kTN > 1 ? j & 1 : wn & 1;
}
template <class C, bool kGated>
__device__ __forceinline__ constexpr int block_col(int wn, int j)
{
    return !kGated ? 32 * (C::kTN * wn + j) : C::kTN > 1 ? 16 * C::kTN * wn + 32 * (j >> 1) : 32 * (wn >> 1);
}

template <class C, bool kGated, int kOut>
__global__ __launch_bounds__(kThreads, 1) void grouped_gemm_i8(const Args a)
{
    constexpr int BN = kGated ? BNB / 2 : BNB;               // output columns per task
    constexpr int kRowBytes = kGated ? 128 : 256;            // one weight k row of one matrix in LDS
    constexpr int kChunks = kRowBytes / 16;
    constexpr int kRowsPerCopy = 64 / kChunks;
    constexpr int BK = C::BK;
    constexpr int kALanes = BK / 16;                         // lanes (16-byte chunks) per A row
    extern __shared__ __attribute__((aligned(256))) unsigned char smem[];
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) unsigned char*)(smem)));
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / C::kWN, wn = wave % C::kWN;
    const int lrow = lane & 31, lh = lane >> 5;
    const int K = a.K, N = a.N;
    const int n_nt = (N + BN - 1) / BN * a.splits;
    const int total = *a.tile_count * n_nt;

    // fragment addresses in stage 0
    uint32_t la_a[BK / 32], la_b[C::kTN];
    {
        const int r0 = 32 * wm + lrow;                       // row blocks interleave over the wave rows
#pragma unroll
        for (int q = 0; q < BK / 32; ++q)
            la_a[q] = lds0 + r0 * BK + 16 * aswz<BK>(2 * q + lh, r0);
        const int g = lane >> 4, sl = lane & 15;
        const int kr = 16 * (g >> 1) + (sl >> 1);
#pragma unroll
        for (int j = 0; j < C::kTN; ++j) {
            const int col = block_col<C, kGated>(wn, j) + 16 * (g & 1) + 8 * (sl & 1);
            la_b[j] = lds0 + C::kABytes + block_mat<C, kGated>(wn, j) * (C::kBBytes / 2) + kr * kRowBytes + 16 * bswz<kGated>(col >> 4, kr) + (col & 15);
        }
    }
    // copy places: A copy j of this wave covers rows kARows (kACopies wave + j) ..; B copy j covers k
    // rows of matrix `mat`
    constexpr int kARows = 64 / kALanes;
    const int mat = kGated ? wave / (kWaves / 2) : 0;
    const int bi0 = kGated ? C::kBCopies * (wave % (kWaves / 2)) : C::kBCopies * wave;
    const uint32_t a_lds = lds0 + C::kACopies * wave * 1024;
    const uint32_t b_lds = lds0 + C::kABytes + mat * (C::kBBytes / 2) + bi0 * 1024;

    for (int t = first_task(); t < total; t += static_cast<int>(gridDim.x)) {
        int nts;
        const MTile tile = decode_task(t, n_nt, a.tiles, nts);
        const int nt = nts / a.splits, split = nts % a.splits;
        const int n0 = nt * BN;
        const int rows = tile.row_end - tile.row_begin;
        const int steps_all = K / BK;
        const int kt0 = static_cast<int>(static_cast<int64_t>(steps_all) * split / a.splits);
        const int steps = static_cast<int>(static_cast<int64_t>(steps_all) * (split + 1) / a.splits) - kt0;

        uint32_t a_voff[C::kACopies], b_voff[C::kBCopies];
#pragma unroll
        for (int j = 0; j < C::kACopies; ++j) {
            const int r = kARows * (C::kACopies * wave + j) + lane / kALanes;
            const int c = aswz<BK>(lane % kALanes, r);
            const int rr = min(r, rows - 1);                 // rows past the tile's end: its last row again
            const int src = a.gather != nullptr ? a.gather[tile.row_begin + rr] / a.gather_k : rr;
            a_voff[j] = static_cast<uint32_t>(src) * static_cast<uint32_t>(K) + 16u * c;
        }
#pragma unroll
        for (int j = 0; j < C::kBCopies; ++j) {
            const int kr = (bi0 + j) * kRowsPerCopy + lane / kChunks;
            const int c = bswz<kGated>(lane % kChunks, kr);
            // columns past N (the second half of the last tile): the tile's first chunk again
            const int cc = n0 + 16 * c < N ? c : 0;
            b_voff[j] = static_cast<uint32_t>(kr) * static_cast<uint32_t>(N) + 16u * cc;
        }
        const int64_t k0 = static_cast<int64_t>(kt0) * BK;
        const uint8_t* ap = a.A + (a.gather != nullptr ? 0 : static_cast<int64_t>(tile.row_begin) * K) + k0;
        const uint8_t* bp = (kGated && mat == 1 ? a.B1 : a.B0) +
                            (static_cast<int64_t>(tile.expert) * K + k0) * N + n0;
        const auto issue = [&](int stage) {
            const uint32_t so = stage * C::kStageBytes;
#pragma unroll
            for (int j = 0; j < C::kACopies; ++j)
                lds_copy16(ap, a_voff[j], a_lds + so + j * 1024);
#pragma unroll
            for (int j = 0; j < C::kBCopies; ++j)
                lds_copy16(bp, b_voff[j], b_lds + so + j * 1024);
            ap += BK;
            bp += static_cast<int64_t>(BK) * N;
        };

        i32x16_t acc[C::kTM][C::kTN];
#pragma unroll
        for (int i = 0; i < C::kTM; ++i)
#pragma unroll
            for (int j = 0; j < C::kTN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    acc[i][j][r] = 0;

#pragma unroll
        for (int p = 0; p < C::kStages - 1; ++p)
            if (p < steps)
                issue(p);
        int stage = 0, fill = C::kStages - 1;
        for (int kt = 0; kt < steps; ++kt) {
            // step kt has landed once the copies of the later steps alone are in flight
            const int later = steps - 1 - kt;
            if (later >= C::kStages - 2)
                step_barrier<C::kCopies * (C::kStages - 2)>();
            else if (C::kStages >= 4 && later == 1)
                step_barrier<C::kCopies>();
            else
                step_barrier<0>();
            // every wave has read step kt - 1: its stage takes step kt + kStages - 1
            if (kt + C::kStages - 1 < steps)
                issue(fill);
            const uint32_t so = stage * C::kStageBytes;
            stage = stage + 1 == C::kStages ? 0 : stage + 1;
            fill = fill + 1 == C::kStages ? 0 : fill + 1;
#pragma unroll
            for (int q = 0; q < BK / 32; ++q) {
                i32x4_t fa[C::kTM], fb[C::kTN];
#pragma unroll
                for (int i = 0; i < C::kTM; ++i)
                    fa[i] = __builtin_bit_cast(i32x4_t, read16(la_a[q] + so + i * (C::kWM * 32 * BK)));
#pragma unroll
                for (int j = 0; j < C::kTN; ++j)
                    fb[j] = read_tr16<kRowBytes>(la_b[j] + so + q * (32 * kRowBytes));
#pragma unroll
                for (int j = 0; j < C::kTN; ++j)
#pragma unroll
                    for (int i = 0; i < C::kTM; ++i)
                        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
            }
        }
        step_barrier<0>();                                   // the stages are free for the next task

        // Epilogue.  Only the stores are under the lane's row test (no other lane-divergent region sits
        // in the task loop); a row past the tile's end reads the last row's scale.
        const float* s0 = a.s0 + static_cast<int64_t>(tile.expert) * N;
        [[maybe_unused]] const float* s1 = kGated ? a.s1 + static_cast<int64_t>(tile.expert) * N : nullptr;
#pragma unroll
        for (int i = 0; i < C::kTM; ++i) {
            const int grow = tile.row_begin + row_block<C::kWM>(i, wm) + lrow;
            const bool live = grow < tile.row_end;
            [[maybe_unused]] float as = 0.0f;
            if constexpr (kOut != kOutPartial) {
                const int r = min(grow, tile.row_end - 1);
                as = a.a_scale[a.gather != nullptr ? a.gather[r] / a.gather_k : r];
            }
#pragma unroll
            for (int j = 0; j < C::kTN; ++j) {
                if constexpr (kOut == kOutPartial) {
                    // int32 sums of this cut of K: [splits, M, N], gated [splits, M, 2 N] (gate, up)
                    const int64_t ld = kGated ? 2 * static_cast<int64_t>(N) : N;
                    const int col = n0 + block_col<C, kGated>(wn, j);
                    int32_t* dst = static_cast<int32_t*>(a.out) + (split * a.M + grow) * ld +
                                   block_mat<C, kGated>(wn, j) * static_cast<int64_t>(N) + col;
                    if (live && col < N)
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            *reinterpret_cast<i32x4_t*>(dst + 8 * g + 4 * lh) =
                                i32x4_t{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
                } else if constexpr (kGated) {
                    static_assert(C::kTN % 2 == 0, "a wave holds the gate and the up block of its outputs");
                    if (j % 2 == 0) {
                        const int col = n0 + block_col<C, kGated>(wn, j);
                        float* dst = static_cast<float*>(a.out) + static_cast<int64_t>(grow) * N + col;
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const int c = 8 * g + 4 * lh;
                            const f32x4_t sg = *reinterpret_cast<const f32x4_t*>(s0 + col + c);
                            const f32x4_t su = *reinterpret_cast<const f32x4_t*>(s1 + col + c);
                            f32x4_t h;
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                h[v] = swiglu(static_cast<float>(acc[i][j][4 * g + v]) * as * sg[v],
                                              static_cast<float>(acc[i][(j + 1) % C::kTN][4 * g + v]) * as * su[v]);
                            if (live)
                                *reinterpret_cast<f32x4_t*>(dst + c) = h;
                        }
                    }
                } else {
                    const int col = n0 + block_col<C, kGated>(wn, j);
                    const float* sc = s0 + (col < N ? col : 0);
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int c = 8 * g + 4 * lh;
                        const f32x4_t s = *reinterpret_cast<const f32x4_t*>(sc + c);
                        f32x4_t v;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = static_cast<float>(acc[i][j][4 * g + e]) * as * s[e];
                        const int64_t at = static_cast<int64_t>(grow) * N + col + c;
                        if (live && col < N) {
                            if constexpr (kOut == kOutF32)
                                *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + at) = v;
                            else
                                *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.out) + at) =
                                    u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                        }
                    }
                }
            }
        }
    }
}

using Large = Config<4, 2, 2, 4, 64, 4>;       // 256 rows
using Mid = Config<2, 4, 2, 2, 128, 3>;        // 128 rows
using Small = Config<1, 8, 2, 1, 128, 3>;      // 64 rows; partial sums only when gated

template <class C, bool kGated, int kOut>
hipError_t launch(const Args& a, hipStream_t s)
{
    static std::atomic<bool> done[64];         // per device: the LDS limit is raised
    int dev = 0;
    if (hipError_t e = hipGetDevice(&dev); e != hipSuccess)
        return e;
    const auto kernel = &grouped_gemm_i8<C, kGated, kOut>;
    if (dev >= 64 || !done[dev]) {
        if (hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
            e != hipSuccess)
            return e;
        if (dev < 64)
            done[dev] = true;
    }
    kernel<<<dim3(device_info().cu_count), dim3(kThreads), C::kSmemBytes, s>>>(a);
    return hipGetLastError();
}

template <bool kGated, int kOut>
hipError_t launch_rows(int bm, const Args& a, hipStream_t s)
{
    if (bm == Large::BM)
        return launch<Large, kGated, kOut>(a, s);
    if (bm == Mid::BM)
        return launch<Mid, kGated, kOut>(a, s);
    if constexpr (!kGated || kOut == kOutPartial)
        return launch<Small, kGated, kOut>(a, s);
    return hipErrorInvalidValue;
}

}  // namespace i8
}  // namespace

bool int8_supported(int64_t K, int64_t N)
{
    return K > 0 && N > 0 && K % 128 == 0 && N % 128 == 0 && K <= kInt8MaxK;
}

Int8Plan int8_plan(int64_t M, int64_t G, int64_t K, int64_t N, bool gated)
{
    // the groups that can hold rows, and the row tiles of each height they make at most
    const int64_t groups = std::max<int64_t>(1, std::min(M, G));
    const int64_t per_group = ceil_div(std::max<int64_t>(M, 1), groups);
    Int8Plan p;
    p.row_tile = per_group <= 64 ? 64 : per_group <= 160 ? 128 : 256;
    const int64_t cols = ceil_div(N, gated ? i8::BNB / 2 : i8::BNB);
    const int64_t tasks = (groups + M / p.row_tile) * cols;
    const int64_t steps = K / 128;
    p.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({steps, 16, 512 / std::max<int64_t>(1, tasks)})));
    if (p.row_tile == 256)
        p.splits = 1;
    p.partial = p.splits > 1 || (gated && p.row_tile == 64);
    return p;
}

hipError_t launch_gemm_i8(const Int8Plan& p, const int8_t* A, const float* a_scale, const int8_t* w0,
                          const float* s0, const int8_t* w1, const float* s1, void* out, int out_dtype,
                          int64_t M, int64_t K, int64_t N, const MTile* tiles, const int32_t* tile_count,
                          const int32_t* gather, int gather_k, hipStream_t s)
{
    i8::Args a{};
    a.A = reinterpret_cast<const uint8_t*>(A);
    a.a_scale = a_scale;
    a.B0 = reinterpret_cast<const uint8_t*>(w0);
    a.B1 = reinterpret_cast<const uint8_t*>(w1);
    a.s0 = s0;
    a.s1 = s1;
    a.out = out;
    a.tiles = tiles;
    a.tile_count = tile_count;
    a.gather = gather;
    a.gather_k = gather_k;
    a.K = static_cast<int>(K);
    a.N = static_cast<int>(N);
    a.splits = p.splits;
    a.M = M;
    const bool gated = w1 != nullptr;
    if (p.partial)
        return gated ? i8::launch_rows<true, i8::kOutPartial>(p.row_tile, a, s)
                     : i8::launch_rows<false, i8::kOutPartial>(p.row_tile, a, s);
    if (gated)
        return i8::launch_rows<true, i8::kOutF32>(p.row_tile, a, s);
    return out_dtype == MOE_F32 ? i8::launch_rows<false, i8::kOutF32>(p.row_tile, a, s)
                                : i8::launch_rows<false, i8::kOutBf16>(p.row_tile, a, s);
}

}  // namespace moe
