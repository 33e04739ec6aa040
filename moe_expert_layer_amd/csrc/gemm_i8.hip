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
//
// Few rows are bound by the weights' bytes: 64-row tiles, copies that run ahead across a workgroup's tasks
// and K cut until the CUs are evenly busy (1000 rows on 128 experts of 2048 x 768: gate and up 73 us for
// at most 403 MB, 5.5 TB/s).  Many rows are bound by the matrix instructions: 256-row tiles (16384 rows, 2
// experts of 4096 x 14336: 0.86-0.93 ms, 2.1-2.2 POP/s).  product_cost below chooses.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <utility>

#include "gemm_common.h"
#include "int8_gate.h"
#include "int8_tiles.h"

namespace moe {
namespace {
namespace i8 {

typedef int i32x16_t __attribute__((ext_vector_type(16)));
typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2_t lds_i32x2_t;

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
constexpr int BNB = 256;                       // weight columns per task (both matrices of a gated task)
constexpr int kOwnTiles = 512;                 // of the table that a workgroup builds for itself: a group per thread
constexpr int kOwnTableBytes = 16 * kOwnTiles + 8 * kWaves;    // and the scan's words
static_assert(kOwnTiles <= kThreads && kMaxExperts < 1 << 23, "the own table's scan and entries");

enum Out { kOutBf16, kOutF32, kOutPartial, kOutHalf };     // kOutHalf: the sums times `unit`, as float16

struct Args {
    const uint8_t* A;                          // int8 rows
    const float* a_scale;
    const uint8_t* B0;                         // int8 [E, K, N]; B1: the up matrix of a gated task
    const uint8_t* B1;
    const float* s0;                           // [E, N]
    const float* s1;
    void* out;                                 // [M, N], or int32 partial sums [splits, M, N or 2N]
    Int8Groups groups;
    const int32_t* gather;                     // may be null: row p of the product is row gather[p] / gather_k of A
    int gather_k;
    int32_t* task_ctr;                         // kXcdCount zeroed counters (large tiles)
    int K, N, splits;
    int64_t M;
    float unit;
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
    static_assert(kSmemBytes + kOwnTableBytes <= 160 * 1024, "LDS");
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

// Neighbouring tasks that one XCD works on at a time (they share weight strips and A rows in its L2): one
// for each of its workgroups, or an eighth of them all where there are fewer, so that every XCD has its
// part of the HBM traffic (64 tasks on two XCDs instead of eight: 111 against 76 us).
__device__ __forceinline__ int xcd_run(int total)
{
    return max(1, min(static_cast<int>(gridDim.x) / kXcdCount, (total + kXcdCount - 1) / kXcdCount));
}
// The workgroup's first task; `total` if it has none.
__device__ __forceinline__ int first_task(int total)
{
    const int xcd = static_cast<int>(blockIdx.x) % kXcdCount, place = static_cast<int>(blockIdx.x) / kXcdCount;
    const int run = xcd_run(total);
    return place < run ? xcd * run + place : total;
}

// A pointer that is the same on every lane, in scalar registers.
__device__ __forceinline__ const uint8_t* scalar(const uint8_t* p)
{
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<int>(v));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<int>(v >> 32));
    return reinterpret_cast<const uint8_t*>(static_cast<uint64_t>(hi) << 32 | lo);
}

// decode_task with its results in scalar registers.
__device__ __forceinline__ MTile uniform_task(int t, int n_nt, const MTile* __restrict__ tiles, int& nt)
{
    int n;
    const MTile m = decode_task(t, n_nt, tiles, n);
    MTile u{};
    u.expert = __builtin_amdgcn_readfirstlane(m.expert);
    u.row_begin = __builtin_amdgcn_readfirstlane(m.row_begin);
    u.row_end = __builtin_amdgcn_readfirstlane(m.row_end);
    nt = __builtin_amdgcn_readfirstlane(n);
    return u;
}

// A tile of the table that a workgroup builds for itself in LDS: first row, rows | expert << 8, and its run.
typedef __attribute__((address_space(3))) i32x4_t lds_tile_t;
__device__ __forceinline__ MTile uniform_task(int t, int n_nt, const lds_tile_t* tiles, int& nt)
{
    const i32x4_t head = tiles[t / n_nt];
    const int local = t - n_nt * head[2];
    nt = __builtin_amdgcn_readfirstlane(local / head[3]);
    const i32x4_t m = tiles[head[2] + local % head[3]];
    MTile u{};
    u.row_begin = __builtin_amdgcn_readfirstlane(m[0]);
    u.row_end = u.row_begin + __builtin_amdgcn_readfirstlane(m[1] & 255);
    u.expert = __builtin_amdgcn_readfirstlane(m[1] >> 8);
    return u;
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

template <class C, bool kGated, int kOut, bool kOwn>
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
    const int n_nt = (N + BN - 1) / BN;
    // The row tiles: a table in memory, or for few groups one that each workgroup builds in LDS, which costs
    // under a microsecond where a launch for the table costs five (1000 rows on 128 experts of 2048 x 1536: 73.8
    // -> 69.7 us; 500 rows on 8 of 2048 x 4096: 22.1 -> 18.6 us)
    [[maybe_unused]] lds_tile_t* const own = reinterpret_cast<lds_tile_t*>(lds0 + C::kSmemBytes);
    int row_tiles;
    if constexpr (kOwn) {
        int* const wave_max = reinterpret_cast<int*>(smem + C::kSmemBytes + 16 * kOwnTiles);
        int* const wave_sum = wave_max + kWaves;
        int reached = 0;
        const GroupRows r = scan_groups<kWaves>(a.groups.offsets, a.groups.expert, 0, a.groups.G, a.groups.E, a.M, C::BM,
                                                reached, wave_max, wave_sum);
        const int R = (r.rows + C::BM - 1) / C::BM;
        for (int i = 0; i < R; ++i) {
            const MTile m = balanced_tile(r.expert, r.begin, r.rows, R, i, r.first);
            own[r.first + i] = i32x4_t{m.row_begin, (m.row_end - m.row_begin) | m.expert << 8, m.run_begin, R};
        }
        const int bad = __syncthreads_or(r.bad ? 1 : 0);
        if (a.groups.status != nullptr && blockIdx.x == 0 && threadIdx.x == 0)
            *a.groups.status = bad ? MOE_ERR_EXPERT_ID_OUT_OF_RANGE : MOE_OK;
        row_tiles = r.total;
    } else {
        row_tiles = *a.groups.tile_count;
    }
    const int total = __builtin_amdgcn_readfirstlane(row_tiles * n_nt * a.splits);
    const auto task_tile = [&](int t, int& nt) {
        if constexpr (kOwn)
            return uniform_task(t / a.splits, n_nt, own, nt);
        else
            return uniform_task(t / a.splits, n_nt, a.groups.tiles, nt);
    };

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

    const int steps_all = K / BK;
    const auto steps_of = [&](int task) {                    // [begin, end) of the task's cut of K
        const int split = task % a.splits;
        return int2{static_cast<int>(static_cast<int64_t>(steps_all) * split / a.splits),
                    static_cast<int>(static_cast<int64_t>(steps_all) * (split + 1) / a.splits)};
    };
    const int grid = static_cast<int>(gridDim.x);

    // The copies run kStages - 1 steps ahead of the products through all of the workgroup's tasks: task
    // pt is the one being copied, its successor's tile entry and slot-list entries are loaded ahead.
    int pt = first_task(total) - grid, left = 0, stage = 0, fill = 0, ahead = 0;
    MTile next_tile{};
    int next_nt = 0;
    int gsrc[C::kACopies] = {};
    const auto fetch = [&](int task) {
        if (task >= total)
            return;
        next_tile = task_tile(task, next_nt);
        const int rows = next_tile.row_end - next_tile.row_begin;
#pragma unroll
        for (int j = 0; j < C::kACopies; ++j)
            gsrc[j] = (kARows * (C::kACopies * wave + j) + lane / kALanes) % rows;   // past the tile's end: its rows again
        if (a.gather != nullptr) {
#pragma unroll
            for (int j = 0; j < C::kACopies; ++j)
                gsrc[j] = a.gather[next_tile.row_begin + gsrc[j]];
            // waited for here: left in flight, they would put a wait for every copy into each step
#pragma unroll
            for (int j = 0; j < C::kACopies; ++j)
                asm volatile("" : "+v"(gsrc[j]));
        }
    };
    uint32_t a_voff[C::kACopies], b_voff[C::kBCopies];
    const uint8_t* ap = nullptr;
    const uint8_t* bp = nullptr;
    const auto issue = [&]() {
        if (left == 0) {
            pt += grid;
            if (pt >= total)
                return;
            const int n0 = next_nt * BN;
#pragma unroll
            for (int j = 0; j < C::kACopies; ++j) {
                const int r = kARows * (C::kACopies * wave + j) + lane / kALanes;
                const int src = a.gather != nullptr ? gsrc[j] / a.gather_k : gsrc[j];
                a_voff[j] = static_cast<uint32_t>(src) * static_cast<uint32_t>(K) + 16u * aswz<BK>(lane % kALanes, r);
            }
#pragma unroll
            for (int j = 0; j < C::kBCopies; ++j) {
                const int kr = (bi0 + j) * kRowsPerCopy + lane / kChunks;
                const int c = bswz<kGated>(lane % kChunks, kr);
                // columns past N (the second half of the last tile): the tile's first chunk again
                b_voff[j] = static_cast<uint32_t>(kr) * static_cast<uint32_t>(N) + 16u * (n0 + 16 * c < N ? c : 0);
            }
            const int2 kt = steps_of(pt);
            left = kt.y - kt.x;
            const int64_t k0 = static_cast<int64_t>(kt.x) * BK;
            ap = scalar(a.A + (a.gather != nullptr ? 0 : static_cast<int64_t>(next_tile.row_begin) * K) + k0);
            bp = scalar((kGated && mat == 1 ? a.B1 : a.B0) + (static_cast<int64_t>(next_tile.expert) * K + k0) * N + n0);
            fetch(pt + grid);
        }
        const uint32_t so = __builtin_amdgcn_readfirstlane(fill) * C::kStageBytes;
#pragma unroll
        for (int j = 0; j < C::kACopies; ++j)
            lds_copy16(ap, a_voff[j], a_lds + so + j * 1024);
#pragma unroll
        for (int j = 0; j < C::kBCopies; ++j)
            lds_copy16(bp, b_voff[j], b_lds + so + j * 1024);
        ap += BK;
        bp += static_cast<int64_t>(BK) * N;
        --left;
        ++ahead;
        fill = fill + 1 == C::kStages ? 0 : fill + 1;
    };
    fetch(pt + grid);
#pragma unroll
    for (int p = 0; p < C::kStages - 1; ++p)
        issue();
    static_assert(C::kStages == 3, "the waits below");

    for (int t = first_task(total); t < total; t += grid) {
        int nt;
        const MTile tile = task_tile(t, nt);
        const int n0 = nt * BN;
        [[maybe_unused]] const int split = t % a.splits;
        const int2 kt = steps_of(t);
        const int steps = kt.y - kt.x;

        i32x16_t acc[C::kTM][C::kTN];
#pragma unroll
        for (int i = 0; i < C::kTM; ++i)
#pragma unroll
            for (int j = 0; j < C::kTN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    acc[i][j][r] = 0;

        for (int k = 0; k < steps; ++k) {
            // this step has landed once the copies of the one after it alone are in flight
            --ahead;
            if (ahead > 0)
                step_barrier<C::kCopies>();
            else
                step_barrier<0>();
            issue();                                         // into the stage that every wave has just finished
            const uint32_t so = stage * C::kStageBytes;
            stage = stage + 1 == C::kStages ? 0 : stage + 1;
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

        // Epilogue.  Only the stores are under the lane's row test (no other lane-divergent region sits
        // in the task loop); a row past the tile's end reads the last row's scale.  All scales are loaded
        // first, in one wait: each wait also waits for the copies in flight and for the stores before it.
        [[maybe_unused]] f32x4_t scale[C::kTN][4];            // of column block j (gated: of its matrix)
        [[maybe_unused]] float row_scale[C::kTM];
        if constexpr (kOut == kOutBf16 || kOut == kOutF32) {
#pragma unroll
            for (int j = 0; j < C::kTN; ++j) {
                const int col = n0 + block_col<C, kGated>(wn, j);
                const float* sc = (kGated && block_mat<C, kGated>(wn, j) == 1 ? a.s1 : a.s0) +
                                  static_cast<int64_t>(tile.expert) * N + (col < N ? col : 0);
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    scale[j][g] = *reinterpret_cast<const f32x4_t*>(sc + 8 * g + 4 * lh);
            }
#pragma unroll
            for (int i = 0; i < C::kTM; ++i) {
                const int r = min(tile.row_begin + row_block<C::kWM>(i, wm) + lrow, tile.row_end - 1);
                row_scale[i] = a.a_scale[a.gather != nullptr ? a.gather[r] / a.gather_k : r];
            }
#pragma unroll
            for (int j = 0; j < C::kTN; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    asm volatile("" : "+v"(scale[j][g]));     // not to be loaded between the stores
#pragma unroll
            for (int i = 0; i < C::kTM; ++i)
                asm volatile("" : "+v"(row_scale[i]));
        }
#pragma unroll
        for (int i = 0; i < C::kTM; ++i) {
            const int grow = tile.row_begin + row_block<C::kWM>(i, wm) + lrow;
            const bool live = grow < tile.row_end;
            [[maybe_unused]] const float as = kOut == kOutBf16 || kOut == kOutF32 ? row_scale[i] : a.unit;
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
                            const int up = (j + 1) % C::kTN;
                            f32x4_t h;
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                h[v] = swiglu(static_cast<float>(acc[i][j][4 * g + v]) * as * scale[j][g][v],
                                              static_cast<float>(acc[i][up][4 * g + v]) * as * scale[up][g][v]);
                            if (live)
                                *reinterpret_cast<f32x4_t*>(dst + c) = h;
                        }
                    }
                } else {
                    const int col = n0 + block_col<C, kGated>(wn, j);
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int c = 8 * g + 4 * lh;
                        f32x4_t v;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = kOut == kOutHalf ? static_cast<float>(acc[i][j][4 * g + e]) * as
                                                    : static_cast<float>(acc[i][j][4 * g + e]) * as * scale[j][g][e];
                        const int64_t at = static_cast<int64_t>(grow) * N + col + c;
                        if (live && col < N) {
                            if constexpr (kOut == kOutF32)
                                *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + at) = v;
                            else
                                *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.out) + at) =
                                    kOut == kOutHalf ? u32x2_t{pack_half2(v[0], v[1]), pack_half2(v[2], v[3])}
                                                     : u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                        }
                    }
                }
            }
        }
    }
}

// ----------------------------------------------------------------------------------- large tiles
//
// 256 rows x 256 weight columns per task (8 waves of 64 x 128, two per SIMD) for K >= 256: the structure
// of the MX large-tile kernel.  A K step is 64 values (two MFMAs per block).  The weights go through
// four stages of one step, A through two stages of a pair of steps (rows of 128 bytes, whole cache
// lines); three steps are in flight.  Each step's MFMAs run in two halves around its one barrier
// (weight blocks 0-1, then 2-3), each followed by its share of the step's copies and fragment reads.
// Tasks are claimed per XCD, and the next task's first copies go out before the current epilogue.
// Measured against the ring kernel above with 256-row tiles: 16384 x 4096 x 14336 1.07 -> 0.92 ms, 65536
// rows on 32 experts of 7168 x 2048 1.95 -> 1.63 ms (gate and up) and 1.28 -> 1.02 ms (down).
namespace big {

constexpr int kWM = 4, kWN = 2, kTM = 2, kTN = 4;
constexpr int BM = kWM * kTM * 32;                    // 256
constexpr int BK = 64;
constexpr int kStages = 4;
constexpr int kBBytes = BK * BNB;                     // one weight stage: 16 KiB
constexpr int kAPairBytes = BM * 2 * BK;              // one A stage: 32 KiB
constexpr int kBRing = 2 * kAPairBytes;               // the A stages, then the weight stages
constexpr int kOutBase = kBRing + kStages * kBBytes;  // 128 KiB
constexpr int kOutWaveBytes = 4096;                   // epilogue staging per wave
constexpr int kSmemBytes = kOutBase + kWaves * kOutWaveBytes;
constexpr int kACopies = kAPairBytes / 1024 / kWaves; // 4 per wave and pair
constexpr int kBCopies = kBBytes / 1024 / kWaves;     // 2 per wave and step
static_assert(kSmemBytes <= 160 * 1024, "LDS");

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// Sources (uniform) and LDS destinations of this wave's copies: A at the next pair, the weights at the
// next step.
struct Copy {
    const uint8_t* a;
    const uint8_t* b;
    uint32_t a_lds, b_lds;
};

// Copies C0 .. C1 - 1 of a step's list: its weights into stage SB when SB >= 0, then the A of a pair into
// pair stage QA when QA >= 0 (the barriers' waits count on this order).
template <int SB, int QA>
constexpr int copy_count() { return (SB >= 0 ? kBCopies : 0) + (QA >= 0 ? kACopies : 0); }
template <int SB, int QA, int C0, int C1>
__device__ __forceinline__ void copies(const Copy& c, const uint32_t (&a_voff)[kACopies],
                                       const uint32_t (&b_voff)[kBCopies])
{
    constexpr int nb = SB >= 0 ? kBCopies : 0;
#pragma unroll
    for (int q = C0; q < C1; ++q) {
        if (q < nb)
            lds_copy16(c.b, b_voff[q], c.b_lds + SB * kBBytes + q * 1024);
        else
            lds_copy16(c.a, a_voff[q - nb], c.a_lds + QA * kAPairBytes + (q - nb) * 1024);
    }
}

// The lane's fragment addresses in stage 0, hidden from the optimiser so that stages and blocks stay
// immediate offsets.
struct LaneAddr {
    uint32_t a[2][2];         // A, pair half hp: chunks 4 hp + h and 4 hp + 2 + h of the lane's row
    uint32_t b[kTN];
};

struct Frag {                 // 64 k of one row or column: the two MFMAs' operands
    i32x4_t k0, k1;
};

template <int p>
__device__ __forceinline__ void read_a(Frag& f, const LaneAddr& la, int i)
{
    constexpr int S = p % kStages;
    const uint32_t o = (S / 2) * kAPairBytes + i * (kWM * 32 * 128);
    f.k0 = __builtin_bit_cast(i32x4_t, read16(la.a[S % 2][0] + o));
    f.k1 = __builtin_bit_cast(i32x4_t, read16(la.a[S % 2][1] + o));
}
template <bool kGated, int p>
__device__ __forceinline__ void read_b(Frag& f, const LaneAddr& la, int j)
{
    constexpr int kRowBytes = kGated ? 128 : 256;
    const uint32_t at = la.b[j] + (p % kStages) * kBBytes;
    f.k0 = read_tr16<kRowBytes>(at);
    f.k1 = read_tr16<kRowBytes>(at + 32 * kRowBytes);
}

// MFMA mm of one half step (all blocks' first 32 k, then their second): block (row i, column j0 + jj).
template <int NB, int J0, int mm>
__device__ __forceinline__ void mfma(i32x16_t (&acc)[kTM][kTN], const Frag (&A)[kTM], const Frag (&b)[2])
{
    constexpr int m = mm % (2 * NB), i = m / 2, jj = m % 2;
    acc[i][J0 + jj] = __builtin_amdgcn_mfma_i32_32x32x32_i8(mm < 2 * NB ? b[jj].k0 : b[jj].k1,
                                                            mm < 2 * NB ? A[i].k0 : A[i].k1, acc[i][J0 + jj], 0, 0, 0);
}

template <bool kGated, int NB, int p, int mm>
__device__ __forceinline__ void before(i32x16_t (&acc)[kTM][kTN], const Frag (&A)[kTM], const Frag (&b01)[2],
                                       Frag (&b23)[2], const LaneAddr& la)
{
    mfma<NB, 0, mm>(acc, A, b01);
    if constexpr (mm < 2)
        read_b<kGated, p>(b23[mm], la, 2 + mm);
    __builtin_amdgcn_sched_barrier(0);
}

// After the barrier: the copies and the next step's reads are spread over the first half of the MFMAs,
// so that the reads land well before the next step needs them.
template <bool kGated, int NB, int p, int SB, int QA, int mm>
__device__ __forceinline__ void after(i32x16_t (&acc)[kTM][kTN], const Frag (&A)[kTM], Frag (&An)[kTM],
                                      const Frag (&b23)[2], Frag (&b01)[2], const LaneAddr& la, const Copy& cp,
                                      const uint32_t (&a_voff)[kACopies], const uint32_t (&b_voff)[kBCopies])
{
    constexpr int half = 2 * NB, NC = copy_count<SB, QA>(), NR = NB + 2;
    constexpr int pn = (p + 1) % kStages;
    mfma<NB, 2, mm>(acc, A, b23);
    if constexpr (mm < half) {
        copies<SB, QA, mm * NC / half, (mm + 1) * NC / half>(cp, a_voff, b_voff);
#pragma unroll
        for (int r = mm * NR / half; r < (mm + 1) * NR / half; ++r) {
            if (r == 0)
                read_a<pn>(An[0], la, 0);
            else if (r < 3)
                read_b<kGated, pn>(b01[r - 1], la, r - 1);
            else
                read_a<pn>(An[NB - 1], la, NB - 1);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
}

// Copies in flight that still let "step t + 1 has landed" hold at the barrier of step t (at position p of
// a unit).  In issue order: setup A pair 0, weights 0 .. 3, pair 1; after barrier t weights t + 4 and, t
// odd, pair (t + 3) / 2.  Even t: what step t + 1 needs was complete a barrier before, but for t = 0, where
// the weights of steps 2, 3 and pair 1 may be open.  Odd t: pair (t + 1) / 2 has only the weights of step
// t + 3 behind it (nothing in a task's last unit).
template <int p, bool kLast>
constexpr int wait() { return p % 2 == 0 ? 2 * kBCopies + kACopies : kLast ? 0 : kBCopies; }
constexpr int kTopWait = 3 * kBCopies + kACopies;     // step 0 has landed

template <bool kGated, int NB, int p, bool kLast, int... Ms>
__device__ __forceinline__ void step(std::integer_sequence<int, Ms...>, i32x16_t (&acc)[kTM][kTN], const Frag (&A)[kTM],
                                     Frag (&An)[kTM], Frag (&b01)[2], Frag (&b23)[2], const LaneAddr& la, Copy& cp,
                                     const uint32_t (&a_voff)[kACopies], const uint32_t (&b_voff)[kBCopies],
                                     int64_t N)
{
    constexpr int SB = kLast ? -1 : p, QA = !kLast && p % 2 == 1 ? ((p + 3) / 2) % 2 : -1;
    __builtin_amdgcn_sched_barrier(0);
    (before<kGated, NB, p, Ms>(acc, A, b01, b23, la), ...);
    if constexpr (!kLast || p + 1 < kStages)
        step_barrier<wait<p, kLast>()>();
    __builtin_amdgcn_sched_barrier(0);
    // after a task's last step the reads take a stale stage, whose fragments are never used
    if constexpr (NB > 0)
        (after<kGated, NB, p, SB, QA, Ms>(acc, A, An, b23, b01, la, cp, a_voff, b_voff), ...);
    else
        copies<SB, QA, 0, copy_count<SB, QA>()>(cp, a_voff, b_voff);
    if constexpr (SB >= 0)
        cp.b += BK * N;
    if constexpr (QA >= 0)
        cp.a += 2 * BK;
    __builtin_amdgcn_sched_barrier(0);
}

// The K loop of one task: KT even, at least 4; an odd number of pairs starts at position 2 (setup puts
// its first copies there).  Every LDS address is a lane base plus a constant.
template <bool kGated, int NB>
__device__ __forceinline__ void k_loop(i32x16_t (&acc)[kTM][kTN], const LaneAddr& la, Copy cp,
                                       const uint32_t (&a_voff)[kACopies], const uint32_t (&b_voff)[kBCopies], int KT,
                                       int64_t N)
{
    constexpr auto ms = std::make_integer_sequence<int, 4 * NB>{};
    Frag A0[kTM], A1[kTM], b01[2], b23[2];
    const bool half = (KT & 2) != 0;
    if constexpr (NB > 0) {
        if (half) {
#pragma unroll
            for (int i = 0; i < NB; ++i)
                read_a<2>(A0[i], la, i);
            read_b<kGated, 2>(b01[0], la, 0);
            read_b<kGated, 2>(b01[1], la, 1);
        } else {
#pragma unroll
            for (int i = 0; i < NB; ++i)
                read_a<0>(A0[i], la, i);
            read_b<kGated, 0>(b01[0], la, 0);
            read_b<kGated, 0>(b01[1], la, 1);
        }
    }
    if (half) {
        step<kGated, NB, 2, false>(ms, acc, A0, A1, b01, b23, la, cp, a_voff, b_voff, N);
        step<kGated, NB, 3, false>(ms, acc, A1, A0, b01, b23, la, cp, a_voff, b_voff, N);
    }
    for (int kt = half ? 2 : 0; kt < KT - kStages; kt += kStages) {
        step<kGated, NB, 0, false>(ms, acc, A0, A1, b01, b23, la, cp, a_voff, b_voff, N);
        step<kGated, NB, 1, false>(ms, acc, A1, A0, b01, b23, la, cp, a_voff, b_voff, N);
        step<kGated, NB, 2, false>(ms, acc, A0, A1, b01, b23, la, cp, a_voff, b_voff, N);
        step<kGated, NB, 3, false>(ms, acc, A1, A0, b01, b23, la, cp, a_voff, b_voff, N);
    }
    step<kGated, NB, 0, true>(ms, acc, A0, A1, b01, b23, la, cp, a_voff, b_voff, N);
    step<kGated, NB, 1, true>(ms, acc, A1, A0, b01, b23, la, cp, a_voff, b_voff, N);
    step<kGated, NB, 2, true>(ms, acc, A0, A1, b01, b23, la, cp, a_voff, b_voff, N);
    step<kGated, NB, 3, true>(ms, acc, A1, A0, b01, b23, la, cp, a_voff, b_voff, N);
}

template <bool kGated, int kOut>
__global__ __launch_bounds__(kThreads, 1) void grouped_gemm_i8_dma(const Args a)
{
    constexpr int BN = kGated ? BNB / 2 : BNB;
    constexpr int kRowBytes = kGated ? 128 : 256;
    constexpr int kChunks = kRowBytes / 16;
    constexpr int kRowsPerCopy = 64 / kChunks;
    using C = Config<kWM, kWN, kTM, kTN, BK, 2>;             // the wave layout, for block_mat / block_col
    extern __shared__ __attribute__((aligned(256))) unsigned char smem[];
    int* const claimed = reinterpret_cast<int*>(smem + kOutBase);   // start of wave 0's staging
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) unsigned char*)(smem)));
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / kWN, wn = wave % kWN;
    const int lrow = lane & 31, lh = lane >> 5;
    const int K = a.K, N = a.N;
    const int KT = K / BK;
    const int n_nt = (N + BN - 1) / BN;
    const int total = __builtin_amdgcn_readfirstlane(*a.groups.tile_count * n_nt);
    const int first = KT & 2;                                // position of a task's first step

    const int mat = kGated ? wave / (kWaves / 2) : 0;
    const int bi0 = kGated ? kBCopies * (wave % (kWaves / 2)) : kBCopies * wave;
    Copy cp{};
    cp.a_lds = lds0 + kACopies * wave * 1024;
    cp.b_lds = lds0 + kBRing + mat * (kBBytes / 2) + bi0 * 1024;
    LaneAddr la;
    {
        const int r0 = 32 * wm + lrow;
#pragma unroll
        for (int hp = 0; hp < 2; ++hp)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                la.a[hp][q] = lds0 + r0 * 128 + 16 * aswz<128>(4 * hp + 2 * q + lh, r0);
        const int g = lane >> 4, sl = lane & 15;
        const int kr = 16 * (g >> 1) + (sl >> 1);
#pragma unroll
        for (int j = 0; j < kTN; ++j) {
            const int col = block_col<C, kGated>(wn, j) + 16 * (g & 1) + 8 * (sl & 1);
            la.b[j] = lds0 + kBRing + block_mat<C, kGated>(wn, j) * (kBBytes / 2) + kr * kRowBytes +
                      16 * bswz<kGated>(col >> 4, kr) + (col & 15);
        }
        asm volatile("" : "+v"(la.a[0][0]), "+v"(la.a[0][1]), "+v"(la.a[1][0]), "+v"(la.a[1][1]));
#pragma unroll
        for (int j = 0; j < kTN; ++j)
            asm volatile("" : "+v"(la.b[j]));
    }

    const int xcd = blockIdx.x % kXcdCount;
    const int blk = xcd_run(total);
    MTile tile{};
    int n0 = 0;
    uint32_t a_voff[kACopies], b_voff[kBCopies];
    // Gathered rows: the slot-list entries of this lane's copy rows, loaded a task ahead.
    int gsrc[kACopies] = {};
    const auto fetch_rows = [&](const MTile& tl) {
        if (a.gather == nullptr)
            return;
        const int last = tl.row_end - tl.row_begin - 1;
#pragma unroll
        for (int j = 0; j < kACopies; ++j)
            gsrc[j] = a.gather[tl.row_begin + min(8 * (kACopies * wave + j) + lane / 8, last)];
    };
    const auto setup = [&](const MTile& tl, int nt) {
        tile = tl;
        n0 = nt * BN;
        const int rows = tile.row_end - tile.row_begin;
#pragma unroll
        for (int j = 0; j < kACopies; ++j) {
            const int r = 8 * (kACopies * wave + j) + lane / 8;      // 8 lanes per 128-byte row
            const int src = a.gather != nullptr ? gsrc[j] / a.gather_k : min(r, rows - 1);
            a_voff[j] = static_cast<uint32_t>(src) * static_cast<uint32_t>(K) + 16u * aswz<128>(lane % 8, r);
        }
#pragma unroll
        for (int j = 0; j < kBCopies; ++j) {
            const int kr = (bi0 + j) * kRowsPerCopy + lane / kChunks;
            const int c = bswz<kGated>(lane % kChunks, kr);
            // columns past N (the second half of the last tile): the tile's first chunk again
            b_voff[j] = static_cast<uint32_t>(kr) * static_cast<uint32_t>(N) + 16u * (n0 + 16 * c < N ? c : 0);
        }
        cp.a = a.A + (a.gather != nullptr ? 0 : static_cast<int64_t>(tile.row_begin) * K);
        cp.b = (kGated && mat == 1 ? a.B1 : a.B0) + static_cast<int64_t>(tile.expert) * K * N + n0;
        // A pair 0, the weights of steps 0 .. 3, A pair 1 (the waits count on this order)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int j = 0; j < kACopies; ++j)
                lds_copy16(cp.a, a_voff[j], cp.a_lds + ((first / 2 + q) & 1) * kAPairBytes + j * 1024);
            cp.a += 2 * BK;
            if (q == 1)
                continue;
#pragma unroll
            for (int st = 0; st < kStages; ++st) {
#pragma unroll
                for (int j = 0; j < kBCopies; ++j)
                    lds_copy16(cp.b, b_voff[j], cp.b_lds + ((first + st) & 3) * kBBytes + j * 1024);
                cp.b += static_cast<int64_t>(BK) * N;
            }
        }
    };

    // Claims: two ahead when gathering rows or running at least four tasks per workgroup (a task's
    // successor is in the claim word at its top barrier, and its tile entry is loaded during its K loop),
    // else one ahead, read after the K loop.
    const bool ahead2 = a.gather != nullptr || total >= 4 * static_cast<int>(gridDim.x);
    int t = claim_task(claimed, a.task_ctr, xcd, blk, wave, lane);
    if (ahead2)
        claim_task(claimed, a.task_ctr, xcd, blk, wave, lane);
    if (t < total) {
        int nt;
        const MTile tl = decode_task(t, n_nt, a.groups.tiles, nt);
        fetch_rows(tl);
        setup(tl, nt);
    }
    while (t < total) {
        const int rows = tile.row_end - tile.row_begin;
        const int nb = __builtin_amdgcn_readfirstlane(min(kTM, max(0, ((rows + 31) / 32 - wm + kWM - 1) / kWM)));
        i32x16_t acc[kTM][kTN];
#pragma unroll
        for (int i = 0; i < kTM; ++i)
#pragma unroll
            for (int j = 0; j < kTN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    acc[i][j][r] = 0;
        // step 0 has landed; past this barrier every wave sees the claim of the following task
        step_barrier<kTopWait>();
        int t_next = total;
        MTile tile_next{};
        int nt_next = 0;
        if (ahead2) {
            const int ci = __builtin_amdgcn_readfirstlane(*claimed);
            t_next = ((ci / blk) * kXcdCount + xcd) * blk + ci % blk;
            if (t_next < total)
                tile_next = decode_task(t_next, n_nt, a.groups.tiles, nt_next);
        }
        const int claim_ret = claim_issue(a.task_ctr, xcd, wave, lane);
        if (t_next < total)
            fetch_rows(tile_next);
        if (nb == 0)
            k_loop<kGated, 0>(acc, la, cp, a_voff, b_voff, KT, N);
        else if (nb == 1)
            k_loop<kGated, 1>(acc, la, cp, a_voff, b_voff, KT, N);
        else
            k_loop<kGated, 2>(acc, la, cp, a_voff, b_voff, KT, N);
        const int claim_after = claim_value(claim_ret, wave);
        if (!ahead2) {
            if (wave == 0)
                *claimed = claim_after;
            __syncthreads();
            const int ci = __builtin_amdgcn_readfirstlane(*claimed);
            t_next = ((ci / blk) * kXcdCount + xcd) * blk + ci % blk;
            if (t_next < total)
                tile_next = decode_task(t_next, n_nt, a.groups.tiles, nt_next);
        }
        const MTile done = tile;
        const int done_n0 = n0;
        t = t_next;
        __syncthreads();                                     // the ring is free, and the claim word read
        if (t < total)
            setup(tile_next, nt_next);

        // Epilogue: scaled blocks through the wave's staging area (rows of 128 bytes, 16-byte chunks
        // XOR-swizzled by row), out as whole 128-byte row pieces.  Only the stores are under a row test.
        const uint32_t stg = lds0 + kOutBase + wave * kOutWaveBytes;
        const float* s0 = a.s0 + static_cast<int64_t>(done.expert) * N;
        [[maybe_unused]] const float* s1 = kGated ? a.s1 + static_cast<int64_t>(done.expert) * N : nullptr;
        constexpr bool kWide = kGated || kOut == kOutF32;    // float32 out: one 32-column block a row piece
        constexpr int kBlocks = kGated ? kTN / 2 : kTN;      // output blocks of this wave's columns
        constexpr int kPiece = kWide ? 1 : 2;                // output blocks per row piece
#pragma unroll
        for (int i = 0; i < kTM; ++i) {
            const int srow = min(done.row_begin + row_block<kWM>(i, wm) + lrow, done.row_end - 1);
            const float as = kOut == kOutHalf ? a.unit : a.a_scale[a.gather != nullptr ? a.gather[srow] / a.gather_k : srow];
#pragma unroll
            for (int ob = 0; ob < kBlocks; ob += kPiece) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int b = 0; b < kPiece; ++b) {
                    const int j = kGated ? 2 * ob : ob + b;
                    const int col = done_n0 + block_col<C, kGated>(wn, j);
                    const float* sc = s0 + (col < N ? col : 0);
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        f32x4_t sg = {1.0f, 1.0f, 1.0f, 1.0f};
                        if constexpr (kOut != kOutHalf)
                            sg = *reinterpret_cast<const f32x4_t*>(sc + 8 * g + 4 * lh);
                        f32x4_t v;
                        if constexpr (kGated) {
                            const f32x4_t su = *reinterpret_cast<const f32x4_t*>(s1 + col + 8 * g + 4 * lh);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                v[e] = swiglu(static_cast<float>(acc[i][j][4 * g + e]) * as * sg[e],
                                              static_cast<float>(acc[i][j + 1][4 * g + e]) * as * su[e]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                v[e] = static_cast<float>(acc[i][j][4 * g + e]) * as * sg[e];
                        }
                        if constexpr (kWide)
                            *reinterpret_cast<__attribute__((address_space(3))) f32x4_t*>(
                                stg + lrow * 128 + (((2 * g + lh) ^ (lrow & 7)) << 4)) = v;
                        else
                            *reinterpret_cast<__attribute__((address_space(3))) u32x2_t*>(
                                stg + lrow * 128 + (((4 * b + g) ^ (lrow & 7)) << 4) + 8 * lh) =
                                kOut == kOutHalf ? u32x2_t{pack_half2(v[0], v[1]), pack_half2(v[2], v[3])}
                                                 : u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                    }
                }
                const int col = done_n0 + block_col<C, kGated>(wn, kGated ? 2 * ob : ob);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int row = (lane >> 3) + 8 * m, chunk = lane & 7;
                    const u32x4_t v = read16(stg + row * 128 + ((chunk ^ (row & 7)) << 4));
                    const int grow = done.row_begin + row_block<kWM>(i, wm) + row;
                    if (grow < done.row_end && col < N)
                        *reinterpret_cast<u32x4_t*>(static_cast<unsigned char*>(a.out) +
                                                    (static_cast<int64_t>(grow) * N + col) * (kWide ? 4 : 2) + 16 * chunk) = v;
                }
            }
        }
        // two ahead: the claim goes out after wave 0's last read of its staging area, which holds the word
        if (ahead2 && wave == 0)
            *claimed = claim_after;
    }
}

}  // namespace big

using Mid = Config<2, 4, 2, 2, 128, 3>;        // 128 rows
using Small = Config<1, 8, 2, 1, 128, 3>;      // 64 rows; partial sums only when gated

// Raises the kernel's LDS limit once per device and launches it, one workgroup per CU.
template <auto kernel, int kSmem>
hipError_t launch(const Args& a, hipStream_t s)
{
    static std::atomic<bool> done[64];
    int dev = 0;
    if (hipError_t e = hipGetDevice(&dev); e != hipSuccess)
        return e;
    if (dev >= 64 || !done[dev]) {
        if (hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, kSmem);
            e != hipSuccess)
            return e;
        if (dev < 64)
            done[dev] = true;
    }
    kernel<<<dim3(device_info().cu_count), dim3(kThreads), kSmem, s>>>(a);
    return hipGetLastError();
}

template <bool kGated, int kOut>
hipError_t launch_rows(int bm, const Args& a, hipStream_t s)
{
    if (bm == big::BM) {
        if constexpr (kOut != kOutPartial)
            return launch<&big::grouped_gemm_i8_dma<kGated, kOut>, big::kSmemBytes>(a, s);
    } else if (bm == Mid::BM) {
        return a.groups.tiles == nullptr
                   ? launch<&grouped_gemm_i8<Mid, kGated, kOut, true>, Mid::kSmemBytes + kOwnTableBytes>(a, s)
                   : launch<&grouped_gemm_i8<Mid, kGated, kOut, false>, Mid::kSmemBytes>(a, s);
    } else if constexpr (!kGated || kOut == kOutPartial) {
        return a.groups.tiles == nullptr
                   ? launch<&grouped_gemm_i8<Small, kGated, kOut, true>, Small::kSmemBytes + kOwnTableBytes>(a, s)
                   : launch<&grouped_gemm_i8<Small, kGated, kOut, false>, Small::kSmemBytes>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace i8
}  // namespace

bool int8_supported(int64_t K, int64_t N)
{
    return K > 0 && N > 0 && K % 128 == 0 && N % 128 == 0 && K <= kInt8MaxK;
}

namespace {

// Estimated microseconds of one grouped product with row tiles of `tile` rows and K in `cuts`, for M rows
// spread evenly at random over G groups: the rounds of tasks over the CUs, each as long as its steps (of
// 128 values of K: between `lone` for a workgroup by itself, latency, and `full` with all CUs busy, LDS
// copies or for 256 rows the MFMAs; 2.5 more steps to fill and to finish) or its share of the weights
// at 5.9 TB/s, and a part of the shorter one; a cut product has its sums written and, by one more
// launch, read.  Constants fitted to 1500 timings of whole calls (K x N of 4096 x 14336, 7168 x 2048, 2048 x
// 768, 1024 x 4096, 1 to 32 groups of 1 to 700 rows, tiles of 64, 128 and 256 rows, 1 to 8 cuts), taken with
// a launch for the tile table in each: the plan chosen was within 12% of the best of them, where a choice by
// rows per group alone lost up to 2.8x (7168 x 2048, one group of 200 rows: 73 us with 256-row tiles, 26 us
// with 64 rows and 8 cuts).  Products of less than some 20 us (2048 x 768, 1024 x 4096 with few groups) all
// timed as the host's part of a call, so theirs is the other shapes' estimate; no shape was left out to check.
struct Spread {                                // M rows over the groups that hold some
    double rows, held, per_group;
    Spread(int64_t M, int64_t G)
    {
        rows = static_cast<double>(std::max<int64_t>(M, 1));
        held = std::max(1.0, static_cast<double>(G) * (1.0 - std::pow(1.0 - 1.0 / static_cast<double>(G), rows)));
        per_group = rows / held;
    }
};

double product_cost(const Spread& x, int64_t K, int64_t N, bool gated, int tile, int cuts)
{
    const double lone = tile == 64 ? 0.47 : tile == 128 ? 0.7 : 1.2, full = tile == 64 ? 0.82 : tile == 128 ? 1.3 : 1.9;
    constexpr double cus = 256;                // a host-only rule: the MI355X's, whatever device is current
    const double tasks = x.held * std::ceil(x.per_group / tile) * static_cast<double>(ceil_div(N, gated ? i8::BNB / 2 : i8::BNB)) * cuts;
    const double weights = x.held * static_cast<double>(K) * static_cast<double>(N) * (gated ? 2 : 1) / 5.9e6 / tasks;
    const double steps = std::ceil(static_cast<double>(K / 128) / cuts) + 2.5;
    const auto round = [&](double n) {
        const double step = (lone + (full - lone) * std::min(1.0, n / cus)) *
                            (tile == 256 ? 0.75 + 0.25 * std::min(1.0, x.per_group / tile) : 1.0);
        return std::max(steps * step, n * weights) + 0.21 * std::min(steps * step, n * weights);
    };
    const double whole = std::floor(tasks / cus), rest = tasks - whole * cus;
    double cost = (whole > 0 ? whole * round(cus) : 0.0) + (rest > 0 ? round(rest) : 0.0);
    const double values = x.rows * static_cast<double>(N) * (gated ? 2 : 1);
    if (cuts > 1 || (gated && tile == 64))
        cost += 8.0 * values * cuts / 5.2e6 + (gated ? 0.0 : 7.6);   // int32 sums out and in; h's quantiser runs anyway
    else if (gated)
        cost += 4.0 * values / 5.2e6;                               // float32 h out and in
    return cost;
}

// The best number of cuts for the tile height, and its cost.
double best_cuts(const Spread& x, int64_t K, int64_t N, bool gated, int tile, int& cuts)
{
    cuts = 1;
    double best = product_cost(x, K, N, gated, tile, 1);
    for (int c : {2, 3, 4, 6, 8, 12, 16}) {
        if (tile == 256 || K / 128 < 4 * c)
            break;
        const double cost = product_cost(x, K, N, gated, tile, c);
        if (cost < best) {
            best = cost;
            cuts = c;
        }
    }
    return best;
}

Int8Plan make_plan(int tile, int cuts, bool gated)
{
    return Int8Plan{tile, cuts, cuts > 1 || (gated && tile == 64)};
}

}  // namespace

Int8Plan int8_plan(int64_t M, int64_t G, int64_t K, int64_t N)
{
    const Spread x(M, G);
    Int8Plan p{};
    double best = 0.0;
    for (int tile : {64, 128, 256}) {
        if (tile == 256 && K < 256)
            break;
        int cuts = 1;
        const double cost = best_cuts(x, K, N, false, tile, cuts);
        if (tile == 64 || cost < best) {
            best = cost;
            p = make_plan(tile, cuts, false);
        }
    }
    return p;
}

void int8_ffn_plans(int64_t M, int64_t G, int64_t H, int64_t F, Int8Plan& fc1, Int8Plan& fc2)
{
    const Spread x(M, G);
    double best = 0.0;
    for (int tile : {64, 128, 256}) {
        if (tile == 256 && std::min(H, F) < 256)
            break;
        int c1 = 1, c2 = 1;
        const double cost = best_cuts(x, H, F, true, tile, c1) + best_cuts(x, F, H, false, tile, c2);
        if (tile == 64 || cost < best) {
            best = cost;
            fc1 = make_plan(tile, c1, true);
            fc2 = make_plan(tile, c2, false);
        }
    }
}

bool int8_own_tiles(const Int8Plan& p, int64_t M, int64_t G)
{
    return p.row_tile != i8::big::BM && max_mtiles(M, G, 0, p.row_tile) <= i8::kOwnTiles;
}

bool int8_tasks_fit(const Int8Plan& p, int64_t M, int64_t G, int64_t N, bool gated)
{
    // the loops over tasks step by the grid and decode_task multiplies back: kept well below 2^31
    return max_mtiles(M, G, 0, p.row_tile) * ceil_div(N, gated ? i8::BNB / 2 : i8::BNB) * p.splits < (int64_t{1} << 30);
}

hipError_t launch_gemm_i8(const Int8Plan& p, const int8_t* A, const float* a_scale, const int8_t* w0,
                          const float* s0, const int8_t* w1, const float* s1, void* out, int out_dtype,
                          int64_t M, int64_t K, int64_t N, const Int8Groups& groups,
                          const int32_t* gather, int gather_k, int32_t* task_ctr, hipStream_t s)
{
    i8::Args a{};
    a.A = reinterpret_cast<const uint8_t*>(A);
    a.a_scale = a_scale;
    a.B0 = reinterpret_cast<const uint8_t*>(w0);
    a.B1 = reinterpret_cast<const uint8_t*>(w1);
    a.s0 = s0;
    a.s1 = s1;
    a.out = out;
    a.groups = groups;
    a.gather = gather;
    a.gather_k = gather_k;
    a.task_ctr = task_ctr;
    a.K = static_cast<int>(K);
    a.N = static_cast<int>(N);
    a.splits = p.splits;
    a.M = M;
    a.unit = int8_half_unit(K);
    const bool gated = w1 != nullptr;
    if (p.partial)
        return gated ? i8::launch_rows<true, i8::kOutPartial>(p.row_tile, a, s)
                     : i8::launch_rows<false, i8::kOutPartial>(p.row_tile, a, s);
    if (gated)
        return i8::launch_rows<true, i8::kOutF32>(p.row_tile, a, s);
    if (out_dtype == kInt8HalfSums)
        return i8::launch_rows<false, i8::kOutHalf>(p.row_tile, a, s);
    return out_dtype == MOE_F32 ? i8::launch_rows<false, i8::kOutF32>(p.row_tile, a, s)
                                : i8::launch_rows<false, i8::kOutBf16>(p.row_tile, a, s);
}

}  // namespace moe
