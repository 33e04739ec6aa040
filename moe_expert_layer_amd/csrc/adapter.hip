// Low-rank adapters of many requests beside a shared projection (moe_adapter_add):
//   v[t] = scale[a] x[t] A[a],  out[t] = base[t] + v[t] B[a],  a = ids[t].
//
// Memory is what bounds it: x and base once, out once, each used adapter's A and B once; the products are R operations a
// byte.  Two ways:
//   - few rows (row_kernel): one launch, a workgroup per (row, run of output columns).  Each computes its row's v for
//     itself, which reads the adapter's A again from the L2 but saves a launch and a pass through memory;
//   - many rows: the rows are sorted by adapter into tiles of up to 64 (plan_kernel, one workgroup), then v and v B run
//     on the matrix cores, tile by tile (shrink_kernel, expand_kernel).  x goes from memory to the MFMA's registers, the
//     adapter's matrices through LDS; K is cut so that there are workgroups enough, the cuts' float32 sums joined when
//     the second product reads them.  v enters that product as two bfloat16 planes (16 bits) for bfloat16 tensors, as
//     three for float32 ones.
// A row's result does not depend on the tile that it falls into, so neither the order in which the plan's counters hand
// out places nor other rows change it.
#include <algorithm>

#include "dropout.h"
#include "planes.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;                 // rows per tile

template <class T>
__device__ __forceinline__ float to_float(T v)
{
    if constexpr (sizeof(T) == 2)
        return bf16_to_f32(v);
    else
        return v;
}

struct Args {
    const void *base, *x, *a, *b;
    void* out;
    const int32_t *ids, *ranks;
    const float* scale;
    int T, K, N, L, R;
    bool vec_k, vec_r, vec_n;             // rows of x, of A, of B / base / out are whole, aligned 16-byte chunks
};

__device__ __forceinline__ int rank_of(const Args& g, int a) { return g.ranks == nullptr ? g.R : min(max(g.ranks[a], 0), g.R); }

// ------------------------------------------------------------------------------------------------ few rows

// Workgroup (t, c): row t, output columns [c cols, (c + 1) cols).  Threads take (k, 8 columns of A) and add over k, then
// (r, 8 columns of B) and add over r, both joined through LDS in a fixed order.
template <class T>
__global__ __launch_bounds__(kThreads) void row_kernel(Args g, int cols)
{
    constexpr int kJoin = 32;                              // partial sums of a column that one thread adds in a row
    __shared__ float part[kThreads * 8];
    __shared__ float v[kMaxRank];
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x;
    const T* const base = static_cast<const T*>(g.base) + t * g.N;
    T* const out = static_cast<T*>(g.out) + t * g.N;
    const int n0 = blockIdx.y * cols, n1 = min(n0 + cols, g.N);
    const int a = g.ids[t];
    const bool on = a >= 0 && a < g.L;
    const int rank = on ? rank_of(g, a) : 0;
    if (rank == 0) {                                       // uniform: the row is copied
        if (g.base != g.out)
            for (int n = n0 + 8 * tid; n < n1; n += 8 * kThreads) {
                float w[8];
                load8(w, base + n, n1 - n, g.vec_n);
                store8(out + n, w, n1 - n, g.vec_n);
            }
        return;
    }
    {
        const T* const x = static_cast<const T*>(g.x) + t * g.K;
        const T* const A = static_cast<const T*>(g.a) + static_cast<int64_t>(a) * g.K * g.R;
        const int chunks = (rank + 7) / 8, lanes = kThreads / chunks;   // threads per column chunk
        const int c = tid % chunks, kk = tid / chunks;
        float sum[8] = {};
        if (kk < lanes) {
#pragma unroll 8
            for (int k = kk; k < g.K; k += lanes) {
                float w[8];
                load8(w, A + static_cast<int64_t>(k) * g.R + 8 * c, rank - 8 * c, g.vec_r);
                const float xk = to_float(x[k]);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sum[i] = fmaf(xk, w[i], sum[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            part[i * kThreads + tid] = sum[i];
        // column r = 8 c + i: parts part[i][c + chunks kk]; halve them until a thread can add them in a row
        int left = lanes;
        while (left > kJoin) {
            __syncthreads();
            const int half = (left + 1) / 2;
            if (kk < left - half)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    part[i * kThreads + tid] += part[i * kThreads + tid + half * chunks];
            left = half;
        }
        __syncthreads();
        if (tid < rank) {
            float s = 0.0f;
            for (int q = 0; q < left; ++q)
                s += part[(tid % 8) * kThreads + tid / 8 + chunks * q];
            v[tid] = g.scale == nullptr ? s : s * g.scale[a];
        }
        __syncthreads();
    }
    const T* const B = static_cast<const T*>(g.b) + static_cast<int64_t>(a) * g.R * g.N;
    // threads per run of 8 output columns: as many as the run of columns leaves, at most the rank
    const int runs = min(kThreads, (n1 - n0 + 7) / 8), lanes = max(1, min(rank, kThreads / runs));
    for (int first = n0; first < n1; first += 8 * runs) {      // the same number of passes for every thread
        const int q = tid % runs, rr = tid / runs, n = first + 8 * q;
        float sum[8] = {};
        if (rr < lanes && n < n1)
#pragma unroll 4
            for (int r = rr; r < rank; r += lanes) {
                float w[8];
                load8(w, B + static_cast<int64_t>(r) * g.N + n, n1 - n, g.vec_n);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sum[i] = fmaf(v[r], w[i], sum[i]);
            }
        if (lanes > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i)
                part[i * kThreads + tid] = sum[i];
            __syncthreads();
            if (rr == 0)
                for (int p = 1; p < lanes; ++p)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sum[i] += part[i * kThreads + tid + p * runs];
        }
        if (rr == 0 && n < n1) {
            float w[8];
            load8(w, base + n, n1 - n, g.vec_n);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] += sum[i];
            store8(out + n, w, n1 - n, g.vec_n);
        }
    }
}

// ------------------------------------------------------------------------------------------------ many rows

struct Tile {
    int adapter, begin, end;              // sorted rows [begin, end); adapter L: rows without one
    int pad;
};

constexpr int kPlanThreads = 1024;
static_assert(kMaxAdapters < kPlanThreads, "one bin a thread, and one for rows without an adapter");

// perm: the rows by adapter (those without one last); tiles, and their number in count[0].
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(const int32_t* __restrict__ ids, int T, int L,
                                                            int32_t* __restrict__ perm, Tile* __restrict__ tiles,
                                                            int32_t* __restrict__ count)
{
    __shared__ int rows[kPlanThreads + 1], tile0[kPlanThreads + 1], place[kPlanThreads], sums[2][kPlanThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    place[tid] = 0;
    __syncthreads();
    for (uint32_t t = tid; t < static_cast<uint32_t>(T); t += kPlanThreads) {   // T + 1024 may pass 2^31
        const int a = ids[t];
        atomicAdd(&place[a >= 0 && a < L ? a : L], 1);
    }
    __syncthreads();
    // exclusive sums over the bins of rows and of tiles
    const int n = place[tid], nt = (n + kTile - 1) / kTile;
    int s0 = n, s1 = nt;
    for (int d = 1; d < 64; d *= 2) {
        const int u0 = __shfl_up(s0, d), u1 = __shfl_up(s1, d);
        if (lane >= d) {
            s0 += u0;
            s1 += u1;
        }
    }
    if (lane == 63) {
        sums[0][wave] = s0;
        sums[1][wave] = s1;
    }
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        s0 += sums[0][w];
        s1 += sums[1][w];
    }
    rows[tid + 1] = s0;
    tile0[tid + 1] = s1;
    if (tid == 0)
        rows[0] = tile0[0] = 0;
    place[tid] = s0 - n;
    __syncthreads();
    for (uint32_t t = tid; t < static_cast<uint32_t>(T); t += kPlanThreads) {   // T + 1024 may pass 2^31
        const int a = ids[t];
        perm[atomicAdd(&place[a >= 0 && a < L ? a : L], 1)] = static_cast<int32_t>(t);
    }
    const int total = tile0[L + 1];
    if (tid == 0)
        count[0] = total;
    for (int i = tid; i < total; i += kPlanThreads) {
        int lo = 0, hi = L;                               // the bin that holds tile i
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (tile0[mid] <= i)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int begin = rows[lo] + (i - tile0[lo]) * kTile;
        tiles[i] = Tile{lo, begin, min(begin + kTile, rows[lo + 1]), 0};
    }
}

struct TileArgs {
    const Tile* tiles;
    const int32_t *count, *perm;
    float* v;                             // partial sums [splits, T, 32 kRB] in sorted order
    int splits, steps;                    // cuts of K, K steps of all of them
};

// The sums of one MFMA step: all products of planes that count.
template <int PA, int PB>
__device__ __forceinline__ f32x16_t mfma_planes(const bf16x8_t (&w)[PB], const bf16x8_t (&r)[PA], f32x16_t acc)
{
    if constexpr (PA == 3 && PB == 3) {
#pragma unroll
        for (int i = 0; i < 6; ++i)
            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[kPlanePairs[i][1]], r[kPlanePairs[i][0]], acc, 0, 0, 0);
    } else {
        static_assert(PB == 1, "bfloat16 weights");
#pragma unroll
        for (int i = PA - 1; i >= 0; --i)
            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[0], r[i], acc, 0, 0, 0);
    }
    return acc;
}

// v of a tile's rows over one cut of K.  Waves: 2 row halves of 32 x 2 halves of each K step; kRB column blocks of 32.
template <class T, int kRB>
__global__ __launch_bounds__(kThreads) void shrink_kernel(Args g, TileArgs p)
{
    constexpr int P = Raw8<T>::kPlanes;
    constexpr int kStep = kRB == 4 ? 64 : 128, kGroups = kStep / 32;       // MFMA steps of 16 k per wave and K step
    constexpr int kCols = 32 * kRB, kRow = 2 * kCols + 16;                 // bytes of one k row in LDS
    constexpr int kPlane = kStep * kRow, kLoads = kStep * kCols / 8 / kThreads;
    __shared__ __attribute__((aligned(16))) unsigned char smem[P * kPlane > 64 * kCols * 4 ? P * kPlane : 64 * kCols * 4];
    if (static_cast<int>(blockIdx.x) >= p.count[0])
        return;
    const Tile tile = p.tiles[blockIdx.x];
    if (tile.adapter >= g.L)
        return;
    const int rank = rank_of(g, tile.adapter);
    if (rank == 0)
        return;
    const int split = blockIdx.y;
    const int step0 = static_cast<int>(static_cast<int64_t>(p.steps) * split / p.splits);
    const int step1 = static_cast<int>(static_cast<int64_t>(p.steps) * (split + 1) / p.splits);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wr = wave >> 1, wk = wave & 1;
    const int n = tile.end - tile.begin;
    const bool busy = 32 * wr < n;                        // this wave has rows
    const int row = p.perm[tile.begin + min(32 * wr + (lane & 31), n - 1)];
    const T* const x = static_cast<const T*>(g.x) + static_cast<int64_t>(row) * g.K;
    const T* const A = static_cast<const T*>(g.a) + static_cast<int64_t>(tile.adapter) * g.K * g.R;
    const uint32_t lds = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned char*)(smem)));

    Raw8<T> xr[kGroups], ar[kLoads];
    const auto fetch = [&](int step) {
        const int k0 = step * kStep;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int c = (tid + i * kThreads) % (kCols / 8), k = k0 + (tid + i * kThreads) / (kCols / 8);
            ar[i] = load_raw(A + static_cast<int64_t>(k) * g.R + 8 * c, k < g.K ? rank - 8 * c : 0, g.vec_r);
        }
        if (busy)
#pragma unroll
            for (int s = 0; s < kGroups; ++s) {
                const int k = k0 + (kStep / 2) * wk + 16 * s + 8 * (lane >> 5);
                xr[s] = load_raw(x + k, g.K - k, g.vec_k);
            }
    };
    f32x16_t acc[kRB];
#pragma unroll
    for (int j = 0; j < kRB; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e)
            acc[j][e] = 0.0f;
    if (step0 < step1)
        fetch(step0);
    for (int step = step0; step < step1; ++step) {
        __syncthreads();                                  // the stage of the step before is read
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = tid + i * kThreads;
            u32x4_t pl[P];
            ar[i].planes(pl);
#pragma unroll
            for (int q = 0; q < P; ++q)
                *reinterpret_cast<u32x4_t*>(smem + q * kPlane + (at / (kCols / 8)) * kRow + 16 * (at % (kCols / 8))) = pl[q];
        }
        u32x4_t xp[kGroups][P];
#pragma unroll
        for (int s = 0; s < kGroups; ++s)
            xr[s].planes(xp[s]);
        __syncthreads();
        if (step + 1 < step1)
            fetch(step + 1);
        if (busy)
#pragma unroll
            for (int s = 0; s < kGroups; ++s) {
                bf16x8_t r[P];
#pragma unroll
                for (int q = 0; q < P; ++q)
                    r[q] = __builtin_bit_cast(bf16x8_t, xp[s][q]);
#pragma unroll
                for (int j = 0; j < kRB; ++j) {
                    bf16x8_t w[P];
#pragma unroll
                    for (int q = 0; q < P; ++q)
                        w[q] = read_tr(lds + q * kPlane + ((kStep / 2) * wk + 16 * s) * kRow + 64 * j + tr_offset(lane, kRow), kRow);
                    acc[j] = mfma_planes<P, P>(w, r, acc[j]);
                }
            }
    }
    // the two K halves join through LDS
    __syncthreads();
    float* const join = reinterpret_cast<float*>(smem) + (32 * wr + (lane & 31)) * kCols + 8 * (lane >> 5);
    if (busy && wk == 1)
#pragma unroll
        for (int j = 0; j < kRB; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float w[8];
                run8(acc[j], h, w);
                store8(join + 32 * j + 16 * h, w, 8, true);
            }
    __syncthreads();
    if (busy && wk == 0) {
        const float f = g.scale == nullptr ? 1.0f : g.scale[tile.adapter];
        float* const v = p.v + (static_cast<int64_t>(split) * g.T + tile.begin + 32 * wr + (lane & 31)) * kCols + 8 * (lane >> 5);
#pragma unroll
        for (int j = 0; j < kRB; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float w[8], u[8];
                run8(acc[j], h, w);
                load8(u, join + 32 * j + 16 * h, 8, true);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i] = (w[i] + u[i]) * f;
                if (32 * wr + (lane & 31) < n)
                    store8(v + 32 * j + 16 * h, w, 8, true);
            }
    }
}

// out of a tile's rows over `cols` columns (a multiple of 128).  Waves: 2 row halves x 2 halves of 128 columns.
template <class T, int kRB>
__global__ __launch_bounds__(kThreads) void expand_kernel(Args g, TileArgs p, int cols)
{
    constexpr int PB = Raw8<T>::kPlanes, PV = PB == 1 ? 2 : 3;
    constexpr int kR = 32 * kRB, kRow = 2 * 128 + 16, kPlane = kR * kRow, kLoads = kR * 16 / kThreads;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    if (static_cast<int>(blockIdx.x) >= p.count[0])
        return;
    const Tile tile = p.tiles[blockIdx.x];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n0 = blockIdx.y * cols, n1 = min(n0 + cols, g.N), n = tile.end - tile.begin;
    const int rank = tile.adapter < g.L ? rank_of(g, tile.adapter) : 0;
    if (rank == 0) {                                      // the rows are copied, a wave each
        if (g.base != g.out)
            for (int r = wave; r < n; r += kThreads / 64) {
                const int64_t at = static_cast<int64_t>(p.perm[tile.begin + r]) * g.N;
                for (int c = n0 + 8 * lane; c < n1; c += 512) {
                    float w[8];
                    load8(w, static_cast<const T*>(g.base) + at + c, n1 - c, g.vec_n);
                    store8(static_cast<T*>(g.out) + at + c, w, n1 - c, g.vec_n);
                }
            }
        return;
    }
    const int wr = wave >> 1, wc = wave & 1;
    const int mine = 32 * wr + (lane & 31), safe = min(mine, n - 1);
    const bool busy = 32 * wr < n, real = mine < n;
    const int64_t row = static_cast<int64_t>(p.perm[tile.begin + safe]) * g.N;
    const T* const B = static_cast<const T*>(g.b) + static_cast<int64_t>(tile.adapter) * g.R * g.N;
    const uint32_t lds = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned char*)(smem)));

    Raw8<T> br[kLoads], base[4];
    const auto fetch = [&](int c0) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = (tid + i * kThreads) / 16, c = c0 + 8 * (tid % 16);
            br[i] = load_raw(B + static_cast<int64_t>(r) * g.N + c, r < rank ? n1 - c : 0, g.vec_n);
        }
        if (busy)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = c0 + 64 * wc + 16 * q + 8 * (lane >> 5);
                base[q] = load_raw(static_cast<const T*>(g.base) + row + c, real ? n1 - c : 0, g.vec_n);
            }
    };
    fetch(n0);
    // v of this lane's row, 8 of every 16 columns, as planes
    bf16x8_t v[2 * kRB][PV];
#pragma unroll
    for (int s = 0; s < 2 * kRB; ++s) {
        float sum[8] = {};
        for (int q = 0; q < p.splits; ++q) {
            float w[8];
            load8(w, p.v + (static_cast<int64_t>(q) * g.T + tile.begin + safe) * kR + 16 * s + 8 * (lane >> 5), 8, true);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum[i] += w[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (16 * s + 8 * (lane >> 5) + i >= rank)
                sum[i] = 0.0f;
        u32x4_t pl[PV];
        split8<PV>(sum, pl);
#pragma unroll
        for (int q = 0; q < PV; ++q)
            v[s][q] = __builtin_bit_cast(bf16x8_t, pl[q]);
    }
    for (int c0 = n0; c0 < n1; c0 += 128) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            u32x4_t pl[PB];
            br[i].planes(pl);
#pragma unroll
            for (int q = 0; q < PB; ++q)
                *reinterpret_cast<u32x4_t*>(smem + q * kPlane + ((tid + i * kThreads) / 16) * kRow + 16 * (tid % 16)) = pl[q];
        }
        Raw8<T> now[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            now[q] = base[q];
        __syncthreads();
        if (c0 + 128 < n1)
            fetch(c0 + 128);
        if (!busy)
            continue;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            f32x16_t acc;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc[e] = 0.0f;
#pragma unroll
            for (int s = 0; s < 2 * kRB; ++s) {
                bf16x8_t w[PB];
#pragma unroll
                for (int q = 0; q < PB; ++q)
                    w[q] = read_tr(lds + q * kPlane + 16 * s * kRow + 2 * (64 * wc + 32 * j) + tr_offset(lane, kRow), kRow);
                acc = mfma_planes<PV, PB>(w, v[s], acc);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float w[8], u[8];
                run8(acc, h, w);
                now[2 * j + h].values(u);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i] += u[i];
                const int c = c0 + 64 * wc + 32 * j + 16 * h + 8 * (lane >> 5);
                if (real && c < n1)
                    store8(static_cast<T*>(g.out) + row + c, w, n1 - c, g.vec_n);
            }
        }
    }
}

// ------------------------------------------------------------------------------------------------ the host's side

// How a call runs.
struct Plan {
    bool rows;                // row_kernel
    int cols;                 // output columns per workgroup
    int blocks;               // column blocks of 32 that hold the rank (1, 2 or 4)
    int splits, steps;
    int64_t max_tiles;
};

Plan plan(const moe_adapter& p)
{
    Plan q{};
    const int64_t size = p.dtype == MOE_F32 ? 4 : 2;
    q.rows = p.K * p.R * size <= (int64_t{1} << 20) && p.T * (p.K + p.N) * p.R * size <= (int64_t{384} << 20);
    if (q.rows) {
        // about 256 workgroups, 64 columns at least
        const int64_t per_row = std::clamp<int64_t>(ceil_div(256, std::max<int64_t>(p.T, 1)), 1, ceil_div(p.N, 64));
        q.cols = static_cast<int>(ceil_div(ceil_div(p.N, per_row), 8) * 8);
        return q;
    }
    q.blocks = p.R <= 32 ? 1 : p.R <= 64 ? 2 : 4;
    q.steps = static_cast<int>(ceil_div(p.K, q.blocks == 4 ? 64 : 128));
    q.max_tiles = ceil_div(p.T, kTile) + std::min(p.T, p.L + 1);
    const int64_t tiles = ceil_div(p.T, kTile);
    q.splits = static_cast<int>(std::clamp<int64_t>(ceil_div(512, tiles), 1, std::clamp<int64_t>(q.steps / 4, 1, 16)));
    const int64_t per_tile = std::clamp<int64_t>(ceil_div(1024, tiles), 1, ceil_div(p.N, 128));
    q.cols = static_cast<int>(ceil_div(ceil_div(p.N, per_tile), 128) * 128);
    return q;
}

template <class T, int kRB>
hipError_t launch_tiles(const Args& g, const TileArgs& t, const Plan& q, hipStream_t s)
{
    constexpr int kExpandLds = Raw8<T>::kPlanes * 32 * kRB * (2 * 128 + 16);
    if (kExpandLds > 65536)
        if (hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&expand_kernel<T, kRB>),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, kExpandLds); e != hipSuccess)
            return e;
    const unsigned tiles = static_cast<unsigned>(q.max_tiles);
    shrink_kernel<T, kRB><<<dim3(tiles, q.splits), kThreads, 0, s>>>(g, t);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    expand_kernel<T, kRB><<<dim3(tiles, static_cast<unsigned>(ceil_div(g.N, q.cols))), kThreads, kExpandLds, s>>>(g, t, q.cols);
    return hipGetLastError();
}

template <class T>
hipError_t launch(const moe_adapter& p, const Args& g, unsigned char* ws, hipStream_t s)
{
    const Plan q = plan(p);
    if (q.rows) {
        row_kernel<T><<<dim3(static_cast<unsigned>(p.T), static_cast<unsigned>(ceil_div(p.N, q.cols))), kThreads, 0, s>>>(g, q.cols);
        return hipGetLastError();
    }
    const AdapterLayout L = adapter_layout(p);
    int32_t* const perm = reinterpret_cast<int32_t*>(ws + L.perm);
    Tile* const tiles = reinterpret_cast<Tile*>(ws + L.tiles);
    int32_t* const count = reinterpret_cast<int32_t*>(ws + L.count);
    plan_kernel<<<1, kPlanThreads, 0, s>>>(g.ids, g.T, g.L, perm, tiles, count);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    const TileArgs t{tiles, count, perm, reinterpret_cast<float*>(ws + L.v), q.splits, q.steps};
    return q.blocks == 1 ? launch_tiles<T, 1>(g, t, q, s) : q.blocks == 2 ? launch_tiles<T, 2>(g, t, q, s)
                                                                         : launch_tiles<T, 4>(g, t, q, s);
}

}  // namespace

AdapterLayout adapter_layout(const moe_adapter& p)
{
    AdapterLayout L;
    const Plan q = plan(p);
    if (q.rows)
        return L;
    size_t off = 0;
    const auto take = [&](size_t& at, size_t bytes) {
        at = off;
        off = align_up(off + bytes);
    };
    take(L.count, sizeof(int32_t));
    take(L.perm, static_cast<size_t>(p.T) * sizeof(int32_t));
    take(L.tiles, static_cast<size_t>(q.max_tiles) * sizeof(Tile));
    take(L.v, static_cast<size_t>(q.splits) * p.T * 32 * q.blocks * sizeof(float));
    L.total = off;
    return L;
}

hipError_t launch_adapter(const moe_adapter& p, const void* base, const void* x, const void* a, const void* b,
                          const int32_t* ids, const float* scale, const int32_t* ranks, void* out, void* workspace,
                          hipStream_t s)
{
    const auto aligned = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
    const int64_t size = p.dtype == MOE_F32 ? 4 : 2;
    Args g{base, x, a, b, out, ids, ranks, scale, static_cast<int>(p.T), static_cast<int>(p.K), static_cast<int>(p.N),
           static_cast<int>(p.L), static_cast<int>(p.R), false, false, false};
    g.vec_k = p.K * size % 16 == 0 && aligned(x);
    g.vec_r = p.R * size % 16 == 0 && aligned(a);
    g.vec_n = p.N * size % 16 == 0 && aligned(b) && aligned(base) && aligned(out);
    unsigned char* const ws = static_cast<unsigned char*>(workspace);
    return p.dtype == MOE_F32 ? launch<float>(p, g, ws, s) : launch<uint16_t>(p, g, ws, s);
}

}  // namespace moe
