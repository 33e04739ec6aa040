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
};

__device__ __forceinline__ int rank_of(const Args& g, int a) { return g.ranks == nullptr ? g.R : min(max(g.ranks[a], 0), g.R); }

// ------------------------------------------------------------------------------------------------ few rows

constexpr int kRowThreads = 1024;         // 16 waves: a CU has one or two of these workgroups, and 128 KiB in flight
constexpr int kRowWaves = kRowThreads / 64;

// Workgroup (t, c): row t, output columns [c cols, (c + 1) cols).  Threads take (k, 8 columns of A) and add over k, then
// (r, 8 columns of B) and add over r; both are joined in a fixed order, within the wave and then through LDS.  Loads go
// out in batches, and what does not wait for v (the first rows of B, base) at the start.
template <class T, bool kWhole>
__global__ __launch_bounds__(kRowThreads) void row_kernel(Args g, int cols)
{
    constexpr int kBatch = 8;
    __shared__ float part[kRowThreads * 8];
    __shared__ float v[kMaxRank];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t t = blockIdx.x;
    const T* const base = static_cast<const T*>(g.base) + t * g.N;
    T* const out = static_cast<T*>(g.out) + t * g.N;
    const int n0 = blockIdx.y * cols, n1 = min(n0 + cols, g.N);
    const int a = g.ids[t];
    const bool on = a >= 0 && a < g.L;
    const int rank = on ? rank_of(g, a) : 0;
    if (rank == 0) {                                       // uniform: the row is copied
        if (g.base != g.out)
            for (int n = n0 + 8 * tid; n < n1; n += 8 * kRowThreads) {
                float w[8];
                load8(w, base + n, n1 - n);
                store8(out + n, w, n1 - n);
            }
        return;
    }
    const float scale = g.scale == nullptr ? 1.0f : g.scale[a];
    // threads per run of 8 output columns: as many as the run of columns leaves, at most the rank
    const T* const B = static_cast<const T*>(g.b) + static_cast<int64_t>(a) * g.R * g.N;
    const int runs = min(kRowThreads, (n1 - n0 + 7) / 8), lanes = max(1, min(rank, kRowThreads / runs));
    const int q = tid % runs, rr = tid / runs;
    const int left0 = n1 - n0 - 8 * q;
    Raw8<T> b0 = load_raw<kWhole>(B + static_cast<int64_t>(rr) * g.N + n0 + 8 * q, rr < lanes ? left0 : 0);
    Raw8<T> base0 = load_raw<kWhole>(base + n0 + 8 * q, rr == 0 ? left0 : 0);
    {
        const T* const x = static_cast<const T*>(g.x) + t * g.K;
        const T* const A = static_cast<const T*>(g.a) + static_cast<int64_t>(a) * g.K * g.R;
        // a power of two of column chunks, so that the lanes of one chunk are whole strides of the wave
        const int bits = rank <= 8 ? 0 : 32 - __clz((rank - 1) >> 3), chunks = 1 << bits;
        const int c = tid & (chunks - 1), stride = kRowThreads >> bits;
        const int width = 8 * c < rank ? g.R - 8 * c : 0;
        float sum[8] = {};
        for (int k0 = tid >> bits; k0 < g.K; k0 += kBatch * stride) {
            Raw8<T> w[kBatch];
            T xk[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int k = k0 + i * stride;
                w[i] = load_raw<kWhole>(A + static_cast<int64_t>(k) * g.R + 8 * c, k < g.K ? width : 0);
                xk[i] = x[min(k, g.K - 1)];
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                float f[8];
                w[i].values(f);
                const float m = k0 + i * stride < g.K ? to_float(xk[i]) : 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum[e] = fmaf(m, f[e], sum[e]);
            }
        }
        for (int d = 32; d >= chunks; d >>= 1)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum[i] += __shfl_xor(sum[i], d);
        if (lane < chunks)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                part[wave * kMaxRank + 8 * lane + i] = sum[i];
        __syncthreads();
        if (tid < rank) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kRowWaves; ++w)
                s += part[w * kMaxRank + tid];
            v[tid] = s * scale;
        }
        __syncthreads();
    }
    for (int first = n0; first < n1; first += 8 * runs) {      // the same number of passes for every thread
        const int n = first + 8 * q;
        float sum[8] = {};
        if (rr < lanes && n < n1) {
            if (first != n0)
                b0 = load_raw<kWhole>(B + static_cast<int64_t>(rr) * g.N + n, n1 - n);
            for (int r0 = rr + lanes; ; r0 += kBatch * lanes) {
                Raw8<T> w[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    w[i] = load_raw<kWhole>(B + static_cast<int64_t>(r0 + i * lanes) * g.N + n, r0 + i * lanes < rank ? n1 - n : 0);
                float f[8];
                if (r0 == rr + lanes) {                        // the row that was loaded first
                    b0.values(f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        sum[e] = v[rr] * f[e];
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    w[i].values(f);
                    const float m = r0 + i * lanes < rank ? v[r0 + i * lanes] : 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        sum[e] = fmaf(m, f[e], sum[e]);
                }
                if (r0 + kBatch * lanes >= rank)
                    break;
            }
        }
        if (lanes > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i)
                part[i * kRowThreads + tid] = sum[i];
            __syncthreads();
            if (rr == 0)
                for (int p = 1; p < lanes; ++p)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sum[i] += part[i * kRowThreads + tid + p * runs];
        }
        if (rr == 0 && n < n1) {
            if (first != n0)
                base0 = load_raw<kWhole>(base + n, n1 - n);
            float f[8];
            base0.values(f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum[i] += f[i];
            store8(out + n, sum, n1 - n);
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
    // Adds the lanes' rows to their bins' counters, returns each lane's place.  Rows of one request lie side by side:
    // a wave of one bin adds once (64 additions to one counter would take turns).
    const auto add = [&](uint32_t t) {
        const int a = ids[t], bin = a >= 0 && a < L ? a : L;
        if (__all(bin == __builtin_amdgcn_readfirstlane(bin))) {
            const uint64_t active = __ballot(1);
            const int before = __popcll(active & ((uint64_t{1} << lane) - 1));
            int first = 0;
            if (before == 0)
                first = atomicAdd(&place[bin], __popcll(active));
            return __builtin_amdgcn_readfirstlane(first) + before;
        }
        return atomicAdd(&place[bin], 1);
    };
    place[tid] = 0;
    __syncthreads();
    for (uint32_t t = tid; t < static_cast<uint32_t>(T); t += kPlanThreads)   // T + 1024 may pass 2^31
        add(t);
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
    for (uint32_t t = tid; t < static_cast<uint32_t>(T); t += kPlanThreads)
        perm[add(t)] = static_cast<int32_t>(t);
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
template <class T, int kRB, bool kWhole>
__global__ __launch_bounds__(kThreads) void shrink_kernel(Args g, TileArgs p)
{
    constexpr int P = kPlanesOf<T>;
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
            ar[i] = load_raw<kWhole>(A + static_cast<int64_t>(k) * g.R + 8 * c, k < g.K ? g.R - 8 * c : 0);
        }
    };
    const auto fetch_x = [&](int step, int s) {
        const int k = step * kStep + (kStep / 2) * wk + 16 * s + 8 * (lane >> 5);
        xr[s] = load_raw<kWhole>(x + k, busy ? g.K - k : 0);
    };
    f32x16_t acc[kRB];
#pragma unroll
    for (int j = 0; j < kRB; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e)
            acc[j][e] = 0.0f;
    if (step0 < step1) {
        fetch(step0);
#pragma unroll
        for (int s = 0; s < kGroups; ++s)
            fetch_x(step0, s);
    }
    for (int step = step0; step < step1; ++step) {
        __syncthreads();                                  // the stage of the step before is read
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = tid + i * kThreads;
            u32x4_t pl[P];
            planes8(ar[i], pl);
#pragma unroll
            for (int q = 0; q < P; ++q)
                *reinterpret_cast<u32x4_t*>(smem + q * kPlane + (at / (kCols / 8)) * kRow + 16 * (at % (kCols / 8))) = pl[q];
        }
        __syncthreads();
        if (step + 1 < step1)
            fetch(step + 1);
        if (busy)
#pragma unroll
            for (int s = 0; s < kGroups; ++s) {
                u32x4_t xp[P];
                planes8(xr[s], xp);
                bf16x8_t r[P];
#pragma unroll
                for (int q = 0; q < P; ++q)
                    r[q] = __builtin_bit_cast(bf16x8_t, xp[q]);
                if (step + 1 < step1)
                    fetch_x(step + 1, s);
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
                store8(join + 32 * j + 16 * h, w, 8);
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
                load8(u, join + 32 * j + 16 * h, 8);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i] = (w[i] + u[i]) * f;
                if (32 * wr + (lane & 31) < n)
                    store8(v + 32 * j + 16 * h, w, 8);
            }
    }
}

// out of a tile's rows over `cols` columns (a multiple of 128).  Waves: 2 row halves x 2 halves of 128 columns.
template <class T, int kRB, bool kWhole>
__global__ __launch_bounds__(kThreads) void expand_kernel(Args g, TileArgs p, int cols)
{
    constexpr int PB = kPlanesOf<T>, PV = PB == 1 ? 2 : 3;
    constexpr int kR = 32 * kRB, kRow = 2 * 128 + 16, kPlane = kR * kRow, kLoads = kR * 16 / kThreads;
    constexpr int kVRow = 2 * kR + 16, kVPlane = kTile * kVRow;        // v's planes, after B's
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
                    load8(w, static_cast<const T*>(g.base) + at + c, n1 - c);
                    store8(static_cast<T*>(g.out) + at + c, w, n1 - c);
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
            br[i] = load_raw<kWhole>(B + static_cast<int64_t>(r) * g.N + c, r < rank ? n1 - c : 0);
        }
        if (busy)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = c0 + 64 * wc + 16 * q + 8 * (lane >> 5);
                base[q] = load_raw<kWhole>(static_cast<const T*>(g.base) + row + c, real ? n1 - c : 0);
            }
    };
    fetch(n0);
    // v of the tile's rows as planes, each thread 8 columns of a row at a time
#pragma unroll
    for (int i = 0; i < kTile * kR / 8 / kThreads; ++i) {
        const int r = (tid + i * kThreads) / (kR / 8), c = 8 * ((tid + i * kThreads) % (kR / 8));
        const float* const v = p.v + (static_cast<int64_t>(tile.begin) + min(r, n - 1)) * kR + c;
        float sum[8] = {};
#pragma unroll 4
        for (int q = 0; q < p.splits; ++q) {
            float w[8];
            load8(w, v + static_cast<int64_t>(q) * g.T * kR, 8);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum[e] += w[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e >= rank)
                sum[e] = 0.0f;
        u32x4_t pl[PV];
        split8<PV>(sum, pl);
#pragma unroll
        for (int q = 0; q < PV; ++q)
            *reinterpret_cast<u32x4_t*>(smem + PB * kPlane + q * kVPlane + r * kVRow + 2 * c) = pl[q];
    }
    const unsigned char* const mine_v = smem + PB * kPlane + (32 * wr + (lane & 31)) * kVRow + 16 * (lane >> 5);
    for (int c0 = n0; c0 < n1; c0 += 128) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            u32x4_t pl[PB];
            planes8(br[i], pl);
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
                bf16x8_t w[PB], v[PV];
#pragma unroll
                for (int q = 0; q < PV; ++q)
                    v[q] = *reinterpret_cast<const bf16x8_t*>(mine_v + q * kVPlane + 32 * s);
#pragma unroll
                for (int q = 0; q < PB; ++q)
                    w[q] = read_tr(lds + q * kPlane + 16 * s * kRow + 2 * (64 * wc + 32 * j) + tr_offset(lane, kRow), kRow);
                acc = mfma_planes<PV, PB>(w, v, acc);
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
                    store8(static_cast<T*>(g.out) + row + c, w, n1 - c);
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
    const int64_t per_tile = std::clamp<int64_t>(ceil_div(640, tiles), 1, ceil_div(p.N, 128));
    q.cols = static_cast<int>(ceil_div(ceil_div(p.N, per_tile), 128) * 128);
    return q;
}

bool whole(const moe_adapter& p) { return p.K % 8 == 0 && p.N % 8 == 0 && p.R % 8 == 0; }

template <class T, int kRB, bool kWhole>
hipError_t launch_tiles(const Args& g, const TileArgs& t, const Plan& q, hipStream_t s)
{
    constexpr int kPB = kPlanesOf<T>, kPV = kPB == 1 ? 2 : 3;
    constexpr int kExpandLds = kPB * 32 * kRB * (2 * 128 + 16) + kPV * kTile * (64 * kRB + 16);
    static LdsLimit limit;
    if (hipError_t e = limit.ensure(reinterpret_cast<const void*>(&expand_kernel<T, kRB, kWhole>), kExpandLds); e != hipSuccess)
        return e;
    const unsigned tiles = static_cast<unsigned>(q.max_tiles);
    shrink_kernel<T, kRB, kWhole><<<dim3(tiles, q.splits), kThreads, 0, s>>>(g, t);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    expand_kernel<T, kRB, kWhole><<<dim3(tiles, static_cast<unsigned>(ceil_div(g.N, q.cols))), kThreads, kExpandLds, s>>>(g, t, q.cols);
    return hipGetLastError();
}

template <class T>
hipError_t launch(const moe_adapter& p, const Args& g, unsigned char* ws, hipStream_t s)
{
    const Plan q = plan(p);
    if (q.rows) {
        const dim3 grid(static_cast<unsigned>(p.T), static_cast<unsigned>(ceil_div(p.N, q.cols)));
        if (whole(p))
            row_kernel<T, true><<<grid, kRowThreads, 0, s>>>(g, q.cols);
        else
            row_kernel<T, false><<<grid, kRowThreads, 0, s>>>(g, q.cols);
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
    // rows of whole runs of eight values need no code for a run that ends early
    const auto by_blocks = [&](auto whole) {
        constexpr bool kWhole = decltype(whole)::value;
        return q.blocks == 1 ? launch_tiles<T, 1, kWhole>(g, t, q, s) : q.blocks == 2 ? launch_tiles<T, 2, kWhole>(g, t, q, s)
                                                                                     : launch_tiles<T, 4, kWhole>(g, t, q, s);
    };
    return whole(p) ? by_blocks(std::true_type{}) : by_blocks(std::false_type{});
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
    const Args g{base, x, a, b, out, ids, ranks, scale, static_cast<int>(p.T), static_cast<int>(p.K), static_cast<int>(p.N),
                 static_cast<int>(p.L), static_cast<int>(p.R)};
    unsigned char* const ws = static_cast<unsigned char*>(workspace);
    return p.dtype == MOE_F32 ? launch<float>(p, g, ws, s) : launch<uint16_t>(p, g, ws, s);
}

}  // namespace moe
