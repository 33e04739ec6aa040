// Low-rank adapters of many requests beside a shared projection (moe_adapter_add):
//   v[t] = scale[a] x[t] A[a],  out[t] = base[t] + v[t] B[a],  a = ids[t].
//
// Memory is what bounds it: x and base once, out once, each used adapter's A and B once; the products are R operations a
// byte.  Two ways:
//   - few rows (row_kernel; rule in plan()): one launch, a workgroup per (row, run of output columns).  Each computes its
//     row's v for itself, which reads the adapter's A again from the L2 but saves a launch and a pass through memory;
//   - many rows: the rows are sorted by adapter into tiles of up to 64 (plan_kernel, one workgroup), then v and v B run
//     on the matrix cores, tile by tile (shrink_kernel, expand_kernel).  x goes from memory to the MFMA's registers, the
//     adapter's matrices through LDS; K is cut so that there are workgroups enough, and join_kernel adds the cuts' float32
//     sums.  v enters the second product as two bfloat16 planes (16 bits) for bfloat16 tensors, as three for float32 ones.
// A row's result does not depend on the tile that it falls into, so neither the order in which the plan's counters hand
// out places nor other rows change it.  Planes of infinite values can make a product NaN that is infinite by the formula:
// a sum that comes out NaN is taken again from the values themselves (resum), as single rows have it
// (1% of float32 calls, less of bfloat16 ones: 4000 x 4096 x 4096 of rank 128 187 -> 190 us).
// Measured: one row 4096 -> 14336 of rank 16 7.5 us, 64 rows of 32 adapters 4096 -> 4096 10.5; 8192 rows 14336 -> 4096 of
// rank 64: plan 7, shrink 54-71 (median 71; it fetches 317 MB, x once and A once for each XCD, 4.5 TB/s), join 5, expand 32 (4.4
// TB/s of base, out and v).
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
    int tail;                             // the first adapter whose reads of A may pass the tensor's end (first_tail)
};

__device__ __forceinline__ int rank_of(const Args& g, int a) { return g.ranks == nullptr ? g.R : min(max(g.ranks[a], 0), g.R); }

// Eight values of A from `at` on (values from the tensor's start): what lies past the row belongs to columns that nobody
// reads, and only past the tensor's end (total values, at least 8) the last eight are read and shifted into place.
template <class T>
__device__ __forceinline__ Raw8<T> load_a(const T* a, int64_t at, int64_t total)
{
    return load_raw<true>(a + min(at, total - 8), 8);
}
__device__ __forceinline__ void shift_a(Raw8<uint16_t>& r, int skip)
{
    u32x4_t v = r.w;
    for (int i = 0; i < skip; ++i)
        v = u32x4_t{__builtin_amdgcn_alignbit(v[1], v[0], 16), __builtin_amdgcn_alignbit(v[2], v[1], 16),
                    __builtin_amdgcn_alignbit(v[3], v[2], 16), v[3] >> 16};
    r.w = v;
}
__device__ __forceinline__ void shift_a(Raw8<float>& r, int skip)
{
    for (int i = 0; i < skip; ++i) {
        r.a = f32x4_t{r.a[1], r.a[2], r.a[3], r.b[0]};
        r.b = f32x4_t{r.b[1], r.b[2], r.b[3], 0.0f};
    }
}
__device__ __forceinline__ bool past_end(const Args& g, int a) { return a >= g.tail; }
// How far the load of eight values from `at` on was moved back to end with the tensor.
__device__ __forceinline__ int moved_back(int64_t at, int64_t total)
{
    return static_cast<int>(max(at + 8 - total, static_cast<int64_t>(0)));
}

// Writes eight columns [from, from + 8) of a row, those before `first` left out (they are another thread's).
template <class T>
__device__ __forceinline__ void store_from(T* row, int from, int first, const float (&v)[8])
{
    if (from == first) {
        store8<T, true>(row + from, v, 8);
        return;
    }
#pragma unroll
    for (int i = 1; i < 8; ++i)
        if (from + i >= first) {
            if constexpr (sizeof(T) == 2)
                row[from + i] = f32_to_bf16(v[i]);
            else
                row[from + i] = v[i];
        }
}

// ------------------------------------------------------------------------------------------------ few rows

constexpr int kRowThreads = 1024;         // 16 waves: a CU has one or two of these workgroups, and 128 KiB in flight
constexpr int kRowWaves = kRowThreads / 64;
// Rows and bytes of A and B up to which row_kernel is taken (us of single rows against tiles with 1.5 between launches).
// Rows: 128 -> 128 of rank 8 bfloat16, 700 rows 14.6 / 17.4, 1024 rows 19.0 / 17.8; 1024 -> 1024 of rank 16, 700 rows 19.2
// / 22.5, 1000 rows 25.3 / 23.2.  Bytes, 4096 -> 4096: bfloat16 of rank 16, 131 MB 18.3 / 24.3, 184 MB 24.6 / 25.2, of rank
// 64, 157 MB 30.3 / 25.5; float32, whose planes make the tiles dearer, of rank 16, 268 MB 25.5 / 44.8.
constexpr int64_t kMaxRowTokens = 896;
constexpr int64_t max_row_reads(int64_t size) { return int64_t{size == 2 ? 144 : 256} << 20; }

// Workgroup (t, c): row t, output columns [c cols, (c + 1) cols).  Threads take (k, 8 columns of A) and add over k, then
// (r, 8 columns of B) and add over r; both are joined in a fixed order, within the wave and then through LDS.  Loads go
// out in batches, and what does not wait for v (the first rows of B, base) at the start.  A run of 8 columns that would
// pass the row's end is the row's last 8.
template <class T>
__global__ __launch_bounds__(kRowThreads) void row_kernel(Args g, int cols)
{
    constexpr int kBatch = sizeof(T) == 2 ? 8 : 4;         // 128 registers a thread
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
                const int from = min(n, g.N - 8);
                load_raw<true>(base + from, 8).values(w);
                store_from(out, from, n, w);
            }
        return;
    }
    const float scale = g.scale == nullptr ? 1.0f : g.scale[a];
    // threads per run of 8 output columns: as many as the run of columns leaves, at most the rank
    const T* const B = static_cast<const T*>(g.b) + static_cast<int64_t>(a) * g.R * g.N;
    const int runs = min(kRowThreads, (n1 - n0 + 7) / 8), lanes = max(1, min(rank, kRowThreads / runs));
    const int q = tid % runs, rr = min(tid / runs, lanes);
    const int first = n0 + 8 * q, from0 = min(first, g.N - 8);
    Raw8<T> b0 = load_raw<true>(B + static_cast<int64_t>(min(rr, rank - 1)) * g.N + from0, 8);
    Raw8<T> base0 = load_raw<true>(base + from0, 8);
    {
        const T* const x = static_cast<const T*>(g.x) + t * g.K;
        const T* const A = static_cast<const T*>(g.a);
        const int64_t a0 = static_cast<int64_t>(a) * g.K * g.R, total = static_cast<int64_t>(g.L) * g.K * g.R;
        // a power of two of column chunks, so that the lanes of one chunk are whole strides of the wave
        const int bits = rank <= 8 ? 0 : 32 - __clz((rank - 1) >> 3), chunks = 1 << bits;
        const int c = 8 * min(tid & (chunks - 1), (rank - 1) >> 3), stride = kRowThreads >> bits;
        float sum[8] = {};
        for (int k0 = tid >> bits; k0 < g.K; k0 += kBatch * stride) {
            Raw8<T> w[kBatch];
            T xk[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int k = min(k0 + i * stride, g.K - 1);
                w[i] = load_a(A, a0 + static_cast<int64_t>(k) * g.R + c, total);
                xk[i] = x[k];
            }
            if (past_end(g, a))
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    shift_a(w[i], moved_back(a0 + static_cast<int64_t>(min(k0 + i * stride, g.K - 1)) * g.R + c, total));
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                float f[8];
                w[i].values(f);
                const float m = to_float(xk[i]);
                if (k0 + i * stride < g.K)
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
    for (int pass = n0; pass < n1; pass += 8 * runs) {         // the same number of passes for every thread
        const int n = pass + 8 * q, from = min(n, g.N - 8);
        float sum[8] = {};
        if (rr < lanes && n < n1) {
            if (pass != n0) {
                b0 = load_raw<true>(B + static_cast<int64_t>(rr) * g.N + from, 8);
                base0 = load_raw<true>(base + from, 8);
            }
            float f[8];
            b0.values(f);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum[e] = v[rr] * f[e];
            for (int r0 = rr + lanes; r0 < rank; r0 += kBatch * lanes) {
                Raw8<T> w[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    w[i] = load_raw<true>(B + static_cast<int64_t>(min(r0 + i * lanes, rank - 1)) * g.N + from, 8);
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    w[i].values(f);
                    const int r = r0 + i * lanes;
                    if (r < rank)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            sum[e] = fmaf(v[r], f[e], sum[e]);
                }
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
            float f[8];
            base0.values(f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum[i] += f[i];
            store_from(out, from, n, sum);
        }
    }
}

// Rows of fewer than 8 columns, or fewer than 8 values of A in all: nothing that is read 8 values at a time exists.  A column of
// A after the other, for the sizes that nothing else takes: 4096 -> 7 of rank 16, 64 rows 50 us, 4096 rows 468.
template <class T>
__global__ __launch_bounds__(kThreads) void narrow_kernel(Args g)
{
    __shared__ float part[kThreads], v[kMaxRank];
    const int tid = threadIdx.x;
    for (int64_t t = blockIdx.x; t < g.T; t += gridDim.x) {
        const int a = g.ids[t], rank = a >= 0 && a < g.L ? rank_of(g, a) : 0;
        const T* const x = static_cast<const T*>(g.x) + t * g.K;
        for (int r = 0; r < rank; ++r) {
            const T* const A = static_cast<const T*>(g.a) + static_cast<int64_t>(a) * g.K * g.R + r;
            float s = 0.0f;
            for (int k = tid; k < g.K; k += kThreads)
                s = fmaf(to_float(x[k]), to_float(A[static_cast<int64_t>(k) * g.R]), s);
            part[tid] = s;
            for (int d = kThreads / 2; d > 0; d /= 2) {
                __syncthreads();
                if (tid < d)
                    part[tid] += part[tid + d];
            }
            if (tid == 0)
                v[r] = g.scale == nullptr ? part[0] : part[0] * g.scale[a];
            __syncthreads();
        }
        const T* const B = static_cast<const T*>(g.b) + static_cast<int64_t>(rank > 0 ? a : 0) * g.R * g.N;
        for (int n = tid; n < g.N; n += kThreads) {
            float s = 0.0f;
            for (int r = 0; r < rank; ++r)
                s = fmaf(v[r], to_float(B[static_cast<int64_t>(r) * g.N + n]), s);
            s += to_float(static_cast<const T*>(g.base)[t * g.N + n]);
            if constexpr (sizeof(T) == 2)
                static_cast<T*>(g.out)[t * g.N + n] = f32_to_bf16(s);
            else
                static_cast<T*>(g.out)[t * g.N + n] = s;
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
    const auto add = [&](int a) {
        const int bin = a >= 0 && a < L ? a : L;
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
    // Runs over this thread's rows, the loads of eight at a time ahead of their counters (one by one 8192 rows took 10 us).
    const auto each = [&](auto use) {
        constexpr int kAhead = 8;
        for (int t0 = tid; t0 < T; t0 += kAhead * kPlanThreads) {
            int id[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                id[i] = ids[min(t0 + i * kPlanThreads, T - 1)];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (t0 + i * kPlanThreads < T)
                    use(id[i], t0 + i * kPlanThreads);
        }
    };
    place[tid] = 0;
    __syncthreads();
    each([&](int a, int) { add(a); });
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
    each([&](int a, int t) { perm[add(a)] = t; });
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
    float* part;                          // sums over one cut of K each, [splits, T, 32 kRB] in sorted order
    uint16_t* v;                          // v's planes [2 or 3, T, 32 kRB] in sorted order
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

// sum[0 .. 7] = the sums over i in [i0, i1) of factor(i) times the first n of eight values at p + i ld.
template <class T, class F>
__device__ __forceinline__ void resum(float (&sum)[8], int i0, int i1, F factor, const T* p, int64_t ld, int n)
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        sum[e] = 0.0f;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        const float f = factor(i);
        float w[8];
        load8(w, p + i * ld, n);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum[e] = fmaf(f, w[e], sum[e]);
    }
}

// Eight values of v as the planes that enter the second product.
template <class T>
__device__ __forceinline__ void store_v(uint16_t* p, int64_t plane, const float (&w)[8])
{
    constexpr int PV = kPlanesOf<T> == 1 ? 2 : 3;
    u32x4_t pl[PV];
    split8<PV, true>(w, pl);
#pragma unroll
    for (int q = 0; q < PV; ++q)
        *reinterpret_cast<u32x4_t*>(p + q * plane) = pl[q];
}

// v of a tile's rows over one cut of K.  Waves: 2 row halves of 32 x 2 halves of each K step; kRB column blocks of 32.
template <class T, int kRB>
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
    const T* const A = static_cast<const T*>(g.a);
    const int64_t a0 = static_cast<int64_t>(tile.adapter) * g.K * g.R, total = static_cast<int64_t>(g.L) * g.K * g.R;
    const uint32_t lds = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned char*)(smem)));

    // Steps of whole kStep run with kSets of them in flight: unconditional loads (past the rank's and the last step's end
    // they repeat what is there), each into the registers that its step's predecessor has just left.
    constexpr int kSets = P == 1 ? 2 : 1;
    Raw8<T> xr[kSets][kGroups], ar[kSets][kLoads];
    const auto place = [&](int step, int i) {              // of this thread's value i of A in a step, from the tensor's start
        const int c = (tid + i * kThreads) % (kCols / 8), k = step * kStep + (tid + i * kThreads) / (kCols / 8);
        return a0 + static_cast<int64_t>(min(k, g.K - 1)) * g.R + min(8 * c, (g.R - 1) / 8 * 8);
    };
    const auto fetch_a = [&](Raw8<T>& r, int step, int i) { r = load_a(A, place(step, i), total); };
    const auto fetch_x = [&](Raw8<T>& r, int step, int s, bool partial) {
        const int k = step * kStep + (kStep / 2) * wk + 16 * s + 8 * (lane >> 5);
        r = partial ? load_raw<false>(x + k, g.K - k) : load_raw<true>(x + k, 8);
    };
    f32x16_t acc[kRB];
#pragma unroll
    for (int j = 0; j < kRB; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e)
            acc[j][e] = 0.0f;
    // one step from one set of registers, which then take step `next` (more: there is one)
    const auto run = [&](auto more, Raw8<T> (&av)[kLoads], Raw8<T> (&xv)[kGroups], int step, int next) {
        constexpr bool kMore = decltype(more)::value;
        if (past_end(g, tile.adapter))
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                shift_a(av[i], moved_back(place(step, i), total));
        __syncthreads();                                  // the stage of the step before is read
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = tid + i * kThreads;
            u32x4_t pl[P];
            planes8(av[i], pl);
#pragma unroll
            for (int q = 0; q < P; ++q)
                *reinterpret_cast<u32x4_t*>(smem + q * kPlane + (at / (kCols / 8)) * kRow + 16 * (at % (kCols / 8))) =
                    step * kStep + at / (kCols / 8) < g.K ? pl[q] : u32x4_t{0, 0, 0, 0};
        }
        __syncthreads();
        if constexpr (kMore)
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                fetch_a(av[i], next, i);
#pragma unroll
        for (int s = 0; s < kGroups; ++s) {
            u32x4_t xp[P];
            planes8(xv[s], xp);
            bf16x8_t r[P];
#pragma unroll
            for (int q = 0; q < P; ++q)
                r[q] = __builtin_bit_cast(bf16x8_t, xp[q]);
            if constexpr (kMore)
                fetch_x(xv[s], next, s, false);
#pragma unroll
            for (int j = 0; j < kRB; ++j) {
                bf16x8_t w[P];
#pragma unroll
                for (int q = 0; q < P; ++q)
                    w[q] = read_tr(lds + q * kPlane + ((kStep / 2) * wk + 16 * s) * kRow + 64 * j + tr_offset(lane, kRow), kRow);
                acc[j] = mfma_planes<P, P>(w, r, acc[j]);
            }
        }
    };
    const int whole1 = min(step1, g.K / kStep);            // steps [step0, whole1) lie within K
    if (step0 < whole1) {
#pragma unroll
        for (int u = 0; u < kSets; ++u) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                fetch_a(ar[u][i], min(step0 + u, whole1 - 1), i);
#pragma unroll
            for (int s = 0; s < kGroups; ++s)
                fetch_x(xr[u][s], min(step0 + u, whole1 - 1), s, false);
        }
        int step = step0;
        for (; step + kSets <= whole1; step += kSets)
#pragma unroll
            for (int u = 0; u < kSets; ++u)
                run(std::true_type{}, ar[u], xr[u], step + u, min(step + u + kSets, whole1 - 1));
        if (step < whole1)
            run(std::false_type{}, ar[0], xr[0], step, 0);
    }
    if (whole1 < step1) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            fetch_a(ar[0][i], whole1, i);
#pragma unroll
        for (int s = 0; s < kGroups; ++s)
            fetch_x(xr[0][s], whole1, s, true);
        run(std::false_type{}, ar[0], xr[0], whole1, 0);
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
        const int64_t at = static_cast<int64_t>(tile.begin + 32 * wr + (lane & 31)) * kCols;
#pragma unroll
        for (int j = 0; j < kRB; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = 32 * j + 16 * h + 8 * (lane >> 5);
                float w[8], u[8];
                run8(acc[j], h, w);
                load8(u, join + 32 * j + 16 * h, 8);
                if (32 * wr + (lane & 31) >= n)
                    continue;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i] = c + i < rank ? w[i] + u[i] : 0.0f;
                if constexpr (P > 1)
                    if (any_nan(w))                       // of columns below the rank
                        resum(w, step0 * kStep, min(step1 * kStep, g.K), [&](int k) { return x[k]; }, A + a0 + c, g.R, rank - c);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i] = c + i < rank ? w[i] * f : 0.0f;
                if (p.splits == 1)
                    store_v<T>(p.v + at + c, static_cast<int64_t>(g.T) * kCols, w);
                else
                    store8(p.part + static_cast<int64_t>(split) * g.T * kCols + at + c, w, 8);
            }
    }
}

// v from the cuts' sums; n groups of 8 values.
template <class T>
__global__ __launch_bounds__(kThreads) void join_kernel(const float* __restrict__ part, uint16_t* __restrict__ v, int splits,
                                                        int64_t n)
{
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (at >= n)
        return;
    constexpr int kAhead = 4;                             // cuts whose loads go out together
    float sum[8] = {};
    for (int q0 = 0; q0 < splits; q0 += kAhead) {
        Raw8<float> w[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            w[i] = load_raw<true>(part + 8 * (at + (q0 + i) * n), q0 + i < splits ? 8 : 0);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            float f[8];
            w[i].values(f);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum[e] += f[e];
        }
    }
    store_v<T>(v + 8 * at, 8 * n, sum);
}

// LDS of expand_kernel: B's rows of one run, then v's planes.  The run's product takes the place of B once that is read.
template <class T, int kRB>
struct ExpandLds {
    static constexpr int PB = kPlanesOf<T>, PV = PB == 1 ? 2 : 3, kR = 32 * kRB;
    static constexpr int kRow = 2 * 128 + 16, kPlane = kR * kRow;         // B: bytes of a row, of a plane
    static constexpr int kOutRow = 4 * 128 + 16;                           // the product, float32
    static constexpr int kVRow = 2 * kR + 16, kVPlane = kTile * kVRow;
    static constexpr int kV = PB * kPlane > kTile * kOutRow ? PB * kPlane : kTile * kOutRow;   // where v begins
    static constexpr int kBytes = kV + PV * kVPlane;
    // Workgroups: those resident, three per CU at most (8192 x 4096, rank 64: 32 us, 512 of them 35, 1024 36; rank 100,
    // where two fit: 2000 x 11776 36, 768 of them 41).
    static constexpr int kGrid = 256 * (160 * 1024 / kBytes < 3 ? 160 * 1024 / kBytes : 3);
};

// out.  The work is the (tile, run of 128 columns) pairs in order, in equal shares for the workgroups of the grid.  For the
// product each of the four waves takes 32 columns of all 64 rows; for base and out, whole rows of a run (256 or 512 bytes;
// with pieces of 32 rows, as the accumulators hold them, 8192 x 4096 of rank 64 took 6 us longer).
template <class T, int kRB>
__global__ __launch_bounds__(kThreads) void expand_kernel(Args g, TileArgs p)
{
    using M = ExpandLds<T, kRB>;
    constexpr int PB = M::PB, PV = M::PV, kR = M::kR, kLoads = kR * 16 / kThreads;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t lds = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned char*)(smem)));
    const uint32_t runs = (g.N + 127) / 128;
    const int col = 8 * (tid % 16), row0 = tid / 16;   // this thread: rows row0 + 16 i
    // T N is at most 2^37: fewer than 2^32 pairs
    const uint32_t items = static_cast<uint32_t>(p.count[0]) * runs, per = items / gridDim.x, more = items % gridDim.x;
    const uint32_t item1 = per * (blockIdx.x + 1) + min(blockIdx.x + 1, more);
    for (uint32_t item = per * blockIdx.x + min(blockIdx.x, more); item < item1;) {
        const int ti = static_cast<int>(item / runs), run0 = static_cast<int>(item - static_cast<uint32_t>(ti) * runs);
        const int run1 = static_cast<int>(min(runs, run0 + item1 - item));
        item += run1 - run0;
        const Tile tile = p.tiles[ti];
        const int n0 = 128 * run0, n1 = min(128 * run1, g.N), n = tile.end - tile.begin;
        const int rank = tile.adapter < g.L ? rank_of(g, tile.adapter) : 0;
        if (rank == 0 && g.base == g.out)
            continue;
        int64_t at[4];                                    // rows past the last repeat it and are not written
#pragma unroll
        for (int i = 0; i < 4; ++i)
            at[i] = static_cast<int64_t>(p.perm[tile.begin + min(row0 + 16 * i, n - 1)]) * g.N;
        Raw8<T> bv[kLoads], base[4];
        if (rank == 0) {                                  // the rows are copied (one by one a tile took 9 us)
            for (int c = n0 + col; c < n1; c += 128) {
                const int from = min(c, g.N - 8);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    base[i] = load_raw<true>(static_cast<const T*>(g.base) + at[i] + from, 8);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float w[8];
                    base[i].values(w);
                    if (row0 + 16 * i < n)
                        store_from(static_cast<T*>(g.out) + at[i], from, c, w);
                }
            }
            continue;
        }
        const T* const B = static_cast<const T*>(g.b) + static_cast<int64_t>(tile.adapter) * g.R * g.N;
        const auto fetch = [&](int c0) {
            const int from = min(c0 + col, g.N - 8);      // the row's last 8 columns where these would pass its end
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                bv[i] = load_raw<true>(B + static_cast<int64_t>(min(row0 + 16 * i, rank - 1)) * g.N + from, 8);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                base[i] = load_raw<true>(static_cast<const T*>(g.base) + at[i] + from, 8);
        };
        fetch(n0);
        // v of the tile's rows (once the tile before is done with its own)
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTile * kR / 8 / kThreads; ++i) {
            const int r = (tid + i * kThreads) / (kR / 8), c = 8 * ((tid + i * kThreads) % (kR / 8));
            const uint16_t* const v = p.v + (static_cast<int64_t>(tile.begin) + min(r, n - 1)) * kR + c;
#pragma unroll
            for (int q = 0; q < PV; ++q)
                *reinterpret_cast<u32x4_t*>(smem + M::kV + q * M::kVPlane + r * M::kVRow + 2 * c) =
                    *reinterpret_cast<const u32x4_t*>(v + static_cast<int64_t>(q) * g.T * kR);
        }
        const unsigned char* const mine_v = smem + M::kV + (lane & 31) * M::kVRow + 16 * (lane >> 5);
        for (int c0 = n0; c0 < n1; c0 += 128) {
            __syncthreads();                              // the product of the run before is read
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {            // B's rows from the rank on are zero
                u32x4_t pl[PB];
                planes8(bv[i], pl);
#pragma unroll
                for (int q = 0; q < PB; ++q)
                    *reinterpret_cast<u32x4_t*>(smem + q * M::kPlane + (row0 + 16 * i) * M::kRow + 2 * col) =
                        row0 + 16 * i < rank ? pl[q] : u32x4_t{0, 0, 0, 0};
            }
            __syncthreads();
            f32x16_t acc[2];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    acc[b][e] = 0.0f;
#pragma unroll
            for (int k = 0; k < 2 * kRB; ++k) {
                bf16x8_t w[PB];
#pragma unroll
                for (int q = 0; q < PB; ++q)
                    w[q] = read_tr(lds + q * M::kPlane + 16 * k * M::kRow + 64 * wave + tr_offset(lane, M::kRow), M::kRow);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    bf16x8_t v[PV];
#pragma unroll
                    for (int q = 0; q < PV; ++q)
                        v[q] = *reinterpret_cast<const bf16x8_t*>(mine_v + q * M::kVPlane + 32 * b * M::kVRow + 32 * k);
                    acc[b] = mfma_planes<PV, PB>(w, v, acc[b]);
                }
            }
            __syncthreads();
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int q = 0; q < 4; ++q)               // columns 8 q + 4 (lane / 32) .. + 3 of the wave's 32
                    *reinterpret_cast<f32x4_t*>(smem + (32 * b + (lane & 31)) * M::kOutRow +
                                                4 * (32 * wave + 8 * q + 4 * (lane >> 5))) =
                        f32x4_t{acc[b][4 * q], acc[b][4 * q + 1], acc[b][4 * q + 2], acc[b][4 * q + 3]};
            __syncthreads();
            // rows whose sums are looked at together: a branch at each would part their loads, four of float32 take registers
            // of a third workgroup
            constexpr int kTogether = PB == 1 ? 4 : 2;
#pragma unroll
            for (int i0 = 0; i0 < 4; i0 += kTogether) {
                float sum[kTogether][8];
                bool nan = false;
#pragma unroll
                for (int i = 0; i < kTogether; ++i) {
                    load8(sum[i], reinterpret_cast<const float*>(smem + (row0 + 16 * (i0 + i)) * M::kOutRow) + col, 8);
                    nan |= any_nan(sum[i]);
                }
                if (nan)
#pragma unroll
                    for (int i = 0; i < kTogether; ++i) {
                        const unsigned char* const v = smem + M::kV + (row0 + 16 * (i0 + i)) * M::kVRow;
                        const auto value = [&](int r) {
                            float f = 0.0f;
#pragma unroll
                            for (int q = PV - 1; q >= 0; --q)
                                f += bf16_to_f32(*reinterpret_cast<const uint16_t*>(v + q * M::kVPlane + 2 * r));
                            return f;
                        };
                        if (any_nan(sum[i]))
                            resum(sum[i], 0, rank, value, B + min(c0 + col, g.N - 8), g.N, 8);
                    }
#pragma unroll
                for (int i = 0; i < kTogether; ++i) {
                    float u[8];
                    base[i0 + i].values(u);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        u[e] += sum[i][e];
                    if (row0 + 16 * (i0 + i) < n && c0 + col < g.N)
                        store_from(static_cast<T*>(g.out) + at[i0 + i], min(c0 + col, g.N - 8), c0 + col, u);
                }
            }
            // the next run's values are loaded when their registers are free: copying them would wait for the loads
            __builtin_amdgcn_sched_barrier(0);
            if (c0 + 128 < n1)
                fetch(c0 + 128);
        }
    }
}

// ------------------------------------------------------------------------------------------------ the host's side

// The first adapter with fewer than eight values of A behind it, where rows are not whole runs of eight: loads of eight
// values from inside such an adapter on may pass the tensor's end.
int first_tail(const moe_adapter& p)
{
    return static_cast<int>(p.R % 8 == 0 ? p.L : std::max<int64_t>(p.L - ceil_div(8, p.K * p.R), 0));
}

// How a call runs.
struct Plan {
    bool narrow;              // narrow_kernel
    bool rows;                // row_kernel
    int cols;                 // row_kernel: output columns per workgroup
    int blocks;               // column blocks of 32 that hold the rank (1, 2 or 4)
    int splits, steps;
    int64_t max_tiles;
};

Plan plan(const moe_adapter& p)
{
    Plan q{};
    const int64_t size = p.dtype == MOE_F32 ? 4 : 2;
    q.narrow = p.N < 8 || p.L * p.K * p.R < 8;
    if (q.narrow)
        return q;
    q.rows = p.T <= kMaxRowTokens && p.K * p.R * size <= (int64_t{1} << 20) &&
             p.T * (p.K + p.N) * p.R * size <= max_row_reads(size);
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
    // about 1024 workgroups of the shrink (512: 5000 x 11776 of rank 32 52 us against 40, float32 of rank 128 105 against 80)
    q.splits = static_cast<int>(std::clamp<int64_t>(ceil_div(1024, tiles), 1, std::clamp<int64_t>(q.steps / 4, 1, 16)));
    return q;
}

template <class T, int kRB>
hipError_t launch_tiles(const Args& g, const TileArgs& t, const Plan& q, hipStream_t s)
{
    constexpr int kExpandLds = ExpandLds<T, kRB>::kBytes;
    static LdsLimit limit;
    if (hipError_t e = limit.ensure(reinterpret_cast<const void*>(&expand_kernel<T, kRB>), kExpandLds); e != hipSuccess)
        return e;
    const unsigned tiles = static_cast<unsigned>(q.max_tiles);
    shrink_kernel<T, kRB><<<dim3(tiles, q.splits), kThreads, 0, s>>>(g, t);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    if (t.splits > 1) {
        const int64_t n = static_cast<int64_t>(g.T) * 4 * kRB;
        join_kernel<T><<<dim3(static_cast<unsigned>(ceil_div(n, kThreads))), kThreads, 0, s>>>(t.part, t.v, t.splits, n);
        if (hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
    }
    const int64_t items = q.max_tiles * ceil_div(g.N, 128);
    expand_kernel<T, kRB><<<dim3(static_cast<unsigned>(std::min<int64_t>(items, ExpandLds<T, kRB>::kGrid))), kThreads, kExpandLds, s>>>(g, t);
    return hipGetLastError();
}

template <class T>
hipError_t launch(const moe_adapter& p, const Args& g, unsigned char* ws, hipStream_t s)
{
    const Plan q = plan(p);
    if (q.narrow) {
        narrow_kernel<T><<<dim3(static_cast<unsigned>(std::min<int64_t>(p.T, 65536))), kThreads, 0, s>>>(g);
        return hipGetLastError();
    }
    if (q.rows) {
        const dim3 grid(static_cast<unsigned>(p.T), static_cast<unsigned>(ceil_div(p.N, q.cols)));
        row_kernel<T><<<grid, kRowThreads, 0, s>>>(g, q.cols);
        return hipGetLastError();
    }
    const AdapterLayout L = adapter_layout(p);
    int32_t* const perm = reinterpret_cast<int32_t*>(ws + L.perm);
    Tile* const tiles = reinterpret_cast<Tile*>(ws + L.tiles);
    int32_t* const count = reinterpret_cast<int32_t*>(ws + L.count);
    plan_kernel<<<1, kPlanThreads, 0, s>>>(g.ids, g.T, g.L, perm, tiles, count);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    const TileArgs t{tiles, count, perm, reinterpret_cast<float*>(ws + L.part), reinterpret_cast<uint16_t*>(ws + L.v), q.splits,
                     q.steps};
    return q.blocks == 1 ? launch_tiles<T, 1>(g, t, q, s) : q.blocks == 2 ? launch_tiles<T, 2>(g, t, q, s)
                                                                         : launch_tiles<T, 4>(g, t, q, s);
}

}  // namespace

AdapterLayout adapter_layout(const moe_adapter& p)
{
    AdapterLayout L;
    const Plan q = plan(p);
    if (q.narrow || q.rows)
        return L;
    size_t off = 0;
    const auto take = [&](size_t& at, size_t bytes) {
        at = off;
        off = align_up(off + bytes);
    };
    take(L.count, sizeof(int32_t));
    take(L.perm, static_cast<size_t>(p.T) * sizeof(int32_t));
    take(L.tiles, static_cast<size_t>(q.max_tiles) * sizeof(Tile));
    take(L.v, static_cast<size_t>(p.dtype == MOE_F32 ? 3 : 2) * p.T * 32 * q.blocks * sizeof(uint16_t));
    if (q.splits > 1)
        take(L.part, static_cast<size_t>(q.splits) * p.T * 32 * q.blocks * sizeof(float));
    L.total = off;
    return L;
}

hipError_t launch_adapter(const moe_adapter& p, const void* base, const void* x, const void* a, const void* b,
                          const int32_t* ids, const float* scale, const int32_t* ranks, void* out, void* workspace,
                          hipStream_t s)
{
    const Args g{base, x, a, b, out, ids, ranks, scale, static_cast<int>(p.T), static_cast<int>(p.K), static_cast<int>(p.N),
                 static_cast<int>(p.L), static_cast<int>(p.R), first_tail(p)};
    unsigned char* const ws = static_cast<unsigned char*>(workspace);
    return p.dtype == MOE_F32 ? launch<float>(p, g, ws, s) : launch<uint16_t>(p, g, ws, s);
}

}  // namespace moe
