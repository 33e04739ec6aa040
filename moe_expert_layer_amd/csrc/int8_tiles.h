// Device side shared by the int8 kernels: the rows of each group, a group's balanced row tiles, float16 values.
#pragma once

#include "common.h"
#include "internal.h"

namespace moe {

// Two floats to float16, round to nearest even, lo in the low half; and back.
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi)
{
    return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<_Float16>(lo))) |
           static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<_Float16>(hi))) << 16;
}
__device__ __forceinline__ float half_to_f32(uint16_t h)
{
    return static_cast<float>(__builtin_bit_cast(_Float16, h));
}

// What a thread's group holds: its rows, the tiles before it and the tiles of all groups of the pass.
struct GroupRows {
    int begin, rows, expert, first, total;
    bool bad;                                                 // rows of an expert that does not exist: skipped
};

// Groups base + threadIdx.x of a workgroup of kWaves waves, with row tiles of bm.  A group begins no earlier
// than any offset before it (`reached`: the largest one of earlier passes), so that no row is in two groups
// and all tiles together are at most max_mtiles, whatever the offsets.  wave_max and wave_sum: LDS, kWaves
// words each.  All threads call it; two barriers, after which a further pass may follow at once.
template <int kWaves>
__device__ __forceinline__ GroupRows scan_groups(const int32_t* __restrict__ offsets,
                                                 const int32_t* __restrict__ group_expert, int base, int G, int E,
                                                 int64_t M, int bm, int& reached, int* wave_max, int* wave_sum)
{
    const int me = threadIdx.x, lane = me & 63, wave = me >> 6, limit = static_cast<int>(M);
    const bool mine = base + me < G;
    const int g = mine ? base + me : 0;
    const int o = mine ? min(max(offsets[g], 0), limit) : 0;
    const int end = mine ? min(max(offsets[g + 1], 0), limit) : 0;
    GroupRows r;
    r.expert = mine ? (group_expert != nullptr ? group_expert[g] : g) : 0;
    int rb = o;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1)
        rb = max(rb, __shfl_up(rb, off));                     // a lane below `off` gets its own value
    if (lane == 63)
        wave_max[wave] = rb;
    __syncthreads();
    rb = max(rb, reached);
    for (int w = 0; w < kWaves; ++w) {
        rb = w < wave ? max(rb, wave_max[w]) : rb;
        reached = max(reached, wave_max[w]);
    }
    r.begin = rb;
    r.rows = max(end - rb, 0);
    r.bad = false;
    if (r.expert < 0 || r.expert >= E) {
        r.bad = r.rows > 0;
        r.rows = 0;
    }
    const int count = (r.rows + bm - 1) / bm;
    int before = count;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(before, off);
        before += lane >= off ? v : 0;
    }
    if (lane == 63)
        wave_sum[wave] = before;
    __syncthreads();
    r.first = before - count;
    r.total = 0;
    for (int w = 0; w < kWaves; ++w) {
        r.first += w < wave ? wave_sum[w] : 0;
        r.total += wave_sum[w];
    }
    return r;
}

// Tile i of the R balanced ones of a group of n rows from row `begin`: its 32-row blocks are dealt as
// evenly as possible, the last tile ends the group (the in-run table of launch_build_tiles).
__device__ __forceinline__ MTile balanced_tile(int expert, int begin, int n, int R, int i, int run_begin)
{
    const int blocks = (n + 31) / 32, each = blocks / R, more = blocks % R;
    MTile t;
    t.expert = expert;
    t.row_begin = begin + 32 * (each * i + min(i, more));
    t.row_end = i == R - 1 ? begin + n : begin + 32 * (each * (i + 1) + min(i + 1, more));
    t.chunk = 0;
    t.run_begin = run_begin;
    t.run_len = R;
    t.pad0 = t.pad1 = 0;
    return t;
}

}  // namespace moe
