// Host-side internals of the gate and the int8 operators: launchers shared by api.cpp and the kernels.
#pragma once

#include "internal.h"
#include "moe_expert_layer.h"

namespace moe {

// gate.hip: the gate with scores, bias, groups and renormalised weights, and its gradient
// (moe_router_gate, moe_router_gate_backward); dtype MOE_F32 or MOE_BF16 logits.
hipError_t launch_gate(const moe_gate& o, const void* logits, int dtype, const float* bias, int64_t T,
                       int64_t E, int64_t k, int32_t* ids, float* probs, hipStream_t s);
hipError_t launch_gate_backward(const moe_gate& o, const void* logits, int dtype, int64_t T, int64_t E,
                                int64_t k, const int32_t* ids, const float* dprobs, void* dlogits, hipStream_t s);

// gemm_i8.hip: grouped GEMMs on int8 rows and weights, scales per row and per (expert, column).
constexpr int64_t kInt8MaxK = 130944;  // |sum of K products of -128 .. 127| stays below 2^31
bool int8_supported(int64_t K, int64_t N);
// How a grouped product of M rows in at most G groups with [K, N] weights (gated: two of them) runs:
// the tile table's height, the cuts of K, and whether the kernel leaves int32 partial sums
// ([splits, M, N], gated [splits, M, 2 N]) for launch_int8_finish / launch_int8_swiglu_partial.
struct Int8Plan {
    int row_tile;
    int splits;
    bool partial;
};
Int8Plan int8_plan(int64_t M, int64_t G, int64_t K, int64_t N);
// The same for the two products of an FFN, which share a tile table.
void int8_ffn_plans(int64_t M, int64_t G, int64_t H, int64_t F, Int8Plan& fc1, Int8Plan& fc2);
// Whether the plan's tasks (row tiles x column tiles x cuts) can be numbered in 32 bits.
bool int8_tasks_fit(const Int8Plan& p, int64_t M, int64_t G, int64_t N, bool gated);
// The groups of a product's M rows (offsets [G + 1]; expert [G], null: group g is expert g).  tiles: the table of
// launch_int8_tiles with its count; null, where int8_own_tiles allows it: each workgroup builds the table for
// itself, and the first one writes the status word unless that is null.
struct Int8Groups {
    const int32_t* offsets;
    const int32_t* expert;
    int G, E;
    int32_t* status;
    const MTile* tiles;
    const int32_t* tile_count;
};
bool int8_own_tiles(const Int8Plan& p, int64_t M, int64_t G);
// The layer keeps the down projection's sums as float16, times a power of two (of K) that brings the largest
// possible one, 127 * 128 * K, to at most 2^15: 11 bits of each sum, where a scaled bfloat16 row would keep 8.
constexpr int kInt8HalfSums = 100;          // out_dtype of launch_gemm_i8, beside the public ones
inline float int8_half_unit(int64_t K)
{
    int bits = 0;
    while ((int64_t{1} << bits) < K)
        ++bits;
    return bits > 1 ? 1.0f / static_cast<float>(1 << (bits - 1)) : 1.0f;
}
// out: [M, N] of out_dtype (MOE_F32 / MOE_BF16 / kInt8HalfSums), gated (w1 not null) float32 swiglu of the two
// products, or the partial sums.  gather (may be null): row p of the product is row
// gather[p] / gather_k of A and a_scale, whose rows then lie within 2^32 bytes.  task_ctr: kXcdCount zeroed
// counters for this launch (256-row tiles).
hipError_t launch_gemm_i8(const Int8Plan& p, const int8_t* A, const float* a_scale, const int8_t* w0,
                          const float* s0, const int8_t* w1, const float* s1, void* out, int out_dtype,
                          int64_t M, int64_t K, int64_t N, const Int8Groups& groups,
                          const int32_t* gather, int gather_k, int32_t* task_ctr, hipStream_t s);
// quant_i8.hip.  Rows of float32 or bfloat16 -> int8 codes and one scale per row (moe_int8_quantize).
hipError_t launch_int8_quantize(int dtype, const void* x, int64_t rows, int64_t cols, int8_t* codes,
                                float* scales, hipStream_t s);
// The rows that a group holds (offsets, group_expert as for launch_build_tiles; row_experts, where not
// null, says each row's expert, -1 for none) from the gated partial sums [splits, M, 2 F]: h =
// swiglu(gate, up), quantised.
hipError_t launch_int8_swiglu_partial(const int32_t* partial, int splits, const float* a_scale,
                                      const int32_t* gather, int gather_k, const float* sg, const float* su,
                                      const int32_t* row_experts, const int32_t* offsets,
                                      const int32_t* group_expert, int64_t G, int64_t E, int64_t M,
                                      int64_t F, int8_t* codes, float* scales, hipStream_t s);
// The table of balanced row tiles alone (the in-run table of launch_build_tiles, with its count at
// tile_count, the counters and the status word as there), at most max_mtiles of them whatever the offsets.
hipError_t launch_int8_tiles(const int32_t* offsets, const int32_t* group_expert, int64_t G, int64_t E, int64_t M,
                             int bm, MTile* tiles, int32_t* tile_count, int32_t* task_ctr, int32_t* status,
                             bool write_status, hipStream_t s);
// The routing (as launch_route_* leave it, and each row's expert), the table of balanced row tiles of
// height bm with its count, and with x not null the quantised token rows, in one launch; at most
// kInt8SmallSlots slots.  tiles null: no table.
constexpr int64_t kInt8SmallSlots = 256;
hipError_t launch_int8_prologue(const int32_t* ids, int64_t T, int64_t k, int64_t E, int32_t* counts, int32_t* offsets,
                                int32_t* perm, int32_t* pos, int32_t* row_experts, int32_t* status, int bm,
                                MTile* tiles, int32_t* tile_count, const uint16_t* x, int64_t H, int8_t* codes, float* scales,
                                hipStream_t s);
// The layer's output [T, N] bfloat16 from the down projection's sums: partial sums [splits, T k, N] int32, or with
// splits 0 float16 rows [T k, N] (kInt8HalfSums).  K: the down projection's, for the rows' unit.
hipError_t launch_int8_combine(const void* sums, int splits, int64_t K, const float* a_scale, const float* w_scale,
                               const int32_t* expert_ids, const int32_t* pos, const float* probs, int64_t T, int64_t k,
                               int64_t N, uint16_t* out, hipStream_t s);
// out [M, N] from the partial sums [splits, M, N] of the rows that a group holds.
hipError_t launch_int8_finish(const int32_t* partial, int splits, const float* a_scale, const float* w_scale,
                              const int32_t* offsets, const int32_t* group_expert, int64_t G, int64_t E,
                              int64_t M, int64_t N, void* out, int out_dtype, hipStream_t s);

}  // namespace moe
