// The gated block of a shared expert and its gradient on gfx950 MFMA (moe_gated_projection,
// moe_gated_projection_backward):
//
//   forward    g = x Wg, u = x Wu, h = D(act(g) u)                 x [T, H], Wg / Wu [H, F], h [T, F]
//   backward   d = D(dh), dg = d u act'(g), du = d act(g)
//              dx = dg Wg^T + du Wu^T, dWg = x^T dg, dWu = x^T du
//
// All products run through one kernel, gemm<>, C [M, N] = sum over segments of A B, whose operands lie either with K
// contiguous (kKC: rows of K values) or as K rows of contiguous columns (kNC):
//   forward  A = x (kKC), B = Wg and Wu (kNC), both in one tile: the epilogue holds g and u of the same columns
//   dx       A = dg, then du (kKC), B = Wg, then Wu (kKC): two segments of one sum
//   dWg|dWu  A = x (kNC, M = H), B = dg | du (kNC): K = T
// bfloat16 operands go to v_mfma_f32_32x32x16_bf16 as they are, float32 operands as three bfloat16 planes (planes.h): six
// segments of one sum, the small products first, so that the partial sums stay small until the last sixth of the additions.
#include <algorithm>
#include <atomic>
#include <utility>

#include "dropout.h"
#include "planes.h"

namespace moe {
namespace {

enum Layout { kKC = 0, kNC = 1 };
enum Epi {
    kEpiGated,       // h, and g and u where they are kept
    kEpiGatedBwd,    // dg and du
    kEpiOut          // the product itself
};

constexpr int kBK = 64;                         // K values per step: 128-byte rows of a kKC operand, whole cache lines
constexpr uint32_t kOob = 0xC0000000u;          // a buffer offset past any num_records used here: reads as zero

// Tile shape: kWM x kWN waves, each kTM x kTN accumulator blocks of 32 x 32.
template <int kWM_, int kWN_, int kTM_, int kTN_, int kBlocks_>
struct Shape {
    static constexpr int kWM = kWM_, kWN = kWN_, kTM = kTM_, kTN = kTN_, kBlocks = kBlocks_;
    static constexpr int kWaves = kWM * kWN, kThreads = kWaves * 64;
    static constexpr int BM = 32 * kWM * kTM, BNB = 32 * kWN * kTN;    // rows, staged columns of B
    static constexpr int kABytes = BM * kBK * 2, kBBytes = BNB * kBK * 2, kStage = kABytes + kBBytes;
    static constexpr int kSmem = 2 * kStage;
    static constexpr int kAC = kABytes / 1024 / kWaves, kBC = kBBytes / 1024 / kWaves;   // 1 KiB copies per wave
    static_assert(kAC * kWaves * 1024 == kABytes && kBC * kWaves * 1024 == kBBytes, "whole copies");
    static_assert(kAC % 2 == 0 && kBC % 2 == 0 && kWaves % 2 == 0 && kTN % 2 == 0, "pairs");
};

struct GemmArgs {
    // operand planes: segment s multiplies plane (a_idx >> 4 s) & 15 of a with plane (b_idx >> 4 s) & 7 of b0, or of
    // b1 where bit 3 is set; a gated tile, and the second half of the column tiles with mats = 2, take the other one
    const uint16_t *a, *b0, *b1;
    int64_t a_plane, b_plane;                   // values between planes
    uint64_t a_idx, b_idx;
    int nseg, kt;                               // segments, steps of kBK per segment
    int lda, ldb;                               // values between rows, multiples of 8
    int M, N, K;                                // rows, columns (of one matrix), the rows of a kNC operand
    int mt, nt, mats;                           // row tiles, column tiles (of one matrix), matrices of columns
    // epilogue
    void *o0, *o1;                              // outputs of matrix 0 and 1 (kEpiOut), h (kEpiGated)
    int ldo;
    void *save_g, *save_u;                      // g and u, laid out as h (or null)
    const void* dh;                             // kEpiGatedBwd: [M, ld_dh], of which n_dh columns exist
    int ld_dh;
    uint16_t* dgu;                              // planes of dg, then of du, [M, ldb] each
    int64_t dgu_plane;
    int act;
    Dropout drop;
};

__device__ __forceinline__ void copy16(const i32x4_t& rsrc, uint32_t voff, uint32_t lds)
{
    // LDS DMA of 16 bytes per lane through a buffer resource: lane i writes LDS byte lds + 16 i; offsets past the
    // resource's end read as zero.  Counts in vmcnt; the waits are explicit (step_barrier).
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :: "v"(voff), "s"(rsrc), "s"(lds) : "memory");
}

// This wave's copies and LDS reads are complete, then the workgroup's.
__device__ __forceinline__ void step_barrier()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ i32x4_t make_rsrc(const uint16_t* p, int64_t bytes)
{
    const uint64_t q = reinterpret_cast<uint64_t>(p);
    return i32x4_t{__builtin_amdgcn_readfirstlane(static_cast<int>(q)),
                   __builtin_amdgcn_readfirstlane(static_cast<int>(q >> 32) & 0xFFFF),
                   __builtin_amdgcn_readfirstlane(static_cast<int>(bytes)), 0x00027000};
}

// One operand's share of an LDS stage: kCols rows (kKC) or columns (kNC) of 64 k.
//   kKC: row r is 128 bytes, its 16-byte chunk c (8 k) lies at c ^ ((r >> 1) & 7): 16 rows' reads of one chunk cover
//        all 16 bank groups
//   kNC: k row kr is 2 kCols bytes, chunk c (8 columns) lies at c ^ swizzle(kr): the four k rows of a transposing read
//        land in four different 64-byte quarters of a 256-byte bank window
template <int kLayout, int kCols>
struct Region {
    static constexpr int kRow = kLayout == kKC ? 128 : 2 * kCols;
    static constexpr int kChunks = kRow / 16;
    static constexpr int kRowsPerCopy = 64 / kChunks;
    static constexpr int kBytes = kCols * kBK * 2;
    static_assert(kLayout == kKC || kChunks == 8 || kChunks == 16 || kChunks == 32, "swizzle");
    static __device__ __forceinline__ int swizzle(int r)
    {
        if constexpr (kLayout == kKC)
            return (r >> 1) & 7;
        else
            return kChunks == 8 ? 4 * ((r >> 1) & 1) : 4 * (r & 3);
    }
    // Buffer offset of this lane's 16 bytes in copy ci (1 KiB of the region).  kNC: columns from `limit` on are not read.
    static __device__ __forceinline__ uint32_t voff(int ci, int lane, int ld, int limit)
    {
        const int r = ci * kRowsPerCopy + lane / kChunks;
        const int c = (lane % kChunks) ^ swizzle(r);
        const uint32_t v = static_cast<uint32_t>(r) * static_cast<uint32_t>(ld) * 2u + 16u * c;
        return kLayout == kKC || 8 * c < limit ? v : kOob;
    }
    // LDS addresses of this lane's fragment reads, from the region's start.  kKC: by sub-step of 16 k (block i of 32
    // rows: + 32 i rows).  kNC: by block (sub-step s, half h: + (16 s + 4 h) rows).
    static __device__ __forceinline__ uint32_t read_base(int lane, int i, int block0)
    {
        if constexpr (kLayout == kKC) {
            const int r = lane & 31;
            return (32 * block0 + r) * 128 + 16 * ((2 * i + (lane >> 5)) ^ swizzle(r));
        } else {
            const int g = lane >> 4, e = (lane >> 2) & 3, q = lane & 3;
            const int kr = 8 * (g >> 1) + e, col = 32 * (block0 + i) + 16 * (g & 1) + 4 * q;
            return kr * kRow + 16 * ((col >> 3) ^ swizzle(kr)) + 2 * (col & 7);
        }
    }
    static constexpr int bases(int blocks) { return kLayout == kKC ? 4 : blocks; }
};

// The kernel for one tile shape, operand layouts and epilogue.
template <class S, int kLA, int kLB, int kEpi, bool kF32>
struct Gemm {
    static constexpr bool kDual = kEpi != kEpiOut;
    static constexpr int BN = kDual ? S::BNB / 2 : S::BNB;               // output columns per tile
    using RA = Region<kLA, S::BM>;
    using RB = Region<kLB, BN>;                                          // one matrix's columns
    static constexpr int kNA = RA::bases(S::kTM), kNB = RB::bases(S::kTN);
    static constexpr int kReadsA = kLA == kKC ? 1 : 2, kReadsB = kLB == kKC ? 1 : 2;   // LDS reads per fragment
    static constexpr int kReads = S::kTM * kReadsA + S::kTN * kReadsB;
    static_assert(!kDual || kLB == kNC, "gated tiles take N-contiguous weights");

    struct Frags {
        bf16x8_t a[S::kTM], b[S::kTN];
        i16x4_t lo;
    };
    struct Lane {
        uint32_t a_voff[S::kAC], b_voff[S::kBC];
        uint32_t a_base[kNA], b_base[kNB];
        int k8[2];                       // kKC: the k of this lane's chunk, by the copy's parity
        uint32_t a_lds, b_lds;           // this wave's first copies in the stage being filled
        i32x4_t ra, rb;
    };

    template <int kLayout, class R, int kSub, int kHalf>
    static __device__ __forceinline__ void read_frag(bf16x8_t& f, i16x4_t& lo, uint32_t base)
    {
        if constexpr (kLayout == kKC) {
            f = *reinterpret_cast<const __attribute__((address_space(3))) bf16x8_t*>(base);
        } else {
            const i16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                reinterpret_cast<lds_i16x4_t*>(base + (16 * kSub + 4 * kHalf) * R::kRow));
            if constexpr (kHalf == 0)
                lo = v;
            else
                f = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, v, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }

    // Read Q of a sub-step, in the order the MFMAs take them: A block 0, the B blocks, the other A blocks.
    template <int kSub, int Q>
    static __device__ __forceinline__ void read_one(Frags& f, const Lane& ln)
    {
        constexpr int kB0 = kReadsA, kA1 = kReadsA + S::kTN * kReadsB;
        if constexpr (Q >= kB0 && Q < kA1) {
            constexpr int j = (Q - kB0) / kReadsB, h = (Q - kB0) % kReadsB;
            if constexpr (kLB == kKC)
                read_frag<kKC, RB, kSub, 0>(f.b[j], f.lo, ln.b_base[kSub] + j * 32 * 128);
            else
                read_frag<kNC, RB, kSub, h>(f.b[j], f.lo, ln.b_base[j]);
        } else {
            constexpr int q = Q < kB0 ? Q : Q - S::kTN * kReadsB;
            constexpr int i = q / kReadsA, h = q % kReadsA;
            if constexpr (kLA == kKC)
                read_frag<kKC, RA, kSub, 0>(f.a[i], f.lo, ln.a_base[kSub] + i * 32 * 128);
            else
                read_frag<kNC, RA, kSub, h>(f.a[i], f.lo, ln.a_base[i]);
        }
    }

    template <int kSub, int Q0, int... Is>
    static __device__ __forceinline__ void reads(std::integer_sequence<int, Is...>, Frags& f, const Lane& ln)
    {
        (read_one<kSub, Q0 + Is>(f, ln), ...);
    }

    // Copy C of a step: A's, then B's.  krem: K values left from the step's first one (kKC chunks past them read zero).
    template <int C>
    static __device__ __forceinline__ void copy_one(const Lane& ln, int krem)
    {
        if constexpr (C < S::kAC) {
            uint32_t v = ln.a_voff[C];
            if constexpr (kLA == kKC)
                v = ln.k8[C % 2] < krem ? v : kOob;
            copy16(ln.ra, v, ln.a_lds + C * 1024);
        } else {
            constexpr int j = C - S::kAC;
            uint32_t v = ln.b_voff[j];
            if constexpr (kLB == kKC)
                v = ln.k8[j % 2] < krem ? v : kOob;
            copy16(ln.rb, v, ln.b_lds + j * 1024);
        }
    }

    template <int C0, int... Is>
    static __device__ __forceinline__ void copies(std::integer_sequence<int, Is...>, const Lane& ln, int krem)
    {
        (copy_one<C0 + Is>(ln, krem), ...);
    }

    // MFMA M of a sub-step, then this slot's share of the fragment reads of sub-step kNext (over the first half of the
    // MFMAs, so that they have landed when the sub-step ends) and of the copies (over all of them).
    template <int kNext, bool kCopy, int M>
    static __device__ __forceinline__ void slot(f32x16_t (&acc)[S::kTM][S::kTN], const Frags& use, Frags& load,
                                                const Lane& ln, int krem)
    {
        constexpr int NM = S::kTM * S::kTN, RF = NM / 2, NC = kCopy ? S::kAC + S::kBC : 0;
        constexpr int i = M / S::kTN, j = M % S::kTN;
        // B as the first operand: the block is transposed, a lane holds one row of C and runs of four columns
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(use.b[j], use.a[i], acc[i][j], 0, 0, 0);
        if constexpr (M < RF)
            reads<kNext, M * kReads / RF>(std::make_integer_sequence<int, (M + 1) * kReads / RF - M * kReads / RF>{}, load, ln);
        copies<M * NC / NM>(std::make_integer_sequence<int, (M + 1) * NC / NM - M * NC / NM>{}, ln, krem);
        __builtin_amdgcn_sched_barrier(0);
    }

    template <int kNext, bool kCopy, int... Ms>
    static __device__ __forceinline__ void slots(std::integer_sequence<int, Ms...>, f32x16_t (&acc)[S::kTM][S::kTN],
                                                 const Frags& use, Frags& load, const Lane& ln, int krem)
    {
        __builtin_amdgcn_sched_barrier(0);
        (slot<kNext, kCopy, Ms>(acc, use, load, ln, krem), ...);
        __builtin_amdgcn_sched_barrier(0);
    }

    // The next step to copy: segment and first k.
    struct Feed {
        int seg, kk;
    };

    // Points the lane's buffer resources at step f (nothing is read past the last segment), returns the K values left.
    static __device__ __forceinline__ int aim(const GemmArgs& g, const Feed& f, Lane& ln, int m0, int n0, int mat)
    {
        const int seg = f.seg;
        const uint16_t* a = g.a + ((g.a_idx >> (4 * seg)) & 15) * g.a_plane;
        const int bi = static_cast<int>((g.b_idx >> (4 * seg)) & 15);
        const uint16_t* b = ((bi >> 3) ^ mat ? g.b1 : g.b0) + (bi & 7) * g.b_plane;
        const bool on = seg < g.nseg;
        // kKC: rows [m0, M) of lda values from kk on; kNC: rows [kk, K) from column m0 on
        const int64_t an = kLA == kKC ? min(S::BM, g.M - m0) : min(kBK, g.K - f.kk);
        const int64_t bn = kLB == kKC ? min(BN, g.N - n0) : min(kBK, g.K - f.kk);
        a += kLA == kKC ? static_cast<int64_t>(m0) * g.lda + f.kk : static_cast<int64_t>(f.kk) * g.lda + m0;
        b += kLB == kKC ? static_cast<int64_t>(n0) * g.ldb + f.kk : static_cast<int64_t>(f.kk) * g.ldb + n0;
        ln.ra = make_rsrc(a, on && an > 0 ? 2 * (an * g.lda - (kLA == kKC ? f.kk : m0)) : 0);
        ln.rb = make_rsrc(b, on && bn > 0 ? 2 * (bn * g.ldb - (kLB == kKC ? f.kk : n0)) : 0);
        return (kLA == kKC ? g.lda : g.ldb) - f.kk;
    }

    static __device__ __forceinline__ void advance(const GemmArgs& g, Feed& f)
    {
        f.kk += kBK;
        if (f.kk >= g.kt * kBK) {
            f.kk = 0;
            ++f.seg;
        }
    }

    // The sum of the tile's steps.
    static __device__ __forceinline__ void k_loop(const GemmArgs& g, f32x16_t (&acc)[S::kTM][S::kTN], int m0, int n0,
                                                  int mat0)
    {
        extern __shared__ __attribute__((aligned(256))) unsigned char smem[];
        const uint32_t lds0 = static_cast<uint32_t>(
            reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned char*)(smem)));
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int wm = wave / S::kWN, wn = wave % S::kWN;

        Lane ln;
        // in a gated tile the first half of the waves copies the gate columns, the others the up columns
        const int mat = kDual ? (wave >= S::kWaves / 2 ? 1 : 0) : mat0;
        const int ci_b = S::kBC * (kDual ? wave % (S::kWaves / 2) : wave);
#pragma unroll
        for (int j = 0; j < S::kAC; ++j)
            ln.a_voff[j] = RA::voff(S::kAC * wave + j, lane, g.lda, g.M - m0);
#pragma unroll
        for (int j = 0; j < S::kBC; ++j)
            ln.b_voff[j] = RB::voff(ci_b + j, lane, g.ldb, g.N - n0);
#pragma unroll
        for (int j = 0; j < 2; ++j)                        // the swizzle's row part: 8 j + lane / 8
            ln.k8[j] = 8 * ((lane & 7) ^ ((4 * j + (lane >> 4)) & 7));
        ln.a_lds = lds0 + S::kAC * wave * 1024;
        ln.b_lds = lds0 + S::kABytes + S::kBC * wave * 1024;
#pragma unroll
        for (int i = 0; i < kNA; ++i) {
            ln.a_base[i] = lds0 + RA::read_base(lane, i, wm * S::kTM);
            asm volatile("" : "+v"(ln.a_base[i]));
        }
#pragma unroll
        for (int i = 0; i < kNB; ++i) {
            // gated: block i is matrix i % 2, block (wn kTN + i) / 2 of its columns
            if constexpr (kDual)
                ln.b_base[i] = lds0 + S::kABytes + (i & 1) * RB::kBytes + RB::read_base(lane, 0, (wn * S::kTN + i) / 2);
            else
                ln.b_base[i] = lds0 + S::kABytes + RB::read_base(lane, i, wn * S::kTN);
            asm volatile("" : "+v"(ln.b_base[i]));
        }

        constexpr int kC = S::kAC + S::kBC;
        using AllCopies = std::make_integer_sequence<int, kC>;
        using AllMfmas = std::make_integer_sequence<int, S::kTM * S::kTN>;
        Feed f{0, 0};
        int krem = aim(g, f, ln, m0, n0, mat);
        copies<0>(AllCopies{}, ln, krem);
        advance(g, f);
        krem = aim(g, f, ln, m0, n0, mat);
        ln.a_lds += S::kStage;
        ln.b_lds += S::kStage;
        copies<0>(AllCopies{}, ln, krem);
        advance(g, f);
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" :: "n"(kC) : "memory");

        Frags f0, f1;
        reads<0, 0>(std::make_integer_sequence<int, kReads>{}, f0, ln);
        int delta = S::kStage;
        const int steps = g.nseg * g.kt;
        for (int t = 0; t < steps; ++t) {
            slots<1, false>(AllMfmas{}, acc, f0, f1, ln, 0);
            slots<2, false>(AllMfmas{}, acc, f1, f0, ln, 0);
            krem = aim(g, f, ln, m0, n0, mat);
            slots<3, false>(AllMfmas{}, acc, f0, f1, ln, 0);
            step_barrier();               // step t + 1 has landed, step t's stage is free
#pragma unroll
            for (int i = 0; i < kNA; ++i)
                ln.a_base[i] += delta;
#pragma unroll
            for (int i = 0; i < kNB; ++i)
                ln.b_base[i] += delta;
            ln.a_lds -= delta;
            ln.b_lds -= delta;
            slots<0, true>(AllMfmas{}, acc, f1, f0, ln, krem);
            advance(g, f);
            delta = -delta;
        }
        // the copies past the last step (of nothing, into LDS) end before the workgroup does
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    }
};

// act(g) and its slope.  silu and gelu's tanh form are g s(z) with the logistic function s: z = g, and
// z = 2 sqrt(2 / pi) (g + 0.044715 g^3) since (1 + tanh y) / 2 = s(2 y).  bfloat16 results take exponential and quotient
// from the hardware's 1-ulp units, float32 ones from the exact functions.
template <bool kF32>
__device__ __forceinline__ void activation(int act, float g, float& value, float& slope)
{
    if (act == MOE_ACT_GELU) {
        const float c = 0.5f * erfcf(-0.70710678118654752f * g);
        value = g * c;
        const float e = kF32 ? expf(-0.5f * g * g) : __builtin_amdgcn_exp2f(-0.72134752044448170f * g * g);
        slope = c + (e == 0.0f ? 0.0f : g * e * 0.39894228040143268f);
        return;
    }
    constexpr float kA = 1.5957691216057308f, kB = 0.044715f;
    const float z = act == MOE_ACT_SILU ? g : kA * (g + kB * g * g * g);
    const float dz = act == MOE_ACT_SILU ? 1.0f : kA * (1.0f + 3.0f * kB * g * g);
    float s, t;                                                // s(z) and 1 - s(z)
    if constexpr (kF32) {
        const float e = expf(-fabsf(z)), r = 1.0f / (1.0f + e);
        s = z < 0.0f ? e * r : r;
        t = z < 0.0f ? r : e * r;
    } else {
        const float e = __builtin_amdgcn_exp2f(-1.4426950408889634f * fabsf(z)), r = __builtin_amdgcn_rcpf(1.0f + e);
        s = z < 0.0f ? e * r : r;
        t = z < 0.0f ? r : e * r;
    }
    value = g * s;
    const float st = s * t;
    slope = s + (st == 0.0f ? 0.0f : g * st * dz);
}

// Eight values to the planes at p (one bfloat16 plane, rounded, or three); p aligned to 16 bytes.
template <bool kF32>
__device__ __forceinline__ void store_planes(uint16_t* p, int64_t plane, const float (&v)[8])
{
    if constexpr (kF32) {
        u32x4_t q[3];
        split8<3>(v, q);
#pragma unroll
        for (int i = 0; i < 3; ++i)
            *reinterpret_cast<u32x4_t*>(p + i * plane) = q[i];
    } else {
        *reinterpret_cast<u32x4_t*>(p) = pack8_bf16(v);
    }
}

template <bool kF32>
using Value = std::conditional_t<kF32, float, uint16_t>;

// h of eight columns from col on in one row (col < F), and g and u where they are kept.
template <bool kF32>
__device__ __forceinline__ void finish_gated(const GemmArgs& e, const DropKey& key, float (&g)[8], const float (&u)[8],
                                             int64_t row, int col)
{
    using T = Value<kF32>;
    const int n = e.N - col;
    const int64_t at = row * e.ldo + col;
    if (e.save_g != nullptr) {
        store8(static_cast<T*>(e.save_g) + at, g, n);
        store8(static_cast<T*>(e.save_u) + at, u, n);
    }
    float h[8], slope;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        activation<kF32>(e.act, g[i], h[i], slope);
        h[i] *= u[i];
    }
    if (e.drop.threshold != 0)
        drop8(h, e.drop, key, static_cast<uint32_t>(col >> 3), static_cast<uint32_t>(row));
    store8(static_cast<T*>(e.o0) + at, h, n);
}

// dg and du of eight columns; columns from N on (up to ldb) are written as zero, they pad the products' K.
template <bool kF32>
__device__ __forceinline__ void finish_gated_bwd(const GemmArgs& e, const DropKey& key, float (&g)[8], float (&u)[8],
                                                 int64_t row, int col)
{
    using T = Value<kF32>;
    const int n = e.N - col;
    float d[8];
    load8(d, static_cast<const T*>(e.dh) + row * e.ld_dh + col, n);
    if (e.drop.threshold != 0)
        drop8(d, e.drop, key, static_cast<uint32_t>(col >> 3), static_cast<uint32_t>(row));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float value, slope;
        activation<kF32>(e.act, g[i], value, slope);
        // a dropped place has no gradient whatever its g and u
        g[i] = d[i] == 0.0f || i >= n ? 0.0f : d[i] * u[i] * slope;
        u[i] = d[i] == 0.0f || i >= n ? 0.0f : d[i] * value;
    }
    constexpr int kPlanes = kF32 ? 3 : 1;
    uint16_t* const p = e.dgu + row * e.ldb + col;
    store_planes<kF32>(p, e.dgu_plane, g);
    store_planes<kF32>(p + kPlanes * e.dgu_plane, e.dgu_plane, u);
}

template <class S, int kLA, int kLB, int kEpi, bool kF32>
__global__ __launch_bounds__(S::kThreads, S::kBlocks) void gemm(GemmArgs g)
{
    using G = Gemm<S, kLA, kLB, kEpi, kF32>;
    // consecutive tiles go to one XCD (workgroup b runs on XCD b % 8), in groups of 8 row tiles, so that the
    // workgroups of an XCD share rows of A and columns of B in its L2
    const int cols = g.nt * g.mats, total = g.mt * cols;
    const int per = (total + kXcdCount - 1) / kXcdCount;
    const int t = static_cast<int>(blockIdx.x % kXcdCount) * per + static_cast<int>(blockIdx.x / kXcdCount);
    if (static_cast<int>(blockIdx.x / kXcdCount) >= per || t >= total)
        return;
    constexpr int kGroup = 8;
    const int band = t / (kGroup * cols), in_band = t - band * kGroup * cols;
    const int height = min(kGroup, g.mt - band * kGroup);
    const int m0 = (band * kGroup + in_band % height) * S::BM;
    const int ct = in_band / height;
    const int mat = ct >= g.nt ? 1 : 0;
    const int n0 = (ct - mat * g.nt) * G::BN;

    f32x16_t acc[S::kTM][S::kTN];
#pragma unroll
    for (int i = 0; i < S::kTM; ++i)
#pragma unroll
        for (int j = 0; j < S::kTN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                acc[i][j][r] = 0.0f;
    G::k_loop(g, acc, m0, n0, mat);

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / S::kWN, wn = wave % S::kWN;
    const DropKey key = drop_key(g.drop);
#pragma unroll
    for (int i = 0; i < S::kTM; ++i) {
        const int64_t row = m0 + 32 * (wm * S::kTM + i) + (lane & 31);
#pragma unroll
        for (int j = 0; j < S::kTN; j += G::kDual ? 2 : 1) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                __builtin_amdgcn_sched_barrier(0);   // not every block's values in registers at once
                const int block = wn * S::kTN + j;
                const int col = n0 + 32 * (G::kDual ? block / 2 : block) + 16 * p + 8 * (lane >> 5);
                float v[8], w[8];
                run8(acc[i][j], p, v);
                if constexpr (G::kDual)
                    run8(acc[i][j + 1], p, w);
                if (row >= g.M || col >= (kEpi == kEpiGatedBwd ? g.ldb : g.N))
                    continue;
                if constexpr (kEpi == kEpiGated)
                    finish_gated<kF32>(g, key, v, w, row, col);
                else if constexpr (kEpi == kEpiGatedBwd)
                    finish_gated_bwd<kF32>(g, key, v, w, row, col);
                else
                    store8(static_cast<Value<kF32>*>(mat ? g.o1 : g.o0) + row * g.ldo + col, v, g.N - col);
            }
        }
    }
}

// dg and du from the kept g and u.
template <bool kF32>
__global__ __launch_bounds__(256) void act_grad_kernel(GemmArgs e, Divisor groups, int n, int64_t row0)
{
    using T = Value<kF32>;
    const int at = blockIdx.x * 256 + threadIdx.x;
    if (at >= n)
        return;
    const int r = static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(at)) * groups.m) >> groups.shift);
    const int col = 8 * (at - r * groups.d);
    const int64_t row = row0 + r;
    float g[8], u[8];
    load8(g, static_cast<const T*>(e.save_g) + row * e.ldo + col, e.N - col);
    load8(u, static_cast<const T*>(e.save_u) + row * e.ldo + col, e.N - col);
    finish_gated_bwd<kF32>(e, drop_key(e.drop), g, u, row, col);
}

// A matrix [rows, cols] of any alignment as planes [rows, ld] of bfloat16, the columns from cols on zero.
template <bool kF32>
__global__ __launch_bounds__(256) void pack_kernel(const Value<kF32>* __restrict__ src, uint16_t* __restrict__ dst,
                                                   int64_t plane, Divisor groups, int n, int64_t row0, int cols, int ld)
{
    const int at = blockIdx.x * 256 + threadIdx.x;
    if (at >= n)
        return;
    const int r = static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(at)) * groups.m) >> groups.shift);
    const int col = 8 * (at - r * groups.d);
    const int64_t row = row0 + r;
    float v[8];
    load8(v, src + row * cols + col, cols - col);
    store_planes<kF32>(dst + row * ld + col, plane, v);
}

// Runs `launch(first row, groups of 8 columns, ...)` over rows of `groups` groups, below 2^31 groups a launch.
template <class F>
hipError_t for_groups(int64_t rows, int64_t groups, F launch)
{
    const int64_t step = ((int64_t{1} << 31) - 256) / groups;
    for (int64_t r = 0; r < rows; r += step) {
        const int n = static_cast<int>(std::min(step, rows - r) * groups);
        launch(r, n, dim3(static_cast<unsigned>(ceil_div(n, 256))));
        if (hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

// A matrix as the products take it: planes of bfloat16, rows of ld values.
struct Planes {
    const uint16_t* p;
    int64_t plane;
    int ld;
};

int planes_of(int dtype) { return dtype == MOE_F32 ? 3 : 1; }
int64_t padded(int64_t cols) { return (cols + 7) / 8 * 8; }
// Whether a matrix of that width has to be laid out anew.
bool needs_pack(int dtype, int64_t cols) { return dtype == MOE_F32 || cols % 8 != 0; }

hipError_t prepare(int dtype, const void* src, int64_t rows, int64_t cols, void* room, Planes& out, hipStream_t s)
{
    const int64_t ld = padded(cols);
    out = Planes{static_cast<const uint16_t*>(src), 0, static_cast<int>(ld)};
    if (!needs_pack(dtype, cols))
        return hipSuccess;
    uint16_t* const dst = static_cast<uint16_t*>(room);
    out = Planes{dst, rows * ld, static_cast<int>(ld)};
    const Divisor div = divisor(static_cast<int>(ld / 8));
    return for_groups(rows, ld / 8, [&](int64_t r, int n, dim3 grid) {
        if (dtype == MOE_F32)
            pack_kernel<true><<<grid, 256, 0, s>>>(static_cast<const float*>(src), dst, rows * ld, div, n, r,
                                                   static_cast<int>(cols), static_cast<int>(ld));
        else
            pack_kernel<false><<<grid, 256, 0, s>>>(static_cast<const uint16_t*>(src), dst, rows * ld, div, n, r,
                                                    static_cast<int>(cols), static_cast<int>(ld));
    });
}

using Small = Shape<2, 2, 2, 2, 2>;

template <class S, int kLA, int kLB, int kEpi, bool kF32>
hipError_t launch_shape(GemmArgs g, hipStream_t s)
{
    using G = Gemm<S, kLA, kLB, kEpi, kF32>;
    g.mt = static_cast<int>(ceil_div(g.M, S::BM));
    g.nt = static_cast<int>(ceil_div(kEpi == kEpiGatedBwd ? g.ldb : g.N, G::BN));
    const int64_t total = static_cast<int64_t>(g.mt) * g.nt * g.mats;
    gemm<S, kLA, kLB, kEpi, kF32><<<dim3(static_cast<unsigned>(ceil_div(total, kXcdCount) * kXcdCount)), S::kThreads,
                                    S::kSmem, s>>>(g);
    return hipGetLastError();
}

template <int kLA, int kLB, int kEpi>
hipError_t launch_gemm(const GemmArgs& g, int dtype, hipStream_t s)
{
    return dtype == MOE_F32 ? launch_shape<Small, kLA, kLB, kEpi, true>(g, s) : launch_shape<Small, kLA, kLB, kEpi, false>(g, s);
}

// The segments of a product of planes: one for bfloat16, six for float32, small products first.  a0, b0: added to the
// plane numbers (four bits each).
void add_segments(GemmArgs& g, int dtype, int a0, int b0)
{
    for (int i = dtype == MOE_F32 ? 0 : 5; i < 6; ++i) {
        g.a_idx |= static_cast<uint64_t>(a0 + kPlanePairs[i][0]) << (4 * g.nseg);
        g.b_idx |= static_cast<uint64_t>(b0 + kPlanePairs[i][1]) << (4 * g.nseg);
        ++g.nseg;
    }
}

// dx's two sums interleaved by size: the small products of both first.
void add_segments_pair(GemmArgs& g, int dtype, int a1)
{
    for (int i = dtype == MOE_F32 ? 0 : 5; i < 6; ++i)
        for (int m = 0; m < 2; ++m) {
            g.a_idx |= static_cast<uint64_t>(m * a1 + kPlanePairs[i][0]) << (4 * g.nseg);
            g.b_idx |= static_cast<uint64_t>(8 * m + kPlanePairs[i][1]) << (4 * g.nseg);
            ++g.nseg;
        }
}

}  // namespace

GatedLayout gated_layout(const moe_gated& g, bool backward)
{
    GatedLayout L;
    const int64_t P = planes_of(g.dtype);
    size_t off = 0;
    const auto take = [&](size_t& at, int64_t values) {
        at = off;
        off = align_up(off + static_cast<size_t>(values) * 2);
    };
    if (needs_pack(g.dtype, g.H))
        take(L.x, P * g.T * padded(g.H));
    if (needs_pack(g.dtype, g.F)) {
        take(L.wg, P * g.H * padded(g.F));
        take(L.wu, P * g.H * padded(g.F));
    }
    if (backward)
        take(L.dgu, 2 * P * g.T * padded(g.F));
    L.total = off;
    return L;
}

namespace {

// x and both weights laid out for the products.
hipError_t prepare_all(const moe_gated& q, const void* x, const void* wg, const void* wu, const GatedLayout& L,
                       unsigned char* ws, Planes& px, Planes& pg, Planes& pu, hipStream_t s)
{
    if (hipError_t e = prepare(q.dtype, x, q.T, q.H, ws + L.x, px, s); e != hipSuccess)
        return e;
    if (hipError_t e = prepare(q.dtype, wg, q.H, q.F, ws + L.wg, pg, s); e != hipSuccess)
        return e;
    return prepare(q.dtype, wu, q.H, q.F, ws + L.wu, pu, s);
}

GemmArgs forward_args(const moe_gated& q, const Dropout& d, const Planes& px, const Planes& pg, const Planes& pu)
{
    GemmArgs g{};
    g.a = px.p;
    g.b0 = pg.p;
    g.b1 = pu.p;
    g.a_plane = px.plane;
    g.b_plane = pg.plane;
    add_segments(g, q.dtype, 0, 0);
    g.kt = static_cast<int>(ceil_div(q.H, kBK));
    g.lda = px.ld;
    g.ldb = pg.ld;
    g.M = static_cast<int>(q.T);
    g.N = static_cast<int>(q.F);
    g.K = static_cast<int>(q.H);
    g.mats = 1;
    g.act = q.activation;
    g.drop = d;
    return g;
}

}  // namespace

hipError_t launch_gated(const moe_gated& q, const Dropout& d, const void* x, const void* wg, const void* wu, void* h,
                        void* saved_gu, void* workspace, hipStream_t s)
{
    const GatedLayout L = gated_layout(q, false);
    Planes px, pg, pu;
    if (hipError_t e = prepare_all(q, x, wg, wu, L, static_cast<unsigned char*>(workspace), px, pg, pu, s); e != hipSuccess)
        return e;
    const int64_t size = q.dtype == MOE_F32 ? 4 : 2;
    GemmArgs g = forward_args(q, d, px, pg, pu);
    g.o0 = h;
    g.ldo = static_cast<int>(q.F);
    g.save_g = saved_gu;
    g.save_u = saved_gu == nullptr ? nullptr : static_cast<unsigned char*>(saved_gu) + q.T * q.F * size;
    return launch_gemm<kKC, kNC, kEpiGated>(g, q.dtype, s);
}

hipError_t launch_gated_backward(const moe_gated& q, const Dropout& d, const void* x, const void* wg, const void* wu,
                                 const void* dh, const void* saved_gu, void* dx, void* dwg, void* dwu, void* workspace,
                                 hipStream_t s)
{
    const GatedLayout L = gated_layout(q, true);
    unsigned char* const ws = static_cast<unsigned char*>(workspace);
    Planes px, pg, pu;
    if (hipError_t e = prepare_all(q, x, wg, wu, L, ws, px, pg, pu, s); e != hipSuccess)
        return e;
    const int64_t size = q.dtype == MOE_F32 ? 4 : 2, ldf = padded(q.F);
    const int P = planes_of(q.dtype);
    uint16_t* const dgu = reinterpret_cast<uint16_t*>(ws + L.dgu);
    const int64_t dgu_plane = q.T * ldf;
    if (q.T > 0) {
        GemmArgs g = forward_args(q, d, px, pg, pu);
        g.ldb = static_cast<int>(ldf);
        g.dh = dh;
        g.ld_dh = static_cast<int>(q.F);
        g.dgu = dgu;
        g.dgu_plane = dgu_plane;
        if (saved_gu == nullptr) {
            if (hipError_t e = launch_gemm<kKC, kNC, kEpiGatedBwd>(g, q.dtype, s); e != hipSuccess)
                return e;
        } else {
            g.save_g = const_cast<void*>(saved_gu);
            g.save_u = const_cast<unsigned char*>(static_cast<const unsigned char*>(saved_gu)) + q.T * q.F * size;
            g.ldo = static_cast<int>(q.F);
            const Divisor div = divisor(static_cast<int>(ldf / 8));
            const hipError_t e = for_groups(q.T, ldf / 8, [&](int64_t r, int n, dim3 grid) {
                if (q.dtype == MOE_F32)
                    act_grad_kernel<true><<<grid, 256, 0, s>>>(g, div, n, r);
                else
                    act_grad_kernel<false><<<grid, 256, 0, s>>>(g, div, n, r);
            });
            if (e != hipSuccess)
                return e;
        }
        // dx [T, H]: K = F, the gate part, then the up part
        GemmArgs c{};
        c.a = dgu;
        c.a_plane = dgu_plane;
        c.b0 = pg.p;
        c.b1 = pu.p;
        c.b_plane = pg.plane;
        add_segments_pair(c, q.dtype, P);
        c.kt = static_cast<int>(ceil_div(ldf, kBK));
        c.lda = c.ldb = static_cast<int>(ldf);
        c.M = static_cast<int>(q.T);
        c.N = static_cast<int>(q.H);
        c.mats = 1;
        c.o0 = dx;
        c.ldo = static_cast<int>(q.H);
        if (hipError_t e = launch_gemm<kKC, kKC, kEpiOut>(c, q.dtype, s); e != hipSuccess)
            return e;
    }
    // dWg and dWu [H, F]: K = T
    GemmArgs w{};
    w.a = px.p;
    w.a_plane = px.plane;
    w.b0 = dgu;
    w.b1 = dgu + P * dgu_plane;
    w.b_plane = dgu_plane;
    add_segments(w, q.dtype, 0, 0);
    w.kt = static_cast<int>(ceil_div(q.T, kBK));
    w.lda = px.ld;
    w.ldb = static_cast<int>(ldf);
    w.M = static_cast<int>(q.H);
    w.N = static_cast<int>(q.F);
    w.K = static_cast<int>(q.T);
    w.mats = 2;
    w.o0 = dwg;
    w.o1 = dwu;
    w.ldo = static_cast<int>(q.F);
    return launch_gemm<kNC, kNC, kEpiOut>(w, q.dtype, s);
}

}  // namespace moe
