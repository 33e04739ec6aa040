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
// bfloat16 operands go to v_mfma_f32_32x32x16_bf16 as they are, float32 operands as three bfloat16 planes (planes.h), all
// of them in one stage: the product of the first planes has a sum of its own, the five small ones share another.
#include <algorithm>
#include <utility>

#include "gated_epilogue.h"

namespace moe {
namespace {

enum Layout { kKC = 0, kNC = 1 };
constexpr uint32_t kOob = 0xC0000000u;          // a buffer offset past any num_records used here: reads as zero

// Tile shape: kWM x kWN waves, each kTM x kTN accumulator blocks of 32 x 32; kP planes of kBK values of K per stage,
// kStages of them in LDS.
template <int kWM_, int kWN_, int kTM_, int kTN_, int kBlocks_, int kBK_, int kP_, int kStages_>
struct Shape {
    static constexpr int kWM = kWM_, kWN = kWN_, kTM = kTM_, kTN = kTN_, kBlocks = kBlocks_, kBK = kBK_, kP = kP_;
    static constexpr int kStages = kStages_, kSubs = kBK / 16;         // sub-steps: one MFMA of 16 k deep
    static constexpr int kWaves = kWM * kWN, kThreads = kWaves * 64;
    static constexpr int BM = 32 * kWM * kTM, BNB = 32 * kWN * kTN;    // rows, staged columns of B
    static constexpr int kAPlane = BM * kBK * 2, kBPlane = BNB * kBK * 2;
    static constexpr int kABytes = kP * kAPlane, kStage = kABytes + kP * kBPlane, kSmem = kStages * kStage;
    static constexpr int kAC = kAPlane / 1024 / kWaves, kBC = kBPlane / 1024 / kWaves;   // 1 KiB copies per wave and plane
    static constexpr int kPairs = kP == 1 ? 1 : 6, kSums = kP == 1 ? 1 : 2;
    static constexpr int kMfmas = kPairs * kTM * kTN;                  // per wave and sub-step
    static_assert(kAC * kWaves * 1024 == kAPlane && kBC * kWaves * 1024 == kBPlane, "whole copies");
    static_assert(kAC % 2 == 0 && kBC % 2 == 0 && kWaves % 2 == 0 && kTN % 2 == 0 && kSubs % 2 == 0, "pairs");
    static_assert(kSmem * kBlocks <= 160 * 1024, "LDS of one CU");
};

struct GemmArgs {
    // segment s multiplies a[s] with b[s]; a gated tile's second columns, and the second half of the column tiles with
    // mats = 2, take the other of b
    const uint16_t *a[2], *b[2];
    int nseg, kt;                               // segments, steps of K per segment
    int lda, ldb;                               // values between rows, multiples of 8
    int a_plane, b_plane;                       // values between the planes of a row
    int M, N;                                   // rows, columns (of one matrix)
    int K, kc;                                  // the rows of a kNC operand, the values of a kKC operand's row (K, padded)
    int mt, nt, mats;                           // row tiles, column tiles (of one matrix), matrices of columns
    EpiArgs e;
};

__device__ __forceinline__ void copy16(const i32x4_t& rsrc, uint32_t voff, uint32_t soff, uint32_t lds)
{
    // LDS DMA of 16 bytes per lane through a buffer resource: lane i writes LDS byte lds + 16 i; offsets past the
    // resource's end read as zero.  Counts in vmcnt; the waits are explicit (step_barrier).
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :: "v"(voff), "s"(rsrc), "s"(soff), "s"(lds) : "memory");
}

// This wave's copies but the last kLater and its LDS reads are complete, then the workgroup's.
template <int kLater>
__device__ __forceinline__ void step_barrier()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(kLater) : "memory");
}

__device__ __forceinline__ i32x4_t make_rsrc(const uint16_t* p, int64_t bytes)
{
    const uint64_t q = reinterpret_cast<uint64_t>(p);
    return i32x4_t{__builtin_amdgcn_readfirstlane(static_cast<int>(q)),
                   __builtin_amdgcn_readfirstlane(static_cast<int>(q >> 32) & 0xFFFF),
                   __builtin_amdgcn_readfirstlane(static_cast<int>(bytes)), 0x00027000};
}

// One operand plane's share of an LDS stage: kCols rows (kKC) or columns (kNC) of kBK k.
//   kKC: row r is 128 (64) bytes, its 16-byte chunk c (8 k) lies at c ^ ((r >> 1) & 7) (c ^ ((r >> 2) & 3)): 16 rows'
//        reads of one chunk cover all 16 bank groups
//   kNC: k row kr is 2 kCols bytes, chunk c (8 columns) lies at c ^ swizzle(kr): the four k rows of a transposing read
//        land in four different 64-byte quarters of a 256-byte bank window
template <int kLayout, int kCols, int kBK>
struct Region {
    static_assert(kBK == 64 || kBK == 32, "rows of 8 or 4 chunks");
    static constexpr int kRow = kLayout == kKC ? 2 * kBK : 2 * kCols;
    static constexpr int kChunks = kRow / 16;
    static constexpr int kRowsPerCopy = 64 / kChunks;
    static constexpr int kBytes = kCols * kBK * 2;
    static_assert(kLayout == kKC || kChunks == 8 || kChunks == 16 || kChunks == 32, "swizzle");
    static __device__ __forceinline__ int swizzle(int r)
    {
        if constexpr (kLayout == kKC)
            return kBK == 64 ? (r >> 1) & 7 : (r >> 2) & 3;
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
            return (32 * block0 + r) * kRow + 16 * ((2 * i + (lane >> 5)) ^ swizzle(r));
        } else {
            const int g = lane >> 4, e = (lane >> 2) & 3, q = lane & 3;
            const int kr = 8 * (g >> 1) + e, col = 32 * (block0 + i) + 16 * (g & 1) + 4 * q;
            return kr * kRow + 16 * ((col >> 3) ^ swizzle(kr)) + 2 * (col & 7);
        }
    }
    static constexpr int bases(int blocks) { return kLayout == kKC ? kBK / 16 : blocks; }
    // The k of this lane's chunk in copy ci (kKC).
    static __device__ __forceinline__ int chunk_k(int ci, int lane)
    {
        return 8 * ((lane % kChunks) ^ swizzle(ci * kRowsPerCopy + lane / kChunks));
    }
};

// The kernel for one tile shape, operand layouts and epilogue.
template <class S, int kLA, int kLB, int kEpi>
struct Gemm {
    static constexpr bool kDual = kEpi != kEpiOut;
    static constexpr int kBK = S::kBK;
    static constexpr int BN = kDual ? S::BNB / 2 : S::BNB;               // output columns per tile
    using RA = Region<kLA, S::BM, kBK>;
    using RB = Region<kLB, BN, kBK>;                                     // one matrix's columns
    static constexpr int kNA = RA::bases(S::kTM), kNB = RB::bases(S::kTN);
    static constexpr int kReadsA = kLA == kKC ? 1 : 2, kReadsB = kLB == kKC ? 1 : 2;   // LDS reads per fragment
    static constexpr int kReadsPlane = S::kTM * kReadsA + S::kTN * kReadsB, kReads = S::kP * kReadsPlane;
    static constexpr int kC = S::kP * (S::kAC + S::kBC);                 // copies per wave and step
    static_assert(!kDual || kLB == kNC, "gated tiles take N-contiguous weights");
    static_assert((S::kStages - 1) * kC < 64, "vmcnt");

    struct Frags {
        bf16x8_t a[S::kP][S::kTM], b[S::kP][S::kTN];
        i16x4_t lo;
    };
    using Acc = f32x16_t[S::kSums][S::kTM][S::kTN];
    struct Lane {
        uint32_t a_voff[S::kAC], b_voff[S::kBC];
        uint32_t a_base[kNA], b_base[kNB];
        int k8[2];                       // kKC: the k of this lane's chunk, by the copy's parity
        uint32_t a_lds, b_lds;           // this wave's first copies in the stage being filled
        uint32_t a_plane, b_plane;       // bytes between planes
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

    // Read Q of a sub-step, plane by plane in the order the MFMAs take them: A block 0, the B blocks, the other A blocks.
    template <int kSub, int Q>
    static __device__ __forceinline__ void read_one(Frags& f, const Lane& ln)
    {
        constexpr int p = Q / kReadsPlane, Q1 = Q % kReadsPlane, kB0 = kReadsA, kA1 = kReadsA + S::kTN * kReadsB;
        if constexpr (Q1 >= kB0 && Q1 < kA1) {
            constexpr int j = (Q1 - kB0) / kReadsB, h = (Q1 - kB0) % kReadsB;
            if constexpr (kLB == kKC)
                read_frag<kKC, RB, kSub, 0>(f.b[p][j], f.lo, ln.b_base[kSub] + p * S::kBPlane + j * 32 * RB::kRow);
            else
                read_frag<kNC, RB, kSub, h>(f.b[p][j], f.lo, ln.b_base[j] + p * S::kBPlane);
        } else {
            constexpr int q = Q1 < kB0 ? Q1 : Q1 - S::kTN * kReadsB;
            constexpr int i = q / kReadsA, h = q % kReadsA;
            if constexpr (kLA == kKC)
                read_frag<kKC, RA, kSub, 0>(f.a[p][i], f.lo, ln.a_base[kSub] + p * S::kAPlane + i * 32 * RA::kRow);
            else
                read_frag<kNC, RA, kSub, h>(f.a[p][i], f.lo, ln.a_base[i] + p * S::kAPlane);
        }
    }

    template <int kSub, int Q0, int... Is>
    static __device__ __forceinline__ void reads(std::integer_sequence<int, Is...>, Frags& f, const Lane& ln)
    {
        (read_one<kSub, Q0 + Is>(f, ln), ...);
    }

    // Copy C of a step: A's planes, then B's.  krem: K values left from the step's first one (kKC chunks past them read
    // zero).
    template <int C>
    static __device__ __forceinline__ void copy_one(const Lane& ln, int krem)
    {
        if constexpr (C < S::kP * S::kAC) {
            constexpr int p = C / S::kAC, i = C % S::kAC;
            uint32_t v = ln.a_voff[i];
            if constexpr (kLA == kKC)
                v = ln.k8[i % 2] < krem ? v : kOob;
            copy16(ln.ra, v, p * ln.a_plane, ln.a_lds + p * S::kAPlane + i * 1024);
        } else {
            constexpr int p = (C - S::kP * S::kAC) / S::kBC, j = (C - S::kP * S::kAC) % S::kBC;
            uint32_t v = ln.b_voff[j];
            if constexpr (kLB == kKC)
                v = ln.k8[j % 2] < krem ? v : kOob;
            copy16(ln.rb, v, p * ln.b_plane, ln.b_lds + p * S::kBPlane + j * 1024);
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
    static __device__ __forceinline__ void slot(Acc& acc, const Frags& use, Frags& load, const Lane& ln, int krem)
    {
        constexpr int NM = S::kMfmas, RF = NM / 2, NC = kCopy ? kC : 0;
        constexpr int pair = M / (S::kTM * S::kTN), i = M / S::kTN % S::kTM, j = M % S::kTN;
        constexpr int pa = S::kP == 1 ? 0 : kPlanePairs[pair][0], pb = S::kP == 1 ? 0 : kPlanePairs[pair][1];
        f32x16_t& sum = acc[S::kP > 1 && pa + pb > 0 ? 1 : 0][i][j];
        // B as the first operand: the block is transposed, a lane holds one row of C and runs of four columns
        sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(use.b[pb][j], use.a[pa][i], sum, 0, 0, 0);
        if constexpr (M < RF)
            reads<kNext, M * kReads / RF>(std::make_integer_sequence<int, (M + 1) * kReads / RF - M * kReads / RF>{}, load, ln);
        copies<M * NC / NM>(std::make_integer_sequence<int, (M + 1) * NC / NM - M * NC / NM>{}, ln, krem);
        __builtin_amdgcn_sched_barrier(0);
    }

    template <int kNext, bool kCopy, int... Ms>
    static __device__ __forceinline__ void slots(std::integer_sequence<int, Ms...>, Acc& acc, const Frags& use, Frags& load,
                                                 const Lane& ln, int krem)
    {
        __builtin_amdgcn_sched_barrier(0);
        (slot<kNext, kCopy, Ms>(acc, use, load, ln, krem), ...);
        __builtin_amdgcn_sched_barrier(0);
    }

    // The next step to copy: segment, first k, and the steps left.
    struct Feed {
        int seg, kk, left;
    };

    // Points the lane's buffer resources at step f (nothing is read past the last step), returns the K values left.
    static __device__ __forceinline__ int aim(const GemmArgs& g, const Feed& f, Lane& ln, int m0, int n0, int mat)
    {
        const int seg = f.seg;
        const uint16_t* a = seg != 0 ? g.a[1] : g.a[0];
        const uint16_t* b = (seg ^ mat) & 1 ? g.b[1] : g.b[0];
        const bool on = f.left > 0;
        // kKC: rows [m0, M) of lda values from kk on; kNC: rows [kk, K) from column m0 on
        const int64_t an = kLA == kKC ? min(S::BM, g.M - m0) : min(kBK, g.K - f.kk);
        const int64_t bn = kLB == kKC ? min(BN, g.N - n0) : min(kBK, g.K - f.kk);
        a += kLA == kKC ? static_cast<int64_t>(m0) * g.lda + f.kk : static_cast<int64_t>(f.kk) * g.lda + m0;
        b += kLB == kKC ? static_cast<int64_t>(n0) * g.ldb + f.kk : static_cast<int64_t>(f.kk) * g.ldb + n0;
        ln.ra = make_rsrc(a, on && an > 0 ? 2 * (an * g.lda - (kLA == kKC ? f.kk : m0)) : 0);
        ln.rb = make_rsrc(b, on && bn > 0 ? 2 * (bn * g.ldb - (kLB == kKC ? f.kk : n0)) : 0);
        return g.kc - f.kk;
    }

    static __device__ __forceinline__ void advance(const GemmArgs& g, Feed& f)
    {
        --f.left;
        f.kk += kBK;
        if (f.kk >= g.kt * kBK) {
            f.kk = 0;
            ++f.seg;
        }
    }

    // Sub-steps kSub - 1 .. kSubs - 2 of a step with the reads of their successors; the last one's use is left.
    template <int kSub>
    static __device__ __forceinline__ void inner(Acc& acc, Frags& f0, Frags& f1, const Lane& ln)
    {
        using All = std::make_integer_sequence<int, S::kMfmas>;
        if constexpr (kSub < S::kSubs) {
            slots<kSub, false>(All{}, acc, kSub % 2 ? f0 : f1, kSub % 2 ? f1 : f0, ln, 0);
            inner<kSub + 1>(acc, f0, f1, ln);
        }
    }

    // The sum of the tile's steps [step0, step1).
    static __device__ __forceinline__ void k_loop(const GemmArgs& g, Acc& acc, int m0, int n0, int mat0, int step0, int step1)
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
        for (int j = 0; j < 2; ++j)                        // a wave's first copy has an even number
            ln.k8[j] = Region<kKC, S::BM, kBK>::chunk_k(j, lane);
        const uint32_t a_lds = lds0 + S::kAC * wave * 1024, b_lds = lds0 + S::kABytes + S::kBC * wave * 1024;
        ln.a_plane = 2 * static_cast<uint32_t>(g.a_plane);
        ln.b_plane = 2 * static_cast<uint32_t>(g.b_plane);
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

        using AllCopies = std::make_integer_sequence<int, kC>;
        using AllMfmas = std::make_integer_sequence<int, S::kMfmas>;
        Feed f{g.kt > 0 ? step0 / g.kt : 0, g.kt > 0 ? step0 % g.kt * kBK : 0, step1 - step0};
#pragma unroll
        for (int i = 0; i < S::kStages; ++i) {
            ln.a_lds = a_lds + i * S::kStage;
            ln.b_lds = b_lds + i * S::kStage;
            const int krem = aim(g, f, ln, m0, n0, mat);
            copies<0>(AllCopies{}, ln, krem);
            advance(g, f);
        }
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" :: "n"((S::kStages - 1) * kC) : "memory");

        Frags f0, f1;
        reads<0, 0>(std::make_integer_sequence<int, kReads>{}, f0, ln);
        int stage = 0;                    // the step's own; its successor's fragments come from the next one
        for (int t = step0; t < step1; ++t) {
            inner<1>(acc, f0, f1, ln);
            const int krem = aim(g, f, ln, m0, n0, mat);
            step_barrier<(S::kStages - 2) * kC>();         // step t + 1 has landed, step t's stage is free
            const int next = stage + 1 == S::kStages ? 0 : stage + 1, delta = (next - stage) * S::kStage;
#pragma unroll
            for (int i = 0; i < kNA; ++i)
                ln.a_base[i] += delta;
#pragma unroll
            for (int i = 0; i < kNB; ++i)
                ln.b_base[i] += delta;
            ln.a_lds = a_lds + stage * S::kStage;
            ln.b_lds = b_lds + stage * S::kStage;
            slots<0, true>(AllMfmas{}, acc, f1, f0, ln, krem);
            advance(g, f);
            stage = next;
        }
        // the copies past the last step (of nothing, into LDS) end before the workgroup does
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    }
};

// Workgroup `block` of one product.
template <class S, int kLA, int kLB, int kEpi>
__device__ __forceinline__ void gemm_block(const GemmArgs& g, unsigned block)
{
    using G = Gemm<S, kLA, kLB, kEpi>;
    // consecutive tiles go to one XCD (workgroup b runs on XCD b % 8), in groups of 8 row tiles, so that the
    // workgroups of an XCD share rows of A and columns of B in its L2
    const int cols = g.nt * g.mats, tiles = g.mt * cols, total = tiles * g.e.parts;
    const int per = (total + kXcdCount - 1) / kXcdCount;
    const int id = static_cast<int>(block % kXcdCount) * per + static_cast<int>(block / kXcdCount);
    if (id >= total)
        return;
    const int part = id / tiles, t = id - part * tiles;
    constexpr int kGroup = 8;
    const int band = t / (kGroup * cols), in_band = t - band * kGroup * cols;
    const int height = min(kGroup, g.mt - band * kGroup);
    const int m0 = (band * kGroup + in_band % height) * S::BM;
    const int ct = in_band / height;
    const int mat = ct >= g.nt ? 1 : 0;
    const int n0 = (ct - mat * g.nt) * G::BN;

    typename G::Acc acc;
#pragma unroll
    for (int q = 0; q < S::kSums; ++q)
#pragma unroll
        for (int i = 0; i < S::kTM; ++i)
#pragma unroll
            for (int j = 0; j < S::kTN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    acc[q][i][j][r] = 0.0f;
    const int64_t steps = static_cast<int64_t>(g.nseg) * g.kt;
    G::k_loop(g, acc, m0, n0, mat, static_cast<int>(steps * part / g.e.parts), static_cast<int>(steps * (part + 1) / g.e.parts));

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / S::kWN, wn = wave % S::kWN;
    const EpiArgs& e = g.e;
    const DropKey key = kEpi == kEpiOut ? DropKey{} : drop_key(e.drop);
    if constexpr (S::kSums == 2)
#pragma unroll
        for (int i = 0; i < S::kTM; ++i)
#pragma unroll
            for (int j = 0; j < S::kTN; ++j)
                acc[0][i][j] += acc[1][i][j];
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
                run8(acc[0][i][j], p, v);
                if constexpr (G::kDual)
                    run8(acc[0][i][j + 1], p, w);
                if (row >= g.M || col >= g.N)
                    continue;
                if (e.partial != nullptr) {
                    store8(partial_at(e, part, mat, row, col), v, 8);
                    if constexpr (G::kDual)
                        store8(partial_at(e, part, 1, row, col), w, 8);
                } else {
                    finish8<kEpi, (S::kP > 1)>(e, key, v, w, mat, row, col);
                }
            }
        }
    }
}

template <class S, int kLA, int kLB, int kEpi>
__global__ __launch_bounds__(S::kThreads, S::kBlocks) void gemm(GemmArgs g)
{
    gemm_block<S, kLA, kLB, kEpi>(g, blockIdx.x);
}

// dx (workgroups below `first`, a multiple of the XCDs) and the weights' gradients in one launch: neither waits for the
// other.
template <class S>
__global__ __launch_bounds__(S::kThreads, S::kBlocks) void gemm_pair(GemmArgs dx, GemmArgs dw, unsigned first)
{
    if (blockIdx.x < first)
        gemm_block<S, kKC, kKC, kEpiOut>(dx, blockIdx.x);
    else
        gemm_block<S, kNC, kNC, kEpiOut>(dw, blockIdx.x - first);
}

// dg and du from the kept g and u.
template <bool kF32>
__global__ __launch_bounds__(256) void act_grad_kernel(EpiArgs e, Divisor groups, int n, int64_t row0)
{
    using T = Value<kF32>;
    const int at = blockIdx.x * 256 + threadIdx.x;
    if (at >= n)
        return;
    const int r = static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(at)) * groups.m) >> groups.shift);
    const int col = 8 * (at - r * groups.d);
    const int64_t row = row0 + r;
    float g[8], u[8];
    load8(g, static_cast<const T*>(e.save_g) + row * e.N + col, e.N - col);
    load8(u, static_cast<const T*>(e.save_u) + row * e.N + col, e.N - col);
    finish_gated_bwd<kF32>(e, drop_key(e.drop), g, u, row, col);
}

// Matrices [rows, cols] of any alignment as bfloat16, the planes of a row one after the other, each one's columns from cols
// up to the next multiple of 8 zero; up to three matrices in one launch (blockIdx.y).
struct PackArgs {
    struct One {
        const void* src;
        uint16_t* dst;
        int plane;                                // values between the planes of a row
        Divisor groups;
        int n, cols, ld;                          // groups of 8 columns in all, columns, values between rows of dst
    } m[3];
    int64_t row0;
};
template <bool kF32>
__global__ __launch_bounds__(256) void pack_kernel(PackArgs g)
{
    const PackArgs::One& m = blockIdx.y == 0 ? g.m[0] : blockIdx.y == 1 ? g.m[1] : g.m[2];
    const int at = blockIdx.x * 256 + threadIdx.x;
    if (at >= m.n)
        return;
    const int r = static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(at)) * m.groups.m) >> m.groups.shift);
    const int col = 8 * (at - r * m.groups.d);
    const int64_t row = g.row0 + r;
    float v[8];
    load8(v, static_cast<const Value<kF32>*>(m.src) + row * m.cols + col, m.cols - col);
    store_planes<kF32>(m.dst + row * m.ld + col, m.plane, v);
}

// A matrix as the products take it: rows of ld values, the planes of a row `plane` values apart.
struct Planes {
    const uint16_t* p;
    int plane, ld;
};

int planes_of(int dtype) { return dtype == MOE_F32 ? 3 : 1; }
int64_t padded(int64_t cols) { return (cols + 7) / 8 * 8; }
// Values per plane of a row of what is laid out here: whole cache lines (rows that start inside one cost the copies of K
// up to a third: 512 x 1024 x 2056, two segments, 46 against 60 us).
int64_t own_plane(int64_t cols) { return (cols + 63) / 64 * 64; }
int64_t own_ld(int dtype, int64_t cols) { return planes_of(dtype) * own_plane(cols); }
// Whether a matrix of that width has to be laid out anew.
bool needs_pack(int dtype, int64_t cols) { return dtype == MOE_F32 || cols % 8 != 0; }

struct Source {
    const void* src;
    int64_t rows, cols;
    void* room;
};

// Lays out up to three matrices where their widths need it.
template <int kCount>
hipError_t prepare(int dtype, const Source (&in)[kCount], Planes* (&out)[kCount], hipStream_t s)
{
    int64_t first[3], most = 0, widest = 1;
    PackArgs a{};
    int count = 0;
    for (int i = 0; i < kCount; ++i) {
        const Source& q = in[i];
        *out[i] = Planes{static_cast<const uint16_t*>(q.src), 0, static_cast<int>(q.cols)};
        if (!needs_pack(dtype, q.cols))
            continue;
        const int ld = static_cast<int>(own_ld(dtype, q.cols)), plane = static_cast<int>(own_plane(q.cols));
        uint16_t* const dst = static_cast<uint16_t*>(q.room);
        *out[i] = Planes{dst, plane, ld};
        const int64_t groups = ceil_div(q.cols, 8);
        a.m[count] = PackArgs::One{q.src, dst, plane, divisor(static_cast<int>(groups)), 0, static_cast<int>(q.cols), ld};
        first[count++] = q.rows;
        most = std::max(most, q.rows);
        widest = std::max(widest, groups);
    }
    const int64_t step = ((int64_t{1} << 31) - 256) / widest;              // rows per launch: fewer than 2^31 groups
    for (int64_t r = 0; r < most; r += step) {
        int64_t threads = 0;
        a.row0 = r;
        for (int i = 0; i < count; ++i) {
            a.m[i].n = static_cast<int>(std::clamp<int64_t>(first[i] - r, 0, step) * a.m[i].groups.d);
            threads = std::max<int64_t>(threads, a.m[i].n);
        }
        const dim3 grid(static_cast<unsigned>(ceil_div(threads, 256)), count);
        if (dtype == MOE_F32)
            pack_kernel<true><<<grid, 256, 0, s>>>(a);
        else
            pack_kernel<false><<<grid, 256, 0, s>>>(a);
        if (hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

// bfloat16: large tiles of 256 x 256, 8 waves of 64 x 128, one workgroup per CU.  4096 tokens, H = 4096, F = 14336: the
// gated product 810-860 us, dx 740-770, dWg and dWu 790-835 (1.1-1.3 PF).  The matrix cores are busy 60-66% of the cycles
// at the 1.75-1.9 GHz that the chip's power leaves (2.5 GHz in short products), which is not all that holds dx back: the
// library's product of its operands takes 630-700.  Stages of 32 k, four or five of them, took 4-8%
// longer, other groupings of tiles, orders of the copies and wave priorities nothing off.
// Small ones of 128 x 128, 4 waves of 64 x 64, two workgroups per CU, for products that leave CUs without a large tile: LDS
// bounds them (16 KiB of fragments per 16 MFMAs); 4 stages of 32 k: the same times.
// float32: 128 x 128, 4 waves of 64 x 64, one.  A stage holds all planes, so six products come of the reads that one plane
// product takes twice: 1000 x 1001 x 1365 54 us with the products one after the other, 46 so; the matrix cores are busy
// 41-50% of the cycles of the CUs that have a tile.  Planes interleaved in memory, for longer runs: the same time.
using Large = Shape<4, 2, 2, 4, 1, 64, 1, 2>;
using Small = Shape<2, 2, 2, 2, 2, 64, 1, 2>;
using Float = Shape<2, 2, 2, 2, 1, 32, 3, 3>;

// Steps of a sum over K values.
int64_t steps_of(int dtype, int64_t K) { return ceil_div(K, dtype == MOE_F32 ? Float::kBK : Small::kBK); }
static_assert(Large::kBK == Small::kBK, "one K step for bfloat16");

// A product's size: M rows, N staged columns in all (both matrices'), steps of K.
struct Size {
    int64_t M, N, steps;
    int64_t small() const { return ceil_div(M, Small::BM) * ceil_div(N, Small::BNB); }
};
static_assert(Float::BM == Small::BM && Float::BNB == Small::BNB, "counted alike");

// How a product runs: its tiles, and into how many parts its steps are cut.
struct GemmPlan {
    bool large;
    int parts;
    double time;
};

// The times that decide, in us, are measured ones (4096 x 4096 x 28672 and 512 x 1024 x 4096): a step of a large tile 1.75;
// of a small one 0.7, or 1.05 for two that share a CU; of a float32 one 1.3; a workgroup's start and end 8 and 6.
constexpr int64_t kCus = 256;
int64_t slots_of(int dtype) { return dtype == MOE_F32 ? kCus : 2 * kCus; }
double step_time(int dtype, int64_t tiles) { return dtype == MOE_F32 ? 1.3 : tiles <= kCus ? 0.7 : 1.05; }
// Parts cost a launch of 4 and two passes of float32 sums at 3.5 TB/s, and give workgroups to CUs that had none: a product
// is cut only where all of its workgroups are resident at once, two together up to twice as many (22 x 2880 x 602, float32:
// 230 workgroups of one step beside 23 of 38).
double parts_time(const Size& z, int64_t parts)
{
    return parts == 1 ? 0.0 : 4.0 + static_cast<double>(8 * parts * z.M * z.N) / 3.5e6;
}
constexpr int64_t kParts[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16};

GemmPlan plan_gemm(int dtype, const Size& z)
{
    const int64_t large = ceil_div(z.M, Large::BM) * ceil_div(z.N, Large::BNB), small = z.small(), slots = slots_of(dtype);
    GemmPlan best{true, 1, 1e30};
    if (dtype != MOE_F32)
        best.time = static_cast<double>(ceil_div(large, kCus)) * (1.75 * static_cast<double>(z.steps) + 8.0);
    for (int64_t p : kParts) {
        if (p > 1 && (small * p > slots || z.steps < 3 * p))
            break;
        const int64_t tiles = small * p, rest = tiles % slots;
        const double rounds = step_time(dtype, slots) * static_cast<double>(tiles / slots) + (rest == 0 ? 0.0 : step_time(dtype, rest));
        const double t = rounds * static_cast<double>(ceil_div(z.steps, p)) + 6.0 * static_cast<double>(ceil_div(tiles, slots)) +
                         parts_time(z, p);
        if (t < best.time)
            best = GemmPlan{false, static_cast<int>(p), t};
    }
    return best;
}

// How dx and the weights' gradients run: both in one launch of small tiles, or one after the other (5 us between them).
struct PairPlan {
    bool together;
    GemmPlan dx, dw;
};
PairPlan plan_pair(int dtype, const Size& x, const Size& w)
{
    PairPlan best{false, plan_gemm(dtype, x), plan_gemm(dtype, w)};
    double time = dtype == MOE_F32 ? 1e30 : best.dx.time + 5.0 + best.dw.time;
    const int64_t slots = slots_of(dtype);
    for (int64_t p : kParts)
        for (int64_t q : kParts) {
            const int64_t tx = x.small() * p, tw = w.small() * q, tiles = tx + tw;
            if ((p > 1 && x.steps < 3 * p) || (q > 1 && w.steps < 3 * q) || (p * q > 1 && tiles > 2 * slots))
                break;
            const int64_t nx = ceil_div(x.steps, p), nw = ceil_div(w.steps, q);
            // a launch of more workgroups than are resident evens out but for its last ones
            const double steps = tiles <= slots ? static_cast<double>(std::max(nx, nw))
                                                : static_cast<double>(tx * nx + tw * nw) / static_cast<double>(slots) +
                                                      0.5 * static_cast<double>(std::max(nx, nw));
            const double t = step_time(dtype, tiles) * steps + 6.0 * static_cast<double>(ceil_div(tiles, slots)) +
                             parts_time(x, p) + parts_time(w, q);
            if (t < time) {
                time = t;
                best = PairPlan{true, {false, static_cast<int>(p), 0.0}, {false, static_cast<int>(q), 0.0}};
            }
        }
    return best;
}

// Bytes of a product's partial sums.
int64_t partial_bytes(const Size& z, int parts) { return parts > 1 ? int64_t{4} * parts * z.M * z.N : 0; }

// The rest of a product's arguments, by its plan.
void set_plan(GemmArgs& g, const GemmPlan& plan, float* partial)
{
    g.e.M = g.M;
    g.e.N = g.N;
    g.e.mats = g.mats;
    g.e.parts = plan.parts;
    g.e.partial = plan.parts > 1 ? partial : nullptr;
    g.e.ld_part = static_cast<int>(padded(g.N));
}

// Tiles of shape S, BN output columns each; returns the workgroups.
template <class S>
int64_t set_tiles(GemmArgs& g, int BN)
{
    g.mt = static_cast<int>(ceil_div(g.M, S::BM));
    g.nt = static_cast<int>(ceil_div(g.N, BN));
    return ceil_div(static_cast<int64_t>(g.mt) * g.nt * g.mats * g.e.parts, kXcdCount) * kXcdCount;
}

// A gated product's two matrices are columns of one tile.
template <class S, int kLA, int kLB, int kEpi>
hipError_t launch_shape(GemmArgs g, hipStream_t s)
{
    using G = Gemm<S, kLA, kLB, kEpi>;
    static LdsLimit limit;
    if (hipError_t e = limit.ensure(reinterpret_cast<const void*>(&gemm<S, kLA, kLB, kEpi>), S::kSmem); e != hipSuccess)
        return e;
    if (G::kDual)
        g.mats = 1;
    const int64_t blocks = set_tiles<S>(g, G::BN);
    gemm<S, kLA, kLB, kEpi><<<dim3(static_cast<unsigned>(blocks)), S::kThreads, S::kSmem, s>>>(g);
    return hipGetLastError();
}

// Parts of K leave their sums; a second launch makes the results of them.
hipError_t finish_parts(Epi epi, int dtype, const GemmArgs& g, hipStream_t s)
{
    return g.e.parts == 1 ? hipSuccess : launch_gated_finish(epi, dtype, g.e, s);
}

// A product by its plan (float32 gradients run together, launch_pair).
template <int kLA, int kLB, int kEpi>
hipError_t launch_gemm(GemmArgs g, int dtype, const GemmPlan& plan, float* partial, hipStream_t s)
{
    if (g.M == 0)
        return hipSuccess;
    set_plan(g, plan, partial);
    hipError_t e = hipSuccess;
    if (plan.large)
        e = launch_shape<Large, kLA, kLB, kEpi>(g, s);
    else if (dtype != MOE_F32)
        e = launch_shape<Small, kLA, kLB, kEpi>(g, s);
    else if constexpr (kEpi != kEpiOut)
        e = launch_shape<Float, kLA, kLB, kEpi>(g, s);
    return e != hipSuccess ? e : finish_parts(static_cast<Epi>(kEpi), dtype, g, s);
}

template <class S>
hipError_t launch_together(GemmArgs& dx, GemmArgs& dw, hipStream_t s)
{
    static LdsLimit limit;
    if (hipError_t e = limit.ensure(reinterpret_cast<const void*>(&gemm_pair<S>), S::kSmem); e != hipSuccess)
        return e;
    const int64_t first = set_tiles<S>(dx, S::BNB), rest = set_tiles<S>(dw, S::BNB);
    gemm_pair<S><<<dim3(static_cast<unsigned>(first + rest)), S::kThreads, S::kSmem, s>>>(dx, dw, static_cast<unsigned>(first));
    return hipGetLastError();
}

// dx and the weights' gradients by their plan.
hipError_t launch_pair(GemmArgs& dx, GemmArgs& dw, int dtype, const PairPlan& plan, float* partial, int64_t dx_bytes,
                       hipStream_t s)
{
    float* const dw_partial = partial + dx_bytes / 4;
    if (!plan.together) {
        const hipError_t e = launch_gemm<kKC, kKC, kEpiOut>(dx, dtype, plan.dx, partial, s);
        return e != hipSuccess ? e : launch_gemm<kNC, kNC, kEpiOut>(dw, dtype, plan.dw, dw_partial, s);
    }
    set_plan(dx, plan.dx, partial);
    set_plan(dw, plan.dw, dw_partial);
    hipError_t e = dtype == MOE_F32 ? launch_together<Float>(dx, dw, s) : launch_together<Small>(dx, dw, s);
    if (e == hipSuccess)
        e = finish_parts(kEpiOut, dtype, dx, s);
    return e != hipSuccess ? e : finish_parts(kEpiOut, dtype, dw, s);
}

// The products of a call.
Size size_gu(const moe_gated& g) { return {g.T, 2 * padded(g.F), steps_of(g.dtype, g.H)}; }
Size size_dx(const moe_gated& g) { return {g.T, padded(g.H), 2 * steps_of(g.dtype, g.F)}; }
Size size_dw(const moe_gated& g) { return {g.H, 2 * padded(g.F), steps_of(g.dtype, g.T)}; }
PairPlan plan_backward(const moe_gated& g) { return plan_pair(g.dtype, size_dx(g), size_dw(g)); }

// Whether g and u come from the kernels for few rows.
bool few_rows(const moe_gated& g) { return g.T <= kMaxRows && g.F >= kMinCols; }

}  // namespace

GatedLayout gated_layout(const moe_gated& g, bool backward)
{
    GatedLayout L;
    size_t off = 0;
    const auto take = [&](size_t& at, int64_t bytes) {
        at = off;
        off = align_up(off + static_cast<size_t>(bytes));
    };
    const bool rows = few_rows(g);                  // the forward product takes its operands as they are
    if (needs_pack(g.dtype, g.H) && (backward || !rows))
        take(L.x, 2 * g.T * own_ld(g.dtype, g.H));
    if (needs_pack(g.dtype, g.F) && (backward || !rows)) {
        take(L.wg, 2 * g.H * own_ld(g.dtype, g.F));
        take(L.wu, 2 * g.H * own_ld(g.dtype, g.F));
    }
    if (backward)
        take(L.dgu, 2 * 2 * g.T * own_ld(g.dtype, g.F));
    int64_t partial = 0;                                  // of one product after the other
    if (g.T > 0) {
        const int64_t parts = rows ? gated_rows_parts(g.dtype, g.T, g.H, g.F) : 1;
        partial = rows ? parts > 1 ? 4 * 2 * parts * g.T * padded(g.F) : 0
                       : partial_bytes(size_gu(g), plan_gemm(g.dtype, size_gu(g)).parts);
    }
    if (backward) {
        const PairPlan p = plan_backward(g);
        L.dx_partial = partial_bytes(size_dx(g), p.dx.parts);
        partial = std::max(partial, L.dx_partial + partial_bytes(size_dw(g), p.dw.parts));
    }
    take(L.partial, partial);
    L.total = off;
    return L;
}

namespace {

struct Prepared {
    Planes x, wg, wu;
};

// x and both weights laid out for the products.
hipError_t prepare_all(const moe_gated& q, const void* x, const void* wg, const void* wu, const GatedLayout& L,
                       unsigned char* ws, Prepared& p, hipStream_t s)
{
    const Source in[3] = {{x, q.T, q.H, ws + L.x}, {wg, q.H, q.F, ws + L.wg}, {wu, q.H, q.F, ws + L.wu}};
    Planes* out[3] = {&p.x, &p.wg, &p.wu};
    return prepare(q.dtype, in, out, s);
}

// g and u of all rows with epilogue kEpi (kEpiGated or kEpiGatedBwd); p is not read for few rows.
template <int kEpi>
hipError_t launch_gu(const moe_gated& q, const void* x, const void* wg, const void* wu, const Prepared& p, EpiArgs e,
                     float* partial, hipStream_t s)
{
    e.M = static_cast<int>(q.T);
    e.N = static_cast<int>(q.F);
    e.mats = 2;
    e.act = q.activation;
    if (few_rows(q)) {
        e.parts = gated_rows_parts(q.dtype, q.T, q.H, q.F);
        e.partial = e.parts > 1 ? partial : nullptr;
        e.ld_part = static_cast<int>(padded(q.F));
        const hipError_t err = launch_gated_rows(static_cast<Epi>(kEpi), q.dtype, RowsArgs{x, wg, wu, static_cast<int>(q.H), e}, s);
        return err != hipSuccess || e.parts == 1 ? err : launch_gated_finish(static_cast<Epi>(kEpi), q.dtype, e, s);
    }
    GemmArgs g{};
    g.a[0] = p.x.p;
    g.b[0] = p.wg.p;
    g.b[1] = p.wu.p;
    g.a_plane = p.x.plane;
    g.b_plane = p.wg.plane;
    g.nseg = 1;
    g.kt = static_cast<int>(steps_of(q.dtype, q.H));
    g.lda = p.x.ld;
    g.ldb = p.wg.ld;
    g.M = static_cast<int>(q.T);
    g.N = static_cast<int>(q.F);
    g.K = static_cast<int>(q.H);
    g.kc = static_cast<int>(padded(q.H));
    g.mats = 2;
    g.e = e;
    return launch_gemm<kKC, kNC, kEpi>(g, q.dtype, plan_gemm(q.dtype, size_gu(q)), partial, s);
}

}  // namespace

hipError_t launch_gated(const moe_gated& q, const Dropout& d, const void* x, const void* wg, const void* wu, void* h,
                        void* saved_gu, void* workspace, hipStream_t s)
{
    const GatedLayout L = gated_layout(q, false);
    unsigned char* const ws = static_cast<unsigned char*>(workspace);
    Prepared p{};
    if (!few_rows(q))
        if (hipError_t e = prepare_all(q, x, wg, wu, L, ws, p, s); e != hipSuccess)
            return e;
    const int64_t size = q.dtype == MOE_F32 ? 4 : 2;
    EpiArgs e{};
    e.o0 = h;
    e.save_g = saved_gu;
    e.save_u = saved_gu == nullptr ? nullptr : static_cast<unsigned char*>(saved_gu) + q.T * q.F * size;
    e.drop = d;
    return launch_gu<kEpiGated>(q, x, wg, wu, p, e, reinterpret_cast<float*>(ws + L.partial), s);
}

hipError_t launch_gated_backward(const moe_gated& q, const Dropout& d, const void* x, const void* wg, const void* wu,
                                 const void* dh, const void* saved_gu, void* dx, void* dwg, void* dwu, void* workspace,
                                 hipStream_t s)
{
    const GatedLayout L = gated_layout(q, true);
    unsigned char* const ws = static_cast<unsigned char*>(workspace);
    Prepared p{};
    if (q.T > 0)                                          // without tokens x and the weights may be null
        if (hipError_t e = prepare_all(q, x, wg, wu, L, ws, p, s); e != hipSuccess)
            return e;
    const int64_t size = q.dtype == MOE_F32 ? 4 : 2, ldf = own_ld(q.dtype, q.F);
    float* const partial = reinterpret_cast<float*>(ws + L.partial);
    uint16_t* const dg = reinterpret_cast<uint16_t*>(ws + L.dgu);
    uint16_t* const du = dg + q.T * ldf;
    const int plane = static_cast<int>(own_plane(q.F));
    if (q.T > 0) {
        EpiArgs e{};
        e.dh = dh;
        e.dg = dg;
        e.du = du;
        e.d_plane = plane;
        e.ld_d = static_cast<int>(ldf);
        e.drop = d;
        if (saved_gu == nullptr) {
            if (hipError_t err = launch_gu<kEpiGatedBwd>(q, x, wg, wu, p, e, partial, s);
                err != hipSuccess)
                return err;
        } else {
            e.M = static_cast<int>(q.T);
            e.N = static_cast<int>(q.F);
            e.act = q.activation;
            e.save_g = const_cast<void*>(saved_gu);
            e.save_u = static_cast<unsigned char*>(e.save_g) + q.T * q.F * size;
            const Divisor div = divisor(static_cast<int>(ceil_div(q.F, 8)));
            const hipError_t err = for_groups(q.T, ceil_div(q.F, 8), [&](int64_t r, int n, unsigned grid) {
                if (q.dtype == MOE_F32)
                    act_grad_kernel<true><<<grid, 256, 0, s>>>(e, div, n, r);
                else
                    act_grad_kernel<false><<<grid, 256, 0, s>>>(e, div, n, r);
            });
            if (err != hipSuccess)
                return err;
        }
    }
    // dx [T, H]: K = F, the gate part, then the up part
    GemmArgs c{};
    c.a[0] = dg;
    c.a[1] = du;
    c.a_plane = plane;
    c.b[0] = p.wg.p;
    c.b[1] = p.wu.p;
    c.b_plane = p.wg.plane;
    c.nseg = 2;
    c.kt = static_cast<int>(steps_of(q.dtype, q.F));
    c.kc = static_cast<int>(padded(q.F));
    c.lda = static_cast<int>(ldf);
    c.ldb = p.wg.ld;
    c.M = static_cast<int>(q.T);
    c.N = static_cast<int>(q.H);
    c.mats = 1;
    c.e.o0 = dx;
    // dWg and dWu [H, F]: K = T
    GemmArgs w{};
    w.a[0] = p.x.p;
    w.a_plane = p.x.plane;
    w.b[0] = dg;
    w.b[1] = du;
    w.b_plane = plane;
    w.nseg = 1;
    w.kt = static_cast<int>(steps_of(q.dtype, q.T));
    w.lda = p.x.ld;
    w.ldb = static_cast<int>(ldf);
    w.M = static_cast<int>(q.H);
    w.N = static_cast<int>(q.F);
    w.K = static_cast<int>(q.T);
    w.mats = 2;
    w.e.o0 = dwg;
    w.e.o1 = dwu;
    return launch_pair(c, w, q.dtype, plan_backward(q), partial, L.dx_partial, s);
}

}  // namespace moe
