// Counter-based dropout shared by the kernels that apply it: the mask is a function of the seed, the offset and
// the place (row, column) alone, so the forward, the backward and a recomputation draw it again instead of storing it.
//
// Philox 4x32 with 10 rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011):
// key = seed, counter = (column / 8, row, offset low, offset high); its 128 bits serve the 8 columns of the group, 16
// bits each, the low half of a word first.  A value is dropped where its 16 bits are below `threshold`.  16 bits per
// value (not 32) halve the rounds: one call is about 20 32-bit multiply pairs, which for 4 values a call would take
// as long as moving 4 bfloat16 values in and out of memory at 5.7 TB/s.
#pragma once

#include <stdint.h>

#include "shared_expert.h"
#include "vec8.h"

namespace moe {

// The key and the offset half of the counter, the same for every value of a call (rng may be null without dropout).
struct DropKey {
    uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ DropKey drop_key(const Dropout& d)
{
    if (d.threshold == 0)
        return DropKey{};
    const uint64_t seed = static_cast<uint64_t>(d.rng[0]), offset = static_cast<uint64_t>(d.rng[1]);
    return DropKey{static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32), static_cast<uint32_t>(offset),
                   static_cast<uint32_t>(offset >> 32)};
}

// The 8 x 16 bits of one group of columns.
__device__ __forceinline__ u32x4_t drop_bits(const DropKey& k, uint32_t group, uint32_t row)
{
    uint32_t c0 = group, c1 = row, c2 = k.o0, c3 = k.o1, k0 = k.k0, k1 = k.k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u, p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
        c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
        c1 = static_cast<uint32_t>(p1);
        c3 = static_cast<uint32_t>(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4_t{c0, c1, c2, c3};
}

// v[0 .. 7] of one group: kept values times the factor, dropped ones zero whatever they were (infinities and NaN too).
__device__ __forceinline__ void drop8(float (&v)[8], const Dropout& d, const DropKey& k, uint32_t group, uint32_t row)
{
    const u32x4_t bits = drop_bits(k, group, row);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = i % 2 == 0 ? bits[i / 2] & 0xFFFFu : bits[i / 2] >> 16;
        v[i] = b >= d.threshold ? v[i] * d.scale : 0.0f;
    }
}

}  // namespace moe
