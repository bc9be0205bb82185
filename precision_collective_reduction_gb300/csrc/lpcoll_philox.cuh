// lpcoll_philox.cuh -- dropout's random words: Philox4x32 with 10 rounds (J. K.
// Salmon, M. A. Moraes, R. O. Dror, D. E. Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC 2011), a counter-based generator, so that the gradient
// makes the forward pass's words again instead of reading a mask.
//
// A counter gives the words of four neighbouring columns. Its first 64 bits
// count the groups of four, ceil(hidden / 4) in a row, so that a group never
// spans rows and any part of the rows can be made alone; the others are the
// caller's offset. An element is kept if its word is not below p 2^32.
#pragma once

#include "lpcoll_layers.cuh"

namespace lpc {

struct Philox {
    uint32_t key0, key1, offset0, offset1, least;
    unsigned long long first_row, groups;

    __device__ __forceinline__ Philox(const DropArgs &a, size_t hidden)
    {
        unsigned long long seed = 0, offset = 0;
        if (a.least != 0 && LPC_READ_OK(a.rng, 16)) {
            seed = a.rng[0];
            offset = a.rng[1];
        }
        key0 = static_cast<uint32_t>(seed);
        key1 = static_cast<uint32_t>(seed >> 32);
        offset0 = static_cast<uint32_t>(offset);
        offset1 = static_cast<uint32_t>(offset >> 32);
        least = a.least;
        first_row = a.first_row;
        groups = (hidden + 3) / 4;
    }
    // First group of row t.
    __device__ __forceinline__ unsigned long long row(size_t t) const
    {
        return (first_row + t) * groups;
    }
    // Bit j: column j of the group is kept.
    __device__ __forceinline__ uint32_t keep4(unsigned long long group) const
    {
        uint32_t c0 = static_cast<uint32_t>(group), c1 = static_cast<uint32_t>(group >> 32);
        uint32_t c2 = offset0, c3 = offset1, k0 = key0, k1 = key1;
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const unsigned long long a = static_cast<unsigned long long>(c0) * 0xD2511F53u;
            const unsigned long long b = static_cast<unsigned long long>(c2) * 0xCD9E8D57u;
            c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
            c1 = static_cast<uint32_t>(b);
            c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
            c3 = static_cast<uint32_t>(a);
            k0 += 0x9E3779B9u;
            k1 += 0xBB67AE85u;
        }
        return (c0 >= least ? 1u : 0u) | (c1 >= least ? 2u : 0u) | (c2 >= least ? 4u : 0u) |
               (c3 >= least ? 8u : 0u);
    }
};

}  // namespace lpc
