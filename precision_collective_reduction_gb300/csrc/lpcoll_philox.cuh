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

// Made by whole warps.
struct Philox {
    uint32_t key0, key1, offset0, offset1, least;
    unsigned long long first_row, groups;

    // uniform: the offset kept out of the lanes' registers as well, and with it the first
    // round's product of it, which is the same for all counters. Norms of 8192 x 8192 BF16
    // 104 -> 100 us, their gradients 137 -> 134; the kernel without a norm, which is held
    // to 32 or 40 registers, spills more for it (FP32 59 -> 61). The second round's
    // too, made once a row for both upper words that the row's counters can have, takes the
    // registers of the norms' pipelines: 104 and 143 us.
    __device__ __forceinline__ Philox(const DropArgs &a, size_t hidden, bool uniform)
    {
        unsigned long long seed = 0, offset = 0;
        if (a.least != 0 && LPC_READ_OK(a.rng, 16)) {
            seed = a.rng[0];
            offset = a.rng[1];
        }
        // the same in every lane: said by a warp-wide OR, it keeps the rounds' keys out
        // of the lanes' registers
        key0 = __reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(seed));
        key1 = __reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(seed >> 32));
        offset0 = static_cast<uint32_t>(offset);
        offset1 = static_cast<uint32_t>(offset >> 32);
        if (uniform) {
            offset0 = __reduce_or_sync(0xFFFFFFFFu, offset0);
            offset1 = __reduce_or_sync(0xFFFFFFFFu, offset1);
        }
        least = a.least;
        first_row = a.first_row;
        groups = (hidden + 3) / 4;
    }
    // First group of row t.
    __device__ __forceinline__ unsigned long long row(size_t t) const
    {
        return (first_row + t) * groups;
    }
    // The words of N groups, round by round side by side: their keys are the same,
    // and one chain of products alone would wait for itself.
    template <int N>
    __device__ __forceinline__ void words(const unsigned long long (&group)[N],
                                          uint32_t (&w)[4 * N]) const
    {
        uint32_t k0 = key0, k1 = key1;
#pragma unroll
        for (int g = 0; g < N; ++g) {
            w[4 * g] = static_cast<uint32_t>(group[g]);
            w[4 * g + 1] = static_cast<uint32_t>(group[g] >> 32);
            w[4 * g + 2] = offset0;
            w[4 * g + 3] = offset1;
        }
#pragma unroll
        for (int i = 0; i < 10; ++i) {
#pragma unroll
            for (int g = 0; g < N; ++g) {
                uint32_t *const c = w + 4 * g;
                const unsigned long long a = static_cast<unsigned long long>(c[0]) * 0xD2511F53u;
                const unsigned long long b = static_cast<unsigned long long>(c[2]) * 0xCD9E8D57u;
                c[0] = static_cast<uint32_t>(b >> 32) ^ c[1] ^ k0;
                c[1] = static_cast<uint32_t>(b);
                c[2] = static_cast<uint32_t>(a >> 32) ^ c[3] ^ k1;
                c[3] = static_cast<uint32_t>(a);
            }
            k0 += 0x9E3779B9u;
            k1 += 0xBB67AE85u;
        }
    }
    // 0 where a column is dropped, whatever it holds.
    __device__ __forceinline__ float keep(float x, uint32_t word) const
    {
        return word >= least ? x : 0.0f;
    }
};

}  // namespace lpc
