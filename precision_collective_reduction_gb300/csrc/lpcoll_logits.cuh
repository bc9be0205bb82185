// lpcoll_logits.cuh -- a token's logits, one warp or part of one per token: what the router and
// the balance loss share. Internal linkage: each translation unit has its own.
#pragma once

#include "lpcoll_layers.cuh"

namespace lpc {

namespace {

// The PER experts of a lane come in runs of kRun consecutive ones, run r at
// (r * LANES + lane) * kRun for the LANES lanes of a token, so that a run is one
// access where rows of logits are a multiple of a run.
template <int DT, int PER> constexpr int kRun = PER < Fmt<DT>::kVec ? PER : Fmt<DT>::kVec;

template <int DT, int PER, int LANES = 32> __device__ __forceinline__ int expert_of(int i, int lane)
{
    constexpr int R = kRun<DT, PER>;
    return (i / R * LANES + lane) * R + i % R;
}

template <int BYTES> struct RunBytes;
template <> struct RunBytes<4> {
    using Raw = uint32_t;
};
template <> struct RunBytes<8> {
    using Raw = uint2;
};
template <> struct RunBytes<16> {
    using Raw = uint4;
};

// -infinity where there is no expert.
template <int DT, int PER, int LANES = 32>
__device__ __forceinline__ void load_logits(const void *logits, size_t t, int experts, int lane,
                                            float (&x)[PER])
{
    constexpr int R = kRun<DT, PER>;
    constexpr int kEs = kOne<DT>;
    using Raw = typename RunBytes<R * kEs>::Raw;
    const char *row = static_cast<const char *>(logits) + t * experts * kEs;
    if (experts % R == 0) {
#pragma unroll
        for (int r = 0; r < PER / R; ++r) {
            const int e = (r * LANES + lane) * R;
            typename Pack<DT, kEs>::Raw v[R];
            if (e < experts && LPC_READ_OK(row + e * kEs, R * kEs)) {
                const Raw raw = *reinterpret_cast<const Raw *>(row + e * kEs);
                memcpy(v, &raw, sizeof(raw));
            }
#pragma unroll
            for (int j = 0; j < R; ++j) {
                float one[1];
                widen_pack<DT, kEs>(v[j], one);
                x[r * R + j] = e < experts ? one[0] : -INFINITY;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = expert_of<DT, PER, LANES>(i, lane);
            float one[1] = {-INFINITY};
            if (e < experts)
                widen_pack<DT, kEs>(load_pack<DT, kEs>(row, e), one);
            x[i] = one[0];
        }
    }
}

}  // namespace

}  // namespace lpc
