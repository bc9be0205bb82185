// lpcoll_dropout.cu -- residual_dropout without a norm, and the gradient of that:
//   x' = x + d(sum_r h_r)     dh = d(dx')
// with the mask made from the counters of lpcoll_philox.cuh both times.
//
// A lane takes 16 bytes of a row whatever the width of its accesses, so that it
// uses all words of the counters that it makes (two groups of four columns in
// BF16, one in FP32).
#include "lpcoll_layernorm.cuh"

namespace lpc {

namespace {

constexpr int kLanes = 256;  // of a CTA

// Lanes per row: rows share a CTA where they are short.
struct Rows {
    unsigned segs;      // CTAs of a row
    int lanes, per_cta;  // lanes of a row in a CTA, rows of a CTA
};

template <int DT, int W>
__global__ void __launch_bounds__(kLanes)
dropout_kernel(const __grid_constant__ LayerNormArgs a, const Rows rows)
{
    wait_prior_grid();
    constexpr int kN = Pack<DT, W>::kN;      // columns of an access
    constexpr int kCols = Fmt<DT>::kVec;     // of a lane
    constexpr int kPacks = kCols / kN;
    const int which = static_cast<int>(threadIdx.x) / rows.lanes;
    const int lane = static_cast<int>(threadIdx.x) - which * rows.lanes;
    const size_t t = static_cast<size_t>(blockIdx.x / rows.segs) * rows.per_cta + which;
    const size_t col = (static_cast<size_t>(blockIdx.x % rows.segs) * rows.lanes + lane) * kCols;
    if (t >= a.tokens || col >= static_cast<size_t>(a.hidden))
        return;
    const Philox rnd(a.drop, a.hidden);
    const size_t e0 = t * a.hidden + col;
    const auto has = [&](int i) { return W == 16 || col + i * kN < static_cast<size_t>(a.hidden); };
    Vec<kN> x[kPacks], h[kPacks];
#pragma unroll
    for (int i = 0; i < kPacks; ++i) {
        if (!has(i))
            continue;
        h[i] = load_vec_of<DT, W>(a.h[0], e0 + i * kN);
        if (a.x != nullptr)
            x[i] = load_vec_of<DT, W>(a.x, e0 + i * kN);
    }
#pragma unroll 4
    for (int r = 1; r < a.nranks; ++r)
#pragma unroll
        for (int i = 0; i < kPacks; ++i)
            if (has(i))
                h[i] = plus(h[i], load_vec_of<DT, W>(a.h[r], e0 + i * kN));
    uint32_t bits = 0;
    if (a.drop.least != 0) {
        const unsigned long long group = rnd.row(t) + col / 4;
#pragma unroll
        for (int q = 0; q < kCols / 4; ++q)
            bits |= rnd.keep4(group + q) << (q * 4);
    }
#pragma unroll
    for (int i = 0; i < kPacks; ++i) {
        if (!has(i))
            continue;
        if (a.dx != nullptr)  // gradient: of the residual, dx' itself
            store_vec_of<DT, W>(a.dx, e0 + i * kN, h[i]);
        if (a.x_out == nullptr)
            continue;
        Vec<kN> v = a.drop.least != 0 ? dropped(h[i], a.drop.scale, bits >> (i * kN)) : h[i];
        if (a.x != nullptr)
            v = plus(x[i], v);
        store_vec_of<DT, W>(a.x_out, e0 + i * kN, v);
    }
}

template <int DT, int W> cudaError_t dropout_dt(const LayerNormArgs &a, cudaStream_t st)
{
    const size_t lanes = (static_cast<size_t>(a.hidden) + Fmt<DT>::kVec - 1) / Fmt<DT>::kVec;
    Rows r;
    r.segs = static_cast<unsigned>((lanes + kLanes - 1) / kLanes);
    r.lanes = static_cast<int>((lanes + r.segs - 1) / r.segs);
    r.per_cta = kLanes / r.lanes;
    const size_t ctas = (a.tokens + r.per_cta - 1) / r.per_cta * r.segs;
    return launch_kernel_block(dropout_kernel<DT, W>, ctas, r.lanes * r.per_cta, 0, st, a, r);
}

}  // namespace

cudaError_t launch_dropout(const LayerNormArgs &a, cudaStream_t st)
{
    return LPC_BY_ROW(dropout_dt, a.dtype, static_cast<size_t>(a.hidden), a, st);
}

}  // namespace lpc
