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
#ifndef DR_A
#define DR_A 1
#endif
#ifndef DR_C
#define DR_C 6
#endif
constexpr int kAhead = DR_A;    // pieces that a lane has in flight

// How rows are dealt out: `lanes` lanes of each of `segs` CTAs go through a row in
// pieces of 16 bytes, `pieces` of them; short rows share a CTA, `rows` of them.
struct Cut {
    unsigned segs, pieces;
    int lanes, rows;
};

template <int DT, int W>
__global__ void __launch_bounds__(kLanes, DR_C)
dropout_kernel(const __grid_constant__ LayerNormArgs a, const Cut cut)
{
    wait_prior_grid();
    constexpr int kN = Pack<DT, W>::kN;   // columns of an access
    constexpr int kCols = Fmt<DT>::kVec;  // of a piece
    constexpr int kPacks = kCols / kN;
    constexpr int kGroups = kCols / 4;
    size_t t = blockIdx.x;
    unsigned piece = threadIdx.x;
    if (cut.segs > 1) {
        t = blockIdx.x / cut.segs;
        piece += blockIdx.x % cut.segs * cut.lanes;
    } else if (cut.rows > 1) {
        const unsigned which = threadIdx.x / cut.lanes;
        t = t * cut.rows + which;
        piece -= which * cut.lanes;
    }
    const Philox rnd(a.drop, a.hidden);
    if (t >= a.tokens || (cut.segs == 1 && threadIdx.x >= static_cast<unsigned>(cut.lanes * cut.rows)))
        return;
    const unsigned step = cut.segs * cut.lanes;
    const unsigned long long row = rnd.row(t);
    const size_t e0 = t * a.hidden;
    const bool drop = a.drop.least != 0;
    for (; piece < cut.pieces; piece += kAhead * step) {
        Vec<kN> h[kAhead][kPacks], x[kAhead][kPacks];
        const auto col = [&](int u, int i) { return (piece + u * step) * kCols + i * kN; };
        const auto has = [&](int u, int i) {
            return W == 16 ? (u == 0 || piece + u * step < cut.pieces)
                           : col(u, i) < static_cast<unsigned>(a.hidden);
        };
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int i = 0; i < kPacks; ++i)
                if (has(u, i)) {
                    h[u][i] = load_vec_of<DT, W>(a.h[0], e0 + col(u, i));
                    if (a.x != nullptr)
                        x[u][i] = load_vec_of<DT, W>(a.x, e0 + col(u, i));
                }
#pragma unroll 4
        for (int r = 1; r < a.nranks; ++r)
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
#pragma unroll
                for (int i = 0; i < kPacks; ++i)
                    if (has(u, i))
                        h[u][i] = plus(h[u][i], load_vec_of<DT, W>(a.h[r], e0 + col(u, i)));
        uint32_t word[kAhead * kCols];
        if (drop) {
            unsigned long long group[kAhead * kGroups];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
#pragma unroll
                for (int q = 0; q < kGroups; ++q)
                    group[u * kGroups + q] = row + (piece + u * step) * kGroups + q;
            rnd.words(group, word);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int i = 0; i < kPacks; ++i) {
                if (!has(u, i))
                    continue;
                Vec<kN> v = h[u][i];
                if (a.dx != nullptr)  // gradient: of the residual, dx' itself
                    store_vec_of<DT, W>(a.dx, e0 + col(u, i), v);
                if (a.x_out == nullptr)
                    continue;
                if (drop) {
                    v = mul(a.drop.scale, v);
#pragma unroll
                    for (int j = 0; j < kN; ++j)
                        v.v[j] = rnd.keep(v.v[j], word[u * kCols + i * kN + j]);
                }
                if (a.x != nullptr)
                    v = plus(x[u][i], v);
                store_vec_of<DT, W>(a.x_out, e0 + col(u, i), v);
            }
    }
}

// A row's lanes have kAhead pieces or more; where there are few rows, more CTAs
// share one and its lanes have one piece.
template <int DT, int W> cudaError_t dropout_dt(const LayerNormArgs &a, cudaStream_t st)
{
    const size_t pieces = (a.hidden + Fmt<DT>::kVec - 1) / Fmt<DT>::kVec;
    Cut c;
    c.pieces = static_cast<unsigned>(pieces);
    const bool few = a.tokens * pieces < static_cast<size_t>(kSms) * 4 * kLanes * kAhead;
    const size_t lanes = few ? pieces : (pieces + kAhead - 1) / kAhead;
    c.segs = few ? static_cast<unsigned>((pieces + kLanes - 1) / kLanes) : 1;
    c.lanes = static_cast<int>(lanes < kLanes ? lanes : kLanes);
    c.rows = c.segs > 1 ? 1 : kLanes / c.lanes;
    const size_t ctas = (a.tokens + c.rows - 1) / c.rows * c.segs;
    // whole warps, whose lanes behind the rows' do nothing
    return launch_kernel_block(dropout_kernel<DT, W>, ctas, round_up(c.lanes * c.rows, 32), 0, st, a, c);
}

}  // namespace

cudaError_t launch_dropout(const LayerNormArgs &a, cudaStream_t st)
{
    return LPC_BY_ROW(dropout_dt, a.dtype, static_cast<size_t>(a.hidden), a, st);
}

}  // namespace lpc
