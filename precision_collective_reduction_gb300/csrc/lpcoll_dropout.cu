// lpcoll_dropout.cu -- residual_dropout without a norm, and the gradient of that:
//   x' = x + d(sum_r h_r)     dh = d(dx')
// with the mask made from the counters of lpcoll_philox.cuh both times.
//
// A lane takes 16 bytes of a row whatever the width of its accesses, so that it
// uses all words of the counters that it makes (two groups of four columns in
// BF16, one in FP32).
//
// The generator's 20 wide products per four columns go at 32 lanes a clock and SM
// (measured: 0.165 SM clocks a column), 38 us of 8192 x 8192 columns on a GB300, beside
// some 15 other instructions a column. FP32 hides them behind its bytes: 8192 x 4096
// with residual 59 us (floor 59). BF16 has half the bytes: 8192 x 8192 with
// residual 76 us (floor 59), its gradient 72 (floor 40): 70% of the issue slots. Six
// CTAs of 256 lanes an SM at 40 registers (8 at 32 in FP32) were faster than 4 and 5
// without spills; two pieces in flight and the next piece's loads ahead were not.
#include "lpcoll_layernorm.cuh"

namespace lpc {

namespace {

constexpr int kLanes = 256;  // of a CTA
// How rows are dealt out: `lanes` lanes of each of `segs` CTAs go through a row in
// pieces of 16 bytes, `pieces` of them; short rows share a CTA, `rows` of them.
struct Cut {
    unsigned segs, pieces;
    int lanes, rows;
};

template <int DT, int W>
__global__ void __launch_bounds__(kLanes, DT == LPCOLL_F32 ? 8 : 6)
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
    const Philox rnd(a.drop, a.hidden, false);
    if (t >= a.tokens || threadIdx.x >= static_cast<unsigned>(cut.lanes * cut.rows))
        return;
    const unsigned long long row = rnd.row(t);
    const bool drop = a.drop.least != 0;
    for (; piece < cut.pieces; piece += cut.segs * cut.lanes) {
        const unsigned col = piece * kCols;
        const size_t e0 = t * a.hidden + col;
        const auto has = [&](int i) {
            return W == 16 || col + i * kN < static_cast<unsigned>(a.hidden);
        };
        Vec<kN> h[kPacks], x[kPacks];
#pragma unroll
        for (int i = 0; i < kPacks; ++i)
            if (has(i)) {
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
        uint32_t word[kCols];
        if (drop) {
            unsigned long long group[kGroups];
#pragma unroll
            for (int q = 0; q < kGroups; ++q)
                group[q] = row + piece * kGroups + q;
            rnd.words(group, word);
        }
#pragma unroll
        for (int i = 0; i < kPacks; ++i) {
            if (!has(i))
                continue;
            Vec<kN> v = h[i];
            if (a.dx != nullptr)  // gradient: of the residual, dx' itself
                store_vec_of<DT, W>(a.dx, e0 + i * kN, v);
            if (a.x_out == nullptr)
                continue;
            if (drop) {
                v = mul(a.drop.scale, v);
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    v.v[j] = rnd.keep(v.v[j], word[i * kN + j]);
            }
            if (a.x != nullptr)
                v = plus(x[i], v);
            store_vec_of<DT, W>(a.x_out, e0 + i * kN, v);
        }
    }
}

// A CTA of 256 lanes goes through a row, piece after piece; where there are few rows,
// several CTAs share one.
template <int DT, int W> cudaError_t dropout_dt(const LayerNormArgs &a, cudaStream_t st)
{
    const size_t pieces = (a.hidden + Fmt<DT>::kVec - 1) / Fmt<DT>::kVec;
    Cut c;
    c.pieces = static_cast<unsigned>(pieces);
    const bool few = a.tokens * pieces < static_cast<size_t>(kSms) * 16 * kLanes;
    const size_t turns = (pieces + kLanes - 1) / kLanes;  // evenly, not full ones and a rest
    c.segs = few ? static_cast<unsigned>(turns) : 1;
    c.lanes = static_cast<int>((pieces + turns - 1) / turns);
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
