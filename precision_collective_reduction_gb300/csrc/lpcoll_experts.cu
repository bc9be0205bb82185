// lpcoll_experts.cu -- tokens sent out as rows sorted by expert
// (expert_dispatch, exact or as FP8 payloads), the weighted way back
// (expert_combine) and its gradient.
//
// All three only move rows: out[slot_row[t, k]] = x[t], y[t] = sum_k w[t, k]
// rows[slot_row[t, k]]. The HBM traffic bounds them, so each goes through the
// tokens and reads or writes a token's row once for its K choices. A map
// entry outside [0, nrows) counts as "no row": nothing is read or written for
// it. Rows that no slot uses are written as zeros by CTAs of the same launch.
#include "lpcoll_layers.cuh"
#include "lpcoll_wide.cuh"

namespace lpc {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
// Rows whose use one warp checks (and clears where they are unused).
constexpr int kClearRows = 8;
// Rows that a lane of the combine kernels loads before it adds them.
constexpr int kCombineChunk = 4;

__device__ __forceinline__ bool has_row(int row, const RowsArgs &a)
{
    return static_cast<unsigned>(row) < static_cast<unsigned>(a.nrows);
}

// Bit i: row r0 + i (i < kClearRows) exists and is used by no slot.
__device__ __forceinline__ unsigned unused_rows(const RowsArgs &a, size_t r0, int lane)
{
    bool unused = false;
    if (lane < kClearRows && r0 + lane < a.nrows) {
        const int s = load_i32(a.row_slot + r0 + lane);
        unused = s < 0 || static_cast<size_t>(s) >= a.tokens * a.topk;
    }
    return __ballot_sync(kAll, unused);
}

// Warp `warp` of the clearing part of a grid: zeros into its unused rows.
template <int DT, bool VEC>
__device__ __forceinline__ void clear_rows(const RowsArgs &a, void *out, size_t warp, int lane)
{
    constexpr int kN = Pack<DT, VEC>::kN;
    const size_t r0 = warp * kClearRows;
    for (unsigned m = unused_rows(a, r0, lane); m != 0; m &= m - 1) {
        const size_t row = r0 + __ffs(m) - 1;
        for (size_t i = static_cast<size_t>(lane) * kN; i < a.hidden; i += 32 * kN)
            store_pack<DT, VEC>(out, row * a.hidden + i, typename Pack<DT, VEC>::Raw{});
    }
}

size_t clear_ctas(size_t nrows)
{
    constexpr size_t kPerCta = kClearRows * kWarpsPerCta;
    return (nrows + kPerCta - 1) / kPerCta;
}

// CTA c < tokens * segs: segment c % segs of token c / segs, one pack a lane.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
dispatch_kernel(const RowsArgs a, unsigned segs, size_t token_ctas)
{
    wait_prior_grid();
    constexpr int kN = Pack<DT, VEC>::kN;
    if (blockIdx.x >= token_ctas) {
        const size_t warp = (blockIdx.x - token_ctas) * kWarpsPerCta + (threadIdx.x >> 5);
        clear_rows<DT, VEC>(a, a.out, warp, threadIdx.x & 31);
        return;
    }
    const size_t t = blockIdx.x / segs;
    const size_t i = (static_cast<size_t>(blockIdx.x % segs) * kThreads + threadIdx.x) * kN;
    if (i >= a.hidden)
        return;
    const auto v = load_pack<DT, VEC>(a.x, t * a.hidden + i);
    for (int k = 0; k < a.topk; ++k) {
        const int row = load_i32(a.slot_row + t * a.topk + k);
        if (has_row(row, a))
            store_pack<DT, VEC>(a.out, static_cast<size_t>(row) * a.hidden + i, v);
    }
}

// 16 elements of a row from element i on (missing ones read 0).
template <int DT, bool VEC>
__device__ __forceinline__ void load_row16(const void *base, size_t row, size_t hidden, size_t i,
                                           float (&x)[kWideElems])
{
    constexpr int V = Fmt<DT>::kVec;
    uint4 raw[kWideElems / V];
#pragma unroll
    for (int j = 0; j < kWideElems / V; ++j) {
        const int cnt = lane_count<DT>(hidden, i + j * V);
        raw[j] = cnt > 0 ? load_vec<DT>(base, row * hidden + i + j * V, access_count<DT>(cnt, VEC))
                         : make_uint4(0u, 0u, 0u, 0u);
    }
    wide_widen<DT>(raw, x);
}

__device__ __forceinline__ size_t row_blocks(size_t hidden) { return (hidden + kBlock - 1) / kBlock; }

// Low precision: a lane quantizes 16 consecutive elements, 8 lanes a block of
// 128, once per token, and writes codes and scales into the K rows. codes are
// stored 16 at a time where rows of codes start on 16 bytes.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
dispatch_lp_kernel(const RowsArgs a, unsigned segs, size_t token_ctas)
{
    wait_prior_grid();
    const int lane = threadIdx.x & 31;
    const size_t nb = row_blocks(a.hidden);
    if (blockIdx.x >= token_ctas) {
        const size_t r0 =
            ((blockIdx.x - token_ctas) * kWarpsPerCta + (threadIdx.x >> 5)) * kClearRows;
        for (unsigned m = unused_rows(a, r0, lane); m != 0; m &= m - 1) {
            const size_t row = r0 + __ffs(m) - 1;
            const uint32_t zero[4] = {0u, 0u, 0u, 0u};
            for (size_t i = static_cast<size_t>(lane) * kWideElems; i < a.hidden; i += kWideItem)
                wide_store_codes(a.codes + row * a.hidden, a.hidden, i, zero);
            for (size_t b = lane; b < nb; b += 32)
                store_scale(a.scales + row * nb + b, 0.0f);
        }
        return;
    }
    const size_t t = blockIdx.x / segs;
    const size_t i =
        (static_cast<size_t>(blockIdx.x % segs) * kThreads + threadIdx.x) * kWideElems;
    float x[kWideElems];
    if (i < a.hidden) {
        load_row16<DT, VEC>(a.x, t, a.hidden, i, x);
    } else {
#pragma unroll
        for (int j = 0; j < kWideElems; ++j)
            x[j] = 0.0f;
    }
    uint32_t w[4];
    float s;
    wide_quantize(x, w, s);  // all 32 lanes take part
    if (i >= a.hidden)
        return;
    for (int k = 0; k < a.topk; ++k) {
        const int row = load_i32(a.slot_row + t * a.topk + k);
        if (!has_row(row, a))
            continue;
        wide_store_codes(a.codes + static_cast<size_t>(row) * a.hidden, a.hidden, i, w);
        if (lane % kWideGroup == 0)
            store_scale(a.scales + row * nb + i / kBlock, s);
    }
}

// y[t] = sum_k w[t, k] rows[slot_row[t, k]], k ascending, one FP32 fused
// multiply-add each, rounded once at the end. A lane holds one pack of the
// result and loads kCombineChunk rows ahead.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) combine_kernel(const RowsArgs a, unsigned segs)
{
    wait_prior_grid();
    constexpr int kN = Pack<DT, VEC>::kN;
    constexpr int C = kCombineChunk;
    const size_t t = blockIdx.x / segs;
    const size_t i = (static_cast<size_t>(blockIdx.x % segs) * kThreads + threadIdx.x) * kN;
    if (i >= a.hidden)
        return;
    float acc[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j)
        acc[j] = 0.0f;
    for (int k0 = 0; k0 < a.topk; k0 += C) {
        typename Pack<DT, VEC>::Raw v[C];
        float w[C];
        bool there[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const size_t s = t * a.topk + k0 + c;
            const int row = k0 + c < a.topk ? load_i32(a.slot_row + s) : -1;
            there[c] = has_row(row, a);
            if (there[c]) {
                w[c] = a.weights != nullptr ? load_f32(a.weights + s) : 1.0f;
                v[c] = load_pack<DT, VEC>(a.rows, static_cast<size_t>(row) * a.hidden + i);
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (there[c]) {
                float x[kN];
                widen_pack<DT, VEC>(v[c], x);
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    acc[j] = fmaf(w[c], x[j], acc[j]);
            }
        }
    }
    store_pack<DT, VEC>(a.out, t * a.hidden + i, narrow_pack<DT, VEC>(acc));
}

// 16 codes of a row from element i on (missing ones read 0).
__device__ __forceinline__ uint4 load_row_codes(const uint8_t *codes, size_t row, size_t hidden,
                                                size_t i, bool aligned)
{
    const uint8_t *p = codes + row * hidden;
    if (aligned)
        return wide_load_codes(p, hidden, i);
    const size_t n = hidden - i < kWideElems ? hidden - i : kWideElems;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (LPC_READ_OK(p + i, n)) {
#pragma unroll
        for (int j = 0; j < kWideElems; ++j)
            if (static_cast<size_t>(j) < n)
                w[j / 4] |= static_cast<uint32_t>(p[i + j]) << (8 * (j % 4));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The same from FP8 payloads: a row's value is fl(e4m3(code) * scale).
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) combine_lp_kernel(const RowsArgs a, unsigned segs)
{
    wait_prior_grid();
    constexpr int C = kCombineChunk;
    constexpr int V = Fmt<DT>::kVec;
    const size_t t = blockIdx.x / segs;
    const size_t i =
        (static_cast<size_t>(blockIdx.x % segs) * kThreads + threadIdx.x) * kWideElems;
    if (i >= a.hidden)
        return;
    const size_t nb = row_blocks(a.hidden);
    const bool aligned = a.hidden % 16 == 0;
    float acc[kWideElems];
#pragma unroll
    for (int j = 0; j < kWideElems; ++j)
        acc[j] = 0.0f;
    for (int k0 = 0; k0 < a.topk; k0 += C) {
        uint4 v[C];
        float w[C], sc[C];
        bool there[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const size_t s = t * a.topk + k0 + c;
            const int row = k0 + c < a.topk ? load_i32(a.slot_row + s) : -1;
            there[c] = has_row(row, a);
            if (there[c]) {
                w[c] = a.weights != nullptr ? load_f32(a.weights + s) : 1.0f;
                sc[c] = load_scale(a.scales + row * nb + i / kBlock);
                v[c] = load_row_codes(a.codes, static_cast<size_t>(row), a.hidden, i, aligned);
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (there[c]) {
                float x[kWideElems];
                wide_dequant(v[c], sc[c], x);
#pragma unroll
                for (int j = 0; j < kWideElems; ++j)
                    acc[j] = fmaf(w[c], x[j], acc[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kWideElems / V; ++j) {
        const int cnt = lane_count<DT>(a.hidden, i + j * V);
        float y[V];
#pragma unroll
        for (int q = 0; q < V; ++q)
            y[q] = acc[j * V + q];
        if (cnt > 0)
            store_vec<DT>(a.out, t * a.hidden + i + j * V, access_count<DT>(cnt, VEC),
                          narrow<DT>(y));
    }
}

// CTA c < tokens * parts: choices [p kper, (p + 1) kper) of token c / parts,
// p = c % parts. For each choice the CTA goes through the row once:
// drows = w dy and the partial products of dw = <rows, dy>, which the warps
// add up in shared memory at the end. dy comes from L1 after the first choice.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
combine_backward_kernel(const RowsArgs a, unsigned parts, int kper, size_t token_ctas)
{
    wait_prior_grid();
    __shared__ float dot[LPCOLL_MAX_TOPK][kWarpsPerCta];
    constexpr int kN = Pack<DT, VEC>::kN;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x >= token_ctas) {
        clear_rows<DT, VEC>(a, a.out, (blockIdx.x - token_ctas) * kWarpsPerCta + warp, lane);
        return;
    }
    const size_t t = blockIdx.x / parts;
    const int k_lo = static_cast<int>(blockIdx.x % parts) * kper;
    const int k_hi = min(k_lo + kper, a.topk);
    for (int k = k_lo; k < k_hi; ++k) {
        const size_t s = t * a.topk + k;
        const int row = load_i32(a.slot_row + s);
        float sum = 0.0f;
        if (has_row(row, a)) {
            const float w = a.weights != nullptr ? load_f32(a.weights + s) : 1.0f;
            const size_t r0 = static_cast<size_t>(row) * a.hidden;
#pragma unroll 4
            for (size_t i = static_cast<size_t>(threadIdx.x) * kN; i < a.hidden;
                 i += static_cast<size_t>(kThreads) * kN) {
                float g[kN], x[kN];
                widen_pack<DT, VEC>(load_pack<DT, VEC>(a.x, t * a.hidden + i), g);
                if (a.dweights != nullptr) {
                    widen_pack<DT, VEC>(load_pack<DT, VEC>(a.rows, r0 + i), x);
#pragma unroll
                    for (int j = 0; j < kN; ++j)
                        sum = fmaf(x[j], g[j], sum);
                }
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    g[j] = __fmul_rn(w, g[j]);
                store_pack<DT, VEC>(a.out, r0 + i, narrow_pack<DT, VEC>(g));
            }
        }
        sum = warp_sum(sum);
        if (lane == 0)
            dot[k - k_lo][warp] = sum;
    }
    if (a.dweights == nullptr)
        return;
    __syncthreads();
    const int k = k_lo + static_cast<int>(threadIdx.x);
    if (k < k_hi) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarpsPerCta; ++w)
            sum += dot[threadIdx.x][w];
        store_f32(a.dweights + t * a.topk + k, sum);
    }
}

unsigned segments(size_t hidden, int per_lane)
{
    const size_t per = static_cast<size_t>(per_lane) * kThreads;
    return static_cast<unsigned>((hidden + per - 1) / per);
}

template <int DT, bool VEC>
cudaError_t dispatch_dt(const RowsArgs &a, bool lp, cudaStream_t st)
{
    const unsigned segs = segments(a.hidden, lp ? kWideElems : Pack<DT, VEC>::kN);
    const size_t ctas = a.tokens * segs;
    return launch_kernel_block(lp ? dispatch_lp_kernel<DT, VEC> : dispatch_kernel<DT, VEC>,
                               ctas + clear_ctas(a.nrows), kThreads, 0, st, a, segs, ctas);
}

template <int DT, bool VEC>
cudaError_t combine_dt(const RowsArgs &a, bool lp, cudaStream_t st)
{
    const unsigned segs = segments(a.hidden, lp ? kWideElems : Pack<DT, VEC>::kN);
    return launch_kernel_block(lp ? combine_lp_kernel<DT, VEC> : combine_kernel<DT, VEC>,
                               a.tokens * segs, kThreads, 0, st, a, segs);
}

template <int DT, bool VEC>
cudaError_t combine_backward_dt(const RowsArgs &a, cudaStream_t st)
{
    const int kper = a.topk;
    const unsigned parts = 1;
    const size_t ctas = a.tokens * parts;
    return launch_kernel_block(combine_backward_kernel<DT, VEC>, ctas + clear_ctas(a.nrows),
                               kThreads, 0, st, a, parts, kper, ctas);
}

}  // namespace

#define LPC_BY_TYPE(fn, ...)                                                         \
    (a.dtype == LPCOLL_F32                                                           \
         ? (rows_aligned(a.hidden, a.dtype) ? fn<LPCOLL_F32, true>(__VA_ARGS__)      \
                                            : fn<LPCOLL_F32, false>(__VA_ARGS__))    \
         : (rows_aligned(a.hidden, a.dtype) ? fn<LPCOLL_BF16, true>(__VA_ARGS__)     \
                                            : fn<LPCOLL_BF16, false>(__VA_ARGS__)))

cudaError_t launch_dispatch(const RowsArgs &a, bool lp, cudaStream_t st)
{
    return LPC_BY_TYPE(dispatch_dt, a, lp, st);
}

cudaError_t launch_combine(const RowsArgs &a, bool lp, cudaStream_t st)
{
    return LPC_BY_TYPE(combine_dt, a, lp, st);
}

cudaError_t launch_combine_backward(const RowsArgs &a, cudaStream_t st)
{
    return LPC_BY_TYPE(combine_backward_dt, a, st);
}

}  // namespace lpc
