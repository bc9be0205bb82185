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

// Choice k's row, in lane k (topk <= 32); -1 in the other lanes.
__device__ __forceinline__ int lane_row(const RowsArgs &a, size_t t, int lane)
{
    return lane < a.topk ? load_i32(a.slot_row + t * a.topk + lane) : -1;
}

// Choice k's weight, in lane k.
__device__ __forceinline__ float lane_weight(const RowsArgs &a, size_t t, int lane)
{
    return a.weights != nullptr && lane < a.topk ? load_f32(a.weights + t * a.topk + lane) : 1.0f;
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

// CTA `cta` of the clearing part of a grid: zeros into its unused rows.
template <int DT, int W>
__device__ __forceinline__ void clear_rows(const RowsArgs &a, void *out, size_t cta)
{
    constexpr int kN = Pack<DT, W>::kN;
    const int lane = threadIdx.x & 31;
    const size_t r0 = (cta * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kClearRows;
    for (unsigned m = unused_rows(a, r0, lane); m != 0; m &= m - 1) {
        const size_t row = r0 + __ffs(m) - 1;
        for (size_t i = static_cast<size_t>(lane) * kN; i < a.hidden; i += 32 * kN)
            store_pack<DT, W>(out, row * a.hidden + i, typename Pack<DT, W>::Raw{});
    }
}

size_t clear_ctas(size_t nrows, int threads)
{
    const size_t per_cta = static_cast<size_t>(kClearRows) * (threads / 32);
    return (nrows + per_cta - 1) / per_cta;
}

// How a token's row is cut: `segs` CTAs of `threads` lanes, each lane with
// `per_lane` elements, evenly, so that the last CTA is not nearly empty.
struct Cut {
    unsigned segs;
    int threads;
};
Cut cut_row(size_t hidden, int per_lane)
{
    const size_t lanes = (hidden + per_lane - 1) / per_lane;
    const size_t segs = (lanes + kThreads - 1) / kThreads;
    const size_t each = (lanes + segs - 1) / segs;
    return {static_cast<unsigned>(segs), static_cast<int>((each + 31) / 32 * 32)};
}

// Accesses per lane, so that a lane moves 16 bytes at any access width.
template <int W> constexpr int kPer = 16 / W;

// CTA c < token_ctas: segment c % segs of token c / segs, in accesses of W
// bytes, the lanes' accesses side by side.
template <int DT, int W>
__global__ void __launch_bounds__(kThreads)
dispatch_kernel(const RowsArgs a, unsigned segs, size_t token_ctas)
{
    wait_prior_grid();
    constexpr int kN = Pack<DT, W>::kN;
    if (blockIdx.x >= token_ctas) {
        clear_rows<DT, W>(a, a.out, blockIdx.x - token_ctas);
        return;
    }
    const size_t t = blockIdx.x / segs;
    const size_t base = static_cast<size_t>(blockIdx.x % segs) * blockDim.x * kPer<W>;
    const int rows = lane_row(a, t, threadIdx.x & 31);
    typename Pack<DT, W>::Raw v[kPer<W>];
#pragma unroll
    for (int u = 0; u < kPer<W>; ++u) {
        const size_t i = (base + u * blockDim.x + threadIdx.x) * kN;
        if (i < a.hidden)
            v[u] = load_pack<DT, W>(a.x, t * a.hidden + i);
    }
    for (int k = 0; k < a.topk; ++k) {
        const int row = __shfl_sync(kAll, rows, k);
        if (!has_row(row, a))
            continue;
#pragma unroll
        for (int u = 0; u < kPer<W>; ++u) {
            const size_t i = (base + u * blockDim.x + threadIdx.x) * kN;
            if (i < a.hidden)
                store_pack<DT, W>(a.out, static_cast<size_t>(row) * a.hidden + i, v[u]);
        }
    }
}

// 16 elements of a row from element i on (missing ones read 0).
template <int DT, int W>
__device__ __forceinline__ void load_row16(const void *base, size_t row, size_t hidden, size_t i,
                                           float (&x)[kWideElems])
{
    constexpr int V = Fmt<DT>::kVec;
    uint4 raw[kWideElems / V];
#pragma unroll
    for (int j = 0; j < kWideElems / V; ++j) {
        const int cnt = lane_count<DT>(hidden, i + j * V);
        raw[j] = cnt > 0 ? load_vec<DT>(base, row * hidden + i + j * V,
                                        access_count<DT>(cnt, W == 16))
                         : make_uint4(0u, 0u, 0u, 0u);
    }
    wide_widen<DT>(raw, x);
}

__device__ __forceinline__ size_t row_blocks(size_t hidden) { return (hidden + kBlock - 1) / kBlock; }

// Low precision: a lane quantizes 16 consecutive elements, 8 lanes a block of
// 128, once per token, and writes codes and scales into the K rows. codes are
// stored 16 at a time where rows of codes start on 16 bytes.
template <int DT, int W>
__global__ void __launch_bounds__(kThreads)
dispatch_lp_kernel(const RowsArgs a, unsigned segs, size_t token_ctas)
{
    wait_prior_grid();
    const int lane = threadIdx.x & 31;
    const size_t nb = row_blocks(a.hidden);
    if (blockIdx.x >= token_ctas) {
        const size_t r0 =
            ((blockIdx.x - token_ctas) * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kClearRows;
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
        (static_cast<size_t>(blockIdx.x % segs) * blockDim.x + threadIdx.x) * kWideElems;
    const int rows = lane_row(a, t, lane);
    float x[kWideElems];
    if (i < a.hidden) {
        load_row16<DT, W>(a.x, t, a.hidden, i, x);
    } else {
#pragma unroll
        for (int j = 0; j < kWideElems; ++j)
            x[j] = 0.0f;
    }
    uint32_t w[4];
    float s;
    wide_quantize(x, w, s);  // all 32 lanes take part
    for (int k = 0; k < a.topk; ++k) {
        const int row = __shfl_sync(kAll, rows, k);
        if (!has_row(row, a) || i >= a.hidden)
            continue;
        wide_store_codes(a.codes + static_cast<size_t>(row) * a.hidden, a.hidden, i, w);
        if (lane % kWideGroup == 0)
            store_scale(a.scales + row * nb + i / kBlock, s);
    }
}

// y[t] = sum_k w[t, k] rows[slot_row[t, k]], k ascending, one FP32 fused
// multiply-add each, rounded once at the end. A lane loads its part of
// kCombineChunk rows before it adds them.
template <int DT, int W>
__global__ void __launch_bounds__(kThreads) combine_kernel(const RowsArgs a, unsigned segs)
{
    wait_prior_grid();
    constexpr int kN = Pack<DT, W>::kN;
    constexpr int C = kCombineChunk;
    const int lane = threadIdx.x & 31;
    const size_t t = blockIdx.x / segs;
    const size_t base = static_cast<size_t>(blockIdx.x % segs) * blockDim.x * kPer<W>;
    const int rows = lane_row(a, t, lane);
    const float weights = lane_weight(a, t, lane);
    float acc[kPer<W>][kN];
#pragma unroll
    for (int u = 0; u < kPer<W>; ++u)
#pragma unroll
        for (int j = 0; j < kN; ++j)
            acc[u][j] = 0.0f;
    for (int k0 = 0; k0 < a.topk; k0 += C) {
        typename Pack<DT, W>::Raw v[C][kPer<W>];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int row = __shfl_sync(kAll, rows, (k0 + c) & 31);
#pragma unroll
            for (int u = 0; u < kPer<W>; ++u) {
                const size_t i = (base + u * blockDim.x + threadIdx.x) * kN;
                if (k0 + c < a.topk && has_row(row, a) && i < a.hidden)
                    v[c][u] = load_pack<DT, W>(a.rows, static_cast<size_t>(row) * a.hidden + i);
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int row = __shfl_sync(kAll, rows, (k0 + c) & 31);
            const float w = __shfl_sync(kAll, weights, (k0 + c) & 31);
            if (k0 + c < a.topk && has_row(row, a)) {
#pragma unroll
                for (int u = 0; u < kPer<W>; ++u) {
                    float x[kN];
                    widen_pack<DT, W>(v[c][u], x);
#pragma unroll
                    for (int j = 0; j < kN; ++j)
                        acc[u][j] = fmaf(w, x[j], acc[u][j]);
                }
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kPer<W>; ++u) {
        const size_t i = (base + u * blockDim.x + threadIdx.x) * kN;
        if (i < a.hidden)
            store_pack<DT, W>(a.out, t * a.hidden + i, narrow_pack<DT, W>(acc[u]));
    }
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
template <int DT, int W>
__global__ void __launch_bounds__(kThreads) combine_lp_kernel(const RowsArgs a, unsigned segs)
{
    wait_prior_grid();
    constexpr int C = kCombineChunk;
    constexpr int V = Fmt<DT>::kVec;
    const int lane = threadIdx.x & 31;
    const size_t t = blockIdx.x / segs;
    const size_t i =
        (static_cast<size_t>(blockIdx.x % segs) * blockDim.x + threadIdx.x) * kWideElems;
    const int rows = lane_row(a, t, lane);
    const float weights = lane_weight(a, t, lane);
    const size_t nb = row_blocks(a.hidden);
    const bool aligned = a.hidden % 16 == 0, inside = i < a.hidden;
    float acc[kWideElems];
#pragma unroll
    for (int j = 0; j < kWideElems; ++j)
        acc[j] = 0.0f;
    for (int k0 = 0; k0 < a.topk; k0 += C) {
        uint4 v[C];
        float sc[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int row = __shfl_sync(kAll, rows, (k0 + c) & 31);
            if (k0 + c < a.topk && has_row(row, a) && inside) {
                sc[c] = load_scale(a.scales + row * nb + i / kBlock);
                v[c] = load_row_codes(a.codes, static_cast<size_t>(row), a.hidden, i, aligned);
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int row = __shfl_sync(kAll, rows, (k0 + c) & 31);
            const float w = __shfl_sync(kAll, weights, (k0 + c) & 31);
            if (k0 + c < a.topk && has_row(row, a) && inside) {
                float x[kWideElems];
                wide_dequant(v[c], sc[c], x);
#pragma unroll
                for (int j = 0; j < kWideElems; ++j)
                    acc[j] = fmaf(w, x[j], acc[j]);
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
            store_vec<DT>(a.out, t * a.hidden + i + j * V, access_count<DT>(cnt, W == 16),
                          narrow<DT>(y));
    }
}

// Accesses of a row that a lane of the gradient kernel has in flight.
constexpr int kBackBatch = 4;

// CTA c < token_ctas: choices [p kper, (p + 1) kper) of token c / parts, p =
// c % parts. The CTA goes through the token's row in batches; with dy's batch
// in registers it takes one choice after the other: the row's batch is read,
// drows = w dy written and the partial products of dw = <row, dy> added up,
// over a warp with shuffles, over the warps in shared memory at the end.
template <int DT, int W>
__global__ void __launch_bounds__(1024)
combine_backward_kernel(const RowsArgs a, unsigned parts, int kper, size_t token_ctas)
{
    wait_prior_grid();
    __shared__ float dot[LPCOLL_MAX_TOPK][32];
    constexpr int kN = Pack<DT, W>::kN;
    constexpr int B = kBackBatch;
    using Raw = typename Pack<DT, W>::Raw;
    if (blockIdx.x >= token_ctas) {
        clear_rows<DT, W>(a, a.out, blockIdx.x - token_ctas);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const size_t t = blockIdx.x / parts;
    const int k_lo = static_cast<int>(blockIdx.x % parts) * kper;
    const int k_hi = min(k_lo + kper, a.topk);
    const int rows = lane_row(a, t, lane);
    const float weights = lane_weight(a, t, lane);
    const bool dots = a.dweights != nullptr;
    const size_t step = static_cast<size_t>(blockDim.x) * kN;
    for (size_t i0 = static_cast<size_t>(threadIdx.x) * kN, b0 = 0; b0 < a.hidden;
         i0 += B * step, b0 += B * step) {
        Raw g[B];
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (i0 + b * step < a.hidden)
                g[b] = load_pack<DT, W>(a.x, t * a.hidden + i0 + b * step);
        for (int k = k_lo; k < k_hi; ++k) {
            const int row = __shfl_sync(kAll, rows, k);
            const float w = __shfl_sync(kAll, weights, k);
            float sum = 0.0f;
            if (has_row(row, a)) {
                const size_t r0 = static_cast<size_t>(row) * a.hidden + i0;
                Raw v[B];
                if (dots) {
#pragma unroll
                    for (int b = 0; b < B; ++b)
                        if (i0 + b * step < a.hidden)
                            v[b] = load_pack<DT, W>(a.rows, r0 + b * step);
                }
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    if (i0 + b * step < a.hidden) {
                        float y[kN], x[kN];
                        widen_pack<DT, W>(g[b], y);
                        if (dots) {
                            widen_pack<DT, W>(v[b], x);
#pragma unroll
                            for (int j = 0; j < kN; ++j)
                                sum = fmaf(x[j], y[j], sum);
                        }
#pragma unroll
                        for (int j = 0; j < kN; ++j)
                            y[j] = __fmul_rn(w, y[j]);
                        store_pack<DT, W>(a.out, r0 + b * step, narrow_pack<DT, W>(y));
                    }
                }
            }
            if (dots) {
                sum = warp_sum(sum);
                if (lane == 0)
                    dot[k - k_lo][warp] = b0 == 0 ? sum : dot[k - k_lo][warp] + sum;
            }
        }
    }
    if (!dots)
        return;
    __syncthreads();
    for (int k = k_lo + warp; k < k_hi; k += blockDim.x >> 5) {
        const float sum = warp_sum(lane < (blockDim.x >> 5) ? dot[k - k_lo][lane] : 0.0f);
        if (lane == 0)
            store_f32(a.dweights + t * a.topk + k, a.hidden > 0 ? sum : 0.0f);
    }
}

template <int DT, int W>
cudaError_t dispatch_dt(const RowsArgs &a, bool lp, cudaStream_t st)
{
    const Cut c = cut_row(a.hidden, lp ? kWideElems : 16 / kOne<DT>);
    const size_t ctas = a.tokens * c.segs;
    return launch_kernel_block(lp ? dispatch_lp_kernel<DT, W> : dispatch_kernel<DT, W>,
                               ctas + clear_ctas(a.nrows, c.threads), c.threads, 0, st, a, c.segs,
                               ctas);
}

template <int DT, int W>
cudaError_t combine_dt(const RowsArgs &a, bool lp, cudaStream_t st)
{
    const Cut c = cut_row(a.hidden, lp ? kWideElems : 16 / kOne<DT>);
    return launch_kernel_block(lp ? combine_lp_kernel<DT, W> : combine_kernel<DT, W>,
                               a.tokens * c.segs, c.threads, 0, st, a, c.segs);
}

template <int DT, int W>
cudaError_t combine_backward_dt(const RowsArgs &a, cudaStream_t st)
{
    constexpr int kLane = Pack<DT, W>::kN * kBackBatch;  // elements of a lane's batch
    const size_t lanes = (a.hidden + kLane - 1) / kLane;
    const int threads = static_cast<int>(lanes < 32 ? 32 : (lanes > 1024 ? 1024 : (lanes + 31) / 32 * 32));
    const int kper = a.topk;
    const unsigned parts = 1;
    const size_t ctas = a.tokens * parts;
    return launch_kernel_block(combine_backward_kernel<DT, W>,
                               ctas + clear_ctas(a.hidden > 0 ? a.nrows : 0, threads), threads, 0,
                               st, a, parts, kper, ctas);
}

}  // namespace

cudaError_t launch_dispatch(const RowsArgs &a, bool lp, cudaStream_t st)
{
    return LPC_BY_ROW(dispatch_dt, a.dtype, a.hidden, a, lp, st);
}

cudaError_t launch_combine(const RowsArgs &a, bool lp, cudaStream_t st)
{
    return LPC_BY_ROW(combine_dt, a.dtype, a.hidden, a, lp, st);
}

cudaError_t launch_combine_backward(const RowsArgs &a, cudaStream_t st)
{
    return LPC_BY_ROW(combine_backward_dt, a.dtype, a.hidden, a, st);
}

}  // namespace lpc
