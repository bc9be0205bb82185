// lpcoll_experts.cu -- tokens sent out as rows sorted by expert
// (expert_dispatch, exact or as FP8 payloads), the weighted way back
// (expert_combine) and its gradient.
//
// All three only move rows: out[slot_row[t, k]] = x[t], y[t] = sum_k w[t, k]
// rows[slot_row[t, k]]. The HBM traffic bounds them, so each goes through the
// tokens and reads or writes a token's row once for its K choices. A map
// entry outside [0, nrows) counts as "no row": nothing is read or written for
// it. Rows that no slot uses are written as zeros by the first CTAs of the same
// launch (last, their long runs of stores were its tail).
//
// Measured on one GB300, 8192 tokens and 4 rows of 8192 BF16 each: dispatch 99 us
// and combine 97 us (6.7 TB/s), as FP8 payloads 76 and 85 us; the gradient of
// 4001 tokens and 8 rows of 4100 FP32 178 us (6.2 TB/s). DRAM bounds all of them
// but the FP8 combine (instructions: 73% issue active, DRAM at 43%).
#include "lpcoll_dda.cuh"
#include "lpcoll_layers.cuh"
#include "lpcoll_wide.cuh"

namespace lpc {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
// Rows whose use one warp checks (and clears where they are unused).
constexpr int kClearRows = 4;
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

// How a token's row is cut: `segs` CTAs of `threads` lanes each (up to `most`), a
// lane with `per_lane` elements, evenly, so that the last CTA is not nearly
// empty. Short rows share a CTA, `tokens` of them.
struct Cut {
    unsigned segs;
    int threads, tokens;
    size_t ctas(size_t all_tokens) const { return (all_tokens + tokens - 1) / tokens * segs; }
    int block() const { return threads * tokens; }
};
Cut cut_row(size_t hidden, int per_lane, int most)
{
    const size_t lanes = (hidden + per_lane - 1) / per_lane;
    const size_t segs = (lanes + most - 1) / most;
    const size_t each = (lanes + segs - 1) / segs;
    Cut c;
    c.segs = static_cast<unsigned>(segs);
    c.threads = static_cast<int>((each + 31) / 32 * 32);
    c.tokens = segs > 1 ? 1 : most / c.threads;
    return c;
}

// The token and the lane among the token's lanes of a thread.
struct Place {
    size_t t;
    unsigned seg;
    int lane;
};
__device__ __forceinline__ Place place_of(unsigned cta, const Cut &c)
{
    Place p;
    const int which = static_cast<int>(threadIdx.x) / c.threads;
    p.t = static_cast<size_t>(cta / c.segs) * c.tokens + which;
    p.seg = cta % c.segs;
    p.lane = static_cast<int>(threadIdx.x) - which * c.threads;
    return p;
}

// Accesses per lane, so that a lane moves 16 bytes at any access width.
template <int W> constexpr int kPer = 16 / W;

// The lanes of a token, after the clearing CTAs, in accesses of W bytes side by
// side.
template <int DT, int W>
__global__ void __launch_bounds__(kThreads)
dispatch_kernel(const RowsArgs a, const Cut cut, unsigned clear)
{
    wait_prior_grid();
    constexpr int kN = Pack<DT, W>::kN;
    if (blockIdx.x < clear) {
        clear_rows<DT, W>(a, a.out, blockIdx.x);
        return;
    }
    const Place me = place_of(blockIdx.x - clear, cut);
    if (me.t >= a.tokens)
        return;
    const size_t base = static_cast<size_t>(me.seg) * cut.threads * kPer<W> + me.lane;
    const int rows = lane_row(a, me.t, threadIdx.x & 31);
    typename Pack<DT, W>::Raw v[kPer<W>];
#pragma unroll
    for (int u = 0; u < kPer<W>; ++u) {
        const size_t i = (base + u * cut.threads) * kN;
        if (i < a.hidden)
            v[u] = load_pack<DT, W>(a.x, me.t * a.hidden + i);
    }
    for (int k = 0; k < a.topk; ++k) {
        const int row = __shfl_sync(kAll, rows, k);
        if (!has_row(row, a))
            continue;
#pragma unroll
        for (int u = 0; u < kPer<W>; ++u) {
            const size_t i = (base + u * cut.threads) * kN;
            if (i < a.hidden)
                store_pack<DT, W>(a.out, static_cast<size_t>(row) * a.hidden + i, v[u]);
        }
    }
}

// Long aligned rows: a CTA takes a part of a token's row, or the rows of
// several tokens, into shared memory and sends it to the K rows, one thread and
// one bulk copy each.
__global__ void __launch_bounds__(kThreads)
dispatch_bulk_kernel(const RowsArgs a, unsigned row_bytes, unsigned segs, unsigned part_bytes,
                     unsigned tokens_per_cta, unsigned clear)
{
    wait_prior_grid();
    extern __shared__ uint4 chunk[];
    if (blockIdx.x < clear) {
        // a row of 16-byte zeros, whatever its type
        RowsArgs z = a;
        z.hidden = row_bytes / 4;
        clear_rows<LPCOLL_F32, 16>(z, a.out, blockIdx.x);
        return;
    }
    const unsigned cta = blockIdx.x - clear;
    const size_t t0 = static_cast<size_t>(cta / segs) * tokens_per_cta;
    const unsigned count = static_cast<unsigned>(
        a.tokens - t0 < tokens_per_cta ? a.tokens - t0 : tokens_per_cta);
    // bytes [off, off + len) of each row; several rows only if they are whole
    const unsigned off = cta % segs * part_bytes;
    const unsigned len = row_bytes - off < part_bytes ? row_bytes - off : part_bytes;
    const char *src = static_cast<const char *>(a.x) + t0 * row_bytes + off;
    for (unsigned b = threadIdx.x * 16; b < len * count; b += kThreads * 16) {
        char *dst = reinterpret_cast<char *>(chunk) + b;
        if (LPC_READ_OK(src + b, 16))
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                         "l"(src + b)
                         : "memory");
    }
    // the first destinations, while the row is on its way
    const unsigned sends = count * a.topk;
    int row = threadIdx.x < sends ? load_i32(a.slot_row + t0 * a.topk + threadIdx.x) : -1;
    asm volatile("cp.async.wait_all;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    for (unsigned s = threadIdx.x; s < sends; s += kThreads) {
        if (s != threadIdx.x)
            row = load_i32(a.slot_row + t0 * a.topk + s);
        if (has_row(row, a))
            bulk_store(static_cast<char *>(a.out) + static_cast<size_t>(row) * row_bytes + off,
                       reinterpret_cast<const char *>(chunk) + s / a.topk * len, len);
    }
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// N words from byte address p on, of any alignment, by aligned words; the bytes
// from `end` on read 0. p and `end` lie in one buffer that starts on a word.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, const uint8_t *end, uint32_t (&w)[N])
{
    const unsigned off = static_cast<unsigned>(reinterpret_cast<uintptr_t>(p) & 3u);
    const uint8_t *base = p - off;
    uint32_t v[N + 1];
    if (base + 4 * (N + 1) <= end && LPC_READ_OK(base, 4 * (N + 1))) {
#pragma unroll
        for (int k = 0; k <= N; ++k)
            v[k] = reinterpret_cast<const uint32_t *>(base)[k];
    } else {
#pragma unroll
        for (int k = 0; k <= N; ++k) {
            v[k] = 0u;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (base + 4 * k + b < end && LPC_READ_OK(base + 4 * k + b, 1))
                    v[k] |= static_cast<uint32_t>(base[4 * k + b]) << (8 * b);
        }
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
        w[k] = __funnelshift_r(v[k], v[k + 1], 8 * off);
}

// 16 elements of row `row` of a [rows][hidden] matrix from element i on (missing
// ones read 0).
template <int DT, int W>
__device__ __forceinline__ void load_row16(const void *base, size_t rows, size_t row,
                                           size_t hidden, size_t i, float (&x)[kWideElems])
{
    constexpr int V = Fmt<DT>::kVec;
    uint4 raw[kWideElems / V];
    if constexpr (W == 16) {
#pragma unroll
        for (int j = 0; j < kWideElems / V; ++j) {
            const int cnt = lane_count<DT>(hidden, i + j * V);
            raw[j] = cnt > 0 ? load_vec<DT>(base, row * hidden + i + j * V, cnt)
                             : make_uint4(0u, 0u, 0u, 0u);
        }
    } else {
        constexpr int kEs = 16 / V;
        const uint8_t *first = static_cast<const uint8_t *>(base);
        uint32_t w[kWideElems * kEs / 4];
        load_words(first + (row * hidden + i) * kEs, first + rows * hidden * kEs, w);
        // elements of the next row are not this one's
#pragma unroll
        for (int j = 0; j < kWideElems * kEs / 4; ++j) {
            if (i + (j + 1) * 4 / kEs > hidden)
                w[j] = i + j * 4 / kEs < hidden ? w[j] & 0xFFFFu : 0u;
        }
        memcpy(raw, w, sizeof(w));
    }
    wide_widen<DT>(raw, x);
}

// Stores the 16 codes of every lane of a warp at p (of any alignment, lane after
// lane; n of them are the row's) in aligned words: a lane's last word takes the
// bytes it misses from the next lane.
__device__ __forceinline__ void store_codes16(uint8_t *p, int n, const uint32_t (&w)[4], int lane)
{
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 3u);
    const int head = (4 - off) & 3;  // bytes before the lane's first aligned word
    const uint32_t next = __shfl_down_sync(kAll, w[0], 1);
    const int n_next = __shfl_down_sync(kAll, n, 1);
    const auto byte = [&](int b) {
        if (LPC_WRITE_OK(p + b, 1))
            p[b] = static_cast<uint8_t>(w[b / 4] >> (8 * (b % 4)));
    };
    // bytes that go out one by one: the head, unless the lane before takes it,
    // and what no whole word holds
    const int first = lane > 0 && n >= head ? head : 0;
    const bool shared = head == 0 || (lane < 31 && n_next >= head);
    int words = n < head ? 0 : (n - head) / 4;
    if (n == kWideElems && shared)
        words = 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t v = __funnelshift_r(w[k], k < 3 ? w[k < 3 ? k + 1 : 3] : next, 8 * head);
        if (k < words && LPC_WRITE_OK(p + head + 4 * k, 4))
            *reinterpret_cast<uint32_t *>(p + head + 4 * k) = v;
    }
#pragma unroll
    for (int b = 0; b < kWideElems; ++b)
        if (b < n && b >= first && (b < head || b >= head + 4 * words))
            byte(b);
}

__device__ __forceinline__ size_t row_blocks(size_t hidden) { return (hidden + kBlock - 1) / kBlock; }

// Low precision: a lane quantizes 16 consecutive elements, 8 lanes a block of
// 128, once per token, and writes codes and scales into the K rows. (Quantizing
// takes 68% of the issue slots, so it must not be done per row.)
template <int DT, int W>
__global__ void __launch_bounds__(kThreads)
dispatch_lp_kernel(const RowsArgs a, const Cut cut, unsigned clear)
{
    wait_prior_grid();
    const int lane = threadIdx.x & 31;
    const size_t nb = row_blocks(a.hidden);
    if (blockIdx.x < clear) {
        const size_t r0 =
            (static_cast<size_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kClearRows;
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
    const Place me = place_of(blockIdx.x - clear, cut);
    const size_t t = me.t;
    if (t >= a.tokens)
        return;
    const size_t i = (static_cast<size_t>(me.seg) * cut.threads + me.lane) * kWideElems;
    const int rows = lane_row(a, t, lane);
    float x[kWideElems];
    if (i < a.hidden) {
        load_row16<DT, W>(a.x, a.tokens, t, a.hidden, i, x);
    } else {
#pragma unroll
        for (int j = 0; j < kWideElems; ++j)
            x[j] = 0.0f;
    }
    uint32_t w[4];
    float s;
    wide_quantize(x, w, s);  // all 32 lanes take part
    const bool aligned = a.hidden % kWideElems == 0;
    const int n = i >= a.hidden ? 0
                                : static_cast<int>(a.hidden - i < kWideElems ? a.hidden - i
                                                                             : kWideElems);
    for (int k = 0; k < a.topk; ++k) {
        const int row = __shfl_sync(kAll, rows, k);
        if (!has_row(row, a))
            continue;
        uint8_t *const codes = a.codes + static_cast<size_t>(row) * a.hidden;
        if (!aligned)
            store_codes16(codes + i, n, w, lane);
        else if (n > 0)
            wide_store_codes(codes, a.hidden, i, w);
        if (n > 0 && lane % kWideGroup == 0)
            store_scale(a.scales + row * nb + i / kBlock, s);
    }
}

// y[t] = sum_k w[t, k] rows[slot_row[t, k]], k ascending, one FP32 fused
// multiply-add each, rounded once at the end. A lane loads its U parts of
// kCombineChunk rows before it adds them.
template <int DT, int W, int U>
__global__ void __launch_bounds__(kThreads) combine_kernel(const RowsArgs a, const Cut cut)
{
    wait_prior_grid();
    constexpr int kN = Pack<DT, W>::kN;
    constexpr int C = kCombineChunk;
    const Place me = place_of(blockIdx.x, cut);
    if (me.t >= a.tokens)
        return;
    const int lane = threadIdx.x & 31;
    const size_t base = static_cast<size_t>(me.seg) * cut.threads * U + me.lane;
    const int rows = lane_row(a, me.t, lane);
    const float weights = lane_weight(a, me.t, lane);
    float acc[U][kN];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < kN; ++j)
            acc[u][j] = 0.0f;
    for (int k0 = 0; k0 < a.topk; k0 += C) {
        typename Pack<DT, W>::Raw v[C][U];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int row = __shfl_sync(kAll, rows, (k0 + c) & 31);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const size_t i = (base + u * cut.threads) * kN;
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
                for (int u = 0; u < U; ++u) {
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
    for (int u = 0; u < U; ++u) {
        const size_t i = (base + u * cut.threads) * kN;
        if (i < a.hidden)
            store_pack<DT, W>(a.out, me.t * a.hidden + i, narrow_pack<DT, W>(acc[u]));
    }
}

// 16 codes of row `row` from element i < hidden on; those past the row's end are
// of no use.
__device__ __forceinline__ uint4 load_row_codes(const RowsArgs &a, int row, size_t i, bool aligned)
{
    const uint8_t *p = a.codes + static_cast<size_t>(row) * a.hidden;
    if (aligned)
        return wide_load_codes(p, a.hidden, i);
    uint32_t w[4];
    load_words(p + i, static_cast<const uint8_t *>(a.codes) + a.nrows * a.hidden, w);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The same from FP8 payloads, with fl(weight * scale) as the factor of a code's
// value. A lane holds 16 consecutive elements (with 8, 118 us where 16 took 93, now 85); a
// warp's results go through shared memory, so that its stores are consecutive.
template <int DT, int W>
__global__ void __launch_bounds__(kThreads) combine_lp_kernel(const RowsArgs a, const Cut cut)
{
    wait_prior_grid();
    __shared__ uint4 stage_all[kWarpsPerCta][kWideElems * 32 / Fmt<DT>::kVec];
    constexpr int C = kCombineChunk;
    const Place me = place_of(blockIdx.x, cut);
    if (me.t >= a.tokens)
        return;
    const int lane = threadIdx.x & 31;
    const size_t i = (static_cast<size_t>(me.seg) * cut.threads + me.lane) * kWideElems;
    const int rows = lane_row(a, me.t, lane);
    const float weights = lane_weight(a, me.t, lane);
    const size_t nb = row_blocks(a.hidden);
    const bool aligned = a.hidden % 16 == 0, inside = i < a.hidden;
    float2 acc[kWideElems / 2];
#pragma unroll
    for (int j = 0; j < kWideElems / 2; ++j)
        acc[j] = make_float2(0.0f, 0.0f);
    for (int k0 = 0; k0 < a.topk; k0 += C) {
        uint4 v[C];
        float sc[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int row = __shfl_sync(kAll, rows, (k0 + c) & 31);
            if (k0 + c < a.topk && has_row(row, a) && inside) {
                sc[c] = load_scale(a.scales + row * nb + i / kBlock);
                v[c] = load_row_codes(a, row, i, aligned);
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int row = __shfl_sync(kAll, rows, (k0 + c) & 31);
            const float w = __shfl_sync(kAll, weights, (k0 + c) & 31);
            if (k0 + c < a.topk && has_row(row, a) && inside) {
                const float f = __fmul_rn(w, sc[c]);
                const uint32_t codes[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                for (int j = 0; j < kWideElems / 2; ++j)
                    acc[j] = fma_pair(make_float2(f, f), dec2(codes[j / 2] >> (16 * (j % 2))),
                                      acc[j]);
            }
        }
    }
    float y[kWideElems];
#pragma unroll
    for (int j = 0; j < kWideElems / 2; ++j) {
        y[2 * j] = acc[j].x;
        y[2 * j + 1] = acc[j].y;
    }
    char *const out = static_cast<char *>(a.out) + me.t * a.hidden * (16 / Fmt<DT>::kVec);
    wide_store_results<DT, W == 16>(out, a.hidden, i - static_cast<size_t>(lane) * kWideElems, y,
                                    stage_all[threadIdx.x >> 5], lane);
}

// Accesses of a row and choices that a lane of the gradient kernel has in
// flight: kBackBatch of one choice (narrow ones are more, so that a lane's batch
// is 64 or 32 bytes), or, for rows of at most one access per lane of 128, one
// access of kBackChoices choices.
template <int W> constexpr int kBackBatch = W == 16 ? 4 : (W == 8 ? 8 : 16);
constexpr int kBackChoices = 4;
constexpr int kBackThreads = 1024, kBackShort = 128;

// The lanes of a token go through its row in batches; with dy's batch in
// registers they take one choice after the other: the row's batch is read,
// drows = w dy written and the partial products of dw = <row, dy> added up,
// over a warp with shuffles, over the warps in shared memory at the end. dy is
// read once for all choices. A second choice's batch in flight took 124
// registers and 203 instead of 190 us.
template <int DT, int W, int B, int C>
__global__ void __launch_bounds__(B == 1 ? kThreads : kBackThreads)
combine_backward_kernel(const RowsArgs a, const Cut cut, unsigned clear)
{
    wait_prior_grid();
    __shared__ float dot[LPCOLL_MAX_TOPK][kBackThreads / 32];
    constexpr int kN = Pack<DT, W>::kN;
    using Raw = typename Pack<DT, W>::Raw;
    if (blockIdx.x < clear) {
        clear_rows<DT, W>(a, a.out, blockIdx.x);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Place me = place_of(blockIdx.x - clear, cut);
    const bool live = me.t < a.tokens;
    const int rows = live ? lane_row(a, me.t, lane) : -1;
    const float weights = live ? lane_weight(a, me.t, lane) : 0.0f;
    const bool dots = a.dweights != nullptr;
    const size_t step = static_cast<size_t>(cut.threads) * kN;
    for (size_t i0 = static_cast<size_t>(me.lane) * kN, b0 = 0; live && b0 < a.hidden;
         i0 += B * step, b0 += B * step) {
        Raw g[B];
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (i0 + b * step < a.hidden)
                g[b] = load_pack<DT, W>(a.x, me.t * a.hidden + i0 + b * step);
        for (int k0 = 0; k0 < a.topk; k0 += C) {
            Raw v[C][B];
            if (dots) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int row = __shfl_sync(kAll, rows, (k0 + c) & 31);
                    if (k0 + c < a.topk && has_row(row, a)) {
#pragma unroll
                        for (int b = 0; b < B; ++b)
                            if (i0 + b * step < a.hidden)
                                v[c][b] = load_pack<DT, W>(
                                    a.rows, static_cast<size_t>(row) * a.hidden + i0 + b * step);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = k0 + c;
                if (k >= a.topk)
                    break;
                const int row = __shfl_sync(kAll, rows, k);
                const float w = __shfl_sync(kAll, weights, k);
                float sum = 0.0f;
                if (has_row(row, a)) {
                    const size_t r0 = static_cast<size_t>(row) * a.hidden + i0;
#pragma unroll
                    for (int b = 0; b < B; ++b) {
                        if (i0 + b * step < a.hidden) {
                            float y[kN], x[kN];
                            widen_pack<DT, W>(g[b], y);
                            if (dots) {
                                widen_pack<DT, W>(v[c][b], x);
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
                        dot[k][warp] = b0 == 0 ? sum : dot[k][warp] + sum;
                }
            }
        }
    }
    if (!dots)
        return;
    __syncthreads();
    if (!live)
        return;
    const int warps = cut.threads >> 5, first = warp / warps * warps;
    for (int k = warp - first; k < a.topk; k += warps) {
        const float sum = warp_sum(lane < warps ? dot[k][first + lane] : 0.0f);
        if (lane == 0)
            store_f32(a.dweights + me.t * a.topk + k, a.hidden > 0 ? sum : 0.0f);
    }
}

// 16-byte vectors from which on a call is bound by traffic, not by latency: 2048
// for each SM.
constexpr size_t kManyVectors = 152 * 2048;

size_t row_vectors(const RowsArgs &a) { return a.tokens * (a.hidden * dtype_bytes(a.dtype) / 16); }

// Shortest row, in bytes, that dispatch sends with bulk copies, and the shared
// memory of a CTA that does. 8192 tokens to 4 rows of 16 KB each took 99 us
// against 131 us with the lanes' own stores (floor 99), 32 tokens to 8 rows 4.0
// against 2.1 us, so bulk copies are for large calls.
constexpr size_t kBulkRow = 1024, kBulkChunk = 16 * 1024;

cudaError_t dispatch_bulk(const RowsArgs &a, size_t row_bytes, cudaStream_t st)
{
    const size_t segs = (row_bytes + kBulkChunk - 1) / kBulkChunk;
    const size_t part = ((row_bytes + segs - 1) / segs + 15) / 16 * 16;
    const size_t per_cta = segs > 1 ? 1 : kBulkChunk / row_bytes;
    const size_t ctas = (a.tokens + per_cta - 1) / per_cta * segs;
    const size_t clear = clear_ctas(a.nrows, kThreads);
    return launch_kernel_block(dispatch_bulk_kernel, clear + ctas, kThreads, per_cta * part, st, a,
                               static_cast<unsigned>(row_bytes), static_cast<unsigned>(segs),
                               static_cast<unsigned>(part), static_cast<unsigned>(per_cta),
                               static_cast<unsigned>(clear));
}

template <int DT, int W>
cudaError_t dispatch_dt(const RowsArgs &a, bool lp, cudaStream_t st)
{
    const size_t row_bytes = a.hidden * dtype_bytes(DT);
    if (W == 16 && !lp && row_bytes >= kBulkRow && row_bytes <= 64 * kBulkChunk &&
        row_vectors(a) >= kManyVectors)
        return dispatch_bulk(a, row_bytes, st);
    // CTAs of 128 lanes for payloads: 4097 elements 69 against 75 us with 256
    const Cut c = lp ? cut_row(a.hidden, kWideElems, kThreads / 2)
                     : cut_row(a.hidden, 16 / kOne<DT>, kThreads);
    const size_t clear = clear_ctas(a.nrows, c.block());
    return launch_kernel_block(lp ? dispatch_lp_kernel<DT, W> : dispatch_kernel<DT, W>,
                               clear + c.ctas(a.tokens), c.block(), 0, st, a, c,
                               static_cast<unsigned>(clear));
}

template <int DT, int W>
cudaError_t combine_dt(const RowsArgs &a, bool lp, cudaStream_t st)
{
    // CTAs of 64 lanes: 8192 tokens of 4 rows of 8192 BF16 take 97 us against 101
    // with 256, from FP8 payloads 85 against 89
    constexpr int kLanes = 64;
    if (lp) {
        const Cut c = cut_row(a.hidden, kWideElems, kLanes);
        return launch_kernel_block(combine_lp_kernel<DT, W>, c.ctas(a.tokens), c.block(), 0, st,
                                   a, c);
    }
    if constexpr (W == 16) {
        // four vectors a lane once there is enough to do: 8192 tokens of 4 rows
        // of 8192 BF16 101 against 109 us, 32 tokens of 8 rows 3.6 against 2.3
        if (row_vectors(a) >= kManyVectors) {
            const Cut c = cut_row(a.hidden, 4 * Fmt<DT>::kVec, kLanes);
            return launch_kernel_block(combine_kernel<DT, W, 4>, c.ctas(a.tokens), c.block(), 0,
                                       st, a, c);
        }
    }
    const Cut c = cut_row(a.hidden, Fmt<DT>::kVec, kLanes);
    return launch_kernel_block(combine_kernel<DT, W, kPer<W>>, c.ctas(a.tokens), c.block(), 0, st,
                               a, c);
}

template <int DT, int W>
cudaError_t combine_backward_dt(const RowsArgs &a, cudaStream_t st)
{
    constexpr int kN = Pack<DT, W>::kN;
    const size_t packs = (a.hidden + kN - 1) / kN;
    const bool brief = packs <= kBackShort;
    const size_t lanes = brief ? packs : (packs + kBackBatch<W> - 1) / kBackBatch<W>;
    Cut c;
    c.segs = 1;
    c.threads = static_cast<int>(lanes < 32 ? 32
                                            : (lanes > kBackThreads ? kBackThreads
                                                                    : (lanes + 31) / 32 * 32));
    c.tokens = c.threads > kThreads ? 1 : kThreads / c.threads;
    const size_t clear = clear_ctas(a.hidden > 0 ? a.nrows : 0, c.block());
    return launch_kernel_block(brief ? combine_backward_kernel<DT, W, 1, kBackChoices>
                                     : combine_backward_kernel<DT, W, kBackBatch<W>, 1>,
                               clear + c.ctas(a.tokens), c.block(), 0, st, a, c,
                               static_cast<unsigned>(clear));
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
