// lpcoll_route.cu -- the router of an expert layer (softmax over the experts,
// the K largest of each token, and the gradient) and the stable counting sort
// of the (token, choice) slots by expert.
//
// Router: one warp per token. A lane holds the logits of experts lane,
// lane + 32, ... as order-preserving 32-bit keys; a choice is the largest key
// of the warp and, among the experts that hold it, the lowest index: two
// warp-wide integer reductions. Every sum is FP32 in a fixed order.
#include "lpcoll_layers.cuh"

namespace lpc {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
// Keys up to this one are "no expert": -infinity, a choice taken, padding.
constexpr uint32_t kKeyNone = 0x007FFFFFu;
constexpr uint32_t kKeyNan = 0xFFFFFFFFu;

// Order-preserving key of a logit: -0 equals +0, a NaN is above +infinity.
__device__ __forceinline__ uint32_t logit_key(float x)
{
    if (isnan(x))
        return kKeyNan;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((b >> 31) != 0 ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ float key_logit(uint32_t k)
{
    return k == kKeyNan ? __uint_as_float(0x7FC00000u)
                        : __uint_as_float(k ^ ((k >> 31) != 0 ? 0x80000000u : 0xFFFFFFFFu));
}

template <int DT, int PER>
__device__ __forceinline__ void load_logits(const void *logits, size_t t, int experts, int lane,
                                            float (&x)[PER])
{
    float one[1];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 32 + lane;
        x[i] = -INFINITY;
        if (e < experts) {
            widen_pack<DT, kOne<DT>>(load_pack<DT, kOne<DT>>(logits, t * experts + e), one);
            x[i] = one[0];
        }
    }
}

template <int DT, int PER>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs a)
{
    wait_prior_grid();
    const int lane = threadIdx.x & 31;
    const size_t t = (static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    if (t >= a.tokens)
        return;
    float x[PER];
    uint32_t key[PER];
    load_logits<DT, PER>(a.logits, t, a.experts, lane, x);
#pragma unroll
    for (int i = 0; i < PER; ++i)
        key[i] = logit_key(x[i]);

    int my_id = -1;
    uint32_t my_key = 0, top = 0;
    for (int j = 0; j < a.topk; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t most = __reduce_max_sync(kAll, best);
        if (most <= kKeyNone)
            break;
        const int mine = best == most ? at * 32 + lane : INT32_MAX;
        const int id = __reduce_min_sync(kAll, mine);
        if (j == 0)
            top = most;
        if (lane == j) {
            my_id = id;
            my_key = most;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i * 32 + lane == id)
                key[i] = 0;
    }

    float w = 0.0f;
    if (top > kKeyNone) {  // the same in all lanes
        const float m = key_logit(top);
        w = my_id >= 0 ? expf(key_logit(my_key) - m) : 0.0f;
        float sum = w;
        if (!a.renormalize) {
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                sum += expf(x[i] - m);
        }
        w = __fdiv_rn(w, warp_sum(sum));
    }
    if (lane < a.topk) {
        store_i32(a.ids + t * a.topk + lane, my_id);
        store_f32(a.weights + t * a.topk + lane, my_id >= 0 ? w : 0.0f);
    }
}

// dl_e = [e chosen as j] w_j dw_j - p_e sum_j w_j dw_j, with p = w at the
// chosen and 0 elsewhere when the weights were renormalised.
template <int DT, int PER>
__global__ void __launch_bounds__(kThreads) route_backward_kernel(const RouteArgs a)
{
    wait_prior_grid();
    const int lane = threadIdx.x & 31;
    const size_t t = (static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    if (t >= a.tokens)
        return;
    int id = -1;
    float w = 0.0f, g = 0.0f;
    if (lane < a.topk) {
        id = load_i32(a.ids + t * a.topk + lane);
        if (id >= 0 && id < a.experts) {
            w = load_f32(a.weights + t * a.topk + lane);
            g = __fmul_rn(w, load_f32(a.dweights + t * a.topk + lane));
        }
    }
    const float mean = warp_sum(g);
    float d[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        d[i] = 0.0f;
    if (a.renormalize) {
        g = fmaf(-w, mean, g);
    } else {
        float x[PER];
        load_logits<DT, PER>(a.logits, t, a.experts, lane, x);
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            most = max(most, logit_key(x[i]));
        most = __reduce_max_sync(kAll, most);
        if (most > kKeyNone) {
            const float m = key_logit(most);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                x[i] = expf(x[i] - m);
                sum += x[i];
            }
            const float f = __fdiv_rn(-mean, warp_sum(sum));
#pragma unroll
            for (int i = 0; i < PER; ++i)
                d[i] = __fmul_rn(f, x[i]);
        }
    }
    for (int j = 0; j < a.topk; ++j) {
        const int e = __shfl_sync(kAll, id, j);
        const float v = __shfl_sync(kAll, g, j);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i * 32 + lane == e)
                d[i] += v;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 32 + lane;
        const float one[1] = {d[i]};
        if (e < a.experts)
            store_pack<DT, kOne<DT>>(a.dlogits, t * a.experts + e,
                                     narrow_pack<DT, kOne<DT>>(one));
    }
}

// ---------------------------------------------------------------------------
// Stable counting sort. The slots are cut into chunks, one CTA each. With more
// than one chunk a first launch counts the experts of each chunk; the placing
// launch adds up the counts of the chunks before its own, so that no CTA waits
// on another, then each of its warps takes a contiguous part of the chunk and
// gives its slots their ranks in order, 32 at a time. Integer sums only: the
// result does not depend on the order in which anything runs.
// ---------------------------------------------------------------------------

// The largest sort of one launch, in one CTA, and the smallest chunk of others:
// 8 warps of 8, or of 2, steps of 32 slots.
constexpr int kSortOne = 2048;
constexpr int kSortChunk = 512;
constexpr int kSortMaxChunks = 128;

__device__ __forceinline__ int slot_expert(const SortArgs &a, int s)
{
    const int e = load_i32(a.ids + s);
    return static_cast<unsigned>(e) < static_cast<unsigned>(a.experts) ? e : -1;
}

__global__ void __launch_bounds__(kThreads) sort_count_kernel(const SortArgs a)
{
    __shared__ int hist[LPCOLL_MAX_EXPERTS];
    for (int e = threadIdx.x; e < a.experts; e += kThreads)
        hist[e] = 0;
    __syncthreads();
    wait_prior_grid();
    const long long lo = static_cast<long long>(blockIdx.x) * a.chunk_len;
    const int end = static_cast<int>(min(lo + a.chunk_len, static_cast<long long>(a.slots)));
    for (long long s = lo + threadIdx.x; s < end; s += kThreads) {
        const int e = slot_expert(a, static_cast<int>(s));
        if (e >= 0)
            atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kThreads)
        store_i32(a.chunk_counts + static_cast<size_t>(blockIdx.x) * a.experts + e, hist[e]);
}

__global__ void __launch_bounds__(kThreads) sort_place_kernel(const SortArgs a)
{
    // next[w][e]: rank within expert e of warp w's next slot
    __shared__ int next[kWarpsPerCta][LPCOLL_MAX_EXPERTS];
    __shared__ int first[LPCOLL_MAX_EXPERTS];  // first row of an expert
    __shared__ int total[LPCOLL_MAX_EXPERTS];  // slots of an expert
    __shared__ int warp_total[kWarpsPerCta];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int E = a.experts;
    for (int e = tid; e < E; e += kThreads)
#pragma unroll
        for (int w = 0; w < kWarpsPerCta; ++w)
            next[w][e] = 0;
    __syncthreads();
    wait_prior_grid();

    const long long lo = static_cast<long long>(blockIdx.x) * a.chunk_len;
    const long long end = min(lo + a.chunk_len, static_cast<long long>(a.slots));
    const int part = (a.chunk_len / kWarpsPerCta + 31) & ~31;
    const long long w_lo = lo + static_cast<long long>(warp) * part;
    const long long w_end = min(w_lo + part, end);
    for (long long s = w_lo + lane; s < w_end; s += 32) {
        const int e = slot_expert(a, static_cast<int>(s));
        if (e >= 0)
            atomicAdd(&next[warp][e], 1);
    }
    __syncthreads();
    for (int e = tid; e < E; e += kThreads) {
        int sum = 0, before = 0;
        if (a.chunks > 1) {
#pragma unroll 8
            for (int c = 0; c < a.chunks; ++c) {
                const int v = load_i32(a.chunk_counts + static_cast<size_t>(c) * E + e);
                sum += v;
                before += c < static_cast<int>(blockIdx.x) ? v : 0;
            }
        }
        int run = before;
#pragma unroll
        for (int w = 0; w < kWarpsPerCta; ++w) {
            const int v = next[w][e];
            next[w][e] = run;
            run += v;
        }
        total[e] = a.chunks > 1 ? sum : run;
    }
    __syncthreads();

    // exclusive sum over the experts, 4 consecutive ones per thread
    constexpr int kPer = LPCOLL_MAX_EXPERTS / kThreads;
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        sum += tid * kPer + i < E ? total[tid * kPer + i] : 0;
    int scan = sum;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int v = __shfl_up_sync(kAll, scan, m);
        scan += lane >= m ? v : 0;
    }
    if (lane == 31)
        warp_total[warp] = scan;
    __syncthreads();
    int before = scan - sum, used = 0;
#pragma unroll
    for (int w = 0; w < kWarpsPerCta; ++w) {
        before += w < warp ? warp_total[w] : 0;
        used += warp_total[w];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = tid * kPer + i;
        if (e < E) {
            first[e] = a.capacity > 0 ? e * a.capacity : before;
            before += total[e];
        }
    }
    __syncthreads();

    const int limit = a.capacity > 0 ? a.capacity : INT32_MAX;
    for (long long s0 = w_lo; s0 < w_end; s0 += 32) {
        const long long s = s0 + lane;
        const int e = s < w_end ? slot_expert(a, static_cast<int>(s)) : -1;
        const unsigned same = __match_any_sync(kAll, e);
        if (e >= 0) {
            const int rank = next[warp][e] + __popc(same & ((1u << lane) - 1u));
            const int row = rank < limit ? first[e] + rank : -1;
            store_i32(a.slot_row + s, row);
            if (row >= 0)
                store_i32(a.row_slot + row, static_cast<int>(s));
        } else if (s < w_end) {
            store_i32(a.slot_row + s, -1);
        }
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1)
            next[warp][e] += __popc(same);
        __syncwarp();
    }

    // rows that no slot took
    const long long stride = static_cast<long long>(gridDim.x) * kThreads;
    const long long r0 = static_cast<long long>(blockIdx.x) * kThreads + tid;
    if (a.capacity > 0) {
        for (long long r = r0; r < a.rows; r += stride) {
            const int e = static_cast<int>(r) / a.capacity;
            if (static_cast<int>(r) - e * a.capacity >= total[e])
                store_i32(a.row_slot + r, -1);
        }
    } else {
        for (long long r = used + r0; r < a.rows; r += stride)
            store_i32(a.row_slot + r, -1);
    }
    if (blockIdx.x == 0) {
        for (int e = tid; e < E; e += kThreads) {
            store_i32(a.offsets + e, first[e]);
            store_i32(a.counts + e, min(total[e], limit));
        }
        if (tid == 0)
            store_i32(a.offsets + E, a.capacity > 0 ? a.rows : used);
    }
}

size_t token_ctas(size_t tokens) { return (tokens + kWarpsPerCta - 1) / kWarpsPerCta; }

template <int DT, int PER>
cudaError_t route_per(const RouteArgs &a, bool backward, cudaStream_t st)
{
    return launch_kernel_block(backward ? route_backward_kernel<DT, PER> : route_kernel<DT, PER>,
                               token_ctas(a.tokens), kThreads, 0, st, a);
}

// Logits per lane: the smallest power of two that holds the experts.
template <int DT>
cudaError_t route_dt(const RouteArgs &a, bool backward, cudaStream_t st)
{
    if (a.experts <= 64)
        return route_per<DT, 2>(a, backward, st);
    if (a.experts <= 128)
        return route_per<DT, 4>(a, backward, st);
    if (a.experts <= 256)
        return route_per<DT, 8>(a, backward, st);
    if (a.experts <= 512)
        return route_per<DT, 16>(a, backward, st);
    return route_per<DT, 32>(a, backward, st);
}

}  // namespace

cudaError_t launch_route(const RouteArgs &a, cudaStream_t st)
{
    return a.dtype == LPCOLL_F32 ? route_dt<LPCOLL_F32>(a, false, st)
                                 : route_dt<LPCOLL_BF16>(a, false, st);
}

cudaError_t launch_route_backward(const RouteArgs &a, cudaStream_t st)
{
    return a.dtype == LPCOLL_F32 ? route_dt<LPCOLL_F32>(a, true, st)
                                 : route_dt<LPCOLL_BF16>(a, true, st);
}

static int sort_chunk_len(size_t slots)
{
    if (slots <= kSortOne)
        return kSortOne;
    const size_t even = (slots + kSortMaxChunks - 1) / kSortMaxChunks;
    const size_t len = (even + kThreads - 1) / kThreads * kThreads;
    return static_cast<int>(len > kSortChunk ? len : kSortChunk);
}

int sort_chunks(size_t slots)
{
    const size_t len = static_cast<size_t>(sort_chunk_len(slots));
    return slots == 0 ? 1 : static_cast<int>((slots + len - 1) / len);
}

cudaError_t launch_sort(SortArgs a, cudaStream_t st)
{
    a.chunk_len = sort_chunk_len(static_cast<size_t>(a.slots));
    a.chunks = sort_chunks(static_cast<size_t>(a.slots));
    if (a.chunks > 1) {
        const cudaError_t e = launch_kernel_block(sort_count_kernel, a.chunks, kThreads, 0, st, a);
        if (e != cudaSuccess)
            return e;
    }
    return launch_kernel_block(sort_place_kernel, a.chunks, kThreads, 0, st, a);
}

}  // namespace lpc
