// lpcoll_route.cu -- the router of an expert layer (softmax over the experts,
// the K largest of each token, and the gradient) and the stable counting sort
// of the (token, choice) slots by expert.
//
// Router: one warp per token, the logits of a lane's experts as
// order-preserving integers. Instructions bound it, not the logits'
// traffic, so a choice is one warp-wide integer maximum: 22 bits of the logit
// and 10 of the expert's index make one unsigned number whose order is that
// of the logits, lower index first. For BF16 the 22 bits hold the whole logit;
// for FP32 a token in which two neighbours of the choice agree in them, and
// not in the rest, is chosen again with both parts apart. A lane sorts its
// numbers once, and the winner of a choice moves up its list. Every sum is
// FP32 in a fixed order. Measured on one GB300, 32768 tokens of 256 FP32 logits,
// 8 choices: 16.4 us (some 400 instructions per token, 70% issue active; with keys
// and indexes apart 30 us; 18.8 for logits of BF16 values, whose ties are chosen again), the gradient 13.2 us (0.78 of the copy rate).
#include "lpcoll_logits.cuh"

namespace lpc {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
// Keys up to this one are "no expert": -infinity, a choice taken, padding.
constexpr uint32_t kKeyNone = 0x007FFFFFu;

// 2^x, 2 ulp; results below the normal range are 0.
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A term e^d of a softmax's sum, d <= 0. The constant is 0.224 2^-24 of itself off and
// the product rounds by up to 2^-24 of itself, which moves a term by up to 1.224 |d| 2^-24
// of itself, beside the 2 ulp of 2^x. Of the sum, whose largest term is 1, that is at most
// 1.224 |d| e^d 2^-24 <= 0.45 2^-24 a term: enough for a sum, not for a probability.
__device__ __forceinline__ float exp_term(float d)
{
    return exp2_fast(__fmul_rn(d, 1.44269504f));
}

// Order-preserving key of a logit: -0 equals +0, and every NaN is the largest
// key, since an addition returns all of them as 0x7FFFFFFF.
__device__ __forceinline__ uint32_t logit_key(float x)
{
    const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_logit(uint32_t k)
{
    return __uint_as_float(k ^ ((k >> 31) != 0 ? 0x80000000u : 0xFFFFFFFFu));
}

// Descending order of v[LO .. LO + N) (Batcher's odd-even merge sort); merge_down
// does it for the elements R apart, whose halves are in order.
template <int P, int Q, int PER> __device__ __forceinline__ void order(uint32_t (&v)[PER])
{
    const uint32_t hi = max(v[P], v[Q]);
    v[Q] = min(v[P], v[Q]);
    v[P] = hi;
}

template <int LO, int END, int STEP, int R, int PER>
__device__ __forceinline__ void order_each(uint32_t (&v)[PER])
{
    if constexpr (LO + R < END) {
        order<LO, LO + R>(v);
        order_each<LO + STEP, END, STEP, R>(v);
    }
}

template <int LO, int N, int R, int PER>
__device__ __forceinline__ void merge_down(uint32_t (&v)[PER])
{
    if constexpr (2 * R < N) {
        merge_down<LO, N, 2 * R>(v);
        merge_down<LO + R, N, 2 * R>(v);
        order_each<LO + R, LO + N, 2 * R, R>(v);
    } else {
        order<LO, LO + R>(v);
    }
}

template <int LO, int N, int PER> __device__ __forceinline__ void sort_down(uint32_t (&v)[PER])
{
    if constexpr (N > 1) {
        sort_down<LO, N / 2>(v);
        sort_down<LO + N / 2, N / 2>(v);
        merge_down<LO, N, 1>(v);
    }
}

constexpr uint32_t kIndexBits = 0x3FFu;
static_assert(LPCOLL_MAX_EXPERTS == kIndexBits + 1, "an expert's index has 10 bits");

// The topk choices by logit and index apart: expert in lane j, -1 from the
// first lane on that finds none left.
template <int DT, int PER>
__device__ __noinline__ int choose_apart(const void *logits, size_t t, int experts, int topk,
                                         int lane)
{
    float x[PER];
    uint32_t key[PER];
    load_logits<DT, PER>(logits, t, experts, lane, x);
#pragma unroll
    for (int i = 0; i < PER; ++i)
        key[i] = logit_key(x[i]);
    int my_id = -1;
    for (int j = 0; j < topk; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] > best) {
                best = key[i];
                at = expert_of<DT, PER>(i, lane);
            }
        const uint32_t most = __reduce_max_sync(kAll, best);
        if (most <= kKeyNone)
            break;
        const int id = __reduce_min_sync(kAll, best == most ? at : INT32_MAX);
        if (lane == j)
            my_id = id;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (expert_of<DT, PER>(i, lane) == id)
                key[i] = 0;
    }
    return my_id;
}

// MOST: choices that the kernel is made for. For few (kFew) the steps are unrolled
// and a lane's list is kept, and moved up, only as far as later steps can reach
// (32768 tokens of 256 FP32 17.7 -> 16.6 us, 16384 of 384 BF16 14.5 -> 11.6); with
// 4 logits a lane or fewer there is nothing to save.
constexpr int kFew = 8;

template <int DT, int PER, int MOST>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs a)
{
    wait_prior_grid();
    // the number after the last choice tells whether that one was sure
    constexpr int L = PER < MOST + 1 ? PER : MOST + 1;
    const int lane = threadIdx.x & 31;
    const size_t t = (static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    if (t >= a.tokens)
        return;
    float x[PER];
    load_logits<DT, PER>(a.logits, t, a.experts, lane, x);

    uint32_t list[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        // a number of -infinity, of an expert that is not there too, stays
        // below kKeyNone
        list[i] = (logit_key(x[i]) & ~kIndexBits) | (kIndexBits - expert_of<DT, PER>(i, lane));
    }
    sort_down<0, PER>(list);
    uint32_t mine = 0;
    const auto step = [&](int j) {
        const uint32_t most = __reduce_max_sync(kAll, list[0]);
        if (lane == j && most > kKeyNone)
            mine = most;
        const bool won = list[0] == most;
#pragma unroll
        for (int i = 0; i < L; ++i)
            if (MOST != kFew || i < MOST - j)
                list[i] = won ? (i + 1 < L ? list[i + 1] : 0u) : list[i];
    };
    if constexpr (MOST == kFew) {
#pragma unroll
        for (int j = 0; j < MOST; ++j)
            if (j < a.topk)
                step(j);
    } else {
        for (int j = 0; j < a.topk; ++j)
            step(j);
    }
    int my_id = mine != 0 ? static_cast<int>(kIndexBits - (mine & kIndexBits)) : -1;
    const auto logit_of = [&](int id) {
        float one[1] = {-INFINITY};
        if (id >= 0)
            widen_pack<DT, kOne<DT>>(load_pack<DT, kOne<DT>>(a.logits, t * a.experts + id), one);
        return one[0];
    };
    float z = logit_of(my_id);
    if constexpr (DT == LPCOLL_F32) {
        // neighbours in the order, the last choice and the next one among them
        const uint32_t next = __reduce_max_sync(kAll, list[0]);
        const uint32_t before = __shfl_up_sync(kAll, mine, 1);
        const float z_before = __shfl_up_sync(kAll, z, 1);
        const bool unsure =
            (lane > 0 && mine != 0 && (mine ^ before) <= kIndexBits &&
             logit_key(z) != logit_key(z_before)) ||
            (lane == a.topk - 1 && mine != 0 && next > kKeyNone &&
             (mine ^ next) <= kIndexBits);
        if (__any_sync(kAll, unsure)) {
            my_id = choose_apart<DT, PER>(a.logits, t, a.experts, a.topk, lane);
            z = logit_of(my_id);
        }
    }

    float w = 0.0f;
    if (__any_sync(kAll, my_id >= 0)) {
        const float m = __shfl_sync(kAll, z, 0);
        w = my_id >= 0 ? expf(z - m) : 0.0f;
        float sum = w;
        if (!a.renormalize) {
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                sum += exp_term(x[i] - m);
        }
        w = __fdiv_rn(w, warp_sum(sum));
    }
    if (lane < a.topk) {
        store_i32(a.ids + t * a.topk + lane, my_id);
        store_f32(a.weights + t * a.topk + lane, my_id >= 0 ? w : 0.0f);
    }
}

// Tokens of a warp of the gradient kernel, whose logits it loads together.
template <int PER> constexpr int kPairs = PER <= 8 ? 2 : 1;

// dl_e = [e chosen as j] w_j dw_j - p_e sum_j w_j dw_j, with p = w at the
// chosen and 0 elsewhere when the weights were renormalised. The chosen
// experts' terms go through a row in shared memory.
template <int DT, int PER>
__global__ void __launch_bounds__(kThreads) route_backward_kernel(const RouteArgs a)
{
    wait_prior_grid();
    constexpr int R = kRun<DT, PER>;
    constexpr int kEs = kOne<DT>;
    using Raw = typename RunBytes<R * kEs>::Raw;
    __shared__ __align__(16) float chosen_all[kWarpsPerCta][PER * 32];
    float *const chosen = chosen_all[threadIdx.x >> 5];
    const int lane = threadIdx.x & 31;
    const size_t t0 =
        ((static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5) * kPairs<PER>;
    float x[kPairs<PER>][PER], w[kPairs<PER>], g[kPairs<PER>];
    int id[kPairs<PER>];
#pragma unroll
    for (int q = 0; q < kPairs<PER>; ++q) {
        id[q] = -1;
        w[q] = g[q] = 0.0f;
        const size_t t = t0 + q;
        if (t < a.tokens) {
            if (!a.renormalize)
                load_logits<DT, PER>(a.logits, t, a.experts, lane, x[q]);
            if (lane < a.topk) {
                id[q] = load_i32(a.ids + t * a.topk + lane);
                w[q] = load_f32(a.weights + t * a.topk + lane);
                g[q] = load_f32(a.dweights + t * a.topk + lane);
            }
        }
    }
#pragma unroll
    for (int q = 0; q < kPairs<PER>; ++q) {
        const size_t t = t0 + q;
        if (t >= a.tokens)
            return;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            chosen[i * 32 + lane] = 0.0f;
        const bool there = id[q] >= 0 && id[q] < a.experts;
        g[q] = there ? __fmul_rn(w[q], g[q]) : 0.0f;
        const float mean = warp_sum(g[q]);
        __syncwarp();
        if (there)
            chosen[id[q]] = a.renormalize ? fmaf(-w[q], mean, g[q]) : g[q];
        __syncwarp();
        float d[PER];
#pragma unroll
        for (int r = 0; r < PER / R; ++r) {
            const float *p = chosen + (r * 32 + lane) * R;
            if constexpr (R % 4 == 0) {
#pragma unroll
                for (int j = 0; j < R; j += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(p + j);
                    d[r * R + j] = v.x;
                    d[r * R + j + 1] = v.y;
                    d[r * R + j + 2] = v.z;
                    d[r * R + j + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < R; ++j)
                    d[r * R + j] = p[j];
            }
        }
        __syncwarp();
        if (!a.renormalize) {
            // a NaN logit does not reach the maximum, but makes the sum NaN
            float most = -INFINITY;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                most = fmaxf(most, x[q][i]);
            const uint32_t key = __reduce_max_sync(kAll, logit_key(most));
            const float m = key > kKeyNone ? key_logit(key) : 0.0f;
            // expf, not exp_term: here a term is a probability as well, of which that
            // one is off by |d| 2^-24 and 0 below 2^-126 (it took 12.2 us, not 13.2)
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                x[q][i] = expf(x[q][i] - m);
                sum += x[q][i];
            }
            sum = warp_sum(sum);
            if (sum != 0.0f) {  // else no expert is left: zeros
                const float f = __fdiv_rn(-mean, sum);
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    d[i] = fmaf(f, x[q][i], d[i]);
            }
        }
        char *row = static_cast<char *>(a.dlogits) + t * a.experts * kEs;
#pragma unroll
        for (int r = 0; r < PER / R; ++r) {
            const int e = (r * 32 + lane) * R;
            typename Pack<DT, kEs>::Raw v[R];
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const float one[1] = {d[r * R + j]};
                v[j] = narrow_pack<DT, kEs>(one);
            }
            if (a.experts % R == 0) {
                Raw raw;
                memcpy(&raw, v, sizeof(raw));
                if (e < a.experts && LPC_WRITE_OK(row + e * kEs, R * kEs))
                    *reinterpret_cast<Raw *>(row + e * kEs) = raw;
            } else {
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (e + j < a.experts)
                        store_pack<DT, kEs>(row, e + j, v[j]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Stable counting sort. The slots are cut into chunks, one CTA each. With more
// than one chunk a first launch counts the experts of each chunk; the placing
// launch adds up the counts of the chunks before its own, so that no CTA waits
// on another, then each of its warps takes a contiguous part of the chunk and
// gives its slots their ranks in order, 32 at a time. Integer sums only: the
// result does not depend on the order in which anything runs. Latency bounds it:
// 4.6 us for 256 slots in one launch, 6.3 for 32768 and 7.0 for 131072 in two.
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
        store_i32(a.chunk_counts + static_cast<size_t>(e) * a.chunks + blockIdx.x, hist[e]);
}

__global__ void __launch_bounds__(kThreads) sort_place_kernel(const SortArgs a)
{
    // next[w][e]: rank within expert e of warp w's next slot
    __shared__ int next[kWarpsPerCta][LPCOLL_MAX_EXPERTS];
    // first row of an expert; before that, its slots in the chunks before
    __shared__ int first[LPCOLL_MAX_EXPERTS];
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
    if (a.chunks > 1) {
        // slots of each expert in all chunks, and in those before this one: a
        // warp for kAhead experts at a time, a lane per chunk
        constexpr int kAhead = 4, kSteps = kSortMaxChunks / 32;
        for (int e0 = warp * kAhead; e0 < E; e0 += kWarpsPerCta * kAhead) {
            int v[kAhead][kSteps];
#pragma unroll
            for (int q = 0; q < kAhead; ++q)
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const int c = i * 32 + lane;
                    v[q][i] = e0 + q < E && c < a.chunks
                                  ? load_i32(a.chunk_counts +
                                             static_cast<size_t>(e0 + q) * a.chunks + c)
                                  : 0;
                }
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                int sum = 0, before = 0;
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    sum += v[q][i];
                    before += i * 32 + lane < static_cast<int>(blockIdx.x) ? v[q][i] : 0;
                }
                sum = __reduce_add_sync(kAll, sum);
                before = __reduce_add_sync(kAll, before);
                if (lane == 0 && e0 + q < E) {
                    total[e0 + q] = sum;
                    first[e0 + q] = before;
                }
            }
        }
        __syncthreads();
    }
    for (int e = tid; e < E; e += kThreads) {
        int run = a.chunks > 1 ? first[e] : 0;
#pragma unroll
        for (int w = 0; w < kWarpsPerCta; ++w) {
            const int v = next[w][e];
            next[w][e] = run;
            run += v;
        }
        if (a.chunks == 1)
            total[e] = run;
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

size_t token_ctas(size_t tokens, int per_warp)
{
    const size_t per_cta = static_cast<size_t>(kWarpsPerCta) * per_warp;
    return (tokens + per_cta - 1) / per_cta;
}

template <int DT, int PER>
cudaError_t route_per(const RouteArgs &a, bool backward, cudaStream_t st)
{
    if (backward)
        return launch_kernel_block(route_backward_kernel<DT, PER>,
                                   token_ctas(a.tokens, kPairs<PER>), kThreads, 0, st, a);
    const size_t ctas = token_ctas(a.tokens, 1);
    if constexpr (PER >= kFew) {
        if (a.topk <= kFew)
            return launch_kernel_block(route_kernel<DT, PER, kFew>, ctas, kThreads, 0, st, a);
    }
    return launch_kernel_block(route_kernel<DT, PER, LPCOLL_MAX_TOPK>, ctas, kThreads, 0, st, a);
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
