// lpcoll_balance.cu -- the balance loss of a router (expert_balance) and its
// gradient.
//
//   p_t = softmax(z_t);  P = sum of p_t, n_e = slots at expert e, over valid tokens
//   loss = c E sum_e (n_e / S) (P_e / V),   S = sum_e n_e, V valid tokens
//   dz_tj = dloss (c E / (S V)) p_tj (n_j - sum_e n_e p_te)
//
// One warp per token, its lanes' probabilities added up in registers over the
// warp's tokens. A CTA adds up its warps in order and leaves one row of sums and
// counts; the rows meet in one cluster, which adds them in order, so the same call
// gives the same bits. Few tokens take that cluster alone: its CTAs make the rows
// too, with a cluster barrier in between.
#include "lpcoll_logits.cuh"

namespace lpc {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kSms = 152;
constexpr int kWide = 1024;            // threads of a CTA that makes sums
constexpr int kWarps = kWide / 32;
constexpr int kJoin = 8;               // CTAs of the cluster that joins the rows
constexpr int kRows = 8;               // warps whose sums are in shared memory at a time
constexpr size_t kOneLaunch = 1024;    // tokens that the cluster takes alone

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
        v = fmaxf(v, __shfl_xor_sync(kAll, v, m));
    return v;
}

__device__ __forceinline__ bool is_valid(const BalanceArgs &a, size_t t)
{
    return a.valid == nullptr || (LPC_READ_OK(a.valid + t, 1) && a.valid[t] != 0);
}

// Softmax of a token in place; all zeros where no logit is above -infinity.
template <int PER> __device__ __forceinline__ void softmax(float (&x)[PER])
{
    float m = x[0];
#pragma unroll
    for (int i = 1; i < PER; ++i)
        m = fmaxf(m, x[i]);
    m = warp_max(m);
    // a NaN logit is no maximum, but its term is NaN, and so is the sum
    if (m == -INFINITY)
        m = 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        x[i] = expf(x[i] - m);
        sum += x[i];
    }
    sum = warp_sum(sum);
    const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
#pragma unroll
    for (int i = 0; i < PER; ++i)
        x[i] = x[i] * inv;
}

// Row `cta` of the workspace: sums [experts], then counts [experts] and the number
// of valid tokens.
__device__ __forceinline__ float *sums_row(const BalanceArgs &a, int cta)
{
    return a.rows + static_cast<size_t>(cta) * (2 * a.experts + 1);
}

struct MakeSmem {
    float part[kRows][LPCOLL_MAX_EXPERTS];
    int hist[LPCOLL_MAX_EXPERTS];
    int tokens;
};

// The sums and counts of the tokens of CTA `cta` of `ctas`.
template <int DT, int PER>
__device__ __forceinline__ void make_row(const BalanceArgs &a, MakeSmem &sm, int cta, int ctas)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < a.experts; e += kWide)
        sm.hist[e] = 0;
    if (tid == 0)
        sm.tokens = 0;
    __syncthreads();
    float acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        acc[i] = 0.0f;
    int tokens = 0;
    const size_t step = static_cast<size_t>(ctas) * kWarps;
    for (size_t t = static_cast<size_t>(cta) * kWarps + warp; t < a.tokens; t += step) {
        if (!is_valid(a, t))
            continue;
        ++tokens;
        float x[PER];
        load_logits<DT, PER>(a.logits, t, a.experts, lane, x);
        if (lane < a.topk) {
            const int e = load_i32(a.ids + t * a.topk + lane);
            if (static_cast<unsigned>(e) < static_cast<unsigned>(a.experts))
                atomicAdd(&sm.hist[e], 1);
        }
        softmax(x);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            acc[i] += x[i];
    }
    if (lane == 0 && tokens != 0)
        atomicAdd(&sm.tokens, tokens);
    float sum = 0.0f;  // of expert tid
    for (int w0 = 0; w0 < kWarps; w0 += kRows) {
        if (warp >= w0 && warp < w0 + kRows)
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = expert_of<DT, PER>(i, lane);
                if (e < a.experts)
                    sm.part[warp - w0][e] = acc[i];
            }
        __syncthreads();
        if (tid < a.experts)
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                sum += sm.part[r][tid];
        __syncthreads();
    }
    float *const row = sums_row(a, cta);
    int32_t *const counts = reinterpret_cast<int32_t *>(row) + a.experts;
    if (tid < a.experts) {
        store_f32(row + tid, sum);
        store_i32(counts + tid, sm.hist[tid]);
    }
    if (tid == 0)
        store_i32(counts + a.experts, sm.tokens);
}

struct JoinSmem {
    float sums[kWarps][33];
    int counts[kWarps][33];
    float dot[kWarps];        // sum of n_e P_e, of a warp's experts
    long long slots[kWarps];  // and of n_e
    float cta_dot;
    long long cta_slots;
};

__device__ __forceinline__ unsigned join_rank()
{
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void join_barrier()
{
    asm volatile("barrier.cluster.arrive.release;\n\t"
                 "barrier.cluster.wait.acquire;" ::: "memory");
}

template <class T> __device__ __forceinline__ T join_load(const T *p, unsigned rank)
{
    static_assert(sizeof(T) == 4 || sizeof(T) == 8, "one 32- or 64-bit value");
    const uint32_t local = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    T v;
    if constexpr (sizeof(T) == 4) {
        uint32_t raw;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(raw) : "r"(remote) : "memory");
        memcpy(&v, &raw, 4);
    } else {
        unsigned long long raw;
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(raw) : "r"(remote) : "memory");
        memcpy(&v, &raw, 8);
    }
    return v;
}

// Adds up the rows, 32 experts of a CTA of the cluster at a time: 32 warps take
// every 32nd row, and a warp adds up an expert's 32.
__device__ __forceinline__ void join_rows(const BalanceArgs &a, JoinSmem &sm, int rows)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int E = a.experts;
    const unsigned rank = join_rank();
    float dot = 0.0f;
    long long slots = 0;
    for (int e0 = static_cast<int>(rank) * 32; e0 < E; e0 += kJoin * 32) {
        float sum = 0.0f;
        int count = 0;
        if (e0 + lane < E) {
#pragma unroll 10
            for (int r = warp; r < rows; r += kWarps) {
                const float *row = sums_row(a, r) + e0 + lane;
                sum += load_f32(row);
                count += load_i32(reinterpret_cast<const int32_t *>(row) + E);
            }
        }
        sm.sums[warp][lane] = sum;
        sm.counts[warp][lane] = count;
        __syncthreads();
        sum = warp_sum(sm.sums[lane][warp]);
        count = __reduce_add_sync(kAll, sm.counts[lane][warp]);
        if (lane == 0 && e0 + warp < E) {
            store_f32(a.prob_sums + e0 + warp, sum);
            store_i32(a.counts + e0 + warp, count);
            dot = fmaf(static_cast<float>(count), sum, dot);
            slots += count;
        }
        __syncthreads();
    }
    if (lane == 0) {
        sm.dot[warp] = dot;
        sm.slots[warp] = slots;
    }
    __syncthreads();
    if (tid == 0) {
        float d = 0.0f;
        long long s = 0;
        for (int w = 0; w < kWarps; ++w) {
            d += sm.dot[w];
            s += sm.slots[w];
        }
        sm.cta_dot = d;
        sm.cta_slots = s;
    }
    join_barrier();
    if (rank == 0 && warp == 0) {
        int tokens = 0;
        for (int r = lane; r < rows; r += 32)
            tokens += load_i32(reinterpret_cast<const int32_t *>(sums_row(a, r)) + 2 * E);
        tokens = __reduce_add_sync(kAll, tokens);
        if (lane == 0) {
            float d = 0.0f;
            long long s = 0;
            for (unsigned c = 0; c < kJoin; ++c) {
                d += join_load(&sm.cta_dot, c);
                s += join_load(&sm.cta_slots, c);
            }
            const float of = static_cast<float>(s) * static_cast<float>(tokens);
            store_i32(a.counts + E, tokens);
            store_f32(a.loss, of == 0.0f ? 0.0f
                                         : __fdiv_rn(a.coef * static_cast<float>(E) * d, of));
        }
    }
    join_barrier();  // no CTA leaves while its sums are read
}

template <int DT, int PER>
__global__ void __launch_bounds__(kWide) balance_rows_kernel(const __grid_constant__ BalanceArgs a)
{
    wait_prior_grid();
    __shared__ MakeSmem sm;
    make_row<DT, PER>(a, sm, blockIdx.x, gridDim.x);
}

__global__ void __launch_bounds__(kWide) balance_join_kernel(const __grid_constant__ BalanceArgs a, int rows)
{
    wait_prior_grid();
    __shared__ JoinSmem sm;
    join_rows(a, sm, rows);
}

template <int DT, int PER>
__global__ void __launch_bounds__(kWide) balance_one_kernel(const __grid_constant__ BalanceArgs a)
{
    wait_prior_grid();
    __shared__ union {
        MakeSmem make;
        JoinSmem join;
    } sm;
    make_row<DT, PER>(a, sm.make, blockIdx.x, kJoin);
    join_barrier();  // the rows are in global memory, and shared memory is free
    join_rows(a, sm.join, kJoin);
}

// Gradient: a warp per token, with the counts of its experts in registers.
template <int DT, int PER>
__global__ void __launch_bounds__(kThreads)
balance_backward_kernel(const __grid_constant__ BalanceArgs a)
{
    wait_prior_grid();
    constexpr int R = kRun<DT, PER>;
    constexpr int kEs = kOne<DT>;
    using Raw = typename RunBytes<R * kEs>::Raw;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.experts;
    float n[PER], all = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = expert_of<DT, PER>(i, lane);
        n[i] = e < E ? static_cast<float>(load_i32(a.counts + e)) : 0.0f;
        all += n[i];
    }
    const float of = warp_sum(all) * static_cast<float>(load_i32(a.counts + E));
    const float rate =
        of == 0.0f ? 0.0f
                   : __fdiv_rn(load_f32(a.dloss) * a.coef * static_cast<float>(E), of);
    const size_t step = static_cast<size_t>(gridDim.x) * kWarpsPerCta;
    for (size_t t = static_cast<size_t>(blockIdx.x) * kWarpsPerCta + warp; t < a.tokens; t += step) {
        const bool valid = is_valid(a, t);
        if (!valid && a.accumulate)
            continue;
        float x[PER];
        if (valid) {
            load_logits<DT, PER>(a.logits, t, E, lane, x);
            softmax(x);
            float mean = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                mean = fmaf(n[i], x[i], mean);
            mean = warp_sum(mean);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                x[i] = of == 0.0f ? 0.0f : rate * x[i] * (n[i] - mean);
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                x[i] = 0.0f;
        }
        if (a.accumulate) {
            float y[PER];
            load_logits<DT, PER>(a.dlogits, t, E, lane, y);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                x[i] += y[i];
        }
        char *const row = static_cast<char *>(a.dlogits) + t * E * kEs;
#pragma unroll
        for (int r = 0; r < PER / R; ++r) {
            const int e = (r * 32 + lane) * R;
            typename Pack<DT, kEs>::Raw v[R];
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const float one[1] = {x[r * R + j]};
                v[j] = narrow_pack<DT, kEs>(one);
            }
            if (E % R == 0) {
                if (e < E && LPC_WRITE_OK(row + e * kEs, R * kEs)) {
                    Raw raw;
                    memcpy(&raw, v, sizeof(raw));
                    *reinterpret_cast<Raw *>(row + e * kEs) = raw;
                }
            } else {
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (e + j < E)
                        store_pack<DT, kEs>(row, e + j, v[j]);
            }
        }
    }
}

template <int DT, int PER>
cudaError_t balance_per(const BalanceArgs &a, bool backward, cudaStream_t st)
{
    if (backward) {
        const size_t need = (a.tokens + kWarpsPerCta - 1) / kWarpsPerCta;
        const size_t most = static_cast<size_t>(kSms) * 8;
        return launch_kernel_block(balance_backward_kernel<DT, PER>, need < most ? need : most,
                                   kThreads, 0, st, a);
    }
    const int rows = balance_rows(a.tokens);
    if (rows == 1)
        return launch_kernel_cluster(balance_one_kernel<DT, PER>, kJoin, kWide, kJoin, 0, st, a);
    const cudaError_t e =
        launch_kernel_block(balance_rows_kernel<DT, PER>, rows, kWide, 0, st, a);
    if (e != cudaSuccess)
        return e;
    return launch_kernel_cluster(balance_join_kernel, kJoin, kWide, kJoin, 0, st, a, rows);
}

// Logits per lane: the smallest power of two that holds the experts.
template <int DT> cudaError_t balance_dt(const BalanceArgs &a, bool backward, cudaStream_t st)
{
    if (a.experts <= 64)
        return balance_per<DT, 2>(a, backward, st);
    if (a.experts <= 128)
        return balance_per<DT, 4>(a, backward, st);
    if (a.experts <= 256)
        return balance_per<DT, 8>(a, backward, st);
    if (a.experts <= 512)
        return balance_per<DT, 16>(a, backward, st);
    return balance_per<DT, 32>(a, backward, st);
}

}  // namespace

int balance_rows(size_t tokens)
{
    if (tokens <= kOneLaunch)
        return 1;
    const size_t need = (tokens + kWarps - 1) / kWarps;
    const size_t most = static_cast<size_t>(kSms) * 2;
    return static_cast<int>(need < most ? need : most);
}

size_t balance_workspace(size_t tokens, int experts)
{
    const int rows = balance_rows(tokens);
    return static_cast<size_t>(rows == 1 ? kJoin : rows) * (2 * experts + 1) * sizeof(float);
}

cudaError_t launch_balance(const BalanceArgs &a, cudaStream_t st)
{
    return a.dtype == LPCOLL_F32 ? balance_dt<LPCOLL_F32>(a, false, st)
                                 : balance_dt<LPCOLL_BF16>(a, false, st);
}

cudaError_t launch_balance_backward(const BalanceArgs &a, cudaStream_t st)
{
    return a.dtype == LPCOLL_F32 ? balance_dt<LPCOLL_F32>(a, true, st)
                                 : balance_dt<LPCOLL_BF16>(a, true, st);
}

}  // namespace lpc
