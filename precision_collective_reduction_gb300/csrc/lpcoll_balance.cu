// lpcoll_balance.cu -- the balance loss of a router (expert_balance) and its
// gradient.
//
//   p_t = softmax(z_t);  P = sum of p_t, n_e = slots at expert e, over valid tokens
//   loss = c E sum_e (n_e / S) (P_e / V),   S = sum_e n_e, V valid tokens
//   dz_tj = dloss (c E / (S V)) p_tj (n_j - sum_e n_e p_te)
//
// 8 to 32 lanes per token, at 8 experts a lane and more, add up its probabilities in
// registers over their tokens. A CTA adds up its warps in order and leaves one row of sums and
// counts; the rows meet in one cluster, which adds them in order, so the same call
// gives the same bits. Few tokens take that cluster alone: its CTAs read one another's
// rows from shared memory.
//
// Measured on one GB300, 32768 tokens of 256 FP32 logits (5.1 us of bytes): 16.0 us, some
// 11 for the rows (62% issue active at half of the warps: exponentials and the two warp-wide
// steps of a softmax) and 5 for the cluster (latency); the gradient 12.1 us (9.9). 512 tokens
// of 64 BF16: 5.9 us in one launch (latency). 8192 tokens of 1024 FP32: 24.4 us (5.0), with 32
// logits and 32 sums a lane, which spill at 64 registers, and 152 rows of 2049 numbers. Tried
// with the hardware's 2^x, which took 14.6 us at the first size but loses digits of small
// probabilities: two CTAs of rows per SM 18.6 us, a warp per token for 64 experts 12.8 instead
// of 9.1 (32768 tokens), the next tokens' logits ahead 15.5 (spills).
#include "lpcoll_logits.cuh"

namespace lpc {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kSms = 152;
constexpr int kWide = 1024;            // threads of a CTA that makes sums
constexpr int kWarps = kWide / 32;
constexpr int kJoin = 8;               // CTAs of the cluster that joins the rows
constexpr int kRows = 8;               // warps whose sums are in shared memory at a time
// Tokens that the cluster takes alone: 512 of 64 BF16 6.6 us, two launches 7.5; of 256 FP32
// 7.2 and 7.5, 1024 of them 9.5 and 7.5; 512 of 1000 17 and 16.
constexpr size_t kOneLaunch = 512;

// Largest of, and sum over, the G lanes of a token; the same bits in each.
template <int G> __device__ __forceinline__ float group_largest(float v)
{
#pragma unroll
    for (int m = G / 2; m >= 1; m >>= 1)
        v = fmaxf(v, __shfl_xor_sync(kAll, v, m));
    return v;
}
template <int G> __device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int m = G / 2; m >= 1; m >>= 1)
        v += __shfl_xor_sync(kAll, v, m);
    return v;
}

__device__ __forceinline__ bool is_valid(const BalanceArgs &a, size_t t)
{
    return a.valid == nullptr || (LPC_READ_OK(a.valid + t, 1) && a.valid[t] != 0);
}

// Softmax of N tokens in place, side by side; all zeros where no logit is above
// -infinity. The same for the loss and its gradient, with expf: small probabilities have
// all their digits.
template <int PER, int G, int N> __device__ __forceinline__ void softmax(float (&x)[N][PER])
{
    float m[N], sum[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        m[u] = x[u][0];
#pragma unroll
        for (int i = 1; i < PER; ++i)
            m[u] = fmaxf(m[u], x[u][i]);
    }
#pragma unroll
    for (int u = 0; u < N; ++u)
        m[u] = group_largest<G>(m[u]);
#pragma unroll
    for (int u = 0; u < N; ++u) {
        // a NaN logit is no maximum, but its term is NaN, and so is the sum
        if (m[u] == -INFINITY)
            m[u] = 0.0f;
        sum[u] = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            x[u][i] = expf(x[u][i] - m[u]);
            sum[u] += x[u][i];
        }
    }
#pragma unroll
    for (int u = 0; u < N; ++u)
        sum[u] = group_sum<G>(sum[u]);
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const float inv = sum[u] == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum[u]);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            x[u][i] = x[u][i] * inv;
    }
}

// Loads the logits of token t if `there`, else -infinity.
template <int DT, int PER, int G>
__device__ __forceinline__ void load_token(const BalanceArgs &a, const void *logits, size_t t,
                                           bool there, int lane, float (&x)[PER])
{
    if (there) {
        load_logits<DT, PER, G>(logits, t, a.experts, lane, x);
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            x[i] = -INFINITY;
    }
}

// Tokens that the lanes of a token take at a time, so that their loads and sums do
// not wait for one another.
template <int PER> constexpr int kPair = PER <= 8 ? 2 : 1;

// Row `cta` of the workspace: sums [experts], then counts [experts] and the number
// of valid tokens.
__device__ __forceinline__ float *sums_row(const BalanceArgs &a, int cta)
{
    return a.rows + static_cast<size_t>(cta) * (2 * a.experts + 1);
}

struct MakeSmem {
    float part[kRows][LPCOLL_MAX_EXPERTS];
    float sums[LPCOLL_MAX_EXPERTS];
    int hist[LPCOLL_MAX_EXPERTS];
    int tokens;
};

// The sums and counts of the tokens of CTA `cta` of `ctas`, left in shared memory.
template <int DT, int PER, int G>
__device__ __forceinline__ void make_row(const BalanceArgs &a, MakeSmem &sm, int cta, int ctas)
{
    constexpr int N = kPair<PER>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int place = lane % G;  // among the token's lanes
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
    const size_t step = static_cast<size_t>(ctas) * (kWide / G);
    const size_t first = static_cast<size_t>(cta) * (kWide / G);  // of the CTA
    for (size_t t0 = first; t0 < a.tokens; t0 += N * step) {
        float x[N][PER];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const size_t t = t0 + u * step + tid / G;
            const bool there = t < a.tokens && is_valid(a, t);
            load_token<DT, PER, G>(a, a.logits, t, there, place, x[u]);
            if (there) {
                tokens += place == 0 ? 1 : 0;
                for (int k = place; k < a.topk; k += G) {
                    const int e = load_i32(a.ids + t * a.topk + k);
                    if (static_cast<unsigned>(e) < static_cast<unsigned>(a.experts))
                        atomicAdd(&sm.hist[e], 1);
                }
            }
        }
        softmax<PER, G, N>(x);
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int i = 0; i < PER; ++i)
                acc[i] += x[u][i];
    }
    // the tokens of a warp
#pragma unroll
    for (int m = G; m < 32; m <<= 1)
#pragma unroll
        for (int i = 0; i < PER; ++i)
            acc[i] += __shfl_xor_sync(kAll, acc[i], m);
    tokens = __reduce_add_sync(kAll, tokens);
    if (lane == 0 && tokens != 0)
        atomicAdd(&sm.tokens, tokens);
    float sum = 0.0f;  // of expert tid
    for (int w0 = 0; w0 < kWarps; w0 += kRows) {
        if (warp >= w0 && warp < w0 + kRows)
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = expert_of<DT, PER, G>(i, place);
                if (lane < G && e < a.experts)
                    sm.part[warp - w0][e] = acc[i];
            }
        __syncthreads();
        if (tid < a.experts)
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                sum += sm.part[r][tid];
        __syncthreads();
    }
    if (tid < a.experts)
        sm.sums[tid] = sum;
}

// What the CTAs of a cluster make the loss from.
struct LossSmem {
    float dot[kWarps];  // sum of n_e P_e, of a warp's experts
    int slots[kWarps];  // and of n_e
    float cta_dot;
    int cta_slots;
};

struct JoinSmem {
    float sums[kWarps][33];
    int counts[kWarps][33];
    LossSmem loss;
};

// A kernel has 48 KB of static shared memory for certain.
constexpr size_t kStaticSmem = 48 * 1024;
static_assert(sizeof(MakeSmem) + sizeof(LossSmem) <= kStaticSmem, "balance_one_kernel's");
static_assert(sizeof(JoinSmem) <= kStaticSmem, "balance_join_kernel's");

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

__device__ __forceinline__ uint32_t join_address(const void *p, unsigned rank)
{
    const uint32_t local = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    return remote;
}

__device__ __forceinline__ float join_load(const float *p, unsigned rank)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(join_address(p, rank)) : "memory");
    return v;
}

__device__ __forceinline__ int join_load(const int *p, unsigned rank)
{
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(join_address(p, rank)) : "memory");
    return v;
}

// The loss, from each warp's part of sum n_e P_e and sum n_e (in its lane 0). All
// threads of the cluster come here; the first thread of all has `tokens`.
__device__ __forceinline__ void write_loss(const BalanceArgs &a, LossSmem &sm, unsigned rank,
                                           float dot, int slots, int tokens)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (lane == 0) {
        sm.dot[warp] = dot;
        sm.slots[warp] = slots;
    }
    __syncthreads();
    if (warp == 0) {
        dot = warp_sum(sm.dot[lane]);
        slots = __reduce_add_sync(kAll, sm.slots[lane]);
        if (lane == 0) {
            sm.cta_dot = dot;
            sm.cta_slots = slots;
        }
    }
    join_barrier();
    if (rank == 0 && warp == 0) {
        dot = warp_sum(lane < kJoin ? join_load(&sm.cta_dot, lane) : 0.0f);
        slots = __reduce_add_sync(kAll, lane < kJoin ? join_load(&sm.cta_slots, lane) : 0);
        if (lane == 0) {
            const float of = static_cast<float>(slots) * static_cast<float>(tokens);
            store_i32(a.counts + a.experts, tokens);
            store_f32(a.loss, of == 0.0f ? 0.0f
                                         : __fdiv_rn(a.coef * static_cast<float>(a.experts) * dot, of));
        }
    }
    join_barrier();  // no CTA leaves while its sums are read
}

// Adds up the rows, 32 experts of a CTA of the cluster at a time: 32 warps take
// every 32nd row, and a warp adds up an expert's 32.
__device__ __forceinline__ void join_rows(const BalanceArgs &a, JoinSmem &sm, int rows)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int E = a.experts;
    const unsigned rank = join_rank();
    int tokens = 0;
    if (rank == 0 && warp == 0) {
#pragma unroll 5
        for (int r = lane; r < rows; r += 32)
            tokens += load_i32(reinterpret_cast<const int32_t *>(sums_row(a, r)) + 2 * E);
        tokens = __reduce_add_sync(kAll, tokens);
    }
    float dot = 0.0f;
    int slots = 0;
    for (int e0 = static_cast<int>(rank) * 32; e0 < E; e0 += kJoin * 32) {
        float sum = 0.0f;
        int count = 0;
        if (e0 + lane < E) {
#pragma unroll 5
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
    write_loss(a, sm.loss, rank, dot, slots, tokens);
}

template <int DT, int PER, int G>
__global__ void __launch_bounds__(kWide) balance_rows_kernel(const __grid_constant__ BalanceArgs a)
{
    wait_prior_grid();
    __shared__ MakeSmem sm;
    make_row<DT, PER, G>(a, sm, blockIdx.x, gridDim.x);
    float *const row = sums_row(a, blockIdx.x);
    int32_t *const counts = reinterpret_cast<int32_t *>(row) + a.experts;
    const int tid = threadIdx.x;
    if (tid < a.experts) {
        store_f32(row + tid, sm.sums[tid]);
        store_i32(counts + tid, sm.hist[tid]);
    }
    if (tid == 0)
        store_i32(counts + a.experts, sm.tokens);
}

__global__ void __launch_bounds__(kWide) balance_join_kernel(const __grid_constant__ BalanceArgs a, int rows)
{
    wait_prior_grid();
    __shared__ JoinSmem sm;
    join_rows(a, sm, rows);
}

// Few tokens: the CTAs of one cluster make their rows and read them from one another's
// shared memory, each an eighth of the experts.
template <int DT, int PER, int G>
__global__ void __launch_bounds__(kWide) balance_one_kernel(const __grid_constant__ BalanceArgs a)
{
    wait_prior_grid();
    __shared__ MakeSmem sm;
    __shared__ LossSmem of_loss;
    make_row<DT, PER, G>(a, sm, blockIdx.x, kJoin);
    join_barrier();
    const unsigned rank = join_rank();
    const int tid = threadIdx.x, each = (a.experts + kJoin - 1) / kJoin;
    const int e = static_cast<int>(rank) * each + tid;
    float dot = 0.0f;
    int slots = 0, tokens = 0;
    if (tid < each && e < a.experts) {
        float p[kJoin];
#pragma unroll
        for (unsigned c = 0; c < kJoin; ++c) {
            p[c] = join_load(&sm.sums[e], c);
            slots += join_load(&sm.hist[e], c);
        }
        float sum = 0.0f;
#pragma unroll
        for (unsigned c = 0; c < kJoin; ++c)
            sum += p[c];
        store_f32(a.prob_sums + e, sum);
        store_i32(a.counts + e, slots);
        dot = static_cast<float>(slots) * sum;
    }
    if (rank == 0 && tid == 0)
#pragma unroll
        for (unsigned c = 0; c < kJoin; ++c)
            tokens += join_load(&sm.tokens, c);
    // write_loss ends with a barrier of the cluster, behind all of these reads
    write_loss(a, of_loss, rank, warp_sum(dot), __reduce_add_sync(kAll, slots), tokens);
}

// Gradient: the counts of a lane's experts stay in its registers.
template <int DT, int PER, int G>
__global__ void __launch_bounds__(kThreads)
balance_backward_kernel(const __grid_constant__ BalanceArgs a)
{
    wait_prior_grid();
    constexpr int N = kPair<PER>;
    constexpr int R = kRun<DT, PER>;
    constexpr int kEs = kOne<DT>;
    using Raw = typename RunBytes<R * kEs>::Raw;
    const int place = threadIdx.x % G;
    const int E = a.experts;
    float n[PER], all = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = expert_of<DT, PER, G>(i, place);
        n[i] = e < E ? static_cast<float>(load_i32(a.counts + e)) : 0.0f;
        all += n[i];
    }
    const float of = group_sum<G>(all) * static_cast<float>(load_i32(a.counts + E));
    const float rate =
        of == 0.0f ? 0.0f
                   : __fdiv_rn(load_f32(a.dloss) * a.coef * static_cast<float>(E), of);
    const size_t step = static_cast<size_t>(gridDim.x) * (kThreads / G);
    const size_t first = static_cast<size_t>(blockIdx.x) * (kThreads / G);
    for (size_t t0 = first; t0 < a.tokens; t0 += N * step) {
        float x[N][PER];
        bool there[N], valid[N];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const size_t t = t0 + u * step + threadIdx.x / G;
            there[u] = t < a.tokens;
            valid[u] = there[u] && is_valid(a, t);
            load_token<DT, PER, G>(a, a.logits, t, valid[u], place, x[u]);
        }
        softmax<PER, G, N>(x);
        float mean[N];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            mean[u] = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                mean[u] = fmaf(n[i], x[u][i], mean[u]);
        }
#pragma unroll
        for (int u = 0; u < N; ++u)
            mean[u] = group_sum<G>(mean[u]);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            if (!there[u] || (a.accumulate && !valid[u]))
                continue;
            const size_t t = t0 + u * step + threadIdx.x / G;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                // padding is 0 beside an infinite rate too
                x[u][i] = of == 0.0f || !valid[u] ? 0.0f : rate * x[u][i] * (n[i] - mean[u]);
            if (a.accumulate) {
                float y[PER];
                load_logits<DT, PER, G>(a.dlogits, t, E, place, y);
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    x[u][i] += y[i];
            }
            char *const row = static_cast<char *>(a.dlogits) + t * E * kEs;
#pragma unroll
            for (int r = 0; r < PER / R; ++r) {
                const int e = (r * G + place) * R;
                typename Pack<DT, kEs>::Raw v[R];
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    const float one[1] = {x[u][r * R + j]};
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
}

template <int DT, int PER, int G>
cudaError_t balance_per(const BalanceArgs &a, bool backward, cudaStream_t st)
{
    if (backward) {
        const size_t need = (a.tokens + kThreads / G - 1) / (kThreads / G);
        const size_t most = static_cast<size_t>(kSms) * 8;
        return launch_kernel_block(balance_backward_kernel<DT, PER, G>, need < most ? need : most,
                                   kThreads, 0, st, a);
    }
    const int rows = balance_rows(a.tokens);
    if (rows == 1)
        return launch_kernel_cluster(balance_one_kernel<DT, PER, G>, kJoin, kWide, kJoin, 0, st, a);
    const cudaError_t e =
        launch_kernel_block(balance_rows_kernel<DT, PER, G>, rows, kWide, 0, st, a);
    if (e != cudaSuccess)
        return e;
    return launch_kernel_cluster(balance_join_kernel, kJoin, kWide, kJoin, 0, st, a, rows);
}

// 8 logits a lane, and lanes that hold the experts, up to a warp; then more logits.
template <int DT> cudaError_t balance_dt(const BalanceArgs &a, bool backward, cudaStream_t st)
{
    if (a.experts <= 64)
        return balance_per<DT, 8, 8>(a, backward, st);
    if (a.experts <= 128)
        return balance_per<DT, 8, 16>(a, backward, st);
    if (a.experts <= 256)
        return balance_per<DT, 8, 32>(a, backward, st);
    if (a.experts <= 512)
        return balance_per<DT, 16, 32>(a, backward, st);
    return balance_per<DT, 32, 32>(a, backward, st);
}

}  // namespace

int balance_rows(size_t tokens)
{
    if (tokens <= kOneLaunch)
        return 1;
    const size_t need = (tokens + kWarps - 1) / kWarps;
    const size_t most = kSms;
    return static_cast<int>(need < most ? need : most);
}

size_t balance_workspace(size_t tokens, int experts)
{
    const int rows = balance_rows(tokens);
    return rows == 1 ? 0 : static_cast<size_t>(rows) * (2 * experts + 1) * sizeof(float);
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
