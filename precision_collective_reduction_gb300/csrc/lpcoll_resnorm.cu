// lpcoll_resnorm.cu -- the end of a transformer block in one pass: the sum of
// the ranks' partial products, the norm after the block, gate, residual and
// the norm before the next block (residual_norm), and the gradients
// (residual_norm_backward).
//
//   h  = sum_r h_r                                    (rank order)
//   u  = h r1 w_post,   r1 = 1 / sqrt(mean h^2 + eps)   (or u = h)
//   x' = alpha x + beta g u
//   n  = x' r2 w_pre,   r2 = 1 / sqrt(mean x'^2 + eps)
//
// Every input is read and every output written once; all arithmetic and sums
// are FP32, rounded once at each output. HBM traffic bounds both directions
// once there are enough tokens.
//
// A row belongs to a "team" of whole warps: a part of a CTA for short rows, a
// CTA, or the CTAs of a cluster, which add up their sums through distributed
// shared memory. A thread of a team always holds the same columns, so what
// the weights and gates of a channel give stays in its registers, and a team
// goes through its rows one after the other while its next rows are on their
// way into shared memory (cp.async): each thread copies and reads its own
// columns only, so no barrier guards them. Where shared memory holds one row of a
// team (8 ranks of 4096 or 8192 BF16 columns, the FP32 gradient of 8192), a forward
// team sends for its next row once this one's columns are read, before the sums
// meet, and a gradient's team at the row's end. Rows of that many bytes keep DRAM
// busy all the same: 8192 x 8192 of 8 ranks 238 us, 4096 x 8192 FP32 gradient 132 us
// (bytes at the copy rate: 238 and 119).
//
// Measured on one GB300, BF16: 16384 x 8192 forward 161 us (6.7 TB/s, DRAM), the
// gradient of 8192 x 8192 131 us (6.1 TB/s; a team's phases between barriers), 32
// x 8192 of 8 ranks 5.9 us (latency).
#include "lpcoll_layers.cuh"

namespace lpc {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kSms = 152;
// A thread holds kElems = 8 or 16 columns, at 64 or 128 registers, so that an SM
// holds kThreadsOne threads: a CTA, or several smaller ones. Short rows share a
// CTA of up to half as many.
template <int kElems> constexpr int kThreadsOne = 8192 / kElems;
constexpr int kWideThreads = 1024;
constexpr int kMaxWarps = kWideThreads / 32;

// Forms of both kernels. kPlain is for calls without clusters in which every
// thread has all its columns, both norms are there, one rank's h, no full gate
// and, in the gradient, dx_out: without the conditions around every access the compiler
// interleaves a thread's accesses (gradient of 8192 x 8192 BF16 143 -> 134 us). Calls
// without it pay: 16384 x 8192 BF16 with the second norm alone 216 us, with both 161.
// kWide is for the forward pass of rows of more than 8192 columns, in a CTA of
// 1024 threads with 16 columns each at 64 registers a thread, the weights from
// L1 each time (8192 x 12288 BF16: 167 us, 241 with a cluster of two CTAs and the
// weights in registers; the gradient of 4096 rows, which keeps its sums too, 268
// against 174; 180 now, the price of the unaligned cluster barriers).
enum Mode { kGeneral, kPlain, kWide };

constexpr int kMaxStages = 4;
constexpr int kMaxCluster = 8;
constexpr int kMaxCtas = 3;  // per SM

// How rows are dealt out: `threads` lanes of each of `cluster` CTAs share a
// row, `packs` accesses of it per CTA; a CTA has `groups` such teams and a
// ring of `stages` rows for each.
struct Deal {
    int threads, groups, cluster, packs, stages;
};

__device__ __forceinline__ unsigned cluster_rank()
{
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;\n\t"
                 "barrier.cluster.wait.acquire;" ::: "memory");
}

// The float at `p` of this CTA's shared memory in CTA `rank` of the cluster.
__device__ __forceinline__ float cluster_load(const float *p, unsigned rank)
{
    const uint32_t local = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    uint32_t remote;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
    return v;
}

// Waits for the threads of this team: of all CTAs of its cluster, of its CTA,
// or of its part of a CTA (barrier 1 + team of the CTA). The compiler may let a
// warp's lanes, of which some have no columns, run apart up to here. A counted
// bar.sync, an aligned form, would then count every part of a warp as a whole one
// and could open before the last warp has written its sums; so could an aligned
// cluster barrier. Hence the unaligned forms. __syncthreads() needs none: CUDA has it
// wait until every thread of the CTA has come, whatever its warp's lanes do
// (barrier.cta.sync 0 in its place: 161 -> 162 us for 16384 x 8192 BF16, the gradient
// of 8192 x 8192 131.6 -> 132.6).
__device__ __forceinline__ void team_barrier(const Deal &deal)
{
    if (deal.cluster > 1)
        cluster_barrier();
    else if (deal.groups == 1)
        __syncthreads();
    else  // teams of 64 threads or more, 8 of them at most
        asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + static_cast<int>(threadIdx.x) / deal.threads),
                     "r"(deal.threads)
                     : "memory");
}

template <int N> constexpr int kSplit = N == 1 ? 1 : (N == 2 ? 2 : 8);

// Sums over a team of N <= 8 values per thread, the same bits in every thread
// of the team and in every run. The lanes of a warp split the values between
// them (each step halves both the values a lane holds and the lanes that share
// one: 9 shuffles for 6 values instead of 30); the warps' sums then meet in
// `red`. The caller alternates between two `red`, so that one barrier per sum
// is enough. first_warp: the team's first in its CTA.
template <int N>
__device__ __forceinline__ void team_sums(float (&v)[N], float (*red)[8], const Deal &deal,
                                          int first_warp)
{
    constexpr int P = kSplit<N>;
    const int lane = threadIdx.x & 31;
    const int warps = deal.threads >> 5;
    float s[P];
#pragma unroll
    for (int i = 0; i < P; ++i)
        s[i] = i < N ? v[i < N ? i : 0] : 0.0f;
#pragma unroll
    for (int half = P / 2; half >= 1; half >>= 1) {
        const bool up = (lane & half) != 0;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float give = up ? s[i] : s[i + half];
            const float keep = up ? s[i + half] : s[i];
            s[i] = keep + __shfl_xor_sync(kAll, give, half);
        }
    }
    float sum = s[0];
#pragma unroll
    for (int m = P; m < 32; m <<= 1)
        sum += __shfl_xor_sync(kAll, sum, m);
    if (warps > 1 || deal.cluster > 1) {
        if (lane < P)
            red[threadIdx.x >> 5][lane] = sum;
        __syncwarp();
        team_barrier(deal);
        sum = 0.0f;
        if (deal.cluster == 1) {
            for (int w = lane / P; w < warps; w += 32 / P)
                sum += red[first_warp + w][lane % P];
        } else {
            for (int w = lane / P; w < warps; w += 32 / P) {
                float far[kMaxCluster];
#pragma unroll
                for (int c = 0; c < kMaxCluster; ++c)
                    far[c] = c < deal.cluster ? cluster_load(&red[w][lane % P], c) : 0.0f;
#pragma unroll
                for (int c = 0; c < kMaxCluster; ++c)
                    sum += far[c];
            }
        }
#pragma unroll
        for (int m = P; m < 32; m <<= 1)
            sum += __shfl_xor_sync(kAll, sum, m);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = P == 1 ? sum : __shfl_sync(kAll, sum, i);
}

// 1 / sqrt(mean of squares + eps); rsqrtf is good to 2 ulp.
__device__ __forceinline__ float inv_rms(float sum, float per_hidden, float eps)
{
    return rsqrtf(fmaf(sum, per_hidden, eps));
}

// N FP32 values, multiplied and added two at a time where N is even.
template <int N> struct Vec {
    float v[N];
};

template <int N> __device__ __forceinline__ Vec<N> splat(float x)
{
    Vec<N> r;
#pragma unroll
    for (int j = 0; j < N; ++j)
        r.v[j] = x;
    return r;
}

template <int N>
__device__ __forceinline__ Vec<N> mul(const Vec<N> &a, const Vec<N> &b)
{
    Vec<N> r;
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float2 p = mul_pair(make_float2(a.v[j], a.v[j + 1]),
                                      make_float2(b.v[j], b.v[j + 1]));
            r.v[j] = p.x;
            r.v[j + 1] = p.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            r.v[j] = __fmul_rn(a.v[j], b.v[j]);
    }
    return r;
}

template <int N> __device__ __forceinline__ Vec<N> mul(float a, const Vec<N> &b)
{
    return mul(splat<N>(a), b);
}

// a b + c
template <int N>
__device__ __forceinline__ Vec<N> fma(const Vec<N> &a, const Vec<N> &b, const Vec<N> &c)
{
    Vec<N> r;
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float2 p = fma_pair(make_float2(a.v[j], a.v[j + 1]),
                                      make_float2(b.v[j], b.v[j + 1]),
                                      make_float2(c.v[j], c.v[j + 1]));
            r.v[j] = p.x;
            r.v[j + 1] = p.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            r.v[j] = __fmaf_rn(a.v[j], b.v[j], c.v[j]);
    }
    return r;
}

template <int N> __device__ __forceinline__ Vec<N> fma(float a, const Vec<N> &b, const Vec<N> &c)
{
    return fma(splat<N>(a), b, c);
}

template <int N> __device__ __forceinline__ Vec<N> add(const Vec<N> &a, const Vec<N> &b)
{
    return fma(splat<N>(1.0f), a, b);
}

// Partial sums of a thread's products: two, or one where values come singly.
template <int N> using Acc = Vec<N % 2 == 0 ? 2 : 1>;

template <int N>
__device__ __forceinline__ void add_products(Acc<N> &acc, const Vec<N> &a, const Vec<N> &b)
{
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int j = 0; j < N; j += 2)
            acc = fma(Vec<2>{{a.v[j], a.v[j + 1]}}, Vec<2>{{b.v[j], b.v[j + 1]}}, acc);
    } else {
        acc = fma(a, b, acc);
    }
}

__device__ __forceinline__ float fold(const Vec<2> &a) { return a.v[0] + a.v[1]; }
__device__ __forceinline__ float fold(const Vec<1> &a) { return a.v[0]; }

template <int DT, int W>
__device__ __forceinline__ Vec<Pack<DT, W>::kN> unpack(typename Pack<DT, W>::Raw raw)
{
    Vec<Pack<DT, W>::kN> r;
    widen_pack<DT, W>(raw, r.v);
    return r;
}

template <int DT, int W>
__device__ __forceinline__ Vec<Pack<DT, W>::kN> load_vec_of(const void *base, size_t e0)
{
    return unpack<DT, W>(load_pack<DT, W>(base, e0));
}

template <int DT, int W>
__device__ __forceinline__ void store_vec_of(void *base, size_t e0,
                                             const Vec<Pack<DT, W>::kN> &x)
{
    store_pack<DT, W>(base, e0, narrow_pack<DT, W>(x.v));
}

// W (16, 8 or 4) bytes from global into this thread's place in shared memory.
template <int W>
__device__ __forceinline__ void copy_async(void *dst, const void *src)
{
    if (!LPC_READ_OK(src, W)) {
#pragma unroll
        for (int i = 0; i < W / 2; ++i)
            static_cast<uint16_t *>(dst)[i] = 0;
        return;
    }
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    if constexpr (W == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else if constexpr (W == 8)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(src) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Waits until at most `pending` of this thread's copy groups are under way.
__device__ __forceinline__ void copy_wait(int pending)
{
    static_assert(kMaxStages == 4, "one case per number of stages");
    if (pending >= 3)
        asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (pending == 2)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (pending == 1)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <int DT>
__device__ __forceinline__ float load_one(const void *base, size_t e)
{
    float one[1];
    widen_pack<DT, kOne<DT>>(load_pack<DT, kOne<DT>>(base, e), one);
    return one[0];
}

// Shared memory of a warp's part of an odd row, of kElems columns per lane: its
// words, and one more.
__host__ __device__ constexpr int odd_warp_bytes(int elems) { return elems * 32 * 2 + 16; }

// Shared memory of a CTA's part of a row, a multiple of 16 bytes.
__host__ __device__ constexpr int row_part_bytes(int width, int packs, int threads, int elems)
{
    return width == 2 ? threads / 32 * odd_warp_bytes(elems) : (packs * width + 15) & ~15;
}

// What a thread of a team works on: its warp's part of a row is kElems * 32
// consecutive columns, access c of all lanes side by side. kAlone: known to have
// no cluster (for the plain gradient 132 against 135 us at 8192 x 8192 BF16; the
// plain forward pass is compiled to a slower kernel with it, 168 against 161).
template <int DT, int W, int kElems, int kMode, bool kAlone> struct Member {
    static constexpr int kN = Pack<DT, W>::kN;
    static constexpr int NV = kElems / kN;
    int group;         // team of the CTA
    int first_warp;    // of the team
    int col0;          // first column of the thread
    int packs;         // accesses from there to the end of the CTA's part of a row
    size_t t0, step;   // first row of the team, distance to its next
    int hidden;
    char *place;       // this thread's place in the team's ring
    int row_bytes, stage_bytes;
    // Rows of an odd number of BF16 elements (W = 2): a warp copies the aligned
    // words that its columns lie in, lane for lane, and reads them from the
    // element on that the row begins with; `end` is the tensors' end.
    int warp_col;
    size_t end;

    __device__ __forceinline__ Member(const Deal &deal, const NormArgs &a, int streams, char *smem)
    {
        hidden = a.hidden;
        group = static_cast<int>(threadIdx.x) / deal.threads;
        const int id = static_cast<int>(threadIdx.x) - group * deal.threads;
        first_warp = group * (deal.threads >> 5);
        const bool alone = kAlone || deal.cluster == 1;
        const int part = alone ? 0 : static_cast<int>(cluster_rank()) * deal.packs;
        const int p0 = (id >> 5) * NV * 32 + (id & 31);
        col0 = (part + p0) * kN;
        packs = min(deal.packs, (hidden + kN - 1) / kN - part) - p0;
        step = static_cast<size_t>(alone ? gridDim.x : gridDim.x / deal.cluster) * deal.groups;
        t0 = static_cast<size_t>(alone ? blockIdx.x : blockIdx.x / deal.cluster) * deal.groups +
             group;
        row_bytes = row_part_bytes(W, deal.packs, deal.threads, kElems);
        stage_bytes = row_bytes * streams;
        place = smem + static_cast<size_t>(group) * stage_bytes * deal.stages;
        if constexpr (W == 2) {
            warp_col = part + (id >> 5) * NV * 32;
            end = a.tokens * hidden;
            place += (id >> 5) * odd_warp_bytes(kElems) + (id & 31) * W;
        } else {
            place += p0 * W;
        }
    }
    __device__ __forceinline__ bool has(int c) const { return kMode == kPlain || c * 32 < packs; }
    __device__ __forceinline__ int col(int c) const { return col0 + c * 32 * kN; }
    // Element of access c of row t.
    __device__ __forceinline__ size_t elem(size_t t, int c) const
    {
        return (t * hidden + col0) + c * 32 * kN;
    }
    // Where access c of row t is, in its stage and stream.
    __device__ __forceinline__ char *at(size_t t, int stage, int stream, int c) const
    {
        char *p = place + stage * stage_bytes + stream * row_bytes + c * 32 * W;
        if constexpr (W == 2)
            p += (t * hidden + warp_col) % 2 * W;
        return p;
    }
    __device__ __forceinline__ Vec<kN> read(size_t t, int stage, int stream, int c) const
    {
        return unpack<DT, W>(
            *reinterpret_cast<const typename Pack<DT, W>::Raw *>(at(t, stage, stream, c)));
    }
    // f w_post gate and w_pre of access c.
    __device__ __forceinline__ Vec<kN> scale(const NormArgs &a, bool post, bool channel, float f,
                                             int c) const
    {
        Vec<kN> q = splat<kN>(f);
        if (post)
            q = mul(q, load_vec_of<DT, W>(a.w_post, col(c)));
        if (channel)
            q = mul(q, load_vec_of<DT, W>(a.gate, col(c)));
        return q;
    }
    // Both for all of this thread's columns, as far as they are there. All loads
    // go out before the first value is used.
    __device__ __forceinline__ void weights(const NormArgs &a, bool post, bool channel, bool pre,
                                            float f, Vec<kN> (&wq)[NV],
                                            typename Pack<DT, W>::Raw (&wp)[NV]) const
    {
        typename Pack<DT, W>::Raw rw[NV], rg[NV];
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            rw[c] = rg[c] = wp[c] = {};
            if (has(c)) {
                if (post)
                    rw[c] = load_pack<DT, W>(a.w_post, col(c));
                if (channel)
                    rg[c] = load_pack<DT, W>(a.gate, col(c));
                if (pre)
                    wp[c] = load_pack<DT, W>(a.w_pre, col(c));
            }
        }
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            wq[c] = splat<kN>(f);
            if (post)
                wq[c] = mul(wq[c], unpack<DT, W>(rw[c]));
            if (channel)
                wq[c] = mul(wq[c], unpack<DT, W>(rg[c]));
        }
    }
    // FP32 values in the place of an access and, if its elements are shorter,
    // of the next stream's.
    __device__ __forceinline__ void keep(size_t t, int stage, int stream, int c,
                                         const Vec<kN> &x) const
    {
        using Raw = typename Pack<DT, W>::Raw;
        constexpr int kParts = kN * 4 / W;
        Raw raw[kParts];
        memcpy(raw, x.v, sizeof(x.v));
#pragma unroll
        for (int i = 0; i < kParts; ++i)
            *reinterpret_cast<Raw *>(at(t, stage, stream + i, c)) = raw[i];
    }
    __device__ __forceinline__ Vec<kN> kept(size_t t, int stage, int stream, int c) const
    {
        using Raw = typename Pack<DT, W>::Raw;
        constexpr int kParts = kN * 4 / W;
        Raw raw[kParts];
#pragma unroll
        for (int i = 0; i < kParts; ++i)
            raw[i] = *reinterpret_cast<const Raw *>(at(t, stage, stream + i, c));
        Vec<kN> x;
        memcpy(x.v, raw, sizeof(x.v));
        return x;
    }
    // Starts the copy of this thread's part of row t.
    __device__ __forceinline__ void copy(int stage, int stream, const void *base, size_t t) const
    {
        if constexpr (W >= 4) {
            using Raw = typename Pack<DT, W>::Raw;
            const Raw *src = static_cast<const Raw *>(base) + (t * hidden + col0) / kN;
#pragma unroll
            for (int c = 0; c < NV; ++c)
                if (has(c))
                    copy_async<W>(at(t, stage, stream, c), src + c * 32);
        } else {
            const int lane = static_cast<int>(threadIdx.x) & 31;
            const int n = min(packs + lane, NV * 32);  // columns of the warp
            const size_t e0 = t * hidden + warp_col, first = e0 & ~static_cast<size_t>(1);
            const int words = n > 0 ? static_cast<int>(e0 - first + n + 1) / 2 : 0;
            const uint16_t *src = static_cast<const uint16_t *>(base) + first;
            uint16_t *dst = reinterpret_cast<uint16_t *>(place + stage * stage_bytes +
                                                         stream * row_bytes) - lane;
            __syncwarp();  // the words' last readers are done
            for (int w = lane; w < words; w += 32) {
                if (first + 2 * w + 1 < end)
                    copy_async<4>(dst + 2 * w, src + 2 * w);
                else  // the tensor's last element, alone in its word
                    dst[2 * w] = load_pack<DT, 2>(src, 2 * w);
            }
        }
    }
    // Waits for a row's copies, this thread's or, where they share them, the
    // warp's.
    __device__ __forceinline__ void ready(int pending) const
    {
        copy_wait(pending);
        if constexpr (W == 2)
            __syncwarp();
    }
};

// Streams of a row: x, a full gate if there is one, then the ranks' h.
template <int DT, int W, int kElems, int kMode>
__global__ void __launch_bounds__(kMode == kWide ? kWideThreads : kThreadsOne<kElems>, 1)
residual_norm_kernel(const __grid_constant__ NormArgs a, const Deal deal, int streams)
{
    wait_prior_grid();
    extern __shared__ uint4 ring_smem[];
    __shared__ float red[2][kMaxWarps][8];
    constexpr int kN = Pack<DT, W>::kN;
    constexpr int NV = kElems / kN;
    const Member<DT, W, kElems, kMode, false> me(deal, a, streams, reinterpret_cast<char *>(ring_smem));
    const bool post = kMode == kPlain || a.w_post != nullptr;
    const bool pre = kMode == kPlain || a.w_pre != nullptr;
    const bool full = kMode != kPlain && a.gate_kind == LPCOLL_GATE_FULL;
    const int h0 = full ? 2 : 1, nranks = kMode == kPlain ? 1 : a.nranks;
    void *const h_sum = kMode == kPlain ? nullptr : a.h_sum;
    const float per_hidden = __fdiv_rn(1.0f, static_cast<float>(a.hidden));
    const auto fetch = [&](size_t t, int stage) {
        if (t < a.tokens) {
            for (int r = 0; r < nranks; ++r)
                me.copy(stage, h0 + r, a.h[r], t);
            me.copy(stage, 0, a.x, t);
            if (full)
                me.copy(stage, 1, a.gate, t);
        }
        copy_commit();
    };
    for (int s = 0; s < deal.stages; ++s)
        fetch(me.t0 + s * me.step, s);

    Vec<kN> wq[NV];  // beta w_post, times a channel's gate
    typename Pack<DT, W>::Raw wp[NV];
    const bool channel = a.gate_kind == LPCOLL_GATE_CHANNEL;
    if constexpr (kMode != kWide)
        me.weights(a, post, channel, pre, a.branch_scale, wq, wp);
    const auto scale = [&](int c) {
        if constexpr (kMode == kWide)
            return me.scale(a, post, channel, a.branch_scale, c);
        else
            return wq[c];
    };
    const auto w_pre = [&](int c) {
        if constexpr (kMode == kWide)
            return load_vec_of<DT, W>(a.w_pre, me.col(c));
        else
            return unpack<DT, W>(wp[c]);
    };

    // The ranks' sum for the row in `stage`, left in FP32 in the place of the
    // first ranks' values, and this thread's part of the sum of its squares.
    const auto sum_ranks = [&](size_t t, int stage) {
        Acc<kN> sq = {};
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
            Vec<kN> h = me.read(t, stage, h0, c);
            if (nranks > 1) {
#pragma unroll 4
                for (int r = 1; r < nranks; ++r)
                    h = add(h, me.read(t, stage, h0 + r, c));
                me.keep(t, stage, h0, c, h);
            }
            add_products(sq, h, h);
        }
        return fold(sq);
    };

    // Each turn ends row t and takes the next row's sum of squares of h with
    // its own of x', so that there is one barrier per row.
    int stage = 0, turn = 0;
    float r1 = 1.0f;
    me.ready(deal.stages - 1);
    const bool summed = post || nranks > 1;
    if (summed) {
        float s[1] = {me.t0 < a.tokens ? sum_ranks(me.t0, 0) : 0.0f};
        if (post) {
            team_sums(s, red[1], deal, me.first_warp);
            r1 = inv_rms(s[0], per_hidden, a.eps);
        }
    }
    for (size_t t = me.t0; t < a.tokens; t += me.step, turn ^= 1) {
        const float gate_t = a.gate_kind == LPCOLL_GATE_TOKEN ? load_one<DT>(a.gate, t) : 1.0f;
        const float f = r1 * gate_t;
        Vec<kN> v[NV];
        Acc<kN> sq = {};
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
            v[c] = nranks > 1 ? me.kept(t, stage, h0, c) : me.read(t, stage, h0, c);
            if (h_sum != nullptr)
                store_vec_of<DT, W>(h_sum, me.elem(t, c), v[c]);
            Vec<kN> u = mul(mul(f, scale(c)), v[c]);
            if (full)
                u = mul(u, me.read(t, stage, 1, c));
            v[c] = fma(a.res_scale, me.read(t, stage, 0, c), u);
            add_products(sq, v[c], v[c]);
            store_vec_of<DT, W>(a.x_out, me.elem(t, c), v[c]);
        }
        fetch(t + deal.stages * me.step, stage);
        stage = stage + 1 == deal.stages ? 0 : stage + 1;
        me.ready(deal.stages - 1);
        float s[2] = {fold(sq), summed && t + me.step < a.tokens ? sum_ranks(t + me.step, stage) : 0.0f};
        if (post || pre)
            team_sums(s, red[turn], deal, me.first_warp);
        r1 = post ? inv_rms(s[1], per_hidden, a.eps) : 1.0f;
        if (pre) {
            const float r2 = inv_rms(s[0], per_hidden, a.eps);
#pragma unroll
            for (int c = 0; c < NV; ++c)
                if (me.has(c))
                    store_vec_of<DT, W>(a.n_out, me.elem(t, c),
                                        mul(mul(r2, w_pre(c)), v[c]));
        }
    }
    if (kMode != kPlain && deal.cluster > 1)
        cluster_barrier();  // no CTA leaves while another reads its sums
}

// ---------------------------------------------------------------------------
// Gradients. With q = dn w_pre and c2 = r2^2 mean(q x'), the gradient of x' is
// D = dx' + r2 (q - x' c2). The gradient through the first norm needs the sum
// of beta g w_post D h, which is linear in D; so with P = g w_post h (g without
// a token's own gate) the six sums h^2, x'^2, q x', P dx', P q, P x' of one
// pass over the row give every factor of the second:
//   sum(P D) = sum(P dx') + r2 (sum(P q) - c2 sum(P x')).
// A thread keeps the sums over tokens of its columns in registers, S = sum
// beta r1 h D (times a gate that differs by token) and dw_pre = sum dn x' r2,
// and the CTA leaves them in the workspace, [2][CTAs][hidden]; a second launch
// adds those up in order: dw_post = g S, and dgate = w_post S for a gate per
// channel.
// ---------------------------------------------------------------------------

// Row streams of a stage.
enum Stream { kH = 0, kDx = 1, kX = 2, kDn = 3, kGate = 4 };

template <int DT, int W, int kElems, int kMode>
__global__ void __launch_bounds__(kThreadsOne<kElems>, 1)
residual_norm_backward_kernel(const __grid_constant__ NormArgs a, const Deal deal, int streams)
{
    wait_prior_grid();
    extern __shared__ uint4 ring_smem[];
    __shared__ float red[2][kMaxWarps][8];
    constexpr int kN = Pack<DT, W>::kN;
    constexpr int NV = kElems / kN;
    const Member<DT, W, kElems, kMode, kMode == kPlain> me(deal, a, streams, reinterpret_cast<char *>(ring_smem));
    const bool post = kMode == kPlain || a.w_post != nullptr;
    const bool pre = kMode == kPlain || a.w_pre != nullptr;
    const bool given = kMode == kPlain || a.dx_out != nullptr;
    const bool full = kMode != kPlain && a.gate_kind == LPCOLL_GATE_FULL;
    const int H = a.hidden;
    const float per_hidden = __fdiv_rn(1.0f, static_cast<float>(H));
    const auto fetch = [&](size_t t, int stage) {
        if (t < a.tokens) {
            me.copy(stage, kH, a.h[0], t);
            if (given)
                me.copy(stage, kDx, a.dx_out, t);
            if (pre) {
                me.copy(stage, kX, a.x, t);
                me.copy(stage, kDn, a.dn_out, t);
            }
            if (full)
                me.copy(stage, kGate, a.gate, t);
        }
        copy_commit();
    };
    for (int s = 0; s < deal.stages; ++s)
        fetch(me.t0 + s * me.step, s);

    Vec<kN> wq[NV];                    // w_post times a channel's gate
    typename Pack<DT, W>::Raw wp[NV];  // w_pre
    Vec<kN> S[NV], s_pre[NV];
    me.weights(a, post, a.gate_kind == LPCOLL_GATE_CHANNEL, pre, 1.0f, wq, wp);
#pragma unroll
    for (int c = 0; c < NV; ++c)
        S[c] = s_pre[c] = splat<kN>(0.0f);

    // a token's gate, read a row ahead
    const auto gate_of = [&](size_t t) {
        return a.gate_kind == LPCOLL_GATE_TOKEN && t < a.tokens ? load_one<DT>(a.gate, t) : 1.0f;
    };

    // a thread's part of the six sums of the row in `stage`
    const auto row_sums = [&](size_t t, int stage, float (&s)[6]) {
        Acc<kN> v[6] = {};
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
            const Vec<kN> h = me.read(t, stage, kH, c);
            Vec<kN> p = mul(wq[c], h);
            add_products(v[0], h, h);
            if (full)
                p = mul(p, me.read(t, stage, kGate, c));
            if (given)
                add_products(v[3], p, me.read(t, stage, kDx, c));
            if (pre) {
                const Vec<kN> x = me.read(t, stage, kX, c);
                const Vec<kN> q = mul(me.read(t, stage, kDn, c), unpack<DT, W>(wp[c]));
                add_products(v[1], x, x);
                add_products(v[2], q, x);
                add_products(v[4], p, q);
                add_products(v[5], p, x);
            }
        }
#pragma unroll
        for (int i = 0; i < 6; ++i)
            s[i] = fold(v[i]);
    };

    int stage = 0, turn = 0;
    float gate_next = gate_of(me.t0);
    for (size_t t = me.t0; t < a.tokens; t += me.step, turn ^= 1) {
        const float gate_t = gate_next;
        gate_next = gate_of(t + me.step);
        me.ready(deal.stages - 1);
        float s[6];
        row_sums(t, stage, s);
        team_sums(s, red[turn], deal, me.first_warp);
        const float r1 = post ? inv_rms(s[0], per_hidden, a.eps) : 1.0f;
        const float r2 = pre ? inv_rms(s[1], per_hidden, a.eps) : 0.0f;
        const float c2 = pre ? r2 * r2 * s[2] * per_hidden : 0.0f;
        const float pd = fmaf(r2, fmaf(-c2, s[5], s[4]), s[3]);
        const float bt = a.branch_scale * gate_t;
        // dh = f1 wq g D - f2 h;  S += f1 g h D
        const float f1 = r1 * bt;
        const float f2 = post ? r1 * (r1 * r1 * bt * pd * per_hidden) : 0.0f;
        if (a.gate_kind == LPCOLL_GATE_TOKEN && a.dgate != nullptr && me.col0 == 0)
            store_f32(static_cast<float *>(a.dgate) + t, a.branch_scale * r1 * pd);
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
            Vec<kN> d = splat<kN>(0.0f);
            if (given)
                d = me.read(t, stage, kDx, c);
            if (pre) {
                const Vec<kN> x = me.read(t, stage, kX, c), dn = me.read(t, stage, kDn, c);
                const Vec<kN> q = mul(dn, unpack<DT, W>(wp[c]));
                s_pre[c] = fma(mul(r2, dn), x, s_pre[c]);
                d = fma(r2, fma(-c2, x, q), d);
            }
            const Vec<kN> dx = mul(a.res_scale, d);
            const Vec<kN> h = me.read(t, stage, kH, c);
            if (full) {
                if (a.dgate != nullptr)
                    store_vec_of<DT, W>(a.dgate, me.elem(t, c),
                                        mul(mul(mul(f1, wq[c]), h), d));
                d = mul(d, me.read(t, stage, kGate, c));
            }
            const Vec<kN> e = mul(f1, d);
            S[c] = fma(h, e, S[c]);
            store_vec_of<DT, W>(a.dx, me.elem(t, c), dx);
            store_vec_of<DT, W>(a.dh, me.elem(t, c), fma(wq[c], e, mul(-f2, h)));
        }
        fetch(t + deal.stages * me.step, stage);
        stage = stage + 1 == deal.stages ? 0 : stage + 1;
    }
    copy_wait(0);
    if (kMode != kPlain && deal.cluster > 1)
        cluster_barrier();  // no CTA leaves while another reads its sums

    // The CTA's sums over its tokens: the groups add theirs in order in shared
    // memory (the rows are done with), then the CTA writes one row per gradient.
    if (a.partial == nullptr)
        return;
    const size_t part = static_cast<size_t>(gridDim.x / deal.cluster) * H;
    float *const out = a.partial + static_cast<size_t>(blockIdx.x / deal.cluster) * H;
    float *const sums = reinterpret_cast<float *>(ring_smem);
    for (int g = 0; g < deal.groups; ++g) {
        __syncthreads();
        if (me.group != g)
            continue;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const int i = me.col(c) + j;
                float v0 = s_pre[c].v[j], v1 = S[c].v[j];
                if (g > 0) {
                    v0 = sums[2 * i] + v0;
                    v1 = sums[2 * i + 1] + v1;
                }
                if (g + 1 < deal.groups) {
                    sums[2 * i] = v0;
                    sums[2 * i + 1] = v1;
                } else {
                    store_f32(out + i, v0);
                    store_f32(out + part + i, v1);
                }
            }
        }
    }
}

// Column sums of the workspace: a CTA adds 32 columns of one of the two sums.
// 32 threads per column take every 32nd CTA's part, all in flight at once (kPer
// of them, for as many CTAs per SM), and a warp adds up a column's 32.
constexpr int kPer = (kSms + 31) / 32;

template <int DT, int kPerSm>
__global__ void __launch_bounds__(1024)
norm_column_sums_kernel(const __grid_constant__ NormArgs a, int parts, int column_ctas)
{
    wait_prior_grid();
    __shared__ float red[32][33];
    const int which = blockIdx.x / column_ctas;
    const bool channel = a.gate_kind == LPCOLL_GATE_CHANNEL;
    float *const dgate = channel ? static_cast<float *>(a.dgate) : nullptr;
    if (which == 0 ? a.dw_pre == nullptr : a.dw_post == nullptr && dgate == nullptr)
        return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first = (blockIdx.x % column_ctas) * 32;
    const float *p = a.partial + static_cast<size_t>(which) * parts * a.hidden + first + lane;
    constexpr int kParts = kPer * kPerSm;
    float v[kParts];
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        const int q = i * 32 + warp;
        v[i] = q < parts && first + lane < a.hidden
                   ? load_f32(p + static_cast<size_t>(q) * a.hidden)
                   : 0.0f;
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kParts; ++i)
        sum += v[i];
    red[warp][lane] = sum;
    __syncthreads();
    sum = warp_sum(red[lane][warp]);
    const int col = first + warp;
    if (lane != 0 || col >= a.hidden)
        return;
    if (which == 0 || parts == 0) {  // no tokens: zeros, whatever the weights hold
        if (which == 0)
            store_f32(a.dw_pre + col, sum);
        else if (a.dw_post != nullptr)
            store_f32(a.dw_post + col, 0.0f);
        if (which == 1 && dgate != nullptr)
            store_f32(dgate + col, 0.0f);
        return;
    }
    if (a.dw_post != nullptr)
        store_f32(a.dw_post + col, channel ? sum * load_one<DT>(a.gate, col) : sum);
    if (dgate != nullptr)
        store_f32(dgate + col, a.w_post != nullptr ? sum * load_one<DT>(a.w_post, col) : sum);
}

int round_up(int n, int to) { return (n + to - 1) / to * to; }

struct Plan {
    Deal deal;
    int elems;    // columns of a thread
    bool even;    // every thread has all its columns
    bool wide;    // kWide (forward only)
    int ctas;     // CTAs, or clusters of them, that share the rows
    size_t smem;  // dynamic shared memory of a CTA
};

// Shared memory of the rings of a CTA, for one to kMaxCtas CTAs per SM.
constexpr size_t kSmem[kMaxCtas] = {224 * 1024, 110 * 1024, 72 * 1024};
constexpr size_t kSmemOne = kSmem[0];

// A row is one CTA's, or, where there are few tokens or the row does not fit
// one, a cluster's. 16 columns a thread halve what a row costs besides its
// columns (sums, addresses), 8 columns give twice the warps. 8192 columns in
// BF16: the gradients of 8192 tokens take 134 us with 16 and 177 with 8, the
// forward pass of 16384 tokens 183 and 160 (8192 tokens of 8 ranks at 4096 columns
// 121 and 125). 8 are also faster where latency counts (32 tokens: 5.6 against 6.1 us)
// and for the shortest rows (128 columns: 7.2 against 9.0 us).
Plan make_plan(size_t tokens, int hidden, int dtype, int streams, bool gradient)
{
    const int width = row_width(hidden, dtype);
    const int kn = width / static_cast<int>(dtype_bytes(dtype));
    constexpr int kRow = 8192;  // columns of the largest CTA but kWide's
    Plan p;
    p.wide = !gradient && tokens > kSms && hidden > kRow && width == 16 &&
             static_cast<size_t>(hidden) * width / kn * streams <= kSmemOne;
    int cluster = hidden > kRow && !p.wide ? 2 : 1;
    // few tokens: a row over up to 8 CTAs, while there are SMs left and a CTA
    // keeps two warps
    while (cluster < kMaxCluster && tokens * cluster * 2 <= kSms && hidden >= 512 * cluster * 2)
        cluster *= 2;
    // many ranks: until a row of all streams fits the shared memory
    while (!p.wide && cluster < kMaxCluster &&
           (static_cast<size_t>(hidden) * width / kn / cluster + 2048) * streams > kSmemOne)
        cluster *= 2;
    const bool light =
        !gradient && streams <= 2 && hidden <= kRow && dtype == LPCOLL_BF16;
    p.elems = !p.wide && (hidden <= 256 || tokens <= kSms || light) ? 8 : 16;
    Deal &d = p.deal;
    d.cluster = cluster;
    d.packs = ((hidden + kn - 1) / kn + cluster - 1) / cluster;
    d.threads = round_up((d.packs + p.elems / kn - 1) / (p.elems / kn), 32);
    const int room = p.wide ? kWideThreads : (p.elems == 8 ? kThreadsOne<8> : kThreadsOne<16>);
    d.groups = cluster > 1 || d.threads * 4 > room ? 1 : room / 2 / d.threads;
    // one row of each of a CTA's teams, in all streams
    const size_t row =
        static_cast<size_t>(row_part_bytes(width, d.packs, d.threads, p.elems)) * streams;
    while (d.groups > 1 && row * d.groups > kSmem[1])
        d.groups /= 2;
    p.even = width == 16 && hidden % kn == 0 && d.packs * cluster * kn == hidden &&
             d.packs % (32 * (p.elems / kn)) == 0;
    int per_sm = room / (d.threads * d.groups);
    per_sm = per_sm < 1 ? 1 : (per_sm > kMaxCtas ? kMaxCtas : per_sm);
    while (per_sm > 1 && row * d.groups > kSmem[per_sm - 1])
        --per_sm;
    const size_t steps = (tokens + d.groups - 1) / d.groups;
    const size_t most = static_cast<size_t>(kSms) * per_sm / cluster;
    p.ctas = static_cast<int>(steps < most ? steps : most);
    const size_t stage = row * d.groups;
    // as many rows under way as fit, and no more than a team has
    size_t stages = kSmem[per_sm - 1] / stage;
    const size_t rows = (steps + p.ctas - 1) / p.ctas;
    stages = stages > kMaxStages ? kMaxStages : stages;
    stages = stages > rows ? rows : stages;
    d.stages = stages < 1 ? 1 : static_cast<int>(stages);
    // the groups of a CTA add up their sums over tokens in shared memory
    const size_t sums =
        gradient && d.groups > 1 ? static_cast<size_t>(hidden) * 2 * sizeof(float) : 0;
    p.smem = d.stages * stage > sums ? d.stages * stage : sums;
    return p;
}

template <class Kernel>
cudaError_t launch_plan(Kernel kernel, const NormArgs &a, const Plan &p, int streams,
                        cudaStream_t st)
{
    // 48 KB hold the kernels' static shared memory too
    if (p.smem > 44 * 1024) {
        // always the same value: calls of several threads must not undo each other's
        const cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemOne));
        if (e != cudaSuccess)
            return e;
    }
    return launch_kernel_cluster(kernel, static_cast<size_t>(p.ctas) * p.deal.cluster,
                                 p.deal.threads * p.deal.groups, p.deal.cluster, p.smem, st, a,
                                 p.deal, streams);
}

Plan backward_plan(size_t tokens, int hidden, int dtype, int gate_kind)
{
    const int streams = gate_kind == LPCOLL_GATE_FULL ? 5 : 4;
    return make_plan(tokens, hidden, dtype, streams, true);
}

template <int DT, int W>
cudaError_t backward_dt(const NormArgs &a, const Plan &p, cudaStream_t st)
{
    const bool full = a.gate_kind == LPCOLL_GATE_FULL;
    const int streams = full ? 5 : 4;
    if constexpr (W == 16) {
        if (p.even && p.deal.cluster == 1 && !full && a.w_post != nullptr && a.w_pre != nullptr &&
            a.dx_out != nullptr)
            return launch_plan(p.elems == 8 ? residual_norm_backward_kernel<DT, W, 8, kPlain>
                                            : residual_norm_backward_kernel<DT, W, 16, kPlain>,
                               a, p, streams, st);
    }
    return launch_plan(p.elems == 8 ? residual_norm_backward_kernel<DT, W, 8, kGeneral>
                                    : residual_norm_backward_kernel<DT, W, 16, kGeneral>,
                       a, p, streams, st);
}

template <int DT, int W>
cudaError_t forward_dt(const NormArgs &a, cudaStream_t st)
{
    const bool full = a.gate_kind == LPCOLL_GATE_FULL;
    const int streams = a.nranks + 1 + (full ? 1 : 0);
    const Plan p = make_plan(a.tokens, a.hidden, a.dtype, streams, false);
    if constexpr (W == 16) {
        if (p.wide)
            return launch_plan(residual_norm_kernel<DT, W, 16, kWide>, a, p, streams, st);
        if (p.even && p.deal.cluster == 1 && !full && a.w_post != nullptr && a.w_pre != nullptr &&
            a.nranks == 1 && a.h_sum == nullptr)
            return launch_plan(p.elems == 8 ? residual_norm_kernel<DT, W, 8, kPlain>
                                            : residual_norm_kernel<DT, W, 16, kPlain>,
                               a, p, streams, st);
    }
    return launch_plan(p.elems == 8 ? residual_norm_kernel<DT, W, 8, kGeneral>
                                    : residual_norm_kernel<DT, W, 16, kGeneral>,
                       a, p, streams, st);
}

template <int DT> cudaError_t column_sums(const NormArgs &a, int parts, cudaStream_t st)
{
    static_assert(kMaxCtas == 3, "one kernel per number of CTAs per SM");
    const int ctas = (a.hidden + 31) / 32;
    const auto kernel = parts <= kSms ? norm_column_sums_kernel<DT, 1>
                                      : (parts <= 2 * kSms ? norm_column_sums_kernel<DT, 2>
                                                           : norm_column_sums_kernel<DT, 3>);
    return launch_kernel_block(kernel, static_cast<size_t>(2) * ctas, 1024, 0, st, a, parts, ctas);
}

}  // namespace

int norm_backward_parts(size_t tokens, size_t hidden, int dtype)
{
    if (hidden == 0 || tokens == 0)
        return 0;
    // the same workspace for every kind of gate
    const int h = static_cast<int>(hidden);
    const int some = backward_plan(tokens, h, dtype, LPCOLL_GATE_NONE).ctas;
    const int full = backward_plan(tokens, h, dtype, LPCOLL_GATE_FULL).ctas;
    return some > full ? some : full;
}

cudaError_t launch_residual_norm(const NormArgs &a, cudaStream_t st)
{
    return LPC_BY_ROW(forward_dt, a.dtype, static_cast<size_t>(a.hidden), a, st);
}

cudaError_t launch_residual_norm_backward(const NormArgs &args, cudaStream_t st)
{
    NormArgs a = args;
    const bool sums = a.dw_pre != nullptr || a.dw_post != nullptr ||
                      (a.gate_kind == LPCOLL_GATE_CHANNEL && a.dgate != nullptr);
    if (!sums)
        a.partial = nullptr;
    int parts = 0;
    if (a.tokens > 0) {
        const Plan p = backward_plan(a.tokens, a.hidden, a.dtype, a.gate_kind);
        parts = p.ctas;
        const cudaError_t e =
            LPC_BY_ROW(backward_dt, a.dtype, static_cast<size_t>(a.hidden), a, p, st);
        if (e != cudaSuccess)
            return e;
    }
    if (!sums)
        return cudaSuccess;
    return a.dtype == LPCOLL_F32 ? column_sums<LPCOLL_F32>(a, parts, st)
                                 : column_sums<LPCOLL_BF16>(a, parts, st);
}

}  // namespace lpc
