// lpcoll_rows.cuh -- what the kernels that normalise rows share: teams of warps
// that own a row, their sums, rows on their way through shared memory, and how
// rows are dealt out to CTAs. Internal linkage: each translation unit has its own.
//
// A row belongs to a "team" of whole warps: a part of a CTA for short rows, a
// CTA, or the CTAs of a cluster. A thread of a team always holds the same
// columns, and copies (cp.async) and reads its own columns only, so no barrier
// guards the rows in shared memory.
#pragma once

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

// Forms of the kernels: any call; one in which every thread has all its columns and
// nothing is left out; rows of more than 8192 columns in a CTA of 1024 threads.
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

    template <class Args>
    __device__ __forceinline__ Member(const Deal &deal, const Args &a, int streams, char *smem)
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
// FP32 values of an access at column `col` of a row of FP32 numbers, in the widest
// accesses that rows of the access's own width leave aligned.
template <int DT, int W>
__device__ __forceinline__ void store_floats(float *row, int col, const Vec<Pack<DT, W>::kN> &x)
{
    constexpr int kN = Pack<DT, W>::kN;
    constexpr int kF = kN < 4 ? kN : 4;
#pragma unroll
    for (int j = 0; j < kN; j += kF) {
        Vec<kF> v;
#pragma unroll
        for (int i = 0; i < kF; ++i)
            v.v[i] = x.v[j + i];
        store_vec_of<LPCOLL_F32, 4 * kF>(row, col + j, v);
    }
}

// Leaves two sums over a CTA's tokens of each of its columns in the workspace,
// [2][CTAs][hidden]: the teams add theirs in order in shared memory (the rows are
// done with), then the CTA, or each of a cluster for its columns, writes a row of both.
template <int DT, int W, class M, int kN, int NV>
__device__ __forceinline__ void leave_sums(const M &me, const Deal &deal, Vec<kN> (&s0)[NV],
                                           Vec<kN> (&s1)[NV], float *partial, float *sums)
{
    const int H = me.hidden;
    const size_t part = static_cast<size_t>(gridDim.x / deal.cluster) * H;
    float *const out = partial + static_cast<size_t>(blockIdx.x / deal.cluster) * H;
    for (int g = 0; g < deal.groups; ++g) {
        __syncthreads();
        if (me.group != g)
            continue;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
            if (deal.groups > 1)
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    const int i = me.col(c) + j;
                    if (g > 0) {
                        s0[c].v[j] = sums[2 * i] + s0[c].v[j];
                        s1[c].v[j] = sums[2 * i + 1] + s1[c].v[j];
                    }
                    if (g + 1 < deal.groups) {
                        sums[2 * i] = s0[c].v[j];
                        sums[2 * i + 1] = s1[c].v[j];
                    }
                }
            if (g + 1 == deal.groups) {
                store_floats<DT, W>(out, me.col(c), s0[c]);
                store_floats<DT, W>(out + part, me.col(c), s1[c]);
            }
        }
    }
}

inline int round_up(int n, int to) { return (n + to - 1) / to * to; }

struct Plan {
    Deal deal;
    int elems;    // columns of a thread
    bool even;    // every thread has all its columns
    bool wide;    // kWide (forward only)
    int ctas;     // CTAs, or clusters of them, that share the rows
    int rows;     // that a team takes at a time
    size_t smem;  // dynamic shared memory of a CTA
};

// Shared memory of the rings of a CTA, for one to kMaxCtas CTAs per SM.
constexpr size_t kSmem[kMaxCtas] = {224 * 1024, 110 * 1024, 72 * 1024};
constexpr size_t kSmemOne = kSmem[0];

// What deal_rows works with beside the call's sizes.
struct Room {
    int threads;       // that an SM holds
    int multiple = 1;  // accesses that a CTA's part of a row is a multiple of
    int rows = 1;      // that a team takes at a time
    int least = 1;     // stages that a team needs
};

// The rest of a plan whose columns per thread and form are chosen, for rows over
// `cluster` CTAs. `gradient`: the teams of a CTA add up two sums of every column at
// the end.
inline Plan deal_rows(Plan p, int cluster, size_t tokens, int hidden, int dtype, int streams,
                      bool gradient, const Room &room)
{
    p.rows = room.rows;
    streams *= room.rows;
    const int width = row_width(hidden, dtype);
    const int kn = width / static_cast<int>(dtype_bytes(dtype));
    Deal &d = p.deal;
    d.cluster = cluster;
    d.packs = round_up(((hidden + kn - 1) / kn + cluster - 1) / cluster, room.multiple);
    d.threads = round_up((d.packs + p.elems / kn - 1) / (p.elems / kn), 32);
    d.groups = cluster > 1 || d.threads * 4 > room.threads ? 1 : room.threads / 2 / d.threads;
    // the rows that each of a CTA's teams takes at a time, in all streams
    const size_t row =
        static_cast<size_t>(row_part_bytes(width, d.packs, d.threads, p.elems)) * streams;
    while (d.groups > 1 && row * d.groups * room.least > kSmem[1])
        d.groups /= 2;
    p.even = width == 16 && hidden % kn == 0 && d.packs * cluster * kn == hidden &&
             d.packs % (32 * (p.elems / kn)) == 0;
    int per_sm = room.threads / (d.threads * d.groups);
    per_sm = per_sm < 1 ? 1 : (per_sm > kMaxCtas ? kMaxCtas : per_sm);
    while (per_sm > 1 && row * d.groups * room.least > kSmem[per_sm - 1])
        --per_sm;
    const size_t at_once = static_cast<size_t>(d.groups) * room.rows;
    const size_t steps = (tokens + at_once - 1) / at_once;
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

template <class Kernel, class Args>
cudaError_t launch_plan(Kernel kernel, const Args &a, const Plan &p, int streams,
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

}  // namespace

}  // namespace lpc
