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
// shared memory. A thread of a team always holds the same columns.
#include "lpcoll_layers.cuh"

namespace lpc {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kSms = 152;
constexpr int kNormThreads = 512;  // largest CTA
constexpr int kNormWarps = kNormThreads / 32;

// How rows are dealt out: `threads` lanes of each of `cluster` CTAs share a
// row, `packs` accesses of it per CTA; a CTA has `groups` such teams.
struct Deal {
    int threads, groups, cluster, packs;
};

__device__ __forceinline__ unsigned cluster_rank()
{
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
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

// Sums over a team of N <= 8 values per thread, the same bits in every thread
// of the team and in every run. The lanes first split the values between them
// (each step halves both the values a lane holds and the lanes that share
// one), 9 shuffles instead of 5 N; the warps' sums then meet in `red`. The
// caller alternates between two `red`, so that one barrier is enough.
template <int N>
__device__ __forceinline__ void team_sums(float (&v)[N], float (*red)[8], const Deal &deal)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = deal.threads >> 5;
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        s[i] = i < N ? v[i < N ? i : 0] : 0.0f;
    // after this lane l holds the sum of value (l & 7) over 4 of the 32 lanes
#pragma unroll
    for (int half = 4; half >= 1; half >>= 1) {
        const bool up = (lane & half) != 0;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float give = up ? s[i] : s[i + half];
            const float keep = up ? s[i + half] : s[i];
            s[i] = keep + __shfl_xor_sync(kAll, give, half);
        }
    }
    float sum = s[0];
    sum += __shfl_xor_sync(kAll, sum, 8);
    sum += __shfl_xor_sync(kAll, sum, 16);
    const int entries = warps * deal.cluster;
    if (entries > 1) {
        if (lane < 8)
            red[warp][lane] = sum;
        if (deal.cluster > 1)
            cluster_barrier();
        else
            __syncthreads();
        const int first = warp / warps * warps;  // of this team in its CTA
        sum = 0.0f;
        for (int e = lane >> 3; e < entries; e += 4) {
            const float *p = &red[first + e % warps][lane & 7];
            sum += deal.cluster > 1 ? cluster_load(p, e / warps) : *p;
        }
        sum += __shfl_xor_sync(kAll, sum, 8);
        sum += __shfl_xor_sync(kAll, sum, 16);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = __shfl_sync(kAll, sum, i);
}

// 1 / sqrt(mean of squares + eps)
__device__ __forceinline__ float inv_rms(float sum, int hidden, float eps)
{
    return __frsqrt_rn(__fdiv_rn(sum, static_cast<float>(hidden)) + eps);
}

template <int DT>
__device__ __forceinline__ float load_one(const void *base, size_t e)
{
    float one[1];
    if constexpr (DT == LPCOLL_F32)
        widen_pack<DT, 4>(load_pack<DT, 4>(base, e), one);
    else
        widen_pack<DT, 2>(load_pack<DT, 2>(base, e), one);
    return one[0];
}

// One row per team.
template <int DT, int W, int NV>
__global__ void __launch_bounds__(kNormThreads)
residual_norm_kernel(const __grid_constant__ NormArgs a, const Deal deal)
{
    wait_prior_grid();
    __shared__ float red[2][kNormWarps][8];
    constexpr int kN = Pack<DT, W>::kN;
    using Raw = typename Pack<DT, W>::Raw;
    const int group = threadIdx.x / deal.threads;
    const int member = threadIdx.x - group * deal.threads;
    const unsigned rank = deal.cluster > 1 ? cluster_rank() : 0;
    const size_t t =
        static_cast<size_t>(blockIdx.x / deal.cluster) * deal.groups + group;
    const size_t row = t * a.hidden;
    const bool live = t < a.tokens;
    int col[NV];  // first column of each access, or -1
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int p = c * deal.threads + member;
        const int i = (static_cast<int>(rank) * deal.packs + p) * kN;
        col[c] = live && p < deal.packs && i < a.hidden ? i : -1;
    }
    float v[NV][kN];
    Raw x[NV];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
#pragma unroll
        for (int j = 0; j < kN; ++j)
            v[c][j] = 0.0f;
        x[c] = Raw{};
        if (col[c] >= 0) {
            x[c] = load_pack<DT, W>(a.x, row + col[c]);
            widen_pack<DT, W>(load_pack<DT, W>(a.h[0], row + col[c]), v[c]);
        }
    }
#pragma unroll 4
    for (int r = 1; r < a.nranks; ++r) {
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (col[c] >= 0) {
                float p[kN];
                widen_pack<DT, W>(load_pack<DT, W>(a.h[r], row + col[c]), p);
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    v[c][j] += p[j];
            }
        }
    }
    float r1[1] = {1.0f};
    if (a.w_post != nullptr) {
        r1[0] = 0.0f;
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int j = 0; j < kN; ++j)
                r1[0] = fmaf(v[c][j], v[c][j], r1[0]);
        team_sums(r1, red[0], deal);
        r1[0] = inv_rms(r1[0], a.hidden, a.eps);
    }
    const float gate_t =
        a.gate_kind == LPCOLL_GATE_TOKEN && live ? load_one<DT>(a.gate, t) : 1.0f;
    float r2[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        if (col[c] < 0)
            continue;
        if (a.h_sum != nullptr)
            store_pack<DT, W>(a.h_sum, row + col[c], narrow_pack<DT, W>(v[c]));
        float w[kN], g[kN], xf[kN];
        if (a.w_post != nullptr) {
            widen_pack<DT, W>(load_pack<DT, W>(a.w_post, col[c]), w);
#pragma unroll
            for (int j = 0; j < kN; ++j)
                v[c][j] = __fmul_rn(__fmul_rn(v[c][j], r1[0]), w[j]);
        }
#pragma unroll
        for (int j = 0; j < kN; ++j)
            g[j] = gate_t;
        if (a.gate_kind == LPCOLL_GATE_CHANNEL)
            widen_pack<DT, W>(load_pack<DT, W>(a.gate, col[c]), g);
        else if (a.gate_kind == LPCOLL_GATE_FULL)
            widen_pack<DT, W>(load_pack<DT, W>(a.gate, row + col[c]), g);
        widen_pack<DT, W>(x[c], xf);
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            v[c][j] = fmaf(__fmul_rn(a.branch_scale, g[j]), v[c][j],
                           __fmul_rn(a.res_scale, xf[j]));
            r2[0] = fmaf(v[c][j], v[c][j], r2[0]);
        }
        store_pack<DT, W>(a.x_out, row + col[c], narrow_pack<DT, W>(v[c]));
    }
    if (a.w_pre != nullptr) {
        team_sums(r2, red[1], deal);
        r2[0] = inv_rms(r2[0], a.hidden, a.eps);
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (col[c] < 0)
                continue;
            float w[kN];
            widen_pack<DT, W>(load_pack<DT, W>(a.w_pre, col[c]), w);
#pragma unroll
            for (int j = 0; j < kN; ++j)
                w[j] = __fmul_rn(__fmul_rn(v[c][j], r2[0]), w[j]);
            store_pack<DT, W>(a.n_out, row + col[c], narrow_pack<DT, W>(w));
        }
    }
    if (deal.cluster > 1)
        cluster_barrier();  // no CTA leaves while another reads its sums
}

// ---------------------------------------------------------------------------
// Gradients. With q = dn w_pre and c2 = r2^2 mean(q x'), the gradient of x' is
// D = dx' + r2 (q - x' c2). The gradient through the first norm needs the sum
// of beta g w_post D h, which is linear in D; so with P = g w_post h (g without
// a token's own gate) the six sums h^2, x'^2, q x', P dx', P q, P x' of one
// pass over the row give every factor of the second:
//   sum(P D) = sum(P dx') + r2 (sum(P q) - c2 sum(P x')).
// A team goes through its tokens one after the other, its next rows on their
// way into shared memory (cp.async) meanwhile: each thread copies and reads its
// own columns only, so that no barrier guards a stage. It keeps the sums over
// tokens of its columns in registers, S = sum beta r1 h D (times a gate that
// differs by token) and dw_pre = sum dn x' r2, and the CTA leaves them in the
// workspace, [2][CTAs][hidden]; a second launch adds those up in order:
// dw_post = g S and dgate = w_post S for a gate per channel.
// ---------------------------------------------------------------------------

// Row streams of a stage.
enum Stream { kH = 0, kDx = 1, kX = 2, kDn = 3, kGate = 4 };

template <int W>
__device__ __forceinline__ void copy_async(void *dst, const void *src)
{
    if (!LPC_READ_OK(src, W)) {
#pragma unroll
        for (int i = 0; i < W / 2; ++i)
            static_cast<uint16_t *>(dst)[i] = 0;
        return;
    }
    if constexpr (W >= 4) {
        const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
        if constexpr (W == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(src) : "memory");
    } else {
        *static_cast<uint16_t *>(dst) = *static_cast<const uint16_t *>(src);
    }
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Waits until at most `pending` of this thread's copy groups are under way.
__device__ __forceinline__ void copy_wait(int pending)
{
    if (pending >= 2)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (pending == 1)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <int DT, int W, int NV>
__global__ void __launch_bounds__(kNormThreads, NV * Pack<DT, W>::kN <= 8 ? 2 : 1)
residual_norm_backward_kernel(const __grid_constant__ NormArgs a, const Deal deal, int stages,
                              int streams)
{
    wait_prior_grid();
    extern __shared__ uint4 stage_smem[];
    __shared__ float red[2][kNormWarps][8];
    constexpr int kN = Pack<DT, W>::kN;
    constexpr size_t kEs = sizeof(typename Pack<DT, W>::Raw) / kN;
    using Raw = typename Pack<DT, W>::Raw;
    const int group = threadIdx.x / deal.threads;
    const int member = threadIdx.x - group * deal.threads;
    const unsigned rank = deal.cluster > 1 ? cluster_rank() : 0;
    const bool post = a.w_post != nullptr, pre = a.w_pre != nullptr, given = a.dx_out != nullptr;
    const bool full = a.gate_kind == LPCOLL_GATE_FULL;
    const int H = a.hidden;
    // shared memory: [stage][group][stream][packs], a stream's part padded to 16 bytes
    const int stream_bytes = (deal.packs * W + 15) & ~15;
    const int group_bytes = stream_bytes * streams;
    char *const mine = reinterpret_cast<char *>(stage_smem) + group * group_bytes;
    const int stage_bytes = group_bytes * deal.groups;

    int col[NV];          // first column of each access, or -1
    float wq[NV][kN];     // w_post times a channel's gate
    Raw wp[NV];           // w_pre
    float S[NV][kN], s_pre[NV][kN];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int p = c * deal.threads + member;
        const int i = (static_cast<int>(rank) * deal.packs + p) * kN;
        col[c] = p < deal.packs && i < H ? i : -1;
        wp[c] = Raw{};
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            S[c][j] = s_pre[c][j] = 0.0f;
            wq[c][j] = 1.0f;
        }
        if (col[c] >= 0) {
            if (post)
                widen_pack<DT, W>(load_pack<DT, W>(a.w_post, i), wq[c]);
            if (pre)
                wp[c] = load_pack<DT, W>(a.w_pre, i);
            if (a.gate_kind == LPCOLL_GATE_CHANNEL) {
                float g[kN];
                widen_pack<DT, W>(load_pack<DT, W>(a.gate, i), g);
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    wq[c][j] = __fmul_rn(wq[c][j], g[j]);
            }
        }
    }

    const size_t step = static_cast<size_t>(gridDim.x / deal.cluster) * deal.groups;
    const size_t t0 = static_cast<size_t>(blockIdx.x / deal.cluster) * deal.groups + group;
    const auto fetch = [&](size_t t, int stage) {
        if (t < a.tokens) {
            const size_t row = t * H;
            char *dst = mine + stage * stage_bytes;
#pragma unroll
            for (int c = 0; c < NV; ++c) {
                if (col[c] < 0)
                    continue;
                char *d = dst + (c * deal.threads + member) * W;
                const size_t off = (row + col[c]) * kEs;
                copy_async<W>(d, static_cast<const char *>(a.h[0]) + off);
                if (given)
                    copy_async<W>(d + kDx * stream_bytes, static_cast<const char *>(a.dx_out) + off);
                if (pre) {
                    copy_async<W>(d + kX * stream_bytes, static_cast<const char *>(a.x) + off);
                    copy_async<W>(d + kDn * stream_bytes, static_cast<const char *>(a.dn_out) + off);
                }
                if (full)
                    copy_async<W>(d + kGate * stream_bytes, static_cast<const char *>(a.gate) + off);
            }
        }
        copy_commit();
    };
    for (int s = 0; s < stages; ++s)
        fetch(t0 + s * step, s);

    int stage = 0, turn = 0;
    // the same number of turns for all teams of the CTA and of the cluster
    for (size_t t = t0; t - group < a.tokens; t += step, turn ^= 1) {
        copy_wait(stages - 1);
        const bool live = t < a.tokens;
        const char *src = mine + stage * stage_bytes;
        const auto read = [&](int stream, int c, float (&out)[kN]) {
            widen_pack<DT, W>(*reinterpret_cast<const Raw *>(
                                  src + stream * stream_bytes + (c * deal.threads + member) * W),
                              out);
        };
        float s[6] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!live || col[c] < 0)
                continue;
            float h[kN], p[kN];
            read(kH, c, h);
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                p[j] = __fmul_rn(wq[c][j], h[j]);
                s[0] = fmaf(h[j], h[j], s[0]);
            }
            if (full) {
                float g[kN];
                read(kGate, c, g);
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    p[j] = __fmul_rn(p[j], g[j]);
            }
            if (given) {
                float d[kN];
                read(kDx, c, d);
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    s[3] = fmaf(p[j], d[j], s[3]);
            }
            if (pre) {
                float x[kN], q[kN], w[kN];
                read(kX, c, x);
                read(kDn, c, q);
                widen_pack<DT, W>(wp[c], w);
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    q[j] = __fmul_rn(q[j], w[j]);
                    s[1] = fmaf(x[j], x[j], s[1]);
                    s[2] = fmaf(q[j], x[j], s[2]);
                    s[4] = fmaf(p[j], q[j], s[4]);
                    s[5] = fmaf(p[j], x[j], s[5]);
                }
            }
        }
        team_sums(s, red[turn], deal);
        const float gate_t =
            a.gate_kind == LPCOLL_GATE_TOKEN && live ? load_one<DT>(a.gate, t) : 1.0f;
        const float r1 = post ? inv_rms(s[0], H, a.eps) : 1.0f;
        const float r2 = pre ? inv_rms(s[1], H, a.eps) : 0.0f;
        const float c2 = pre ? __fdiv_rn(r2 * r2 * s[2], static_cast<float>(H)) : 0.0f;
        const float pd = fmaf(r2, fmaf(-c2, s[5], s[4]), s[3]);
        const float bt = a.branch_scale * gate_t;
        // dh = f1 wq g D - f2 h;  S += f1 g h D
        const float f1 = r1 * bt;
        const float f2 = post ? r1 * __fdiv_rn(r1 * r1 * bt * pd, static_cast<float>(H)) : 0.0f;
        if (a.gate_kind == LPCOLL_GATE_TOKEN && a.dgate != nullptr && live && member == 0 &&
            rank == 0)
            store_f32(static_cast<float *>(a.dgate) + t, a.branch_scale * r1 * pd);
        const size_t row = t * H;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!live || col[c] < 0)
                continue;
            float d[kN], o[kN], h[kN];
#pragma unroll
            for (int j = 0; j < kN; ++j)
                d[j] = 0.0f;
            if (given)
                read(kDx, c, d);
            if (pre) {
                float x[kN], q[kN], w[kN];
                read(kX, c, x);
                read(kDn, c, q);
                widen_pack<DT, W>(wp[c], w);
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    s_pre[c][j] = fmaf(__fmul_rn(q[j], r2), x[j], s_pre[c][j]);
                    d[j] = fmaf(r2, fmaf(-c2, x[j], __fmul_rn(q[j], w[j])), d[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < kN; ++j)
                o[j] = __fmul_rn(a.res_scale, d[j]);
            store_pack<DT, W>(a.dx, row + col[c], narrow_pack<DT, W>(o));
            read(kH, c, h);
            if (full) {
                float g[kN];
                read(kGate, c, g);
                if (a.dgate != nullptr) {
#pragma unroll
                    for (int j = 0; j < kN; ++j)
                        o[j] = __fmul_rn(__fmul_rn(__fmul_rn(f1, wq[c][j]), h[j]), d[j]);
                    store_pack<DT, W>(a.dgate, row + col[c], narrow_pack<DT, W>(o));
                }
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    d[j] = __fmul_rn(d[j], g[j]);
            }
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                S[c][j] = fmaf(__fmul_rn(f1, h[j]), d[j], S[c][j]);
                o[j] = fmaf(__fmul_rn(f1, wq[c][j]), d[j], -__fmul_rn(f2, h[j]));
            }
            store_pack<DT, W>(a.dh, row + col[c], narrow_pack<DT, W>(o));
        }
        fetch(t + stages * step, stage);
        stage = stage + 1 == stages ? 0 : stage + 1;
    }
    copy_wait(0);
    if (deal.cluster > 1)
        cluster_barrier();  // no CTA leaves while another reads its sums

    // The CTA's sums over its tokens: the groups add theirs in order in shared
    // memory (the stages are free), then the CTA writes one row per gradient.
    if (a.partial == nullptr)
        return;
    const size_t part = static_cast<size_t>(gridDim.x / deal.cluster) * H;
    float *const out = a.partial + static_cast<size_t>(blockIdx.x / deal.cluster) * H;
    float *const sums = reinterpret_cast<float *>(stage_smem);
    for (int g = 0; g + 1 < deal.groups; ++g) {
        __syncthreads();
        if (group == g) {
#pragma unroll
            for (int c = 0; c < NV; ++c) {
                if (col[c] < 0)
                    continue;
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    float *p = sums + 2 * (col[c] + j);
                    p[0] = g > 0 ? p[0] + s_pre[c][j] : s_pre[c][j];
                    p[1] = g > 0 ? p[1] + S[c][j] : S[c][j];
                }
            }
        }
    }
    __syncthreads();
    if (group != deal.groups - 1)
        return;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        if (col[c] < 0)
            continue;
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            const int i = col[c] + j;
            float v0 = s_pre[c][j], v1 = S[c][j];
            if (deal.groups > 1) {
                v0 = sums[2 * i] + v0;
                v1 = sums[2 * i + 1] + v1;
            }
            store_f32(out + i, v0);
            store_f32(out + part + i, v1);
        }
    }
}

// Column sums of the workspace: a CTA adds 32 columns of one of the two sums,
// 8 threads per column that each take every 8th CTA's part, in order.
template <int DT>
__global__ void __launch_bounds__(kThreads)
norm_column_sums_kernel(const __grid_constant__ NormArgs a, int parts, int column_ctas)
{
    wait_prior_grid();
    __shared__ float red[8][33];
    const int which = blockIdx.x / column_ctas;
    const bool channel = a.gate_kind == LPCOLL_GATE_CHANNEL;
    float *const dgate = channel ? static_cast<float *>(a.dgate) : nullptr;
    if (which == 0 ? a.dw_pre == nullptr : a.dw_post == nullptr && dgate == nullptr)
        return;
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
    const int col = (blockIdx.x % column_ctas) * 32 + lane;
    float sum = 0.0f;
    if (col < a.hidden) {
        const float *p = a.partial + static_cast<size_t>(which) * parts * a.hidden + col;
#pragma unroll 8
        for (int q = group; q < parts; q += 8)
            sum += load_f32(p + static_cast<size_t>(q) * a.hidden);
    }
    red[group][lane] = sum;
    __syncthreads();
    if (group != 0 || col >= a.hidden)
        return;
    sum = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q)
        sum += red[q][lane];
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

// Accesses per thread of the backward kernel: 8 elements where a CTA then
// holds the row, else 16 (and up to 4 CTAs of a cluster for the longest rows).
template <int DT, int W> constexpr int kFew = 8 / Pack<DT, W>::kN;
template <int DT, int W> constexpr int kMany = 16 / Pack<DT, W>::kN;

// Team of `nv` accesses per thread for a row, over `cluster` CTAs.
Deal deal_row(int hidden, int kn, int nv, int cluster, int most_threads)
{
    Deal d;
    d.cluster = cluster;
    d.packs = ((hidden + kn - 1) / kn + cluster - 1) / cluster;
    d.threads = round_up((d.packs + nv - 1) / nv, 32);
    d.groups = cluster > 1 || d.threads * 2 > most_threads ? 1 : most_threads / d.threads;
    return d;
}

struct BackwardPlan {
    Deal deal;
    bool few;
    int parts;  // CTAs, or clusters of them
};

BackwardPlan backward_plan(size_t tokens, int hidden, int dtype)
{
    const int width = row_width(hidden, dtype);
    const int kn = width / static_cast<int>(dtype_bytes(dtype));
    BackwardPlan p;
    p.few = hidden <= 8 * kNormThreads;
    const int per_cta = 16 * kNormThreads;
    const int cluster = hidden > per_cta ? 2 : 1;
    p.deal = deal_row(hidden, kn, (p.few ? 8 : 16) / kn, cluster, kNormThreads);
    const size_t steps = (tokens + p.deal.groups - 1) / p.deal.groups;
    const size_t most = static_cast<size_t>(kSms) * (p.few ? 2 : 1) / cluster;
    p.parts = static_cast<int>(steps < most ? steps : most);
    return p;
}

template <int DT, int W, int NV>
cudaError_t backward_nv(const NormArgs &a, const BackwardPlan &p, cudaStream_t st)
{
    // shared memory of a CTA beside its static part, for one or two CTAs per SM
    constexpr size_t kLimit = 225 * 1024, kHalf = 112 * 1024;
    const int streams = a.gate_kind == LPCOLL_GATE_FULL ? 5 : 4;
    const size_t stage = static_cast<size_t>(round_up(p.deal.packs * W, 16)) * streams * p.deal.groups;
    // the sums that the groups of a CTA add up at the end
    const size_t sums = p.deal.groups > 1 ? static_cast<size_t>(a.hidden) * 2 * sizeof(float) : 0;
    const size_t room = p.few ? kHalf : kLimit;
    int stages = static_cast<int>(room / stage);
    stages = stages > 3 ? 3 : (stages < 1 ? 1 : stages);
    const size_t smem = stages * stage > sums ? stages * stage : sums;
    auto kernel = residual_norm_backward_kernel<DT, W, NV>;
    // always the same value: calls of several threads must not undo each other's
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kLimit));
    if (e != cudaSuccess)
        return e;
    return launch_kernel_cluster(kernel, static_cast<size_t>(p.parts) * p.deal.cluster,
                                 p.deal.threads * p.deal.groups, p.deal.cluster, smem, st, a,
                                 p.deal, stages, streams);
}

template <int DT, int W>
cudaError_t backward_dt(const NormArgs &a, const BackwardPlan &p, cudaStream_t st)
{
    return p.few ? backward_nv<DT, W, kFew<DT, W>>(a, p, st)
                 : backward_nv<DT, W, kMany<DT, W>>(a, p, st);
}

template <int DT, int W>
cudaError_t forward_dt(const NormArgs &a, cudaStream_t st)
{
    constexpr int kN = Pack<DT, W>::kN;
    const bool few = a.hidden <= 8 * kNormThreads;
    const int cluster = a.hidden > 16 * kNormThreads ? 2 : 1;
    const Deal d = deal_row(a.hidden, kN, few ? kFew<DT, W> : kMany<DT, W>, cluster, 256);
    const size_t grid = (a.tokens + d.groups - 1) / d.groups * cluster;
    return launch_kernel_cluster(few ? residual_norm_kernel<DT, W, kFew<DT, W>>
                                     : residual_norm_kernel<DT, W, kMany<DT, W>>,
                                 grid, d.threads * d.groups, cluster, 0, st, a, d);
}

}  // namespace

int norm_backward_parts(size_t tokens, size_t hidden, int dtype)
{
    return hidden == 0 || tokens == 0
               ? 0
               : backward_plan(tokens, static_cast<int>(hidden), dtype).parts;
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
        const BackwardPlan p = backward_plan(a.tokens, a.hidden, a.dtype);
        parts = p.parts;
        const cudaError_t e =
            LPC_BY_ROW(backward_dt, a.dtype, static_cast<size_t>(a.hidden), a, p, st);
        if (e != cudaSuccess)
            return e;
    }
    if (!sums)
        return cudaSuccess;
    const int ctas = (a.hidden + 31) / 32;
    return launch_kernel_block(a.dtype == LPCOLL_F32 ? norm_column_sums_kernel<LPCOLL_F32>
                                                     : norm_column_sums_kernel<LPCOLL_BF16>,
                               static_cast<size_t>(2) * ctas, kThreads, 0, st, a, parts, ctas);
}

}  // namespace lpc
