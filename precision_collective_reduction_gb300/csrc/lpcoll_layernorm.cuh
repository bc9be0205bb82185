// lpcoll_layernorm.cuh -- kernels of layer_norm and of residual_dropout with its
// norm, and of their gradients, compiled in lpcoll_layernorm.cu and
// lpcoll_dropnorm.cu.
//
//   x' = x                                         (layer_norm)
//   x' = x + d(sum_r h_r),  d(h) = kept ? h / (1 - p) : 0   (residual_dropout)
//   n  = (x' - m) r w + b,  m = mean x', r = 1 / sqrt(mean (x' - m)^2 + eps)
//
// and with q = dn w, xh = (x' - m) r:
//   D  = dx' + r (q - mean q - xh mean(q xh)),  dx = D,  dh = d(D)
//   dw = sum_t dn xh,  db = sum_t dn
//
// Every input is read and every output written once, all sums are FP32. The
// squares are summed about a mean, never about 0: a warp takes the mean of its
// own columns first, sums the squares (and the gradient's q x') about that, and the
// warps' sums are moved to the row's mean where they meet, behind the row's only
// barrier:
//   sum (x - m)^2 = sum_w [M2_w + n_w (m_w - m)^2],
//   sum q (x - m) = sum_w [A_w + (m_w - m) Q_w].
#pragma once

#include "lpcoll_philox.cuh"
#include "lpcoll_rows.cuh"

namespace lpc {

namespace {

__device__ __forceinline__ float2 cluster_load2(const float2 *p, unsigned rank)
{
    const float *f = reinterpret_cast<const float *>(p);
    return make_float2(cluster_load(f, rank), cluster_load(f + 1, rank));
}

__device__ __forceinline__ float4 cluster_load4(const float4 *p, unsigned rank)
{
    const float *f = reinterpret_cast<const float *>(p);
    return make_float4(cluster_load(f, rank), cluster_load(f + 1, rank),
                       cluster_load(f + 2, rank), cluster_load(f + 3, rank));
}

// Columns that warp `w` of a team has in its CTA's part of the row that starts at
// access `part`, as a float (0 where the row ends before).
template <int NV, int kN>
__device__ __forceinline__ float warp_columns(const Deal &deal, int hidden, int part, int w)
{
    const int left = min(deal.packs, hidden / kN - part) - w * NV * 32;
    return static_cast<float>(max(0, min(left, NV * 32)) * kN);
}

// What a lane knows of the columns that the sums are over: its own warp's, and
// those of the warp whose sums it reads (of each CTA of the cluster).
template <int NV, int kN, bool kAlone> struct Shares {
    float inv_own;   // 1 / columns of this warp
    float n0, inv0;  // columns of the warp that this lane reads, without a cluster
    __device__ __forceinline__ Shares(const Deal &deal, int hidden, int first_warp)
    {
        const int lane = threadIdx.x & 31, warps = deal.threads >> 5;
        const int own = static_cast<int>(threadIdx.x >> 5) - first_warp;
        const int part =
            kAlone || deal.cluster == 1 ? 0 : static_cast<int>(cluster_rank()) * deal.packs;
        inv_own = inverse(warp_columns<NV, kN>(deal, hidden, part, own));
        n0 = lane < warps ? warp_columns<NV, kN>(deal, hidden, 0, lane) : 0.0f;
        inv0 = inverse(n0);
    }
    static __device__ __forceinline__ float inverse(float n)
    {
        return n > 0.0f ? __fdiv_rn(1.0f, n) : 0.0f;
    }
    // Columns of warp `lane` of CTA c of the cluster.
    static __device__ __forceinline__ float columns(const Deal &deal, int hidden, int c)
    {
        return warp_columns<NV, kN>(deal, hidden, c * deal.packs, threadIdx.x & 31);
    }
};

// Mean and sum of squares about it of a row, from each warp's sum s and squares q
// about its own mean. The same bits in every thread of the team and every run.
template <class S>
__device__ __forceinline__ void team_moments(float s, float q, const S &share, float2 *red,
                                             const Deal &deal, int first_warp, int hidden,
                                             float per_hidden, bool alone, float &mean, float &m2)
{
    const int lane = threadIdx.x & 31, warps = deal.threads >> 5;
    if (warps == 1 && alone) {
        mean = s * share.inv_own;
        m2 = q;
        return;
    }
    if (lane == 0)
        red[threadIdx.x >> 5] = make_float2(s, q);
    __syncwarp();
    team_barrier(deal);
    if (alone) {
        const float2 v = lane < warps ? red[first_warp + lane] : make_float2(0.0f, 0.0f);
        mean = warp_sum(v.x) * per_hidden;
        const float d = fmaf(v.x, share.inv0, -mean);
        m2 = warp_sum(fmaf(share.n0 * d, d, v.y));
        return;
    }
    float2 v[kMaxCluster];
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
        v[c] = c < deal.cluster && lane < warps ? cluster_load2(red + lane, c)
                                                : make_float2(0.0f, 0.0f);
        sum += v[c].x;
    }
    mean = warp_sum(sum) * per_hidden;
    float sq = 0.0f;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
        if (c >= deal.cluster)
            break;
        const float n = share.columns(deal, hidden, c);
        const float d = fmaf(v[c].x, share.inverse(n), -mean);
        if (lane < warps && n > 0.0f)
            sq += fmaf(n * d, d, v[c].y);
    }
    m2 = warp_sum(sq);
}

// The bits of this thread's columns in row t that dropout keeps, access c's kN
// from bit c kN on. Where an access has fewer than a group's four columns, the
// lanes of a group share its words: each makes the group of one access in turn.
// (A CTA's first column is a multiple of 4: plans deal out whole groups.)
template <int kElems, int kN, class M>
__device__ __forceinline__ uint32_t keep_bits(const Philox &rnd, const M &me, size_t t)
{
    constexpr int NV = kElems / kN;
    const unsigned long long row = rnd.row(t);
    uint32_t bits = 0;
    if constexpr (kN >= 4) {
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
#pragma unroll
            for (int q = 0; q < kN / 4; ++q)
                bits |= rnd.keep4(row + (me.col(c) / 4 + q)) << (c * kN + q * 4);
        }
    } else {
        constexpr int Q = 4 / kN;  // lanes of a group
        const int lane = threadIdx.x & 31, place = lane % Q;
#pragma unroll
        for (int c = 0; c < NV; c += Q) {
            const int col = me.col(c) + place * (32 - 1) * kN;  // of the group's first lane, access c + place
            const uint32_t four = rnd.keep4(row + static_cast<unsigned>(col) / 4);
#pragma unroll
            for (int j = 0; j < Q; ++j) {
                const uint32_t other = __shfl_sync(kAll, four, (lane & ~(Q - 1)) + j);
                bits |= (other >> (place * kN) & ((1u << kN) - 1u)) << ((c + j) * kN);
            }
        }
    }
    return bits;
}

// a + b in one rounding each.
template <int N> __device__ __forceinline__ Vec<N> plus(const Vec<N> &a, const Vec<N> &b)
{
    Vec<N> r;
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float2 p = add_pair(make_float2(a.v[j], a.v[j + 1]),
                                      make_float2(b.v[j], b.v[j + 1]));
            r.v[j] = p.x;
            r.v[j + 1] = p.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            r.v[j] = __fadd_rn(a.v[j], b.v[j]);
    }
    return r;
}

// d of access c: 0 where a column is dropped, whatever it holds.
template <int kN>
__device__ __forceinline__ Vec<kN> dropped(const Vec<kN> &x, float scale, uint32_t bits)
{
    Vec<kN> r;
#pragma unroll
    for (int j = 0; j < kN; ++j)
        r.v[j] = (bits >> j & 1u) != 0 ? __fmul_rn(x.v[j], scale) : 0.0f;
    return r;
}

// Streams of a row: x if there is one, then the ranks' h.
template <int DT, int W, int kElems, int kMode, bool kDrop>
__global__ void __launch_bounds__(kMode == kWide ? kWideThreads : kThreadsOne<kElems>, 1)
layer_norm_kernel(const __grid_constant__ LayerNormArgs a, const Deal deal, int streams)
{
    wait_prior_grid();
    extern __shared__ uint4 ring_smem[];
    __shared__ float2 red[2][kMaxWarps];
    constexpr int kN = Pack<DT, W>::kN;
    constexpr int NV = kElems / kN;
    const Member<DT, W, kElems, kMode, false> me(deal, a, streams, reinterpret_cast<char *>(ring_smem));
    const Shares<NV, kN, kMode == kPlain> share(deal, a.hidden, me.first_warp);
    const bool given = kMode == kPlain || a.x != nullptr;
    const bool weighted = kMode == kPlain || a.w != nullptr;
    const bool biased = kMode == kPlain || a.b != nullptr;
    const int h0 = given ? 1 : 0, nranks = !kDrop ? 0 : (kMode == kPlain ? 1 : a.nranks);
    const bool drop = kDrop && a.drop.least != 0;
    const Philox rnd(a.drop, a.hidden);
    const float per_hidden = __fdiv_rn(1.0f, static_cast<float>(a.hidden));
    const auto fetch = [&](size_t t, int stage) {
        if (t < a.tokens) {
            for (int r = 0; r < nranks; ++r)
                me.copy(stage, h0 + r, a.h[r], t);
            if (given)
                me.copy(stage, 0, a.x, t);
        }
        copy_commit();
    };
    for (int s = 0; s < deal.stages; ++s)
        fetch(me.t0 + s * me.step, s);

    typename Pack<DT, W>::Raw w[NV], b[NV];
    if constexpr (kMode != kWide) {
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            w[c] = b[c] = {};
            if (me.has(c)) {
                if (weighted)
                    w[c] = load_pack<DT, W>(a.w, me.col(c));
                if (biased)
                    b[c] = load_pack<DT, W>(a.b, me.col(c));
            }
        }
    }

    int stage = 0, turn = 0;
    for (size_t t = me.t0; t < a.tokens; t += me.step, turn ^= 1) {
        const uint32_t bits = drop ? keep_bits<kElems, kN>(rnd, me, t) : 0u;
        me.ready(deal.stages - 1);
        Vec<kN> v[NV];
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
            if constexpr (kDrop) {
                Vec<kN> h = me.read(t, stage, h0, c);
#pragma unroll 4
                for (int r = 1; r < nranks; ++r)
                    h = plus(h, me.read(t, stage, h0 + r, c));
                if (drop)
                    h = dropped(h, a.drop.scale, bits >> (c * kN));
                v[c] = given ? plus(me.read(t, stage, 0, c), h) : h;
                store_vec_of<DT, W>(a.x_out, me.elem(t, c), v[c]);
            } else {
                v[c] = me.read(t, stage, 0, c);
            }
#pragma unroll
            for (int j = 0; j < kN; ++j)
                sum += v[c].v[j];
        }
        fetch(t + deal.stages * me.step, stage);
        stage = stage + 1 == deal.stages ? 0 : stage + 1;
        sum = warp_sum(sum);
        const Vec<kN> about = splat<kN>(-(sum * share.inv_own));
        Acc<kN> sq = {};
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
            const Vec<kN> d = plus(v[c], about);
            add_products(sq, d, d);
        }
        float mean, m2;
        team_moments(sum, warp_sum(fold(sq)), share, red[turn], deal, me.first_warp, a.hidden,
                     per_hidden, kMode == kPlain || deal.cluster == 1, mean, m2);
        const float r = inv_rms(m2, per_hidden, a.eps);
        const Vec<kN> centre = splat<kN>(-mean);
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
            Vec<kN> n = mul(r, plus(v[c], centre));
            if constexpr (kMode == kWide) {
                if (weighted)
                    n = mul(n, load_vec_of<DT, W>(a.w, me.col(c)));
                if (biased)
                    n = plus(n, load_vec_of<DT, W>(a.b, me.col(c)));
            } else if (weighted && biased) {
                n = fma(n, unpack<DT, W>(w[c]), unpack<DT, W>(b[c]));
            } else if (weighted) {
                n = mul(n, unpack<DT, W>(w[c]));
            } else if (biased) {
                n = plus(n, unpack<DT, W>(b[c]));
            }
            store_vec_of<DT, W>(a.n_out, me.elem(t, c), n);
        }
    }
    if (kMode != kPlain && deal.cluster > 1)
        cluster_barrier();  // no CTA leaves while another reads its sums
}

// ---------------------------------------------------------------------------
// Gradients. A thread keeps the sums over tokens of its columns, of dn xh and
// of dn, in registers; the CTA leaves them in the workspace, [2][CTAs][hidden],
// and a second launch adds those up in order.
// ---------------------------------------------------------------------------

// Row streams of a stage.
enum GradStream { kGradX = 0, kGradDn = 1, kGradDx = 2 };

// The sums of a row in the gradient: s, and about the warp's mean the squares m2
// and a = sum q (x - mean_w), and q.
template <class S>
__device__ __forceinline__ float4 team_grad_sums(float4 mine, const S &share, float4 *red,
                                                 const Deal &deal, int first_warp, int hidden,
                                                 float per_hidden, bool alone)
{
    const int lane = threadIdx.x & 31, warps = deal.threads >> 5;
    if (warps == 1 && alone)
        return make_float4(mine.x * share.inv_own, mine.y, mine.z, mine.w);
    if (lane == 0)
        red[threadIdx.x >> 5] = mine;
    __syncwarp();
    team_barrier(deal);
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (alone) {
        const float4 v = lane < warps ? red[first_warp + lane] : zero;
        const float mean = warp_sum(v.x) * per_hidden;
        const float d = fmaf(v.x, share.inv0, -mean);
        return make_float4(mean, warp_sum(fmaf(share.n0 * d, d, v.y)), warp_sum(fmaf(d, v.w, v.z)),
                           warp_sum(v.w));
    }
    float4 v[kMaxCluster];
    float sum = 0.0f, q = 0.0f, m2 = 0.0f, at = 0.0f;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
        v[c] = c < deal.cluster && lane < warps ? cluster_load4(red + lane, c) : zero;
        sum += v[c].x;
        q += v[c].w;
    }
    const float mean = warp_sum(sum) * per_hidden;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
        if (c >= deal.cluster)
            break;
        const float n = share.columns(deal, hidden, c);
        const float d = fmaf(v[c].x, share.inverse(n), -mean);
        if (lane < warps && n > 0.0f) {
            m2 += fmaf(n * d, d, v[c].y);
            at += fmaf(d, v[c].w, v[c].z);
        }
    }
    return make_float4(mean, warp_sum(m2), warp_sum(at), warp_sum(q));
}

template <int DT, int W, int kElems, int kMode, bool kDrop>
__global__ void __launch_bounds__(kThreadsOne<kElems>, 1)
layer_norm_backward_kernel(const __grid_constant__ LayerNormArgs a, const Deal deal, int streams)
{
    wait_prior_grid();
    extern __shared__ uint4 ring_smem[];
    __shared__ float4 red[2][kMaxWarps];
    constexpr int kN = Pack<DT, W>::kN;
    constexpr int NV = kElems / kN;
    const Member<DT, W, kElems, kMode, kMode == kPlain> me(deal, a, streams, reinterpret_cast<char *>(ring_smem));
    const Shares<NV, kN, kMode == kPlain> share(deal, a.hidden, me.first_warp);
    const bool weighted = kMode == kPlain || a.w != nullptr;
    const bool given = kDrop && (kMode == kPlain || a.dx_out != nullptr);
    const bool want_dx = kMode == kPlain || a.dx != nullptr;
    const bool want_dh = kDrop && (kMode == kPlain || a.dh != nullptr);
    const bool drop = want_dh && a.drop.least != 0;
    const Philox rnd(a.drop, a.hidden);
    const float per_hidden = __fdiv_rn(1.0f, static_cast<float>(a.hidden));
    const auto fetch = [&](size_t t, int stage) {
        if (t < a.tokens) {
            me.copy(stage, kGradX, a.x, t);
            me.copy(stage, kGradDn, a.dn_out, t);
            if (given)
                me.copy(stage, kGradDx, a.dx_out, t);
        }
        copy_commit();
    };
    for (int s = 0; s < deal.stages; ++s)
        fetch(me.t0 + s * me.step, s);

    typename Pack<DT, W>::Raw w[NV];
    Vec<kN> s_w[NV], s_b[NV];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        w[c] = {};
        if (weighted && me.has(c))
            w[c] = load_pack<DT, W>(a.w, me.col(c));
        s_w[c] = s_b[c] = splat<kN>(0.0f);
    }

    int stage = 0, turn = 0;
    for (size_t t = me.t0; t < a.tokens; t += me.step, turn ^= 1) {
        const uint32_t bits = drop ? keep_bits<kElems, kN>(rnd, me, t) : 0u;
        me.ready(deal.stages - 1);
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
            const Vec<kN> x = me.read(t, stage, kGradX, c);
#pragma unroll
            for (int j = 0; j < kN; ++j)
                s.x += x.v[j];
        }
        s.x = warp_sum(s.x);
        const Vec<kN> about = splat<kN>(-(s.x * share.inv_own));
        Acc<kN> sq = {}, sa = {};
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
            const Vec<kN> d = plus(me.read(t, stage, kGradX, c), about);
            Vec<kN> q = me.read(t, stage, kGradDn, c);
            if (weighted)
                q = mul(q, unpack<DT, W>(w[c]));
            add_products(sq, d, d);
            add_products(sa, q, d);
#pragma unroll
            for (int j = 0; j < kN; ++j)
                s.w += q.v[j];
        }
        s = team_grad_sums(make_float4(s.x, warp_sum(fold(sq)), warp_sum(fold(sa)), warp_sum(s.w)),
                           share, red[turn], deal, me.first_warp, a.hidden, per_hidden,
                           kMode == kPlain || deal.cluster == 1);
        const float r = inv_rms(s.y, per_hidden, a.eps);
        const float c1 = s.w * per_hidden, c2 = r * r * (s.z * per_hidden);
        const Vec<kN> centre = splat<kN>(-s.x);
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
            const Vec<kN> d = plus(me.read(t, stage, kGradX, c), centre);
            const Vec<kN> dn = me.read(t, stage, kGradDn, c);
            s_w[c] = fma(mul(r, d), dn, s_w[c]);
            s_b[c] = plus(s_b[c], dn);
            Vec<kN> q = dn;
            if (weighted)
                q = mul(q, unpack<DT, W>(w[c]));
            q = fma(-c2, d, plus(q, splat<kN>(-c1)));
            q = given ? fma(r, q, me.read(t, stage, kGradDx, c)) : mul(r, q);
            if (want_dx)
                store_vec_of<DT, W>(a.dx, me.elem(t, c), q);
            if (want_dh)
                store_vec_of<DT, W>(a.dh, me.elem(t, c),
                                    drop ? dropped(q, a.drop.scale, bits >> (c * kN)) : q);
        }
        fetch(t + deal.stages * me.step, stage);
        stage = stage + 1 == deal.stages ? 0 : stage + 1;
    }
    copy_wait(0);
    if (kMode != kPlain && deal.cluster > 1)
        cluster_barrier();  // no CTA leaves while another reads its sums
    if (a.partial != nullptr)
        leave_sums(me, deal, s_w, s_b, a.partial, reinterpret_cast<float *>(ring_smem));
}

// Accesses that share a group of four columns.
inline int group_packs(int hidden, int dtype)
{
    const int kn = row_width(hidden, dtype) / static_cast<int>(dtype_bytes(dtype));
    return kn < 4 ? 4 / kn : 1;
}

Plan layer_norm_plan(size_t tokens, int hidden, int dtype, int streams, bool gradient)
{
    const int width = row_width(hidden, dtype);
    const int kn = width / static_cast<int>(dtype_bytes(dtype));
    constexpr int kRow = 8192;  // columns of the largest CTA
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
    p.elems = !p.wide && (hidden <= 256 || tokens <= kSms) ? 8 : 16;
    return deal_rows(p, cluster, tokens, hidden, dtype, streams, gradient,
                     group_packs(hidden, dtype));
}

template <int DT, int W, bool kDrop>
cudaError_t layer_norm_dt(const LayerNormArgs &a, cudaStream_t st)
{
    const int streams = a.nranks + (a.x != nullptr ? 1 : 0);
    const Plan p = layer_norm_plan(a.tokens, a.hidden, a.dtype, streams, false);
    if constexpr (W == 16) {
        if (p.wide)
            return launch_plan(layer_norm_kernel<DT, W, 16, kWide, kDrop>, a, p, streams, st);
        if (p.even && p.deal.cluster == 1 && a.w != nullptr && a.b != nullptr && a.x != nullptr &&
            a.nranks <= 1)
            return launch_plan(p.elems == 8 ? layer_norm_kernel<DT, W, 8, kPlain, kDrop>
                                            : layer_norm_kernel<DT, W, 16, kPlain, kDrop>,
                               a, p, streams, st);
    }
    return launch_plan(p.elems == 8 ? layer_norm_kernel<DT, W, 8, kGeneral, kDrop>
                                    : layer_norm_kernel<DT, W, 16, kGeneral, kDrop>,
                       a, p, streams, st);
}

// The gradients' plan: the same for a residual_dropout with dx_out and without,
// since their workspace is.
Plan layer_norm_backward_plan(size_t tokens, int hidden, int dtype, bool dropout)
{
    return layer_norm_plan(tokens, hidden, dtype, dropout ? 3 : 2, true);
}

template <int DT, int W, bool kDrop>
cudaError_t layer_norm_backward_dt(const LayerNormArgs &a, const Plan &p, cudaStream_t st)
{
    const int streams = kDrop ? 3 : 2;
    if constexpr (W == 16) {
        if (p.even && p.deal.cluster == 1 && a.w != nullptr && a.dx != nullptr &&
            (!kDrop || (a.dx_out != nullptr && a.dh != nullptr)))
            return launch_plan(p.elems == 8 ? layer_norm_backward_kernel<DT, W, 8, kPlain, kDrop>
                                            : layer_norm_backward_kernel<DT, W, 16, kPlain, kDrop>,
                               a, p, streams, st);
    }
    return launch_plan(p.elems == 8 ? layer_norm_backward_kernel<DT, W, 8, kGeneral, kDrop>
                                    : layer_norm_backward_kernel<DT, W, 16, kGeneral, kDrop>,
                       a, p, streams, st);
}

template <int DT, int W> cudaError_t forward_plain(const LayerNormArgs &a, cudaStream_t st)
{
    return layer_norm_dt<DT, W, false>(a, st);
}
template <int DT, int W> cudaError_t forward_drop(const LayerNormArgs &a, cudaStream_t st)
{
    return layer_norm_dt<DT, W, true>(a, st);
}
template <int DT, int W>
cudaError_t backward_plain(const LayerNormArgs &a, const Plan &p, cudaStream_t st)
{
    return layer_norm_backward_dt<DT, W, false>(a, p, st);
}
template <int DT, int W>
cudaError_t backward_drop(const LayerNormArgs &a, const Plan &p, cudaStream_t st)
{
    return layer_norm_backward_dt<DT, W, true>(a, p, st);
}

}  // namespace

}  // namespace lpc
