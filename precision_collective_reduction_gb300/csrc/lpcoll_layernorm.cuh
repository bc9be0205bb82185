// lpcoll_layernorm.cuh -- kernels of layer_norm and of residual_dropout with its
// norm, and of their gradients, compiled in lpcoll_layernorm.cu,
// lpcoll_dropnorm.cu and lpcoll_dropnorm_backward.cu.
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
//
// What bounds them: HBM traffic, and behind it the phases of a row, since a row of 8192
// columns takes the threads of a whole SM (512 of 16 columns, at up to 128 registers) from
// one barrier to the next. Two rows at a time in the forward pass, and the next row's
// sums beside the last row's outputs in the gradient, fill one another's waits. Measured
// on one GB300, 8192 rows of 8192 columns of BF16 (bytes at the copy rate in brackets):
// layer_norm 45 us (40), one row at a time 51, also as two CTAs an SM at 64 registers. Its
// gradient 77 us (59), of which 6 are the launch that adds up the sums over tokens; while
// that took 14, this form took 84, one row after the other 94, with all of a row's values
// in registers 91, with 8 or 32 columns a thread 109 or 148. residual_dropout 100 us (79)
// and 92 with p = 0, its gradient 133 (99) and 122: the generator's products do not all fit
// under the copies. FP32, 8192 rows of 4096: 48 us (40), 71 (59), 93 (79), 113 (99).
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

// What dropout keeps of this thread's columns of a row. An access of four columns
// or more makes its groups' words where they are used. Where an access has fewer,
// the lanes of a group share its words: each makes the group of one access in turn,
// and a row's columns are one bit each. (A CTA's first column is a multiple of 4:
// plans deal out whole groups.)
template <int kElems, int kN> struct Keep {
    unsigned long long row;
    uint32_t bits;

    template <class M>
    __device__ __forceinline__ void make(const Philox &rnd, const M &me, size_t t)
    {
        row = rnd.row(t);
        if constexpr (kN < 4) {
            constexpr int Q = 4 / kN;  // lanes of a group
            constexpr int kGroups = kElems / 4;
            const int lane = threadIdx.x & 31, place = lane % Q;
            bits = 0;
            // access g Q + place of the group's first lane, two groups at a time
            static_assert(kGroups % 2 == 0, "pairs of groups");
#pragma unroll
            for (int g0 = 0; g0 < kGroups; g0 += 2) {
                unsigned long long group[2];
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    group[g] = row + static_cast<unsigned>(me.col((g0 + g) * Q) +
                                                           place * (32 - 1) * kN) / 4;
                uint32_t w[8];
                rnd.words(group, w);
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    uint32_t four = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        four |= w[4 * g + j] >= rnd.least ? 1u << j : 0u;
#pragma unroll
                    for (int j = 0; j < Q; ++j) {
                        const uint32_t other = __shfl_sync(kAll, four, (lane & ~(Q - 1)) + j);
                        bits |= (other >> (place * kN) & ((1u << kN) - 1u))
                                << (((g0 + g) * Q + j) * kN);
                    }
                }
            }
        }
    }
    // d of access c.
    template <class M>
    __device__ __forceinline__ Vec<kN> apply(const Philox &rnd, const M &me, const Vec<kN> &x,
                                             float scale, int c) const
    {
        Vec<kN> r = mul(scale, x);
        if constexpr (kN >= 4) {
            unsigned long long group[kN / 4];
#pragma unroll
            for (int g = 0; g < kN / 4; ++g)
                group[g] = row + static_cast<unsigned>(me.col(c) / 4 + g);
            uint32_t w[kN];
            rnd.words(group, w);
#pragma unroll
            for (int j = 0; j < kN; ++j)
                r.v[j] = rnd.keep(r.v[j], w[j]);
        } else {
#pragma unroll
            for (int j = 0; j < kN; ++j)
                r.v[j] = (bits >> (c * kN + j) & 1u) != 0 ? r.v[j] : 0.0f;
        }
        return r;
    }
};

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

// warp_sum of N values side by side.
template <int N> __device__ __forceinline__ void warp_sums(float (&x)[N])
{
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
        float y[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            y[i] = __shfl_xor_sync(kAll, x[i], m);
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] += y[i];
    }
}

// Sums over a warp of three values of every lane: lane l returns that of value l % 4
// (0 for 3), with 6 shuffles instead of 15.
struct Three {
    float v[3];
};
__device__ __forceinline__ float split_first(const Three &x, float &s1)
{
    const bool up = (threadIdx.x & 2) != 0;
    const float g0 = up ? x.v[0] : x.v[2], g1 = up ? x.v[1] : 0.0f;
    const float k0 = up ? x.v[2] : x.v[0], k1 = up ? 0.0f : x.v[1];
    s1 = k1 + __shfl_xor_sync(kAll, g1, 2);
    return k0 + __shfl_xor_sync(kAll, g0, 2);
}
__device__ __forceinline__ float split_second(float s0, float s1)
{
    const bool up = (threadIdx.x & 1) != 0;
    const float give = up ? s0 : s1, keep = up ? s1 : s0;
    return keep + __shfl_xor_sync(kAll, give, 1);
}
__device__ __forceinline__ float split_sum(const Three &x)
{
    float s1;
    const float s0 = split_first(x, s1);
    float s = split_second(s0, s1);
#pragma unroll
    for (int m = 4; m <= 16; m <<= 1)
        s += __shfl_xor_sync(kAll, s, m);
    return s;
}
// The sums of a row in the gradient.
struct RowSums {
    float mean, m2, a, q;
};

// Two of them side by side.
__device__ __forceinline__ void split_sums(const Three &x, const Three &y, float &a, float &b)
{
    float a1, b1;
    const float a0 = split_first(x, a1), b0 = split_first(y, b1);
    float s[2] = {split_second(a0, a1), split_second(b0, b1)};
#pragma unroll
    for (int m = 4; m <= 16; m <<= 1) {
        const float u = __shfl_xor_sync(kAll, s[0], m), v = __shfl_xor_sync(kAll, s[1], m);
        s[0] += u;
        s[1] += v;
    }
    a = s[0];
    b = s[1];
}

// The sum of a thread's values as an accumulator of products with 1.
template <int N> __device__ __forceinline__ void add_values(Acc<N> &acc, const Vec<N> &a)
{
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int j = 0; j < N; j += 2)
            acc = plus(acc, Vec<2>{{a.v[j], a.v[j + 1]}});
    } else {
        acc = plus(acc, a);
    }
}

// A weight of ones, or a bias of zeros.
template <int DT, int W> __device__ __forceinline__ typename Pack<DT, W>::Raw all_of(float v)
{
    float x[Pack<DT, W>::kN];
#pragma unroll
    for (int j = 0; j < Pack<DT, W>::kN; ++j)
        x[j] = v;
    return narrow_pack<DT, W>(x);
}

constexpr int kTeamThreads = 512;  // most threads of a CTA

// Forms of the kernels beside rows.cuh's: kEven has all its columns as kPlain has,
// but any number of ranks, and the residual or not.
constexpr int kEven = kWide + 1;  // (kWide is residual_norm's)
// kRagged: rows of any length in teams without a cluster. All warps but a team's last have
// all their columns; the steps that go through the columns exist with and without the
// question, and a warp takes its own.
constexpr int kRagged = kEven + 1;

struct Full {
    static constexpr bool kAll = true;
};
struct Partial {
    static constexpr bool kAll = false;
};

// step(Full) where the warp has all of its columns, else step(Partial).
template <int kMode, class Step>
__device__ __forceinline__ void for_columns(bool full, const Step &step)
{
    if constexpr (kMode == kPlain || kMode == kEven) {
        step(Full{});
    } else if constexpr (kMode == kRagged) {
        if (full)
            step(Full{});
        else
            step(Partial{});
    } else {
        step(Partial{});
    }
}

// A team takes R rows at a time: with two, the steps of one fill the waits of the
// other, and one barrier serves both. Streams of a row: x if there is one, then the
// ranks' h.
template <int DT, int W, int kElems, int kMode, bool kDrop, int R>
__global__ void __launch_bounds__(kTeamThreads, 1)
layer_norm_kernel(const __grid_constant__ LayerNormArgs a, const Deal deal, int streams)
{
    wait_prior_grid();
    extern __shared__ uint4 ring_smem[];
    constexpr int kN = Pack<DT, W>::kN;
    constexpr int NV = kElems / kN;
    constexpr bool kAlone = kMode == kPlain || kMode == kEven || kMode == kRagged;
    constexpr int kHas = kMode == kPlain || kMode == kEven ? kPlain : kGeneral;
    __shared__ float2 red[2][R][kMaxWarps];
    const Member<DT, W, kElems, kHas, kAlone> me(deal, a, streams * R, reinterpret_cast<char *>(ring_smem));
    const Shares<NV, kN, kAlone> share(deal, a.hidden, me.first_warp);
    const bool given = kMode == kPlain || !kDrop || a.x != nullptr;
    const int h0 = given ? 1 : 0, nranks = !kDrop ? 0 : (kMode == kPlain ? 1 : a.nranks);
    const bool drop = kDrop && a.drop.least != 0;
    const Philox rnd(a.drop, a.hidden, true);
    const float per_hidden = __fdiv_rn(1.0f, static_cast<float>(a.hidden));
    const int lane = threadIdx.x & 31, warps = deal.threads >> 5;
    const bool full = __all_sync(kAll, me.has(NV - 1));
    const auto fetch = [&](size_t t, int stage) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const size_t row = t + i * me.step;
            if (row >= a.tokens)
                break;
            for (int r = 0; r < nranks; ++r)
                me.copy(stage, i * streams + h0 + r, a.h[r], row);
            if (given)
                me.copy(stage, i * streams, a.x, row);
        }
        copy_commit();
    };
    for (int s = 0; s < deal.stages; ++s)
        fetch(me.t0 + s * R * me.step, s);

    Vec<kN> w[NV], b[NV];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        w[c] = a.w != nullptr && me.has(c) ? load_vec_of<DT, W>(a.w, me.col(c)) : splat<kN>(1.0f);
        b[c] = a.b != nullptr && me.has(c) ? load_vec_of<DT, W>(a.b, me.col(c)) : splat<kN>(0.0f);
    }

    int stage = 0, turn = 0;
    for (size_t t = me.t0; t < a.tokens; t += R * me.step, turn ^= 1) {
        me.ready(deal.stages - 1);
        Vec<kN> v[R][NV];
        float sum[R], sq[R];
        for_columns<kMode>(full, [&](auto all) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const size_t row = t + i * me.step;
                Keep<kElems, kN> keep;
                if (drop)
                    keep.make(rnd, me, row);
                Acc<kN> total = {};
#pragma unroll
                for (int c = 0; c < NV; ++c) {
                    if (!decltype(all)::kAll && !me.has(c))
                        continue;
                    if constexpr (kDrop) {
                        Vec<kN> h = me.read(row, stage, i * streams + h0, c);
#pragma unroll 4
                        for (int r = 1; r < nranks; ++r)
                            h = plus(h, me.read(row, stage, i * streams + h0 + r, c));
                        if (drop)
                            h = keep.apply(rnd, me, h, a.drop.scale, c);
                        v[i][c] = given ? plus(me.read(row, stage, i * streams, c), h) : h;
                        if (R == 1 || row < a.tokens)
                            store_vec_of<DT, W>(a.x_out, me.elem(row, c), v[i][c]);
                    } else {
                        v[i][c] = me.read(row, stage, i, c);
                    }
                    add_values<kN>(total, v[i][c]);
                }
                sum[i] = fold(total);
            }
        });
        fetch(t + deal.stages * R * me.step, stage);
        stage = stage + 1 == deal.stages ? 0 : stage + 1;
        warp_sums(sum);
        for_columns<kMode>(full, [&](auto all) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const Vec<kN> about = splat<kN>(-(sum[i] * share.inv_own));
                Acc<kN> squares = {};
#pragma unroll
                for (int c = 0; c < NV; ++c) {
                    if (!decltype(all)::kAll && !me.has(c))
                        continue;
                    const Vec<kN> d = plus(v[i][c], about);
                    add_products(squares, d, d);
                }
                sq[i] = fold(squares);
            }
        });
        warp_sums(sq);
        float mean[R], m2[R];
        if constexpr (kAlone) {
            float2 e[R];
#pragma unroll
            for (int i = 0; i < R; ++i)
                e[i] = lane == 0 ? make_float2(sum[i], sq[i]) : make_float2(0.0f, 0.0f);
            if (warps > 1) {
                if (lane == 0)
#pragma unroll
                    for (int i = 0; i < R; ++i)
                        red[turn][i][threadIdx.x >> 5] = e[i];
                __syncwarp();
                team_barrier(deal);
                if (lane < warps)
#pragma unroll
                    for (int i = 0; i < R; ++i)
                        e[i] = red[turn][i][me.first_warp + lane];
            }
#pragma unroll
            for (int i = 0; i < R; ++i)
                mean[i] = e[i].x;
            warp_sums(mean);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                mean[i] *= per_hidden;
                const float d = fmaf(e[i].x, share.inv0, -mean[i]);
                m2[i] = fmaf(share.n0 * d, d, e[i].y);
            }
            warp_sums(m2);
        } else {
            team_moments(sum[0], sq[0], share, red[turn][0], deal, me.first_warp, a.hidden,
                         per_hidden, deal.cluster == 1, mean[0], m2[0]);
        }
        for_columns<kMode>(full, [&](auto all) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const size_t row = t + i * me.step;
                if (R > 1 && row >= a.tokens)
                    break;
                const float r = inv_rms(m2[i], per_hidden, a.eps);
                const Vec<kN> centre = splat<kN>(-mean[i]);
#pragma unroll
                for (int c = 0; c < NV; ++c) {
                    if (!decltype(all)::kAll && !me.has(c))
                        continue;
                    const Vec<kN> n = mul(r, plus(v[i][c], centre));
                    store_vec_of<DT, W>(a.n_out, me.elem(row, c), fma(n, w[c], b[c]));
                }
            }
        });
    }
    copy_wait(0);
    if (!kAlone && deal.cluster > 1)
        cluster_barrier();  // no CTA leaves while another reads its sums
}

// ---------------------------------------------------------------------------
// Gradients. A thread keeps the sums over tokens of its columns, of dn xh and
// of dn, in registers; the CTA leaves them in the workspace, [2][CTAs][hidden],
// and a second launch adds those up in order.
// ---------------------------------------------------------------------------

// Row streams of a stage.
enum GradStream { kGradX = 0, kGradDn = 1, kGradDx = 2 };

// The sums of a row in the gradient: about the warp's mean the squares m2 and
// a = sum q (x - mean_w), then q, and the sum of x. A warp leaves them as four floats,
// lane l < 4 value l; `mine` is that value.
constexpr int kSumOfX = 3;

template <class S>
__device__ __forceinline__ Three moved(const float4 &v, const S &share, float mean)
{
    const float d = fmaf(v.w, share.inv0, -mean);
    return {{fmaf(share.n0 * d, d, v.x), fmaf(d, v.z, v.y), v.z}};
}

__device__ __forceinline__ RowSums spread(float mean, float mine)
{
    return {mean, __shfl_sync(kAll, mine, 0), __shfl_sync(kAll, mine, 1),
            __shfl_sync(kAll, mine, 2)};
}

template <class S>
__device__ __forceinline__ RowSums cluster_grad_sums(float mine, float sum, const S &share,
                                                     float4 *red, const Deal &deal, int hidden,
                                                     float per_hidden)
{
    const int lane = threadIdx.x & 31, warps = deal.threads >> 5;
    if (lane < 4)
        reinterpret_cast<float *>(red + (threadIdx.x >> 5))[lane] = lane == kSumOfX ? sum : mine;
    __syncwarp();
    cluster_barrier();
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float4 v[kMaxCluster];
    float all = 0.0f;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
        v[c] = c < deal.cluster && lane < warps ? cluster_load4(red + lane, c) : zero;
        all += v[c].w;
    }
    const float mean = warp_sum(all) * per_hidden;
    Three s = {};
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
        if (c >= deal.cluster)
            break;
        const float n = share.columns(deal, hidden, c);
        const float d = fmaf(v[c].w, share.inverse(n), -mean);
        if (lane < warps && n > 0.0f) {
            s.v[0] += fmaf(n * d, d, v[c].x);
            s.v[1] += fmaf(d, v[c].z, v[c].y);
            s.v[2] += v[c].z;
        }
    }
    return spread(mean, split_sum(s));
}

// The gradient of rows over a cluster of CTAs.
template <int DT, int W, int kElems, bool kDrop>
__global__ void __launch_bounds__(kTeamThreads, 1)
layer_norm_backward_kernel(const __grid_constant__ LayerNormArgs a, const Deal deal, int streams)
{
    wait_prior_grid();
    extern __shared__ uint4 ring_smem[];
    __shared__ float4 red[2][kMaxWarps];
    constexpr int kN = Pack<DT, W>::kN;
    constexpr int NV = kElems / kN;
    const Member<DT, W, kElems, kGeneral, false> me(deal, a, streams, reinterpret_cast<char *>(ring_smem));
    const Shares<NV, kN, false> share(deal, a.hidden, me.first_warp);
    const bool given = kDrop && a.dx_out != nullptr;
    const bool want_dx = a.dx != nullptr;
    const bool want_dh = kDrop && a.dh != nullptr;
    const bool drop = want_dh && a.drop.least != 0;
    const Philox rnd(a.drop, a.hidden, true);
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
        w[c] = a.w != nullptr && me.has(c) ? load_pack<DT, W>(a.w, me.col(c)) : all_of<DT, W>(1.0f);
        s_w[c] = s_b[c] = splat<kN>(0.0f);
    }

    int stage = 0, turn = 0;
    for (size_t t = me.t0; t < a.tokens; t += me.step, turn ^= 1) {
        me.ready(deal.stages - 1);
        Acc<kN> total = {}, sq = {}, sa = {}, sqs = {};
#pragma unroll
        for (int c = 0; c < NV; ++c)
            if (me.has(c))
                add_values<kN>(total, me.read(t, stage, kGradX, c));
        const float sum = warp_sum(fold(total));
        const Vec<kN> about = splat<kN>(-(sum * share.inv_own));  // the warp's mean
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
            const Vec<kN> d = plus(me.read(t, stage, kGradX, c), about);
            const Vec<kN> q = mul(me.read(t, stage, kGradDn, c), unpack<DT, W>(w[c]));
            add_products(sq, d, d);
            add_products(sa, q, d);
            add_values<kN>(sqs, q);
        }
        const RowSums s = cluster_grad_sums(split_sum({{fold(sq), fold(sa), fold(sqs)}}), sum, share,
                                            red[turn], deal, a.hidden, per_hidden);
        Keep<kElems, kN> keep;
        if (drop)
            keep.make(rnd, me, t);
        const float r = inv_rms(s.m2, per_hidden, a.eps);
        const float c1 = s.q * per_hidden, c2 = r * r * (s.a * per_hidden);
        const Vec<kN> centre = splat<kN>(-s.mean);
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
            const Vec<kN> d = plus(me.read(t, stage, kGradX, c), centre);
            const Vec<kN> dn = me.read(t, stage, kGradDn, c);
            s_w[c] = fma(mul(r, d), dn, s_w[c]);
            s_b[c] = plus(s_b[c], dn);
            Vec<kN> q = fma(-c2, d, fma(dn, unpack<DT, W>(w[c]), splat<kN>(-c1)));
            q = given ? fma(r, q, me.read(t, stage, kGradDx, c)) : mul(r, q);
            if (want_dx)
                store_vec_of<DT, W>(a.dx, me.elem(t, c), q);
            if (want_dh)
                store_vec_of<DT, W>(a.dh, me.elem(t, c),
                                    drop ? keep.apply(rnd, me, q, a.drop.scale, c) : q);
        }
        fetch(t + deal.stages * me.step, stage);
        stage = stage + 1 == deal.stages ? 0 : stage + 1;
    }
    copy_wait(0);
    cluster_barrier();  // no CTA leaves while another reads its sums
    if (a.partial != nullptr)
        leave_sums<DT, W>(me, deal, s_w, s_b, a.partial, reinterpret_cast<float *>(ring_smem));
}

// The gradient without clusters (kPlain: every thread has all its columns, and nothing is
// left out; kRagged). A turn of a team joins the sums of its row t, makes
// those of its next row, which depend on nothing of row t, and writes row t: so the
// steps of the one fill the waits of the other. With no next row the stage's old
// values are summed and not used. (One warp more that joins the sums for all, with
// the sums of a row handed over in shared memory, left 96 registers a thread and was
// slower: 8192 x 8192 BF16 95 us, 216 with dropout.)
template <int DT, int W, int kElems, int kMode, bool kDrop>
__global__ void __launch_bounds__(kTeamThreads, 1)
layer_norm_backward_team_kernel(const __grid_constant__ LayerNormArgs a, const Deal deal, int streams)
{
    wait_prior_grid();
    extern __shared__ uint4 ring_smem[];
    __shared__ float4 red[2][kMaxWarps];
    constexpr int kN = Pack<DT, W>::kN;
    constexpr int NV = kElems / kN;
    constexpr int kHas = kMode == kRagged ? kGeneral : kPlain;
    const Member<DT, W, kElems, kHas, true> me(deal, a, streams, reinterpret_cast<char *>(ring_smem));
    const Shares<NV, kN, true> share(deal, a.hidden, me.first_warp);
    const bool given = kDrop && (kMode == kPlain || a.dx_out != nullptr);
    const bool want_dx = kMode == kPlain || a.dx != nullptr;
    const bool want_dh = kDrop && (kMode == kPlain || a.dh != nullptr);
    const bool drop = want_dh && a.drop.least != 0;
    const Philox rnd(a.drop, a.hidden, true);
    const float per_hidden = __fdiv_rn(1.0f, static_cast<float>(a.hidden));
    const int lane = threadIdx.x & 31, warps = deal.threads >> 5;
    const bool full = __all_sync(kAll, me.has(NV - 1));
    // columns of this thread
    int own = 0;
#pragma unroll
    for (int c = 0; c < NV; ++c)
        own += me.has(c) ? kN : 0;
    const float n = kMode == kPlain ? static_cast<float>(kElems) : static_cast<float>(own);
    const float inv_n = kMode == kPlain ? 1.0f / kElems : share.inverse(n);
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
        w[c] = a.w != nullptr && me.has(c) ? load_pack<DT, W>(a.w, me.col(c)) : all_of<DT, W>(1.0f);
        s_w[c] = s_b[c] = splat<kN>(0.0f);
    }

    // This thread's parts of the sums of the row in `stage`, in one pass about its
    // first column x0: with d = x - x0, m = mean d of its n columns,
    //   sum (x - x0 - m)^2 = sum d^2 - m sum d,  sum q (x - x0 - m) = sum q d - m sum q.
    // n (x0 - mean)^2 is at most n times those squares, so of their digits no more
    // are lost than the sum of a row's terms may lose anyway.
    struct Part {
        float sum, mean, m2, a, q;
    };
    const auto add_up = [&](size_t t, int stage) {
        Acc<kN> total = {}, sq = {}, sa = {}, sqs = {};
        float x0 = 0.0f;
        for_columns<kMode>(full, [&](auto all) {
#pragma unroll
            for (int c = 0; c < NV; ++c) {
                if (!decltype(all)::kAll && !me.has(c))
                    continue;
                const Vec<kN> x = me.read(t, stage, kGradX, c);
                if (c == 0)
                    x0 = x.v[0];
                const Vec<kN> d = plus(x, splat<kN>(-x0));
                const Vec<kN> q = mul(me.read(t, stage, kGradDn, c), unpack<DT, W>(w[c]));
                add_values<kN>(total, d);
                add_products(sq, d, d);
                add_products(sa, q, d);
                add_values<kN>(sqs, q);
            }
        });
        const float sum = fold(total), m = sum * inv_n, qs = fold(sqs);
        return Part{fmaf(n, x0, sum), x0 + m, fmaf(-m, sum, fold(sq)), fmaf(-m, qs, fold(sa)), qs};
    };
    // The same about the warp's mean.
    const auto about_warp = [&](const Part &p, float warp_mean) {
        const float d = p.mean - warp_mean;
        return Three{{fmaf(n * d, d, p.m2), fmaf(d, p.q, p.a), p.q}};
    };

    int stage = 0, turn = 0;
    me.ready(deal.stages - 1);
    Part part = add_up(me.t0, 0);
    float sum = warp_sum(part.sum);
    float mine = split_sum(about_warp(part, sum * share.inv_own));
    for (size_t t = me.t0; t < a.tokens; t += me.step, turn ^= 1) {
        const int after = stage + 1 == deal.stages ? 0 : stage + 1;
        const size_t t2 = t + me.step;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (warps > 1) {
            if (lane < 4)
                reinterpret_cast<float *>(&red[turn][threadIdx.x >> 5])[lane] =
                    lane == kSumOfX ? sum : mine;
            __syncwarp();
            team_barrier(deal);
            if (lane < warps)
                v = red[turn][me.first_warp + lane];
        } else {
            const RowSums own = spread(sum, mine);
            if (lane == 0)
                v = make_float4(own.m2, own.a, own.q, sum);
        }
        me.ready(deal.stages - 2);
        part = add_up(t2, after);
        float pair[2] = {v.w, part.sum};
        warp_sums(pair);
        const float mean = pair[0] * per_hidden;
        sum = pair[1];
        float joined;
        split_sums(moved(v, share, mean), about_warp(part, sum * share.inv_own), joined, mine);
        const RowSums s = spread(mean, joined);
        Keep<kElems, kN> keep;
        if (drop)
            keep.make(rnd, me, t);
        // x - mean first: a mean that is large beside the spread costs no digits but its own
        const float r = inv_rms(s.m2, per_hidden, a.eps);
        const float c1 = s.q * per_hidden, c2 = r * r * (s.a * per_hidden);
        const Vec<kN> centre = splat<kN>(-s.mean);
        for_columns<kMode>(full, [&](auto all) {
#pragma unroll
            for (int c = 0; c < NV; ++c) {
                if (!decltype(all)::kAll && !me.has(c))
                    continue;
                const Vec<kN> d = plus(me.read(t, stage, kGradX, c), centre);
                const Vec<kN> dn = me.read(t, stage, kGradDn, c);
                s_w[c] = fma(mul(r, d), dn, s_w[c]);
                s_b[c] = plus(s_b[c], dn);
                Vec<kN> q = fma(-c2, d, fma(dn, unpack<DT, W>(w[c]), splat<kN>(-c1)));
                q = given ? fma(r, q, me.read(t, stage, kGradDx, c)) : mul(r, q);
                if (want_dx)
                    store_vec_of<DT, W>(a.dx, me.elem(t, c), q);
                if (want_dh)
                    store_vec_of<DT, W>(a.dh, me.elem(t, c),
                                        drop ? keep.apply(rnd, me, q, a.drop.scale, c) : q);
            }
        });
        fetch(t + deal.stages * me.step, stage);
        stage = after;
    }
    copy_wait(0);
    if (a.partial != nullptr)
        leave_sums<DT, W>(me, deal, s_w, s_b, a.partial, reinterpret_cast<float *>(ring_smem));
}

// Accesses that share a group of four columns.
inline int group_packs(int hidden, int dtype)
{
    const int kn = row_width(hidden, dtype) / static_cast<int>(dtype_bytes(dtype));
    return kn < 4 ? 4 / kn : 1;
}

// Rows that a team of 8 columns a thread takes at a time: 32768 x 768 BF16 34 us with one,
// 25 with two, 22 with four; in FP32 and with dropout, whose registers four rows fill,
// two are as fast or faster (FP32 33 us, 35 with four).
template <int DT, bool kDrop> constexpr int kShortRows = DT == LPCOLL_BF16 && !kDrop ? 4 : 2;

// Rows that fill their teams may be taken several at a time, `short_rows` where a thread
// has 8 columns; with `ragged` others two at a time (layer_norm of 4096 x 4097 BF16 40 ->
// 32 us; with dropout, whose ranks and words leave no registers for a second row, one at
// a time is faster: 4 ranks of 4096 x 4100 72 us, 84 with two).
Plan layer_norm_plan(size_t tokens, int hidden, int dtype, int streams, bool gradient,
                     int short_rows = 1, bool ragged = false)
{
    const int width = row_width(hidden, dtype);
    const int kn = width / static_cast<int>(dtype_bytes(dtype));
    constexpr int kRow = 16 * kTeamThreads;
    Plan p;
    p.wide = false;
    // rows above 8192 columns in one CTA all the same, at 24 or 32 columns a thread, if
    // their copies fit (2048 x 12288 BF16, norm, with dropout, and their gradients: 20, 50,
    // 40 and 72 us; in a CTA of 1024 threads that reads its weights for every row 26 and 62,
    // over a cluster of two 82 and 110)
    const int least = gradient ? 2 : 1;
    const bool longer = hidden > kRow && tokens > kSms && width == 16 &&
                        least * streams * static_cast<size_t>(hidden) * dtype_bytes(dtype) <= kSmemOne;
    int cluster = hidden > kRow && !longer ? 2 : 1;
    // few tokens: a row over up to 8 CTAs, while there are SMs left and a CTA
    // keeps two warps
    while (cluster < kMaxCluster && tokens * cluster * 2 <= kSms && hidden >= 512 * cluster * 2)
        cluster *= 2;
    // many ranks: until a row of all streams fits the shared memory
    while (!longer && cluster < kMaxCluster &&
           (static_cast<size_t>(hidden) * width / kn / cluster + 2048) * streams > kSmemOne)
        cluster *= 2;
    p.elems = hidden <= 256 || (tokens <= kSms && hidden <= kRow / 2 * cluster) ? 8 : 16;
    if (longer)
        p.elems = hidden <= 24 * kTeamThreads ? 24 : 32;
    // 8 columns a thread also where they fill the threads and 16 do not
    if (cluster == 1 && width == 16 && hidden <= kRow / 2 && hidden % 512 != 0 && hidden % 256 == 0)
        p.elems = 8;
    Room room{kTeamThreads, group_packs(hidden, dtype)};
    room.least = least;
    if (!gradient && cluster == 1 && tokens > kSms && !longer) {
        Room some = room;
        some.rows = p.elems == 8 ? short_rows : 2;
        Plan several = deal_rows(p, cluster, tokens, hidden, dtype, streams, false, some);
        if (!several.even && some.rows != 2) {
            some.rows = 2;
            several = deal_rows(p, cluster, tokens, hidden, dtype, streams, false, some);
        }
        if ((several.even || ragged) && several.smem <= kSmemOne)
            return several;
    }
    return deal_rows(p, cluster, tokens, hidden, dtype, streams, gradient, room);
}

template <int DT, int W, bool kDrop>
cudaError_t layer_norm_dt(const LayerNormArgs &a, cudaStream_t st)
{
    const int streams = a.nranks + (a.x != nullptr ? 1 : 0);
    constexpr int kShort = kShortRows<DT, kDrop>;
    const Plan p = layer_norm_plan(a.tokens, a.hidden, a.dtype, streams, false, kShort, !kDrop);
    if constexpr (W == 16) {
        if (p.elems > 16)
            return launch_plan(p.elems == 24 ? layer_norm_kernel<DT, W, 24, kRagged, kDrop, 1>
                                             : layer_norm_kernel<DT, W, 32, kRagged, kDrop, 1>,
                               a, p, streams, st);
        if (p.even && p.deal.cluster == 1) {
            const bool plain = a.x != nullptr && a.nranks <= 1;
            if (plain && p.elems == 8)
                return launch_plan(p.rows > 1 ? layer_norm_kernel<DT, W, 8, kPlain, kDrop, kShort>
                                               : layer_norm_kernel<DT, W, 8, kPlain, kDrop, 1>,
                                   a, p, streams, st);
            if (plain && p.rows == 2)
                return launch_plan(layer_norm_kernel<DT, W, 16, kPlain, kDrop, 2>, a, p, streams, st);
            if constexpr (kDrop) {
                if (p.elems == 8)
                    return launch_plan(p.rows > 1 ? layer_norm_kernel<DT, W, 8, kEven, true, kShort>
                                                   : layer_norm_kernel<DT, W, 8, kEven, true, 1>,
                                       a, p, streams, st);
                return launch_plan(p.rows == 2 ? layer_norm_kernel<DT, W, 16, kEven, true, 2>
                                               : layer_norm_kernel<DT, W, 16, kEven, true, 1>,
                                   a, p, streams, st);
            }
        }
    }
    if constexpr (!kDrop) {
        if (p.rows == 2)
            return launch_plan(p.elems == 8 ? layer_norm_kernel<DT, W, 8, kRagged, false, 2>
                                            : layer_norm_kernel<DT, W, 16, kRagged, false, 2>,
                               a, p, streams, st);
    }
    // Accesses of 2 or 4 columns: 8192 x 2050 BF16 63 -> 52 us, 8192 x 4100 FP32 110 -> 101.
    // Of 8 columns equal. Of one column, whose words are handed round, slower where there
    // is little else to do (4096 x 4097 BF16 114 us, 121), with 4 ranks 183 -> 165.
    constexpr int kN = Pack<DT, W>::kN;
    if constexpr (kDrop && kN < 8) {
        if (p.elems == 16 && p.deal.cluster == 1 && (kN > 1 || a.nranks > 1))
            return launch_plan(layer_norm_kernel<DT, W, 16, kRagged, true, 1>, a, p, streams, st);
    }
    return launch_plan(p.elems == 8 ? layer_norm_kernel<DT, W, 8, kGeneral, kDrop, 1>
                                    : layer_norm_kernel<DT, W, 16, kGeneral, kDrop, 1>,
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
    if (p.deal.cluster > 1)
        return launch_plan(p.elems == 8 ? layer_norm_backward_kernel<DT, W, 8, kDrop>
                                        : layer_norm_backward_kernel<DT, W, 16, kDrop>,
                           a, p, streams, st);
    if constexpr (W == 16) {
        if (p.elems > 16)
            return launch_plan(p.elems == 24 ? layer_norm_backward_team_kernel<DT, W, 24, kRagged, kDrop>
                                             : layer_norm_backward_team_kernel<DT, W, 32, kRagged, kDrop>,
                               a, p, streams, st);
        if (p.even && a.dx != nullptr && (!kDrop || (a.dx_out != nullptr && a.dh != nullptr)))
            return launch_plan(p.elems == 8 ? layer_norm_backward_team_kernel<DT, W, 8, kPlain, kDrop>
                                            : layer_norm_backward_team_kernel<DT, W, 16, kPlain, kDrop>,
                               a, p, streams, st);
    }
    return launch_plan(p.elems == 8 ? layer_norm_backward_team_kernel<DT, W, 8, kRagged, kDrop>
                                    : layer_norm_backward_team_kernel<DT, W, 16, kRagged, kDrop>,
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
