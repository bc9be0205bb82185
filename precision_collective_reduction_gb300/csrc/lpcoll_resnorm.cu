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
// A CTA holds a token's row in registers, kN elements per thread and access,
// so that every input is read and every output written once; all arithmetic
// and sums are FP32, rounded once at each output.
#include "lpcoll_layers.cuh"

namespace lpc {

namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMaxWarps = kMaxThreads / 32;

// Sums of N values over the CTA, the same bits in every thread and run. The
// caller alternates `red` so that no barrier is needed before the next use.
template <int N>
__device__ __forceinline__ void cta_sums(float (&v)[N], float (*red)[kMaxWarps])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = warp_sum(v[i]);
        if (lane == 0)
            red[i][warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = warp_sum(lane < warps ? red[i][lane] : 0.0f);
}

// 1 / sqrt(mean of squares + eps)
__device__ __forceinline__ float inv_rms(float sum, int hidden, float eps)
{
    return __frsqrt_rn(__fdiv_rn(sum, static_cast<float>(hidden)) + eps);
}

template <int DT, bool VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads)
residual_norm_kernel(const __grid_constant__ NormArgs a)
{
    wait_prior_grid();
    __shared__ float red[2][1][kMaxWarps];
    constexpr int kN = Pack<DT, VEC>::kN;
    using Raw = typename Pack<DT, VEC>::Raw;
    const size_t t = blockIdx.x;
    const size_t row = t * a.hidden;
    const int H = a.hidden;
    float v[NV][kN];
    Raw x[NV];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int i = (c * blockDim.x + threadIdx.x) * kN;
#pragma unroll
        for (int j = 0; j < kN; ++j)
            v[c][j] = 0.0f;
        x[c] = Raw{};
        if (i < H) {
            x[c] = load_pack<DT, VEC>(a.x, row + i);
            widen_pack<DT, VEC>(load_pack<DT, VEC>(a.h[0], row + i), v[c]);
        }
    }
    for (int r = 1; r < a.nranks; ++r) {
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int i = (c * blockDim.x + threadIdx.x) * kN;
            if (i < H) {
                float p[kN];
                widen_pack<DT, VEC>(load_pack<DT, VEC>(a.h[r], row + i), p);
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
        cta_sums(r1, red[0]);
        r1[0] = inv_rms(r1[0], H, a.eps);
    }
    const float gate_t = a.gate_kind == LPCOLL_GATE_TOKEN ? [&] {
        float g[1];
        widen_pack<DT, false>(load_pack<DT, false>(a.gate, t), g);
        return g[0];
    }() : 1.0f;
    float r2[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int i = (c * blockDim.x + threadIdx.x) * kN;
        if (i >= H)
            continue;
        if (a.h_sum != nullptr)
            store_pack<DT, VEC>(a.h_sum, row + i, narrow_pack<DT, VEC>(v[c]));
        float w[kN], g[kN], xf[kN];
        if (a.w_post != nullptr) {
            widen_pack<DT, VEC>(load_pack<DT, VEC>(a.w_post, i), w);
#pragma unroll
            for (int j = 0; j < kN; ++j)
                v[c][j] = __fmul_rn(__fmul_rn(v[c][j], r1[0]), w[j]);
        }
#pragma unroll
        for (int j = 0; j < kN; ++j)
            g[j] = gate_t;
        if (a.gate_kind == LPCOLL_GATE_CHANNEL)
            widen_pack<DT, VEC>(load_pack<DT, VEC>(a.gate, i), g);
        else if (a.gate_kind == LPCOLL_GATE_FULL)
            widen_pack<DT, VEC>(load_pack<DT, VEC>(a.gate, row + i), g);
        widen_pack<DT, VEC>(x[c], xf);
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            v[c][j] = fmaf(__fmul_rn(a.branch_scale, g[j]), v[c][j],
                           __fmul_rn(a.res_scale, xf[j]));
            r2[0] = fmaf(v[c][j], v[c][j], r2[0]);
        }
        store_pack<DT, VEC>(a.x_out, row + i, narrow_pack<DT, VEC>(v[c]));
    }
    if (a.w_pre == nullptr)
        return;
    cta_sums(r2, red[1]);
    r2[0] = inv_rms(r2[0], H, a.eps);
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int i = (c * blockDim.x + threadIdx.x) * kN;
        if (i >= H)
            continue;
        float w[kN];
        widen_pack<DT, VEC>(load_pack<DT, VEC>(a.w_pre, i), w);
#pragma unroll
        for (int j = 0; j < kN; ++j)
            w[j] = __fmul_rn(__fmul_rn(v[c][j], r2[0]), w[j]);
        store_pack<DT, VEC>(a.n_out, row + i, narrow_pack<DT, VEC>(w));
    }
}

// Gradients. With gw = dn w_pre and c2 = r2^2 mean(gw x'), the gradient of x'
// is D = dx' + r2 (gw - x' c2). The gradient through the first norm needs
// sum(q h) with q = beta g w_post D, which is linear in D; so with
// P = g w_post h (g without a token's own gate) the six sums h^2, x'^2, gw x',
// P dx', P gw, P x' of one pass over the row give every factor of the second:
//   sum(P D) = sum(P dx') + r2 (sum(P gw) - c2 sum(P x')).
// The CTAs go through the tokens with the grid as stride; a thread keeps the
// sums over tokens of its own columns in registers and leaves them in the
// workspace, [3][CTAs][hidden], for a second launch to add up in order.
template <int DT, bool VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads)
residual_norm_backward_kernel(const __grid_constant__ NormArgs a)
{
    wait_prior_grid();
    __shared__ float red[2][6][kMaxWarps];
    constexpr int kN = Pack<DT, VEC>::kN;
    const int H = a.hidden;
    const bool post = a.w_post != nullptr, pre = a.w_pre != nullptr;
    float s_pre[NV][kN], s_post[NV][kN], s_gate[NV][kN];
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int j = 0; j < kN; ++j)
            s_pre[c][j] = s_post[c][j] = s_gate[c][j] = 0.0f;
    int turn = 0;
    for (size_t t = blockIdx.x; t < a.tokens; t += gridDim.x, turn ^= 1) {
        const size_t row = t * H;
        float h[NV][kN], x[NV][kN], d[NV][kN], gw[NV][kN], g[NV][kN];
        float s[6] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        float gate_t = 1.0f;
        if (a.gate_kind == LPCOLL_GATE_TOKEN) {
            float one[1];
            widen_pack<DT, false>(load_pack<DT, false>(a.gate, t), one);
            gate_t = one[0];
        }
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int i = (c * blockDim.x + threadIdx.x) * kN;
            if (i < H) {
                widen_pack<DT, VEC>(load_pack<DT, VEC>(a.h[0], row + i), h[c]);
                if (a.dx_out != nullptr) {
                    widen_pack<DT, VEC>(load_pack<DT, VEC>(a.dx_out, row + i), d[c]);
                } else {
#pragma unroll
                    for (int j = 0; j < kN; ++j)
                        d[c][j] = 0.0f;
                }
                if (a.gate_kind == LPCOLL_GATE_CHANNEL) {
                    widen_pack<DT, VEC>(load_pack<DT, VEC>(a.gate, i), g[c]);
                } else if (a.gate_kind == LPCOLL_GATE_FULL) {
                    widen_pack<DT, VEC>(load_pack<DT, VEC>(a.gate, row + i), g[c]);
                } else {
#pragma unroll
                    for (int j = 0; j < kN; ++j)
                        g[c][j] = 1.0f;
                }
                float p[kN];
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    p[j] = __fmul_rn(g[c][j], h[c][j]);
                if (post) {
                    float w[kN];
                    widen_pack<DT, VEC>(load_pack<DT, VEC>(a.w_post, i), w);
#pragma unroll
                    for (int j = 0; j < kN; ++j) {
                        p[j] = __fmul_rn(p[j], w[j]);
                        s[0] = fmaf(h[c][j], h[c][j], s[0]);
                    }
                }
                if (pre) {
                    float w[kN];
                    widen_pack<DT, VEC>(load_pack<DT, VEC>(a.x, row + i), x[c]);
                    widen_pack<DT, VEC>(load_pack<DT, VEC>(a.dn_out, row + i), gw[c]);
                    widen_pack<DT, VEC>(load_pack<DT, VEC>(a.w_pre, i), w);
#pragma unroll
                    for (int j = 0; j < kN; ++j) {
                        const float q = __fmul_rn(gw[c][j], w[j]);
                        s[1] = fmaf(x[c][j], x[c][j], s[1]);
                        s[2] = fmaf(q, x[c][j], s[2]);
                        s[4] = fmaf(p[j], q, s[4]);
                        s[5] = fmaf(p[j], x[c][j], s[5]);
                    }
                }
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    s[3] = fmaf(p[j], d[c][j], s[3]);
            }
        }
        cta_sums(s, red[turn]);
        const float r1 = post ? inv_rms(s[0], H, a.eps) : 1.0f;
        const float r2 = pre ? inv_rms(s[1], H, a.eps) : 0.0f;
        const float c2 = pre ? __fdiv_rn(r2 * r2 * s[2], static_cast<float>(H)) : 0.0f;
        const float pd = fmaf(r2, fmaf(-c2, s[5], s[4]), s[3]);
        const float bt = a.branch_scale * gate_t;
        const float c1 = __fdiv_rn(r1 * r1 * bt * pd, static_cast<float>(H));
        if (a.gate_kind == LPCOLL_GATE_TOKEN && a.dgate != nullptr && threadIdx.x == 0)
            store_f32(static_cast<float *>(a.dgate) + t, a.branch_scale * r1 * pd);
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int i = (c * blockDim.x + threadIdx.x) * kN;
            if (i >= H)
                continue;
            float w[kN], o[kN];
            if (pre) {
                widen_pack<DT, VEC>(load_pack<DT, VEC>(a.w_pre, i), w);
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    s_pre[c][j] = fmaf(gw[c][j], __fmul_rn(x[c][j], r2), s_pre[c][j]);
                    const float q = __fmul_rn(gw[c][j], w[j]);
                    d[c][j] = fmaf(r2, fmaf(-c2, x[c][j], q), d[c][j]);
                }
            }
#pragma unroll
            for (int j = 0; j < kN; ++j)
                o[j] = __fmul_rn(a.res_scale, d[c][j]);
            store_pack<DT, VEC>(a.dx, row + i, narrow_pack<DT, VEC>(o));
            if (post) {
                widen_pack<DT, VEC>(load_pack<DT, VEC>(a.w_post, i), w);
            } else {
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    w[j] = 1.0f;
            }
            float dg[kN];
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const float hh = __fmul_rn(h[c][j], r1);
                const float du = __fmul_rn(__fmul_rn(bt, g[c][j]), d[c][j]);
                dg[j] = __fmul_rn(__fmul_rn(__fmul_rn(hh, w[j]), a.branch_scale), d[c][j]);
                s_gate[c][j] += dg[j];
                s_post[c][j] = fmaf(du, hh, s_post[c][j]);
                o[j] = post ? __fmul_rn(r1, fmaf(-c1, h[c][j], __fmul_rn(du, w[j]))) : du;
            }
            store_pack<DT, VEC>(a.dh, row + i, narrow_pack<DT, VEC>(o));
            if (a.gate_kind == LPCOLL_GATE_FULL && a.dgate != nullptr)
                store_pack<DT, VEC>(a.dgate, row + i, narrow_pack<DT, VEC>(dg));
        }
    }
    const size_t part = static_cast<size_t>(gridDim.x) * H;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int i = (c * blockDim.x + threadIdx.x) * kN;
        if (i >= H)
            continue;
        float *p = a.partial + static_cast<size_t>(blockIdx.x) * H + i;
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            if (a.dw_pre != nullptr)
                store_f32(p + j, s_pre[c][j]);
            if (a.dw_post != nullptr)
                store_f32(p + part + j, s_post[c][j]);
            if (a.gate_kind == LPCOLL_GATE_CHANNEL && a.dgate != nullptr)
                store_f32(p + 2 * part + j, s_gate[c][j]);
        }
    }
}

// Column sums of the workspace: CTA (32 columns, one of the three gradients),
// 8 threads per column that each take every 8th partial sum, in order.
__global__ void __launch_bounds__(kThreads)
norm_column_sums_kernel(const float *partial, int parts, int hidden, float *dw_pre, float *dw_post,
                        float *dgate, int column_ctas)
{
    wait_prior_grid();
    __shared__ float red[8][33];
    const int which = blockIdx.x / column_ctas;
    float *out = which == 0 ? dw_pre : (which == 1 ? dw_post : dgate);
    if (out == nullptr)
        return;
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
    const int col = (blockIdx.x % column_ctas) * 32 + lane;
    float sum = 0.0f;
    if (col < hidden) {
        const float *p = partial + static_cast<size_t>(which) * parts * hidden + col;
#pragma unroll 8
        for (int q = group; q < parts; q += 8)
            sum += load_f32(p + static_cast<size_t>(q) * hidden);
    }
    red[group][lane] = sum;
    __syncthreads();
    if (group == 0 && col < hidden) {
        sum = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q)
            sum += red[q][lane];
        store_f32(out + col, sum);
    }
}

int row_threads(int hidden, int per_thread)
{
    const int n = (hidden + per_thread - 1) / per_thread;
    return (n + 31) / 32 * 32;
}

template <int DT, bool VEC, int NV>
cudaError_t norm_nv(const NormArgs &a, bool backward, cudaStream_t st)
{
    const int threads = row_threads(a.hidden, NV * Pack<DT, VEC>::kN);
    if (!backward)
        return launch_kernel_block(residual_norm_kernel<DT, VEC, NV>, a.tokens, threads, 0, st, a);
    const int parts = norm_backward_parts(a.tokens, a.hidden, a.dtype);
    return launch_kernel_block(residual_norm_backward_kernel<DT, VEC, NV>, parts, threads, 0, st,
                               a);
}

// Accesses per thread and row: as few as keep a CTA within 512 threads, or
// within 1024 for the longest rows.
template <int DT, bool VEC>
cudaError_t norm_dt(const NormArgs &a, bool backward, cudaStream_t st)
{
    constexpr int kN = Pack<DT, VEC>::kN;
    if (a.hidden <= 512 * kN)
        return norm_nv<DT, VEC, 1>(a, backward, st);
    if constexpr (kN >= 8) {
        return norm_nv<DT, VEC, 2>(a, backward, st);
    } else if constexpr (kN >= 4) {
        if (a.hidden <= 512 * kN * 2)
            return norm_nv<DT, VEC, 2>(a, backward, st);
        return norm_nv<DT, VEC, 4>(a, backward, st);
    } else {
        if (a.hidden <= 512 * kN * 4)
            return norm_nv<DT, VEC, 4>(a, backward, st);
        return norm_nv<DT, VEC, 16>(a, backward, st);
    }
}

cudaError_t norm_any(const NormArgs &a, bool backward, cudaStream_t st)
{
    const bool vec = rows_aligned(a.hidden, a.dtype);
    if (a.dtype == LPCOLL_F32)
        return vec ? norm_dt<LPCOLL_F32, true>(a, backward, st)
                   : norm_dt<LPCOLL_F32, false>(a, backward, st);
    return vec ? norm_dt<LPCOLL_BF16, true>(a, backward, st)
               : norm_dt<LPCOLL_BF16, false>(a, backward, st);
}

}  // namespace

int norm_backward_parts(size_t tokens, size_t, int)
{
    constexpr size_t kParts = 304;
    return static_cast<int>(tokens < kParts ? tokens : kParts);
}

cudaError_t launch_residual_norm(const NormArgs &a, cudaStream_t st)
{
    return norm_any(a, false, st);
}

cudaError_t launch_residual_norm_backward(const NormArgs &a, cudaStream_t st)
{
    if (a.tokens > 0) {
        const cudaError_t e = norm_any(a, true, st);
        if (e != cudaSuccess)
            return e;
    }
    float *dgate = a.gate_kind == LPCOLL_GATE_CHANNEL ? static_cast<float *>(a.dgate) : nullptr;
    if (a.dw_pre == nullptr && a.dw_post == nullptr && dgate == nullptr)
        return cudaSuccess;
    const int ctas = (a.hidden + 31) / 32;
    return launch_kernel_block(norm_column_sums_kernel, static_cast<size_t>(3) * ctas, kThreads, 0,
                               st, static_cast<const float *>(a.partial),
                               a.tokens > 0 ? norm_backward_parts(a.tokens, a.hidden, a.dtype) : 0,
                               a.hidden, a.dw_pre, a.dw_post, dgate, ctas);
}

}  // namespace lpc
