// lpcoll_layernorm.cu -- layer_norm and its gradients (kernels in
// lpcoll_layernorm.cuh), and the sums over tokens that both operators' gradients
// end with.
#include "lpcoll_layernorm.cuh"

namespace lpc {

namespace {

// Column sums of the workspace: a CTA adds 32 columns of one of the two sums.
// 32 threads per column take every 32nd part, all in flight at once (kPer of
// them, for as many CTAs per SM), and a warp adds up a column's 32.
constexpr int kPer = (kSms + 31) / 32;

template <int kPerSm>
__global__ void __launch_bounds__(1024)
layer_norm_sums_kernel(const float *partial, float *dw, float *db, int hidden, int parts,
                       int column_ctas)
{
    wait_prior_grid();
    __shared__ float red[32][33];
    const int which = blockIdx.x / column_ctas;
    float *const out = which == 0 ? dw : db;
    if (out == nullptr)
        return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first = (blockIdx.x % column_ctas) * 32;
    const float *p = partial + static_cast<size_t>(which) * parts * hidden + first + lane;
    constexpr int kParts = kPer * kPerSm;
    float v[kParts];
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        const int q = i * 32 + warp;
        v[i] = q < parts && first + lane < hidden ? load_f32(p + static_cast<size_t>(q) * hidden)
                                                  : 0.0f;
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kParts; ++i)
        sum += v[i];
    red[warp][lane] = sum;
    __syncthreads();
    sum = warp_sum(red[lane][warp]);
    if (lane == 0 && first + warp < hidden)
        store_f32(out + first + warp, sum);
}

}  // namespace

int layer_norm_parts(size_t tokens, size_t hidden, int dtype, bool dropout)
{
    if (tokens == 0 || hidden == 0)
        return 0;
    return layer_norm_backward_plan(tokens, static_cast<int>(hidden), dtype, dropout).ctas;
}

cudaError_t launch_layer_norm_sums(const LayerNormArgs &a, int parts, cudaStream_t st)
{
    static_assert(kMaxCtas == 3, "one kernel per number of CTAs per SM");
    const int ctas = (a.hidden + 31) / 32;
    const auto kernel = parts <= kSms ? layer_norm_sums_kernel<1>
                                      : (parts <= 2 * kSms ? layer_norm_sums_kernel<2>
                                                           : layer_norm_sums_kernel<3>);
    return launch_kernel_block(kernel, static_cast<size_t>(2) * ctas, 1024, 0, st, a.partial, a.dw,
                               a.db, a.hidden, parts, ctas);
}

cudaError_t launch_layer_norm(const LayerNormArgs &a, cudaStream_t st)
{
    return LPC_BY_ROW(forward_plain, a.dtype, static_cast<size_t>(a.hidden), a, st);
}

cudaError_t launch_layer_norm_backward(const LayerNormArgs &args, cudaStream_t st)
{
    LayerNormArgs a = args;
    const bool sums = a.dw != nullptr || a.db != nullptr;
    if (!sums)
        a.partial = nullptr;
    int parts = 0;
    if (a.tokens > 0) {
        const Plan p = layer_norm_backward_plan(a.tokens, a.hidden, a.dtype, false);
        parts = p.ctas;
        const cudaError_t e =
            LPC_BY_ROW(backward_plain, a.dtype, static_cast<size_t>(a.hidden), a, p, st);
        if (e != cudaSuccess)
            return e;
    }
    return sums ? launch_layer_norm_sums(a, parts, st) : cudaSuccess;
}

}  // namespace lpc
