// lpcoll_layernorm.cu -- layer_norm and its gradients (kernels in
// lpcoll_layernorm.cuh), and the sums over tokens that both operators' gradients
// end with.
#include "lpcoll_layernorm.cuh"

namespace lpc {

namespace {

// Column sums of the workspace: a CTA adds 32 columns of one of the two sums. Of a
// part, kVec columns a thread; the CTA's threads take as many parts at once as they
// can, each thread all of its own with their loads in flight together, and a warp adds
// up a column's threads. Measured with the stores that leave the parts: 8192 columns of
// 152 CTAs 14 us with 4-byte accesses and 1024 threads.
template <int kVec> constexpr int kSumThreads = kVec == 4 ? 256 : 1024;

template <int kVec>
__global__ void __launch_bounds__(kSumThreads<kVec>)
layer_norm_sums_kernel(const float *partial, float *dw, float *db, int hidden, int parts,
                       int column_ctas)
{
    wait_prior_grid();
    constexpr int kAcross = 32 / kVec;                // threads of a part's 32 columns
    constexpr int kDown = kSumThreads<kVec> / kAcross;  // parts at once
    static_assert(kDown == 32, "a warp adds up a column");
    constexpr int kSteps = (kMaxCtas * kSms + kDown - 1) / kDown;
    __shared__ float red[kDown][33];
    const int which = blockIdx.x / column_ctas;
    float *const out = which == 0 ? dw : db;
    if (out == nullptr)
        return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int first = (blockIdx.x % column_ctas) * 32;
    const int across = tid % kAcross, down = tid / kAcross;
    const int col = first + across * kVec;
    const float *const p = partial + static_cast<size_t>(which) * parts * hidden;
    Vec<kVec> v[kSteps], sum = {};
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int q = i * kDown + down;
        v[i] = {};
        if (q < parts && col < hidden)
            v[i] = load_vec_of<LPCOLL_F32, 4 * kVec>(p, static_cast<size_t>(q) * hidden + col);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
        sum = plus(sum, v[i]);
#pragma unroll
    for (int j = 0; j < kVec; ++j)
        red[down][across * kVec + j] = sum.v[j];
    __syncthreads();
    for (int c = warp; c < 32; c += kSumThreads<kVec> / 32) {
        const float all = warp_sum(red[lane][c]);
        if (lane == 0 && first + c < hidden)
            store_f32(out + first + c, all);
    }
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
    const int ctas = (a.hidden + 31) / 32;
    if (a.hidden % 4 == 0)
        return launch_kernel_block(layer_norm_sums_kernel<4>, static_cast<size_t>(2) * ctas,
                                   kSumThreads<4>, 0, st, a.partial, a.dw, a.db, a.hidden, parts, ctas);
    return launch_kernel_block(layer_norm_sums_kernel<1>, static_cast<size_t>(2) * ctas,
                               kSumThreads<1>, 0, st, a.partial, a.dw, a.db, a.hidden, parts, ctas);
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
