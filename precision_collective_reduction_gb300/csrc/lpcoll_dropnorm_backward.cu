// lpcoll_dropnorm_backward.cu -- the gradients of residual_dropout with its norm
// (kernels in lpcoll_layernorm.cuh).
#include "lpcoll_layernorm.cuh"

namespace lpc {

cudaError_t launch_dropout_norm_backward(const LayerNormArgs &args, cudaStream_t st)
{
    LayerNormArgs a = args;
    const bool sums = a.dw != nullptr || a.db != nullptr;
    if (!sums)
        a.partial = nullptr;
    int parts = 0;
    if (a.tokens > 0) {
        const Plan p = layer_norm_backward_plan(a.tokens, a.hidden, a.dtype, true);
        parts = p.ctas;
        const cudaError_t e =
            LPC_BY_ROW(backward_drop, a.dtype, static_cast<size_t>(a.hidden), a, p, st);
        if (e != cudaSuccess)
            return e;
    }
    return sums ? launch_layer_norm_sums(a, parts, st) : cudaSuccess;
}

}  // namespace lpc
