// lpcoll_dropnorm.cu -- residual_dropout with its norm (kernels in
// lpcoll_layernorm.cuh).
#include "lpcoll_layernorm.cuh"

namespace lpc {

cudaError_t launch_dropout_norm(const LayerNormArgs &a, cudaStream_t st)
{
    return LPC_BY_ROW(forward_drop, a.dtype, static_cast<size_t>(a.hidden), a, st);
}

}  // namespace lpc
