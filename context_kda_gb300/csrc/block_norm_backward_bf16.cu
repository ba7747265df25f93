// Block norms, backward, activations in bf16 (kernels in block_norm.cuh).
#include "block_norm.cuh"

namespace kda {
namespace norm {

cudaError_t backward_bf16(int rtype, Shape s, const NormIn &a, const void *dro, int64_t lddro, const void *dy, int64_t lddy, const NormGrads &g, float *part, int *grid, cudaStream_t stream)
{
    return rtype == KDA_TYPE_F32 ? pick_backward<float, __nv_bfloat16>(s, a, dro, lddro, dy, lddy, g, part, grid, stream)
                                 : pick_backward<__nv_bfloat16, __nv_bfloat16>(s, a, dro, lddro, dy, lddy, g, part, grid, stream);
}

}  // namespace norm
}  // namespace kda
