// Block norms, forward, activations in bf16 (kernels in block_norm.cuh).
#include "block_norm.cuh"

namespace kda {
namespace norm {

cudaError_t forward_bf16(int rtype, Shape s, const NormIn &a, void *r_out, int64_t ldro, void *y, int64_t ldy, cudaStream_t stream)
{
    return rtype == KDA_TYPE_F32 ? pick_forward<float, __nv_bfloat16>(s, a, r_out, ldro, y, ldy, stream)
                                 : pick_forward<__nv_bfloat16, __nv_bfloat16>(s, a, r_out, ldro, y, ldy, stream);
}

}  // namespace norm
}  // namespace kda
