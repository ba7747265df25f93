// Block norms: activations in fp32, the CTAs' column sums, and the dispatch by type (kernels in
// block_norm.cuh).
#include "block_norm.cuh"

namespace kda {
namespace norm {

cudaError_t forward_f32(int, Shape s, const NormIn &a, void *r_out, int64_t ldro, void *y, int64_t ldy, cudaStream_t stream)
{
    return pick_forward<float, float>(s, a, r_out, ldro, y, ldy, stream);
}

cudaError_t backward_f32(int, Shape s, const NormIn &a, const void *dro, int64_t lddro, const void *dy, int64_t lddy,
                         const NormGrads &g, float *part, int *grid, cudaStream_t stream)
{
    return pick_backward<float, float>(s, a, dro, lddro, dy, lddy, g, part, grid, stream);
}

namespace {

constexpr int RT = 1024, STRANDS = RT / 32;   // threads: 32 columns x 32 strands of CTAs

// Column c of [dw_post | dls | dw_pre] (G + 2 D of them): the CTAs' sums, strand by strand, the strands added up in order.
// Its blocks are dispatched while the last of those CTAs fold their sums; every thread has all of its loads in flight
// (8192 x 2048 gradients 51.9 us, 53.8 us with 8 strands a column that load one after the other).
__global__ void __launch_bounds__(RT) reduce(int ctas, int D, int G, const float *part, float *dw_post, float *dls, float *dw_pre)
{
    __shared__ float s[STRANDS][33];
    tc::grid_dep_wait();
    const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5, width = G + 2 * D;
    int c = blockIdx.x * 32 + lane;
    float v[(MAX_GRID + STRANDS - 1) / STRANDS];
#pragma unroll
    for (int k = 0; k < (MAX_GRID + STRANDS - 1) / STRANDS; ++k) {
        const int b = strand + k * STRANDS;
        v[k] = c < width && b < ctas ? part[static_cast<size_t>(b) * width + c] : 0.f;
    }
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < (MAX_GRID + STRANDS - 1) / STRANDS; ++k) sum += v[k];
    s[strand][lane] = sum;
    __syncthreads();
    // a warp a column now: the strands' sums, a lane each
    sum = s[lane][strand];
#pragma unroll
    for (int m = 16; m; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    c = blockIdx.x * 32 + strand;
    if (lane || c >= width) return;
    if (c < G) {
        if (dw_post) dw_post[c] = sum;
    } else if (c < G + D) {
        if (dls) dls[c - G] = sum;
    } else if (dw_pre) {
        dw_pre[c - G - D] = sum;
    }
}

}  // namespace
}  // namespace norm

size_t norm_workspace_bytes(int D) { return static_cast<size_t>(norm::MAX_GRID) * 3 * D * 4; }

cudaError_t launch_norm_forward(int64_t T, int D, int rtype, int type, const NormIn &a, void *r_out, int64_t ldro, void *y,
                                int64_t ldy, cudaStream_t stream)
{
    norm::Shape s = {};
    s.T = static_cast<uint32_t>(T);
    s.D = D;
    s.G = a.group ? a.group : D;
    s.inv_d = 1.f / D;
    s.inv_g = 1.f / s.G;
    s.wide_w = norm::rows_on(a.w_post, 0, 4) && norm::rows_on(a.ls, 0, 4) && norm::rows_on(a.w_pre, 0, 4);
    if (type == KDA_TYPE_F32) return norm::forward_f32(rtype, s, a, r_out, ldro, y, ldy, stream);
    if (type == KDA_TYPE_F16) return norm::forward_f16(rtype, s, a, r_out, ldro, y, ldy, stream);
    return norm::forward_bf16(rtype, s, a, r_out, ldro, y, ldy, stream);
}

cudaError_t launch_norm_backward(int64_t T, int D, int rtype, int type, const NormIn &a, const void *dr_out, int64_t lddro,
                                 const void *dy, int64_t lddy, const NormGrads &g, void *ws, cudaStream_t stream)
{
    norm::Shape s = {};
    s.T = static_cast<uint32_t>(T);
    s.D = D;
    s.G = a.group ? a.group : D;
    s.inv_d = 1.f / D;
    s.inv_g = 1.f / s.G;
    s.wide_w = norm::rows_on(a.w_post, 0, 4) && norm::rows_on(a.ls, 0, 4) && norm::rows_on(a.w_pre, 0, 4);
    float *part = static_cast<float *>(ws);
    int grid = 0;
    if (T > 0) {
        const cudaError_t e =
            type == KDA_TYPE_F32   ? norm::backward_f32(rtype, s, a, dr_out, lddro, dy, lddy, g, part, &grid, stream)
            : type == KDA_TYPE_F16 ? norm::backward_f16(rtype, s, a, dr_out, lddro, dy, lddy, g, part, &grid, stream)
                                   : norm::backward_bf16(rtype, s, a, dr_out, lddro, dy, lddy, g, part, &grid, stream);
        if (e != cudaSuccess) return e;
    }
    if (!g.dw_post && !g.dls && !g.dw_pre) return cudaSuccess;
    const int width = s.G + 2 * D;
    return launch_dependent(norm::reduce, dim3((width + 31) / 32), dim3(norm::RT), 0, stream, grid, D, s.G, part, g.dw_post, g.dls,
                            g.dw_pre);
}

}  // namespace kda
