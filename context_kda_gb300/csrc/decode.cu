// One KDA token per slot, from and into the slot's fp32 state (K x V per head):
//     S~ = Diag(exp g) S,  d = beta (v - S~^T k),  S = S~ + k d^T,  o = scale S^T q.
//
// One CTA per (token, head), one thread per value column: it reads its column twice (for S~^T k, then
// for the update) and writes it once.
#include "elem.cuh"
#include "kda_internal.cuh"

namespace kda {
namespace {

__device__ int g_decode_status;

template <typename E>
__global__ void __launch_bounds__(VD) decode_step(int B, int H, const int32_t *slots, int num_slots, DecodeIn in, float scale,
                                                  float *state, void *o_, int64_t ldo)
{
    __shared__ float s_a[KD], s_k[KD], s_q[KD];
    const int h = blockIdx.y, c = threadIdx.x;
    const int64_t b = blockIdx.x;
    const int slot = slots ? slots[b] : static_cast<int>(b);
    E *o = static_cast<E *>(o_) + b * ldo + h * VD + c;
    if (slot < 0 || slot >= num_slots) {
        *o = from_f32<E>(0.f);
        if (slot >= num_slots && c == 0) record_status(&g_decode_status, KDA_ERR_INVALID_ARG);
        return;
    }
    s_a[c] = expf(in.g[b * in.ldg + h * KD + c]);
    s_k[c] = to_f32(static_cast<const E *>(in.k)[b * in.ldk + h * KD + c]);
    s_q[c] = to_f32(static_cast<const E *>(in.q)[b * in.ldq + h * KD + c]);
    __syncthreads();
    float *S = state + (static_cast<int64_t>(slot) * H + h) * KD * VD + c;
    float u = 0.f;
    for (int k = 0; k < KD; ++k) u = fmaf(s_k[k], s_a[k] * S[k * VD], u);
    const float d = in.beta[b * in.ldb + h] * (to_f32(static_cast<const E *>(in.v)[b * in.ldv + h * VD + c]) - u);
    float y = 0.f;
    for (int k = 0; k < KD; ++k) {
        const float v = fmaf(s_k[k], d, s_a[k] * S[k * VD]);
        S[k * VD] = v;
        y = fmaf(s_q[k], v, y);
    }
    *o = from_f32<E>(scale * y);
}

}  // namespace

cudaError_t launch_decode_step(int B, int H, int type, const int32_t *slots, int num_slots, const DecodeIn &in, float scale,
                               float *state, void *o, int64_t ldo, cudaStream_t stream)
{
    const dim3 grid(B, H);
    if (type == KDA_TYPE_F32) decode_step<float><<<grid, VD, 0, stream>>>(B, H, slots, num_slots, in, scale, state, o, ldo);
    else if (type == KDA_TYPE_F16) decode_step<__half><<<grid, VD, 0, stream>>>(B, H, slots, num_slots, in, scale, state, o, ldo);
    else decode_step<__nv_bfloat16><<<grid, VD, 0, stream>>>(B, H, slots, num_slots, in, scale, state, o, ldo);
    return cudaGetLastError();
}

int take_decode_status()
{
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_decode_status, sizeof(int)) != cudaSuccess) return KDA_ERR_CUDA;
    if (v != 0 && cudaMemcpyToSymbol(g_decode_status, &z, sizeof(int)) != cudaSuccess) return KDA_ERR_CUDA;
    return v;
}

}  // namespace kda
