// One KDA token per slot, from and into the slot's fp32 state (K x V per head):
//     S~ = Diag(exp g) S,  d = beta (v - S~^T k),  S = S~ + k d^T,  o = scale S^T q.
//
// The state is 64 KiB a head and is read and written once; nothing else matters, so the kernel is a copy
// with a product on the way.  Value columns do not depend on one another: a CTA takes 64 columns of
// one (token, head), its 256 threads load them in 16-byte pieces (all before the first use) and hold
// them in registers.  S~^T k and S~^T q come from one pass over the registers, and
//     o = scale (S~^T q + (q . k) d),
// so that the columns are summed once, before the update.
// Bound by memory: 256 tokens x 32 heads in bf16 take 160 us (6.79 TB/s, the rate of a copy) with 64 columns a CTA, 164 us
// with 128 and 171 us with 32; 2 x 16 heads take 3.5 us, the launch and one trip to memory.
#include "elem.cuh"
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int CT = 64;                   // value columns of a CTA

__device__ int g_decode_status;

template <typename E>
__global__ void __launch_bounds__(THREADS) decode_step(int H, const int32_t *slots, int num_slots, DecodeIn in, float scale,
                                                       float *state, void *o_, int64_t ldo)
{
    constexpr int LANES = CT / 4;            // lanes of a row's columns
    constexpr int ROWS = THREADS / LANES;    // rows of one load of the CTA
    constexpr int R = KD / ROWS;             // rows of a thread
    __shared__ float4 s_row[KD];             // exp g, k, q of a row
    __shared__ float s_sum[2][WARPS][CT];
    __shared__ float s_dot[KD / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c0 = blockIdx.x * CT, h = blockIdx.y;
    const int64_t b = blockIdx.z;
    const int slot = slots ? slots[b] : static_cast<int>(b);
    E *o = static_cast<E *>(o_) + b * ldo + h * VD + c0;
    if (slot < 0 || slot >= num_slots) {
        if (tid < CT) o[tid] = from_f32<E>(0.f);
        if (slot >= num_slots && tid == 0) record_status(&g_decode_status, KDA_ERR_INVALID_ARG);
        return;
    }
    const int col = (tid % LANES) * 4, row0 = tid / LANES;
    float *S = state + ((static_cast<int64_t>(slot) * H + h) * KD + row0) * VD + c0 + col;
    float4 s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = *reinterpret_cast<const float4 *>(S + r * ROWS * VD);
    if (tid < KD) {
        const float a = expf(in.g[b * in.ldg + h * KD + tid]);
        const float k = to_f32(static_cast<const E *>(in.k)[b * in.ldk + h * KD + tid]);
        const float q = to_f32(static_cast<const E *>(in.q)[b * in.ldq + h * KD + tid]);
        s_row[tid] = make_float4(a, k, q, 0.f);
        float dot = q * k;
        for (int m = 16; m; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
        if (lane == 0) s_dot[warp] = dot;
    }
    float v = 0.f, beta = 0.f;
    if (tid < CT) {
        v = to_f32(static_cast<const E *>(in.v)[b * in.ldv + h * VD + c0 + tid]);
        beta = in.beta[b * in.ldb + h];
    }
    __syncthreads();
    float u[4] = {}, w[4] = {};
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float4 p = s_row[row0 + r * ROWS];
        s[r].x *= p.x;
        s[r].y *= p.x;
        s[r].z *= p.x;
        s[r].w *= p.x;
        u[0] = fmaf(p.y, s[r].x, u[0]);
        u[1] = fmaf(p.y, s[r].y, u[1]);
        u[2] = fmaf(p.y, s[r].z, u[2]);
        u[3] = fmaf(p.y, s[r].w, u[3]);
        w[0] = fmaf(p.z, s[r].x, w[0]);
        w[1] = fmaf(p.z, s[r].y, w[1]);
        w[2] = fmaf(p.z, s[r].z, w[2]);
        w[3] = fmaf(p.z, s[r].w, w[3]);
    }
#pragma unroll
    for (int m = LANES; m < 32; m *= 2)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u[j] += __shfl_xor_sync(0xffffffffu, u[j], m);
            w[j] += __shfl_xor_sync(0xffffffffu, w[j], m);
        }
    if (lane < LANES) {
        *reinterpret_cast<float4 *>(&s_sum[0][warp][col]) = make_float4(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<float4 *>(&s_sum[1][warp][col]) = make_float4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();
    if (tid < CT) {
        float su = 0.f, sw = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < WARPS; ++j) {
            su += s_sum[0][j][tid];
            sw += s_sum[1][j][tid];
        }
#pragma unroll
        for (int j = 0; j < KD / 32; ++j) dot += s_dot[j];
        const float d = beta * (v - su);
        o[tid] = from_f32<E>(scale * fmaf(dot, d, sw));
        s_sum[0][0][tid] = d;      // read above by this thread alone
    }
    __syncthreads();
    const float4 d = *reinterpret_cast<const float4 *>(&s_sum[0][0][col]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float k = s_row[row0 + r * ROWS].y;
        s[r].x = fmaf(k, d.x, s[r].x);
        s[r].y = fmaf(k, d.y, s[r].y);
        s[r].z = fmaf(k, d.z, s[r].z);
        s[r].w = fmaf(k, d.w, s[r].w);
        *reinterpret_cast<float4 *>(S + r * ROWS * VD) = s[r];
    }
}

template <typename E>
cudaError_t launch(int B, int H, const int32_t *slots, int num_slots, const DecodeIn &in, float scale, float *state, void *o,
                   int64_t ldo, cudaStream_t stream)
{
    // grid.z is at most 65535: more tokens go in several launches
    for (int64_t b = 0; b < B; b += 65535) {
        const int n = static_cast<int>(B - b < 65535 ? B - b : 65535);
        DecodeIn p = in;
        p.q = static_cast<const E *>(in.q) + b * in.ldq;
        p.k = static_cast<const E *>(in.k) + b * in.ldk;
        p.v = static_cast<const E *>(in.v) + b * in.ldv;
        p.g = in.g + b * in.ldg;
        p.beta = in.beta + b * in.ldb;
        const int32_t *sl = slots ? slots + b : nullptr;
        float *st = slots ? state : state + b * H * KD * VD;
        E *out = static_cast<E *>(o) + b * ldo;
        decode_step<E><<<dim3(VD / CT, H, n), THREADS, 0, stream>>>(H, sl, num_slots, p, scale, st, out, ldo);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_step(int B, int H, int type, const int32_t *slots, int num_slots, const DecodeIn &in, float scale,
                               float *state, void *o, int64_t ldo, cudaStream_t stream)
{
    if (type == KDA_TYPE_F32) return launch<float>(B, H, slots, num_slots, in, scale, state, o, ldo, stream);
    if (type == KDA_TYPE_F16) return launch<__half>(B, H, slots, num_slots, in, scale, state, o, ldo, stream);
    return launch<__nv_bfloat16>(B, H, slots, num_slots, in, scale, state, o, ldo, stream);
}

int take_decode_status()
{
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_decode_status, sizeof(int)) != cudaSuccess) return KDA_ERR_CUDA;
    if (v != 0 && cudaMemcpyToSymbol(g_decode_status, &z, sizeof(int)) != cudaSuccess) return KDA_ERR_CUDA;
    return v;
}

}  // namespace kda
