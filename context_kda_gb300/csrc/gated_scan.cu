// Gated linear recurrence over packed sequences, per channel:
//     h_t = exp(g_t) h_{t-1} + i_t x_t,   h_{-1} = h0 of the sequence,
// its gradients and its single-token step.
//
// One thread walks one channel of one sequence.  The backward takes the states before every 128th
// token, recomputes the 128 states of a tile from them and walks the tile backwards:
//     G_t = dh_t + exp(g_{t+1}) G_{t+1}   (+ dfinal at the last token of a sequence),
//     dx = i G, di = x G, dg = exp(g_t) h_{t-1} G_t, dh0 = exp(g) G at the first token.
#include "elem.cuh"
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int TILE = KDA_SCAN_TILE;
constexpr int THREADS = 128;

__device__ int g_scan_status;

template <typename E>
__global__ void __launch_bounds__(THREADS) scan_forward(const int32_t *plan, PlanSig sig, int D, ScanIn in, void *h_,
                                                        int64_t ldh, float *final_state, float *states)
{
    if (!plan_matches(plan, sig)) {
        if (threadIdx.x == 0) record_status(&g_scan_status, KDA_ERR_INVALID_ARG);
        return;
    }
    const PlanView pv{plan};
    const int d = blockIdx.x * THREADS + threadIdx.x, T = pv.T();
    if (d >= D) return;
    const E *x = static_cast<const E *>(in.x) + d, *i = static_cast<const E *>(in.i);
    E *h = static_cast<E *>(h_) + d;
    if (i) i += d;
    for (int n = blockIdx.y; n < pv.N(); n += gridDim.y) {
        float s = in.h0 ? in.h0[static_cast<int64_t>(n) * D + d] : 0.f;
        const int t0 = pv.cu()[n], t1 = pv.cu()[n + 1];
        if (states && t0 == 0) states[d] = 0.f;
        for (int64_t t = t0; t < t1; ++t) {
            const float u = i ? to_f32(i[t * in.ldi]) * to_f32(x[t * in.ldx]) : to_f32(x[t * in.ldx]);
            s = fmaf(expf(in.g[t * in.ldg + d]), s, u);
            h[t * ldh] = from_f32<E>(s);
            if (states && (t + 1) % TILE == 0 && t + 1 < T) states[(t + 1) / TILE * D + d] = s;
        }
        if (final_state) final_state[static_cast<int64_t>(n) * D + d] = s;
    }
}

template <typename E>
__global__ void __launch_bounds__(THREADS) scan_backward(const int32_t *plan, PlanSig sig, int D, ScanIn in,
                                                         const float *states, const void *dh_, int64_t lddh,
                                                         const float *dfinal, ScanGrads out)
{
    if (!plan_matches(plan, sig)) {
        if (threadIdx.x == 0) record_status(&g_scan_status, KDA_ERR_INVALID_ARG);
        return;
    }
    const PlanView pv{plan};
    const int d = blockIdx.x * THREADS + threadIdx.x;
    if (d >= D) return;
    const E *x = static_cast<const E *>(in.x) + d, *i = static_cast<const E *>(in.i);
    const E *dh = static_cast<const E *>(dh_) + d;
    E *dx = static_cast<E *>(out.dx) + d, *di = static_cast<E *>(out.di);
    if (i) i += d;
    if (di) di += d;
    for (int n = blockIdx.y; n < pv.N(); n += gridDim.y) {
        const int t0 = pv.cu()[n], t1 = pv.cu()[n + 1];
        const float first = in.h0 ? in.h0[static_cast<int64_t>(n) * D + d] : 0.f;
        float G = dfinal ? dfinal[static_cast<int64_t>(n) * D + d] : 0.f;
        for (int64_t j = (t1 - 1) / TILE; j >= t0 / TILE; --j) {
            const int64_t a = max(j * TILE, static_cast<int64_t>(t0)), b = min((j + 1) * TILE, static_cast<int64_t>(t1));
            float before[TILE];
            float s = a == t0 ? first : states[j * D + d];
            for (int64_t t = a; t < b; ++t) {
                before[t - a] = s;
                const float u = i ? to_f32(i[t * in.ldi]) * to_f32(x[t * in.ldx]) : to_f32(x[t * in.ldx]);
                s = fmaf(expf(in.g[t * in.ldg + d]), s, u);
            }
            for (int64_t t = b - 1; t >= a; --t) {
                G += to_f32(dh[t * lddh]);
                const float xv = to_f32(x[t * in.ldx]), iv = i ? to_f32(i[t * in.ldi]) : 1.f;
                const float e = expf(in.g[t * in.ldg + d]) * G;
                dx[t * out.lddx] = from_f32<E>(iv * G);
                if (di) di[t * out.lddi] = from_f32<E>(xv * G);
                out.dg[t * out.lddg + d] = before[t - a] * e;
                G = e;
            }
        }
        if (out.dh0) out.dh0[static_cast<int64_t>(n) * D + d] = G;
    }
}

// One token per row, each the next one of its slot's state (updated in place).
template <typename E>
__global__ void __launch_bounds__(THREADS) scan_step(int B, int D, const int32_t *slots, int num_slots, ScanIn in,
                                                     float *state, void *h_, int64_t ldh)
{
    const int d = blockIdx.x * THREADS + threadIdx.x;
    if (d >= D) return;
    for (int64_t b = blockIdx.y; b < B; b += gridDim.y) {
        const int slot = slots ? slots[b] : static_cast<int>(b);
        E *h = static_cast<E *>(h_) + b * ldh + d;
        if (slot < 0 || slot >= num_slots) {
            *h = from_f32<E>(0.f);
            if (slot >= num_slots && d == 0) record_status(&g_scan_status, KDA_ERR_INVALID_ARG);
            continue;
        }
        const float x = to_f32(static_cast<const E *>(in.x)[b * in.ldx + d]);
        const float u = in.i ? x * to_f32(static_cast<const E *>(in.i)[b * in.ldi + d]) : x;
        float *s = state + static_cast<int64_t>(slot) * D + d;
        const float v = fmaf(expf(in.g[b * in.ldg + d]), *s, u);
        *s = v;
        *h = from_f32<E>(v);
    }
}

template <typename F>
cudaError_t by_type(int type, F f)
{
    if (type == KDA_TYPE_F32) f(float{});
    else if (type == KDA_TYPE_F16) f(__half{});
    else f(__nv_bfloat16{});
    return cudaGetLastError();
}

dim3 walk_grid(int D, int64_t rows)
{
    return dim3((D + THREADS - 1) / THREADS, static_cast<unsigned>(rows < 65535 ? rows : 65535));
}

}  // namespace

size_t scan_workspace_bytes(int64_t, int) { return 0; }

cudaError_t launch_scan_forward(const int32_t *plan_host, const int32_t *plan_dev, int D, int type, const ScanIn &in,
                                void *h, int64_t ldh, float *final_state, float *states, void *, cudaStream_t stream)
{
    return by_type(type, [&](auto e) {
        scan_forward<decltype(e)><<<walk_grid(D, plan_host[KDA_PH_N]), THREADS, 0, stream>>>(
            plan_dev, plan_sig(plan_host), D, in, h, ldh, final_state, states);
    });
}

cudaError_t launch_scan_backward(const int32_t *plan_host, const int32_t *plan_dev, int D, int type, const ScanIn &in,
                                 const float *states, const void *dh, int64_t lddh, const float *dfinal,
                                 const ScanGrads &out, void *, cudaStream_t stream)
{
    return by_type(type, [&](auto e) {
        scan_backward<decltype(e)><<<walk_grid(D, plan_host[KDA_PH_N]), THREADS, 0, stream>>>(
            plan_dev, plan_sig(plan_host), D, in, states, dh, lddh, dfinal, out);
    });
}

cudaError_t launch_scan_step(int B, int D, int type, const int32_t *slots, int num_slots, const ScanIn &in,
                             float *state, void *h, int64_t ldh, cudaStream_t stream)
{
    return by_type(type, [&](auto e) {
        scan_step<decltype(e)><<<walk_grid(D, B), THREADS, 0, stream>>>(B, D, slots, num_slots, in, state, h, ldh);
    });
}

int take_scan_status()
{
    int v = KDA_OK, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_scan_status, sizeof v) != cudaSuccess) return KDA_ERR_CUDA;
    if (v != KDA_OK && cudaMemcpyToSymbol(g_scan_status, &z, sizeof z) != cudaSuccess) return KDA_ERR_CUDA;
    return v;
}

}  // namespace kda
