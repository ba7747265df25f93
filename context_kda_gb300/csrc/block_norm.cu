// The norms around a block, fused with the block's gate and the residual:
//     n = o * inv_o * w_post,   inv_o = 1 / sqrt(mean_group(o^2) + eps)     (n = o without w_post)
//     u = act(z) * n,           act = 1, sigmoid or silu
//     r' = r + scale * ls * u                                                (stored in the residual's type)
//     y = r' * inv_r * w_pre,   inv_r = 1 / sqrt(mean_row(r'^2) + eps)       (of r' before it is rounded)
// and the gradients of r, o, z, w_post, ls and w_pre from those of r' and y.
//
// The gradient through v -> v / rms(v), for e = the gradient of v / rms, is written so that what cancels
// exactly (a group of one channel) cancels exactly in fp32 too:
//     (e_j - v_j inv^2 mean(e v)) inv = inv^3 (e_j (mean(v^2) - v_j^2 / G + eps) - v_j (sum(e v) - e_j v_j) / G).
//
// One CTA per row, a row's values in shared memory between its passes.  The backward's column sums
// are kept per CTA in the workspace and added up in a fixed order by a second kernel.
#include "elem.cuh"
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;

// Sum over the CTA; every thread gets it.  'buf' holds WARPS floats.
__device__ __forceinline__ float block_sum(float v, float *buf)
{
    for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < WARPS; ++w) s += buf[w];
    return s;
}

__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

// The gate's value and, times what follows it, its derivative.
__device__ __forceinline__ void gate_of(int kind, float z, float &act, float &slope)
{
    act = 1.f;
    slope = 0.f;
    if (kind == KDA_GATE_NONE) return;
    const float p = sigmoid(z);
    act = kind == KDA_GATE_SIGMOID ? p : z * p;
    slope = kind == KDA_GATE_SIGMOID ? p * (1.f - p) : p * (1.f + z * (1.f - p));
}

// The gradient of v through v / rms from e, the gradient of v / rms (formula at the top): ss = sum of the
// group's v^2, ev = sum of its e v; the products are rounded as the sums' terms were.
__device__ __forceinline__ float unit_grad(float e, float v, float inv, float ss, float ev, int G, float eps)
{
    return inv * inv * inv * (e * ((ss - __fmul_rn(v, v)) / G + eps) - v * ((ev - __fmul_rn(e, v)) / G));
}

// inv[group] = f(sum over the group of v(col)) for every group of G columns (G = D, or a multiple of 32).
template <typename V, typename F>
__device__ __forceinline__ void group_sums(int D, int G, V v, F f, float *seg, float *inv, float *buf)
{
    if (G == D) {
        float s = 0.f;
        for (int c = threadIdx.x; c < D; c += THREADS) s += v(c);
        s = block_sum(s, buf);
        if (threadIdx.x == 0) inv[0] = f(s);
        __syncthreads();
        return;
    }
    for (int c = threadIdx.x; c < D; c += THREADS) {   // D is a multiple of 32: whole warps
        float s = v(c);
        for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(__activemask(), s, m);
        if ((threadIdx.x & 31) == 0) seg[c >> 5] = s;
    }
    __syncthreads();
    for (int j = threadIdx.x; j < D / G; j += THREADS) {
        float s = 0.f;
        for (int k = 0; k < G / 32; ++k) s += seg[j * (G / 32) + k];
        inv[j] = f(s);
    }
    __syncthreads();
}

template <typename R, typename E>
__global__ void __launch_bounds__(THREADS) norm_forward(int64_t T, int D, NormIn a, void *r_out, int64_t ldro, void *y,
                                                        int64_t ldy)
{
    extern __shared__ float sm[];
    float *row = sm, *seg = row + D, *inv = seg + D / 32 + 1, *buf = inv + D / 32 + 1;
    const int G = a.group ? a.group : D;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const E *o = static_cast<const E *>(a.o), *z = static_cast<const E *>(a.z);
        const R *r = static_cast<const R *>(a.r);
        if (o) o += t * a.ldo;
        if (z) z += t * a.ldz;
        if (r) r += t * a.ldr;
        if (o && a.w_post)
            group_sums(D, G, [&](int c) { const float v = to_f32(o[c]); return v * v; },
                       [&](float s) { return 1.f / sqrtf(s / G + a.eps); }, seg, inv, buf);
        float ss = 0.f;
        for (int c = threadIdx.x; c < D; c += THREADS) {
            float v = r ? to_f32(r[c]) : 0.f;
            if (o) {
                float n = to_f32(o[c]), act = 1.f, slope;
                if (a.w_post) n *= inv[c / G] * a.w_post[c % G];
                if (z) gate_of(a.gate, to_f32(z[c]), act, slope);
                v += a.scale * (a.ls ? a.ls[c] : 1.f) * act * n;
            }
            row[c] = v;
            ss += v * v;
            if (r_out) static_cast<R *>(r_out)[t * ldro + c] = from_f32<R>(v);
        }
        if (y) {
            const float inv_r = 1.f / sqrtf(block_sum(ss, buf) / D + a.eps);
            for (int c = threadIdx.x; c < D; c += THREADS)
                static_cast<E *>(y)[t * ldy + c] = from_f32<E>(row[c] * inv_r * a.w_pre[c]);
        }
        __syncthreads();
    }
}

// part: [grid][3][D], this CTA's column sums of w_post (per column), ls and w_pre.
template <typename R, typename E>
__global__ void __launch_bounds__(THREADS) norm_backward(int64_t T, int D, NormIn a, const void *dr_out_,
                                                         int64_t lddro, const void *dy_, int64_t lddy, NormGrads g,
                                                         float *part)
{
    extern __shared__ float sm[];
    float *row = sm, *seg = row + D, *sq = seg + D / 32 + 1, *proj = sq + D / 32 + 1, *buf = proj + D / 32 + 1;
    const int G = a.group ? a.group : D;
    part += static_cast<size_t>(blockIdx.x) * 3 * D;
    for (int c = threadIdx.x; c < 3 * D; c += THREADS) part[c] = 0.f;
    __syncthreads();
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const E *o = static_cast<const E *>(a.o), *z = static_cast<const E *>(a.z), *dy = static_cast<const E *>(dy_);
        const R *r = static_cast<const R *>(a.r), *dro = static_cast<const R *>(dr_out_);
        if (o) o += t * a.ldo;
        if (z) z += t * a.ldz;
        float inv_r = 0.f, ss = 0.f, ev = 0.f;
        if (a.w_pre) {
            r += t * a.ldr;
            dy += t * lddy;
            float s = 0.f, p = 0.f;
            for (int c = threadIdx.x; c < D; c += THREADS) {
                const float v = to_f32(r[c]);
                s += v * v;
                p += to_f32(dy[c]) * a.w_pre[c] * v;
            }
            ss = block_sum(s, buf);
            ev = block_sum(p, buf);
            inv_r = 1.f / sqrtf(ss / D + a.eps);
        }
        if (dro) dro += t * lddro;
        for (int c = threadIdx.x; c < D; c += THREADS) {
            float v = dro ? to_f32(dro[c]) : 0.f;
            if (a.w_pre) {
                const float rv = to_f32(r[c]), d = to_f32(dy[c]);
                part[2 * D + c] += d * rv * inv_r;
                v += unit_grad(d * a.w_pre[c], rv, inv_r, ss, ev, D, a.eps);
            }
            row[c] = v;
            if (g.dr) static_cast<R *>(g.dr)[t * g.lddr + c] = from_f32<R>(v);
        }
        if (!o) {
            __syncthreads();
            continue;
        }
        if (a.w_post)
            group_sums(D, G, [&](int c) { const float v = to_f32(o[c]); return v * v; }, [&](float s) { return s; }, seg, sq, buf);
        for (int c = threadIdx.x; c < D; c += THREADS) {
            const float hat = to_f32(o[c]) * (a.w_post ? 1.f / sqrtf(sq[c / G] / G + a.eps) : 1.f);
            const float w = a.w_post ? a.w_post[c % G] : 1.f;
            float act = 1.f, slope = 0.f;
            if (z) gate_of(a.gate, to_f32(z[c]), act, slope);
            const float tt = a.scale * row[c];
            if (a.ls) part[D + c] += tt * act * hat * w;
            const float du = a.ls ? tt * a.ls[c] : tt;
            if (g.dz) static_cast<E *>(g.dz)[t * g.lddz + c] = from_f32<E>(du * hat * w * slope);
            const float dn = du * act;
            if (a.w_post) part[c] += dn * hat;
            row[c] = dn * w;
        }
        __syncthreads();
        if (a.w_post)
            group_sums(D, G, [&](int c) { return row[c] * to_f32(o[c]); }, [&](float s) { return s; }, seg, proj, buf);
        for (int c = threadIdx.x; c < D; c += THREADS) {
            float v = row[c];
            if (a.w_post) {
                const float ss = sq[c / G];
                v = unit_grad(v, to_f32(o[c]), 1.f / sqrtf(ss / G + a.eps), ss, proj[c / G], G, a.eps);
            }
            static_cast<E *>(g.d_o)[t * g.lddo + c] = from_f32<E>(v);
        }
        __syncthreads();
    }
}

// The CTAs' column sums added up in order; w_post's also over the groups.
__global__ void __launch_bounds__(THREADS) norm_reduce(int ctas, int D, int G, const float *part, float *dw_post, float *dls,
                                                       float *dw_pre)
{
    const int c = blockIdx.x * THREADS + threadIdx.x;
    if (c >= D) return;
    float ls = 0.f, pre = 0.f;
    for (int b = 0; b < ctas; ++b) {
        ls += part[(static_cast<size_t>(b) * 3 + 1) * D + c];
        pre += part[(static_cast<size_t>(b) * 3 + 2) * D + c];
    }
    if (dls) dls[c] = ls;
    if (dw_pre) dw_pre[c] = pre;
    if (!dw_post || c >= G) return;
    float s = 0.f;
    for (int b = 0; b < ctas; ++b)
        for (int k = c; k < D; k += G) s += part[static_cast<size_t>(b) * 3 * D + k];
    dw_post[c] = s;
}

template <typename F>
cudaError_t by_types(int rtype, int type, F f)
{
    if (rtype == KDA_TYPE_F32) {
        if (type == KDA_TYPE_F32) return f(float{}, float{});
        if (type == KDA_TYPE_F16) return f(float{}, __half{});
        return f(float{}, __nv_bfloat16{});
    }
    if (rtype == KDA_TYPE_F16) return f(__half{}, __half{});
    return f(__nv_bfloat16{}, __nv_bfloat16{});
}

size_t smem_bytes(int D) { return (static_cast<size_t>(D) + 3 * (D / 32 + 1) + WARPS) * 4; }

constexpr int MAX_GRID = 304;   // CTAs of a launch: rows of the backward's column sums

}  // namespace

size_t norm_workspace_bytes(int D) { return static_cast<size_t>(MAX_GRID) * 3 * D * 4; }

cudaError_t launch_norm_forward(int64_t T, int D, int rtype, int type, const NormIn &a, void *r_out, int64_t ldro, void *y,
                                int64_t ldy, cudaStream_t stream)
{
    return by_types(rtype, type, [&](auto r, auto e) {
        auto fn = norm_forward<decltype(r), decltype(e)>;
        if (cudaError_t err = set_dynamic_smem(reinterpret_cast<const void *>(fn), static_cast<int>(smem_bytes(D)))) return err;
        fn<<<static_cast<unsigned>(T < 4096 ? T : 4096), THREADS, smem_bytes(D), stream>>>(T, D, a, r_out, ldro, y, ldy);
        return cudaGetLastError();
    });
}

cudaError_t launch_norm_backward(int64_t T, int D, int rtype, int type, const NormIn &a, const void *dr_out, int64_t lddro,
                                 const void *dy, int64_t lddy, const NormGrads &g, void *ws, cudaStream_t stream)
{
    const int grid = static_cast<int>(T < MAX_GRID ? T : MAX_GRID);
    float *part = static_cast<float *>(ws);
    if (grid) {
        const cudaError_t err = by_types(rtype, type, [&](auto r, auto e) {
            auto fn = norm_backward<decltype(r), decltype(e)>;
            if (cudaError_t x = set_dynamic_smem(reinterpret_cast<const void *>(fn), static_cast<int>(smem_bytes(D)))) return x;
            fn<<<grid, THREADS, smem_bytes(D), stream>>>(T, D, a, dr_out, lddro, dy, lddy, g, part);
            return cudaGetLastError();
        });
        if (err != cudaSuccess) return err;
    }
    norm_reduce<<<(D + THREADS - 1) / THREADS, THREADS, 0, stream>>>(grid, D, a.group ? a.group : D, part, g.dw_post, g.dls,
                                                                    g.dw_pre);
    return cudaGetLastError();
}

}  // namespace kda
