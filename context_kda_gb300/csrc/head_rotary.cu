// Norms of the query and key heads with the position rotation in the same pass, and the gradients.
//
//     n = x / sqrt(mean(x^2) + eps) * w,     (a, b) -> (a cos - b sin, a sin + b cos) for every pair of rotated channels,
//
// the angle position * frequency.  The frequency comes as a 64-bit fraction of a turn, so that the product modulo 2^64
// is the reduced angle itself, exact at any position; its top 32 bits go to sincospi.
//
// A lane holds 8 adjacent channels of a head (16 bytes of a 16-bit type), a head is d / 8 lanes, and a warp works one token's
// heads: the norm's sum is a few shuffles, the other channel of a pair is in the lane itself (adjacent pairs) or a
// fixed lane away (halves).  The angles of a token are the same for all its heads: they are made once a token, two or so
// a lane, and go through shared memory.  Few tokens are cut into parts of their heads, so that a decoding step
// fills more than a few warps.
// Bound by memory: 65536 tokens x 40 heads of 128 in bf16 take 236 us (84 % of a copy), gradients of 8192 x 32 heads 58 us (51 %: 16
// warps an SM is what their registers allow), 8 tokens 6 us.  Chunks fetched ahead by bulk copies (as in the
// attention's step) bring nothing: they leave the gradients at 59 us, and the forward, whose registers they take, at 327 us.
#include "elem.cuh"
#include "kda_internal.cuh"
#include "tc.cuh"

namespace kda {
namespace {

constexpr int V = 8;                    // channels of a lane
constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int MAX_GRID = 512;           // CTAs whose sums of the weights' gradients the workspace holds

struct Work {
    HeadIn in;
    int64_t tasks;                      // tokens x parts
    int parts, steps, per_part;         // warp steps (32 / (d / 8) heads each) of a token, of a part
};

// 8 channels as they lie in memory.
template <typename E> struct Raw {
    uint4 v[sizeof(E) / 2];
};

template <typename E, bool ALIGNED> __device__ __forceinline__ void load(Raw<E> &r, const E *p)
{
    if constexpr (ALIGNED) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(E) / 2); ++i) r.v[i] = reinterpret_cast<const uint4 *>(p)[i];
    } else {
        E *e = reinterpret_cast<E *>(&r);
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = p[j];
    }
}

template <typename E> __device__ __forceinline__ void widen(const Raw<E> &r, float (&x)[V])
{
    const E *e = reinterpret_cast<const E *>(&r);
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = to_f32(e[j]);
}

template <typename E, bool ALIGNED> __device__ __forceinline__ void store(E *p, const float (&x)[V])
{
    Raw<E> r;
    E *e = reinterpret_cast<E *>(&r);
#pragma unroll
    for (int j = 0; j < V; ++j) e[j] = from_f32<E>(x[j]);
    if constexpr (ALIGNED) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(E) / 2); ++i) reinterpret_cast<uint4 *>(p)[i] = r.v[i];
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) p[j] = e[j];
    }
}

// A lane's rotation: its channels times 'c' plus their partners times 's' (the sign of the pair's member in it).
struct Turn {
    float c[V], s[V];
    int partner;                        // lane of the other channels; adjacent pairs: -1
    bool on;
};

// The token's angles, through 'tab' (d / 2 entries of this warp).  dir: 1 or, for the gradients, -1.
template <int D> __device__ __forceinline__ void make_turn(const HeadIn &in, int64_t t, float dir, float2 *tab, Turn &turn)
{
    const int lane = threadIdx.x & 31, l = lane % (D / V), half = in.rot / 2;
    if (in.rot == 0) return;
    const uint64_t pos = static_cast<uint64_t>(static_cast<int64_t>(in.positions[t]));
    __syncwarp();
    for (int i = lane; i < half; i += 32) {
        const int32_t top = static_cast<int32_t>((pos * in.phases[i]) >> 32);
        float s, c;
        sincospif(static_cast<float>(top) * 0x1p-31f, &s, &c);
        tab[i] = make_float2(c, s);
    }
    __syncwarp();
    if (!turn.on) return;
    if (in.adjacent) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            const float2 a = tab[l * (V / 2) + j];
            turn.c[2 * j] = turn.c[2 * j + 1] = a.x;
            turn.s[2 * j] = -dir * a.y;
            turn.s[2 * j + 1] = dir * a.y;
        }
    } else {
        const bool second = l * V >= half;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 a = tab[l * V + j - (second ? half : 0)];
            turn.c[j] = a.x;
            turn.s[j] = (second ? dir : -dir) * a.y;
        }
    }
}

template <int D> __device__ __forceinline__ void init_turn(const HeadIn &in, Turn &turn)
{
    const int lane = threadIdx.x & 31, l = lane % (D / V), half = in.rot / 2;
    turn.on = l * V < in.rot;
    turn.partner = in.adjacent ? -1 : !turn.on ? lane : l * V < half ? lane + half / V : lane - half / V;
}

// Channels that are not rotated keep their values, whatever the others are.
__device__ __forceinline__ void rotate(const Turn &t, float (&x)[V])
{
    if (t.partner < 0) {
        if (t.on) {
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                const float a = x[j], b = x[j + 1];
                x[j] = fmaf(b, t.s[j], a * t.c[j]);
                x[j + 1] = fmaf(a, t.s[j + 1], b * t.c[j + 1]);
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float o = __shfl_sync(0xffffffffu, x[j], t.partner);
        if (t.on) x[j] = fmaf(o, t.s[j], x[j] * t.c[j]);
    }
}

// The same of values as they came: the others' come in their own type, half as many shuffles for 16 bits.
template <typename E> __device__ __forceinline__ void rotate(const Turn &t, const Raw<E> &r, float (&x)[V])
{
    widen<E>(r, x);
    if (t.partner < 0) {
        rotate(t, x);
        return;
    }
    Raw<E> other;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(E) / 2); ++i) {
        other.v[i].x = __shfl_sync(0xffffffffu, r.v[i].x, t.partner);
        other.v[i].y = __shfl_sync(0xffffffffu, r.v[i].y, t.partner);
        other.v[i].z = __shfl_sync(0xffffffffu, r.v[i].z, t.partner);
        other.v[i].w = __shfl_sync(0xffffffffu, r.v[i].w, t.partner);
    }
    float o[V];
    widen<E>(other, o);
    if (t.on) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const float2 y = fma2(make_float2(o[j], o[j + 1]), make_float2(t.s[j], t.s[j + 1]),
                                  mul2(make_float2(x[j], x[j + 1]), make_float2(t.c[j], t.c[j + 1])));
            x[j] = y.x, x[j + 1] = y.y;
        }
    }
}

template <int D> __device__ __forceinline__ float head_sum(float v)
{
#pragma unroll
    for (int m = D / V / 2; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

template <int D> __device__ __forceinline__ void weights(const float *w, float (&x)[V])
{
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = w ? w[(threadIdx.x & 31) % (D / V) * V + j] : 1.f;
}

// The steps [lo, hi) of n heads of one token in x.
template <typename E, int D, bool ALIGNED>
__device__ __forceinline__ void forward_heads(const HeadIn &in, const E *x, E *out, int n, int lo, int hi, const float (&w)[V],
                                              const Turn &turn)
{
    constexpr int LANES = D / V, HEADS = 32 / LANES, U = 4;        // steps whose rows are fetched together
    const int lane = threadIdx.x & 31, at = (lane % LANES) * V;
    for (int i = lo; i < hi; i += U) {
        Raw<E> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = (i + u) * HEADS + lane / LANES;
            if (i + u < hi && h < n) load<E, ALIGNED>(r[u], x + h * D + at);
            else r[u] = {};
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // (a step behind the last one is worked on zeros: without a branch the compiler interleaves the batch's steps)
            const int h = (i + u) * HEADS + lane / LANES;
            float v[V];
            widen<E>(r[u], v);
            if (in.norm) {
                float2 ss = mul2(make_float2(v[0], v[1]), make_float2(v[0], v[1]));
#pragma unroll
                for (int j = 2; j < V; j += 2) ss = fma2(make_float2(v[j], v[j + 1]), make_float2(v[j], v[j + 1]), ss);
                const float inv = rsqrtf(fmaf(head_sum<D>(ss.x + ss.y), 1.f / D, in.eps));
#pragma unroll
                for (int j = 0; j < V; j += 2) {
                    const float2 y = mul2(mul2(make_float2(v[j], v[j + 1]), make_float2(inv, inv)), make_float2(w[j], w[j + 1]));
                    v[j] = y.x, v[j + 1] = y.y;
                }
            }
            if (in.rot) rotate(turn, v);
            if (i + u < hi && h < n) store<E, ALIGNED>(out + h * D + at, v);
        }
    }
}

template <typename E, int D, bool ALIGNED>
__global__ void __launch_bounds__(THREADS, 3) head_forward(const Work p, const HeadOut out)
{
    constexpr int HEADS = 32 / (D / V);
    __shared__ float2 s_tab[WARPS][D / 2];
    const HeadIn &in = p.in;
    const int warp = threadIdx.x >> 5, q_steps = (in.H + HEADS - 1) / HEADS;
    float w_q[V], w_k[V];
    weights<D>(in.w_q, w_q);
    weights<D>(in.w_k, w_k);
    Turn turn;
    init_turn<D>(in, turn);
    for (int64_t task = static_cast<int64_t>(blockIdx.x) * WARPS + warp; task < p.tasks; task += static_cast<int64_t>(gridDim.x) * WARPS) {
        const int64_t t = p.parts == 1 ? task : task / p.parts;
        const int lo = static_cast<int>(task - t * p.parts) * p.per_part, hi = min(lo + p.per_part, p.steps);
        make_turn<D>(in, t, 1.f, s_tab[warp], turn);
        forward_heads<E, D, ALIGNED>(in, static_cast<const E *>(in.q) + t * in.ldq, static_cast<E *>(out.q) + t * out.ldq, in.H,
                                     min(lo, q_steps), min(hi, q_steps), w_q, turn);
        forward_heads<E, D, ALIGNED>(in, static_cast<const E *>(in.k) + t * in.ldk, static_cast<E *>(out.k) + t * out.ldk, in.Hk,
                                     max(lo - q_steps, 0), max(hi - q_steps, 0), w_k, turn);
    }
}

// The gradients of the steps [lo, hi): dx from the gradient g of the output, and the sums of the weights' gradients.
template <typename E, int D, bool ALIGNED>
__device__ __forceinline__ void backward_heads(const HeadIn &in, const E *x, const E *g, E *dx, int n, int lo, int hi, const float (&w)[V],
                                               float (&dw)[V], const Turn &turn)
{
    constexpr int LANES = D / V, HEADS = 32 / LANES, U = 2;        // (4: 72 us for 60 at 8192 x 32 heads)
    const int lane = threadIdx.x & 31, at = (lane % LANES) * V;
    for (int i = lo; i < hi; i += U) {
        Raw<E> rx[U], rg[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = (i + u) * HEADS + lane / LANES;
            rx[u] = {};
            rg[u] = {};
            if (i + u < hi && h < n) {
                if (in.norm) load<E, ALIGNED>(rx[u], x + h * D + at);
                load<E, ALIGNED>(rg[u], g + h * D + at);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // (a step behind the last one is worked on zeros, as in the forward; the weights get nothing from it)
            const int h = (i + u) * HEADS + lane / LANES;
            const bool real = i + u < hi && h < n;
            float e[V];
            if (in.rot) rotate<E>(turn, rg[u], e);
            else widen<E>(rg[u], e);
            if (in.norm) {
                float v[V];
                widen<E>(rx[u], v);
                float2 ew[V / 2], ss = make_float2(0.f, 0.f), dot = ss;
#pragma unroll
                for (int j = 0; j < V; j += 2) {
                    const float2 x2 = make_float2(v[j], v[j + 1]);
                    ew[j / 2] = mul2(make_float2(e[j], e[j + 1]), make_float2(w[j], w[j + 1]));
                    ss = fma2(x2, x2, ss);
                    dot = fma2(ew[j / 2], x2, dot);
                }
                const float square = head_sum<D>(ss.x + ss.y);        // (by all lanes)
                const float inv = real ? rsqrtf(fmaf(square, 1.f / D, in.eps)) : 0.f;
                const float mean = head_sum<D>(dot.x + dot.y) * inv * (1.f / D);        // of e w x / rms
                const float2 inv2 = make_float2(inv, inv), less = make_float2(-mean, -mean);
#pragma unroll
                for (int j = 0; j < V; j += 2) {
                    const float2 hat = mul2(make_float2(v[j], v[j + 1]), inv2);
                    const float2 s = fma2(make_float2(e[j], e[j + 1]), hat, make_float2(dw[j], dw[j + 1]));
                    dw[j] = s.x, dw[j + 1] = s.y;
                    const float2 d = mul2(inv2, fma2(hat, less, ew[j / 2]));
                    e[j] = d.x, e[j + 1] = d.y;
                }
            }
            if (real) store<E, ALIGNED>(dx + h * D + at, e);
        }
    }
}

template <typename E, int D, bool ALIGNED>
__global__ void __launch_bounds__(THREADS, 2) head_backward(const Work p, const HeadOut g, const HeadOut dx, float *part)
{
    constexpr int LANES = D / V, HEADS = 32 / LANES;
    __shared__ float2 s_tab[WARPS][D / 2];
    __shared__ float s_sum[WARPS][2 * D];
    const HeadIn &in = p.in;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q_steps = (in.H + HEADS - 1) / HEADS;
    float w_q[V], w_k[V], dw_q[V] = {}, dw_k[V] = {};
    weights<D>(in.w_q, w_q);
    weights<D>(in.w_k, w_k);
    Turn turn;
    init_turn<D>(in, turn);
    for (int64_t task = static_cast<int64_t>(blockIdx.x) * WARPS + warp; task < p.tasks; task += static_cast<int64_t>(gridDim.x) * WARPS) {
        const int64_t t = p.parts == 1 ? task : task / p.parts;
        const int lo = static_cast<int>(task - t * p.parts) * p.per_part, hi = min(lo + p.per_part, p.steps);
        make_turn<D>(in, t, -1.f, s_tab[warp], turn);
        backward_heads<E, D, ALIGNED>(in, static_cast<const E *>(in.q) + t * in.ldq, static_cast<const E *>(g.q) + t * g.ldq,
                                      static_cast<E *>(dx.q) + t * dx.ldq, in.H, min(lo, q_steps), min(hi, q_steps), w_q, dw_q, turn);
        backward_heads<E, D, ALIGNED>(in, static_cast<const E *>(in.k) + t * in.ldk, static_cast<const E *>(g.k) + t * g.ldk,
                                      static_cast<E *>(dx.k) + t * dx.ldk, in.Hk, max(lo - q_steps, 0), max(hi - q_steps, 0), w_k, dw_k, turn);
    }
    tc::grid_dep_launch();
    if (!part) return;
    // the lanes of the same channels, then the warps in order
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int m = LANES; m < 32; m *= 2) {
            dw_q[j] += __shfl_xor_sync(0xffffffffu, dw_q[j], m);
            dw_k[j] += __shfl_xor_sync(0xffffffffu, dw_k[j], m);
        }
        if (lane < LANES) {
            s_sum[warp][lane * V + j] = dw_q[j];
            s_sum[warp][D + lane * V + j] = dw_k[j];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * D; c += THREADS) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) sum += s_sum[i][c];
        part[static_cast<size_t>(blockIdx.x) * 2 * D + c] = sum;
    }
}

constexpr int RT = 1024, STRANDS = RT / 32;   // threads: 32 columns x 32 strands of CTAs

// Column c of [dw_q | dw_k]: the CTAs' sums, strand by strand, the strands added up in a fixed order.
__global__ void __launch_bounds__(RT) head_reduce(int ctas, int D, const float *part, float *dw_q, float *dw_k)
{
    __shared__ float s[STRANDS][33];
    tc::grid_dep_wait();
    const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5;
    int c = blockIdx.x * 32 + lane;
    float v[MAX_GRID / STRANDS], sum = 0.f;
#pragma unroll
    for (int k = 0; k < MAX_GRID / STRANDS; ++k) {
        const int b = strand + k * STRANDS;
        v[k] = b < ctas ? part[static_cast<size_t>(b) * 2 * D + c] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < MAX_GRID / STRANDS; ++k) sum += v[k];
    s[strand][lane] = sum;
    __syncthreads();
    sum = s[lane][strand];        // a warp a column now
#pragma unroll
    for (int m = 16; m; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    c = blockIdx.x * 32 + strand;
    if (lane) return;
    if (c < D) {
        if (dw_q) dw_q[c] = sum;
    } else if (dw_k) {
        dw_k[c - D] = sum;
    }
}

bool on16(const void *p, int64_t ld, int64_t T, int e)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (T < 2 || (ld * e & 15) == 0);
}

// How many warps share a token: one, unless that leaves the device's 'warps' fewer than six tokens each, the last of which
// would leave many of them idle.  A part is four steps at least where there are enough tokens for all warps: each part makes its angles anew
// (gradients of 8192 x 32 heads: two parts 58 us, three, which is what eight tokens each would ask for, 61 us).
Work make_work(const HeadIn &in, int heads, int64_t warps)
{
    Work p{in, in.T, 1, 0, 0};
    p.steps = (in.H + heads - 1) / heads + (in.Hk + heads - 1) / heads;
    if (in.T < 6 * warps)
        p.parts = static_cast<int>(min(static_cast<int64_t>(in.T < warps ? p.steps : (p.steps + 3) / 4), (6 * warps + in.T - 1) / in.T));
    p.per_part = (p.steps + p.parts - 1) / p.parts;
    p.parts = (p.steps + p.per_part - 1) / p.per_part;
    p.tasks = in.T * p.parts;
    return p;
}

template <typename E, int D, bool ALIGNED>
cudaError_t forward(const HeadIn &in, const HeadOut &out, cudaStream_t stream)
{
    const int64_t most = static_cast<int64_t>(sm_count()) * 3;
    const Work p = make_work(in, 32 / (D / V), most * WARPS);
    const int64_t ctas = (p.tasks + WARPS - 1) / WARPS;
    head_forward<E, D, ALIGNED><<<static_cast<int>(min(most, ctas)), THREADS, 0, stream>>>(p, out);
    return cudaGetLastError();
}

template <typename E, int D, bool ALIGNED>
cudaError_t backward(const HeadIn &in, const HeadOut &g, const HeadOut &dx, float *dw_q, float *dw_k, float *part, cudaStream_t stream)
{
    int grid = 0;
    if (!dw_q && !dw_k) part = nullptr;
    if (in.T > 0) {
        const int64_t most = min(sm_count() * 2, MAX_GRID);
        const Work p = make_work(in, 32 / (D / V), most * WARPS);
        const int64_t ctas = (p.tasks + WARPS - 1) / WARPS;
        grid = static_cast<int>(min(most, ctas));
        head_backward<E, D, ALIGNED><<<grid, THREADS, 0, stream>>>(p, g, dx, part);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (!part) return cudaSuccess;
    return launch_dependent(head_reduce, dim3(2 * D / 32), dim3(RT), 0, stream, grid, D, static_cast<const float *>(part), dw_q, dw_k);
}

// Calls f<E, D, ALIGNED>.
#define PICK_D(f, E, AL, ...)                               \
    switch (in.d) {                                         \
    case 32: return f<E, 32, AL>(__VA_ARGS__);              \
    case 64: return f<E, 64, AL>(__VA_ARGS__);              \
    case 128: return f<E, 128, AL>(__VA_ARGS__);            \
    default: return f<E, 256, AL>(__VA_ARGS__);             \
    }
#define PICK(f, aligned, type, ...)                                         \
    if (type == KDA_TYPE_F32) {                                             \
        if (aligned) { PICK_D(f, float, true, __VA_ARGS__) }                \
        PICK_D(f, float, false, __VA_ARGS__)                                \
    } else if (type == KDA_TYPE_F16) {                                      \
        if (aligned) { PICK_D(f, __half, true, __VA_ARGS__) }               \
        PICK_D(f, __half, false, __VA_ARGS__)                               \
    } else {                                                                \
        if (aligned) { PICK_D(f, __nv_bfloat16, true, __VA_ARGS__) }        \
        PICK_D(f, __nv_bfloat16, false, __VA_ARGS__)                        \
    }

}  // namespace

size_t head_workspace_bytes(int d) { return static_cast<size_t>(MAX_GRID) * 2 * d * 4; }

cudaError_t launch_head_forward(const HeadIn &in, int type, const HeadOut &out, cudaStream_t stream)
{
    const int e = elem_bytes(type);
    const bool al = on16(in.q, in.ldq, in.T, e) && on16(in.k, in.ldk, in.T, e) && on16(out.q, out.ldq, in.T, e) && on16(out.k, out.ldk, in.T, e);
    PICK(forward, al, type, in, out, stream)
}

cudaError_t launch_head_backward(const HeadIn &in, int type, const HeadOut &g, const HeadOut &dx, float *dw_q, float *dw_k, void *ws,
                                 cudaStream_t stream)
{
    const int e = elem_bytes(type);
    const bool al = on16(in.q, in.ldq, in.T, e) && on16(in.k, in.ldk, in.T, e) && on16(g.q, g.ldq, in.T, e) && on16(g.k, g.ldk, in.T, e) &&
                    on16(dx.q, dx.ldq, in.T, e) && on16(dx.k, dx.ldk, in.T, e);
    PICK(backward, al, type, in, g, dx, dw_q, dw_k, static_cast<float *>(ws), stream)
}

}  // namespace kda
