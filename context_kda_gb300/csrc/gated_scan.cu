// Gated linear recurrence: forward and single-token step (gated_scan.cuh).
#include "gated_scan.cuh"

namespace kda {
namespace {

// ---- forward --------------------------------------------------------------------------------------------

template <typename E, bool SH, int G> struct __align__(16) ForwardShared {
    Rows<float, SH> g;
    Rows<E, SH> x, i;
    Shared<G> s;
};

template <typename E, bool SH, bool ADJ, bool CHAIN, int G>
__global__ void __launch_bounds__(THREADS, ctas_of<ForwardShared<E, SH, G>>()) scan_forward(const int32_t *plan, PlanSig sig, int D, ScanIn in, Chain ch, void *h_,
                                                              int64_t ldh, float *final_state, float *states)
{
    extern __shared__ __align__(16) unsigned char smem_raw[];
    auto &sm = *reinterpret_cast<ForwardShared<E, SH, G> *>(smem_raw);
    if (!plan_matches(plan, sig)) {
        if (threadIdx.x == 0) record_status(&g_scan_status, KDA_ERR_INVALID_ARG);
        return;
    }
    const PlanView pv{plan};
    const int T = pv.T(), nT = tiles_of(T), run = threadIdx.x / 16, l = threadIdx.x % 16;
    const E *x = static_cast<const E *>(in.x), *ig = static_cast<const E *>(in.i);
    E *h_out = static_cast<E *>(h_);
    const bool pair = !ADJ || pairs(h_out, ldh);

    auto load = [&](const Tile &t, int part) {
        if (part == 1) return;
        fill(sm.g, in.g, in.ldg, t.t0, T, t.col0, D);
        fill(sm.x, x, in.ldx, t.t0, T, t.col0, D);
        if (ig) fill(sm.i, ig, in.ldi, t.t0, T, t.col0, D);
    };
    auto work = [&](const Tile &t, const Bounds &b, auto release) {
        const int left = D - t.col0, rows = T - t.t0 - run * RUN, place = b.place();
        const int kind = kind_of(b, rows >= RUN && left >= C && pair);
        float h0[V] = {};
        if (kind != ANY) seq_row<ADJ>(in.h0, b.first, D, t.col0, l, b.starts != 0, h0);
        const Run<float, SH> gr(sm.g, run, in.g, in.ldg, t.t0);
        const Run<E, SH> xr(sm.x, run, x, in.ldx, t.t0), ir(sm.i, run, ig, in.ldi, t.t0);
        float a[RUN][V], u[RUN][V];
        gr.each([&](int j, const float *row) {
            float gv[V];
            get<ADJ>(row, l, gv);
            set(a[j], decay2(both(gv)));
        });
        xr.each([&](int j, const E *row) { get<ADJ>(row, l, u[j]); });
        if (ig)
            ir.each([&](int j, const E *row) {
                float iv[V];
                get<ADJ>(row, l, iv);
                set(u[j], mul2(both(u[j]), both(iv)));
            });
        // a becomes the product of the decays up to the token (of no use from the first boundary on), u the state from zero, or
        // from its sequence's start
        by_inner_kind(kind, [&](auto k) {
            constexpr int K = decltype(k)::value;
            float A[V] = {1.f, 1.f}, B[V] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < RUN; ++j) {
                if constexpr (K == ANY)
                    if (b.starts >> j & 1) seq_row<ADJ>(in.h0, b.seq(j), D, t.col0, l, true, B);
                if constexpr (K == ONE)
#pragma unroll
                    for (int v = 0; v < V; ++v) B[v] = j == place ? h0[v] : B[v];
                const float2 b2 = fma2(both(a[j]), both(B), both(u[j])), a2 = mul2(both(A), both(a[j]));
                set(B, b2);
                set(u[j], b2);
                set(A, a2);
                set(a[j], both(A));
            }
        });
#pragma unroll
        for (int v = 0; v < V; ++v) sm.s.map[run][chan<ADJ>(l, v)] = make_float2(b.starts ? FORGET : a[RUN - 1][v], u[RUN - 1][v]);
        // A product that leaves fp32's range is infinite, or NaN, from there on.  If that is before the run's first boundary, the
        // products are made again from 2^-k instead of one, and the state that enters is multiplied by 2^k: both are exact, and
        // what the one loses among the small products the other would lose in the state.
        int far[V] = {};           // k
        if (__any_sync(0xffffffffu, !(a[RUN - 1][0] <= MOST_RUN) || !(a[RUN - 1][1] <= MOST_RUN))) {
            sm.s.far = t.rt;
            double p[V];
            far_products<ADJ>(gr, l, place < RUN ? place : RUN, p, far);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (far[v] && !b.starts) sm.s.map[run][chan<ADJ>(l, v)].x = product_of(p[v]);
            if (__any_sync(0xffffffffu, far[0] | far[1])) {
                float A[V] = {two_to(-far[0]), two_to(-far[1])};
                gr.each([&](int j, const float *row) {
                    float gv[V];
                    get<ADJ>(row, l, gv);
                    set(a[j], decay2(both(gv)));
                });
#pragma unroll
                for (int j = 0; j < RUN; ++j) {
                    set(A, mul2(both(A), both(a[j])));
#pragma unroll
                    for (int v = 0; v < V; ++v) a[j][v] = fminf(A[v], MOST);
                }
            }
        }
        __syncthreads();
        if (!incoming<CHAIN, false>(sm.s, ch, t.rt, t.col0, t.tt == nT - 1, release)) return false;
        float h[V], s[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = sm.s.state[run][chan<ADJ>(l, v)];
            if (far[v]) h[v] *= two_to(far[v]);
        }
        E *row = h_out + (static_cast<int64_t>(t.t0) + run * RUN) * ldh + t.col0;
        by_kind(kind, [&](auto k) {
            constexpr int K = decltype(k)::value;
            E *at = row + chan<ADJ>(l, 0);
            float *fin = nullptr;
            if constexpr (K == ONE || K == EDGE)
                if (final_state && place >= 1 && place <= RUN) fin = final_state + static_cast<int64_t>(b.first - 1) * D + t.col0;
#pragma unroll
            for (int j = 0; j < RUN; ++j) {
                set(s, fma2(both(a[j]), both(h), both(u[j])));
                if constexpr (K != PLAIN)
#pragma unroll
                    for (int v = 0; v < V; ++v) s[v] = j >= place ? u[j][v] : s[v];
                if constexpr (K == EDGE) {
                    if (j < rows) put<ADJ>(at - chan<ADJ>(l, 0), l, s, left);
                    if (fin && j + 1 == place) put<ADJ>(fin, l, s, left);
                } else if constexpr (K == ANY) {
                    if (j < rows) put<ADJ>(at - chan<ADJ>(l, 0), l, s, left);
                    if ((b.mask >> (j + 1) & 1) && final_state) put<ADJ>(final_state + (b.seq(j + 1) - 1) * D + t.col0, l, s, left);
                } else {
                    put_all<ADJ>(at, s);
                    if constexpr (K == ONE)
                        if (fin && j + 1 == place) {
                            fin[chan<ADJ>(l, 0)] = s[0];
                            fin[chan<ADJ>(l, 1)] = s[1];
                        }
                }
                at += ldh;
            }
        });
        if (states) {
            if (run == RUNS - 1 && t.tt + 1 < nT) put<ADJ>(states + (static_cast<int64_t>(t.tt) + 1) * D + t.col0, l, s, left);
            if (run == 0 && t.tt == 0) {
                const float zero[V] = {};
                put<ADJ>(states + t.col0, l, zero, left);
            }
        }
        return true;
    };
    walk<CHAIN, false>(sm.s, ch, pv, D, load, work);
}

// ---- one token --------------------------------------------------------------------------------------------

// One token per row, each the next one of its slot's state (updated in place).  Four channels a thread: adjacent ones
// where all rows start on four elements and D is a multiple of four (VEC), else STEP_THREADS apart, so that a warp's
// are adjacent.  Bound by memory, or by the launch (2048 x 4096 in bf16: 21 us, the rate of a copy; 27 us at 4095 channels;
// with one channel a thread, too few loads in flight, 84 us).
constexpr int STEP_THREADS = 128, STEP_N = 4;
__device__ __forceinline__ void get_four(const float *p, float (&v)[4])
{
    const float4 q = *reinterpret_cast<const float4 *>(p);
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
}
template <typename X> __device__ __forceinline__ void get_four(const X *p, float (&v)[4])
{
    const uint2 q = *reinterpret_cast<const uint2 *>(p);
    float w[2];
    unpack(q.x, w, p);
    v[0] = w[0], v[1] = w[1];
    unpack(q.y, w, p);
    v[2] = w[0], v[3] = w[1];
}
__device__ __forceinline__ void put_four(float *p, const float (&v)[4]) { *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]); }
template <typename X> __device__ __forceinline__ void put_four(X *p, const float (&v)[4])
{
    X e[4] = {from_f32<X>(v[0]), from_f32<X>(v[1]), from_f32<X>(v[2]), from_f32<X>(v[3])};
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(e);
}
template <bool VEC, typename X> __device__ __forceinline__ void get_row(const X *row, int d, int D, float (&v)[STEP_N])
{
    if constexpr (VEC) {
        get_four(row + d, v);
    } else {
#pragma unroll
        for (int k = 0; k < STEP_N; ++k) v[k] = d + k * STEP_THREADS < D ? to_f32(row[d + k * STEP_THREADS]) : 0.f;
    }
}
template <bool VEC, typename X> __device__ __forceinline__ void put_row(X *row, int d, int D, const float (&v)[STEP_N])
{
    if constexpr (VEC) {
        put_four(row + d, v);
    } else {
#pragma unroll
        for (int k = 0; k < STEP_N; ++k)
            if (d + k * STEP_THREADS < D) row[d + k * STEP_THREADS] = from_f32<X>(v[k]);
    }
}
template <typename E, bool VEC>
__global__ void __launch_bounds__(STEP_THREADS) scan_step(int B, int D, const int32_t *slots, int num_slots, ScanIn in,
                                                          float *state, void *h_, int64_t ldh)
{
    const int d = blockIdx.x * (STEP_THREADS * STEP_N) + threadIdx.x * (VEC ? STEP_N : 1);
    if (d >= D) return;
    for (int64_t b = blockIdx.y; b < B; b += gridDim.y) {
        // the row's inputs are requested along with its slot, not after it
        float g[STEP_N], u[STEP_N], i[STEP_N];
        get_row<VEC>(in.g + b * in.ldg, d, D, g);
        get_row<VEC>(static_cast<const E *>(in.x) + b * in.ldx, d, D, u);
        if (in.i) get_row<VEC>(static_cast<const E *>(in.i) + b * in.ldi, d, D, i);
        const int slot = slots ? slots[b] : static_cast<int>(b);
        const bool live = slot >= 0 && slot < num_slots;
        float s[STEP_N] = {};
        if (live) {
            float *at = state + static_cast<int64_t>(slot) * D;
            get_row<VEC>(at, d, D, s);
#pragma unroll
            for (int j = 0; j < STEP_N; ++j) s[j] = fmaf(decay(g[j]), s[j], in.i ? u[j] * i[j] : u[j]);
            put_row<VEC>(at, d, D, s);
        } else if (slot >= num_slots && d == 0) {
            record_status(&g_scan_status, KDA_ERR_INVALID_ARG);
        }
        put_row<VEC>(static_cast<E *>(h_) + b * ldh, d, D, s);
    }
}

}  // namespace

size_t scan_workspace_bytes(int64_t T, int D) { return T <= MAX_CLUSTER * L ? 0 : layout_of(T, D).end; }

cudaError_t launch_scan_forward(const int32_t *plan_host, const int32_t *plan_dev, int D, int type, const ScanIn &in,
                                void *h, int64_t ldh, float *final_state, float *states, void *ws, cudaStream_t stream)
{
    return by_type(type, [&](auto ev) {
        using E = decltype(ev);
        return by_lie(Lie().with(in.x, in.ldx, sizeof(E)).with(in.i, in.ldi, sizeof(E)).with(in.g, in.ldg, 4), [&](auto shift, auto adj) {
            constexpr bool SH = decltype(shift)::value, ADJ = decltype(adj)::value;
            auto form = [](auto chain, auto group) {
                constexpr bool CHAIN = decltype(chain)::value;
                constexpr int G = decltype(group)::value;
                using Sh = ForwardShared<E, SH, G>;
                using K = decltype(&scan_forward<E, SH, ADJ, CHAIN, G>);
                return Form<K>{scan_forward<E, SH, ADJ, CHAIN, G>, static_cast<int>(sizeof(Sh)), ctas_of<Sh>()};
            };
            using Wide = std::integral_constant<int, WIDE_GROUP>;
            using Narrow = std::integral_constant<int, NARROW_GROUP>;
            return run(form(std::false_type{}, Wide{}), form(std::true_type{}, Wide{}), form(std::true_type{}, Narrow{}), plan_host, plan_dev, D, ws,
                       stream, in, h, ldh, final_state, states);
        });
    });
}

cudaError_t launch_scan_step(int B, int D, int type, const int32_t *slots, int num_slots, const ScanIn &in,
                             float *state, void *h, int64_t ldh, cudaStream_t stream)
{
    return by_type(type, [&](auto ev) {
        using E = decltype(ev);
        auto on_four = [](const void *p, int64_t ld, uintptr_t bytes) {
            return !p || ((reinterpret_cast<uintptr_t>(p) & (4 * bytes - 1)) == 0 && (ld & 3) == 0);
        };
        const bool four = D % 4 == 0 && on_four(in.x, in.ldx, sizeof(E)) && on_four(in.i, in.ldi, sizeof(E)) && on_four(in.g, in.ldg, 4) &&
                          on_four(state, 0, 4) && on_four(h, ldh, sizeof(E));
        const dim3 grid((D + STEP_THREADS * STEP_N - 1) / (STEP_THREADS * STEP_N), B < 65535 ? B : 65535);
        if (four) scan_step<E, true><<<grid, STEP_THREADS, 0, stream>>>(B, D, slots, num_slots, in, state, h, ldh);
        else scan_step<E, false><<<grid, STEP_THREADS, 0, stream>>>(B, D, slots, num_slots, in, state, h, ldh);
        return cudaGetLastError();
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
