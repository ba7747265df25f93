// Gated linear recurrence: gradients (gated_scan.cuh).
#include "gated_scan.cuh"

namespace kda {
namespace {

// ---- backward -------------------------------------------------------------------------------------------

template <typename E, bool SH, int G> struct __align__(16) BackwardShared {
    Rows<float, SH> g;
    Rows<E, SH> x, i, dh;
    float2 fmap[RUNS][C];          // the runs' maps of the states, forwards
    float fstate[RUNS][C];         // the state that enters each run
    Shared<G> s;
};

template <typename E, bool SH, bool ADJ, bool CHAIN, int G>
__global__ void __launch_bounds__(THREADS, ctas_of<BackwardShared<E, SH, G>>()) scan_backward(const int32_t *plan, PlanSig sig, int D, ScanIn in, Chain ch,
                                                                                    const float *states, const void *dh_, int64_t lddh,
                                                                                    const float *dfinal, ScanGrads out)
{
    extern __shared__ __align__(16) unsigned char smem_raw[];
    auto &sm = *reinterpret_cast<BackwardShared<E, SH, G> *>(smem_raw);
    if (!plan_matches(plan, sig)) {
        if (threadIdx.x == 0) record_status(&g_scan_status, KDA_ERR_INVALID_ARG);
        return;
    }
    const PlanView pv{plan};
    const int T = pv.T(), run = threadIdx.x / 16, l = threadIdx.x % 16, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const E *x = static_cast<const E *>(in.x), *ig = static_cast<const E *>(in.i), *dh = static_cast<const E *>(dh_);
    E *dx = static_cast<E *>(out.dx), *di = static_cast<E *>(out.di);
    const bool pair = !ADJ || (pairs(dx, out.lddx) && (!di || pairs(di, out.lddi)) && pairs(out.dg, out.lddg));

    // part 0: the decays, which a tile takes to registers; part 1: what it reads again for the gradients
    auto load = [&](const Tile &t, int part) {
        if (part == 0) {
            fill(sm.g, in.g, in.ldg, t.t0, T, t.col0, D);
            return;
        }
        fill(sm.x, x, in.ldx, t.t0, T, t.col0, D);
        if (ig) fill(sm.i, ig, in.ldi, t.t0, T, t.col0, D);
        fill(sm.dh, dh, lddh, t.t0, T, t.col0, D);
    };
    auto work = [&](const Tile &t, const Bounds &b, auto release) {
        const int left = D - t.col0, rows = T - t.t0 - run * RUN, place = b.place();
        const uint32_t ends = b.mask >> 1;
        const int kind = kind_of(b, rows >= RUN && left >= C && pair);
        float h0[V] = {}, df[V] = {};
        if (kind != ANY) {
            seq_row<ADJ>(in.h0, b.first, D, t.col0, l, b.starts != 0, h0);
            seq_row<ADJ>(dfinal, b.first - 1, D, t.col0, l, ends != 0, df);
        }
        // the state before the tile, for the warp that folds the states' maps
        float f0 = 0.f;
        if (warp == WARPS - 1 && lane < left) f0 = states[static_cast<int64_t>(t.tt) * D + t.col0 + lane];
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
        const Run<E, SH> hr(sm.dh, run, dh, lddh, t.t0);
        float P[V] = {1.f, 1.f}, F[V] = {0.f, 0.f}, B[V] = {0.f, 0.f};   // (P, F): of the states; (P, B): of the gradients
        by_inner_kind(kind, [&](auto k) {
            constexpr int K = decltype(k)::value;
#pragma unroll
            for (int j = RUN - 1; j >= 0; --j) {
                float d[V];
                get<ADJ>(hr(j), l, d);
                if constexpr (K == ANY)
                    if (ends >> j & 1) seq_row<ADJ>(dfinal, b.seq(j + 1) - 1, D, t.col0, l, true, B);
                if constexpr (K == ONE)
#pragma unroll
                    for (int v = 0; v < V; ++v) B[v] = j + 1 == place ? df[v] : B[v];
                set(B, mul2(both(a[j]), add2(both(d), both(B))));
            }
#pragma unroll
            for (int j = 0; j < RUN; ++j) {
                if constexpr (K == ANY)
                    if (b.starts >> j & 1) seq_row<ADJ>(in.h0, b.seq(j), D, t.col0, l, true, F);
                if constexpr (K == ONE)
#pragma unroll
                    for (int v = 0; v < V; ++v) F[v] = j == place ? h0[v] : F[v];
                set(P, mul2(both(P), both(a[j])));
                set(F, fma2(both(a[j]), both(F), both(u[j])));
            }
        });
        if (__any_sync(0xffffffffu, !(P[0] <= MOST_RUN) || !(P[1] <= MOST_RUN))) {
            sm.s.far = t.rt;
            double p[V];
            int k[V];
            far_products<ADJ>(gr, l, RUN, p, k);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (!(P[v] <= MOST)) P[v] = product_of(p[v]);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sm.s.map[run][chan<ADJ>(l, v)] = make_float2(ends ? FORGET : P[v], B[v]);
            sm.fmap[run][chan<ADJ>(l, v)] = make_float2(b.starts ? FORGET : P[v], F[v]);
        }
        __syncthreads();
        // While the tile's map travels: the states before each token, in place of the tokens' own terms.
        auto meanwhile = [&] {
            release();
            if (warp == WARPS - 1) {
                auto fold = [&](int r, auto f) {
                    const float2 m = sm.fmap[r][lane];
                    sm.fstate[r][lane] = f0;
                    f0 = f(m, f0);
                };
                if (sm.s.far == t.rt) {
#pragma unroll 1
                    for (int r = 0; r < RUNS; ++r) fold(r, any_apply);
                } else {
#pragma unroll
                    for (int r = 0; r < RUNS; ++r) fold(r, apply);
                }
            }
            __syncthreads();
            float f[V];
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] = sm.fstate[run][chan<ADJ>(l, v)];
            by_inner_kind(kind, [&](auto k) {
                constexpr int K = decltype(k)::value;
#pragma unroll
                for (int j = 0; j < RUN; ++j) {
                    if constexpr (K == ANY)
                        if (b.starts >> j & 1) seq_row<ADJ>(in.h0, b.seq(j), D, t.col0, l, true, f);
                    if constexpr (K == ONE)
#pragma unroll
                        for (int v = 0; v < V; ++v) f[v] = j == place ? h0[v] : f[v];
                    const float2 next = fma2(both(a[j]), both(f), both(u[j]));
                    set(u[j], both(f));
                    set(f, next);
                }
            });
        };
        if (!incoming<CHAIN, true>(sm.s, ch, t.rt, t.col0, t.tt == 0, meanwhile)) return false;
        float e[V];
#pragma unroll
        for (int v = 0; v < V; ++v) e[v] = sm.s.state[run][chan<ADJ>(l, v)];
        const int64_t last = static_cast<int64_t>(t.t0) + run * RUN + RUN - 1;
        const int c0 = t.col0 + chan<ADJ>(l, 0);
        E *px = dx + last * out.lddx + c0, *pi = di ? di + last * out.lddi + c0 : nullptr;
        float *pg = out.dg + last * out.lddg + c0;
        by_kind(kind, [&](auto k) {
            constexpr int K = decltype(k)::value;
            float *first = nullptr;
            if constexpr (K == ONE || K == EDGE)
                if (out.dh0 && b.starts) first = out.dh0 + static_cast<int64_t>(b.first) * D + t.col0;
#pragma unroll
            for (int j = RUN - 1; j >= 0; --j) {
                float Gr[V], gx[V], gi[V], gg[V];
                get<ADJ>(hr(j), l, Gr);
                get<ADJ>(xr(j), l, gi);
                if constexpr (K == ANY)
                    if (ends >> j & 1) seq_row<ADJ>(dfinal, b.seq(j + 1) - 1, D, t.col0, l, true, e);
                if constexpr (K == ONE || K == EDGE)
#pragma unroll
                    for (int v = 0; v < V; ++v) e[v] = j + 1 == place ? df[v] : e[v];
                set(Gr, add2(both(Gr), both(e)));
                set(e, mul2(both(a[j]), both(Gr)));
                set(gi, mul2(both(gi), both(Gr)));
                set(gg, mul2(both(u[j]), both(e)));
                set(gx, both(Gr));
                if (ig) {
                    get<ADJ>(ir(j), l, gx);
                    set(gx, mul2(both(gx), both(Gr)));
                }
                if constexpr (K == ANY || K == EDGE) {
                    if (j < rows) {
                        put<ADJ>(px - chan<ADJ>(l, 0), l, gx, left);
                        if (di) put<ADJ>(pi - chan<ADJ>(l, 0), l, gi, left);
                        put<ADJ>(pg - chan<ADJ>(l, 0), l, gg, left);
                    }
                    if constexpr (K == EDGE) {
                        if (first && j == place) put<ADJ>(first, l, e, left);
                    } else if ((b.starts >> j & 1) && out.dh0) put<ADJ>(out.dh0 + b.seq(j) * D + t.col0, l, e, left);
                } else {
                    put_all<ADJ>(px, gx);
                    if (di) put_all<ADJ>(pi, gi);
                    put_all<ADJ>(pg, gg);
                    if constexpr (K == ONE)
                        if (first && j == place) {
                            first[chan<ADJ>(l, 0)] = e[0];
                            first[chan<ADJ>(l, 1)] = e[1];
                        }
                }
                px -= out.lddx;
                pi -= out.lddi;
                pg -= out.lddg;
            }
        });
        __syncthreads();
        return true;
    };
    walk<CHAIN, true>(sm.s, ch, pv, D, load, work);
}

}  // namespace

cudaError_t launch_scan_backward(const int32_t *plan_host, const int32_t *plan_dev, int D, int type, const ScanIn &in,
                                 const float *states, const void *dh, int64_t lddh, const float *dfinal,
                                 const ScanGrads &out, void *ws, cudaStream_t stream)
{
    return by_type(type, [&](auto ev) {
        using E = decltype(ev);
        const Lie lie = Lie().with(in.x, in.ldx, sizeof(E)).with(in.i, in.ldi, sizeof(E)).with(in.g, in.ldg, 4).with(dh, lddh, sizeof(E));
        return by_lie(lie, [&](auto shift, auto adj) {
            constexpr bool SH = decltype(shift)::value, ADJ = decltype(adj)::value;
            auto form = [](auto chain, auto group) {
                constexpr bool CHAIN = decltype(chain)::value;
                constexpr int G = decltype(group)::value;
                using Sh = BackwardShared<E, SH, G>;
                using K = decltype(&scan_backward<E, SH, ADJ, CHAIN, G>);
                return Form<K>{scan_backward<E, SH, ADJ, CHAIN, G>, static_cast<int>(sizeof(Sh)), ctas_of<Sh>()};
            };
            using Wide = std::integral_constant<int, WIDE_GROUP>;
            using Narrow = std::integral_constant<int, NARROW_GROUP>;
            return run(form(std::false_type{}, Wide{}), form(std::true_type{}, Wide{}), form(std::true_type{}, Narrow{}), plan_host, plan_dev, D, ws,
                       stream, in, states, dh, lddh, dfinal, out);
        });
    });
}

int take_scan_backward_status()
{
    int v = KDA_OK, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_scan_status, sizeof v) != cudaSuccess) return KDA_ERR_CUDA;
    if (v != KDA_OK && cudaMemcpyToSymbol(g_scan_status, &z, sizeof z) != cudaSuccess) return KDA_ERR_CUDA;
    return v;
}

}  // namespace kda
