// Gradients of the window attention.  With p_ij = exp(scale q_i . k_j - lse_i), D_i = do_i . o_i:
//     dp_ij = do_i . v_j,   ds_ij = p_ij (dp_ij - D_i),
//     dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_{i, heads} ds_ij q_i,   dv_j = sum_{i, heads} p_ij do_i.
//
// Three kernels, and no atomics on sums, so that the same call gives the same bits: the rows' D; a kernel whose CTAs own 128
// queries and go over their keys (dq); and one whose CTAs own 128 keys and go over the queries that see them, of all heads of
// the group (dk, dv).  Scores and dp are computed in both: seven products for each pair of tiles where one kernel with a shared dq would take five.
// The last two are one kernel of two kinds.  Its own rows X1, X2 (keys and values, or queries and do) stay in shared
// memory; tiles of 64 of the other side, Y1, Y2, come by TMA four deep:
//     S = X1 Y1^T,  P' = X2 Y2^T           to TMEM, two buffers that alternate between two groups of four warps,
//     p, ds                                 a thread a row, back to TMEM in their places, as A operands of
//     A2 += ds Y1  (dk or dq),   A1 += p Y2  (dv).
//
// D_i from the output carries that output's rounding.  Where a row sees many keys the rest hides it, where it sees few it would be as large as
// the rounding of ds.  Queries whose tiles are DRY or fewer (the first rows of a sequence, narrow windows) go over them twice: sum_j ds_ij,
// which is zero with the right D, corrects D first, and the corrected D is left for the keys.
//
// Sinks are seen by every later query of their sequence.  Their tile's window part is worked as any other; the rest is cut into
// pieces of CHUNK queries, each a CTA's, which leave sums in fp32 in the workspace, and a last kernel adds those in order.
//
// fp16 has a narrow range: p is kept times 2^10, ds times a power of two for each key head, from the longest rows of do and v
// (|ds| <= 2 |do| |v|), so that it neither overflows nor fades.  bf16 needs neither.
#include "window_attention.cuh"

namespace kda {
namespace {

using namespace attn;

__device__ int g_window_back_status;

constexpr int THREADS = 384;
constexpr int SUB = 64;                   // rows of a tile of the other side
constexpr int STAGES = 4;
constexpr int DRY = 3;                    // tiles of the other side that queries go over twice
constexpr int CHUNK = 1024;               // queries of a piece of the sinks' work
constexpr uint32_t SBOX = SUB * 128;      // 64 rows of 64 columns

template <int D> struct Smem {
    static constexpr uint32_t X_BYTES = D / 64 * BOX, Y_BYTES = D / 64 * SBOX;
    static constexpr uint32_t X = 0, Y = 2 * X_BYTES, BYTES = Y + STAGES * 2 * Y_BYTES, ALLOC = BYTES + 1024;
    static_assert(ALLOC <= 227 * 1024, "shared memory");
};
// TMEM columns: two buffers of S and P', then the sums
constexpr uint32_t TM_ACC = 256, TM_COLS = 512;

struct Back {
    const float *lse;                     // [H][T]
    float *delta;                         // [H][T]
    float *most;                          // fp16: [2][Hk], the longest rows of do and of v
    float *first, *rest;                  // sinks: the window's part [N][Hk][2][S][d], the pieces' [slots][Hk][2][S][d]
    int window_blocks;                    // blocks of windows' tiles; the others are the sinks' pieces
};

// ds is kept times this in fp16: 2 |do| |v| becomes 2^14 to 2^15.
__device__ __forceinline__ float ds_factor(float most_do, float most_v)
{
    const float bound = 2.f * most_do * most_v;
    if (!(bound > 0.f) || !isfinite(bound)) return 1.f;
    int e;
    frexpf(bound, &e);                    // bound < 2^e
    return exp2f(static_cast<float>(min(max(15 - e, -100), 100)));
}

// KEYS: the CTA owns keys (dk, dv); else queries (dq).
template <typename E, int D, bool KEYS>
__global__ void __launch_bounds__(THREADS, 1)
    window_back(const __grid_constant__ CUtensorMap mx1, const __grid_constant__ CUtensorMap mx2, const __grid_constant__ CUtensorMap my1,
                const __grid_constant__ CUtensorMap my2, const Shape p, const Back k, E *out1, int64_t ld1, E *out2, int64_t ld2)
{
    using L = Smem<D>;
    constexpr bool F16 = !Pair<E>::BF16;
    constexpr float P_EXP = F16 ? 10.f : 0.f;            // p is kept times 2^P_EXP
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t s_x, s_full[STAGES], s_fix[STAGES], s_free[STAGES], s_s[2], s_p[2], s_end;
    __shared__ float4 s_row[2][2][SUB / 4][2];           // (KEYS) the queries' lse and D, by group and buffer
    __shared__ float s_dry[KEYS ? 1 : 2][KEYS ? 1 : TILE];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (!plan_matches(p.plan, p.sig)) {
        if (tid == 0 && blockIdx.x == 0) record_status(&g_window_back_status, KDA_ERR_INVALID_ARG);
        return;
    }
    // ---- the CTA's work
    const int g = p.H / p.Hk;
    Place at;
    bool sinks = false;                                  // a piece of the sinks' work
    int head, slot = 0;                                  // key head (KEYS) or query head
    if (KEYS && static_cast<int>(blockIdx.x) >= k.window_blocks) {
        const int i = blockIdx.x - k.window_blocks;
        sinks = true;
        head = i % p.Hk;
        slot = i / p.Hk;
        if (!find_tile(p, slot, CHUNK, at)) return;
    } else {
        const int works = KEYS ? p.Hk : p.H, i = (KEYS ? k.window_blocks : static_cast<int>(gridDim.x)) - 1 - blockIdx.x;
        head = i % works;
        if (!find_tile(p, i / works, TILE, at)) return;
    }
    const int W = min(p.W, at.len), x0 = sinks ? 0 : at.t0, rows = min(TILE, at.len - x0);      // own rows [x0, x0 + rows)
    const bool has_sinks = p.S > 0 && W < at.len;        // some query has left a sink behind its window
    // tiles of the other side: [lo, hi], then (queries) those of the sinks
    int lo, hi, extra = 0;
    if (KEYS) {
        lo = (sinks ? max(at.t0, W) : x0) / SUB;
        hi = (sinks ? min(at.t0 + CHUNK, at.len) - 1 : static_cast<int>(min(static_cast<int64_t>(x0) + TILE - 1 + W, static_cast<int64_t>(at.len)) - 1)) / SUB;
        if (sinks && (!has_sinks || lo > hi)) return;
    } else {
        lo = max(0, x0 - W + 1) / SUB;
        hi = (x0 + rows - 1) / SUB;
        if (has_sinks && x0 + rows - 1 >= W) extra = (p.S + SUB - 1) / SUB;
    }
    const int per_head = hi - lo + 1, tiles = KEYS ? g * per_head : per_head + extra;
    const int dry = !KEYS && tiles <= DRY ? tiles : 0, n = dry + tiles;      // steps, the first 'dry' of them for D alone
    const int xh = head, yh = KEYS ? head * g : head / g;                        // heads of the own rows and of the other side
    auto tile = [&](int i) {
        if (KEYS) return lo + i % per_head;
        if (i >= dry) i -= dry;
        return i < per_head ? hi - i : i - per_head;
    };
    auto y_head = [&](int i) { return KEYS ? yh + i / per_head : yh; };
    auto is_sink = [&](int i) { return KEYS ? sinks : (i >= dry ? i - dry : i) >= per_head; };
    // whether all own rows and all rows of tile i see each other
    auto whole = [&](int i) {
        const int y0 = tile(i) * SUB;
        if (is_sink(i)) return false;
        if (KEYS) return y0 >= x0 + TILE - 1 && y0 + SUB - 1 - x0 < W && y0 + SUB <= at.len;
        return y0 + SUB - 1 <= x0 && x0 + TILE - 1 - y0 < W;
    };
    // columns [a, b] of tile i that go with own row r
    auto visible = [&](int i, int r, int &a, int &b) {
        const int y0 = tile(i) * SUB, x = x0 + r;
        if (KEYS) {
            a = is_sink(i) ? (x < p.S ? x + W - y0 : SUB) : x - y0;
            b = min(SUB - 1, (is_sink(i) ? at.len - 1 : static_cast<int>(min(static_cast<int64_t>(x) + W, static_cast<int64_t>(at.len)) - 1)) - y0);
        } else {
            a = is_sink(i) ? 0 : x - W + 1 - y0;
            b = min(SUB - 1, (is_sink(i) ? min(p.S - 1, x - W) : x) - y0);
        }
        a = max(a, 0);
    };

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *const basep = smem_raw + (base - smem_u32(smem_raw));
    if (tid == 0) {
        mbar_init(smem_u32(&s_x), 1);
        for (int i = 0; i < STAGES; ++i) mbar_init(smem_u32(&s_full[i]), 1), mbar_init(smem_u32(&s_fix[i]), 2), mbar_init(smem_u32(&s_free[i]), 1);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&s_s[i]), 1), mbar_init(smem_u32(&s_p[i]), 4);
        mbar_init(smem_u32(&s_end), 1);
        s_abort = 0;
    }
    if (warp == 0) tmem_alloc(smem_u32(&s_tmem), TM_COLS);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem;
    volatile int *const abort_flag = &s_abort;
    auto give_up = [&] {
        record_status(&g_window_back_status, KDA_ERR_TIMEOUT);
        *abort_flag = 1;
    };
    auto y1 = [&](int i) { return base + L::Y + (i % STAGES) * 2 * L::Y_BYTES; };
    int fetched = 0;

    if (warp == 0) {
        // ---- fetch
        if (lane == 0) {
            const uint32_t bx = smem_u32(&s_x);
            mbar_arrive_expect_tx(bx, 2 * L::X_BYTES);
            for (int c = 0; c < D / 64; ++c) {
                tma_load_3d(base + L::X + c * BOX, &mx1, c * 64, xh, at.start + x0, bx);
                tma_load_3d(base + L::X + L::X_BYTES + c * BOX, &mx2, c * 64, xh, at.start + x0, bx);
            }
            bool ok = true;
            for (int i = 0; i < n; ++i) {
                const int s = i % STAGES;
                if (i >= STAGES) ok = wait_thread(smem_u32(&s_free[s]), (i / STAGES - 1) & 1);
                if (!ok) break;
                const uint32_t bar = smem_u32(&s_full[s]);
                mbar_arrive_expect_tx(bar, 2 * L::Y_BYTES);
                for (int c = 0; c < D / 64; ++c) {
                    tma_load_3d(y1(i) + c * SBOX, &my1, c * 64, y_head(i), at.start + tile(i) * SUB, bar);
                    tma_load_3d(y1(i) + L::Y_BYTES + c * SBOX, &my2, c * 64, y_head(i), at.start + tile(i) * SUB, bar);
                }
                ++fetched;
            }
            if (!ok) give_up();
        }
    } else if (warp == 1) {
        // ---- products.  TMEM addresses start at 0: the CTA has all of it
        constexpr uint32_t ID_S = idesc<E>(TILE, SUB, 0), ID_A = idesc<E>(TILE, D, 1);
        const uint32_t xd = desc_k(base + L::X);
        auto scores = [&](int buf, uint32_t y) {
            const uint32_t yd = desc_k(y);
            if (elect()) {
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                    for (int s = 0; s < D / 16; ++s)
                        product(buf * 128 + w * SUB, xd + ((w * L::X_BYTES + (s / 4) * BOX + (s % 4) * 32) >> 4),
                                yd + ((w * L::Y_BYTES + (s / 4) * SBOX + (s % 4) * 32) >> 4), ID_S, s > 0);
                commit(smem_u32(&s_s[buf]));
            }
            __syncwarp();
        };
        bool ok = wait_warp(smem_u32(&s_x), 0);
        int next = 0, next_parity = 0;              // stage and parity of the next tile to be multiplied
        auto step_next = [&] {
            if (++next == STAGES) next = 0, next_parity ^= 1;
        };
        for (int i = 0; i < 2 && i < n && ok; ++i) {
            ok = wait_warp(smem_u32(&s_fix[next]), next_parity);
            if (!ok) break;
            fence_after();
            scores(i, base + L::Y + next * 2 * L::Y_BYTES);
            step_next();
        }
        int stage = 0;
        for (int i = 0; i < n && ok; ++i) {
            ok = wait_warp(smem_u32(&s_p[i & 1]), (i >> 1) & 1);
            if (!ok) break;
            fence_after();
            const uint32_t d = (i & 1) * 128, y = base + L::Y + stage * 2 * L::Y_BYTES, y1d = desc_mn(y, SBOX), y2d = desc_mn(y + L::Y_BYTES, SBOX);
            if (elect()) {
                if (i >= dry)
#pragma unroll
                    for (int s = 0; s < SUB / 16; ++s) product_ta(TM_ACC, d + SUB + s * 8, y1d + s * (2048 >> 4), ID_A, i > dry || s > 0);
                if (KEYS)
#pragma unroll
                    for (int s = 0; s < SUB / 16; ++s) product_ta(TM_ACC + D, d + s * 8, y2d + s * (2048 >> 4), ID_A, i > 0 || s > 0);
                commit(smem_u32(&s_free[stage]));
            }
            __syncwarp();
            if (++stage == STAGES) stage = 0;
            if (i + 2 < n) {
                ok = wait_warp(smem_u32(&s_fix[next]), next_parity);
                if (!ok) break;
                fence_after();
                scores(i & 1, base + L::Y + next * 2 * L::Y_BYTES);
                step_next();
            }
        }
        if (!ok && lane == 0) give_up();
        if (elect()) commit(smem_u32(&s_end));
        __syncwarp();
        if (!ok) wait_warp(smem_u32(&s_end), 0);     // the products in flight end before the memory is given back
    } else if (warp < 4) {
        // ---- rows behind the sequence's end: zeros, so that a factor of zero meets no infinity or NaN there
        bool ok = true;
        for (int i = 0; i < n && ok; ++i) {
            ok = wait_warp(smem_u32(&s_full[i % STAGES]), (i / STAGES) & 1);
            if (!ok) break;
            const int real = at.len - tile(i) * SUB;
            if (real < SUB) {
                unsigned char *const y = basep + (y1(i) - base) + (warp - 2) * L::Y_BYTES;
                for (int r = real + lane / 8; r < SUB; r += 4)
                    for (int c = 0; c < D / 64; ++c) *reinterpret_cast<uint4 *>(y + c * SBOX + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s_fix[i % STAGES]));
        }
        if (!ok && lane == 0) give_up();
    } else {
        // ---- p and ds, a thread a row; the two groups take turns
        const int x = (warp >> 2) - 1, t = tid & 127, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + x * 128, tp = ts + SUB;
        const float factor = F16 ? ds_factor(k.most[KEYS ? head : yh], k.most[p.Hk + (KEYS ? head : yh)]) : 1.f;
        const float ds_mul = factor * (F16 ? 0x1p-10f : 1.f);
        const float2 cc = make_float2(p.c, p.c), ff = make_float2(ds_mul, ds_mul);
        // KEYS: thread t holds lse (t < 64) or D of query t % 64 of the group's next tile; else every thread those of its own row
        auto row_value = [&](int i) {
            const int y = tile(i) * SUB + (t & 63);
            const int64_t at_row = static_cast<int64_t>(y_head(i)) * p.T + at.start + y;
            if (y >= at.len) return 0.f;
            return t < 64 ? P_EXP - k.lse[at_row] * 1.44269504088896340736f : -k.delta[at_row];
        };
        float next = 0.f;
        float2 l2 = make_float2(0.f, 0.f), d2 = make_float2(0.f, 0.f);
        if (KEYS) {
            if (x < n) next = row_value(x);
        } else if (r < rows) {
            const int64_t at_row = static_cast<int64_t>(head) * p.T + at.start + x0 + r;
            l2.x = l2.y = P_EXP - k.lse[at_row] * 1.44269504088896340736f;
            d2.x = d2.y = -k.delta[at_row];
        }
        bool ok = true;
        float off = 0.f;                                // (dry steps) sum of ds
        bool corrected = false;
        auto correct = [&](bool ok) {                    // D by what both groups have found; everyone of them comes here once
            s_dry[x][r] = off * (F16 ? 0x1p-10f : 1.f);
            if (bar_or(3, 256, !ok)) return false;
            d2.x -= s_dry[0][r] + s_dry[1][r];
            d2.y = d2.x;
            if (x == 0 && r < rows) k.delta[static_cast<int64_t>(head) * p.T + at.start + x0 + r] = -d2.x;
            return true;
        };
        for (int i = x; i < n; i += 2) {
            if (!KEYS && i >= dry && dry > 0 && !corrected) {
                corrected = true;
                ok = correct(true);
                if (!ok) break;
            }
            const int turn = (i >> 1) & 1;
            if (KEYS) reinterpret_cast<float *>(s_row[x][turn])[(t & 63) / 4 * 8 + (t >> 6) * 4 + (t & 3)] = next;
            ok = wait_warp(smem_u32(&s_s[x]), turn);
            if (KEYS) ok = !bar_or(1 + x, 128, !ok);
            if (!ok) break;
            if (KEYS && i + 2 < n) next = row_value(i + 2);
            fence_after();
            int a = 0, b = SUB - 1;
            const bool all = whole(i);
            if (!all) visible(i, r, a, b);
            const unsigned len = b >= a ? b - a + 1 : 0;
            if (!KEYS && i < dry) {
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    uint32_t s[32], q[32];
                    tmem_ld32_nowait(ts + c * 32, s);
                    tmem_ld32_nowait(tp + c * 32, q);
                    tmem_wait_ld();
                    reg_fence32(s);
                    reg_fence32(q);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (static_cast<unsigned>(c * 32 + e - a) < len)
                            off = fmaf(ex2_ftz(fmaf(__uint_as_float(s[e]), p.c, l2.x)), __uint_as_float(q[e]) + d2.x, off);
                }
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&s_p[x]));
                continue;
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t s[32], q[32];
                tmem_ld32_nowait(ts + c * 32, s);
                tmem_ld32_nowait(tp + c * 32, q);
                tmem_wait_ld();
                reg_fence32(s);
                reg_fence32(q);
                uint32_t ep[16], es[16];
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    float2 lj[2] = {l2, l2}, dj[2] = {d2, d2};
                    if (KEYS) {
                        const float4 l4 = s_row[x][turn][c * 8 + j / 4][0], d4 = s_row[x][turn][c * 8 + j / 4][1];
                        lj[0] = make_float2(l4.x, l4.y), lj[1] = make_float2(l4.z, l4.w);
                        dj[0] = make_float2(d4.x, d4.y), dj[1] = make_float2(d4.z, d4.w);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int e = j + 2 * h;
                        float2 v = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), cc, lj[h]);
                        v.x = ex2_ftz(v.x);
                        v.y = ex2_ftz(v.y);
                        float2 w = add2(make_float2(__uint_as_float(q[e]), __uint_as_float(q[e + 1])), dj[h]);
                        if (F16) w = mul2(w, ff);
                        w = mul2(w, v);
                        if (!all) {
                            if (static_cast<unsigned>(c * 32 + e - a) >= len) v.x = w.x = 0.f;
                            if (static_cast<unsigned>(c * 32 + e + 1 - a) >= len) v.y = w.y = 0.f;
                        }
                        if (KEYS) ep[e / 2] = Pair<E>::pack(v.x, v.y);
                        es[e / 2] = Pair<E>::pack(w.x, w.y);
                    }
                }
                if (KEYS) tmem_st16_nowait(ts + c * 16, ep);
                tmem_st16_nowait(tp + c * 16, es);
            }
            tmem_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s_p[x]));
        }
        if (!KEYS && dry > 0 && !corrected && !correct(ok)) ok = false;      // a wait gave up in the dry steps, or no step of this group's follows
        if (ok) ok = wait_warp(smem_u32(&s_end), 0);
        if (!ok && lane == 0) give_up();
        // ---- the sums: the first group writes dk or dq, the second dv; rounded once, rows by way of shared memory (the own rows are
        // no longer needed), the sinks' in fp32 into the workspace
        if (ok && (KEYS || x == 0)) {
            fence_after();
            const float mul = x == 0 ? p.scale / factor : F16 ? 0x1p-10f : 1.f;
            unsigned char *const stage = basep + L::X + x * L::X_BYTES;
            const int keep = KEYS && has_sinks && x0 == 0 ? min(p.S, rows) : 0;      // rows that go into the workspace
            float *const part = sinks ? k.rest + ((static_cast<int64_t>(slot) * p.Hk + head) * 2 + x) * p.S * D
                                      : k.first + ((static_cast<int64_t>(at.seq) * p.Hk + head) * 2 + x) * p.S * D;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tmem_ld32_nowait(tmem + lanes + TM_ACC + x * D + c * 32, v);
                tmem_wait_ld();
                reg_fence32(v);
                float f[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]) * mul;
                if (r < keep)
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        *reinterpret_cast<float4 *>(part + static_cast<int64_t>(r) * D + c * 32 + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint4 y;
                    y.x = Pair<E>::pack(f[8 * q], f[8 * q + 1]);
                    y.y = Pair<E>::pack(f[8 * q + 2], f[8 * q + 3]);
                    y.z = Pair<E>::pack(f[8 * q + 4], f[8 * q + 5]);
                    y.w = Pair<E>::pack(f[8 * q + 6], f[8 * q + 7]);
                    *reinterpret_cast<uint4 *>(stage + r * (2 * D) + (((c * 4 + q) ^ (r & 7)) << 4)) = y;
                }
            }
            __syncwarp();
            if (!sinks) {
                constexpr int CH = D / 8, RPI = 32 / CH;
                const int ch = lane % CH;
                const int64_t ld = x == 0 ? ld1 : ld2;
                E *const dst = (x == 0 ? out1 : out2) + (static_cast<int64_t>(at.start) + x0) * ld + head * D + ch * 8;
#pragma unroll 4
                for (int j = 0; j < 32; j += RPI) {
                    const int row = (warp & 3) * 32 + j + lane / CH;
                    if (row >= keep && row < rows)
                        *reinterpret_cast<uint4 *>(dst + row * ld) = *reinterpret_cast<const uint4 *>(stage + row * (2 * D) + ((ch ^ (row & 7)) << 4));
                }
            }
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 0) {
        if (s_abort && lane == 0) {     // the copies in flight end before the memory is given back
            mbar_wait(smem_u32(&s_x), 0);
            for (int i = 0; i < STAGES && i < fetched; ++i) mbar_wait(smem_u32(&s_full[i]), ((fetched - 1 - i) / STAGES) & 1);
        }
        __syncwarp();
        tmem_dealloc(tmem, TM_COLS);
    }
}

// D of every row: d / 8 lanes a head's row.  fp16: also the longest rows of do and v of each key head.
template <typename E, int D>
__global__ void __launch_bounds__(256) window_delta(const Shape p, const E *o, int64_t ldo, const E *d_o, int64_t lddo, const E *v, int64_t ldv, Back k)
{
    constexpr int LANES = D / 8;
    const int lane = threadIdx.x & 31, l = lane % LANES;
    const int heads = p.H + (Pair<E>::BF16 ? 0 : p.Hk);      // the value heads behind the query heads
    const int64_t n = static_cast<int64_t>(p.T) * heads, all = (n * LANES + 31) / 32 * 32;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < all; i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t row = i / LANES, t = row / heads;
        const int h = static_cast<int>(row - t * heads);
        float dot = 0.f, sq = 0.f;
        if (row < n) {
            const uint4 a = *reinterpret_cast<const uint4 *>(h < p.H ? d_o + t * lddo + h * D + l * 8 : v + t * ldv + (h - p.H) * D + l * 8);
            const uint4 b = h < p.H ? *reinterpret_cast<const uint4 *>(o + t * ldo + h * D + l * 8) : a;
            const E *const x = reinterpret_cast<const E *>(&a), *const y = reinterpret_cast<const E *>(&b);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float u = to_f32(x[j]);
                dot = fmaf(u, to_f32(y[j]), dot);
                if (!Pair<E>::BF16) sq = fmaf(u, u, sq);
            }
        }
#pragma unroll
        for (int m = LANES / 2; m; m >>= 1) {
            dot += __shfl_xor_sync(0xffffffffu, dot, m);
            if (!Pair<E>::BF16) sq += __shfl_xor_sync(0xffffffffu, sq, m);
        }
        if (l == 0 && row < n) {
            if (h < p.H) k.delta[static_cast<int64_t>(h) * p.T + t] = dot;
            if (!Pair<E>::BF16 && isfinite(sq)) {      // numbers above zero compare as their bits do
                int *const to = reinterpret_cast<int *>(k.most) + (h < p.H ? h / (p.H / p.Hk) : p.Hk + h - p.H);
                const int bits = __float_as_int(sqrtf(sq));
                if (bits > *static_cast<volatile int *>(to)) atomicMax(to, bits);
            }
        }
    }
}

// The sinks' rows of dk and dv: the window's part and the pieces', in order.
template <typename E>
__global__ void __launch_bounds__(256) window_sinks(const Shape p, const Back k, int D, E *dk, int64_t lddk, E *dv, int64_t lddv)
{
    if (!plan_matches(p.plan, p.sig)) return;
    const int32_t *cu = p.plan + p.off_cu;
    const int seq = blockIdx.x / p.Hk, head = blockIdx.x % p.Hk, start = cu[seq], len = cu[seq + 1] - start;
    if (len <= p.W) return;
    const int keep = min(p.S, len), slot0 = start / CHUNK + seq;
    const int64_t size = static_cast<int64_t>(p.S) * D;
    for (int i = threadIdx.x; i < 2 * keep * D; i += blockDim.x) {
        const int x = i / (keep * D), e = i - x * keep * D;
        float sum = k.first[((static_cast<int64_t>(seq) * p.Hk + head) * 2 + x) * size + e];
        for (int c = p.W / CHUNK; c <= (len - 1) / CHUNK; ++c)
            sum += k.rest[((static_cast<int64_t>(slot0 + c) * p.Hk + head) * 2 + x) * size + e];
        E *const to = x == 0 ? dk + (static_cast<int64_t>(start) + e / D) * lddk : dv + (static_cast<int64_t>(start) + e / D) * lddv;
        to[head * D + e % D] = from_f32<E>(sum);
    }
}

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Regions of the workspace: D, the longest rows, the sinks' parts; off[4]: its size.
void layout(int T, int N, int H, int Hk, int d, int W, int S, size_t off[5])
{
    const size_t part = static_cast<size_t>(Hk) * 2 * S * d * 4, some = S > 0 && W < T;
    off[0] = 0;
    off[1] = round256(static_cast<size_t>(H) * T * 4);
    off[2] = round256(off[1] + static_cast<size_t>(2) * Hk * 4);
    off[3] = round256(off[2] + some * N * part);
    off[4] = round256(off[3] + some * static_cast<size_t>(tile_slots(T, N, CHUNK)) * part);
}

template <typename E, int D>
cudaError_t backward(const Shape &p, const WindowIn &in, const WindowGrads &g, void *ws, cudaStream_t stream)
{
    const bool bf16 = Pair<E>::BF16;
    size_t off[5];
    layout(p.T, p.N, p.H, p.Hk, D, p.W, p.S, off);
    char *const b = static_cast<char *>(ws);
    Back k{g.lse, reinterpret_cast<float *>(b + off[0]), reinterpret_cast<float *>(b + off[1]), reinterpret_cast<float *>(b + off[2]),
           reinterpret_cast<float *>(b + off[3]), 0};
    const bool sinks = p.S > 0 && p.W < p.T;
    const int64_t slots = tile_slots(p.T, p.N, TILE), pieces = sinks ? static_cast<int64_t>(tile_slots(p.T, p.N, CHUNK)) * p.Hk : 0;
    if (slots * p.H > INT32_MAX || slots * p.Hk + pieces > INT32_MAX || static_cast<int64_t>(p.N) * p.Hk > INT32_MAX)
        return cudaErrorInvalidConfiguration;
    k.window_blocks = static_cast<int>(slots * p.Hk);
    CUtensorMap m[8];      // queries, do, keys, values: tiles of 128 rows, then of 64
    for (int i = 0; i < 2; ++i) {
        const uint32_t rows = i ? SUB : TILE;
        if (!encode_heads(&m[4 * i], in.q, bf16, D, p.H, p.T, in.ldq, rows) || !encode_heads(&m[4 * i + 1], g.d_o, bf16, D, p.H, p.T, g.lddo, rows) ||
            !encode_heads(&m[4 * i + 2], in.k, bf16, D, p.Hk, p.T, in.ldk, rows) ||
            !encode_heads(&m[4 * i + 3], in.v, bf16, D, p.Hk, p.T, in.ldv, rows))
            return cudaErrorInvalidValue;
    }
    cudaError_t e;
    if (!bf16 && (e = cudaMemsetAsync(k.most, 0, static_cast<size_t>(2) * p.Hk * 4, stream)) != cudaSuccess) return e;
    const int64_t rows = static_cast<int64_t>(p.T) * (p.H + (bf16 ? 0 : p.Hk)) * (D / 8);
    const int grid = static_cast<int>(min((rows + 255) / 256, static_cast<int64_t>(sm_count()) * 16));
    window_delta<E, D><<<grid, 256, 0, stream>>>(p, static_cast<const E *>(g.o), g.ldo, static_cast<const E *>(g.d_o), g.lddo,
                                                 static_cast<const E *>(in.v), in.ldv, k);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const void *fk = reinterpret_cast<const void *>(&window_back<E, D, true>), *fq = reinterpret_cast<const void *>(&window_back<E, D, false>);
    if ((e = set_dynamic_smem(fk, Smem<D>::ALLOC)) != cudaSuccess || (e = set_dynamic_smem(fq, Smem<D>::ALLOC)) != cudaSuccess) return e;
    window_back<E, D, false><<<static_cast<int>(slots * p.H), THREADS, Smem<D>::ALLOC, stream>>>(
        m[0], m[1], m[6], m[7], p, k, static_cast<E *>(g.dq), g.lddq, nullptr, 0);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    window_back<E, D, true><<<static_cast<int>(slots * p.Hk + pieces), THREADS, Smem<D>::ALLOC, stream>>>(
        m[2], m[3], m[4], m[5], p, k, static_cast<E *>(g.dk), g.lddk, static_cast<E *>(g.dv), g.lddv);
    if ((e = cudaGetLastError()) != cudaSuccess || !sinks) return e;
    window_sinks<E><<<p.N * p.Hk, 256, 0, stream>>>(p, k, D, static_cast<E *>(g.dk), g.lddk, static_cast<E *>(g.dv), g.lddv);
    return cudaGetLastError();
}

}  // namespace

size_t window_workspace_bytes(int T, int N, int H, int Hk, int d, int W, int S)
{
    size_t off[5];
    layout(T, N, H, Hk, d, W, S, off);
    return off[4];
}

cudaError_t launch_window_backward(const int32_t *plan_host, const int32_t *plan_dev, int type, const WindowIn &in, const WindowGrads &g, void *ws,
                                   cudaStream_t stream)
{
    const Shape p = window_shape(plan_host, plan_dev, in);
    if (type == KDA_TYPE_F16) return in.d == 64 ? backward<__half, 64>(p, in, g, ws, stream) : backward<__half, 128>(p, in, g, ws, stream);
    return in.d == 64 ? backward<__nv_bfloat16, 64>(p, in, g, ws, stream) : backward<__nv_bfloat16, 128>(p, in, g, ws, stream);
}

int take_window_back_status()
{
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_window_back_status, sizeof(int)) != cudaSuccess) return KDA_ERR_CUDA;
    if (v != 0 && cudaMemcpyToSymbol(g_window_back_status, &z, sizeof(int)) != cudaSuccess) return KDA_ERR_CUDA;
    return v;
}

}  // namespace kda
