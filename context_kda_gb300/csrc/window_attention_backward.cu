// Gradients of the window attention.  With p_ij = exp(scale q_i . k_j - lse_i), D_i = do_i . o_i:
//     dp_ij = do_i . v_j,   ds_ij = p_ij (dp_ij - D_i),
//     dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_{i, heads} ds_ij q_i,   dv_j = sum_{i, heads} p_ij do_i.
//
// Three kernels, and no atomics on sums, so that the same call gives the same bits: the rows' D; a kernel whose CTAs own 128
// queries and go over their keys (dq); and one whose CTAs own 128 keys and go over the queries that see them, of all heads of
// the group (dk, dv).  Scores and dp are computed in both: seven products for each pair of tiles where one kernel with a shared dq
// would take five.
// The last two are one kernel of two kinds.  Its own rows X1, X2 (keys and values, or queries and do) stay in shared
// memory; tiles of 128 of the other side, Y1, Y2, come by TMA.  Per pair of tiles
//     S = X1 Y1^T, P' = X2 Y2^T             to TMEM,
//     p, then ds                            two threads a row; both back to TMEM in the places of S and P', as A operands of
//     A2 += p Y2 (dv), A1 += ds Y1 (dk or dq).
// For keys the tensor cores run A2(i), S(i+1), A1(i), P'(i+1) in turn: p(i+1) is computed during A1(i) and P'(i+1), ds(i) during
// A2(i) and S(i+1), so one buffer each is enough.  Queries have one sum and room for a second P': S(i+1), P'(i+1), A1(i), and p and ds
// of a step are computed while the scores of the next are.  (Tiles of 64 with two buffers of everything fit too, but products
// with N = 64 are bound by shared memory: 57 cycles where 32 would do.)
//
// D_i from the output carries that output's rounding (and that of its probabilities): u sum_c |do_c| (sum_j p_ij |v_jc| + |o_ic|) at most,
// and ds_ij is off by p_ij times that.  In a row that spreads its weight over many keys the rounding of ds itself is larger; in one that
// sees few, or puts nearly all its weight on few of many, ds is next to nothing and the error stays: it is the larger one
// there.  Rows that see few can be told beforehand: the first queries of a sequence, and all with a narrow window, go over their
// tiles twice: sum_j ds_ij, which is zero with the right D, corrects D first, and the corrected D is left for the keys.  The others keep
// the output's D, since a second pass over all tiles is two products more for seven.  dq of random rows of 2000 keys in bf16 is off by 0.24 %
// against 64 bits, as with an exact D; with scores 4 times as wide by 0.37 % (exact 0.24 %), 16 times 0.67 %.
//
// Sinks are seen by every later query of their sequence.  Their tile's window part is worked as any other; the rest is cut into
// pieces of CHUNK queries, each a CTA's, which leave sums in fp32 in the workspace, and a last kernel adds those in order.
//
// Bound by the products and, beside them, p and ds, and by the ends of the two launches: 8192 tokens x 16 heads (4 key heads) of 128, window 1024,
// bf16, 240 us, 36 % of the dense rate (half of it, counting the two products done twice); 8 heads of 64 in fp16, documents of any length, 150 to
// 180 us (14 to 16 %).  Tiles are launched last to first.  For queries that is most work first; for keys it is the reverse: the first ones are
// seen by the most queries and start last, and with shared key heads a CTA walks all heads of its group.  A list schedule of the documents'
// keys takes 46 to 62 steps where 40 to 47 are the mean, of 8192 x (16, 4) heads with everything visible 363 for 221.
//
// fp16 has a narrow range: p is kept times 2^10, ds times a power of two for each key head, from the longest rows of do and v
// (|ds| <= 2 |do| |v|), so that it neither overflows nor fades.  bf16 needs neither.
#include "window_attention.cuh"

namespace kda {
namespace {

using namespace attn;

__device__ int g_window_back_status;

constexpr int THREADS = 384;
constexpr int REGS_OTHER = 72, REGS_SOFTMAX = 216;     // of 168 at the launch: 128 x 72 + 256 x 216 = 384 x 168
constexpr int HALF = TILE / 2;            // columns of a thread
constexpr int NARROW = 32;                // windows up to this are narrow
constexpr int CHUNK = 1024;               // queries of a piece of the sinks' work (tiles and pieces are found by shifts: 2^7, 2^10)

template <int D> struct Smem {
    static constexpr uint32_t T_BYTES = D / 64 * BOX;
    static constexpr int N1 = 3, N2 = 2;      // stages of Y1 (read first and last in a round) and of Y2
    static constexpr uint32_t X = 0, Y1 = 2 * T_BYTES, Y2 = Y1 + N1 * T_BYTES, BYTES = Y2 + N2 * T_BYTES;
    static_assert(BYTES + 3 * 1024 <= 227 * 1024, "shared memory");      // with the static part
};
// TMEM columns: S (p), P' (ds), the sums
constexpr uint32_t TM_S = 0, TM_P = 128, TM_ACC = 256, TM_P2 = 384, TM_COLS = 512;      // (queries: TM_P2 for odd steps)

struct Back {
    const float *lse;                     // [H][T]
    float *delta;                         // [H][T]
    float *most;                          // fp16: [2][Hk], the longest rows of do and of v
    float *first, *rest;                  // sinks: the window's part [N][Hk][2][S][d], the pieces' [slots][Hk][2][S][d]
    int window_blocks;                    // blocks of windows' tiles; the others are the sinks' pieces
};

// ds is kept times this in fp16: 2 |do| |v| becomes 2^14 to 2^15, so that |ds| from 2^-27 of |do| |v| up is a normal number (2^-14).
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
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ uint64_t s_x, s_y1[L::N1], s_free1[L::N1], s_y2[L::N2], s_free2[L::N2], s_go, s_s, s_pp[2], s_a, s_b[2], s_rows[2], s_rfree[2], s_end;
    __shared__ float4 s_row[2][TILE / 4][2];             // KEYS: four queries' lse, then D, of two tiles; else: sums of ds
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) prefetch_map(mx1), prefetch_map(mx2), prefetch_map(my1), prefetch_map(my2);
    // A device plan of another launch: no gradient is written.  Where the starts come with the launch nothing depends on it before.
    const bool right = plan_matches(p.plan, p.sig);
    if (p.N > FEW && !right) {
        if (tid == 0 && blockIdx.x == 0) record_status(&g_window_back_status, KDA_ERR_INVALID_ARG);
        grid_dep_wait();                                 // the rows' D is still being written: the call ends when that has
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
        if (!find_tile(p, slot, 10, at)) return;
    } else {
        const int works = KEYS ? p.Hk : p.H, i = (KEYS ? k.window_blocks : static_cast<int>(gridDim.x)) - 1 - blockIdx.x;
        head = i % works;
        if (!find_tile(p, i / works, 7, at)) return;
    }
    const int W = min(p.W, at.len), x0 = sinks ? 0 : at.t0, rows = min(TILE, at.len - x0);      // own rows [x0, x0 + rows)
    const bool has_sinks = p.S > 0 && W < at.len;        // some query has left a sink behind its window
    // tiles of the other side: [lo, hi], then (queries) that of the sinks
    int lo, hi, extra = 0;
    if (KEYS) {
        const int64_t end = sinks ? at.t0 + CHUNK : static_cast<int64_t>(x0) + TILE - 1 + W;
        lo = (sinks ? max(at.t0, W) : x0) / TILE;
        hi = static_cast<int>((min(end, static_cast<int64_t>(at.len)) - 1) / TILE);
        if (sinks && (!has_sinks || lo > hi)) return;
    } else {
        lo = max(0, x0 - W + 1) / TILE;
        hi = x0 / TILE;
        extra = has_sinks && x0 + rows - 1 >= W;
    }
    const int tiles = KEYS ? g * (hi - lo + 1) : hi - lo + 1 + extra;
    const int dry = !KEYS && (tiles == 1 || W <= NARROW) ? tiles : 0, n = dry + tiles;      // steps, the first 'dry' of them for D alone
    const int xh = head, yh = KEYS ? head * g : head / g;                        // heads of the own rows and of the other side
    // The steps in order: keys go over the tiles of each query head from lo up; queries from the diagonal down, the sinks last.
    struct Iter {
        int tile, head;
        bool sink;
    };
    auto first = [&] { return Iter{KEYS ? lo : hi, yh, KEYS && sinks}; };
    auto advance = [&](Iter &i) {
        if (KEYS) {
            if (++i.tile > hi) i.tile = lo, ++i.head;
        } else if (i.sink || (i.tile == lo && !extra)) {
            i = first();
        } else if (i.tile == lo) {
            i.tile = 0, i.sink = true;
        } else {
            --i.tile;
        }
    };
    // whether all own rows and all rows of the tile see each other
    auto whole = [&](const Iter &i) {
        const int y0 = i.tile * TILE;
        if (i.sink) return false;
        if (KEYS) return y0 >= x0 + TILE - 1 && y0 + TILE - 1 - x0 < W && y0 + TILE <= at.len;
        return y0 + TILE - 1 <= x0 && x0 + TILE - 1 - y0 < W;
    };
    // columns [a, b] of the tile that go with own row r
    auto visible = [&](const Iter &i, int r, int &a, int &b) {
        const int y0 = i.tile * TILE, x = x0 + r;
        if (KEYS) {
            a = i.sink ? (x < p.S ? x + W - y0 : TILE) : x - y0;
            b = (i.sink ? at.len - 1 : static_cast<int>(min(static_cast<int64_t>(x) + W, static_cast<int64_t>(at.len)) - 1)) - y0;
        } else {
            a = i.sink ? 0 : x - W + 1 - y0;
            b = (i.sink ? min(p.S - 1, x - W) : x) - y0;
        }
    };

    const uint32_t base = smem_u32(smem);
    unsigned char *const basep = smem;
    if (base & 1023u) {                                  // the swizzle counts from there
        if (tid == 0) record_status(&g_window_back_status, KDA_ERR_UNSUPPORTED);
        return;
    }
    int fetched[2] = {0, 0};                             // (the fetching thread) tiles of Y1 and of Y2
    auto load = [&](const CUtensorMap &m, uint32_t dst, int h, int row, uint32_t bar) {
        for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * BOX, &m, c * 64, h, at.start + row, bar);
    };
    auto fetch = [&](const CUtensorMap &m, uint32_t to, const Iter &i, uint64_t &full) {
        mbar_arrive_expect_tx(smem_u32(&full), L::T_BYTES);
        load(m, base + to, i.head, i.tile * TILE, smem_u32(&full));
    };
    if (tid == 0) {
        mbar_init(smem_u32(&s_x), 1);
        for (int i = 0; i < L::N1; ++i) mbar_init(smem_u32(&s_y1[i]), 1), mbar_init(smem_u32(&s_free1[i]), 1);
        for (int i = 0; i < L::N2; ++i) mbar_init(smem_u32(&s_y2[i]), 1), mbar_init(smem_u32(&s_free2[i]), 1);
        mbar_init(smem_u32(&s_go), 1);
        mbar_init(smem_u32(&s_s), 1);
        for (int i = 0; i < 2; ++i) {                    // of even and odd steps: nobody can fall a whole round behind
            mbar_init(smem_u32(&s_pp[i]), 1);
            mbar_init(smem_u32(&s_b[i]), KEYS ? 9 : 8);
            mbar_init(smem_u32(&s_rows[i]), 1);
            mbar_init(smem_u32(&s_rfree[i]), 8);
        }
        mbar_init(smem_u32(&s_a), 9);
        mbar_init(smem_u32(&s_end), 1);
        s_abort = 0;
        // the first tiles are on their way before anything else
        const uint32_t bx = smem_u32(&s_x);
        mbar_arrive_expect_tx(bx, 2 * L::T_BYTES);
        load(mx1, base + L::X, xh, x0, bx);
        const Iter i = first();
        fetch(my1, L::Y1, i, s_y1[0]);
        load(mx2, base + L::X + L::T_BYTES, xh, x0, bx);
        fetch(my2, L::Y2, i, s_y2[0]);
        fetched[0] = fetched[1] = 1;
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
    if (warp < 4) fewer_registers<REGS_OTHER>();

    if (warp == 0) {
        // ---- fetch
        if (lane == 0) {
            bool ok = true;
            Iter it = first();
            for (int i = 1, s1 = 1, s2 = 1 % L::N2, r1 = 0, r2 = 0; i < n; ++i) {      // stages, and rounds through them
                advance(it);
                if (i >= L::N1) ok = wait_thread(smem_u32(&s_free1[s1]), (r1 - 1) & 1);
                if (!ok) break;
                fetch(my1, L::Y1 + s1 * L::T_BYTES, it, s_y1[s1]);
                ++fetched[0];
                if (i >= L::N2) ok = wait_thread(smem_u32(&s_free2[s2]), (r2 - 1) & 1);
                if (!ok) break;
                fetch(my2, L::Y2 + s2 * L::T_BYTES, it, s_y2[s2]);
                ++fetched[1];
                if (++s1 == L::N1) s1 = 0, ++r1;
                if (++s2 == L::N2) s2 = 0, ++r2;
            }
            if (!ok) give_up();
        }
    } else if (warp == 1) {
        // ---- products.  TMEM addresses start at 0: the CTA has all of it
        constexpr uint32_t ID_S = idesc<E>(TILE, TILE, 0), ID_A = idesc<E>(TILE, D, 1);
        auto scores = [&](uint32_t to, uint32_t x, uint32_t y, uint64_t &bar) {
            const uint32_t xd = desc_k(x), yd = desc_k(y);
            if (elect()) {
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t off = ((s / 4) * BOX + (s % 4) * 32) >> 4;
                    product(to, xd + off, yd + off, ID_S, s > 0);
                }
                commit(smem_u32(&bar));
            }
            __syncwarp();
        };
        auto add = [&](uint32_t to, uint32_t from, uint32_t y, bool more) {
            const uint32_t yd = desc_mn(y, BOX);
            if (elect()) {
#pragma unroll
                for (int s = 0; s < TILE / 16; ++s)
                    product_ta(to, from + (s / 4) * HALF + (s % 4) * 8, yd + s * (2048 >> 4), ID_A, more || s > 0);
            }
            __syncwarp();
        };
        auto signal = [&](uint64_t &bar) {
            if (elect()) commit(smem_u32(&bar));
            __syncwarp();
        };
        bool ok = wait_warp(smem_u32(&s_x), 0) && wait_warp(smem_u32(&s_go), 0);
        if (ok) {
            fence_after();
            scores(TM_S, base + L::X, base + L::Y1, s_s);
            scores(TM_P, base + L::X + L::T_BYTES, base + L::Y2, s_pp[0]);
            if (!KEYS) signal(s_free2[0]);
        }
        int c1 = 0, c2 = 0;                              // stages of step i
        for (int i = 0; i < n && ok; ++i) {
            const int d1 = c1 + 1 == L::N1 ? 0 : c1 + 1, d2 = c2 + 1 == L::N2 ? 0 : c2 + 1;
            const bool next = i + 1 < n;
            const uint32_t p_now = KEYS || !(i & 1) ? TM_P : TM_P2, p_next = KEYS || (i & 1) ? TM_P : TM_P2;
            ok = wait_warp(smem_u32(&s_a), i & 1);       // S(i) is read (keys: and p in its place); Y1(i + 1), for queries Y2(i + 1) too, is there
            if (!ok) break;
            fence_after();
            if (KEYS) {
                add(TM_ACC + D, TM_S, base + L::Y2 + c2 * L::T_BYTES, i > 0);
                signal(s_free2[c2]);
            }
            if (next) scores(TM_S, base + L::X, base + L::Y1 + d1 * L::T_BYTES, s_s);
            if (next && !KEYS) {
                scores(p_next, base + L::X + L::T_BYTES, base + L::Y2 + d2 * L::T_BYTES, s_pp[(i + 1) & 1]);
                signal(s_free2[d2]);
            }
            ok = wait_warp(smem_u32(&s_b[i & 1]), i >> 1 & 1);       // ds in the place of P'(i); keys: Y2(i + 1) is there
            if (!ok) break;
            fence_after();
            if (i >= dry) add(TM_ACC, p_now, base + L::Y1 + c1 * L::T_BYTES, i > dry);
            signal(s_free1[c1]);
            if (next && KEYS) scores(TM_P, base + L::X + L::T_BYTES, base + L::Y2 + d2 * L::T_BYTES, s_pp[(i + 1) & 1]);
            c1 = d1;
            c2 = d2;
        }
        if (!ok && lane == 0) give_up();
        signal(s_end);
        if (!ok) wait_warp(smem_u32(&s_end), 0);         // the products in flight end before the memory is given back
    } else if (warp == 2) {
        // ---- rows behind the sequence's end: zeros, so that a factor of zero meets no infinity or NaN there.  Tells the products
        // when the next tiles are there
        bool ok = true;
        Iter it = first();
        int s1 = 0, s2 = 0, r1 = 0, r2 = 0;
        auto there = [&](uint64_t &full, int round, uint32_t to) {
            ok = wait_warp(smem_u32(&full), round & 1);
            const int real = at.len - it.tile * TILE;
            if (!ok || real >= TILE) return;
            for (int r = real + lane / 8; r < TILE; r += 4)
                for (int c = 0; c < D / 64; ++c)
                    *reinterpret_cast<uint4 *>(basep + to + c * BOX + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
            fence_async_smem();
            __syncwarp();
        };
        there(s_y1[0], 0, L::Y1);
        if (ok) there(s_y2[0], 0, L::Y2);
        if (ok && lane == 0) mbar_arrive(smem_u32(&s_go));
        for (int i = 0; i < n && ok; ++i) {
            if (++s1 == L::N1) s1 = 0, ++r1;
            if (++s2 == L::N2) s2 = 0, ++r2;
            advance(it);
            // (an arrival waits for the step's scores, which are issued when the arrivals of the step before are complete; queries'
            // P'(i + 1) does not wait for s_b(i), so there is no arrival here)
            if (i + 1 < n) there(s_y1[s1], r1, L::Y1 + s1 * L::T_BYTES);
            if (!KEYS && ok && i + 1 < n) there(s_y2[s2], r2, L::Y2 + s2 * L::T_BYTES);
            ok = ok && wait_warp(smem_u32(&s_s), i & 1);
            if (!ok) break;
            if (lane == 0) mbar_arrive(smem_u32(&s_a));
            if (!KEYS) continue;
            if (i + 1 < n) there(s_y2[s2], r2, L::Y2 + s2 * L::T_BYTES);
            ok = ok && wait_warp(smem_u32(&s_pp[i & 1]), i >> 1 & 1);
            if (!ok) break;
            if (lane == 0) mbar_arrive(smem_u32(&s_b[i & 1]));
        }
        if (!ok && lane == 0) give_up();
    } else if (warp == 3 && KEYS) {
        // ---- the queries' lse and D, a tile ahead
        grid_dep_wait();
        bool ok = true;
        Iter it = first();
        for (int i = 0; i < n; ++i, advance(it)) {
            float v[2][TILE / 32];
#pragma unroll
            for (int j = 0; j < TILE / 32; ++j) {
                const int y = it.tile * TILE + j * 32 + lane;
                const int64_t row = static_cast<int64_t>(it.head) * p.T + at.start + y;
                v[0][j] = v[1][j] = 0.f;
                if (y < at.len) v[0][j] = k.lse[row], v[1][j] = k.delta[row];
            }
            // the tile before last has been read by all
            if (i > 1) ok = wait_warp(smem_u32(&s_rfree[i & 1]), (i >> 1) - 1 & 1);
            if (!ok) break;
            float *const to = reinterpret_cast<float *>(s_row[i & 1]) + lane / 4 * 8 + (lane & 3);
#pragma unroll
            for (int j = 0; j < TILE / 32; ++j) {
                to[j * 64] = fmaf(-v[0][j], 1.44269504088896340736f, P_EXP);
                to[j * 64 + 4] = -v[1][j];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s_rows[i & 1]));
        }
        if (!ok && lane == 0) give_up();
    } else if (warp > 3) {
        // ---- p and ds, two threads a row
        more_registers<REGS_SOFTMAX>();
        const int x = (warp >> 2) - 1, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + TM_S + x * HALF;
        grid_dep_wait();                                 // D (and what goes with it) is the kernel's before
        const float factor = F16 ? ds_factor(k.most[KEYS ? head : yh], k.most[p.Hk + (KEYS ? head : yh)]) : 1.f;
        const float ds_mul = factor * (F16 ? 0x1p-10f : 1.f);
        const float2 cc = make_float2(p.c, p.c), ff = make_float2(ds_mul, ds_mul);
        Iter it = first();
        float2 l2 = make_float2(0.f, 0.f), d2 = make_float2(0.f, 0.f);      // queries: of the thread's own row
        if (!KEYS && r < rows) {
            const int64_t at_row = static_cast<int64_t>(head) * p.T + at.start + x0 + r;
            l2.x = l2.y = P_EXP - k.lse[at_row] * 1.44269504088896340736f;
            d2.x = d2.y = -k.delta[at_row];
        }
        bool ok = true, corrected = false;
        float off = 0.f;                                 // (dry steps) sum of ds
        float *const s_dry = reinterpret_cast<float *>(s_row);
        for (int i = 0; i < n; ++i, advance(it)) {
            if (!KEYS && dry > 0 && i == dry) {          // D by what both threads of the row have found
                corrected = true;
                s_dry[x * TILE + r] = off * (F16 ? 0x1p-10f : 1.f);
                bar_or(3, 256, false);
                d2.x -= s_dry[r] + s_dry[TILE + r];
                d2.y = d2.x;
                if (x == 0 && r < rows) k.delta[static_cast<int64_t>(head) * p.T + at.start + x0 + r] = -d2.x;
            }
            const bool all = whole(it);
            int a = 0, b = TILE - 1;
            if (!all) visible(it, r, a, b);
            a -= x * HALF;
            b -= x * HALF;
            const uint32_t tp = tmem + lanes + (KEYS || !(i & 1) ? TM_P : TM_P2) + x * HALF;
            ok = (!KEYS || wait_warp(smem_u32(&s_rows[i & 1]), i >> 1 & 1)) && wait_warp(smem_u32(&s_s), i & 1);
            if (!ok) break;
            const float4 (*const row)[2] = s_row[i & 1] + x * (HALF / 4);
            fence_after();
            uint32_t u[2][32];
            tmem_ld32_nowait(ts, u[0]);
            tmem_ld32_nowait(ts + 32, u[1]);
            tmem_wait_ld();
            reg_fence32(u[0]);
            reg_fence32(u[1]);
            if (!KEYS) {
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&s_a));
            }
            float2 pr[HALF / 2];
#pragma unroll
            for (int j = 0; j < HALF; j += 4) {
                float4 l4 = make_float4(l2.x, l2.y, l2.x, l2.y);
                if (KEYS) l4 = row[j / 4][0];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int e = j + 2 * h;
                    float2 v = fma2(make_float2(__uint_as_float(u[e / 32][e % 32]), __uint_as_float(u[e / 32][e % 32 + 1])), cc,
                                    h ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y));
                    v.x = ex2_ftz(v.x);
                    v.y = ex2_ftz(v.y);
                    pr[e / 2] = v;
                }
            }
            if (!all) {
                // a bound that no row of the warp meets costs nothing.  (ds is zero where p is: the other side's rows are finite
                // behind the sequence's end)
#pragma unroll
                for (int c = 0; c < HALF; c += 32) {
                    if (__any_sync(0xffffffffu, a > c)) {
#pragma unroll
                        for (int e = c; e < c + 32; ++e)
                            if (e < a) (e & 1 ? pr[e / 2].y : pr[e / 2].x) = 0.f;
                    }
                    if (__any_sync(0xffffffffu, b < c + 31)) {
#pragma unroll
                        for (int e = c; e < c + 32; ++e)
                            if (e > b) (e & 1 ? pr[e / 2].y : pr[e / 2].x) = 0.f;
                    }
                }
            }
            if (KEYS) {
                uint32_t w[32];
#pragma unroll
                for (int e = 0; e < HALF / 2; ++e) w[e] = Pair<E>::pack(pr[e].x, pr[e].y);
                tmem_st32_nowait(ts, w);
                tmem_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&s_a));
            }
            ok = wait_warp(smem_u32(&s_pp[i & 1]), i >> 1 & 1);
            if (!ok) break;
            fence_after();
            tmem_ld32_nowait(tp, u[0]);
            tmem_ld32_nowait(tp + 32, u[1]);
            tmem_wait_ld();
            reg_fence32(u[0]);
            reg_fence32(u[1]);
            if (!KEYS && i < dry) {
#pragma unroll
                for (int e = 0; e < HALF; ++e)
                    off = fmaf(e & 1 ? pr[e / 2].y : pr[e / 2].x, __uint_as_float(u[e / 32][e % 32]) + d2.x, off);
            } else {
                float2 ds[HALF / 2];
#pragma unroll
                for (int j = 0; j < HALF; j += 4) {
                    float4 d4 = make_float4(d2.x, d2.y, d2.x, d2.y);
                    if (KEYS) d4 = row[j / 4][1];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int e = j + 2 * h;
                        float2 v = add2(make_float2(__uint_as_float(u[e / 32][e % 32]), __uint_as_float(u[e / 32][e % 32 + 1])),
                                        h ? make_float2(d4.z, d4.w) : make_float2(d4.x, d4.y));
                        if (F16) v = mul2(v, ff);
                        ds[e / 2] = mul2(v, pr[e / 2]);
                    }
                }
                uint32_t w[32];
#pragma unroll
                for (int e = 0; e < HALF / 2; ++e) w[e] = Pair<E>::pack(ds[e].x, ds[e].y);
                tmem_st32_nowait(tp, w);
                tmem_wait_st();
            }
            fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&s_b[i & 1]));
                if (KEYS) mbar_arrive(smem_u32(&s_rfree[i & 1]));
            }
        }
        if (!KEYS && dry > 0 && !corrected) bar_or(3, 256, true);       // a wait gave up: whoever waits for this warp goes on
        if (ok) ok = wait_warp(smem_u32(&s_end), 0);
        if (!ok && lane == 0) give_up();
        // ---- the sums: keys: the first group writes dk, the second dv; queries: half of dq's columns each.  Rounded once, rows by way of
        // shared memory (the own rows are no longer needed), the sinks' in fp32 into the workspace
        if (!right && lane == 0) record_status(&g_window_back_status, KDA_ERR_INVALID_ARG);
        if (ok && right) {
            constexpr int COLS = KEYS ? D : D / 2, CH = COLS / 8, RPI = 32 / CH, SWZ = CH < 8 ? CH - 1 : 7;
            fence_after();
            const float mul = KEYS && x == 1 ? (F16 ? 0x1p-10f : 1.f) : p.scale / factor;
            unsigned char *const stage = basep + L::X + x * L::T_BYTES;
            const int keep = KEYS && has_sinks && x0 == 0 ? min(p.S, rows) : 0;      // rows that go into the workspace
            float *const part = sinks ? k.rest + ((static_cast<int64_t>(slot) * p.Hk + head) * 2 + x) * p.S * D
                                      : k.first + ((static_cast<int64_t>(at.seq) * p.Hk + head) * 2 + x) * p.S * D;
#pragma unroll
            for (int c = 0; c < COLS / 32; ++c) {
                uint32_t v[32];
                tmem_ld32_nowait(tmem + lanes + TM_ACC + x * COLS + c * 32, v);
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
                    *reinterpret_cast<uint4 *>(stage + r * (2 * COLS) + (((c * 4 + q) ^ (r & SWZ)) << 4)) = y;
                }
            }
            __syncwarp();
            if (!sinks) {
                const int ch = lane % CH;
                const int64_t ld = KEYS && x == 1 ? ld2 : ld1;
                E *const dst = (KEYS && x == 1 ? out2 : out1) + (static_cast<int64_t>(at.start) + x0) * ld + head * D + (KEYS ? 0 : x * COLS) + ch * 8;
#pragma unroll
                for (int j = 0; j < 32; j += RPI) {
                    const int row = (warp & 3) * 32 + j + lane / CH;
                    if (row >= keep && row < rows)
                        *reinterpret_cast<uint4 *>(dst + row * ld) = *reinterpret_cast<const uint4 *>(stage + row * (2 * COLS) + ((ch ^ (row & SWZ)) << 4));
                }
            }
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    grid_dep_launch();
    if (warp == 0) {
        if (s_abort && lane == 0) {     // the copies in flight end before the memory is given back
            mbar_wait(smem_u32(&s_x), 0);
            for (int i = 0; i < L::N1 && i < fetched[0]; ++i) mbar_wait(smem_u32(&s_y1[i]), ((fetched[0] - 1 - i) / L::N1) & 1);
            for (int i = 0; i < L::N2 && i < fetched[1]; ++i) mbar_wait(smem_u32(&s_y2[i]), ((fetched[1] - 1 - i) / L::N2) & 1);
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
    const int64_t n = static_cast<int64_t>(p.T) * heads;
    constexpr int U = 4, ROWS = 32 / LANES;                  // steps in flight, rows of a warp's step
    const int64_t warps = static_cast<int64_t>(gridDim.x) * blockDim.x / 32;
    for (int64_t first = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / 32 * ROWS; first < n; first += U * warps * ROWS) {
        uint4 a[U], b[U];
        int64_t t[U];
        int h[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = first + u * warps * ROWS + lane / LANES;
            t[u] = row / heads;
            h[u] = row < n ? static_cast<int>(row - t[u] * heads) : -1;
            a[u] = b[u] = make_uint4(0, 0, 0, 0);
            if (h[u] >= p.H) {
                a[u] = b[u] = *reinterpret_cast<const uint4 *>(v + t[u] * ldv + (h[u] - p.H) * D + l * 8);
            } else if (h[u] >= 0) {
                a[u] = *reinterpret_cast<const uint4 *>(d_o + t[u] * lddo + h[u] * D + l * 8);
                b[u] = *reinterpret_cast<const uint4 *>(o + t[u] * ldo + h[u] * D + l * 8);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const E *const x = reinterpret_cast<const E *>(&a[u]), *const y = reinterpret_cast<const E *>(&b[u]);
            float dot = 0.f, sq = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float w = to_f32(x[j]);
                dot = fmaf(w, to_f32(y[j]), dot);
                if (!Pair<E>::BF16) sq = fmaf(w, w, sq);
            }
#pragma unroll
            for (int m = LANES / 2; m; m >>= 1) {
                dot += __shfl_xor_sync(0xffffffffu, dot, m);
                if (!Pair<E>::BF16) sq += __shfl_xor_sync(0xffffffffu, sq, m);
            }
            if (l == 0 && h[u] >= 0) {
                if (h[u] < p.H) k.delta[static_cast<int64_t>(h[u]) * p.T + t[u]] = dot;
                if (!Pair<E>::BF16 && isfinite(sq)) {      // numbers above zero compare as their bits do
                    int *const to = reinterpret_cast<int *>(k.most) + (h[u] < p.H ? h[u] / (p.H / p.Hk) : p.Hk + h[u] - p.H);
                    const int bits = __float_as_int(sqrtf(sq));
                    if (bits > *static_cast<volatile int *>(to)) atomicMax(to, bits);
                }
            }
        }
    }
    grid_dep_launch();
}

// The sinks' rows of dk and dv: the window's part and the pieces', in order.
template <typename E>
__global__ void __launch_bounds__(128) window_sinks(const Shape p, const Back k, int D, E *dk, int64_t lddk, E *dv, int64_t lddv)
{
    grid_dep_wait();
    if (!plan_matches(p.plan, p.sig)) return;
    const int32_t *cu = p.plan + p.off_cu;
    const int seq = blockIdx.x / p.Hk, head = blockIdx.x % p.Hk, start = cu[seq], len = cu[seq + 1] - start;
    if (len <= p.W) return;
    const int keep = min(p.S, len), slot0 = start / CHUNK + seq;
    const int64_t size = static_cast<int64_t>(p.S) * D, step = static_cast<int64_t>(p.Hk) * 2 * size;
    for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < 2 * keep * D; i += gridDim.y * blockDim.x) {
        const int x = i / (keep * D), e = i - x * keep * D;
        float sum = k.first[((static_cast<int64_t>(seq) * p.Hk + head) * 2 + x) * size + e];
        const float *const rest = k.rest + ((static_cast<int64_t>(slot0) * p.Hk + head) * 2 + x) * size + e;
        const int last = (len - 1) / CHUNK;
#pragma unroll 8
        for (int c = p.W / CHUNK; c <= last; ++c) sum += rest[c * step];
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
    CUtensorMap mq, mdo, mk, mv;
    if (!encode_heads(&mq, in.q, bf16, D, p.H, p.T, in.ldq, TILE) || !encode_heads(&mdo, g.d_o, bf16, D, p.H, p.T, g.lddo, TILE) ||
        !encode_heads(&mk, in.k, bf16, D, p.Hk, p.T, in.ldk, TILE) || !encode_heads(&mv, in.v, bf16, D, p.Hk, p.T, in.ldv, TILE))
        return cudaErrorInvalidValue;
    cudaError_t e;
    if (!bf16 && (e = cudaMemsetAsync(k.most, 0, static_cast<size_t>(2) * p.Hk * 4, stream)) != cudaSuccess) return e;
    const int64_t rows = static_cast<int64_t>(p.T) * (p.H + (bf16 ? 0 : p.Hk)) * (D / 8);
    const int grid = static_cast<int>(min((rows + 1023) / 1024, static_cast<int64_t>(sm_count()) * 8));
    window_delta<E, D><<<grid, 256, 0, stream>>>(p, static_cast<const E *>(g.o), g.ldo, static_cast<const E *>(g.d_o), g.lddo,
                                                 static_cast<const E *>(in.v), in.ldv, k);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const void *fk = reinterpret_cast<const void *>(&window_back<E, D, true>), *fq = reinterpret_cast<const void *>(&window_back<E, D, false>);
    if ((e = set_dynamic_smem(fk, Smem<D>::BYTES)) != cudaSuccess || (e = set_dynamic_smem(fq, Smem<D>::BYTES)) != cudaSuccess) return e;
    // each of the others begins while the last CTAs of the one before it end
    e = launch_dependent(window_back<E, D, false>, dim3(static_cast<unsigned>(slots * p.H)), dim3(THREADS), Smem<D>::BYTES, stream, mq, mdo, mk, mv, p, k,
                         static_cast<E *>(g.dq), g.lddq, static_cast<E *>(nullptr), static_cast<int64_t>(0));
    if (e != cudaSuccess) return e;
    e = launch_dependent(window_back<E, D, true>, dim3(static_cast<unsigned>(slots * p.Hk + pieces)), dim3(THREADS), Smem<D>::BYTES, stream, mk, mv, mq,
                         mdo, p, k, static_cast<E *>(g.dk), g.lddk, static_cast<E *>(g.dv), g.lddv);
    if (e != cudaSuccess || !sinks) return e;
    const unsigned share = static_cast<unsigned>(min(16, (2 * p.S * D + 127) / 128));      // blocks of a sequence and head
    return launch_dependent(window_sinks<E>, dim3(p.N * p.Hk, share), dim3(128), 0, stream, p, k, D, static_cast<E *>(g.dk), g.lddk,
                            static_cast<E *>(g.dv), g.lddv);
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
