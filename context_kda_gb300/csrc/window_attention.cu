// Attention over a sliding window with sinks, forward: o = softmax(scale q k^T) v over the visible keys, one pass over the
// keys with the running maximum and sum of every row.
//
// A CTA works two tiles of 128 query rows against the same tiles of keys: two heads that share a key head, or else two
// neighbouring tiles of one head.  Warp 0 fetches (TMA), warp 1 issues the products (tcgen05), warp 2 looks after the
// values (below), and four warps a row tile do its softmax, a thread a row.  Scores S = Q K^T lie in
// TMEM; a row's probabilities take the scores' place there as the A operand of O += P V.  While one row tile's
// probabilities are computed, the tensor cores work for the other.  They take the next product hardly before
// the last is done, so whatever the issuing warp waits for stands still: it waits for probabilities only, and warp 2 adds
// its arrival to theirs once the tile's values and the next keys are there.  One warp issues for both row tiles in turn; two
// warps that issue as they can drift into step, and both row tiles' softmax then meets idle tensor cores (329 us for 261).
// A row's maximum is followed lazily (a published method for this hardware, as two row tiles in turn are): O is multiplied up only when
// the maximum has grown by more than 2^8 since, which fp32 sums and 16-bit probabilities hold easily; the diagonal tile comes
// first, so that there always is a maximum (minus infinity where a row's scores are).
// Probabilities are rounded to the activations' type (half a step of it relative, as the output itself); their sum is kept in fp32 from
// the values before rounding.  fp16 has no numbers below 2^-24, and very many small probabilities count: there they are kept
// times 2^7, each off by half a step or 2^-32 of the row's largest.
// Bound by the tensor cores' issue where much is visible: 8192 tokens x 16 heads (4 key heads) of 128, all visible, 201 us, 73 % of the dense
// bf16 rate counted over visible pairs; by the way in and out of a CTA where little is: 32768 tokens in 24 sequences, window 1024, 258 us
// (38 %); 1024 x 8 heads 19 us.
//
// Values behind a masked place are multiplied by a probability of zero, which an infinity or NaN would survive.  Warp 2
// therefore looks through the value tiles that some row sees only a part of, puts zeros in the place of such values (and of the rows
// behind the sequence's end) and leaves a mark; the rows that do see one add it at the end, from memory.
#include "window_attention.cuh"

namespace kda {
namespace {

using namespace attn;

__device__ int g_window_status;

constexpr int THREADS = 384;
constexpr int REGS_OTHER = 72, REGS_SOFTMAX = 216;     // of 168 at the launch: 128 x 72 + 256 x 216 = 384 x 168
constexpr float LAZY = 8.f;               // growth of a row's maximum, in powers of two, that O is not corrected for
constexpr float F16_EXP = 7.f;            // 2^LAZY times that is 2^15, fp16's last power of two
constexpr float FAR = 65536.f;            // exponents that are not made from products of their own: off by 2^-8 at most below

template <int D> struct Smem {
    static constexpr uint32_t T_BYTES = D / 64 * BOX;
    static constexpr int KS = D == 128 ? 3 : 4, VS = D == 128 ? 2 : 4;
    static constexpr uint32_t Q = 0, K = 2 * T_BYTES, V = K + KS * T_BYTES, BYTES = V + VS * T_BYTES, ALLOC = BYTES + 1024;
    static_assert(ALLOC + 2048 <= 227 * 1024, "shared memory");      // with the static part
};

// TMEM columns: scores (probabilities in their first half), outputs
constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;

// What the roles know of a CTA's work: its row tiles x = 0, 1 and the key tiles, from the diagonal down, the sinks' last.
struct Rows {
    int count, t0, head;                  // rows that exist, first row in the sequence
    int lo, hi;                           // key tiles of the window; none: lo > hi
    bool sink;
};
struct Tiles {
    int top, n_win, n;                    // highest key tile, tiles of the windows, all tiles

    __device__ __forceinline__ bool is_sink(int i) const { return i >= n_win; }
    __device__ __forceinline__ int tile(int i) const { return i < n_win ? top - i : 0; }
    __device__ __forceinline__ bool active(const Rows &x, int i) const { return is_sink(i) ? x.sink : tile(i) >= x.lo && tile(i) <= x.hi; }
    // Keys [a, b] of tile i that row r of x sees.
    __device__ __forceinline__ void visible(const Rows &x, int i, int r, int W, int S, int &a, int &b) const
    {
        const int row = x.t0 + r, j0 = tile(i) * TILE;
        a = is_sink(i) ? 0 : max(0, row - W + 1 - j0);           // (row - W is above -2^31)
        b = is_sink(i) ? min(S - 1, row - W) : min(TILE - 1, row - j0);
    }
    // Whether some row of x sees only a part of tile i, or the tile passes the sequence's end.
    __device__ __forceinline__ bool masked(const Rows &x, int i, int len, int W) const
    {
        const int j0 = tile(i) * TILE;
        return is_sink(i) || j0 + TILE - 1 > x.t0 || j0 < x.t0 + TILE - W || j0 + TILE > len;
    }
};

template <typename E, int D>
__global__ void __launch_bounds__(THREADS, 1)
    window_forward(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                   const Shape p, bool two_heads, const E *v_rows, int64_t ldv, E *o, int64_t ldo, float *lse)
{
    using L = Smem<D>;
    constexpr float P_EXP = Pair<E>::BF16 ? 0.f : F16_EXP;      // probabilities are kept times 2^P_EXP
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t s_q, s_kfull[L::KS], s_kfree[L::KS], s_vfull[L::VS], s_vfree[L::VS], s_s[2], s_p[2], s_o[2], s_end;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) prefetch_map(mq), prefetch_map(mk), prefetch_map(mv);
    // A device plan of another launch: nothing is written.  Where the starts come with the launch nothing depends on it before.
    const bool right = plan_matches(p.plan, p.sig);
    if (p.N > FEW && !right) {
        if (tid == 0 && blockIdx.x == 0) record_status(&g_window_status, KDA_ERR_INVALID_ARG);
        return;
    }
    Place at;
    const int works = two_heads ? p.H / 2 : p.H, slot = (gridDim.x - 1 - blockIdx.x) / works, work = (gridDim.x - 1 - blockIdx.x) % works;
    if (!find_tile(p, slot, two_heads ? 7 : 8, at)) return;      // the last rows of a sequence, which see the most, come first
    auto make_rows = [&](int x) {
        Rows y;
        y.head = two_heads ? 2 * work + x : work;
        y.t0 = at.t0 + (two_heads ? 0 : x * TILE);
        y.count = min(TILE, at.len - y.t0);
        y.hi = y.count > 0 ? y.t0 / TILE : -1;
        y.lo = max(0, y.t0 - p.W + 1) / TILE;
        y.sink = y.count > 0 && p.S > 0 && y.t0 + y.count - 1 >= p.W;
        return y;
    };
    const Rows x0 = make_rows(0), x1 = make_rows(1);
    Tiles w;
    w.top = max(x0.hi, x1.hi);
    w.n_win = w.top - x0.lo + 1;
    w.n = w.n_win + (x0.sink || x1.sink);
    const int hk = x0.head / (p.H / p.Hk);
    auto look_after = [&](int i) {        // tile i's values
        return (w.active(x0, i) && w.masked(x0, i, at.len, p.W)) || (w.active(x1, i) && w.masked(x1, i, at.len, p.W));
    };

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *const basep = smem_raw + (base - smem_u32(smem_raw));
    int fetched[2] = {0, 0};              // (the fetching thread) tiles of keys and of values
    auto load = [&](const CUtensorMap &m, uint32_t dst, int head, int row, uint32_t bar) {
        for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * BOX, &m, c * 64, head, at.start + row, bar);
    };
    auto fetch = [&](const CUtensorMap &m, uint32_t to, int i, uint64_t &full) {      // tile i of keys or values
        mbar_arrive_expect_tx(smem_u32(&full), L::T_BYTES);
        load(m, base + to, hk, w.tile(i) * TILE, smem_u32(&full));
    };
    if (tid == 0) {
        mbar_init(smem_u32(&s_q), 1);
        for (int i = 0; i < L::KS; ++i) mbar_init(smem_u32(&s_kfull[i]), 1), mbar_init(smem_u32(&s_kfree[i]), 1);
        for (int i = 0; i < L::VS; ++i) mbar_init(smem_u32(&s_vfull[i]), 1), mbar_init(smem_u32(&s_vfree[i]), 1);
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_u32(&s_s[x]), 1);
            mbar_init(smem_u32(&s_p[x]), 5);
            mbar_init(smem_u32(&s_o[x]), 1);
        }
        mbar_init(smem_u32(&s_end), 1);
        s_abort = 0;
        s_bad = 0;
        // the first tiles are on their way before anything else
        const uint32_t bq = smem_u32(&s_q);
        mbar_arrive_expect_tx(bq, (x1.count > 0 ? 2 : 1) * L::T_BYTES);
        load(mq, base + L::Q, x0.head, x0.t0, bq);
        fetch(mk, L::K, 0, s_kfull[0]);
        if (x1.count > 0) load(mq, base + L::Q + L::T_BYTES, x1.head, x1.t0, bq);
        fetch(mv, L::V, 0, s_vfull[0]);
        fetched[0] = fetched[1] = 1;
    }
    if (warp == 0) tmem_alloc(smem_u32(&s_tmem), TM_COLS);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem;
    volatile int *const abort_flag = &s_abort;
    auto give_up = [&] {
        record_status(&g_window_status, KDA_ERR_TIMEOUT);
        *abort_flag = 1;
    };

    if (warp < 4) fewer_registers<REGS_OTHER>();
    if (warp == 0) {
        // ---- fetch
        if (lane == 0) {
            bool ok = true;
            for (int i = 1; i <= w.n; ++i) {             // keys a tile ahead of the values
                if (i < w.n) {
                    const int s = i % L::KS;
                    if (i >= L::KS) ok = wait_thread(smem_u32(&s_kfree[s]), (i / L::KS - 1) & 1);
                    if (!ok) break;
                    fetch(mk, L::K + s * L::T_BYTES, i, s_kfull[s]);
                    ++fetched[0];
                }
                if (i > 1) {
                    const int s = (i - 1) % L::VS;
                    if (i - 1 >= L::VS) ok = wait_thread(smem_u32(&s_vfree[s]), ((i - 1) / L::VS - 1) & 1);
                    if (!ok) break;
                    fetch(mv, L::V + s * L::T_BYTES, i - 1, s_vfull[s]);
                    ++fetched[1];
                }
            }
            if (!ok) give_up();
        }
    } else if (warp == 1) {
        // ---- products.  TMEM addresses start at 0: the CTA has all of it
        constexpr uint32_t ID_S = idesc<E>(TILE, TILE, 0), ID_O = idesc<E>(TILE, D, 1);
        auto scores = [&](int x, int stage, bool last) {      // last: of this tile of keys
            const uint32_t qd = desc_k(base + L::Q + x * L::T_BYTES), kd = desc_k(base + L::K + stage * L::T_BYTES);
            if (elect()) {
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t off = ((s / 4) * BOX + (s % 4) * 32) >> 4;
                    product(TM_S + x * 128, qd + off, kd + off, ID_S, s > 0);
                }
                commit(smem_u32(&s_s[x]));
                if (last) commit(smem_u32(&s_kfree[stage]));
            }
            __syncwarp();
        };
        auto signal = [&](uint64_t &bar) {
            if (elect()) commit(smem_u32(&bar));
            __syncwarp();
        };
        bool ok = wait_warp(smem_u32(&s_q), 0) && wait_warp(smem_u32(&s_kfull[0]), 0);
        if (ok) {
            fence_after();
            if (w.active(x0, 0)) scores(0, 0, !w.active(x1, 0));
            if (w.active(x1, 0)) scores(1, 0, true);
        }
        int ks = 1 % L::KS, kp = 1 / L::KS & 1, vs = 0;      // stage (and parity) of the next keys and values
        int done[2] = {0, 0};
        for (int i = 0; i < w.n && ok; ++i) {
            const bool more = i + 1 < w.n;
            // of the sinks' tile only the rows that hold sinks
            const int steps = w.is_sink(i) ? (p.S + 15) / 16 : TILE / 16;
            const uint32_t vd = desc_mn(base + L::V + vs * L::T_BYTES, BOX);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const Rows &rows = x ? x1 : x0;
                const bool next = more && w.active(rows, i + 1);
                // the last of the two that work a tile gives its stage back
                const bool last = x == 1 || !w.active(x1, i), last_next = x == 1 || !(more && w.active(x1, i + 1));
                if (w.active(rows, i)) {
                    ok = ok && wait_warp(smem_u32(&s_p[x]), done[x] & 1);
                    if (!ok) continue;
                    fence_after();
                    if (elect()) {
#pragma unroll
                        for (int s = 0; s < TILE / 16; ++s)
                            if (s < steps) product_ta(TM_O + x * D, TM_S + x * 128 + s * 8, vd + s * (2048 >> 4), ID_O, done[x] > 0 || s > 0);
                        if (last) commit(smem_u32(&s_vfree[vs]));
                    }
                    __syncwarp();
                    ++done[x];
                } else if (next) {
                    ok = ok && wait_warp(smem_u32(&s_kfull[ks]), kp);
                    fence_after();
                }
                if (ok && next) scores(x, ks, last_next);
            }
            if (!ok) break;
            if (++vs == L::VS) vs = 0;
            if (++ks == L::KS) ks = 0, kp ^= 1;
        }
        if (ok) {
            signal(s_o[0]);
            signal(s_o[1]);
        } else {
            if (lane == 0) give_up();
            signal(s_end);                     // the products in flight end before the memory is given back
            wait_warp(smem_u32(&s_end), 0);
        }
    } else if (warp == 2) {
        // ---- values behind masked places; tells the products that a tile's values and the next keys are there
        bool ok = true;
        int seen[2] = {0, 0};
        auto there = [&](int i) {
            if (i + 1 < w.n) ok = wait_warp(smem_u32(&s_kfull[(i + 1) % L::KS]), ((i + 1) / L::KS) & 1);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (!ok || !w.active(x ? x1 : x0, i)) continue;
                ok = wait_warp(smem_u32(&s_s[x]), seen[x]++ & 1);     // the last round's arrivals are complete
                if (ok && lane == 0) mbar_arrive(smem_u32(&s_p[x]));
            }
        };
        for (int i = 0; i < w.n && ok; ++i) {
            ok = wait_warp(smem_u32(&s_vfull[i % L::VS]), (i / L::VS) & 1);
            if (!ok) break;
            if (!look_after(i)) {
                there(i);
                continue;
            }
            unsigned char *const v = basep + L::V + (i % L::VS) * L::T_BYTES;
            const int real = at.len - w.tile(i) * TILE;     // rows of the sequence
            // times zero, added up: NaN where one is infinite or NaN
            uint4 *const mine = reinterpret_cast<uint4 *>(v + (lane / 8) * 128 + (lane & 7) * 16);
            uint32_t sum[4] = {0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll 8
                for (int r = 0; r < 32; ++r) {
                    const uint4 x = mine[c * (BOX / 16) + r * 32];
                    sum[0] = Pair<E>::times_zero(x.x, sum[0]);
                    sum[1] = Pair<E>::times_zero(x.y, sum[1]);
                    sum[2] = Pair<E>::times_zero(x.z, sum[2]);
                    sum[3] = Pair<E>::times_zero(x.w, sum[3]);
                }
            bool bad = ((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7FFF7FFFu) != 0;
            if (__any_sync(0xffffffffu, bad) || real < TILE) {
                constexpr uint32_t INF = Pair<E>::INF;
                bad = false;
#pragma unroll 1
                for (int i = 0; i < D / 64 * 32; ++i) {
                    const int r = i % 32;
                    uint4 x = mine[i / 32 * (BOX / 16) + r * 32];
                    uint32_t *const e = reinterpret_cast<uint32_t *>(&x);
                    bool hit = false;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t lo = (e[j] & INF) == INF ? 0xFFFFu : 0u, hi = (e[j] & (INF << 16)) == (INF << 16) ? 0xFFFF0000u : 0u;
                        hit |= (lo | hi) != 0;
                        e[j] &= ~(lo | hi);
                    }
                    if (r * 4 + lane / 8 >= real) mine[i / 32 * (BOX / 16) + r * 32] = make_uint4(0, 0, 0, 0);
                    else if (hit) mine[i / 32 * (BOX / 16) + r * 32] = x, bad = true;
                }
                bad = __any_sync(0xffffffffu, bad);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0 && bad) {
                *static_cast<volatile int *>(&s_bad) = 1;
                __threadfence_block();
            }
            there(i);
        }
        if (!ok && lane == 0) give_up();
    } else if (warp > 3) {
        // ---- softmax, a thread a row
        more_registers<REGS_SOFTMAX>();
        const int x = (warp >> 2) - 1, r = (warp & 3) * 32 + lane;
        const Rows rows = make_rows(x);
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + TM_S + x * 128, to = tmem + lanes + TM_O + x * D;
        float m = -INFINITY, sum = 0.f;      // the row's maximum (of the scores) and sum of probabilities
        int n = 0;
        bool ok = true;
        for (int i = 0; i < w.n; ++i) {
            if (!w.active(rows, i)) continue;
            ok = wait_warp(smem_u32(&s_s[x]), n & 1);
            if (!ok) break;
            fence_after();
            uint32_t u[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32_nowait(ts + c * 32, u[c]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 4; ++c) reg_fence32(u[c]);
            if (w.masked(rows, i, at.len, p.W)) {
                int a, b;
                w.visible(rows, i, r, p.W, p.S, a, b);
                if (__any_sync(0xffffffffu, a > 0)) {
#pragma unroll
                    for (int j = 0; j < TILE; ++j)
                        if (j < a) u[j / 32][j % 32] = 0xFF800000u;
                }
#pragma unroll
                for (int j = 0; j < TILE; ++j)
                    if (j > b) u[j / 32][j % 32] = 0xFF800000u;
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < 32; j += 2)
#pragma unroll
                for (int c = 0; c < 4; ++c) top[c] = max3(top[c], __uint_as_float(u[c][j]), __uint_as_float(u[c][j + 1]));
            const float new_m = max3(m, fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            // each row by its own growth, whatever the warp's others do: rows share a warp with other sequences' too
            const bool grown = (new_m - m) * p.c > LAZY;
            if (n == 0) {
                m = new_m;
            } else if (__any_sync(0xffffffffu, grown)) {
                // the products before this tile's scores are complete, O among them
                const float f = grown ? ex2_ftz((m - new_m) * p.c) : 1.f;
                m = grown ? new_m : m;
                sum *= f;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t t[32];
                    tmem_ld32_nowait(to + c * 32, t);
                    tmem_wait_ld();
                    reg_fence32(t);
#pragma unroll
                    for (int j = 0; j < 32; ++j) t[j] = __float_as_uint(__uint_as_float(t[j]) * f);
                    tmem_st32_nowait(to + c * 32, t);
                }
            }
            // Exponents (s - m) c come as s c - m c in one instruction, off by half a step of m c for all of the row, which cancels; where m c
            // is far from zero, so that this would pass fp32's range (2^32) or fp16's, the difference is taken first.  (So it is
            // where all scores have been minus infinity: probabilities of zero.)
            const bool far = fabsf(m * p.c) > FAR;
            if (__any_sync(0xffffffffu, far)) {
                const float less = far && m != -INFINITY ? m : 0.f;
#pragma unroll
                for (int j = 0; j < TILE; ++j) u[j / 32][j % 32] = __float_as_uint(__uint_as_float(u[j / 32][j % 32]) - less);
            }
            const float off = far ? P_EXP : fmaf(-m, p.c, P_EXP);
            const float2 cc = make_float2(p.c, p.c), mc = make_float2(off, off);
            float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t e[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const int k = h * 64 + 2 * j;
                    float2 v = fma2(make_float2(__uint_as_float(u[k / 32][k % 32]), __uint_as_float(u[k / 32][k % 32 + 1])), cc, mc);
                    v.x = ex2_ftz(v.x);
                    v.y = ex2_ftz(v.y);
                    s2[j & 1] = add2(s2[j & 1], v);
                    e[j] = Pair<E>::pack(v.x, v.y);
                }
                tmem_st32_nowait(ts + h * 32, e);
            }
            tmem_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s_p[x]));
            sum += (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
            ++n;
        }
        if (ok && n > 0) ok = wait_warp(smem_u32(&s_o[x]), 0);
        if (!ok && lane == 0) give_up();
        if (ok && n > 0) {
            fence_after();
            const int64_t token = at.start + rows.t0 + r;
            const bool real = r < rows.count && right;
            if (!right && lane == 0) record_status(&g_window_status, KDA_ERR_INVALID_ARG);
            if (lse && real) lse[static_cast<int64_t>(rows.head) * p.T + token] = fmaf(m, p.c, log2f(sum) - P_EXP) * 0.69314718055994530942f;
            const float inv = 1.f / sum;
            const int bad = *static_cast<volatile int *>(&s_bad);
            unsigned char *const out = basep + L::Q + x * L::T_BYTES;      // the queries are no longer needed: rows of D, chunks swizzled
            uint32_t t[D / 32][32];
#pragma unroll
            for (int c = 0; c < D / 32; ++c) tmem_ld32_nowait(to + c * 32, t[c]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) reg_fence32(t[c]);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                float f[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(t[c][j]) * inv;
                if (bad && real) {
                    // values that are infinite or NaN: what the row sees of them
                    for (int i = 0; i < w.n; ++i) {
                        if (!w.active(rows, i)) continue;
                        int a, b;
                        w.visible(rows, i, r, p.W, p.S, a, b);
                        for (int j = a; j <= b; ++j) {
                            const E *const v = v_rows + (at.start + w.tile(i) * TILE + j) * ldv + hk * D + c * 32;
#pragma unroll
                            for (int q = 0; q < 32; ++q) {
                                const float val = to_f32(v[q]);
                                if (!isfinite(val)) f[q] += val;
                            }
                        }
                    }
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int chunk = c * 4 + q;
                    uint4 y;
                    y.x = Pair<E>::pack(f[8 * q], f[8 * q + 1]);
                    y.y = Pair<E>::pack(f[8 * q + 2], f[8 * q + 3]);
                    y.z = Pair<E>::pack(f[8 * q + 4], f[8 * q + 5]);
                    y.w = Pair<E>::pack(f[8 * q + 6], f[8 * q + 7]);
                    *reinterpret_cast<uint4 *>(out + r * (2 * D) + ((chunk ^ (r & 7)) << 4)) = y;
                }
            }
            __syncwarp();
            constexpr int CH = D / 8, RPI = 32 / CH;     // 16-byte pieces of a row, rows of one store of the warp
            const int r0 = (warp & 3) * 32, ch = lane % CH;
            E *const dst = o + (static_cast<int64_t>(at.start) + rows.t0) * ldo + rows.head * D + ch * 8;
#pragma unroll
            for (int k = 0; k < 32; k += RPI) {
                const int row = r0 + k + lane / CH;
                if (row < rows.count && right)
                    *reinterpret_cast<uint4 *>(dst + row * ldo) = *reinterpret_cast<const uint4 *>(out + row * (2 * D) + ((ch ^ (row & 7)) << 4));
            }
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 0) {
        if (s_abort && lane == 0) {     // the copies in flight end before the memory is given back
            mbar_wait(smem_u32(&s_q), 0);
            for (int i = 0; i < L::KS && i < fetched[0]; ++i) mbar_wait(smem_u32(&s_kfull[i]), ((fetched[0] - 1 - i) / L::KS) & 1);
            for (int i = 0; i < L::VS && i < fetched[1]; ++i) mbar_wait(smem_u32(&s_vfull[i]), ((fetched[1] - 1 - i) / L::VS) & 1);
        }
        __syncwarp();
        tmem_dealloc(tmem, TM_COLS);
    }
}

template <typename E, int D>
cudaError_t forward(const Shape &p, const WindowIn &in, void *o, int64_t ldo, float *lse, cudaStream_t stream)
{
    CUtensorMap mq, mk, mv;
    const bool bf16 = Pair<E>::BF16;
    if (!encode_heads(&mq, in.q, bf16, D, p.H, p.T, in.ldq, TILE) || !encode_heads(&mk, in.k, bf16, D, p.Hk, p.T, in.ldk, TILE) ||
        !encode_heads(&mv, in.v, bf16, D, p.Hk, p.T, in.ldv, TILE))
        return cudaErrorInvalidValue;
    const void *fn = reinterpret_cast<const void *>(&window_forward<E, D>);
    const cudaError_t e = set_dynamic_smem(fn, Smem<D>::ALLOC);
    if (e != cudaSuccess) return e;
    const bool two_heads = p.H / p.Hk % 2 == 0;
    const int64_t grid = static_cast<int64_t>(two_heads ? p.H / 2 : p.H) * tile_slots(p.T, p.N, two_heads ? TILE : 2 * TILE);
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    window_forward<E, D><<<static_cast<int>(grid), THREADS, Smem<D>::ALLOC, stream>>>(mq, mk, mv, p, two_heads, static_cast<const E *>(in.v), in.ldv,
                                                                    static_cast<E *>(o), ldo, lse);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_forward(const int32_t *plan_host, const int32_t *plan_dev, int type, const WindowIn &in, void *o, int64_t ldo,
                                  float *lse, cudaStream_t stream)
{
    const Shape p = window_shape(plan_host, plan_dev, in);
    if (type == KDA_TYPE_F16)
        return in.d == 64 ? forward<__half, 64>(p, in, o, ldo, lse, stream) : forward<__half, 128>(p, in, o, ldo, lse, stream);
    return in.d == 64 ? forward<__nv_bfloat16, 64>(p, in, o, ldo, lse, stream) : forward<__nv_bfloat16, 128>(p, in, o, ldo, lse, stream);
}

int take_window_status()
{
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_window_status, sizeof(int)) != cudaSuccess) return KDA_ERR_CUDA;
    if (v != 0 && cudaMemcpyToSymbol(g_window_status, &z, sizeof(int)) != cudaSuccess) return KDA_ERR_CUDA;
    return v;
}

}  // namespace kda
