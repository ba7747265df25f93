// Gated linear recurrence over packed sequences, per channel:
//     h_t = exp(g_t) h_{t-1} + i_t x_t,   h_{-1} = h0 of the sequence,
// its gradients (the same recurrence backwards in time) and its single-token step.
//
// One pass over the data.  Over a run of tokens the recurrence is the map h -> A h + B with A the product
// of the decays and B the run's state from zero, and maps compose as (A2, B2) o (A1, B1) = (A1 A2, A2 B1 + B2);
// a run in which a sequence starts forgets what came before (h -> B, marked by A = -1: decays are not
// negative), so nothing of another sequence, infinities and NaN included, is ever multiplied in.
//   - The stream is cut into tiles of 128 tokens x C channels.  A CTA copies a tile to shared memory
//     (cp.async), each of its eight warps folds 16 tokens in registers, the warps' maps are folded in
//     shared memory, and the tile's map is published; with the tile's incoming state known, every warp
//     runs its 16 tokens again from registers and writes the results.  Inputs are read once.
//   - Up to 8 tiles of tokens ('cluster'): the CTAs of a channel range are one cluster; they exchange the
//     maps through distributed shared memory.  One launch and no workspace, for short inputs, where
//     latency counts.
//   - More ('chain'): CTAs take tiles in time order from a ticket, so that a tile waits only for tiles
//     taken before it by CTAs that run.  A tile's incoming state is folded, always in the same order,
//     from the state at its group's start and the maps of the group's earlier tiles (groups of 16
//     tiles); the group's last tile publishes the next group's state.  Only that last step is serial in time,
//     once in 2048 tokens.  Published words carry their own validity (they are all ones until written,
//     which no published value is), so that one 8-byte store and one load pass a map on.  A kernel before
//     the main one sets them, the ticket and each tile's sequence starts.
//   - Waits give up after about two seconds (KDA_ERR_TIMEOUT through kda_device_status).
//
// The backward takes the states before every 128th token that the forward saved, so a tile recomputes its
// states without waiting; its own recurrence is
//     G_t = dh_t + e_{t+1},  e_t = exp(g_t) G_t   (e_{t+1} = dfinal at the last token of a sequence),
//     dx = i G, di = x G, dg = e_t h_{t-1}, dh0 = e at the first token,
// with tiles taken from the last to the first.
#include <type_traits>

#include "elem.cuh"
#include "kda_internal.cuh"
#include "tc.cuh"

namespace kda {
namespace {

constexpr int L = KDA_SCAN_TILE;    // tokens of a tile
constexpr int THREADS = 256, WARPS = THREADS / 32, W = L / WARPS;   // W: tokens of a warp
constexpr int MIN_GROUP = 8, MAX_GROUP = 16;   // tiles of a group: see run()
constexpr int MAX_CLUSTER = 8;      // tiles that a cluster covers
constexpr int DPAD = 64;            // channels are padded to this in the workspace
constexpr long long SPIN = 4000000000LL;   // clocks of a wait: about two seconds

__device__ int g_scan_status;

// Workspace of the chain (bytes).
struct Layout {
    size_t starts, state, map, end;   // each tile's sequence starts; groups' states; tiles' maps
};
// The sequence starts of a tile: bit j: a sequence starts at its token j; 'first': the lowest such sequence.
// The end of the stream counts as the start of sequence N.
struct __align__(16) Starts {
    uint32_t bits[L / 32];
    int first, pad[3];
};
static_assert(sizeof(Starts) == 32, "two 16-byte loads");
__host__ __device__ inline int tiles_of(int T) { return (T + L - 1) / L; }
inline Layout layout_of(int64_t T, int D)
{
    const size_t nT = static_cast<size_t>(T + L - 1) / L, Dp = static_cast<size_t>(D + DPAD - 1) / DPAD * DPAD;
    auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
    Layout l;
    l.starts = 256;                                  // the ticket comes first
    l.state = up(l.starts + (nT + 1) * sizeof(Starts));
    l.map = up(l.state + (nT / MIN_GROUP + 1) * Dp * 4);
    l.end = l.map + nT * Dp * 8;
    return l;
}
struct Chain {
    int *ticket;
    Starts *starts;       // [tiles + 1]
    uint32_t *state;      // [groups][Dp], all ones until published
    uint64_t *map;        // [tiles][Dp], low word A, high word B
    int Dp, group;        // padded channels; tiles of a group
};
inline Chain chain_of(void *ws, int64_t T, int D)
{
    char *b = static_cast<char *>(ws);
    const Layout l = layout_of(T, D);
    return Chain{reinterpret_cast<int *>(b), reinterpret_cast<Starts *>(b + l.starts), reinterpret_cast<uint32_t *>(b + l.state),
                 reinterpret_cast<uint64_t *>(b + l.map), (D + DPAD - 1) / DPAD * DPAD, MAX_GROUP};
}

__global__ void __launch_bounds__(256) chain_init(const int32_t *plan, PlanSig sig, int nT, int *ticket, Starts *starts, uint4 *words,
                                                  size_t n)
{
    tc::grid_dep_launch();
    const size_t id = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x, step = static_cast<size_t>(gridDim.x) * blockDim.x;
    if (!plan_matches(plan, sig)) return;   // the main kernel records it
    for (size_t j = id; j < n; j += step) words[j] = make_uint4(~0u, ~0u, ~0u, ~0u);
    if (id == 0) *ticket = 0;
    const PlanView pv{plan};
    const int32_t *cu = pv.cu();
    const int lane = threadIdx.x & 31, N = pv.N();
    for (size_t j = id / 32; j <= static_cast<size_t>(nT); j += step / 32) {     // a warp a tile
        const int64_t t0 = static_cast<int64_t>(j) * L;
        int lo = 0, hi = N + 1;                                // first n with cu[n] >= t0 (N + 1: none)
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] < t0) lo = mid + 1;
            else hi = mid;
        }
        uint32_t mine[L / 32] = {};
        for (int k = 0; k < L / 32; ++k) {                     // at most a start a token
            const int m = lo + k * 32 + lane;
            const int64_t t = m <= N ? cu[m] - t0 : L;
#pragma unroll
            for (int w = 0; w < L / 32; ++w)
                if (t >> 5 == w) mine[w] |= 1u << (t & 31);
        }
#pragma unroll
        for (int w = 0; w < L / 32; ++w) mine[w] = __reduce_or_sync(0xffffffffu, mine[w]);
        if (lane == 0) {
            Starts st = {};
#pragma unroll
            for (int w = 0; w < L / 32; ++w) st.bits[w] = mine[w];
            st.first = lo;
            starts[j] = st;
        }
    }
}

// ---- copies of a tile --------------------------------------------------------------------------------

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp16_all(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Tokens t0.. (zeros from T on), channels c0.. (zeros from D on) of a tensor of rows into [L][C].  WIDE:
// every row starts on 16 bytes; otherwise 4-byte elements are copied one by one and 2-byte elements pass
// through registers.
template <typename X, int C, bool WIDE>
__device__ __forceinline__ void fill(X *dst, const X *src, int64_t ld, int t0, int T, int c0, int D)
{
    if constexpr (WIDE) {
        constexpr int EPC = 16 / sizeof(X), CPR = C / EPC, STEP = THREADS / CPR;   // per copy, per row; rows per step
        const int row = threadIdx.x / CPR, ch = threadIdx.x % CPR;
        const int left = (D - c0 - ch * EPC) * static_cast<int>(sizeof(X));
        const int bytes = left < 0 ? 0 : left > 16 ? 16 : left;
        const X *p = src + (t0 + row) * ld + c0 + ch * EPC;
        const uint32_t s = tc::smem_u32(dst + row * C + ch * EPC);
        if (t0 + L <= T && c0 + C <= D) {
            const int64_t hop = STEP * ld;
#pragma unroll
            for (int k = 0; k < L / STEP; ++k) {
                cp16_all(s + k * STEP * C * sizeof(X), p);
                p += hop;
            }
            return;
        }
#pragma unroll 4
        for (int k = 0; k < L / STEP; ++k) {
            const bool in = t0 + row + k * STEP < T && bytes > 0;
            cp16(s + k * STEP * C * sizeof(X), in ? p + k * STEP * ld : src, in ? bytes : 0);
        }
    } else {
        constexpr int STEP = THREADS / C;
        const int row = threadIdx.x / C, c = threadIdx.x % C;
        const X *p = src + (t0 + row) * ld + c0 + c;
        X *s = dst + row * C + c;
        const bool col = c0 + c < D;
        if constexpr (sizeof(X) == 4) {
            for (int k = 0; k < L / STEP; ++k) {
                const bool in = col && t0 + row + k * STEP < T;
                cp4(tc::smem_u32(s + k * STEP * C), in ? p + k * STEP * ld : src, in ? 4 : 0);
            }
        } else {
#pragma unroll 16
            for (int k = 0; k < L / STEP; ++k)
                s[k * STEP * C] = col && t0 + row + k * STEP < T ? p[k * STEP * ld] : from_f32<X>(0.f);
        }
    }
}

// ---- channels of a lane --------------------------------------------------------------------------------
// V = C / 32 channels a lane: adjacent ones when copies are wide (pairs are loaded and stored as one),
// 32 apart otherwise (single elements of a warp are adjacent).
template <int V, bool WIDE> __device__ __forceinline__ int chan(int lane, int v) { return WIDE ? lane * V + v : lane + 32 * v; }

template <int V, bool WIDE> __device__ __forceinline__ void get(const float *row, int lane, float (&o)[V])
{
    if constexpr (V == 2 && WIDE) {
        const float2 p = reinterpret_cast<const float2 *>(row)[lane];
        o[0] = p.x;
        o[1] = p.y;
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = row[chan<V, WIDE>(lane, v)];
    }
}
template <int V, bool WIDE> __device__ __forceinline__ void get(const __nv_bfloat16 *row, int lane, float (&o)[V])
{
    if constexpr (V == 2 && WIDE) {
        const uint32_t p = reinterpret_cast<const uint32_t *>(row)[lane];
        o[0] = __uint_as_float(p << 16);
        o[1] = __uint_as_float(p & 0xFFFF0000u);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = to_f32(row[chan<V, WIDE>(lane, v)]);
    }
}
template <int V, bool WIDE> __device__ __forceinline__ void get(const __half *row, int lane, float (&o)[V])
{
    if constexpr (V == 2 && WIDE) {
        const float2 p = __half22float2(reinterpret_cast<const __half2 *>(row)[lane]);
        o[0] = p.x;
        o[1] = p.y;
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = to_f32(row[chan<V, WIDE>(lane, v)]);
    }
}

__device__ __forceinline__ void put2(float *p, float a, float b) { *reinterpret_cast<float2 *>(p) = make_float2(a, b); }
__device__ __forceinline__ void put2(__half *p, float a, float b) { *reinterpret_cast<__half2 *>(p) = __floats2half2_rn(a, b); }
__device__ __forceinline__ void put2(__nv_bfloat16 *p, float a, float b)
{
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(a, b);
}
// A lane's channels of one row: 'left' channels from the row's address on exist; 'pair': rows start on pairs.
template <int V, bool WIDE, typename X>
__device__ __forceinline__ void put(X *row, int lane, const float (&o)[V], int left, bool pair)
{
    if constexpr (V == 2 && WIDE) {
        if (pair && 2 * lane + 1 < left) {
            put2(row + 2 * lane, o[0], o[1]);
            return;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (chan<V, WIDE>(lane, v) < left) row[chan<V, WIDE>(lane, v)] = from_f32<X>(o[v]);
}
// The same where all channels exist and, for two adjacent ones, rows start on pairs.
template <int V, bool WIDE, typename X> __device__ __forceinline__ void put_all(X *row, int lane, const float (&o)[V])
{
    if constexpr (V == 2 && WIDE) {
        put2(row + 2 * lane, o[0], o[1]);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) row[chan<V, WIDE>(lane, v)] = from_f32<X>(o[v]);
    }
}
template <typename X> __host__ __device__ inline bool pairs(const X *p, int64_t ld)
{
    return (reinterpret_cast<uintptr_t>(p) & (2 * sizeof(X) - 1)) == 0 && (ld & 1) == 0;
}

// exp(g) as 2^(g log2 e): the product's rounding moves the result by |g| 2^-24 relative, which is below the
// exponential's own 2^-22 for every g that leaves anything to remember.
__device__ __forceinline__ float decay(float g) { return tc::ex2_ftz(g * 1.4426950408889634f); }

// ---- maps ---------------------------------------------------------------------------------------------

// One map more: (A, B) becomes (a, b) o (A, B).
__device__ __forceinline__ void then(float &A, float &B, float a, float b)
{
    B = a < 0.f ? b : fmaf(a, B, b);
    A = a < 0.f || A < 0.f ? -1.f : A * a;
}
__device__ __forceinline__ float apply(float a, float b, float h) { return a < 0.f ? b : fmaf(a, h, b); }

// A float as a word that is not all ones (one NaN pattern gives way to another).
__device__ __forceinline__ uint32_t word(float x)
{
    const uint32_t u = __float_as_uint(x);
    return u == ~0u ? 0x7FFFFFFFu : u;
}
__device__ __forceinline__ uint64_t ld_relaxed(const uint64_t *p)
{
    uint64_t v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_relaxed(const uint32_t *p)
{
    uint32_t v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_relaxed(uint64_t *p, uint64_t v)
{
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ void st_relaxed(uint32_t *p, uint32_t v)
{
    asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// V published words of a lane; false when they did not come.
template <int V, typename U> __device__ __forceinline__ bool poll(const U *p, U (&v)[V], const int (&at)[V])
{
    const long long began = clock64();
    while (true) {
        bool all = true;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            v[j] = ld_relaxed(p + at[j]);
            all = all && v[j] != static_cast<U>(~static_cast<U>(0));
        }
        if (all) return true;
        if (clock64() - began > SPIN) return false;
    }
}

// What the tiles of a channel range pass on: shared memory of both directions.
template <int C> struct Shared {
    float2 map[WARPS][C];          // the warps' maps
    float2 before[MAX_GROUP - 1][C];       // maps of the tiles before this one (cluster: this tile's in [0])
    float state[C];                // the tile's incoming state
    int seq[L + 4];                // cluster, per token (one more than the tile's): the sequence that starts there, or -1
    int next, bad;
};

__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float2 ld_cluster(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The state that enters each warp's tokens of tile 'rt' (tiles numbered in the direction of the recurrence), from the
// warps' maps in sh.map; warps are counted in that direction too.  Warp 'last', the tile's last, does what one
// warp can: it folds the maps (each becomes that of the warps before it), passes the tile's on and folds the state
// that enters the tile, left in sh.state.  False: a wait ran out.  All threads call it, behind a barrier after the
// maps were written; meanwhile() runs once this tile's map is on its way and before others are waited for.
template <int C, int V, bool WIDE, bool CHAIN, bool REVERSE, typename Meanwhile>
__device__ __forceinline__ bool incoming(Shared<C> &sh, const Chain &ch, int rt, int col0, bool last, float (&h)[V], Meanwhile meanwhile)
{
    const int lane = threadIdx.x & 31, warp = REVERSE ? WARPS - 1 - (threadIdx.x >> 5) : threadIdx.x >> 5;
    constexpr int last_warp = WARPS - 1;
    int at[V];
#pragma unroll
    for (int v = 0; v < V; ++v) at[v] = chan<V, WIDE>(lane, v);
    float Am[V], Bm[V];
    if (warp == last_warp) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            Am[v] = 1.f;
            Bm[v] = 0.f;
        }
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float2 m = sh.map[w][at[v]];
                sh.map[w][at[v]] = make_float2(Am[v], Bm[v]);
                then(Am[v], Bm[v], m.x, m.y);
            }
    }
    if constexpr (CHAIN) {
        const int grp = rt / ch.group, pos = rt - grp * ch.group;
        if (warp == last_warp && pos < ch.group - 1 && !last) {   // the group's last tile publishes a state instead
            uint64_t *p = ch.map + static_cast<size_t>(rt) * ch.Dp + col0;
#pragma unroll
            for (int v = 0; v < V; ++v)
                st_relaxed(p + at[v], static_cast<uint64_t>(word(Bm[v])) << 32 | __float_as_uint(Am[v]));
        }
        meanwhile();
        bool ok = true;
        for (int p = warp; p < pos && ok; p += WARPS) {
            uint64_t w[V];
            ok = poll<V>(ch.map + static_cast<size_t>(grp * ch.group + p) * ch.Dp + col0, w, at);
#pragma unroll
            for (int v = 0; v < V; ++v)
                sh.before[p][at[v]] = make_float2(__uint_as_float(static_cast<uint32_t>(w[v])), __uint_as_float(static_cast<uint32_t>(w[v] >> 32)));
        }
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = 0.f;
        if (warp == last_warp && grp > 0 && ok) {
            uint32_t w[V];
            ok = poll<V>(ch.state + static_cast<size_t>(grp) * ch.Dp + col0, w, at);
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = __uint_as_float(w[v]);
        }
        if (!ok) sh.bad = 1;
        __syncthreads();
        if (sh.bad) return false;
        if (warp == last_warp) {
#pragma unroll 5
            for (int p = 0; p < pos; ++p)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float2 m = sh.before[p][at[v]];
                    h[v] = apply(m.x, m.y, h[v]);
                }
            if (pos == ch.group - 1 && !last) {
                uint32_t *p = ch.state + static_cast<size_t>(grp + 1) * ch.Dp + col0;
#pragma unroll
                for (int v = 0; v < V; ++v) st_relaxed(p + at[v], word(apply(Am[v], Bm[v], h[v])));
            }
#pragma unroll
            for (int v = 0; v < V; ++v) sh.state[at[v]] = h[v];
        }
    } else {
        if (warp == last_warp)
#pragma unroll
            for (int v = 0; v < V; ++v) sh.before[0][at[v]] = make_float2(Am[v], Bm[v]);
        cluster_arrive();
        meanwhile();
        cluster_wait();
        if (warp == last_warp) {
            float2 m[MAX_CLUSTER - 1][V];
#pragma unroll
            for (int p = 0; p < MAX_CLUSTER - 1; ++p)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    m[p][v] = p < rt ? ld_cluster(mapa(tc::smem_u32(&sh.before[0][at[v]]), p)) : make_float2(1.f, 0.f);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float s = 0.f;
#pragma unroll
                for (int p = 0; p < MAX_CLUSTER - 1; ++p) s = p < rt ? apply(m[p][v].x, m[p][v].y, s) : s;
                sh.state[at[v]] = s;
            }
        }
        cluster_arrive();   // paired with the wait at the kernel's end: no CTA leaves while its map is read
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float2 m = sh.map[warp][at[v]];
        h[v] = apply(m.x, m.y, sh.state[at[v]]);
    }
    return true;
}

// The sequence starts among a warp's tokens and the token after them: bit j of 'mask'; the start at bit j is that of
// sequence first + (number of bits below j).
struct Bounds {
    uint32_t mask;
    int first;
    __device__ __forceinline__ int64_t seq(int j) const { return first + __popc(mask & ((1u << j) - 1)); }
};
// Chain: from the tile's words and the next tile's first bit (a tile ahead of their use).
struct Words {
    uint4 bits;
    uint32_t after;
    int first;
    __device__ __forceinline__ void load(const Starts *st, int tt)
    {
        bits = *reinterpret_cast<const uint4 *>(st[tt].bits);
        first = st[tt].first;
        after = st[tt + 1].bits[0];
    }
    __device__ __forceinline__ Bounds of_warp(int warp) const
    {
        constexpr int PER = 32 / W;            // warps of a word
        const int w = warp / PER, at = warp % PER * W;
        const uint32_t b[6] = {bits.x, bits.y, bits.z, bits.w, after, 0u};
        uint32_t cur = 0, next = 0;
        int below = 0;
#pragma unroll
        for (int k = 0; k < L / 32; ++k) {
            if (k == w) cur = b[k], next = b[k + 1];
            if (k < w) below += __popc(b[k]);
        }
        Bounds r;
        r.mask = __funnelshift_r(cur, next, at) & ((2u << W) - 1);
        r.first = first + below + __popc(cur & ((1u << at) - 1));
        return r;
    }
};
static_assert(32 % W == 0 && L == 128, "whole warps a word, four words a tile");
// Cluster: the starts are marked in shared memory (seq holds -1 everywhere) and read a warp at a time.
__device__ __forceinline__ void mark_starts(int *seq, const PlanView &pv, int t0)
{
    const int32_t *cu = pv.cu();
    for (int n = threadIdx.x; n <= pv.N(); n += THREADS) {
        const int t = cu[n] - t0;
        if (t >= 0 && t <= L) seq[t] = n;
    }
}
__device__ __forceinline__ Bounds marked(const int *seq)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = lane <= W ? seq[warp * W + lane] : -1;
    Bounds r;
    r.mask = __ballot_sync(0xffffffffu, n >= 0);
    r.first = __shfl_sync(0xffffffffu, n, r.mask ? __ffs(r.mask) - 1 : 0);
    return r;
}

// The tile whose number in the direction of the recurrence is rt and whose channels start at col0.
struct Tile {
    int rt, tt, t0, col0;
};
template <int C, bool REVERSE> __device__ __forceinline__ Tile tile_of(int k, int nT, int nC)
{
    Tile t;
    t.rt = k / nC;
    t.tt = REVERSE ? nT - 1 - t.rt : t.rt;
    t.t0 = t.tt * L;
    t.col0 = (k % nC) * C;
    return t;
}

// Walks the tiles of a CTA: load(tile, part) starts the copies of a tile in two parts, work(tile, bounds, release)
// computes it; release runs within it, once part 0's copies may be overwritten, part 1's may when it is done.  work
// returns false when a wait ran out.
template <int C, bool CHAIN, bool REVERSE, typename Load, typename Work>
__device__ __forceinline__ void walk(Shared<C> &sh, const Chain &ch, const PlanView &pv, int D, Load load, Work work)
{
    const int T = pv.T(), nT = tiles_of(T), nC = (D + C - 1) / C;
    if (threadIdx.x == 0) sh.bad = 0;
    if constexpr (!CHAIN) {
        for (int j = threadIdx.x; j < L + 4; j += THREADS) sh.seq[j] = -1;
        uint32_t cs, rank;
        asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(cs));
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        const int cc = blockIdx.x / cs;
        const Tile t = tile_of<C, REVERSE>(static_cast<int>(rank) * nC + cc, nT, nC);
        const bool real = t.rt < nT;      // clusters are a power of two: some CTAs may be past the end
        if (real) {
            load(t, 0);
            load(t, 1);
        }
        __syncthreads();
        if (real) mark_starts(sh.seq, pv, t.t0);
        cp_wait();
        __syncthreads();
        if (real) {
            work(t, marked(sh.seq), [] {});
        } else {
            cluster_arrive();
            cluster_wait();
            cluster_arrive();
        }
        cluster_wait();
    } else {
        // Tickets are drawn ahead (k: in work, k2: next, then the one drawn while k is in work), so that neither the
        // draw nor a tile's starts are waited for; the second only once the first tile's copies are on their way, when
        // all CTAs have drawn their first.  A CTA works its tiles in the order drawn, so the lowest unfinished tile is
        // always in work with nothing to wait for.
        const int n = nT * nC;
        tc::grid_dep_wait();
        int drawn = 0;
        if (threadIdx.x == 0) sh.next = atomicAdd(ch.ticket, 1);
        __syncthreads();
        int k = sh.next;
        Words words = {};
        if (k < n) {
            const Tile t = tile_of<C, REVERSE>(k, nT, nC);
            load(t, 0);
            load(t, 1);
            words.load(ch.starts, t.tt);
            if (threadIdx.x == 0) drawn = atomicAdd(ch.ticket, 1);
        }
        while (k < n) {
            const Tile t = tile_of<C, REVERSE>(k, nT, nC);
            __syncthreads();                 // everyone has read 'next'
            if (threadIdx.x == 0) sh.next = drawn;
            cp_wait();
            __syncthreads();
            const int k2 = sh.next;
            const Bounds bounds = words.of_warp(threadIdx.x >> 5);
            const bool ok = work(t, bounds, [&] {
                // called behind a barrier of the CTA: the copies' buffers are free
                if (threadIdx.x == 0 && k2 < n) drawn = atomicAdd(ch.ticket, 1);
                if (k2 < n) {
                    const Tile u = tile_of<C, REVERSE>(k2, nT, nC);
                    load(u, 0);
                    words.load(ch.starts, u.tt);
                }
            });
            if (!ok) {
                cp_wait();
                if (threadIdx.x == 0) record_status(&g_scan_status, KDA_ERR_TIMEOUT);
                return;
            }
            if (k2 < n) load(tile_of<C, REVERSE>(k2, nT, nC), 1);
            k = k2;
        }
    }
}

// ---- forward --------------------------------------------------------------------------------------------

template <typename E, int C> struct __align__(16) ForwardShared {
    float g[L][C];
    E x[L][C], i[L][C];
    Shared<C> s;
};

template <typename E, int C, bool WIDE, bool CHAIN>
__global__ void __launch_bounds__(THREADS, 2) scan_forward(const int32_t *plan, PlanSig sig, int D, ScanIn in, Chain ch, void *h_,
                                                           int64_t ldh, float *final_state, float *states)
{
    constexpr int V = C / 32;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    auto &sm = *reinterpret_cast<ForwardShared<E, C> *>(smem_raw);
    if (!plan_matches(plan, sig)) {
        if (threadIdx.x == 0) record_status(&g_scan_status, KDA_ERR_INVALID_ARG);
        return;
    }
    const PlanView pv{plan};
    const int T = pv.T(), nT = tiles_of(T), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const E *x = static_cast<const E *>(in.x), *ig = static_cast<const E *>(in.i);
    E *h_out = static_cast<E *>(h_);
    const bool pair = V == 1 || !WIDE || pairs(h_out, ldh);

    auto load = [&](const Tile &t, int part) {
        if (part == 1) return;
        fill<E, C, WIDE>(&sm.x[0][0], x, in.ldx, t.t0, T, t.col0, D);
        if (ig) fill<E, C, WIDE>(&sm.i[0][0], ig, in.ldi, t.t0, T, t.col0, D);
        fill<float, C, WIDE>(&sm.g[0][0], in.g, in.ldg, t.t0, T, t.col0, D);
    };
    auto work = [&](const Tile &t, const Bounds &bounds, auto release) {
        const int r0 = warp * W, left = D - t.col0;
        float a[W][V], u[W][V];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float gv[V];
            get<V, WIDE>(sm.g[r0 + j], lane, gv);
            get<V, WIDE>(sm.x[r0 + j], lane, u[j]);
#pragma unroll
            for (int v = 0; v < V; ++v) a[j][v] = decay(gv[v]);
        }
        if (ig) {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                float iv[V];
                get<V, WIDE>(sm.i[r0 + j], lane, iv);
#pragma unroll
                for (int v = 0; v < V; ++v) u[j][v] *= iv[v];
            }
        }
        // bit j: a sequence starts at the warp's token j (bit W: at the token after its last)
        const uint32_t mask = bounds.mask;
        const int rows = T - t.t0 - r0;      // tokens from the warp's first on
        const uint32_t starts = mask & (rows >= W ? (1u << W) - 1 : rows > 0 ? (1u << rows) - 1 : 0u);
        float A[V], B[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            A[v] = a[0][v];
            B[v] = u[0][v];
        }
        if (starts) {
            const float *h0 = in.h0 ? in.h0 + t.col0 : nullptr;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if (!(starts >> j & 1)) continue;
                const int64_t n = bounds.seq(j);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (h0 && chan<V, WIDE>(lane, v) < left) u[j][v] = fmaf(a[j][v], h0[n * D + chan<V, WIDE>(lane, v)], u[j][v]);
            }
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) B[v] = j == 0 || (starts >> j & 1) ? u[j][v] : fmaf(a[j][v], B[v], u[j][v]);
#pragma unroll
            for (int v = 0; v < V; ++v) A[v] = -1.f;
        } else {
            // a becomes the product of the decays up to the token, u the state from zero
#pragma unroll
            for (int j = 1; j < W; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    u[j][v] = B[v] = fmaf(a[j][v], B[v], u[j][v]);
                    a[j][v] = A[v] *= a[j][v];
                }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) sm.s.map[warp][chan<V, WIDE>(lane, v)] = make_float2(A[v], B[v]);
        __syncthreads();
        float h[V];
        if (!incoming<C, V, WIDE, CHAIN, false>(sm.s, ch, t.rt, t.col0, t.tt == nT - 1, h, release)) return false;
        E *row = h_out + (t.t0 + r0) * ldh + t.col0;
        if (starts) {
#pragma unroll
            for (int j = 0; j < W; ++j) {
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = starts >> j & 1 ? u[j][v] : fmaf(a[j][v], h[v], u[j][v]);
                if (j < rows) put<V, WIDE>(row, lane, h, left, pair);
                row += ldh;
                if ((mask >> (j + 1) & 1) && final_state)
                    put<V, WIDE>(final_state + (bounds.seq(j + 1) - 1) * D + t.col0, lane, h, left, false);
            }
        } else {
            float s[V];
            if (rows >= W && left >= C && pair) {
#pragma unroll
                for (int j = 0; j < W; ++j) {
#pragma unroll
                    for (int v = 0; v < V; ++v) s[v] = fmaf(a[j][v], h[v], u[j][v]);
                    put_all<V, WIDE>(row, lane, s);
                    row += ldh;
                }
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j) {
#pragma unroll
                    for (int v = 0; v < V; ++v) s[v] = fmaf(a[j][v], h[v], u[j][v]);
                    if (j < rows) put<V, WIDE>(row, lane, s, left, pair);
                    row += ldh;
                }
            }
            if (mask && final_state) {         // no start among the warp's tokens: the one behind the last, or the stream's end
                const int j = __ffs(mask) - 2;
#pragma unroll
                for (int k = 0; k < W; ++k)
                    if (k == j)
#pragma unroll
                        for (int v = 0; v < V; ++v) s[v] = fmaf(a[k][v], h[v], u[k][v]);
                if (j >= 0) put<V, WIDE>(final_state + (bounds.seq(j + 1) - 1) * D + t.col0, lane, s, left, false);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = fmaf(a[W - 1][v], h[v], u[W - 1][v]);
        }
        if (states) {
            if (warp == WARPS - 1 && t.tt + 1 < nT)
                put<V, WIDE>(states + static_cast<int64_t>(t.tt + 1) * D + t.col0, lane, h, left, false);
            if (warp == 0 && t.tt == 0) {
                const float zero[V] = {};
                put<V, WIDE>(states + t.col0, lane, zero, left, false);
            }
        }
        return true;
    };
    walk<C, CHAIN, false>(sm.s, ch, pv, D, load, work);
}

// ---- backward -------------------------------------------------------------------------------------------

template <typename E, int C> struct __align__(16) BackwardShared {
    float g[L][C];
    E x[L][C], i[L][C], dh[L][C];
    float2 fmap[WARPS][C];         // the warps' maps of the states, forwards
    Shared<C> s;
};

template <typename E, int C, bool WIDE, bool CHAIN>
__global__ void __launch_bounds__(THREADS, 2) scan_backward(const int32_t *plan, PlanSig sig, int D, ScanIn in, Chain ch,
                                                            const float *states, const void *dh_, int64_t lddh,
                                                            const float *dfinal, ScanGrads out)
{
    constexpr int V = C / 32;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    auto &sm = *reinterpret_cast<BackwardShared<E, C> *>(smem_raw);
    if (!plan_matches(plan, sig)) {
        if (threadIdx.x == 0) record_status(&g_scan_status, KDA_ERR_INVALID_ARG);
        return;
    }
    const PlanView pv{plan};
    const int T = pv.T(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const E *x = static_cast<const E *>(in.x), *ig = static_cast<const E *>(in.i), *dh = static_cast<const E *>(dh_);
    E *dx = static_cast<E *>(out.dx), *di = static_cast<E *>(out.di);
    const bool pair = V == 1 || !WIDE || (pairs(dx, out.lddx) && pairs(di, out.lddi) && pairs(out.dg, out.lddg));

    // part 0: the decays, which a tile takes to registers; part 1: what it reads again for the gradients
    auto load = [&](const Tile &t, int part) {
        if (part == 0) {
            fill<float, C, WIDE>(&sm.g[0][0], in.g, in.ldg, t.t0, T, t.col0, D);
            return;
        }
        fill<E, C, WIDE>(&sm.dh[0][0], dh, lddh, t.t0, T, t.col0, D);
        fill<E, C, WIDE>(&sm.x[0][0], x, in.ldx, t.t0, T, t.col0, D);
        if (ig) fill<E, C, WIDE>(&sm.i[0][0], ig, in.ldi, t.t0, T, t.col0, D);
    };
    auto work = [&](const Tile &t, const Bounds &bounds, auto release) {
        const int r0 = warp * W, left = D - t.col0, rows = T - t.t0 - r0;
        const uint32_t mask = bounds.mask;
        const uint32_t starts = mask & (rows >= W ? (1u << W) - 1 : rows > 0 ? (1u << rows) - 1 : 0u);
        const uint32_t ends = mask >> 1;
        const bool plain = mask == 0 && rows >= W && left >= C && pair;
        // row n of h0 or dfinal at this lane's channels
        auto seq_row = [&](const float *p, int64_t n, float (&o)[V]) {
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = p && chan<V, WIDE>(lane, v) < left ? p[n * D + t.col0 + chan<V, WIDE>(lane, v)] : 0.f;
        };
        float hin[V];                    // the state before the tile
        seq_row(states, t.tt, hin);
        float a[W][V], u[W][V];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float gv[V];
            get<V, WIDE>(sm.g[r0 + j], lane, gv);
            get<V, WIDE>(sm.x[r0 + j], lane, u[j]);
#pragma unroll
            for (int v = 0; v < V; ++v) a[j][v] = decay(gv[v]);
        }
        if (ig) {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                float iv[V];
                get<V, WIDE>(sm.i[r0 + j], lane, iv);
#pragma unroll
                for (int v = 0; v < V; ++v) u[j][v] *= iv[v];
            }
        }
        float P[V], fb[V], B[V];         // maps of the states (P, fb; forwards) and of the gradients (P, B; backwards)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P[v] = 1.f;
            fb[v] = B[v] = 0.f;
        }
        auto maps = [&](auto bounded) {
            constexpr bool bnd = decltype(bounded)::value;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if constexpr (bnd)
                    if (starts >> j & 1) seq_row(in.h0, bounds.seq(j), fb);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    P[v] *= a[j][v];
                    fb[v] = fmaf(a[j][v], fb[v], u[j][v]);
                }
            }
#pragma unroll
            for (int j = W - 1; j >= 0; --j) {
                float d[V];
                get<V, WIDE>(sm.dh[r0 + j], lane, d);
                if constexpr (bnd)
                    if (ends >> j & 1) seq_row(dfinal, bounds.seq(j + 1) - 1, B);
#pragma unroll
                for (int v = 0; v < V; ++v) B[v] = a[j][v] * (d[v] + B[v]);
            }
        };
        if (mask == 0) maps(std::false_type{});
        else maps(std::true_type{});
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = chan<V, WIDE>(lane, v);
            sm.fmap[warp][c] = make_float2(starts ? -1.f : P[v], fb[v]);
            sm.s.map[WARPS - 1 - warp][c] = make_float2(ends ? -1.f : P[v], B[v]);
        }
        __syncthreads();
        // the last warp in time has nothing to wait for: it folds the maps of the states (each becomes that of the
        // warps before it)
        if (warp == WARPS - 1) {
            float A[V], S[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                A[v] = 1.f;
                S[v] = 0.f;
            }
#pragma unroll
            for (int w = 0; w < WARPS; ++w)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int c = chan<V, WIDE>(lane, v);
                    const float2 m = sm.fmap[w][c];
                    sm.fmap[w][c] = make_float2(A[v], S[v]);
                    then(A[v], S[v], m.x, m.y);
                }
        }
        float e[V];
        if (!incoming<C, V, WIDE, CHAIN, true>(sm.s, ch, t.rt, t.col0, t.tt == 0, e, release)) return false;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float2 m = sm.fmap[warp][chan<V, WIDE>(lane, v)];
            hin[v] = apply(m.x, m.y, hin[v]);
        }
        const int64_t last = t.t0 + r0 + W - 1;
        E *px = dx + last * out.lddx + t.col0, *pi = di ? di + last * out.lddi + t.col0 : nullptr;
        float *pg = out.dg + last * out.lddg + t.col0;
        // the states before each token (in place of u), then the gradients of each token from that of the next state
        auto finish = [&](auto bounded) {
            constexpr bool bnd = decltype(bounded)::value;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if constexpr (bnd)
                    if (starts >> j & 1) seq_row(in.h0, bounds.seq(j), hin);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float h = fmaf(a[j][v], hin[v], u[j][v]);
                    u[j][v] = hin[v];
                    hin[v] = h;
                }
            }
#pragma unroll
            for (int j = W - 1; j >= 0; --j) {
                float G[V], gx[V], gi[V], gg[V];
                get<V, WIDE>(sm.dh[r0 + j], lane, G);
                get<V, WIDE>(sm.x[r0 + j], lane, gi);
                if constexpr (bnd)
                    if (ends >> j & 1) seq_row(dfinal, bounds.seq(j + 1) - 1, e);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    G[v] += e[v];
                    e[v] = a[j][v] * G[v];
                    gi[v] *= G[v];
                    gg[v] = u[j][v] * e[v];
                    gx[v] = G[v];
                }
                if (ig) {
                    get<V, WIDE>(sm.i[r0 + j], lane, gx);
#pragma unroll
                    for (int v = 0; v < V; ++v) gx[v] *= G[v];
                }
                if constexpr (bnd) {
                    if (j < rows) {
                        put<V, WIDE>(px, lane, gx, left, pair);
                        if (di) put<V, WIDE>(pi, lane, gi, left, pair);
                        put<V, WIDE>(pg, lane, gg, left, pair);
                    }
                    if ((starts >> j & 1) && out.dh0) put<V, WIDE>(out.dh0 + bounds.seq(j) * D + t.col0, lane, e, left, false);
                } else {
                    put_all<V, WIDE>(px, lane, gx);
                    if (di) put_all<V, WIDE>(pi, lane, gi);
                    put_all<V, WIDE>(pg, lane, gg);
                }
                px -= out.lddx;
                pi -= out.lddi;
                pg -= out.lddg;
            }
        };
        if (plain) finish(std::false_type{});
        else finish(std::true_type{});
        __syncthreads();
        return true;
    };
    walk<C, CHAIN, true>(sm.s, ch, pv, D, load, work);
}

// ---- one token --------------------------------------------------------------------------------------------

// One token per row, each the next one of its slot's state (updated in place).
constexpr int STEP_THREADS = 128;
template <typename E>
__global__ void __launch_bounds__(STEP_THREADS) scan_step(int B, int D, const int32_t *slots, int num_slots, ScanIn in,
                                                          float *state, void *h_, int64_t ldh)
{
    const int d = blockIdx.x * STEP_THREADS + threadIdx.x;
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

// ---- launches ---------------------------------------------------------------------------------------------

template <typename F> cudaError_t by_type(int type, F f)
{
    if (type == KDA_TYPE_F32) return f(float{});
    if (type == KDA_TYPE_F16) return f(__half{});
    return f(__nv_bfloat16{});
}

// Every row of the tensor starts on 16 bytes.
bool wide(const void *p, int64_t ld, int bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * bytes & 15) == 0;
}

// Runs a tile kernel in the form that the number of tiles asks for.  cluster / chain: the two instances.
template <typename K, typename... Args>
cudaError_t run(K cluster, K chain, int C, int smem, const int32_t *plan_host, const int32_t *plan_dev, int D, void *ws,
                cudaStream_t stream, const ScanIn &in, Args... args)
{
    const int T = plan_host[KDA_PH_T], nT = tiles_of(T), nC = (D + C - 1) / C;
    const PlanSig sig = plan_sig(plan_host);
    K fn = nT <= MAX_CLUSTER ? cluster : chain;
    if (cudaError_t e = set_dynamic_smem(reinterpret_cast<const void *>(fn), smem)) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    Chain ch = {};
    if (nT <= MAX_CLUSTER) {
        int cs = 1;
        while (cs < nT) cs *= 2;
        cfg.gridDim = dim3(static_cast<unsigned>(nC) * cs);
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = cs;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    } else {
        ch = chain_of(ws, T, D);
        // A short group folds fewer maps a tile (measured at 64 channel ranges: 115.0 us with 8, 117.0 us with 16); a
        // long one passes the state on less often, which is what bounds narrow inputs.
        ch.group = nC >= 32 ? MIN_GROUP : MAX_GROUP;
        const Layout l = layout_of(T, D);
        const size_t words = (l.end - l.state) / 16;
        const size_t want = (words + 4 * 256 - 1) / (4 * 256), most = 4 * static_cast<size_t>(sm_count());
        chain_init<<<static_cast<unsigned>(want < most ? want : most), 256, 0, stream>>>(
            plan_dev, sig, nT, ch.ticket, ch.starts, reinterpret_cast<uint4 *>(ch.state), words);
        if (cudaError_t e = cudaGetLastError()) return e;
        const int64_t tiles = static_cast<int64_t>(nT) * nC, grid = 2 * static_cast<int64_t>(sm_count());
        cfg.gridDim = dim3(static_cast<unsigned>(tiles < grid ? tiles : grid));
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
    }
    return cudaLaunchKernelEx(&cfg, fn, plan_dev, sig, D, in, ch, args...);
}

}  // namespace

size_t scan_workspace_bytes(int64_t T, int D) { return T <= MAX_CLUSTER * L ? 0 : layout_of(T, D).end; }

cudaError_t launch_scan_forward(const int32_t *plan_host, const int32_t *plan_dev, int D, int type, const ScanIn &in,
                                void *h, int64_t ldh, float *final_state, float *states, void *ws, cudaStream_t stream)
{
    return by_type(type, [&](auto ev) {
        using E = decltype(ev);
        constexpr int C = 64;
        const int smem = sizeof(ForwardShared<E, C>);
        const bool w = wide(in.x, in.ldx, sizeof(E)) && (!in.i || wide(in.i, in.ldi, sizeof(E))) && wide(in.g, in.ldg, 4);
        return w ? run(scan_forward<E, C, true, false>, scan_forward<E, C, true, true>, C, smem, plan_host, plan_dev, D, ws, stream,
                       in, h, ldh, final_state, states)
                 : run(scan_forward<E, C, false, false>, scan_forward<E, C, false, true>, C, smem, plan_host, plan_dev, D, ws,
                       stream, in, h, ldh, final_state, states);
    });
}

cudaError_t launch_scan_backward(const int32_t *plan_host, const int32_t *plan_dev, int D, int type, const ScanIn &in,
                                 const float *states, const void *dh, int64_t lddh, const float *dfinal,
                                 const ScanGrads &out, void *ws, cudaStream_t stream)
{
    return by_type(type, [&](auto ev) {
        using E = decltype(ev);
        constexpr int C = sizeof(E) == 4 ? 32 : 64;    // two CTAs' tiles fit an SM
        const int smem = sizeof(BackwardShared<E, C>);
        const bool w = wide(in.x, in.ldx, sizeof(E)) && (!in.i || wide(in.i, in.ldi, sizeof(E))) && wide(in.g, in.ldg, 4) &&
                       wide(dh, lddh, sizeof(E));
        return w ? run(scan_backward<E, C, true, false>, scan_backward<E, C, true, true>, C, smem, plan_host, plan_dev, D, ws,
                       stream, in, states, dh, lddh, dfinal, out)
                 : run(scan_backward<E, C, false, false>, scan_backward<E, C, false, true>, C, smem, plan_host, plan_dev, D, ws,
                       stream, in, states, dh, lddh, dfinal, out);
    });
}

cudaError_t launch_scan_step(int B, int D, int type, const int32_t *slots, int num_slots, const ScanIn &in,
                             float *state, void *h, int64_t ldh, cudaStream_t stream)
{
    const dim3 grid((D + STEP_THREADS - 1) / STEP_THREADS, B < 65535 ? B : 65535);
    return by_type(type, [&](auto e) {
        scan_step<decltype(e)><<<grid, STEP_THREADS, 0, stream>>>(B, D, slots, num_slots, in, state, h, ldh);
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
