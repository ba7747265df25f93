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
//     the main one sets them, the ticket and each tile's first sequence.
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
constexpr int GROUP = 16;           // tiles of a group
constexpr int MAX_CLUSTER = 8;      // tiles that a cluster covers
constexpr int DPAD = 64;            // channels are padded to this in the workspace
constexpr long long SPIN = 4000000000LL;   // clocks of a wait: about two seconds

__device__ int g_scan_status;

// Workspace of the chain (bytes).
struct Layout {
    size_t first, state, map, end;   // each tile's first sequence; groups' states; tiles' maps
};
__host__ __device__ inline int tiles_of(int T) { return (T + L - 1) / L; }
inline Layout layout_of(int64_t T, int D)
{
    const size_t nT = static_cast<size_t>(T + L - 1) / L, Dp = static_cast<size_t>(D + DPAD - 1) / DPAD * DPAD;
    auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
    Layout l;
    l.first = 256;                                   // the ticket comes first
    l.state = up(l.first + (nT + 1) * 4);
    l.map = up(l.state + (nT + GROUP - 1) / GROUP * Dp * 4);
    l.end = l.map + nT * Dp * 8;
    return l;
}
struct Chain {
    int *ticket;
    const int *first;
    uint32_t *state;      // [groups][Dp], all ones until published
    uint64_t *map;        // [tiles][Dp], low word A, high word B
    int Dp;
};
inline Chain chain_of(void *ws, int64_t T, int D)
{
    char *b = static_cast<char *>(ws);
    const Layout l = layout_of(T, D);
    return Chain{reinterpret_cast<int *>(b), reinterpret_cast<int *>(b + l.first), reinterpret_cast<uint32_t *>(b + l.state),
                 reinterpret_cast<uint64_t *>(b + l.map), (D + DPAD - 1) / DPAD * DPAD};
}

__global__ void __launch_bounds__(256) chain_init(const int32_t *plan, PlanSig sig, int nT, int *ticket, int *first, uint4 *words,
                                                  size_t n)
{
    tc::grid_dep_launch();
    const size_t id = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x, step = static_cast<size_t>(gridDim.x) * blockDim.x;
    if (!plan_matches(plan, sig)) return;   // the main kernel records it
    for (size_t j = id; j < n; j += step) words[j] = make_uint4(~0u, ~0u, ~0u, ~0u);
    if (id == 0) *ticket = 0;
    const PlanView pv{plan};
    const int32_t *cu = pv.cu();
    for (size_t j = id; j <= static_cast<size_t>(nT); j += step) {
        const int64_t t = static_cast<int64_t>(j) * L;     // first n with cu[n] >= t (N + 1: none)
        int lo = 0, hi = pv.N() + 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] < t) lo = mid + 1;
            else hi = mid;
        }
        first[j] = lo;
    }
}

// ---- copies of a tile --------------------------------------------------------------------------------

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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
#pragma unroll
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
    float2 before[GROUP][C];       // maps of the tiles before this one (cluster: this tile's in [0])
    float state[C];                // the tile's incoming state
    int seq[2][L + 4];             // per token (one more than the tile's): the sequence that starts there, or -1
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

// The state that enters tile 'rt' (tiles numbered in the direction of the recurrence), left in sh.state for all
// threads.  (Am, Bm): this tile's map, in the warp 'last_warp', the last one of the tile in that direction.  False: a
// wait ran out.
template <int C, int V, bool WIDE, bool CHAIN>
__device__ __forceinline__ bool incoming(Shared<C> &sh, const Chain &ch, int rt, int col0, bool last, int last_warp,
                                         const float (&Am)[V], const float (&Bm)[V])
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int at[V];
#pragma unroll
    for (int v = 0; v < V; ++v) at[v] = chan<V, WIDE>(lane, v);
    if constexpr (CHAIN) {
        const int pos = rt % GROUP, grp = rt / GROUP;
        if (warp == last_warp && pos < GROUP - 1 && !last) {   // the group's last tile publishes a state instead
            uint64_t *p = ch.map + static_cast<size_t>(rt) * ch.Dp + col0;
#pragma unroll
            for (int v = 0; v < V; ++v)
                st_relaxed(p + at[v], static_cast<uint64_t>(word(Bm[v])) << 32 | __float_as_uint(Am[v]));
        }
        bool ok = true;
        for (int p = warp; p < pos && ok; p += WARPS) {
            uint64_t w[V];
            ok = poll<V>(ch.map + static_cast<size_t>(grp * GROUP + p) * ch.Dp + col0, w, at);
#pragma unroll
            for (int v = 0; v < V; ++v)
                sh.before[p][at[v]] = make_float2(__uint_as_float(static_cast<uint32_t>(w[v])), __uint_as_float(static_cast<uint32_t>(w[v] >> 32)));
        }
        float h[V];
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
            if (pos == GROUP - 1 && !last) {
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
                float h = 0.f;
#pragma unroll
                for (int p = 0; p < MAX_CLUSTER - 1; ++p) h = p < rt ? apply(m[p][v].x, m[p][v].y, h) : h;
                sh.state[at[v]] = h;
            }
        }
        cluster_arrive();   // paired with the wait at the kernel's end: no CTA leaves while its map is read
    }
    __syncthreads();
    return true;
}

// Marks the tile's sequence starts: seq[j] = n where token t0 + j is sequence n's first (n = N at token T).
// 'first': the first n with cu[n] >= t0, or -1 to look at all of them.  seq must hold -1 everywhere.
__device__ __forceinline__ void mark_starts(int *seq, const PlanView &pv, int first, int t0)
{
    const int32_t *cu = pv.cu();
    const int N = pv.N();
    if (first >= 0) {
        const int n = first + threadIdx.x;    // a start a token at most: L + 1 of them
        if (threadIdx.x <= L && n <= N) {
            const int t = cu[n] - t0;
            if (t <= L) seq[t] = n;
        }
        return;
    }
    for (int n = threadIdx.x; n <= N; n += THREADS) {
        const int t = cu[n] - t0;
        if (t >= 0 && t <= L) seq[t] = n;
    }
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

// Walks the tiles of a CTA: load(tile) starts the copies of a tile, work(tile, seq, release) computes it and calls
// release() once the copied data may be overwritten.  work returns false when a wait ran out.
template <int C, bool CHAIN, bool REVERSE, typename Load, typename Work>
__device__ __forceinline__ void walk(Shared<C> &sh, const Chain &ch, const PlanView &pv, int D, Load load, Work work)
{
    const int T = pv.T(), nT = tiles_of(T), nC = (D + C - 1) / C;
    for (int j = threadIdx.x; j < 2 * (L + 4); j += THREADS) (&sh.seq[0][0])[j] = -1;
    if (threadIdx.x == 0) sh.bad = 0;
    if constexpr (!CHAIN) {
        uint32_t cs, rank;
        asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(cs));
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        const int cc = blockIdx.x / cs;
        const Tile t = tile_of<C, REVERSE>(static_cast<int>(rank) * nC + cc, nT, nC);
        const bool real = t.rt < nT;      // clusters are a power of two: some CTAs may be past the end
        if (real) load(t);
        __syncthreads();
        if (real) mark_starts(sh.seq[0], pv, -1, t.t0);
        cp_wait();
        __syncthreads();
        if (real) {
            work(t, sh.seq[0], [] {});
        } else {
            cluster_arrive();
            cluster_wait();
            cluster_arrive();
        }
        cluster_wait();
    } else {
        tc::grid_dep_wait();
        const int n = nT * nC;
        if (threadIdx.x == 0) sh.next = atomicAdd(ch.ticket, 1);
        __syncthreads();
        int k = sh.next, at = 0;
        if (k < n) {
            const Tile t = tile_of<C, REVERSE>(k, nT, nC);
            load(t);
            mark_starts(sh.seq[0], pv, ch.first[t.tt], t.t0);
        }
        while (k < n) {
            const Tile t = tile_of<C, REVERSE>(k, nT, nC);
            __syncthreads();                 // everyone has read 'next'
            if (threadIdx.x == 0) sh.next = atomicAdd(ch.ticket, 1);
            cp_wait();
            __syncthreads();
            const int k2 = sh.next;
            const bool ok = work(t, sh.seq[at], [&] {
                // called between two barriers of the CTA: the copies' buffers are free
                if (k2 < n) load(tile_of<C, REVERSE>(k2, nT, nC));
            });
            if (!ok) {
                cp_wait();
                if (threadIdx.x == 0) record_status(&g_scan_status, KDA_ERR_TIMEOUT);
                return;
            }
            at ^= 1;
            if (k2 < n) {
                const Tile u = tile_of<C, REVERSE>(k2, nT, nC);
                mark_starts(sh.seq[at], pv, ch.first[u.tt], u.t0);
            }
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

    auto load = [&](const Tile &t) {
        fill<E, C, WIDE>(&sm.x[0][0], x, in.ldx, t.t0, T, t.col0, D);
        if (ig) fill<E, C, WIDE>(&sm.i[0][0], ig, in.ldi, t.t0, T, t.col0, D);
        fill<float, C, WIDE>(&sm.g[0][0], in.g, in.ldg, t.t0, T, t.col0, D);
    };
    auto work = [&](const Tile &t, int *seq, auto release) {
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
        const int sv = lane <= W ? seq[r0 + lane] : -1;
        const uint32_t mask = __ballot_sync(0xffffffffu, sv >= 0);
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
                const int64_t n = __shfl_sync(0xffffffffu, sv, j);
                if (!(starts >> j & 1)) continue;
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
#pragma unroll
            for (int j = 1; j < W; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    A[v] *= a[j][v];
                    B[v] = fmaf(a[j][v], B[v], u[j][v]);
                }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) sm.s.map[warp][chan<V, WIDE>(lane, v)] = make_float2(A[v], B[v]);
        __syncthreads();
        release();
        if (threadIdx.x <= L) seq[threadIdx.x] = -1;
        float pa[V], pb[V], h[V];      // the map of the warps before this one
#pragma unroll
        for (int v = 0; v < V; ++v) {
            pa[v] = 1.f;
            pb[v] = 0.f;
        }
        for (int w = 0; w < warp; ++w)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float2 m = sm.s.map[w][chan<V, WIDE>(lane, v)];
                then(pa[v], pb[v], m.x, m.y);
            }
#pragma unroll
        for (int v = 0; v < V; ++v) {      // and with it: the tile's in the last warp
            const float b = A[v] < 0.f ? B[v] : fmaf(A[v], pb[v], B[v]);
            A[v] = A[v] < 0.f || pa[v] < 0.f ? -1.f : A[v] * pa[v];
            B[v] = b;
        }
        if (!incoming<C, V, WIDE, CHAIN>(sm.s, ch, t.rt, t.col0, t.tt == nT - 1, WARPS - 1, A, B)) return false;
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = apply(pa[v], pb[v], sm.s.state[chan<V, WIDE>(lane, v)]);
        E *row = h_out + (t.t0 + r0) * ldh + t.col0;
        if (mask == 0 && rows >= W && left >= C && pair) {
#pragma unroll
            for (int j = 0; j < W; ++j) {
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = fmaf(a[j][v], h[v], u[j][v]);
                put_all<V, WIDE>(row, lane, h);
                row += ldh;
            }
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) {
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = starts >> j & 1 ? u[j][v] : fmaf(a[j][v], h[v], u[j][v]);
                if (j < rows) put<V, WIDE>(row, lane, h, left, pair);
                row += ldh;
                const int64_t n = __shfl_sync(0xffffffffu, sv, j + 1) - 1;
                if ((mask >> (j + 1) & 1) && final_state) put<V, WIDE>(final_state + n * D + t.col0, lane, h, left, false);
            }
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

    auto load = [&](const Tile &t) {
        fill<float, C, WIDE>(&sm.g[0][0], in.g, in.ldg, t.t0, T, t.col0, D);
        fill<E, C, WIDE>(&sm.dh[0][0], dh, lddh, t.t0, T, t.col0, D);
        fill<E, C, WIDE>(&sm.x[0][0], x, in.ldx, t.t0, T, t.col0, D);
        if (ig) fill<E, C, WIDE>(&sm.i[0][0], ig, in.ldi, t.t0, T, t.col0, D);
    };
    auto work = [&](const Tile &t, int *seq, auto release) {
        const int r0 = warp * W, left = D - t.col0, rows = T - t.t0 - r0;
        const int sv = lane <= W ? seq[r0 + lane] : -1;
        const uint32_t mask = __ballot_sync(0xffffffffu, sv >= 0);
        const uint32_t starts = mask & (rows >= W ? (1u << W) - 1 : rows > 0 ? (1u << rows) - 1 : 0u);
        const uint32_t ends = mask >> 1;
        const bool plain = mask == 0 && rows >= W && left >= C && pair;
        // row n of h0 or dfinal at this lane's channels
        auto seq_row = [&](const float *p, int64_t n, float (&o)[V]) {
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = p && chan<V, WIDE>(lane, v) < left ? p[n * D + t.col0 + chan<V, WIDE>(lane, v)] : 0.f;
        };
        auto u_of = [&](int j, float (&u)[V]) {
            get<V, WIDE>(sm.x[r0 + j], lane, u);
            if (ig) {
                float iv[V];
                get<V, WIDE>(sm.i[r0 + j], lane, iv);
#pragma unroll
                for (int v = 0; v < V; ++v) u[v] *= iv[v];
            }
        };
        float hin[V];                    // the state before the tile
        seq_row(states, t.tt, hin);
        float a[W][V];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float gv[V];
            get<V, WIDE>(sm.g[r0 + j], lane, gv);
#pragma unroll
            for (int v = 0; v < V; ++v) a[j][v] = decay(gv[v]);
        }
        float P[V], fb[V], B[V];         // maps of the states (P, fb; forwards) and of the gradients (P, B; backwards)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P[v] = 1.f;
            fb[v] = B[v] = 0.f;
        }
        if (mask == 0) {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                float u[V];
                u_of(j, u);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    P[v] *= a[j][v];
                    fb[v] = fmaf(a[j][v], fb[v], u[v]);
                }
            }
#pragma unroll
            for (int j = W - 1; j >= 0; --j) {
                float d[V];
                get<V, WIDE>(sm.dh[r0 + j], lane, d);
#pragma unroll
                for (int v = 0; v < V; ++v) B[v] = a[j][v] * (d[v] + B[v]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                float u[V];
                u_of(j, u);
                const int64_t n = __shfl_sync(0xffffffffu, sv, j);
                if (starts >> j & 1) seq_row(in.h0, n, fb);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    P[v] *= a[j][v];
                    fb[v] = fmaf(a[j][v], fb[v], u[v]);
                }
            }
#pragma unroll
            for (int j = W - 1; j >= 0; --j) {
                float d[V];
                get<V, WIDE>(sm.dh[r0 + j], lane, d);
                const int64_t n = __shfl_sync(0xffffffffu, sv, j + 1) - 1;
                if (ends >> j & 1) seq_row(dfinal, n, B);
#pragma unroll
                for (int v = 0; v < V; ++v) B[v] = a[j][v] * (d[v] + B[v]);
            }
        }
        float A[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = chan<V, WIDE>(lane, v);
            A[v] = ends ? -1.f : P[v];
            sm.fmap[warp][c] = make_float2(starts ? -1.f : P[v], fb[v]);
            sm.s.map[warp][c] = make_float2(A[v], B[v]);
        }
        __syncthreads();
        if (threadIdx.x <= L) seq[threadIdx.x] = -1;
        float pa[V], pb[V], e[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            pa[v] = 1.f;
            pb[v] = 0.f;
        }
        for (int w = WARPS - 1; w > warp; --w)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float2 m = sm.s.map[w][chan<V, WIDE>(lane, v)];
                then(pa[v], pb[v], m.x, m.y);
            }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float b = A[v] < 0.f ? B[v] : fmaf(A[v], pb[v], B[v]);
            A[v] = A[v] < 0.f || pa[v] < 0.f ? -1.f : A[v] * pa[v];
            B[v] = b;
        }
        if (!incoming<C, V, WIDE, CHAIN>(sm.s, ch, t.rt, t.col0, t.tt == 0, 0, A, B)) return false;
#pragma unroll
        for (int v = 0; v < V; ++v) e[v] = apply(pa[v], pb[v], sm.s.state[chan<V, WIDE>(lane, v)]);
        for (int w = 0; w < warp; ++w)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float2 m = sm.fmap[w][chan<V, WIDE>(lane, v)];
                hin[v] = apply(m.x, m.y, hin[v]);
            }
        float before[W][V];              // the state before each token
        const int64_t last = t.t0 + r0 + W - 1;
        E *px = dx + last * out.lddx + t.col0, *pi = di ? di + last * out.lddi + t.col0 : nullptr;
        float *pg = out.dg + last * out.lddg + t.col0;
        // token j's gradients from that of the next state; e becomes that of the one before
        auto grads = [&](int j, float (&gx)[V], float (&gi)[V], float (&gg)[V]) {
            float d[V], iv[V];
            get<V, WIDE>(sm.dh[r0 + j], lane, d);
            get<V, WIDE>(sm.x[r0 + j], lane, gi);
            if (ig) get<V, WIDE>(sm.i[r0 + j], lane, iv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float G = d[v] + e[v];
                e[v] = a[j][v] * G;
                gx[v] = ig ? iv[v] * G : G;
                gi[v] *= G;
                gg[v] = before[j][v] * e[v];
            }
        };
        if (plain) {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                float u[V];
                u_of(j, u);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    before[j][v] = hin[v];
                    hin[v] = fmaf(a[j][v], hin[v], u[v]);
                }
            }
#pragma unroll
            for (int j = W - 1; j >= 0; --j) {
                float gx[V], gi[V], gg[V];
                grads(j, gx, gi, gg);
                put_all<V, WIDE>(px, lane, gx);
                put_all<V, WIDE>(pg, lane, gg);
                px -= out.lddx;
                pg -= out.lddg;
                if (di) {
                    put_all<V, WIDE>(pi, lane, gi);
                    pi -= out.lddi;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                float u[V];
                u_of(j, u);
                const int64_t n = __shfl_sync(0xffffffffu, sv, j);
                if (starts >> j & 1) seq_row(in.h0, n, hin);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    before[j][v] = hin[v];
                    hin[v] = fmaf(a[j][v], hin[v], u[v]);
                }
            }
#pragma unroll
            for (int j = W - 1; j >= 0; --j) {
                float gx[V], gi[V], gg[V];
                const int64_t n = __shfl_sync(0xffffffffu, sv, j + 1) - 1;
                if (ends >> j & 1) seq_row(dfinal, n, e);
                grads(j, gx, gi, gg);
                if (j < rows) {
                    put<V, WIDE>(px, lane, gx, left, pair);
                    if (di) put<V, WIDE>(pi, lane, gi, left, pair);
                    put<V, WIDE>(pg, lane, gg, left, pair);
                }
                px -= out.lddx;
                pi -= out.lddi;
                pg -= out.lddg;
                const int64_t m = __shfl_sync(0xffffffffu, sv, j);
                if ((starts >> j & 1) && out.dh0) put<V, WIDE>(out.dh0 + m * D + t.col0, lane, e, left, false);
            }
        }
        __syncthreads();
        release();
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
        const Layout l = layout_of(T, D);
        const size_t words = (l.end - l.state) / 16;
        const size_t want = (words + 4 * 256 - 1) / (4 * 256), most = 4 * static_cast<size_t>(sm_count());
        chain_init<<<static_cast<unsigned>(want < most ? want : most), 256, 0, stream>>>(
            plan_dev, sig, nT, ch.ticket, const_cast<int *>(ch.first), reinterpret_cast<uint4 *>(ch.state), words);
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
