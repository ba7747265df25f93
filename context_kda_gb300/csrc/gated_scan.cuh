// Gated linear recurrence over packed sequences, per channel:
//     h_t = exp(g_t) h_{t-1} + i_t x_t,   h_{-1} = h0 of the sequence,
// its gradients (the same recurrence backwards in time) and its single-token step.
//
// One pass over the data.  Over a run of tokens the recurrence is the map h -> A h + B with A the product
// of the decays and B the run's state from zero, and maps compose as (A2, B2) o (A1, B1) = (A1 A2, A2 B1 + B2);
// a run in which a sequence starts forgets what came before (h -> B, marked by A = -1: decays are not
// negative), so nothing of another sequence, infinities and NaN included, is ever multiplied in.  Decays may be above one
// and their product beyond fp32's range, where a state may still be small: such an A is kept scaled, as a negative number.
//
// The stream is cut into tiles of 128 tokens x 32 channels, a tile into 8 runs of 16 tokens (half a warp each, two
// channels a lane).  A CTA of four warps copies a tile to shared memory (cp.async), folds each run in
// registers, folds the runs' maps in shared memory and publishes the tile's; with the tile's incoming state known,
// every run is finished from registers and the results are written.  Inputs are read from memory once.  The
// kernel waits rather than computes (for copies, for other tiles' maps), so four CTAs share an SM, each in another phase;
// a tile's copies are requested as soon as the last tile's have gone to registers.
//
// Measured on the device (bf16, share of a copy's 6.79 TB/s): wide inputs are bound by memory, 65536 x 4096 413 us (96 %),
// 16384 x 4096 110 us (90 %) and its gradients 201 us (89 %), as first built with two CTAs of 256 threads an SM 119 and 277 us;
// what is left is the first tiles' way in and the last ones' way out.  Narrow inputs are bound by the state's way along the
// chain, about a microsecond a group: 49274 x 128 26 us (36 %), 16384 x 1024 38 us (66 %).  Rows that do not start on 16 bytes
// are bound by instructions, 16384 x 1001 50 us (48 %) and its gradients 88 us (49 %); the smallest by the launch,
// 1024 x 512 5.4 us.
//   - Up to 8 tiles of tokens ('cluster'): the CTAs of a channel range are one cluster; they exchange the
//     maps through distributed shared memory.  One launch and no workspace, for short inputs, where
//     latency counts.
//   - More ('chain'): CTAs draw all their tiles in time order from a ticket, so that a tile waits only for tiles drawn
//     before it by CTAs that run, and progress needs one CTA on the device, not the grid.  A tile's incoming state is folded, always in the same order, from the
//     state at its group's start and the maps of the group's earlier tiles; the group's last tile publishes
//     the next group's state.  Only that last step is serial in time, once a group.  Published words
//     carry their own validity (they are all ones until written, which no published value is), so that one
//     8-byte store and one load pass a map on.  A kernel before the main one sets them, the ticket and each
//     tile's sequence starts.
//   - Waits give up after about two seconds (KDA_ERR_TIMEOUT through kda_device_status).
//
// The backward takes the states before every 128th token that the forward saved, so a tile recomputes its
// states without waiting; its own recurrence is
//     G_t = dh_t + e_{t+1},  e_t = exp(g_t) G_t   (e_{t+1} = dfinal at the last token of a sequence),
//     dx = i G, di = x G, dg = e_t h_{t-1}, dh0 = e at the first token,
// with tiles taken from the last to the first.
#pragma once

#include <type_traits>

#include "elem.cuh"
#include "kda_internal.cuh"
#include "tc.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int L = KDA_SCAN_TILE;             // tokens of a tile
constexpr int C = 32;                        // channels of a tile
constexpr int RUN = 16, RUNS = L / RUN;      // tokens of a run, runs of a tile
constexpr int V = 2;                         // channels of a lane
constexpr int WARPS = RUNS / 2, THREADS = WARPS * 32;
// CTAs of an SM: four, or as many as their shared memory allows.
template <typename Sh> constexpr int ctas_of() { return 233472 / (static_cast<int>(sizeof(Sh)) + 1024) < 4 ? 233472 / (static_cast<int>(sizeof(Sh)) + 1024) : 4; }
// Tiles of a group.  Narrow inputs wait for the state's way from group to group, which a long group shortens, at the cost
// of more maps that a tile reads and folds (bf16, groups of 8 / 16: 65536 tokens x 4096 channels, 128 ranges of channels, 411 / 420 us
// and gradients of 16384 x 4096 200 / 206 us; 16384 x 1024, 32 ranges, 39 / 37 us; 49274 x 128, 4 ranges, 39 / 26 us; of 32, the
// last takes 22 us and the others are slower than with 16: a third length for a few ranges would take that, at the cost of another
// instance of every kernel).
constexpr int WIDE_GROUP = 8, NARROW_GROUP = 16, WIDE_RANGES = 64;
// Tiles that a cluster covers: 512 tokens in bf16 take 5.2 us, by a chain 6.7 us, at 512 channels, and 6.1 and 7.8 us at 4096;
// 1024 tokens 5.4 and 6.8 us, and 10.6 and 10.9 us.
constexpr int MAX_CLUSTER = 8;
constexpr long long SPIN = 4000000000LL;     // clocks of a wait: about two seconds

__device__ int g_scan_status;

// The sequence starts of a tile: bit j: a sequence starts at its token j; 'first': the lowest such sequence.
// The end of the stream counts as the start of sequence N.
struct __align__(16) Starts {
    uint32_t bits[L / 32];
    int first, pad[3];
};
static_assert(sizeof(Starts) == 32 && L == 128 && RUN == 16, "two runs a word, four words a tile");

// Workspace of the chain (bytes).
struct Layout {
    size_t starts, state, map, end;   // each tile's sequence starts; groups' states; tiles' maps
};
__host__ __device__ inline int tiles_of(int T) { return static_cast<int>((static_cast<int64_t>(T) + L - 1) / L); }
inline int padded(int D) { return (D + C - 1) / C * C; }
inline Layout layout_of(int64_t T, int D)
{
    const size_t nT = static_cast<size_t>(T + L - 1) / L, Dp = padded(D);
    auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
    Layout l;
    l.starts = 256;                                  // the ticket comes first
    l.state = up(l.starts + (nT + 1) * sizeof(Starts));
    l.map = up(l.state + (nT / WIDE_GROUP + 1) * Dp * 4);
    l.end = l.map + nT * Dp * 8;
    return l;
}
struct Chain {
    int *ticket;
    Starts *starts;       // [tiles + 1]
    uint32_t *state;      // [groups][Dp], all ones until published
    uint64_t *map;        // [tiles][Dp], low word A, high word B
    int Dp;               // padded channels
};
inline Chain chain_of(void *ws, int64_t T, int D)
{
    char *b = static_cast<char *>(ws);
    const Layout l = layout_of(T, D);
    return Chain{reinterpret_cast<int *>(b), reinterpret_cast<Starts *>(b + l.starts), reinterpret_cast<uint32_t *>(b + l.state),
                 reinterpret_cast<uint64_t *>(b + l.map), padded(D)};
}

__global__ void __launch_bounds__(256) chain_init(const int32_t *plan, PlanSig sig, int nT, int *ticket, Starts *starts,
                                                  uint4 *words, size_t n)
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

// ---- a tile in shared memory ----------------------------------------------------------------------------

// Rows of one tensor, run by run.  SH: rows that do not all start on 16 bytes are copied with the 16 bytes they start in,
// so a row takes one copy more and its channels start at an offset.  Runs are moved against each other where a
// warp, which reads two runs at once, would find both in the same banks.
template <typename X, bool SH> struct __align__(16) Rows {
    static constexpr int EPC = 16 / static_cast<int>(sizeof(X));            // elements of a copy
    static constexpr int PITCH = (C + (SH ? EPC : 0)) * static_cast<int>(sizeof(X));
    static constexpr int RUN_BYTES = RUN * PITCH + (SH || sizeof(X) == 2 ? 64 : 0);
    unsigned char b[RUNS * RUN_BYTES];
    __device__ __forceinline__ X *row(int run, int j) { return reinterpret_cast<X *>(b + run * RUN_BYTES + j * PITCH); }
};
// The row of a run's j-th token in shared memory, from its first channel on.
template <typename X, bool SH> struct Run {
    Rows<X, SH> &rows;
    int run;
    uint32_t first, ld;        // element the run's first row starts at, and between rows (modulo a copy)
    __device__ __forceinline__ Run(Rows<X, SH> &r, int n, const X *src, int64_t stride, int t0) : rows(r), run(n), first(0), ld(0)
    {
        if constexpr (SH) {
            first = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src) / sizeof(X)) + static_cast<uint32_t>(t0 + n * RUN) * static_cast<uint32_t>(stride);
            ld = static_cast<uint32_t>(stride);
        }
    }
    __device__ __forceinline__ const X *operator()(int j) const
    {
        // rows a copy's elements apart start alike
        constexpr int EPC = Rows<X, SH>::EPC;
        return rows.row(run, j) + (SH ? (first + (j % EPC) * ld) & (EPC - 1) : 0u);
    }
    // f(j, row) for all tokens, those that start alike one after the other
    template <typename F> __device__ __forceinline__ void each(F f) const
    {
        constexpr int P = SH ? Rows<X, SH>::EPC : 1;
#pragma unroll
        for (int k = 0; k < P; ++k) {
#pragma unroll
            for (int j = k; j < RUN; j += P) f(j, (*this)(j));
        }
    }
};
// What the runs and tiles of a channel range pass on; G: tiles of a group.
template <int G> struct Shared {
    float2 map[RUNS][C];           // the runs' maps
    float state[RUNS][C];          // the state that enters each run
    float2 before[G - 1][C];   // maps of the group's tiles before this one (cluster: this tile's in [0])
    Starts starts;                 // cluster: the tile's sequence starts
    uint32_t after;
    int next, bad;
    int far;                       // the last tile (its number, rt) that met great products
};

// ---- copies ---------------------------------------------------------------------------------------------

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Tokens t0.. (zeros from T on), channels c0.. (zeros from D on) of a tensor of rows.
template <typename X, bool SH>
__device__ __forceinline__ void fill(Rows<X, SH> &dst, const X *src, int64_t ld, int t0, int T, int c0, int D)
{
    using R = Rows<X, SH>;
    if constexpr (!SH) {
        constexpr int CPR = C / R::EPC, STEP = THREADS / CPR;      // copies of a row, rows of a step
        const int row = threadIdx.x / CPR, c = threadIdx.x % CPR * R::EPC;
        const X *p = src + (static_cast<int64_t>(t0) + row) * ld + c0 + c;
        const int64_t hop = STEP * ld;
        const int left = D - c0 - c;
        const int bytes = (left < 0 ? 0 : left > R::EPC ? R::EPC : left) * static_cast<int>(sizeof(X));
        const int rows = bytes ? T - t0 - row : 0;                 // of this thread, from its first on
        // the k-th row's place is a constant from the first's: steps never leave the first row's place within its run
        static_assert(STEP % RUN == 0 || RUN % STEP == 0, "whole runs a step or whole steps a run");
        const uint32_t to = smem_u32(dst.row(row / RUN, row % RUN) + c);
        auto place = [](int k) { return k * STEP / RUN * R::RUN_BYTES + k * STEP % RUN * R::PITCH; };
        if (rows >= L) {
#pragma unroll
            for (int k = 0; k < L / STEP; ++k) {
                copy16(to + place(k), p, bytes);
                p += hop;
            }
        } else {
#pragma unroll 4
            for (int k = 0; k < L / STEP; ++k) {
                const bool in = k * STEP < rows;
                copy16(to + place(k), in ? p : src, in ? bytes : 0);
                p += hop;
            }
        }
    } else {
        constexpr int CPR = C / R::EPC, STEP = THREADS / CPR;      // whole copies of a row, rows of a step; a row takes one copy more
        static_assert(THREADS == L, "the last copies are one a thread");
        const char *base = reinterpret_cast<const char *>(src);
        const int64_t pitch = ld * static_cast<int64_t>(sizeof(X));
        const char *tile = base + t0 * pitch + c0 * static_cast<int64_t>(sizeof(X));
        if (t0 > 0 && T - t0 > L && D - c0 >= C) {
            // rows before and after the tile's: whole copies stay within the tensor, their ends belong to other channels
            const int row = threadIdx.x / CPR, c = threadIdx.x % CPR;
            const uint32_t to = smem_u32(dst.row(row / RUN, row % RUN) + c * R::EPC);
            auto from = [](const char *p) { return reinterpret_cast<const char *>(reinterpret_cast<uintptr_t>(p) & ~static_cast<uintptr_t>(15)); };
            const char *p = tile + row * pitch;
            const int64_t hop = STEP * pitch;
#pragma unroll
            for (int k = 0; k < L / STEP; ++k) {
                copy16(to + k * STEP / RUN * R::RUN_BYTES + k * STEP % RUN * R::PITCH, from(p) + c * 16, 16);
                p += hop;
            }
            copy16(smem_u32(dst.row(threadIdx.x / RUN, threadIdx.x % RUN) + C), from(tile + threadIdx.x * pitch) + C * sizeof(X), 16);
            return;
        }
        const int width = (D - c0 < C ? D - c0 : C) * static_cast<int>(sizeof(X));
#pragma unroll 1
        for (int k = threadIdx.x; k < L * (CPR + 1); k += THREADS) {
            const int row = k / (CPR + 1), ch = k % (CPR + 1);
            const char *p = tile + row * pitch;
            const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u);
            const int left = row < T - t0 ? off + width - ch * 16 : 0;
            const int bytes = left < 0 ? 0 : left > 16 ? 16 : left;
            const char *at = p - off + ch * 16;
            X *to = dst.row(row / RUN, row % RUN) + ch * R::EPC;
            if (bytes && at < base) {        // the tensor starts within this copy: nothing before it is read
                const int skip = static_cast<int>(base - at) / static_cast<int>(sizeof(X));
                for (int e = 0; e < R::EPC; ++e)
                    to[e] = e >= skip && e * static_cast<int>(sizeof(X)) < bytes ? reinterpret_cast<const X *>(at)[e] : from_f32<X>(0.f);
            } else {
                copy16(smem_u32(to), bytes ? at : base - (reinterpret_cast<uintptr_t>(base) & 15u), bytes);
            }
        }
    }
}

// ---- channels of a lane ---------------------------------------------------------------------------------
// Adjacent ones where a pair can be loaded and stored as one (ADJ), 16 apart otherwise (single elements of half a
// warp are adjacent).
template <bool ADJ> __device__ __forceinline__ int chan(int lane, int v) { return ADJ ? lane * 2 + v : lane + 16 * v; }

__device__ __forceinline__ void unpack(uint32_t w, float (&o)[V], const __nv_bfloat16 *)
{
    o[0] = __uint_as_float(w << 16);
    o[1] = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void unpack(uint32_t w, float (&o)[V], const __half *)
{
    const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    o[0] = p.x;
    o[1] = p.y;
}
template <bool ADJ, typename X> __device__ __forceinline__ void get(const X *row, int lane, float (&o)[V])
{
    if constexpr (ADJ && sizeof(X) == 4) {
        const float2 p = reinterpret_cast<const float2 *>(row)[lane];
        o[0] = p.x;
        o[1] = p.y;
    } else if constexpr (ADJ) {
        unpack(reinterpret_cast<const uint32_t *>(row)[lane], o, row);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = to_f32(row[chan<ADJ>(lane, v)]);
    }
}

__device__ __forceinline__ void put2(float *p, float a, float b) { *reinterpret_cast<float2 *>(p) = make_float2(a, b); }
__device__ __forceinline__ void put2(__half *p, float a, float b) { *reinterpret_cast<__half2 *>(p) = __floats2half2_rn(a, b); }
__device__ __forceinline__ void put2(__nv_bfloat16 *p, float a, float b)
{
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(a, b);
}
// A lane's channels of one row, from its first one's address, where all of the tile's channels exist and, if adjacent,
// rows start on pairs.
template <bool ADJ, typename X> __device__ __forceinline__ void put_all(X *at, const float (&o)[V])
{
    if constexpr (ADJ) {
        put2(at, o[0], o[1]);
    } else {
        at[0] = from_f32<X>(o[0]);
        at[16] = from_f32<X>(o[1]);
    }
}
// The same where 'left' channels exist.
template <bool ADJ, typename X> __device__ __forceinline__ void put(X *row, int lane, const float (&o)[V], int left)
{
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (chan<ADJ>(lane, v) < left) row[chan<ADJ>(lane, v)] = from_f32<X>(o[v]);
}
template <typename X> __device__ __forceinline__ bool pairs(const X *p, int64_t ld)
{
    return (reinterpret_cast<uintptr_t>(p) & (2 * sizeof(X) - 1)) == 0 && (ld & 1) == 0;
}

// exp(g) as 2^(g log2 e): the product's rounding moves the result by |g| 2^-24 relative, which is below the exponential's own
// error for every g that leaves anything to remember.  That is 2^-22 at most; measured against 64 bits, in units of 2^-24: 1.4 for
// g in -1e-7 .. -1e-3, where states are longest remembered, 2.1 down to -0.2, 3.8 down to -3 (torch's fp32 exponential 1.5, 1.8
// and 2.4, a correctly rounded one 0.5 to 1).
__device__ __forceinline__ float decay(float g) { return ex2_ftz(g * 1.4426950408889634f); }

// A lane's two channels in one instruction (gradients of 16384 x 4096 in bf16: 4 us of 201 less than in scalar ones).
static_assert(V == 2, "pairs");
__device__ __forceinline__ float2 both(const float (&v)[V]) { return make_float2(v[0], v[1]); }
__device__ __forceinline__ void set(float (&v)[V], float2 p) { v[0] = p.x, v[1] = p.y; }
__device__ __forceinline__ float2 decay2(float2 g)
{
    g = mul2(g, make_float2(1.4426950408889634f, 1.4426950408889634f));
    return make_float2(ex2_ftz(g.x), ex2_ftz(g.y));
}

// ---- maps -----------------------------------------------------------------------------------------------

// A map's A as a float: a product of decays of up to fp32's largest number is itself, -1 marks a map that forgets, and a
// greater product is scaled: minus its 2^-127th part, from -2 on.  Minus infinity stands for 2^254 and more, which takes every
// state but zero (and fp32's denormal numbers) past fp32's range; zero stays zero (a decay that is infinite by itself makes a NaN
// of the map's other half).
constexpr float MOST = 3.402823466e38f, FORGET = -1.f;
constexpr float MOST_RUN = 32768.f;     // the runs' products up to which a tile's is in range
static_assert(RUNS == 8, "2^(15 * 8) < 2^128");
__device__ __forceinline__ float product_of(double p)
{
    return !(p > MOST) ? static_cast<float>(p) : p < 0x1p254 ? -static_cast<float>(p * 0x1p-127) : __int_as_float(static_cast<int>(0xFF800000u));
}
// A run whose products may leave fp32's range: the product of its first n decays, kept at 2^1000 beyond that, and, for a channel
// whose products in fp32 do leave it, the k that brings all of them to 2^121 and less (126 at most; else 0).  Decays that are
// infinite by themselves, or NaN, do not count: they leave NaN behind them, and must change nothing before them.
template <bool ADJ, typename R> __device__ __forceinline__ void far_products(const R &rows, int l, int n, double (&p)[V], int (&k)[V])
{
    constexpr double MAX = 0x1p1000;
    float q[V] = {1.f, 1.f};
    double peak[V] = {1.0, 1.0};
    bool over[V] = {};
    p[0] = p[1] = 1.0;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
        float g[V];
        get<ADJ>(rows(j), l, g);
        set(g, decay2(both(g)));
#pragma unroll
        for (int v = 0; v < V; ++v) g[v] = g[v] <= MOST ? g[v] : 1.f;
        set(q, mul2(both(q), both(g)));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            over[v] = over[v] || !(q[v] <= MOST);
            p[v] = p[v] < MAX ? fmin(p[v] * g[v], MAX) : MAX;
            peak[v] = fmax(peak[v], p[v]);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) k[v] = over[v] ? max(0, min((__double2hiint(peak[v]) >> 20) - 1023 - 120, 126)) : 0;
}
__device__ __forceinline__ float two_to(int k) { return __int_as_float((127 + k) << 23); }     // |k| <= 126
// A state behind a map.  Scaled ones (any_apply) are rare and the folds are what tiles wait for: who makes or fetches a map that
// may lead to one leaves a mark, and folds go by 'apply' where there is none (65536 x 4096 in bf16: 428 us with the cases
// looked at in every step, 421 us with a tile's product looked at behind its fold, 413 us).
__device__ __forceinline__ float apply(float2 m, float h) { return m.x < 0.f ? m.y : fmaf(m.x, h, m.y); }
__device__ __forceinline__ bool scaled(float lowest) { return lowest < FORGET; }
__device__ __forceinline__ float any_apply(float2 m, float h)
{
    if (!scaled(m.x)) return apply(m, h);
    if (m.x < -MOST) return h == 0.f ? m.y : fmaf(h, -m.x, m.y);
    return fmaf(0x1p64f * h * -m.x, 0x1p63f, m.y);      // neither product leaves the range before the result does
}
// One map more: (A, B) becomes m o (A, B).
__device__ __forceinline__ void then(float &A, float &B, float2 m)
{
    B = apply(m, B);
    A = m.x < 0.f || A < 0.f ? FORGET : A * m.x;
}
// (a call: its double arithmetic in the kernels' code costs gradients of 16384 x 4096 half a percent)
__device__ __noinline__ float any_join(float A, float a)
{
    auto whole = [](float x) { return x < 0.f ? fmin(static_cast<double>(x) * -0x1p127, 0x1p600) : static_cast<double>(x); };
    return A == FORGET || a == FORGET ? FORGET : product_of(whole(A) * whole(a));
}
__device__ __forceinline__ void any_then(float &A, float &B, float2 m)
{
    B = any_apply(m, B);
    A = any_join(A, m.x);
}

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

// The tile whose number in the direction of the recurrence is rt and whose channels start at col0.
struct Tile {
    int rt, tt, t0, col0;
};
template <bool REVERSE> __device__ __forceinline__ Tile tile_of(int k, int nT, int nC)
{
    Tile t;
    t.rt = k / nC;
    t.tt = REVERSE ? nT - 1 - t.rt : t.rt;
    t.t0 = t.tt * L;
    t.col0 = (k - t.rt * nC) * C;
    return t;
}

// The sequence starts among a run's tokens and the token after them: bit j of 'mask'; the start at bit j is that of
// sequence first + (number of bits below j).  'starts': those among the run's tokens.
struct Bounds {
    uint32_t mask, starts;
    int first;
    __device__ __forceinline__ Bounds(const uint4 &bits, int first_seq, uint32_t after, int run, int rows)
    {
        const int w = run / 2;             // = the warp
        const uint32_t b[6] = {bits.x, bits.y, bits.z, bits.w, after, 0u};
        uint32_t cur = 0, next = 0;
        int below = first_seq;
#pragma unroll
        for (int k = 0; k < L / 32; ++k) {
            if (k == w) cur = b[k], next = b[k + 1];
            if (k < w) below += __popc(b[k]);
        }
        const int at = run % 2 * RUN;
        mask = __funnelshift_r(cur, next, at) & ((2u << RUN) - 1);
        first = below + __popc(cur & ((1u << at) - 1));
        starts = mask & (rows >= RUN ? (1u << RUN) - 1 : rows > 0 ? (1u << rows) - 1 : 0u);
    }
    __device__ __forceinline__ int64_t seq(int j) const { return first + __popc(mask & ((1u << j) - 1)); }
    // the first boundary's place, beyond the run if there is none
    __device__ __forceinline__ int place() const { return mask ? __ffs(mask) - 1 : 2 * RUN; }
};
// How a warp's two runs are worked.  Boundaries between sequences are rare, but later tiles wait for the tiles that
// hold them: a run with one takes it by selections (its rows of h0 and dfinal are requested before anything else).
// Runs at the tensor's edges do the same (tokens past the end leave a state as it is: their decay is one and their term
// zero) and look at what they may write; only runs with several boundaries look at every token.
enum { PLAIN = 0, ONE = 1, EDGE = 2, ANY = 3 };
__device__ __forceinline__ int kind_of(const Bounds &b, bool inside)
{
    if (__any_sync(0xffffffffu, __popc(b.mask) > 1)) return ANY;
    if (__any_sync(0xffffffffu, !inside)) return EDGE;
    return __any_sync(0xffffffffu, b.mask != 0) ? ONE : PLAIN;
}
template <int K> using Kind = std::integral_constant<int, K>;
template <typename F> __device__ __forceinline__ void by_kind(int kind, F f)
{
    if (kind == PLAIN) f(Kind<PLAIN>{});
    else if (kind == ONE) f(Kind<ONE>{});
    else if (kind == EDGE) f(Kind<EDGE>{});
    else f(Kind<ANY>{});
}
// The same for what writes nothing.
template <typename F> __device__ __forceinline__ void by_inner_kind(int kind, F f)
{
    if (kind == PLAIN) f(Kind<PLAIN>{});
    else if (kind == ANY) f(Kind<ANY>{});
    else f(Kind<ONE>{});
}
// Row n of [N][D] at a lane's channels (zeros past D, without the tensor, or where it is not wanted).
template <bool ADJ> __device__ __forceinline__ void seq_row(const float *p, int64_t n, int D, int col0, int l, bool wanted, float (&o)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = p && wanted && col0 + chan<ADJ>(l, v) < D ? p[n * D + col0 + chan<ADJ>(l, v)] : 0.f;
}

// ---- tiles in turn ----------------------------------------------------------------------------------------

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
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
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ float2 map_of(uint64_t w)
{
    return make_float2(__uint_as_float(static_cast<uint32_t>(w)), __uint_as_float(static_cast<uint32_t>(w >> 32)));
}

// The state that enters each run of tile 'rt' (tiles and runs numbered in the direction of the recurrence), from the
// runs' maps in sh.map, left in sh.state.  The warp 'one' does what one warp can, a channel a lane: it folds the maps, passes the
// tile's on and folds the state that enters the tile.  meanwhile() runs once this tile's map is on its way and before
// others are waited for.  False: a wait ran out.  All threads call it, behind a barrier after the maps were written.
template <bool CHAIN, bool REVERSE, int G, typename Meanwhile>
__device__ __forceinline__ bool incoming(Shared<G> &sh, const Chain &ch, int rt, int col0, bool last, Meanwhile meanwhile)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int one = REVERSE ? 0 : WARPS - 1;
    float A = 1.f, B = 0.f, h = 0.f;
    bool far = sh.far == rt;           // a map may be scaled
    if (warp == one) {
        if (far) {
#pragma unroll 1
            for (int r = 0; r < RUNS; ++r) any_then(A, B, sh.map[REVERSE ? RUNS - 1 - r : r][lane]);
        } else {
#pragma unroll
            for (int r = 0; r < RUNS; ++r) then(A, B, sh.map[REVERSE ? RUNS - 1 - r : r][lane]);
        }
    }
    if constexpr (CHAIN) {
        const int grp = rt / G, pos = rt - grp * G;
        uint64_t *own = ch.map + static_cast<size_t>(rt) * ch.Dp + col0 + lane;
        if (warp == one && pos < G - 1 && !last)      // the group's last tile publishes a state instead
            st_relaxed(own, static_cast<uint64_t>(word(B)) << 32 | __float_as_uint(A));
        meanwhile();
        constexpr int WORDS = (G - 1 + WARPS - 1) / WARPS;
        uint64_t w[WORDS];
        const long long began = clock64();
        const uint32_t *state = ch.state + static_cast<size_t>(grp) * ch.Dp + col0 + lane;
        uint32_t from = warp == one && grp > 0 ? ld_relaxed(state) : 0u;
        // only what has not come yet is read again: words that many CTAs wait for are few enough as it is
#pragma unroll
        for (int k = 0; k < WORDS; ++k) w[k] = warp + k * WARPS < pos ? ~0ull : 0ull;
        while (true) {
            bool all = true;
#pragma unroll
            for (int k = 0; k < WORDS; ++k)
                if (__any_sync(0xffffffffu, w[k] == ~0ull)) w[k] = ld_relaxed(own - static_cast<size_t>(pos - warp - k * WARPS) * ch.Dp);
#pragma unroll
            for (int k = 0; k < WORDS; ++k) all = all && w[k] != ~0ull;
            if (__all_sync(0xffffffffu, all)) break;
            if (__any_sync(0xffffffffu, clock64() - began > SPIN)) {
                sh.bad = 1;
                break;
            }
        }
#pragma unroll
        for (int k = 0; k < WORDS; ++k)
            if (warp + k * WARPS < pos) {
                const float2 m = map_of(w[k]);
                sh.before[warp + k * WARPS][lane] = m;
                if (scaled(m.x)) sh.far = rt;
            }
        __syncthreads();
        far = far || sh.far == rt;
        if (sh.bad) return false;
        if (warp == one) {
            // the group's state may come last, and the next group's follows from it: no barrier stands in between
            while (__any_sync(0xffffffffu, from == ~0u)) {
                if (__any_sync(0xffffffffu, clock64() - began > SPIN)) {
                    sh.bad = 1;
                    break;
                }
                from = ld_relaxed(state);
            }
            h = __uint_as_float(from);
            auto pass_on = [&](auto f) {
                if (pos == G - 1 && !last && !sh.bad)
                    st_relaxed(ch.state + static_cast<size_t>(grp + 1) * ch.Dp + col0 + lane, word(f(make_float2(A, B), h)));
            };
            if (far) {
#pragma unroll 1
                for (int p = 0; p < pos; ++p) h = any_apply(sh.before[p][lane], h);
                pass_on(any_apply);
            } else {
#pragma unroll 5
                for (int p = 0; p < pos; ++p) h = apply(sh.before[p][lane], h);
                pass_on(apply);
            }
        }
    } else {
        if (warp == one) sh.before[0][lane] = make_float2(A, B);
        cluster_arrive();
        meanwhile();
        cluster_wait();
        if (warp == one) {
            float2 m[MAX_CLUSTER - 1];
#pragma unroll
            for (int p = 0; p < MAX_CLUSTER - 1; ++p)
                m[p] = p < rt ? ld_cluster(mapa(smem_u32(&sh.before[0][lane]), p)) : make_float2(1.f, 0.f);
            float lowest = 0.f;
#pragma unroll
            for (int p = 0; p < MAX_CLUSTER - 1; ++p) {
                h = p < rt ? apply(m[p], h) : h;
                lowest = fminf(lowest, m[p].x);
            }
            if (scaled(lowest)) {
                h = 0.f;
#pragma unroll
                for (int p = 0; p < MAX_CLUSTER - 1; ++p) h = p < rt ? any_apply(m[p], h) : h;
            }
        }
        cluster_arrive();   // paired with the wait at the kernel's end: no CTA leaves while its map is read
    }
    if (warp == one) {
        auto fold = [&](int k, auto f) {
            const int r = REVERSE ? RUNS - 1 - k : k;
            const float2 m = sh.map[r][lane];
            sh.state[r][lane] = h;
            h = f(m, h);
        };
        if (far) {
#pragma unroll 1
            for (int k = 0; k < RUNS; ++k) fold(k, any_apply);
        } else {
#pragma unroll
            for (int k = 0; k < RUNS; ++k) fold(k, apply);
        }
    }
    __syncthreads();
    return sh.bad == 0;
}

// Walks the tiles of a CTA: load(tile, part) starts the copies of a tile in two parts, work(tile, bounds, release)
// computes it; release runs within it, once part 0's copies may be overwritten, part 1's may when it is done.  work
// returns false when a wait ran out.
template <bool CHAIN, bool REVERSE, int G, typename Load, typename Work>
__device__ __forceinline__ void walk(Shared<G> &sh, const Chain &ch, const PlanView &pv, int D, Load load, Work work)
{
    const int T = pv.T(), nT = tiles_of(T), nC = (D + C - 1) / C;
    const int run = threadIdx.x / 16;
    if (threadIdx.x == 0) sh.bad = 0, sh.far = -1;
    if constexpr (!CHAIN) {
        uint32_t cs, rank;
        asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(cs));
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        const Tile t = tile_of<REVERSE>(static_cast<int>(rank) * nC + static_cast<int>(blockIdx.x / cs), nT, nC);
        if (t.rt < nT) {
            load(t, 0);
            load(t, 1);
            if (threadIdx.x < L / 32) sh.starts.bits[threadIdx.x] = 0;
            if (threadIdx.x == 32) sh.starts.first = 0x7FFFFFFF;
            if (threadIdx.x == 33) sh.after = 0;
            __syncthreads();
            for (int n = threadIdx.x; n <= pv.N(); n += THREADS) {
                const int pos = pv.cu()[n] - t.t0;
                if (pos < 0 || pos > L) continue;
                if (pos < L) atomicOr(&sh.starts.bits[pos >> 5], 1u << (pos & 31));
                else sh.after = 1;
                atomicMin(&sh.starts.first, n);
            }
            cp_wait_all();
            __syncthreads();
            work(t, Bounds(*reinterpret_cast<const uint4 *>(sh.starts.bits), sh.starts.first, sh.after, run, T - t.t0 - run * RUN), [] {});
        } else {                    // clusters are a power of two: some CTAs may be past the end
            cluster_arrive();
            cluster_wait();
            cluster_arrive();
        }
        cluster_wait();
    } else {
        // Every tile goes by a ticket, the first one too, so a tile belongs to a CTA that runs, however few of the grid do (a
        // kernel on another stream may hold the rest of the device for as long as it likes).  Later tickets are drawn ahead (k: in
        // work, k2: next, then the one drawn while k is in work), so that neither the draw nor a tile's starts are waited
        // for.  A CTA works its tiles in the order drawn, so the lowest unfinished tile is always in work, and all that it
        // waits for has been published.
        const int n = nT * nC;
        grid_dep_wait();                     // the kernel before sets the ticket
        if (threadIdx.x == 0) sh.next = atomicAdd(ch.ticket, 1);
        __syncthreads();
        int drawn = 0, k = sh.next;
        uint4 bits = {};
        uint32_t after = 0;
        int first = 0;
        auto words = [&](const Tile &t) {
            bits = *reinterpret_cast<const uint4 *>(ch.starts[t.tt].bits);
            first = ch.starts[t.tt].first;
            after = ch.starts[t.tt + 1].bits[0];
        };
        if (k < n) {
            const Tile t = tile_of<REVERSE>(k, nT, nC);
            load(t, 0);
            load(t, 1);
            words(t);
            if (threadIdx.x == 0) drawn = atomicAdd(ch.ticket, 1);
        }
        while (k < n) {
            const Tile t = tile_of<REVERSE>(k, nT, nC);
            __syncthreads();                 // everyone has read 'next'
            if (threadIdx.x == 0) sh.next = drawn;
            cp_wait_all();
            __syncthreads();
            const int k2 = sh.next;
            const bool ok = work(t, Bounds(bits, first, after, run, T - t.t0 - run * RUN), [&] {
                // called behind a barrier of the CTA: part 0's buffers are free
                if (threadIdx.x == 0 && k2 < n) drawn = atomicAdd(ch.ticket, 1);
                if (k2 < n) {
                    const Tile u = tile_of<REVERSE>(k2, nT, nC);
                    load(u, 0);
                    words(u);
                }
            });
            if (!ok) {
                cp_wait_all();
                if (threadIdx.x == 0) record_status(&g_scan_status, KDA_ERR_TIMEOUT);
                return;
            }
            if (k2 < n) load(tile_of<REVERSE>(k2, nT, nC), 1);
            k = k2;
        }
    }
}

// ---- launches ---------------------------------------------------------------------------------------------

template <typename F> cudaError_t by_type(int type, F f)
{
    if (type == KDA_TYPE_F32) return f(float{});
    if (type == KDA_TYPE_F16) return f(__half{});
    return f(__nv_bfloat16{});
}

// How a tensor's rows lie: all on 16 bytes, all on pairs of elements.
struct Lie {
    bool wide = true, even = true;
    Lie &with(const void *p, int64_t ld, int bytes)
    {
        if (!p) return *this;
        const uintptr_t at = reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * bytes);
        wide = wide && (at & 15) == 0;
        even = even && (at & (2 * bytes - 1)) == 0;
        return *this;
    }
};
// Calls f(copies with an offset, channels in pairs) for how the rows lie.
template <typename F> cudaError_t by_lie(const Lie &lie, F f)
{
    if (lie.wide) return f(std::false_type{}, std::true_type{});
    if (lie.even) return f(std::true_type{}, std::true_type{});
    return f(std::true_type{}, std::false_type{});
}

// A form of a tile kernel: a cluster for few tiles, chains with groups of either length.
template <typename K> struct Form {
    K fn;
    int smem, ctas;         // shared memory, CTAs of an SM
};
// Runs a tile kernel in the form that the numbers of tiles and of channel ranges ask for.
template <typename K, typename... Args>
cudaError_t run(Form<K> cluster, Form<K> wide, Form<K> narrow, const int32_t *plan_host, const int32_t *plan_dev, int D, void *ws, cudaStream_t stream,
                const ScanIn &in, Args... args)
{
    const int T = plan_host[KDA_PH_T], nT = tiles_of(T), nC = (D + C - 1) / C;
    const PlanSig sig = plan_sig(plan_host);
    const Form<K> form = nT <= MAX_CLUSTER ? cluster : nC >= WIDE_RANGES ? wide : narrow;
    if (cudaError_t e = set_dynamic_smem(reinterpret_cast<const void *>(form.fn), form.smem)) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = form.smem;
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
        const int64_t tiles = static_cast<int64_t>(nT) * nC, all = static_cast<int64_t>(form.ctas) * sm_count();
        cfg.gridDim = dim3(static_cast<unsigned>(tiles < all ? tiles : all));
        chain_init<<<static_cast<unsigned>(want < most ? want : most), 256, 0, stream>>>(
            plan_dev, sig, nT, ch.ticket, ch.starts, reinterpret_cast<uint4 *>(ch.state), words);
        if (cudaError_t e = cudaGetLastError()) return e;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
    }
    return cudaLaunchKernelEx(&cfg, form.fn, plan_dev, sig, D, in, ch, args...);
}

}  // namespace
}  // namespace kda
