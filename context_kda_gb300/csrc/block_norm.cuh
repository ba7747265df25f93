// The norms around a block, fused with the block's gate and the residual:
//     n = o * inv_o * w_post,   inv_o = 1 / sqrt(mean_group(o^2) + eps)     (n = o without w_post)
//     u = act(z) * n,           act = 1, sigmoid or silu
//     r' = r + scale * ls * u                                                (stored in the residual's type)
//     y = r' * inv_r * w_pre,   inv_r = 1 / sqrt(mean_row(r'^2) + eps)       (of r' before it is rounded)
// and the gradients of r, o, z, w_post, ls and w_pre from those of r' and y.  Bound by memory: a row is
// read once and stays in registers between its two norms.
//
// The gradient through v -> v / rms(v) is inv (e - hat mean(e hat)) for e = the gradient of hat = v inv.  In a group
// of one channel the two terms cancel down to inv^3 eps e, which is then what is computed.
// Reciprocals and square roots are the hardware's approximations (about 2^-22 relative): fp32 results keep 1e-6.
//
// A CTA of BLOCK threads takes R rows at a time (NT threads a row, 8 NC channels a thread) and walks over
// all its rows, which are copied to a ring in shared memory (cp.async) up to two steps ahead, as many as fit.  With an fp32
// residual above 8192 channels (gradients: 4096, and 8192 all in 16 bits) one step fits: none is ahead, and rows that do not start
// on 16 bytes are read from memory as they are needed, as are all in gradients above 8192 channels with an fp32 residual.
// Sums over a row take one barrier each (none when a row is a warp or less).  U is the run of adjacent channels of a thread: 8 (4 where the
// residual is fp32) where rows start on 16 bytes (a thread copies what it reads itself, without a barrier), else 2 where they
// start on pairs and 1 anywhere (8192 rows in bf16, forward of 3970 channels: 83 us in pairs, 92 us one by one; gradients
// of 1002 channels with an fp32 residual: 50 and 55 us, all in scalar instructions).
// FULL instances are for the usual call: every part but the gate is there and, unless U = 1, D is a multiple of U and
// outputs lie as inputs do.  They decide nothing about that per row, which is a third of the instructions of the
// others and bounds them (16384 x 2048 gradients in bf16: 114 us, 92 us with FULL, both in scalar instructions).
// Column sums (the weights' gradients) stay in registers over all rows of a CTA, are folded over its R rows
// and its groups at the end, and a second kernel adds up the CTAs in order.
//
// Measured on the device (share of a copy's 6.79 TB/s): forward of 65536 x 4096 in bf16 with an fp32 residual 540 us (103 %),
// of 16384 x 4096 all in bf16 84 us (95 %); gradients of 16384 x 4096 with an fp32 residual 216 us (101 %), of 16384 x 2048 in
// bf16 88 us (90 %), of 8192 x 2048 50 us (80 %): the launches, the first rows' way in and the column sums take 6 us of
// any call.  Unaligned rows are bound by instructions, gradients of 8198 x 1001 in fp32 56 us (69 %); above 4096 channels the weights
// are read again for every row, 8192 x 8192 in bf16 115 to 119 us (83 to 86 %) and gradients 346 us (46 %: the column sums leave
// no registers for the row, and some of it is kept in local memory, most above 8192 channels: 4096 x 16384 1022 us, 15 %).
#pragma once

#include <type_traits>

#include "elem.cuh"
#include "kda_internal.cuh"
#include "tc.cuh"

namespace kda {
namespace norm {

constexpr int MAX_GRID = 304;   // CTAs of a launch: rows of the backward's column sums

// What both directions take besides NormIn.
struct Shape {
    uint32_t T;
    int D, G, NT;                // channels, channels of a group, threads of a row
    bool wide_w;                 // weights start on 16 bytes
    bool wide_r, wide_a, wide_b; // outputs whose rows start on 16 bytes: residual, the others
    float inv_d, inv_g;          // 1 / D, 1 / G
};

template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void unpack(uint32_t w, float *v, const __nv_bfloat16 *)
{
    v[0] = __uint_as_float(w << 16);
    v[1] = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void unpack(uint32_t w, float *v, const __half *)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    v[0] = f.x;
    v[1] = f.y;
}
__device__ __forceinline__ void unpack(uint32_t w, float *v, const float *) { v[0] = __uint_as_float(w); }

// Channel j of a thread's NE of its row.  U > 2: runs of U, NT threads apart.  U <= 2: W threads take W NE adjacent channels,
// their runs W threads apart, so that all but a thread's first are at offsets that the compiler knows; W is a warp, or half
// of one for rows of up to 128 channels (gradients of 46838 x 113 in fp32: 32 us, 45 us with W = 32).
template <int U, int NE, int W> __device__ __forceinline__ int channel_of(int ti, int NT, int j)
{
    if constexpr (U > 2) return (ti + j / U * NT) * U + j % U;
    else return ti / W * (W * NE) + ti % W * U + j / U * (W * U) + j % U;
}

// A thread's channels of a row of X, in runs of U: run q starts at channel (ti + q NT) U.  U = 8, or 4 where the
// residual is fp32: rows start on 16 bytes; every thread copies its own channels into its own slots.  A run is one
// copy, so that a warp's copies and stores are adjacent bytes: with 8 channels of fp32 a thread, in two pieces each,
// every sector moved twice (16384 x 2048 in fp32: 157 us, 109 us with 4).
template <typename X, int BLOCK, int NC, int U, int W> struct Row {
    static constexpr int NE = 8 * NC, NU = NE / U, RUN = U * static_cast<int>(sizeof(X));     // runs, bytes of a run
    static constexpr int BYTES = NE * static_cast<int>(sizeof(X)) * BLOCK;                    // of the CTA, per step
    static_assert(RUN == 16 || RUN == 8, "one copy a run");
    static __device__ __forceinline__ void copy(uint32_t dst, const X *src, int bytes)
    {
        if constexpr (RUN == 16) copy16(dst, src, bytes);
        else copy8(dst, src, bytes);
    }

    // Copies the row's channels below D to the slots at 'base'; 'row' is the row's first channel.
    static __device__ __forceinline__ void fetch(uint32_t base, const X *row, const X *, int ti, int NT, int D, bool)
    {
#pragma unroll
        for (int q = 0; q < NU; ++q) {
            const int c = (ti + q * NT) * U, left = (D - c) * static_cast<int>(sizeof(X));
            const int bytes = left < 0 ? 0 : left > RUN ? RUN : left;
            copy(base + (q * BLOCK + threadIdx.x) * RUN, bytes ? row + c : row, bytes);
        }
    }
    // The same where D is a multiple of 8 (zeros from D on).
    static __device__ __forceinline__ void fetch_full(uint32_t base, const X *row, const X *, int ti, int NT, int D, bool)
    {
#pragma unroll
        for (int q = 0; q < NU; ++q) {
            const bool there = (ti + q * NT) * U < D;
            copy(base + (q * BLOCK + threadIdx.x) * RUN, there ? row + (ti + q * NT) * U : row, there ? RUN : 0);
        }
    }
    // Zeros in place of a row past the end ('any': some address of the tensor).
    static __device__ __forceinline__ void fetch_none(uint32_t base, const X *any)
    {
#pragma unroll
        for (int q = 0; q < NU; ++q) copy(base + (q * BLOCK + threadIdx.x) * RUN, any, 0);
    }
    // The channels as fp32 (zeros from D on): from the slots, or from the row where there is no ring.
    template <bool RING>
    static __device__ __forceinline__ void read(const unsigned char *base, const X *row, int ti, int NT, int D, bool in, float (&v)[NE])
    {
        if constexpr (RING) {
            constexpr int EPW = 4 / static_cast<int>(sizeof(X));
#pragma unroll
            for (int q = 0; q < NU; ++q) {
                const unsigned char *at = base + (q * BLOCK + threadIdx.x) * RUN;
                if constexpr (RUN == 16) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(at);
                    unpack(w.x, v + q * U, row);
                    unpack(w.y, v + q * U + EPW, row);
                    unpack(w.z, v + q * U + 2 * EPW, row);
                    unpack(w.w, v + q * U + 3 * EPW, row);
                } else {
                    const uint2 w = *reinterpret_cast<const uint2 *>(at);
                    unpack(w.x, v + q * U, row);
                    unpack(w.y, v + q * U + EPW, row);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < NE; ++j) {
                const int c = channel_of<U, NE, W>(ti, NT, j);
                v[j] = in && c < D ? to_f32(row[c]) : 0.f;
            }
        }
    }
    // The channels below D; FULL: D is a multiple of 8 and the row starts on 16 bytes (else as 'wide' says).
    template <bool FULL> static __device__ __forceinline__ void write(X *row, int ti, int NT, int D, bool wide, const float (&v)[NE])
    {
#pragma unroll
        for (int q = 0; q < NU; ++q) {
            const int c = (ti + q * NT) * U;
            X e[U];
#pragma unroll
            for (int j = 0; j < U; ++j) e[j] = from_f32<X>(v[q * U + j]);
            if (FULL ? c < D : wide && c + U <= D) {
                if constexpr (RUN == 16) *reinterpret_cast<uint4 *>(row + c) = *reinterpret_cast<const uint4 *>(e);
                else *reinterpret_cast<uint2 *>(row + c) = *reinterpret_cast<const uint2 *>(e);
            } else if (!FULL) {
#pragma unroll
                for (int j = 0; j < U; ++j)
                    if (c + j < D) row[c + j] = e[j];
            }
        }
    }
};

// U = 1: any rows; U = 2: D is even and rows start on pairs.  A row is copied 16 bytes at a time with the 16 bytes it
// starts in, by all of its threads, so it is read behind a barrier of them, from an offset.
template <typename X, int BLOCK, int NC, int U, int W> struct Staged {
    static constexpr int NE = 8 * NC, SIZE = static_cast<int>(sizeof(X)), EPC = 16 / SIZE;
    using Pair = typename std::conditional<SIZE == 4, uint2, uint32_t>::type;
    static constexpr int BYTES = BLOCK * NE * SIZE + BLOCK / W * 16;     // of the CTA, per step: a row has W threads at least
    static __device__ __forceinline__ int place(int NT) { return static_cast<int>(threadIdx.x / NT) * (NT * NE * SIZE + 16); }

    // 'inner': 16 bytes before and behind the row belong to the tensor's rows, so whole copies may be read.
    static __device__ __forceinline__ void fetch(uint32_t base, const X *row, const X *tensor, int ti, int NT, int D, bool inner)
    {
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u), end = off + D * SIZE;
        const char *p = reinterpret_cast<const char *>(row) - off;
        base += place(NT);
        if (inner) {
#pragma unroll
            for (int k = 0; k <= NE * SIZE / 16; ++k) {
                const int at = (ti + k * NT) * 16;
                if (at < end) copy16(base + at, p + at, 16);
            }
            return;
        }
#pragma unroll 1
        for (int k = 0; k <= NE * SIZE / 16; ++k) {
            const int at = (ti + k * NT) * 16;
            if (at >= end) break;
            const int bytes = end - at > 16 ? 16 : end - at;
            if (p + at < reinterpret_cast<const char *>(tensor)) {     // the tensor starts here: nothing before it is read
                for (int e = off / SIZE; e < EPC && at + e * SIZE < end; ++e)
                    store(base + at + e * SIZE, reinterpret_cast<const X *>(p + at)[e]);
            } else {
                copy16(base + at, p + at, bytes);
            }
        }
    }
    static __device__ __forceinline__ void store(uint32_t at, X v)
    {
        if constexpr (SIZE == 4)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(to_f32(v)) : "memory");
        else
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(*reinterpret_cast<const unsigned short *>(&v)) : "memory");
    }
    static __device__ __forceinline__ void fetch_full(uint32_t base, const X *row, const X *tensor, int ti, int NT, int D, bool inner)
    {
        fetch(base, row, tensor, ti, NT, D, inner);
    }
    static __device__ __forceinline__ void fetch_none(uint32_t, const X *) {}
    template <bool RING>
    static __device__ __forceinline__ void read(const unsigned char *base, const X *row, int ti, int NT, int D, bool in, float (&v)[NE])
    {
        const X *p = RING ? reinterpret_cast<const X *>(base + place(NT) + (reinterpret_cast<uintptr_t>(row) & 15u)) : row;
        const int some = in ? D : 0;
        if constexpr (U == 2) {
#pragma unroll
            for (int j = 0; j < NE; j += 2) {
                const int c = channel_of<U, NE, W>(ti, NT, j);
                X e[2] = {from_f32<X>(0.f), from_f32<X>(0.f)};
                if (c < some) *reinterpret_cast<Pair *>(e) = *reinterpret_cast<const Pair *>(p + c);
                v[j] = to_f32(e[0]);
                v[j + 1] = to_f32(e[1]);
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            const int c = channel_of<U, NE, W>(ti, NT, j);
            v[j] = c < some ? to_f32(p[c]) : 0.f;
        }
    }
    template <bool> static __device__ __forceinline__ void write(X *row, int ti, int NT, int D, bool, const float (&v)[NE])
    {
        if constexpr (U == 2) {
#pragma unroll
            for (int j = 0; j < NE; j += 2) {
                const int c = channel_of<U, NE, W>(ti, NT, j);
                const X e[2] = {from_f32<X>(v[j]), from_f32<X>(v[j + 1])};
                if (c < D) *reinterpret_cast<Pair *>(row + c) = *reinterpret_cast<const Pair *>(e);
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < NE; ++j)
            if (channel_of<U, NE, W>(ti, NT, j) < D) row[channel_of<U, NE, W>(ti, NT, j)] = from_f32<X>(v[j]);
    }
};
template <typename X, int BLOCK, int NC, int W> struct Row<X, BLOCK, NC, 1, W> : Staged<X, BLOCK, NC, 1, W> {};
template <typename X, int BLOCK, int NC, int W> struct Row<X, BLOCK, NC, 2, W> : Staged<X, BLOCK, NC, 2, W> {};

// Sums over a row's NT threads (a power of two); every thread gets them.  Rows wider than a warp take one barrier: the
// warps' sums go to one of two buffers in turn, 'turn' being the number of the CTA's step.  An object serves one sum a
// step, whichever others the call has: a warp writes a buffer again two steps later, behind the barrier of the step in
// between, which no warp reaches before it has read what the first of them left.
template <int BLOCK> struct Sums {
    float part[2][2][BLOCK / 32];
    static __device__ __forceinline__ float xor_add(float v, int m) { return v + __shfl_xor_sync(0xffffffffu, v, m); }
    // A sum over the lanes that differ in the bits of n - 1 (n a power of two).
    static __device__ __forceinline__ float lanes(float v, int n)
    {
        if (n > 16) v = xor_add(v, 16);
        if (n > 8) v = xor_add(v, 8);
        if (n > 4) v = xor_add(v, 4);
        if (n > 2) v = xor_add(v, 2);
        if (n > 1) v = xor_add(v, 1);
        return v;
    }
    __device__ __forceinline__ float over_row(float v, int NT, int turn)
    {
        v = lanes(v, NT < 32 ? NT : 32);
        if (NT <= 32) return v;
        const int warp = threadIdx.x >> 5, n = NT >> 5, w0 = warp & ~(n - 1);
        if ((threadIdx.x & 31) == 0) part[turn & 1][0][warp] = v;
        __syncthreads();
        return lanes(part[turn & 1][0][w0 + (threadIdx.x & (n - 1))], n);
    }
    // Two sums at once: each half of a warp takes one of them.
    __device__ __forceinline__ void over_row(float &u, float &v, int NT, int turn)
    {
        if (NT < 32) {
            u = lanes(u, NT);
            v = lanes(v, NT);
            return;
        }
        const bool upper = threadIdx.x & 16;
        float w = (upper ? v : u) + __shfl_xor_sync(0xffffffffu, upper ? u : v, 16);
        w = lanes(w, 16);
        if (NT > 32) {
            const int warp = threadIdx.x >> 5, n = NT >> 5, w0 = warp & ~(n - 1);
            if ((threadIdx.x & 15) == 0) part[turn & 1][upper][warp] = w;
            __syncthreads();
            if (n == 32) {       // more partial sums than lanes of a half
                u = lanes(part[turn & 1][0][threadIdx.x & 31], 32);
                v = lanes(part[turn & 1][1][threadIdx.x & 31], 32);
                return;
            }
            w = lanes(part[turn & 1][upper][w0 + (threadIdx.x & (n - 1))], n);
        }
        u = __shfl_sync(0xffffffffu, w, 0);
        v = __shfl_sync(0xffffffffu, w, 16);
    }
};

// Row t of a tensor of rows 'ld' bytes apart.
template <typename X> __device__ __forceinline__ X *row_at(X *p, uint32_t t, uint32_t ld)
{
    using Byte = typename std::conditional<std::is_const<X>::value, const char, char>::type;
    return reinterpret_cast<X *>(reinterpret_cast<Byte *>(p) + static_cast<uint64_t>(t) * ld);
}

// Sums over each run's group of G channels (G < D), in place.  U > 2: G spans G / U lanes of consecutive threads, which
// may be two warps when U = 4 (NT U is then at least G; buffers in turn as above, so an object serves one sum a row).  U <= 2: a
// run's lanes, and several runs of its W threads where a run of them is less.
template <int BLOCK, int NU, int U, int W> struct GroupSums {
    float part[U == 4 ? 2 : 1][U == 4 ? NU : 1][BLOCK / 32];
    static __device__ __forceinline__ void fold(float (&v)[NU], int m)
    {
#pragma unroll
        for (int q = 0; q < NU; ++q) v[q] += __shfl_xor_sync(0xffffffffu, v[q], m);
    }
    // Sums of n adjacent runs.
    static __device__ __forceinline__ void join(float (&v)[NU], int n)
    {
#pragma unroll
        for (int m = 1; m < NU; m *= 2) {
            if (m >= n) return;
#pragma unroll
            for (int q = 0; q < NU; ++q)
                if (!(q & m)) v[q] = v[q | m] = v[q] + v[q | m];
        }
    }
    __device__ __forceinline__ void over_group(float (&v)[NU], int G, int turn)
    {
        const int lanes = G / U;
#pragma unroll 1
        for (int m = (lanes < W ? lanes : W) >> 1; m > 8; m >>= 1) fold(v, m);
        if (lanes >= 16) fold(v, 8);
        if (lanes >= 8) fold(v, 4);
        fold(v, 2);        // a group is four lanes at least
        fold(v, 1);
        if constexpr (U <= 2) join(v, lanes / W);
        if constexpr (U == 4) {
            if (lanes <= 32) return;
            const int warp = threadIdx.x >> 5, n = lanes >> 5, w0 = warp & ~(n - 1);
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int q = 0; q < NU; ++q) part[turn & 1][q][warp] = v[q];
            __syncthreads();
#pragma unroll
            for (int q = 0; q < NU; ++q) {
                float s = 0.f;
                for (int w = 0; w < n; ++w) s += part[turn & 1][q][w0 + w];
                v[q] = s;
            }
        }
    }
};

__device__ __forceinline__ float rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float inv_rms(float mean_sq, float eps) { return rsqrtf(mean_sq + eps); }

// Two channels in one instruction (16384 x 2048 gradients in bf16: 88 us, 92 us in scalar ones; forward of 8192 x 3970
// 80 and 83 us).
__device__ __forceinline__ float2 two(float x) { return make_float2(x, x); }
template <int N> __device__ __forceinline__ float2 at(const float (&v)[N], int j) { return make_float2(v[j], v[j + 1]); }
template <int N> __device__ __forceinline__ void set(float (&v)[N], int j, float2 p) { v[j] = p.x, v[j + 1] = p.y; }
__device__ __forceinline__ float2 sigmoid2(float2 z)
{
    const float2 w = mul2(z, two(-1.4426950408889634f));
    const float2 d = fma2(make_float2(tc::ex2_ftz(w.x), tc::ex2_ftz(w.y)), two(1.f), two(1.f));
    return make_float2(rcp(d.x), rcp(d.y));      // exp = infinity: 0
}
// Sums over runs of U of products that come in pairs of channels.
template <int NE, int U> struct RunSums {
    float2 s[U == 1 ? NE / 2 : NE / U];
    __device__ __forceinline__ RunSums()
    {
#pragma unroll
        for (float2 &p : s) p = two(0.f);
    }
    __device__ __forceinline__ void add(int j, float2 a, float2 b)
    {
        float2 &p = s[U == 1 ? j / 2 : j / U];
        p = fma2(a, b, p);
    }
    __device__ __forceinline__ float run(int q) const { return U == 1 ? (q % 2 ? s[q / 2].y : s[q / 2].x) : s[q].x + s[q].y; }
};

// The gradient of a group of one channel from e, the gradient of hat = v inv.
__device__ __forceinline__ float unit_grad_of_one(float e, float inv, float eps) { return e * (eps * inv) * (inv * inv); }

// A weight's values at a thread's channels (1 where it is absent), times 'scale': kept in registers when they are few,
// read again for every row otherwise, four at a time where the weight starts on 16 bytes ('wide') and D allows.
template <int NE, int U, int W, typename I>
__device__ __forceinline__ void weights(const float *w, float scale, I index, int ti, int NT, int D, bool wide, float (&v)[NE])
{
    if constexpr (U >= 4) {
        if (w && wide && D % U == 0) {
#pragma unroll
            for (int j = 0; j < NE; j += 4) {
                const int c = channel_of<U, NE, W>(ti, NT, j);
                const float4 f = c < D ? __ldg(reinterpret_cast<const float4 *>(w + index(c))) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[j] = scale * f.x;
                v[j + 1] = scale * f.y;
                v[j + 2] = scale * f.z;
                v[j + 3] = scale * f.w;
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        const int c = channel_of<U, NE, W>(ti, NT, j);
        v[j] = c < D ? scale * (w ? __ldg(w + index(c)) : 1.f) : 0.f;
    }
}

// ---- forward ----------------------------------------------------------------------------------------------

template <typename R, typename E, int BLOCK, int NC, int U, int W> struct Forward {
    using RowR = Row<R, BLOCK, NC, U, W>;
    using RowE = Row<E, BLOCK, NC, U, W>;
    static constexpr int NE = 8 * NC, NU = NE / U;
    static constexpr int STEP = RowR::BYTES + 2 * RowE::BYTES;
    static constexpr int CTAS = NC == 1 ? 1024 / BLOCK : 1;                       // of an SM
    static constexpr int FIT = 220 / CTAS * 1024 / STEP;
    static constexpr int S = FIT > 3 ? 3 : FIT == 1 && U <= 2 ? 0 : FIT;      // steps in the ring; 0: no ring
    static constexpr int SMEM = S * STEP;
};

template <typename R, typename E, int BLOCK, int NC, int U, bool FULL, int W>
__global__ void __launch_bounds__(BLOCK, Forward<R, E, BLOCK, NC, U, W>::CTAS) forward(Shape s, NormIn a, R *r_out, int64_t ldro, E *y, int64_t ldy)
{
    using F = Forward<R, E, BLOCK, NC, U, W>;
    using RowR = typename F::RowR;
    using RowE = typename F::RowE;
    constexpr int NE = F::NE, NU = F::NU, S = F::S;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ Sums<BLOCK> sums, sums_o;
    __shared__ GroupSums<BLOCK, NU, U, W> groups;
    const R *r = static_cast<const R *>(a.r);
    const E *o = static_cast<const E *>(a.o), *z = static_cast<const E *>(a.z);
    const int D = s.D, G = s.G, NT = s.NT, ti = threadIdx.x & (NT - 1), rows = BLOCK / NT, rr = threadIdx.x / NT;
    const float inv_d = s.inv_d, inv_g = s.inv_g;
    const uint32_t step = gridDim.x * rows;
    const uint32_t lr = a.ldr * sizeof(R), lo = a.ldo * sizeof(E), lz = a.ldz * sizeof(E);
    const uint32_t base = tc::smem_u32(ring);
    const bool has_r = FULL || r, has_o = FULL || o, has_post = FULL || a.w_post, has_out = FULL || r_out, has_y = FULL || y;

    auto fetch = [&](int slot, uint32_t t) {
        const uint32_t b = base + slot * F::STEP;
        if (t < s.T) {
            const bool inner = t >= 16 && t + 16 < s.T;      // rows are two bytes at least
            if constexpr (FULL) {
                RowR::fetch_full(b, row_at(r, t, lr), r, ti, NT, D, inner);
                RowE::fetch_full(b + RowR::BYTES, row_at(o, t, lo), o, ti, NT, D, inner);
                if (z) RowE::fetch_full(b + RowR::BYTES + RowE::BYTES, row_at(z, t, lz), z, ti, NT, D, inner);
            } else {
                if (r) RowR::fetch(b, row_at(r, t, lr), r, ti, NT, D, inner);
                if (o) RowE::fetch(b + RowR::BYTES, row_at(o, t, lo), o, ti, NT, D, inner);
                if (z) RowE::fetch(b + RowR::BYTES + RowE::BYTES, row_at(z, t, lz), z, ti, NT, D, inner);
            }
        } else {
            if (has_r) RowR::fetch_none(b, r);
            if (has_o) RowE::fetch_none(b + RowR::BYTES, o);
            if (z) RowE::fetch_none(b + RowR::BYTES + RowE::BYTES, z);
        }
    };
    uint32_t t0 = blockIdx.x * rows;
    if constexpr (S > 0)
        for (int k = 0; k < S - 1; ++k) {
            fetch(k, t0 + rr + k * step);
            cp_commit();
        }
    auto in_group = [&](int c) { return G == D ? c : c & (G - 1); };
    auto in_row = [&](int c) { return c; };
    float wl[NE], wr[NE];      // scale * ls * w_post, w_pre
    auto branch_weights = [&] {
        weights<NE, U, W>(a.ls, a.scale, in_row, ti, NT, D, s.wide_w, wl);
        if (has_post) {
            float wg[NE];
            weights<NE, U, W>(a.w_post, 1.f, in_group, ti, NT, D, s.wide_w, wg);
#pragma unroll
            for (int j = 0; j < NE; ++j) wl[j] *= wg[j];
        }
    };
    if constexpr (NC == 1) {
        branch_weights();
        if (has_y) weights<NE, U, W>(a.w_pre, 1.f, in_row, ti, NT, D, s.wide_w, wr);
    }
    int slot = 0, turn = 0;
    for (; t0 < s.T; t0 += step) {
        const uint32_t t = t0 + rr;
        const bool in = t < s.T;
        auto ahead = [&] {
            fetch(slot == 0 ? S - 1 : slot - 1, t + (S - 1) * step);
            cp_commit();
        };
        if constexpr (S > 0 && U > 2) {
            ahead();
            cp_wait<S - 1>();
        } else if constexpr (S > 0) {
            cp_wait<S - 2>();
            if (NT > 32) __syncthreads();      // the row is there, and the one before it has been read
            else __syncwarp();
            ahead();
        }
        const unsigned char *b = ring + slot * F::STEP;
        float v[NE];
        if (has_r) {
            RowR::template read<(S > 0)>(b, row_at(r, t, lr), ti, NT, D, in, v);
        } else {
#pragma unroll
            for (int j = 0; j < NE; ++j) v[j] = 0.f;
        }
        if (has_o) {
            float n[NE];
            RowE::template read<(S > 0)>(b + RowR::BYTES, row_at(o, t, lo), ti, NT, D, in, n);
            float g[NE];
            if (z) RowE::template read<(S > 0)>(b + RowR::BYTES + RowE::BYTES, row_at(z, t, lz), ti, NT, D, in, g);
            if (has_post) {
                float ss[NU];
                RunSums<NE, U> n2;
#pragma unroll
                for (int j = 0; j < NE; j += 2) n2.add(j, at(n, j), at(n, j));
#pragma unroll
                for (int q = 0; q < NU; ++q) ss[q] = n2.run(q);
                if (G == D) {
                    float all = 0.f;
#pragma unroll
                    for (int q = 0; q < NU; ++q) all += ss[q];
                    const float inv = inv_rms(sums_o.over_row(all, NT, turn) * inv_g, a.eps);
#pragma unroll
                    for (int j = 0; j < NE; j += 2) set(n, j, mul2(at(n, j), two(inv)));
                } else {
                    groups.over_group(ss, G, turn);
#pragma unroll
                    for (int q = 0; q < NU; ++q) {
                        const float inv = inv_rms(ss[q] * inv_g, a.eps);
#pragma unroll
                        for (int j = 0; j < U; ++j) n[q * U + j] *= inv;
                    }
                }
            }
            if (a.gate == KDA_GATE_SIGMOID) {
#pragma unroll
                for (int j = 0; j < NE; j += 2) set(n, j, mul2(at(n, j), sigmoid2(at(g, j))));
            } else if (a.gate == KDA_GATE_SILU) {
#pragma unroll
                for (int j = 0; j < NE; j += 2) set(n, j, mul2(at(n, j), mul2(at(g, j), sigmoid2(at(g, j)))));
            }
            if constexpr (NC > 1) branch_weights();
#pragma unroll
            for (int j = 0; j < NE; j += 2) set(v, j, fma2(at(wl, j), at(n, j), at(v, j)));
        }
        if (has_out && in) RowR::template write<FULL>(row_at(r_out, t, static_cast<uint32_t>(ldro * sizeof(R))), ti, NT, D, s.wide_r, v);
        if (has_y) {
            float2 s2 = two(0.f);
#pragma unroll
            for (int j = 0; j < NE; j += 2) s2 = fma2(at(v, j), at(v, j), s2);
            const float ss = s2.x + s2.y;
            const float inv = inv_rms(sums.over_row(ss, NT, turn) * inv_d, a.eps);
            if constexpr (NC > 1) weights<NE, U, W>(a.w_pre, 1.f, in_row, ti, NT, D, s.wide_w, wr);
#pragma unroll
            for (int j = 0; j < NE; j += 2) set(v, j, mul2(at(v, j), mul2(two(inv), at(wr, j))));
            if (in) RowE::template write<FULL>(row_at(y, t, static_cast<uint32_t>(ldy * sizeof(E))), ti, NT, D, s.wide_a, v);
        }
        ++turn;
        if constexpr (S > 0) slot = slot + 1 == S ? 0 : slot + 1;
    }
}

// ---- backward ---------------------------------------------------------------------------------------------

template <typename R, typename E, int BLOCK, int NC, int U, int W> struct Backward {
    using RowR = Row<R, BLOCK, NC, U, W>;
    using RowE = Row<E, BLOCK, NC, U, W>;
    static constexpr int NE = 8 * NC, NU = NE / U;
    static constexpr int STEP = 2 * RowR::BYTES + 3 * RowE::BYTES;
    static constexpr int CTAS = BLOCK == 256 ? 2 : 1;                             // of an SM
    static constexpr int FIT = 220 / CTAS * 1024 / STEP;
    static constexpr int S = FIT > 3 ? 3 : FIT == 1 && U <= 2 ? 0 : FIT;
    static constexpr int FOLD = BLOCK * NE * 4;      // the column sums of the CTA, folded at the end
    static constexpr int SMEM = S * STEP > FOLD ? S * STEP : FOLD;
};

// part: [grid][G + 2 D], the CTA's sums for w_post, ls and w_pre.
template <typename R, typename E, int BLOCK, int NC, int U, bool FULL, int W>
__global__ void __launch_bounds__(BLOCK, Backward<R, E, BLOCK, NC, U, W>::CTAS) backward(Shape s, NormIn a, const R *dro, int64_t lddro,
                                                                                      const E *dy, int64_t lddy, NormGrads g, float *part)
{
    using B = Backward<R, E, BLOCK, NC, U, W>;
    using RowR = typename B::RowR;
    using RowE = typename B::RowE;
    constexpr int NE = B::NE, NU = B::NU, S = B::S;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ Sums<BLOCK> sums, sums_o, sums_e;
    __shared__ GroupSums<BLOCK, NU, U, W> groups_o, groups_e;
    const R *r = static_cast<const R *>(a.r);
    const E *o = static_cast<const E *>(a.o), *z = static_cast<const E *>(a.z);
    R *dr = static_cast<R *>(g.dr);
    E *d_o = static_cast<E *>(g.d_o), *dz = static_cast<E *>(g.dz);
    const int D = s.D, G = s.G, NT = s.NT, ti = threadIdx.x & (NT - 1), rows = BLOCK / NT, rr = threadIdx.x / NT;
    const float inv_d = s.inv_d, inv_g = s.inv_g;
    const uint32_t step = gridDim.x * rows;
    const uint32_t lr = a.ldr * sizeof(R), lo = a.ldo * sizeof(E), lz = a.ldz * sizeof(E);
    const uint32_t ldr = lddro * sizeof(R), ldy = lddy * sizeof(E);
    const uint32_t base = tc::smem_u32(ring);
    constexpr int O_DRO = RowR::BYTES, O_DY = 2 * RowR::BYTES, O_O = O_DY + RowE::BYTES, O_Z = O_O + RowE::BYTES;
    const bool has_pre = FULL || a.w_pre, has_dro = FULL || dro, has_o = FULL || o, has_post = FULL || a.w_post;

    auto fetch = [&](int slot, uint32_t t) {
        const uint32_t b = base + slot * B::STEP;
        if (t < s.T) {
            const bool inner = t >= 16 && t + 16 < s.T;      // rows are two bytes at least
            if constexpr (FULL) {
                RowR::fetch_full(b, row_at(r, t, lr), r, ti, NT, D, inner);
                RowE::fetch_full(b + O_DY, row_at(dy, t, ldy), dy, ti, NT, D, inner);
                RowR::fetch_full(b + O_DRO, row_at(dro, t, ldr), dro, ti, NT, D, inner);
                RowE::fetch_full(b + O_O, row_at(o, t, lo), o, ti, NT, D, inner);
                if (z) RowE::fetch_full(b + O_Z, row_at(z, t, lz), z, ti, NT, D, inner);
            } else {
                if (a.w_pre) {
                    RowR::fetch(b, row_at(r, t, lr), r, ti, NT, D, inner);
                    RowE::fetch(b + O_DY, row_at(dy, t, ldy), dy, ti, NT, D, inner);
                }
                if (dro) RowR::fetch(b + O_DRO, row_at(dro, t, ldr), dro, ti, NT, D, inner);
                if (o) RowE::fetch(b + O_O, row_at(o, t, lo), o, ti, NT, D, inner);
                if (z) RowE::fetch(b + O_Z, row_at(z, t, lz), z, ti, NT, D, inner);
            }
        } else {
            if (has_pre) {
                RowR::fetch_none(b, r);
                RowE::fetch_none(b + O_DY, dy);
            }
            if (has_dro) RowR::fetch_none(b + O_DRO, dro);
            if (has_o) RowE::fetch_none(b + O_O, o);
            if (z) RowE::fetch_none(b + O_Z, z);
        }
    };
    uint32_t t0 = blockIdx.x * rows;
    if constexpr (S > 0)
        for (int k = 0; k < S - 1; ++k) {
            fetch(k, t0 + rr + k * step);
            cp_commit();
        }
    auto in_group = [&](int c) { return G == D ? c : c & (G - 1); };
    auto in_row = [&](int c) { return c; };
    float acc_g[NE], acc_l[NE], acc_r[NE];
#pragma unroll
    for (int j = 0; j < NE; ++j) acc_g[j] = acc_l[j] = acc_r[j] = 0.f;
    float wg[NE], wl[NE], wr[NE];
    if constexpr (NC == 1) {
        weights<NE, U, W>(a.w_post, 1.f, in_group, ti, NT, D, s.wide_w, wg);
        weights<NE, U, W>(a.ls, a.scale, in_row, ti, NT, D, s.wide_w, wl);
        weights<NE, U, W>(a.w_pre, 1.f, in_row, ti, NT, D, s.wide_w, wr);
    }
    int slot = 0, turn = 0;
    for (; t0 < s.T; t0 += step) {
        const uint32_t t = t0 + rr;
        const bool in = t < s.T;
        auto ahead = [&] {
            fetch(slot == 0 ? S - 1 : slot - 1, t + (S - 1) * step);
            cp_commit();
        };
        if constexpr (S > 0 && U > 2) {
            ahead();
            cp_wait<S - 1>();
        } else if constexpr (S > 0) {
            cp_wait<S - 2>();
            if (NT > 32) __syncthreads();      // the row is there, and the one before it has been read
            else __syncwarp();
            ahead();
        }
        const unsigned char *b = ring + slot * B::STEP;
        float ov[NE], rv[NE], e[NE];
        float ss = 0.f, ev_r = 0.f;             // sums of r^2 and of e r over the row
        float so[NU];                           // of o^2 over the groups
        auto inverse = [&](float sum) { return in ? inv_rms(sum * inv_g, a.eps) : 0.f; };     // no row: zeros, also with eps = 0
        if (has_pre) {
            RowR::template read<(S > 0)>(b, row_at(r, t, lr), ti, NT, D, in, rv);
            RowE::template read<(S > 0)>(b + O_DY, row_at(dy, t, ldy), ti, NT, D, in, e);
            if constexpr (NC > 1) weights<NE, U, W>(a.w_pre, 1.f, in_row, ti, NT, D, s.wide_w, wr);
            float2 s2 = two(0.f), e2 = two(0.f);
#pragma unroll
            for (int j = 0; j < NE; j += 2) {
                s2 = fma2(at(rv, j), at(rv, j), s2);
                e2 = fma2(mul2(at(e, j), at(wr, j)), at(rv, j), e2);
            }
            ss = s2.x + s2.y;
            ev_r = e2.x + e2.y;
        }
        if (has_o) {
            RowE::template read<(S > 0)>(b + O_O, row_at(o, t, lo), ti, NT, D, in, ov);
            if (has_post) {
                float all = 0.f;
                RunSums<NE, U> o2;
#pragma unroll
                for (int j = 0; j < NE; j += 2) o2.add(j, at(ov, j), at(ov, j));
#pragma unroll
                for (int q = 0; q < NU; ++q) all += so[q] = o2.run(q);
                if (G == D) {
                    all = sums_o.over_row(all, NT, turn);
                    if constexpr (U <= 2) all = inverse(all);      // one for all of the thread's runs
#pragma unroll
                    for (int q = 0; q < NU; ++q) so[q] = all;
                } else {
                    groups_o.over_group(so, G, turn);
                    if constexpr (U <= 2)
#pragma unroll
                        for (int q = 0; q < NU; ++q) so[q] = inverse(so[q]);
                }
            }
        }
        float v[NE];                            // the gradient of r', then that of o
        if (has_dro) {
            RowR::template read<(S > 0)>(b + O_DRO, row_at(dro, t, ldr), ti, NT, D, in, v);
        } else {
#pragma unroll
            for (int j = 0; j < NE; ++j) v[j] = 0.f;
        }
        if (has_pre) {
            sums.over_row(ss, ev_r, NT, turn);
            const float inv = in ? inv_rms(ss * inv_d, a.eps) : 0.f, mean = ev_r * inv_d * inv;   // no row: as above
            if ((!FULL || U == 1) && D == 1) {
                v[0] += unit_grad_of_one(e[0] * wr[0], inv, a.eps);
                acc_r[0] = fmaf(e[0], rv[0] * inv, acc_r[0]);
            } else {
#pragma unroll
                for (int j = 0; j < NE; j += 2) {
                    const float2 hat = mul2(at(rv, j), two(inv));
                    set(acc_r, j, fma2(at(e, j), hat, at(acc_r, j)));
                    set(v, j, fma2(two(inv), fma2(hat, two(-mean), mul2(at(e, j), at(wr, j))), at(v, j)));
                }
            }
        }
        if (dr && in) RowR::template write<FULL>(row_at(dr, t, static_cast<uint32_t>(g.lddr * sizeof(R))), ti, NT, D, s.wide_r, v);
        if (has_o) {
            float gz[NE];
            if (z) RowE::template read<(S > 0)>(b + O_Z, row_at(z, t, lz), ti, NT, D, in, gz);
            if constexpr (NC > 1) {
                weights<NE, U, W>(a.w_post, 1.f, in_group, ti, NT, D, s.wide_w, wg);
                weights<NE, U, W>(a.ls, a.scale, in_row, ti, NT, D, s.wide_w, wl);
            }
            float ev[NU], inv[NU];
#pragma unroll
            for (int q = 0; q < NU; ++q) inv[q] = !has_post ? 1.f : U <= 2 ? so[q] : inverse(so[q]);
            auto inv2 = [&](int j) { return make_float2(inv[j / U], inv[(j + 1) / U]); };
            RunSums<NE, U> e2;
            // channels j and j + 1 with the gate's value and derivative times v: v becomes the gradient of hat, ov becomes hat
            auto channels = [&](int j, float2 va, float2 vs) {
                const float2 hat = mul2(at(ov, j), inv2(j)), n = mul2(hat, at(wg, j)), dn = mul2(va, at(wl, j));
                set(acc_l, j, fma2(va, n, at(acc_l, j)));      // times the scale, at the end
                set(acc_g, j, fma2(dn, hat, at(acc_g, j)));
                set(gz, j, mul2(mul2(vs, at(wl, j)), n));
                const float2 dhat = mul2(dn, at(wg, j));
                set(v, j, dhat);
                set(ov, j, hat);
                e2.add(j, dhat, hat);
            };
            if (a.gate == KDA_GATE_SIGMOID) {
#pragma unroll
                for (int j = 0; j < NE; j += 2) {
                    const float2 p = sigmoid2(at(gz, j)), va = mul2(at(v, j), p);
                    channels(j, va, mul2(va, fma2(p, two(-1.f), two(1.f))));
                }
            } else if (a.gate == KDA_GATE_SILU) {
#pragma unroll
                for (int j = 0; j < NE; j += 2) {
                    const float2 z2 = at(gz, j), p = sigmoid2(z2), va = mul2(at(v, j), p);
                    channels(j, mul2(va, z2), mul2(va, fma2(z2, fma2(p, two(-1.f), two(1.f)), two(1.f))));
                }
            } else {
#pragma unroll
                for (int j = 0; j < NE; j += 2) channels(j, at(v, j), two(0.f));
            }
#pragma unroll
            for (int q = 0; q < NU; ++q) ev[q] = e2.run(q);
            if (dz && in) RowE::template write<FULL>(row_at(dz, t, static_cast<uint32_t>(g.lddz * sizeof(E))), ti, NT, D, s.wide_b, gz);
            if (has_post) {
                if (G == D) {
                    float all = 0.f;
#pragma unroll
                    for (int q = 0; q < NU; ++q) all += ev[q];
                    all = sums_e.over_row(all, NT, turn);
#pragma unroll
                    for (int q = 0; q < NU; ++q) ev[q] = all;
                } else {
                    groups_e.over_group(ev, G, turn);
                }
                if ((!FULL || U == 1) && G == 1) {
                    v[0] = unit_grad_of_one(v[0], inv[0], a.eps);
                } else {
#pragma unroll
                    for (int q = 0; q < NU; ++q) ev[q] *= -inv_g;
#pragma unroll
                    for (int j = 0; j < NE; j += 2)
                        set(v, j, mul2(inv2(j), fma2(at(ov, j), make_float2(ev[j / U], ev[(j + 1) / U]), at(v, j))));
                }
            }
            if (in) RowE::template write<FULL>(row_at(d_o, t, static_cast<uint32_t>(g.lddo * sizeof(E))), ti, NT, D, s.wide_a, v);
        }
        ++turn;
        if constexpr (S > 0) slot = slot + 1 == S ? 0 : slot + 1;
    }
    // the CTA's column sums, over its rows (and over the groups for w_post); the kernel that adds them up may be dispatched
    tc::grid_dep_launch();
    cp_wait<0>();
    float *fold = reinterpret_cast<float *>(ring);     // [rows][8 NC NT]
    const int width = NT * NE;
    part += static_cast<size_t>(blockIdx.x) * (G + 2 * static_cast<size_t>(D));
    auto put = [&](const float (&acc)[NE]) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NE; ++j) fold[(threadIdx.x / NT) * width + channel_of<U, NE, W>(ti, NT, j)] = acc[j];
        __syncthreads();
    };
    if (g.dw_post) {
        put(acc_g);
        for (int c = threadIdx.x; c < G; c += BLOCK) {
            float v = 0.f;
            for (int k = 0; k < rows; ++k)
                for (int j = c; j < D; j += G) v += fold[k * width + j];
            part[c] = v;
        }
    }
    auto out = [&](float *p, float by) {
        for (int c = threadIdx.x; c < D; c += BLOCK) {
            float v = 0.f;
            for (int k = 0; k < rows; ++k) v += fold[k * width + c];
            p[c] = by * v;
        }
    };
    if (g.dls) {
        put(acc_l);
        out(part + G, a.scale);
    }
    if (g.dw_pre) {
        put(acc_r);
        out(part + G + D, 1.f);
    }
}

// ---- launches ---------------------------------------------------------------------------------------------

// Every row of the tensor starts on 'on' bytes.
inline bool rows_on(const void *p, int64_t ld, int elem, int on = 16)
{
    return !p || ((reinterpret_cast<uintptr_t>(p) & (on - 1)) == 0 && (ld * elem & (on - 1)) == 0);
}

// Threads of a row: as many as hold it in 8 nc channels each; W at least where runs are short, a group's where they
// are four channels.
inline int threads_of_row(int D, int G, int nc, int U, int W)
{
    int nt = U <= 2 ? W : 4;
    while (static_cast<int64_t>(nt) * 8 * nc < D) nt *= 2;
    if (G < D && U > 2)
        while (nt * U < G) nt *= 2;
    return nt;
}

template <typename R, typename E, int BLOCK, int NC, int U, bool FULL = false, int W = 32>
cudaError_t run_forward(Shape s, const NormIn &a, void *r_out, int64_t ldro, void *y, int64_t ldy, cudaStream_t stream)
{
    using F = Forward<R, E, BLOCK, NC, U, W>;
    s.NT = threads_of_row(s.D, s.G, NC, U, W);
    auto fn = forward<R, E, BLOCK, NC, U, FULL, W>;
    if (cudaError_t e = set_dynamic_smem(reinterpret_cast<const void *>(fn), F::SMEM)) return e;
    // With one barrier a row, fewer CTAs read and write the rows more nearly in order and are faster (16384 x 4096 with a
    // residual in fp32: 164 us on one CTA of 512 threads an SM, 177 us on two); with two barriers a row the second CTA
    // is needed to fill the waits (all in bf16: 86 us on two, 109 us on one).
    const int ctas = F::CTAS > 1 && !(a.w_post && s.G == s.D) ? F::CTAS / 2 : F::CTAS;
    const int64_t rows = BLOCK / s.NT, want = (s.T + rows - 1) / rows, most = static_cast<int64_t>(ctas) * sm_count();
    fn<<<static_cast<unsigned>(want < most ? want : most), BLOCK, F::SMEM, stream>>>(s, a, static_cast<R *>(r_out), ldro,
                                                                                      static_cast<E *>(y), ldy);
    return cudaGetLastError();
}

template <typename R, typename E, int BLOCK, int NC, int U, bool FULL = false, int W = 32>
cudaError_t run_backward(Shape s, const NormIn &a, const void *dro, int64_t lddro, const void *dy, int64_t lddy, const NormGrads &g,
                         float *part, int *grid, cudaStream_t stream)
{
    using B = Backward<R, E, BLOCK, NC, U, W>;
    s.NT = threads_of_row(s.D, s.G, NC, U, W);
    auto fn = backward<R, E, BLOCK, NC, U, FULL, W>;
    if (cudaError_t e = set_dynamic_smem(reinterpret_cast<const void *>(fn), B::SMEM)) return e;
    const int64_t rows = BLOCK / s.NT, want = (s.T + rows - 1) / rows, full = B::CTAS * sm_count(), most = full < MAX_GRID ? full : MAX_GRID;
    *grid = static_cast<int>(want < most ? want : most);
    fn<<<*grid, BLOCK, B::SMEM, stream>>>(s, a, static_cast<const R *>(dro), lddro, static_cast<const E *>(dy), lddy, g, part);
    return cudaGetLastError();
}

// The instance for a width and a run: CTAs of 256 threads for rows of up to 2048 channels, 512 up to 4096, 512 with
// twice the channels a thread up to 8192, 1024 with those up to 16384.
#define KDA_NORM_PICK(FN, R, E, U, ...)                \
    (s.D <= 2048   ? FN<R, E, 256, 1, U>(__VA_ARGS__)  \
     : s.D <= 4096 ? FN<R, E, 512, 1, U>(__VA_ARGS__)  \
     : s.D <= 8192 ? FN<R, E, 512, 2, U>(__VA_ARGS__)  \
                   : FN<R, E, 1024, 2, U>(__VA_ARGS__))

// Channels of a run where rows start on 16 bytes.
template <typename R> constexpr int WIDE = sizeof(R) == 4 ? 4 : 8;

template <typename R, typename E>
cudaError_t pick_forward(Shape s, const NormIn &a, void *r_out, int64_t ldro, void *y, int64_t ldy, cudaStream_t stream)
{
    constexpr int re = sizeof(R), e = sizeof(E);
    if (rows_on(a.r, a.ldr, re) && rows_on(a.o, a.ldo, e) && rows_on(a.z, a.ldz, e)) {
        s.wide_r = rows_on(r_out, ldro, re);
        s.wide_a = rows_on(y, ldy, e);
        // above 4096 channels: 8192 x 8192 in bf16 115 us on one CTA of 1024 threads with 8 channels each, 162 us on 512 with 16
        if (a.r && a.o && a.w_post && r_out && y && s.wide_r && s.wide_a && s.D % 8 == 0 && s.D <= 8192)
            return s.D <= 2048   ? run_forward<R, E, 256, 1, WIDE<R>, true>(s, a, r_out, ldro, y, ldy, stream)
                   : s.D <= 4096 ? run_forward<R, E, 512, 1, WIDE<R>, true>(s, a, r_out, ldro, y, ldy, stream)
                                 : run_forward<R, E, 1024, 1, WIDE<R>, true>(s, a, r_out, ldro, y, ldy, stream);
        return KDA_NORM_PICK(run_forward, R, E, WIDE<R>, s, a, r_out, ldro, y, ldy, stream);
    }
    if (a.r && a.o && a.w_post && r_out && y && s.D <= 4096) {
        if (s.D % 2 == 0 && rows_on(a.r, a.ldr, re, 2 * re) && rows_on(a.o, a.ldo, e, 2 * e) && rows_on(a.z, a.ldz, e, 2 * e) &&
            rows_on(r_out, ldro, re, 2 * re) && rows_on(y, ldy, e, 2 * e))
            return s.D <= 128    ? run_forward<R, E, 256, 1, 2, true, 16>(s, a, r_out, ldro, y, ldy, stream)
                   : s.D <= 2048 ? run_forward<R, E, 256, 1, 2, true>(s, a, r_out, ldro, y, ldy, stream)
                               : run_forward<R, E, 512, 1, 2, true>(s, a, r_out, ldro, y, ldy, stream);
        return s.D <= 128    ? run_forward<R, E, 256, 1, 1, true, 16>(s, a, r_out, ldro, y, ldy, stream)
               : s.D <= 2048 ? run_forward<R, E, 256, 1, 1, true>(s, a, r_out, ldro, y, ldy, stream)
                           : run_forward<R, E, 512, 1, 1, true>(s, a, r_out, ldro, y, ldy, stream);
    }
    return KDA_NORM_PICK(run_forward, R, E, 1, s, a, r_out, ldro, y, ldy, stream);
}

template <typename R, typename E>
cudaError_t pick_backward(Shape s, const NormIn &a, const void *dro, int64_t lddro, const void *dy, int64_t lddy, const NormGrads &g,
                          float *part, int *grid, cudaStream_t stream)
{
    constexpr int re = sizeof(R), e = sizeof(E);
    const bool pre = !a.w_pre || (rows_on(a.r, a.ldr, re) && rows_on(dy, lddy, e));
    if (pre && rows_on(dro, lddro, re) && rows_on(a.o, a.ldo, e) && rows_on(a.z, a.ldz, e)) {
        s.wide_r = rows_on(g.dr, g.lddr, re);
        s.wide_a = rows_on(g.d_o, g.lddo, e);
        s.wide_b = rows_on(g.dz, g.lddz, e);
        // above 4096 channels the other way round, registers being short: 346 us on 512 threads, 457 us on 1024
        if (a.w_pre && dro && a.o && a.w_post && s.wide_r && s.wide_a && s.wide_b && s.D % 8 == 0 && s.D <= 8192)
            return s.D <= 2048   ? run_backward<R, E, 256, 1, WIDE<R>, true>(s, a, dro, lddro, dy, lddy, g, part, grid, stream)
                   : s.D <= 4096 ? run_backward<R, E, 512, 1, WIDE<R>, true>(s, a, dro, lddro, dy, lddy, g, part, grid, stream)
                                 : run_backward<R, E, 512, 2, WIDE<R>, true>(s, a, dro, lddro, dy, lddy, g, part, grid, stream);
        return KDA_NORM_PICK(run_backward, R, E, WIDE<R>, s, a, dro, lddro, dy, lddy, g, part, grid, stream);
    }
    if (a.w_pre && dro && a.o && a.w_post && s.D <= 4096) {
        if (s.D % 2 == 0 && rows_on(a.r, a.ldr, re, 2 * re) && rows_on(dro, lddro, re, 2 * re) && rows_on(dy, lddy, e, 2 * e) &&
            rows_on(a.o, a.ldo, e, 2 * e) && rows_on(a.z, a.ldz, e, 2 * e) && rows_on(g.dr, g.lddr, re, 2 * re) &&
            rows_on(g.d_o, g.lddo, e, 2 * e) && rows_on(g.dz, g.lddz, e, 2 * e))
            return s.D <= 128    ? run_backward<R, E, 256, 1, 2, true, 16>(s, a, dro, lddro, dy, lddy, g, part, grid, stream)
                   : s.D <= 2048 ? run_backward<R, E, 256, 1, 2, true>(s, a, dro, lddro, dy, lddy, g, part, grid, stream)
                               : run_backward<R, E, 512, 1, 2, true>(s, a, dro, lddro, dy, lddy, g, part, grid, stream);
        return s.D <= 128    ? run_backward<R, E, 256, 1, 1, true, 16>(s, a, dro, lddro, dy, lddy, g, part, grid, stream)
               : s.D <= 2048 ? run_backward<R, E, 256, 1, 1, true>(s, a, dro, lddro, dy, lddy, g, part, grid, stream)
                           : run_backward<R, E, 512, 1, 1, true>(s, a, dro, lddro, dy, lddy, g, part, grid, stream);
    }
    return KDA_NORM_PICK(run_backward, R, E, 1, s, a, dro, lddro, dy, lddy, g, part, grid, stream);
}

// One translation unit per activation type.
cudaError_t forward_bf16(int rtype, Shape s, const NormIn &a, void *r_out, int64_t ldro, void *y, int64_t ldy, cudaStream_t stream);
cudaError_t forward_f16(int rtype, Shape s, const NormIn &a, void *r_out, int64_t ldro, void *y, int64_t ldy, cudaStream_t stream);
cudaError_t forward_f32(int rtype, Shape s, const NormIn &a, void *r_out, int64_t ldro, void *y, int64_t ldy, cudaStream_t stream);
cudaError_t backward_bf16(int rtype, Shape s, const NormIn &a, const void *dro, int64_t lddro, const void *dy, int64_t lddy,
                          const NormGrads &g, float *part, int *grid, cudaStream_t stream);
cudaError_t backward_f16(int rtype, Shape s, const NormIn &a, const void *dro, int64_t lddro, const void *dy, int64_t lddy,
                         const NormGrads &g, float *part, int *grid, cudaStream_t stream);
cudaError_t backward_f32(int rtype, Shape s, const NormIn &a, const void *dro, int64_t lddro, const void *dy, int64_t lddy,
                         const NormGrads &g, float *part, int *grid, cudaStream_t stream);

}  // namespace norm
}  // namespace kda
