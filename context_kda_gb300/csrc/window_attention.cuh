// Attention over a sliding window with sinks: what its forward and its gradients share.
//
// In a sequence, query i sees the keys j <= i with i - j < W, and of the others the first S (the sinks).  Tiles of 128 keys
// start at multiples of 128 from the sequence's start.  A tile of rows works the tiles of its window, whose mask is
// i - W < j <= i, and, once a row has left them behind, the sinks' tile with the mask j < S, j <= i - W: no pair twice.
#pragma once

#include "elem.cuh"
#include "kda_internal.cuh"
#include "tc.cuh"

namespace kda {
namespace attn {

using namespace tc;

constexpr int TILE = 128;                 // rows of a tile, of queries and of keys
constexpr uint32_t BOX = TILE * 128;      // 128 rows of 64 16-bit columns, as a box with the 128-byte swizzle lands

// Sequences whose starts come with the launch.  Finding a tile in the device plan takes three trips to the L2 cache, 2300 cycles
// before a CTA knows what to fetch; from the launch's constants it is hardly any.
constexpr int FEW = 32;

struct Shape {
    const int32_t *plan;
    PlanSig sig;
    int N, off_cu, T;                     // of the plan
    int32_t cu[FEW + 1];                  // the host plan's, where N <= FEW
    int H, Hk, W, S;
    float c;                              // scale * log2(e): scores to exponents of two
    float scale;
};

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Named barrier 'id' over 'threads' threads with an OR of v: everyone gets the same answer.
__device__ __forceinline__ bool bar_or(int id, uint32_t threads, bool v)
{
    uint32_t r;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbarrier.cta.red.or.pred q, %2, %3, p;\nselp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(v)), "r"(id), "r"(threads)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap &m) { asm volatile("prefetch.tensormap [%0];" ::"l"(&m) : "memory"); }

// Registers of a warpgroup's threads, after the launch gave every thread the same.
template <int N> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

inline Shape window_shape(const int32_t *plan_host, const int32_t *plan_dev, const WindowIn &in)
{
    Shape p{plan_dev, plan_sig(plan_host), plan_host[KDA_PH_N], plan_host[KDA_PH_OFF_CU], plan_host[KDA_PH_T], {}, in.H, in.Hk, in.W, in.S,
            in.scale * 1.44269504088896340736f, in.scale};
    for (int n = 0; n <= p.N && p.N <= FEW; ++n) p.cu[n] = plan_host[p.off_cu + n];
    return p;
}

template <typename E> struct Pair;        // two values rounded to a packed pair (a in the low half); x 0 + c of such pairs
template <> struct Pair<__nv_bfloat16> {
    static constexpr bool BF16 = true;
    static constexpr uint32_t INF = 0x7F80u;
    static __device__ __forceinline__ uint32_t times_zero(uint32_t x, uint32_t c)
    {
        uint32_t d;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(x), "r"(0u), "r"(c));
        return d;
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) { return bf16x2_bits(a, b); }
};
template <> struct Pair<__half> {
    static constexpr bool BF16 = false;
    static constexpr uint32_t INF = 0x7C00u;
    static __device__ __forceinline__ uint32_t times_zero(uint32_t x, uint32_t c)
    {
        uint32_t d;
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(x), "r"(0u), "r"(c));
        return d;
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};

// Instruction descriptor of kind::f16 with operands of type E; b_mn: B is MN-major.
template <typename E> __host__ __device__ constexpr uint32_t idesc(int M, int N, int b_mn)
{
    return idesc_bf16(M, N, 0, b_mn) & (Pair<E>::BF16 ? ~0u : ~((1u << 7) | (1u << 10)));
}

// Shared-memory descriptors in the 128-byte swizzle layout, by halves: rows of 128 bytes, 8-row groups 1024 bytes apart (the
// upper half: that, version 1, the swizzle).  K-major operands: a K step of 16 columns advances the start by 32 bytes.  MN-major
// ones (rows are the contraction index): the next 64 columns are 'lbo' bytes on, and a K step of 16 rows advances the start
// by 2048 bytes.
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | (lbo >> 4 << 16); }

// The products are issued by a whole warp whose values are the same in every lane, so that they stay in uniform registers, one
// elected lane doing it: a lone thread's products took 100 cycles each to issue, twice what the tensor cores need for them.
__device__ __forceinline__ bool elect()
{
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}
// D[tmem] (+)= A B^T, one K step: A in shared memory, or (ta) in TMEM.
__device__ __forceinline__ void product(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate)
{
    asm volatile("{\n.reg .pred p;\n.reg .b64 a, b;\nmov.b64 a, {%1, %3};\nmov.b64 b, {%2, %3};\nsetp.ne.b32 p, %5, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}\n" ::"r"(d),
                 "r"(a), "r"(b), "n"(DESC_HI), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)));
}
__device__ __forceinline__ void product_ta(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate)
{
    asm volatile("{\n.reg .pred p;\n.reg .b64 b;\nmov.b64 b, {%2, %3};\nsetp.ne.b32 p, %5, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(d),
                 "r"(a), "r"(b), "n"(DESC_HI), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)));
}

__device__ __forceinline__ bool look(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_thread(uint32_t bar, uint32_t parity) { return look(bar, parity) || mbar_wait(bar, parity); }
// A bounded wait of a whole warp, the same answer in every lane; the clock is read only where the first look fails.  All lanes
// look: a branch to one lane and back costs more than the look itself.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity)
{
    if (__all_sync(0xffffffffu, look(bar, parity))) return true;
    const long long t0 = clock64();
    while (!__all_sync(0xffffffffu, look(bar, parity)))
        if (__any_sync(0xffffffffu, clock64() - t0 > 4000000000LL)) return false;
    return true;
}

// The sequence and tile of slot 'slot'.  Sequence n has its tiles of 'rows' = 2^log_rows tokens from slot cu[n] / rows + n on, which
// leaves room for all of them without a prefix sum; a slot behind a sequence's last tile is empty (false).  Whole warps call it.
struct Place {
    int seq, start, len, t0;              // the sequence, its first token and length, first row of the tile in it
};
__device__ __forceinline__ bool find_tile(const Shape &p, int slot, int log_rows, Place &at)
{
    const int lane = threadIdx.x & 31;
    int lo = 0;
    if (p.N <= FEW) {
        lo = __popc(__ballot_sync(0xffffffffu, lane < p.N && (p.cu[lane] >> log_rows) + lane <= slot)) - 1;
        at.start = p.cu[lo];
        at.len = p.cu[lo + 1] - at.start;
    } else {
        const int32_t *cu = p.plan + p.off_cu;
        for (int count = p.N;;) {         // 32 candidates at a time, evenly spread over the rest
            const int stride = (count + 31) / 32, n = lo + lane * stride;
            const bool in = lane * stride < count && (cu[n] >> log_rows) + n <= slot;
            const int last = __popc(__ballot_sync(0xffffffffu, in)) - 1;
            lo += last * stride;
            count = min(stride, count - last * stride);
            if (stride == 1) break;
        }
        at.start = cu[lo];
        at.len = cu[lo + 1] - at.start;
    }
    at.seq = lo;
    at.t0 = (slot - ((at.start >> log_rows) + lo)) << log_rows;
    // the same in every lane; said so that the compiler knows
    at.seq = __shfl_sync(0xffffffffu, at.seq, 0);
    at.start = __shfl_sync(0xffffffffu, at.start, 0);
    at.len = __shfl_sync(0xffffffffu, at.len, 0);
    at.t0 = __shfl_sync(0xffffffffu, at.t0, 0);
    return at.t0 < at.len;
}
inline int tile_slots(int T, int N, int rows) { return T / rows + N; }

// Tensor map of [T][heads][d] 16-bit values with a token stride: boxes of 64 columns x 1 head x 'rows' tokens.
inline bool encode_heads(CUtensorMap *m, const void *p, bool bf16, int d, int heads, int64_t T, int64_t ld, uint32_t rows)
{
    auto fn = tmap_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(T)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(ld) * 2};
    const cuuint32_t box[3] = {64, 1, rows}, es[3] = {1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(p), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace attn
}  // namespace kda
