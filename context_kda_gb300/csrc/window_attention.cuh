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

struct Shape {
    const int32_t *plan;
    PlanSig sig;
    int N, off_cu, T;                     // of the plan
    int H, Hk, W, S;
    float c;                              // scale * log2(e): scores to exponents of two
    float scale;
};

// Registers of a warpgroup's threads, after the launch gave every thread the same.
template <int N> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

inline Shape window_shape(const int32_t *plan_host, const int32_t *plan_dev, const WindowIn &in)
{
    return Shape{plan_dev, plan_sig(plan_host), plan_host[KDA_PH_N], plan_host[KDA_PH_OFF_CU], plan_host[KDA_PH_T], in.H, in.Hk, in.W, in.S,
                 in.scale * 1.44269504088896340736f, in.scale};
}

template <typename E> struct Pair;        // two values rounded to a packed pair (a in the low half)
template <> struct Pair<__nv_bfloat16> {
    static constexpr bool BF16 = true;
    static constexpr uint32_t INF = 0x7F80u;
    static __device__ __forceinline__ uint32_t pack(float a, float b) { return bf16x2_bits(a, b); }
};
template <> struct Pair<__half> {
    static constexpr bool BF16 = false;
    static constexpr uint32_t INF = 0x7C00u;
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

// Descriptor of an MN-major operand in the 128-byte swizzle layout: rows (the contraction index) of 128 bytes, 8-row groups
// 1024 bytes apart, the next 64 columns 'lbo' bytes on.  A K step of 16 rows advances the start by 2048 bytes.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t lbo)
{
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// The sequence and tile of slot 'slot'.  Sequence n has its tiles of 'rows' tokens from slot cu[n] / rows + n on, which
// leaves room for all of them without a prefix sum; a slot behind a sequence's last tile is empty (false).  Whole warps call it.
struct Place {
    int seq, start, len, t0;              // the sequence, its first token and length, first row of the tile in it
};
__device__ __forceinline__ bool find_tile(const Shape &p, int slot, int rows, Place &at)
{
    const int32_t *cu = p.plan + p.off_cu;
    const int lane = threadIdx.x & 31;
    int lo = 0, count = p.N;
    while (true) {                        // 32 candidates at a time, evenly spread over the rest
        const int stride = (count + 31) / 32, n = lo + lane * stride;
        const bool in = lane * stride < count && cu[n] / rows + n <= slot;
        const int last = __popc(__ballot_sync(0xffffffffu, in)) - 1;
        lo += last * stride;
        count = min(stride, count - last * stride);
        if (stride == 1) break;
    }
    at.seq = lo;
    at.start = cu[lo];
    at.len = cu[lo + 1] - at.start;
    at.t0 = (slot - (at.start / rows + lo)) * rows;
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
