// The window attention a token at a time, from and into a ring cache, and the fill of that cache from packed sequences.
//
// A slot's cache holds, for each key head, S rows for the first S positions and W rows that are used in turn:
// position p is in row p if p < S, else in row S + (p - S) mod W.  So the rows that the next token sees are the first
// min(p + 1, S + W), its own among them, in whatever order; attention does not ask for it.
//
// The step is bound by memory: every visible row is read once, for all heads of its group.  A cluster of CTAs shares
// the rows of one (token, key head); a warp takes 16 rows at a time, which are contiguous, as one bulk copy of keys and one of
// values, STAGES of them in turn, each warp with its own barriers.  How the bytes are asked for is what decides: without any work on
// them, the 807 MB of 64 tokens x 8 key heads over up to 4100 rows of 128 take 133 us as bulk copies of 4 KB, 160 us a row at a time and
// 180 us with 16 bytes a lane (cp.async).  With the work and as separate calls 123 to 131 us, 6.1 to 6.5 TB/s, where a copy runs at 6.8.
// The products (mma, whose rate does not matter here) may take channels and rows in any order, so a lane's 16 bytes of keys are
// its part of two K steps, and its 16 bytes each of four rows of values, interleaved, are its part of eight N tiles: no lane needs
// another's bytes.  Rows follow one another without a gap, so lanes of odd rows take their pieces in another order and swap them
// afterwards: keys without bank conflicts, values (128 channels) with two to a bank.  Scores leave the first product where the
// second one wants its A operand.  Each warp keeps its own running maximum, sum and outputs; they are joined in shared memory
// and then over the cluster, in a fixed order.  Probabilities are rounded to the activations' type for their product; in fp16, which has no
// numbers below 2^-24, they are kept times 2^15, since very many small ones count.
// The new token's row is laid over the cache's in shared memory, and the CTA whose rows it is among writes it to the cache.
#include <type_traits>

#include "elem.cuh"
#include "kda_internal.cuh"
#include "tc.cuh"

namespace kda {
namespace {

__device__ int g_cache_status;

constexpr int WARPS = 4, THREADS = WARPS * 32;
constexpr int ROWS = 16;                  // of a warp's step
constexpr int MAX_SPLIT = 8;              // CTAs of a cluster
constexpr int STAGES = 3;                 // of a warp's queue, 16 rows each: two CTAs an SM have up to 192 KiB on their way

template <int D> constexpr uint32_t STAGE = 2 * ROWS * D * 2;      // bytes: 16 rows of keys, 16 of values
template <int D> constexpr uint32_t QUEUE = STAGES * STAGE<D>;     // of a warp
// A warp's sums, for the join: channel ch of a head at at_ch(ch), heads PITCH apart, so that its 8 heads x 4 groups of channels meet 32 banks.
template <int D> constexpr int PITCH = D + 33;
template <int D> __device__ __forceinline__ int at_ch(int ch) { return ch + 8 * (ch / (D / 4)); }
template <int D, int HG> constexpr uint32_t SUMS = HG * PITCH<D> * 4;
template <int D, int HG> constexpr uint32_t SMEM = WARPS * (QUEUE<D> > SUMS<D, HG> ? QUEUE<D> : SUMS<D, HG>);

__device__ __forceinline__ void swap_if(bool yes, uint4 &a, uint4 &b)
{
    const uint4 x = a;
    a.x = yes ? b.x : a.x, a.y = yes ? b.y : a.y, a.z = yes ? b.z : a.z, a.w = yes ? b.w : a.w;
    b.x = yes ? x.x : b.x, b.y = yes ? x.y : b.y, b.z = yes ? x.z : b.z, b.w = yes ? x.w : b.w;
}

template <typename E>
__device__ __forceinline__ void mma(float &c0, float &c1, float &c2, float &c3, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1);
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float &c0, float &c1, float &c2, float &c3, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                   uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c0), "+f"(c1), "+f"(c2), "+f"(c3)
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<__half>(float &c0, float &c1, float &c2, float &c3, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c0), "+f"(c1), "+f"(c2), "+f"(c3)
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) { return tc::bf16x2_bits(a, b); }
__device__ __forceinline__ uint32_t pack2(float a, float b, __half)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float load_rank(const float *p, uint32_t rank)     // the same place in another CTA of the cluster
{
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

struct Step {
    StepIn in;
    int g, blocks, split;                 // heads of a group, blocks of HG heads in it, CTAs of a cluster
    float c;                              // scale * log2(e)
    int64_t ldo;
};

// HG: query heads worked together, 8 or 16 (the product's M).
template <typename E, int D, int HG>
__global__ void __launch_bounds__(THREADS, 2) window_step(const Step p, E *cache_k, E *cache_v, E *o)
{
    constexpr int KC = D / 32, VC = D / 64;       // 16-byte pieces of a lane: of a row of keys, of a row of values
    constexpr float P_EXP = std::is_same<E, __half>::value ? 15.f : 0.f;      // probabilities (one at most) are kept times 2^P_EXP
    extern __shared__ __align__(16) unsigned char smem[];
    auto s_o = reinterpret_cast<float (*)[HG][PITCH<D>]>(smem);      // [WARPS], once the queues are empty
    __shared__ float s_m[WARPS][HG], s_l[WARPS][HG], s_mc[HG], s_lc[HG];
    __shared__ alignas(8) uint64_t s_full[WARPS][STAGES];
    const StepIn &in = p.in;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, hd = lane >> 2, c4 = lane & 3;
    const int part = blockIdx.x % p.split;
    const int64_t unit = blockIdx.x / p.split;    // (token, key head, block of its heads)
    const int block = static_cast<int>(unit % p.blocks), hk = static_cast<int>(unit / p.blocks % in.Hk);
    const int64_t b = unit / p.blocks / in.Hk;
    const int h0 = hk * p.g + block * HG, heads = min(HG, p.g - block * HG);
    const int cap = in.S + in.W, slot = in.slots ? in.slots[b] : static_cast<int>(b), len = in.lengths[b];
    E *const out = o + b * p.ldo + static_cast<int64_t>(h0) * D;
    if (slot < 0 || slot >= in.num_slots || len < 0) {
        for (int i = tid + part * THREADS; i < heads * D; i += THREADS * p.split) out[i] = from_f32<E>(0.f);
        if (slot >= 0 && tid == 0) record_status(&g_cache_status, KDA_ERR_INVALID_ARG);
        return;      // the whole cluster
    }
    const int fresh = len < in.S ? len : in.S + (len - in.S) % in.W;       // the new token's row
    const int n = len < cap ? len + 1 : cap;
    const int64_t first = (static_cast<int64_t>(slot) * in.Hk + hk) * cap;
    const E *const k_new = static_cast<const E *>(in.k) + b * in.ldk + static_cast<int64_t>(hk) * D;
    const E *const v_new = static_cast<const E *>(in.v) + b * in.ldv + static_cast<int64_t>(hk) * D;
    const int per = ((n + p.split - 1) / p.split + ROWS - 1) / ROWS * ROWS, lo = part * per, hi = min(n, lo + per);

    // queries: the A operand, heads hd and hd + 8
    uint32_t qa[KC][4], qb[HG == 16 ? KC : 1][4];
#pragma unroll
    for (int i = 0; i < KC; ++i) {
        const E *const q = static_cast<const E *>(in.q) + b * in.ldq + static_cast<int64_t>(h0) * D + (c4 + 4 * i) * 8;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (hd < heads) x = *reinterpret_cast<const uint4 *>(q + hd * D);
        qa[i][0] = x.x, qa[i][1] = x.y, qa[i][2] = x.z, qa[i][3] = x.w;
        if constexpr (HG == 16) {
            x = make_uint4(0, 0, 0, 0);
            if (hd + 8 < heads) x = *reinterpret_cast<const uint4 *>(q + (hd + 8) * D);
            qb[i][0] = x.x, qb[i][1] = x.y, qb[i][2] = x.z, qb[i][3] = x.w;
        }
    }
    float acc[D / 8][2], acc2[HG == 16 ? D / 8 : 1][2], m = -INFINITY, l = 0.f, m2 = -INFINITY, l2 = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        acc[i][0] = acc[i][1] = 0.f;
        if constexpr (HG == 16) acc2[i][0] = acc2[i][1] = 0.f;
    }

    const uint32_t full = tc::smem_u32(&s_full[warp][0]), queue = tc::smem_u32(smem) + warp * QUEUE<D>;
    unsigned char *const mine = smem + warp * QUEUE<D>;
    if (lane == 0)
        for (int s = 0; s < STAGES; ++s) tc::mbar_init(full + s * 8, 1);
    auto fetch = [&](int r0, int stage) {         // by lane 0
        const uint32_t bytes = min(ROWS, hi - r0) * D * 2, to = queue + stage * STAGE<D>;
        tc::mbar_arrive_expect_tx(full + stage * 8, 2 * bytes);
        tc::bulk_g2s(to, cache_k + (first + r0) * D, bytes, full + stage * 8);
        tc::bulk_g2s(to + STAGE<D> / 2, cache_v + (first + r0) * D, bytes, full + stage * 8);
    };
    constexpr int STRIDE = WARPS * ROWS;
    int r0 = lo + warp * ROWS;
    if (lane == 0)
        for (int s = 0; s < STAGES - 1; ++s)
            if (r0 + s * STRIDE < hi) fetch(r0 + s * STRIDE, s);
    __syncwarp();
    uint32_t parity = 0;
    for (int stage = 0; r0 < hi; r0 += STRIDE, stage = stage == STAGES - 1 ? 0 : stage + 1) {
        __syncwarp();                             // the stage before this one has been read
        if (lane == 0 && r0 + (STAGES - 1) * STRIDE < hi) fetch(r0 + (STAGES - 1) * STRIDE, stage == 0 ? STAGES - 1 : stage - 1);
        __syncwarp();
        if (!__all_sync(0xffffffffu, tc::mbar_wait(full + stage * 8, parity >> stage & 1))) {
            if (lane == 0) record_status(&g_cache_status, KDA_ERR_TIMEOUT);
            for (int i = 0, s = stage; i < STAGES; ++i, s = s == STAGES - 1 ? 0 : s + 1)      // copies on their way, before this memory is used again
                if (r0 + i * STRIDE < hi) tc::mbar_wait(full + s * 8, parity >> s & 1);
            l = l2 = NAN;
            break;
        }
        parity ^= 1u << stage;
        unsigned char *const rows = mine + stage * STAGE<D>;
        if (fresh >= r0 && fresh < r0 + ROWS && fresh < hi) {
            if (lane < 2 * D / 8) {
                const bool is_v = lane >= D / 8;
                const int ch = lane % (D / 8) * 8;
                *reinterpret_cast<uint4 *>(rows + is_v * (STAGE<D> / 2) + ((fresh - r0) * D + ch) * 2) = *reinterpret_cast<const uint4 *>((is_v ? v_new : k_new) + ch);
            }
            tc::fence_async_smem();               // before the next copy to this place
        }
        if (r0 + ROWS > hi)                       // no values there: a probability of zero, but what lies there may be NaN
            for (int i = (hi - r0) * (D / 8) + lane; i < ROWS * D / 8; i += 32)
                *reinterpret_cast<uint4 *>(rows + STAGE<D> / 2 + i * 16) = make_uint4(0, 0, 0, 0);
        __syncwarp();
        float s[2][4] = {};
#pragma unroll
        for (int t = 0; t < 2; ++t) {             // keys of rows r0 + hd, + 8
            uint4 kr[KC];
#pragma unroll
            for (int i = 0; i < KC; ++i) kr[i] = *reinterpret_cast<const uint4 *>(rows + (t * 8 + hd) * D * 2 + (c4 + 4 * (i ^ (hd & 1))) * 16);
#pragma unroll
            for (int i = 0; i < KC; i += 2) swap_if(hd & 1, kr[i], kr[i + 1]);
#pragma unroll
            for (int i = 0; i < KC; ++i) {
                const uint4 y = kr[i];
                const uint32_t b0[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    mma<E>(s[t][0], s[t][1], s[t][2], s[t][3], qa[i][2 * h], HG == 16 ? qb[HG == 16 ? i : 0][2 * h] : 0u, qa[i][2 * h + 1],
                           HG == 16 ? qb[HG == 16 ? i : 0][2 * h + 1] : 0u, b0[2 * h], b0[2 * h + 1]);
            }
        }
        // s[t][0, 1]: head hd, rows r0 + 8 t + 2 c4, + 1;  s[t][2, 3]: head hd + 8
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (r0 + t * 8 + c4 * 2 + j >= hi) s[t][j] = s[t][j + 2] = -INFINITY;
        auto follow = [&](float &m, float &l, float (*a)[2], int j) {      // the running maximum and sum; s becomes probabilities
            float top = fmaxf(fmaxf(s[0][j], s[0][j + 1]), fmaxf(s[1][j], s[1][j + 1]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            top = fmaxf(top, m);
            if (__any_sync(0xffffffffu, top > m)) {
                const float f = m == -INFINITY ? 0.f : tc::ex2_ftz((m - top) * p.c);
                l *= f;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) a[i][0] *= f, a[i][1] *= f;
                m = top;
            }
            const float less = m == -INFINITY ? 0.f : m;      // (no maximum yet: scores of minus infinity alone, probabilities of zero)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    s[t][j + k] = tc::ex2_ftz(fmaf(s[t][j + k] - less, p.c, P_EXP));      // (the difference first: scores may be of any size)
                    l += s[t][j + k];
                }
        };
        follow(m, l, acc, 0);
        if constexpr (HG == 16) follow(m2, l2, acc2, 2);
        const uint32_t a0 = pack2(s[0][0], s[0][1], E()), a2 = pack2(s[1][0], s[1][1], E());
        const uint32_t a1 = HG == 16 ? pack2(s[0][2], s[0][3], E()) : 0u, a3 = HG == 16 ? pack2(s[1][2], s[1][3], E()) : 0u;
        uint4 vr[VC][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {             // values of rows r0 + 2 c4, + 1, + 8, + 9
            const unsigned char *const row = rows + STAGE<D> / 2 + ((t >> 1) * 8 + c4 * 2 + (t & 1)) * D * 2 + hd * VC * 16;
#pragma unroll
            for (int i = 0; i < VC; ++i) vr[i][t] = *reinterpret_cast<const uint4 *>(row + (VC == 1 ? 0 : (i ^ (c4 & 1)) * 16));
            if constexpr (VC == 2) swap_if(c4 & 1, vr[0][t], vr[1][t]);
        }
#pragma unroll
        for (int i = 0; i < VC; ++i) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t y[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) y[t] = w == 0 ? vr[i][t].x : w == 1 ? vr[i][t].y : w == 2 ? vr[i][t].z : vr[i][t].w;
#pragma unroll
                for (int h = 0; h < 2; ++h) {     // channel 2 w + h of the lane's 8
                    const uint32_t b0 = __byte_perm(y[0], y[1], h ? 0x7632 : 0x5410), b1 = __byte_perm(y[2], y[3], h ? 0x7632 : 0x5410);
                    const int j = i * 8 + 2 * w + h;
                    float d2 = 0.f, d3 = 0.f;
                    if constexpr (HG == 16) mma<E>(acc[j][0], acc[j][1], acc2[j][0], acc2[j][1], a0, a1, a2, a3, b0, b1);
                    else mma<E>(acc[j][0], acc[j][1], d2, d3, a0, 0u, a2, 0u, b0, b1);
                }
            }
        }
    }
    __syncthreads();
    // ---- the new row into the cache, by the CTA whose rows it is among
    if (block == 0 && fresh >= lo && fresh < hi && tid < 2 * D / 8) {
        const int ch = tid % (D / 8) * 8;
        const bool is_v = tid >= D / 8;
        *reinterpret_cast<uint4 *>((is_v ? cache_v : cache_k) + (first + fresh) * D + ch) = *reinterpret_cast<const uint4 *>((is_v ? v_new : k_new) + ch);
    }
    // ---- the warps of the CTA, then the CTAs of the cluster
    auto leave = [&](int head, float m, float l, float (*a)[2]) {
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (c4 == 0) s_m[warp][head] = m, s_l[warp][head] = l;
#pragma unroll
        for (int j = 0; j < D / 8; ++j)           // n = 2 c4 + e is channel (n VC + j / 8) * 8 + j % 8
#pragma unroll
            for (int e = 0; e < 2; ++e) s_o[warp][head][at_ch<D>(((2 * c4 + e) * VC + j / 8) * 8 + j % 8)] = a[j][e];
    };
    leave(hd, m, l, acc);
    if constexpr (HG == 16) leave(hd + 8, m2, l2, acc2);
    __syncthreads();
    for (int i = tid; i < heads * D; i += THREADS) {
        const int h = i / D, ch = i % D;
        float top = s_m[0][h], sum = 0.f, v = 0.f;
#pragma unroll
        for (int w = 1; w < WARPS; ++w) top = fmaxf(top, s_m[w][h]);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float f = s_m[w][h] == -INFINITY && !(s_l[w][h] > 0.f || s_l[w][h] != s_l[w][h]) ? 0.f : tc::ex2_ftz((s_m[w][h] - top) * p.c);
            sum = fmaf(f, s_l[w][h], sum);
            v = fmaf(f, s_o[w][h][at_ch<D>(ch)], v);
        }
        if (p.split == 1) out[i] = from_f32<E>(v / sum);
        else s_o[0][h][at_ch<D>(ch)] = v;
        if (ch == 0) s_mc[h] = top, s_lc[h] = sum;
    }
    if (p.split == 1) return;
    cluster_sync();
    for (int i = tid + static_cast<int>(cluster_rank()) * THREADS; i < heads * D; i += THREADS * p.split) {
        const int h = i / D, ch = i % D;
        float ms[MAX_SPLIT], ls[MAX_SPLIT], vs[MAX_SPLIT], top = -INFINITY, sum = 0.f, v = 0.f;
#pragma unroll
        for (int r = 0; r < MAX_SPLIT; ++r)
            if (r < p.split) {
                ms[r] = load_rank(&s_mc[h], r), ls[r] = load_rank(&s_lc[h], r), vs[r] = load_rank(&s_o[0][h][at_ch<D>(ch)], r);
                top = fmaxf(top, ms[r]);
            }
#pragma unroll
        for (int r = 0; r < MAX_SPLIT; ++r)
            if (r < p.split) {
                const float f = ms[r] == -INFINITY && ls[r] == 0.f ? 0.f : tc::ex2_ftz((ms[r] - top) * p.c);
                sum = fmaf(f, ls[r], sum);
                v = fmaf(f, vs[r], v);
            }
        out[i] = from_f32<E>(v / sum);
    }
    cluster_sync();          // nobody leaves while its shared memory is read
}

template <typename E, int D, int HG>
cudaError_t step(Step p, void *cache_k, void *cache_v, void *o, cudaStream_t stream)
{
    const StepIn &in = p.in;
    p.blocks = (p.g + HG - 1) / HG;
    const int64_t units = static_cast<int64_t>(in.B) * in.Hk * p.blocks;
    // three rounds of CTAs (two an SM) and more, since lengths differ, but none with fewer than 64 rows of a full cache (its way in and out
    // would take longer): 64 tokens x 8 key heads over up to 4100 rows of 128, any length, 123 to 134 us, with half as many CTAs 138 us,
    // twice as many 130 us; with all caches full, where nothing is uneven, 170, 158 and 172 us.  2 tokens x 4 over 1028 rows: 8.2 us
    p.split = 1;
    while (p.split < MAX_SPLIT && units * p.split < 6 * sm_count() && (in.W + in.S) / (2 * p.split) >= 64) p.split *= 2;
    const cudaError_t e = set_dynamic_smem(reinterpret_cast<const void *>(&window_step<E, D, HG>), SMEM<D, HG>);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(units * p.split));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM<D, HG>;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, window_step<E, D, HG>, p, static_cast<E *>(cache_k), static_cast<E *>(cache_v), static_cast<E *>(o));
}

// A warp a token of the packed sequences: its key and value heads into the sequence's slot, where the window still holds it.
template <int D>
__global__ void __launch_bounds__(256) cache_fill(const int32_t *plan, PlanSig sig, int N, int off_cu, int T, const FillIn in, uint4 *cache_k,
                                                  uint4 *cache_v)
{
    constexpr int CH = D / 8;                // 16-byte pieces of a head
    if (!plan_matches(plan, sig)) {
        if (threadIdx.x == 0 && blockIdx.x == 0) record_status(&g_cache_status, KDA_ERR_INVALID_ARG);
        return;
    }
    const int32_t *cu = plan + off_cu;
    const int lane = threadIdx.x & 31, cap = in.S + in.W;
    for (int64_t t = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / 32; t < T; t += static_cast<int64_t>(gridDim.x) * blockDim.x / 32) {
        int lo = 0, count = N;               // the token's sequence, 32 candidates at a time
        while (true) {
            const int stride = (count + 31) / 32;
            const bool before = lane * stride < count && cu[lo + lane * stride] <= t;
            const int last = __popc(__ballot_sync(0xffffffffu, before)) - 1;
            lo += last * stride;
            count = min(stride, count - last * stride);
            if (stride == 1) break;
        }
        const int pos = static_cast<int>(t - cu[lo]), len = cu[lo + 1] - cu[lo], slot = in.slots ? in.slots[lo] : lo;
        if (slot < 0) continue;
        if (slot >= in.num_slots) {
            if (lane == 0) record_status(&g_cache_status, KDA_ERR_INVALID_ARG);
            continue;
        }
        if (pos >= in.S && pos < len - in.W) continue;
        const int row = pos < in.S ? pos : in.S + (pos - in.S) % in.W;
        const uint4 *const k = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(in.k) + t * in.ldk);
        const uint4 *const v = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(in.v) + t * in.ldv);
        for (int i = lane; i < in.Hk * CH; i += 32) {
            const int64_t to = ((static_cast<int64_t>(slot) * in.Hk + i / CH) * cap + row) * CH + i % CH;
            cache_k[to] = k[i];
            cache_v[to] = v[i];
        }
    }
}

}  // namespace

cudaError_t launch_window_step(int type, const StepIn &in, void *cache_k, void *cache_v, void *o, int64_t ldo, cudaStream_t stream)
{
    const Step p{in, in.H / in.Hk, 1, 1, in.scale * 1.44269504088896340736f, ldo};
    if (type == KDA_TYPE_F16) {
        if (in.d == 64) return p.g > 8 ? step<__half, 64, 16>(p, cache_k, cache_v, o, stream) : step<__half, 64, 8>(p, cache_k, cache_v, o, stream);
        return p.g > 8 ? step<__half, 128, 16>(p, cache_k, cache_v, o, stream) : step<__half, 128, 8>(p, cache_k, cache_v, o, stream);
    }
    if (in.d == 64)
        return p.g > 8 ? step<__nv_bfloat16, 64, 16>(p, cache_k, cache_v, o, stream) : step<__nv_bfloat16, 64, 8>(p, cache_k, cache_v, o, stream);
    return p.g > 8 ? step<__nv_bfloat16, 128, 16>(p, cache_k, cache_v, o, stream) : step<__nv_bfloat16, 128, 8>(p, cache_k, cache_v, o, stream);
}

cudaError_t launch_window_fill(const int32_t *plan_host, const int32_t *plan_dev, const FillIn &in, void *cache_k, void *cache_v, cudaStream_t stream)
{
    const int T = plan_host[KDA_PH_T];
    const int grid = static_cast<int>(min((static_cast<int64_t>(T) + 7) / 8, static_cast<int64_t>(sm_count()) * 8));
    auto fill = in.d == 64 ? cache_fill<64> : cache_fill<128>;
    fill<<<grid, 256, 0, stream>>>(plan_dev, plan_sig(plan_host), plan_host[KDA_PH_N], plan_host[KDA_PH_OFF_CU], T, in, static_cast<uint4 *>(cache_k),
                                   static_cast<uint4 *>(cache_v));
    return cudaGetLastError();
}

int take_cache_status()
{
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_cache_status, sizeof(int)) != cudaSuccess) return KDA_ERR_CUDA;
    if (v != 0 && cudaMemcpyToSymbol(g_cache_status, &z, sizeof(int)) != cudaSuccess) return KDA_ERR_CUDA;
    return v;
}

}  // namespace kda
