// C ABI entry points of libkda (declared and documented in include/kda.h).
//
// Every call validates its arguments on the host and enqueues nothing when it
// rejects them; no call allocates, frees or synchronises.  There is no
// fallback path (cuLA PR #110, "feat(cp): add opt-in NVSHMEM CP state handoff",
// §Supported configuration: request an error instead of fallback).
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <mutex>
#include <utility>

#include "elem.cuh"
#include "kda_internal.cuh"

namespace {

thread_local int g_last_cuda_error = 0;

int cuda_status(cudaError_t e)
{
    if (e == cudaSuccess) return KDA_OK;
    g_last_cuda_error = static_cast<int>(e);
    return KDA_ERR_CUDA;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A host plan is accepted when kda_plan_check accepts it.  The check re-plans, so the plans
// already accepted are remembered by (length, checksum, T, N, S); a plan whose words hash to a
// remembered entry is accepted after the O(length) checksum pass alone.
struct PlanKey {
    int32_t total, checksum, T, N, S;
    bool operator==(const PlanKey &o) const
    {
        return total == o.total && checksum == o.checksum && T == o.T && N == o.N && S == o.S;
    }
};
std::mutex g_plan_mutex;
PlanKey g_plan_seen[16];
int g_plan_seen_n = 0, g_plan_seen_next = 0;

bool plan_ok(const int32_t *plan)
{
    if (!plan) return false;
    if (plan[KDA_PH_MAGIC] != KDA_PLAN_MAGIC || plan[KDA_PH_VERSION] != KDA_PLAN_VERSION) return false;
    if (plan[KDA_PH_TOTAL] < KDA_PLAN_HEADER_WORDS) return false;
    const uint32_t sum = kda::plan_checksum_words(plan, static_cast<size_t>(plan[KDA_PH_TOTAL]));
    if (sum != static_cast<uint32_t>(plan[KDA_PH_CHECKSUM])) return false;
    const PlanKey key{plan[KDA_PH_TOTAL], plan[KDA_PH_CHECKSUM], plan[KDA_PH_T], plan[KDA_PH_N], plan[KDA_PH_S]};
    {
        std::lock_guard<std::mutex> lock(g_plan_mutex);
        for (int i = 0; i < g_plan_seen_n; ++i)
            if (g_plan_seen[i] == key) return true;
    }
    if (kda_plan_check(plan) != KDA_OK) return false;
    std::lock_guard<std::mutex> lock(g_plan_mutex);
    g_plan_seen[g_plan_seen_next] = key;
    g_plan_seen_next = (g_plan_seen_next + 1) % 16;
    if (g_plan_seen_n < 16) ++g_plan_seen_n;
    return true;
}

size_t round256(size_t x) { return (x + 255u) & ~static_cast<size_t>(255u); }

constexpr int kBlockedMinSegments = 16;   // fewer segments always compose by the chain

bool layout(const int32_t *plan, int32_t H, size_t off[7])
{
    if (!plan_ok(plan) || H < 1) return false;
    const size_t h = static_cast<size_t>(H), K = kda::KD, V = kda::VD;
    const size_t sizes[6] = {
        h * static_cast<size_t>(plan[KDA_PH_TCONT]) * K * 2,                 // qhat (bf16)
        static_cast<size_t>(plan[KDA_PH_NFIN]) * h * K * K * 4,              // fin transitions
        static_cast<size_t>(plan[KDA_PH_NCHUNKS]) * h * KDA_PACKAGE_BYTES,   // chunk packages
        static_cast<size_t>(plan[KDA_PH_S]) * h * K * K * 4,                 // A
        static_cast<size_t>(plan[KDA_PH_S]) * h * K * V * 4,                 // B
        static_cast<size_t>(plan[KDA_PH_S]) * h * K * V * 4,                 // S_in
    };
    size_t pos = 0;
    for (int i = 0; i < 6; ++i) {
        off[i] = pos;
        pos = round256(pos + sizes[i]);
    }
    // from 16 segments on, room for the two-level scan's group totals and incoming states after S_in
    if (plan[KDA_PH_S] >= kBlockedMinSegments) pos = round256(pos + kda::scan_scratch_bytes(plan, H));
    off[6] = pos;
    return true;
}

// The composition schedule of the fused entry points: the two-level scan where its estimated depth,
// counted in products per CTA over the waves the device's SMs need, is below the chain's.
bool use_blocked_scan(const int32_t *plan, int32_t H)
{
    const long long S = plan[KDA_PH_S];
    if (S < kBlockedMinSegments) return false;
    const long long sm = kda::sm_count(), m = kda::scan_group_size(static_cast<int>(S)), G = (S + m - 1) / m;
    auto waves = [&](long long ctas) { return (ctas + sm - 1) / sm; };
    const long long chain = waves(4LL * H) * S;
    const long long blocked = waves(8LL * H * G) * (m + 1) + (G - 1) + waves(4LL * H * G) * (m + 1);
    return blocked < chain;
}

bool inputs_ok(const void *q, const void *k, const void *v, const float *g, const float *beta,
               const float *h0)
{
    if (!q || !k || !v || !g || !beta) return false;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(beta)) return false;
    if (h0 && !aligned16(h0)) return false;
    return true;
}

size_t S_in_bytes(const int32_t *plan, int32_t H)
{
    return static_cast<size_t>(plan[KDA_PH_S]) * static_cast<size_t>(H) * kda::KD * kda::VD * 4;
}

kda::Workspace carve(void *ws, const size_t off[7])
{
    char *b = static_cast<char *>(ws);
    return kda::Workspace{reinterpret_cast<uint16_t *>(b + off[0]), reinterpret_cast<float *>(b + off[1]),
                          reinterpret_cast<unsigned char *>(b + off[2]), reinterpret_cast<float *>(b + off[3]),
                          reinterpret_cast<float *>(b + off[4]), reinterpret_cast<float *>(b + off[5])};
}

// Bytes of the qhat + fin regions that kda_apply_boundary reads.
size_t boundary_bytes(const size_t off[7]) { return off[2]; }
// Bytes of the qhat + fin + package regions that kda_segment_forward uses.
size_t segment_bytes(const size_t off[7]) { return off[3]; }

}  // namespace

extern "C" const char *kda_status_string(int status)
{
    switch (status) {
    case KDA_OK: return "ok";
    case KDA_ERR_INVALID_ARG: return "invalid argument";
    case KDA_ERR_UNSUPPORTED: return "unsupported configuration";
    case KDA_ERR_WORKSPACE: return "buffer too small";
    case KDA_ERR_CUDA: return "CUDA error";
    case KDA_ERR_TIMEOUT: return "device wait timed out";
    case KDA_ERR_RANGE: return "decay out of the chunkwise range";
    default: return "unknown status";
    }
}

extern "C" int kda_last_cuda_error(void) { return g_last_cuda_error; }

extern "C" int kda_selftest_wait_expiry(void *stream)
{
    return cuda_status(kda::launch_wait_expiry_probe(static_cast<cudaStream_t>(stream)));
}

extern "C" int kda_selftest_state_abort(const int32_t *plan, const int32_t *plan_dev, int32_t H,
                                        const kda_bf16 *q, const kda_bf16 *k, const kda_bf16 *v, const float *g,
                                        const float *beta, const float *h0, float scale, kda_bf16 *o, float *A,
                                        float *B, float *final_state, void *ws, size_t ws_bytes, void *stream)
{
    size_t off[7];
    if (!layout(plan, H, off) || !plan_dev) return KDA_ERR_INVALID_ARG;
    if (plan[KDA_PH_MAXPIECE] <= KDA_CHUNK) return KDA_ERR_INVALID_ARG;   // needs a piece of two chunks
    if (!inputs_ok(q, k, v, g, beta, h0)) return KDA_ERR_INVALID_ARG;
    if (!o || !A || !B || !final_state || !aligned16(o) || !aligned16(A) || !aligned16(B) ||
        !aligned16(final_state))
        return KDA_ERR_INVALID_ARG;
    if (!ws || !aligned16(ws)) return KDA_ERR_INVALID_ARG;
    if (ws_bytes < off[3]) return KDA_ERR_WORKSPACE;
    const kda::Workspace w = carve(ws, off);
    return cuda_status(kda::launch_state_abort_selftest(plan, plan_dev, H, q, k, v, g, beta, h0, scale, o, A, B,
                                                        final_state, w.qhat, w.afin, w.pkg,
                                                        static_cast<cudaStream_t>(stream)));
}

extern "C" int kda_device_status(void)
{
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        g_last_cuda_error = static_cast<int>(e);
        return KDA_ERR_CUDA;
    }
    int worst = KDA_OK;
    for (int st : {kda::take_prep_status(), kda::take_state_status(), kda::take_compose_status(),
                   kda::take_boundary_status(), kda::take_backward_status(), kda::take_reverse_status(),
                   kda::take_scan_status(), kda::take_scan_backward_status(), kda::take_decode_status(), kda::take_window_status(), kda::take_window_back_status(),
                   kda::take_cache_status()})
        if (st != KDA_OK && worst == KDA_OK) worst = st;
    return worst;
}

namespace kda {
void record_cuda_error(int err) { g_last_cuda_error = err; }

PFN_cuTensorMapEncodeTiled_v12000 tmap_encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

bool encode_f32_rows(CUtensorMap *m, const void *ptr, uint64_t rows, uint32_t cols, uint32_t box_rows)
{
    auto fn = tmap_encode_fn();
    if (!fn || rows == 0) return false;
    const cuuint64_t dims[2] = {cols, static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 4};
    const cuuint32_t box[2] = {32, box_rows};
    const cuuint32_t es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void *>(ptr), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_f32_rows128(CUtensorMap *m, const void *ptr, uint64_t rows, uint32_t box_rows)
{
    return encode_f32_rows(m, ptr, rows, 128, box_rows);
}

bool encode_rows_3d(CUtensorMap *m, const void *ptr, CUtensorMapDataType dt, uint32_t elem, int H, int T,
                    uint32_t inner, uint32_t box_rows)
{
    auto fn = tmap_encode_fn();
    if (!fn || T <= 0) return false;
    const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T)};
    const cuuint64_t strides[2] = {128ull * elem, 128ull * elem * static_cast<cuuint64_t>(H)};
    const cuuint32_t box[3] = {inner, 1, box_rows};
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(m, dt, 3, const_cast<void *>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Unique id of the calling thread's current context (driver entry points, looked up once).
cudaError_t current_context_id(unsigned long long *id)
{
    using GetCurrent = CUresult (*)(CUcontext *);
    using GetId = CUresult (*)(CUcontext, unsigned long long *);
    static GetCurrent get_current = nullptr;
    static GetId get_id = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_current = reinterpret_cast<GetCurrent>(p);
        p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_id = reinterpret_cast<GetId>(p);
    });
    if (!get_current || !get_id) return cudaErrorNotSupported;
    CUcontext ctx = nullptr;
    if (get_current(&ctx) != CUDA_SUCCESS) return cudaErrorDeviceUninitialized;
    if (!ctx) {   // nothing current yet on this thread: the runtime would use the primary context
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaSetDevice(dev);   // initialises and binds the primary context
        if (e != cudaSuccess) return e;
        if (get_current(&ctx) != CUDA_SUCCESS || !ctx) return cudaErrorDeviceUninitialized;
    }
    if (get_id(ctx, id) != CUDA_SUCCESS) return cudaErrorDeviceUninitialized;
    return cudaSuccess;
}

// The dynamic shared-memory limit of a kernel, set once per (kernel, context): the attribute
// belongs to the function in the current context, so after cudaDeviceReset (a new context id) it
// is set again.
cudaError_t set_dynamic_smem(const void *fn, int bytes)
{
    unsigned long long ctx = 0;
    cudaError_t e = current_context_id(&ctx);
    if (e != cudaSuccess) return e;
    struct Done {
        const void *fn;
        unsigned long long ctx;
        int bytes;
    };
    static std::mutex mu;
    static Done done[64];
    static int n_done = 0, next = 0;
    {
        std::lock_guard<std::mutex> lock(mu);
        for (int i = 0; i < n_done; ++i)
            if (done[i].fn == fn && done[i].ctx == ctx && done[i].bytes >= bytes) return cudaSuccess;
    }
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    done[next] = Done{fn, ctx, bytes};
    next = (next + 1) % 64;
    if (n_done < 64) ++n_done;
    return cudaSuccess;
}

int sm_count()
{
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
    if (cached[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
        cached[dev] = n;
    }
    return cached[dev];
}
}  // namespace kda

extern "C" int kda_workspace_layout(const int32_t *plan, int32_t H, size_t off[7])
{
    if (!off) return KDA_ERR_INVALID_ARG;
    return layout(plan, H, off) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

extern "C" size_t kda_workspace_bytes(const int32_t *plan, int32_t H)
{
    size_t off[7];
    return layout(plan, H, off) ? off[6] : 0;
}

extern "C" int kda_segment_forward(const int32_t *plan, const int32_t *plan_dev, int32_t H,
                                   const kda_bf16 *q, const kda_bf16 *k, const kda_bf16 *v,
                                   const float *g, const float *beta, const float *h0, float scale,
                                   kda_bf16 *o, float *A, float *B, float *final_state,
                                   void *ws, size_t ws_bytes, void *stream)
{
    size_t off[7];
    if (!layout(plan, H, off) || !plan_dev) return KDA_ERR_INVALID_ARG;
    if (!inputs_ok(q, k, v, g, beta, h0)) return KDA_ERR_INVALID_ARG;
    if (!o || !A || !B || !final_state || !aligned16(o) || !aligned16(A) || !aligned16(B) ||
        !aligned16(final_state))
        return KDA_ERR_INVALID_ARG;
    if (segment_bytes(off) > 0 && (!ws || !aligned16(ws))) return KDA_ERR_INVALID_ARG;
    if (ws_bytes < segment_bytes(off)) return KDA_ERR_WORKSPACE;
    const kda::Workspace w = carve(ws, off);
    return cuda_status(kda::launch_chunk_forward(plan, plan_dev, H, q, k, v, g, beta, h0, scale, o, A, B,
                                                 final_state, w.qhat, w.afin, w.pkg,
                                                 static_cast<cudaStream_t>(stream)));
}

extern "C" int kda_compose_summaries(const int32_t *plan, const int32_t *plan_dev, int32_t H,
                                     const float *A, const float *B, const float *h0, float *S_in,
                                     void *stream)
{
    size_t off[7];
    if (!layout(plan, H, off) || !plan_dev) return KDA_ERR_INVALID_ARG;
    if (!A || !B || !S_in || !aligned16(A) || !aligned16(B) || !aligned16(S_in)) return KDA_ERR_INVALID_ARG;
    if (h0 && !aligned16(h0)) return KDA_ERR_INVALID_ARG;
    return cuda_status(kda::launch_compose(plan, plan_dev, H, A, B, h0, S_in, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t kda_scan_workspace_bytes(const int32_t *plan, int32_t H)
{
    size_t off[7];
    if (!layout(plan, H, off)) return 0;
    return kda::scan_scratch_bytes(plan, H);
}

extern "C" int kda_compose_summaries_blocked(const int32_t *plan, const int32_t *plan_dev, int32_t H,
                                             const float *A, const float *B, const float *h0, float *S_in,
                                             void *ws, size_t ws_bytes, void *stream)
{
    size_t off[7];
    if (!layout(plan, H, off) || !plan_dev) return KDA_ERR_INVALID_ARG;
    if (!A || !B || !S_in || !aligned16(A) || !aligned16(B) || !aligned16(S_in)) return KDA_ERR_INVALID_ARG;
    if (h0 && !aligned16(h0)) return KDA_ERR_INVALID_ARG;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return KDA_ERR_INVALID_ARG;
    if (ws_bytes < kda::scan_scratch_bytes(plan, H)) return KDA_ERR_WORKSPACE;
    return cuda_status(kda::launch_compose_blocked(plan, plan_dev, H, A, B, h0, S_in, ws,
                                                   static_cast<cudaStream_t>(stream)));
}

extern "C" int kda_apply_boundary(const int32_t *plan, const int32_t *plan_dev, int32_t H,
                                  const float *S_in, const void *ws, size_t ws_bytes, kda_bf16 *o,
                                  float *final_state, void *stream)
{
    size_t off[7];
    if (!layout(plan, H, off) || !plan_dev) return KDA_ERR_INVALID_ARG;
    if (!S_in || !o || !final_state || !aligned16(S_in) || !aligned16(o) || !aligned16(final_state))
        return KDA_ERR_INVALID_ARG;
    if (boundary_bytes(off) > 0 && (!ws || !aligned16(ws))) return KDA_ERR_INVALID_ARG;
    if (ws_bytes < boundary_bytes(off)) return KDA_ERR_WORKSPACE;
    const kda::Workspace w = carve(const_cast<void *>(ws), off);
    return cuda_status(kda::launch_boundary(plan, plan_dev, H, S_in, w.qhat, w.afin, o, final_state,
                                            static_cast<cudaStream_t>(stream)));
}

extern "C" int kda_forward_segmented(const int32_t *plan, const int32_t *plan_dev, int32_t H,
                                     const kda_bf16 *q, const kda_bf16 *k, const kda_bf16 *v,
                                     const float *g, const float *beta, const float *h0, float scale,
                                     kda_bf16 *o, float *final_state, void *ws, size_t ws_bytes,
                                     void *stream)
{
    size_t off[7];
    if (!layout(plan, H, off) || !plan_dev) return KDA_ERR_INVALID_ARG;
    if (!inputs_ok(q, k, v, g, beta, h0)) return KDA_ERR_INVALID_ARG;
    if (!o || !final_state || !aligned16(o) || !aligned16(final_state)) return KDA_ERR_INVALID_ARG;
    if (!ws || !aligned16(ws)) return KDA_ERR_INVALID_ARG;
    if (ws_bytes < off[6]) return KDA_ERR_WORKSPACE;
    const kda::Workspace w = carve(ws, off);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int rc = cuda_status(kda::launch_chunk_forward(plan, plan_dev, H, q, k, v, g, beta, h0, scale, o, w.A, w.B,
                                                   final_state, w.qhat, w.afin, w.pkg, s));
    if (rc != KDA_OK) return rc;
    rc = cuda_status(use_blocked_scan(plan, H)
                         ? kda::launch_compose_blocked(plan, plan_dev, H, w.A, w.B, h0, w.S_in,
                                                       static_cast<char *>(ws) + round256(off[5] + S_in_bytes(plan, H)), s)
                         : kda::launch_compose(plan, plan_dev, H, w.A, w.B, h0, w.S_in, s));
    if (rc != KDA_OK) return rc;
    return cuda_status(kda::launch_boundary(plan, plan_dev, H, w.S_in, w.qhat, w.afin, o, final_state, s));
}

extern "C" int kda_forward_two_pass(const int32_t *plan, const int32_t *plan_dev, int32_t H,
                                    const kda_bf16 *q, const kda_bf16 *k, const kda_bf16 *v,
                                    const float *g, const float *beta, const float *h0, float scale,
                                    kda_bf16 *o, float *final_state, void *ws, size_t ws_bytes, void *stream)
{
    size_t off[7];
    if (!layout(plan, H, off) || !plan_dev) return KDA_ERR_INVALID_ARG;
    if (!inputs_ok(q, k, v, g, beta, h0)) return KDA_ERR_INVALID_ARG;
    if (!o || !final_state || !aligned16(o) || !aligned16(final_state)) return KDA_ERR_INVALID_ARG;
    if (!ws || !aligned16(ws)) return KDA_ERR_INVALID_ARG;
    if (ws_bytes < off[6]) return KDA_ERR_WORKSPACE;
    const kda::Workspace w = carve(ws, off);
    return cuda_status(kda::launch_two_pass(plan, plan_dev, H, q, k, v, g, beta, h0, scale, o, w.A, w.B, w.S_in,
                                            final_state, w.pkg, static_cast<cudaStream_t>(stream)));
}

namespace {

constexpr int kBackwardGrid = 152;   // CTAs of the backward's chunk and piece kernels (grid-stride)

// Regions of the backward's workspace after the forward's: o and final states of the forward run it
// needs (not returned), the chunk start states and end gradients, the segment end gradients and
// continuing pieces' incoming-state gradients, the CTAs' scratch, and each chunk's terms for the chains.
bool backward_layout(const int32_t *plan, int32_t H, size_t off[10])
{
    size_t fw[7];
    if (!layout(plan, H, fw)) return false;
    const size_t h = static_cast<size_t>(H), K = kda::KD, V = kda::VD;
    const size_t T = static_cast<size_t>(plan[KDA_PH_T]), N = static_cast<size_t>(plan[KDA_PH_N]);
    const size_t S = static_cast<size_t>(plan[KDA_PH_S]), C = static_cast<size_t>(plan[KDA_PH_NCHUNKS]);
    const size_t sizes[9] = {T * h * V * 2, N * h * K * V * 4, h * C * K * V * 4, h * C * K * V * 4,
                             S * h * K * V * 4, S * h * K * V * 4,
                             static_cast<size_t>(kBackwardGrid) * kda::backward_scratch_floats() * 4,
                             h * C * kda::BT_FLOATS * 4, h * C * kda::RIMG_UNIT};
    size_t pos = fw[6];
    for (int i = 0; i < 9; ++i) {
        off[i] = pos;
        pos = round256(pos + sizes[i]);
    }
    off[9] = pos;
    return true;
}

}  // namespace

extern "C" size_t kda_backward_workspace_bytes(const int32_t *plan, int32_t H)
{
    size_t off[10];
    return backward_layout(plan, H, off) ? off[9] : 0;
}

extern "C" int kda_backward_segmented(const int32_t *plan, const int32_t *plan_dev, int32_t H,
                                      const kda_bf16 *q, const kda_bf16 *k, const kda_bf16 *v, const float *g,
                                      const float *beta, const float *h0, float scale, const kda_bf16 *dout,
                                      const float *dfinal, float *dq, float *dk, float *dv, float *dg,
                                      float *dbeta, float *dh0, void *ws, size_t ws_bytes, void *stream)
{
    size_t fw[7], off[10];
    if (!layout(plan, H, fw) || !backward_layout(plan, H, off) || !plan_dev) return KDA_ERR_INVALID_ARG;
    if (!inputs_ok(q, k, v, g, beta, h0)) return KDA_ERR_INVALID_ARG;
    if (!dout || !aligned16(dout) || (dfinal && !aligned16(dfinal)) || (dh0 && !aligned16(dh0)))
        return KDA_ERR_INVALID_ARG;
    if (!dq || !dk || !dv || !dg || !dbeta || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
        !aligned16(dg) || !aligned16(dbeta))
        return KDA_ERR_INVALID_ARG;
    if (!ws || !aligned16(ws)) return KDA_ERR_INVALID_ARG;
    if (ws_bytes < off[9]) return KDA_ERR_WORKSPACE;
    const kda::Workspace w = carve(ws, fw);
    char *b = static_cast<char *>(ws);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    // the forward's local pass and composition: S_in, the segment transitions A and the final-state
    // transitions of continuing pieces
    // (its preparation in backward mode also leaves each chunk's FP32 terms and operand images)
    int rc = cuda_status(kda::launch_chunk_forward(plan, plan_dev, H, q, k, v, g, beta, h0, scale,
                                                   reinterpret_cast<uint16_t *>(b + off[0]), w.A, w.B,
                                                   reinterpret_cast<float *>(b + off[1]), w.qhat, w.afin, w.pkg, s,
                                                   reinterpret_cast<unsigned char *>(b + off[8]),
                                                   reinterpret_cast<float *>(b + off[7])));
    if (rc != KDA_OK) return rc;
    rc = cuda_status(use_blocked_scan(plan, H)
                         ? kda::launch_compose_blocked(plan, plan_dev, H, w.A, w.B, h0, w.S_in,
                                                       b + round256(fw[5] + S_in_bytes(plan, H)), s)
                         : kda::launch_compose(plan, plan_dev, H, w.A, w.B, h0, w.S_in, s));
    if (rc != KDA_OK) return rc;
    // every piece again from its true incoming state, recording each chunk's start state
    rc = cuda_status(kda::launch_state_record(plan, plan_dev, H, h0, w.S_in, w.pkg,
                                              reinterpret_cast<uint16_t *>(b + off[0]),
                                              reinterpret_cast<float *>(b + off[1]),
                                              reinterpret_cast<float *>(b + off[2]), s));
    if (rc != KDA_OK) return rc;
    return cuda_status(kda::launch_backward(
        plan, plan_dev, H, q, k, v, g, beta, scale, dout, dfinal, w.A, w.afin,
        reinterpret_cast<const float *>(b + off[2]), reinterpret_cast<float *>(b + off[3]),
        reinterpret_cast<float *>(b + off[4]), reinterpret_cast<float *>(b + off[5]), w.S_in,
        reinterpret_cast<const float *>(b + off[1]), reinterpret_cast<float *>(b + off[7]),
        reinterpret_cast<unsigned char *>(b + off[8]),
        reinterpret_cast<float *>(b + off[6]), kBackwardGrid, dq, dk, dv, dg, dbeta, dh0, s));
}

// ---- the operators around the KDA layer ------------------------------------------------------------

namespace {

// A tensor of rows: present, aligned to its elements, its rows at least 'width' apart.
bool rows_ok(const void *p, int64_t ld, int64_t width, int bytes)
{
    return p && (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes)) == 0 && ld >= width;
}
bool rows_ok_or_null(const void *p, int64_t ld, int64_t width, int bytes) { return !p || rows_ok(p, ld, width, bytes); }
bool floats_ok_or_null(const float *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool scan_in_ok(int32_t D, int32_t type, const kda::ScanIn &in)
{
    const int e = kda::elem_bytes(type);
    return D >= 1 && e && rows_ok(in.x, in.ldx, D, e) && rows_ok_or_null(in.i, in.ldi, D, e) &&
           rows_ok(in.g, in.ldg, D, 4) && floats_ok_or_null(in.h0);
}

// The workspace, where the call needs one.
int scan_ws_ok(const int32_t *plan, int32_t D, const void *ws, size_t ws_bytes)
{
    const size_t need = kda::scan_workspace_bytes(plan[KDA_PH_T], D);
    if (need && (!ws || !aligned16(ws))) return KDA_ERR_INVALID_ARG;
    return ws_bytes < need ? KDA_ERR_WORKSPACE : KDA_OK;
}

bool norm_group_ok(int32_t D, int32_t group)
{
    return group == 0 || group == D ||
           ((group == 32 || group == 64 || group == 128 || group == 256) && D % group == 0);
}

// The block norm's kernels count rows in 32 bits and step between them by a 32-bit number of bytes.
bool norm_steps_ok(int64_t T, std::initializer_list<std::pair<int64_t, int>> strides)
{
    for (const auto &s : strides)
        if (s.first > INT32_MAX / s.second) return false;
    return T <= INT32_MAX;
}

// What both directions of the block norm check of the arguments they share.
int norm_in_ok(int64_t T, int32_t D, int32_t rtype, int32_t type, const kda::NormIn &a, float eps)
{
    const int e = kda::elem_bytes(type), re = kda::elem_bytes(rtype);
    if (T < 0 || D < 1 || !e || !re || !(eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    if (rtype != type && rtype != KDA_TYPE_F32) return KDA_ERR_UNSUPPORTED;
    if (D > kda::NORM_MAX_D || !norm_group_ok(D, a.group)) return KDA_ERR_UNSUPPORTED;
    if (a.gate != KDA_GATE_NONE && a.gate != KDA_GATE_SIGMOID && a.gate != KDA_GATE_SILU) return KDA_ERR_INVALID_ARG;
    if (T == 0) return KDA_OK;   // no rows: their addresses do not matter
    if ((a.gate != KDA_GATE_NONE) != (a.z != nullptr)) return KDA_ERR_INVALID_ARG;
    if (!a.o && (a.z || a.w_post || a.ls)) return KDA_ERR_INVALID_ARG;
    if (!rows_ok_or_null(a.r, a.ldr, D, re) || !rows_ok_or_null(a.o, a.ldo, D, e) || !rows_ok_or_null(a.z, a.ldz, D, e))
        return KDA_ERR_INVALID_ARG;
    if (!floats_ok_or_null(a.w_post) || !floats_ok_or_null(a.ls) || !floats_ok_or_null(a.w_pre)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

}  // namespace

extern "C" size_t kda_gated_scan_workspace_bytes(const int32_t *plan, int32_t D)
{
    return plan_ok(plan) && D >= 1 && D <= kda::SCAN_MAX_D ? kda::scan_workspace_bytes(plan[KDA_PH_T], D) : 0;
}

extern "C" int kda_gated_scan_forward(const int32_t *plan, const int32_t *plan_dev, int32_t D, int32_t type,
                                      const void *x, int64_t ldx, const void *i, int64_t ldi, const float *g, int64_t ldg,
                                      const float *h0, void *h, int64_t ldh, float *final_state, float *states,
                                      void *ws, size_t ws_bytes, void *stream)
{
    const kda::ScanIn in{x, i, g, h0, ldx, ldi, ldg};
    if (!plan_ok(plan) || !plan_dev || !scan_in_ok(D, type, in)) return KDA_ERR_INVALID_ARG;
    if (!rows_ok(h, ldh, D, kda::elem_bytes(type)) || !floats_ok_or_null(final_state) || !floats_ok_or_null(states))
        return KDA_ERR_INVALID_ARG;
    if (D > kda::SCAN_MAX_D) return KDA_ERR_UNSUPPORTED;
    if (const int rc = scan_ws_ok(plan, D, ws, ws_bytes)) return rc;
    return cuda_status(kda::launch_scan_forward(plan, plan_dev, D, type, in, h, ldh, final_state, states, ws,
                                                static_cast<cudaStream_t>(stream)));
}

extern "C" int kda_gated_scan_backward(const int32_t *plan, const int32_t *plan_dev, int32_t D, int32_t type,
                                       const void *x, int64_t ldx, const void *i, int64_t ldi, const float *g, int64_t ldg,
                                       const float *h0, const float *states, const void *dh, int64_t lddh,
                                       const float *dfinal, void *dx, int64_t lddx, void *di, int64_t lddi, float *dg,
                                       int64_t lddg, float *dh0, void *ws, size_t ws_bytes, void *stream)
{
    const kda::ScanIn in{x, i, g, h0, ldx, ldi, ldg};
    const kda::ScanGrads out{dx, di, dg, dh0, lddx, lddi, lddg};
    if (!plan_ok(plan) || !plan_dev || !scan_in_ok(D, type, in)) return KDA_ERR_INVALID_ARG;
    const int e = kda::elem_bytes(type);
    if (!states || !floats_ok_or_null(states) || !rows_ok(dh, lddh, D, e) || !floats_ok_or_null(dfinal))
        return KDA_ERR_INVALID_ARG;
    if (!rows_ok(dx, lddx, D, e) || !rows_ok_or_null(di, lddi, D, e) || !rows_ok(dg, lddg, D, 4) || !floats_ok_or_null(dh0))
        return KDA_ERR_INVALID_ARG;
    if (di && !i) return KDA_ERR_INVALID_ARG;
    if (D > kda::SCAN_MAX_D) return KDA_ERR_UNSUPPORTED;
    if (const int rc = scan_ws_ok(plan, D, ws, ws_bytes)) return rc;
    return cuda_status(kda::launch_scan_backward(plan, plan_dev, D, type, in, states, dh, lddh, dfinal, out, ws,
                                                 static_cast<cudaStream_t>(stream)));
}

extern "C" int kda_gated_scan_step(int32_t B, int32_t D, int32_t type, const int32_t *slots, int32_t num_slots,
                                   const void *x, int64_t ldx, const void *i, int64_t ldi, const float *g, int64_t ldg,
                                   float *state, void *h, int64_t ldh, void *stream)
{
    const kda::ScanIn in{x, i, g, nullptr, ldx, ldi, ldg};
    if (B < 0 || num_slots < 0 || (!slots && B > num_slots)) return KDA_ERR_INVALID_ARG;
    if (B == 0) return D >= 1 && kda::elem_bytes(type) ? KDA_OK : KDA_ERR_INVALID_ARG;
    if (!scan_in_ok(D, type, in) || !state || !floats_ok_or_null(state) || !rows_ok(h, ldh, D, kda::elem_bytes(type)) ||
        (reinterpret_cast<uintptr_t>(slots) & 3u))
        return KDA_ERR_INVALID_ARG;
    if (D > kda::SCAN_MAX_D) return KDA_ERR_UNSUPPORTED;
    return cuda_status(kda::launch_scan_step(B, D, type, slots, num_slots, in, state, h, ldh,
                                             static_cast<cudaStream_t>(stream)));
}

extern "C" size_t kda_block_norm_workspace_bytes(int32_t D)
{
    return D >= 1 && D <= kda::NORM_MAX_D ? kda::norm_workspace_bytes(D) : 0;
}

extern "C" int kda_block_norm_forward(int64_t T, int32_t D, int32_t res_type, int32_t type, const void *r, int64_t ldr,
                                      const void *o, int64_t ldo, const void *z, int64_t ldz, int32_t gate, int32_t group,
                                      const float *w_post, float scale, const float *ls, const float *w_pre, float eps,
                                      void *r_out, int64_t ldr_out, void *y, int64_t ldy, void *stream)
{
    const kda::NormIn a{r, o, z, ldr, ldo, ldz, w_post, ls, w_pre, gate, group, scale, eps};
    const int rc = norm_in_ok(T, D, res_type, type, a, eps);
    if (rc != KDA_OK || T == 0) return rc;
    if ((y != nullptr) != (w_pre != nullptr) || (!y && !r_out)) return KDA_ERR_INVALID_ARG;
    if (!r && !o) return KDA_ERR_INVALID_ARG;
    if (!rows_ok_or_null(r_out, ldr_out, D, kda::elem_bytes(res_type)) || !rows_ok_or_null(y, ldy, D, kda::elem_bytes(type)))
        return KDA_ERR_INVALID_ARG;
    const int e = kda::elem_bytes(type), re = kda::elem_bytes(res_type);
    if (!norm_steps_ok(T, {{r ? ldr : 0, re}, {o ? ldo : 0, e}, {z ? ldz : 0, e}, {r_out ? ldr_out : 0, re}, {y ? ldy : 0, e}}))
        return KDA_ERR_UNSUPPORTED;
    return cuda_status(kda::launch_norm_forward(T, D, res_type, type, a, r_out, ldr_out, y, ldy,
                                                static_cast<cudaStream_t>(stream)));
}

extern "C" int kda_block_norm_backward(int64_t T, int32_t D, int32_t res_type, int32_t type, const void *r_out,
                                       int64_t ldr_out, const void *o, int64_t ldo, const void *z, int64_t ldz,
                                       int32_t gate, int32_t group, const float *w_post, float scale, const float *ls,
                                       const float *w_pre, float eps, const void *dr_out, int64_t lddr_out, const void *dy,
                                       int64_t lddy, void *dr, int64_t lddr, void *d_o, int64_t lddo, void *dz,
                                       int64_t lddz, float *dw_post, float *dls, float *dw_pre, void *ws, size_t ws_bytes,
                                       void *stream)
{
    const kda::NormIn a{r_out, o, z, ldr_out, ldo, ldz, w_post, ls, w_pre, gate, group, scale, eps};
    const kda::NormGrads g{dr, d_o, dz, lddr, lddo, lddz, dw_post, dls, dw_pre};
    if (const int rc = norm_in_ok(T, D, res_type, type, a, eps)) return rc;
    const int e = kda::elem_bytes(type), re = kda::elem_bytes(res_type);
    if ((dw_post && !w_post) || (dls && !ls) || (dw_pre && !w_pre)) return KDA_ERR_INVALID_ARG;
    if (!floats_ok_or_null(dw_post) || !floats_ok_or_null(dls) || !floats_ok_or_null(dw_pre)) return KDA_ERR_INVALID_ARG;
    if (T > 0) {
        if ((dy != nullptr) != (w_pre != nullptr) || (!dy && !dr_out) || (w_pre && !r_out)) return KDA_ERR_INVALID_ARG;
        if ((d_o != nullptr) != (o != nullptr) || (!dr && !d_o) || (dz && !z))
            return KDA_ERR_INVALID_ARG;
        if (!rows_ok_or_null(dr_out, lddr_out, D, re) || !rows_ok_or_null(dy, lddy, D, e) || !rows_ok_or_null(dr, lddr, D, re) ||
            !rows_ok_or_null(d_o, lddo, D, e) || !rows_ok_or_null(dz, lddz, D, e))
            return KDA_ERR_INVALID_ARG;
    }
    if (!norm_steps_ok(T, {{r_out ? ldr_out : 0, re}, {o ? ldo : 0, e}, {z ? ldz : 0, e}, {dr_out ? lddr_out : 0, re},
                           {dy ? lddy : 0, e}, {dr ? lddr : 0, re}, {d_o ? lddo : 0, e}, {dz ? lddz : 0, e}}))
        return KDA_ERR_UNSUPPORTED;
    if (!ws || !aligned16(ws)) return KDA_ERR_INVALID_ARG;
    if (ws_bytes < kda::norm_workspace_bytes(D)) return KDA_ERR_WORKSPACE;
    return cuda_status(kda::launch_norm_backward(T, D, res_type, type, a, dr_out, lddr_out, dy, lddy, g, ws,
                                                 static_cast<cudaStream_t>(stream)));
}

extern "C" int kda_decode_step(int32_t B, int32_t H, int32_t type, const int32_t *slots, int32_t num_slots, const void *q,
                               int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv, const float *g,
                               int64_t ldg, const float *beta, int64_t ldb, float scale, float *state, void *o, int64_t ldo,
                               void *stream)
{
    const int e = kda::elem_bytes(type);
    if (B < 0 || H < 1 || !e || num_slots < 0 || (!slots && B > num_slots)) return KDA_ERR_INVALID_ARG;
    if (H > 65535) return KDA_ERR_UNSUPPORTED;
    if (B == 0) return KDA_OK;
    const int64_t w = static_cast<int64_t>(H) * kda::KD;
    if (!rows_ok(q, ldq, w, e) || !rows_ok(k, ldk, w, e) || !rows_ok(v, ldv, w, e) || !rows_ok(g, ldg, w, 4) ||
        !rows_ok(beta, ldb, H, 4) || !rows_ok(o, ldo, w, e) || !state || !aligned16(state) ||
        (reinterpret_cast<uintptr_t>(slots) & 3u))
        return KDA_ERR_INVALID_ARG;
    const kda::DecodeIn in{q, k, v, g, beta, ldq, ldk, ldv, ldg, ldb};
    return cuda_status(kda::launch_decode_step(B, H, type, slots, num_slots, in, scale, state, o, ldo,
                                               static_cast<cudaStream_t>(stream)));
}

// ---- the attention layer beside the KDA layer -----------------------------------------------------------

namespace {

// What both directions of the head norms check of the arguments they share; 'x': whether q and k are read.
int head_in_ok(const kda::HeadIn &a, int32_t type, int32_t pairs, bool x)
{
    const int e = kda::elem_bytes(type);
    if (a.T < 0 || a.H < 1 || a.Hk < 0 || a.d < 1 || !e || a.rot < 0) return KDA_ERR_INVALID_ARG;
    if ((a.norm != 0 && a.norm != 1) || (pairs != KDA_PAIRS_HALVES && pairs != KDA_PAIRS_ADJACENT)) return KDA_ERR_INVALID_ARG;
    if (a.d != 32 && a.d != 64 && a.d != 128 && a.d != 256) return KDA_ERR_UNSUPPORTED;
    if (a.rot > a.d || a.rot % 16) return KDA_ERR_UNSUPPORTED;
    if (a.H > INT32_MAX / a.d || a.Hk > INT32_MAX / a.d) return KDA_ERR_UNSUPPORTED;     // a row's channels are counted in 32 bits
    if (a.norm ? !(a.eps >= 0.f) : (a.w_q || a.w_k)) return KDA_ERR_INVALID_ARG;
    if (!floats_ok_or_null(a.w_q) || !floats_ok_or_null(a.w_k) || (!a.Hk && a.w_k)) return KDA_ERR_INVALID_ARG;
    if (a.T == 0) return KDA_OK;   // no rows: their addresses do not matter
    if (a.rot && (!a.positions || (reinterpret_cast<uintptr_t>(a.positions) & 3u) || !a.phases || (reinterpret_cast<uintptr_t>(a.phases) & 7u)))
        return KDA_ERR_INVALID_ARG;
    const int64_t w = static_cast<int64_t>(a.H) * a.d, wk = static_cast<int64_t>(a.Hk) * a.d;
    if (x && (!rows_ok(a.q, a.ldq, w, e) || (a.Hk ? !rows_ok(a.k, a.ldk, wk, e) : a.k != nullptr))) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}
bool head_rows_ok(const kda::HeadIn &a, int32_t type, const kda::HeadOut &x)
{
    const int e = kda::elem_bytes(type);
    return rows_ok(x.q, x.ldq, static_cast<int64_t>(a.H) * a.d, e) &&
           (a.Hk ? rows_ok(x.k, x.ldk, static_cast<int64_t>(a.Hk) * a.d, e) : x.k == nullptr);
}

}  // namespace

// A frequency over 2 pi as two doubles, 107 bits of it: with 53 alone the fraction of a turn is off by 2^-53 of itself, which the position
// multiplies.  Each of the two is cut into 32-bit halves exactly (a remainder and a difference without rounding), of either sign.
extern "C" int kda_rotary_phases(const double *frequencies, int32_t n, uint64_t *phases)
{
    if (n < 0 || (n && (!frequencies || !phases))) return KDA_ERR_INVALID_ARG;
    constexpr double inv_high = 0x1.45f306dc9c883p-3, inv_low = -0x1.6b01ec5417056p-57;      // 1 / (2 pi)
    for (int32_t i = 0; i < n; ++i) {
        const double f = frequencies[i];
        if (!std::isfinite(f)) return KDA_ERR_INVALID_ARG;
        const double turns = f * inv_high, rest = std::fma(f, inv_low, std::fma(f, inv_high, -turns));
        uint64_t high = 0;
        double low = 0.0;
        for (const double x : {turns, rest}) {
            const double part = std::fmod(x, 1.0), top = std::trunc(std::ldexp(part, 32));
            high += static_cast<uint64_t>(static_cast<int64_t>(top));
            low += std::ldexp(part, 64) - std::ldexp(top, 32);
        }
        phases[i] = (high << 32) + static_cast<uint64_t>(static_cast<int64_t>(std::llrint(low)));
    }
    return KDA_OK;
}

extern "C" size_t kda_head_norm_rotary_workspace_bytes(int32_t d)
{
    return d == 32 || d == 64 || d == 128 || d == 256 ? kda::head_workspace_bytes(d) : 0;
}

extern "C" int kda_head_norm_rotary_forward(int64_t T, int32_t H, int32_t Hk, int32_t d, int32_t type, const void *q, int64_t ldq,
                                            const void *k, int64_t ldk, int32_t norm, const float *w_q, const float *w_k, float eps,
                                            const int32_t *positions, const uint64_t *phases, int32_t rot, int32_t pairs, void *q_out,
                                            int64_t ldq_out, void *k_out, int64_t ldk_out, void *stream)
{
    const kda::HeadIn in{q, k, ldq, ldk, T, w_q, w_k, positions, phases, H, Hk, d, rot, pairs, norm, eps};
    const kda::HeadOut out{q_out, k_out, ldq_out, ldk_out};
    const int rc = head_in_ok(in, type, pairs, true);
    if (rc != KDA_OK || T == 0) return rc;
    if (!head_rows_ok(in, type, out)) return KDA_ERR_INVALID_ARG;
    return cuda_status(kda::launch_head_forward(in, type, out, static_cast<cudaStream_t>(stream)));
}

extern "C" int kda_head_norm_rotary_backward(int64_t T, int32_t H, int32_t Hk, int32_t d, int32_t type, const void *q, int64_t ldq,
                                             const void *k, int64_t ldk, int32_t norm, const float *w_q, const float *w_k, float eps,
                                             const int32_t *positions, const uint64_t *phases, int32_t rot, int32_t pairs,
                                             const void *dq_out, int64_t lddq_out, const void *dk_out, int64_t lddk_out, void *dq,
                                             int64_t lddq, void *dk, int64_t lddk, float *dw_q, float *dw_k, void *ws, size_t ws_bytes,
                                             void *stream)
{
    const kda::HeadIn in{q, k, ldq, ldk, T, w_q, w_k, positions, phases, H, Hk, d, rot, pairs, norm, eps};
    const kda::HeadOut g{const_cast<void *>(dq_out), const_cast<void *>(dk_out), lddq_out, lddk_out}, dx{dq, dk, lddq, lddk};
    if (const int rc = head_in_ok(in, type, pairs, norm != 0)) return rc;
    if ((dw_q && !w_q) || (dw_k && !w_k) || !floats_ok_or_null(dw_q) || !floats_ok_or_null(dw_k)) return KDA_ERR_INVALID_ARG;
    if (T > 0 && (!head_rows_ok(in, type, g) || !head_rows_ok(in, type, dx))) return KDA_ERR_INVALID_ARG;
    if (dw_q || dw_k) {
        if (!ws || !aligned16(ws)) return KDA_ERR_INVALID_ARG;
        if (ws_bytes < kda::head_workspace_bytes(d)) return KDA_ERR_WORKSPACE;
    }
    return cuda_status(kda::launch_head_backward(in, type, g, dx, dw_q, dw_k, ws, static_cast<cudaStream_t>(stream)));
}

namespace {

// Rows on 16 bytes: what the copies of the attention's tiles take.
bool rows16_ok(const void *p, int64_t ld, int64_t width) { return p && aligned16(p) && ld >= width && ld % 8 == 0; }

bool map_stride_ok(int64_t ld) { return ld < (int64_t(1) << 39); }

int window_shape_ok(const kda::WindowIn &in, int32_t type)
{
    if (in.H < 1 || in.Hk < 1 || in.H % in.Hk || in.d < 1 || !kda::elem_bytes(type) || in.W < 1 || in.S < 0) return KDA_ERR_INVALID_ARG;
    const float c = in.scale * 1.44269504088896340736f;
    if (!(c > 0.f) || !std::isnormal(c)) return KDA_ERR_INVALID_ARG;
    if (type == KDA_TYPE_F32 || (in.d != 64 && in.d != 128) || in.S > KDA_WINDOW_MAX_SINKS) return KDA_ERR_UNSUPPORTED;
    if (in.H > INT32_MAX / in.d) return KDA_ERR_UNSUPPORTED;      // a token's channels are counted in 32 bits
    return KDA_OK;
}

// What the forward and the backward check of the arguments they share.
int window_in_ok(const int32_t *plan, const int32_t *plan_dev, const kda::WindowIn &in, int32_t type)
{
    if (!plan_ok(plan) || !plan_dev) return KDA_ERR_INVALID_ARG;
    if (const int rc = window_shape_ok(in, type)) return rc;
    const int64_t w = static_cast<int64_t>(in.H) * in.d, wk = static_cast<int64_t>(in.Hk) * in.d;
    if (!rows16_ok(in.q, in.ldq, w) || !rows16_ok(in.k, in.ldk, wk) || !rows16_ok(in.v, in.ldv, wk)) return KDA_ERR_INVALID_ARG;
    if (!kda::window_sizes_ok(plan[KDA_PH_T], plan[KDA_PH_N], in.H)) return KDA_ERR_UNSUPPORTED;
    // tensor maps hold strides below 2^40 bytes
    if (!map_stride_ok(in.ldq) || !map_stride_ok(in.ldk) || !map_stride_ok(in.ldv)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace

extern "C" int kda_window_attention_forward(const int32_t *plan, const int32_t *plan_dev, int32_t H, int32_t Hk, int32_t d, int32_t type,
                                            const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                                            float scale, int32_t window, int32_t sinks, void *o, int64_t ldo, float *lse, void *stream)
{
    const kda::WindowIn in{q, k, v, ldq, ldk, ldv, H, Hk, d, window, sinks, scale};
    if (const int rc = window_in_ok(plan, plan_dev, in, type)) return rc;
    if (!rows16_ok(o, ldo, static_cast<int64_t>(H) * d) || !floats_ok_or_null(lse)) return KDA_ERR_INVALID_ARG;
    return cuda_status(kda::launch_window_forward(plan, plan_dev, type, in, o, ldo, lse, static_cast<cudaStream_t>(stream)));
}

namespace {

// A ring cache's rows are counted in 32 bits, up to two rounds of a CTA's warps behind the last one.
bool cache_ok(const void *k, const void *v, int32_t window, int32_t sinks)
{
    return k && v && aligned16(k) && aligned16(v) && window <= INT32_MAX - 512 - sinks;
}

}  // namespace

extern "C" int kda_window_cache_fill(const int32_t *plan, const int32_t *plan_dev, int32_t Hk, int32_t d, int32_t type, const int32_t *slots,
                                     int32_t num_slots, const void *k, int64_t ldk, const void *v, int64_t ldv, int32_t window,
                                     int32_t sinks, void *cache_k, void *cache_v, void *stream)
{
    const kda::WindowIn shape{nullptr, k, v, 0, ldk, ldv, Hk, Hk, d, window, sinks, 1.f};
    if (!plan_ok(plan) || !plan_dev) return KDA_ERR_INVALID_ARG;
    if (const int rc = window_shape_ok(shape, type)) return rc;
    const int64_t wk = static_cast<int64_t>(Hk) * d;
    if (num_slots < 0 || (!slots && plan[KDA_PH_N] > num_slots) || (reinterpret_cast<uintptr_t>(slots) & 3u)) return KDA_ERR_INVALID_ARG;
    if (!rows16_ok(k, ldk, wk) || !rows16_ok(v, ldv, wk) || !cache_ok(cache_k, cache_v, window, sinks)) return KDA_ERR_INVALID_ARG;
    if (wk > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    const kda::FillIn in{k, v, ldk, ldv, slots, num_slots, Hk, d, window, sinks};
    return cuda_status(kda::launch_window_fill(plan, plan_dev, in, cache_k, cache_v, static_cast<cudaStream_t>(stream)));
}

extern "C" int kda_window_attention_step(int32_t B, int32_t H, int32_t Hk, int32_t d, int32_t type, const int32_t *slots, int32_t num_slots,
                                         const int32_t *lengths, const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v,
                                         int64_t ldv, float scale, int32_t window, int32_t sinks, void *cache_k, void *cache_v, void *o,
                                         int64_t ldo, void *stream)
{
    const kda::WindowIn shape{q, k, v, ldq, ldk, ldv, H, Hk, d, window, sinks, scale};
    if (B < 0 || num_slots < 0 || (!slots && B > num_slots)) return KDA_ERR_INVALID_ARG;
    if (const int rc = window_shape_ok(shape, type)) return rc;
    if (B == 0) return KDA_OK;
    const int64_t w = static_cast<int64_t>(H) * d, wk = static_cast<int64_t>(Hk) * d;
    if ((reinterpret_cast<uintptr_t>(slots) & 3u) || !lengths || (reinterpret_cast<uintptr_t>(lengths) & 3u)) return KDA_ERR_INVALID_ARG;
    if (!rows16_ok(q, ldq, w) || !rows16_ok(k, ldk, wk) || !rows16_ok(v, ldv, wk) || !rows16_ok(o, ldo, w) ||
        !cache_ok(cache_k, cache_v, window, sinks))
        return KDA_ERR_INVALID_ARG;
    const int64_t blocks = (H / Hk + 7) / 8;
    if (static_cast<int64_t>(B) * Hk > INT32_MAX / (8 * blocks)) return KDA_ERR_UNSUPPORTED;
    const kda::StepIn in{q, k, v, ldq, ldk, ldv, slots, lengths, B, num_slots, H, Hk, d, window, sinks, scale};
    return cuda_status(kda::launch_window_step(type, in, cache_k, cache_v, o, ldo, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t kda_window_attention_workspace_bytes(const int32_t *plan, int32_t H, int32_t Hk, int32_t d, int32_t window, int32_t sinks)
{
    const kda::WindowIn shape{nullptr, nullptr, nullptr, 0, 0, 0, H, Hk, d, window, sinks, 1.f};
    if (!plan_ok(plan) || window_shape_ok(shape, KDA_TYPE_BF16) != KDA_OK) return 0;
    return kda::window_workspace_bytes(plan[KDA_PH_T], plan[KDA_PH_N], H, Hk, d, window, sinks);
}

extern "C" int kda_window_attention_backward(const int32_t *plan, const int32_t *plan_dev, int32_t H, int32_t Hk, int32_t d, int32_t type,
                                             const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv, float scale,
                                             int32_t window, int32_t sinks, const void *o, int64_t ldo, const float *lse, const void *d_o,
                                             int64_t lddo, void *dq, int64_t lddq, void *dk, int64_t lddk, void *dv, int64_t lddv, void *ws,
                                             size_t ws_bytes, void *stream)
{
    const kda::WindowIn in{q, k, v, ldq, ldk, ldv, H, Hk, d, window, sinks, scale};
    const kda::WindowGrads g{o, d_o, ldo, lddo, lse, dq, dk, dv, lddq, lddk, lddv};
    if (const int rc = window_in_ok(plan, plan_dev, in, type)) return rc;
    const int64_t w = static_cast<int64_t>(H) * d, wk = static_cast<int64_t>(Hk) * d;
    if (!rows16_ok(o, ldo, w) || !rows16_ok(d_o, lddo, w) || !lse || !floats_ok_or_null(lse)) return KDA_ERR_INVALID_ARG;
    if (!rows16_ok(dq, lddq, w) || !rows16_ok(dk, lddk, wk) || !rows16_ok(dv, lddv, wk) || !ws || !aligned16(ws)) return KDA_ERR_INVALID_ARG;
    if (!map_stride_ok(lddo)) return KDA_ERR_UNSUPPORTED;
    if (ws_bytes < kda::window_workspace_bytes(plan[KDA_PH_T], plan[KDA_PH_N], H, Hk, d, window, sinks)) return KDA_ERR_WORKSPACE;
    return cuda_status(kda::launch_window_backward(plan, plan_dev, type, in, g, ws, static_cast<cudaStream_t>(stream)));
}
