// operators.cu -- host side of the operators beside the layer: routing from given logits,
// MXFP4 rows and expert products, and the weighted combine (include/ds4moe.h).
//
// The stateless calls launch on the caller's current device and stream and keep nothing; the
// ds4moe_mxfp4 handle holds the packed matrices of one projection of E experts on one device.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>
#include <string>

#include "../../include/ds4moe.h"
#include "combine.cuh"
#include "mxfp4.cuh"
#include "mxfp4_product.cuh"
#include "scored_router.cuh"

using namespace ds4;

struct ds4moe_mxfp4 {
    int device = 0;
    ds4moe_mxfp4_config cfg{};
    int num_sms = 148;
    cudaStream_t last_stream = nullptr;
    bool loaded = false;
    std::string err;
    uint8_t *packed = nullptr;
    size_t expert_bytes = 0;
    int *status = nullptr;
};

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
bool injected(const char *what) {
    const char *v = getenv("DS4MOE_FAULT");
    return v && strcmp(v, what) == 0;
}
bool float_type(int t) { return t == DS4MOE_F32 || t == DS4MOE_BF16 || t == DS4MOE_F16; }
size_t size_of(int t) { return t == DS4MOE_F32 ? 4 : 2; }

ds4moe_status fail(ds4moe_mxfp4 *h, ds4moe_status st, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    h->err = buf;
    return st;
}

#define CK(h, call)                                                                                          \
    do {                                                                                                     \
        cudaError_t e_ = (call);                                                                             \
        if (e_ != cudaSuccess)                                                                               \
            return fail((h), e_ == cudaErrorMemoryAllocation ? DS4MOE_ENOMEM : DS4MOE_ECUDA, "%s: %s (%s:%d)", \
                        #call, cudaGetErrorString(e_), __FILE__, __LINE__);                                  \
    } while (0)

// The handle's device for the length of a call; the caller's current device again after it.
struct OnDevice {
    int before = -1;
    cudaError_t err;
    explicit OnDevice(int device) {
        err = cudaGetDevice(&before);
        if (err == cudaSuccess && before != device) err = cudaSetDevice(device);
        else if (err == cudaSuccess) before = -1;
    }
    ~OnDevice() {
        if (before >= 0) cudaSetDevice(before);
    }
};

bool aligned32(const void *p) { return ((uintptr_t)p & 31u) == 0; }

// CTAs of 128 threads: an item a thread where there are few, up to `most` where there are many
// (a row's index arithmetic and indexes are then shared by its items).
RowSplit split_rows(int64_t rows, int items, int most) {
    int each = (int)std::min<int64_t>(std::max<int64_t>(rows * items / (148 * 2048), 1), most);
    RowSplit s{items, (items + 128 * each - 1) / (128 * each), 0};
    if (rows * s.segments > INT32_MAX) s.segments = 1;
    s.per = ((items + s.segments - 1) / s.segments + 1) & ~1;
    return s;
}
// A launch that may begin before the kernel ahead of it in the stream has ended; every kernel
// here waits for that end itself.
template <class... P, class... A>
cudaError_t launch_ahead(void (*kernel)(P...), int grid, int block, size_t smem, cudaStream_t st, A &&...args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(grid);
    lc.blockDim = dim3(block);
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    lc.attrs = at;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, static_cast<P>(args)...);
}
ds4moe_status launched(cudaError_t e) {
    if (e != cudaSuccess) cudaGetLastError();   // the next call's launch does not report it
    return e == cudaSuccess ? DS4MOE_OK : DS4MOE_ECUDA;
}
int blocks_for(int64_t threads) { return (int)std::min<int64_t>((threads + 255) / 256, 148 * 64); }

// ------------------------------------------------------------------ routing from logits
bool router_ok(const ds4moe_router *r) {
    return r && r->n_experts >= 1 && r->n_experts <= SR_MAX_EXPERTS && r->top_k >= 1 && r->top_k <= SR_MAX_TOPK &&
           r->score >= DS4MOE_SCORE_SOFTMAX && r->score <= DS4MOE_SCORE_SQRT_SOFTPLUS && r->n_groups >= 1 &&
           r->n_groups <= SR_MAX_GROUPS && r->n_experts % r->n_groups == 0 && r->topk_groups >= 1 &&
           r->topk_groups <= r->n_groups && r->top_k <= r->n_experts / r->n_groups * r->topk_groups &&
           r->group_score >= DS4MOE_GROUP_MAX && r->group_score <= DS4MOE_GROUP_TOP2 &&
           (r->renormalise == 0 || r->renormalise == 1) && r->scale - r->scale == 0.0f;
}
// Tokens a block: up to four blocks an SM where there are tokens for it (three are resident at once).
int route_block(int T) {
    int TB = T <= 64 ? 64 : SR_MIN_BLOCK;
    while (TB < SR_MAX_BLOCK && T / TB > 592) TB *= 2;
    return TB;
}
// Counts of every block, the totals, and the blocks' masks.
size_t route_workspace(const ds4moe_router *r, int T) {
    const int TB = route_block(T);
    const size_t NB = ((size_t)T + TB - 1) / TB, pitch = (r->n_experts + 3) / 4 * 4;
    return NB <= 1 ? 0 : ((NB + 1) * pitch + NB * (TB / 32) * r->n_experts) * 4;
}

// ------------------------------------------------------------------ MXFP4 products
// Tensor map of the rows' codes, [rows][K / 2] bytes, with boxes of 128 bytes (one K step) x
// box_rows and the 128-byte swizzle.
bool row_map(CUtensorMap *m, const void *codes, int rows, int K, int box_rows) {
    static const PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
        cudaDriverEntryPointQueryResult q;
        void *f = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)K / 2, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)K / 2};
    cuuint32_t box[2] = {MX_TK / 2, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(codes), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class C>
ds4moe_status run_product(ds4moe_mxfp4 *h, const MxArgs &a, cudaStream_t st) {
    const int64_t row_tiles = a.rows / C::NT + a.E, m_tiles = ((int64_t)a.N * (a.gated ? 2 : 1) + MX_TM - 1) / MX_TM;
    if (row_tiles * m_tiles + h->num_sms > INT32_MAX) return fail(h, DS4MOE_EINVAL, "too many tiles for one call");
    CUtensorMap tm[3];
    const int boxes[3] = {C::NT, C::BOX0, C::BOX1};
    for (int i = 0; i < 3; ++i)
        if (!row_map(&tm[i], a.a_codes, a.rows, a.K, boxes[i])) return fail(h, DS4MOE_ECUDA, "tensor map of the rows");
    CK(h, launch_ahead(mxfp4_product_kernel<C>, h->num_sms, MX_THREADS, C::SMEM, st, tm[0], tm[1], tm[2], a));
    return DS4MOE_OK;
}
// Tiles of up to 32 rows, two steps a stage, where experts have few rows; of up to 192, one step a
// stage, elsewhere.  Measured (us, 32 / 192 rows a tile; 64 experts, 4096 x 4096, by the mean rows
// an expert): 8 rows 106 / 106, 24 106 / 107, 32 106 / 108, 40 115 / 109; one row each of 8 of 256
// experts (gated, 2048 x 4096) 17.6 / 22.3, 40 rows of 32 experts 21.9 / 26.0, one expert with 16
// rows 9.2 / 10.4 (all before kernels were launched ahead; now 24, 32 and 40 rows each 89, 92 and
// 93).  These loads are even.  The rule sees the mean over all experts, idle ones included, so many
// rows of few among many experts get narrow tiles, and their weights come from L2 once for each 32
// rows: 4096 rows of 20 of 256 experts take 101 us, of 20 of 20 experts (wide tiles) 55.  Two steps
// a stage (half the barriers) took one row of one expert from 10.4 to 8.9 us; with wide tiles they
// leave three stages of 128 rows or two of 192: 94 and 91 against 90 us at 8191 x 4096 x 4096.
template <bool GATED>
using FewRows = MxCfg<32, 16, 8, 4, 2, GATED>;
template <bool GATED>
using ManyRows = MxCfg<192, 128, 64, 5, 1, GATED>;
template <bool GATED>
ds4moe_status pick_product(ds4moe_mxfp4 *h, const MxArgs &a, cudaStream_t st) {
    if (a.rows <= 24ll * std::min(a.rows, a.E)) return run_product<FewRows<GATED>>(h, a, st);
    return run_product<ManyRows<GATED>>(h, a, st);
}
// The product kernels' shared memory on the current device (once, when a handle is made).
template <class C>
cudaError_t allow_smem() {
    return cudaFuncSetAttribute(mxfp4_product_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
}
template <bool GATED>
cudaError_t prepare_product() {
    const cudaError_t e = allow_smem<FewRows<GATED>>();
    return e == cudaSuccess ? allow_smem<ManyRows<GATED>>() : e;
}

}  // namespace

extern "C" {

size_t ds4moe_route_logits_workspace(const ds4moe_router *r, int32_t T) {
    return router_ok(r) && T > 0 ? route_workspace(r, T) : 0;
}

ds4moe_status ds4moe_route_logits(const ds4moe_router *r, const void *logits_dev, int32_t logits_type, int64_t ld,
                                  int32_t T, const float *bias_dev, int32_t *topk_idx_dev, float *topk_w_dev,
                                  int32_t *expert_offsets_dev, int32_t *sorted_token_dev, int32_t *sorted_slot_dev,
                                  int32_t *inv_pos_dev, void *workspace_dev, size_t workspace_bytes, void *cuda_stream) {
    if (!router_ok(r) || T < 0 || !float_type(logits_type) || ld < r->n_experts) return DS4MOE_EINVAL;
    if ((int64_t)T * r->top_k > INT32_MAX) return DS4MOE_EINVAL;
    if (injected("launch")) return DS4MOE_ECUDA;
    const bool permute = expert_offsets_dev || sorted_token_dev || sorted_slot_dev || inv_pos_dev;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
    if (T == 0) {
        // no pair: the offsets are all zero
        if (expert_offsets_dev &&
            cudaMemsetAsync(expert_offsets_dev, 0, (r->n_experts + 1) * sizeof(int32_t), st) != cudaSuccess)
            return DS4MOE_ECUDA;
        return DS4MOE_OK;
    }
    if (!logits_dev || (uintptr_t)logits_dev % size_of(logits_type) || !topk_idx_dev || !topk_w_dev) return DS4MOE_EINVAL;
    ScoredArgs a{};
    a.E = r->n_experts; a.k = r->top_k; a.score = r->score; a.G = r->n_groups; a.topk_groups = r->topk_groups;
    a.top2 = r->group_score == DS4MOE_GROUP_TOP2; a.renormalise = r->renormalise; a.scale = r->scale;
    a.logits = logits_dev; a.type = logits_type; a.ld = ld;
    a.T = T; a.TB = route_block(T); a.NB = (int)(((int64_t)T + a.TB - 1) / a.TB);
    a.bias = bias_dev;
    a.topk_idx = topk_idx_dev; a.topk_w = topk_w_dev;
    a.offsets = expert_offsets_dev; a.sorted_token = sorted_token_dev; a.sorted_slot = sorted_slot_dev; a.inv_pos = inv_pos_dev;
    if (permute && a.NB > 1) {
        if (!workspace_dev || !aligned16(workspace_dev) || workspace_bytes < route_workspace(r, T)) return DS4MOE_EINVAL;
        a.cnt = static_cast<int *>(workspace_dev);
        a.pitch = (a.E + 3) / 4 * 4;
        a.total = a.cnt + (size_t)a.NB * a.pitch;
        a.mask = reinterpret_cast<uint32_t *>(a.total + a.pitch);
    }
    // one block, or fewer than the SMs: more warps a block, two tokens a warp
    const bool few = a.NB <= 148;
    const int warps = few ? std::min(std::max(std::min(T, a.TB) / 2, SR_WARPS), SR_MAX_WARPS) : SR_WARPS;
    cudaError_t err = cudaSuccess;
    auto launch = [&](auto many, auto lone, int npl) {
        auto kernel = few ? lone : many;
        const size_t smem = (a.G > 1 ? (size_t)warps * 32 * npl * 8 : 0) + (size_t)a.E * (a.TB / 32 + 1) * 4;
        // The leave is the kernel's, for every thread of the process, so it is always for the most
        // that any call takes: it never falls below what another thread is about to launch with.
        if (smem > SR_PLAIN_SMEM)
            err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SR_MOST_SMEM);
        if (err == cudaSuccess) err = launch_ahead(kernel, a.NB, 32 * warps, smem, st, a);
    };
    static_assert(SR_MOST_SMEM + 4096 <= 227 * 1024, "shared memory per CTA");
    auto typed = [&](auto v) {
        using E = decltype(v);
        // a lane's logits as one aligned piece: the common counts of experts
        const bool vec = (uintptr_t)logits_dev % 16 == 0 && ld * sizeof(E) % 16 == 0;
        if (a.E <= 32) launch(scored_topk_kernel<1, E, false, false>, scored_topk_kernel<1, E, false, true>, 1);
        else if (a.E <= 64) launch(scored_topk_kernel<2, E, false, false>, scored_topk_kernel<2, E, false, true>, 2);
        else if (a.E == 128 && vec) launch(scored_topk_kernel<4, E, true, false>, scored_topk_kernel<4, E, true, true>, 4);
        else if (a.E <= 128) launch(scored_topk_kernel<4, E, false, false>, scored_topk_kernel<4, E, false, true>, 4);
        else if (a.E == 256 && vec) launch(scored_topk_kernel<8, E, true, false>, scored_topk_kernel<8, E, true, true>, 8);
        else if (a.E <= 256) launch(scored_topk_kernel<8, E, false, false>, scored_topk_kernel<8, E, false, true>, 8);
        else if (a.E == 512 && vec) launch(scored_topk_kernel<16, E, true, false>, scored_topk_kernel<16, E, true, true>, 16);
        else launch(scored_topk_kernel<16, E, false, false>, scored_topk_kernel<16, E, false, true>, 16);
    };
    if (logits_type == DS4MOE_F32) typed(float{});
    else if (logits_type == DS4MOE_BF16) typed(__nv_bfloat16{});
    else typed(__half{});
    if (err != cudaSuccess || !permute || a.NB == 1) return launched(err);
    const int scanned = a.NB > SR_DIRECT;
    if (scanned && (err = launch_ahead(scored_scan_kernel, (a.E + 31) / 32, 1024, 0, st, a)) != cudaSuccess) return launched(err);
    const size_t sums = scanned ? 0 : (size_t)2 * (SR_PERMUTE_THREADS / (a.pitch / 4)) * a.pitch;
    static_assert((2 * SR_MAX_EXPERTS + 2 * 4 * SR_PERMUTE_THREADS + SR_MAX_EXPERTS * (SR_MAX_BLOCK / 32)) * 4 <= 48 * 1024,
                  "shared memory of the permutation");
    return launched(launch_ahead(scored_permute_kernel, a.NB, SR_PERMUTE_THREADS,
                                 (2 * a.pitch + sums + (size_t)a.E * (a.TB / 32)) * 4, st, a, scanned));
}

ds4moe_status ds4moe_mxfp4_quantize(const void *x_dev, int32_t x_type, int64_t ld, int32_t rows, int32_t K,
                                    const int32_t *inv_pos_dev, int32_t top_k, int32_t out_rows, uint8_t *codes_dev,
                                    uint8_t *scales_dev, void *cuda_stream) {
    if (rows < 0 || out_rows < 0 || K <= 0 || K % MX_BLOCK || !float_type(x_type) || ld < K) return DS4MOE_EINVAL;
    if (inv_pos_dev ? top_k < 1 || top_k > SR_MAX_TOPK : out_rows < rows) return DS4MOE_EINVAL;
    if (injected("launch")) return DS4MOE_ECUDA;
    if (rows == 0 || out_rows == 0) return DS4MOE_OK;
    if (!x_dev || (uintptr_t)x_dev % size_of(x_type) || !codes_dev || !aligned16(codes_dev) || !scales_dev) return DS4MOE_EINVAL;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
    const bool vec = aligned32(x_dev) && ld * size_of(x_type) % 32 == 0;
    const RowSplit split = split_rows(rows, K / 16, 4);
    cudaError_t err = cudaSuccess;
    auto go = [&](auto kernel, auto *x) {
        err = launch_ahead(kernel, rows * split.segments, 128, 0, st, x, ld, K, split, inv_pos_dev, top_k, out_rows, codes_dev,
                           scales_dev);
    };
    if (x_type == DS4MOE_F32) {
        auto *x = static_cast<const float *>(x_dev);
        if (vec) go(mxfp4_quantize_kernel<float, true>, x); else go(mxfp4_quantize_kernel<float, false>, x);
    } else if (x_type == DS4MOE_BF16) {
        auto *x = static_cast<const __nv_bfloat16 *>(x_dev);
        if (vec) go(mxfp4_quantize_kernel<__nv_bfloat16, true>, x); else go(mxfp4_quantize_kernel<__nv_bfloat16, false>, x);
    } else {
        auto *x = static_cast<const __half *>(x_dev);
        if (vec) go(mxfp4_quantize_kernel<__half, true>, x); else go(mxfp4_quantize_kernel<__half, false>, x);
    }
    return launched(err);
}

ds4moe_status ds4moe_mxfp4_dequantize(const uint8_t *codes_dev, const uint8_t *scales_dev, int32_t rows, int32_t K,
                                      void *out_dev, int32_t out_type, int64_t ld, void *cuda_stream) {
    if (rows < 0 || K <= 0 || K % MX_BLOCK || !float_type(out_type) || ld < K) return DS4MOE_EINVAL;
    if (injected("launch")) return DS4MOE_ECUDA;
    if (rows == 0) return DS4MOE_OK;
    if (!codes_dev || !aligned16(codes_dev) || !scales_dev || !out_dev || (uintptr_t)out_dev % size_of(out_type)) return DS4MOE_EINVAL;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
    const bool vec = aligned32(out_dev) && ld * size_of(out_type) % 32 == 0;
    const RowSplit split = split_rows(rows, K / 16, 4);
    cudaError_t err = cudaSuccess;
    auto go = [&](auto kernel, auto *out) {
        err = launch_ahead(kernel, rows * split.segments, 128, 0, st, codes_dev, scales_dev, K, split, out, ld);
    };
    if (out_type == DS4MOE_F32) {
        auto *o = static_cast<float *>(out_dev);
        if (vec) go(mxfp4_dequantize_kernel<float, true>, o); else go(mxfp4_dequantize_kernel<float, false>, o);
    } else if (out_type == DS4MOE_BF16) {
        auto *o = static_cast<__nv_bfloat16 *>(out_dev);
        if (vec) go(mxfp4_dequantize_kernel<__nv_bfloat16, true>, o); else go(mxfp4_dequantize_kernel<__nv_bfloat16, false>, o);
    } else {
        auto *o = static_cast<__half *>(out_dev);
        if (vec) go(mxfp4_dequantize_kernel<__half, true>, o); else go(mxfp4_dequantize_kernel<__half, false>, o);
    }
    return launched(err);
}

ds4moe_status ds4moe_combine(const void *o_dev, int32_t o_type, int64_t o_rows, int32_t T, int32_t top_k, int32_t H,
                             const int32_t *inv_pos_dev, const float *topk_w_dev, const void *add_dev, int32_t add_type,
                             void *y_dev, int32_t y_type, void *cuda_stream) {
    if (T < 0 || H <= 0 || top_k < 1 || top_k > SR_MAX_TOPK || o_rows < 0 || !float_type(o_type) || !float_type(y_type) ||
        (add_dev && !float_type(add_type)))
        return DS4MOE_EINVAL;
    if (injected("launch")) return DS4MOE_ECUDA;
    if (T == 0) return DS4MOE_OK;
    if ((o_rows > 0 && !o_dev) || !inv_pos_dev || !topk_w_dev || !y_dev) return DS4MOE_EINVAL;
    if ((uintptr_t)o_dev % size_of(o_type) || (uintptr_t)y_dev % size_of(y_type) ||
        (add_dev && (uintptr_t)add_dev % size_of(add_type)))
        return DS4MOE_EINVAL;
    CombineArgs a{o_dev, o_rows, T, top_k, H, inv_pos_dev, topk_w_dev, add_dev, add_type, y_dev};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
    const int64_t per = 32 / size_of(o_type);   // columns of a 32-byte piece
    const bool vec = H % per == 0 && aligned32(o_dev) && H * size_of(o_type) % 32 == 0 && aligned32(y_dev) &&
                     H * size_of(y_type) % 16 == 0 && (!add_dev || aligned16(add_dev));
    const int64_t piece = 16 / size_of(o_type);   // in 64 bits: H goes up to 2^31 - 1
    const RowSplit split = split_rows(T, (int)(vec ? H / per : (H + piece - 1) / piece), 4);
    cudaError_t err = cudaSuccess;
    auto go = [&](auto kernel) { err = launch_ahead(kernel, T * split.segments, 128, 0, st, a, split); };
    auto with = [&](auto o) {
        using TO = decltype(o);
        auto to = [&](auto y) {
            using TY = decltype(y);
            if (vec) go(combine_kernel<TO, TY>);
            else go(combine_shifted_kernel<TO, TY>);
        };
        if (y_type == DS4MOE_F32) to(float{});
        else if (y_type == DS4MOE_BF16) to(__nv_bfloat16{});
        else to(__half{});
    };
    if (o_type == DS4MOE_F32) with(float{});
    else if (o_type == DS4MOE_BF16) with(__nv_bfloat16{});
    else with(__half{});
    return launched(err);
}

const char *ds4moe_mxfp4_last_error(const ds4moe_mxfp4 *h) { return h ? h->err.c_str() : "null handle"; }

ds4moe_status ds4moe_mxfp4_create(const ds4moe_mxfp4_config *cfg, int cuda_device, ds4moe_mxfp4 **out) {
    if (!cfg || !out) return DS4MOE_EINVAL;
    *out = nullptr;
    if (cfg->n_experts < 1 || cfg->n_experts > SR_MAX_EXPERTS || cfg->n_out < 1 || cfg->n_out > 65536 || cfg->n_in < MX_BLOCK ||
        cfg->n_in > 65536 || cfg->n_in % MX_BLOCK || (cfg->gated != 0 && cfg->gated != 1))
        return DS4MOE_EINVAL;
    if (injected("alloc")) return DS4MOE_ENOMEM;
    ds4moe_mxfp4 *h = new (std::nothrow) ds4moe_mxfp4();
    if (!h) return DS4MOE_ENOMEM;
    h->cfg = *cfg;
    h->device = cuda_device;
    h->expert_bytes = mx_expert_bytes(cfg->n_out * (cfg->gated ? 2 : 1), cfg->n_in);
    OnDevice on(cuda_device);
    cudaError_t e = on.err;
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, cuda_device);
    if (e == cudaSuccess) e = cfg->gated ? prepare_product<true>() : prepare_product<false>();
    if (e == cudaSuccess) e = cudaMalloc(&h->packed, h->expert_bytes * cfg->n_experts);
    if (e == cudaSuccess) e = cudaMalloc(&h->status, 256);
    if (e == cudaSuccess) e = cudaMemset(h->status, 0, 256);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        cudaGetLastError();
        if (h->packed) cudaFree(h->packed);
        if (h->status) cudaFree(h->status);
        delete h;
        return e == cudaErrorMemoryAllocation ? DS4MOE_ENOMEM : DS4MOE_ECUDA;
    }
    *out = h;
    return DS4MOE_OK;
}

void ds4moe_mxfp4_destroy(ds4moe_mxfp4 *h) {
    if (!h) return;
    OnDevice on(h->device);
    cudaDeviceSynchronize();
    cudaFree(h->packed);
    cudaFree(h->status);
    delete h;
}

ds4moe_status ds4moe_mxfp4_load(ds4moe_mxfp4 *h, const uint8_t *codes_dev, const uint8_t *scales_dev,
                                const uint8_t *up_codes_dev, const uint8_t *up_scales_dev, void *cuda_stream) {
    if (!h) return DS4MOE_EINVAL;
    const ds4moe_mxfp4_config &g = h->cfg;
    if (!codes_dev || !scales_dev || (g.gated && (!up_codes_dev || !up_scales_dev)))
        return fail(h, DS4MOE_EINVAL, "null weight pointer");
    if (!g.gated && (up_codes_dev || up_scales_dev)) return fail(h, DS4MOE_EINVAL, "a second matrix for a handle that is not gated");
    if (!aligned16(codes_dev) || (g.gated && !aligned16(up_codes_dev))) return fail(h, DS4MOE_EINVAL, "codes must be 16-byte aligned");
    if (injected("h2d")) return fail(h, DS4MOE_ECUDA, "weight packing failed (injected: DS4MOE_FAULT=h2d)");
    OnDevice on(h->device);
    CK(h, on.err);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
    const int64_t n = (int64_t)g.n_experts * (h->expert_bytes / MX_TILE_BYTES) * MX_TM * (MX_TK / MX_BLOCK);
    CK(h, launch_ahead(mxfp4_pack_kernel, blocks_for(n), 256, 0, st, codes_dev, scales_dev, g.gated ? up_codes_dev : nullptr,
                       g.gated ? up_scales_dev : nullptr, g.n_experts, g.n_out, g.n_in, h->packed));
    h->loaded = true;
    h->last_stream = st;
    return DS4MOE_OK;
}

ds4moe_status ds4moe_mxfp4_product(ds4moe_mxfp4 *h, const uint8_t *a_codes_dev, const uint8_t *a_scales_dev, int32_t rows,
                                   const int32_t *expert_offsets_dev, void *out_dev, int32_t out_type, int64_t ld,
                                   uint8_t *out_scales_dev, void *cuda_stream) {
    if (!h) return DS4MOE_EINVAL;
    const ds4moe_mxfp4_config &g = h->cfg;
    if (injected("launch")) return fail(h, DS4MOE_ECUDA, "kernel launch failed (injected: DS4MOE_FAULT=launch)");
    if (!h->loaded) return fail(h, DS4MOE_ESTATE, "no weights loaded");
    if (rows < 0 || rows > MX_MOST_ROWS) return fail(h, DS4MOE_EINVAL, "rows=%d is not in 0 .. %d", rows, MX_MOST_ROWS);
    if (!float_type(out_type) && out_type != DS4MOE_MXFP4) return fail(h, DS4MOE_EINVAL, "unknown output type %d", out_type);
    if (out_type == DS4MOE_MXFP4 ? g.n_out % MX_BLOCK != 0 || ld != g.n_out || !out_scales_dev : out_scales_dev != nullptr)
        return fail(h, DS4MOE_EINVAL, "an MXFP4 output needs n_out %% 32 == 0, ld == n_out and scales; the others take no scales");
    if (ld < g.n_out) return fail(h, DS4MOE_EINVAL, "ld is below n_out");
    if (!expert_offsets_dev && g.n_experts != 1) return fail(h, DS4MOE_EINVAL, "expert offsets are required");
    if (rows == 0) return DS4MOE_OK;
    if (!a_codes_dev || !a_scales_dev || !out_dev) return fail(h, DS4MOE_EINVAL, "null buffer");
    if (!aligned16(a_codes_dev)) return fail(h, DS4MOE_EINVAL, "codes must be 16-byte aligned");
    if ((uintptr_t)out_dev % (out_type == DS4MOE_MXFP4 ? 16 : size_of(out_type)))
        return fail(h, DS4MOE_EINVAL, "the output is not aligned to its elements (MXFP4: to 16 bytes)");
    OnDevice on(h->device);
    CK(h, on.err);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
    h->last_stream = st;
    MxArgs a{};
    a.w = h->packed; a.expert_bytes = h->expert_bytes;
    a.E = g.n_experts; a.N = g.n_out; a.K = g.n_in; a.gated = g.gated;
    a.a_codes = a_codes_dev; a.a_scales = a_scales_dev; a.rows = rows; a.offsets = expert_offsets_dev;
    a.out = out_dev; a.out_scales = out_scales_dev; a.out_type = out_type; a.ld = ld;
    a.status = h->status;
    return g.gated ? pick_product<true>(h, a, st) : pick_product<false>(h, a, st);
}

ds4moe_status ds4moe_mxfp4_sync_status(ds4moe_mxfp4 *h) {
    if (!h) return DS4MOE_EINVAL;
    OnDevice on(h->device);
    CK(h, on.err);
    CK(h, cudaStreamSynchronize(h->last_stream));
    int st = 0;
    CK(h, cudaMemcpy(&st, h->status, 4, cudaMemcpyDeviceToHost));
    if (st != 0) {
        CK(h, cudaMemset(h->status, 0, 4));
        return fail(h, (ds4moe_status)st, "device status %d", st);
    }
    return DS4MOE_OK;
}

}  // extern "C"
