// mxfp4_product.cuh -- products of MXFP4 rows, grouped by expert, with the experts' MXFP4 matrices.
#pragma once
#include "mxfp4.cuh"
#include "scan.cuh"
#include "tcgen.cuh"

namespace ds4 {

struct MxArgs {
    const uint8_t *w;          // packed matrices
    size_t expert_bytes;
    int E, N, K, gated;        // N outputs (a gated matrix has 2N packed rows)
    const uint8_t *a_codes, *a_scales;
    int rows;                  // rows of a
    const int *offsets;        // [E + 1], or null: one expert takes every row
    void *out;
    uint8_t *out_scales;       // MXFP4 output
    int out_type;
    int64_t ld;                // elements between output rows (MXFP4: packed, ld = N)
    int vec_out;               // 16-byte stores are aligned
    int *status;
};

// Rows [first, last) of expert e, clipped to the rows there are.
__device__ __forceinline__ void mx_group(const MxArgs &p, int e, int &first, int &last) {
    first = p.offsets ? min(max(p.offsets[e], 0), p.rows) : 0;
    last = p.offsets ? min(max(p.offsets[e + 1], first), p.rows) : p.rows;
}

// ------------------------------------------------------------------ tcgen05
// A persistent kernel, one CTA per SM, over tiles of 128 packed weight rows (the MMA's M) x up
// to NT rows of a (the MMA's N): each expert's rows are cut into equal tiles of at most NT, and
// the tiles that share weight rows follow one another, so the weights cross HBM once.  One
// K step is 256 inputs: a weight tile with its scales (one contiguous bulk copy), the rows'
// codes (TMA, 128-byte swizzle, only the boxes that hold rows of the tile) and the rows'
// scales, then four block-scaled MMAs of 64 inputs (kind::mxf4, E2M1 x E2M1 with an E8M0 scale
// per 32, exact products, fp32 accumulators in tensor memory).
//   warp 0     producer of weight tiles and row codes
//   warp 1     allocates tensor memory; copies the step's scales there (tcgen05.cp) and issues
//              the MMAs.  Every stage has its own scale columns, so a copy never meets an MMA
//              that still reads the columns' last contents
//   warp 2     rows' scales: plain loads (rows start anywhere, K / 32 is any number), laid out
//              in shared memory as the copy wants them
//   warps 4-7  epilogue: accumulators -> silu(g) * u -> shared memory -> rows of the output
// The accumulators are double buffered, so a tile's epilogue overlaps the next tile.
// Every wait is bounded, as in the layer's grouped GEMM: on a timeout the CTA records
// ETIMEOUT, waits for its own copies and MMAs, frees tensor memory and returns.
constexpr int MX_THREADS = 256;
constexpr int MX_CHUNK = 32;             // rows of a that pass through shared memory at a time

template <int NT_, int BOX_, int STAGES_, bool GATED_>
struct MxCfg {
    static constexpr int NT = NT_, BOX = BOX_, STAGES = STAGES_;
    static constexpr bool GATED = GATED_;
    static constexpr int SF_CHUNKS = (NT + 127) / 128;                 // 512-byte scale chunks of the rows per 128 inputs
    static constexpr int B_BYTES = (NT * 128 + 1023) / 1024 * 1024;
    static constexpr int SFB_BYTES = 2 * SF_CHUNKS * 512;
    // weight codes | weight scales | row scales | (to 1024) | row codes
    static constexpr int B_OFF = (MX_TILE_BYTES + SFB_BYTES + 1023) / 1024 * 1024;
    static constexpr int STAGE_BYTES = B_OFF + B_BYTES;
    static constexpr int SF_COLS = 8 + 8 * SF_CHUNKS;                  // tensor memory columns of a stage's scales
    static constexpr int COLS = 2 * NT + STAGES * SF_COLS;
    static constexpr int TMEM = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    static constexpr int F = GATED ? 64 : 128;                         // outputs of a tile
    static constexpr int PITCH = F + 4;                                // floats between rows of the epilogue buffer
    static constexpr int EPI_BYTES = MX_CHUNK * PITCH * 4;
    static constexpr int S_BYTES = (SR_MAX_EXPERTS + 1) * 4;
    static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + EPI_BYTES + 512 + S_BYTES;
    static_assert(COLS <= 512, "tensor memory");
    static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
    static_assert(NT % 16 == 0 && NT % BOX == 0 && BOX % 8 == 0, "row tiles");
};

// Instruction descriptor of kind::mxf4: E2M1 A and B (K-major), E8M0 scales, fp32 D, M = 128, N;
// sf: the first scale byte (0 or 2) of the columns' four that this MMA takes.
__device__ __forceinline__ uint32_t mxf4_idesc(int N, uint32_t sf) {
    return (sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | (1u << 27) | (sf << 29);
}
__device__ __forceinline__ void mx_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}
// 512 bytes of scales from shared memory to four columns, repeated in each quarter of the lanes.
__device__ __forceinline__ void mx_copy_scales(uint32_t tmem, uint32_t smem) {
    // no swizzle; 8-row groups of 16-byte rows 128 bytes apart
    const uint64_t d = (uint64_t)((smem & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(d) : "memory");
}

struct MxTile {
    int e, m, row0, n;   // expert, weight row tile, first row of a, rows
};

// Tile t: S[e] counts the row tiles of the experts before e.
__device__ __forceinline__ MxTile mx_tile(const MxArgs &p, const int *S, int64_t t, int MT, int NT) {
    const int u = (int)(t / MT);
    int lo = 0, hi = p.E;   // S[lo] <= u < S[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (S[mid] <= u) lo = mid; else hi = mid;
    }
    MxTile x;
    x.e = lo;
    const int s0 = S[lo], nt = S[lo + 1] - s0;
    const int64_t local = t - (int64_t)s0 * MT;
    x.m = (int)(local / nt);
    const int i = (int)(local - (int64_t)x.m * nt);
    int first, last;
    mx_group(p, lo, first, last);
    const int per = min(NT, ((last - first + nt - 1) / nt + 15) & ~15);
    x.row0 = first + i * per;
    x.n = min(per, last - x.row0);   // at least 1: nt tiles of per rows are needed
    return x;
}

// y (8 consecutive outputs of row r from output f) -> the output, plain types.
template <class T>
__device__ __forceinline__ void mx_store8(const MxArgs &p, size_t o, int f, const float (&y)[8], bool vec) {
    T *out = reinterpret_cast<T *>(p.out) + o;
    if (vec && f + 8 <= p.N) {
        store_row<T, 8, true>(out, y);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (f + j < p.N) out[j] = from_f32<T>(y[j]);
    }
}

template <class C>
__global__ void __launch_bounds__(MX_THREADS, 1) mxfp4_product_kernel(const __grid_constant__ CUtensorMap tm_a, MxArgs p) {
    extern __shared__ __align__(1024) uint8_t mx_smem_raw[];
    uint8_t *stages = mx_smem_raw + ((1024u - (smem_u32(mx_smem_raw) & 1023u)) & 1023u);
    float *epi = reinterpret_cast<float *>(stages + C::STAGES * C::STAGE_BYTES);
    uint64_t *bars = reinterpret_cast<uint64_t *>(reinterpret_cast<uint8_t *>(epi) + C::EPI_BYTES);
    uint64_t *full = bars;                       // [S] producer (with the bytes) and the scale warp
    uint64_t *empty = full + C::STAGES;          // [S] MMA commit
    uint64_t *acc_full = empty + C::STAGES;      // [2] MMA commit
    uint64_t *acc_empty = acc_full + 2;          // [2] 4 epilogue warps
    uint64_t *drain = acc_empty + 2;             // MMA commit at exit
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(drain + 2);
    int *part = reinterpret_cast<int *>(drain + 3);          // [8]
    int *S = reinterpret_cast<int *>(bars + 64);
    static_assert((2 * C::STAGES + 8) * 8 + 32 <= 512, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(full + s), 2);
            mbar_init(smem_u32(empty + s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(acc_full + b), 1);
            mbar_init(smem_u32(acc_empty + b), 4);
        }
        mbar_init(smem_u32(drain), 1);
        *abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)), "n"(C::TMEM)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    for (int e = threadIdx.x; e < p.E; e += MX_THREADS) {
        int first, last;
        mx_group(p, e, first, last);
        S[e] = (last - first + C::NT - 1) / C::NT;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const int units = block_scan(S, p.E, part);
    if (threadIdx.x == 0) S[p.E] = units;
    __syncthreads();

    const int packed_rows = C::GATED ? 2 * p.N : p.N;
    const int MT = (packed_rows + MX_TM - 1) / MX_TM, KT = (p.K + MX_TK - 1) / MX_TK;
    const int64_t tiles = (int64_t)units * MT;

    if (warp == 0) {
        // ------------------------------------------------------------------- producer
        uint32_t it = 0;
        bool ok = true;
        for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const MxTile x = mx_tile(p, S, t, MT, C::NT);
            const uint8_t *w = p.w + (size_t)x.e * p.expert_bytes + (size_t)x.m * KT * MX_TILE_BYTES;
            const int boxes = (x.n + C::BOX - 1) / C::BOX;
            for (int kt = 0; kt < KT; ++kt, ++it) {
                const uint32_t s = it % C::STAGES;
                if (!(ok = mbar_wait(smem_u32(empty + s), ((it / C::STAGES) & 1) ^ 1, abort, p.status))) break;
                if (elect_one()) {
                    const uint32_t st = smem_u32(stages + s * C::STAGE_BYTES), bar = smem_u32(full + s);
                    mbar_expect_tx(bar, (uint32_t)(MX_TILE_BYTES + boxes * C::BOX * 128));
                    bulk_g2s(st, w + (size_t)kt * MX_TILE_BYTES, MX_TILE_BYTES, bar);
                    for (int j = 0; j < boxes; ++j)
                        tma_load_2d(st + C::B_OFF + j * C::BOX * 128, &tm_a, kt * (MX_TK / 2), x.row0 + j * C::BOX, bar);
                }
                __syncwarp();
            }
        }
        if (!ok)   // no copy of this CTA may still be writing shared memory (a stage also waits for the scale warp)
            for (uint32_t i = it > C::STAGES ? it - C::STAGES : 0; i < it; ++i)
                mbar_drain(smem_u32(full + i % C::STAGES), (i / C::STAGES) & 1, p.status);
    } else if (warp == 1) {
        // ------------------------------------------------------------------------ MMA
        uint32_t it = 0, tc = 0;
        bool ok = true;
        for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++tc) {
            const MxTile x = mx_tile(p, S, t, MT, C::NT);
            const uint32_t b = tc & 1;
            if (!(ok = mbar_wait(smem_u32(acc_empty + b), ((tc >> 1) & 1) ^ 1, abort, p.status))) break;
            tc_fence_after();
            const int N = (x.n + 15) & ~15;
            const int chunks = (N + 127) >> 7;
            const uint32_t d = tmem + b * C::NT;
            for (int kt = 0; kt < KT; ++kt, ++it) {
                const uint32_t s = it % C::STAGES;
                if (!(ok = mbar_wait(smem_u32(full + s), (it / C::STAGES) & 1, abort, p.status))) break;
                tc_fence_after();
                const uint32_t st = smem_u32(stages + s * C::STAGE_BYTES);
                const uint32_t sfa = tmem + 2 * C::NT + s * C::SF_COLS, sfb = sfa + 8;
                const uint64_t ad = sw128_desc(st), bd = sw128_desc(st + C::B_OFF);
                const int steps = min(4, (p.K - kt * MX_TK + 63) >> 6);
                if (elect_one()) {
                    for (int g = 0; g < (steps + 1) / 2; ++g) {
                        mx_copy_scales(sfa + 4 * g, st + MX_CODE_BYTES + 512 * g);
                        for (int c = 0; c < chunks; ++c)
                            mx_copy_scales(sfb + 4 * (g * C::SF_CHUNKS + c), st + MX_TILE_BYTES + 512 * (g * C::SF_CHUNKS + c));
                    }
                    for (int kk = 0; kk < steps; ++kk)
                        mx_mma(d, ad + 2 * kk, bd + 2 * kk, mxf4_idesc(N, 2 * (kk & 1)), sfa + 4 * (kk >> 1),
                               sfb + 4 * C::SF_CHUNKS * (kk >> 1), (kt | kk) != 0);
                    tc_commit(smem_u32(empty + s));
                }
                __syncwarp();
            }
            if (ok && elect_one()) tc_commit(smem_u32(acc_full + b));
            __syncwarp();
        }
        if (elect_one()) tc_commit(smem_u32(drain));
        __syncwarp();
        mbar_drain(smem_u32(drain), 0, p.status);
    } else if (warp == 2) {
        // ----------------------------------------------------------------- row scales
        // Chunk (g, c) of a stage: lane l holds the four bytes of rows 128 c + 32 j + l, j < 4.
        // A step's words are loaded one step ahead of their stage.
        constexpr int WORDS = 2 * 4 * C::SF_CHUNKS;
        const int kb = p.K / MX_BLOCK;
        const bool wide = kb % 8 == 0 && ((uintptr_t)p.a_scales & 7) == 0;
        uint32_t w[WORDS];
        auto load = [&](const MxTile &x, int kt) {
#pragma unroll
            for (int j = 0; j < WORDS / 2; ++j) {
                const int r = 32 * j + lane;
                uint32_t v[2] = {0x7f7f7f7fu, 0x7f7f7f7fu};
                if (r < x.n) {
                    const uint8_t *src = p.a_scales + (size_t)(x.row0 + r) * kb + kt * 8;
                    if (wide) {
                        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(src));
                        v[0] = u.x;
                        v[1] = u.y;
                    } else {
                        for (int i = 0; i < 8 && kt * 8 + i < kb; ++i)
                            v[i >> 2] = (v[i >> 2] & ~(0xffu << (8 * (i & 3)))) | ((uint32_t)__ldg(src + i) << (8 * (i & 3)));
                    }
                }
                w[j] = v[0];
                w[WORDS / 2 + j] = v[1];
            }
        };
        uint32_t it = 0;
        bool ok = true;
        int64_t t = blockIdx.x;
        MxTile x{};
        if (t < tiles) {
            x = mx_tile(p, S, t, MT, C::NT);
            load(x, 0);
        }
        int kt = 0;
        while (t < tiles) {
            const uint32_t s = it % C::STAGES;
            if (!(ok = mbar_wait(smem_u32(empty + s), ((it / C::STAGES) & 1) ^ 1, abort, p.status))) break;
            const uint32_t dst = smem_u32(stages + s * C::STAGE_BYTES) + MX_TILE_BYTES + lane * 16;
#pragma unroll
            for (int c = 0; c < WORDS / 4; ++c)
                sts_v4(dst + 512 * c, make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]));
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(full + s));
            ++it;
            if (++kt == KT) {
                kt = 0;
                t += gridDim.x;
                if (t >= tiles) break;
                x = mx_tile(p, S, t, MT, C::NT);
            }
            load(x, kt);
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------------- epilogue
        const int q = warp - 4, et = threadIdx.x - 128;
        const bool vec = p.vec_out != 0;
        uint32_t tc = 0;
        for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x, ++tc) {
            const MxTile x = mx_tile(p, S, t, MT, C::NT);
            const uint32_t b = tc & 1;
            // the four warps leave together: they meet at barriers below
            uint32_t ok = mbar_wait(smem_u32(acc_full + b), (tc >> 1) & 1, abort, p.status, nullptr, 0, 0, 64);
            asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %0, 0;\n\tbarrier.cta.red.and.pred b, 1, 128, a;\n\t"
                         "selp.u32 %0, 1, 0, b;\n\t}" : "+r"(ok)::"memory");
            if (!ok) break;
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + b * C::NT;
            for (int c0 = 0; c0 < x.n; c0 += MX_CHUNK) {
                float v[32];
                tc_ld32(acc + c0, v);
                tc_wait_ld();
                if (c0 + MX_CHUNK >= x.n) {   // the tile's last columns are read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(acc_empty + b));
                }
                if (C::GATED) {
                    // lane 2i holds gate i, lane 2i + 1 up i: the even lane takes row j, the odd one row j + 1
                    float *dst = epi + (lane & 1) * C::PITCH + q * 16 + (lane >> 1);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? v[j] : v[j + 1], 1);
                        const float g = (lane & 1) ? got : v[j], u = (lane & 1) ? v[j + 1] : got;
                        dst[j * C::PITCH] = silu(g) * u;
                    }
                } else {
                    float *dst = epi + q * 32 + lane;
#pragma unroll
                    for (int j = 0; j < 32; ++j) dst[j * C::PITCH] = v[j];
                }
                asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
                const int rows = min(MX_CHUNK, x.n - c0);
                // items of 8 outputs of a row, a row's items on consecutive threads
                for (int i = et; i < rows * (C::F / 8); i += 128) {
                    const int r = i / (C::F / 8), g8 = i % (C::F / 8), f = x.m * C::F + g8 * 8;
                    float y[8];
                    const float4 y0 = *reinterpret_cast<const float4 *>(epi + r * C::PITCH + g8 * 8);
                    const float4 y1 = *reinterpret_cast<const float4 *>(epi + r * C::PITCH + g8 * 8 + 4);
                    y[0] = y0.x; y[1] = y0.y; y[2] = y0.z; y[3] = y0.w;
                    y[4] = y1.x; y[5] = y1.y; y[6] = y1.z; y[7] = y1.w;
                    const size_t row = (size_t)x.row0 + c0 + r;
                    if (p.out_type == DT_MXFP4) {
                        // four threads hold a block of 32 outputs (rows * F / 8 is a multiple of 8)
                        uint32_t amax = 0;
#pragma unroll
                        for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(y[j]) & 0x7fffffffu);
                        const unsigned team = 0xfu << (threadIdx.x & 28);
                        amax = max(amax, __shfl_xor_sync(team, amax, 1));
                        amax = max(amax, __shfl_xor_sync(team, amax, 2));
                        const uint32_t sc = mx_scale_byte(amax);
                        uint32_t c = 0x77777777u;
                        if (sc != 255u) {
                            const float inv = mx_inverse(sc);
                            c = 0;
#pragma unroll
                            for (int j = 0; j < 4; ++j) c |= e2m1x2_code(y[2 * j] * inv, y[2 * j + 1] * inv) << (8 * j);
                        }
                        if (f < p.N) {   // N % 32 == 0: a block is all in or all out
                            *reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(p.out) + row * (p.N / 2) + f / 2) = c;
                            if ((g8 & 3) == 0) p.out_scales[row * (p.N / MX_BLOCK) + f / MX_BLOCK] = (uint8_t)sc;
                        }
                    } else if (p.out_type == DT_F32) {
                        mx_store8<float>(p, row * p.ld + f, f, y, vec);
                    } else if (p.out_type == DT_BF16) {
                        mx_store8<__nv_bfloat16>(p, row * p.ld + f, f, y, vec);
                    } else {
                        mx_store8<__half>(p, row * p.ld + f, f, y, vec);
                    }
                }
                asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::TMEM));
    }
}

}  // namespace ds4
