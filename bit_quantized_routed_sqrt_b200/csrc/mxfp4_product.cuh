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
    int *status;
};

// Rows [first, last) of expert e, clipped to the rows there are.
__device__ __forceinline__ void mx_group(const MxArgs &p, int e, int &first, int &last) {
    first = p.offsets ? min(max(p.offsets[e], 0), p.rows) : 0;
    last = p.offsets ? min(max(p.offsets[e + 1], first), p.rows) : p.rows;
}

// ------------------------------------------------------------------ tcgen05
// out[r][n] = sum_k a[r][k] W[n][k] over each expert's rows: products of two E2M1 values and two
// powers of two are exact, the sums are fp32.  The weights bound it where an expert has few rows
// (17/32 byte a weight: 6.3 TB/s at 128 rows of 256 experts, 97% of a copy's rate), the steps of
// the ring below where it has many (3.1 PFLOP/s at 8191 x 4096 x 4096, 87 to 89 us).
//
// A persistent kernel, one CTA per SM, over tiles of 128 packed weight rows (the MMA's M) x up
// to NT rows of a (the MMA's N): each expert's rows are cut into equal tiles of at most NT, and
// the tiles that share weight rows follow one another, so the weights cross HBM once.  One
// K step is 256 inputs: a weight tile with its scales (one contiguous bulk copy), the rows'
// codes (TMA, 128-byte swizzle) and the rows' scales, then four block-scaled MMAs of 64 inputs
// (kind::mxf4: E2M1 x E2M1 with an E8M0 scale per 32, fp32 accumulators in tensor memory).  A
// stage of the ring holds one or two such steps.
//   warps 0, 3 producers of weight tiles and of row codes
//   warp 1     allocates tensor memory; copies the step's scales there (tcgen05.cp) and issues
//              the MMAs.  Every stage has its own scale columns, so a copy never meets an MMA
//              that still reads the columns' last contents
//   warps 2,12 rows' scales (rows start anywhere, K / 32 is any number), laid out in shared
//              memory as the copy wants them
//   warps 4-11 epilogue, in two groups of four that take chunks of 32 rows in turn: accumulators
//              -> silu(g) * u -> output.  A lane is an output, so a warp stores 32 (gated: two
//              times 16) neighbouring elements of a row at once: 740 cycles a chunk, where a store
//              under a test of its row each took 3000 and made the epilogue the bound (1.06 against
//              0.95 ms at 65536 rows x 7168 x 2048)
// The accumulators are double buffered, so a tile's epilogue overlaps the next tile.
// Every wait is bounded, as in the layer's grouped GEMM: on a timeout the CTA records
// ETIMEOUT, waits for its own copies and MMAs, frees tensor memory and returns.
//
// What a step costs beside its MMAs (130 to 510 cycles) is the roles' serial work: a successful
// barrier test takes 150 cycles, the issue of a bulk copy 55 and of a TMA load 100 more.  Pairs
// of CTAs (cta_group::2, half the rows' traffic) measured 5% faster at 8191 x 4096 x 4096 and 7%
// slower at 65536 x 7168 x 2048; two steps at a time in the MMA warp 8% slower at both.
constexpr int MX_THREADS = 416;
constexpr int MX_CHUNK = 32;             // rows of a (accumulator columns) that an epilogue warp takes at a time
// MXFP4 output: of each pair of epilogue warps, two buffers of the codes of 32 rows x 32
// outputs and of each warp's scale bytes
constexpr int MX_PAIR_BYTES = 2 * (32 * 16 + 2 * 32);

// BOX1 < BOX0 < NT: the row counts that one TMA load can bring (a tile takes the least that holds it).
// PER: input tiles (of 256) a stage.
template <int NT_, int BOX0_, int BOX1_, int STAGES_, int PER_, bool GATED_>
struct MxCfg {
    static constexpr int PER = PER_;
    static constexpr int NT = NT_, BOX0 = BOX0_, BOX1 = BOX1_, STAGES = STAGES_;
    static constexpr bool GATED = GATED_;
    static constexpr int SF_CHUNKS = (NT + 127) / 128;                 // 512-byte scale chunks of the rows per 128 inputs
    static constexpr int B_BYTES = (NT * 128 + 1023) / 1024 * 1024;
    static constexpr int SFB_BYTES = 2 * SF_CHUNKS * 512;
    // PER of each: weight tiles (codes, scales) | row scales | (to 1024) | row codes
    static constexpr int SFB_OFF = PER * MX_TILE_BYTES;
    static constexpr int B_OFF = (SFB_OFF + PER * SFB_BYTES + 1023) / 1024 * 1024;
    static constexpr int STAGE_BYTES = B_OFF + PER * B_BYTES;
    static constexpr int TILE_COLS = 8 + 8 * SF_CHUNKS;                // tensor memory columns of an input tile's scales
    static constexpr int SF_COLS = PER * TILE_COLS;                    // and of a stage's
    static constexpr int COLS = 2 * NT + STAGES * SF_COLS;
    static constexpr int TMEM = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    static constexpr int F = GATED ? 64 : 128;                         // outputs of a tile
    static constexpr int EPI_BYTES = 4 * MX_PAIR_BYTES;
    static constexpr int BAR_BYTES = 256;
    static constexpr int S_BYTES = 3 * (SR_MAX_EXPERTS + 1) * 4;
    static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + EPI_BYTES + BAR_BYTES + S_BYTES;
    static_assert(COLS <= 512, "tensor memory");
    static_assert(PER <= 2 && STAGES * PER >= 4, "a scale warp waits on every other pair of input tiles");
    static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
    static_assert(NT <= 255 && NT % 16 == 0 && NT > BOX0 && BOX0 > BOX1 && BOX1 % 8 == 0, "row tiles");
    static_assert((2 * STAGES + 5) * 8 + 16 + 32 + 4 * STAGES <= BAR_BYTES, "barrier area");
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

// Flags beside the rows of a step's tile.
constexpr uint32_t MX_HALF = 1u << 29, MX_FIRST = 1u << 30, MX_LAST = 1u << 31;   // half: one input tile

// Whether the phase of that parity has completed, without waiting.
__device__ __forceinline__ uint32_t mx_test(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done;
}

constexpr int MX_MOST_ROWS = INT32_MAX - 255;   // a box of rows that begins at the last one ends within 31 bits

// An expert's rows (up to 2^31 - 1) are cut into equal tiles of at most NT: how many tiles, and the
// rows of each but the last, a multiple of 16.
__host__ __device__ constexpr int mx_row_tiles(int rows, int NT) { return (int)(((uint32_t)rows + NT - 1) / NT); }
__host__ __device__ constexpr int mx_tile_rows(int rows, int tiles, int NT) {
    const int even = (int)((((uint32_t)rows + tiles - 1) / tiles + 15) & ~15u);
    return even < NT ? even : NT;
}

struct MxTile {
    int e, m, row0, n;   // expert, weight row tile, first row of a, rows
};

// The tiles of one CTA in order, for one warp: S[e] counts the row tiles of the experts before
// e, lo[e] and hi[e] are its rows, MT is the number of weight row tiles.  Tiles and their
// counts fit 31 bits (the host checks).
template <int NT>
struct MxTiles {
    const int *S, *row_lo, *row_hi;
    uint32_t MT, t, tiles, lo, hi;   // the expert's tiles: [lo, hi)
    int E, e, nt, first, last, per;

    __device__ __forceinline__ MxTiles(const int *S_, int E_, int MT_, uint32_t tiles_)
        : S(S_), row_lo(S_ + SR_MAX_EXPERTS + 1), row_hi(S_ + 2 * (SR_MAX_EXPERTS + 1)), MT(MT_), t(blockIdx.x),
          tiles(tiles_), lo(0), hi(0), E(E_), e(-1) {}
    __device__ __forceinline__ bool more() const { return t < tiles; }
    __device__ __forceinline__ void next() { t += gridDim.x; }
    __device__ __forceinline__ MxTile get() {
        if (t >= hi) {
            // The last expert behind e with S * MT <= t, 32 candidates at a time: it is E - 1 at
            // most, and S[e + 1] * MT <= t holds (the tiles of e end there).
            const int lane = threadIdx.x & 31;
            int l = e + 1;
            const int step = (E - l + 31) >> 5;   // at most 16
            int i = l + lane * step;
            l += (__popc(__ballot_sync(0xffffffffu, i < E && (uint32_t)S[min(i, E)] * MT <= t)) - 1) * step;
            i = l + lane;
            l += __popc(__ballot_sync(0xffffffffu, lane < step && i < E && (uint32_t)S[min(i, E)] * MT <= t)) - 1;
            e = l;
            lo = (uint32_t)S[e] * MT;
            nt = S[e + 1] - S[e];
            hi = lo + nt * MT;
            first = row_lo[e];
            last = row_hi[e];
            per = mx_tile_rows(last - first, nt, NT);
        }
        MxTile x;
        x.e = e;
        const uint32_t local = t - lo;
        x.m = nt == 1 ? local : local / (uint32_t)nt;
        x.row0 = first + (int)(local - (uint32_t)x.m * nt) * per;
        x.n = min(per, last - x.row0);   // at least 1: nt tiles of per rows are needed
        return x;
    }
};

// silu(g) u = g u / (1 + e^-g).  Below SILU_FAR e^-g leaves the range where __fdividef divides (its
// result is 0 for divisors above 2^126), though the product may be a normal value; there 1 + e^-g is
// e^-g to the last bit, and each half of e^g goes to one factor.  The operands of one quotient are
// selected: selecting the quotient itself makes a branch of it (16384 rows, 2 x 2048 x 4096: 454 us
// against 480).
constexpr float SILU_FAR = -87.0f;
__device__ __forceinline__ float silu_times(float g, float u) {
    const bool far = g < SILU_FAR;
    const float e = expf(far ? 0.5f * g : -g);
    return __fdividef(far ? g * e : g, far ? 1.0f : 1.0f + e) * (far ? u * e : u);
}

// The gated values of a chunk: lane 2i holds gate i, lane 2i + 1 up i; h[j] is row 2j in the even
// lane, row 2j + 1 in the odd one.
__device__ __forceinline__ void mx_gated(const float (&v)[32], float (&h)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const float got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? v[2 * j] : v[2 * j + 1], 1);
        h[j] = silu_times((lane & 1) ? got : v[2 * j], (lane & 1) ? v[2 * j + 1] : got);
    }
}

// One chunk of an epilogue warp: rows row0 .. row0 + rows - 1 (rows <= 32) from accumulator
// columns v, outputs from f0 on (this warp's: 32, gated 16).
template <bool GATED, class T>
__device__ __forceinline__ void mx_store_chunk(const MxArgs &p, const float (&v)[32], size_t row0, int rows, int f0) {
    const int lane = threadIdx.x & 31;
    const int f = f0 + (GATED ? lane >> 1 : lane);
    T *out = reinterpret_cast<T *>(p.out) + (row0 + (GATED ? lane & 1 : 0)) * p.ld + f;
    const int64_t step = (GATED ? 2 : 1) * p.ld;
    float y[GATED ? 16 : 32];
    if constexpr (GATED) {
        mx_gated(v, y);
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) y[j] = v[j];
    }
    constexpr int J = GATED ? 16 : 32;
    if (rows == MX_CHUNK && f0 + (GATED ? 16 : 32) <= p.N) {   // a whole chunk: no predicates
#pragma unroll
        for (int j = 0; j < J; ++j, out += step) *out = from_f32<T>(y[j]);
    } else if (f < p.N) {
        const int mine = GATED ? (rows - (lane & 1) + 1) >> 1 : rows;
#pragma unroll
        for (int j = 0; j < J; ++j, out += step)
            if (j < mine) *out = from_f32<T>(y[j]);
    }
}

// The same for MXFP4 output.  Gated, a pair of warps holds the 32 outputs of a block, 16 each
// (half: which): they exchange their scale bytes and put their codes into one buffer,
// at two barriers of the pair; otherwise a warp holds a whole block and uses a buffer alone.
template <bool GATED>
__device__ __forceinline__ void mx_store_chunk_mxfp4(const MxArgs &p, const float (&v)[32], size_t row0, int rows, int f0,
                                                     uint8_t *buf, int bar, int half) {
    const int lane = threadIdx.x & 31;
    uint8_t *codes = buf;                                        // [32 rows][16]
    uint8_t *sc = buf + 512;                                     // [2][32 rows]
    if (GATED) {
        float h[16];
        uint32_t m[16];
        mx_gated(v, h);
#pragma unroll
        for (int j = 0; j < 16; ++j) m[j] = __float_as_uint(h[j]) & 0x7fffffffu;
#pragma unroll
        for (int o = 2; o < 32; o <<= 1)
#pragma unroll
            for (int j = 0; j < 16; ++j) m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], o));
        if (lane < 2)
#pragma unroll
            for (int j = 0; j < 16; ++j) sc[half * 32 + 2 * j + lane] = (uint8_t)mx_scale_byte(m[j]);
        asm volatile("barrier.cta.sync %0, 64;" ::"r"(bar) : "memory");
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int r = 2 * j + (lane & 1);
            const uint32_t s = max(mx_scale_byte(m[j]), (uint32_t)sc[(half ^ 1) * 32 + r]);   // monotonic in the magnitude
            const float y = s == 255u ? 6.0f : h[j] * mx_inverse(s);
            const float next = __shfl_xor_sync(0xffffffffu, y, 2);
            if ((lane & 2) == 0) codes[r * 16 + half * 8 + (lane >> 2)] = (uint8_t)e2m1x2_code(y, next);
        }
        asm volatile("barrier.cta.sync %0, 64;" ::"r"(bar) : "memory");
        if (half == 0 && lane < rows && f0 < p.N) {
            *reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(p.out) + (row0 + lane) * (p.N / 2) + f0 / 2) =
                *reinterpret_cast<const uint4 *>(codes + lane * 16);
        } else if (half == 1 && lane < rows && f0 - 16 < p.N) {
            p.out_scales[(row0 + lane) * (p.N / MX_BLOCK) + (f0 - 16) / MX_BLOCK] =
                max(sc[lane], sc[32 + lane]);
        }
    } else {
        uint32_t my_scale = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const uint32_t s = mx_scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(v[j]) & 0x7fffffffu));
            const float y = s == 255u ? 6.0f : v[j] * mx_inverse(s);
            const float next = __shfl_xor_sync(0xffffffffu, y, 1);
            if ((lane & 1) == 0) codes[j * 16 + (lane >> 1)] = (uint8_t)e2m1x2_code(y, next);
            if (lane == j) my_scale = s;
        }
        __syncwarp();
        if (lane < rows && f0 < p.N) {
            *reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(p.out) + (row0 + lane) * (p.N / 2) + f0 / 2) =
                *reinterpret_cast<const uint4 *>(codes + lane * 16);
            p.out_scales[(row0 + lane) * (p.N / MX_BLOCK) + f0 / MX_BLOCK] = (uint8_t)my_scale;
        }
        __syncwarp();
    }
}

template <class C>
__global__ void __launch_bounds__(MX_THREADS, 1)
    mxfp4_product_kernel(const __grid_constant__ CUtensorMap tm_nt, const __grid_constant__ CUtensorMap tm_box0,
                         const __grid_constant__ CUtensorMap tm_box1, const __grid_constant__ MxArgs p) {
    next_kernel_may_start();
    extern __shared__ __align__(1024) uint8_t mx_smem_raw[];
    uint8_t *stages = mx_smem_raw + ((1024u - (smem_u32(mx_smem_raw) & 1023u)) & 1023u);
    uint8_t *epi = stages + C::STAGES * C::STAGE_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(epi + C::EPI_BYTES);
    uint64_t *full = bars;                       // [S] two producers (with their bytes) and a scale warp
    uint64_t *empty = full + C::STAGES;          // [S] MMA commit
    uint64_t *acc_full = empty + C::STAGES;      // [2] MMA commit
    uint64_t *acc_empty = acc_full + 2;          // [2] 8 epilogue warps
    uint64_t *drain = acc_empty + 2;             // MMA commit at exit
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(drain + 2);
    int *part = reinterpret_cast<int *>(drain + 3);          // [8]
    volatile uint32_t *meta = reinterpret_cast<volatile uint32_t *>(part + 8);   // [S] rows | MX_FIRST | MX_LAST
    int *S = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(bars) + C::BAR_BYTES);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(full + s), 3);
            mbar_init(smem_u32(empty + s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(acc_full + b), 1);
            mbar_init(smem_u32(acc_empty + b), 8);
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
    wait_for_kernel_before();
    int decreasing = 0;   // groups would overlap and their tiles could outnumber what the host checked
    for (int e = threadIdx.x; e < p.E; e += MX_THREADS) {
        int first, last;
        if (p.offsets && p.offsets[e] > p.offsets[e + 1]) decreasing = 1;
        mx_group(p, e, first, last);
        S[e] = mx_row_tiles(last - first, C::NT);
        S[SR_MAX_EXPERTS + 1 + e] = first;
        S[2 * (SR_MAX_EXPERTS + 1) + e] = last;
    }
    tc_fence_before();
    decreasing = __syncthreads_or(decreasing);
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    int units = block_scan(S, p.E, part);
    if (decreasing) {   // no tile at all
        units = 0;
        if (threadIdx.x == 0) set_status(p.status, ST_EDEVICE);
    }
    if (threadIdx.x == 0) S[p.E] = units;
    __syncthreads();

    const int packed_rows = C::GATED ? 2 * p.N : p.N;
    const int MT = (packed_rows + MX_TM - 1) / MX_TM, KT = (p.K + MX_TK - 1) / MX_TK, KS = (KT + C::PER - 1) / C::PER;
    const uint32_t tiles = (uint32_t)units * MT;
    MxTiles<C::NT> walk(S, p.E, MT, tiles);

    if (warp == 0 || warp == 3) {
        // ---------------------------------------------------- producers: weights, row codes
        // Issuing one TMA load takes about 100 cycles after 150 for the wait, so each producer
        // has one load a step: one box holds all of a tile's rows.
        const bool weights = warp == 0;
        uint32_t it = 0;
        bool ok = true;
        for (; walk.more() && ok; walk.next()) {
            const MxTile x = walk.get();
            const uint8_t *w = p.w + (size_t)x.e * p.expert_bytes + (size_t)x.m * KT * MX_TILE_BYTES;
            const CUtensorMap *map = x.n <= C::BOX1 ? &tm_box1 : x.n <= C::BOX0 ? &tm_box0 : &tm_nt;
            const uint32_t bytes = weights ? MX_TILE_BYTES : 128 * (x.n <= C::BOX1 ? C::BOX1 : x.n <= C::BOX0 ? C::BOX0 : C::NT);
            for (int ks = 0; ks < KS; ++ks, ++it) {
                const uint32_t s = it % C::STAGES;
                if (!(ok = mbar_wait(smem_u32(empty + s), ((it / C::STAGES) & 1) ^ 1, abort, p.status))) break;
                const bool half = C::PER == 2 && 2 * ks + 1 == KT;
                if (elect_one()) {
                    const uint32_t st = smem_u32(stages + s * C::STAGE_BYTES), bar = smem_u32(full + s);
                    if (!weights)
                        meta[s] = x.n | (ks == 0 ? MX_FIRST : 0u) | (ks == KS - 1 ? MX_LAST : 0u) | (half ? MX_HALF : 0u);
                    mbar_expect_tx(bar, half ? bytes : C::PER * bytes);   // releases meta to the MMA warp
                    if (weights) {
                        bulk_g2s(st, w + (size_t)ks * C::PER * MX_TILE_BYTES, half ? bytes : C::PER * bytes, bar);
                    } else {
                        tma_load_2d(st + C::B_OFF, map, ks * C::PER * (MX_TK / 2), x.row0, bar);
                        if (C::PER == 2 && !half)
                            tma_load_2d(st + C::B_OFF + C::B_BYTES, map, ks * MX_TK + MX_TK / 2, x.row0, bar);
                    }
                }
                __syncwarp();
            }
        }
        if (!ok)   // no copy of this CTA may still be writing shared memory (a stage also waits for the other roles)
            for (uint32_t i = it > C::STAGES ? it - C::STAGES : 0; i < it; ++i)
                mbar_drain(smem_u32(full + i % C::STAGES), (i / C::STAGES) & 1, p.status);
    } else if (warp == 1) {
        // ------------------------------------------------------------------------ MMA
        // A step's rows and whether it begins or ends a tile come with its stage (meta), and
        // the next stage's barrier is asked before this step's MMAs are issued, so that this
        // warp, the one that bounds a step, neither walks the tiles (700 cycles each) nor waits
        // out the 150 cycles of a successful barrier test.
        const uint32_t mine = walk.more() ? (tiles - 1 - blockIdx.x) / gridDim.x + 1 : 0, total = mine * (uint32_t)KS;
        uint32_t tc = 0, idesc0 = 0, idesc2 = 0, d = tmem, b = 0;
        bool ok = true, ready = false;
        for (uint32_t it = 0; it < total; ++it) {
            const uint32_t s = it % C::STAGES;
            if (!ready && !(ok = mbar_wait(smem_u32(full + s), (it / C::STAGES) & 1, abort, p.status))) break;
            const uint32_t m = lds_u32(smem_u32(const_cast<const uint32_t *>(meta + s)));
            if (m & MX_FIRST) {
                b = tc & 1;
                if (!(ok = mbar_wait(smem_u32(acc_empty + b), ((tc >> 1) & 1) ^ 1, abort, p.status))) break;
                const int N = ((int)(m & 0xffffu) + 15) & ~15;
                idesc0 = mxf4_idesc(N, 0);
                idesc2 = mxf4_idesc(N, 2);
                d = tmem + b * C::NT;
            }
            const uint32_t asked = mx_test(smem_u32(full + (it + 1) % C::STAGES), ((it + 1) / C::STAGES) & 1);
            tc_fence_after();
            const uint32_t st = smem_u32(stages + s * C::STAGE_BYTES);
            const uint32_t sfa = tmem + 2 * C::NT + s * C::SF_COLS, sfb = sfa + 8;
            const uint64_t ad = sw128_desc(st), bd = sw128_desc(st + C::B_OFF);
            if (elect_one()) {
                // Unrolled, with every operand a constant off the stage's base: a loop with
                // run-time bounds moved each instruction's operands to uniform registers
                // one by one and took 1000 cycles a tile of 256 inputs where the MMAs take 160
                // to 510.  Inputs past K are zeros, so the last tile runs whole as well.
#pragma unroll
                for (int h = 0; h < C::PER; ++h) {
                    if (h == 1 && (m & MX_HALF)) break;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        mx_copy_scales(sfa + h * C::TILE_COLS + 4 * g, st + h * MX_TILE_BYTES + MX_CODE_BYTES + 512 * g);
#pragma unroll
                        for (int c = 0; c < C::SF_CHUNKS; ++c)
                            mx_copy_scales(sfb + h * C::TILE_COLS + 4 * (g * C::SF_CHUNKS + c),
                                           st + C::SFB_OFF + h * C::SFB_BYTES + 512 * (g * C::SF_CHUNKS + c));
                    }
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mx_mma(d, ad + h * (MX_TILE_BYTES >> 4) + 2 * kk, bd + h * (C::B_BYTES >> 4) + 2 * kk, kk & 1 ? idesc2 : idesc0,
                               sfa + h * C::TILE_COLS + 4 * (kk >> 1), sfb + h * C::TILE_COLS + 4 * C::SF_CHUNKS * (kk >> 1),
                               (h | kk) != 0 || !(m & MX_FIRST));
                }
                tc_commit(smem_u32(empty + s));
                if (m & MX_LAST) tc_commit(smem_u32(acc_full + b));
            }
            if (m & MX_LAST) ++tc;
            ready = __all_sync(0xffffffffu, asked);
        }
        if (elect_one()) tc_commit(smem_u32(drain));
        __syncwarp();
        mbar_drain(smem_u32(drain), 0, p.status);
    } else if (warp == 2 || warp == 12) {
        // ----------------------------------------------------------------- row scales
        // Chunk (g, c) of an input tile: 16 bytes for each l < 32, the four bytes of rows
        // 128 c + 32 j + l, j < 4.  A lane takes the 16 bytes of a row that two input tiles need;
        // the two warps take such pairs of tiles in turn and load one ahead, so the loads have
        // four tiles to arrive.  (4-byte asynchronous copies, one for each word, took 1140 cycles
        // an input tile at 192 rows: 32 lines each.)
        constexpr int R = (C::NT + 31) / 32;
        const uint32_t which = warp == 2 ? 0 : 1;
        const int kb = p.K / MX_BLOCK, PT = (KT + 1) / 2;
        const uint8_t *a_scales = after_wait(p.a_scales);
        const bool aligned = kb % 16 == 0 && ((uintptr_t)a_scales & 15) == 0;
        uint32_t cur[R][4], nxt[R][4];
        uint32_t it0 = 0;        // stages before this tile
        uint32_t g = 0;          // pairs before the one in nxt, all tiles
        MxTile x{};
        int pt = -1;             // the pair's place in the tile
        bool ok = true;
        auto load = [&]() {
#pragma unroll
            for (int j = 0; j < R; ++j) {
                if (32 * j >= x.n) break;
                const uint8_t *src = a_scales + (size_t)(x.row0 + min(32 * j + lane, x.n - 1)) * kb + pt * 16;
                if (aligned) {
                    const uint4 u = ld_input(reinterpret_cast<const uint4 *>(src));
                    nxt[j][0] = u.x; nxt[j][1] = u.y; nxt[j][2] = u.z; nxt[j][3] = u.w;
                } else {
                    // aligned words that hold any of the row's bytes, shifted; bytes past K are 0
                    const int left = kb - pt * 16;   // at least 1
                    const uint32_t *word = reinterpret_cast<const uint32_t *>((uintptr_t)src & ~(uintptr_t)3);
                    const int off = (int)((uintptr_t)src & 3);
                    uint32_t v[5];
#pragma unroll
                    for (int i = 0; i < 5; ++i) v[i] = 4 * i < off + min(left, 16) ? ld_input(word + i) : 0u;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int valid = left - 4 * i;
                        nxt[j][i] = __funnelshift_r(v[i], v[i + 1], 8 * off) &
                                    (valid >= 4 ? 0xffffffffu : valid <= 0 ? 0u : (1u << (8 * valid)) - 1u);
                    }
                }
            }
        };
        // moves to this warp's next pair, at or behind pair g, and loads it
        auto advance = [&]() {
            while (walk.more()) {
                if (pt < 0) x = walk.get();
                for (++pt; pt < PT; ++pt, ++g)
                    if ((g & 1) == which) return load();
                pt = -1;
                it0 += KS;
                walk.next();
            }
        };
        advance();
        while (walk.more() && ok) {
            const int rows = x.n, first = 2 * pt;
            const uint32_t it = it0 + first / C::PER;
#pragma unroll
            for (int j = 0; j < R; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) cur[j][i] = nxt[j][i];
            ++g;
            advance();
#pragma unroll
            for (int h = 0; h < 2 / C::PER; ++h) {   // the pair's stages
                if (first + h >= KT) break;
                const uint32_t s = (it + h) % C::STAGES;
                if (!(ok = mbar_wait(smem_u32(empty + s), (((it + h) / C::STAGES) & 1) ^ 1, abort, p.status))) break;
                const uint32_t dst = smem_u32(stages + s * C::STAGE_BYTES) + C::SFB_OFF + lane * 16;
#pragma unroll
                for (int c = 0; c < C::SF_CHUNKS; ++c) {
                    if (128 * c >= rows) break;
                    auto word = [&](int j, int i) { return 4 * c + j < R ? cur[4 * c + j < R ? 4 * c + j : 0][2 * h + i] : 0u; };
#pragma unroll
                    for (int i = 0; i < 2 * C::PER; ++i)   // input tile i / 2, 128 inputs i % 2 of it
                        sts_v4(dst + (i >> 1) * C::SFB_BYTES + 512 * ((i & 1) * C::SF_CHUNKS + c),
                               make_uint4(word(0, i), word(1, i), word(2, i), word(3, i)));
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(full + s));
            }
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------------- epilogue
        const int q = warp & 3, group = (warp - 4) >> 2, pair = group * 2 + (q >> 1);
        uint8_t *pair_buf = epi + pair * MX_PAIR_BYTES;
        const int bar = 1 + pair;
        uint32_t tc = 0, used = 0;
        for (; walk.more(); walk.next(), ++tc) {
            const MxTile x = walk.get();
            const uint32_t b = tc & 1;
            // the two warps of a pair leave together: they meet at barriers in their chunks
            uint32_t ok = mbar_wait(smem_u32(acc_full + b), (tc >> 1) & 1, abort, p.status, nullptr, 0, 0, 64);
            asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %0, 0;\n\tbarrier.cta.red.and.pred b, %1, 64, a;\n\t"
                         "selp.u32 %0, 1, 0, b;\n\t}" : "+r"(ok) : "r"(bar) : "memory");
            if (!ok) break;
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + b * C::NT;
            const int f0 = x.m * C::F + q * (C::F / 4);
            const int chunks = (x.n + MX_CHUNK - 1) / MX_CHUNK;
            const int first = (group ^ tc) & 1;   // a tile of one chunk goes to either group in turn
            for (int c = first; c < chunks; c += 2) {
                float v[32];
                tc_ld32(acc + c * MX_CHUNK, v);
                tc_wait_ld();
                if (c + 2 >= chunks) {   // this warp's last columns are read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(acc_empty + b));
                }
                const size_t row0 = (size_t)x.row0 + c * MX_CHUNK;
                const int rows = min(MX_CHUNK, x.n - c * MX_CHUNK);
                if (p.out_type == DT_F32) mx_store_chunk<C::GATED, float>(p, v, row0, rows, f0);
                else if (p.out_type == DT_BF16) mx_store_chunk<C::GATED, __nv_bfloat16>(p, v, row0, rows, f0);
                else if (p.out_type == DT_F16) mx_store_chunk<C::GATED, __half>(p, v, row0, rows, f0);
                else {
                    // gated: the pair's buffers in turn; else each warp its own
                    const uint32_t which = C::GATED ? used & 1 : q & 1;
                    mx_store_chunk_mxfp4<C::GATED>(p, v, row0, rows, f0, pair_buf + which * (MX_PAIR_BYTES / 2), bar, q & 1);
                    ++used;
                }
            }
            if (first >= chunks) {
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(acc_empty + b));
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
