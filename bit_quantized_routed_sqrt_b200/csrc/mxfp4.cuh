// mxfp4.cuh -- MXFP4 rows: quantisation, dequantisation and the packed layout of weights.
//
// MXFP4 (the OCP microscaling format): 32 consecutive inputs of a row share one scale byte s
// (E8M0, the value 2^(s - 127); 255 is NaN) and are E2M1 codes: sign bit, then the index of
// one of 0, 0.5, 1, 1.5, 2, 3, 4, 6.  Element 2i of a row is the low nibble of code byte i.
#pragma once
#include "common.cuh"

namespace ds4 {

constexpr int MX_BLOCK = 32;        // inputs that share a scale

enum : int { DT_F32 = 0, DT_BF16 = 1, DT_F16 = 2, DT_MXFP4 = 3 };

// The value of a scale byte in fp32 (2^-127 is a subnormal).
__device__ __forceinline__ float e8m0_value(uint32_t s) {
    return __uint_as_float(s == 255u ? 0x7fc00000u : s == 0u ? 0x00400000u : s << 23);
}
// Two codes (low nibble first) -> two fp16 values, exactly.
__device__ __forceinline__ __half2 e2m1x2_value(uint32_t byte) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(byte));
    return *reinterpret_cast<__half2 *>(&r);
}
// Two fp32 values -> codes (lo in the low nibble), nearest even, saturated at +-6.
__device__ __forceinline__ uint32_t e2m1x2_code(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
    return r & 0xFFu;
}

// The scale byte of a block from the largest |x| of it, as fp32 bits: the exponent of the
// largest magnitude less 2 (6 is the largest E2M1 value, 4 its power of two), at least -127.
// A block that holds a NaN or an infinity gets the NaN scale.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return 255u;
    const int e = (int)(amax_bits >> 23);   // a subnormal's 0 ends below 2 as well
    return e > 2 ? (uint32_t)(e - 2) : 0u;
}
// 2^-(s - 127) for a scale byte 0..252 (the largest of a finite block: 254 - 2): exact, so x times it is x over the scale.
__device__ __forceinline__ float mx_inverse(uint32_t s) { return __uint_as_float((254u - s) << 23); }

// ------------------------------------------------------------------ row types
template <class T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Loads of a kernel's inputs.  They are ordinary loads: the read-only path (ld.global.nc, __ldg) is
// for data that nothing writes while the kernel lives, and a kernel here is alive while the one
// before it writes them (see next_kernel_may_start).  A load without volatile may move, but not
// ahead of the wait that its address comes from (after_wait).
__device__ __forceinline__ int ld_input(const int *p) {
    int v;
    asm("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ld_input(const uint32_t *p) {
    uint32_t v;
    asm("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ float ld_input(const float *p) {
    float v;
    asm("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ld_input(const uint8_t *p) {
    uint32_t v;
    asm("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ld_input(const uint2 *p) {
    uint2 v;
    asm("ld.global.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 ld_input(const uint4 *p) {
    uint4 v;
    asm("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
// 16 bytes that are read once.
__device__ __forceinline__ uint4 ld_once_v4(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
// 32 bytes at once (32-byte aligned): a lane's load is a whole sector.
__device__ __forceinline__ void ld_once_v8(const void *p, uint32_t (&r)[8]) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
}
__device__ __forceinline__ void st_v8(void *p, const uint32_t (&r)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
                 "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// N consecutive values; VEC: the address is 32-byte aligned and N * sizeof(T) a multiple of 32.
template <class T, int N, bool VEC>
__device__ __forceinline__ void load_row(const T *p, float (&v)[N]) {
    if constexpr (VEC) {
        constexpr int PER = 32 / sizeof(T);
#pragma unroll
        for (int i = 0; i < N / PER; ++i) {
            uint32_t u[8];
            ld_once_v8(p + i * PER, u);
            const T *t = reinterpret_cast<const T *>(u);
#pragma unroll
            for (int j = 0; j < PER; ++j) v[i * PER + j] = to_f32<T>(t[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = to_f32<T>(p[i]);
    }
}
template <class T, int N, bool VEC>
__device__ __forceinline__ void store_row(T *p, const float (&v)[N]) {
    if constexpr (VEC) {
        constexpr int PER = 32 / sizeof(T);
#pragma unroll
        for (int i = 0; i < N / PER; ++i) {
            uint32_t u[8];
            T *t = reinterpret_cast<T *>(u);
#pragma unroll
            for (int j = 0; j < PER; ++j) t[j] = from_f32<T>(v[i * PER + j]);
            st_v8(p + i * PER, u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = from_f32<T>(v[i]);
    }
}

// Programmatic dependent launch: a kernel here lets the one behind it start at once, and waits
// for the whole of the one before it, before it reads or writes any memory that both can see.
// What overlaps is the launch and the set-up of barriers and tensor memory: one token's gated
// product 17.5 -> 15.7 us, the routing of 2048 tokens (two kernels) 12.3 -> 10.0.
__device__ __forceinline__ void next_kernel_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// A pointer whose loads (those of ld_input may move past other memory operations) cannot move
// ahead of that wait.
template <class T>
__device__ __forceinline__ T *after_wait(T *p) {
    asm volatile("" : "+l"(p)::"memory");
    return p;
}

// Rows cut into segments of items, a CTA per segment (rows * segments CTAs): item i of a row on
// thread i % blockDim.x.  Keeps a row's index arithmetic out of the items.
struct RowSplit {
    int items, segments, per;   // items a row, segments a row, items a segment
    __device__ __forceinline__ void place(int &row, int &first, int &last) const {
        row = segments == 1 ? blockIdx.x : blockIdx.x / segments;
        const int s = blockIdx.x - row * segments;
        first = s * per;
        last = min(items, first + per);
    }
};

// ------------------------------------------------------------------ quantise
// A thread takes 16 inputs (one or two 32-byte loads), two neighbours a block of 32.  Row r goes
// to row r of the output, or to the rows inv_pos[r * k + j], j < k (entries outside [0, out_rows)
// are skipped): the row is read and rounded once however many places it goes to.  Bound by
// memory: 2048 x 4096 bf16 to 8 places each take 12.7 us cold (52 MB, 8 us at a copy's rate),
// 8192 x 7168 70 us (56); with 8 inputs a thread and 16-byte loads 18 and 93.
template <class T, bool VEC>
__global__ void __launch_bounds__(128) mxfp4_quantize_kernel(const T *x, int64_t ld, int K, RowSplit split,
                                                             const int *inv_pos, int k, int out_rows,
                                                             uint8_t *codes, uint8_t *scales) {
    next_kernel_may_start();
    wait_for_kernel_before();
    x = after_wait(x);
    inv_pos = after_wait(inv_pos);
    int r, first, last;
    split.place(r, first, last);
    // items are K / 16 and segments even: the two threads of a block of 32 are in or out together
    for (int g = first + threadIdx.x; g < last; g += blockDim.x) {
        float v[16];
        load_row<T, 16, VEC>(x + r * ld + g * 16, v);
        uint32_t amax = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7fffffffu);
        amax = max(amax, __shfl_xor_sync(3u << (threadIdx.x & 30), amax, 1));
        const uint32_t s = mx_scale_byte(amax);
        uint2 c = make_uint2(0x77777777u, 0x77777777u);
        if (s != 255u) {
            const float inv = mx_inverse(s);
            c = make_uint2(0, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c.x |= e2m1x2_code(v[2 * j] * inv, v[2 * j + 1] * inv) << (8 * j);
                c.y |= e2m1x2_code(v[8 + 2 * j] * inv, v[9 + 2 * j] * inv) << (8 * j);
            }
        }
        const size_t code_at = (size_t)g * 8, scale_at = g >> 1;
        if (!inv_pos) {
            *reinterpret_cast<uint2 *>(codes + (size_t)r * (K / 2) + code_at) = c;
            if ((g & 1) == 0) scales[(size_t)r * (K / MX_BLOCK) + scale_at] = (uint8_t)s;
        } else {
#pragma unroll 4
            for (int j = 0; j < k; ++j) {
                const int p = ld_input(inv_pos + (size_t)r * k + j);
                if (p < 0 || p >= out_rows) continue;
                *reinterpret_cast<uint2 *>(codes + (size_t)p * (K / 2) + code_at) = c;
                if ((g & 1) == 0) scales[(size_t)p * (K / MX_BLOCK) + scale_at] = (uint8_t)s;
            }
        }
    }
}

// ------------------------------------------------------------------ dequantise
// A thread takes 16 values: 8 bytes of codes and their scale byte to one or two 32-byte stores.
// Bound by memory: 65536 x 7168 to bf16 take 183 us (181 at a copy's rate); with 8 values a
// thread and 16-byte stores 259.
template <class T, bool VEC>
__global__ void __launch_bounds__(128) mxfp4_dequantize_kernel(const uint8_t *codes,
                                                               const uint8_t *scales, int K, RowSplit split,
                                                               T *out, int64_t ld) {
    next_kernel_may_start();
    wait_for_kernel_before();
    codes = after_wait(codes);
    scales = after_wait(scales);
    int r, first, last;
    split.place(r, first, last);
#pragma unroll 2
    for (int g = first + threadIdx.x; g < last; g += blockDim.x) {
        const uint2 c = ld_input(reinterpret_cast<const uint2 *>(codes + (size_t)r * (K / 2)) + g);
        const float s = e8m0_value(ld_input(scales + (size_t)r * (K / MX_BLOCK) + (g >> 1)));
        float v[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 f = __half22float2(e2m1x2_value(((j < 4 ? c.x : c.y) >> (8 * (j & 3))) & 0xFFu));
            v[2 * j] = f.x * s;
            v[2 * j + 1] = f.y * s;
        }
        store_row<T, 16, VEC>(out + r * ld + g * 16, v);
    }
}

// ------------------------------------------------------------------ packed weights
// An expert's matrix [N][K] is cut into tiles of 128 rows x 256 inputs (both filled up with
// zeros), ordered (row tile, input tile), 17408 contiguous bytes each:
//   bytes [0, 16384):     the codes as shared memory wants them: row r at r * 128, its 16-byte
//                         chunk c (32 inputs) at chunk c ^ (r % 8)  (128-byte swizzle)
//   bytes [16384, 17408): the scales, 512 bytes for each 128 inputs: four bytes (one per 32
//                         inputs) of row r at (r % 32) * 16 + (r / 32) * 4
// Gated matrices hold 2N rows: gate row i in row 2i, up row i in row 2i + 1.
constexpr int MX_TM = 128, MX_TK = 256;
constexpr int MX_CODE_BYTES = MX_TM * MX_TK / 2;
constexpr int MX_TILE_BYTES = MX_CODE_BYTES + MX_TM * MX_TK / MX_BLOCK;   // 17408
__host__ __device__ constexpr size_t mx_expert_bytes(int rows, int K) {
    return (size_t)((rows + MX_TM - 1) / MX_TM) * ((K + MX_TK - 1) / MX_TK) * MX_TILE_BYTES;
}
__host__ __device__ constexpr uint32_t mx_code_off(int r, int chunk) { return (uint32_t)(r * 128 + ((chunk ^ (r & 7)) << 4)); }
__host__ __device__ constexpr uint32_t mx_scale_off(int r, int blk) {
    return (uint32_t)(MX_CODE_BYTES + (blk >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (blk & 3));
}

// One thread per (expert, packed row, block of 32 inputs), filler included.
__global__ void __launch_bounds__(256) mxfp4_pack_kernel(const uint8_t *c0, const uint8_t *s0,
                                                         const uint8_t *c1, const uint8_t *s1,
                                                         int E, int N, int K, uint8_t *packed) {
    next_kernel_may_start();
    wait_for_kernel_before();
    c0 = after_wait(c0);
    s0 = after_wait(s0);
    c1 = after_wait(c1);
    s1 = after_wait(s1);
    const int mats = c1 ? 2 : 1, rows = N * mats;
    const int row_tiles = (rows + MX_TM - 1) / MX_TM, k_tiles = (K + MX_TK - 1) / MX_TK;
    const int64_t per_tile = MX_TM * (MX_TK / MX_BLOCK);
    const int64_t total = (int64_t)E * row_tiles * k_tiles * per_tile;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t tile = i / per_tile;
        const int in = (int)(i - tile * per_tile), r = in >> 3, blk = in & 7;
        const int kt = (int)(tile % k_tiles);
        const int64_t rest = tile / k_tiles;
        const int rt = (int)(rest % row_tiles), e = (int)(rest / row_tiles);
        const int row = rt * MX_TM + r, kb = kt * (MX_TK / MX_BLOCK) + blk;
        uint4 c = make_uint4(0, 0, 0, 0);
        uint8_t s = 127;
        if (row < rows && kb < K / MX_BLOCK) {
            const uint8_t *cs = mats == 2 && (row & 1) ? c1 : c0, *ss = mats == 2 && (row & 1) ? s1 : s0;
            const size_t src = ((size_t)e * N + (mats == 2 ? row >> 1 : row)) * (K / MX_BLOCK) + kb;
            c = *reinterpret_cast<const uint4 *>(cs + src * 16);
            s = ss[src];
        }
        uint8_t *t = packed + (size_t)tile * MX_TILE_BYTES;
        *reinterpret_cast<uint4 *>(t + mx_code_off(r, blk)) = c;
        t[mx_scale_off(r, blk)] = s;
    }
}

}  // namespace ds4
