// mxfp4_product.cuh -- products of MXFP4 rows, grouped by expert, with the experts' MXFP4 matrices.
#pragma once
#include "mxfp4.cuh"

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

// One warp per (row, 32 outputs), a lane per output: the plain order of the sum, 32 products
// of a block added in fp32, then scaled.
__global__ void __launch_bounds__(256) mxfp4_product_simple_kernel(MxArgs p) {
    const int lane = threadIdx.x & 31;
    const int n_blocks = (p.N + 31) / 32, kb = p.K / MX_BLOCK, k_tiles = (p.K + MX_TK - 1) / MX_TK;
    const int64_t total = (int64_t)p.rows * n_blocks;
    for (int64_t i = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; i < total;
         i += ((int64_t)gridDim.x * blockDim.x) >> 5) {
        const int r = (int)(i / n_blocks), n = (int)(i % n_blocks) * 32 + lane;
        int e = 0, first = 0, last = p.rows;
        for (; e < p.E; ++e) {
            mx_group(p, e, first, last);
            if (r >= first && r < last) break;
        }
        if (e == p.E) continue;   // a row behind the last group
        float v[2] = {0.0f, 0.0f};
        for (int m = 0; m < (p.gated ? 2 : 1); ++m) {
            const int row = p.gated ? 2 * n + m : n;
            if (n >= p.N) break;
            const uint8_t *tile = p.w + (size_t)e * p.expert_bytes + (size_t)(row / MX_TM) * k_tiles * MX_TILE_BYTES;
            for (int b = 0; b < kb; ++b) {
                const uint8_t *t = tile + (size_t)(b >> 3) * MX_TILE_BYTES;
                const uint4 w4 = *reinterpret_cast<const uint4 *>(t + mx_code_off(row % MX_TM, b & 7));
                const uint4 a4 = *reinterpret_cast<const uint4 *>(p.a_codes + (size_t)r * (p.K / 2) + b * 16);
                const uint32_t ws[4] = {w4.x, w4.y, w4.z, w4.w}, as[4] = {a4.x, a4.y, a4.z, a4.w};
                float acc = 0.0f;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float2 f = __half22float2(__hmul2(e2m1x2_value((ws[j >> 2] >> (8 * (j & 3))) & 0xFFu),
                                                            e2m1x2_value((as[j >> 2] >> (8 * (j & 3))) & 0xFFu)));
                    acc += f.x;
                    acc += f.y;
                }
                v[m] += acc * e8m0_value(t[mx_scale_off(row % MX_TM, b & 7)]) * e8m0_value(p.a_scales[(size_t)r * kb + b]);
            }
        }
        const float y = p.gated ? silu(v[0]) * v[1] : v[0];
        if (p.out_type == DT_MXFP4) {
            uint32_t amax = __float_as_uint(y) & 0x7fffffffu;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const uint32_t s = mx_scale_byte(amax);
            const float inv = s == 255u ? 1.0f : mx_inverse(s);
            const float next = __shfl_down_sync(0xffffffffu, y, 1);
            if ((lane & 1) == 0)
                reinterpret_cast<uint8_t *>(p.out)[(size_t)r * (p.N / 2) + n / 2] =
                    s == 255u ? 0x77 : (uint8_t)e2m1x2_code(y * inv, next * inv);
            if (lane == 0) p.out_scales[(size_t)r * (p.N / MX_BLOCK) + n / 32] = (uint8_t)s;
        } else if (n < p.N) {
            const size_t o = (size_t)r * p.ld + n;
            if (p.out_type == DT_F32) reinterpret_cast<float *>(p.out)[o] = y;
            else if (p.out_type == DT_BF16) reinterpret_cast<__nv_bfloat16 *>(p.out)[o] = __float2bfloat16_rn(y);
            else reinterpret_cast<__half *>(p.out)[o] = __float2half_rn(y);
        }
    }
}

}  // namespace ds4
