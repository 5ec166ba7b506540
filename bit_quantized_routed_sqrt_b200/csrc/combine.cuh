// combine.cuh -- the weighted sum of each token's expert rows.
#pragma once
#include "mxfp4.cuh"

namespace ds4 {

struct CombineArgs {
    const void *o;           // [o_rows][H] expert rows
    int64_t o_rows;
    int T, k, H;
    const int *inv_pos;      // [T][k]
    const float *w;          // [T][k]
    const void *add;         // [T][H] or null
    int add_type;
    void *y;                 // [T][H]
};

__device__ __forceinline__ float load_typed(const void *p, int type, size_t i) {
    return type == DT_F32 ? reinterpret_cast<const float *>(p)[i]
           : type == DT_BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i])
                             : __half2float(reinterpret_cast<const __half *>(p)[i]);
}

// acc += N values by 16-byte loads (coherent ones: add may be y).
template <class T, int N>
__device__ __forceinline__ void add_row(const T *p, float (&acc)[N]) {
    constexpr int PER = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < N / PER; ++i) {
        uint4 u;
        asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p + i * PER));
        const T *v = reinterpret_cast<const T *>(&u);
#pragma unroll
        for (int j = 0; j < PER; ++j) acc[i * PER + j] += to_f32<T>(v[j]);
    }
}

// y[t] = add[t] + sum_j w[t, j] o[inv_pos[t, j]]: the slots in order, in fp32, then add; a slot
// whose row is outside [0, o_rows) adds nothing.  Bound by memory: every row of o is read once.
// A thread takes the columns of 32 bytes of a token; the rows of eight slots are in flight
// together: 8192 x 7168 of 8, bf16 with an fp32 add, take 217 us (215 at a copy's rate; a column
// a thread took 516).  Asking for add before the rows cost registers: 232 us.
template <class TO, class TY>
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ CombineArgs p, RowSplit split) {
    next_kernel_may_start();
    wait_for_kernel_before();
    int t, first, last;
    split.place(t, first, last);
    const TO *o = reinterpret_cast<const TO *>(p.o);
    TY *y = reinterpret_cast<TY *>(p.y) + (size_t)t * p.H;
    const int *inv = after_wait(p.inv_pos) + (size_t)t * p.k;
    const float *w = after_wait(p.w) + (size_t)t * p.k;
    constexpr int PER = 32 / sizeof(TO);   // a 32-byte load a row
    for (int g = first + threadIdx.x; g < last; g += blockDim.x) {
        float acc[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = 0.0f;
        for (int j0 = 0; j0 < p.k; j0 += 8) {
            uint32_t u[8][8];
            float wt[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = j0 + j < p.k ? ld_input(inv + j0 + j) : -1;
                const bool on = r >= 0 && r < p.o_rows;
                wt[j] = on ? ld_input(w + j0 + j) : 0.0f;
                if (on) ld_once_v8(o + (size_t)r * p.H + g * PER, u[j]);
                else
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[j][i] = 0u;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const TO *v = reinterpret_cast<const TO *>(u[j]);
#pragma unroll
                for (int i = 0; i < PER; ++i) acc[i] = fmaf(wt[j], to_f32<TO>(v[i]), acc[i]);
            }
        }
        if (p.add) {
            const size_t at = (size_t)t * p.H + g * PER;
            if (p.add_type == DT_F32) add_row<float, PER>(reinterpret_cast<const float *>(p.add) + at, acc);
            else if (p.add_type == DT_BF16) add_row<__nv_bfloat16, PER>(reinterpret_cast<const __nv_bfloat16 *>(p.add) + at, acc);
            else add_row<__half, PER>(reinterpret_cast<const __half *>(p.add) + at, acc);
        }
        if constexpr (PER * sizeof(TY) % 32 == 0) {
            store_row<TY, PER, true>(y + g * PER, acc);
        } else {   // fp32 rows, 16-bit result: 16 bytes
            uint4 u;
            TY *v = reinterpret_cast<TY *>(&u);
#pragma unroll
            for (int i = 0; i < PER; ++i) v[i] = from_f32<TY>(acc[i]);
            *reinterpret_cast<uint4 *>(y + g * PER) = u;
        }
    }
}

// The same for rows that begin at any element.  A thread takes 16 bytes of every row: they lie in
// one or two aligned 16-byte pieces (the same offset for all threads of a row), which it loads
// whole and shifts together; a piece is loaded only where it holds some byte of o.  The results
// go through shared memory, so that their stores (and the loads of add) are of neighbours.
// One column a load instead took 325 us where this takes 129 at 5000 x 6001 of 8, bf16.
template <class TO, class TY>
__global__ void __launch_bounds__(128) combine_shifted_kernel(const __grid_constant__ CombineArgs p, RowSplit split) {
    constexpr int PER = 16 / sizeof(TO);
    __shared__ float buf[4][32 * (PER + 1)];
    next_kernel_may_start();
    wait_for_kernel_before();
    int t, first, last;
    split.place(t, first, last);
    const uintptr_t base = (uintptr_t)after_wait(p.o), end = base + (size_t)p.o_rows * p.H * sizeof(TO);
    const int *inv = after_wait(p.inv_pos) + (size_t)t * p.k;
    const float *w = after_wait(p.w) + (size_t)t * p.k;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int g0 = first + 32 * warp; g0 < last; g0 += 128) {   // 32 pieces a warp
        const int g = g0 + lane;
        float acc[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = 0.0f;
        for (int j0 = 0; j0 < p.k; j0 += 4) {
            uint4 lo[4], hi[4];
            float wt[4];
            uint32_t m[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = j0 + j < p.k ? ld_input(inv + j0 + j) : -1;
                const bool on = r >= 0 && r < p.o_rows;
                const uintptr_t at = base + ((size_t)(on ? r : 0) * p.H + (size_t)g * PER) * sizeof(TO), piece = at & ~(uintptr_t)15;
                m[j] = (uint32_t)at & 15u;
                wt[j] = on ? ld_input(w + j0 + j) : 0.0f;
                lo[j] = hi[j] = make_uint4(0, 0, 0, 0);
                if (on && g < last && piece < end) lo[j] = ld_once_v4(reinterpret_cast<const void *>(piece));
                if (on && g < last && m[j] && piece + 16 < end) hi[j] = ld_input(reinterpret_cast<const uint4 *>(piece + 16));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j0 + j >= p.k) break;
                uint32_t v[8] = {lo[j].x, lo[j].y, lo[j].z, lo[j].w, hi[j].x, hi[j].y, hi[j].z, hi[j].w};
                if (m[j] & 8u) { v[0] = v[2]; v[1] = v[3]; v[2] = v[4]; v[3] = v[5]; v[4] = v[6]; }
                if (m[j] & 4u) { v[0] = v[1]; v[1] = v[2]; v[2] = v[3]; v[3] = v[4]; v[4] = (m[j] & 8u) ? v[7] : v[5]; }
                uint32_t u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) u[i] = __funnelshift_r(v[i], v[i + 1], 8 * (m[j] & 3u));
                const TO *x = reinterpret_cast<const TO *>(u);
                // what a row's end leaves of the next row is not stored; a slot without a row adds nothing
#pragma unroll
                    for (int i = 0; i < PER; ++i) acc[i] = fmaf(wt[j], to_f32<TO>(x[i]), acc[i]);
            }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < PER; ++i) buf[warp][lane * (PER + 1) + i] = acc[i];
        __syncwarp();
        const int c0 = g0 * PER, n = min((min(last, g0 + 32) - g0) * PER, p.H - c0);   // last * PER can pass 2^31
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = 32 * i + lane;
            if (c >= n) break;
            const size_t at = (size_t)t * p.H + c0 + c;
            float y = buf[warp][c / PER * (PER + 1) + c % PER];
            if (p.add) y += load_typed(p.add, p.add_type, at);
            reinterpret_cast<TY *>(p.y)[at] = from_f32<TY>(y);
        }
    }
}

}  // namespace ds4
