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

// N values by 16-byte loads (coherent ones: add may be y).
template <class T, int N>
__device__ __forceinline__ void load_add(const T *p, float (&a)[N]) {
    constexpr int PER = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < N / PER; ++i) {
        uint4 u;
        asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p + i * PER));
        const T *v = reinterpret_cast<const T *>(&u);
#pragma unroll
        for (int j = 0; j < PER; ++j) a[i * PER + j] = to_f32<T>(v[j]);
    }
}

// y[t] = add[t] + sum_j w[t, j] o[inv_pos[t, j]]: the slots in order, in fp32, then add; a slot
// whose row is outside [0, o_rows) adds nothing.  Bound by memory: every row of o is read once.
// A thread takes 16 columns of a token; the rows of eight slots are in flight together.
template <class TO, class TY>
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ CombineArgs p, RowSplit split) {
    int t, first, last;
    split.place(t, first, last);
    const TO *o = reinterpret_cast<const TO *>(p.o);
    TY *y = reinterpret_cast<TY *>(p.y) + (size_t)t * p.H;
    const int *inv = p.inv_pos + (size_t)t * p.k;
    const float *w = p.w + (size_t)t * p.k;
    constexpr int PER = 32 / sizeof(TO);   // a 32-byte load a row
    for (int g = first + threadIdx.x; g < last; g += blockDim.x) {
        float acc[PER], extra[PER];   // add is asked for before the rows are known
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = extra[i] = 0.0f;
        if (p.add) {
            const size_t at = (size_t)t * p.H + g * PER;
            if (p.add_type == DT_F32) load_add<float, PER>(reinterpret_cast<const float *>(p.add) + at, extra);
            else if (p.add_type == DT_BF16) load_add<__nv_bfloat16, PER>(reinterpret_cast<const __nv_bfloat16 *>(p.add) + at, extra);
            else load_add<__half, PER>(reinterpret_cast<const __half *>(p.add) + at, extra);
        }
        for (int j0 = 0; j0 < p.k; j0 += 8) {
            uint32_t u[8][8];
            float wt[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = j0 + j < p.k ? __ldg(inv + j0 + j) : -1;
                const bool on = r >= 0 && r < p.o_rows;
                wt[j] = on ? __ldg(w + j0 + j) : 0.0f;
                if (on) ld_stream_v8(o + (size_t)r * p.H + g * PER, u[j]);
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
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] += extra[i];
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

// The same column by column, where rows are not 32-byte aligned.
template <class TO, class TY>
__global__ void __launch_bounds__(128) combine_columns_kernel(const __grid_constant__ CombineArgs p, RowSplit split) {
    int t, first, last;
    split.place(t, first, last);
    const TO *o = reinterpret_cast<const TO *>(p.o);
    const int *inv = p.inv_pos + (size_t)t * p.k;
    const float *w = p.w + (size_t)t * p.k;
    for (int c = first + threadIdx.x; c < last; c += blockDim.x) {
        float acc = 0.0f;
#pragma unroll 8
        for (int j = 0; j < p.k; ++j) {
            const int r = __ldg(inv + j);
            if (r >= 0 && r < p.o_rows) acc = fmaf(__ldg(w + j), to_f32<TO>(o[(size_t)r * p.H + c]), acc);
        }
        if (p.add) acc += load_typed(p.add, p.add_type, (size_t)t * p.H + c);
        reinterpret_cast<TY *>(p.y)[(size_t)t * p.H + c] = from_f32<TY>(acc);
    }
}

}  // namespace ds4
