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

// y[t] = add[t] + sum_j w[t, j] o[inv_pos[t, j]], slots in order, in fp32; a slot whose row is
// outside [0, o_rows) adds nothing.
template <class TO, class TY>
__global__ void __launch_bounds__(256) combine_kernel(CombineArgs p) {
    const int64_t total = (int64_t)p.T * p.H;
    const TO *o = reinterpret_cast<const TO *>(p.o);
    TY *y = reinterpret_cast<TY *>(p.y);
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int t = (int)(i / p.H), c = (int)(i - (int64_t)t * p.H);
        float acc = p.add ? load_typed(p.add, p.add_type, (size_t)i) : 0.0f;
        for (int j = 0; j < p.k; ++j) {
            const int r = p.inv_pos[(size_t)t * p.k + j];
            if (r < 0 || r >= p.o_rows) continue;
            acc = fmaf(p.w[(size_t)t * p.k + j], to_f32<TO>(o[(size_t)r * p.H + c]), acc);
        }
        y[i] = from_f32<TY>(acc);
    }
}

}  // namespace ds4
