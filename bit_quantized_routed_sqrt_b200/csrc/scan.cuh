// scan.cuh -- a block-wide scan over experts.
#pragma once
#include <cuda_runtime.h>

namespace ds4 {

constexpr int SR_MAX_EXPERTS = 512;
constexpr int SCAN_THREADS = 256;
static_assert(SR_MAX_EXPERTS <= 2 * SCAN_THREADS, "two experts a thread");

// Exclusive scan of v[0..E) in place by the block (E <= SR_MAX_EXPERTS; the first SCAN_THREADS threads hold
// two experts each, any others none); the total to every thread.
__device__ __forceinline__ int block_scan(int *v, int E, int *part) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int a = 2 * tid < E ? v[2 * tid] : 0, b = 2 * tid + 1 < E ? v[2 * tid + 1] : 0;
    int s = a + b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31 && warp < SCAN_THREADS / 32) part[warp] = s;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < SCAN_THREADS / 32; ++w) {
        if (w < warp) before += part[w];
        total += part[w];
    }
    const int ex = before + s - a - b;
    if (2 * tid < E) v[2 * tid] = ex;
    if (2 * tid + 1 < E) v[2 * tid + 1] = ex + a;
    __syncthreads();
    return total;
}

}  // namespace ds4
