// scored_router.cuh -- routing from given logits: softmax, sigmoid or sqrt-softplus scores, a
// bias on the choice, groups, top-k, renormalised weights, and the token -> expert permutation.
#pragma once
#include "combine.cuh"
#include "scan.cuh"

namespace ds4 {

constexpr int SR_MAX_TOPK = 32;
constexpr int SR_MAX_GROUPS = 32;
constexpr int SR_WARPS = SCAN_THREADS / 32;

enum : int { SCORE_SOFTMAX = 0, SCORE_SIGMOID = 1, SCORE_SQRT_SOFTPLUS = 2 };

struct ScoredArgs {
    int E, k, score, G, topk_groups, top2, renormalise;
    float scale;
    const void *logits;
    int type;
    int64_t ld;
    int T, TB, NB;           // tokens, tokens per block, blocks
    const float *bias;       // [E] or null
    int *topk_idx;           // [T][k]
    float *topk_w;
    int *offsets, *sorted_token, *sorted_slot, *inv_pos;   // each may be null
    int *cnt;                // workspace [NB][E]
    uint32_t *mask;          // workspace [NB][E][TB / 32]
};

// Score of a logit in fp64; m and inv_sum are the softmax's maximum and 1 / sum.
__device__ __forceinline__ double score64(int kind, double l, double m, double inv_sum) {
    if (kind == SCORE_SOFTMAX) return exp(l - m) * inv_sum;
    if (kind == SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
    return sqrt(fmax(l, 0.0) + log1p(exp(-fabs(l))));
}

// Score up to a factor common to a token's experts, so that a token whose scores all
// underflow still has weights: exp(-m) times the score (sqrt-softplus: exp(-m / 2)), with m
// the largest chosen logit (softmax), or that where it is negative and 0 elsewhere.
__device__ __forceinline__ double relative_score64(int kind, double l, double m) {
    if (kind == SCORE_SOFTMAX) return exp(l - m);
    if (kind == SCORE_SIGMOID) return l >= 0.0 ? 1.0 / (1.0 + exp(-l)) : exp(l - m) / (1.0 + exp(l));
    if (l >= 0.0) return sqrt(l + log1p(exp(-l)));
    const double t = exp(l);
    return exp(0.5 * (l - m)) * (t > 0.0 ? sqrt(log1p(t) / t) : 1.0);
}

__device__ __forceinline__ double warp_max64(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Best (value, index) of a warp: the larger value, the lower index among equals.
__device__ __forceinline__ void warp_best(double &v, int &i) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const double ov = __shfl_xor_sync(0xffffffffu, v, o);
        const int oi = __shfl_xor_sync(0xffffffffu, i, o);
        if (ov > v || (ov == v && oi < i)) { v = ov; i = oi; }
    }
}

// One token, one warp; lane holds experts lane + 32 i.  Returns to lane j < k the expert of
// slot j (-1: no candidate was left) and its weight.
template <int NPL>
__device__ void scored_token(const ScoredArgs &p, int64_t t, double *scratch, int &my_e, float &my_w) {
    const int lane = threadIdx.x & 31;
    double l[NPL], c[NPL];
    double m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        const float v = e < p.E ? load_typed(p.logits, p.type, t * p.ld + e) : -INFINITY;
        // NaN and -inf: no candidate.  +inf counts as the largest finite value.
        l[i] = v > -INFINITY ? (double)fminf(v, 3.402823466e38f) : -INFINITY;
        m = fmax(m, l[i]);
    }
    const bool by_score = p.bias || (p.G > 1 && p.top2);
    double inv_sum = 0.0;
    if (p.score == SCORE_SOFTMAX && (by_score || !p.renormalise)) {
        m = warp_max64(m);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) sum += l[i] > -INFINITY ? exp(l[i] - m) : 0.0;
        inv_sum = 1.0 / warp_sum(sum);
    }
    // what is ranked: score + bias; without a bias the logit, which orders as its score does
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        c[i] = l[i];
        if (by_score && l[i] > -INFINITY) {
            c[i] = score64(p.score, l[i], m, inv_sum);
            if (p.bias) c[i] += (double)p.bias[e];
            if (!(c[i] > -INFINITY)) c[i] = l[i] = -INFINITY;
        }
    }
    if (p.G > 1) {
        const int per = p.E / p.G;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (lane + 32 * i < p.E) scratch[lane + 32 * i] = c[i];
        __syncwarp();
        double best = -INFINITY, next = -INFINITY;
        if (lane < p.G)
            for (int j = 0; j < per; ++j) {
                const double v = scratch[lane * per + j];
                if (v > best) { next = best; best = v; }
                else if (v > next) next = v;
            }
        double g = p.top2 && next > -INFINITY ? best + next : best;
        unsigned kept = 0;
        for (int j = 0; j < p.topk_groups; ++j) {
            double v = g;
            int gi = lane;
            warp_best(v, gi);
            if (!(v > -INFINITY)) break;
            kept |= 1u << gi;
            if (lane == gi) g = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane + 32 * i;
            if (e < p.E && !((kept >> (e / per)) & 1u)) c[i] = -INFINITY;
            else if (!p.bias) c[i] = l[i];
        }
    }
    my_e = -1;
    double my_l = -INFINITY;
    for (int j = 0; j < p.k; ++j) {
        double v = -INFINITY;
        int e = lane;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (c[i] > v) { v = c[i]; e = lane + 32 * i; }
        warp_best(v, e);
        if (!(v > -INFINITY)) break;
        double pl = 0.0;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (e == lane + 32 * i) { c[i] = -INFINITY; pl = l[i]; }
        pl = __shfl_sync(0xffffffffu, pl, e & 31);
        if (lane == j) { my_e = e; my_l = pl; }
    }
    double w = 0.0;
    if (p.renormalise) {
        double top = warp_max64(my_l);
        if (p.score != SCORE_SOFTMAX) top = fmin(top, 0.0);
        if (my_e >= 0) w = relative_score64(p.score, my_l, top);
        const double sum = warp_sum(w);
        if (my_e >= 0) w = w / sum;
    } else if (my_e >= 0) {
        w = score64(p.score, my_l, m, inv_sum);
    }
    my_w = (float)(w * (double)p.scale);
}

// Positions of one block's pairs, given the first position of each expert's pairs of this
// block (base) and the block's token masks.
__device__ __forceinline__ void scored_scatter(const ScoredArgs &p, int t0, int nt, const int *base, const uint32_t *mask) {
    const int W = p.TB / 32;
    for (int i = threadIdx.x; i < nt * p.k; i += blockDim.x) {
        const int tl = i / p.k, j = i - tl * p.k;
        const size_t pair = (size_t)t0 * p.k + i;
        const int e = p.topk_idx[pair];
        int pos = -1;
        if (e >= 0) {
            pos = base[e];
            const uint32_t *me = mask + e * W;
            for (int w = 0; w < tl / 32; ++w) pos += __popc(me[w]);
            pos += __popc(me[tl / 32] & ((1u << (tl & 31)) - 1u));
            if (p.sorted_token) p.sorted_token[pos] = t0 + tl;
            if (p.sorted_slot) p.sorted_slot[pos] = j;
        }
        if (p.inv_pos) p.inv_pos[pair] = pos;
    }
}

// Top-k of TB tokens a block.  With one block the permutation follows at once; otherwise the
// block leaves its counts and masks to scored_permute_kernel.
template <int NPL>
__global__ void __launch_bounds__(32 * SR_WARPS) scored_topk_kernel(ScoredArgs p) {
    extern __shared__ __align__(16) uint8_t sr_smem[];
    double *scratch = reinterpret_cast<double *>(sr_smem);                       // [8][E], groups only
    uint32_t *mask = reinterpret_cast<uint32_t *>(scratch + (p.G > 1 ? SR_WARPS * p.E : 0));   // [E][TB / 32]
    int *base = reinterpret_cast<int *>(mask + p.E * (p.TB / 32));               // [E]
    __shared__ int part[SR_WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * p.TB, nt = min(p.TB, p.T - t0), W = p.TB / 32;
    for (int i = threadIdx.x; i < p.E * W; i += blockDim.x) mask[i] = 0;
    __syncthreads();
    for (int tl = warp; tl < nt; tl += SR_WARPS) {
        int e;
        float w;
        scored_token<NPL>(p, t0 + tl, scratch + (p.G > 1 ? warp * p.E : 0), e, w);
        if (lane < p.k) {
            const size_t pair = (size_t)(t0 + tl) * p.k + lane;
            p.topk_idx[pair] = e;
            p.topk_w[pair] = w;
            if (e >= 0) atomicOr(&mask[e * W + tl / 32], 1u << (tl & 31));
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        int n = 0;
        for (int w = 0; w < W; ++w) n += __popc(mask[e * W + w]);
        base[e] = n;
        if (p.NB > 1 && p.cnt) p.cnt[(size_t)blockIdx.x * p.E + e] = n;
    }
    if (p.NB > 1) {
        if (p.cnt)
            for (int i = threadIdx.x; i < p.E * W; i += blockDim.x) p.mask[(size_t)blockIdx.x * p.E * W + i] = mask[i];
        return;
    }
    __syncthreads();
    const int total = block_scan(base, p.E, part);
    if (p.offsets) {
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.offsets[e] = base[e];
        if (threadIdx.x == 0) p.offsets[p.E] = total;
    }
    scored_scatter(p, t0, nt, base, mask);
}

__global__ void __launch_bounds__(32 * SR_WARPS) scored_permute_kernel(ScoredArgs p) {
    extern __shared__ __align__(16) uint8_t sr_smem[];
    int *base = reinterpret_cast<int *>(sr_smem), *before = base + p.E;   // [E] each
    __shared__ int part[SR_WARPS];
    const int t0 = blockIdx.x * p.TB, nt = min(p.TB, p.T - t0), W = p.TB / 32;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        int all = 0, mine = 0;
        for (int b = 0; b < p.NB; ++b) {
            const int n = p.cnt[(size_t)b * p.E + e];
            if (b < blockIdx.x) mine += n;
            all += n;
        }
        base[e] = all;
        before[e] = mine;
    }
    __syncthreads();
    const int total = block_scan(base, p.E, part);
    if (p.offsets && blockIdx.x == 0) {
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.offsets[e] = base[e];
        if (threadIdx.x == 0) p.offsets[p.E] = total;
    }
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) base[e] += before[e];
    __syncthreads();
    scored_scatter(p, t0, nt, base, p.mask + (size_t)blockIdx.x * p.E * W);
}

}  // namespace ds4
