// scored_router.cuh -- routing from given logits: softmax, sigmoid or sqrt-softplus scores, a
// bias on the choice, groups, top-k, renormalised weights, and the token -> expert permutation.
#pragma once
#include "combine.cuh"
#include "scan.cuh"

namespace ds4 {

constexpr int SR_MAX_TOPK = 32;
constexpr int SR_MAX_GROUPS = 32;
constexpr int SR_BLOCK = 64, SR_WORDS = SR_BLOCK / 32;   // tokens a CTA
constexpr int SR_WARPS = 8, SR_MAX_WARPS = 16;           // warps a CTA (a lone CTA: up to 16)
constexpr int SR_DIRECT = 64;                            // blocks whose counts every CTA adds up itself

enum : int { SCORE_SOFTMAX = 0, SCORE_SIGMOID = 1, SCORE_SQRT_SOFTPLUS = 2 };

struct ScoredArgs {
    int E, k, score, G, topk_groups, top2, renormalise;
    float scale;
    const void *logits;
    int type;
    int64_t ld;
    int T, NB;               // tokens, blocks
    const float *bias;       // [E] or null
    int *topk_idx;           // [T][k]
    float *topk_w;
    int *offsets, *sorted_token, *sorted_slot, *inv_pos;   // each may be null
    int *cnt;                // workspace [NB][E]
    uint32_t *mask;          // workspace [NB][E][SR_WORDS]
    int *total;              // workspace [E]
};

// Score of a logit in fp64; m and inv_sum are the softmax's maximum and 1 / sum.
__device__ __forceinline__ double score64(int kind, double l, double m, double inv_sum) {
    if (kind == SCORE_SOFTMAX) return exp(l - m) * inv_sum;
    if (kind == SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
    return sqrt(fmax(l, 0.0) + log1p(exp(-fabs(l))));
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

// The choice of one token in fp64, by one warp; lane holds experts lane + 32 i.  Returns to
// lane j < k the expert of slot j (-1: no candidate was left).  About 3000 instructions a
// token at 256 experts: it runs where scored_choice finds two values too close.
template <int NPL>
__device__ __noinline__ int scored_choice64(const ScoredArgs &p, int64_t t, double *scratch) {
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
    if (p.score == SCORE_SOFTMAX && by_score) {
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
    int my_e = -1;
    for (int j = 0; j < p.k; ++j) {
        double v = -INFINITY;
        int e = lane;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (c[i] > v) { v = c[i]; e = lane + 32 * i; }
        warp_best(v, e);
        if (!(v > -INFINITY)) break;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (e == lane + 32 * i) c[i] = -INFINITY;
        if (lane == j) my_e = e;
    }
    return my_e;
}

// ------------------------------------------------------------------ the choice in fp32
// An approximate choice value a_i of every expert with a bound M on its distance from the
// exact one, as a 32-bit key: the ordered bits of a_i, cut to make room for the expert's index
// (larger for the lower index), so that keys are unique and one integer maximum finds the best
// expert with its tie rule.  Each lane sorts its keys (a network of integer minima and maxima);
// a slot is then one warp maximum over the lanes' heads and a shift in the lane that had it.
// The order is certain where neighbours (the first expert left out among them) differ by more
// than 2 M and the cut; anything closer, exact ties of fp32 logits among it, is decided by
// scored_choice64.  Without a bias the values are the logits themselves: M is 0, and for fp16
// and bf16 logits the cut drops nothing, so nothing is left to decide.

__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) { return __uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k); }
__device__ __forceinline__ float warp_max_f32(float v) { return order_value(__reduce_max_sync(0xffffffffu, order_key(v))); }

__device__ __forceinline__ float approx_rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float approx_sqrt(float x) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// log(1 + t), 0 <= t <= 1, as 2 atanh(z) = 2 (z + z^3/3 + ...), z = t / (2 + t) <= 1/3: the series
// to z^13 is short of it by less than 2e-8 of it; rounding and the reciprocal add some 2^-22.
__device__ __forceinline__ float log1p_unit(float t, float rcp_2_t) {
    const float z = t * rcp_2_t, q = z * z;
    float s = fmaf(q, 1.0f / 13, 1.0f / 11);
    s = fmaf(s, q, 1.0f / 9);
    s = fmaf(s, q, 1.0f / 7);
    s = fmaf(s, q, 1.0f / 5);
    s = fmaf(s, q, 1.0f / 3);
    return 2.0f * fmaf(s * q, z, z);
}

// Sorts v descending (odd-even merges).
template <int N>
__device__ __forceinline__ void sort_network(uint32_t (&v)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t a = v[i + j], b = v[i + j + k];
                        v[i + j] = max(a, b);
                        v[i + j + k] = min(a, b);
                    }
}

// The choice of one token by one warp: to lane j < k the expert of slot j, or -1.
template <int NPL>
__device__ __forceinline__ int scored_choice(const ScoredArgs &p, int64_t t, double *scratch) {
    constexpr uint32_t LOW = NPL <= 8 ? 255u : 511u;   // room for the index
    const int lane = threadIdx.x & 31;
    const bool by_score = p.bias || (p.G > 1 && p.top2);
    float l[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < p.E ? load_typed(p.logits, p.type, t * p.ld + e) : -INFINITY;
    }
    float a[NPL], M = 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) a[i] = l[i] > -INFINITY ? fminf(l[i], 3.402823466e38f) : -INFINITY;   // NaN: out
    if (by_score) {
        // M: each score is off by at most (16 + |x|) 2^-22 of itself, x the exponential's
        // argument (ex2.approx 2^-22, its argument's rounding 1.5 |x| 2^-24, reciprocal, root,
        // series and sum less than 2^-21 together), the sum with the bias by 2^-24; below
        // e^-87 the exponentials may be flushed to 0, a score (a root) of up to 1.3e-19.
        float off = 0.0f, size = 0.0f, top = 0.0f, scale = 1.0f;
        if (p.score == SCORE_SOFTMAX) {
            top = -INFINITY;
#pragma unroll
            for (int i = 0; i < NPL; ++i) top = fmaxf(top, a[i]);
            top = warp_max_f32(top);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) sum += a[i] > -INFINITY ? __expf(a[i] - top) : 0.0f;
            scale = approx_rcp(warp_sum(sum));
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            if (!(a[i] > -INFINITY)) continue;
            const float x = p.score == SCORE_SOFTMAX ? a[i] - top : p.score == SCORE_SIGMOID ? -a[i] : -fabsf(a[i]);
            const float ex = __expf(x);
            float s;
            if (p.score == SCORE_SOFTMAX) s = ex * scale;
            else if (p.score == SCORE_SIGMOID) s = approx_rcp(1.0f + ex);
            else s = approx_sqrt(fmaxf(a[i], 0.0f) + log1p_unit(ex, approx_rcp(2.0f + ex)));
            off = fmaxf(off, s * (16.0f + fminf(fabsf(x), 1e4f)));
            if (p.bias) s += p.bias[lane + 32 * i];
            a[i] = s > -INFINITY ? s : -INFINITY;
            size = fmaxf(size, fabsf(s));   // of a NaN: not taken
        }
        M = warp_max_f32(fmaf(off, 2.384185791e-7f, fmaf(size, 1.192092896e-7f, 2e-19f)));
    }
    bool sure = true;
    uint32_t key[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i)
        key[i] = a[i] > -INFINITY ? (order_key(a[i]) & ~LOW) | (LOW - (uint32_t)(lane + 32 * i)) : 0u;
    if (p.G > 1) {
        // group values by lane, from the experts' values in shared memory (padded: no conflicts)
        const int per = p.E / p.G;
        float *v = reinterpret_cast<float *>(scratch);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (lane + 32 * i < p.E) v[33 * i + lane] = a[i];
        __syncwarp();
        float best = -INFINITY, next = -INFINITY;
        if (lane < p.G) {
            int at = lane * per;
            for (int j = 0; j < per; ++j, ++at) {
                const float x = v[at + (at >> 5)];
                next = fmaxf(next, fminf(best, x));
                best = fmaxf(best, x);
            }
        }
        const float g = p.top2 && next > -INFINITY ? best + next : best;
        int rank = 0;
        for (int h = 0; h < p.G; ++h) {
            const float o = __shfl_sync(0xffffffffu, g, h);
            rank += o > g || (o == g && h < lane);
        }
        const bool in = g > -INFINITY && rank < p.topk_groups;
        const unsigned kept = __ballot_sync(0xffffffffu, in);
        if (by_score) {
            const float least = -warp_max_f32(in ? -g : -INFINITY);
            const float left = warp_max_f32(!in ? g : -INFINITY);
            sure = !(left > -INFINITY) || least - left > 4.0f * M + 2.4e-7f * (fabsf(least) + fabsf(left));
        }
        const float inv = 1.0f / (float)per;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            // (e + 1/2) / per is at least 1/2 / 512 from a whole number: the product's rounding cannot cross it
            const int of = (int)(((float)(lane + 32 * i) + 0.5f) * inv);
            if (!((kept >> of) & 1u)) key[i] = 0u;
            else if (!p.bias && by_score && key[i])   // ranked by the logit, chosen groups by their scores
                key[i] = (order_key(fminf(l[i], 3.402823466e38f)) & ~LOW) | (LOW - (uint32_t)(lane + 32 * i));
        }
        if (!p.bias) M = 0.0f;
    }
    sort_network<NPL>(key);
    uint32_t mine = 0, last = 0;
    for (int j = 0; j <= p.k; ++j) {
        const uint32_t best = __reduce_max_sync(0xffffffffu, key[0]);
        if (j == p.k) { last = best; break; }
        if (lane == j) mine = best;
        if (key[0] == best) {
#pragma unroll
            for (int i = 0; i + 1 < NPL; ++i) key[i] = key[i + 1];
            key[NPL - 1] = 0u;
        }
    }
    if (p.bias || p.type == DT_F32) {
        uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1);
        if (lane == p.k - 1) next = last;
        // the value is at least what its key's upper bits say, the next one below their successor
        const float low = order_value(mine & ~LOW), high = order_value((next & ~LOW) + LOW + 1u);
        sure = __all_sync(0xffffffffu, lane >= p.k || next == 0u || low - high >= 2.0f * M) && sure;
    }
    if (!sure) return scored_choice64<NPL>(p, t, scratch);
    return lane < p.k && mine ? (int)(LOW - (mine & LOW)) : -1;
}

// x - y and what its rounding left.
__device__ __forceinline__ float exact_diff(float x, float y, float &rest) {
    const float d = x - y, b = d - x;
    rest = (x - (d - b)) - (y + b);
    return d;
}
__device__ __forceinline__ float exp_diff(float x, float y, float half) {   // exp(half (x - y))
    float rest;
    const float d = exact_diff(x, y, rest);
    return half * d > -200.0f ? expf(half * d) * (1.0f + half * rest) : 0.0f;   // far below any sum (and d may be -inf)
}

// Weights of the chosen experts: lane j < k has slot j's expert (or -1) and gets its weight.
// Renormalised, scores count up to a factor common to the token, exp(-m) (sqrt-softplus:
// exp(-m / 2)) with m the largest chosen logit (softmax) or that where it is negative and 0
// elsewhere: tokens whose scores all underflow have weights too.
template <int NPL>
__device__ __forceinline__ float scored_weight(const ScoredArgs &p, int64_t t, int e) {
    const int lane = threadIdx.x & 31;
    const bool on = e >= 0;
    const float l = on ? fminf(load_typed(p.logits, p.type, t * p.ld + e), 3.402823466e38f) : -INFINITY;
    float m = 0.0f;
    double sum = 0.0;
    if (p.score == SCORE_SOFTMAX && !p.renormalise) {
        // the denominator takes every expert
        float v[NPL];
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int o = lane + 32 * i;
            const float x = o < p.E ? load_typed(p.logits, p.type, t * p.ld + o) : -INFINITY;
            v[i] = x > -INFINITY ? fminf(x, 3.402823466e38f) : -INFINITY;
            m = fmaxf(m, v[i]);
        }
        m = warp_max_f32(m);
#pragma unroll
        for (int i = 0; i < NPL; ++i) sum += v[i] > -INFINITY ? (double)expf(v[i] - m) : 0.0;
        sum = warp_sum(sum);
    } else if (p.renormalise) {
        m = warp_max_f32(l);
        if (p.score != SCORE_SOFTMAX) m = fminf(m, 0.0f);
    }
    float w = 0.0f;
    if (on) {
        if (p.score == SCORE_SOFTMAX) {
            w = exp_diff(l, m, 1.0f);
        } else {
            const float ex = expf(-fabsf(l));
            if (p.score == SCORE_SIGMOID) w = (l >= 0.0f ? 1.0f : exp_diff(l, m, 1.0f)) / (1.0f + ex);
            else if (l >= 0.0f) w = sqrtf(l + log1p_unit(ex, 1.0f / (2.0f + ex)));
            else w = exp_diff(l, m, 0.5f) * (ex > 1e-30f ? sqrtf(log1p_unit(ex, 1.0f / (2.0f + ex)) / ex) : 1.0f);
        }
    }
    if (p.renormalise) w = w / warp_sum(w);
    else if (p.score == SCORE_SOFTMAX) w = (float)((double)w / sum);
    return on ? w * p.scale : 0.0f;
}

// Positions of one block's pairs, given the first position of each expert's pairs of this
// block (base) and the block's token masks.
__device__ __forceinline__ void scored_scatter(const ScoredArgs &p, int t0, int nt, const int *base, const uint32_t *mask) {
    for (int i = threadIdx.x; i < nt * p.k; i += blockDim.x) {
        const int tl = i / p.k, j = i - tl * p.k;
        const size_t pair = (size_t)t0 * p.k + i;
        const int e = p.topk_idx[pair];
        int pos = -1;
        if (e >= 0) {
            pos = base[e];
            const uint32_t *me = mask + e * SR_WORDS;
            for (int w = 0; w < tl / 32; ++w) pos += __popc(me[w]);
            pos += __popc(me[tl / 32] & ((1u << (tl & 31)) - 1u));
            if (p.sorted_token) p.sorted_token[pos] = t0 + tl;
            if (p.sorted_slot) p.sorted_slot[pos] = j;
        }
        if (p.inv_pos) p.inv_pos[pair] = pos;
    }
}

// Top-k of SR_BLOCK tokens a block.  With one block the permutation follows at once; otherwise
// the block leaves its counts and masks to the kernels below.
template <int NPL>
__global__ void __launch_bounds__(32 * SR_MAX_WARPS) scored_topk_kernel(const __grid_constant__ ScoredArgs p) {
    extern __shared__ __align__(16) uint8_t sr_smem[];
    const int warps = blockDim.x >> 5;
    double *scratch = reinterpret_cast<double *>(sr_smem);                       // [warps][32 NPL], groups only
    uint32_t *mask = reinterpret_cast<uint32_t *>(scratch + (p.G > 1 ? warps * 32 * NPL : 0));   // [E][SR_WORDS]
    int *base = reinterpret_cast<int *>(mask + p.E * SR_WORDS);                  // [E]
    __shared__ int part[SCAN_THREADS / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * SR_BLOCK, nt = min(SR_BLOCK, p.T - t0);
    for (int i = threadIdx.x; i < p.E * SR_WORDS; i += blockDim.x) mask[i] = 0;
    __syncthreads();
    for (int tl = warp; tl < nt; tl += warps) {
        const int e = scored_choice<NPL>(p, t0 + tl, scratch + (p.G > 1 ? warp * 32 * NPL : 0));
        const float w = scored_weight<NPL>(p, t0 + tl, e);
        if (lane < p.k) {
            const size_t pair = (size_t)(t0 + tl) * p.k + lane;
            p.topk_idx[pair] = e;
            p.topk_w[pair] = w;
            if (e >= 0) atomicOr(&mask[e * SR_WORDS + tl / 32], 1u << (tl & 31));
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < SR_WORDS; ++w) n += __popc(mask[e * SR_WORDS + w]);
        base[e] = n;
        if (p.NB > 1 && p.cnt) p.cnt[(size_t)blockIdx.x * p.E + e] = n;
    }
    if (p.NB > 1) {
        if (p.cnt)
            for (int i = threadIdx.x; i < p.E * SR_WORDS; i += blockDim.x) p.mask[(size_t)blockIdx.x * p.E * SR_WORDS + i] = mask[i];
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

// Counts of the blocks -> the counts before each block, in place, and the totals.  A warp per
// expert, eight neighbours a CTA (they share the counts' 32-byte sectors), each lane a run of
// up to 32 blocks at a time.
__global__ void __launch_bounds__(256) scored_scan_kernel(const __grid_constant__ ScoredArgs p) {
    const int e = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (e >= p.E) return;
    int carry = 0;
    for (int b0 = 0; b0 < p.NB; b0 += 1024) {
        const int each = (min(p.NB - b0, 1024) + 31) / 32, first = b0 + lane * each;
        int v[32], sum = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = i < each && first + i < p.NB ? p.cnt[(size_t)(first + i) * p.E + e] : 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) sum += v[i];
        int before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += u;
        }
        const int all = __shfl_sync(0xffffffffu, before, 31);
        int at = carry + before - sum;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            if (i < each && first + i < p.NB) p.cnt[(size_t)(first + i) * p.E + e] = at;
            at += v[i];
        }
        carry += all;
    }
    if (lane == 0) p.total[e] = carry;
}

// Offsets and the places of one block's pairs.  scanned: cnt and total are those of
// scored_scan_kernel; otherwise cnt holds the blocks' own counts, which every CTA adds up.
__global__ void __launch_bounds__(SCAN_THREADS) scored_permute_kernel(const __grid_constant__ ScoredArgs p, int scanned) {
    extern __shared__ __align__(16) uint8_t sr_smem[];
    int *base = reinterpret_cast<int *>(sr_smem), *before = base + p.E;   // [E] each
    uint32_t *mask = reinterpret_cast<uint32_t *>(before + p.E);          // [E][SR_WORDS]
    __shared__ int part[SCAN_THREADS / 32];
    const int t0 = blockIdx.x * SR_BLOCK, nt = min(SR_BLOCK, p.T - t0);
    for (int i = threadIdx.x; i < p.E * SR_WORDS; i += blockDim.x) mask[i] = p.mask[(size_t)blockIdx.x * p.E * SR_WORDS + i];
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        if (scanned) {
            base[e] = p.total[e];
            before[e] = p.cnt[(size_t)blockIdx.x * p.E + e];
        } else {
            int all = 0, mine = 0;
#pragma unroll 16
            for (int b = 0; b < p.NB; ++b) {
                const int n = p.cnt[(size_t)b * p.E + e];
                mine += b < blockIdx.x ? n : 0;
                all += n;
            }
            base[e] = all;
            before[e] = mine;
        }
    }
    __syncthreads();
    const int total = block_scan(base, p.E, part);
    if (p.offsets && blockIdx.x == 0) {
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.offsets[e] = base[e];
        if (threadIdx.x == 0) p.offsets[p.E] = total;
    }
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) base[e] += before[e];
    __syncthreads();
    scored_scatter(p, t0, nt, base, mask);
}

}  // namespace ds4
