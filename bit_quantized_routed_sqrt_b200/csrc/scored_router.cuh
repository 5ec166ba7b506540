// scored_router.cuh -- routing from given logits: softmax, sigmoid or sqrt-softplus scores, a
// bias on the choice, groups, top-k, renormalised weights, and the token -> expert permutation.
//
// s = softmax(l), sigmoid(l) or sqrt(log(1 + e^l)); the choice goes by s + bias (without a bias by
// l, which orders alike), the weight is that of s.  A warp per token.  65536 tokens of 256 experts
// with a bias take 76 us for the choice and 87 with the permutation where their 78 MB take 12 at a
// copy's rate.  700 instructions a token (300 the scores, 160 the sort and the k picks, 120 the
// weights; 460 without a bias) are 39 us of issue.  In the rest, not measured apart: three blocks an
// SM are resident, so the last of 512 run in a second turn; registers spill (72 bytes stored a thread
// in this build, 136 for rows that are not aligned pieces); 31% of the warps' places are active.
// Scores in fp64 throughout took 520.  A single token takes 4.4 us of the GPU.
#pragma once
#include "combine.cuh"
#include "scan.cuh"

namespace ds4 {

constexpr int SR_MAX_TOPK = 32;
constexpr int SR_MAX_GROUPS = 32;
constexpr int SR_MIN_BLOCK = 32, SR_MAX_BLOCK = 256;     // tokens a CTA
constexpr int SR_WARPS = 8, SR_MAX_WARPS = 16;           // warps a CTA (up to 16 where there are at most 148 CTAs)
constexpr int SR_DIRECT = 256;                           // blocks whose counts every CTA adds up itself
constexpr int SR_PERMUTE_THREADS = 512;
// Dynamic shared memory that a launch may have without leave: 48 KB less what the kernel has
// beside it, 32 bytes that the compiler makes 1 KB of (with room for more of both).
constexpr int SR_PLAIN_SMEM = 44 * 1024;
// the most dynamic shared memory of one: values of every warp's experts (groups), masks and counts
constexpr int SR_MOST_SMEM = SR_MAX_WARPS * SR_MAX_EXPERTS * 8 + SR_MAX_EXPERTS * (SR_MAX_BLOCK / 32 + 1) * 4;

enum : int { SCORE_SOFTMAX = 0, SCORE_SIGMOID = 1, SCORE_SQRT_SOFTPLUS = 2 };

struct ScoredArgs {
    int E, k, score, G, topk_groups, top2, renormalise;
    float scale;
    const void *logits;
    int type;
    int64_t ld;
    int T, TB, NB;           // tokens, tokens a block (a power of two), blocks
    const float *bias;       // [E] or null
    int *topk_idx;           // [T][k]
    float *topk_w;
    int *offsets, *sorted_token, *sorted_slot, *inv_pos;   // each may be null
    int pitch;               // E rounded up to 4
    int *cnt;                // workspace [NB][pitch], 16-byte aligned
    uint32_t *mask;          // workspace [NB][E][words of TB bits]
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

// One token's exact values in fp64, by one warp; lane holds experts lane + 32 i.  Returns the mask
// of the groups that the token may choose from, and to each lane its experts' choice values
// (-inf: no candidate, or not in those groups).
template <int NPL>
__device__ __forceinline__ unsigned scored_values64(const ScoredArgs &p, int64_t t, double *scratch, double (&c)[NPL]) {
    const int lane = threadIdx.x & 31;
    double l[NPL];
    double m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        const float v = e < p.E ? load_typed(p.logits, p.type, t * p.ld + e) : -INFINITY;
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
    if (p.G == 1) return 1u;
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
            next = fmax(next, fmin(best, v));
            best = fmax(best, v);
        }
    const double g = p.top2 && next > -INFINITY ? best + next : best;
    int rank = 0;
    for (int h = 0; h < p.G; ++h) {
        const double o = __shfl_sync(0xffffffffu, g, h);
        rank += o > g || (o == g && h < lane);
    }
    const unsigned kept = __ballot_sync(0xffffffffu, g > -INFINITY && rank < p.topk_groups);
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        if (e < p.E && !((kept >> (e / per)) & 1u)) c[i] = -INFINITY;
        else if (!p.bias) c[i] = l[i];
    }
    return kept;
}

// The groups of one token, exactly: for scored_choice, where two groups are too close.
template <int NPL>
__device__ __noinline__ unsigned scored_groups64(const ScoredArgs &p, int64_t t, double *scratch) {
    double c[NPL];
    return scored_values64<NPL>(p, t, scratch, c);
}

// The choice of one token in fp64: to lane j < k the expert of slot j (-1: no candidate was
// left).  It runs where scored_choice and scored_rank cannot tell.
template <int NPL>
__device__ __noinline__ int scored_choice64(const ScoredArgs &p, int64_t t, double *scratch) {
    const int lane = threadIdx.x & 31;
    double c[NPL];
    scored_values64<NPL>(p, t, scratch, c);
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
// than 2 M and the cut; where some are closer, exact ties of fp32 logits among them, scored_rank
// orders all that may be among the first k by their fp64 values (scored_choice64 does the whole
// token where they are too many); where groups are too close, scored_groups64 chooses them.  Without a bias the values are the logits themselves: M is 0, and for fp16
// and bf16 logits the cut drops nothing, so nothing is left to decide.

constexpr uint32_t SR_LIVE = 0x00800000u;   // the lowest key of a finite value

// Bits that order as the values do, -0 below +0: where the two are a tie (logits; a score is not -0,
// nor its sum with a bias) 0 is added to the value first.
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
__device__ __forceinline__ float approx_exp(float x) {   // ex2.approx(x log2 e), below 2^-126 zero
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.442695041f));
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

// Sorts v descending (Batcher's odd-even merge sort).
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

// A token's logits in one lane: experts lane * NPL + i where a lane's are one aligned piece of
// the row (VEC: E = 32 NPL), otherwise lane + 32 i.
template <int NPL, class T, bool VEC>
struct LaneLogits {
    static constexpr int BYTES = NPL * (int)sizeof(T);
    static constexpr int WORDS = VEC ? (BYTES + 3) / 4 : 1;
    uint32_t w[WORDS];
    T v[VEC ? 1 : NPL];

    __device__ __forceinline__ static int expert(int lane, int i) { return VEC ? lane * NPL + i : lane + 32 * i; }
    __device__ __forceinline__ void load(const ScoredArgs &p, const T *logits, int64_t t) {
        const int lane = threadIdx.x & 31;
        const T *row = logits + t * p.ld;
        if constexpr (VEC) {
            const uint8_t *src = reinterpret_cast<const uint8_t *>(row) + lane * BYTES;
            if constexpr (BYTES % 16 == 0) {
#pragma unroll
                for (int i = 0; i < BYTES / 16; ++i) {
                    const uint4 u = ld_input(reinterpret_cast<const uint4 *>(src) + i);
                    w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
                }
            } else {
                const uint2 u = ld_input(reinterpret_cast<const uint2 *>(src));
                w[0] = u.x; w[1] = u.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (lane + 32 * i < p.E) v[i] = row[lane + 32 * i];
        }
    }
    // NaN and -inf: no candidate, -inf; +inf counts as the largest finite value.
    __device__ __forceinline__ float get(const ScoredArgs &p, int i) const {
        float x;
        if constexpr (VEC) {
            if constexpr (sizeof(T) == 4) x = __uint_as_float(w[i]);
            else {
                const uint16_t h = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
                x = to_f32<T>(*reinterpret_cast<const T *>(&h));
            }
        } else {
            x = (threadIdx.x & 31) + 32 * i < p.E ? to_f32<T>(v[i]) : -INFINITY;
        }
        return fminf(fmaxf(x, -INFINITY), 3.402823466e38f);   // fmaxf drops a NaN
    }
};

// Lane j < n holds candidate e (or -1): to lane j < k the j-th best of them by the exact choice
// values (fp64), ties to the lower expert.
template <int NPL, class T, bool VEC>
__device__ __noinline__ int scored_rank(const ScoredArgs &p, int64_t t, const LaneLogits<NPL, T, VEC> &logits, int e, int n) {
    const int lane = threadIdx.x & 31;
    const bool on = lane < n && e >= 0;
    double l = on ? (double)fminf(to_f32<T>(reinterpret_cast<const T *>(p.logits)[t * p.ld + e]), 3.402823466e38f) : -INFINITY;
    double v = l;
    if (p.bias) {   // otherwise ranked by the logits
        double m = 0.0, inv_sum = 0.0;
        if (p.score == SCORE_SOFTMAX) {
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < NPL; ++i) top = fmaxf(top, logits.get(p, i));
            m = (double)warp_max_f32(top);
            double sum = 0.0;
            for (int i = 0; i < NPL; ++i) sum += logits.get(p, i) > -INFINITY ? exp((double)logits.get(p, i) - m) : 0.0;
            inv_sum = 1.0 / warp_sum(sum);
        }
        if (on) v = score64(p.score, l, m, inv_sum) + (double)p.bias[e];
    }
    int rank = 0;
    for (int h = 0; h < n; ++h) {
        const double ov = __shfl_sync(0xffffffffu, v, h);
        const int oe = __shfl_sync(0xffffffffu, on ? e : -1, h);
        rank += oe >= 0 && (ov > v || (ov == v && oe < e));
    }
    int got = -1;
    for (int h = 0; h < n; ++h) {
        const int r = __shfl_sync(0xffffffffu, on ? rank : -1, h), oe = __shfl_sync(0xffffffffu, e, h);
        if (r == lane) got = oe;
    }
    return lane < p.k ? got : -1;
}

// The choice of one token by one warp: to lane j < k the expert of slot j, or -1.  bias: the
// lane's experts' (0 without one, -inf for a NaN); bias_size: the largest magnitude of all.
template <int NPL, class T, bool VEC>
__device__ __forceinline__ int scored_choice(const ScoredArgs &p, int64_t t, const LaneLogits<NPL, T, VEC> &logits,
                                             const float (&bias)[NPL], float bias_size, double *scratch) {
    using L = LaneLogits<NPL, T, VEC>;
    constexpr uint32_t LOW = NPL <= 8 ? 255u : 511u;   // room for the index
    const int lane = threadIdx.x & 31;
    const bool by_score = p.bias || (p.G > 1 && p.top2);
    float a[NPL], M = 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) a[i] = logits.get(p, i);
    if (by_score) {
        // M: each score is off by at most (4 + |x|) 2^-22 of itself, x the exponential's argument
        // (ex2.approx 2^-22, its argument's rounding 1.5 |x| 2^-24, reciprocal and root 2^-23
        // each, the series' roundings 2^-22; a root halves what comes before it), 4 more where a
        // sum of 512 is in it (13 additions, its terms' errors, its reciprocal), and the sum with
        // the bias is off by 2^-24; below e^-87 the exponentials may be flushed to 0, a score (a
        // root) of up to 1.3e-19.  Score times (4 or 8 + |x|) grows with the logit, whichever the
        // score, so the largest logit's bounds every expert's.
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NPL; ++i) top = fmaxf(top, a[i]);
        top = fmaxf(warp_max_f32(top), -3.402823466e38f);
        float most, off;   // the largest score, and it times (4 or 8 + |x|)
        auto take = [&](int i, float s) { a[i] = a[i] > -INFINITY ? s + bias[i] : -INFINITY; };
        // (one loop for each score: a test inside the loop costs as much as a score)
        if (p.score == SCORE_SOFTMAX) {
            float sum = 0.0f, e[NPL];
#pragma unroll
            for (int i = 0; i < NPL; ++i) sum += e[i] = approx_exp(a[i] - top);   // of -inf: 0
            most = approx_rcp(warp_sum(sum));
            off = 8.0f * most;
#pragma unroll
            for (int i = 0; i < NPL; ++i) take(i, e[i] * most);
        } else if (p.score == SCORE_SIGMOID) {
            auto score = [](float l) { return approx_rcp(1.0f + approx_exp(-l)); };
            most = score(top);
            off = most * (4.0f + fabsf(top));
#pragma unroll
            for (int i = 0; i < NPL; ++i) take(i, score(a[i]));
        } else {
            auto score = [](float l) {
                const float ex = approx_exp(-fabsf(l));
                return approx_sqrt(fmaxf(l, 0.0f) + log1p_unit(ex, approx_rcp(2.0f + ex)));
            };
            most = score(top);
            off = most * (4.0f + fabsf(top));
#pragma unroll
            for (int i = 0; i < NPL; ++i) take(i, score(a[i]));
        }
        M = fmaf(off, 2.384185791e-7f, fmaf(most + bias_size, 1.192092896e-7f, 2e-19f));
    } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) a[i] += 0.0f;   // -0 and +0 are equal logits
    }
    uint32_t key[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i)
        key[i] = (order_key(a[i]) & ~LOW) | (LOW - (uint32_t)L::expert(lane, i));   // of -inf: below SR_LIVE
    if (p.G > 1) {
        // group values by lane, from the experts' values in shared memory (padded: no conflicts)
        const int per = p.E / p.G;
        float *v = reinterpret_cast<float *>(scratch);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (L::expert(lane, i) < p.E) v[L::expert(lane, i) + (L::expert(lane, i) >> 5)] = a[i];
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
        unsigned kept = __ballot_sync(0xffffffffu, in);
        if (by_score) {
            const float least = -warp_max_f32(in ? -g : -INFINITY);
            const float left = warp_max_f32(!in ? g : -INFINITY);
            if (left > -INFINITY && !(least - left > 4.0f * M + 2.4e-7f * (fabsf(least) + fabsf(left))))
                kept = scored_groups64<NPL>(p, t, scratch);
        }
        const float inv = 1.0f / (float)per;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            // (e + 1/2) / per is at least 1/2 / 512 from a whole number: the product's rounding cannot cross it
            const int of = (int)(((float)L::expert(lane, i) + 0.5f) * inv);
            if (!((kept >> (of & 31)) & 1u)) key[i] = 0u;
            else if (!p.bias && by_score && key[i] >= SR_LIVE)   // ranked by the logit, chosen groups by their scores
                key[i] = (order_key(logits.get(p, i) + 0.0f) & ~LOW) | (LOW - (uint32_t)L::expert(lane, i));
        }
        if (!p.bias) M = 0.0f;
    }
    sort_network<NPL>(key);
    auto pop = [&]() {   // the best key left, taken out
        const uint32_t best = __reduce_max_sync(0xffffffffu, key[0]);
        const bool had = key[0] == best;
#pragma unroll
        for (int i = 0; i + 1 < NPL; ++i) key[i] = had ? key[i + 1] : key[i];
        key[NPL - 1] = had ? 0u : key[NPL - 1];
        return best;
    };
    uint32_t mine = 0, last = 0;
    for (int j = 0; j < p.k; ++j) {
        const uint32_t best = pop();
        if (lane == j) mine = best;
    }
    if (p.bias || sizeof(T) == 4) {
        last = __reduce_max_sync(0xffffffffu, key[0]);
        uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1);
        if (lane == p.k - 1) next = last;
        // the value is at least what its key's upper bits say, the next one below their successor
        const float low = order_value(mine & ~LOW), high = order_value((next & ~LOW) + LOW + 1u);
        if (!__all_sync(0xffffffffu, lane >= p.k || next < SR_LIVE || low - high >= 2.0f * M)) {
            // Every expert that may be among the first k, one a lane, by its exact value.
            const float least = __shfl_sync(0xffffffffu, low, p.k - 1);   // the k-th is not below this less M
            int n = p.k;
            for (; last >= SR_LIVE && !(least - order_value((last & ~LOW) + LOW + 1u) >= 2.0f * M); ++n) {
                if (n == 32) return scored_choice64<NPL>(p, t, scratch);
                if (lane == n) mine = last;
                pop();
                last = __reduce_max_sync(0xffffffffu, key[0]);
            }
            return scored_rank<NPL, T, VEC>(p, t, logits, mine >= SR_LIVE ? (int)(LOW - (mine & LOW)) : -1, n);
        }
    }
    return lane < p.k && mine >= SR_LIVE ? (int)(LOW - (mine & LOW)) : -1;
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
// In half steps of fp32 (expf and each approximate function 2, a quotient by __fdividef 4) a softmax
// score is off by at most 4, a sigmoid score 11, a sqrt-softplus score 14; the weight by that, what
// the sum has (the same and 5 for up to 32 terms), the quotient's 4 and the scale's 1: 38 at most.
template <int NPL, class T, bool VEC>
__device__ __forceinline__ float scored_weight(const ScoredArgs &p, int64_t t, const LaneLogits<NPL, T, VEC> &logits, int e) {
    const bool on = e >= 0;
    const float l = on ? fminf(to_f32<T>(reinterpret_cast<const T *>(p.logits)[t * p.ld + e]), 3.402823466e38f) : -INFINITY;
    float m = 0.0f;
    double sum = 0.0;
    if (p.score == SCORE_SOFTMAX && !p.renormalise) {
        // the denominator takes every expert
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NPL; ++i) m = fmaxf(m, logits.get(p, i));
        m = warp_max_f32(m);
#pragma unroll
        for (int i = 0; i < NPL; ++i) sum += logits.get(p, i) > -INFINITY ? (double)expf(logits.get(p, i) - m) : 0.0;
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
            if (p.score == SCORE_SIGMOID) {
                w = __fdividef(l >= 0.0f ? 1.0f : exp_diff(l, m, 1.0f), 1.0f + ex);
            } else {
                const float lp = log1p_unit(ex, approx_rcp(2.0f + ex));
                if (l >= 0.0f) w = approx_sqrt(l + lp);
                else w = exp_diff(l, m, 0.5f) * (ex > 1e-30f ? approx_sqrt(__fdividef(lp, ex)) : 1.0f);
            }
        }
    }
    if (p.renormalise) w = __fdividef(w, warp_sum(w));
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
            const uint32_t *me = mask + e * (p.TB / 32);
            for (int w = 0; w < tl / 32; ++w) pos += __popc(me[w]);
            pos += __popc(me[tl / 32] & ((1u << (tl & 31)) - 1u));
            if (p.sorted_token) p.sorted_token[pos] = t0 + tl;
            if (p.sorted_slot) p.sorted_slot[pos] = j;
        }
        if (p.inv_pos) p.inv_pos[pair] = pos;
    }
}

// Top-k of TB tokens a block.  With one block the permutation follows at once; otherwise the
// block leaves its counts and masks to the kernels below.  The next token's logits are loaded
// before the present one is chosen from.
template <int NPL, class T, bool VEC, bool LONE>
__global__ void __launch_bounds__(32 * (LONE ? SR_MAX_WARPS : SR_WARPS), LONE || NPL > 8 ? 1 : 3) scored_topk_kernel(const __grid_constant__ ScoredArgs p) {
    next_kernel_may_start();
    wait_for_kernel_before();
    extern __shared__ __align__(16) uint8_t sr_smem[];
    const int warps = blockDim.x >> 5, W = p.TB / 32;
    double *scratch = reinterpret_cast<double *>(sr_smem);                       // [warps][32 NPL], groups only
    uint32_t *mask = reinterpret_cast<uint32_t *>(scratch + (p.G > 1 ? warps * 32 * NPL : 0));   // [E][W]
    int *base = reinterpret_cast<int *>(mask + p.E * W);                         // [E]
    __shared__ int part[SCAN_THREADS / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * p.TB, nt = min(p.TB, p.T - t0);
    LaneLogits<NPL, T, VEC> now, next;
    const T *logits = after_wait(reinterpret_cast<const T *>(p.logits));
    if (warp < nt) next.load(p, logits, t0 + warp);
    float bias[NPL], bias_size = 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = LaneLogits<NPL, T, VEC>::expert(lane, i);
        bias[i] = p.bias && e < p.E ? fmaxf(p.bias[e], -INFINITY) : 0.0f;   // fmaxf drops a NaN
        if (bias[i] > -INFINITY) bias_size = fmaxf(bias_size, fabsf(bias[i]));
    }
    bias_size = warp_max_f32(bias_size);
    for (int i = threadIdx.x; i < p.E * W; i += blockDim.x) mask[i] = 0;
    __syncthreads();
    for (int tl = warp; tl < nt; tl += warps) {
        now = next;
        if (tl + warps < nt) next.load(p, logits, t0 + tl + warps);
        const int e = scored_choice<NPL, T, VEC>(p, t0 + tl, now, bias, bias_size, scratch + (p.G > 1 ? warp * 32 * NPL : 0));
        const float w = scored_weight<NPL, T, VEC>(p, t0 + tl, now, e);
        if (lane < p.k) {
            const size_t pair = (size_t)(t0 + tl) * p.k + lane;
            p.topk_idx[pair] = e;
            p.topk_w[pair] = w;
            if (e >= 0) atomicOr(&mask[e * W + tl / 32], 1u << (tl & 31));
        }
    }
    if (p.NB > 1 && !p.cnt) return;   // no permutation
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        int n = 0;
        for (int w = 0; w < W; ++w) n += __popc(mask[e * W + w]);
        base[e] = n;
        if (p.NB > 1) p.cnt[(size_t)blockIdx.x * p.pitch + e] = n;
    }
    if (p.NB > 1) {
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

// Counts of the blocks -> the counts before each block, in place, and the totals.  A CTA has 32
// experts, one a lane; its warps take runs of blocks.
__global__ void __launch_bounds__(1024) scored_scan_kernel(const __grid_constant__ ScoredArgs p) {
    next_kernel_may_start();
    wait_for_kernel_before();
    __shared__ int sums[32][33];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.x * 32 + lane;
    const bool on = e < p.E;
    int carry = 0;
    for (int b0 = 0; b0 < p.NB; b0 += 512) {
        const int each = (min(p.NB - b0, 512) + 31) / 32, first = b0 + warp * each;
        int v[16], sum = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = on && i < each && first + i < p.NB ? p.cnt[(size_t)(first + i) * p.pitch + e] : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum += v[i];
        sums[warp][lane] = sum;
        __syncthreads();
        int at = carry, all = 0;
#pragma unroll
        for (int w = 0; w < 32; ++w) {
            const int n = sums[w][lane];
            at += w < warp ? n : 0;
            all += n;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (on && i < each && first + i < p.NB) p.cnt[(size_t)(first + i) * p.pitch + e] = at;
            at += v[i];
        }
        carry += all;
        __syncthreads();
    }
    if (on && warp == 0) p.total[e] = carry;
}

// Offsets and the places of one block's pairs.  scanned: cnt and total are those of
// scored_scan_kernel; otherwise cnt holds the blocks' own counts, which every CTA adds up: four
// experts a thread, the blocks dealt out to the strips of threads that the experts leave.
__global__ void __launch_bounds__(SR_PERMUTE_THREADS) scored_permute_kernel(const __grid_constant__ ScoredArgs p, int scanned) {
    next_kernel_may_start();
    wait_for_kernel_before();
    extern __shared__ __align__(16) uint8_t sr_smem[];
    const int W = p.TB / 32, fours = p.pitch / 4, strips = SR_PERMUTE_THREADS / fours;
    int *base = reinterpret_cast<int *>(sr_smem), *before = base + p.pitch;   // [pitch] each
    int *sums = before + p.pitch;                                             // [2][strips][pitch]
    uint32_t *mask = reinterpret_cast<uint32_t *>(sums + (scanned ? 0 : 2 * strips * p.pitch));   // [E][W]
    __shared__ int part[SCAN_THREADS / 32];
    const int t0 = blockIdx.x * p.TB, nt = min(p.TB, p.T - t0);
    for (int i = threadIdx.x; i < p.E * W; i += blockDim.x) mask[i] = p.mask[(size_t)blockIdx.x * p.E * W + i];
    if (scanned) {
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
            base[e] = p.total[e];
            before[e] = p.cnt[(size_t)blockIdx.x * p.pitch + e];
        }
    } else {
        const int strip = threadIdx.x / fours, f = threadIdx.x - strip * fours;
        if (strip < strips) {
            int4 all = make_int4(0, 0, 0, 0), mine = make_int4(0, 0, 0, 0);
#pragma unroll 8
            for (int b = strip; b < p.NB; b += strips) {
                const int4 n = *reinterpret_cast<const int4 *>(p.cnt + (size_t)b * p.pitch + 4 * f);
                all.x += n.x; all.y += n.y; all.z += n.z; all.w += n.w;
                if (b < blockIdx.x) { mine.x += n.x; mine.y += n.y; mine.z += n.z; mine.w += n.w; }
            }
            *reinterpret_cast<int4 *>(sums + strip * p.pitch + 4 * f) = all;
            *reinterpret_cast<int4 *>(sums + (strips + strip) * p.pitch + 4 * f) = mine;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
            int a = 0, m = 0;
            for (int i = 0; i < strips; ++i) {
                a += sums[i * p.pitch + e];
                m += sums[(strips + i) * p.pitch + e];
            }
            base[e] = a;
            before[e] = m;
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
