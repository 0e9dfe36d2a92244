// Routing by scores and the gradient of its weights.
//   s_e = sigmoid(l_e), or softmax over all of a token's experts
//   c_e = s_e + bias_e                                     decides who is chosen
//   groups of E / n_group consecutive experts: the sum of their group_top
//   (1 or 2) largest c; only the topk_group best groups are kept
//   chosen: the top_k largest c; w_j = scale s_j, or scale s_j / sum of the chosen s
//
// One wave routes one token: the choice is top_k + 1 dependent reductions, and a
// reduction over 64 lanes by DPP and scalar registers costs what one over 16 does.
// What bounds it: instructions, at few tokens their latency.  Measured: 16 tokens
// of 256 experts in 8 groups 6.6 us (decided in 64 bits throughout 13.9), 8192
// tokens of 288 experts, softmax with a bias, 16.3 (25.5): 13 and the about 20
// tokens that FP32 does not decide, whose waves end last.  That is with a bias that
// differs from expert to expert.  Where equal logits give equal choice scores (a bias
// of zeros, or group sums without a bias) FP32 does not decide those tokens either:
// of BF16 logits of that spread 37% have a tie among their nine largest, and the
// same call takes 21.3 us (FP16: 5%, 18.7; FP32: none, 16.1).  Without bias and sums
// logits are compared, and ties are decided: 11.3.  Reading the logits (4.7 MB)
// takes 1.
#include <algorithm>

#include "common.h"
#include "router.h"
#include "tiles.h"
#include "wave.h"

namespace moe {

namespace {

template <int DT>
__device__ __forceinline__ float load_logit(const void *p, int64_t i) {
    if constexpr (DT == kDtF32) return static_cast<const float *>(p)[i];
    else if constexpr (DT == kDtF16) return (float)static_cast<const _Float16 *>(p)[i];
    else return bf16_bits_to_f32(static_cast<const uint16_t *>(p)[i]);
}

template <int DT>
__device__ __forceinline__ void store_grad(void *p, int64_t i, float v) {
    if constexpr (DT == kDtF32) static_cast<float *>(p)[i] = v;
    else if constexpr (DT == kDtF16) static_cast<_Float16 *>(p)[i] = (_Float16)v;
    else static_cast<uint16_t *>(p)[i] = (uint16_t)f32_to_bf16_bits(v);
}

// FP64 -> uint64 with the same order; -0 and +0 are one value.
__device__ __forceinline__ uint64_t ordered64(double d) {
    const uint64_t u = (uint64_t)__double_as_longlong(d + 0.0);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
    return v;
}

// A logit that can be chosen: neither NaN nor -infinity.  (+infinity counts as
// the largest finite value, so that a softmax stays defined.)
__device__ __forceinline__ bool usable(float l) { return l > -INFINITY; }
__device__ __forceinline__ float finite(float l) { return fminf(l, 3.402823466e38f); }

__device__ __forceinline__ double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }

// ------------------------------------------------------------------ forward

// Lane layout: a group's experts lie with 2^sh lanes; lane p of group g holds
// experts g n + p, g n + p + 2^sh, ... (n experts a group).
struct Lanes {
    int n, g, p, sh;
    __device__ __forceinline__ int expert(int i) const { return g * n + p + (i << sh); }
    __device__ __forceinline__ bool holds(int i) const { return p + (i << sh) < n; }
};

template <int CTRL>
__device__ __forceinline__ uint64_t dpp64(uint64_t v) {
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, 0xF, 0xF, false);
    return (uint64_t)hi << 32 | (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

// Chooses in 64 bits: lane r < top_k gets the expert of rank r (-1: none is
// left).  mx: the largest logit.
template <int NPL>
__device__ __forceinline__ int choose64(const ScoreArgs &a, const Lanes &ln, const float (&l)[NPL],
                                        const float (&bias)[NPL], float mx) {
    const int lane = threadIdx.x & 63;
    const bool soft = a.score == kScoreSoftmax;
    double s[NPL], total = 0.0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        s[i] = exp(soft ? (double)l[i] - (double)mx : -(double)l[i]);      // (no branches: one chain beside the other)
        total += s[i];
    }
    if (soft) total = wave_sum(total);
    uint64_t key[NPL];                           // 0: not to be chosen
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const double c = (soft ? s[i] : 1.0) / (soft ? total : 1.0 + s[i]) + (double)bias[i];
        key[i] = usable(l[i]) && c > -INFINITY ? ordered64(c) : 0;
    }
    auto value = [](uint64_t k) {
        return __longlong_as_double((long long)((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
    };
    if (a.topk_group < a.n_group) {
        uint64_t b1 = 0, b2 = 0;                 // the two largest of the group
        auto merge = [&](uint64_t o1, uint64_t o2) {
            const uint64_t lo = b1 < o1 ? b1 : o1, hi = b1 < o1 ? o1 : b1, two = b2 < o2 ? o2 : b2;
            b1 = hi;
            b2 = lo < two ? two : lo;
        };
#pragma unroll
        for (int i = 0; i < NPL; ++i) merge(key[i], 0);
        if (ln.sh > 0) merge(dpp64<0xB1>(b1), dpp64<0xB1>(b2));       // quad [1,0,3,2]
        if (ln.sh > 1) merge(dpp64<0x4E>(b1), dpp64<0x4E>(b2));       // quad [2,3,0,1]
        if (ln.sh > 2) merge(dpp64<0x141>(b1), dpp64<0x141>(b2));     // half-row mirror
        if (ln.sh > 3) merge(dpp64<0x140>(b1), dpp64<0x140>(b2));     // row mirror
        for (int d = 16; d < 1 << ln.sh; d <<= 1) {
            const uint64_t o1 = __shfl_xor(b1, d, 64), o2 = __shfl_xor(b2, d, 64);
            merge(o1, o2);
        }
        uint64_t sc = 0;
        if (b1) sc = a.group_top == 2 && b2 ? ordered64(value(b1) + value(b2)) : b1;
        int rank = 0;
        for (int h = 0; h < a.n_group; ++h) {
            const uint64_t o = (uint64_t)__builtin_amdgcn_readlane((uint32_t)(sc >> 32), h << ln.sh) << 32 |
                               (uint32_t)__builtin_amdgcn_readlane((uint32_t)sc, h << ln.sh);
            rank += o > sc || (o == sc && h < ln.g);
        }
        if (rank >= a.topk_group) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) key[i] = 0;
        }
    }
    int sel = -1;
    for (int r = 0; r < a.top_k; ++r) {
        uint64_t bk = key[0];
        int bi = 0;                              // of equals the first
#pragma unroll
        for (int i = 1; i < NPL; ++i) {
            bi = key[i] > bk ? i : bi;
            bk = key[i] > bk ? key[i] : bk;
        }
        // the largest high halves, of those the largest low halves, of those the
        // lowest expert
        const uint32_t hi = (uint32_t)(bk >> 32), top = wave_max_u32(hi);
        if (top == 0) break;                     // nobody is left
        uint64_t who = __ballot(hi == top);
        if (who & (who - 1)) {
            const uint32_t lo = hi == top ? (uint32_t)bk : 0u, low = wave_max_u32(lo);
            who = __ballot(hi == top && lo == low);
        }
        const int be = ln.expert(bi);
        if (who & (who - 1)) {
            const uint32_t first = wave_min_u32((who >> lane) & 1 ? (uint32_t)be : 0xFFFFFFFFu);
            who = __ballot(((who >> lane) & 1) && (uint32_t)be == first);
        }
        const int w = __builtin_ctzll(who);
        const int e = __builtin_amdgcn_readlane(be, w);
        if (lane == r) sel = e;
        const int out = lane == w ? bi : -1;
#pragma unroll
        for (int i = 0; i < NPL; ++i) key[i] = i == out ? 0 : key[i];
    }
    return sel;
}

__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// The two largest of a group's values in every lane of the group (v1 >= v2 are
// the lane's own): in rows of 16 lanes by DPP, beyond by permutes.
__device__ __forceinline__ void group_top2(float &v1, float &v2, int sh) {
    auto merge = [&](float o1, float o2) {
        const float lo = fminf(v1, o1);
        v1 = fmaxf(v1, o1);
        v2 = fmaxf(lo, fmaxf(v2, o2));
    };
#define MOE_TOP2(ctrl)                                                                                          \
    merge(__uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v1), ctrl, 0xF, 0xF, false)),          \
          __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v2), ctrl, 0xF, 0xF, false)))
    if (sh > 0) MOE_TOP2(0xB1);                  // quad [1,0,3,2]
    if (sh > 1) MOE_TOP2(0x4E);                  // quad [2,3,0,1]
    if (sh > 2) MOE_TOP2(0x141);                 // half-row mirror
    if (sh > 3) MOE_TOP2(0x140);                 // row mirror
#undef MOE_TOP2
    for (int d = 16; d < 1 << sh; d <<= 1) {
        const float o1 = __shfl_xor(v1, d, 64), o2 = __shfl_xor(v2, d, 64);
        merge(o1, o2);
    }
}

// The same choice in FP32 where it is sure to be the one in 64 bits; `sure` says
// whether it is.  Two cases:
//   plain  no bias and no sums of scores: larger logits have larger scores, so the
//          logits themselves are compared.  Sure if the logits lie where 64 bits
//          tell the scores of different ones apart ([-700, 20], and a softmax's
//          within 700 of the largest) and those compared are equal or 2^-40 apart.
//   else   choice scores in FP32.  A sigmoid is off by less than 8 * 2^-24 of itself
//          (its exponent is exact; exp, sum and quotient), a softmax's score by
//          less than (D + NPL + 16) 2^-24 (the exponent, up to D, is rounded; NPL + 6
//          additions of the denominator), the sum with the bias by 2^-24 more of the
//          result, and a score is at most |c| + |bias|.  Sure if those compared are
//          further apart than both errors (a group's score has two of each).
// Compared are neighbours in the ranking, the last one chosen and the best one
// not chosen, and the worst group kept and the best one not kept.
template <int NPL>
__device__ __forceinline__ int choose32(const ScoreArgs &a, const Lanes &ln, const float (&l)[NPL],
                                        const float (&bias)[NPL], float mx, bool &sure) {
    const int lane = threadIdx.x & 63;
    const bool grouped = a.topk_group < a.n_group;
    const bool plain = !a.bias && !(grouped && a.group_top == 2);
    const bool soft = a.score == kScoreSoftmax;
    float c[NPL], bmax = 0.f, tol = 0x1p-20f;
    sure = true;
    float low = 0.f;                             // the smallest usable logit
    if (plain || soft) {
        low = INFINITY;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (usable(l[i])) low = fminf(low, l[i]);
        low = unordered(wave_min_u32(ordered_bits(low)));
    }
    if (plain) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) c[i] = l[i];
        // (nobody usable: mx = -inf)
        sure = soft ? mx - low < 700.f || mx == -INFINITY : mx <= 20.f && low >= -700.f;
    } else {
        float inv = 0.f;
        float e[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            e[i] = usable(l[i]) ? (soft ? expf(l[i] - mx) : 1.0f / (1.0f + expf(-l[i]))) : 0.f;
        if (soft) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) sum += e[i];
            inv = 1.0f / wave_sum(sum);
            tol = (fminf(mx - low, 104.f) + (float)(NPL + 16)) * 0x1p-23f;
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            c[i] = -INFINITY;
            if (!usable(l[i])) continue;
            c[i] = (soft ? e[i] * inv : e[i]) + bias[i];
            if (!(c[i] > -INFINITY)) c[i] = -INFINITY;
            else bmax = fmaxf(bmax, fabsf(bias[i]));
        }
        bmax = unordered(wave_max_u32(ordered_bits(bmax)));
        // (an infinite bias: bmax = inf, nothing is sure)
        sure = bmax < INFINITY;
    }
    auto apart = [&](float hi, float lo, float biases) {     // hi >= lo; a negative one is at most its biases
        const float gap = hi - lo;
        return plain ? gap == 0.f || gap >= 0x1p-40f : gap > tol * (fabsf(hi) + biases * bmax) + 0x1p-120f;
    };
    if (grouped) {
        float v1 = -INFINITY, v2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            v2 = fmaxf(v2, fminf(v1, c[i]));
            v1 = fmaxf(v1, c[i]);
        }
        group_top2(v1, v2, ln.sh);
        const float sc = a.group_top == 2 && v2 > -INFINITY ? v1 + v2 : v1;
        int rank = 0;
        for (int h = 0; h < a.n_group; ++h) {
            const float o = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sc), h << ln.sh));
            rank += o > sc || (o == sc && h < ln.g);
        }
        const bool there = ln.g < a.n_group, kept = rank < a.topk_group;
        const float worst = unordered(wave_min_u32(ordered_bits(there && kept ? sc : INFINITY)));
        const float best = unordered(wave_max_u32(ordered_bits(there && !kept ? sc : -INFINITY)));
        if (best > -INFINITY) sure = sure && apart(worst, best, 4.f);
        if (!kept) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) c[i] = -INFINITY;
        }
    }
    if (!sure) return -1;
    uint32_t key[NPL];                           // 0: not to be chosen
#pragma unroll
    for (int i = 0; i < NPL; ++i) key[i] = c[i] > -INFINITY ? ordered_bits(c[i] + 0.0f) : 0u;
    int sel = -1, n = 0;                         // ranks with an expert, one past the last chosen among them
    float v = 0.f;                               // the value of the lane's rank
    for (int r = 0; r <= a.top_k; ++r) {
        uint32_t bk = key[0];
        int bi = 0;                              // of equals the first
#pragma unroll
        for (int i = 1; i < NPL; ++i) {
            bi = key[i] > bk ? i : bi;
            bk = max(bk, key[i]);
        }
        const uint32_t top = wave_max_u32(bk);
        if (top == 0) break;
        n = r + 1;
        if (lane == r) v = unordered(top);
        if (r == a.top_k) break;
        const int be = ln.expert(bi);
        uint64_t who = __ballot(bk == top);
        if (who & (who - 1)) {
            if (!plain) {                        // equal scores
                sure = false;
                break;
            }
            const uint32_t first = wave_min_u32(bk == top ? (uint32_t)be : 0xFFFFFFFFu);
            who = __ballot(bk == top && (uint32_t)be == first);
        }
        const int w = __builtin_ctzll(who);
        const int e = __builtin_amdgcn_readlane(be, w);
        if (lane == r) sel = e;
        const int out = lane == w ? bi : -1;
#pragma unroll
        for (int i = 0; i < NPL; ++i) key[i] = i == out ? 0u : key[i];
    }
    // all neighbours at once
    const float below = __shfl_down(v, 1, 64);
    if (__ballot(lane + 1 < n && !apart(v, below, 2.f))) sure = false;
    return sel;
}

template <int DT, int NPL>
__global__ void __launch_bounds__(256)
route_scored_kernel(ScoreArgs a, int sh) {
    __shared__ int chosen[4][32];
    __shared__ float most[4];
    __shared__ double totals[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, kk = a.top_k + a.n_shared;
    {
        const int64_t t = (int64_t)blockIdx.x * 4 + wave;
        const Lanes ln = {a.E / a.n_group, lane >> sh, lane & ((1 << sh) - 1), sh};
        float l[NPL], bias[NPL];
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const bool there = ln.g < a.n_group && ln.holds(i);
            l[i] = there && t < a.M ? load_logit<DT>(a.logits, t * a.ld + ln.expert(i)) : -INFINITY;
            bias[i] = there && a.bias ? a.bias[ln.expert(i)] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            l[i] = usable(l[i]) ? finite(l[i]) : -INFINITY;
            mx = fmaxf(mx, l[i]);
        }
        mx = unordered(wave_max_u32(ordered_bits(mx)));
        double total = 0.0;
        if (a.score == kScoreSoftmax && !a.renorm) {         // (renormalised weights need no denominator)
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (usable(l[i])) total += exp((double)l[i] - (double)mx);
            total = wave_sum(total);
        }
        bool sure;
        int sel = choose32(a, ln, l, bias, mx, sure);
        if (!sure) sel = choose64(a, ln, l, bias, mx);
        if (lane < 32) chosen[wave][lane] = lane < a.top_k ? sel : -1;
        if (lane == 0) {
            most[wave] = mx;
            totals[wave] = total;
        }
        if (t < a.M && lane < a.top_k) a.ids[t * kk + lane] = sel;
        else if (t < a.M && lane < kk) {         // the shared expert
            a.ids[t * kk + lane] = a.E;
            a.w[t * kk + lane] = 1.0f;
        }
    }
    // The weights of all four tokens at once, 16 or 32 lanes a token: lane j of
    // them holds slot j.  (In every wave for its own token they took 1.4 of 17.4 us for 8192 tokens.)
    __syncthreads();
    const int width = a.top_k <= 16 ? 16 : 32, q = (int)threadIdx.x / width, j = lane & (width - 1);
    if (wave * 64 >= 4 * width) return;
    const int64_t t = (int64_t)blockIdx.x * 4 + q;
    const int sel = chosen[q][j];
    double s = 0.0;
    const float ls = sel >= 0 ? finite(load_logit<DT>(a.logits, t * a.ld + sel)) : -INFINITY;
    if (a.renorm) {
        // up to a factor that renormalising takes out, so that not all underflow
        uint32_t bits = row_max_u32(ordered_bits(ls));
        if (width == 32) bits = max(bits, (uint32_t)__shfl_xor((int)bits, 16, 64));
        const float top = unordered(bits);
        const float m = a.score == kScoreSoftmax ? top : fminf(top, 0.f);
        if (sel >= 0)
            s = a.score == kScoreSoftmax ? exp((double)ls - (double)m)
                                         : 1.0 / (exp((double)m) + exp((double)m - (double)ls));
        double sum = s;                          // over the lanes that hold a slot
        for (int d = 1; d < a.top_k; d <<= 1) sum += __shfl_xor(sum, d, 64);
        s = sum > 0.0 ? s / sum : 0.0;
    } else if (sel >= 0) {
        s = a.score == kScoreSoftmax ? exp((double)ls - (double)most[q]) / totals[q] : sigmoid64(ls);
    }
    if (t < a.M && j < a.top_k) a.w[t * kk + j] = (float)(s * (double)a.scale);
}

// ----------------------------------------------------------------- backward

// With a_j = scale dL/dw_j for the token's slots j that hold an expert:
//   softmax                dl_e = p_e sum_f p_f (A_e - A_f) over all experts f, A_e = sum_{j: e_j = e} a_j:
//                          p_e (A_e sum_{f in no slot} p_f + sum_{f in a slot} p_f (A_e - A_f)) for one in a slot,
//                          -p_e sum_f p_f A_f for the others
//   softmax, renormalised  dl_e = sum_{j: e_j = e} p_j sum_{i: e_i != e} p_i (a_j - a_i), p over the slots
//   sigmoid                dl_e = sum_{j: e_j = e} s_j (1 - s_j) a_j
//   sigmoid, renormalised  ... with sum_{i: e_i != e} s_i (a_j - a_i) / S^2 in the place of a_j, S = sum s
//                          (the differences between slots of one expert cancel, and are left out)
// (1 - s is the sigmoid of -l: no cancellation where s is near 1; the differences
// of a or A are taken first, and the p of experts in no slot added up, not taken from
// 1: none where one expert holds nearly the whole sum, and a single slot's gradient
// is 0 with renormalised weights.)
// One wave a token, for gradients that every logit has (2048 tokens of 512
// experts, BF16: 6.5 us, 4.2 MB, bound by its latency; without the differences 6.3)
// and for more than 16 slots.
template <int DT, int NPL>
__global__ void __launch_bounds__(256)
route_scored_bwd_kernel(ScoreArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= a.M) return;
    const int64_t row = t * a.ld;
    const bool dense = a.score == kScoreSoftmax && !a.renorm;
    // lane j holds slot j
    int id = -1;
    float av = 0.f;
    if (lane < a.slots) {
        id = a.ids[t * a.slots + lane];
        if (id < 0 || id >= a.E) id = -1;
        if (id >= 0) av = a.dw[t * a.slots + lane] * a.scale;
    }
    float ls = id >= 0 ? load_logit<DT>(a.logits, row + id) : -INFINITY;
    if (!usable(ls)) id = -1;                    // never chosen: weight 0, whatever its logit
    ls = id >= 0 ? finite(ls) : -INFINITY;
    if (id < 0) av = 0.f;
    auto value = [](float x, int j) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), j)); };
    auto apart = [&](float s) {                  // sum_{i: e_i != e_j} s_i (a_j - a_i)
        float sum = 0.f;
        for (int i = 0; i < a.slots; ++i) {
            const float si = value(s, i), ai = value(av, i);
            if (__builtin_amdgcn_readlane(id, i) != id) sum = fmaf(si, av - ai, sum);
        }
        return sum;
    };
    if (dense) {
        float p[NPL], mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane + 64 * i;
            p[i] = e < a.E ? load_logit<DT>(a.logits, row + e) : -INFINITY;
            p[i] = usable(p[i]) ? finite(p[i]) : -INFINITY;
            mx = fmaxf(mx, p[i]);
        }
        mx = wave_max(mx);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            p[i] = usable(p[i]) ? expf(p[i] - mx) : 0.f;
            sum += p[i];
        }
        sum = wave_sum(sum);
        const float inv = sum > 0.f ? 1.0f / sum : 0.f;
        // of the lane's slot: A, and p where it is the first one of its expert
        const float ps = id >= 0 ? expf(ls - mx) * inv : 0.f;
        float A = av, pf = ps, diff = 0.f;       // diff: sum_{f in a slot} p_f (A - A_f)
        int slot[NPL];                           // the last slot of the lane's experts
#pragma unroll
        for (int i = 0; i < NPL; ++i) slot[i] = -1;
        for (int j = 0; j < a.slots; ++j) {
            const int ej = __builtin_amdgcn_readlane(id, j);
            const float pj = value(pf, j), aj = value(A, j);
            if (ej != id) diff = fmaf(pj, A - aj, diff);
#pragma unroll
            for (int i = 0; i < NPL; ++i) slot[i] = lane + 64 * i == ej ? j : slot[i];
        }
        float rest = 0.f;                        // of the experts in no slot
        int listed = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            rest += slot[i] < 0 ? p[i] : 0.f;
            listed += __builtin_popcountll(__ballot(slot[i] >= 0));
        }
        rest = wave_sum(rest) * inv;
        if (listed < __builtin_popcountll(__ballot(id >= 0))) {        // an expert twice
            A = diff = 0.f;
            for (int j = 0; j < a.slots; ++j) {
                const float aj = value(av, j);
                if (__builtin_amdgcn_readlane(id, j) == id) {
                    A += aj;
                    if (j < lane) pf = 0.f;
                }
            }
            for (int j = 0; j < a.slots; ++j) {
                const float pj = value(pf, j), aj = value(A, j);
                if (__builtin_amdgcn_readlane(id, j) != id) diff = fmaf(pj, A - aj, diff);
            }
        }
        const float dot = wave_sum(pf * A);
        diff = fmaf(A, rest, diff);
        const float v = ps * diff;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane + 64 * i;
            const float of = __shfl(v, slot[i], 64);
            if (e < a.E) store_grad<DT>(a.dl, t * a.ld_dl + e, slot[i] < 0 ? -(p[i] * inv * dot) : of);
        }
        return;
    }
    float v;
    if (a.score == kScoreSoftmax) {
        const float m = wave_max(ls);
        const float ex = id >= 0 ? expf(ls - m) : 0.f;
        const float sum = wave_sum(ex);
        const float q = sum > 0.f ? ex / sum : 0.f;
        v = q * apart(q);
    } else {
        // renormalised: s up to a factor, which cancels, so that not all underflow
        const float m = a.renorm ? fminf(wave_max(ls), 0.f) : 0.f;
        const float s = id >= 0 ? 1.0f / (expf(m) + expf(m - ls)) : 0.f;
        const float rest = id >= 0 ? 1.0f / (1.0f + expf(ls)) : 0.f;
        if (a.renorm) {
            const float S = wave_sum(s);
            av = S > 0.f ? apart(s) / S / S : 0.f;
        }
        v = s * rest * av;
    }
    float d[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) d[i] = 0.f;
    for (int j = 0; j < a.slots; ++j) {
        const int ej = __builtin_amdgcn_readlane(id, j);
        const float vj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), j));
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (lane + 64 * i == ej) d[i] += vj;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane + 64 * i;
        if (e < a.E) store_grad<DT>(a.dl, t * a.ld_dl + e, d[i]);
    }
}

// The same for weights whose gradient is 0 outside the slots, up to 16 of them: a
// row of 16 lanes takes a token (its sums are DPP steps), a wave four.  The rows
// of d_logits are put together in LDS and stored 16 bytes a lane: it is their
// writing that bounds the kernel (16384 tokens of 256 experts, FP32, 16.8 MB: 6.5 us;
// one wave a token took 12.9).
constexpr int kRowWaves = 2;

// The sum over the lane's row of 16.
__device__ __forceinline__ float row_sum(float v) {
    v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0xB1, 0xF, 0xF, false));
    v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x4E, 0xF, 0xF, false));
    v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x141, 0xF, 0xF, false));
    v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x140, 0xF, 0xF, false));
    return v;
}

// The value of lane J of the lane's row.
template <int J>
__device__ __forceinline__ int row_lane(int v) {
    return __builtin_amdgcn_update_dpp(0, v, 0x150 + J, 0xF, 0xF, false);      // row broadcast
}
template <int J>
__device__ __forceinline__ float row_lane(float v) {
    return __uint_as_float(row_lane<J>((int)__float_as_uint(v)));
}

// n += the row's lanes from J on, up to lane 15, that hold the same expert
template <int J>
__device__ __forceinline__ void count_same(int id, int slots, int &n) {
    if constexpr (J < 16) {
        if (J < slots) {
            n += row_lane<J>(id) == id;
            count_same<J + 1>(id, slots, n);
        }
    }
}

// sum += s_i (a - a_i) over the row's lanes i from J on, up to lane 15; TWICE: that
// hold another expert
template <bool TWICE, int J = 0>
__device__ __forceinline__ void add_apart(int id, float s, float a, int slots, float &sum) {
    if constexpr (J < 16) {
        if (J < slots) {
            const int ej = TWICE ? row_lane<J>(id) : -1;
            const float more = fmaf(row_lane<J>(s), a - row_lane<J>(a), sum);
            sum = TWICE && ej == id ? sum : more;
            add_apart<TWICE, J + 1>(id, s, a, slots, sum);
        }
    }
}

// s += v of row lane J where that holds the same expert; up to lane 15
template <int J>
__device__ __forceinline__ void add_same(int id, float v, int slots, float &s) {
    if constexpr (J < 16) {
        if (J < slots) {
            const int ej = row_lane<J>(id);
            const float vj = row_lane<J>(v);     // (in every lane, before the choice)
            s += ej == id ? vj : 0.f;
            add_same<J + 1>(id, v, slots, s);
        }
    }
}

typedef u32x4 u32x4_any __attribute__((aligned(2)));

template <int DT>
__global__ void __launch_bounds__(64 * kRowWaves)
route_scored_bwd_rows_kernel(ScoreArgs a, int pitch) {
    extern __shared__ __attribute__((aligned(16))) float rows[];      // [4 kRowWaves][pitch], pitch >= E, a multiple of 8
    const int lane = threadIdx.x & 63, j = lane & 15;
    const int64_t t0 = ((int64_t)blockIdx.x * kRowWaves + (threadIdx.x >> 6)) * 4, t = t0 + (lane >> 4);
    float *const mine = rows + (threadIdx.x >> 6) * 4 * pitch;
    for (int i = lane * 4; i < 4 * pitch; i += 256) *reinterpret_cast<v4f *>(mine + i) = v4f{0.f, 0.f, 0.f, 0.f};
    int id = -1;
    float av = 0.f, ls = -INFINITY;
    if (t < a.M && j < a.slots) {
        id = a.ids[t * a.slots + j];
        av = a.dw[t * a.slots + j] * a.scale;
        if (id < 0 || id >= a.E) id = -1;
        if (id >= 0) ls = load_logit<DT>(a.logits, t * a.ld + id);
    }
    // whether a token of the wave lists an expert twice (while the logits arrive)
    int same = 0;
    count_same<0>(id, a.slots, same);
    const bool twice = __ballot(id >= 0 && same > 1) != 0;
    if (!usable(ls)) id = -1;                    // never chosen: weight 0, whatever its logit
    ls = id >= 0 ? finite(ls) : -INFINITY;
    if (id < 0) av = 0.f;
    auto apart = [&](float s) {
        float d = 0.f;
        if (twice) add_apart<true>(id, s, av, a.slots, d);
        else add_apart<false>(id, s, av, a.slots, d);
        return d;
    };
    const float top = unordered(row_max_u32(ordered_bits(ls)));
    float v;
    if (a.score == kScoreSoftmax) {
        const float ex = id >= 0 ? expf(ls - top) : 0.f;
        const float sum = row_sum(ex);
        const float q = sum > 0.f ? ex / sum : 0.f;
        v = q * apart(q);
    } else {
        // renormalised: s up to a factor, which cancels, so that not all underflow
        const float m = a.renorm ? fminf(top, 0.f) : 0.f;
        const float s = id >= 0 ? 1.0f / (expf(m) + expf(m - ls)) : 0.f;
        const float rest = id >= 0 ? 1.0f / (1.0f + expf(ls)) : 0.f;
        if (a.renorm) {
            const float S = row_sum(s);
            av = S > 0.f ? apart(s) / S / S : 0.f;
        }
        v = s * rest * av;
    }
    float d = v;
    if (twice) {                                 // both lanes hold the same sum
        d = 0.f;
        add_same<0>(id, v, a.slots, d);
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);          // the zeros are written
    __builtin_amdgcn_wave_barrier();
    if (id >= 0) mine[(lane >> 4) * pitch + id] = d;
    __builtin_amdgcn_wave_barrier();
    constexpr int per = DT == kDtF32 ? 4 : 8;    // values of a 16-byte store
    for (int r = 0; r < 4 && t0 + r < a.M; ++r)
        for (int e = lane * per; e < a.E; e += 64 * per) {
            const float *p = mine + r * pitch + e;
            const int64_t at = (t0 + r) * a.ld_dl + e;
            if (e + per <= a.E) {
                u32x4 o;
                if constexpr (DT == kDtF32) {
                    o = *reinterpret_cast<const u32x4 *>(p);
                    *reinterpret_cast<u32x4_any *>(static_cast<float *>(a.dl) + at) = o;
                } else {
                    float f[8];
                    for (int i = 0; i < 8; ++i) f[i] = p[i];
                    o = narrow8<DT == kDtF16>(f);
                    *reinterpret_cast<u32x4_any *>(static_cast<uint16_t *>(a.dl) + at) = o;
                }
            } else {
                for (int i = 0; e + i < a.E; ++i) store_grad<DT>(a.dl, at + i, p[i]);
            }
        }
}

template <int DT, int NPL>
hipError_t launch_fwd(const ScoreArgs &a, int sh, hipStream_t st) {
    route_scored_kernel<DT, NPL><<<(unsigned)((a.M + 3) / 4), 256, 0, st>>>(a, sh);
    return hipGetLastError();
}
template <int DT, int NPL>
hipError_t launch_bwd(const ScoreArgs &a, hipStream_t st) {
    route_scored_bwd_kernel<DT, NPL><<<(unsigned)((a.M + 3) / 4), 256, 0, st>>>(a);
    return hipGetLastError();
}

template <int DT>
hipError_t fwd(const ScoreArgs &a, hipStream_t st) {
    int sh = 6;                                  // log2 of a group's lanes
    while (sh > 0 && (a.n_group << sh) > 64) --sh;
    const int n = a.E / a.n_group, npl = (n + (1 << sh) - 1) >> sh;
    // Experts of a lane, rounded up to a width with code.  Powers of two, and 5: what
    // one group of 257 to 320 experts takes (8192 tokens of 288, FP32 logits, 14.8 us,
    // in code for 8 18.0; of 320 16.2, 20.1).  8192 tokens of 384 and 512 experts in
    // one group (8) take 20.2 and 20.9, of 576 and 1024 (16) 33.5 and 35.6, of 1024 in
    // 32 groups (16) 58; more than 16 only where the number of groups is no power of
    // two and lanes are left over (1023 in 33 groups, a lane each: 105).
    if (npl <= 2) return launch_fwd<DT, 2>(a, sh, st);
    if (npl <= 4) return launch_fwd<DT, 4>(a, sh, st);
    if (npl <= 5) return launch_fwd<DT, 5>(a, sh, st);
    if (npl <= 8) return launch_fwd<DT, 8>(a, sh, st);
    if (npl <= 16) return launch_fwd<DT, 16>(a, sh, st);
    return launch_fwd<DT, 32>(a, sh, st);
}
template <int DT>
hipError_t bwd(const ScoreArgs &a, hipStream_t st) {
    if (!(a.score == kScoreSoftmax && !a.renorm) && a.slots <= 16) {
        const int pitch = (a.E + 7) / 8 * 8;
        const int64_t wgs = (a.M + 4 * kRowWaves - 1) / (4 * kRowWaves);
        route_scored_bwd_rows_kernel<DT><<<(unsigned)wgs, 64 * kRowWaves, (size_t)pitch * 16 * kRowWaves, st>>>(a, pitch);
        return hipGetLastError();
    }
    if (a.E <= 128) return launch_bwd<DT, 2>(a, st);
    if (a.E <= 256) return launch_bwd<DT, 4>(a, st);
    if (a.E <= 512) return launch_bwd<DT, 8>(a, st);
    return launch_bwd<DT, 16>(a, st);
}

}  // namespace

namespace {

// A launch counts its threads in 32 bits: at most 2^25 tokens each.
template <typename F>
hipError_t in_parts(ScoreArgs a, F launch) {
    const int64_t M = a.M, part = (int64_t)1 << 25, size = a.dtype == kDtF32 ? 4 : 2;
    const int64_t slots = a.slots ? a.slots : a.top_k + a.n_shared;
    for (int64_t t = 0; t < M; t += part) {
        a.M = std::min(part, M - t);
        const hipError_t e = launch(a);
        if (e != hipSuccess) return e;
        a.logits = static_cast<const uint8_t *>(a.logits) + part * a.ld * size;
        a.ids += part * slots;
        if (a.w) a.w += part * slots;
        if (a.dw) a.dw += part * slots;
        if (a.dl) a.dl = static_cast<uint8_t *>(a.dl) + part * a.ld_dl * size;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_route_scored(const ScoreArgs &a, hipStream_t st) {
    return in_parts(a, [st](const ScoreArgs &p) {
        return p.dtype == kDtF32 ? fwd<kDtF32>(p, st) : p.dtype == kDtF16 ? fwd<kDtF16>(p, st) : fwd<kDtBf16>(p, st);
    });
}
hipError_t launch_route_scored_bwd(const ScoreArgs &a, hipStream_t st) {
    return in_parts(a, [st](const ScoreArgs &p) {
        return p.dtype == kDtF32 ? bwd<kDtF32>(p, st) : p.dtype == kDtF16 ? bwd<kDtF16>(p, st) : bwd<kDtBf16>(p, st);
    });
}

}  // namespace moe
