// Routing with scores: softmax or sigmoid of the router logits over all
// experts, a bias and groups for the choice, the k best, their weights, and
// the gradient of the logits (include/moe.h: moe_route_forward).  The layer's
// own routing, plain top-k of the logits, is k_topk_route; the pages feed it
// Gaussian logits (alphalab.site "Mixture-of-Kittens" sections 一 and 四).
#include <cfloat>

#include "common.h"
#include "launch.h"
#include "profile.h"
#include "rows.h"

namespace moe {

// ---------------------------------------------------------------- wave reductions
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
    return v;
}

// Between a wave's LDS accesses of which one lane's read what another's wrote: they are done in
// order, and the fences keep the compiler from carrying a lane's own values past this place.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ float no_nan(float v) { return v == v ? v : -INFINITY; }
__device__ __forceinline__ double no_nan(double v) { return v == v ? v : -(double)INFINITY; }

// exp(v - m) with m the largest of the v: 1 for the largest (infinite ones
// too), 0 for -inf (where all are)
__device__ __forceinline__ float soft_exp(float v, float m) {
    const float top = fmaxf(m, -FLT_MAX);
    return expf(v == top ? 0.f : v - top);
}
__device__ __forceinline__ double soft_exp(double v, double m) {
    return v == -(double)INFINITY ? 0.0 : v == m ? 1.0 : exp(v - m);
}

// ---------------------------------------------------------------- lanes of experts
// A wave per token.  Groups take lanes of their own: `per` lanes (a power of
// two, 64 / n_group or less) of EPL neighbouring experts each, so that a
// group's lanes meet in shuffles of a few steps and a lower lane (and in it a
// lower place) is a lower expert.
struct Lanes {
    int per;                  // lanes of a group
    int Eg;                   // experts of a group
};

template <int EPL>
__device__ __forceinline__ int first_expert(const Lanes& L, int n_group, int lane, int& count) {
    const int g = lane / L.per, in = (lane & (L.per - 1)) * EPL;
    count = g < n_group ? min(max(L.Eg - in, 0), EPL) : 0;
    return count > 0 ? g * L.Eg + in : 0;
}

// ================================================================ forward
// Whole numbers in the order of floats (-0 as 0, NaN as -inf), none of them 0
__device__ __forceinline__ uint32_t order(float v) {
    const int b = __float_as_int(v + 0.f);
    return (uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __int_as_float((int)(o ^ ((o & 0x80000000u) ? 0x80000000u : ~0u)));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_or0(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ uint32_t wave_most(uint32_t v) {
    v = max(v, dpp_or0<0x111, 0xf>(v));
    v = max(v, dpp_or0<0x112, 0xf>(v));
    v = max(v, dpp_or0<0x114, 0xf>(v));
    v = max(v, dpp_or0<0x118, 0xf>(v));
    v = max(v, dpp_or0<0x142, 0xa>(v));
    v = max(v, dpp_or0<0x143, 0xc>(v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// ---------------------------------------------------------------- where 32 bits do not tell
// The scores of a token in 64 bits
struct Exact {
    double m, z;
    __device__ __forceinline__ double operator()(const RouteArgs& a, const float* row, int e) const {
        const double v = no_nan(row[e]);
        const double s = a.score == SCORE_SIGMOID ? 1.0 / (1.0 + exp(-v)) : z > 0.0 ? soft_exp(v, m) / z : 0.0;
        return no_nan(s + (a.bias ? (double)a.bias[e] : 0.0));
    }
};

// The groups kept by their scores in 64 bits: whether this lane's is
__device__ __forceinline__ bool kept64(const RouteArgs& a, const Lanes& L, const Exact& exact, const float* row, int e0,
                                       int n, int lane) {
    double t1 = -(double)INFINITY, t2 = t1;
    for (int j = 0; j < n; ++j) {
        const double c = exact(a, row, e0 + j);
        t2 = fmax(t2, fmin(t1, c));
        t1 = fmax(t1, c);
    }
    for (int off = L.per >> 1; off >= 1; off >>= 1) {
        const double o1 = __shfl_xor(t1, off), o2 = __shfl_xor(t2, off);
        t2 = fmax(fmax(t2, o2), fmin(t1, o1));
        t1 = fmax(t1, o1);
    }
    const double score = a.group_top == 2 ? no_nan(t1 + t2) : t1;
    int better = 0;
    for (int g = 0; g < a.n_group; ++g) {
        const double o = __shfl(score, g * L.per);
        better += o > score || (o == score && g < lane / L.per);
    }
    return better < a.topk_group;
}

// The choice among the places of `key`, each c off by less than err + 2^-23 |c|: k rounds of
// the largest, and where others are as close to it as both errors, the largest of those in
// 64 bits, the lower index first.  kept: 1 or 0, or -1 where the groups are not sure either.
template <int EPL>
__device__ __forceinline__ int choose_close(const RouteArgs& a, const Lanes& L, const float* row, const uint32_t (&key)[EPL],
                                            float err, int e0, int n, int kept, int lane) {
    Exact exact{0.0, 0.0};
    if (a.score == SCORE_SOFTMAX) {
        float m = -INFINITY;
        for (int j = 0; j < n; ++j) m = fmaxf(m, no_nan(row[e0 + j]));
        exact.m = wave_most(m);
        for (int j = 0; j < n; ++j) exact.z += soft_exp((double)no_nan(row[e0 + j]), exact.m);
        exact.z = wave_sum(exact.z);
    }
    if (kept < 0) kept = kept64(a, L, exact, row, e0, n, lane);
    uint32_t open = !kept ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;       // the places still to be chosen
    int sel = 0;
    for (int r = 0; r < a.k; ++r) {
        uint32_t best = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) best = max(best, open >> j & 1u ? key[j] : 0u);
        best = wave_most(best);
        const float c = value_of(best);
        // (three errors: those of the others are a little larger, and the difference is rounded itself)
        const uint32_t thr = fabsf(c) < INFINITY ? order(c - 3.f * (err + 0x1p-23f * fabsf(c))) : best;
        uint32_t close = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) close |= (key[j] >= thr ? 1u : 0u) << j;
        close &= open;
        int at = close ? e0 + __builtin_ctz(close) : 0x7fffffff;
        const uint64_t who = __ballot(close != 0);
        if ((__ballot((close & (close - 1)) != 0) || (who & (who - 1))) && fabsf(c) < INFINITY) {
            double b = -(double)INFINITY;
            for (uint32_t left = close; left; left &= left - 1) {
                const double x = exact(a, row, e0 + __builtin_ctz(left));
                if (x > b) { b = x; at = e0 + __builtin_ctz(left); }
            }
            for (int off = 32; off >= 1; off >>= 1) {
                const double ob = __shfl_xor(b, off);
                const int oat = __shfl_xor(at, off);
                if (ob > b || (ob == b && oat < at)) { b = ob; at = oat; }
            }
        } else {
            at = lane_value(at, __builtin_ctzll(who));
        }
        if (n > 0 && at >= e0 && at < e0 + n) open &= ~(1u << (at - e0));
        if (lane == r) sel = at;
    }
    return sel;
}

// The choice is the one in 64 bits.  Without a bias (and sums of two in the groups) it is
// that of the logits, exactly.  Else c is computed in 32 bits, off by less than `err` for
// the score and 2^-23 |c| for the sum, and where two that the choice tells apart, neighbours among the k + 1
// best or a kept group's and another's, are closer than both errors, the token is done
// again in 64 bits (16384 x 512, sigmoid and bias: one token in a thousand).  In half steps
// of 1 (2^-24):
//   sigmoid: exp(-v) by exp2 is off by 1.5 |v| + 2 relative, the score by s (1 - s) times
//     that, below 0.5 + 0.5, and by 3 s from 1 + exp and the reciprocal; 8 are taken;
//   softmax: s (|v - m| + EPL + 16), 1 / z the largest s: |v - m| and 2 from the exponential, 2 and
//     at most 4.5 in z from those of all experts (the mean of |v - m| weighted by the scores, 4.44
//     at the most for 1024), EPL - 1 and 6 from its sum in a lane and over the wave, 2 from the
//     reciprocal and the product; s |v - m| <= 0.37 goes as 1;
//   both: the rounding of c, |c|; 2 |c| are taken.  (It is c's own size that counts, not the
//     largest of the biases: one of -10^9 or fp32's lowest, for an expert that is not to be
//     chosen, would leave no token sure, 235 us instead of 28 for 16384 x 512.)
//
// 34 MB are read once, yet the instructions bound it, 950 vector and 400 scalar ones a
// token (with sigmoid, bias and groups), of which ten rounds of the choice are 220 (16384 x 512:
// softmax 21 us, with sigmoid and bias 28, with 8 groups 32, with all scores out 32 by
// softmax; the bytes alone 5.5).  Rounds that look at all of a lane's keys each time and a choice
// in 64 bits from the start for the tokens that are not sure took 50, all in 64 bits 75:
// the second way's registers left four waves a SIMD instead of eight.  4 tokens take
// what a launch takes (10 us a call).
template <int EPL, bool SCORES>
__global__ __launch_bounds__(256) void k_route(RouteArgs a, Lanes L, bool vec) {
    const int lane = lane_id();
    int n;
    const int e0 = first_expert<EPL>(L, a.n_group, lane, n);
    const bool softmax = a.score == SCORE_SOFTMAX;
    const bool groups = a.n_group > 1, two = groups && a.group_top == 2;
    const bool by_logit = !a.bias && !two;
    const int64_t t = block_number() * 4 + wave_id();
    if (t >= a.T) return;
    const float* row = a.logits + t * a.E;
    // (vec: rows, groups and bias in whole chunks of four)
    auto load = [&](const float* p, float none, float (&to)[EPL]) {
        if (EPL % 4 == 0 && vec) {
#pragma unroll
            for (int j = 0; j + 3 < EPL; j += 4) {
                f32x4 q = {none, none, none, none};
                if (j < n) q = *(const f32x4*)(p + e0 + j);
#pragma unroll
                for (int i = 0; i < 4; ++i) to[j + i] = q[i];
            }
        } else {
#pragma unroll
            for (int j = 0; j < EPL; ++j) to[j] = j < n ? p[e0 + j] : none;
        }
    };
    float v[EPL], bias[EPL];
    load(row, -INFINITY, v);
    float m = -INFINITY;
    if (a.bias) {
        load(a.bias, 0.f, bias);
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) bias[j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) v[j] = no_nan(v[j]);
    float z = 0.f;
    if (softmax && (SCORES || !by_logit || !a.renorm)) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) m = fmaxf(m, v[j]);
        m = wave_most(m);
#pragma unroll
        for (int j = 0; j < EPL; ++j) z += soft_exp(v[j], m);
        z = wave_total(z);
    }
    const float rz = z > 0.f ? 1.f / z : 0.f;
    uint32_t key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        float c = v[j];
        if (SCORES || !by_logit) {
            float s;
            if (softmax) s = soft_exp(v[j], m) * rz;
            else if (SCORES) s = 1.f / (1.f + expf(-v[j]));
            else s = __builtin_amdgcn_rcpf(1.f + __expf(-v[j]));
            if (SCORES && j < n) a.scores[t * a.E + e0 + j] = s;
            if (!by_logit) c = no_nan(s + bias[j]);
        }
        key[j] = j < n ? order(c) : 0u;
    }
    const float err = softmax ? 0x1p-24f * (1.f + (EPL + 16) * rz) : 0x1p-21f;
    bool kept = true, sure = true;
    if (groups) {
        uint32_t t1 = 0, t2 = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            t2 = max(t2, min(t1, key[j]));
            t1 = max(t1, key[j]);
        }
        for (int off = L.per >> 1; off >= 1; off >>= 1) {
            const uint32_t o1 = __shfl_xor(t1, off), o2 = __shfl_xor(t2, off);
            t2 = max(max(t2, o2), min(t1, o1));
            t1 = max(t1, o1);
        }
        const bool mine = lane / L.per < a.n_group;
        const uint32_t score = !mine ? 0 : two ? order(no_nan(value_of(t1) + value_of(t2))) : t1;
        int better = 0;
        for (int g = 0; g < a.n_group; ++g) {
            const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)score, g * L.per);
            better += o > score || (o == score && g < lane / L.per);
        }
        kept = mine && better < a.topk_group;
        if (!by_logit && a.topk_group < a.n_group) {
            // the worst kept at its least and the best other at its most; of sums of two each
            // has its rounding, and the sum, which is no larger than both
            float size = fabsf(value_of(t1)), c = value_of(score);
            if (two) size = 2.f * (size + fabsf(value_of(t2)));
            size = size < INFINITY ? 0x1p-23f * size : 0.f;
            const float lo = value_of(~wave_most(kept ? ~order(c - size) : 0u));
            const float hi = value_of(wave_most(mine && !kept ? order(c + size) : 0u));
            sure = lo - hi > (two ? 4.f : 2.f) * err;      // (equal infinities: not sure)
        }
    }
    // Rounds of the wave's largest.  A lane has its two largest at hand and looks at its
    // keys again when both are taken: what is left of them comes after the last one taken.
    int sel = 0;                                           // lane r < k: the r-th choice
    const bool groups_sure = sure;
    if (sure) {
        uint32_t b1 = 0, b2 = 0;
        int e1 = 0, e2 = 0;
        auto largest_two = [&](uint32_t last, int e) {
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const bool after = (key[j] < last) | ((key[j] == last) & (e0 + j > e));
                const uint32_t c = after ? key[j] : 0u;
                const bool first = c > b1;
                e2 = first ? e1 : c > b2 ? e0 + j : e2;
                b2 = max(b2, min(b1, c));
                e1 = first ? e0 + j : e1;
                b1 = max(b1, c);
            }
        };
        if (kept) largest_two(~0u, 0);
        float above = INFINITY, gap = INFINITY;            // (infinite ones need no 64 bits: NaN, left out)
        for (int r = 0;; ++r) {
            const uint32_t most = wave_most(b1);
            if (!by_logit && most) {
                const float c = value_of(most);
                gap = fminf(gap, fmaf(-0x1p-22f, fmaxf(fabsf(above), fabsf(c)), above - c));
                above = c;
            }
            if (r == a.k) break;
            const int owner = __builtin_ctzll(__ballot(b1 == most));
            const int e = lane_value(e1, owner);
            if (lane == r) sel = e;
            if (lane == owner) {
                b1 = b2;
                e1 = e2;
                b2 = 0;
            }
            if (EPL > 2 && lane_value((int)b1, owner) == 0 && lane == owner) largest_two(most, e);
        }
        sure = gap > 2.f * err;
    }
    if (!by_logit && !sure) sel = choose_close<EPL>(a, L, row, key, err, e0, n, groups_sure ? kept : -1, lane);
    // the weights
    const bool in = lane < a.k;
    const float l = in ? no_nan(row[sel]) : -INFINITY;
    float p;
    if (a.renorm) {
        // only the ratios of the chosen matter: the scores relative to the largest of
        // them, so that none is lost where all are tiny
        const float ml = wave_most(l);
        if (softmax) p = soft_exp(l, ml);
        else {
            const float c = fminf(ml, 0.f);
            p = l == -INFINITY ? 0.f : l < 0.f ? expf(l - c) / (1.f + expf(l)) : expf(-c) / (1.f + expf(-l));
        }
        const float sum = wave_total(in ? p : 0.f);
        p = sum > 0.f ? p / sum : 0.f;
    } else {
        p = softmax ? soft_exp(l, m) * rz : 1.f / (1.f + expf(-l));
    }
    if (in) {
        a.idx[t * a.k + lane] = sel;
        a.w[t * a.k + lane] = a.scale * p;
    }
}

// ================================================================ backward
// With a_j the gradient of the weights times the score of choice j,
//   renorm: t_j = s_j / sum s, a_j = scale t_j (dw_j - sum_i t_i dw_i)   (they sum to 0)
//   else    a_j = scale dw_j s_j,
// the logits' is
//   sigmoid: (d_scores s + a) (1 - s)
//   softmax: d_scores s + a - s sum over all experts of (d_scores s + a).
// A wave per token; the row is put together in LDS, where the k choices are
// added to what all experts have.  HBM bounds it: 16384 x 512 with d_scores, 102 MB
// in 21 us, 4.9 TB/s.
template <int V, int NI>
__global__ __launch_bounds__(256) void k_route_bwd(RouteArgs a) {
    __shared__ __attribute__((aligned(16))) float rows[4][64 * V * NI];
    const int64_t t = block_number() * 4 + wave_id();
    if (t >= a.T) return;
    typedef float fv __attribute__((ext_vector_type(V)));
    const int lane = lane_id();
    const float* row = a.logits + t * a.E;
    float* out = rows[wave_id()];
    const bool softmax = a.score == SCORE_SOFTMAX;
    int e = -1;
    float dw = 0.f, l = -INFINITY;
    if (lane < a.k) {
        const int at = a.idx[t * a.k + lane];
        if ((unsigned)at < (unsigned)a.E) {
            e = at;
            dw = a.dw[t * a.k + lane];
            l = no_nan(row[e]);
        } else {
            raise_err(a.err, ERR_BAD_EXPERT);
        }
    }
    // all scores, where something needs them
    const bool dense = a.d_scores || (softmax && !a.renorm);
    fv s[NI], g[NI];
    float m = -INFINITY, z = 0.f;
    if (dense) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int c = (i * 64 + lane) * V;
            fv x = c < a.E ? *(const fv*)(row + c) : fv(-INFINITY);
            g[i] = a.d_scores && c < a.E ? *(const fv*)(a.d_scores + t * a.E + c) : fv(0.f);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                s[i][q] = no_nan(x[q]);
                m = fmaxf(m, s[i][q]);
            }
        }
        if (softmax) {
            m = wave_most(m);
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    s[i][q] = soft_exp(s[i][q], m);
                    z += s[i][q];
                }
            z = wave_sum(z);
        }
    }
    const float rz = z > 0.f ? 1.f / z : 0.f;
    float p = 0.f;
    if (a.renorm) {
        const float ml = wave_most(l);
        if (softmax) p = soft_exp(l, ml);
        else if (l != -INFINITY) {
            const float c = fminf(ml, 0.f);
            p = l < 0.f ? expf(l - c) / (1.f + expf(l)) : expf(-c) / (1.f + expf(-l));
        }
        const float sum = wave_total(p);
        p = sum > 0.f ? p / sum : 0.f;
        p = a.scale * p * (dw - wave_total(p * dw));
    } else {
        p = a.scale * dw * (softmax ? soft_exp(l, m) * rz : 1.f / (1.f + expf(-l)));
    }
    if (e < 0) p = 0.f;
    float dot = softmax && !a.renorm ? wave_total(p) : 0.f;
    if (!softmax) p *= 1.f / (1.f + expf(l));
    if (softmax && a.d_scores) {
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int q = 0; q < V; ++q) d = fmaf(g[i][q], s[i][q] * rz, d);
        dot += wave_total(d);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        fv o = fv(0.f);
        if (dense) {
#pragma unroll
            for (int q = 0; q < V; ++q) {
                if (softmax) o[q] = s[i][q] * rz * (g[i][q] - dot);
                else {
                    const float x = s[i][q];
                    o[q] = g[i][q] * (1.f / (1.f + expf(-x))) * (1.f / (1.f + expf(x)));
                }
            }
        }
        *(fv*)(out + (i * 64 + lane) * V) = o;
    }
    // a choice that a caller's table names more than once: the first of them adds them all
    float mine = 0.f;
    bool first = e >= 0;
    for (int j = 0; j < a.k; ++j) {
        const int ej = lane_value(e, j);
        const float pj = lane_value(p, j);
        if (ej == e) {
            mine += pj;
            if (j < lane) first = false;
        }
    }
    wave_lds_order();
    if (first) out[e] += mine;
    wave_lds_order();
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int c = (i * 64 + lane) * V;
        if (c < a.E) *(fv*)(a.d_logits + t * a.E + c) = *(const fv*)(out + c);
    }
}

// ================================================================ launchers
template <int EPL>
static int route_(const RouteArgs& a, const Lanes& L, hipStream_t st) {
    const bool vec = L.Eg % 4 == 0 && ((uintptr_t)a.logits | (uintptr_t)a.bias) % 16 == 0;
    const dim3 grid = rows_grid(((int64_t)a.T + 3) / 4);
    if (a.scores) k_route<EPL, true><<<grid, 256, 0, st>>>(a, L, vec);
    else k_route<EPL, false><<<grid, 256, 0, st>>>(a, L, vec);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_route(const RouteArgs& a, hipStream_t st) {
    ProfScope prof_(st, "route");
    Lanes L{64, a.E / a.n_group};
    for (int g = 1; g < a.n_group; g <<= 1) L.per >>= 1;
    const int need = (L.Eg + L.per - 1) / L.per;
    if (need <= 1) return route_<1>(a, L, st);
    if (need <= 2) return route_<2>(a, L, st);
    if (need <= 4) return route_<4>(a, L, st);
    if (need <= 8) return route_<8>(a, L, st);
    if (need <= 16) return route_<16>(a, L, st);
    return route_<32>(a, L, st);
}

int launch_route_bwd(const RouteArgs& a, hipStream_t st) {
    ProfScope prof_(st, "route_bwd");
    const dim3 grid = rows_grid(((int64_t)a.T + 3) / 4);
    auto go = [&](auto kern) {
        kern<<<grid, 256, 0, st>>>(a);
        return hipGetLastError() == hipSuccess ? 0 : -1;
    };
    if (a.E % 4 == 0 && ((uintptr_t)a.logits | (uintptr_t)a.d_scores | (uintptr_t)a.d_logits) % 16 == 0) {
        if (a.E <= 256) return go(k_route_bwd<4, 1>);
        if (a.E <= 512) return go(k_route_bwd<4, 2>);
        return go(k_route_bwd<4, 4>);
    }
    if (a.E <= 64) return go(k_route_bwd<1, 1>);
    if (a.E <= 256) return go(k_route_bwd<1, 4>);
    return go(k_route_bwd<1, 16>);
}

}  // namespace moe
