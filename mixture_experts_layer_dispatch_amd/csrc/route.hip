// Routing with scores: softmax or sigmoid of the router logits over all
// experts, a bias and groups for the choice, the k best, their weights, and
// the gradient of the logits (include/moe.h: moe_route_forward).  The layer's
// own routing, plain top-k of the logits, is k_topk_route; the pages feed it
// Gaussian logits (alphalab.site "Mixture-of-Kittens" sections 一 and 四).
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

__device__ __forceinline__ float no_nan(float v) { return v == v ? v : -INFINITY; }
__device__ __forceinline__ double no_nan(double v) { return v == v ? v : -(double)INFINITY; }

// exp(v - m) with m the largest of the v: 1 for the largest (infinite ones
// too), 0 for -inf
__device__ __forceinline__ float soft_exp(float v, float m) { return v == -INFINITY ? 0.f : v == m ? 1.f : expf(v - m); }
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
template <int EPL>
__global__ __launch_bounds__(256) void k_route(RouteArgs a, Lanes L) {
    const int64_t t = block_number() * 4 + wave_id();
    if (t >= a.T) return;
    const int lane = lane_id();
    const float* row = a.logits + t * a.E;
    int n;
    const int e0 = first_expert<EPL>(L, a.n_group, lane, n);
    float v[EPL];
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        v[j] = j < n ? no_nan(row[e0 + j]) : -INFINITY;
        m = fmaxf(m, v[j]);
    }
    const bool softmax = a.score == SCORE_SOFTMAX;
    const bool groups = a.n_group > 1, two = groups && a.group_top == 2;
    const bool by_logit = !a.bias && !two;
    double key[EPL];
    double z = 0.0;
    m = wave_most(m);
    if (softmax) {
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (j < n) z += soft_exp((double)v[j], (double)m);
        z = wave_sum(z);
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        key[j] = v[j];
        if (j < n && (a.scores || !by_logit)) {
            const double s = !softmax ? 1.0 / (1.0 + exp(-(double)v[j])) : z > 0.0 ? soft_exp((double)v[j], (double)m) / z : 0.0;
            if (a.scores) a.scores[t * a.E + e0 + j] = (float)s;
            if (!by_logit) key[j] = no_nan(s + (a.bias ? (double)a.bias[e0 + j] : 0.0));
        }
    }
    // the places still to be chosen
    uint32_t open = n >= 32 ? ~0u : (1u << n) - 1u;
    if (groups) {
        double t1 = -(double)INFINITY, t2 = t1;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            if (j < n) {
                t2 = fmax(t2, fmin(t1, key[j]));
                t1 = fmax(t1, key[j]);
            }
        }
        for (int off = L.per >> 1; off >= 1; off >>= 1) {
            const double o1 = __shfl_xor(t1, off), o2 = __shfl_xor(t2, off);
            t2 = fmax(fmax(t2, o2), fmin(t1, o1));
            t1 = fmax(t1, o1);
        }
        const double score = two ? no_nan(t1 + t2) : t1;
        bool left = lane / L.per < a.n_group, kept = false;
        for (int r = 0; r < a.topk_group; ++r) {
            double b = score;
            int at = left ? lane / L.per : 64;
            for (int off = 32; off >= 1; off >>= 1) {
                const double ob = __shfl_xor(b, off);
                const int oat = __shfl_xor(at, off);
                if (oat < 64 && (at == 64 || ob > b || (ob == b && oat < at))) { b = ob; at = oat; }
            }
            if (lane / L.per == at) { kept = true; left = false; }
        }
        if (!kept) open = 0;
    }
    int sel = 0;                                   // lane r < k: the r-th choice
    for (int r = 0; r < a.k; ++r) {
        double b = -(double)INFINITY;
        int at = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if ((open >> j & 1u) && (at == 0x7fffffff || key[j] > b)) { b = key[j]; at = e0 + j; }
        for (int off = 32; off >= 1; off >>= 1) {
            const double ob = __shfl_xor(b, off);
            const int oat = __shfl_xor(at, off);
            if (oat != 0x7fffffff && (at == 0x7fffffff || ob > b || (ob == b && oat < at))) { b = ob; at = oat; }
        }
        if (n > 0 && at >= e0 && at < e0 + n) open &= ~(1u << (at - e0));
        if (lane == r) sel = at;
    }
    // the weights, in 64 bits: k of them
    const bool in = lane < a.k;
    const double l = in ? (double)no_nan(row[sel]) : -(double)INFINITY;
    double p = 0.0, sum = 1.0;
    if (a.renorm) {
        // only the ratios of the chosen matter: the scores relative to the largest of
        // them, so that none is lost where all are tiny
        double ml = l;
        for (int off = 32; off >= 1; off >>= 1) ml = fmax(ml, __shfl_xor(ml, off));
        if (softmax) p = soft_exp(l, ml);
        else {
            const double c = fmin(ml, 0.0);
            p = l == -(double)INFINITY ? 0.0 : l < 0.0 ? exp(l - c) / (1.0 + exp(l)) : exp(-c) / (1.0 + exp(-l));
        }
        sum = 0.0;
        for (int r = 0; r < a.k; ++r) sum += __shfl(p, r);
    } else if (softmax) {
        p = soft_exp(l, (double)m);
        sum = z;
    } else {
        p = 1.0 / (1.0 + exp(-l));
    }
    if (in) {
        a.idx[t * a.k + lane] = sel;
        a.w[t * a.k + lane] = sum > 0.0 ? (float)(a.scale * p / sum) : 0.f;
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
// added to what all experts have.
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
    __builtin_amdgcn_wave_barrier();
    if (first) out[e] += mine;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int c = (i * 64 + lane) * V;
        if (c < a.E) *(fv*)(a.d_logits + t * a.E + c) = *(const fv*)(out + c);
    }
}

// ================================================================ launchers
int launch_route(const RouteArgs& a, hipStream_t st) {
    ProfScope prof_(st, "route");
    Lanes L{64, a.E / a.n_group};
    for (int g = 1; g < a.n_group; g <<= 1) L.per >>= 1;
    const int need = (L.Eg + L.per - 1) / L.per;
    const dim3 grid = rows_grid(((int64_t)a.T + 3) / 4);
    if (need <= 1) k_route<1><<<grid, 256, 0, st>>>(a, L);
    else if (need <= 2) k_route<2><<<grid, 256, 0, st>>>(a, L);
    else if (need <= 4) k_route<4><<<grid, 256, 0, st>>>(a, L);
    else if (need <= 8) k_route<8><<<grid, 256, 0, st>>>(a, L);
    else if (need <= 16) k_route<16><<<grid, 256, 0, st>>>(a, L);
    else k_route<32><<<grid, 256, 0, st>>>(a, L);
    return hipGetLastError() == hipSuccess ? 0 : -1;
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
