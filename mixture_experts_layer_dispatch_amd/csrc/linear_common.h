// What the products of linear.hip and linear_w4.hip share: activations, the
// tiles of grouped rows, and the epilogue of a few outputs.
#pragma once

#include "dtype.h"
#include "launch.h"

namespace moe {

// ================================================================ activations
// (reciprocals by v_rcp_f32, 1 ulp: an IEEE division is ten instructions, and
// with erff the epilogue of a 256 x 256 tile took 15 percent of a 4096-deep product)
__device__ __forceinline__ float sigm(float v) { return __builtin_amdgcn_rcpf(1.0f + __expf(-v)); }

constexpr float kInvSqrt2Pi = 0.39894228040143268f;   // 1 / sqrt(2 pi)
constexpr float kTanhC = 0.79788456080286536f;        // sqrt(2 / pi)
constexpr float kTanhA = 0.044715f;

// The standard normal's distribution function, as 2^p(|z|) below zero and one
// minus that above: log2 of the tail is nearly a parabola, and p is its
// least-squares fit of degree 7, reweighted towards the least largest error,
// over |z| <= 6: the tail's relative error is below 6.5e-6 and |z| times its
// error below 5.6e-7 (with the evaluation in fp32); beyond 6 the tail (1e-9)
// is taken as 0.  One transcendental instruction and seven fused
// multiply-adds where erff takes about 40 instructions.
__device__ __forceinline__ float normal_cdf(float z) {
    const float a = fabsf(z);
    float p = -1.834812566e-06f;
    p = fmaf(p, a, 6.159831682e-05f);
    p = fmaf(p, a, -9.305250343e-04f);
    p = fmaf(p, a, 8.507891679e-03f);
    p = fmaf(p, a, -5.396007077e-02f);
    p = fmaf(p, a, -4.584643916e-01f);
    p = fmaf(p, a, -1.151251046e+00f);
    p = fmaf(p, a, -9.999952944e-01f);
    const float q = a <= 6.0f ? __builtin_amdgcn_exp2f(p) : 0.0f;
    return z < 0.f ? q : 1.0f - q;
}

// gelu_tanh: (1 + tanh u) / 2 = sigmoid(2 u), u = sqrt(2 / pi) (z + a z^3)
template <int ACT>
__device__ __forceinline__ float act(float z) {
    if constexpr (ACT == LIN_RELU) return z < 0.f ? 0.f : z;
    else if constexpr (ACT == LIN_GELU) return z * normal_cdf(z);
    else if constexpr (ACT == LIN_GELU_TANH) return z * sigm(2.0f * kTanhC * (z + kTanhA * z * z * z));
    else if constexpr (ACT == LIN_SILU) return z * sigm(z);
    else return z;
}

template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
    if constexpr (ACT == LIN_RELU) return z > 0.f ? 1.f : 0.f;
    else if constexpr (ACT == LIN_GELU) return normal_cdf(z) + z * __expf(-0.5f * z * z) * kInvSqrt2Pi;
    else if constexpr (ACT == LIN_GELU_TANH) {
        const float p = sigm(2.0f * kTanhC * (z + kTanhA * z * z * z)), d = p * (1.0f - p);
        // (where the sigmoid is 0 or 1, z^2 may be infinite)
        return d == 0.f ? p : p + z * d * 2.0f * kTanhC * (1.0f + 3.0f * kTanhA * z * z);
    } else if constexpr (ACT == LIN_SILU) {
        const float p = sigm(z);
        return p * (1.0f + z * (1.0f - p));
    } else return 1.f;
}

// ================================================================ row tiles
// The rows of group e, 0 if its offsets are not ascending inside the matrix.
__device__ __forceinline__ int group_rows(const LinTiles& t, int e, int& lo, bool tell) {
    const int a = t.offsets[e], b = t.offsets[e + 1];
    lo = a;
    if (a < 0 || b < a || b > t.rows) {
        if (tell) raise_err(t.err, ERR_BAD_OFFSETS);
        return 0;
    }
    return b - a;
}

__device__ __forceinline__ int group_tiles(const LinTiles& t, int n) { return (n + t.tm - 1) / t.tm; }

// Upper bound of the tiles of a set: ceil(n / tm) <= (n + tm - 1) / tm for each
// of at most min(rows, E) groups with rows.  Grids and workspaces are made for
// it, so numbers of tiles are cut to it: offsets that descend somewhere
// (refused there) can make the other groups overlap.
__host__ __device__ static inline int64_t max_tiles(const LinTiles& t) {
    if (t.tm == 0) return 0;
    if (t.E == 0) return ((int64_t)t.rows + t.tm - 1) / t.tm;
    const int64_t groups = t.rows < t.E ? t.rows : t.E;
    return (t.rows + groups * (t.tm - 1)) / t.tm;
}

// The tiles before each group, found by one wave, for at most 64 groups: lane e has group e's first row,
// rows and the tiles before it; returns their number.  Saves a launch where the
// product itself is short (grouped products of few tiles: 15 -> 11 us a call).
struct WaveTiles {
    int lo, n, pre, total;
};
__device__ __forceinline__ WaveTiles wave_tiles(const LinTiles& t, bool tell) {
    const int lane = lane_id();
    WaveTiles w{0, 0, 0, 0};
    if (lane < t.E) w.n = group_rows(t, lane, w.lo, tell);
    const int n = lane < t.E ? group_tiles(t, w.n) : 0;
    int incl = n;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(incl, off);
        if (lane >= off) incl += o;
    }
    const int most = (int)max_tiles(t);
    w.pre = min(incl - n, most);
    w.total = min(__builtin_amdgcn_readlane(incl, 63), most);
    return w;
}

// 256 x 256 tiles behind the last whole round of 256 that are computed as four
// 128 x 128 tiles each: up to 64 make one round of those, up to 128 two, which
// take 0.4 and 0.8 of the time of a round of the large tiles (4096 -> 4096, 5120
// rows: 320 tiles, 178 -> 143 us; 5632 rows, 352 tiles, 179 -> 169; 6144, 384,
// 181 -> 179).
constexpr int kRest256 = 128;

// The tile L of block b of `total`; with `quarter`, the quarter of it for a tile
// that is computed in quarters, else -1.
__device__ __forceinline__ bool rest_tile(int total, int b, int* quarter, int& L) {
    const int rest = total & 255, whole = total - rest;
    const bool split = quarter && rest <= kRest256;
    if (split && b >= whole) {
        if (b >= whole + 4 * rest) return false;
        const int s = xcd_remap(b - whole, 4 * rest);
        L = whole + (s >> 2);
        *quarter = s & 3;
        return true;
    }
    if (b >= total) return false;
    L = xcd_remap(b, split ? whole : total);
    if (quarter) *quarter = -1;
    return true;
}

// Block b's tile: expert e, rows lo .. hi - 1, column tile nt, and its number
// mt among the row tiles.  An XCD's consecutive tiles are BAND row tiles by the
// column tiles one after the other: with BAND 4, 4 by 8 for its 32 CUs, so that
// its L2 holds 12 operand strips for 32 tiles (1024 x 4096 x 4096 in 128 x 128
// tiles, 1 by 32: 45 -> 38 us; dW's 256 x 256 tiles 386 -> 377).
template <int TM, int BAND>
__device__ __forceinline__ bool lin_tile(const LinTiles& t, int nNt, int b, int& e, int& lo, int& hi, int& nt,
                                         int& mt, int* quarter = nullptr) {
    WaveTiles w;
    int ntiles;
    if (!t.offsets) ntiles = (t.rows + TM - 1) / TM;
    else if (t.list) ntiles = t.list[t.E];
    else {
        w = wave_tiles(t, b == 0);
        ntiles = w.total;
    }
    int L;
    if (!rest_tile(ntiles * nNt, b, quarter, L)) return false;
    // (small groups share weights within a group only: no bands)
    const int B = TM < 256 && t.offsets ? 1 : BAND;
    const int band = L / (B * nNt), r = L - band * B * nNt, rows = min(B, ntiles - B * band);
    nt = r / rows;
    mt = B * band + (r - nt * rows);
    if (!t.offsets) {
        e = 0;
        lo = mt * TM;
        hi = min(lo + TM, t.rows);
        return true;
    }
    if (t.list) {
        // the last group whose tiles start at or before mt, in two loads: 64
        // groups apart, then those between (a binary search is ten loads that
        // wait for each other, 0.5 us each: 1518 x 1520 x 944 at
        // 425 experts 289 instead of 253 us)
        const int per = (t.E + 63) >> 6, lane = lane_id();
        const bool far = lane * per < t.E && t.list[min(lane * per, t.E)] <= mt;
        const int e0 = per * (63 - __builtin_clzll(__ballot(far)));
        const bool near = lane < per && e0 + lane < t.E;
        const int pre = t.list[min(e0 + lane, t.E)];
        const int i = 63 - __builtin_clzll(__ballot(near && pre <= mt));
        e = e0 + i;
        const int a0 = t.offsets[e];
        lo = a0 + (mt - __builtin_amdgcn_readlane(pre, i)) * TM;
        hi = min(lo + TM, t.offsets[e + 1]);
    } else {
        // the last group whose tiles start at or before mt (one without tiles starts where the next one does)
        const uint64_t m = __ballot(lane_id() < t.E && w.pre <= mt);
        e = 63 - __builtin_clzll(m);
        const int a0 = __builtin_amdgcn_readlane(w.lo, e), n = __builtin_amdgcn_readlane(w.n, e);
        lo = a0 + (mt - __builtin_amdgcn_readlane(w.pre, e)) * TM;
        hi = min(lo + TM, a0 + n);
    }
    return true;
}

// ================================================================ outputs
// Four consecutive output columns from col, values packed: the bias of expert
// e, the activation with the residual of a row (both zero past the last column).
template <class D>
__device__ __forceinline__ uint2 pack4(const f32x4& v) {
    return make_uint2(D::pack2(v[0], v[1]), D::pack2(v[2], v[3]));
}
template <class D>
__device__ __forceinline__ f32x4 unpack4(const uint2& b) {
    return f32x4{D::lo(b.x), D::hi(b.x), D::lo(b.y), D::hi(b.y)};
}
template <class D>
__device__ __forceinline__ f32x4 bias4(const LinFwdArgs& a, int e, int col) {
    return col < a.N ? unpack4<D>(*(const uint2*)(a.bias + (int64_t)e * a.N + col)) : f32x4{0.f, 0.f, 0.f, 0.f};
}
template <class D, int ACT>
__device__ __forceinline__ f32x4 act_residual(const LinFwdArgs& a, int row, int rows, int col, f32x4 v) {
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = act<ACT>(v[r]);
    if (a.residual && row < rows && col < a.N) v += unpack4<D>(*(const uint2*)(a.residual + (int64_t)row * a.N + col));
    return v;
}
// all of it, stored
template <class D, int ACT>
__device__ __forceinline__ void lin_out(const LinFwdArgs& a, int e, int row, int col, f32x4 v) {
    const int64_t at = (int64_t)row * a.N + col;
    if (a.bias) v += bias4<D>(a, e, col);
    if (a.z) *(uint2*)(a.z + at) = pack4<D>(v);
    *(uint2*)(a.y + at) = pack4<D>(act_residual<D, ACT>(a, row, row + 1, col, v));
}

// ================================================================ launches
static int ok() { return hipGetLastError() == hipSuccess ? 0 : -1; }

template <class F>
static int with_act(int act, const F& f) {
    switch (act) {
        case LIN_RELU: return f(std::integral_constant<int, LIN_RELU>{});
        case LIN_GELU: return f(std::integral_constant<int, LIN_GELU>{});
        case LIN_GELU_TANH: return f(std::integral_constant<int, LIN_GELU_TANH>{});
        case LIN_SILU: return f(std::integral_constant<int, LIN_SILU>{});
        default: return f(std::integral_constant<int, LIN_NONE>{});
    }
}

template <class K, class A>
static int go(K kern, int64_t grid, int threads, const A& a, hipStream_t st) {
    if (grid <= 0) return 0;
    kern<<<(unsigned)grid, threads, 0, st>>>(a);
    return ok();
}

}  // namespace moe
