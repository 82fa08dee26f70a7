// y = act(x W^T + b) + residual, dense or grouped by expert, and its backward:
//
//   z  = x W^T + b          x [M, K], W [N, K] (per expert), b [N]
//   y  = act(z) + residual
//   dz = dy act'(z)
//   dx = dz W,  dW = dz^T x,  db = sum over the rows of dz
//
// The products of experts that are not the layer's SwiGLU (alphalab.site
// "Mixture-of-Kittens" section 一: each expert runs its FFN on the rows routed
// to it) and the dense projections in front of and behind the layer.  Groups
// are the rows offsets[e] .. offsets[e + 1] of one macrobatch; no count
// reaches the host (arex-research.com "Cursor 放出 MoK", design section, second
// decision): the grid covers an upper bound of tiles and each block finds its
// tile in a prefix that k_linear_prefix builds.
//
// N and K are multiples of 8 (16-byte rows), M and the groups are any size:
// operand chunks past a row's end, a group's end or a matrix's end are read
// as zeros, results past them are not stored.  Products are sums of fp32 MFMA
// steps in ascending order of the reduction index; bias, activation and
// residual are applied to the fp32 sum, which is rounded once.
#include "dtype.h"
#include "gemm_common.h"
#include "profile.h"
#include "tile256.h"

namespace moe {

// ================================================================ activations
// (reciprocals by v_rcp_f32, 1 ulp: an IEEE division is ten instructions, and
// with erff the epilogue of a 256 x 256 tile took 15 percent of a 4096-deep product)
__device__ __forceinline__ float sigm(float v) { return __builtin_amdgcn_rcpf(1.0f + __expf(-v)); }

constexpr float kInvSqrt2Pi = 0.39894228040143268f;   // 1 / sqrt(2 pi)
constexpr float kTanhC = 0.79788456080286536f;        // sqrt(2 / pi)
constexpr float kTanhA = 0.044715f;

// The standard normal's distribution function, and e = exp(-z^2 / 2).  With
// x = |z| / sqrt(2): Phi(-|z|) = erfc(x) / 2 = e erfcx(x) / 2, and erfcx(x) is a
// polynomial of degree 8 in t = 1 / (1 + 0.43 x), without a constant term,
// fitted by iteratively reweighted least squares to a relative error of 8.4e-8
// over x in [0, 9.5] (4.0e-7 with its evaluation in fp32).
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    e = __expf(-0.5f * z * z);
    const float t = __builtin_amdgcn_rcpf(fmaf(0.304055916f, fabsf(z), 1.0f));
    float p = 3.685406223e-02f;
    p = fmaf(p, t, -1.551871300e-01f);
    p = fmaf(p, t, 1.918536574e-01f);
    p = fmaf(p, t, -4.286365956e-02f);
    p = fmaf(p, t, 1.234226599e-01f);
    p = fmaf(p, t, 1.024754047e-01f);
    p = fmaf(p, t, 1.221877486e-01f);
    p = fmaf(p, t, 1.212573051e-01f);
    const float q = e * (p * t);
    return z < 0.f ? q : 1.0f - q;
}

// gelu_tanh: (1 + tanh u) / 2 = sigmoid(2 u), u = sqrt(2 / pi) (z + a z^3)
template <int ACT>
__device__ __forceinline__ float act(float z) {
    if constexpr (ACT == LIN_RELU) return z < 0.f ? 0.f : z;
    else if constexpr (ACT == LIN_GELU) {
        float e;
        return z * normal_cdf(z, e);
    } else if constexpr (ACT == LIN_GELU_TANH) return z * sigm(2.0f * kTanhC * (z + kTanhA * z * z * z));
    else if constexpr (ACT == LIN_SILU) return z * sigm(z);
    else return z;
}

template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
    if constexpr (ACT == LIN_RELU) return z > 0.f ? 1.f : 0.f;
    else if constexpr (ACT == LIN_GELU) {
        float e;
        const float c = normal_cdf(z, e);
        return c + z * e * kInvSqrt2Pi;
    } else if constexpr (ACT == LIN_GELU_TANH) {
        const float p = sigm(2.0f * kTanhC * (z + kTanhA * z * z * z));
        return p + z * p * (1.0f - p) * 2.0f * kTanhC * (1.0f + 3.0f * kTanhA * z * z);
    } else if constexpr (ACT == LIN_SILU) {
        const float p = sigm(z);
        return p * (1.0f + z * (1.0f - p));
    } else return 1.f;
}

// ================================================================ tile prefixes
// One block: for each list q, out[q][e] = sum over e' < e of
// ceil(n_e' / tm[q]) over the groups with lo[q] <= n < hi[q] rows.
__global__ __launch_bounds__(1024) void k_linear_prefix(const int32_t* __restrict__ offsets, int E, int rows,
                                                        LinPrefix p, int32_t* __restrict__ err) {
    __shared__ int32_t wsum[16];
    const int e = threadIdx.x, lane = lane_id(), wv = threadIdx.x >> 6;
    int cnt = 0;
    if (e < E) {
        const int a = offsets[e], b = offsets[e + 1];
        if (a < 0 || b < a || b > rows) raise_err(err, ERR_BAD_OFFSETS);
        else cnt = b - a;
    }
    for (int q = 0; q < p.n; ++q) {
        const int n = cnt >= p.lo[q] && cnt < p.hi[q] ? (cnt + p.tm[q] - 1) / p.tm[q] : 0;
        int incl = n;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int o = __shfl_up(incl, off);
            if (lane >= off) incl += o;
        }
        if (lane == 63) wsum[wv] = incl;
        __syncthreads();
        int pre = incl - n;
        for (int v = 0; v < wv; ++v) pre += wsum[v];
        if (e < E) p.out[q][e] = pre;
        if (e == E - 1) p.out[q][E] = pre + n;
        __syncthreads();
    }
}

// ================================================================ 64 / 128 x 128 tiles
// stages of the ring: two blocks of 64-row tiles share a CU
template <int TM>
constexpr int lin_stages() { return TM == 64 ? 3 : 4; }

// Four consecutive output columns of one row: bias, activation, residual.
template <class D, int ACT>
__device__ __forceinline__ void lin_out(const LinFwdArgs& a, int e, int64_t row, int col, const f32x4& s) {
    const int64_t at = row * a.N + col;
    float z[4] = {s[0], s[1], s[2], s[3]};
    if (a.bias) {
        const uint2 b = *(const uint2*)(a.bias + (int64_t)e * a.N + col);
        z[0] += D::lo(b.x); z[1] += D::hi(b.x); z[2] += D::lo(b.y); z[3] += D::hi(b.y);
    }
    if (a.z) *(uint2*)(a.z + at) = make_uint2(D::pack2(z[0], z[1]), D::pack2(z[2], z[3]));
#pragma unroll
    for (int r = 0; r < 4; ++r) z[r] = act<ACT>(z[r]);
    if (a.residual) {
        const uint2 b = *(const uint2*)(a.residual + at);
        z[0] += D::lo(b.x); z[1] += D::hi(b.x); z[2] += D::lo(b.y); z[3] += D::hi(b.y);
    }
    *(uint2*)(a.y + at) = make_uint2(D::pack2(z[0], z[1]), D::pack2(z[2], z[3]));
}

template <class D, int ACT, int TM>
__global__ __launch_bounds__(kT1Threads, TM == 64 ? 2 : 1) void k_linear_fwd(LinFwdArgs a) {
    constexpr int TN = 128;
    int e, lo, hi, nt;
    if (!map_mtile<TM>(a.g, (a.N + TN - 1) / TN, blockIdx.x, e, lo, hi, nt)) return;
    const int n0 = nt * TN;
    T1_RING(ring, TM, lin_stages<TM>());
    T1Acc<TM> acc;
    {
        const TileOperand<false, TM, 1, kT1Threads> oa(a.x, a.K, lo, hi);
        const TileOperand<false, TN, 1, kT1Threads> ob(a.w + (int64_t)e * a.N * a.K, a.K, n0, a.N);
        t1_mainloop<D, false, false, TM, lin_stages<TM>()>(oa, ob, a.K, acc, ring);
    }
    AccPos<TM, TN> pos;
#pragma unroll
    for (int mb = 0; mb < TM / 32; ++mb) {
        const int row = lo + pos.m(mb);
        if (row >= hi) continue;
#pragma unroll
        for (int nb = 0; nb < TN / 32; ++nb) {
            const int col = n0 + pos.n(nb);
            if (col < a.N) lin_out<D, ACT>(a, e, row, col, acc[mb][nb]);
        }
    }
}

// ================================================================ few rows
// A handful of rows: the weights are read once and everything else is small,
// so the product is a stream.  A block computes 16 MB rows by 16 NB columns;
// its W waves split the reduction, each reading pieces of S * 64 bytes of every
// weight row (neighbouring waves neighbouring pieces) straight into MFMA
// fragments: no LDS and no barrier until the waves' sums are added, in wave
// order, at the end.  The loads run one unit ahead.
template <class D, int ACT, int MB, int NB, int S, int W>
__global__ __launch_bounds__(64 * W) void k_linear_stream(LinFwdArgs a) {
    constexpr int TM = 16 * MB, TN = 16 * NB, U = 32 * S;
    __shared__ f32x4 sums[W][MB * NB][64];
    int e, lo, hi, nt;
    if (!map_mtile<TM>(a.g, (a.N + TN - 1) / TN, blockIdx.x, e, lo, hi, nt)) return;
    const int lane = lane_id(), wv = wave_id(), j = lane & 15, kg = 8 * (lane >> 4);
    const uint16_t *xp[MB], *wp[NB];
#pragma unroll
    for (int m = 0; m < MB; ++m) xp[m] = a.x + (int64_t)min(lo + 16 * m + j, hi - 1) * a.K + kg;
#pragma unroll
    for (int n = 0; n < NB; ++n)
        wp[n] = a.w + ((int64_t)e * a.N + min(nt * TN + 16 * n + j, a.N - 1)) * a.K + kg;
    f32x4 acc[MB][NB];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    struct Unit {
        uint4 x[MB][S], w[NB][S];
    } u0, u1;
    auto load = [&](Unit& u, int k0) {
        if (k0 + U <= a.K) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
#pragma unroll
                for (int n = 0; n < NB; ++n) u.w[n][s] = *(const uint4*)(wp[n] + k0 + 32 * s);
#pragma unroll
                for (int m = 0; m < MB; ++m) u.x[m][s] = *(const uint4*)(xp[m] + k0 + 32 * s);
            }
        } else {                                           // the last unit: zeros behind the row
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const bool in = k0 + 32 * s + kg < a.K;
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    u.w[n][s] = in ? *(const uint4*)(wp[n] + k0 + 32 * s) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int m = 0; m < MB; ++m)
                    u.x[m][s] = in ? *(const uint4*)(xp[m] + k0 + 32 * s) : make_uint4(0, 0, 0, 0);
            }
        }
    };
    auto add = [&](const Unit& u) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int n = 0; n < NB; ++n) acc[m][n] = D::mfma(u.w[n][s], u.x[m][s], acc[m][n]);
    };
    int k0 = wv * U;
    if (k0 < a.K) {
        load(u0, k0);
        for (;;) {
            const int k1 = k0 + W * U, k2 = k1 + W * U;
            if (k1 < a.K) load(u1, k1);
            add(u0);
            if (k1 >= a.K) break;
            if (k2 < a.K) load(u0, k2);
            add(u1);
            if (k2 >= a.K) break;
            k0 = k2;
        }
    }
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n) sums[wv][m * NB + n][lane] = acc[m][n];
    __syncthreads();
    for (int i = threadIdx.x; i < MB * NB * 64; i += 64 * W) {
        const int b = i >> 6, l = i & 63;
        f32x4 v = sums[0][b][l];
#pragma unroll
        for (int q = 1; q < W; ++q) v += sums[q][b][l];
        const int row = lo + 16 * (b / NB) + (l & 15), col = nt * TN + 16 * (b % NB) + 4 * (l >> 4);
        if (row < hi && col < a.N) lin_out<D, ACT>(a, e, row, col, v);
    }
}

// ================================================================ backward, small tiles
// dx = dz W: W read with its row (the reduction index n) as the memory row
template <class D, int TM>
__device__ __forceinline__ void dx_tile(const LinBwdArgs& a, int block, const T1Ring& ring) {
    constexpr int TN = 128;
    int e, lo, hi, nt;
    if (!map_mtile<TM>(a.g, (a.K + TN - 1) / TN, block, e, lo, hi, nt)) return;
    const int n0 = nt * TN;
    T1Acc<TM> acc;
    {
        const TileOperand<false, TM, 1, kT1Threads> oa(a.dz, a.N, lo, hi);
        const TileOperand<true, TN, 1, kT1Threads> ob(a.w + (int64_t)e * a.N * a.K, a.K, n0, a.K);
        t1_mainloop<D, false, true, TM, lin_stages<TM>()>(oa, ob, a.N, acc, ring);
    }
    AccPos<TM, TN> pos;
#pragma unroll
    for (int mb = 0; mb < TM / 32; ++mb) {
        const int row = lo + pos.m(mb);
        if (row >= hi) continue;
#pragma unroll
        for (int nb = 0; nb < TN / 32; ++nb) {
            const int col = n0 + pos.n(nb);
            const f32x4 v = acc[mb][nb];
            if (col < a.K)
                *(uint2*)(a.dx + (int64_t)row * a.K + col) = make_uint2(D::pack2(v[0], v[1]), D::pack2(v[2], v[3]));
        }
    }
}

template <class D, int TM>
__global__ __launch_bounds__(kT1Threads, TM == 64 ? 2 : 1) void k_linear_dx(LinBwdArgs a) {
    T1_RING(ring, TM, lin_stages<TM>());
    dx_tile<D, TM>(a, blockIdx.x, ring);
}

// dW = dz^T x over a group's rows: both operands with the row as the memory row
template <class D>
__device__ __forceinline__ void dw_tile(const LinBwdArgs& a, int block, const T1Ring& ring) {
    constexpr int TM = 128, TN = 128;
    int e, mt, nt, lo, n;
    if (!map_ktile(a.g, (a.N + TM - 1) / TM, (a.K + TN - 1) / TN, block, e, mt, nt, lo, n)) return;
    const int m0 = mt * TM, n0 = nt * TN;
    T1Acc<TM> acc;
    {
        const TileOperand<true, TM, 1, kT1Threads> oa(a.dz + (int64_t)lo * a.N, a.N, m0, a.N);
        const TileOperand<true, TN, 1, kT1Threads> ob(a.x + (int64_t)lo * a.K, a.K, n0, a.K);
        t1_mainloop<D, true, true, TM, lin_stages<TM>()>(oa, ob, n, acc, ring);
    }
    AccPos<TM, TN> pos;
    uint16_t* out = a.dw + (int64_t)e * a.N * a.K;
#pragma unroll
    for (int mb = 0; mb < TM / 32; ++mb) {
        const int row = m0 + pos.m(mb);
        if (row >= a.N) continue;
#pragma unroll
        for (int nb = 0; nb < TN / 32; ++nb) {
            const int col = n0 + pos.n(nb);
            const f32x4 v = acc[mb][nb];
            if (col < a.K)
                *(uint2*)(out + (int64_t)row * a.K + col) = make_uint2(D::pack2(v[0], v[1]), D::pack2(v[2], v[3]));
        }
    }
}

template <class D>
__global__ __launch_bounds__(kT1Threads, 1) void k_linear_dw(LinBwdArgs a) {
    T1_RING(ring, 128, 4);
    dw_tile<D>(a, blockIdx.x, ring);
}

// Groups of few rows: dW's write is all the work.  Blocks of 32 KB of LDS,
// four to a CU, so that some wait for their operands while others store: one
// stage, no ring; the tile goes out through LDS as whole 256-byte row pieces.
// (The ring form, a block to a CU, took 3160 us where 512 experts of 40 rows
// write 4.3 GB, register-staged tiles stored from their fragments 1540 us.)
template <class D>
__global__ __launch_bounds__(kT1Threads, 4) void k_linear_dw_few(LinBwdArgs a) {
    constexpr int TM = 128, TN = 128;
    __shared__ __attribute__((aligned(16))) uint16_t sm[TM * TN];
    static_assert(TM * TN == 2 * kT2Half, "the operands' stage and the tile take the same LDS");
    int e, mt, nt, lo, n;
    if (!map_ktile(a.g, (a.N + TM - 1) / TM, (a.K + TN - 1) / TN, blockIdx.x, e, mt, nt, lo, n)) return;
    const int m0 = mt * TM, n0 = nt * TN;
    uint16_t *const sa = sm, *const sb = sm + kT2Half;
    T1Acc<TM> acc;
    {
        const TileOperand<true, TM, 1, kT1Threads> oa(a.dz + (int64_t)lo * a.N, a.N, m0, a.N);
        const TileOperand<true, TN, 1, kT1Threads> ob(a.x + (int64_t)lo * a.K, a.K, n0, a.K);
        T1Loop<D, true, true, TM, 3> l(oa, ob, acc);
        const int nk = n / kTK, left = n % kTK;
        for (int kt = 0; kt < nk; ++kt) {
            oa.copy(0, kt, sa);
            ob.copy(0, kt, sb);
            t2_wait<0>();
            t2_barrier();
            l.product(sa, sb);
            __syncthreads();
        }
        if (left > 0) {
            oa.copy_tail(0, nk, left, sa);
            ob.copy_tail(0, nk, left, sb);
            __syncthreads();
            l.product(sa, sb);
            __syncthreads();
        }
    }
    // 16-byte chunk c of row r at slot c ^ (r & 15)
    AccPos<TM, TN> pos;
#pragma unroll
    for (int mb = 0; mb < TM / 32; ++mb)
#pragma unroll
        for (int nb = 0; nb < TN / 32; ++nb) {
            const int r = pos.m(mb), c = pos.n(nb);
            const f32x4 v = acc[mb][nb];
            *(uint2*)(sm + r * TN + (((c >> 3) ^ (r & 15)) << 3) + (c & 7)) =
                make_uint2(D::pack2(v[0], v[1]), D::pack2(v[2], v[3]));
        }
    __syncthreads();
    const int c = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    if (n0 + 8 * c >= a.K) return;
    uint16_t* out = a.dw + ((int64_t)e * a.N + m0) * a.K + n0 + 8 * c;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const int r = r0 + 16 * q;
        if (m0 + r < a.N) *(uint4*)(out + (int64_t)r * a.K) = *(const uint4*)(sm + r * TN + ((c ^ (r & 15)) << 3));
    }
}

// db[e] = the sum of its tiles' partial rows (k_linear_dz): 64 columns of an
// expert, `waves` waves over the tiles
template <class D>
__device__ __forceinline__ void db_columns(const float* part, const GroupRows& g, int N, int block, int waves,
                                           float* sums, uint16_t* db) {
    const int nc = (N + 63) / 64;
    const int e = block / nc, col = (block % nc) * 64 + lane_id(), wv = wave_id();
    int t0 = 0, t1 = (g.dense_rows + kLinDzRows - 1) / kLinDzRows;
    if (g.tile_off) {
        t0 = g.tile_off[e];
        t1 = g.tile_off[e + 1];
    }
    float s = 0.f;
    if (col < N)
        for (int t = t0 + wv; t < t1; t += waves) s += part[(int64_t)t * N + col];
    sums[wv * 64 + lane_id()] = s;
    __syncthreads();
    if (wv > 0 || col >= N) return;
    for (int v = 1; v < waves; ++v) s += sums[v * 64 + lane_id()];
    db[(int64_t)e * N + col] = (uint16_t)D::pack2(s, 0.f);
}

// All that follows dz in one launch, for products whose tiles leave CUs idle:
// blocks of dW's tiles, dx's tiles and db's columns.
template <class D>
__global__ __launch_bounds__(kT1Threads, 1) void k_linear_bwd(LinBwdArgs a) {
    T1_RING(ring, 128, 4);
    int b = blockIdx.x;
    if (b < a.ndw) {
        dw_tile<D>(a, b, ring);
        return;
    }
    b -= a.ndw;
    if (b < a.ndx) dx_tile<D, 128>(a, b, ring);
    else db_columns<D>(a.part, a.grows, a.N, b - a.ndx, kT1Threads / 64, (float*)ring.a0, a.db);
}

// ================================================================ 256 x 256 tiles
// Tile b of the groups in tile_big (or of the dense group) with nNt column
// tiles: an XCD's consecutive tiles are 4 row tiles by 8 column tiles, so that
// its L2 holds 12 operand strips for 32 tiles.
__device__ __forceinline__ bool map_tile256(const GroupRows& g, int nNt, int b, int& e, int& lo, int& hi, int& nt) {
    const int ntiles = g.tile_off ? g.tile_big[g.E] : (g.dense_rows + 255) / 256;
    if (b >= ntiles * nNt) return false;
    const int L = xcd_remap(b, ntiles * nNt);
    const int band = L / (4 * nNt), r = L - band * 4 * nNt, rows = min(4, ntiles - 4 * band);
    nt = r / rows;
    const int mt = 4 * band + (r - nt * rows);
    if (!g.tile_off) {
        e = 0;
        lo = mt * 256;
        hi = min(lo + 256, g.dense_rows);
        return true;
    }
    int a = 0, z = g.E;
    while (z - a > 1) {
        const int mid = (a + z) >> 1;
        if (g.tile_big[mid] <= mt) a = mid;
        else z = mid;
    }
    e = a;
    lo = g.offsets[e] + (mt - g.tile_big[e]) * 256;
    hi = min(lo + 256, g.offsets[e + 1]);
    return true;
}

template <class D, int ACT>
__global__ __launch_bounds__(kT2Threads, 2) void k_linear_fwd256(LinFwdArgs a) {
    int e, lo, hi, nt;
    if (!map_tile256(a.g, (a.N + 255) / 256, blockIdx.x, e, lo, hi, nt)) return;
    T2_LDS(lds);
    T2Acc acc;
    {
        const T2Operand<false> oa(a.x, a.K, lo, hi);
        const T2Operand<false> ob(a.w + (int64_t)e * a.N * a.K, a.K, nt * 256, a.N);
        t2_mainloop<D, false, false>(oa, ob, a.K, acc, lds);
    }
    if (a.bias) {
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int nb = 0; nb < 2; ++nb) {
                const int col = nt * 256 + t2_col(hb, nb);
                const uint2 b = col < a.N ? *(const uint2*)(a.bias + (int64_t)e * a.N + col) : make_uint2(0, 0);
                const f32x4 v{D::lo(b.x), D::hi(b.x), D::lo(b.y), D::hi(b.y)};
#pragma unroll
                for (int ha = 0; ha < 2; ++ha)
#pragma unroll
                    for (int mb = 0; mb < 4; ++mb) acc[ha][hb][mb][nb] += v;
            }
    }
    auto pack = [](const f32x4& v) { return make_uint2(D::pack2(v[0], v[1]), D::pack2(v[2], v[3])); };
    if (a.z)
        t2_put(lds, a.z, lo, hi, nt * 256, a.N,
               [&](int ha, int hb, int mb, int nb) { return pack(acc[ha][hb][mb][nb]); });
    t2_put(lds, a.y, lo, hi, nt * 256, a.N, [&](int ha, int hb, int mb, int nb) {
        f32x4 v = acc[ha][hb][mb][nb];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = act<ACT>(v[r]);
        if (a.residual) {
            const int row = lo + t2_row(ha, mb), col = nt * 256 + t2_col(hb, nb);
            if (row < hi && col < a.N) {
                const uint2 b = *(const uint2*)(a.residual + (int64_t)row * a.N + col);
                v += f32x4{D::lo(b.x), D::hi(b.x), D::lo(b.y), D::hi(b.y)};
            }
        }
        return pack(v);
    });
}

template <class D>
__device__ __forceinline__ void t2_store(const T2Lds& lds, uint16_t* out, int r0, int r1, int c0, int ncol,
                                         const T2Acc& acc) {
    t2_put(lds, out, r0, r1, c0, ncol, [&](int ha, int hb, int mb, int nb) {
        const f32x4 v = acc[ha][hb][mb][nb];
        return make_uint2(D::pack2(v[0], v[1]), D::pack2(v[2], v[3]));
    });
}

template <class D>
__global__ __launch_bounds__(kT2Threads, 2) void k_linear_dx256(LinBwdArgs a) {
    int e, lo, hi, nt;
    if (!map_tile256(a.g, (a.K + 255) / 256, blockIdx.x, e, lo, hi, nt)) return;
    T2_LDS(lds);
    T2Acc acc;
    {
        const T2Operand<false> oa(a.dz, a.N, lo, hi);
        const T2Operand<true> ob(a.w + (int64_t)e * a.N * a.K, a.K, nt * 256, a.K);
        t2_mainloop<D, false, true>(oa, ob, a.N, acc, lds);
    }
    t2_store<D>(lds, a.dx, lo, hi, nt * 256, a.K, acc);
}

template <class D>
__global__ __launch_bounds__(kT2Threads, 2) void k_linear_dw256(LinBwdArgs a) {
    int e, mt, nt, lo, n;
    if (!map_ktile(a.g, (a.N + 255) / 256, (a.K + 255) / 256, blockIdx.x, e, mt, nt, lo, n)) return;
    T2_LDS(lds);
    T2Acc acc;
    {
        const T2Operand<true> oa(a.dz + (int64_t)lo * a.N, a.N, mt * 256, a.N);
        const T2Operand<true> ob(a.x + (int64_t)lo * a.K, a.K, nt * 256, a.K);
        t2_mainloop<D, true, true>(oa, ob, n, acc, lds);
    }
    t2_store<D>(lds, a.dw + (int64_t)e * a.N * a.K, mt * 256, a.N, nt * 256, a.K, acc);
}

// ================================================================ dz and db
// A block takes a tile of TR rows by 512 columns (8 per lane, rows round
// robin over four waves): dz = dy act'(z) (rounded once, to the type the
// products read), and the column sums of the unrounded dz, in fp32, one
// partial row per tile.
template <class D, int ACT, int TR>
__global__ __launch_bounds__(256) void k_linear_dz(LinDzArgs a) {
    __shared__ float sums[3][64][8];
    int e, lo, hi, nt;
    if (!map_mtile<TR>(a.g, (a.N + 511) / 512, blockIdx.x, e, lo, hi, nt)) return;
    const int lane = lane_id(), wv = wave_id();
    const int col = nt * 512 + lane * 8;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (col < a.N) {
#pragma unroll 4
        for (int r = lo + wv; r < hi; r += 4) {
            const int64_t at = (int64_t)r * a.N + col;
            float g[8], z[8];
            D::unpack(*(const uint4*)(a.dy + at), g);
            if constexpr (ACT != LIN_NONE) {
                D::unpack(*(const uint4*)(a.z + at), z);
#pragma unroll
                for (int q = 0; q < 8; ++q) g[q] *= act_grad<ACT>(z[q]);
                *(uint4*)(a.dz + at) = D::pack(g);
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) s[q] += g[q];
        }
    }
    if (!a.part) return;
    if (wv > 0) {
#pragma unroll
        for (int q = 0; q < 8; ++q) sums[wv - 1][lane][q] = s[q];
    }
    __syncthreads();
    if (wv > 0 || col >= a.N) return;
#pragma unroll
    for (int v = 0; v < 3; ++v)
#pragma unroll
        for (int q = 0; q < 8; ++q) s[q] += sums[v][lane][q];
    const int tile = a.g.tile_off ? a.g.tile_off[e] + (lo - a.g.offsets[e]) / TR : lo / TR;
    float* p = a.part + (int64_t)tile * a.N + col;
    *(float4*)p = make_float4(s[0], s[1], s[2], s[3]);
    *(float4*)(p + 4) = make_float4(s[4], s[5], s[6], s[7]);
}

template <class D>
__global__ __launch_bounds__(1024) void k_linear_db(LinBwdArgs a) {
    __shared__ float sums[16 * 64];
    db_columns<D>(a.part, a.grows, a.N, blockIdx.x, 16, sums, a.db);
}

// ================================================================ launchers
// upper bound of the row tiles of the groups (or of the dense group)
static int64_t row_tiles(const GroupRows& g, int tm) {
    if (!g.tile_off) return ((int64_t)g.dense_rows + tm - 1) / tm;
    const int64_t b = ((int64_t)g.rows + (int64_t)g.E * (tm - 1)) / tm;
    return b < g.rows ? b : g.rows;
}

static int ok() { return hipGetLastError() == hipSuccess ? 0 : -1; }

int launch_linear_prefix(const int32_t* offsets, int E, int rows, const LinPrefix& p, int32_t* err, hipStream_t st) {
    ProfScope prof_(st, "linear_prefix");
    k_linear_prefix<<<1, 1024, 0, st>>>(offsets, E, rows, p, err);
    return ok();
}

template <class D, class F>
static int with_act(int act, const F& f) {
    switch (act) {
        case LIN_RELU: return f(std::integral_constant<int, LIN_RELU>{});
        case LIN_GELU: return f(std::integral_constant<int, LIN_GELU>{});
        case LIN_GELU_TANH: return f(std::integral_constant<int, LIN_GELU_TANH>{});
        case LIN_SILU: return f(std::integral_constant<int, LIN_SILU>{});
        default: return f(std::integral_constant<int, LIN_NONE>{});
    }
}

// The groups in tiles of 256 rows come first, the others follow in a launch
// of their own; a dense product is one or the other.
static int64_t big_tiles(const GroupRows& g) {
    if (!g.tile_off) return g.tm == 256 ? ((int64_t)g.dense_rows + 255) / 256 : 0;
    if (!g.tile_big) return 0;
    // groups of n >= 256 rows take ceil(n / 256) <= n / 128 tiles
    const int64_t x = (int64_t)g.rows / 128, y = ((int64_t)g.rows + (int64_t)g.E * 255) / 256;
    return x < y ? x : y;
}

// Row tiles and forms of x W^T with C output columns (or, `dx`, of dz W).
LinForm linear_form(int M, int E, int C, bool dx) {
    const int64_t groups = E > 0 ? E : 1;
    LinForm f{};
    f.small = M >= 128 * groups ? 128 : 64;
    if (!dx && (E == 0 ? M <= 512 : M <= 8 * groups)) {
        f.stream = true;
        f.small = E > 0 || M <= 16 ? 16 : M <= 32 ? 32 : 64;
        return f;
    }
    if (E == 0) f.dense_big = ((int64_t)(M + 255) / 256) * ((C + 255) / 256) >= 128;
    else f.split = M >= 192 * groups;
    return f;
}

// Forms of dW: 256 x 256 tiles, the ring of 128 x 128 tiles, or the form of few rows.
int linear_dw_form(int M, int E, int N, int K) {
    const int64_t groups = E > 0 ? E : 1;
    if (M >= 256 * groups)
        return groups * ((N + 255) / 256) * ((K + 255) / 256) >= 128 ? LIN_DW_256 : LIN_DW_RING;
    return LIN_DW_FEW;
}

template <class D>
static int fwd_(const LinFwdArgs& a, hipStream_t st) {
    return with_act<D>(a.act, [&](auto A) {
        const int64_t big = big_tiles(a.g) * ((a.N + 255) / 256);
        if (big > 0) {
            k_linear_fwd256<D, A()><<<(unsigned)big, kT2Threads, 0, st>>>(a);
            if (ok()) return -1;
        }
        if (a.g.tm == 256) return 0;
        if (a.stream) {
            auto go = [&](auto kern, int tn, int waves) {
                kern<<<(unsigned)(row_tiles(a.g, a.g.tm) * ((a.N + tn - 1) / tn)), 64 * waves, 0, st>>>(a);
                return ok();
            };
            const bool dense = !a.g.tile_off;
            if (a.g.tm == 16) {
                if (dense) return go(k_linear_stream<D, A(), 1, 1, 4, 8>, 16, 8);
                return go(k_linear_stream<D, A(), 1, 2, 4, 8>, 32, 8);
            }
            if (a.g.tm == 32) return go(k_linear_stream<D, A(), 2, 1, 4, 8>, 16, 8);
            if (a.g.dense_rows <= 64) return go(k_linear_stream<D, A(), 4, 1, 2, 8>, 16, 8);
            return go(k_linear_stream<D, A(), 4, 4, 2, 8>, 64, 8);
        }
        const int64_t grid = row_tiles(a.g, a.g.tm) * ((a.N + 127) / 128);
        if (a.g.tm == 128) k_linear_fwd<D, A(), 128><<<(unsigned)grid, 256, 0, st>>>(a);
        else k_linear_fwd<D, A(), 64><<<(unsigned)grid, 256, 0, st>>>(a);
        return ok();
    });
}

int launch_linear_fwd(const LinFwdArgs& a, hipStream_t st) {
    ProfScope prof_(st, "linear_fwd");
    return a.dtype == 0 ? fwd_<Bf16>(a, st) : fwd_<Fp16>(a, st);
}

template <class D>
static int dx_(const LinBwdArgs& a, hipStream_t st) {
    const int64_t big = big_tiles(a.g) * ((a.K + 255) / 256);
    if (big > 0) {
        k_linear_dx256<D><<<(unsigned)big, kT2Threads, 0, st>>>(a);
        if (ok()) return -1;
    }
    if (a.g.tm == 256) return 0;
    const int64_t grid = row_tiles(a.g, a.g.tm) * ((a.K + 127) / 128);
    if (a.g.tm == 128) k_linear_dx<D, 128><<<(unsigned)grid, 256, 0, st>>>(a);
    else k_linear_dx<D, 64><<<(unsigned)grid, 256, 0, st>>>(a);
    return ok();
}

template <class D>
static int dw_(const LinBwdArgs& a, hipStream_t st) {
    const int64_t groups = a.g.offsets ? a.g.E : 1;
    if (a.dw_form == LIN_DW_256) {
        const int64_t grid = groups * ((a.N + 255) / 256) * ((a.K + 255) / 256);
        k_linear_dw256<D><<<(unsigned)grid, kT2Threads, 0, st>>>(a);
        return ok();
    }
    const int64_t grid = groups * ((a.N + 127) / 128) * ((a.K + 127) / 128);
    if (a.dw_form == LIN_DW_RING) k_linear_dw<D><<<(unsigned)grid, kT1Threads, 0, st>>>(a);
    else k_linear_dw_few<D><<<(unsigned)grid, kT1Threads, 0, st>>>(a);
    return ok();
}

template <class D>
static int db_(const LinBwdArgs& a, hipStream_t st) {
    const int64_t grid = (int64_t)(a.grows.tile_off ? a.grows.E : 1) * ((a.N + 63) / 64);
    k_linear_db<D><<<(unsigned)grid, 1024, 0, st>>>(a);
    return ok();
}

template <class D>
static int bwd_(LinBwdArgs a, hipStream_t st) {
    const int64_t groups = a.g.offsets ? a.g.E : 1;
    const int64_t ndw = a.dw ? groups * ((a.N + 127) / 128) * ((a.K + 127) / 128) : 0;
    const int64_t ndx = a.dx ? row_tiles(a.g, 128) * ((a.K + 127) / 128) : 0;
    const int64_t ndb = a.db ? groups * ((a.N + 63) / 64) : 0;
    if (a.g.tm == 128 && !a.g.tile_big && (ndw > 0) + (ndx > 0) + (ndb > 0) > 1 && ndw + ndx + ndb <= 512) {
        ProfScope prof_(st, "linear_bwd");
        a.ndw = (int)ndw;
        a.ndx = (int)ndx;
        k_linear_bwd<D><<<(unsigned)(ndw + ndx + ndb), kT1Threads, 0, st>>>(a);
        return ok();
    }
    if (a.db) {
        ProfScope prof_(st, "linear_db");
        if (db_<D>(a, st)) return -1;
    }
    if (a.dw) {
        ProfScope prof_(st, "linear_dw");
        if (dw_<D>(a, st)) return -1;
    }
    if (a.dx) {
        ProfScope prof_(st, "linear_dx");
        if (dx_<D>(a, st)) return -1;
    }
    return 0;
}

int launch_linear_bwd(const LinBwdArgs& a, hipStream_t st) { return a.dtype == 0 ? bwd_<Bf16>(a, st) : bwd_<Fp16>(a, st); }

template <class D>
static int dz_(const LinDzArgs& a, hipStream_t st) {
    const int64_t grid = row_tiles(a.g, kLinDzRows) * ((a.N + 511) / 512);
    return with_act<D>(a.act, [&](auto A) {
        k_linear_dz<D, A(), kLinDzRows><<<(unsigned)grid, 256, 0, st>>>(a);
        return ok();
    });
}

int launch_linear_dz(const LinDzArgs& a, hipStream_t st) {
    ProfScope prof_(st, "linear_dz");
    return a.dtype == 0 ? dz_<Bf16>(a, st) : dz_<Fp16>(a, st);
}

}  // namespace moe
