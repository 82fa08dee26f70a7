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
// tile from the offsets.
//
// N and K are multiples of 8 (16-byte rows), M and the groups are any size:
// reduction indices past a row's or a group's end are read as zeros, rows and
// columns past an operand's last are read from its last one and their results
// are not stored.  Products are sums of fp32 MFMA steps in ascending order of
// the reduction index (or of a few ascending parts, added in order); bias,
// activation and residual are applied to the fp32 sum, which is rounded once.
#include "dtype.h"
#include "gemm_common.h"
#include "linear_common.h"
#include "profile.h"
#include "tile256.h"

namespace moe {

// One block: for each of up to three sets of tiles, list[e] = the tiles of the
// groups before e, list[E] their number.
__global__ __launch_bounds__(1024) void k_linear_prefix(LinPrefix p) {
    __shared__ int32_t wsum[16];
    const int E = p.t[0].E, e = threadIdx.x, lane = lane_id(), wv = threadIdx.x >> 6;
    int lo, cnt = 0;
    if (e < E) cnt = group_rows(p.t[0], e, lo, true);
    for (int q = 0; q < p.n; ++q) {
        const int n = e < E ? group_tiles(p.t[q], cnt) : 0;
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
        int32_t* out = const_cast<int32_t*>(p.t[q].list);
        const int most = (int)max_tiles(p.t[q]);
        if (e < E) out[e] = min(pre, most);
        if (e == E - 1) out[E] = min(pre + n, most);
        __syncthreads();
    }
}

// dW: block b's expert e, tile (mt, nt) of nMt by nNt, and the expert's rows lo,
// n; tiles in bands of BAND row tiles, as above.
template <int BAND>
__device__ __forceinline__ bool lin_wtile(const LinTiles& t, int nMt, int nNt, int b, int& e, int& mt, int& nt,
                                          int& lo, int& n, int* quarter = nullptr) {
    const int per = nMt * nNt, total = (t.offsets ? t.E : 1) * per;
    int L;
    if (!rest_tile(total, b, quarter, L)) return false;
    const int rem = L % per;
    e = L / per;
    const int band = rem / (BAND * nNt), r = rem - band * BAND * nNt, rows = min(BAND, nMt - BAND * band);
    nt = r / rows;
    mt = BAND * band + (r - nt * rows);
    lo = 0;
    n = t.rows;
    if (t.offsets) n = group_rows(t, e, lo, true);
    return true;
}

// ================================================================ 64 / 128 x 128 tiles
// stages of the ring: two blocks of 64-row tiles share a CU
template <int TM>
constexpr int lin_stages() { return TM == 64 ? 3 : 4; }
template <int TM>
constexpr int lin_waves() { return TM == 64 ? 4 : 8; }

// ONCE: a weight tile feeds one row tile, so it is copied non-temporally (512
// experts of 40 rows, 4.3 GB of weights: 801 -> 698 us, 6.45 TB/s; where two
// row tiles read it: 39 -> 46 us).  Weight rows have to be whole 128-byte lines
// for that: pieces of a line that two steps read come twice (K = 4072: 1122
// non-temporally, 916 plainly).
template <class D, int ACT, int TM, bool ONCE>
__device__ __forceinline__ void fwd_tile(const LinFwdArgs& a, int e, int lo, int hi, int n0, const T1Ring& ring) {
    constexpr int TN = 128;
    T1Acc<TM, lin_waves<TM>()> acc;
    {
        const TileOperand<false, TM, 1, 64 * lin_waves<TM>()> oa(a.x, a.K, lo, hi);
        const TileOperand<false, TN, 1, 64 * lin_waves<TM>(), ONCE> ob(a.w + (int64_t)e * a.N * a.K, a.K, n0, a.N);
        t1_mainloop<D, false, false, TM, lin_stages<TM>(), lin_waves<TM>(), ONCE>(oa, ob, a.K, acc, ring);
    }
    T1Pos<TM, lin_waves<TM>()> pos;
    if (a.bias) {
#pragma unroll
        for (int nb = 0; nb < t1_nb<lin_waves<TM>()>(); ++nb) {
            const f32x4 v = bias4<D>(a, e, n0 + pos.n(nb));
#pragma unroll
            for (int mb = 0; mb < TM / 32; ++mb) acc[mb][nb] += v;
        }
    }
    const bool nt_out = many((int64_t)a.t.rows * a.N);
    if (a.z)
        t1_put<TM, lin_waves<TM>()>(ring, nt_out, a.z, lo, hi, n0, a.N,
                                    [&](int mb, int nb) { return pack4<D>(acc[mb][nb]); });
    t1_put<TM, lin_waves<TM>()>(ring, nt_out, a.y, lo, hi, n0, a.N, [&](int mb, int nb) {
        return pack4<D>(act_residual<D, ACT>(a, lo + pos.m(mb), hi, n0 + pos.n(nb), acc[mb][nb]));
    });
}
template <class D, int ACT, int TM, bool ONCE>
__global__ __launch_bounds__(64 * lin_waves<TM>(), TM == 64 ? 2 : 1) void k_linear_fwd(LinFwdArgs a) {
    int e, lo, hi, nt, mt;
    if (!lin_tile<TM, TM == 128 ? 4 : 1>(a.t, (a.N + 127) / 128, blockIdx.x, e, lo, hi, nt, mt)) return;
    T1_RING(ring, TM, lin_stages<TM>());
    fwd_tile<D, ACT, TM, ONCE>(a, e, lo, hi, nt * 128, ring);
}

// ================================================================ split reductions
// Too few tiles for the chip: each tile's reduction is split into ksplit
// ascending parts of whole 64-deep steps, a block each, whose fp32 sums
// k_linear_sum adds in order (128 x 4096 x 4096: 39 -> 17 us).  N: output columns,
// K: reduction length, w: [N, K], or (BKS) [K, N].
template <class D, bool BKS, int TM>
__global__ __launch_bounds__(64 * lin_waves<TM>(), 1) void k_linear_part(LinFwdArgs a) {
    constexpr int TN = 128;
    const int part = blockIdx.x % a.ksplit;
    int e, lo, hi, nt, mt;
    if (!lin_tile<TM, 1>(a.t, (a.N + TN - 1) / TN, blockIdx.x / a.ksplit, e, lo, hi, nt, mt)) return;
    const int steps = (a.K + kTK - 1) / kTK, k0 = steps * part / a.ksplit * kTK;
    const int k1 = min(steps * (part + 1) / a.ksplit * kTK, a.K), n0 = nt * TN;
    T1_RING(ring, TM, 4);
    T1Acc<TM, lin_waves<TM>()> acc;
    {
        const TileOperand<false, TM, 1, 64 * lin_waves<TM>()> oa(a.x + k0, a.K, lo, hi);
        const uint16_t* w = a.w + (int64_t)e * a.N * a.K;
        const TileOperand<BKS, TN, 1, 64 * lin_waves<TM>()> ob(BKS ? w + (int64_t)k0 * a.N : w + k0,
                                                               BKS ? a.N : a.K, n0, a.N);
        t1_mainloop<D, false, BKS, TM, 4, lin_waves<TM>()>(oa, ob, k1 - k0, acc, ring);
    }
    T1Pos<TM, lin_waves<TM>()> pos;
#pragma unroll
    for (int mb = 0; mb < TM / 32; ++mb) {
        const int row = lo + pos.m(mb);
        if (row >= hi) continue;
#pragma unroll
        for (int nb = 0; nb < t1_nb<lin_waves<TM>()>(); ++nb) {
            const int col = n0 + pos.n(nb);
            if (col < a.N) *(f32x4*)(a.part + ((int64_t)part * a.t.rows + row) * a.N + col) = acc[mb][nb];
        }
    }
}

// Eight rows of a tile, 128 columns.
template <class D, int ACT, int TM>
__global__ __launch_bounds__(256) void k_linear_sum(LinFwdArgs a) {
    int e, lo, hi, nt, mt;
    if (!lin_tile<TM, 1>(a.t, (a.N + 127) / 128, blockIdx.x / (TM / 8), e, lo, hi, nt, mt)) return;
    const int row = lo + blockIdx.x % (TM / 8) * 8 + (threadIdx.x >> 5), col = nt * 128 + (threadIdx.x & 31) * 4;
    if (row >= hi || col >= a.N) return;
    f32x4 v = *(const f32x4*)(a.part + (int64_t)row * a.N + col);
#pragma unroll 4
    for (int q = 1; q < a.ksplit; ++q) v += *(const f32x4*)(a.part + ((int64_t)q * a.t.rows + row) * a.N + col);
    lin_out<D, ACT>(a, e, row, col, v);
}

// ================================================================ few rows
// A handful of rows: the weights are read once and everything else is small,
// so the product is a stream.  A block computes 16 MB rows by 16 NB columns;
// its W waves split the reduction, each reading pieces of S * 64 bytes of every
// weight row (neighbouring waves neighbouring pieces) straight into MFMA
// fragments: no LDS and no barrier until the waves' sums are added, in wave
// order, at the end.  The loads run one unit ahead.  (Non-temporal loads of the
// weights: 4 x 4096 x 4096 10.1 -> 10.4 us, 160 rows at 512 experts 190 -> 221.)
template <class D, int ACT, int MB, int NB, int S, int W>
__global__ __launch_bounds__(64 * W) void k_linear_stream(LinFwdArgs a) {
    constexpr int TM = 16 * MB, TN = 16 * NB, U = 32 * S;
    __shared__ f32x4 sums[W][MB * NB][64];
    int e, lo, hi, nt, mt;
    if (!lin_tile<TM, 1>(a.t, (a.N + TN - 1) / TN, blockIdx.x, e, lo, hi, nt, mt)) return;
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
        } else {                                           // the last unit: zeros behind the row (masked, as above)
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int k = k0 + 32 * s + kg < a.K ? k0 + 32 * s : a.K - 8 - kg;
                const uint32_t in = k0 + 32 * s + kg < a.K ? ~0u : 0u;
                auto masked = [&](const uint16_t* p) {
                    const uint4 v = *(const uint4*)(p + k);
                    return make_uint4(v.x & in, v.y & in, v.z & in, v.w & in);
                };
#pragma unroll
                for (int n = 0; n < NB; ++n) u.w[n][s] = masked(wp[n]);
#pragma unroll
                for (int m = 0; m < MB; ++m) u.x[m][s] = masked(xp[m]);
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
template <class D, int TM, bool ONCE>
__device__ __forceinline__ void dx_tile(const LinBwdArgs& a, int e, int lo, int hi, int n0, const T1Ring& ring) {
    constexpr int TN = 128;
    T1Acc<TM, lin_waves<TM>()> acc;
    {
        const TileOperand<false, TM, 1, 64 * lin_waves<TM>()> oa(a.dz, a.N, lo, hi);
        const TileOperand<true, TN, 1, 64 * lin_waves<TM>(), ONCE> ob(a.w + (int64_t)e * a.N * a.K, a.K, n0, a.K);
        t1_mainloop<D, false, true, TM, lin_stages<TM>(), lin_waves<TM>(), ONCE>(oa, ob, a.N, acc, ring);
    }
    t1_put<TM, lin_waves<TM>()>(ring, many((int64_t)a.t.rows * a.K), a.dx, lo, hi, n0, a.K,
                                [&](int mb, int nb) { return pack4<D>(acc[mb][nb]); });
}
template <class D, int TM, bool ONCE>
__device__ __forceinline__ void dx_block(const LinBwdArgs& a, int block, const T1Ring& ring) {
    int e, lo, hi, nt, mt;
    if (!lin_tile<TM, TM == 128 ? 4 : 1>(a.t, (a.K + 127) / 128, block, e, lo, hi, nt, mt)) return;
    dx_tile<D, TM, ONCE>(a, e, lo, hi, nt * 128, ring);
}

template <class D, int TM, bool ONCE>
__global__ __launch_bounds__(64 * lin_waves<TM>(), TM == 64 ? 2 : 1) void k_linear_dx(LinBwdArgs a) {
    T1_RING(ring, TM, lin_stages<TM>());
    dx_block<D, TM, ONCE>(a, blockIdx.x, ring);
}

__device__ __forceinline__ int64_t dw_elements(const LinBwdArgs& a) {
    return (int64_t)(a.t.offsets ? a.t.E : 1) * a.N * a.K;
}

// dW = dz^T x over a group's rows: both operands with the row as the memory row
template <class D>
__device__ __forceinline__ void dw_tile(const LinBwdArgs& a, int e, int lo, int n, int m0, int n0, const T1Ring& ring) {
    constexpr int TM = 128, TN = 128;
    T1Acc<TM, lin_waves<TM>()> acc;
    {
        const TileOperand<true, TM, 1, 64 * lin_waves<TM>()> oa(a.dz + (int64_t)lo * a.N, a.N, m0, a.N);
        const TileOperand<true, TN, 1, 64 * lin_waves<TM>()> ob(a.x + (int64_t)lo * a.K, a.K, n0, a.K);
        t1_mainloop<D, true, true, TM, lin_stages<TM>(), lin_waves<TM>()>(oa, ob, n, acc, ring);
    }
    t1_put<TM, lin_waves<TM>()>(ring, many(dw_elements(a)), a.dw + (int64_t)e * a.N * a.K, m0, a.N, n0, a.K,
               [&](int mb, int nb) { return pack4<D>(acc[mb][nb]); });
}

template <class D>
__device__ __forceinline__ void dw_block(const LinBwdArgs& a, int block, const T1Ring& ring) {
    int e, mt, nt, lo, n;
    if (!lin_wtile<4>(a.t, (a.N + 127) / 128, (a.K + 127) / 128, block, e, mt, nt, lo, n)) return;
    dw_tile<D>(a, e, lo, n, mt * 128, nt * 128, ring);
}

template <class D>
__global__ __launch_bounds__(64 * lin_waves<128>(), 1) void k_linear_dw(LinBwdArgs a) {
    T1_RING(ring, 128, 4);
    dw_block<D>(a, blockIdx.x, ring);
}

// Groups of few rows: dW's write is all the work.  Blocks of 32 KB of LDS,
// four to a CU, so that some wait for their operands while others store: one
// stage, no ring; the tile goes out through LDS as whole 256-byte row pieces,
// past the caches.  Where 512 experts of 40 rows write 4.3 GB: 869 us (4.9 TB/s;
// 10 rows each: 644, 6.7 TB/s; the ring form, a block to a CU, 3160 us;
// register-staged tiles stored from their fragments 1540).  Blocks that walk
// eight tiles, dz^T in fragments and the next x loaded ahead (64 KB, two to a
// CU): 807 us, but 774 for 10 rows each and 162 instead of 139 us for 64
// experts of 128 rows.
template <class D>
__global__ __launch_bounds__(256, 4) void k_linear_dw_few(LinBwdArgs a) {
    constexpr int TM = 128, TN = 128;
    __shared__ __attribute__((aligned(16))) uint16_t sm[TM * TN];
    static_assert(TM * TN == 2 * kT2Half, "the operands' stage and the tile take the same LDS");
    int e, mt, nt, lo, n;
    if (!lin_wtile<1>(a.t, (a.N + TM - 1) / TM, (a.K + TN - 1) / TN, blockIdx.x, e, mt, nt, lo, n)) return;
    const int m0 = mt * TM, n0 = nt * TN;
    uint16_t *const sa = sm, *const sb = sm + kT2Half;
    T1Acc<TM, 4> acc;
    {
        const TileOperand<true, TM, 1, 256> oa(a.dz + (int64_t)lo * a.N, a.N, m0, a.N);
        const TileOperand<true, TN, 1, 256> ob(a.x + (int64_t)lo * a.K, a.K, n0, a.K);
        T1Loop<D, true, true, TM, 3, 4> l(oa, ob, acc);
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
    T1Pos<TM, 4> pos;
#pragma unroll
    for (int mb = 0; mb < TM / 32; ++mb)
#pragma unroll
        for (int nb = 0; nb < TN / 32; ++nb) {
            const int r = pos.m(mb), c = pos.n(nb);
            *(uint2*)(sm + r * TN + (((c >> 3) ^ (r & 15)) << 3) + (c & 7)) = pack4<D>(acc[mb][nb]);
        }
    __syncthreads();
    const int c = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    if (n0 + 8 * c >= a.K) return;
    const bool past = many(dw_elements(a));
    uint16_t* out = a.dw + ((int64_t)e * a.N + m0) * a.K + n0 + 8 * c;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const int r = r0 + 16 * q;
        if (m0 + r < a.N) st_out(past, out + (int64_t)r * a.K, sm + r * TN + ((c ^ (r & 15)) << 3));
    }
}

// db[e] = the sum of its tiles' partial rows (k_linear_dz): 64 columns of an
// expert, `waves` waves over the tiles
template <class D>
__device__ __forceinline__ void db_columns(const float* part, const LinTiles& t, int N, int block, int waves,
                                           float* sums, uint16_t* db) {
    const int nc = (N + 63) / 64;
    const int e = block / nc, col = (block % nc) * 64 + lane_id(), wv = wave_id();
    int t0 = 0, t1 = (t.rows + t.tm - 1) / t.tm;
    if (t.offsets && t.list) {
        t0 = t.list[e];
        t1 = t.list[e + 1];
    } else if (t.offsets) {
        const WaveTiles w = wave_tiles(t, false);
        t0 = __builtin_amdgcn_readlane(w.pre, e);
        t1 = min(t0 + group_tiles(t, __builtin_amdgcn_readlane(w.n, e)), w.total);
    }
    float s = 0.f;
    if (col < N)
        for (int i = t0 + wv; i < t1; i += waves) s += part[(int64_t)i * N + col];
    sums[wv * 64 + lane_id()] = s;
    __syncthreads();
    if (wv > 0 || col >= N) return;
    for (int v = 1; v < waves; ++v) s += sums[v * 64 + lane_id()];
    db[(int64_t)e * N + col] = (uint16_t)D::pack2(s, 0.f);
}

// All that follows dz in one launch, for products whose tiles leave CUs idle:
// blocks of dW's tiles, dx's tiles and db's columns.
template <class D>
__global__ __launch_bounds__(64 * lin_waves<128>(), 1) void k_linear_bwd(LinBwdArgs a) {
    T1_RING(ring, 128, 4);
    int b = blockIdx.x;
    if (b < a.ndw) {
        dw_block<D>(a, b, ring);
        return;
    }
    b -= a.ndw;
    if (b < a.ndx) dx_block<D, 128, false>(a, b, ring);
    else db_columns<D>(a.part, a.strips, a.N, b - a.ndx, lin_waves<128>(), (float*)ring.a0, a.db);
}

// ================================================================ 256 x 256 tiles
__device__ __forceinline__ T1Ring t1_ring(const T2Lds& l) {
    return T1Ring{l.h[0], l.h[1], l.h[2], l.h[3], l.h[4], l.h[5], l.h[6], l.h[7]};
}

template <class D, int ACT>
__global__ __launch_bounds__(kT2Threads, 2) void k_linear_fwd256(LinFwdArgs a) {
    int e, lo, hi, nt, mt, q;
    if (!lin_tile<256, 4>(a.t, (a.N + 255) / 256, blockIdx.x, e, lo, hi, nt, mt, &q)) return;
    T2_LDS(lds);
    if (q >= 0) {
        const int r0 = lo + 128 * (q >> 1), n0 = nt * 256 + 128 * (q & 1);
        if (r0 < hi && n0 < a.N) fwd_tile<D, ACT, 128, false>(a, e, r0, min(r0 + 128, hi), n0, t1_ring(lds));
        return;
    }
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
                const f32x4 v = bias4<D>(a, e, nt * 256 + t2_col(hb, nb));
#pragma unroll
                for (int ha = 0; ha < 2; ++ha)
#pragma unroll
                    for (int mb = 0; mb < 4; ++mb) acc[ha][hb][mb][nb] += v;
            }
    }
    const bool nt_out = many((int64_t)a.t.rows * a.N);
    if (a.z)
        t2_put(lds, nt_out, a.z, lo, hi, nt * 256, a.N,
               [&](int ha, int hb, int mb, int nb) { return pack4<D>(acc[ha][hb][mb][nb]); });
    t2_put(lds, nt_out, a.y, lo, hi, nt * 256, a.N, [&](int ha, int hb, int mb, int nb) {
        return pack4<D>(
            act_residual<D, ACT>(a, lo + t2_row(ha, mb), hi, nt * 256 + t2_col(hb, nb), acc[ha][hb][mb][nb]));
    });
}

template <class D>
__device__ __forceinline__ void t2_store(const T2Lds& lds, bool nt, uint16_t* out, int r0, int r1, int c0, int ncol,
                                         const T2Acc& acc) {
    t2_put(lds, nt, out, r0, r1, c0, ncol,
           [&](int ha, int hb, int mb, int nb) { return pack4<D>(acc[ha][hb][mb][nb]); });
}

template <class D>
__global__ __launch_bounds__(kT2Threads, 2) void k_linear_dx256(LinBwdArgs a) {
    T2_LDS(lds);
    if ((int)blockIdx.x < a.ndb) {                 // db's columns first (a launch less)
        db_columns<D>(a.part, a.strips, a.N, blockIdx.x, kT2Threads / 64, (float*)lds.h[0], a.db);
        return;
    }
    int e, lo, hi, nt, mt, q;
    if (!lin_tile<256, 4>(a.t, (a.K + 255) / 256, blockIdx.x - a.ndb, e, lo, hi, nt, mt, &q)) return;
    if (q >= 0) {
        const int r0 = lo + 128 * (q >> 1), n0 = nt * 256 + 128 * (q & 1);
        if (r0 < hi && n0 < a.K) dx_tile<D, 128, false>(a, e, r0, min(r0 + 128, hi), n0, t1_ring(lds));
        return;
    }
    T2Acc acc;
    {
        const T2Operand<false> oa(a.dz, a.N, lo, hi);
        const T2Operand<true> ob(a.w + (int64_t)e * a.N * a.K, a.K, nt * 256, a.K);
        t2_mainloop<D, false, true>(oa, ob, a.N, acc, lds);
    }
    t2_store<D>(lds, many((int64_t)a.t.rows * a.K), a.dx, lo, hi, nt * 256, a.K, acc);
}

template <class D>
__global__ __launch_bounds__(kT2Threads, 2) void k_linear_dw256(LinBwdArgs a) {
    int e, mt, nt, lo, n, q;
    if (!lin_wtile<4>(a.t, (a.N + 255) / 256, (a.K + 255) / 256, blockIdx.x, e, mt, nt, lo, n, &q)) return;
    T2_LDS(lds);
    if (q >= 0) {
        const int m0 = mt * 256 + 128 * (q >> 1), n0 = nt * 256 + 128 * (q & 1);
        if (m0 < a.N && n0 < a.K) dw_tile<D>(a, e, lo, n, m0, n0, t1_ring(lds));
        return;
    }
    T2Acc acc;
    {
        const T2Operand<true> oa(a.dz + (int64_t)lo * a.N, a.N, mt * 256, a.N);
        const T2Operand<true> ob(a.x + (int64_t)lo * a.K, a.K, nt * 256, a.K);
        t2_mainloop<D, true, true>(oa, ob, n, acc, lds);
    }
    t2_store<D>(lds, many(dw_elements(a)), a.dw + (int64_t)e * a.N * a.K, mt * 256, a.N, nt * 256, a.K, acc);
}

// ================================================================ dz and db
// A block takes a tile of TR rows by 512 columns (8 per lane, rows round
// robin over four waves): dz = dy act'(z), and the column sums of the
// unrounded dz, in fp32, one partial row per tile.  dz is rounded once, to the
// 16-bit type that the MFMA multiplies: both products see an operand half a
// step off, as random from element to element as the rounding of their result,
// so dx and dW are off by sqrt(2) times what rounding the result alone costs
// (1111 x 1000 x 1544 fp16: 2.9e-4 of the norm, 2.1e-4 for products of
// unrounded dz).  Keeping more of dz takes a second 16-bit operand and twice
// the products.  Bound by HBM: 20480 x 1024 bf16, 126 MB in 27 us.
template <class D, int ACT, int TR>
__global__ __launch_bounds__(256) void k_linear_dz(LinDzArgs a) {
    __shared__ float sums[3][64][8];
    int e, lo, hi, nt, mt;
    if (!lin_tile<TR, 1>(a.t, (a.N + 511) / 512, blockIdx.x, e, lo, hi, nt, mt)) return;
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
    float* p = a.part + (int64_t)mt * a.N + col;
    *(float4*)p = make_float4(s[0], s[1], s[2], s[3]);
    *(float4*)(p + 4) = make_float4(s[4], s[5], s[6], s[7]);
}

template <class D>
__global__ __launch_bounds__(1024) void k_linear_db(LinBwdArgs a) {
    __shared__ float sums[16 * 64];
    db_columns<D>(a.part, a.strips, a.N, blockIdx.x, 16, sums, a.db);
}

// ================================================================ launchers
// blocks for `tiles` 256 x 256 tiles, or for at most as many (the device counts
// groups' tiles), the ones behind the last whole round in quarters
static int64_t blocks256(int64_t tiles, bool exact) {
    const int64_t rest = tiles % 256;
    return tiles + 3 * (!exact ? kRest256 : rest <= kRest256 ? rest : 0);
}

static int64_t blocks256(const LinTiles& t, int C) {
    return blocks256(max_tiles(t) * ((C + 255) / 256), t.E == 0);
}

// Whether a product of M rows (of E groups, E = 0: dense) and C output columns
// takes 256 x 256 tiles rather than 128 x 128 ones.  A CU works on one of the
// large tiles at a time; a round of 256 of them takes what two rounds of 256
// small tiles do, full or not, and 64 left over go as one round of small ones:
//   4096 -> 1024, 8 groups of 768 rows   87 us, 128 x 128:  82
//                            1024 rows   88                111
//   1536 -> 768, 64 groups of 128 rows   56                 65
//                             512 rows  108                142
//   1024 -> 1024, 16 groups of 384 rows  33                 29
//                              512 rows  34                 41
//   4096 x 4096, dense, 2560 rows        82                109
// (groups of fewer than 128 rows leave half of a large tile empty: 64 of 96,
// 4096 -> 1024: 150 us, 128 x 128: 136)
static bool takes_256(int64_t M, int64_t E, int64_t C) {
    auto tiles = [&](int64_t t) {                  // a group's last tile is half full on average
        return (E > 0 ? M + E * (t / 2) : M + t - 1) / t * ((C + t - 1) / t);
    };
    const int64_t whole = tiles(256) / 256, rest = tiles(256) % 256;
    return whole * 512 + (rest == 0 ? 0 : rest <= 64 ? 256 : 512) < tiles(128);
}

// The parts of a reduction over R that its few tiles are best split into.  A
// step of a lone block takes about 0.45 us; the sum's launch 6 us, and a part
// of a million outputs, written and read, 1.5 us.
//   128 x 4096 x 4096                    39 us, in parts 17
//   8 groups of 16 rows, 4096 -> 1024    34              18
//               64 rows                  31              22
//   1024 x 1024 x 1024                   12              18
//   8 groups of 128 rows, 2048 -> 2048   21              36
static int parts(const LinTiles& t, int R, int C) {
    const int64_t tiles = max_tiles(t) * ((C + 127) / 128);
    const int steps = (R + kTK - 1) / kTK;
    int best = 1;
    float least = 0.45f * steps;
    for (int64_t ks = 2; ks <= 16 && ks * tiles <= 256 && ks * 4 <= steps; ++ks) {
        const float us = 0.45f * steps / ks + 6 + 1.5e-6f * ks * t.rows * C;
        if (us < least) {
            least = us;
            best = (int)ks;
        }
    }
    return best;
}

// The tiles of a product with C output columns and R reduction indices: x W^T,
// or (dx) dz W.
LinPlan linear_plan(int M, int E, int R, int C, bool dx) {
    LinPlan p{};
    p.ksplit = 1;
    p.small = {nullptr, nullptr, E, M, 0, nullptr};
    p.big = p.small;
    if (E > 0) {
        if (M >= 128LL * E && takes_256(M, E, C)) {
            p.big.tm = 256;
            return p;
        }
        // (64 experts of 40 and 64 rows, 4096 -> 1024: 64-row tiles 99 and 148 us,
        // 128-row tiles 105 and 130)
        p.small.tm = M > 48LL * E ? 128 : 64;
        // few rows and few tiles: latency, which the streaming form splits over eight waves
        if (!dx && M <= 8LL * E && (M + 63LL) / 64 * ((C + 127) / 128) < 2048) {
            p.stream = true;
            p.small.tm = 16;
            return p;
        }
        p.once = p.small.tm == 64 && (dx ? C : R) % 64 == 0;
        p.ksplit = parts(p.small, R, C);
        return p;
    }
    if (!dx && M <= 32) {
        p.stream = true;
        p.small.tm = M <= 16 ? 16 : 32;
        return p;
    }
    if (takes_256(M, 0, C)) {
        p.big.tm = 256;
        return p;
    }
    p.small.tm = M <= 64 ? 64 : 128;
    p.ksplit = parts(p.small, R, C);
    return p;
}

size_t linear_part_floats(const LinPlan& p, int M, int C) {
    return p.ksplit > 1 ? (size_t)p.ksplit * M * C : 0;
}

// 32, or 8 where those are too few for the chip (1111 x 1000: 7.3 -> 4.4 us).
int linear_dz_rows(int M, int E, int N) {
    return max_tiles({nullptr, nullptr, E, M, 32, nullptr}) * ((N + 511) / 512) < 256 ? 8 : 32;
}

// Whether the blocks of a product find their tiles themselves (LinTiles.list null)
bool linear_inline_tiles(const LinTiles& t, int C, int tn) {
    return t.E <= 64 && max_tiles(t) * ((C + tn - 1) / tn) <= 2048;
}

int launch_linear_prefix(const LinPrefix& p, hipStream_t st) {
    ProfScope prof_(st, "linear_prefix");
    k_linear_prefix<<<1, 1024, 0, st>>>(p);
    return ok();
}

// the parts of a split product, or of dz W (BKS), and their sum
template <class D, bool BKS>
static int split_(const LinFwdArgs& a, hipStream_t st) {
    const int64_t tiles = max_tiles(a.t) * ((a.N + 127) / 128);
    if (a.t.tm == 128) {
        if (go(k_linear_part<D, BKS, 128>, tiles * a.ksplit, 64 * lin_waves<128>(), a, st)) return -1;
        return with_act(a.act, [&](auto A) { return go(k_linear_sum<D, A(), 128>, tiles * 16, 256, a, st); });
    }
    if (go(k_linear_part<D, BKS, 64>, tiles * a.ksplit, 64 * lin_waves<64>(), a, st)) return -1;
    return with_act(a.act, [&](auto A) { return go(k_linear_sum<D, A(), 64>, tiles * 8, 256, a, st); });
}

template <class D>
static int fwd_(const LinPlan& p, LinFwdArgs a, hipStream_t st) {
    if (p.ksplit > 1) {
        a.t = p.small;
        a.ksplit = p.ksplit;
        return split_<D, false>(a, st);
    }
    return with_act(a.act, [&](auto A) {
        if (p.big.tm) {
            a.t = p.big;
            return go(k_linear_fwd256<D, A()>, blocks256(a.t, a.N), kT2Threads, a, st);
        }
        a.t = p.small;
        const int64_t tiles = max_tiles(a.t);
        if (p.stream) {
            const int n16 = (a.N + 15) / 16;
            if (a.t.tm == 16 && a.t.offsets)
                return go(k_linear_stream<D, A(), 1, 2, 4, 8>, tiles * ((n16 + 1) / 2), 512, a, st);
            if (a.t.tm == 16) return go(k_linear_stream<D, A(), 1, 1, 4, 8>, tiles * n16, 512, a, st);
            return go(k_linear_stream<D, A(), 2, 1, 4, 8>, tiles * n16, 512, a, st);
        }
        const int64_t grid = tiles * ((a.N + 127) / 128);
        if (a.t.tm == 128) return go(k_linear_fwd<D, A(), 128, false>, grid, 64 * lin_waves<128>(), a, st);
        if (p.once) return go(k_linear_fwd<D, A(), 64, true>, grid, 64 * lin_waves<64>(), a, st);
        return go(k_linear_fwd<D, A(), 64, false>, grid, 64 * lin_waves<64>(), a, st);
    });
}

int launch_linear_fwd(const LinPlan& p, const LinFwdArgs& a, hipStream_t st) {
    ProfScope prof_(st, "linear_fwd");
    return a.dtype == 0 ? fwd_<Bf16>(p, a, st) : fwd_<Fp16>(p, a, st);
}

template <class D>
static int dz_(const LinDzArgs& a, hipStream_t st) {
    const int64_t grid = max_tiles(a.t) * ((a.N + 511) / 512);
    return with_act(a.act, [&](auto A) {
        return a.t.tm == 8 ? go(k_linear_dz<D, A(), 8>, grid, 256, a, st)
                           : go(k_linear_dz<D, A(), 32>, grid, 256, a, st);
    });
}

int launch_linear_dz(const LinDzArgs& a, hipStream_t st) {
    ProfScope prof_(st, "linear_dz");
    return a.dtype == 0 ? dz_<Bf16>(a, st) : dz_<Fp16>(a, st);
}

template <class D>
static int dx_(const LinPlan& p, LinBwdArgs a, hipStream_t st) {
    if (p.ksplit > 1) {                        // dz W as the sum of its parts
        LinFwdArgs f{p.small, a.dtype, LIN_NONE, a.K, a.N, a.dz, a.w, nullptr, nullptr, a.dx, nullptr, p.ksplit, a.sums};
        return split_<D, true>(f, st);
    }
    if (p.big.tm) {
        a.t = p.big;
        return go(k_linear_dx256<D>, a.ndb + blocks256(a.t, a.K), kT2Threads, a, st);
    }
    a.t = p.small;
    const int64_t grid = max_tiles(a.t) * ((a.K + 127) / 128);
    if (a.t.tm == 128) return go(k_linear_dx<D, 128, false>, grid, 64 * lin_waves<128>(), a, st);
    if (p.once) return go(k_linear_dx<D, 64, true>, grid, 64 * lin_waves<64>(), a, st);
    return go(k_linear_dx<D, 64, false>, grid, 64 * lin_waves<64>(), a, st);
}

// dW: 256 x 256 tiles, the ring of 128 x 128 tiles, or the form of few rows,
// whose several blocks to a CU hide the stores of tiles with few steps (64
// experts, 1024 x 4096: of 384 rows 285 us, 256 x 256 tiles 320; of 512 347 and
// 364; of 768 500 and 451).
template <class D>
static int dw_(const LinBwdArgs& a, hipStream_t st) {
    const int64_t groups = a.t.offsets ? a.t.E : 1, M = a.t.rows;
    const int64_t t256 = groups * ((a.N + 255) / 256) * ((a.K + 255) / 256);
    const int64_t t128 = groups * ((a.N + 127) / 128) * ((a.K + 127) / 128);
    if (M < 512 * groups) return go(k_linear_dw_few<D>, t128, 256, a, st);
    if (t256 >= 128) return go(k_linear_dw256<D>, blocks256(t256, true), kT2Threads, a, st);
    return go(k_linear_dw<D>, t128, 64 * lin_waves<128>(), a, st);
}

template <class D>
static int bwd_(const LinPlan& p, LinBwdArgs a, hipStream_t st) {
    const int64_t groups = a.t.offsets ? a.t.E : 1;
    const int64_t ndw = a.dw ? groups * ((a.N + 127) / 128) * ((a.K + 127) / 128) : 0;
    // 64-row tiles become 128-row ones in one launch with the rest (blocks that
    // find their tiles themselves can): 40 x 512 x 512 15 -> 11 us
    LinTiles one = p.small;
    if (one.tm == 64 && !one.list) one.tm = 128;
    const int64_t ndx = a.dx ? max_tiles(one) * ((a.K + 127) / 128) : 0;
    const int64_t ndb = a.db ? groups * ((a.N + 63) / 64) : 0;
    // one launch where the tiles leave CUs idle, unless dx's few long ones would be its length
    if (one.tm == 128 && !p.big.tm && (ndw > 0) + (ndx > 0) + (ndb > 0) > 1 && ndw + ndx + ndb <= 512 &&
        (p.ksplit == 1 || a.N <= 24 * kTK)) {
        ProfScope prof_(st, "linear_bwd");
        a.t = one;
        a.ndw = (int)ndw;
        a.ndx = (int)ndx;
        return go(k_linear_bwd<D>, ndw + ndx + ndb, 64 * lin_waves<128>(), a, st);
    }
    if (a.db && a.dx && p.big.tm) {
        a.ndb = (int)ndb;                          // with dx, below
    } else if (a.db) {
        ProfScope prof_(st, "linear_db");
        if (go(k_linear_db<D>, ndb, 1024, a, st)) return -1;
    }
    if (a.dw) {
        ProfScope prof_(st, "linear_dw");
        if (dw_<D>(a, st)) return -1;
    }
    if (a.dx) {
        ProfScope prof_(st, "linear_dx");
        if (dx_<D>(p, a, st)) return -1;
    }
    return 0;
}

int launch_linear_bwd(const LinPlan& p, const LinBwdArgs& a, hipStream_t st) {
    return a.dtype == 0 ? bwd_<Bf16>(p, a, st) : bwd_<Fp16>(p, a, st);
}

}  // namespace moe
