// Rows to experts and back as calls of their own, for callers that run their
// own experts (or exchange rows between ranks) between the two.
//
//   permute             xs[row(t, j)] = x[t]
//   permute backward    dx[t] = sum_j dxs[row(t, j)]
//   unpermute           y[t] = residual[t] + sum_j w[t, j] o[row(t, j)]
//   unpermute backward  do[row(t, j)] = w[t, j] dy[t],
//                       dw[t, j] = <o[row(t, j)], dy[t]>, and through the
//                       softmax over the chosen logits
//                       d_logit[t, idx[t, j]] += w_j (dw_j - sum_i w_i dw_i)
//
// with row = row_of_slot of one schedule table, as the pages have it
// (arex-research.com "Cursor 放出 MoK", design section, first decision: one
// table for dispatch, combine and their reverses; alphalab.site
// "Mixture-of-Kittens" section 二: a fixed accumulation order).
//
// All four are bound by HBM.  Every kernel goes over the token side, so a
// token's own row is read (or written) once for its k expert rows, which are
// whole contiguous rows: T + S rows moved by permute and unpermute (plus T
// of residual), T + 2 S by the unpermute backward, the least there is.
// Sums are fp32, j ascending, rounded once; a row outside the table is
// skipped and raises MOE_DEVERR_BAD_ROW.
#include "common.h"
#include "dtype.h"
#include "launch.h"
#include "profile.h"
#include "rows.h"

namespace moe {

// Lane j < k of the wave holds the row of the token's slot j (-1: bad).
__device__ __forceinline__ int slot_row(const int32_t* __restrict__ row_of_slot, int t, int k, int S, int lane,
                                        int32_t* err) {
    int row = -1;
    if (lane < k) {
        const int r = row_of_slot[(int64_t)t * k + lane];
        if ((unsigned)r < (unsigned)S) row = r;
        else raise_err(err, ERR_BAD_ROW);
    }
    return row;
}

// ================================================================ permute
// A wave takes one 1 KB segment (64 chunks of 16 bytes) of a token's row and
// writes it k times.  (A wave per expert row, reading its token's row, writes in
// order but reads every row k times: 16384 tokens x 10 x 4096 366 us instead of
// 297; four segments to a wave 301.)
template <bool NT>
__global__ __launch_bounds__(256) void k_permute(const uint4* __restrict__ x, int C, int nseg,
                                                 const int32_t* __restrict__ row_of_slot, int T, int k, int S,
                                                 uint4* __restrict__ xs, int32_t* __restrict__ err) {
    const int64_t L = block_number() * 4 + wave_id();
    if (L >= (int64_t)T * nseg) return;
    const int t = (int)(L / nseg);
    const int lane = lane_id(), c = (int)(L % nseg) * 64 + lane;
    const int myrow = slot_row(row_of_slot, t, k, S, lane, err);
    if (c >= C) return;
    const uint4 v = x[(int64_t)t * C + c];
    for (int j = 0; j < k; ++j) {
        const int r = lane_value(myrow, j);
        if (r >= 0) st_row<NT>(xs + (int64_t)r * C + c, v);
    }
}

// ================================================================ unpermute
// A wave takes one segment of a token's row and loads up to KB expert rows'
// segments at once.
template <class D, bool WEIGHT, int KB>
__global__ __launch_bounds__(256) void k_unpermute(const uint4* __restrict__ o, int C, int nseg,
                                                   const int32_t* __restrict__ row_of_slot,
                                                   const float* __restrict__ w, int T, int k, int S,
                                                   const uint4* residual, uint4* y,
                                                   int32_t* __restrict__ err) {
    const int64_t L = block_number() * 4 + wave_id();
    if (L >= (int64_t)T * nseg) return;
    const int t = (int)(L / nseg);
    const int lane = lane_id(), c = (int)(L % nseg) * 64 + lane;
    const int myrow = slot_row(row_of_slot, t, k, S, lane, err);
    float myw = 1.f;
    if (WEIGHT) myw = lane < k ? w[(int64_t)t * k + lane] : 0.f;
    if (c >= C) return;
    float acc[D::PER16];
#pragma unroll
    for (int q = 0; q < D::PER16; ++q) acc[q] = 0.f;
    for (int j0 = 0; j0 < k; j0 += KB) {
        uint4 v[KB];
#pragma unroll
        for (int jj = 0; jj < KB; ++jj) {
            const int r = lane_value(myrow, (j0 + jj) & 63);
            v[jj] = (j0 + jj < k && r >= 0) ? ld_once(o + (int64_t)r * C + c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int jj = 0; jj < KB; ++jj) {
            const int j = (j0 + jj) & 63;
            if (j0 + jj >= k || lane_value(myrow, j) < 0) continue;
            const float wj = WEIGHT ? lane_value(myw, j) : 1.f;
            float f[D::PER16];
            D::unpack(v[jj], f);
#pragma unroll
            for (int q = 0; q < D::PER16; ++q) acc[q] = WEIGHT ? fmaf(wj, f[q], acc[q]) : acc[q] + f[q];
        }
    }
    if (residual) {
        float f[D::PER16];
        D::unpack(residual[(int64_t)t * C + c], f);
#pragma unroll
        for (int q = 0; q < D::PER16; ++q) acc[q] += f[q];
    }
    y[(int64_t)t * C + c] = D::pack(acc);
}

// ================================================================ unpermute backward
// The sum over the wave's 64 lanes of each of N values, N a power of two:
// every step halves either the lanes a value is spread over and the values a
// lane holds (N > 1) or the lanes alone, N - 1 + 6 - log2 N exchanges instead of
// 6 N.  Lane l ends up with the sum of value bitrev(l, log2 N) in v[0]
// (sum_slot); the order is fixed.
template <int N>
__device__ __forceinline__ float sum_many(float (&v)[N], int lane) {
    int off = 1;
#pragma unroll
    for (int n = N; n > 1; n >>= 1, off <<= 1) {
        const bool up = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float keep = up ? v[i + n / 2] : v[i], give = up ? v[i] : v[i + n / 2];
            v[i] = keep + __shfl_xor(give, off);
        }
    }
    float s = v[0];
    for (; off < 64; off <<= 1) s += __shfl_xor(s, off);
    return s;
}
// the value whose sum lane l holds: bit b of l picked the upper half of step b
template <int N>
__device__ __forceinline__ int sum_slot(int lane) {
    int s = 0;
#pragma unroll
    for (int n = N, b = 0; n > 1; n >>= 1, ++b)
        if (lane & (1 << b)) s += n / 2;
    return s;
}

// WPT waves of a block share a token (its segments dealt round robin); KB
// expert rows' segments are loaded at once.
template <class D, int WPT, int KB, bool NT>
__global__ __launch_bounds__(256) void k_unpermute_bwd(const uint4* __restrict__ o, const uint4* __restrict__ dy,
                                                       int C, int nseg, const int32_t* __restrict__ row_of_slot,
                                                       const int32_t* __restrict__ idx,
                                                       const float* __restrict__ w, int T, int k, int E, int S,
                                                       uint4* __restrict__ d_o, float* __restrict__ dw,
                                                       float* __restrict__ d_logits, int32_t* __restrict__ err) {
    constexpr int TPB = 4 / WPT;                          // tokens of a block
    __shared__ float part[4][KB];                         // each wave's dw sums of a batch of slots
    __shared__ float s_dl[TPB][kMaxTopK];
    __shared__ int32_t s_idx[TPB][kMaxTopK];
    const int wv = wave_id(), sub = wv % WPT, tt = wv / WPT, lane = lane_id();
    const int64_t t64 = block_number() * TPB + tt;
    const bool live = t64 < T;
    const int t = live ? (int)t64 : 0;
    const int myrow = live ? slot_row(row_of_slot, t, k, S, lane, err) : -1;
    const float myw = live && lane < k ? w[(int64_t)t * k + lane] : 0.f;
    float mydw = 0.f;                                     // lane j: dw of slot j
    for (int j0 = 0; j0 < k; j0 += KB) {
        float acc[KB];
#pragma unroll
        for (int jj = 0; jj < KB; ++jj) acc[jj] = 0.f;
        for (int sg = sub; sg < nseg && live; sg += WPT) {
            const int c = sg * 64 + lane;
            const bool in = c < C;
            uint4 v[KB];
            const uint4 dv = in ? dy[(int64_t)t * C + c] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int jj = 0; jj < KB; ++jj) {
                const int r = lane_value(myrow, (j0 + jj) & 63);
                v[jj] = (in && j0 + jj < k && r >= 0) ? ld_once(o + (int64_t)r * C + c) : make_uint4(0, 0, 0, 0);
            }
            float g[D::PER16];
            D::unpack(dv, g);
#pragma unroll
            for (int jj = 0; jj < KB; ++jj) {
                const int j = (j0 + jj) & 63;
                const int r = lane_value(myrow, j);
                if (j0 + jj >= k || r < 0) continue;
                float f[D::PER16], h[D::PER16];
                D::unpack(v[jj], f);
                const float wj = lane_value(myw, j);
#pragma unroll
                for (int q = 0; q < D::PER16; ++q) {
                    acc[jj] = fmaf(f[q], g[q], acc[jj]);
                    h[q] = wj * g[q];
                }
                if (in) st_row<NT>(d_o + (int64_t)r * C + c, D::pack(h));
            }
        }
        const float s = sum_many<KB>(acc, lane);
        const int slot = sum_slot<KB>(lane);
        if constexpr (WPT == 1) {
            if (lane < KB) part[wv][slot] = s;            // lanes 0 .. KB - 1 hold all KB values once
            __builtin_amdgcn_wave_barrier();
            if (lane >= j0 && lane < j0 + KB && lane < k) mydw = part[wv][lane - j0];
            __builtin_amdgcn_wave_barrier();
        } else {
            if (lane < KB) part[wv][slot] = s;
            __syncthreads();
            if (lane >= j0 && lane < j0 + KB && lane < k) {
                mydw = part[tt * WPT][lane - j0];
#pragma unroll
                for (int q = 1; q < WPT; ++q) mydw += part[tt * WPT + q][lane - j0];
            }
            __syncthreads();
        }
    }
    if (live && sub == 0 && lane < k) dw[(int64_t)t * k + lane] = mydw;
    if (!d_logits) return;
    float c = 0.f;
    for (int j = 0; j < k; ++j) c = fmaf(lane_value(myw, j), lane_value(mydw, j), c);
    if (live && sub == 0 && lane < k) {
        s_dl[tt][lane] = myw * (mydw - c);
        const int e = idx[(int64_t)t * k + lane];
        s_idx[tt][lane] = e;                              // (compared only: one outside matches nothing below)
        if ((unsigned)e >= (unsigned)E) raise_err(err, ERR_BAD_EXPERT);
    }
    __syncthreads();
    if (!live) return;
    for (int e = sub * 64 + lane; e < E; e += 64 * WPT) {
        float v = 0.f;
        for (int j = 0; j < k; ++j)
            if (s_idx[tt][j] == e) v += s_dl[tt][j];      // (a caller's table may name an expert twice)
        d_logits[(int64_t)t * E + e] = v;
    }
}

// ================================================================ launchers
template <class D, bool WEIGHT>
static int unpermute_(const RowsArgs& a, const void* o, const float* w, const void* residual, void* y,
                      hipStream_t st) {
    const int C = a.H / D::PER16, nseg = (C + 63) / 64;
    const dim3 grid = rows_grid(((int64_t)a.T * nseg + 3) / 4);
    auto go = [&](auto kern) {
        kern<<<grid, 256, 0, st>>>((const uint4*)o, C, nseg, a.row_of_slot, w, a.T, a.k, a.S,
                                   (const uint4*)residual, (uint4*)y, a.err);
    };
    if (a.k <= 2) go(k_unpermute<D, WEIGHT, 2>);
    else go(k_unpermute<D, WEIGHT, 8>);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

template <bool WEIGHT>
static int unpermute_any(const RowsArgs& a, const void* o, const float* w, const void* residual, void* y,
                         hipStream_t st) {
    if (a.dtype == 0) return unpermute_<Bf16, WEIGHT>(a, o, w, residual, y, st);
    if (a.dtype == 1) return unpermute_<Fp16, WEIGHT>(a, o, w, residual, y, st);
    return unpermute_<Fp32, WEIGHT>(a, o, w, residual, y, st);
}

int launch_permute(const RowsArgs& a, const void* x, void* xs, hipStream_t st) {
    ProfScope prof_(st, "permute");
    const int C = a.H * (a.dtype == 2 ? 4 : 2) / 16, nseg = (C + 63) / 64;
    const dim3 grid = rows_grid(((int64_t)a.T * nseg + 3) / 4);
    auto go = [&](auto kern) {
        kern<<<grid, 256, 0, st>>>((const uint4*)x, C, nseg, a.row_of_slot, a.T, a.k, a.S, (uint4*)xs, a.err);
        return hipGetLastError() == hipSuccess ? 0 : -1;
    };
    return (int64_t)a.S * C * 16 > kCacheBytes ? go(k_permute<true>) : go(k_permute<false>);
}

int launch_permute_bwd(const RowsArgs& a, const void* dxs, void* dx, hipStream_t st) {
    ProfScope prof_(st, "permute_bwd");
    return unpermute_any<false>(a, dxs, nullptr, nullptr, dx, st);
}

int launch_unpermute(const RowsArgs& a, const void* o, const float* w, const void* residual, void* y,
                     hipStream_t st) {
    ProfScope prof_(st, "unpermute");
    return unpermute_any<true>(a, o, w, residual, y, st);
}

template <class D>
static int unpermute_bwd_(const RowsArgs& a, const void* o, const void* dy, const int32_t* idx, const float* w,
                          int E, void* d_o, float* dw, float* d_logits, hipStream_t st) {
    const int C = a.H / D::PER16, nseg = (C + 63) / 64;
    auto go = [&](auto kern, int tpb) {
        kern<<<rows_grid(((int64_t)a.T + tpb - 1) / tpb), 256, 0, st>>>(
            (const uint4*)o, (const uint4*)dy, C, nseg, a.row_of_slot, idx, w, a.T, a.k, E, a.S, (uint4*)d_o, dw,
            d_logits, a.err);
    };
    const bool nt = (int64_t)a.S * C * 16 > kCacheBytes;
    auto pick = [&](auto NT) {
        if (nseg == 1) {                                   // one segment: a wave has the whole row
            if (a.k <= 4) go(k_unpermute_bwd<D, 1, 4, NT()>, 4);
            else go(k_unpermute_bwd<D, 1, 8, NT()>, 4);
        } else {
            if (a.k <= 4) go(k_unpermute_bwd<D, 4, 4, NT()>, 1);
            else go(k_unpermute_bwd<D, 4, 8, NT()>, 1);
        }
    };
    if (nt) pick(std::true_type{});
    else pick(std::false_type{});
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_unpermute_bwd(const RowsArgs& a, const void* o, const void* dy, const int32_t* idx, const float* w,
                         int E, void* d_o, float* dw, float* d_logits, hipStream_t st) {
    ProfScope prof_(st, "unpermute_bwd");
    if (a.dtype == 0) return unpermute_bwd_<Bf16>(a, o, dy, idx, w, E, d_o, dw, d_logits, st);
    if (a.dtype == 1) return unpermute_bwd_<Fp16>(a, o, dy, idx, w, E, d_o, dw, d_logits, st);
    return unpermute_bwd_<Fp32>(a, o, dy, idx, w, E, d_o, dw, d_logits, st);
}

}  // namespace moe
