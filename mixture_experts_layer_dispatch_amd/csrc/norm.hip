// Layer norm and rms norm of rows, with the residual added on the way, and
// their gradients (include/moe.h: moe_norm_forward):
//
//   h = x + residual,  xh = (h - mean) rstd,  y = xh gamma + beta
//   g = dy gamma,  dx = rstd (g - sum(g) / H - xh sum(g xh) / H) + d_total
//   dgamma = sum over the rows of dy xh,  dbeta = sum of dy
//
// what stands in front of the router projection and the experts in a block of
// a model.  A row is read once and kept in registers: the mean first, then the
// sum of the squared distances from it, so that a mean far from zero costs no
// digits.
#include "dtype.h"
#include "launch.h"
#include "profile.h"
#include "rows.h"

namespace moe {

// ---------------------------------------------------------------- sums of a row
// A row is W waves; `s` holds a value per wave of the block, for two sums at once.
template <int W>
__device__ __forceinline__ f32x2 row_sums(f32x2 v, f32x2* s) {
    v[0] = wave_total(v[0]);
    v[1] = wave_total(v[1]);
    if constexpr (W > 1) {
        const int wv = wave_id(), first = wv / W * W;
        __syncthreads();                           // (what was there has been read)
        if (lane_id() == 0) s[wv] = v;
        __syncthreads();
        v = s[first];
#pragma unroll
        for (int q = 1; q < W; ++q) v += s[first + q];
    }
    return v;
}

// 16 bytes' worth of parameters from element `at` on
template <class D, class P>
__device__ __forceinline__ void load_params(const void* p, int at, float* f) {
    if constexpr (D::PER16 == P::PER16) {
        P::unpack(*(const uint4*)((const char*)p + (int64_t)at * (16 / P::PER16)), f);
    } else {                                       // 16-bit rows, fp32 parameters
        const uint4* q = (const uint4*)((const float*)p + at);
        Fp32::unpack(q[0], f);
        Fp32::unpack(q[1], f + 4);
    }
}
template <class D, class P>
__device__ __forceinline__ void store_params(void* p, int at, const float* f) {
    if constexpr (D::PER16 == P::PER16) {
        *(uint4*)((char*)p + (int64_t)at * (16 / P::PER16)) = P::pack(f);
    } else {
        uint4* q = (uint4*)((float*)p + at);
        q[0] = Fp32::pack(f);
        q[1] = Fp32::pack(f + 4);
    }
}

// ================================================================ forward
// A block has 4 rows of a wave each (W 1), or one row of W waves; a thread has NC
// chunks of 16 bytes of its row.  HBM bounds it: 16384 x 4096 bf16, 268 MB without a residual
// in 46 to 49 us, 5.5 to 5.8 TB/s; 4 rows take what a launch takes.
template <class D, class P, int W, int NC>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void k_norm(NormArgs a) {
    constexpr int RB = W == 1 ? 4 : 1, PER = D::PER16;
    __shared__ f32x2 sums[RB * W];
    const int wv = wave_id(), C = a.H / PER;
    const int64_t row = block_number() * RB + wv / W;
    if (W > 1 && row >= a.M) return;               // (a whole block)
    const bool live = row < a.M;
    const int c0 = (wv % W) * 64 + lane_id();
    uint4 v[NC];
    const uint4* x = (const uint4*)a.x + row * C;
    const uint4* res = (const uint4*)a.residual + row * C;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = c0 + i * 64 * W;
        v[i] = live && c < C ? x[c] : make_uint4(0, 0, 0, 0);
    }
    if (a.residual) {
        uint4* total = (uint4*)a.total + row * C;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = c0 + i * 64 * W;
            if (!live || c >= C) continue;
            float f[PER], r[PER];
            D::unpack(v[i], f);
            D::unpack(res[c], r);
#pragma unroll
            for (int q = 0; q < PER; ++q) f[q] += r[q];
            v[i] = D::pack(f);
            total[c] = v[i];
        }
    }
    float mean = 0.f;
    if (!a.rms) {
        f32x2 s = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float f[PER];
            D::unpack(v[i], f);                    // (zeros behind the row)
#pragma unroll
            for (int q = 0; q < PER; ++q) s[0] += f[q];
        }
        mean = row_sums<W>(s, sums)[0] / a.H;
    }
    f32x2 s = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = c0 + i * 64 * W;
        if (c >= C) continue;
        float f[PER];
        D::unpack(v[i], f);
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const float d = f[q] - mean;
            s[0] = fmaf(d, d, s[0]);
        }
    }
    const float rstd = 1.f / sqrtf(row_sums<W>(s, sums)[0] / a.H + a.eps);
    if (!live) return;
    uint4* y = (uint4*)a.y + row * C;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = c0 + i * 64 * W;
        if (c >= C) continue;
        float f[PER], g[PER], b[PER];
        D::unpack(v[i], f);
        load_params<D, P>(a.gamma, c * PER, g);
        if (a.beta) load_params<D, P>(a.beta, c * PER, b);
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            f[q] = (f[q] - mean) * rstd * g[q];
            if (a.beta) f[q] += b[q];
        }
        y[c] = D::pack(f);
    }
    if (wv % W == 0 && lane_id() == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

// ================================================================ backward
// A block has RG rows at a time, W waves each (one, or the whole block), and
// goes over the rows RG b, RG b + 1, ..., then RG (b + parts), ...  A thread keeps its
// columns' sums for dgamma and dbeta over its rows; the block adds them up over its
// rows in LDS and writes one part, which k_norm_params adds up block by block.  Latency
// bounds it, with a block of eight waves a CU and no row fetched ahead of the one before:
// 16384 x 4096 bf16 with d_total, 537 MB in 132 us, 4.1 TB/s where the forward reaches 5.8
// (373 with a row per block and parts added in sequence).
template <class D, class P, int W, int NC, int RG>
__global__ __launch_bounds__(64 * W * RG, 1) void k_norm_bwd(NormArgs a, int parts) {
    constexpr int PER = D::PER16, Q = PER / 4;
    __shared__ f32x2 sums[W];
    __shared__ f32x4 cols[RG > 1 ? RG : 1][RG > 1 ? 2 * Q : 1][64 * W];
    const int C = a.H / PER, rg = wave_id() / W, c0 = wave_id() % W * 64 + lane_id();
    const bool params = a.dgamma || a.dbeta;
    float dg[NC][PER], db[NC][PER];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int q = 0; q < PER; ++q) dg[i][q] = db[i][q] = 0.f;
    for (int64_t row = (int64_t)blockIdx.x * RG + rg; row < a.M; row += (int64_t)parts * RG) {
        const uint4* x = (const uint4*)a.x + row * C;
        const uint4* dy = (const uint4*)a.dy + row * C;
        uint4 xv[NC], gv[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = c0 + i * 64 * W;
            xv[i] = c < C ? x[c] : make_uint4(0, 0, 0, 0);
            gv[i] = c < C ? dy[c] : make_uint4(0, 0, 0, 0);
        }
        const float mean = a.mean ? a.mean[row] : 0.f, rstd = a.rstd[row];
        f32x2 s = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = c0 + i * 64 * W;
            if (c >= C) continue;
            float f[PER], d[PER], g[PER];
            D::unpack(xv[i], f);
            D::unpack(gv[i], d);
            load_params<D, P>(a.gamma, c * PER, g);
#pragma unroll
            for (int q = 0; q < PER; ++q) {
                const float xh = (f[q] - mean) * rstd, w = d[q] * g[q];
                dg[i][q] = fmaf(d[q], xh, dg[i][q]);
                db[i][q] += d[q];
                s[0] += w;
                s[1] = fmaf(w, xh, s[1]);
            }
        }
        if (!a.y) continue;
        s = row_sums<W>(s, sums);
        const float mg = a.rms ? 0.f : s[0] / a.H, mx = s[1] / a.H;
        uint4* dx = (uint4*)a.y + row * C;
        const uint4* skip = (const uint4*)a.residual + row * C;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = c0 + i * 64 * W;
            if (c >= C) continue;
            float f[PER], d[PER], g[PER], r[PER];
            D::unpack(xv[i], f);
            D::unpack(gv[i], d);
            load_params<D, P>(a.gamma, c * PER, g);
            if (a.residual) D::unpack(skip[c], r);
#pragma unroll
            for (int q = 0; q < PER; ++q) {
                const float xh = (f[q] - mean) * rstd;
                f[q] = rstd * (d[q] * g[q] - mg - xh * mx);
                if (a.residual) f[q] += r[q];
            }
            dx[c] = D::pack(f);
        }
    }
    if (!params) return;
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.H;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = c0 + i * 64 * W;
        f32x4 v[2 * Q];
#pragma unroll
        for (int q = 0; q < 2 * Q; ++q) {
            const float* f = q < Q ? dg[i] + 4 * q : db[i] + 4 * (q - Q);
            v[q] = f32x4{f[0], f[1], f[2], f[3]};
        }
        if constexpr (RG > 1) {
            if (i > 0) __syncthreads();
#pragma unroll
            for (int q = 0; q < 2 * Q; ++q) cols[rg][q][c0] = v[q];
            __syncthreads();
            // wave rg adds up quad rg
            if (rg < 2 * Q && c < C) {
                f32x4 t = cols[0][rg][c0];
#pragma unroll
                for (int g = 1; g < RG; ++g) t += cols[g][rg][c0];
                *(f32x4*)(part + (rg < Q ? 0 : a.H) + c * PER + 4 * (rg % Q)) = t;
            }
        } else if (c < C) {
#pragma unroll
            for (int q = 0; q < 2 * Q; ++q) *(f32x4*)(part + (q < Q ? 0 : a.H) + c * PER + 4 * (q % Q)) = v[q];
        }
    }
}

// Rows too long for a block's registers beside the sums for dgamma and dbeta: a
// block per row reads it twice, the second time from the caches,
template <class D, class P>
__global__ __launch_bounds__(1024) void k_norm_bwd_long(NormArgs a) {
    constexpr int PER = D::PER16, W = 16;
    __shared__ f32x2 sums[W];
    const int C = a.H / PER;
    const int64_t row = block_number();
    if (row >= a.M) return;
    const uint4* x = (const uint4*)a.x + row * C;
    const uint4* dy = (const uint4*)a.dy + row * C;
    const float mean = a.mean ? a.mean[row] : 0.f, rstd = a.rstd[row];
    f32x2 s = {0.f, 0.f};
    for (int c = threadIdx.x; c < C; c += 64 * W) {
        float f[PER], d[PER], g[PER];
        D::unpack(x[c], f);
        D::unpack(dy[c], d);
        load_params<D, P>(a.gamma, c * PER, g);
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const float w = d[q] * g[q];
            s[0] += w;
            s[1] = fmaf(w, (f[q] - mean) * rstd, s[1]);
        }
    }
    s = row_sums<W>(s, sums);
    const float mg = a.rms ? 0.f : s[0] / a.H, mx = s[1] / a.H;
    uint4* dx = (uint4*)a.y + row * C;
    const uint4* skip = (const uint4*)a.residual + row * C;
    for (int c = threadIdx.x; c < C; c += 64 * W) {
        float f[PER], d[PER], g[PER], r[PER];
        D::unpack(x[c], f);
        D::unpack(dy[c], d);
        load_params<D, P>(a.gamma, c * PER, g);
        if (a.residual) D::unpack(skip[c], r);
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            f[q] = rstd * (d[q] * g[q] - mg - (f[q] - mean) * rstd * mx);
            if (a.residual) f[q] += r[q];
        }
        dx[c] = D::pack(f);
    }
}

// and the sums over the rows have blocks of their own (before dx, which may be dy):
// 64 chunks of columns, four waves that share the part's rows.
template <class D>
__global__ __launch_bounds__(256) void k_norm_cols(NormArgs a, int parts) {
    constexpr int PER = D::PER16, Q = PER / 4;
    __shared__ f32x4 cols[4][2 * Q][64];
    const int C = a.H / PER, c = blockIdx.x * 64 + lane_id(), wv = wave_id();
    float dg[PER] = {}, db[PER] = {};
    if (c < C)
        for (int64_t row = (int64_t)blockIdx.y * 4 + wv; row < a.M; row += (int64_t)parts * 4) {
            const float mean = a.mean ? a.mean[row] : 0.f, rstd = a.rstd[row];
            float f[PER], d[PER];
            D::unpack(((const uint4*)a.x)[row * C + c], f);
            D::unpack(((const uint4*)a.dy)[row * C + c], d);
#pragma unroll
            for (int q = 0; q < PER; ++q) {
                dg[q] = fmaf(d[q], (f[q] - mean) * rstd, dg[q]);
                db[q] += d[q];
            }
        }
#pragma unroll
    for (int q = 0; q < 2 * Q; ++q) {
        const float* f = q < Q ? dg + 4 * q : db + 4 * (q - Q);
        cols[wv][q][lane_id()] = f32x4{f[0], f[1], f[2], f[3]};
    }
    __syncthreads();
    if (wv >= 2 * Q || c >= C) return;
    f32x4 t = cols[0][wv][lane_id()];
#pragma unroll
    for (int g = 1; g < 4; ++g) t += cols[g][wv][lane_id()];
    float* part = a.part + (int64_t)blockIdx.y * 2 * a.H;
    *(f32x4*)(part + (wv < Q ? 0 : a.H) + c * PER + 4 * (wv % Q)) = t;
}

// dgamma (y 0) and dbeta (y 1): a block's 16 quarters of columns, four each, over 64
// slices of the parts, whose sums are added in order.
template <class P>
__global__ __launch_bounds__(1024) void k_norm_params(NormArgs a, int parts) {
    __shared__ f32x4 sums[64][16];
    void* out = blockIdx.y ? a.dbeta : a.dgamma;
    if (!out) return;
    const int col = (blockIdx.x * 16 + (threadIdx.x & 15)) * 4, sl = threadIdx.x >> 4;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (col < a.H) {
        const float* p = a.part + (int64_t)blockIdx.y * a.H + col;
#pragma unroll 4
        for (int b = sl; b < parts; b += 64) v += *(const f32x4*)(p + (int64_t)b * 2 * a.H);
    }
    sums[sl][threadIdx.x & 15] = v;
    __syncthreads();
    if (threadIdx.x >= 16 || col >= a.H) return;
    for (int q = 1; q < min(parts, 64); ++q) v += sums[q][threadIdx.x];
    if constexpr (P::PER16 == 4) *(f32x4*)((float*)out + col) = v;
    else *(uint2*)((uint16_t*)out + col) = make_uint2(P::pack2(v[0], v[1]), P::pack2(v[2], v[3]));
}

// ================================================================ launchers
// The forward's rows: f(W, NC).  (Rows of at most 2^16 elements: 2^13 chunks of
// 16 bits, 2^14 of fp32.)  bf16 rows of 134 MB in all, over and over, us, in (W, NC):
//    512 elements  (1, 1) 47, (4, 1) 136
//   1024           (4, 1) 76, (2, 4) 58, (1, 2) 43
//   2048           (4, 1) 48, (1, 4) 44, (8, 1) 75
//   4096           (4, 2) 43, (1, 8) 46, (8, 1) 49, (16, 1) 86
//   8192           (4, 4) 43, (8, 2) 43, (16, 1) 57
//   16384          (16, 4) 60, (16, 2) 47, (8, 4) 45
//   32768          (16, 4) 58, (8, 8) 50
// and 4 rows of 4096: (4, 2) 3.8, (1, 8) 6.2, (8, 1) 3.5, (16, 1) 3.8.  The first of each
// is taken; at 1024, 16384 and 32768 another is faster.
template <class D, class F>
static int with_shape(int C, const F& f) {
    using std::integral_constant;
    if (C <= 64) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
    if (C <= 256) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
    if (C <= 512) return f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
    if (C <= 1024) return f(integral_constant<int, 4>{}, integral_constant<int, 4>{});
    if (C <= 4096) return f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
    if constexpr (D::PER16 == 4)
        if (C > 8192) return f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
    return f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
}

template <class F>
static int with_types(int dtype, int params, const F& f) {
    if (dtype == 2) return f(Fp32{}, Fp32{});
    if (dtype == 1) return params == 1 ? f(Fp16{}, Fp16{}) : f(Fp16{}, Fp32{});
    return params == 0 ? f(Bf16{}, Bf16{}) : f(Bf16{}, Fp32{});
}

// The backward's rows: up to 512 chunks in a wave, eight rows to a block, up to
// 2048 a block each, f(W, NC, RG); longer ones go over memory twice, f(0, 0, 1).  As above,
// 134 MB each of x, dy and dx, us:
//   512 elements  (1, 1, 8) 125, (8, 1, 1) 378;  1024  (1, 2, 8) 104, (8, 1, 1) 228
//   2048          (1, 4, 8) 92, (8, 1, 1) 137;   4096  (1, 8, 8) 97, (8, 1, 1) 100, (4, 2, 1) 106
//   8192          (8, 2, 1) 97, (16, 1, 1) 111;  16384 (8, 4, 1) 113, (16, 2, 1) 114, twice 139
//   32768         twice 148, (16, 4, 1) 325
template <class F>
static int with_bwd_shape(int C, const F& g) {
    using std::integral_constant;
    if (C <= 64) return g(integral_constant<int, 1>{}, integral_constant<int, 1>{}, integral_constant<int, 8>{});
    if (C <= 128) return g(integral_constant<int, 1>{}, integral_constant<int, 2>{}, integral_constant<int, 8>{});
    if (C <= 256) return g(integral_constant<int, 1>{}, integral_constant<int, 4>{}, integral_constant<int, 8>{});
    if (C <= 512) return g(integral_constant<int, 1>{}, integral_constant<int, 8>{}, integral_constant<int, 8>{});
    if (C <= 1024) return g(integral_constant<int, 8>{}, integral_constant<int, 2>{}, integral_constant<int, 1>{});
    if (C <= 2048) return g(integral_constant<int, 8>{}, integral_constant<int, 4>{}, integral_constant<int, 1>{});
    return g(integral_constant<int, 0>{}, integral_constant<int, 0>{}, integral_constant<int, 1>{});
}

// Blocks of the backward, each with its part.  As above, with 128, 256, 512 and 1024 blocks:
// 128 elements 294, 153, 109, 97 us; 512: 218, 125, 99, 100; 2048: 151, 93, 95, 100; 4096: 141,
// 97, 105, 118; 8192 (a block a row) 176, 106, 98, 106; 16384: 156, 106, 112, 143.
int norm_parts(int M, int H, int dtype) {
    return with_bwd_shape(H / (dtype == 2 ? 4 : 8), [&](auto w, auto n, auto rg) {
        constexpr int RG = decltype(rg)::value, most = RG > 1 ? 256 : decltype(w)::value ? 512 : 64;
        const int blocks = (M + RG - 1) / RG;
        return blocks < most ? blocks : most;
    });
}

int launch_norm(const NormArgs& a, hipStream_t st) {
    ProfScope prof_(st, "norm");
    return with_types(a.dtype, a.params, [&](auto d, auto p) {
        using D = decltype(d);
        using P = decltype(p);
        return with_shape<D>(a.H / D::PER16, [&](auto w, auto n) {
            constexpr int W = decltype(w)::value, RB = W == 1 ? 4 : 1;
            constexpr int threads = W == 1 ? 256 : 64 * W;
            k_norm<D, P, W, decltype(n)::value><<<rows_grid(((int64_t)a.M + RB - 1) / RB, threads), threads, 0, st>>>(a);
            return hipGetLastError() == hipSuccess ? 0 : -1;
        });
    });
}

int launch_norm_bwd(const NormArgs& a, hipStream_t st) {
    const int parts = norm_parts(a.M, a.H, a.dtype);
    {
        ProfScope prof_(st, "norm_bwd");
        const int r = with_types(a.dtype, a.params, [&](auto d, auto p) {
            using D = decltype(d);
            using P = decltype(p);
            return with_bwd_shape(a.H / D::PER16, [&](auto w, auto n, auto rg) {
                constexpr int W = decltype(w)::value, RG = decltype(rg)::value;
                if constexpr (W > 0) {
                    k_norm_bwd<D, P, W, decltype(n)::value, RG><<<parts, 64 * W * RG, 0, st>>>(a, parts);
                } else {
                    if (a.dgamma || a.dbeta)
                        k_norm_cols<D><<<dim3((a.H / D::PER16 + 63) / 64, parts), 256, 0, st>>>(a, parts);
                    if (a.y) k_norm_bwd_long<D, P><<<rows_grid(a.M, 1024), 1024, 0, st>>>(a);
                }
                return hipGetLastError() == hipSuccess ? 0 : -1;
            });
        });
        if (r || (!a.dgamma && !a.dbeta)) return r;
    }
    ProfScope prof_(st, "norm_params");
    const dim3 grid((a.H + 63) / 64, 2);
    if (a.params == 2) k_norm_params<Fp32><<<grid, 1024, 0, st>>>(a, parts);
    else if (a.params == 1) k_norm_params<Fp16><<<grid, 1024, 0, st>>>(a, parts);
    else k_norm_params<Bf16><<<grid, 1024, 0, st>>>(a, parts);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace moe
