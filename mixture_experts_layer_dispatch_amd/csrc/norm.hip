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
// A row is W waves; `s` holds a value per wave and row, for two sums at once.
template <int W>
__device__ __forceinline__ f32x2 row_sums(f32x2 v, f32x2* s) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        v[0] += __shfl_xor(v[0], off);
        v[1] += __shfl_xor(v[1], off);
    }
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
// chunks of 16 bytes of its row.
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
// Block b goes over the rows b, b + parts, ...; a thread keeps its columns'
// sums for dgamma and dbeta, which k_norm_params adds up block by block.
template <class D, class P, int W, int NC>
__global__ __launch_bounds__(64 * W) void k_norm_bwd(NormArgs a, int parts) {
    constexpr int PER = D::PER16;
    __shared__ f32x2 sums[W];
    const int C = a.H / PER, c0 = threadIdx.x;
    const bool params = a.dgamma || a.dbeta;
    float dg[NC][PER], db[NC][PER];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int q = 0; q < PER; ++q) dg[i][q] = db[i][q] = 0.f;
    for (int64_t row = blockIdx.x; row < a.M; row += parts) {
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
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = c0 + i * 64 * W;
        if (c >= C) continue;
        float* p = a.part + (int64_t)blockIdx.x * 2 * a.H + c * PER;
#pragma unroll
        for (int q = 0; q < PER; q += 4) {
            *(f32x4*)(p + q) = f32x4{dg[i][q], dg[i][q + 1], dg[i][q + 2], dg[i][q + 3]};
            *(f32x4*)(p + a.H + q) = f32x4{db[i][q], db[i][q + 1], db[i][q + 2], db[i][q + 3]};
        }
    }
}

// dgamma (y 0) and dbeta (y 1): the parts' sums in order, eight columns a thread
template <class P>
__global__ __launch_bounds__(64) void k_norm_params(NormArgs a, int parts) {
    void* out = blockIdx.y ? a.dbeta : a.dgamma;
    const int at = (blockIdx.x * 64 + threadIdx.x) * 8;
    if (!out || at >= a.H) return;
    float f[8] = {};
    const float* p = a.part + blockIdx.y * a.H + at;
    for (int b = 0; b < parts; ++b) {
        const f32x4 lo = *(const f32x4*)(p + (int64_t)b * 2 * a.H), hi = *(const f32x4*)(p + (int64_t)b * 2 * a.H + 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            f[q] += lo[q];
            f[4 + q] += hi[q];
        }
    }
    if constexpr (P::PER16 == 8) {
        store_params<P, P>(out, at, f);
    } else {
        store_params<P, P>(out, at, f);
        store_params<P, P>(out, at + 4, f + 4);
    }
}

// ================================================================ launchers
// (rows of at most 2^16 elements: 2^14 chunks of fp32, 16 to a thread of 1024)
template <class F>
static int with_shape(int C, const F& f) {
    using std::integral_constant;
    if (C <= 64) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
    if (C <= 256) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
    if (C <= 512) return f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
    if (C <= 1024) return f(integral_constant<int, 4>{}, integral_constant<int, 4>{});
    if (C <= 4096) return f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
    return f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
}

template <class F>
static int with_types(int dtype, int params, const F& f) {
    if (dtype == 2) return f(Fp32{}, Fp32{});
    if (dtype == 1) return params == 1 ? f(Fp16{}, Fp16{}) : f(Fp16{}, Fp32{});
    return params == 0 ? f(Bf16{}, Bf16{}) : f(Bf16{}, Fp32{});
}

int norm_parts(int M, int H, int dtype) {
    return M < 1024 ? M : 1024;
}

int launch_norm(const NormArgs& a, hipStream_t st) {
    ProfScope prof_(st, "norm");
    return with_types(a.dtype, a.params, [&](auto d, auto p) {
        using D = decltype(d);
        using P = decltype(p);
        return with_shape(a.H / D::PER16, [&](auto w, auto n) {
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
            return with_shape(a.H / D::PER16, [&](auto w, auto n) {
                constexpr int W = decltype(w)::value;
                k_norm_bwd<D, P, W, decltype(n)::value><<<parts, 64 * W, 0, st>>>(a, parts);
                return hipGetLastError() == hipSuccess ? 0 : -1;
            });
        });
        if (r || (!a.dgamma && !a.dbeta)) return r;
    }
    ProfScope prof_(st, "norm_params");
    const dim3 grid((a.H + 511) / 512, 2);
    if (a.params == 2) k_norm_params<Fp32><<<grid, 64, 0, st>>>(a, parts);
    else if (a.params == 1) k_norm_params<Fp16><<<grid, 64, 0, st>>>(a, parts);
    else k_norm_params<Bf16><<<grid, 64, 0, st>>>(a, parts);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace moe
