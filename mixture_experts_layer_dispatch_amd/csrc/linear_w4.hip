// y = act(x W^T + b) + residual with weights of 4 bits and a scale (and zero
// point) per group of 32, 64 or 128 inputs, dense or grouped by expert
// (include/moe.h: moe_linear_w4_forward), and the weights' quantiser:
//
//   W[n, k] = scale[k / G, n] (code[n, k] - zero[k / G, n])
//
// the serving form of linear.hip's products, in whose manner tiles are found
// and outputs made.  The matrix instructions multiply x by the whole numbers
// code - zero, which bf16 and fp16 hold exactly, over one group; the group's
// fp32 sum is then multiplied by its scale and added.  So no weight is rounded
// (rounded to 16 bits first they would put as much error into y as y's own
// rounding), and the scale costs one multiply-add per output and group instead of
// one per weight.
#include "dtype.h"
#include "gemm_common.h"
#include "linear_common.h"
#include "profile.h"
#include "rows.h"
#include "tile256.h"

namespace moe {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------- codes
// A lane's 16 bytes of a row are 32 codes in a row, lane quarter q (16 lanes)
// having those from 32 q on.  Transposed over the quarters (4 x 4 words), word s
// has the codes from 32 s + 8 q on: what a lane of an MFMA over 32 s .. 32 s + 31
// supplies.
__device__ __forceinline__ void transpose_quarters(uint4& v) {
    auto swap32 = [](uint32_t& a, uint32_t& b) {
        const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(a, b, false, false));
        a = r[0];
        b = r[1];
    };
    auto swap16 = [](uint32_t& a, uint32_t& b) {
        const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a, b, false, false));
        a = r[0];
        b = r[1];
    };
    swap32(v.x, v.z);
    swap32(v.y, v.w);
    swap16(v.x, v.y);
    swap16(v.z, v.w);
}

// Eight codes (low nibble first) minus zero, as a fragment of D.  A byte of 0 .. 15
// is an E4M3 number of that many times 2^-9 (subnormal or of the smallest exponent),
// so one conversion makes two codes fp32.
template <class D>
__device__ __forceinline__ uint4 codes8(uint32_t w, float zero) {
    const uint32_t even = w & 0x0f0f0f0fu, odd = w >> 4 & 0x0f0f0f0fu;
    const f32x2 e0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)even, 512.f, false);
    const f32x2 e1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)even, 512.f, true);
    const f32x2 o0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)odd, 512.f, false);
    const f32x2 o1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)odd, 512.f, true);
    return make_uint4(D::pack2(e0[0] - zero, o0[0] - zero), D::pack2(e0[1] - zero, o0[1] - zero),
                      D::pack2(e1[0] - zero, o1[0] - zero), D::pack2(e1[1] - zero, o1[1] - zero));
}

// four consecutive outputs from col, the activation chosen at run time
template <class D>
__device__ __forceinline__ void w4_out(const LinFwdArgs& f, int e, int row, int col, const f32x4& v) {
    switch (f.act) {
        case LIN_RELU: return lin_out<D, LIN_RELU>(f, e, row, col, v);
        case LIN_GELU: return lin_out<D, LIN_GELU>(f, e, row, col, v);
        case LIN_GELU_TANH: return lin_out<D, LIN_GELU_TANH>(f, e, row, col, v);
        case LIN_SILU: return lin_out<D, LIN_SILU>(f, e, row, col, v);
        default: return lin_out<D, LIN_NONE>(f, e, row, col, v);
    }
}

// ================================================================ few rows
// 16 rows by 16 columns a block, its W waves split the reduction in units of 128.
template <class D, int G, int W>
__global__ __launch_bounds__(64 * W) void k_w4_stream(W4Args a) {
    __shared__ __attribute__((aligned(16))) float sums[W][16][20];
    const LinFwdArgs& f = a.f;
    int e, lo, hi, nt, mt;
    if (!lin_tile<16, 1>(f.t, (f.N + 15) / 16, blockIdx.x, e, lo, hi, nt, mt)) return;
    const int lane = lane_id(), wv = wave_id(), j = lane & 15, q = lane >> 4;
    const int col = min(nt * 16 + j, f.N - 1), groups = f.K / G;
    const uint16_t* x = f.x + (int64_t)min(lo + j, hi - 1) * f.K;
    const uint8_t* codes = a.codes + ((int64_t)e * f.N + col) * (f.K / 2);
    const uint16_t* scales = a.scales + (int64_t)e * groups * f.N + col;
    const uint8_t* zeros = a.zeros ? a.zeros + (int64_t)e * groups * f.N + col : nullptr;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int k0 = wv * 128; k0 < f.K; k0 += W * 128) {
        // (behind the row: its last codes, times zeros in place of x)
        uint4 c = *(const uint4*)(codes + min(k0 + 32 * q, f.K - 32) / 2);
        transpose_quarters(c);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        f32x4 part = {0.f, 0.f, 0.f, 0.f};
        float scale = 0.f, zero = 8.f;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int k = k0 + 32 * s;
            if (k >= f.K) break;
            if (k % G == 0) {
                part = f32x4{0.f, 0.f, 0.f, 0.f};
                scale = D::lo(scales[(int64_t)(k / G) * f.N]);
                if (zeros) zero = zeros[(int64_t)(k / G) * f.N];
            }
            part = D::mfma(*(const uint4*)(x + k + 8 * q), codes8<D>(w[s], zero), part);
            if ((k + 32) % G == 0)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[r] = fmaf(scale, part[r], acc[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) sums[wv][4 * q + r][j] = acc[r];
    __syncthreads();
    if (threadIdx.x >= 64) return;
    const int r = threadIdx.x >> 2, c = (threadIdx.x & 3) * 4;
    f32x4 v = *(const f32x4*)&sums[0][r][c];
#pragma unroll
    for (int p = 1; p < W; ++p) v += *(const f32x4*)&sums[p][r][c];
    if (lo + r < hi && nt * 16 + c < f.N) w4_out<D>(f, e, lo + r, nt * 16 + c, v);
}

// ================================================================ tiles
// 16 MB rows by 64 NW columns, a wave all the rows of 64 columns: each weight is
// taken apart once per row tile.  x goes through a ring of three LDS stages of 128
// inputs, copied two steps ahead (in two arrays of 64 each; arrays of their own, so
// that reads wait for no copies in flight), the codes two steps ahead into
// registers.  Lane j of a quarter has the columns 4 j .. 4 j + 3 of its wave's 64, one
// to an MFMA, so that scales come and outputs go as four neighbours.
template <int MB>
struct W4Ring {
    uint16_t* h[3][2];
};

template <class D, int G, int MB, int NW>
struct W4Loop {
    static constexpr int NG = 128 / G, KS = G / 32, NC = 2 * MB * 16 * 8 / (64 * NW);
    const W4Args& a;
    const TileOperand<false, 16 * MB, 1, 64 * NW>& x;
    const W4Ring<MB>& ring;
    const uint8_t* codes[4];      // of the lane's four rows, its quarter's 16 bytes
    const uint16_t* scales;       // of its four columns
    const uint8_t* zeros;
    int steps, lane;
    f32x4 acc[MB][4];             // [rows 16 mb + 4 q + r][column 4 j + nb], r in the vector
    uint4 w[3][4];
    uint2 sc[3][NG];
    uint32_t zr[3][NG];

    __device__ __forceinline__ void load(int s, int buf) {
        const int K = a.f.K, q = lane >> 4;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int kt = 2 * s + h;
            if (kt < K / 64) x.copy(0, kt, ring.h[buf][h]);
            else if (kt == K / 64 && K % 64) x.copy_tail(0, kt, K % 64, ring.h[buf][h]);
        }
        __builtin_amdgcn_sched_barrier(0);
        const int at = min(s * 128 + 32 * q, K - 32) / 2;      // (behind the row: not used)
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) w[buf][nb] = *(const uint4*)(codes[nb] + at);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int64_t row = (int64_t)min(s * NG + g, K / G - 1) * a.f.N;
            sc[buf][g] = *(const uint2*)(scales + row);
            zr[buf][g] = zeros ? *(const uint32_t*)(zeros + row) : 0x08080808u;
        }
        t2_fence();
    }
    template <int BUF>
    __device__ __forceinline__ void step(int s) {
        const int left = steps - 1 - s, K = a.f.K;
        if (left > 1 || (left == 1 && K % 128 == 0)) t2_wait<NC + 8>();
        else t2_wait<0>();
        t2_barrier();
        if (left >= 2) load(s + 2, (BUF + 2) % 3);
        const int ksteps = min(4, (K - s * 128) / 32);
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) transpose_quarters(w[BUF][nb]);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (g * KS >= ksteps) break;
            uint4 b[KS][4];
            const f32x4 scale = unpack4<D>(sc[BUF][g]);
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) {
                const float zero = (float)(zr[BUF][g] >> (8 * nb) & 255u);
                const uint32_t c[4] = {w[BUF][nb].x, w[BUF][nb].y, w[BUF][nb].z, w[BUF][nb].w};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) b[ks][nb] = codes8<D>(c[g * KS + ks], zero);
            }
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                f32x4 part[4];
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const int k = g * KS + ks;
                    const uint4 fx = t2_frag<false>(ring.h[BUF][k >> 1], 16 * mb, 32 * (k & 1));
#pragma unroll
                    for (int nb = 0; nb < 4; ++nb)
                        part[nb] = D::mfma(fx, b[ks][nb], ks ? part[nb] : f32x4{0.f, 0.f, 0.f, 0.f});
                }
#pragma unroll
                for (int nb = 0; nb < 4; ++nb)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[mb][nb][r] = fmaf(scale[nb], part[nb][r], acc[mb][nb][r]);
            }
        }
    }
};

template <class D, int G, int MB, int NW>
__global__ __launch_bounds__(64 * NW, 2) void k_w4_tile(W4Args a) {
    constexpr int TM = 16 * MB, TN = 64 * NW;
    __shared__ __attribute__((aligned(16))) uint16_t s00[TM * 64], s01[TM * 64], s10[TM * 64], s11[TM * 64],
        s20[TM * 64], s21[TM * 64];
    const LinFwdArgs& f = a.f;
    int e, lo, hi, nt, mt;
    if (!lin_tile<TM, 1>(f.t, (f.N + TN - 1) / TN, blockIdx.x, e, lo, hi, nt, mt)) return;
    const W4Ring<MB> ring{{{s00, s01}, {s10, s11}, {s20, s21}}};
    const TileOperand<false, TM, 1, 64 * NW> x(f.x, f.K, lo, hi);
    const int lane = lane_id(), col = nt * TN + 64 * wave_id() + 4 * (lane & 15), colc = min(col, f.N - 4);
    const int64_t ge = (int64_t)e * (f.K / G) * f.N + colc;
    W4Loop<D, G, MB, NW> l{a, x, ring, {}, a.scales + ge, a.zeros ? a.zeros + ge : nullptr, (f.K + 127) / 128, lane};
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
        l.codes[nb] = a.codes + ((int64_t)e * f.N + colc + nb) * (f.K / 2);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) l.acc[mb][nb] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    l.load(0, 0);
    if (l.steps > 1) l.load(1, 1);
    for (int s = 0; s < l.steps; s += 3) {
        l.template step<0>(s);
        if (s + 1 < l.steps) l.template step<1>(s + 1);
        if (s + 2 < l.steps) l.template step<2>(s + 2);
    }
    if (col >= f.N) return;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = lo + 16 * mb + 4 * (lane >> 4) + r;
            if (row < hi) w4_out<D>(f, e, row, col, f32x4{l.acc[mb][0][r], l.acc[mb][1][r], l.acc[mb][2][r], l.acc[mb][3][r]});
        }
}

// ================================================================ quantiser
// A wave takes 512 neighbouring weights of a row, eight to a lane; a group is
// G / 8 lanes.  Quotients of two 16-bit numbers are told from the halves between
// whole numbers by fp32's correctly rounded division.
template <class D, int G>
__global__ __launch_bounds__(256) void k_w4_quant(W4QuantArgs a, int64_t total) {
    const int64_t u = block_number() * 4 + wave_id();
    if (u >= total) return;
    const int pieces = (a.K + 511) / 512, lane = lane_id();
    const int64_t row = u / pieces;
    const int k = (int)(u % pieces) * 512 + lane * 8;
    const bool in = k < a.K;                                   // (whole groups: K is a multiple of G)
    float f[8];
    D::unpack(in ? *(const uint4*)(a.w + row * a.K + k) : make_uint4(0, 0, 0, 0), f);
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, f[i]);
        hi = fmaxf(hi, f[i]);
    }
#pragma unroll
    for (int off = G / 16; off >= 1; off >>= 1) {
        lo = fminf(lo, __shfl_xor(lo, off));
        hi = fmaxf(hi, __shfl_xor(hi, off));
    }
    const double range = a.zeros ? ((double)hi - lo) / 15.0 : (double)fmaxf(hi, -lo) / 7.0;
    const uint32_t sbits = D::pack2((float)range, 0.f) & 0xffffu;
    const float scale = D::lo(sbits);
    float zero = 8.f;
    if (a.zeros) zero = scale > 0.f ? fminf(fmaxf(rintf(-lo / scale), 0.f), 15.f) : 0.f;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float c = scale > 0.f ? fminf(fmaxf(rintf(f[i] / scale) + zero, 0.f), 15.f) : zero;
        w |= (uint32_t)c << (4 * i);
    }
    if (!in) return;
    *(uint32_t*)(a.codes + row * (a.K / 2) + k / 2) = w;
    if (k % G == 0) {
        const int64_t e = row / a.N, at = (e * (a.K / G) + k / G) * a.N + row % a.N;
        a.scales[at] = (uint16_t)sbits;
        if (a.zeros) a.zeros[at] = (uint8_t)zero;
    }
}

// ================================================================ launchers
LinTiles w4_tiles(int M, int E, int K, int N) {
    const int tm = (E ? M <= 8LL * E : M <= 16) ? 16 : 64;
    return {nullptr, nullptr, E, M, tm, nullptr};
}

int w4_tile_columns(const LinTiles& t) { return t.tm == 16 ? 16 : 256; }

template <class D, int G>
static int w4_(const W4Args& a, hipStream_t st) {
    const int64_t grid = max_tiles(a.f.t) * ((a.f.N + w4_tile_columns(a.f.t) - 1) / w4_tile_columns(a.f.t));
    if (a.f.t.tm == 16) return go(k_w4_stream<D, G, 8>, grid, 512, a, st);
    return go(k_w4_tile<D, G, 4, 4>, grid, 256, a, st);
}

template <class F>
static int with_group(int G, const F& f) {
    if (G == 32) return f(std::integral_constant<int, 32>{});
    if (G == 64) return f(std::integral_constant<int, 64>{});
    return f(std::integral_constant<int, 128>{});
}

int launch_w4(const W4Args& a, hipStream_t st) {
    ProfScope prof_(st, "linear_w4");
    return with_group(a.G, [&](auto g) {
        return a.f.dtype == 0 ? w4_<Bf16, decltype(g)::value>(a, st) : w4_<Fp16, decltype(g)::value>(a, st);
    });
}

int launch_w4_quant(const W4QuantArgs& a, hipStream_t st) {
    ProfScope prof_(st, "linear_w4_quantize");
    const int64_t total = a.rows * ((a.K + 511) / 512);
    const dim3 grid = rows_grid((total + 3) / 4);
    return with_group(a.G, [&](auto g) {
        if (a.dtype == 0) k_w4_quant<Bf16, decltype(g)::value><<<grid, 256, 0, st>>>(a, total);
        else k_w4_quant<Fp16, decltype(g)::value><<<grid, 256, 0, st>>>(a, total);
        return ok();
    });
}

}  // namespace moe
