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

// Eight codes (low nibble first) minus zero, as a fragment of D.
template <class D>
__device__ __forceinline__ uint4 codes8(uint32_t w, float zero) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (float)(w >> (4 * i) & 15u) - zero;
    return D::pack(f);
}

// ================================================================ few rows
// 16 rows by 16 columns a block, its W waves split the reduction in units of 128.
template <class D, int ACT, int G, int W>
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
    if (lo + r < hi && nt * 16 + c < f.N) lin_out<D, ACT>(f, e, lo + r, nt * 16 + c, v);
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
LinTiles w4_tiles(int M, int E, int K, int N) { return {nullptr, nullptr, E, M, 16, nullptr}; }

int w4_tile_columns(const LinTiles& t) { return 16; }

template <class D, int G>
static int w4_(const W4Args& a, hipStream_t st) {
    return with_act(a.f.act, [&](auto A) {
        return go(k_w4_stream<D, A(), G, 8>, max_tiles(a.f.t) * ((a.f.N + 15) / 16), 512, a, st);
    });
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
