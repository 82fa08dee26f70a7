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

// Eight codes (low nibble first) as they are, 0 .. 15, as a fragment of D.  A byte of
// 0 .. 15 is an E4M3 number of that many times 2^-9 (subnormal or of the smallest
// exponent), so one conversion makes two codes.
template <class D>
__device__ __forceinline__ uint4 codes8(uint32_t w) {
    const uint32_t even = w & 0x0f0f0f0fu, odd = w >> 4 & 0x0f0f0f0fu;
    const int lo = (int)__builtin_amdgcn_perm(odd, even, 0x05010400u);
    const int hi = (int)__builtin_amdgcn_perm(odd, even, 0x07030602u);
    auto two = [](int v, auto upper) {
        if constexpr (std::is_same<D, Bf16>::value)
            return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 512.f, decltype(upper)::value));
        else
            return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 512.f, decltype(upper)::value));
    };
    return make_uint4(two(lo, std::false_type{}), two(lo, std::true_type{}), two(hi, std::false_type{}),
                      two(hi, std::true_type{}));
}

// The same minus zero, exactly: fp16 by pairs, bf16 by way of fp32.
template <class D>
__device__ __forceinline__ uint4 codes8(uint32_t w, float zero) {
    if constexpr (std::is_same<D, Fp16>::value) {
        const uint4 v = codes8<D>(w);
        const f16x2 z = {(_Float16)zero, (_Float16)zero};
        auto sub = [&](uint32_t p) { return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, p) - z); };
        return make_uint4(sub(v.x), sub(v.y), sub(v.z), sub(v.w));
    } else {
        const int even = (int)(w & 0x0f0f0f0fu), odd = (int)(w >> 4 & 0x0f0f0f0fu);
        const f32x2 e0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(even, 512.f, false);
        const f32x2 e1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(even, 512.f, true);
        const f32x2 o0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(odd, 512.f, false);
        const f32x2 o1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(odd, 512.f, true);
        return make_uint4(D::pack2(e0[0] - zero, o0[0] - zero), D::pack2(e0[1] - zero, o0[1] - zero),
                          D::pack2(e1[0] - zero, o1[0] - zero), D::pack2(e1[1] - zero, o1[1] - zero));
    }
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

// f with the activation as a type
template <class F>
__device__ __forceinline__ void dev_act(int act, const F& f) {
    switch (act) {
        case LIN_RELU: f(std::integral_constant<int, LIN_RELU>{}); break;
        case LIN_GELU: f(std::integral_constant<int, LIN_GELU>{}); break;
        case LIN_GELU_TANH: f(std::integral_constant<int, LIN_GELU_TANH>{}); break;
        case LIN_SILU: f(std::integral_constant<int, LIN_SILU>{}); break;
        default: f(std::integral_constant<int, LIN_NONE>{});
    }
}

// what is taken off the codes: 8, by the sums of x; 8, exactly; zeros, exactly
enum { W4_MID, W4_EIGHT, W4_ZEROS };

// By the sums of x, an infinite x makes all outputs of its row NaN, and x beyond 2^128 / (15 G)
// can take sums of the codes past fp32's range where those of code - 8 are inside it.  No sum that
// has left it comes back, so what comes out finite is right, and the waves that have other
// sums replace them by exact ones, straight from memory; but for rows that have a NaN,
// which is what they come out as, so that a padded batch need not be cleared.  2048 x 4096 x
// 4096 takes 76 us; a call with its launch 82, with an infinite x in one row 328, in all 631,
// with one row of random bits 84, with only such rows 110.
__device__ __forceinline__ bool finite(float v) { return fabsf(v) < INFINITY; }

// Which of `rows` (bit j: row row0 + j, 16 of them) have a NaN in x (bf16)
__device__ __forceinline__ uint32_t nan_rows(const LinFwdArgs& f, int row0, int hi, uint32_t rows) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    const int j = lane_id() & 15, q = lane_id() >> 4;
    const uint16_t* x = f.x + (int64_t)min(row0 + j, hi - 1) * f.K + 8 * q;
    uint32_t found = 0;
    for (int k = 0; k < f.K && (rows & ~found); k += 256) {
        u16x2 most = {0, 0};
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint4 v = *(const uint4*)(x + min(k + 32 * u, f.K - 32));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
        }
        uint64_t m = __ballot(most[0] > 0x7f80 || most[1] > 0x7f80);
        m |= m >> 32;
        found |= (uint32_t)(m | m >> 16) & 0xffffu;
    }
    return rows & found;
}

// ================================================================ few rows
// Exact sums of 16 rows from row0 by 16 columns from col0: lane j + 16 q has row j's
// columns 4 q .. 4 q + 3.
template <class D, int G>
__device__ __forceinline__ f32x4 w4_exact16(const W4Args& a, int e, int row0, int hi, int col0) {
    const LinFwdArgs& f = a.f;
    const int j = lane_id() & 15, q = lane_id() >> 4, groups = f.K / G;
    const uint16_t* x = f.x + (int64_t)min(row0 + j, hi - 1) * f.K + 8 * q;
    const uint8_t* codes = a.codes + ((int64_t)e * f.N + min(col0 + j, f.N - 1)) * (f.K / 2) + 4 * q;
    const uint16_t* scales = a.scales + (int64_t)e * groups * f.N + min(col0 + 4 * q, f.N - 4);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int g = 0; g < groups; ++g) {
        f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < G / 32; ++s) {
            const int k = g * G + 32 * s;
            part = D::mfma(codes8<D>(*(const uint32_t*)(codes + k / 2), 8.f), *(const uint4*)(x + k), part);
        }
        const f32x4 scale = unpack4<D>(*(const uint2*)(scales + (int64_t)g * f.N));
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] = fmaf(scale[r], part[r], acc[r]);
    }
    return acc;
}

// A handful of rows: the codes are read once and everything else is small, so the
// product is a stream.  A block computes 16 rows by 16 NB columns; its W waves split
// the reduction in units of 128 inputs, whose codes they read straight into registers,
// UNITS at a time.  A lane quarter reads 16 bytes of a row, 32 inputs in a row; groups of
// 128 are multiplied in that order (word s of every quarter, and the same inputs of x,
// to an MFMA), smaller ones are first transposed over the quarters.  (The second launch bound
// keeps two blocks to a CU; 64 columns are faster without: 4096 -> 65536 27.5 us, 29.5 with it.)
template <class D, int G, int MODE, int NB, int W, int UNITS>
__global__ __launch_bounds__(64 * W, NB == 4 ? 1 : W / 2) void k_w4_stream(W4Args a) {
    constexpr int TN = 16 * NB, NG = 128 / G, PER = G / 32;
    __shared__ __attribute__((aligned(16))) float sums[W][16][TN + 4];
    const LinFwdArgs& f = a.f;
    int e, lo, hi, nt, mt;
    if (!lin_tile<16, 1>(f.t, (f.N + TN - 1) / TN, blockIdx.x, e, lo, hi, nt, mt)) return;
    const int lane = lane_id(), wv = wave_id(), j = lane & 15, q = lane >> 4, groups = f.K / G;
    const uint16_t* x = f.x + (int64_t)min(lo + j, hi - 1) * f.K;
    const uint8_t* codes[NB];
    int64_t ge[NB];
    f32x4 acc[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        const int col = min(nt * TN + 16 * n + j, f.N - 1);
        codes[n] = a.codes + ((int64_t)e * f.N + col) * (f.K / 2);
        ge[n] = (int64_t)e * groups * f.N + col;
        acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const int units = (f.K + 127) / 128;
    for (int u0 = wv; u0 < units; u0 += W * UNITS) {
        uint4 c[UNITS][NB];
        uint16_t sc[UNITS][NB][NG];
        uint8_t zr[UNITS][NB][NG];
        uint4 xv[UNITS][4];
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int k0 = min(u0 + u * W, units - 1) * 128;   // (one behind the last: read, not added)
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                c[u][n] = *(const uint4*)(codes[n] + min(k0 + 32 * q, f.K - 32) / 2);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const int64_t at = ge[n] + (int64_t)min(k0 / G + g, groups - 1) * f.N;
                    sc[u][n][g] = a.scales[at];
                    if (MODE == W4_ZEROS) zr[u][n][g] = a.zeros[at];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int k0 = min(u0 + u * W, units - 1) * 128;
#pragma unroll
            for (int s = 0; s < 4; ++s)
                xv[u][s] = *(const uint4*)(x + (G == 128 ? k0 + 32 * q + 8 * s : min(k0 + 32 * s, f.K - 32) + 8 * q));
        }
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            if (u0 + u * W >= units) break;
            const int k0 = (u0 + u * W) * 128;
#pragma unroll
            for (int n = 0; n < NB; ++n)
                if (G < 128) transpose_quarters(c[u][n]);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if (g > 0 && k0 + g * G >= f.K) break;
                f32x4 start = {0.f, 0.f, 0.f, 0.f};
                if (MODE == W4_MID) {
#pragma unroll
                    for (int s = g * PER; s < (g + 1) * PER; ++s)
                        start = D::mfma(xv[u][s], make_uint4(0xc100c100u, 0xc100c100u, 0xc100c100u, 0xc100c100u), start);
                }
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const uint32_t w[4] = {c[u][n].x, c[u][n].y, c[u][n].z, c[u][n].w};
                    f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = g * PER; s < (g + 1) * PER; ++s) {
                        uint4 b;
                        if constexpr (MODE == W4_MID) b = codes8<D>(w[s]);
                        else b = codes8<D>(w[s], MODE == W4_ZEROS ? (float)zr[u][n][g] : 8.f);
                        part = D::mfma(xv[u][s], b, part);
                    }
                    const float scale = D::lo(sc[u][n][g]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[n][r] = fmaf(scale, MODE == W4_MID ? part[r] + start[r] : part[r], acc[n][r]);
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) sums[wv][4 * q + r][16 * n + j] = acc[n][r];
    __syncthreads();
    if (threadIdx.x >= 64 * NB) return;
    const int r = threadIdx.x / (4 * NB), c = threadIdx.x % (4 * NB) * 4;
    f32x4 v = *(const f32x4*)&sums[0][r][c];
#pragma unroll
    for (int p = 1; p < W; ++p) v += *(const f32x4*)&sums[p][r][c];
    if constexpr (MODE == W4_MID) {
        const bool bad = !(finite(v[0]) && finite(v[1]) && finite(v[2]) && finite(v[3]));
        if (uint64_t m = __ballot(bad && lo + r < hi); __builtin_expect(m != 0, 0)) {
            uint32_t rows = 0;                 // (a wave has whole rows)
            for (; m; m &= m - 1) rows |= 1u << ((64 * wv + __builtin_ctzll(m)) / (4 * NB));
            rows &= ~nan_rows(f, lo, hi, rows);
            for (int n = 0; n < NB && rows; ++n) {
                const f32x4 y = w4_exact16<D, G>(a, e, lo, hi, nt * TN + 16 * n);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float t = __shfl(y[i], r + 16 * (c >> 2 & 3));
                    if (bad && c >> 4 == n) v[i] = t;
                }
            }
        }
    }
    if (lo + r < hi && nt * TN + c < f.N) w4_out<D>(f, e, lo + r, nt * TN + c, v);
}

// ================================================================ tiles
// 64 rows by 512 columns, eight waves with all the rows of 64 columns each (2 x 2 MFMAs
// of 32 x 32), so that each weight is taken apart once per row tile; steps of 128
// inputs.  Lane j of a half wave has the columns 2 j and 2 j + 1 of its wave's 64, one to
// an MFMA.  A pair of MFMA steps, 32 inputs (number c), takes the 16-byte chunk c of a
// weight row: lane half h its words 2 h and 2 h + 1, one to a step, and of x the same
// inputs.
//
// All operands are copied into LDS, two steps ahead and never drained: x in three
// stages that the block shares, a wave's codes in three and its scales and zeros in two
// stages of its own (what a wave copies, only it reads: no barrier).  The stages are
// arrays of their own, since a read waits for the copies in flight into its array.  A
// load into registers in the loop would wait for every copy before it.
//
// MID: the MFMAs multiply the codes themselves, and their sums start at -8 times the
// sum of x over the group, which each wave computes for the eight rows that it copied,
// one step ahead (bf16 codes minus 8 take twice the instructions).
//
// Bounds: two waves a SIMD that convert and multiply in turn.  8192 x 4096 x 4096 takes 283 us,
// 0.97 PFLOP/s: MFMAs are 49 % of the SIMDs' cycles, other vector instructions 50 %, at 2.06 GHz.
// 20480 rows at 512 experts, 4096 -> 1024, 343 us, its 1.3 GB at 3.85 TB/s.  Groups of 32
// multiply and add 64 sums four times a step: 1024 x 4096 x 4096 61 us, 31 % and 59 % (groups
// of 128 49 us, 44 % and 46 %); 1111 x 4104 x 4032 fp16 with zeros 93 us: its 162 tiles leave a
// third of the CUs idle.
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <class D>
__device__ __forceinline__ f32x16 mfma32(const uint4& x, const uint4& w, const f32x16& c) {
    if constexpr (std::is_same<D, Bf16>::value)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, w), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, w), c, 0, 0, 0);
}

// v of the lanes 1, 2 and 7 (in bits) from this one
template <int CTRL>
__device__ __forceinline__ float dpp_lane(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float lane_xor1(float v) { return dpp_lane<0xb1>(v); }
__device__ __forceinline__ float lane_xor2(float v) { return dpp_lane<0x4e>(v); }
__device__ __forceinline__ float lane_xor7(float v) { return dpp_lane<0x141>(v); }

// SIZE bytes a lane (16 or 4) to the wave's part of an LDS array, lane by lane; the
// address a scalar and a 32-bit offset
template <int SIZE>
__device__ __forceinline__ void copy_lds(const char* base, uint32_t o, void* dst) {
    asm volatile("" : "+v"(o));
    if constexpr (SIZE == 16) __builtin_amdgcn_global_load_lds((glb_void_t*)(base + o), (lds_void_t*)dst, 16, 0, 0);
    else __builtin_amdgcn_global_load_lds((glb_void_t*)(base + o), (lds_void_t*)dst, 4, 0, 0);
}

constexpr int kW4Waves = 8, kW4Cols = 64 * kW4Waves;

template <class D, int G, int MODE>
struct W4Loop {
    static constexpr bool MID = MODE == W4_MID;
    static constexpr int NG = 128 / G, PER = G / 16;      // groups of a step, MFMA steps of a group
    static constexpr bool ZEROS = MODE == W4_ZEROS;
    static constexpr int SC = (NG + 1) / 2;               // copies of scales, two groups each
    static constexpr int NS = SC + ZEROS;                 // and with that of zeros
    int K, N, lane;
    int last;                     // the part's steps end here
    uint16_t* xs[3];              // [half of 64 inputs][64 rows]
    uint8_t* ws[3];               // the wave's 4 KB of a stage
    uint8_t* ss[2];               // its 256 NS bytes: [group][column 2 j + n] scales, [group][column] zeros
    float* sums;                  // [2][NG][64] MID: -8 times the sums of x
    const char *x, *codes, *scales, *zeros;               // of the tile's first row, of its expert and first column
    uint32_t xo, xk;              // the thread's row and chunk of x, the chunk's first input in 64
    uint32_t co[4], ck;           // its rows and its chunk of codes, the chunk's place in 64 bytes
    uint32_t so, zo;              // its two columns, the four whose zeros it copies
    uint32_t at[2];               // its columns' first words in a stage
    f32x16 acc[2][2];             // [rows 32 m + 8 (r / 4) + 4 h + r % 4][column 2 j + n]

    // Steps behind the last are the last one again, so that every step has the same copies
    // in flight; inputs behind the rows are their last ones again, and their groups are
    // not added.
    __device__ __forceinline__ void load_x(int s, int buf, int h) {
        s = min(s, last - 1);
        const int k0 = min(s * 128 + 64 * h, (K - 1) / 64 * 64);
        uint32_t back = 0;                                     // (at most the chunk's place in the row)
        if (G < 128 && k0 + 64 > K) back = (uint32_t)max(k0 + (int)xk + 8 - K, 0) * 2;
        copy_lds<16>(x + (int64_t)k0 * 2, xo - back, xs[buf] + h * 4096 + wave_id() * 512);
    }
    __device__ __forceinline__ void load_codes(int s, int buf, int i) {
        s = min(s, last - 1);
        uint32_t back = 0;
        if (G < 128 && s * 128 + 128 > K) back = (uint32_t)max(s * 64 + (int)ck + 16 - K / 2, 0);   // (at most ck)
        copy_lds<16>(codes + s * 64, co[i] - back, ws[buf] + i * 1024);
    }
    __device__ __forceinline__ void load_scales(int s, int buf) {
#pragma unroll
        for (int i = 0; i < SC; ++i) {                         // lane half h: group 2 i + h
            const int row = min(s * NG + min(2 * i + (lane >> 5), NG - 1), K / G - 1);
            copy_lds<4>(scales, ((uint32_t)row * N + so) * 2, ss[buf] + i * 256);
        }
        if (ZEROS) {                                           // lane quarter q: group q
            const int row = min(s * NG + min(lane >> 4, NG - 1), K / G - 1);
            copy_lds<4>(zeros, (uint32_t)row * N + zo, ss[buf] + SC * 256);
        }
    }
    // copy number i of a step's (all of the scales are one), spread over the MFMAs of the
    // step two before: in one place they hold up the wave
    __device__ __forceinline__ void load(int i, int s, int xw, int sb) {
        if (i < 2) load_x(s, xw, i);
        else if (i == 2) load_scales(s, sb);
        else if (i < 7) load_codes(s, xw, i - 3);
    }
    // The sums of the wave's eight rows over a step's groups, by the lanes that copied them:
    // a lane adds its 16 bytes of each half (two inputs an instruction, in fp32) and
    // the eight lanes of a row meet in shuffles.  (By 16 x 16 MFMAs of x and -8, each
    // waiting for the one before: 8192 x 4096 x 4096 298 instead of 286 us.)
    __device__ __forceinline__ void put_sums(int xb, int buf) {
        if constexpr (MID) {
            // (in assembly, with its wait: the compiler would wait for the copies in flight
            // in every second step, and counts them right in the others)
            const uint32_t at = (uint32_t)(uintptr_t)(lds_void_t*)(xs[xb] + wave_id() * 512 + lane * 8);
            typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
            u32x4_t v[2];
            asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %2 offset:8192\n\ts_waitcnt lgkmcnt(0)"
                         : "=&v"(v[0]), "=&v"(v[1])
                         : "v"(at)
                         : "memory");
            float t[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                t[h] = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t two = v[h][i], m8 = 0xc100c100u;            // -8, -8
                    t[h] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, two), __builtin_bit_cast(bf16x2, m8), t[h], false);
                }
            }
            if (G == 128) t[0] += t[1];
            const int row = 8 * wave_id() + (lane >> 3);
#pragma unroll
            for (int h = 0; h < (G == 128 ? 1 : 2); ++h) {
                t[h] += lane_xor1(t[h]);
                t[h] += lane_xor2(t[h]);
                if (G > 32) t[h] += lane_xor7(t[h]);
                // (G of 32: four lanes have chunks 0 .. 3 or 4 .. 7 of the half)
                const int g = G == 32 ? 2 * h + ((lane >> 2 & 1) ^ (row >> 3 & 1)) : h;
                if ((lane & (G == 32 ? 3 : 7)) == 0) sums[(buf * NG + g) * 64 + row] = t[h];
            }
        }
    }
    // x's fragment of 32 rows for MFMA step t = 2 c + u
    __device__ __forceinline__ uint4 frag(int xb, int m, int t) {
        const int j = lane & 31, h = lane >> 5;
        return *(const uint4*)(xs[xb] + (t >> 2) * 4096 + kc_off(32 * m + j, 16 * ((2 * t - (t & 1) + 2 * h) & 7)));
    }
    // In flight at the top of a step: its own copies; then, not waited for, the next
    // step's.  W: s % 3, S: s % 2.
    template <int W, int S>
    __device__ __forceinline__ void step(int s) {
        t2_wait<6 + NS>();
        t2_barrier();
        uint4 b[2][2], fx[4][2];                               // [MFMA step][n or m]
        uint2 w[2];
        uint32_t sc[NG], zr[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            sc[g] = *(const uint32_t*)(ss[S] + g * 128 + (lane & 31) * 4);
            if (ZEROS) zr[g] = *(const uint16_t*)(ss[S] + SC * 256 + g * 64 + (lane & 31) * 2);
        }
        auto take = [&](int t) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                // (at: two addresses that the compiler cannot put together, or it reads both
                // columns' words at once and then waits for the copies in flight, no longer
                // knowing what is read)
                if (t % 2 == 0) w[n] = *(const uint2*)(ws[W] + (at[n] ^ (t / 2 * 16)));
                const uint32_t v = t % 2 ? w[n].y : w[n].x;
                if constexpr (MID) b[t & 1][n] = codes8<D>(v);
                else if constexpr (ZEROS) b[t & 1][n] = codes8<D>(v, (float)(zr[t / PER] >> (8 * n) & 255u));
                else b[t & 1][n] = codes8<D>(v, 8.f);
            }
        };
        auto fetch = [&](int t) {
#pragma unroll
            for (int m = 0; m < 2; ++m) fx[t & 3][m] = frag(W, m, t);
        };
        fetch(0);
        take(0);
        fetch(1);
        f32x16 part[2][2];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            if (t % PER == 0) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            f32x4 v = {0.f, 0.f, 0.f, 0.f};
                            if (MID) v = *(const f32x4*)(sums + (S * NG + t / PER) * 64 + 32 * m + 8 * i + 4 * (lane >> 5));
#pragma unroll
                            for (int r = 0; r < 4; ++r) part[m][n][4 * i + r] = v[r];
                        }
            }
            if (t < 6) fetch(t + 2);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < 2; ++n) part[m][n] = mfma32<D>(fx[t & 3][m], b[t & 1][n], part[m][n]);
            load(t, s + 2, (W + 2) % 3, S);
            if (t < 7) take(t + 1);
            if (MID && t == 6) {
                t2_wait<10 + 2 * NS>();                        // the wave's copies of the next x
                t2_fence();
                put_sums((W + 1) % 3, S ^ 1);
            }
            if (t % PER == PER - 1 && (NG == 1 || s * NG + t / PER < K / G)) {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float scale = n ? D::hi(sc[t / PER]) : D::lo(sc[t / PER]);
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int r = 0; r < 16; ++r) acc[m][n][r] = fmaf(scale, part[m][n][r], acc[m][n][r]);
                }
            }
        }
    }
};

// Exact sums of 32 rows from row0 by the lanes' columns over the groups from g0 to g1, in the layout
// of the loop's (lane halves have the same 32 columns).
template <class D, int G>
__device__ __forceinline__ f32x16 w4_exact32(const W4Args& a, int e, int row0, int hi, int col, int g0, int g1) {
    const LinFwdArgs& f = a.f;
    const int j = lane_id() & 31, h = lane_id() >> 5, groups = f.K / G;
    col = min(col, f.N - 1);
    const uint16_t* x = f.x + (int64_t)min(row0 + j, hi - 1) * f.K + 8 * h;
    const uint8_t* codes = a.codes + ((int64_t)e * f.N + col) * (f.K / 2) + 4 * h;
    const uint16_t* scales = a.scales + (int64_t)e * groups * f.N + col;
    f32x16 acc, part;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.f;
    for (int g = g0; g < min(g1, groups); ++g) {
#pragma unroll
        for (int r = 0; r < 16; ++r) part[r] = 0.f;
#pragma unroll
        for (int s = 0; s < G / 16; ++s) {
            const int k = g * G + 16 * s;
            part = mfma32<D>(*(const uint4*)(x + k), codes8<D>(*(const uint32_t*)(codes + k / 2), 8.f), part);
        }
        const float scale = D::lo(scales[(int64_t)g * f.N]);
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[r] = fmaf(scale, part[r], acc[r]);
    }
    return acc;
}

template <class D, int G, int MODE>
__global__ __launch_bounds__(64 * kW4Waves, 2) void k_w4_tile(W4Args a) {
    typedef W4Loop<D, G, MODE> Loop;
    constexpr int TM = 64, TN = kW4Cols, XS = TM * 128, WS = TN * 64, SS = kW4Waves * Loop::NS * 256;
    __shared__ __attribute__((aligned(16))) uint16_t x0[XS], x1[XS], x2[XS];
    __shared__ __attribute__((aligned(16))) uint8_t w0[WS], w1[WS], w2[WS], s0[SS], s1[SS];
    __shared__ __attribute__((aligned(16))) float sums[Loop::MID ? 2 * Loop::NG * 64 : 4];
    const LinFwdArgs& f = a.f;
    int e, lo, hi, nt, mt;
    const int ks = f.ksplit, part = ks > 1 ? blockIdx.x % ks : 0;
    if (!lin_tile<TM, 1>(f.t, (f.N + TN - 1) / TN, ks > 1 ? blockIdx.x / ks : blockIdx.x, e, lo, hi, nt, mt)) return;
    const int lane = lane_id(), wv = wave_id(), n0 = nt * TN, col = n0 + 64 * wv + 2 * (lane & 31);
    const int64_t ge = (int64_t)e * (f.K / G) * f.N + n0;
    Loop l;
    l.K = f.K;
    l.N = f.N;
    const int steps = (f.K + 127) / 128, first = (int)((int64_t)steps * part / ks);
    l.last = (int)((int64_t)steps * (part + 1) / ks);
    l.lane = lane;
    l.xs[0] = x0; l.xs[1] = x1; l.xs[2] = x2;
    l.ws[0] = w0 + wv * 4096; l.ws[1] = w1 + wv * 4096; l.ws[2] = w2 + wv * 4096;
    l.ss[0] = s0 + wv * Loop::NS * 256; l.ss[1] = s1 + wv * Loop::NS * 256;
    l.sums = sums;
    l.x = (const char*)(f.x + (int64_t)lo * f.K);
    l.codes = (const char*)a.codes + ((int64_t)e * f.N + n0) * (f.K / 2);
    l.scales = (const char*)(a.scales + ge);
    l.zeros = a.zeros ? (const char*)a.zeros + ge : nullptr;
    {
        // chunk c of row r goes to slot c ^ (r / 2 % 8) (kc_off)
        const int r = threadIdx.x >> 3, c = (threadIdx.x & 7) ^ (r >> 1 & 7);
        l.xk = 8 * c;
        l.xo = (uint32_t)min(r, hi - lo - 1) * f.K * 2 + 16 * c;
    }
    l.so = min(64 * wv + 2 * (lane & 31), f.N - 2 - n0);
    l.zo = min(64 * wv + 4 * (lane & 15), f.N - 4 - n0);
    l.ck = 16 * ((lane & 3) ^ (lane >> 4));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // copy i of lane l goes to row 16 i + l / 4 of the wave's stage (column 2 j + n at 32 n + j), slot l % 4
        // with chunk l % 4 ^ j / 4 % 4
        const int r = 16 * i + (lane >> 2), j = r & 31, n = r >> 5;
        l.co[i] = (uint32_t)min(64 * wv + 2 * j + n, f.N - 1 - n0) * (f.K / 2) + l.ck;
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        l.at[n] = n * 2048 + (lane & 31) * 64 + (lane >> 2 & 3) * 16 + (lane >> 5) * 8;
        asm volatile("" : "+v"(l.at[n]));
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int r = 0; r < 16; ++r) l.acc[m][n][r] = 0.f;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 7; ++i) l.load(i, first + s, s, s);
    if (Loop::MID) {
        t2_wait<10 + 2 * Loop::NS>();
        t2_fence();
        l.put_sums(0, 0);
    }
    // (left at once after the last step: the compiler counts what may be in flight at a
    // read over every way that leads there)
    for (int s = first;; s += 6) {
        l.template step<0, 0>(s);
        if (s + 1 >= l.last) break;
        l.template step<1, 1>(s + 1);
        if (s + 2 >= l.last) break;
        l.template step<2, 0>(s + 2);
        if (s + 3 >= l.last) break;
        l.template step<0, 1>(s + 3);
        if (s + 4 >= l.last) break;
        l.template step<1, 0>(s + 4);
        if (s + 5 >= l.last) break;
        l.template step<2, 1>(s + 5);
        if (s + 6 >= l.last) break;
    }
    t2_wait<0>();                              // (the copies of the last step again)
    if constexpr (Loop::MID) {
        f32x4 t = {0.f, 0.f, 0.f, 0.f};        // 0, or NaN where a sum is not finite
#pragma unroll
        for (int i = 0; i < 64; ++i) t[i & 3] = fmaf(l.acc[i >> 5][i >> 4 & 1][i & 15], 0.f, t[i & 3]);
        if (__builtin_expect(__ballot(t[0] + t[1] + t[2] + t[3] != 0.f) != 0, 0)) {
            uint64_t rows = 0;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const uint64_t b = __ballot(!finite(l.acc[m][0][r]) || !finite(l.acc[m][1][r]));
                    rows |= (uint64_t)(((uint32_t)b ? 1 : 0) | (b >> 32 ? 16 : 0)) << (32 * m + 8 * (r >> 2) + (r & 3));
                }
            if (hi - lo < TM) rows &= (1ull << (hi - lo)) - 1;
            for (int i = 0; i < TM; i += 16)
                if (rows >> i & 0xffff) rows &= ~((uint64_t)nan_rows(f, lo + i, hi, (uint32_t)(rows >> i) & 0xffffu) << i);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                if (!(uint32_t)(rows >> 32 * m)) continue;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const f32x16 y = w4_exact32<D, G>(a, e, lo + 32 * m, hi, col + n, first * Loop::NG, l.last * Loop::NG);
#pragma unroll
                    for (int r = 0; r < 16; ++r) l.acc[m][n][r] = finite(l.acc[m][n][r]) ? l.acc[m][n][r] : y[r];
                }
            }
        }
    }
    if (col >= f.N) return;
    if (ks > 1) {                              // k_w4_sum does the rest
        float* out = f.part + (int64_t)part * f.t.rows * f.N + col;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = lo + 32 * m + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
                if (row < hi) *(f32x2*)(out + (int64_t)row * f.N) = f32x2{l.acc[m][0][r], l.acc[m][1][r]};
            }
        return;
    }
    float bias[2] = {0.f, 0.f};
    if (f.bias) {
        const uint32_t v = *(const uint32_t*)(f.bias + (int64_t)e * f.N + col);
        bias[0] = D::lo(v);
        bias[1] = D::hi(v);
    }
    // 16 rows at a time, their residual (which may be y) loaded ahead of their stores
    auto out = [&](auto A) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            uint32_t res[16];
            const int r0 = lo + 32 * m + 4 * (lane >> 5);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = r0 + 8 * (r >> 2) + (r & 3);
                res[r] = f.residual ? *(const uint32_t*)(f.residual + (int64_t)min(row, hi - 1) * f.N + col) : 0u;
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = r0 + 8 * (r >> 2) + (r & 3);
                float v[2];
#pragma unroll
                for (int n = 0; n < 2; ++n) v[n] = act<decltype(A)::value>(l.acc[m][n][r] + bias[n]);
                if (row < hi)
                    *(uint32_t*)(f.y + (int64_t)row * f.N + col) = D::pack2(v[0] + D::lo(res[r]), v[1] + D::hi(res[r]));
            }
        }
    };
    dev_act(f.act, out);
}

// The parts of a split reduction, added in order: eight rows of a tile, 128 columns.
template <class D>
__global__ __launch_bounds__(256) void k_w4_sum(W4Args a) {
    const LinFwdArgs& f = a.f;
    int e, lo, hi, nt, mt;
    if (!lin_tile<64, 1>(f.t, (f.N + 127) / 128, blockIdx.x / 8, e, lo, hi, nt, mt)) return;
    const int row = lo + blockIdx.x % 8 * 8 + (threadIdx.x >> 5), col = nt * 128 + (threadIdx.x & 31) * 4;
    if (row >= hi || col >= f.N) return;
    f32x4 v = *(const f32x4*)(f.part + (int64_t)row * f.N + col);
#pragma unroll 4
    for (int q = 1; q < f.ksplit; ++q) v += *(const f32x4*)(f.part + ((int64_t)q * f.t.rows + row) * f.N + col);
    w4_out<D>(f, e, row, col, v);
}

// ================================================================ quantiser
// v, not negative, as fp32 for a rounding to 16 bits: towards zero, the last bit set where
// something is lost, so that the second rounding is v's own (the quotient of a group with
// zeros can lie closer to halfway between two fp16 numbers than fp32 tells apart).
__device__ __forceinline__ float to_odd(double v) {
    const float f = __double2float_rz(v);
    return (double)f == v ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

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
    const uint32_t sbits = D::pack2(to_odd(range), 0.f) & 0xffffu;
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
// The tiles of a product and the parts of its reduction.  Few rows go as a stream, 16
// at a time (512 experts, 4096 -> 1024: of 8 rows 291 us, in tiles of 64 rows 336; of 12
// 335 both, of 16 395 and 339; dense 4096 x 4096, 32 rows 12 and 18, 64 rows 15 and 19), by the
// groups' mean: the host does not know each (6000 rows at those experts evenly 326 us, by a
// Zipf law with 1136 at most 374).  A round of tiles over the 256 CUs takes 2.3 us a step of 128
// inputs, its beginning and end about 5; parts cost a launch more (6 us) and their sums'
// way through memory.  (The step is that of bf16 in groups of 128; groups of 32 with zeros
// take 2.9, and one cost serves both.)
W4Plan w4_plan(int M, int E, int K, int N) {
    W4Plan p{{nullptr, nullptr, E, M, (E ? M <= 12LL * E : M <= 64) ? 16 : 64, nullptr}, 1};
    if (p.t.tm == 16) return p;
    const int64_t tiles = max_tiles(p.t) * ((N + kW4Cols - 1) / kW4Cols);
    const int steps = (K + 127) / 128;
    float least = 1e30f;
    for (int ks = 1; ks <= 16 && ks * 2 <= steps + 1; ++ks) {
        const float us = (float)((tiles * ks + 255) / 256) * (2.3f * ((steps + ks - 1) / ks) + 5.f) +
                         (ks > 1 ? 6.f + 2.5e-6f * ks * M * N : 0.f);
        if (us < least) {
            least = us;
            p.ksplit = ks;
        }
    }
    return p;
}

int w4_tile_columns(const W4Plan& p) { return p.t.tm == 16 ? 16 : kW4Cols; }

template <class D, int G, int MODE>
static int w4_(const W4Args& a, hipStream_t st) {
    const LinFwdArgs& f = a.f;
    const int64_t tiles = max_tiles(f.t);
    if (f.t.tm == 16) {
        // Several columns of 16 share the loads of x, and few waves a block's beginning and
        // end, where the blocks are enough for the chip.  By 16, 32 and 64 columns, us, K 4096:
        // 4 rows, N 4096 6.1, 7.2, 10.5; 8192 8.6, 7.3, 10.6; 16384 14.2, 11.3, 13.2; 32768 24.3,
        // 18.8, 19.1; 65536 46.6, 31.8, 27.7.  64 rows, N 4096 21.8, 15.0, 14.8; 8192 39.1, 25.9, 21.3;
        // 16384 74, 47, 36.  160 rows at 512 experts, N 1024, 92, 65 to 72, 68 to 70; 40 rows 29, 23.5,
        // 26.5.  (32 columns from 256 blocks on, and 64 from 512 for more than 16 rows, would win too.)
        const int64_t four = tiles * ((f.N + 63) / 64), two = tiles * ((f.N + 31) / 32);
        if (four >= 1024) return go(k_w4_stream<D, G, MODE, 4, 4, 2>, four, 256, a, st);
        if (two >= 512) return go(k_w4_stream<D, G, MODE, 2, 4, 4>, two, 256, a, st);
        return go(k_w4_stream<D, G, MODE, 1, 8, 4>, tiles * ((f.N + 15) / 16), 512, a, st);
    }
    if (go(k_w4_tile<D, G, MODE>, tiles * ((f.N + kW4Cols - 1) / kW4Cols) * f.ksplit, 64 * kW4Waves, a, st)) return -1;
    return f.ksplit > 1 ? go(k_w4_sum<D>, tiles * ((f.N + 127) / 128) * 8, 256, a, st) : 0;
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
        constexpr int G = decltype(g)::value;
        if (a.f.dtype == 0) return a.zeros ? w4_<Bf16, G, W4_ZEROS>(a, st) : w4_<Bf16, G, W4_MID>(a, st);
        return a.zeros ? w4_<Fp16, G, W4_ZEROS>(a, st) : w4_<Fp16, G, W4_EIGHT>(a, st);
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
