// 256 x 256 output tiles on MFMA for products with hundreds of rows or more.
//
// A block is eight waves (two per SIMD) and owns a CU: two LDS stages of
// 64 KB, each four 16 KB halves (rows 0-127 / 128-255 of the A tile, columns
// 0-127 / 128-255 of the B tile, 64 reduction indices deep).  Wave w computes
// 64 + 64 rows (64 (w >> 2) of either half) by 32 + 32 columns (32 (w & 3) of
// either half), four quarters of 64 x 32, one per phase of a step:
//
//   phase 1  reads A half 0 and B half 0,  A0 x B0
//   phase 2  reads B half 1,               A0 x B1
//   phase 3  reads A half 1,               A1 x B1
//   phase 4  reads nothing,                A1 x B0
//
// A phase is a memory part (its LDS reads, and the copies of one half of a
// later step from global memory straight into the half that every wave has
// read) and a product part (16 MFMAs), each ended by a barrier.  Waves 4-7 run
// one barrier behind waves 0-3, so each SIMD has one wave in its product part
// while the other one's reads and copies are issued.  The copies run five
// halves (80 KB) ahead of the reads and are never drained in the loop: each
// memory part waits only until the half the next phase reads has landed
// (vmcnt 10, two copies per thread and half).
//
// 16384 x 4096 x 4096, bf16: x W^T 417 us (1320 TFLOP/s; with gelu 433), dz W
// 389 (1413), dz^T x 383 (1436); the library's products there: 436, 501 and 915.
// MFMA busy 70 percent of x W^T's cycles (62 with gelu and two outputs), at
// 1.94 GHz, what power leaves of the clock; 2 percent of the LDS cycles are bank
// conflicts.  256 x 256 rather than
// 128 x 128 halves the bytes that each product reads from LDS and L2; the
// accumulators then take half of a wave's registers, hence eight waves, one
// block to a CU and the alternating groups instead of several blocks.
//
// Below it, the same operands and layouts for 64 or 128 x 128 tiles over a ring
// of three or four stages (T1).
#pragma once

#include "dtype.h"
#include "gemm_common.h"

namespace moe {

constexpr int kT2Threads = 512;
constexpr int kT2Half = 128 * kTK;             // uint16 of one half: 128 rows (or columns) by kTK

// Compiler fence around the barriers: no LDS access moves across it.
__device__ __forceinline__ void t2_fence() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void t2_barrier() {
    t2_fence();
    __builtin_amdgcn_s_barrier();
    t2_fence();
}
// wait until this wave's LDS reads are done and at most N copies are in flight
template <int N>
__device__ __forceinline__ void t2_wait() {
    __builtin_amdgcn_s_waitcnt((N & 15) | 0x70 | ((N >> 4) << 14));
}

// ---------------------------------------------------------------- operands
// KC: the reduction index is contiguous in memory.  A half is 128 rows of
// 128 bytes; 16-byte chunk c of row r sits at slot c ^ ((r >> 1) & 7) (kc_off).
// KS: the reduction index is the memory row.  A half is 64 memory rows of 128
// columns (256 bytes); chunk c of memory row k sits at slot c ^ 2 s(k),
// s(k) = (k & 3) + 4 ((k >> 3) & 1): the eight memory rows that a 32-lane pass
// of the transpose load reads fall on eight different 32-byte bank windows.
// Copy q of thread t moves chunk q * (threads) + t.  Rows (columns) past the
// operand's last are read from its last one; their results are not stored.
// A tile holds the operand in NH arrays of ROWS rows (columns) each, copied by
// THR threads.  NT: non-temporal copies, for an operand that is read once.
template <bool KS, int ROWS, int NH, int THR, bool NT = false>
struct TileOperand {
    static constexpr int PER = ROWS * (kTK / 8) / THR;
    static_assert(!KS || ROWS == 128, "KS arrays are 128 columns wide");
    const char* base;             // at the tile's first row or column, reduction index 0
    int64_t step;                 // bytes from one 64-deep step to the next
    uint32_t off[NH][PER];        // [array][copy]
    int kpos[PER];                // [copy] the chunk's reduction index (KC: its first of eight)

    // r0: first row (KC) or column (KS) of the tile, n: the operand's count of them
    __device__ __forceinline__ TileOperand(const uint16_t* p, int64_t ld, int r0, int n) {
        base = (const char*)(KS ? p + r0 : p + (int64_t)r0 * ld);
        step = KS ? kTK * ld * 2 : kTK * 2;
        const int t = threadIdx.x;
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int g = q * THR + t;
            if constexpr (KS) {
                const int k = g >> 4, s = (k & 3) | ((k >> 1) & 4);
                const int c = (g & 15) ^ (s << 1);
                kpos[q] = k;
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const int col = min(h * ROWS + c * 8, n - r0 - 8);
                    off[h][q] = (uint32_t)(k * (int)ld + col) * 2;
                }
            } else {
                const int r = g >> 3, c = (g & 7) ^ ((r >> 1) & 7);
                kpos[q] = c * 8;
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const int row = min(h * ROWS + r, n - r0 - 1);
                    off[h][q] = (uint32_t)(row * (int)ld + c * 8) * 2;
                }
            }
        }
    }
    __device__ __forceinline__ void copy(int h, int kt, uint16_t* dst) const {
        const char* b = base + kt * step;
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            uint32_t o = off[h][q];
            asm volatile("" : "+v"(o));            // a scalar base and a 32-bit offset, not 64-bit lane addresses
            __builtin_amdgcn_global_load_lds((glb_void_t*)(b + o),
                                             (lds_void_t*)(dst + (q * THR + wave_id() * 64) * 8), 16, 0, NT ? 2 : 0);
        }
    }
    // the last, partial step through registers: `left` reduction indices, zeros
    // behind them.  Chunks behind them load the last one instead and are masked:
    // loads under a lane's condition are waited for one by one (512 experts of
    // 40 rows, all partial steps: dW 1087 -> 869 us).
    __device__ __forceinline__ void copy_tail(int h, int kt, int left, uint16_t* dst) const {
        const char* b = base + kt * step;
        const int last = KS ? left - 1 : left - 8, unit = KS ? (int)(step / kTK) : 2;
        uint4 v[PER];
#pragma unroll
        for (int q = 0; q < PER; ++q) v[q] = *(const uint4*)(b + off[h][q] - (uint32_t)(max(kpos[q] - last, 0) * unit));
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const uint32_t m = kpos[q] < left ? ~0u : 0u;
            *(uint4*)(dst + (q * THR + threadIdx.x) * 8) = make_uint4(v[q].x & m, v[q].y & m, v[q].z & m, v[q].w & m);
        }
    }
};

template <bool KS>
using T2Operand = TileOperand<KS, 128, 2, kT2Threads>;

// The fragment of 16 rows (columns) from r and the reduction indices ks .. ks + 31 of a half:
// lane l holds row r + (l & 15), reduction indices ks + 8 (l >> 4) + 0 .. 7.
template <bool KS>
__device__ __forceinline__ uint4 t2_frag(const uint16_t* half, int r, int ks) {
    const int lane = lane_id(), g = lane >> 4, j = lane & 15;
    if constexpr (KS) {
        const int s = (j >> 2) | ((g & 1) << 2);
        const int col = r + 4 * (j & 3);
        const uint16_t* p = half + (ks + 8 * g + (j >> 2)) * 128 + ((((col >> 3) ^ (s << 1)) << 3) | (col & 7));
        const v4i16 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)p);
        const v4i16 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(p + 4 * 128));
        return make_uint4(__builtin_bit_cast(uint2, a).x, __builtin_bit_cast(uint2, a).y,
                          __builtin_bit_cast(uint2, b).x, __builtin_bit_cast(uint2, b).y);
    } else {
        return *(const uint4*)(half + kc_off(r + j, 2 * (ks + 8 * g)));
    }
}

// 16 bytes of an output: past the caches if it is too large to be found there
// by whoever reads it next (many: more elements than the 32 MB of the L2s
// hold).  512 experts of 40 rows (y and z of 42 MB each next to 4.3 GB of
// weights) 786 -> 719 us, dx of the same 858 -> 815; 16384 x 4096 x 4096 429 -> 421.
__device__ __forceinline__ bool many(int64_t elements) { return elements > (16 << 20); }
__device__ __forceinline__ void st_out(bool nt, uint16_t* p, const uint16_t* v) {
    if (nt) {
        // (the markers keep the compiler from merging the two stores into a plain one)
        asm volatile("; non-temporal");
        __builtin_nontemporal_store(*(const u32x4*)v, (u32x4*)p);
        asm volatile("; non-temporal");
    } else {
        *(u32x4*)p = *(const u32x4*)v;
    }
}

// A wave's four quarters: acc[ha][hb][mb][nb] is rows 128 ha + 64 (w >> 2) + 16 mb + (lane & 15),
// columns 128 hb + 32 (w & 3) + 16 nb + 4 (lane >> 4) + 0 .. 3.
typedef f32x4 T2Acc[2][2][4][2];

template <class D, bool AKS, bool BKS>
struct T2Loop {
    const T2Operand<AKS>& a;
    const T2Operand<BKS>& b;
    T2Acc& acc;
    int wr, wc;                   // first row / column of the wave in a half
    uint4 fa[4][2], fb[2][2][2];  // fa[mb][ks], fb[half][nb][ks]

    __device__ __forceinline__ T2Loop(const T2Operand<AKS>& a_, const T2Operand<BKS>& b_, T2Acc& acc_)
        : a(a_), b(b_), acc(acc_), wr(64 * (wave_id() >> 2)), wc(32 * (wave_id() & 3)) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int mb = 0; mb < 4; ++mb)
#pragma unroll
                    for (int nb = 0; nb < 2; ++nb) acc[i][j][mb][nb] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    __device__ __forceinline__ void read_a(const uint16_t* half) {
#pragma unroll
        for (int mb = 0; mb < 4; ++mb)
#pragma unroll
            for (int s = 0; s < 2; ++s) fa[mb][s] = t2_frag<AKS>(half, wr + 16 * mb, 32 * s);
    }
    __device__ __forceinline__ void read_b(int h, const uint16_t* half) {
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int s = 0; s < 2; ++s) fb[h][nb][s] = t2_frag<BKS>(half, wc + 16 * nb, 32 * s);
    }
    __device__ __forceinline__ void product(int ha, int hb) {
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int mb = 0; mb < 4; ++mb)
#pragma unroll
                for (int nb = 0; nb < 2; ++nb)
                    acc[ha][hb][mb][nb] = D::mfma(fb[hb][nb][s], fa[mb][s], acc[ha][hb][mb][nb]);
        __builtin_amdgcn_s_setprio(0);
    }
    // Step kt of nk on one stage while the copies of later steps go out: A half
    // 1 of step kt + 1, then A half 0, B half 0 and B half 1 of step kt + 2.
    // The waits leave in flight what was issued after the half the next phase
    // reads: five halves, fewer in the last two steps.
    // FULL: the caller knows that there are two more steps (branches here make
    // the compiler lose track of the copies and drain them all once a step).
    template <bool FULL>
    __device__ __forceinline__ void step(int kt, int nk, uint16_t* a0, const uint16_t* a1, uint16_t* b0,
                                         uint16_t* b1, uint16_t* na1) {
        const bool m1 = FULL || kt + 1 < nk, m2 = FULL || kt + 2 < nk;
        read_b(0, b0);
        read_a(a0);
        if (m1) {
            a.copy(1, kt + 1, na1);
            t2_wait<10>();
        } else {
            t2_wait<2>();
        }
        t2_barrier();
        product(0, 0);
        t2_barrier();
        read_b(1, b1);
        if (m2) {
            a.copy(0, kt + 2, a0);
            t2_wait<10>();
        } else if (m1) {
            t2_wait<8>();
        } else {
            t2_wait<0>();
        }
        t2_barrier();
        product(0, 1);
        t2_barrier();
        read_a(a1);
        if (m2) b.copy(0, kt + 2, b0);
        t2_wait<63>();
        t2_barrier();
        product(1, 1);
        t2_barrier();
        if (m2) {
            b.copy(1, kt + 2, b1);
            t2_wait<10>();
        } else {
            t2_wait<4>();
        }
        t2_barrier();
        product(1, 0);
        t2_barrier();
    }
};

// The stages' halves, each an array of its own: the compiler waits for every
// copy in flight before an LDS read that it cannot tell apart from the copies'
// destination.
struct T2Lds {
    uint16_t* h[8];
};
#define T2_LDS(NAME)                                                                                        \
    __shared__ __attribute__((aligned(16))) uint16_t NAME##0[kT2Half], NAME##1[kT2Half], NAME##2[kT2Half], \
        NAME##3[kT2Half], NAME##4[kT2Half], NAME##5[kT2Half], NAME##6[kT2Half], NAME##7[kT2Half];             \
    const T2Lds NAME{{NAME##0, NAME##1, NAME##2, NAME##3, NAME##4, NAME##5, NAME##6, NAME##7}}

// acc = A (x) B over `len` reduction indices.
template <class D, bool AKS, bool BKS>
__device__ __forceinline__ void t2_mainloop(const T2Operand<AKS>& a, const T2Operand<BKS>& b, int len, T2Acc& acc,
                                            const T2Lds& lds) {
    uint16_t *const a00 = lds.h[0], *const a01 = lds.h[1], *const b00 = lds.h[2], *const b01 = lds.h[3];
    uint16_t *const a10 = lds.h[4], *const a11 = lds.h[5], *const b10 = lds.h[6], *const b11 = lds.h[7];
    T2Loop<D, AKS, BKS> l(a, b, acc);
    const int nk = len / kTK, left = len % kTK;
    const bool late = wave_id() >= 4;
    if (nk > 0) {
        a.copy(0, 0, a00);
        b.copy(0, 0, b00);
        b.copy(1, 0, b01);
        a.copy(1, 0, a01);
        const int k1 = min(1, nk - 1);             // a single step: copied twice, so that the waits count the same
        a.copy(0, k1, a10);
        b.copy(0, k1, b10);
        b.copy(1, k1, b11);
        t2_wait<10>();
        t2_barrier();
        if (late) t2_barrier();
        int kt = 0;
        for (; kt + 3 < nk; kt += 2) {
            l.template step<true>(kt, nk, a00, a01, b00, b01, a11);
            l.template step<true>(kt + 1, nk, a10, a11, b10, b11, a01);
        }
        for (; kt < nk; kt += 2) {                 // the last one to three
            l.template step<false>(kt, nk, a00, a01, b00, b01, a11);
            if (kt + 1 < nk) l.template step<false>(kt + 1, nk, a10, a11, b10, b11, a01);
        }
        if (!late) t2_barrier();
    }
    if (left > 0) {
        __syncthreads();
        a.copy_tail(0, nk, left, a00);
        a.copy_tail(1, nk, left, a01);
        b.copy_tail(0, nk, left, b00);
        b.copy_tail(1, nk, left, b01);
        __syncthreads();
        l.read_b(0, b00);
        l.read_a(a00);
        l.product(0, 0);
        l.read_b(1, b01);
        l.product(0, 1);
        l.read_a(a01);
        l.product(1, 1);
        l.product(1, 0);
    }
}

// rows and columns of acc[ha][hb][mb][nb] in the tile
__device__ __forceinline__ int t2_row(int ha, int mb) {
    return 128 * ha + 64 * (wave_id() >> 2) + 16 * mb + (lane_id() & 15);
}
__device__ __forceinline__ int t2_col(int hb, int nb) {
    return 128 * hb + 32 * (wave_id() & 3) + 16 * nb + 4 * (lane_id() >> 4);
}

// The tile to out [., ncol] at row r0, column c0 (rows below r1): f(ha, hb, mb,
// nb) gives four consecutive values of a row, packed.  It goes out through the
// stages' LDS (32 rows to an array, 16-byte chunk c of row r at slot c ^ (r &
// 31)) as 512-byte row pieces, 16 bytes per lane (stored straight from the
// fragments, 16 rows by 32 bytes an instruction, the same bytes took 32 us
// instead of 22 for 134 MB).
template <class F>
__device__ __forceinline__ void t2_put(const T2Lds& lds, bool nt, uint16_t* out, int r0, int r1, int c0, int ncol,
                                       const F& f) {
    const int wr = wave_id() >> 2, t = threadIdx.x;
    __syncthreads();                           // the LDS is no longer read
#pragma unroll
    for (int ha = 0; ha < 2; ++ha)
#pragma unroll
        for (int mb = 0; mb < 4; ++mb) {
            uint16_t* h = wr ? lds.h[4 * ha + 2 + (mb >> 1)] : lds.h[4 * ha + (mb >> 1)];
            const int r = 16 * (mb & 1) + (lane_id() & 15);
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                for (int nb = 0; nb < 2; ++nb) {
                    const int c = t2_col(hb, nb);
                    *(uint2*)(h + r * 256 + (((c >> 3) ^ r) << 3) + (c & 7)) = f(ha, hb, mb, nb);
                }
        }
    __syncthreads();
    const int c = t & 31;
    if (c0 + 8 * c < ncol) {
        uint16_t* p = out + (int64_t)r0 * ncol + c0 + 8 * c;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const int r = 16 * q + (t >> 5);
            if (r0 + r < r1)
                st_out(nt, p + (int64_t)r * ncol, lds.h[q >> 1] + (r & 31) * 256 + ((c ^ (r & 31)) << 3));
        }
    }
}

// ================================================================ 64 / 128 x 128 tiles
// Fewer rows, or too few 256 x 256 tiles for the chip: NW waves in two rows of
// NW / 2, each TM / 2 rows by 256 / NW columns (64-row tiles: four waves of 64
// columns; 128-row tiles: eight of 32), over a ring of NST stages of 64
// reduction indices that copies fill NST - 1 steps ahead; one barrier a step,
// after which the stage read a step before is filled again.  A block at a time
// on a CU then has up to 96 KB of copies in flight: with one step in flight
// (register-staged) such a product took about 1 us a step, the latency of a
// load from HBM.
// A wave's columns are NB blocks of 16.
template <int NW>
constexpr int t1_nb() { return 16 / NW; }
template <int TM, int NW>
using T1Acc = f32x4[TM / 32][t1_nb<NW>()];

// row and first column in the tile of accumulator (mb, nb): rows 16 apart, four columns each
template <int TM, int NW>
struct T1Pos {
    int m_, n_;
    __device__ __forceinline__ T1Pos()
        : m_((TM / 2) * (wave_id() & 1) + (lane_id() & 15)),
          n_(16 * t1_nb<NW>() * (wave_id() >> 1) + 4 * (lane_id() >> 4)) {}
    __device__ __forceinline__ int m(int mb) const { return m_ + 16 * mb; }
    __device__ __forceinline__ int n(int nb) const { return n_ + 16 * nb; }
};

template <class D, bool AKS, bool BKS, int TM, int NST, int NW, bool NT = false>
struct T1Loop {
    static constexpr int NB = t1_nb<NW>();
    using OpA = TileOperand<AKS, TM, 1, 64 * NW>;
    using OpB = TileOperand<BKS, 128, 1, 64 * NW, NT>;
    static constexpr int PER = OpA::PER + OpB::PER;      // copies per thread and step
    const OpA& a;
    const OpB& b;
    T1Acc<TM, NW>& acc;
    int wm, wn;

    __device__ __forceinline__ T1Loop(const OpA& a_, const OpB& b_, T1Acc<TM, NW>& acc_)
        : a(a_), b(b_), acc(acc_), wm((TM / 2) * (wave_id() & 1)), wn(16 * NB * (wave_id() >> 1)) {
#pragma unroll
        for (int mb = 0; mb < TM / 32; ++mb)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    __device__ __forceinline__ void product(const uint16_t* sa, const uint16_t* sb) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            uint4 fa[TM / 32], fb[NB];
#pragma unroll
            for (int mb = 0; mb < TM / 32; ++mb) fa[mb] = t2_frag<AKS>(sa, wm + 16 * mb, 32 * s);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) fb[nb] = t2_frag<BKS>(sb, wn + 16 * nb, 32 * s);
#pragma unroll
            for (int mb = 0; mb < TM / 32; ++mb)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = D::mfma(fb[nb], fa[mb], acc[mb][nb]);
        }
    }
    // step kt on (sa, sb) while step kt + NST - 1 is copied to (na, nb)
    template <bool FULL>
    __device__ __forceinline__ void step(int kt, int nk, const uint16_t* sa, const uint16_t* sb, uint16_t* na,
                                         uint16_t* nb) {
        const int later = FULL ? NST : nk - 1 - kt;       // steps behind this one
        if (later >= NST - 2) t2_wait<(NST - 2) * PER>();
        else if (NST > 3 && later == 1) t2_wait<PER>();
        else t2_wait<0>();
        t2_barrier();
        if (later >= NST - 1) {
            a.copy(0, kt + NST - 1, na);
            b.copy(0, kt + NST - 1, nb);
        }
        product(sa, sb);
    }
};

// The ring's arrays, each of its own: the compiler waits for every copy in
// flight before an LDS read that it cannot tell apart from the copies'
// destination.  TM * kTK and 128 * kTK elements (a3, b3: with four stages).
struct T1Ring {
    uint16_t *a0, *a1, *a2, *a3, *b0, *b1, *b2, *b3;
};
#define T1_RING(NAME, TM, NST)                                                                             \
    __shared__ __attribute__((aligned(16))) uint16_t NAME##a0[TM * kTK], NAME##a1[TM * kTK], NAME##a2[TM * kTK]; \
    __shared__ __attribute__((aligned(16))) uint16_t NAME##b0[128 * kTK], NAME##b1[128 * kTK], NAME##b2[128 * kTK]; \
    __shared__ __attribute__((aligned(16))) uint16_t NAME##a3[NST == 4 ? TM * kTK : 8];                        \
    __shared__ __attribute__((aligned(16))) uint16_t NAME##b3[NST == 4 ? 128 * kTK : 8];                       \
    const T1Ring NAME{NAME##a0, NAME##a1, NAME##a2, NAME##a3, NAME##b0, NAME##b1, NAME##b2, NAME##b3}

// acc = A (x) B over `len` reduction indices
template <class D, bool AKS, bool BKS, int TM, int NST, int NW, bool NT = false>
__device__ __forceinline__ void t1_mainloop(const TileOperand<AKS, TM, 1, 64 * NW>& a,
                                            const TileOperand<BKS, 128, 1, 64 * NW, NT>& b, int len,
                                            T1Acc<TM, NW>& acc, const T1Ring& r) {
    static_assert(NST == 3 || NST == 4, "");
    uint16_t *const a0 = r.a0, *const a1 = r.a1, *const a2 = r.a2, *const a3 = r.a3;
    uint16_t *const b0 = r.b0, *const b1 = r.b1, *const b2 = r.b2, *const b3 = r.b3;
    T1Loop<D, AKS, BKS, TM, NST, NW, NT> l(a, b, acc);
    const int nk = len / kTK, left = len % kTK;
    if (nk > 0) {
        // steps 0 .. NST - 2; what is past the last one is the last one again,
        // so that the waits count the same
        a.copy(0, 0, a0);
        b.copy(0, 0, b0);
        a.copy(0, min(1, nk - 1), a1);
        b.copy(0, min(1, nk - 1), b1);
        if constexpr (NST == 4) {
            a.copy(0, min(2, nk - 1), a2);
            b.copy(0, min(2, nk - 1), b2);
        }
        int kt = 0;
        if constexpr (NST == 4) {
            for (; kt + 6 < nk; kt += 4) {
                l.template step<true>(kt, nk, a0, b0, a3, b3);
                l.template step<true>(kt + 1, nk, a1, b1, a0, b0);
                l.template step<true>(kt + 2, nk, a2, b2, a1, b1);
                l.template step<true>(kt + 3, nk, a3, b3, a2, b2);
            }
            for (; kt < nk; kt += 4) {
                l.template step<false>(kt, nk, a0, b0, a3, b3);
                if (kt + 1 < nk) l.template step<false>(kt + 1, nk, a1, b1, a0, b0);
                if (kt + 2 < nk) l.template step<false>(kt + 2, nk, a2, b2, a1, b1);
                if (kt + 3 < nk) l.template step<false>(kt + 3, nk, a3, b3, a2, b2);
            }
        } else {
            for (; kt + 4 < nk; kt += 3) {
                l.template step<true>(kt, nk, a0, b0, a2, b2);
                l.template step<true>(kt + 1, nk, a1, b1, a0, b0);
                l.template step<true>(kt + 2, nk, a2, b2, a1, b1);
            }
            for (; kt < nk; kt += 3) {
                l.template step<false>(kt, nk, a0, b0, a2, b2);
                if (kt + 1 < nk) l.template step<false>(kt + 1, nk, a1, b1, a0, b0);
                if (kt + 2 < nk) l.template step<false>(kt + 2, nk, a2, b2, a1, b1);
            }
        }
        t2_wait<0>();                              // (one or two steps: the repeated copies)
    }
    if (left > 0) {
        __syncthreads();
        a.copy_tail(0, nk, left, a0);
        b.copy_tail(0, nk, left, b0);
        __syncthreads();
        l.product(a0, b0);
    }
}

// The tile to out [., ncol] at row r0, column c0 (rows below r1): f(mb, nb) gives
// four consecutive values of a row, packed.  Through the ring's LDS (64 rows to
// an array, 16-byte chunk c of row r at slot c ^ (r & 15)) as 256-byte row
// pieces: stored straight from the fragments (16 rows by 32 bytes an
// instruction) z next to y cost 512 experts of 40 rows 66 us, 42 MB.
template <int TM, int NW, class F>
__device__ __forceinline__ void t1_put(const T1Ring& ring, bool nt, uint16_t* out, int r0, int r1, int c0,
                                       int ncol, const F& f) {
    constexpr int NB = t1_nb<NW>(), RP = 4 * NW;           // rows of a pass
    const int wm = wave_id() & 1, wn = 16 * NB * (wave_id() >> 1), t = threadIdx.x, lane = lane_id();
    __syncthreads();                           // the LDS is no longer read
    uint16_t* h = TM == 128 && wm ? ring.b1 : ring.b0;
#pragma unroll
    for (int mb = 0; mb < TM / 32; ++mb) {
        const int r = (TM == 64 ? 32 * wm : 0) + 16 * mb + (lane & 15);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int c = wn + 16 * nb + 4 * (lane >> 4);
            *(uint2*)(h + r * 128 + (((c >> 3) ^ (r & 15)) << 3) + (c & 7)) = f(mb, nb);
        }
    }
    __syncthreads();
    const int c = t & 15;
    if (c0 + 8 * c < ncol) {
        uint16_t* p = out + (int64_t)r0 * ncol + c0 + 8 * c;
#pragma unroll
        for (int q = 0; q < TM / RP; ++q) {
            const int r = RP * q + (t >> 4);
            if (r0 + r < r1)
                st_out(nt, p + (int64_t)r * ncol,
                       (RP * q < 64 ? ring.b0 : ring.b1) + (r & 63) * 128 + ((c ^ (r & 15)) << 3));
        }
    }
}

}  // namespace moe
