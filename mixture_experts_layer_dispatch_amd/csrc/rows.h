// What the kernels that go over rows or tokens share: grids, values of single
// lanes, accesses past the caches.
#pragma once

#include "common.h"

namespace moe {

// Launches of more than 2^30 threads (2^22 blocks of 256) take a second grid
// dimension: a dimension's threads are counted in 32 bits.
static dim3 rows_grid(int64_t blocks, int threads = 256) {
    const int64_t x = (1 << 30) / threads;
    if (blocks <= x) return dim3((unsigned)blocks);
    return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}
__device__ __forceinline__ int64_t block_number() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

__device__ __forceinline__ int lane_value(int v, int j) { return __builtin_amdgcn_readlane(v, j); }
__device__ __forceinline__ float lane_value(float v, int j) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), j));
}

// ---------------------------------------------------------------- over a wave
// In a fixed order, without the LDS: within rows of 16 lanes by shifts, then
// across them; lane 63 has the result.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or(float v, float other) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(other), __float_as_int(v), CTRL, ROWS, 0xf, false));
}
template <class F>
__device__ __forceinline__ float wave_fold(float v, float none, const F& f) {
    v = f(v, dpp_or<0x111, 0xf>(v, none));         // from the lane 1, 2, 4, 8 below
    v = f(v, dpp_or<0x112, 0xf>(v, none));
    v = f(v, dpp_or<0x114, 0xf>(v, none));
    v = f(v, dpp_or<0x118, 0xf>(v, none));
    v = f(v, dpp_or<0x142, 0xa>(v, none));         // lane 15 of the row below into rows 1 and 3
    v = f(v, dpp_or<0x143, 0xc>(v, none));         // lane 31 into rows 2 and 3
    return lane_value(v, 63);
}
__device__ __forceinline__ float wave_total(float v) {
    return wave_fold(v, 0.f, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_most(float v) {
    return wave_fold(v, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
}

// ---------------------------------------------------------------- non-temporal accesses
// The expert rows are read once: non-temporal loads (16384 tokens x 10 x 4096
// bf16: unpermute 312 -> 291 us, permute backward 287 -> 256; 2048 tokens:
// 38 -> 34, 35 -> 33).  Expert rows that are written are too many to be found
// in a cache later and go past it (NT) once they are more than the 32 MB of the
// L2s: 8192 tokens x 8 x 1024 (134 MB) permute 27.3 -> 24.2 us, unpermute
// backward 56 -> 52; 16384 x 10 x 4096 (1.3 GB) 292 -> 298 and 585 -> 564.
constexpr int64_t kCacheBytes = 32ll << 20;

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint4 ld_once(const uint4* p) {
    return __builtin_bit_cast(uint4, __builtin_nontemporal_load((const u32x4_t*)p));
}
template <bool NT>
__device__ __forceinline__ void st_row(uint4* p, const uint4& v) {
    if constexpr (NT) __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, v), (u32x4_t*)p);
    else *p = v;
}

}  // namespace moe
