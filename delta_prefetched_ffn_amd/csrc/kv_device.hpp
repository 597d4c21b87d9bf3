// Device helpers of the 8-bit key/value cache: e4m3 and 16-bit conversions, row loads, the search
// for a work item's sequence.
#pragma once

#include <hip/hip_fp16.h>

#include "kv_internal.hpp"

namespace np {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 2^e for -126 <= e <= 127.
__device__ inline float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The sequence of a work item: the number of sequences that end at or before it.
__device__ inline int find_item(const KvBatch& b, int item) {
    if (b.n == 1) return 0;
    int c = 0;
    const int lane = threadIdx.x & 63;
    for (int i0 = 0; i0 < b.n; i0 += 64) {
        const int i = i0 + lane;
        c += __popcll(__ballot(i < b.n && b.item0[min(i, b.n - 1) + 1] <= item));
    }
    return __builtin_amdgcn_readfirstlane(c);
}

// The page of table entry `index` of sequence `seq`; -1 where it was dropped (a number outside the
// pool, which the host never writes, counts as dropped too: no address is made of it).
__device__ inline int page_of(const KvView& kv, int seq, int index) {
    const int p = kv.table[(int64_t)seq * kv.max_pages + index];
    return p < kv.n_pages ? p : -1;
}

// N consecutive values of a caller's row, as fp32 (N = 4 or 8; the address is aligned to
// N * sizeof(T) bytes up to 16).
template <int N>
__device__ inline void load_row(float* o, const float* p) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const f32x4 v = reinterpret_cast<const f32x4*>(p)[i];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[4 * i + k] = v[k];
    }
}
template <int N>
__device__ inline void load_row(float* o, const __bf16* p) {
    uint32_t w[N / 2];
    __builtin_memcpy(w, __builtin_assume_aligned(p, 2 * N), 2 * N);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        o[2 * i] = __uint_as_float(w[i] << 16);
        o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
template <int N>
__device__ inline void load_row(float* o, const _Float16* p) {
    _Float16 h[N];
    __builtin_memcpy(h, __builtin_assume_aligned(p, 2 * N), 2 * N);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = (float)h[i];
}

// One value to e4m3 range: beyond +-448 (only infinities get here: the block's exponent covers
// every finite value) saturates, NaN stays.
__device__ inline float sat448(float x) { return x != x ? x : fminf(fmaxf(x, -448.0f), 448.0f); }

// Four fp32 of at most 448 (or NaN) to four e4m3 bytes (round to nearest even).
__device__ inline uint32_t to_e4m3(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    return (uint32_t)w;
}

// Four e4m3 bytes scaled by s and rounded to e4m3 again.
__device__ inline uint32_t rescale_e4m3(uint32_t w, float s) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    return to_e4m3(lo[0] * s, lo[1] * s, hi[0] * s, hi[1] * s);
}

// Whether any of the four e4m3 bytes is NaN (0x7f or 0xff).
__device__ inline uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

}  // namespace np
