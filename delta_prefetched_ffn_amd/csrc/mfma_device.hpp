// Matrix instructions and their operands, shared by the gfx950 kernels that use them: 16-bit operands, codes widened to
// them, fp32 values as sums of them.
#pragma once

#include "kv_device.hpp"

namespace np {

template <typename E>
struct Vec8;
template <>
struct Vec8<__bf16> {
    typedef bf16x8 t;
};
template <>
struct Vec8<_Float16> {
    typedef f16x8 t;
};

__device__ inline f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ inline f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// Eight e4m3 codes (two dwords), each dword times its scale 2^k, to eight 16-bit floats: exact in
// bf16, exact in fp16 while the product stays within its normal range.
template <typename E>
__device__ inline typename Vec8<E>::t widen(uint32_t a, uint32_t b, float sa, float sb);
template <>
__device__ inline bf16x8 widen<__bf16>(uint32_t a, uint32_t b, float sa, float sb) {
    const bf16x2 x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, sa, false), y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, sa, true);
    const bf16x2 z = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, sb, false), w = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, sb, true);
    return bf16x8{x[0], x[1], y[0], y[1], z[0], z[1], w[0], w[1]};
}
template <>
__device__ inline f16x8 widen<_Float16>(uint32_t a, uint32_t b, float sa, float sb) {
    const f16x2 x = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, sa, false), y = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, sa, true);
    const f16x2 z = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, sb, false), w = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, sb, true);
    return f16x8{x[0], x[1], y[0], y[1], z[0], z[1], w[0], w[1]};
}

// x[8] as `N` summands of type E, each the rounding of what the ones before left.
template <typename E, int N>
__device__ inline void split(typename Vec8<E>::t* o, const float* x) {
    float r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = x[k];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const E e = (E)r[k];
            o[n][k] = e;
            if (n + 1 < N) r[k] = r[k] - (float)e;
        }
}

typedef float f32x16 __attribute__((ext_vector_type(16)));
__device__ inline f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
__device__ inline f32x16 mfma(f16x8 a, f16x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }

}  // namespace np
