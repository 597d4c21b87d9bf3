// What the attention kernels over the 8-bit cache share: operand types, the sums' unit, the join of partial results.
#pragma once

#include "mfma_device.hpp"

namespace np {

// What differs by the type of q and out. K codes become Op values (exact), q is held as kTerms
// summands of that type: bf16 and fp16 as they are, fp32 as three bf16 summands (8 + 8 + 8 bits:
// exact). P is rounded to fp16 for 16-bit outputs (2^-11 of the value, below the output's own
// rounding for bf16 and equal to it for fp16) and to three bf16 summands (2^-24) for fp32. In fp16 it
// is held times 2^kLift, so that it is between 2^7 and 2^15 at the row's maximum: weights from 2^-21 of
// that on are rounded by 2^-11 of themselves, smaller ones by at most 2^-32 of the largest (fp16's last
// places). N tokens are then off by at most N * 2^-32 of the row's sum together, half a step of fp16 at
// 2 Mi tokens; without the factor it was at 16 Ki.
template <typename T>
struct AttnKind;
template <>
struct AttnKind<__bf16> {
    typedef __bf16 Q;
    typedef _Float16 P;
    static constexpr int kQ = 1, kP = 1, kLift = 7;
};
template <>
struct AttnKind<_Float16> {
    typedef _Float16 Q;
    typedef _Float16 P;
    static constexpr int kQ = 1, kP = 1, kLift = 7;
};
template <>
struct AttnKind<float> {
    typedef __bf16 Q;
    typedef __bf16 P;
    static constexpr int kQ = 3, kP = 3, kLift = 0;
};

// P's values reach 2^kLazy (times 2^kLift) before the running maximum is raised, so most steps rescale nothing.
constexpr float kLazy = 8.0f;
// O is kept in units of 2^unit; a block's V codes are widened times 2^(ev - unit). Within
// [-kFar, kNear] of the unit every code is a normal fp16 number (2^-9 * 2^-5 = 2^-14 and
// 448 * 2^7 < 65504), so widening is exact; a block further off moves the unit. It moves down by at
// most kDrop from the largest exponent met (O would overflow fp32): blocks below that vanish.
constexpr int kFar = 5, kNear = 7, kDrop = 40;
constexpr int kNoUnit = -1000;  // below every exponent: no block met so far

// x, but made where it stands: what rare paths compute from the lane is not kept in registers across
// the loop for them.
__device__ inline int here(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// Adds a part (maximum mp, sum lp, values v) to a row's join at the maximum mm >= mp. A part that
// saw no token (mp = -inf, lp = 0) adds nothing, whatever mm is.
__device__ inline void join(f32x4& x, float& ll, float mm, float mp, float lp, f32x4 v) {
    if (mp == -__builtin_inff() && lp == 0.0f) return;
    const float f = mp == mm ? 1.0f : __builtin_amdgcn_exp2f(mp - mm);
    ll += f * lp;
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] += f * v[j];
}

}  // namespace np
