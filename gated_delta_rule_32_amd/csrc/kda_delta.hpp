// Device helpers of the gated delta rule's kernels.
#pragma once

#include "kda_delta.h"
#include "kda_scan.hpp"

namespace kda {

constexpr int SC = 32;            // tokens per chunk
constexpr float NORM_EPS = 1e-6f;

// FP32 as two BF16 pieces (to 2^-16) or as three of 8 significant bits each (exactly).
// Of accumulators, two tiles that make one operand at a time: the matrix units take the
// rounded values off again (minus one half of an identity times the operand, which is
// exact), where the vector units would need a conversion back and a subtraction for each.
struct Pieces {
    bf16x8 first, second;   // -1 where the contraction index is the row, in the operand's first or second half
    __device__ __forceinline__ explicit Pieces(int lane) {
        bf16x4 id = to_bf4_neg(from_bf4(identity_frag(lane)));
        const bf16x4 none = __builtin_bit_cast(bf16x4, u32x2{0u, 0u});
        first = cat8(id, none);
        second = cat8(none, id);
    }
    __device__ __forceinline__ bf16x8 take(f32x4& x, f32x4& y) const {
        const bf16x8 a = cat8(to_bf4(x), to_bf4(y));
        x = mma32(first, a, x);
        y = mma32(second, a, y);
        return a;
    }
    __device__ __forceinline__ void split(f32x4 x, f32x4 y, bf16x8 (&p)[3]) const {
        p[0] = take(x, y);
        p[1] = take(x, y);
        p[2] = cat8(to_bf4(x), to_bf4(y));
    }
    __device__ __forceinline__ void split(f32x4 x, bf16x4& a, bf16x4& b) const { split4_rne(x, a, b); }
    __device__ __forceinline__ void split(f32x4 x, bf16x4& a, bf16x4& b, bf16x4& c) const {
        a = take_high(x);
        b = take_high(x);
        c = to_bf4(x);
    }
};

// 2^(Gi - Gj), from the sums' two parts.
__device__ __forceinline__ float decay2(float hi, float li, float hj, float lj) {
    return __builtin_amdgcn_exp2f((hi - hj) + (li - lj));
}

}  // namespace kda
