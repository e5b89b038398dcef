// Device helpers of the gated delta rule's kernels.
#pragma once

#include "kda_delta.h"
#include "kda_scan.hpp"

namespace kda {

constexpr int SC = 32;            // tokens per chunk
constexpr float NORM_EPS = 1e-6f;

// FP32 as three BF16 pieces of 8 significant bits each.
__device__ __forceinline__ void split3(f32x4 x, bf16x4& a, bf16x4& b, bf16x4& c) {
    a = take_high(x);
    b = take_high(x);
    c = to_bf4(x);
}

// 2^(Gi - Gj), from the sums' two parts.
__device__ __forceinline__ float decay2(float hi, float li, float hj, float lj) {
    return __builtin_amdgcn_exp2f((hi - hj) + (li - lj));
}

}  // namespace kda
