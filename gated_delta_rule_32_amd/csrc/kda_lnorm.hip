// Layer norm of token rows, forward and backward:
//     y = w (x - m) r + b,   m = mean x,   r = 1 / sqrt(mean (x - m)^2 + eps),
//     dx = r (d - mean d - h mean(d h)),   d = w dy,   h = (x - m) r,
//     dw = sum dy h,   db = sum dy   (over the rows).
// A row stays in the registers of the threads that share it from its one read to its one
// write, so that the mean is known before the squares around it are summed.  All
// arithmetic is FP32; the only roundings are those of the BF16 outputs.  Bound by HBM.  The
// backward forms m and r anew; its weight gradients are summed per thread over the rows of a
// workgroup, and over the workgroups by a second kernel, all in a fixed order.
#include <algorithm>

#include "kda_common.hpp"
#include "kda_layers.h"

namespace kda {

namespace {

typedef float f32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x8 load8(const bf16* p) { return __builtin_convertvector(*(const bf16x8*)p, f32x8); }
__device__ __forceinline__ f32x8 load8(const float* p) {
    const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 4);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ void store8(float* p, f32x8 x) {
    *(f32x4*)p = f32x4{x[0], x[1], x[2], x[3]};
    *(f32x4*)(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
}
__device__ __forceinline__ void store8(bf16* p, f32x8 x) {
    *(bf16x8*)p = cat8(to_bf4(f32x4{x[0], x[1], x[2], x[3]}), to_bf4(f32x4{x[4], x[5], x[6], x[7]}));
}
__device__ __forceinline__ float sum8(f32x8 x) {
    return ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
}

// Sums of K values over the `kThreads` threads that share a row, the same in all of them.
// `part`: room for K values of each wave of the workgroup; a round of two slots, so that one barrier a
// sum is enough.
template <int kThreads, int K>
__device__ __forceinline__ void row_sum(float (&x)[K], float (*part)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        x[k] = row16_sum(x[k]);
        x[k] += __shfl_xor(x[k], 16, 64);
        x[k] += __shfl_xor(x[k], 32, 64);
    }
    if constexpr (kThreads > 64) {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) part[threadIdx.x >> 6][k] = x[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < kThreads / 64; ++i) s += part[i][k];
            x[k] = s;
        }
    }
}

}  // namespace

// kThreads threads share a row, kVecs groups of 8 channels each; a workgroup of 256 takes
// 256 / kThreads rows where that is more than one.
template <int kThreads, int kVecs>
__global__ __launch_bounds__(kThreads < 256 ? 256 : kThreads) void lnorm_fwd_kernel(LNormArgs a) {
    constexpr int ROWS = kThreads < 256 ? 256 / kThreads : 1;
    static_assert(kThreads == 64 || ROWS == 1, "rows of a workgroup are summed in single waves");
    __shared__ float part[2][kThreads > 64 ? kThreads / 64 : 1][1];
    const int t = threadIdx.x % kThreads;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / kThreads;
    if (row >= a.rows) return;   // (whole waves, and only where no barrier follows)
    const bf16* px = (const bf16*)a.x + row * a.sx;
    f32x8 x[kVecs];
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < kVecs; ++c) {
        const int at = (c * kThreads + t) * 8;
        x[c] = at < a.C ? load8(px + at) : f32x8{};
        s[0] += sum8(x[c]);
    }
    row_sum<kThreads>(s, part[0]);
    const float m = s[0] * a.inv;
    s[0] = 0.0f;
#pragma unroll
    for (int c = 0; c < kVecs; ++c) {
        if ((c * kThreads + t) * 8 < a.C) x[c] -= m;
        s[0] += sum8(x[c] * x[c]);
    }
    row_sum<kThreads>(s, part[1]);
    const float r = rsqrtf(s[0] * a.inv + a.eps);
    bf16* py = (bf16*)a.y + row * a.C;
#pragma unroll
    for (int c = 0; c < kVecs; ++c) {
        const int at = (c * kThreads + t) * 8;
        if (at >= a.C) continue;
        const f32x8 w = load8(a.w + at);
        f32x8 y = x[c] * r * w;
        if (a.b != nullptr) y += load8(a.b + at);
        store8(py + at, y);
    }
}

template <int kThreads, int kVecs>
__global__ __launch_bounds__(kThreads < 256 ? 256 : kThreads) void lnorm_bwd_kernel(LNormArgs a) {
    constexpr int ROWS = kThreads < 256 ? 256 / kThreads : 1;
    static_assert(kThreads == 64 || ROWS == 1, "rows of a workgroup are summed in single waves");
    __shared__ float part1[2][kThreads > 64 ? kThreads / 64 : 1][1];
    __shared__ float part2[kThreads > 64 ? kThreads / 64 : 1][2];
    const int t = threadIdx.x % kThreads;
    f32x8 w[kVecs], dw[kVecs], db[kVecs];
#pragma unroll
    for (int c = 0; c < kVecs; ++c) {
        const int at = (c * kThreads + t) * 8;
        w[c] = at < a.C ? load8(a.w + at) : f32x8{};
        dw[c] = db[c] = f32x8{};
    }
    const int64_t step = (int64_t)gridDim.x * ROWS;
    for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / kThreads; row < a.rows; row += step) {
        const bf16* px = (const bf16*)a.x + row * a.sx;
        const bf16* pd = (const bf16*)a.dy + row * a.C;
        f32x8 x[kVecs], d[kVecs];
        float s[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < kVecs; ++c) {
            const int at = (c * kThreads + t) * 8;
            x[c] = at < a.C ? load8(px + at) : f32x8{};
            d[c] = at < a.C ? load8(pd + at) : f32x8{};
            s[0] += sum8(x[c]);
        }
        row_sum<kThreads>(s, part1[0]);
        const float m = s[0] * a.inv;
        s[0] = 0.0f;
#pragma unroll
        for (int c = 0; c < kVecs; ++c) {
            if ((c * kThreads + t) * 8 < a.C) x[c] -= m;
            s[0] += sum8(x[c] * x[c]);
        }
        row_sum<kThreads>(s, part1[1]);
        const float r = rsqrtf(s[0] * a.inv + a.eps);
        float g[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < kVecs; ++c) {
            x[c] *= r;
            dw[c] += d[c] * x[c];
            db[c] += d[c];
            d[c] *= w[c];
            g[0] += sum8(d[c]);
            g[1] += sum8(d[c] * x[c]);
        }
        row_sum<kThreads>(g, part2);
        const float g0 = g[0] * a.inv, g1 = g[1] * a.inv;
        bf16* dx = (bf16*)a.dx + row * a.C;
#pragma unroll
        for (int c = 0; c < kVecs; ++c) {
            const int at = (c * kThreads + t) * 8;
            if (at < a.C) store8(dx + at, (d[c] - g0 - x[c] * g1) * r);
        }
    }
    // partials: a row of each sum per (workgroup, row of it)
    float* p = a.part + ((int64_t)blockIdx.x * ROWS + threadIdx.x / kThreads) * 2 * a.C;
#pragma unroll
    for (int c = 0; c < kVecs; ++c) {
        const int at = (c * kThreads + t) * 8;
        if (at >= a.C) continue;
        store8(p + at, dw[c]);
        store8(p + a.C + at, db[c]);
    }
}

// Sums of the partials' rows: a workgroup takes 64 columns, each of its four waves every fourth row.
__global__ __launch_bounds__(256) void lnorm_reduce_kernel(const float* part, int rows, int C, float* dw, float* db) {
    __shared__ float sum[4][64];
    const int lane = threadIdx.x & 63, g = threadIdx.x >> 6;
    const int col = blockIdx.x * 64 + lane;   // of 2C
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (col < 2 * C) {
        const float* p = part + col;
        int r = g;
        for (; r + 12 < rows; r += 16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += p[(int64_t)(r + 4 * i) * 2 * C];
        }
        for (; r < rows; r += 4) s[0] += p[(int64_t)r * 2 * C];
    }
    sum[g][lane] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (g == 0 && col < 2 * C) {
        const float v = (sum[0][lane] + sum[1][lane]) + (sum[2][lane] + sum[3][lane]);
        if (col < C)
            dw[col] = v;
        else if (db != nullptr)
            db[col - C] = v;
    }
}

namespace {

// Threads of a row, and groups of 8 channels a thread takes.
struct Shape {
    int threads, vecs;
};
Shape row_shape(int C) {
    const int v = (C + 7) / 8;
    for (int threads : {64, 256, 512, 1024})
        if (v <= threads * (threads == 1024 ? 4 : threads == 64 ? 2 : 3)) return {threads, (v + threads - 1) / threads};
    return {0, 0};
}
// Workgroups of a backward pass.
int bwd_blocks(int64_t rows, int C) {
    const int per = row_shape(C).threads == 64 ? 4 : 1;
    return (int)std::min<int64_t>((rows + per - 1) / per, 512);
}

template <int kThreads, int kVecs>
hipError_t launch(const LNormArgs& a, bool bwd, hipStream_t s) {
    constexpr int ROWS = kThreads < 256 ? 256 / kThreads : 1, BLOCK = kThreads < 256 ? 256 : kThreads;
    if (!bwd) {
        hipLaunchKernelGGL((lnorm_fwd_kernel<kThreads, kVecs>), dim3((unsigned)((a.rows + ROWS - 1) / ROWS)), dim3(BLOCK), 0, s, a);
        return hipGetLastError();
    }
    const int blocks = bwd_blocks(a.rows, a.C);
    hipLaunchKernelGGL((lnorm_bwd_kernel<kThreads, kVecs>), dim3((unsigned)blocks), dim3(BLOCK), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(lnorm_reduce_kernel, dim3((unsigned)((2 * a.C + 63) / 64)), dim3(256), 0, s, a.part, blocks * ROWS, a.C,
                       a.dw, a.db);
    return hipGetLastError();
}

}  // namespace

int64_t lnorm_part_rows(int64_t rows, int C) {
    return (int64_t)bwd_blocks(rows, C) * (row_shape(C).threads == 64 ? 4 : 1);
}

hipError_t launch_lnorm(const LNormArgs& a, bool bwd, hipStream_t s) {
    const Shape h = row_shape(a.C);
    switch (h.threads * 8 + h.vecs) {
        case 64 * 8 + 1: return launch<64, 1>(a, bwd, s);
        case 64 * 8 + 2: return launch<64, 2>(a, bwd, s);
        case 256 * 8 + 1: return launch<256, 1>(a, bwd, s);
        case 256 * 8 + 2: return launch<256, 2>(a, bwd, s);
        case 256 * 8 + 3: return launch<256, 3>(a, bwd, s);
        case 512 * 8 + 2: return launch<512, 2>(a, bwd, s);
        case 512 * 8 + 3: return launch<512, 3>(a, bwd, s);
        case 1024 * 8 + 2: return launch<1024, 2>(a, bwd, s);
        case 1024 * 8 + 3: return launch<1024, 3>(a, bwd, s);
        case 1024 * 8 + 4: return launch<1024, 4>(a, bwd, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace kda
