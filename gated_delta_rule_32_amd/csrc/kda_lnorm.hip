// Layer norm of token rows, forward and backward:
//     y = w (x - m) r + b,   m = mean x,   r = 1 / sqrt(mean (x - m)^2 + eps),
//     dx = r (d - mean d - h mean(d h)),   d = w dy,   h = (x - m) r,
//     dw = sum dy h,   db = sum dy   (over the rows).
// A row stays in the registers of the threads that share it from its one read to its one
// write, so that the mean is known before the squares around it are summed.  All
// arithmetic is FP32; the only roundings are those of the BF16 outputs.  The
// backward forms m and r anew, with mean d and mean(d h) in the sum that gives r; its weight gradients are
// summed per thread over the rows of a workgroup, and over the workgroups by a second kernel, all in a
// fixed order.
// Bound by HBM.  So that it never waits for a row's sums, the next row is on its way meanwhile:
// 8192 x 12288 took 218 us backward with a row at a time and takes 111 (105 at 6.0 TB/s, and 5 for the sums
// over workgroups), forward 103 and 67 (6.0 TB/s).
#include <algorithm>

#include "kda_common.hpp"
#include "kda_layers.h"

namespace kda {

namespace {

typedef float f32x8 __attribute__((ext_vector_type(8)));

// Rows that are read and written once and not found in a cache again (kStream) go past it.
template <bool kStream>
__device__ __forceinline__ bf16x8 load_row(const bf16* p) {
    const bf16x8* q = (const bf16x8*)p;
    return kStream ? __builtin_nontemporal_load(q) : *q;
}
template <bool kStream>
__device__ __forceinline__ void store_row(bf16* p, f32x8 x) {
    const bf16x8 y = cat8(to_bf4(f32x4{x[0], x[1], x[2], x[3]}), to_bf4(f32x4{x[4], x[5], x[6], x[7]}));
    if (kStream)
        __builtin_nontemporal_store(y, (bf16x8*)p);
    else
        *(bf16x8*)p = y;
}
__device__ __forceinline__ f32x8 widen(bf16x8 x) { return __builtin_convertvector(x, f32x8); }
__device__ __forceinline__ f32x8 load8(const float* p) {
    const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 4);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ void store8(float* p, f32x8 x) {
    *(f32x4*)p = f32x4{x[0], x[1], x[2], x[3]};
    *(f32x4*)(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
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
        if constexpr (kThreads > 16) x[k] = rows_sum(x[k]);
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
template <int kThreads, int kVecs, bool kStream>
__global__ __launch_bounds__(kThreads < 256 ? 256 : kThreads) void lnorm_fwd_kernel(LNormArgs a) {
    constexpr int ROWS = kThreads < 256 ? 256 / kThreads : 1;
    static_assert(kThreads <= 64 || ROWS == 1, "rows of a workgroup are summed in single waves");
    // many long rows: a workgroup walks over its rows with w and b in registers and the next row on its way
    constexpr bool kHold = kStream && kThreads < 1024;
    __shared__ float part[2][kThreads > 64 ? kThreads / 64 : 1][1];
    const int t = threadIdx.x % kThreads;
    f32x8 w[kVecs], b[kVecs];
    bf16x8 next[kVecs];
    auto load = [&](int64_t row) __attribute__((always_inline)) {
        const bf16* px = (const bf16*)a.x + row * a.sx;
#pragma unroll
        for (int c = 0; c < kVecs; ++c) {
            const int at = (c * kThreads + t) * 8;
            next[c] = at < a.C ? load_row<kStream>(px + at) : bf16x8{};
        }
    };
    int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / kThreads;
    if (row >= a.rows) return;   // (whole rows, and only where no barrier follows)
    load(row);
    if (kHold) {
#pragma unroll
        for (int c = 0; c < kVecs; ++c) {
            const int at = (c * kThreads + t) * 8;
            w[c] = at < a.C ? load8(a.w + at) : f32x8{};
            b[c] = at < a.C && a.b != nullptr ? load8(a.b + at) : f32x8{};
        }
    }
    const int64_t step = (int64_t)gridDim.x * ROWS;
    for (;;) {
        f32x8 x[kVecs];
        float s[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < kVecs; ++c) {
            x[c] = widen(next[c]);
            s[0] += sum8(x[c]);
        }
        if (kHold && row + step < a.rows) load(row + step);
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
            const f32x8 wc = kHold ? w[c] : load8(a.w + at);
            const f32x8 bc = kHold ? b[c] : a.b != nullptr ? load8(a.b + at) : f32x8{};
            // (one rounding, so that a row's bits do not depend on how many there are)
            store_row<kStream>(py + at, __builtin_elementwise_fma(x[c] * r, wc, bc));
        }
        row += step;
        if (row >= a.rows) break;
        if (!kHold) load(row);
    }
}

template <int kThreads, int kVecs, bool kStream>
__global__ __launch_bounds__(kThreads < 256 ? 256 : kThreads) void lnorm_bwd_kernel(LNormArgs a) {
    constexpr int ROWS = kThreads < 256 ? 256 / kThreads : 1;
    static_assert(kThreads <= 64 || ROWS == 1, "rows of a workgroup are summed in single waves");
    // With 16 waves a thread has 128 registers, of which the sums take half: then x stays in BF16, w
    // is read again, no row is on its way meanwhile, and of the longest rows dw is summed in LDS.
    constexpr bool kLean = kThreads == 1024, kLds = kLean && kVecs > 2;
    __shared__ f32x4 far[kLds ? 2 * kVecs * kThreads : 1];
    __shared__ float part1[kThreads > 64 ? kThreads / 64 : 1][1];
    __shared__ float part2[kThreads > 64 ? kThreads / 64 : 1][3];
    const int t = threadIdx.x % kThreads;
    f32x8 w[kVecs], dw[kVecs], db[kVecs];
    auto weight = [&](int c) __attribute__((always_inline)) {
        const int at = (c * kThreads + t) * 8;
        return at < a.C ? load8(a.w + at) : f32x8{};
    };
#pragma unroll
    for (int c = 0; c < kVecs; ++c) {
        if (!kLean) w[c] = weight(c);
        dw[c] = db[c] = f32x8{};
        if (kLds) far[2 * c * kThreads + t] = far[(2 * c + 1) * kThreads + t] = f32x4{};
    }
    bf16x8 nx[kVecs], nd[kVecs];   // the next row, on its way while this one is summed
    auto load = [&](int64_t row) __attribute__((always_inline)) {
        const bf16* px = (const bf16*)a.x + row * a.sx;
        const bf16* pd = (const bf16*)a.dy + row * a.C;
#pragma unroll
        for (int c = 0; c < kVecs; ++c) {
            const int at = (c * kThreads + t) * 8;
            nx[c] = at < a.C ? load_row<kStream>(px + at) : bf16x8{};
            nd[c] = at < a.C ? load_row<kStream>(pd + at) : bf16x8{};
        }
    };
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / kThreads;
    if (!kLean && row < a.rows) load(row);
    for (; row < a.rows; row += step) {
        if (kLean) load(row);
        f32x8 x[kVecs];
        bf16x8 raw[kVecs], d[kVecs];
        float s[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < kVecs; ++c) {
            raw[c] = nx[c];
            d[c] = nd[c];
            const f32x8 v = widen(raw[c]);
            if (!kLean) x[c] = v;
            s[0] += sum8(v);
        }
        if (!kLean && row + step < a.rows) load(row + step);
        row_sum<kThreads>(s, part1);
        const float m = s[0] * a.inv;
        float g[3] = {0.0f, 0.0f, 0.0f};   // of (x - m)^2, d and d (x - m)
#pragma unroll
        for (int c = 0; c < kVecs; ++c) {
            f32x8 v = kLean ? widen(raw[c]) : x[c];
            if ((c * kThreads + t) * 8 < a.C) v -= m;
            if (!kLean) x[c] = v;
            const f32x8 e = widen(d[c]) * (kLean ? weight(c) : w[c]);
            g[0] += sum8(v * v);
            g[1] += sum8(e);
            g[2] += sum8(e * v);
            if (kLean) __builtin_amdgcn_sched_barrier(0);   // (one group's values at a time)
        }
        row_sum<kThreads>(g, part2);
        const float r = rsqrtf(g[0] * a.inv + a.eps);
        const float g0 = g[1] * a.inv, g1 = g[2] * r * a.inv;
        bf16* dx = (bf16*)a.dx + row * a.C;
#pragma unroll
        for (int c = 0; c < kVecs; ++c) {
            const int at = (c * kThreads + t) * 8;
            const f32x8 h = (kLean ? widen(raw[c]) - m : x[c]) * r, e = widen(d[c]);   // (behind C: e is zero)
            if (kLds) {
                const f32x8 y = e * h;
                far[2 * c * kThreads + t] += f32x4{y[0], y[1], y[2], y[3]};
                far[(2 * c + 1) * kThreads + t] += f32x4{y[4], y[5], y[6], y[7]};
            } else {
                dw[c] += e * h;
            }
            db[c] += e;
            if (at < a.C) store_row<kStream>(dx + at, (e * (kLean ? load8(a.w + at) : w[c]) - g0 - h * g1) * r);
            if (kLean) __builtin_amdgcn_sched_barrier(0);
        }
    }
    // partials: a row of each sum per workgroup
    float* p = a.part + (int64_t)blockIdx.x * 2 * a.C;
    if constexpr (ROWS > 1) {
        __shared__ float all[2 * 8 * kVecs * 256];   // [sum][row][channel]
#pragma unroll
        for (int c = 0; c < kVecs; ++c) {
            const int at = (threadIdx.x / kThreads * kVecs * kThreads + c * kThreads + t) * 8;
            store8(all + at, dw[c]);
            store8(all + 8 * kVecs * 256 + at, db[c]);
        }
        __syncthreads();
        constexpr int W = 8 * kVecs * kThreads;   // channels a row has room for
        for (int i = threadIdx.x; i < 2 * W; i += 256) {
            const int set = i / W, col = i % W;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < ROWS; ++j) sum += all[(set * ROWS + j) * W + col];
            if (col < a.C) p[set * a.C + col] = sum;
        }
    } else {
#pragma unroll
        for (int c = 0; c < kVecs; ++c) {
            const int at = (c * kThreads + t) * 8;
            if (at >= a.C) continue;
            if (kLds) {
                *(f32x4*)(p + at) = far[2 * c * kThreads + t];
                *(f32x4*)(p + at + 4) = far[(2 * c + 1) * kThreads + t];
            } else {
                store8(p + at, dw[c]);
            }
            store8(p + a.C + at, db[c]);
        }
    }
}

// Sums of the partials' rows: a workgroup takes 64 columns, each of its 16 waves every 16th row.
__global__ __launch_bounds__(1024) void lnorm_reduce_kernel(const float* part, int rows, int C, float* dw, float* db) {
    __shared__ float sum[16][64];
    const int lane = threadIdx.x & 63, g = threadIdx.x >> 6;
    const int col = blockIdx.x * 64 + lane;   // of 2C
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (col < 2 * C) {
        const float* p = part + col;
        int r = g;
        for (; r + 48 < rows; r += 64) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += p[(int64_t)(r + 16 * i) * 2 * C];
        }
        for (; r < rows; r += 16) s[0] += p[(int64_t)r * 2 * C];
    }
    sum[g][lane] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (g == 0 && col < 2 * C) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += sum[i][lane];
        if (col < C)
            dw[col] = v;
        else if (db != nullptr)
            db[col - C] = v;
    }
}

namespace {

// Threads of a row, and groups of 8 channels a thread takes: as many as registers hold with the next row.
// In us against a group a thread (forward, backward): 16384 x 1024 14, 24 / 16, 42; 8192 x 4096 24, 40 /
// 24, 44; 8192 x 8192 43, 77 / 50, 125; 8192 x 12288 65, 109 / 94, 146 (in 1024 threads); with few rows
// more threads are faster: 128 x 4096 3.5, 8.3 / 3.1, 7.9.
struct Shape {
    int threads, vecs;
};
Shape row_shape(int C) {
    const int v = (C + 7) / 8;
    if (v <= 16) return {16, 1};
    for (int threads : {64, 256, 512, 1024})
        if (v <= threads * (threads == 1024 ? 4 : threads == 64 ? 2 : 3)) return {threads, (v + threads - 1) / threads};
    return {0, 0};
}
// Workgroups that walk over the rows (a backward pass, and a forward that streams).  In us with 256,
// 512, 1024 of them, backward 8192 x 2048 40, 30, 31, 8192 x 4096 59, 46, 54, 65536 x 1024 80, 75,
// 86; forward 16384 x 6144 87, 68, 75, 32768 x 4096 117, 90, 96, and in workgroups of 512, 8192 x 12288 68, 71, 71.
int walk_blocks(int64_t rows, int C) {
    const int threads = row_shape(C).threads, per = threads < 256 ? 256 / threads : 1;
    return (int)std::min<int64_t>((rows + per - 1) / per, threads > 256 ? 256 : 512);
}

template <int kThreads, int kVecs, bool kStream>
hipError_t launch_stream(const LNormArgs& a, bool bwd, hipStream_t s) {
    constexpr int ROWS = kThreads < 256 ? 256 / kThreads : 1, BLOCK = kThreads < 256 ? 256 : kThreads;
    if (!bwd) {
        int64_t blocks = (a.rows + ROWS - 1) / ROWS;
        if (kStream && kThreads < 1024) blocks = walk_blocks(a.rows, a.C);
        if (kThreads == 1024) blocks = std::min<int64_t>(blocks, 1 << 16);   // (a launch holds less than 2^32 threads)
        hipLaunchKernelGGL((lnorm_fwd_kernel<kThreads, kVecs, kStream>), dim3((unsigned)blocks), dim3(BLOCK), 0, s, a);
        return hipGetLastError();
    }
    const int blocks = walk_blocks(a.rows, a.C);
    hipLaunchKernelGGL((lnorm_bwd_kernel<kThreads, kVecs, kStream>), dim3((unsigned)blocks), dim3(BLOCK), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(lnorm_reduce_kernel, dim3((unsigned)((2 * a.C + 63) / 64)), dim3(1024), 0, s, a.part, blocks, a.C,
                       a.dw, a.db);
    return hipGetLastError();
}
template <int kThreads, int kVecs>
hipError_t launch(const LNormArgs& a, bool bwd, hipStream_t s) {
    return a.rows * a.C * (bwd ? 6 : 4) > kStreamBytes ? launch_stream<kThreads, kVecs, true>(a, bwd, s)
                                                       : launch_stream<kThreads, kVecs, false>(a, bwd, s);
}

}  // namespace

int64_t lnorm_part_rows(int64_t rows, int C) { return walk_blocks(rows, C); }

hipError_t launch_lnorm(const LNormArgs& a, bool bwd, hipStream_t s) {
    const Shape h = row_shape(a.C);
    switch (h.threads * 8 + h.vecs) {
        case 16 * 8 + 1: return launch<16, 1>(a, bwd, s);
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
