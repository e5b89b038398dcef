// Per-head row norms around a linear-attention layer, each in one pass:
// queries and keys are RMS-normed and rotated before it, the heads' outputs
// RMS-normed and gated behind it.  A row is the 128 channels of one (token,
// head); 16 lanes hold it (8 channels a lane), so a row's sums stay inside one
// DPP row, and a wave moves four rows at a time.  All arithmetic is FP32; the
// only roundings are those of the BF16 outputs.  Bound by HBM: every row is
// read once and written once.  The backward recomputes the norms from its
// inputs; the weight gradients are summed per lane over a fixed set of rows,
// per workgroup through LDS, and over the workgroups by a second kernel, all
// in a fixed order.
#include "kda_common.hpp"
#include "kda_layers.h"

namespace kda {

namespace {

constexpr int RN_THREADS = 256;
constexpr int RN_GROUPS = RN_THREADS / 16;   // rows in flight per workgroup

// Workgroups of a backward pass: four per compute unit, fewer when there are
// fewer rows.  (Its partials are one row of sums per workgroup.)  In us, 256, 512, 1024,
// 2048 and 4096 of them: query/key norm of 4099 tokens x 32 heads 34, 26, 24, 28, 31, of 16384
// x 40 167, 105, 93, 94, 98; gated norm of 4099 x 32 42, 34, 32, 35, 36, of 8192 x 96 278, 191,
// 192, 201, 200, of 16384 x 40 232, 153, 161, 170, 164.
constexpr int RN_BWD_BLOCKS = 1024;

// Whether a pass over `rows` rows of that many tensors is too large to be found
// in a cache again.  Gated norm of 96 heads, forward and backward: 8192 tokens 300 -> 280 us
// non-temporal, 4096 tokens 155 -> 145 us; the forward of 2048 tokens (150 MB)
// takes 24.6 us with retention, 26 us without.
bool streams(int64_t rows, int tensors) { return rows * (D * 2) * tensors > kStreamBytes; }

template <bool kStream, class T>
__device__ __forceinline__ T load(const bf16* p) {
    if constexpr (kStream) return __builtin_nontemporal_load((const T*)p);
    return *(const T*)p;
}
template <bool kStream, class T>
__device__ __forceinline__ void store(bf16* p, T v) {
    if constexpr (kStream)
        __builtin_nontemporal_store(v, (T*)p);
    else
        *(T*)p = v;
}

struct Row8 {
    float x[8];
};
__device__ __forceinline__ void unpack(Row8& r, bf16x4 lo, bf16x4 hi) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        r.x[e] = (float)lo[e];
        r.x[4 + e] = (float)hi[e];
    }
}
__device__ __forceinline__ bf16x4 pack4(const float* x) { return to_bf4(f32x4{x[0], x[1], x[2], x[3]}); }

// 1 / sqrt(mean x^2 + eps) of a row.
__device__ __forceinline__ float inv_rms(const Row8& r, float eps) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s += r.x[e] * r.x[e];
    return fast_rsqrt(row16_sum(s) * (1.0f / D) + eps);
}

// The 8 channels of a lane for the rotation: two quads of channels lo .. lo+3
// and hi .. hi+3.  Rotating halves, channel p pairs with p + rot/2, so the
// first rot/8 lanes take quads p and p + rot/2 and no lane needs another's
// values; the remaining lanes hold the channels behind rot.  Rotating
// neighbours, a lane's quads are adjacent.  Either way lane c < rot/8 needs
// angles 4c .. 4c+3.
struct Quads {
    int lo, hi;
    bool turned;
};
__device__ __forceinline__ Quads quads(int c, int rot, bool pairs) {
    const int r8 = rot >> 3;
    Quads q;
    q.turned = c < r8;
    q.lo = pairs || !q.turned ? 8 * c : 4 * c;
    q.hi = pairs || !q.turned ? 8 * c + 4 : 4 * c + (rot >> 1);
    return q;
}

// Rotates (sign 1) or rotates back (sign -1) a lane's 8 channels.
__device__ __forceinline__ void turn(Row8& r, f32x4 cs, f32x4 sn, bool pairs, float sign) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = pairs ? 2 * e : e, j = pairs ? 2 * e + 1 : 4 + e;
        const float u = r.x[i], v = r.x[j], s = sign * sn[e];
        r.x[i] = u * cs[e] - v * s;
        r.x[j] = v * cs[e] + u * s;
    }
}

}  // namespace

// 16 lanes take `per` heads of one token (a unit), so that the position and the
// angles are read once for all of them.
template <bool kPairs, bool kBwd, bool kStream>
__global__ __launch_bounds__(RN_THREADS) void qknorm_kernel(QkNormArgs a) {
    const int c = threadIdx.x & 15, grp = threadIdx.x >> 4;
    const int H = a.Hq + a.Hk, half = a.rot >> 1;
    const Quads qd = quads(c, a.rot, kPairs);
    float wq[8], wk[8], gq[8], gk[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        wq[e] = a.wq[qd.lo + e];
        wq[4 + e] = a.wq[qd.hi + e];
        wk[e] = a.wk[qd.lo + e];
        wk[4 + e] = a.wk[qd.hi + e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) gq[e] = gk[e] = 0.0f;
    const unsigned parts = (unsigned)((H + a.per - 1) / a.per);
    const unsigned units = (unsigned)a.tokens * parts;
    for (unsigned u = blockIdx.x * RN_GROUPS + grp; u < units; u += gridDim.x * RN_GROUPS) {
        const unsigned tok = u / parts;
        const int h0 = (int)(u - tok * parts) * a.per, h1 = min(h0 + a.per, H);
        const int64_t t = tok;
        // a position outside the table turns its token's rows into NaN
        f32x4 cs = {1.f, 1.f, 1.f, 1.f}, sn = zero4();
        const int64_t pos = a.positions != nullptr ? a.positions[t] : t % a.T;
        if (pos < 0 || pos >= a.rows) {
            const float nan = __builtin_nanf("");
            cs = sn = f32x4{nan, nan, nan, nan};
        } else if (qd.turned) {
            cs = *(const f32x4*)(a.cos + pos * half + 4 * c);
            sn = *(const f32x4*)(a.sin + pos * half + 4 * c);
        }
        for (int h = h0; h < h1; ++h) {
            const bool isq = h < a.Hq;
            const bf16* src = isq ? (const bf16*)a.q + t * a.sq + h * D : (const bf16*)a.k + t * a.sk + (h - a.Hq) * D;
            const int64_t out = isq ? (t * a.Hq + h) * D : (t * a.Hk + h - a.Hq) * D;
            Row8 x, dy;
            unpack(x, load<kStream, bf16x4>(src + qd.lo), load<kStream, bf16x4>(src + qd.hi));
            if (kBwd) {
                const bf16* d = (const bf16*)(isq ? a.dyq : a.dyk) + out;
                unpack(dy, load<kStream, bf16x4>(d + qd.lo), load<kStream, bf16x4>(d + qd.hi));
            }
            const float r = inv_rms(x, a.eps);
            if (!kBwd) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x.x[e] = x.x[e] * r * (isq ? wq[e] : wk[e]);
                turn(x, cs, sn, kPairs, 1.0f);
            } else {
                // dn = R^T dy; dw += dn x^; dx = r (w dn - x^ mean(w dn x^))
                turn(dy, cs, sn, kPairs, -1.0f);
                float s = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x.x[e] *= r;
                    const float g = dy.x[e] * x.x[e];
                    gq[e] += isq ? g : 0.0f;
                    gk[e] += isq ? 0.0f : g;
                    dy.x[e] *= isq ? wq[e] : wk[e];
                    s += dy.x[e] * x.x[e];
                }
                s = row16_sum(s) * (1.0f / D);
#pragma unroll
                for (int e = 0; e < 8; ++e) x.x[e] = r * (dy.x[e] - x.x[e] * s);
            }
            bf16* y = kBwd ? (bf16*)(isq ? a.dq : a.dk) + out : (bf16*)(isq ? a.yq : a.yk) + out;
            store<kStream>(y + qd.lo, pack4(x.x));
            store<kStream>(y + qd.hi, pack4(x.x + 4));
        }
    }
    if (kBwd) {
        __shared__ float sums[RN_GROUPS][2 * D];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sums[grp][qd.lo + e] = gq[e];
            sums[grp][qd.hi + e] = gq[4 + e];
            sums[grp][D + qd.lo + e] = gk[e];
            sums[grp][D + qd.hi + e] = gk[4 + e];
        }
        __syncthreads();
        float s = 0.0f;
#pragma unroll
        for (int g = 0; g < RN_GROUPS; ++g) s += sums[g][threadIdx.x];
        a.part[(int64_t)blockIdx.x * 2 * D + threadIdx.x] = s;
    }
}

template <bool kSilu, bool kBwd, bool kStream>
__global__ __launch_bounds__(RN_THREADS) void gnorm_kernel(GNormArgs a) {
    const int c = threadIdx.x & 15, grp = threadIdx.x >> 4;
    const unsigned rows = (unsigned)a.tokens * (unsigned)a.H;
    float w[8], gw[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        w[e] = a.w[8 * c + e];
        gw[e] = 0.0f;
    }
    for (unsigned row = blockIdx.x * RN_GROUPS + grp; row < rows; row += gridDim.x * RN_GROUPS) {
        const unsigned tok = row / (unsigned)a.H;
        const int h = (int)(row - tok * (unsigned)a.H);
        const int64_t t = tok;
        const int64_t out = (int64_t)row * D + 8 * c;
        Row8 x, g, dy;
        const bf16x8 xv = load<kStream, bf16x8>((const bf16*)a.x + t * a.sx + h * D + 8 * c);
        const bf16x8 gv = load<kStream, bf16x8>((const bf16*)a.g + t * a.sg + h * D + 8 * c);
        bf16x8 dv;
        if (kBwd) dv = load<kStream, bf16x8>((const bf16*)a.dy + out);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x.x[e] = (float)xv[e];
            g.x[e] = (float)gv[e];
            if (kBwd) dy.x[e] = (float)dv[e];
        }
        const float r = inv_rms(x, a.eps);
        float act[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float sg = sigmoidf_(g.x[e]);
            // (g = -inf: sigmoid 0, and g sigmoid(g) tends to 0 as well)
            act[e] = kSilu ? (sg > 0.0f ? g.x[e] * sg : g.x[e] < 0.0f ? 0.0f : g.x[e] * sg) : sg;
            if (kBwd) {
                // sigmoid(-g) for 1 - sigmoid(g), whose digits cancel where the gate is open
                // (1% off at a gate of 12, 0 from 17 on)
                const float away = sigmoidf_(-g.x[e]);
                // (g = inf: g sigmoid(-g) tends to 0)
                const float slope = kSilu ? sg + (away > 0.0f ? act[e] * away : 0.0f) : sg * away;
                x.x[e] *= r;
                const float u = dy.x[e] * x.x[e];
                gw[e] += u * act[e];
                g.x[e] = u * w[e] * slope;      // dg
                dy.x[e] *= w[e] * act[e];       // gradient of the normed row
            } else {
                x.x[e] = x.x[e] * r * w[e] * act[e];
            }
        }
        if (!kBwd) {
            store<kStream>((bf16*)a.y + out, cat8(pack4(x.x), pack4(x.x + 4)));
        } else {
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += dy.x[e] * x.x[e];
            s = row16_sum(s) * (1.0f / D);
#pragma unroll
            for (int e = 0; e < 8; ++e) x.x[e] = r * (dy.x[e] - x.x[e] * s);
            store<kStream>((bf16*)a.dx + out, cat8(pack4(x.x), pack4(x.x + 4)));
            store<kStream>((bf16*)a.dg + out, cat8(pack4(g.x), pack4(g.x + 4)));
        }
    }
    if (kBwd) {
        __shared__ float sums[RN_GROUPS][D];
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[grp][8 * c + e] = gw[e];
        __syncthreads();
        if (threadIdx.x < D) {
            float s = 0.0f;
#pragma unroll
            for (int g = 0; g < RN_GROUPS; ++g) s += sums[g][threadIdx.x];
            a.part[(int64_t)blockIdx.x * D + threadIdx.x] = s;
        }
    }
}

// Column sums of part[blocks][cols]: workgroup b takes 8 columns, 32 rows at
// a time, and adds its 32 partial sums in order.  Columns below D go to out0.
__global__ __launch_bounds__(RN_THREADS) void colsum_kernel(const float* part, int blocks, int cols, float* out0,
                                                            float* out1) {
    __shared__ float sums[32][8];
    const int c = threadIdx.x & 7, r = threadIdx.x >> 3;
    const int col = blockIdx.x * 8 + c;
    float s = 0.0f;
#pragma unroll 8
    for (int i = r; i < blocks; i += 32) s += part[(int64_t)i * cols + col];
    sums[r][c] = s;
    __syncthreads();
    if (threadIdx.x < 8) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += sums[i][threadIdx.x];
        if (col < D)
            out0[col] = t;
        else
            out1[col - D] = t;
    }
}

int rownorm_blocks(int64_t rows) {
    const int64_t need = (rows + RN_GROUPS - 1) / RN_GROUPS;
    return (int)(need < RN_BWD_BLOCKS ? need : RN_BWD_BLOCKS);
}

namespace {

// Heads per unit: up to 8, fewer where that would leave a compute unit less than
// four workgroups.  (16384 tokens x 40 heads, forward and backward: 162 us at 8,
// 165 at 4, 178 at 2, 212 at 1, 190 at 16.)
int heads_per_unit(int64_t tokens, int H) {
    int per = 8;
    while (per > 1 && tokens * ((H + per - 1) / per) < (int64_t)RN_GROUPS * 1024) per >>= 1;
    return per;
}

// A forward pass has a group of lanes for every unit or row (up to a launch's
// 2^32 threads, then it loops as well); a backward pass loops, to sum its weight
// gradients.
dim3 forward_grid(int64_t groups) {
    const int64_t need = (groups + RN_GROUPS - 1) / RN_GROUPS, most = (int64_t)1 << 23;
    return dim3((unsigned)(need < most ? need : most));
}

template <bool kPairs, bool kBwd>
void launch_qknorm(const QkNormArgs& a, bool stream, dim3 grid, hipStream_t s) {
    if (stream)
        hipLaunchKernelGGL((qknorm_kernel<kPairs, kBwd, true>), grid, dim3(RN_THREADS), 0, s, a);
    else
        hipLaunchKernelGGL((qknorm_kernel<kPairs, kBwd, false>), grid, dim3(RN_THREADS), 0, s, a);
}
template <bool kSilu, bool kBwd>
void launch_gnorm(const GNormArgs& a, bool stream, dim3 grid, hipStream_t s) {
    if (stream)
        hipLaunchKernelGGL((gnorm_kernel<kSilu, kBwd, true>), grid, dim3(RN_THREADS), 0, s, a);
    else
        hipLaunchKernelGGL((gnorm_kernel<kSilu, kBwd, false>), grid, dim3(RN_THREADS), 0, s, a);
}

}  // namespace

hipError_t launch_qknorm_fwd(const QkNormArgs& args, hipStream_t s) {
    QkNormArgs a = args;
    const int H = a.Hq + a.Hk;
    a.per = heads_per_unit(a.tokens, H);
    const int64_t units = a.tokens * ((H + a.per - 1) / a.per);
    const bool stream = streams(a.tokens * H, 2);
    const dim3 grid = forward_grid(units);
    if (a.interleaved)
        launch_qknorm<true, false>(a, stream, grid, s);
    else
        launch_qknorm<false, false>(a, stream, grid, s);
    return hipGetLastError();
}

hipError_t launch_qknorm_bwd(const QkNormArgs& args, hipStream_t s) {
    QkNormArgs a = args;
    const int H = a.Hq + a.Hk;
    a.per = heads_per_unit(a.tokens, H);
    const bool stream = streams(a.tokens * H, 3);
    const int blocks = rownorm_blocks(a.tokens * H);
    if (a.interleaved)
        launch_qknorm<true, true>(a, stream, dim3(blocks), s);
    else
        launch_qknorm<false, true>(a, stream, dim3(blocks), s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(colsum_kernel, dim3(2 * D / 8), dim3(RN_THREADS), 0, s, (const float*)a.part, blocks, 2 * D,
                       a.dwq, a.dwk);
    return hipGetLastError();
}

hipError_t launch_gnorm_fwd(const GNormArgs& a, hipStream_t s) {
    const int64_t rows = a.tokens * a.H;
    const bool stream = streams(rows, 3);
    const dim3 grid = forward_grid(rows);
    if (a.silu)
        launch_gnorm<true, false>(a, stream, grid, s);
    else
        launch_gnorm<false, false>(a, stream, grid, s);
    return hipGetLastError();
}

hipError_t launch_gnorm_bwd(const GNormArgs& a, hipStream_t s) {
    const int64_t rows = a.tokens * a.H;
    const bool stream = streams(rows, 5);
    const int blocks = rownorm_blocks(rows);
    if (a.silu)
        launch_gnorm<true, true>(a, stream, dim3(blocks), s);
    else
        launch_gnorm<false, true>(a, stream, dim3(blocks), s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(colsum_kernel, dim3(D / 8), dim3(RN_THREADS), 0, s, (const float*)a.part, blocks, D, a.dw, a.dw);
    return hipGetLastError();
}

}  // namespace kda
