// Gated delta rule: training forward and backward scans, prefill, and the token-serial
// form for decode.
//
//     S <- e^{g_t} S;   S <- S + beta_t (v_t - S k_t) k_t^T;   o_t = s S q_t     (S[v][k], FP32)
//
// with one log-decay g_t <= 0 and one beta_t per value head and token.  In a chunk with
// the running sums G_i of g, A_ij = e^{G_i - G_j} k_i.k_j (j < i) and B = diag(beta), the
// rows W = U / beta of what the tokens write solve (1 + A B) W = X, X_i = v_i - e^{G_i} S k_i:
//     W = X - C B X,   C = A - A B C  (strictly lower),
//     o_i = s (e^{G_i} S q_i + sum_{j<=i} e^{G_i - G_j} (q_i.k_j) beta_j W_j),
//     S <- e^{G_n} S + sum_j e^{G_n - G_j} beta_j W_j k_j^T.
// Its adjoint walks backward with Z = dS in place of S: with
//     dU_j = s sum_{i>=j} e^{G_i - G_j} (q_i.k_j) do_i + e^{G_n - G_j} Z k_j,
//     Y = dU - C^T B dU,   dv = B Y,
//     Z <- e^{G_n} Z + s sum_i e^{G_i} do_i q_i^T - sum_i e^{G_i} beta_i Y_i k_i^T.
// C serves both, and does not depend on the state: a kernel of its own forms it for all
// chunks at once.  q and k at unit length enter as they are, with one over their length as
// a factor of their token.
#include "kda_delta_scan.hpp"

namespace kda {

namespace {

// G in base 2 is kept finite, so that a difference of two stays a number: e^-inf and
// 2^-16384 are both 0.
__device__ __forceinline__ double log2_gate(bf16 g) {
    const double x = (double)(float)g * 1.4426950408889634074;
    return x < -16384.0 ? -16384.0 : x;
}

}  // namespace

// One wave per (block of 64 tokens, value head); lane t holds token t's gates, lane 16b + c
// column c of the four diagonal tiles b.  C's diagonal tiles come from forward substitution,
// row after row, the one below from
//     C21 = (1 - C22 B2) A21 (1 - B1 C11)
// by FP32 MFMA.  Bound by the way of k's rows and the records, 12 KB per block and head: 8 x 1024 tokens,
// 96 heads 71 us (5.3 TB/s); 16 q/k and 64 value heads 4.2 TB/s.
constexpr int PREP_WAVES = 4;
constexpr int TS = 260;           // floats between the tiles in LDS: their rows then differ in banks
__global__ __launch_bounds__(64 * PREP_WAVES) void delta_prepare_kernel(DeltaArgs A, int64_t items) {
    __shared__ __align__(16) float tile_[PREP_WAVES][4 * TS];
    __shared__ __align__(16) float tok_[PREP_WAVES][6 * 64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, gq = lane >> 4, n16 = lane & 15;
    const int64_t item = (int64_t)blockIdx.x * PREP_WAVES + wave;
    if (item >= items) return;   // (no workgroup barrier below)
    float* tile = tile_[wave];
    float* tok = tok_[wave];
    const Item it = find_item(A.blocks, item);
    const int Hv = A.blocks.Hv;
    const int64_t at = it.seg * Hv + it.h;

    // rows: block b of 16 tokens, lane (gq, n) channels 32p + 8gq .. + 7 of token n
    auto rows = [&](const bf16* base, int64_t stride, bf16x8 (&r)[4][4]) __attribute__((always_inline)) {
        const bf16* p = base + it.tok0 * stride + (it.h / A.G) * D + 8 * gq;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const bool there = 16 * b + n16 < it.len;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                r[b][c] = there ? *(const bf16x8*)(p + (16 * b + n16) * stride + 32 * c) : bf16x8{};
        }
    };
    bf16x8 k[4][4];
    rows((const bf16*)A.k, A.sk, k);
    // gates: running sums inside each half of the wave, in 64 bits
    const bool valid = lane < it.len;
    const int64_t gat = (it.tok0 + (valid ? lane : 0)) * Hv + it.h;
    double G = valid ? log2_gate(((const bf16*)A.g)[gat]) : 0.0;
    const float beta = valid ? (float)((const bf16*)A.beta)[gat] : 0.0f;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const double y = __shfl_up(G, d, 32);
        if ((lane & 31) >= d) G += y;
    }
    const double last = __shfl(G, 31, 32);
    const float gh = (float)G, gl = (float)(G - (double)(float)G);
    // squared lengths: the diagonals of k k^T and q q^T
    auto diagonal = [&](const bf16x8 (&r)[4][4], float* to) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            f32x4 acc = zero4();
#pragma unroll
            for (int c = 0; c < 4; ++c) acc = mma32(r[b][c], r[b][c], acc);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (4 * gq + e == n16) to[16 * b + n16] = acc[e];
        }
    };
    float rk = 1.0f, rq = 1.0f;
    if (A.unit) {
        diagonal(k, tok);
        if (A.rq) {
            bf16x8 q[4][4];
            rows((const bf16*)A.q, A.sq, q);
            diagonal(q, tok + 64);
        }
        __builtin_amdgcn_wave_barrier();
        rk = rsqrtf(tok[lane] + NORM_EPS);
        if (A.rq) rq = rsqrtf(tok[64 + lane] + NORM_EPS);
        __builtin_amdgcn_wave_barrier();
    }
    if (!valid) rk = rq = 0.0f;
    float* gh_ = tok;
    float* gl_ = tok + 64;
    float* rk_ = tok + 128;
    float* beta_ = tok + 192;
    gh_[lane] = gh;
    gl_[lane] = gl;
    rk_[lane] = rk;
    beta_[lane] = beta;
    __builtin_amdgcn_wave_barrier();

    char* rec = A.rec + at * (2 * REC);
    {
        char* r = rec + (lane >> 5) * REC + (lane & 31) * 4;
        const float from = (float)exp2(G), to = (float)exp2(last - G);
        *(float*)(r + REC_FROM) = from;
        *(float*)(r + REC_FROM_K) = from * rk;
        *(float*)(r + REC_FROM_KB) = from * rk * beta;
        *(float*)(r + REC_TO_K) = to * rk;
        *(float*)(r + REC_TO_KB) = to * rk * beta;
        *(float*)(r + REC_K) = rk;
        *(float*)(r + REC_KB) = rk * beta;
        *(float*)(r + REC_BETA) = beta;
        *(float*)(r + REC_Q) = rq;
        *(float*)(r + REC_GH) = gh;
        *(float*)(r + REC_GL) = gl;
        if ((lane & 31) == 0) {
            const Factor f(exp2(last));
            *(float*)(r + REC_DECAY) = f.f;
            *(float*)(r + REC_DECAY + 4) = f.low;
        }
    }
    // A's tiles.  Diagonal: lane (gq, n) holds rows 4gq + e of column n.  Below: lane (gq, n)
    // holds columns 4gq + e of row n, as the operand of a product needs it.
    f32x4 a21[2];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        f32x4 acc = zero4();
#pragma unroll
        for (int c = 0; c < 4; ++c) acc = mma32(k[b][c], k[b][c], acc);
        const int j = 16 * b + n16;
        const float hj = gh_[j], lj = gl_[j], rj = rk_[j];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 16 * b + 4 * gq + e;
            const float x = acc[e] * decay2(gh_[i], gl_[i], hj, lj) * rk_[i] * rj;
            tile[b * TS + (4 * gq + e) * 16 + n16] = 4 * gq + e > n16 ? x : 0.0f;
        }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        f32x4 acc = zero4();
#pragma unroll
        for (int c = 0; c < 4; ++c) acc = mma32(k[2 * s][c], k[2 * s + 1][c], acc);
        const int i = 32 * s + 16 + n16;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = 32 * s + 4 * gq + e;
            acc[e] *= decay2(gh_[i], gl_[i], gh_[j], gl_[j]) * rk_[i] * rk_[j];
        }
        a21[s] = acc;
    }
    __builtin_amdgcn_wave_barrier();
    // C = A - A B C, tile gq, column n: c_i = A_in - sum_{j<i} A_ij beta_j c_j
    {
        const float* t = tile + gq * TS;
        const float* bt = beta_ + 16 * gq;
        float c[16], bc[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) c[i] = t[i * 16 + n16];
        bc[0] = 0.0f;   // (C's first row is zero)
#pragma unroll
        for (int i = 1; i < 16; ++i) {
#pragma unroll
            for (int j = 1; j < i; ++j) c[i] -= t[i * 16 + j] * bc[j];
            bc[i] = bt[i] * c[i];
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < 16; ++i) tile[gq * TS + i * 16 + n16] = c[i];
        __builtin_amdgcn_wave_barrier();
    }
    // 4 columns of a row of -C's tile, in pieces
    const Pieces pieces(lane);
    auto put = [&](char* to, f32x4 x) __attribute__((always_inline)) {
        bf16x4 p[3];
        pieces.split(-x, p[0], p[1], p[2]);
#pragma unroll
        for (int i = 0; i < 3; ++i) *(bf16x4*)(to + i * REC_TILE + n16 * 32 + gq * 8) = p[i];
    };
#pragma unroll
    for (int b = 0; b < 4; ++b)
        put(rec + (b >> 1) * REC + (b & 1 ? REC_C22 : REC_C11), *(const f32x4*)(tile + b * TS + n16 * 16 + 4 * gq));
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const float* c11 = tile + 2 * s * TS;
        const float* c22 = c11 + TS;
        f32x4 h = zero4();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = 4 * gq + e;
            const float t = (j == n16 ? 1.0f : 0.0f) - beta_[32 * s + j] * c11[j * 16 + n16];
            h = __builtin_amdgcn_mfma_f32_16x16x4f32(a21[s][e], t, h, 0, 0, 0);
        }
        const f32x4 row = *(const f32x4*)(c22 + n16 * 16 + 4 * gq);
        f32x4 r = h;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            r = __builtin_amdgcn_mfma_f32_16x16x4f32(-row[e] * beta_[32 * s + 16 + 4 * gq + e], h[e], r, 0, 0, 0);
        // rows 4gq + e of column n16: through LDS (over tile 2s, which is read) to the rows' order
        __builtin_amdgcn_wave_barrier();
        float* t = tile + 2 * s * TS;
#pragma unroll
        for (int e = 0; e < 4; ++e) t[(4 * gq + e) * 16 + n16] = r[e];
        __builtin_amdgcn_wave_barrier();
        put(rec + s * REC + REC_C21, *(const f32x4*)(t + n16 * 16 + 4 * gq));
    }
}

hipError_t launch_delta_prepare(const DeltaArgs& a, hipStream_t s) {
    const int64_t items = a.blocks.items;
    hipLaunchKernelGGL(delta_prepare_kernel, dim3((unsigned)((items + PREP_WAVES - 1) / PREP_WAVES)),
                       dim3(64 * PREP_WAVES), 0, s, a, items);
    return hipGetLastError();
}

// Four waves with two tiles each spend the least on reading the rows out of LDS.  With one
// workgroup for every second compute unit at most, two of half the columns each shorten a chunk.
// (1024 tokens of 48, 64, 96, 128 sequences and heads, in us: 113, 111, 114, 117 in four waves, 83, 84, 87, 94 in two
// workgroups; of 160, 192, 256: 123, 124, 129 and 128, 130, 142.)
template <int NU, int kParts, int kMode>
__global__ __launch_bounds__(512 / NU / kParts, 2) void delta_scan_kernel(DeltaArgs A) {
    __shared__ __align__(16) char lds[DeltaScanLds<kMode>::TOTAL];
    delta_scan<NU, kParts, kMode>(A, blockIdx.x, gridDim.x, lds);
}

template <int kMode>
static hipError_t launch_scan(const DeltaArgs& a, hipStream_t s) {
    const int64_t items = a.map.items * (kMode == kDeltaState ? 2 : 1);
    if (items <= 128)
        hipLaunchKernelGGL((delta_scan_kernel<1, 2, kMode>), dim3((unsigned)(items * 2)), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((delta_scan_kernel<2, 1, kMode>), dim3((unsigned)items), dim3(256), 0, s, a);
    return hipGetLastError();
}
hipError_t launch_delta_scan(const DeltaArgs& a, hipStream_t s) { return launch_scan<kDeltaOut>(a, s); }

// The states before the segments, S <- S M + Q from one to the next; kReverse: the adjoints behind
// them, Z <- Z M^T + R from the last to the first.  A workgroup per sequence, value head and 16 channels v,
// wave t with their tile of the state as in the scan.  The product is exact to FP32, both
// factors in three BF16 pieces.  Bound by the steps of one segment, 2.6 us: M's pieces, S's way through
// LDS, the products in four sums (in one sum, M taken apart behind the barrier, 3.2 us).  The M's of the
// next two segments are on their way meanwhile.
template <bool kReverse>
__global__ __launch_bounds__(512) void delta_chain_kernel(DeltaArgs A) {
    __shared__ __align__(16) char lds[2][3 * 4 * 1024];   // the state in pieces: [piece][32 channels k][lane][8]
    const int block = xcd_order(blockIdx.x, gridDim.x, 8);   // (the eight that read an M share a cache)
    const Item it = find_item(A.seqs, block >> 3);
    const int64_t slot = A.slot != nullptr ? A.slot[it.n] : it.n;
    if (slot < 0 || slot >= A.slots) return;
    const int Hv = A.map.Hv;
    const int t = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, gq = lane >> 4, n16 = lane & 15;
    const int64_t per = A.map.seg_len;
    const int segs = (int)((it.len + per - 1) / per);
    const int64_t first = A.map.task != nullptr ? A.map.tape_off[it.n] + it.n : it.n * (int64_t)segs;
    // (a place i counts from the chain's start)
    const int64_t item = (first + (kReverse ? segs - 1 : 0)) * Hv + it.h;
    const int64_t step = kReverse ? -Hv : Hv;
    const int64_t size = kReverse ? STATE : 2 * STATE;
    const int at = (16 * (block & 7) + n16) * D + 32 * (t >> 1) + 8 * gq + 4 * (t & 1);
    float* own = (kReverse ? A.behind : A.seg) + item * size + at;
    // of M transposed, [k][k']: 8 values k' of the row k that belongs to lane n, or (reverse) 8 rows k of column k'
    const int row = 32 * (t >> 1) + 8 * (n16 >> 2) + 4 * (t & 1) + (n16 & 3);
    const float* map = A.seg + item * (2 * STATE) + STATE + (kReverse ? 8 * gq * D + row : row * D + 8 * gq);
    auto get_map = [&](int i, f32x4 (&m)[4][2]) __attribute__((always_inline)) {
        const float* from = map + i * step * (2 * STATE);
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (kReverse) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) m[p][j][e] = from[(32 * p + 4 * j + e) * D];
                } else {
                    m[p][j] = *(const f32x4*)(from + 32 * p + 4 * j);
                }
            }
    };
    auto get_own = [&](int i) __attribute__((always_inline)) { return *(const f32x4*)(own + i * step * size); };

    const Pieces pieces(lane);
    f32x4 x = A.s_in != nullptr ? *(const f32x4*)(A.s_in + (slot * Hv + it.h) * (int64_t)STATE + at) : zero4();
    f32x4 m1[4][2], m2[4][2], q0 = zero4(), q1 = zero4(), q2 = zero4();
    if (segs > 1) q0 = get_own(0);
    if (segs > 2) {
        q1 = get_own(1);
        get_map(1, m1);
    }
    if (segs > 3) {
        q2 = get_own(2);
        get_map(2, m2);
    }
    *(f32x4*)own = x;
    if (segs == 1) return;
    x = q0;   // (the first place's own sum starts from s_in)
    auto place = [&](int i, f32x4 (&m)[4][2], f32x4& q, char* to) __attribute__((always_inline)) {
        *(f32x4*)(own + i * step * size) = x;
        if (i + 1 == segs) return false;
        bf16x8 mp[4][3];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            bf16x4 m0[3], m1[3];
            pieces.split(m[p][0], m0[0], m0[1], m0[2]);
            pieces.split(m[p][1], m1[0], m1[1], m1[2]);
#pragma unroll
            for (int d = 0; d < 3; ++d) mp[p][d] = cat8(m0[d], m1[d]);
        }
        bf16x4 a[3];
        pieces.split(x, a[0], a[1], a[2]);
#pragma unroll
        for (int d = 0; d < 3; ++d) *(bf16x4*)(to + ((d * 4 + (t >> 1)) * 64 + lane) * 16 + 8 * (t & 1)) = a[d];
        const f32x4 add = q;
        if (i + 3 < segs) {
            q = get_own(i + 2);
            get_map(i + 2, m);
        }
        barrier_lds();
        f32x4 sum[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            bf16x8 b[3];
#pragma unroll
            for (int d = 0; d < 3; ++d) b[d] = *(const bf16x8*)(to + ((d * 4 + p) * 64 + lane) * 16);
            sum[p] = zero4();
#pragma unroll
            for (int i = 2; i >= 0; --i)
#pragma unroll
                for (int d = 0; d <= i; ++d) sum[p] = mma32(mp[p][d], b[i - d], sum[p]);
        }
        x = add + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
        return true;
    };
    for (int i = 1;; i += 2) {
        if (!place(i, m1, q1, lds[0])) break;
        if (!place(i + 1, m2, q2, lds[1])) break;
    }
}

hipError_t launch_delta_chain(const DeltaArgs& a, bool reverse, hipStream_t s) {
    const dim3 grid((unsigned)(a.seqs.items * 8));
    if (reverse)
        hipLaunchKernelGGL((delta_chain_kernel<true>), grid, dim3(512), 0, s, a);
    else
        hipLaunchKernelGGL((delta_chain_kernel<false>), grid, dim3(512), 0, s, a);
    return hipGetLastError();
}
hipError_t launch_delta_segments(const DeltaArgs& a, hipStream_t s) {
    const hipError_t e = launch_scan<kDeltaState>(a, s);
    return e == hipSuccess ? launch_delta_chain(a, false, s) : e;
}

// Token-serial form on the FP32 state pool (decode, drafted tokens, and sequences of a few
// tokens).  A workgroup takes 32 of the 128 state rows of one (sequence, value head): a half
// wave holds a row (4 channels a lane), each wave 4 pairs of rows, so that every load and
// store moves 1 KiB of contiguous state and S k and S q are sums over the half wave.  Both
// are taken from the decayed state, o = s (S q + u k.q), so that their sums run side by side.
// No LDS, no barrier; everything FP32, the decay as the sum of two values.
// Bound by the states' way in and out; non-temporal (kStream) when that exceeds kStreamBytes.
// 128 sequences x 64 heads, one token: 179 us, 6.1 TB/s; 32 x 32, five drafted tokens: 79 us, 5.3 TB/s.
template <bool kStream>
__global__ __launch_bounds__(256) void delta_token_kernel(DeltaTokenArgs A) {
    const Item it = find_item(A.map, blockIdx.x >> 2);
    const int64_t first = (int64_t)it.n * A.each;
    int64_t slot = it.n;
    if (A.slot != nullptr) {
        const int back = A.accepted != nullptr ? min(max(A.accepted[it.n], 1), A.each) - 1 : 0;
        slot = A.slot[first + back];
    }
    if (slot < 0 || slot >= A.slots) return;
    const int Hv = A.map.Hv;
    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int ch = (lane & 31) * 4;
    const int row0 = (blockIdx.x & 3) * 32 + (tid >> 6) * 2 + half;   // + 8j
    float* S = A.pool + (slot * Hv + it.h) * (int64_t)STATE + ch;
    f32x4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const f32x4* p = (const f32x4*)(S + (row0 + 8 * j) * D);
        x[j] = kStream ? __builtin_nontemporal_load(p) : *p;
    }
    auto put = [&](float* to) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f32x4* p = (f32x4*)(to + (row0 + 8 * j) * D);
            if (kStream)
                __builtin_nontemporal_store(x[j], p);
            else
                *p = x[j];
        }
    };
    auto half_sum = [&](float s) __attribute__((always_inline)) {
        s = row16_sum(s);
        return s + __shfl_xor(s, 16, 64);
    };
    auto dot = [&](f32x4 a, f32x4 b) __attribute__((always_inline)) {
        return a[0] * b[0] + a[1] * b[1] + (a[2] * b[2] + a[3] * b[3]);
    };
    const int hq = it.h / A.G;
    const bf16* q = (const bf16*)A.q + it.tok0 * A.sq + hq * D + ch;
    const bf16* k = (const bf16*)A.k + it.tok0 * A.sk + hq * D + ch;
    const bf16* v = (const bf16*)A.v + it.tok0 * A.sv + it.h * D + row0;
    const bf16* g = (const bf16*)A.g + it.tok0 * Hv + it.h;
    const bf16* beta = (const bf16*)A.beta + it.tok0 * Hv + it.h;
    bf16* o = (bf16*)A.o + (it.tok0 * Hv + it.h) * D + row0;
    for (int64_t t = 0; t < it.len; ++t) {
        const f32x4 qf = from_bf4(*(const bf16x4*)(q + t * A.sq));
        const f32x4 kf = from_bf4(*(const bf16x4*)(k + t * A.sk));
        const Factor decay(exp((double)(float)g[t * Hv]));
        const float b = (float)beta[t * Hv];
        const float kq = half_sum(dot(kf, qf));
        float rq = 1.0f, rk = 1.0f;
        if (A.unit) {
            rq = rsqrtf(half_sum(dot(qf, qf)) + NORM_EPS);
            rk = rsqrtf(half_sum(dot(kf, kf)) + NORM_EPS);
        }
        float sk[4], sq[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[j][e] = decay.apply(x[j][e]);
            sk[j] = half_sum(dot(x[j], kf));
            sq[j] = half_sum(dot(x[j], qf));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float u = b * rk * ((float)v[t * A.sv + 8 * j] - rk * sk[j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[j][e] = fmaf(u, kf[e], x[j][e]);
            if ((lane & 31) == 0) o[t * Hv * D + 8 * j] = (bf16)(A.scale * rq * (sq[j] + u * kq));
        }
        if (A.each > 1) {   // the state after token t, to token t's slot
            const int64_t to = A.slot[first + t];
            if (to >= 0 && to < A.slots) put(A.pool + (to * Hv + it.h) * (int64_t)STATE + ch);
        }
    }
    if (A.each == 1) put(S);
}

hipError_t launch_delta_token(const DeltaTokenArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.map.items * 4));
    if ((1 + a.each) * a.map.items * STATE * 4 > kStreamBytes)
        hipLaunchKernelGGL((delta_token_kernel<true>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((delta_token_kernel<false>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace kda
