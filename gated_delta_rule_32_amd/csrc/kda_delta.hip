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
#include "kda_delta.hpp"

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
// by FP32 MFMA.
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
        bf16x8 q[4][4];
        rows((const bf16*)A.q, A.sq, q);
        diagonal(q, tok + 64);
        __builtin_amdgcn_wave_barrier();
        rk = rsqrtf(tok[lane] + NORM_EPS);
        rq = rsqrtf(tok[64 + lane] + NORM_EPS);
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

    float* rec = A.rec + at * (2 * REC);
    {
        float* r = rec + (lane >> 5) * REC + (lane & 31);
        const float from = (float)exp2(G);
        r[REC_CX] = from * rk;
        r[REC_CE] = (float)exp2(last - G) * rk;
        r[REC_CO] = A.scale * (from * rq);
        r[REC_BETA] = beta;
        r[REC_GH] = gh;
        r[REC_GL] = gl;
        r[REC_A] = A.scale * rq;
        r[REC_RK] = rk;
        if ((lane & 31) == 0) {
            const Factor f(exp2(last));
            float* fac = A.fac + at * 4 + (lane >> 5) * 2;
            fac[0] = f.f;
            fac[1] = f.low;
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
        float* out = rec + (gq >> 1) * REC + (gq & 1 ? REC_C22 : REC_C11) + n16;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            out[i * 16] = c[i];
            tile[gq * TS + i * 16 + n16] = c[i];
        }
        __builtin_amdgcn_wave_barrier();
    }
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
        float* out = rec + s * REC + REC_C21 + n16;
#pragma unroll
        for (int e = 0; e < 4; ++e) out[(4 * gq + e) * 16] = r[e];
    }
}

hipError_t launch_delta_prepare(const DeltaArgs& a, hipStream_t s) {
    const int64_t items = a.blocks.items;
    hipLaunchKernelGGL(delta_prepare_kernel, dim3((unsigned)((items + PREP_WAVES - 1) / PREP_WAVES)),
                       dim3(64 * PREP_WAVES), 0, s, a, items);
    return hipGetLastError();
}

// One workgroup per item (kParts = 2: two, each with half of the state's output channels), a
// wave for every NU tiles of 16 channels v.  A wave keeps its columns of the state as MFMA
// accumulators: tile (t, u) is S^T[k][v] with
//     k = 32(t/2) + 8gq + 4(t%2) + e,   v = 32wv + 8(n/4) + 4u + n%4
// (NU = 1: v = 16wv + n; lane 16gq + n, element e).  The same registers are the operand of
// S K^T from either side, so that X = V - S K^T comes out with tokens along the elements,
// where W = X - C B X and S^T += K^T U take it without leaving the lane, and o^T = S Q^T +
// W^T P^T with 8 neighbouring channels of a token for its store.  Only P = Q K^T passes
// between waves.
// Products are exact to FP32: S and B X go in as three BF16 pieces of 8 bits, C as three, U
// as three; P and W as two where they only meet o.  The rows of the next chunk and its record travel
// to the other of two LDS buffers while this one is computed.
template <int NU, int kParts, int kMode>
__global__ __launch_bounds__(512 / NU / kParts, 2) void delta_scan_kernel(DeltaArgs A) {
    constexpr bool kOut = kMode == kDeltaOut, kRecord = kMode == kDeltaRecord;
    constexpr int NW = 8 / NU / kParts;
    constexpr int SETS = kOut ? 3 : 2, SET = SC * D * 2, LK = 0, LV = 2 * SET, LQ = 4 * SET, LPT = 1024;
    constexpr int ROWS16 = 16 * D * 2;
    __shared__ __align__(16) char lds[2 * SETS * SET];
    __shared__ __align__(16) float lds_r[2][REC];
    __shared__ __align__(16) char lds_p[kOut ? 3 * LPT : 16];

    const int tid = threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63, gq = lane >> 4, n16 = lane & 15;
    int idx = xcd_order(blockIdx.x, (int)gridDim.x, A.G * kParts);
    const int part = idx % kParts;
    idx /= kParts;
    const int wv = w + NW * part;   // this wave among the columns
    const Item it = find_item(A.map, idx);
    const int64_t slot = A.slot != nullptr ? A.slot[it.n] : it.n;
    if (slot < 0 || slot >= A.slots) return;
    const int Hv = A.map.Hv;
    const int64_t soff = (slot * Hv + it.h) * (int64_t)STATE;
    // the item's first block among all blocks
    const int64_t block0 = (A.blocks.task != nullptr ? A.blocks.tape_off[it.n] + it.n
                                                     : (int64_t)it.n * ((A.blocks.len + DB - 1) / DB)) + it.off / DB;

    // Loads: one instruction of a wave moves 4 rows of 256 bytes (16 lanes a row) to 1 KiB of
    // LDS in lane order; a lane fetches the block that belongs there.
    const int lrow = 4 * w + gq;
    constexpr int STEP = 4 * NW;
    const bf16* src[3] = {(const bf16*)A.k, (const bf16*)A.v, (const bf16*)A.q};
    const int64_t stride[3] = {A.sk, A.sv, A.sq};
    const char* pr[SETS];
    unsigned off[SETS];
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
        pr[i] = (const char*)(src[i] + it.tok0 * stride[i] + (i == 1 ? it.h : it.h / A.G) * D);
        off[i] = (unsigned)lrow * (unsigned)(stride[i] * 2) + ((n16 ^ swz(lrow)) << 4);
    }
    static_assert(STEP % 16 == 0, "rows of one lane share their place in a row's order");
    const char* prec = (const char*)(A.rec + (block0 * Hv + it.h) * (2 * REC));
    const float* pfac = A.fac + (block0 * Hv + it.h) * 4;
    auto fetch = [&](char* rows_to, float* rec_to, int t0) __attribute__((always_inline)) {
        const int rem = it.len - t0;
#pragma unroll
        for (int j = 0; j < SC / STEP; ++j) {
            if (rem >= SC || lrow + STEP * j < rem) {
#pragma unroll
                for (int i = 0; i < SETS; ++i)
                    to_lds<false>(pr[i] + j * STEP * 2 * stride[i], off[i], rows_to + 2 * i * SET + (STEP * j + 4 * w) * D * 2);
            } else {   // rows behind the last token are not read and count as zero
#pragma unroll
                for (int i = 0; i < SETS; ++i)
                    *(u32x4*)(rows_to + 2 * i * SET + (STEP * j + 4 * w) * D * 2 + lane * 16) = u32x4{0u, 0u, 0u, 0u};
            }
        }
        if (w < 4) {
            // (a block's second record is behind the first, the next block's Hv blocks on)
            const int c = t0 / SC;
            const char* p = prec + ((int64_t)(c >> 1) * Hv * 2 + (c & 1)) * (REC * 4) + w * 1024;
            to_lds<false>(p, lane * 16, (char*)rec_to + w * 1024);
        }
#pragma unroll
        for (int i = 0; i < SETS; ++i) pr[i] += SC * 2 * stride[i];
    };
    static_assert(NW >= 4, "a record is moved by four waves");
    fetch(lds, lds_r[0], 0);

    f32x4 S[8][NU];
    const int vrow = NU == 2 ? 32 * wv + 8 * (n16 >> 2) + (n16 & 3) : 16 * wv + n16;   // + 4u
    auto krow = [&](int t) __attribute__((always_inline)) { return 32 * (t >> 1) + 8 * gq + 4 * (t & 1); };
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int u = 0; u < NU; ++u)
            S[t][u] = A.s_in != nullptr ? *(const f32x4*)(A.s_in + soff + (vrow + 4 * u) * D + krow(t)) : zero4();

    // LDS offsets (bytes): as in the constant-decay scan
    const int r8 = (n16 * D + ((gq ^ swz(n16)) << 3)) * 2;
    const int trow = 4 * gq + (n16 >> 2), piece = n16 & 3;
    const int tr = (trow * D + ((piece ^ swz(trow)) << 3)) * 2;
    const int trv = NU == 2 ? (trow * D + (((4 * wv + piece) ^ swz(trow)) << 3)) * 2
                            : (trow * D + (((2 * wv + (piece >> 1)) ^ swz(trow)) << 3) + 4 * (piece & 1)) * 2;
    const int64_t sy = (int64_t)Hv * D * 2;
    char* po = (char*)(A.o + (it.tok0 * Hv + it.h) * D);
    const unsigned oy = (unsigned)n16 * (unsigned)sy + (16 * NU * wv + 4 * NU * gq) * 2;

    // One chunk from `buf` and `rec`, the next one on its way into `rows_to` and `rec_to`.
    // (Both pairs are halves of the same arrays; as restrict pointers they show the compiler
    // that what is read through the one need not wait for what is on its way into the other.)
    auto chunk = [&](int t0, const char* __restrict__ buf, const float* __restrict__ rec, char* __restrict__ rows_to,
                     float* __restrict__ rec_to) __attribute__((always_inline)) {
        const int rem = it.len - t0, c = t0 / SC;
        const bool more = rem > SC;
        if (more) fetch(rows_to, rec_to, t0 + SC);
        const float* fac = pfac + (int64_t)(c >> 1) * Hv * 4 + (c & 1) * 2;
        const float f = fac[0], f_low = fac[1];
        if (kOut) {   // P^T tiles: (i, j) = (0, 0), (1, 1), (1, 0)
#pragma unroll
            for (int tile = 0; tile < 3; ++tile) {
                if (w != tile) continue;
                const int bi = tile == 0 ? 0 : 1, bj = tile == 1 ? 1 : 0;
                f32x4 acc = zero4();
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    acc = mma32(*(const bf16x8*)(buf + LK + ((r8 + bj * ROWS16) ^ (64 * p))),
                                *(const bf16x8*)(buf + LQ + ((r8 + bi * ROWS16) ^ (64 * p))), acc);
                const int i = 16 * bi + n16, j = 16 * bj + 4 * gq;
                const float ai = rec[REC_A + i], hi = rec[REC_GH + i], li = rec[REC_GL + i];
                const f32x4 rj = *(const f32x4*)(rec + REC_RK + j), bt = *(const f32x4*)(rec + REC_BETA + j),
                            hj = *(const f32x4*)(rec + REC_GH + j), lj = *(const f32x4*)(rec + REC_GL + j);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = acc[e] * (ai * rj[e] * bt[e]) * decay2(hi, li, hj[e], lj[e]);
                    acc[e] = i >= j + e ? x : 0.0f;
                }
                bf16x4 hi4, lo4;
                split4_rne(acc, hi4, lo4);
                *(bf16x8*)(lds_p + tile * LPT + lane * 16) = cat8(hi4, lo4);
            }
        }
        // S K^T and S Q^T
        f32x4 x[2][NU], y[2][NU];
#pragma unroll
        for (int ti = 0; ti < 2; ++ti)
#pragma unroll
            for (int u = 0; u < NU; ++u) x[ti][u] = y[ti][u] = zero4();
        const bool keep = kRecord && (c & 1) == 0;
        char* planes = kRecord ? (char*)(A.state_planes + ((block0 + (c >> 1)) * Hv + it.h) * (int64_t)(2 * STATE)) : nullptr;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            bf16x8 ak[2], aq[2];
#pragma unroll
            for (int ti = 0; ti < 2; ++ti) {
                ak[ti] = *(const bf16x8*)(buf + LK + ((r8 + ti * ROWS16) ^ (64 * p)));
                if (kOut) aq[ti] = *(const bf16x8*)(buf + LQ + ((r8 + ti * ROWS16) ^ (64 * p)));
            }
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                bf16x4 pc[3][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) split3(S[2 * p + i][u], pc[0][i], pc[1][i], pc[2][i]);
#pragma unroll
                for (int d = 0; d < 3; ++d) {
                    const bf16x8 s = cat8(pc[d][0], pc[d][1]);
#pragma unroll
                    for (int ti = 0; ti < 2; ++ti) x[ti][u] = mma32(ak[ti], s, x[ti][u]);
                    if (kOut && d < 2) {
#pragma unroll
                        for (int ti = 0; ti < 2; ++ti) y[ti][u] = mma32(s, aq[ti], y[ti][u]);
                    }
                    if (kRecord && d < 2 && keep)
                        *(bf16x8*)(planes + d * (STATE * 2) + ((vrow + 4 * u) * D + krow(2 * p)) * 2) = s;
                }
            }
        }
        // X = V - e^G S K^T, W = X - C B X
        f32x4 wr[2][NU];
#pragma unroll
        for (int ti = 0; ti < 2; ++ti) {
            const f32x4 cx = *(const f32x4*)(rec + REC_CX + 16 * ti + 4 * gq);
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const f32x4 v = from_bf4(tr_read(buf + LV + trv + 8 * u + ROWS16 * ti));
#pragma unroll
                for (int e = 0; e < 4; ++e) wr[ti][u][e] = fmaf(-cx[e], x[ti][u][e], v[e]);
            }
        }
        {
            bf16x4 c11[3], c22[3], c21[3];
            const int rm = n16 * 16 + 4 * gq;
            split3(-*(const f32x4*)(rec + REC_C11 + rm), c11[0], c11[1], c11[2]);
            split3(-*(const f32x4*)(rec + REC_C22 + rm), c22[0], c22[1], c22[2]);
            split3(-*(const f32x4*)(rec + REC_C21 + rm), c21[0], c21[1], c21[2]);
            const f32x4 b0 = *(const f32x4*)(rec + REC_BETA + 4 * gq), b1 = *(const f32x4*)(rec + REC_BETA + 16 + 4 * gq);
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                bf16x4 x0[3], x1[3];
                split3(wr[0][u] * b0, x0[0], x0[1], x0[2]);
                split3(wr[1][u] * b1, x1[0], x1[1], x1[2]);
                // pieces (a, b) with a + b <= 2; row block 0 takes two products at once
                wr[0][u] = mma32(cat8(c11[0], c11[0]), cat8(x0[0], x0[1]), wr[0][u]);
                wr[0][u] = mma32(cat8(c11[1], c11[1]), cat8(x0[0], x0[1]), wr[0][u]);
                wr[0][u] = mma32(cat8(c11[0], c11[2]), cat8(x0[2], x0[0]), wr[0][u]);
#pragma unroll
                for (int a = 0; a < 3; ++a)
#pragma unroll
                    for (int b = 0; a + b < 3; ++b)
                        wr[1][u] = mma32(cat8(c21[a], c22[a]), cat8(x0[b], x1[b]), wr[1][u]);
            }
        }
        if (kRecord) {   // the rows W, as planes [v][token]
            char* rp = (char*)(A.row_planes + (((block0 + (c >> 1)) * Hv + it.h) * 2 + (c & 1)) * (int64_t)(2 * D * SC));
#pragma unroll
            for (int ti = 0; ti < 2; ++ti)
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                    bf16x4 hi, lo;
                    split4_rne(wr[ti][u], hi, lo);
                    char* d = rp + ((vrow + 4 * u) * SC + 16 * ti + 4 * gq) * 2;
                    *(bf16x4*)d = hi;
                    *(bf16x4*)(d + D * SC * 2) = lo;
                }
        }
        if (kOut) {
            barrier_lds();
            const bf16x8 p00 = *(const bf16x8*)(lds_p + lane * 16), p11 = *(const bf16x8*)(lds_p + LPT + lane * 16),
                         p10 = *(const bf16x8*)(lds_p + 2 * LPT + lane * 16);
            const bf16x8 p1h = __builtin_shufflevector(p10, p11, 0, 1, 2, 3, 8, 9, 10, 11),
                         p1l = __builtin_shufflevector(p10, p11, 4, 5, 6, 7, 12, 13, 14, 15);
            const float co[2] = {rec[REC_CO + n16], rec[REC_CO + 16 + n16]};
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                bf16x4 h0, l0, h1, l1;
                split4_rne(wr[0][u], h0, l0);
                split4_rne(wr[1][u], h1, l1);
#pragma unroll
                for (int ti = 0; ti < 2; ++ti) y[ti][u] *= co[ti];
                y[0][u] = mma32(cat8(h0, h0), p00, y[0][u]);
                y[0][u] = mma32(cat8(l0, l0), p00, y[0][u]);
                y[1][u] = mma32(cat8(h0, h1), p1h, y[1][u]);
                y[1][u] = mma32(cat8(h0, h1), p1l, y[1][u]);
                y[1][u] = mma32(cat8(l0, l1), p1h, y[1][u]);
            }
#pragma unroll
            for (int ti = 0; ti < 2; ++ti) {
                u32x2 r[NU];
#pragma unroll
                for (int u = 0; u < NU; ++u) r[u] = __builtin_bit_cast(u32x2, to_bf4(y[ti][u]));
                if (16 * ti + n16 < rem) {
                    if constexpr (NU == 2)
                        *row_ptr<u32x4>(po + 16 * ti * sy, oy) = u32x4{r[0][0], r[0][1], r[1][0], r[1][1]};
                    else
                        *row_ptr<u32x2>(po + 16 * ti * sy, oy) = r[0];
                }
            }
            po += SC * sy;
        }
        // S <- e^{G_n} S + K^T U
        bf16x8 u3[3][NU];
        {
            const f32x4 e0 = *(const f32x4*)(rec + REC_CE + 4 * gq) * *(const f32x4*)(rec + REC_BETA + 4 * gq);
            const f32x4 e1 = *(const f32x4*)(rec + REC_CE + 16 + 4 * gq) * *(const f32x4*)(rec + REC_BETA + 16 + 4 * gq);
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                bf16x4 a0[3], a1[3];
                split3(wr[0][u] * e0, a0[0], a0[1], a0[2]);
                split3(wr[1][u] * e1, a1[0], a1[1], a1[2]);
#pragma unroll
                for (int d = 0; d < 3; ++d) u3[d][u] = cat8(a0[d], a1[d]);
            }
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const char* row = buf + LK + (tr ^ (64 * (t >> 1))) + 8 * (t & 1);
            const bf16x8 kt = cat8(tr_read(row), tr_read(row + ROWS16));
#pragma unroll
            for (int u = 0; u < NU; ++u) {
#pragma unroll
                for (int e = 0; e < 4; ++e) S[t][u][e] = fmaf(S[t][u][e], f, S[t][u][e] * f_low);
#pragma unroll
                for (int d = 0; d < 3; ++d) S[t][u] = mma32(kt, u3[d][u], S[t][u]);
            }
        }
        if (more) {
            // the next chunk's rows have arrived when at most this chunk's stores, issued
            // after them, are outstanding (they complete in order)
            wait_vm<kOut ? 2 : 4 * NU>();
            barrier_lds();
        }
    };
    wait_vm<0>();
    barrier_lds();
    for (int t0 = 0, at = 0; t0 < it.len; t0 += SC, at ^= 1)
        chunk(t0, lds + at * SET, lds_r[at], lds + (at ^ 1) * SET, lds_r[at ^ 1]);

    if (A.s_out != nullptr) {
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int u = 0; u < NU; ++u) *(f32x4*)(A.s_out + soff + (vrow + 4 * u) * D + krow(t)) = S[t][u];
    }
}

template <int NU, int kParts>
static void launch_scan(const DeltaArgs& a, DeltaMode mode, hipStream_t s) {
    const dim3 grid((unsigned)(a.map.items * kParts)), block(512 / NU / kParts);
    if (mode == kDeltaOut)
        hipLaunchKernelGGL((delta_scan_kernel<NU, kParts, kDeltaOut>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((delta_scan_kernel<NU, kParts, kDeltaRecord>), grid, block, 0, s, a);
}

hipError_t launch_delta_scan(const DeltaArgs& a, DeltaMode mode, hipStream_t s) {
    if (a.map.items <= 128)
        launch_scan<1, 2>(a, mode, s);
    else if (a.map.items <= 256)
        launch_scan<1, 1>(a, mode, s);
    else
        launch_scan<2, 1>(a, mode, s);
    return hipGetLastError();
}

// Token-serial form on the FP32 state pool (decode, drafted tokens, and sequences of a few
// tokens).  A workgroup takes 32 of the 128 state rows of one (sequence, value head): a half
// wave holds a row (4 channels a lane), each wave 4 pairs of rows, so that every load and
// store moves 1 KiB of contiguous state and S k and S q are sums over the half wave.  Both
// are taken from the decayed state, o = s (S q + u k.q), so that their sums run side by side.
// No LDS, no barrier; everything FP32, the decay as the sum of two values.
// Bound by the states' way in and out; non-temporal (kStream) when that exceeds kStreamBytes.
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
