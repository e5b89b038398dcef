// Gated delta rule, training backward: the adjoint's scan and the gradients of blocks of 64
// tokens.  (The formulas stand in kda_delta.hip.)
#include "kda_delta.hpp"

namespace kda {

// The scan of kda_delta.hip backward in time, Z = dS in place of S and chunks in descending
// order:
//     dU = P^T do + e^{G_n - G} K Z,   Y = dU - C^T B dU,
//     Z <- e^{G_n} Z + Q^T (s e^G do) - K^T (e^G B Y).
// Same distribution and the same exactness: every product that Z or Y takes up is one of three pieces by
// one or by three.  It leaves Z behind every block of 64 tokens and all rows Y for the gradients' kernel.
template <int NU, int kParts>
__global__ __launch_bounds__(512 / NU / kParts, 2) void delta_adjoint_kernel(DeltaArgs A) {
    constexpr int NW = 8 / NU / kParts;
    constexpr int SETS = 3, SET = SC * D * 2, LK = 0, LO = 2 * SET, LQ = 4 * SET, LPT = 3 * 512;
    constexpr int ROWS16 = 16 * D * 2;
    __shared__ __align__(16) char lds[2 * SETS * SET];
    __shared__ __align__(16) float lds_r[2][REC];
    __shared__ __align__(16) char lds_p[3 * LPT];

    const int tid = threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63, gq = lane >> 4, n16 = lane & 15;
    int idx = xcd_order(blockIdx.x, (int)gridDim.x, A.G * kParts);
    const int part = idx % kParts;
    idx /= kParts;
    const int wv = w + NW * part;
    const Item it = find_item(A.map, idx);
    const int Hv = A.map.Hv;
    const int64_t soff = ((int64_t)it.n * Hv + it.h) * (int64_t)STATE;
    const int64_t block0 = (A.blocks.task != nullptr ? A.blocks.tape_off[it.n] + it.n
                                                     : (int64_t)it.n * ((A.blocks.len + DB - 1) / DB)) + it.off / DB;
    const int chunks = (it.len + SC - 1) / SC;

    const int lrow = 4 * w + gq;
    constexpr int STEP = 4 * NW;
    static_assert(STEP % 16 == 0 && NW >= 4, "rows of one lane share their place in a row's order; four waves move a record");
    const bf16* src[3] = {(const bf16*)A.k, (const bf16*)A.d_o, (const bf16*)A.q};
    const int64_t stride[3] = {A.sk, (int64_t)Hv * D, A.sq};
    const char* pr[SETS];
    unsigned off[SETS];
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
        pr[i] = (const char*)(src[i] + (it.tok0 + (int64_t)(chunks - 1) * SC) * stride[i] + (i == 1 ? it.h : it.h / A.G) * D);
        off[i] = (unsigned)lrow * (unsigned)(stride[i] * 2) + ((n16 ^ swz(lrow)) << 4);
    }
    const char* prec = (const char*)(A.rec + (block0 * Hv + it.h) * (2 * REC));
    const float* pfac = A.fac + (block0 * Hv + it.h) * 4;
    auto fetch = [&](char* rows_to, float* rec_to, int c) __attribute__((always_inline)) {
        const int rem = it.len - c * SC;
#pragma unroll
        for (int j = 0; j < SC / STEP; ++j) {
            if (rem >= SC || lrow + STEP * j < rem) {
#pragma unroll
                for (int i = 0; i < SETS; ++i)
                    to_lds<false>(pr[i] + j * STEP * 2 * stride[i], off[i], rows_to + 2 * i * SET + (STEP * j + 4 * w) * D * 2);
            } else {
#pragma unroll
                for (int i = 0; i < SETS; ++i)
                    *(u32x4*)(rows_to + 2 * i * SET + (STEP * j + 4 * w) * D * 2 + lane * 16) = u32x4{0u, 0u, 0u, 0u};
            }
        }
        if (w < 4) {
            const char* p = prec + ((int64_t)(c >> 1) * Hv * 2 + (c & 1)) * (REC * 4) + w * 1024;
            to_lds<false>(p, lane * 16, (char*)rec_to + w * 1024);
        }
#pragma unroll
        for (int i = 0; i < SETS; ++i) pr[i] -= SC * 2 * stride[i];
    };
    fetch(lds, lds_r[0], chunks - 1);

    f32x4 Z[8][NU];
    const int vrow = NU == 2 ? 32 * wv + 8 * (n16 >> 2) + (n16 & 3) : 16 * wv + n16;   // + 4u
    auto krow = [&](int t) __attribute__((always_inline)) { return 32 * (t >> 1) + 8 * gq + 4 * (t & 1); };
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int u = 0; u < NU; ++u)
            Z[t][u] = A.s_in != nullptr ? *(const f32x4*)(A.s_in + soff + (vrow + 4 * u) * D + krow(t)) : zero4();

    const int r8 = (n16 * D + ((gq ^ swz(n16)) << 3)) * 2;
    const int trow = 4 * gq + (n16 >> 2), piece = n16 & 3;
    const int tr = (trow * D + ((piece ^ swz(trow)) << 3)) * 2;
    const int trv = NU == 2 ? (trow * D + (((4 * wv + piece) ^ swz(trow)) << 3)) * 2
                            : (trow * D + (((2 * wv + (piece >> 1)) ^ swz(trow)) << 3) + 4 * (piece & 1)) * 2;

    auto chunk = [&](int c, const char* __restrict__ buf, const float* __restrict__ rec, char* __restrict__ rows_to,
                     float* __restrict__ rec_to) __attribute__((always_inline)) {
        const bool more = c > 0;
        if (more) fetch(rows_to, rec_to, c - 1);
        const int64_t blk = (block0 + (c >> 1)) * Hv + it.h;
        const float* fac = pfac + (int64_t)(c >> 1) * Hv * 4 + (c & 1) * 2;
        const float f = fac[0], f_low = fac[1];
        // P tiles as their transposes' operands: lane (gq, n) rows i = 4gq + e of column j = n,
        // (i, j) = (0, 0), (1, 1), (1, 0)
#pragma unroll
        for (int tile = 0; tile < 3; ++tile) {
            if (w != tile) continue;
            const int bi = tile == 0 ? 0 : 1, bj = tile == 1 ? 1 : 0;
            f32x4 acc = zero4();
#pragma unroll
            for (int p = 0; p < 4; ++p)
                acc = mma32(*(const bf16x8*)(buf + LQ + ((r8 + bi * ROWS16) ^ (64 * p))),
                            *(const bf16x8*)(buf + LK + ((r8 + bj * ROWS16) ^ (64 * p))), acc);
            const int i = 16 * bi + 4 * gq, j = 16 * bj + n16;
            const float rj = rec[REC_RK + j], hj = rec[REC_GH + j], lj = rec[REC_GL + j];
            const f32x4 ai = *(const f32x4*)(rec + REC_A + i), hi = *(const f32x4*)(rec + REC_GH + i),
                        li = *(const f32x4*)(rec + REC_GL + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = acc[e] * (ai[e] * rj) * decay2(hi[e], li[e], hj, lj);
                acc[e] = i + e >= j ? x : 0.0f;
            }
            bf16x4 a, b, d;
            split3(acc, a, b, d);
            char* to = lds_p + tile * LPT + lane * 8;
            *(bf16x4*)to = a;
            *(bf16x4*)(to + 512) = b;
            *(bf16x4*)(to + 1024) = d;
        }
        f32x4 x[2][NU];
#pragma unroll
        for (int ti = 0; ti < 2; ++ti)
#pragma unroll
            for (int u = 0; u < NU; ++u) x[ti][u] = zero4();
        const bool keep = (c & 1) != 0 || c == chunks - 1;   // behind a block
        char* planes = (char*)(A.state_planes + blk * (int64_t)(2 * STATE));
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            bf16x8 ak[2];
#pragma unroll
            for (int ti = 0; ti < 2; ++ti) ak[ti] = *(const bf16x8*)(buf + LK + ((r8 + ti * ROWS16) ^ (64 * p)));
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                bf16x4 pc[3][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) split3(Z[2 * p + i][u], pc[0][i], pc[1][i], pc[2][i]);
#pragma unroll
                for (int d = 0; d < 3; ++d) {
                    const bf16x8 z = cat8(pc[d][0], pc[d][1]);
#pragma unroll
                    for (int ti = 0; ti < 2; ++ti) x[ti][u] = mma32(ak[ti], z, x[ti][u]);
                    if (d < 2 && keep)
                        *(bf16x8*)(planes + d * (STATE * 2) + ((vrow + 4 * u) * D + krow(2 * p)) * 2) = z;
                }
            }
        }
        bf16x4 dof[2][NU];
#pragma unroll
        for (int ti = 0; ti < 2; ++ti)
#pragma unroll
            for (int u = 0; u < NU; ++u) dof[ti][u] = tr_read(buf + LO + trv + 8 * u + ROWS16 * ti);
        barrier_lds();
        // dU, then Y
        bf16x4 pt[3][3];   // tile, piece
#pragma unroll
        for (int tile = 0; tile < 3; ++tile)
#pragma unroll
            for (int d = 0; d < 3; ++d) pt[tile][d] = *(const bf16x4*)(lds_p + tile * LPT + d * 512 + lane * 8);
        const bf16x4 none = __builtin_bit_cast(bf16x4, u32x2{0u, 0u});
        const f32x4 e0 = *(const f32x4*)(rec + REC_CE + 4 * gq), e1 = *(const f32x4*)(rec + REC_CE + 16 + 4 * gq);
        const f32x4 b0 = *(const f32x4*)(rec + REC_BETA + 4 * gq), b1 = *(const f32x4*)(rec + REC_BETA + 16 + 4 * gq);
        bf16x4 c11[3], c22[3], c21[3];   // of -C^T: lane (gq, j) rows i = 4gq + e of column j
        {
            f32x4 m11, m22, m21;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at = (4 * gq + e) * 16 + n16;
                m11[e] = -rec[REC_C11 + at];
                m22[e] = -rec[REC_C22 + at];
                m21[e] = -rec[REC_C21 + at];
            }
            split3(m11, c11[0], c11[1], c11[2]);
            split3(m22, c22[0], c22[1], c22[2]);
            split3(m21, c21[0], c21[1], c21[2]);
        }
        bf16x8 y3[3][NU], o3[3][NU];   // what the state takes up, in pieces
        char* rp = (char*)(A.row_planes + (blk * 2 + (c & 1)) * (int64_t)(2 * D * SC));
        const f32x4 x0_ = *(const f32x4*)(rec + REC_CX + 4 * gq), x1_ = *(const f32x4*)(rec + REC_CX + 16 + 4 * gq);
        const f32x4 o0_ = *(const f32x4*)(rec + REC_CO + 4 * gq), o1_ = *(const f32x4*)(rec + REC_CO + 16 + 4 * gq);
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            f32x4 y0 = x[0][u] * e0, y1 = x[1][u] * e1;
            const bf16x4 d0 = dof[0][u], d1 = dof[1][u];
#pragma unroll
            for (int d = 0; d < 3; ++d) y0 = mma32(cat8(pt[0][d], pt[2][d]), cat8(d0, d1), y0);
            y1 = mma32(cat8(pt[1][0], pt[1][1]), cat8(d1, d1), y1);
            y1 = mma32(cat8(pt[1][2], none), cat8(d1, none), y1);
            bf16x4 q0[3], q1[3];
            split3(y0 * b0, q0[0], q0[1], q0[2]);
            split3(y1 * b1, q1[0], q1[1], q1[2]);
            y1 = mma32(cat8(c22[0], c22[0]), cat8(q1[0], q1[1]), y1);
            y1 = mma32(cat8(c22[1], c22[1]), cat8(q1[0], q1[1]), y1);
            y1 = mma32(cat8(c22[0], c22[2]), cat8(q1[2], q1[0]), y1);
#pragma unroll
            for (int a = 0; a < 3; ++a)
#pragma unroll
                for (int b = 0; a + b < 3; ++b) y0 = mma32(cat8(c11[a], c21[a]), cat8(q0[b], q1[b]), y0);
#pragma unroll
            for (int ti = 0; ti < 2; ++ti) {   // the rows Y, as planes [v][token]
                bf16x4 hi, lo;
                split4_rne(ti == 0 ? y0 : y1, hi, lo);
                char* d = rp + ((vrow + 4 * u) * SC + 16 * ti + 4 * gq) * 2;
                *(bf16x4*)d = hi;
                *(bf16x4*)(d + D * SC * 2) = lo;
            }
            bf16x4 a0[3], a1[3];
            split3(-(y0 * b0) * x0_, a0[0], a0[1], a0[2]);
            split3(-(y1 * b1) * x1_, a1[0], a1[1], a1[2]);
#pragma unroll
            for (int d = 0; d < 3; ++d) y3[d][u] = cat8(a0[d], a1[d]);
            split3(from_bf4(d0) * o0_, a0[0], a0[1], a0[2]);
            split3(from_bf4(d1) * o1_, a1[0], a1[1], a1[2]);
#pragma unroll
            for (int d = 0; d < 3; ++d) o3[d][u] = cat8(a0[d], a1[d]);
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const int at = (tr ^ (64 * (t >> 1))) + 8 * (t & 1);
            const bf16x8 kt = cat8(tr_read(buf + LK + at), tr_read(buf + LK + at + ROWS16));
            const bf16x8 qt = cat8(tr_read(buf + LQ + at), tr_read(buf + LQ + at + ROWS16));
#pragma unroll
            for (int u = 0; u < NU; ++u) {
#pragma unroll
                for (int e = 0; e < 4; ++e) Z[t][u][e] = fmaf(Z[t][u][e], f, Z[t][u][e] * f_low);
#pragma unroll
                for (int d = 0; d < 3; ++d) Z[t][u] = mma32(kt, y3[d][u], Z[t][u]);
#pragma unroll
                for (int d = 0; d < 3; ++d) Z[t][u] = mma32(qt, o3[d][u], Z[t][u]);
            }
        }
        if (more) {
            wait_vm<4 * NU>();
            barrier_lds();
        }
    };
    wait_vm<0>();
    barrier_lds();
    for (int c = chunks - 1, at = 0; c >= 0; --c, at ^= 1)
        chunk(c, lds + at * SET, lds_r[at], lds + (at ^ 1) * SET, lds_r[at ^ 1]);

    if (A.s_out != nullptr) {
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int u = 0; u < NU; ++u) *(f32x4*)(A.s_out + soff + (vrow + 4 * u) * D + krow(t)) = Z[t][u];
    }
}

hipError_t launch_delta_adjoint(const DeltaArgs& a, hipStream_t s) {
    if (a.map.items <= 128)
        hipLaunchKernelGGL((delta_adjoint_kernel<1, 2>), dim3((unsigned)(a.map.items * 2)), dim3(256), 0, s, a);
    else if (a.map.items <= 256)
        hipLaunchKernelGGL((delta_adjoint_kernel<1, 1>), dim3((unsigned)a.map.items), dim3(512), 0, s, a);
    else
        hipLaunchKernelGGL((delta_adjoint_kernel<2, 1>), dim3((unsigned)a.map.items), dim3(256), 0, s, a);
    return hipGetLastError();
}

// Sum over the lanes before this one in its row of 16.
__device__ __forceinline__ float row16_before(float x) {
#define KDA_SHIFTED(n) __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x110 + (n), 0xF, 0xF, true))
    x = KDA_SHIFTED(1);   // (row_shr: zero where there is no lane)
    x += KDA_SHIFTED(1);
    x += KDA_SHIFTED(2);
    x += KDA_SHIFTED(4);
    x += KDA_SHIFTED(8);
#undef KDA_SHIFTED
    return x;
}

// Gradients of a block of 64 tokens of one value head, all blocks at once.  With S the
// state before the block, Z the adjoint behind it, G the running sums from the block's
// start, and q, k at unit length:
//     E = do W^T,   F = Y W^T,   e_ij = s e^{Gi-Gj} beta_j E_ij (i >= j),
//     f_ij = e^{Gi-Gj} beta_i beta_j F_ij (i > j),
//     dq_i = s e^{Gi} S^T do_i + sum_j e_ij k_j,
//     dk_j = -e^{Gj} beta_j S^T Y_j + e^{Gn-Gj} beta_j Z^T W_j + sum_i e_ij q_i - sum_i (f_ij + f_ji) k_i,
//     dbeta_j = F_jj,   dv_j = beta_j Y_j,
// and a decay acts on everything that passes its token:
//     dg_t = e^{Gn} <Z, S> + sum_{j<t} k_j.(e^{Gn-Gj} beta_j Z^T W_j)
//          + sum_{i>=t} (q_i.(s e^{Gi} S^T do_i) - k_i.(e^{Gi} beta_i S^T Y_i))
//          + sum_{i>=t>j} (e_ij q_i.k_j - f_ij k_i.k_j),
// whose terms all hold the decay of token t, so that none has to cancel behind a strong one.
// Four waves; each forms its 32 channels of dq and dk (as D^T: lane (gq, n) holds channels
// 32w + 8gq + 4u + e of token n) and up to three of the ten lower tiles of E and F.  What the scans left
// comes as pairs of BF16 planes, 32 channels v of the sums at a time; products of two pairs take
// three of the four.
constexpr int GS_O = 0, GS_R = 4096, GS_S = GS_R + 16384, GS = GS_S + 32768;   // stage: do, rows, states
constexpr int GM = 32768, GN = GM + 16384, GTOTAL = GN + 16384;                // q, k rows; e; f
__global__ __launch_bounds__(256, 2) void delta_grad_kernel(DeltaGradArgs A) {
    __shared__ __align__(16) char lds[GTOTAL];
    __shared__ float tok[5][DB];            // beta, G as two floats, one over k's and q's length
    __shared__ float dots[5][4][DB];        // per wave: q.(state part of dq), k.(its two parts of dk), then q.dq and k.dk
    __shared__ float sums[2][4][DB];        // of the tiles e q.k - f k.k: of a row, by column tile; of the rows i >= t before column t, by row tile
    __shared__ float diag[DB], whole[4];
    constexpr int TILES = 10;
    static_assert(GTOTAL >= GS, "the products' areas lie over the stage");

    const int tid = threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63, gq = lane >> 4, n16 = lane & 15;
    const Item it = find_item(A.blocks, blockIdx.x);
    const int Hv = A.blocks.Hv;
    const int64_t blk = it.seg * Hv + it.h;
    const float* rec = A.rec + blk * (2 * REC);

    if (w == 0) {
        const float* r = rec + (lane >> 5) * REC + (lane & 31);
        float hi = r[REC_GH], lo = r[REC_GL];
        if (lane >= 32) {   // behind the first chunk's decay: the exact sum of the high parts and the rest
            const float h0 = rec[REC_GH + 31], l0 = rec[REC_GL + 31];
            const float s = h0 + hi, b = s - h0;
            lo = ((h0 - (s - b)) + (hi - b)) + (l0 + lo);
            hi = s;
        }
        tok[0][lane] = r[REC_BETA];
        tok[1][lane] = hi;
        tok[2][lane] = lo;
        tok[3][lane] = r[REC_RK];
        tok[4][lane] = r[REC_A] / A.scale;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) sums[i][w][lane] = 0.0f;

    // tiles (i, j) of E and F: t = w, w + 4, w + 8 of (3,0) (2,0) (1,0) (3,1) (3,2) (2,1) (0,0) (1,1) (2,2) (3,3)
    auto tile_i = [](int t) { return (int)(0x3210233123ull >> (4 * t)) & 15; };
    auto tile_j = [](int t) { return (int)(0x3210121000ull >> (4 * t)) & 15; };

    f32x4 dq[4][2], dks[4][2], dke[4][2], E[3], F[3];
#pragma unroll
    for (int ti = 0; ti < 4; ++ti)
#pragma unroll
        for (int u = 0; u < 2; ++u) dq[ti][u] = dks[ti][u] = dke[ti][u] = zero4();
#pragma unroll
    for (int s = 0; s < 3; ++s) E[s] = F[s] = zero4();
    float zs = 0.0f;

    // Loads: 16 rows of 64 bytes or 4 of 256 an instruction, a lane fetching the 16 bytes that
    // belong in its place.  Rows of 64 bytes: block b of do's row r at b ^ (r/4)%4, of a plane's row
    // at b ^ 2 (r/8)%2; of 256 bytes as in the scans.
    const u32x4 zero = {0u, 0u, 0u, 0u};
    const int r16 = lane >> 2, b4 = lane & 3;
    const int64_t so = (int64_t)Hv * D;
    const bf16* pdo = (const bf16*)A.d_o + ((it.tok0 + 16 * w) * Hv + it.h) * D;
    const unsigned off_o = (unsigned)r16 * (unsigned)(so * 2) + ((b4 ^ ((r16 >> 2) & 3)) << 4);
    // rows W (waves 0, 1) and Y of chunk w % 2; plane w % 2 of S (waves 0, 1) and Z
    const char* prows = (const char*)(w < 2 ? A.w_planes : A.y_planes) + (blk * 2 + (w & 1)) * (int64_t)(2 * D * SC * 2);
    const char* pstate = (const char*)(w < 2 ? A.s_planes : A.z_planes) + (blk * 2 + (w & 1)) * (int64_t)(STATE * 2);
    auto load_stage = [&](int vb) __attribute__((always_inline)) {
        char* o = lds + GS_O + w * 1024;
        if (16 * w + r16 < it.len)
            to_lds<false>((const char*)(pdo + 32 * vb), off_o, o);
        else
            *(u32x4*)(o + lane * 16) = zero;
#pragma unroll
        for (int piece = 0; piece < 2; ++piece)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                char* d = lds + GS_R + (((w >> 1) * 2 + piece) * 2 + (w & 1)) * 2048 + half * 1024;
                if ((w & 1) * SC < it.len)   // (a block may end in its first chunk)
                    to_lds<false>(prows + (piece * D + 32 * vb + 16 * half) * 64, r16 * 64 + ((b4 ^ (((r16 >> 3) & 1) << 1)) << 4), d);
                else
                    *(u32x4*)(d + lane * 16) = zero;
            }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            to_lds<false>(pstate + (32 * vb + 4 * j) * 256, gq * 256 + ((n16 ^ swz(4 * j + gq)) << 4), lds + GS_S + w * 8192 + j * 1024);
    };
    // operands: do, rows (0: W, 1: Y) and states (0: S, 1: Z) of 8 channels v = 32vb + 8gq ..
    auto get_o = [&](int ti) __attribute__((always_inline)) {
        return *(const bf16x8*)(lds + GS_O + (16 * ti + n16) * 64 + ((gq ^ (n16 >> 2)) << 4));
    };
    const int prow = 8 * gq + (n16 >> 2), pa = n16 & 3;   // this lane's row of a transposing read, and its piece there
    auto get_row = [&](int set, int piece, int ti) __attribute__((always_inline)) {
        const char* r = lds + GS_R + ((set * 2 + piece) * 2 + (ti >> 1)) * 2048 + prow * 64 + (((ti ^ gq) & 1) << 5) + 8 * pa;
        return cat8(tr_read(r), tr_read(r + 4 * 64));
    };
    auto get_state = [&](int plane, int u) __attribute__((always_inline)) {
        const char* r = lds + GS_S + plane * 8192 + 8 * u;
        return cat8(tr_read(r + prow * 256 + (((4 * w + pa) ^ swz(prow)) << 4)),
                    tr_read(r + (prow + 4) * 256 + (((4 * w + pa) ^ swz(prow + 4)) << 4)));
    };
    for (int vb = 0; vb < 4; ++vb) {
        if (vb != 0) barrier_lds();
        load_stage(vb);
        wait_vm<0>();
        barrier_lds();
        bf16x8 st[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) st[i][u] = get_state(i, u);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                zs = fmaf((float)st[0][u][e] + (float)st[1][u][e], (float)st[2][u][e] + (float)st[3][u][e], zs);
#pragma unroll
        for (int ti = 0; ti < 4; ++ti) {
            const bf16x8 o = get_o(ti), wh = get_row(0, 0, ti), wl = get_row(0, 1, ti), yh = get_row(1, 0, ti),
                         yl = get_row(1, 1, ti);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                dq[ti][u] = mma32(st[0][u], o, dq[ti][u]);
                dq[ti][u] = mma32(st[1][u], o, dq[ti][u]);
                dks[ti][u] = mma32(st[0][u], yh, dks[ti][u]);
                dks[ti][u] = mma32(st[0][u], yl, dks[ti][u]);
                dks[ti][u] = mma32(st[1][u], yh, dks[ti][u]);
                dke[ti][u] = mma32(st[2][u], wh, dke[ti][u]);
                dke[ti][u] = mma32(st[2][u], wl, dke[ti][u]);
                dke[ti][u] = mma32(st[3][u], wh, dke[ti][u]);
            }
            if (ti == w && 16 * ti + n16 < it.len) {   // dv: 8 channels of a token
                const float b = tok[0][16 * ti + n16];
                f32x4 y0, y1;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y0[e] = b * ((float)yh[e] + (float)yl[e]);
                    y1[e] = b * ((float)yh[4 + e] + (float)yl[4 + e]);
                }
                *(bf16x8*)((bf16*)A.dv + ((it.tok0 + 16 * ti + n16) * Hv + it.h) * D + 32 * vb + 8 * gq) = cat8(to_bf4(y0), to_bf4(y1));
            }
        }
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            if (w + 4 * s >= TILES) continue;
            const int bi = tile_i(w + 4 * s), bj = tile_j(w + 4 * s);
            const bf16x8 o = get_o(bi), yh = get_row(1, 0, bi), yl = get_row(1, 1, bi), wh = get_row(0, 0, bj),
                         wl = get_row(0, 1, bj);
            E[s] = mma32(o, wh, E[s]);
            E[s] = mma32(o, wl, E[s]);
            F[s] = mma32(yh, wh, F[s]);
            F[s] = mma32(yh, wl, F[s]);
            F[s] = mma32(yl, wh, F[s]);
        }
    }
    zs = group_sum<64>(zs);
    if (lane == 0) whole[w] = zs;
    barrier_lds();   // the stage is read; q's and k's rows go over it
    {
        const bf16* src[2] = {(const bf16*)A.q, (const bf16*)A.k};
        const int64_t stride[2] = {A.sq, A.sk};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 16 * w + 4 * j;
                char* d = lds + i * 16384 + r * 256;
                if (r + gq < it.len)
                    to_lds<false>((const char*)(src[i] + (it.tok0 + r) * stride[i] + (it.h / A.G) * D),
                                  (unsigned)gq * (unsigned)(stride[i] * 2) + ((n16 ^ swz(4 * j + gq)) << 4), d);
                else
                    *(u32x4*)(d + lane * 16) = zero;
            }
    }
    wait_vm<0>();
    barrier_lds();
    constexpr int LQ = 0, LK = 16384;
    const int r8 = n16 * 256 + ((gq ^ swz(n16)) << 4);   // 8 channels 32p + 8gq of row n (xor 64p)
    // matrices of 64 rows of 128 bytes: block b of row r at b ^ r % 8; hi at 0, lo at 8192
    auto mat = [&](int base, int row, int block) __attribute__((always_inline)) {
        return lds + base + row * 128 + ((block ^ (row & 7)) << 4);
    };
#pragma unroll
    for (int s = 0; s < 3; ++s) {
        if (w + 4 * s >= TILES) continue;
        const int bi = tile_i(w + 4 * s), bj = tile_j(w + 4 * s);
        f32x4 qk = zero4(), kk = zero4();
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const bf16x8 kj = *(const bf16x8*)(lds + LK + bj * 4096 + (r8 ^ (64 * p)));
            qk = mma32(*(const bf16x8*)(lds + LQ + bi * 4096 + (r8 ^ (64 * p))), kj, qk);
            kk = mma32(*(const bf16x8*)(lds + LK + bi * 4096 + (r8 ^ (64 * p))), kj, kk);
        }
        const int i0 = 16 * bi + 4 * gq, j = 16 * bj + n16;
        const float bj_ = tok[0][j], hj = tok[1][j], lj = tok[2][j], rj = tok[3][j];
        f32x4 m, n, h;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + e;
            const float d = decay2(tok[1][i], tok[2][i], hj, lj) * bj_ * rj;
            const float x = d * (A.scale * tok[4][i]) * E[s][e], y = d * (tok[0][i] * tok[3][i]) * F[s][e];
            m[e] = i >= j ? x : 0.0f;
            n[e] = i > j ? -y : 0.0f;
            h[e] = i > j ? m[e] * qk[e] + n[e] * kk[e] : 0.0f;
            if (i == j) diag[j] = F[s][e];
        }
        // along a row to its columns before t; the rows from t on of that, down column t
        f32x4 along;
        float down = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            along[e] = row16_sum(h[e]);
            const float x = row16_before(h[e]);
            down += bi != bj || 4 * gq + e >= n16 ? x : 0.0f;
        }
        down += __shfl_xor(down, 16, 64);
        down += __shfl_xor(down, 32, 64);
        if (n16 == 0) *(f32x4*)&sums[0][bj][i0] = along;
        if (gq == 0) sums[1][bi][j] = down;
        bf16x4 mh, ml, nh, nl;
        split4_rne(m, mh, ml);
        split4_rne(n, nh, nl);
        {   // e as [j][i], zeros above the diagonal
            char* at = mat(GM, j, 2 * bi + (gq >> 1)) + 8 * (gq & 1);
            *(bf16x4*)at = mh;
            *(bf16x4*)(at + 8192) = ml;
            if (bi != bj) {
                at = mat(GM, 16 * bi + n16, 2 * bj + (gq >> 1)) + 8 * (gq & 1);
                *(u32x2*)at = u32x2{0u, 0u};
                *(u32x2*)(at + 8192) = u32x2{0u, 0u};
            }
        }
        // -f, both ways
        if (bi != bj) {
            char* at = mat(GN, j, 2 * bi + (gq >> 1)) + 8 * (gq & 1);
            *(bf16x4*)at = nh;
            *(bf16x4*)(at + 8192) = nl;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + e;
            char* at = mat(GN, i, j >> 3) + 2 * (j & 7);
            if (i >= j) {
                *(bf16*)at = nh[e];
                *(bf16*)(at + 8192) = nl[e];
            }
            if (bi == bj && i > j) {
                at = mat(GN, j, i >> 3) + 2 * (i & 7);
                *(bf16*)at = nh[e];
                *(bf16*)(at + 8192) = nl[e];
            }
        }
    }
    // the parts that come from the states, and what they say of the decays
    const float hn = tok[1][DB - 1], ln = tok[2][DB - 1];
    const int rch = ((4 * w + gq) ^ swz(n16)) << 4;   // channels 32w + 8gq .. of row n
    auto dot8 = [&](bf16x8 x, const f32x4* y) __attribute__((always_inline)) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) s += (float)x[e] * y[0][e] + (float)x[4 + e] * y[1][e];
        s += __shfl_xor(s, 16, 64);
        return s + __shfl_xor(s, 32, 64);
    };
#pragma unroll
    for (int ti = 0; ti < 4; ++ti) {
        const int t = 16 * ti + n16;
        const float b = tok[0][t], hi = tok[1][t], lo = tok[2][t], rk = tok[3][t], rq = tok[4][t];
        const float from = decay2(hi, lo, 0.0f, 0.0f), to = decay2(hn, ln, hi, lo);
        const float cq = A.scale * from * rq, cs = -from * b * rk, ce = to * b * rk;
        const bf16x8 q8 = *(const bf16x8*)(lds + LQ + ti * 4096 + n16 * 256 + rch);
        const bf16x8 k8 = *(const bf16x8*)(lds + LK + ti * 4096 + n16 * 256 + rch);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            dq[ti][u] *= cq;
            dks[ti][u] *= cs;
            dke[ti][u] *= ce;
        }
        const float s0 = dot8(q8, dq[ti]), s1 = dot8(k8, dks[ti]), s2 = dot8(k8, dke[ti]);
        if (gq == 0) {
            dots[0][w][t] = s0;
            dots[1][w][t] = s1;
            dots[2][w][t] = s2;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) dks[ti][u] += dke[ti][u];
    }
    barrier_lds();
    // the products inside the block
#pragma unroll
    for (int pair = 0; pair < 2; ++pair) {
        const int r0 = 32 * pair + prow, r1 = r0 + 4;
        bf16x8 kt[2], qt[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int a0 = r0 * 256 + (((4 * w + pa) ^ swz(r0 & 15)) << 4) + 8 * u, a1 = r1 * 256 + (((4 * w + pa) ^ swz(r1 & 15)) << 4) + 8 * u;
            kt[u] = cat8(tr_read(lds + LK + a0), tr_read(lds + LK + a1));
            qt[u] = cat8(tr_read(lds + LQ + a0), tr_read(lds + LQ + a1));
        }
#pragma unroll
        for (int ti = 0; ti < 4; ++ti) {
#pragma unroll
            for (int piece = 0; piece < 2; ++piece) {
                if (2 * pair <= ti) {   // sum over j <= i of e_ij k_j
                    const bf16x8 m = cat8(tr_read(mat(GM, r0, 2 * ti + (pa >> 1)) + 8 * (pa & 1) + piece * 8192),
                                          tr_read(mat(GM, r1, 2 * ti + (pa >> 1)) + 8 * (pa & 1) + piece * 8192));
#pragma unroll
                    for (int u = 0; u < 2; ++u) dq[ti][u] = mma32(kt[u], m, dq[ti][u]);
                }
                if (2 * pair + 1 >= ti) {   // sum over i >= j of e_ij q_i
                    const bf16x8 m = *(const bf16x8*)(mat(GM, 16 * ti + n16, 4 * pair + gq) + piece * 8192);
#pragma unroll
                    for (int u = 0; u < 2; ++u) dks[ti][u] = mma32(qt[u], m, dks[ti][u]);
                }
                const bf16x8 n = *(const bf16x8*)(mat(GN, 16 * ti + n16, 4 * pair + gq) + piece * 8192);
#pragma unroll
                for (int u = 0; u < 2; ++u) dks[ti][u] = mma32(kt[u], n, dks[ti][u]);
            }
        }
    }
    // unit length: d - x^ (x^.d), and the rows
    bf16x8 q8[4], k8[4];
#pragma unroll
    for (int ti = 0; ti < 4; ++ti) {
        const int t = 16 * ti + n16;
        q8[ti] = *(const bf16x8*)(lds + LQ + ti * 4096 + n16 * 256 + rch);
        k8[ti] = *(const bf16x8*)(lds + LK + ti * 4096 + n16 * 256 + rch);
        const float s0 = dot8(q8[ti], dq[ti]), s1 = dot8(k8[ti], dks[ti]);
        if (gq == 0) {
            dots[3][w][t] = s0;
            dots[4][w][t] = s1;
        }
    }
    barrier_lds();
#pragma unroll
    for (int ti = 0; ti < 4; ++ti) {
        const int t = 16 * ti + n16;
        if (t >= it.len) continue;
        if (A.unit) {
            const float rk = tok[3][t], rq = tok[4][t];
            const float sq = ((dots[3][0][t] + dots[3][1][t]) + (dots[3][2][t] + dots[3][3][t])) * rq * rq;
            const float sk = ((dots[4][0][t] + dots[4][1][t]) + (dots[4][2][t] + dots[4][3][t])) * rk * rk;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dq[ti][u][e] -= sq * (float)q8[ti][4 * u + e];
                    dks[ti][u][e] -= sk * (float)k8[ti][4 * u + e];
                }
        }
        const int64_t at = (((it.tok0 + t) * Hv + it.h) * D + 32 * w + 8 * gq) * 2;
        u32x2 x[4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            x[u] = A.pack ? pack_quad(dq[ti][u]) : __builtin_bit_cast(u32x2, to_bf4(dq[ti][u]));
            x[2 + u] = A.pack ? pack_quad(dks[ti][u]) : __builtin_bit_cast(u32x2, to_bf4(dks[ti][u]));
        }
        *(u32x4*)((char*)A.dq + at) = u32x4{x[0][0], x[0][1], x[1][0], x[1][1]};
        *(u32x4*)((char*)A.dk + at) = u32x4{x[2][0], x[2][1], x[3][0], x[3][1]};
    }
    if (w == 0) {   // lane t: token t
        const int b = lane >> 4;
        auto four = [&](int i) { return (dots[i][0][lane] + dots[i][1][lane]) + (dots[i][2][lane] + dots[i][3][lane]); };
        float x = __shfl_up(four(2), 1, 64), y = four(0) + four(1);
        if (lane == 0) x = 0.0f;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const float a = __shfl_up(x, d, 64), c = __shfl_down(y, d, 64);
            if (lane >= d) x += a;
            if (lane + d < 64) y += c;
        }
        float dg = decay2(hn, ln, 0.0f, 0.0f) * ((whole[0] + whole[1]) + (whole[2] + whole[3])) + x + y;
        // sum over i >= t > j: of column tile b, and of the column tiles before it
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i >= b) dg += sums[1][i][lane];
#pragma unroll
        for (int c = 0; c < 3; ++c) {
            const float r = sums[0][c][lane];
            float from = r;   // this row and the tile's rows behind it
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) {
                const float z = __shfl_down(from, d, 16);
                if ((lane & 15) + d < 16) from += z;
            }
            float below = 0.0f;
#pragma unroll
            for (int i = 1; i < 4; ++i) {
                const float all = __shfl(from, 16 * i, 64);
                if (i > b) below += all;
            }
            if (c < b) dg += from + below;
        }
        if (lane < it.len) {
            const int64_t at = (it.tok0 + lane) * Hv + it.h;
            ((bf16*)A.dg)[at] = (bf16)dg;
            ((bf16*)A.dbeta)[at] = (bf16)diag[lane];
        }
    }
}

hipError_t launch_delta_grad(const DeltaGradArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(delta_grad_kernel, dim3((unsigned)a.blocks.items), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace kda
