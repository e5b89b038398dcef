// Gated delta rule, training backward: the adjoint's scan and the gradients of blocks of 64
// tokens.  (The formulas stand in kda_delta.hip.)
#include "kda_delta_scan.hpp"

namespace kda {

// Both scans in one launch: neither needs the other, and together they fill the card sooner.
constexpr int BOTH_LDS = DeltaAdjointLds::TOTAL > DeltaScanLds<kDeltaRecord>::TOTAL ? DeltaAdjointLds::TOTAL
                                                                                 : DeltaScanLds<kDeltaRecord>::TOTAL;
template <int NU, int kParts>
__global__ __launch_bounds__(512 / NU / kParts, 2) void delta_both_kernel(DeltaArgs forward, DeltaArgs backward) {
    __shared__ __align__(16) char lds[BOTH_LDS];
    // (the longer chunks of the backward first)
    const int half = gridDim.x / 2;
    if ((int)blockIdx.x < half)
        delta_adjoint<NU, kParts, false>(backward, blockIdx.x, half, lds);
    else
        delta_scan<NU, kParts, kDeltaRecord>(forward, blockIdx.x - half, half, lds);
}

// (As the forward's scan: while two workgroups a compute unit hold both scans' halves.  1024 tokens
// of 48, 64, 96, 128 sequences and heads, in us: 97, 99, 121, 131 in halves, 154, 155, 160, 166 in four waves with two
// tiles each; of 160, 192, 256: 222, 231, 277 and 194, 196, 223.)
hipError_t launch_delta_both(const DeltaArgs& f, const DeltaArgs& b, hipStream_t s) {
    const unsigned items = (unsigned)f.map.items;
    if (items <= 128)
        hipLaunchKernelGGL((delta_both_kernel<1, 2>), dim3(items * 4), dim3(256), 0, s, f, b);
    else
        hipLaunchKernelGGL((delta_both_kernel<2, 1>), dim3(items * 2), dim3(256), 0, s, f, b);
    return hipGetLastError();
}

template <int NU, int kParts>
__global__ __launch_bounds__(512 / NU / kParts, 2) void delta_behind_kernel(DeltaArgs A) {
    __shared__ __align__(16) char lds[DeltaAdjointLds::TOTAL];
    delta_adjoint<NU, kParts, true>(A, blockIdx.x, gridDim.x, lds);
}

hipError_t launch_delta_behind(const DeltaArgs& a, hipStream_t s) {
    const unsigned items = (unsigned)a.map.items;
    if (items <= 256)   // (8 heads x 8192 tokens in 128 segments and heads: the backward 206 us against 228)
        hipLaunchKernelGGL((delta_behind_kernel<1, 2>), dim3(items * 2), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((delta_behind_kernel<2, 1>), dim3(items), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? launch_delta_chain(a, true, s) : e;
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

// Sum over this lane and those behind it in its row of 16.
__device__ __forceinline__ float row16_from(float x) {
#define KDA_SHIFTED(n) __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x100 + (n), 0xF, 0xF, true))
    x += KDA_SHIFTED(1);   // (row_shl: zero where there is no lane)
    x += KDA_SHIFTED(2);
    x += KDA_SHIFTED(4);
    x += KDA_SHIFTED(8);
#undef KDA_SHIFTED
    return x;
}

// Sums over the four rows of lanes of four values: value i's in row i.
__device__ __forceinline__ float rows_sum(const float (&x)[4]) {
    // (a swap of 32 gives lower halves in its first result and upper halves in its second, one of 16
    // even and odd rows)
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x[0]), __float_as_uint(x[2]), false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x[1]), __float_as_uint(x[3]), false, false);
    const float y0 = __uint_as_float(a[0]) + __uint_as_float(a[1]), y1 = __uint_as_float(b[0]) + __uint_as_float(b[1]);
    const auto c = __builtin_amdgcn_permlane16_swap(__float_as_uint(y0), __float_as_uint(y1), false, false);
    return __uint_as_float(c[0]) + __uint_as_float(c[1]);
}

// A partial of dq or dk (value heads that share a q/k head each form one) keeps the upper 24 bits of its FP32
// value, rounded to nearest: off by 2^-17 at most, the upper 16 of them in one array and the lower 8
// in another.  (With 15 bits and a scale for four, 2 bytes in place of 3, dq and dk were off by 4% more than
// one rounding of the exact values.)
__device__ __forceinline__ unsigned round24(float x) {
    const unsigned u = __float_as_uint(x);
    return x != x ? 0x7fc00000u : u + 0x7fu + (u >> 8 & 1u);
}
__device__ __forceinline__ void put_partials(const f32x4 (&x)[2], char* high, char* low) {
    unsigned u[8], h[4], l[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = round24(x[i >> 2][i & 3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __builtin_amdgcn_perm(u[2 * i + 1], u[2 * i], 0x07060302u);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        l[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(u[4 * i + 3], u[4 * i + 2], 0x0c0c0501u),
                                     __builtin_amdgcn_perm(u[4 * i + 1], u[4 * i], 0x0c0c0501u), 0x05040100u);
    *(u32x4*)high = u32x4{h[0], h[1], h[2], h[3]};
    *(u32x2*)low = u32x2{l[0], l[1]};
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
// 32w + 8gq + 4u + e of token n) and up to three of the ten lower tiles of E and F.  What the scans
// left comes 32 channels v of the sums at a time: of the states each wave reads its own columns k, straight
// into the registers where they are operands, ahead by one such part; W, Y and do go through LDS.  A state's value
// becomes two BF16 pieces, as W and Y are, and the products of two pairs take three of the four; so do
// the matrices e and f.
// Bound by HBM: two workgroups share a unit, each with 44 KB on its way (20 of rows and do, 24 of
// states): 8 x 1024 tokens, 96 heads 742 us, 3.3 GB, 4.5 TB/s.  (States through LDS like the rows, as two BF16
// pieces each and 16 channels at a time, 26 KB on their way: 962 us.  States and rows in FP16 took 677 us, and
// results were off by 0.8% more than one rounding of the exact ones.)
constexpr int GS_O = 0, GS_R = 4096, GS = GS_R + 16384;                        // stage: do, rows
constexpr int GS2 = 32768;                                                     // the second stage
constexpr int GM = 32768, GN = GM + 16384, GTOTAL = GN + 16384;                // q, k rows; e; f
__global__ __launch_bounds__(256, 2) void delta_grad_kernel(DeltaGradArgs A) {
    constexpr int TILES = 10;
    __shared__ __align__(16) char lds[GTOTAL];
    __shared__ float tok[5][DB];            // beta, G as two floats, one over k's and q's length
    __shared__ float dots[5][4][DB];        // per wave: q.(state part of dq), k.(its two parts of dk), then q.dq and k.dk
    __shared__ float sums[2][4][DB];        // of the tiles e q.k - f k.k: of a row, by column tile; of the rows i >= t before column t, by row tile
    __shared__ float diag[DB], whole[4];
    static_assert(GS <= GS2 && GTOTAL >= GS2 + GS, "the products' areas lie over the two stages");

    const int tid = threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63, gq = lane >> 4, n16 = lane & 15;
    const Item it = find_item(A.blocks, blockIdx.x);
    const int Hv = A.blocks.Hv;
    const int64_t blk = it.seg * Hv + it.h;
    const char* rec = A.rec + blk * (2 * REC);

    auto put_tokens = [&]() __attribute__((always_inline)) {
        const char* r = rec + (lane >> 5) * REC + (lane & 31) * 4;
        float hi = *(const float*)(r + REC_GH), lo = *(const float*)(r + REC_GL);
        if (lane >= 32) {   // behind the first chunk's decay: the exact sum of the high parts and the rest
            const float h0 = *(const float*)(rec + REC_GH + 124), l0 = *(const float*)(rec + REC_GL + 124);
            const float s = h0 + hi, b = s - h0;
            lo = ((h0 - (s - b)) + (hi - b)) + (l0 + lo);
            hi = s;
        }
        tok[0][lane] = *(const float*)(r + REC_BETA);
        tok[1][lane] = hi;
        tok[2][lane] = lo;
        tok[3][lane] = *(const float*)(r + REC_K);
        tok[4][lane] = *(const float*)(r + REC_Q);
    };
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
    f32x4 zs = zero4();   // of S^T Z, the sum of whose diagonals is <Z, S>

    auto finish = [&](float zs, int lane) __attribute__((always_inline)) {
    const int gq = lane >> 4, n16 = lane & 15, prow = 8 * gq + (n16 >> 2), pa = n16 & 3;
    const float fs = A.forward.scale[blk], fz = A.backward.scale[blk];
    if (lane == 0) whole[w] = zs * (fs * fz);
    constexpr int LQ = 0, LK = 16384;
    const int r8 = n16 * 256 + ((gq ^ swz(n16)) << 4);   // 8 channels 32p + 8gq of row n (xor 64p)
    // matrices of 64 rows of 128 bytes: block b of row r at b ^ r % 8; hi at 0, lo at 8192
    const bf16x4 none = __builtin_bit_cast(bf16x4, u32x2{0u, 0u});
    const bf16x8 id8 = cat8(identity_frag(lane), none);
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
        }
        if (bi == bj) {   // F's diagonal
            const float d01 = n16 & 1 ? F[s][1] : F[s][0], d23 = n16 & 1 ? F[s][3] : F[s][2];
            if (gq == n16 >> 2) diag[j] = n16 & 2 ? d23 : d01;
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
        down = rows_sum(down);
        if (n16 == 0) *(f32x4*)&sums[0][bj][i0] = along;
        if (gq == 0) sums[1][bi][j] = down;
        bf16x4 mh, ml, nh, nl;
        split4_rne(m, mh, ml);
        split4_rne(n, nh, nl);
        char* at = mat(GM, j, 2 * bi + (gq >> 1)) + 8 * (gq & 1);   // e as [j][i], zeros where its pair of tiles goes on above the diagonal
        *(bf16x4*)at = mh;
        *(bf16x4*)(at + 8192) = ml;
        if ((bi & 1) != 0 && bj == bi - 1) {
            at = mat(GM, 16 * bi + n16, 2 * bj + (gq >> 1)) + 8 * (gq & 1);
            *(u32x2*)at = u32x2{0u, 0u};
            *(u32x2*)(at + 8192) = u32x2{0u, 0u};
        }
        if (bi == bj) {   // the sum with its transpose (which the matrix unit forms, exactly)
            nh = to_bf4(mma32(cat8(nh, none), id8, from_bf4(nh)));
            nl = to_bf4(mma32(cat8(nl, none), id8, from_bf4(nl)));
        }
        at = mat(GN, j, 2 * bi + (gq >> 1)) + 8 * (gq & 1);         // -f likewise
        *(bf16x4*)at = nh;
        *(bf16x4*)(at + 8192) = nl;
    }
    // the parts that come from the states, and what they say of the decays
    const float hn = tok[1][DB - 1], ln = tok[2][DB - 1];
    const int rch = ((4 * w + gq) ^ swz(n16)) << 4;   // channels 32w + 8gq .. of row n
    auto dot8 = [&](bf16x8 x, const f32x4* y) __attribute__((always_inline)) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) s += (float)x[e] * y[0][e] + (float)x[4 + e] * y[1][e];
        return s;
    };
    float part[3][4];
#pragma unroll
    for (int ti = 0; ti < 4; ++ti) {
        const int t = 16 * ti + n16;
        const float b = tok[0][t], hi = tok[1][t], lo = tok[2][t], rk = tok[3][t], rq = tok[4][t];
        const float from = decay2(hi, lo, 0.0f, 0.0f), to = decay2(hn, ln, hi, lo);
        const float cq = A.scale * from * rq * fs, cs = -from * b * rk * fs, ce = to * b * rk * fz;
        const bf16x8 q8 = *(const bf16x8*)(lds + LQ + ti * 4096 + n16 * 256 + rch);
        const bf16x8 k8 = *(const bf16x8*)(lds + LK + ti * 4096 + n16 * 256 + rch);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            dq[ti][u] *= cq;
            dks[ti][u] *= cs;
            dke[ti][u] *= ce;
        }
        part[0][ti] = dot8(q8, dq[ti]);
        part[1][ti] = dot8(k8, dks[ti]);
        part[2][ti] = dot8(k8, dke[ti]);
#pragma unroll
        for (int u = 0; u < 2; ++u) dks[ti][u] += dke[ti][u];
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) dots[i][w][lane] = rows_sum(part[i]);
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
                // -sum over i > j of f_ij k_i (tiles from ti on), -sum over i < j of f_ji k_i (those up to ti)
                const bf16x8 n = 2 * pair >= ti
                                     ? *(const bf16x8*)(mat(GN, 16 * ti + n16, 4 * pair + gq) + piece * 8192)
                                     : cat8(tr_read(mat(GN, r0, 2 * ti + (pa >> 1)) + 8 * (pa & 1) + piece * 8192),
                                            tr_read(mat(GN, r1, 2 * ti + (pa >> 1)) + 8 * (pa & 1) + piece * 8192));
#pragma unroll
                for (int u = 0; u < 2; ++u) dks[ti][u] = mma32(kt[u], n, dks[ti][u]);
            }
        }
    }
    // unit length: d - x^ (x^.d), and the rows
    bf16x8 q8[4], k8[4];
#pragma unroll
    for (int ti = 0; ti < 4; ++ti) {
        q8[ti] = *(const bf16x8*)(lds + LQ + ti * 4096 + n16 * 256 + rch);
        k8[ti] = *(const bf16x8*)(lds + LK + ti * 4096 + n16 * 256 + rch);
        part[0][ti] = dot8(q8[ti], dq[ti]);
        part[1][ti] = dot8(k8[ti], dks[ti]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) dots[3 + i][w][lane] = rows_sum(part[i]);
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
        const int64_t at = ((it.tok0 + t) * Hv + it.h) * D + 32 * w + 8 * gq;
        if (A.low != 0) {
            put_partials(dq[ti], (char*)A.dq + 2 * at, (char*)A.dq + A.low + at);
            put_partials(dks[ti], (char*)A.dk + 2 * at, (char*)A.dk + A.low + at);
        } else {
            *(bf16x8*)((bf16*)A.dq + at) = cat8(to_bf4(dq[ti][0]), to_bf4(dq[ti][1]));
            *(bf16x8*)((bf16*)A.dk + at) = cat8(to_bf4(dks[ti][0]), to_bf4(dks[ti][1]));
        }
    }
    if (w == 3) {   // lane t: token t
        const int b = lane >> 4;
        auto at_lane = [&](float x, int i) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), i)); };
        auto four = [&](int i) { return (dots[i][0][lane] + dots[i][1][lane]) + (dots[i][2][lane] + dots[i][3][lane]); };
        // of x the tokens before this one, of y this one and those behind it
        const float x = four(2), y = four(0) + four(1);
        float before = row16_before(x), from = row16_from(y);
        const float x16 = before + x, y16 = from;
        float dg = before + from;
        {
            const float x0 = at_lane(x16, 15), x1 = at_lane(x16, 31), x2 = at_lane(x16, 47);
            const float y1 = at_lane(y16, 16), y2 = at_lane(y16, 32), y3 = at_lane(y16, 48);
            dg += b == 0 ? y1 + y2 + y3 : b == 1 ? x0 + (y2 + y3) : b == 2 ? x0 + x1 + y3 : x0 + x1 + x2;
        }
        dg += decay2(hn, ln, 0.0f, 0.0f) * ((whole[0] + whole[1]) + (whole[2] + whole[3]));
        // sum over i >= t > j: of column tile b, and of the column tiles before it
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i >= b) dg += sums[1][i][lane];
#pragma unroll
        for (int c = 0; c < 3; ++c) {
            const float r = row16_from(sums[0][c][lane]);   // this row and the tile's rows behind it
            const float r2 = at_lane(r, 32), r3 = at_lane(r, 48);
            if (c < b) dg += b == 1 ? r + (r2 + r3) : b == 2 ? r + r3 : r;
        }
        if (lane < it.len) {
            const int64_t at = (it.tok0 + lane) * Hv + it.h;
            ((bf16*)A.dg)[at] = (bf16)dg;
            ((bf16*)A.dbeta)[at] = (bf16)diag[lane];
        }
    }
    };
    // Loads to LDS: 16 rows of 64 bytes or 4 of 256 an instruction, a lane fetching the 16 bytes that
    // belong in its place.  Rows of 64 bytes: block b of do's row r at b ^ (r/4)%4, of W and Y as they are in
    // the planes; of 256 bytes as in the scans.
    const u32x4 zero = {0u, 0u, 0u, 0u};
    const int r16 = lane >> 2, b4 = lane & 3;
    const int64_t so = (int64_t)Hv * D;
    const bf16* pdo = (const bf16*)A.d_o + ((it.tok0 + 16 * w) * Hv + it.h) * D;
    const unsigned off_o = (unsigned)r16 * (unsigned)(so * 2) + ((b4 ^ ((r16 >> 2) & 3)) << 4);
    const bool second = it.len > SC;   // (a block may end in its first chunk)
    // rows W (waves 0, 1) and Y of chunk w % 2
    const char* prows = (w < 2 ? A.forward.rows : A.backward.rows) + (blk * 2 + (w & 1)) * PLANE_ROWS;
    auto load_stage = [&](char* to, int vb) __attribute__((always_inline)) {
        char* o = to + GS_O + w * 1024;
        if (16 * w + r16 < it.len)
            to_lds<false>((const char*)(pdo + 32 * vb), fresh(off_o), o);
        else
            *(u32x4*)(o + lane * 16) = zero;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            char* d = to + GS_R + w * 4096 + i * 1024;
            if ((w & 1) == 0 || second)
                to_lds<false>(prows + vb * 4096 + i * 1024, lane * 16, d);
            else
                *(u32x4*)(d + lane * 16) = zero;
        }
    };
    // S and Z: 8 channels v = 32vb + 8gq .. of column k = 32w + 8(n/4) + 4u + n%4
    const char* pstate[2] = {A.forward.state + blk * PLANE_STATE, A.backward.state + blk * PLANE_STATE};
    const int off_k = (gq >> 1) * (D * 16) + (32 * w + 8 * (n16 >> 2) + (n16 & 3)) * 16 + 8 * (gq & 1);
    u32x4 high[2][2];
    u32x2 low[2][2];
    auto load_states = [&](int vb) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int at = off_k + u * 64;
                high[i][u] = *row_ptr<const u32x4>(pstate[i] + vb * 8192, 2 * at);
                low[i][u] = *row_ptr<const u32x2>(pstate[i] + STATE_LOW + vb * 4096, at);
            }
    };
    auto load_rows = [&]() __attribute__((always_inline)) {
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
    };
    // operands of 8 channels v = 32vb + 8gq ..: rows (0: W, 1: Y), do
    const int pa = n16 & 3;   // this lane's piece of a transposing read
    const int at_row = (8 * gq + (n16 >> 2)) * 64 + pa * 16 + (gq & 1) * 8;
    const int at_o = n16 * 64 + ((gq ^ (n16 >> 2)) << 4);
    auto get_row = [&](const char* from, int set, int ti, int piece) __attribute__((always_inline)) {
        const char* r = from + GS_R + (set * 2 + (ti >> 1)) * 4096 + piece * 2048 + (fresh(at_row) ^ ((ti & 1) * 8));
        return cat8(tr_read(r), tr_read(r + 4 * 64));
    };
    auto get_o = [&](const char* from, int ti) __attribute__((always_inline)) {
        return *(const bf16x8*)(from + GS_O + ti * 1024 + fresh(at_o));
    };
    bf16* pdv = (bf16*)A.dv + ((it.tok0 + 16 * w + n16) * Hv + it.h) * D + 8 * gq;
    auto part = [&](int vb, const char* __restrict__ from, char* __restrict__ to) __attribute__((always_inline)) {
        bf16x8 st[2][2][2];   // S, Z; u; piece
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                st[i][u][0] = __builtin_bit_cast(bf16x8, high[i][u]);
                u32x4 rest;
#pragma unroll
                for (int j = 0; j < 4; ++j) {   // the upper half's value off the whole one is exact, and 8 bits
                    const unsigned h = high[i][u][j], l = low[i][u][j >> 1];
                    const unsigned x0 = __builtin_amdgcn_perm(h, l, j & 1 ? 0x0504020cu : 0x0504000cu),
                                   x1 = __builtin_amdgcn_perm(h, l, j & 1 ? 0x0706030cu : 0x0706010cu);
                    rest[j] = cvt_pk_bf16(__uint_as_float(x0) - __uint_as_float(h << 16),
                                          __uint_as_float(x1) - __uint_as_float(h & 0xffff0000u));
                }
                st[i][u][1] = __builtin_bit_cast(bf16x8, rest);
            }
        __builtin_amdgcn_sched_barrier(0);
        if (vb < 3) {
            load_states(vb + 1);
            load_stage(to, vb + 1);
        } else {   // q's and k's rows, over the first stage
            load_rows();
        }
        {   // dv of the wave's 16 tokens, 8 channels a lane.  (No branch stands behind the sums below: the
            // compiler would move them all past it.)
            const bf16x8 a = get_row(from, 1, w, 0), b = get_row(from, 1, w, 1);
            if (16 * w + n16 < it.len) {
                const float beta = tok[0][16 * w + n16];
                f32x4 y0, y1;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y0[e] = beta * ((float)a[e] + (float)b[e]);
                    y1[e] = beta * ((float)a[4 + e] + (float)b[4 + e]);
                }
                *(bf16x8*)(pdv + 32 * vb) = cat8(to_bf4(y0), to_bf4(y1));
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            zs = mma32(st[0][u][0], st[1][u][0], zs);
            zs = mma32(st[0][u][0], st[1][u][1], zs);
            zs = mma32(st[0][u][1], st[1][u][0], zs);
        }
#pragma unroll
        for (int ti = 0; ti < 4; ++ti) {
            __builtin_amdgcn_sched_barrier(0);   // (the parts of one tile of tokens at a time)
            const bf16x8 o = get_o(from, ti);
            bf16x8 wr[2], yr[2];
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                wr[d] = get_row(from, 0, ti, d);
                yr[d] = get_row(from, 1, ti, d);
            }
#pragma unroll
            for (int d = 0; d < 2; ++d)
#pragma unroll
                for (int u = 0; u < 2; ++u) dq[ti][u] = mma32(st[0][u][d], o, dq[ti][u]);
#pragma unroll
            for (int d = 0; d < 3; ++d)   // (pieces 0 0, 0 1 and 1 0)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    dks[ti][u] = mma32(st[0][u][d >> 1], yr[d & 1], dks[ti][u]);
                    dke[ti][u] = mma32(st[1][u][d >> 1], wr[d & 1], dke[ti][u]);
                }
        }
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            __builtin_amdgcn_sched_barrier(0);
            const int t = min(w + 4 * s, TILES - 1);   // (the last tile again where there is none: its sums are not used)
            const int bi = tile_i(t), bj = tile_j(t);
            const bf16x8 o = get_o(from, bi);
            bf16x8 wr[2], yr[2];
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                wr[d] = get_row(from, 0, bj, d);
                yr[d] = get_row(from, 1, bi, d);
            }
#pragma unroll
            for (int d = 0; d < 2; ++d) E[s] = mma32(o, wr[d], E[s]);
#pragma unroll
            for (int d = 0; d < 3; ++d) F[s] = mma32(yr[d >> 1], wr[d & 1], F[s]);
        }
        wait_vm<0>();
        barrier_lds();
    };
    load_states(0);
    load_stage(lds, 0);
    if (w == 3) put_tokens();
    wait_vm<0>();
    barrier_lds();
    for (int vb = 0; vb < 4; ++vb) part(vb, lds + (vb & 1) * GS2, lds + (~vb & 1) * GS2);
    const float z01 = n16 & 1 ? zs[1] : zs[0], z23 = n16 & 1 ? zs[3] : zs[2];
    finish(group_sum<64>(gq == n16 >> 2 ? (n16 & 2 ? z23 : z01) : 0.0f), fresh(tid & 63));
}

hipError_t launch_delta_grad(const DeltaGradArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(delta_grad_kernel, dim3((unsigned)a.blocks.items), dim3(256), 0, s, a);
    return hipGetLastError();
}

// Sum over the G value heads of a q/k head, in head order, of partials to BF16: 8 channels per thread.
__global__ __launch_bounds__(256) void delta_group_sum_kernel(const char* src0, const char* src1, int64_t low, bf16* dst0,
                                                              bf16* dst1, int64_t vecs, int G) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;   // (token, q/k head, 8 channels)
    if (i >= vecs) return;
    const int64_t row = i >> 4;
    const int c = (int)(i & 15) * 8;
    const char* src = blockIdx.y ? src1 : src0;
    f32x4 a = zero4(), b = zero4();
    for (int g = 0; g < G; ++g) {
        const int64_t at = (row * G + g) * D + c;
        const u32x4 h = *(const u32x4*)(src + 2 * at);
        const u32x2 l = *(const u32x2*)(src + low + at);
#pragma unroll
        for (int j = 0; j < 2; ++j) {   // channels 2j, 2j + 1 of either half
            a[2 * j] += __uint_as_float(__builtin_amdgcn_perm(h[j], l[0], j ? 0x0504020cu : 0x0504000cu));
            a[2 * j + 1] += __uint_as_float(__builtin_amdgcn_perm(h[j], l[0], j ? 0x0706030cu : 0x0706010cu));
            b[2 * j] += __uint_as_float(__builtin_amdgcn_perm(h[2 + j], l[1], j ? 0x0504020cu : 0x0504000cu));
            b[2 * j + 1] += __uint_as_float(__builtin_amdgcn_perm(h[2 + j], l[1], j ? 0x0706030cu : 0x0706010cu));
        }
    }
    *(bf16x8*)((blockIdx.y ? dst1 : dst0) + row * D + c) = cat8(to_bf4(a), to_bf4(b));
}

hipError_t launch_delta_group_sum(const void* src0, const void* src1, int64_t low, bf16_t* dst0, bf16_t* dst1, int64_t tokens,
                                  int Hqk, int G, hipStream_t s) {
    const int64_t vecs = tokens * Hqk * (D / 8);
    hipLaunchKernelGGL(delta_group_sum_kernel, dim3((unsigned)((vecs + 255) / 256), 2), dim3(256), 0, s, (const char*)src0,
                       (const char*)src1, low, (bf16*)dst0, (bf16*)dst1, vecs, G);
    return hipGetLastError();
}

}  // namespace kda
