// The gated delta rule's scans over the chunks of a sequence, forward and backward in time.
// (The formulas stand in kda_delta.hip.)
//
// One workgroup per item (kParts = 2: two, each with half of the state's output channels), a
// wave for every NU tiles of 16 channels v.  A wave keeps its columns of the state as MFMA
// accumulators: tile (t, u) is S^T[k][v] with
//     k = 32(t/2) + 8gq + 4(t%2) + e,   v = 32wv + 8(n/4) + 4u + n%4
// (NU = 1: v = 16wv + n; lane 16gq + n, element e).  The same registers are the operand of
// S K^T from either side, so that X = V - S K^T comes out with tokens along the elements,
// where W = X - C B X and S^T += K^T U take it without leaving the lane, and o^T = S Q^T +
// W^T P^T with 8 neighbouring channels of a token for its store.  Only P = Q K^T passes
// between waves.
// The state is kept divided by the decay since it was last rescaled, so that a chunk only
// adds to it; it is rescaled when that decay falls below 2^-24.
// Products are exact to FP32: S and B X go in as three BF16 pieces, C as three, U as three; P and W
// as two where they only meet o.  The rows of the next chunk and its record travel from
// memory to LDS while this one is computed.
// Bound by the steps of a chunk, each of which needs the one before: 2.4 us with up to one workgroup a
// unit; with two, matrix and vector instructions take 47% and 52% of the time (8 x 1024 tokens, 96 heads:
// forward 327 to 342 us, 3.1 TB/s; both scans of the backward with their planes 720 us, 4.8 TB/s).  The exact
// products are most of it: some 790 matrix instructions a chunk and head, 1.5 us of a unit's four.
// Sequences may be cut into segments, which a launch walks side by side: what a segment adds to a
// state, Q, and what it makes of one, M (the same scan with V = 0 from the identity), are formed first
// (kDeltaState), and chained, S <- S M + Q, by a kernel of its own; so are the adjoints with M^T.
#pragma once

#include "kda_delta.hpp"

namespace kda {

constexpr int DSET = SC * D * 2;        // LDS bytes of a chunk's rows
constexpr int DROWS16 = 16 * D * 2;     // of 16 rows

// LDS (bytes): a chunk's rows and its record in two buffers each; P's tiles (two of two pieces in the
// scan, one of three in the adjoint, with a fourth tile that is not used), q's lengths.
template <bool kThree, int kTiles>
struct DeltaLds {
    static constexpr int K = 0, V = 2 * DSET, Q = 4 * DSET, R = kThree ? 6 * DSET : 4 * DSET, P = R + 2 * REC,
                         X = P + kTiles * 4 * 512, TOTAL = X + 256;
};
template <int kMode>
struct DeltaScanLds : DeltaLds<kMode == kDeltaOut, kMode == kDeltaOut ? 4 : 0> {};
typedef DeltaLds<true, 3> DeltaAdjointLds;   // V: do

// Sum over each 8 lanes, in all of them.
__device__ __forceinline__ float row8_sum(float x) {
    x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0xB1, 0xF, 0xF, true));
    x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x4E, 0xF, 0xF, true));
    x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x141, 0xF, 0xF, true));
    return x;
}
// Where a wave's lanes lie, among the rows and in LDS.
template <int NU, int kParts>
struct DeltaLane {
    static constexpr int NW = 8 / NU / kParts, STEP = 4 * NW;
    static_assert(NW == 4, "four waves: three tiles of P and one to spare, 8 lanes a row for q's length");
    static_assert(STEP % 16 == 0, "rows of one lane share their place in a row's order");
    int w, lane, gq, n16, wv, lrow, vrow, r8, trow, piece, tr, trv;
    __device__ __forceinline__ DeltaLane(int part) {
        w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        lane = threadIdx.x & 63;
        gq = lane >> 4;
        n16 = lane & 15;
        wv = w + NW * part;   // this wave among the columns
        lrow = 4 * w + gq;
        vrow = NU == 2 ? 32 * wv + 8 * (n16 >> 2) + (n16 & 3) : 16 * wv + n16;   // + 4u
        // LDS offsets (bytes): 8 channels (32p + 8gq, xor 64p) of row n; for the transposing reads of row
        // 4gq + n/4 the piece n%4 of K's and Q's channels 32p .. and of the wave's own
        r8 = (n16 * D + ((gq ^ swz(n16)) << 3)) * 2;
        trow = 4 * gq + (n16 >> 2);
        piece = n16 & 3;
        tr = (trow * D + ((piece ^ swz(trow)) << 3)) * 2;
        trv = NU == 2 ? (trow * D + (((4 * wv + piece) ^ swz(trow)) << 3)) * 2
                      : (trow * D + (((2 * wv + (piece >> 1)) ^ swz(trow)) << 3) + 4 * (piece & 1)) * 2;
    }
    __device__ __forceinline__ int krow(int t) const { return 32 * (t >> 1) + 8 * gq + 4 * (t & 1); }
    // One set of a chunk's rows to LDS: an instruction of a wave moves 4 rows of 256 bytes (16
    // lanes a row) to 1 KiB in lane order, a lane fetching the block that belongs there.
    __device__ __forceinline__ void fetch(const char* rows, int64_t bytes, unsigned off, char* to) const {
#pragma unroll
        for (int j = 0; j < SC / STEP; ++j) to_lds<false>(rows + j * STEP * bytes, off, to + (STEP * j + 4 * w) * D * 2);
    }
    // The same of a chunk of `rem` tokens: the rows behind them are not read and count as zero.
    __device__ __forceinline__ void fetch(const char* rows, int64_t bytes, unsigned off, char* to, int rem) const {
#pragma unroll
        for (int j = 0; j < SC / STEP; ++j) {
            char* d = to + (STEP * j + 4 * w) * D * 2;
            if (lrow + STEP * j < rem)
                to_lds<false>(rows + j * STEP * bytes, off, d);
            else
                *(u32x4*)(d + lane * 16) = u32x4{0u, 0u, 0u, 0u};
        }
    }
    // A record, a KiB an instruction, the waves in turn.
    __device__ __forceinline__ void fetch_record(const char* p, char* to) const {
        static_assert(REC % 1024 == 0, "whole instructions");
#pragma unroll
        for (int i = 0; i < REC / 1024; ++i)
            if (i % NW == w) to_lds<false>(p + i * 1024, lane * 16, to + i * 1024);
    }
    __device__ __forceinline__ unsigned offset(int64_t bytes) const {
        return (unsigned)lrow * (unsigned)bytes + ((n16 ^ swz(lrow)) << 4);
    }
};

// The planes of a state, which is `held` times S, and of a chunk's rows.  A store of a wave covers whole 512
// or 256 bytes.  (Both scans of 4 x 4096 tokens of 32 heads, in halves: 488 us; 570 with 32 channels v side by
// side, of which a half's wave has 16.)
template <int NU, int kParts>
struct PlaneWriter {
    const DeltaLane<NU, kParts>& L;
    const Pieces& pieces;
    // The matrix units turn the state around: its pieces times an identity, added up, are 4 channels v of
    // column k = n.
    __device__ __forceinline__ void state(const f32x4 (&S)[8][NU], float held, const DeltaPlanes& to, int64_t blk) const {
        char* p = to.state + blk * PLANE_STATE;
        bf16x8 id[2];   // columns 16i + n of 32
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f32x4 x[2];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j >> 2][j & 3] = 8 * L.gq + j == 16 * i + L.n16 ? 1.0f : 0.0f;
            id[i] = cat8(to_bf4(x[0]), to_bf4(x[1]));
        }
        const int at = NU == 2 ? (2 * L.wv + (L.gq >> 1)) * (D * 16) + L.n16 * 16 + 8 * (L.gq & 1)
                               : L.wv * (D * 16) + L.n16 * 16 + 4 * L.gq;
#pragma unroll
        for (int t = 0; t < 8; t += 2) {
            bf16x8 piece[NU][2];
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                f32x4 x = S[t][u], y = S[t + 1][u];
                piece[u][0] = pieces.take(x, y);
                piece[u][1] = cat8(to_bf4(x), to_bf4(y));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int off = at + 16 * (t + i) * 16;
                unsigned high[2 * NU], low[NU];
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                    const f32x4 x = mma32(piece[u][1], id[i], mma32(piece[u][0], id[i], zero4()));
                    const u32x4 y = __builtin_bit_cast(u32x4, x) + 0x80u;   // (the matrix units' NaN is 0xffc00000)
                    high[2 * u] = __builtin_amdgcn_perm(y[1], y[0], 0x07060302u);
                    high[2 * u + 1] = __builtin_amdgcn_perm(y[3], y[2], 0x07060302u);
                    low[u] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(y[3], y[2], 0x0c0c0501u),
                                                   __builtin_amdgcn_perm(y[1], y[0], 0x0c0c0501u), 0x05040100u);
                }
                if constexpr (NU == 2) {
                    *(u32x4*)(p + 2 * off) = u32x4{high[0], high[1], high[2], high[3]};
                    *(u32x2*)(p + STATE_LOW + off) = u32x2{low[0], low[1]};
                } else {
                    *(u32x2*)(p + 2 * off) = u32x2{high[0], high[1]};
                    *(unsigned*)(p + STATE_LOW + off) = low[0];
                }
            }
        }
        if (threadIdx.x == 0) to.scale[blk] = held;   // (both parts the same)
    }
    __device__ __forceinline__ void rows(const f32x4 (&w)[2][NU], const DeltaPlanes& to, int64_t chunk) const {
        char* p = to.rows + chunk * PLANE_ROWS;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int v = L.vrow + 4 * u;
            const bool odd = (v & 8) != 0;
            bf16x4 a[2], b[2];
            split4_rne(w[0][u], a[0], a[1]);
            split4_rne(w[1][u], b[0], b[1]);
#pragma unroll
            for (int d = 0; d < 2; ++d)
                *(bf16x8*)(p + (v >> 5) * 4096 + d * 2048 + (v & 31) * 64 + 16 * L.gq) = odd ? cat8(b[d], a[d]) : cat8(a[d], b[d]);
        }
    }
};

template <int NU, int kParts, int kMode>
__device__ __forceinline__ void delta_scan(const DeltaArgs& A, int block, int grid, char* lds) {
    constexpr bool kOut = kMode == kDeltaOut, kRecord = kMode == kDeltaRecord, kState = kMode == kDeltaState;
    constexpr int kJobs = kState ? 2 : 1;
    typedef DeltaScanLds<kMode> M;
    constexpr int NW = 8 / NU / kParts;

    int idx = xcd_order(block, grid, A.G * kParts * kJobs);
    const int part = idx % kParts;
    idx /= kParts;
    const bool map_job = kState && (idx & 1) != 0;   // what the segment makes of a state: V zero, from the identity
    idx /= kJobs;
    const DeltaLane<NU, kParts> L(part);
    const int w = L.w, lane = L.lane, gq = L.gq, n16 = L.n16;
    const Item it = find_item(A.map, idx);
    // of a sequence's segments, the last one's state is not needed, nor the first one's map
    const bool last = it.off + it.len >= (A.map.task != nullptr ? A.map.seq_len[it.n] : A.map.len);
    if (kState && (last || (map_job && it.off == 0))) return;
    const int64_t slot = A.slot != nullptr ? A.slot[it.n] : it.n;
    if (slot < 0 || slot >= A.slots) return;
    const int Hv = A.map.Hv;
    const int64_t soff = (slot * Hv + it.h) * (int64_t)STATE;
    float* seg = A.seg == nullptr ? nullptr : A.seg + (it.seg * Hv + it.h) * (int64_t)(2 * STATE);
    const float* s_in = !kState && seg != nullptr ? seg
                        : A.s_in != nullptr && !(kState && (map_job || it.off != 0)) ? A.s_in + soff
                                                                                     : nullptr;
    // the item's first block among all blocks
    const int64_t block0 = (A.blocks.task != nullptr ? A.blocks.tape_off[it.n] + it.n
                                                     : (int64_t)it.n * ((A.blocks.len + DB - 1) / DB)) + it.off / DB;

    // the next chunk's rows and record (a block's second record is behind the first, the next
    // block's Hv blocks on)
    const int64_t bk = A.sk * 2, bv = A.sv * 2, bq = A.sq * 2;
    const char* pk = (const char*)((const bf16*)A.k + it.tok0 * A.sk + (it.h / A.G) * D);
    const char* pv = (const char*)((const bf16*)A.v + it.tok0 * A.sv + it.h * D);
    const char* pq = kOut ? (const char*)((const bf16*)A.q + it.tok0 * A.sq + (it.h / A.G) * D) : nullptr;
    const unsigned ok = L.offset(bk), ov = L.offset(bv), oq = kOut ? L.offset(bq) : 0;
    char* prec = A.rec + (block0 * Hv + it.h) * (2 * REC);
    const int64_t over = (int64_t)(2 * Hv - 1) * REC;
    auto fetch = [&](char* rows_to, char* rec_to, int rem, bool second, auto full) __attribute__((always_inline)) {
        if (decltype(full)::value || rem >= SC) {
            L.fetch(pk, bk, ok, rows_to + M::K);
            L.fetch(pv, bv, ov, rows_to + M::V);
            if (kOut) L.fetch(pq, bq, oq, rows_to + M::Q);
        } else {
            L.fetch(pk, bk, ok, rows_to + M::K, rem);
            L.fetch(pv, bv, ov, rows_to + M::V, rem);
            if (kOut) L.fetch(pq, bq, oq, rows_to + M::Q, rem);
        }
        L.fetch_record(prec, rec_to);
        pk += SC * bk;
        pv += SC * bv;
        if (kOut) pq += SC * bq;
        prec += second ? over : REC;
    };
    fetch(lds, lds + M::R, it.len, false, std::false_type{});

    f32x4 S[8][NU];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int u = 0; u < NU; ++u)
            S[t][u] = s_in != nullptr ? *(const f32x4*)(s_in + (L.vrow + 4 * u) * D + L.krow(t)) : zero4();
    if (map_job)
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[t][u][e] = L.krow(t) + e == L.vrow + 4 * u ? 1.0f : 0.0f;
    const unsigned v_mask = map_job ? 0u : ~0u;

    const Pieces pieces(lane);
    const PlaneWriter<NU, kParts> planes{L, pieces};
    const int64_t sy = (int64_t)Hv * D * 2;
    char* po = kOut ? (char*)(A.o + (it.tok0 * Hv + it.h) * D) : nullptr;
    const unsigned oy = (unsigned)n16 * (unsigned)sy + (16 * NU * L.wv + 4 * NU * gq) * 2;
    double held = 1.0;   // the state is `held` times S

    // One chunk from `rows` and `rec`, the next one on its way into `rows_to` and `rec_to`.
    // (They are halves of the same arrays; as restrict pointers they show the compiler that what is
    // read through the one need not wait for what is on its way into the other.)
    auto chunk = [&](int c, const char* __restrict__ rows, const char* __restrict__ rec, char* __restrict__ rows_to,
                     char* __restrict__ rec_to, auto steady) __attribute__((always_inline)) {
        auto num = [&](int array, int i) __attribute__((always_inline)) { return *(const float*)(rec + array + 4 * i); };
        auto num4 = [&](int array, int i) __attribute__((always_inline)) { return *(const f32x4*)(rec + array + 4 * i); };
        constexpr bool kSteady = decltype(steady)::value;   // a full chunk follows
        const int rem = it.len - c * SC;
        const bool more = kSteady || rem > SC;
        float* lengths = kOut && A.unit && part == 0 && w == 0 ? (float*)(prec - ((c & 1) ? over : REC) + REC_Q) : nullptr;
        if (more) fetch(rows_to, rec_to, rem - SC, (c & 1) == 0, steady);
        const char *k = rows + M::K, *v = rows + M::V, *q = rows + M::Q;
        char* lds_p = lds + M::P + (c & 1) * 4096;
        float* lds_q = (float*)(lds + M::X + (c & 1) * 128);
        // the decay as one more factor of `held`, while that is not below 2^-24
        const float before = (float)held;   // of the state that the chunk meets
        held *= (double)num(REC_DECAY, 0) + (double)num(REC_DECAY, 1);
        const float down = (float)held;
        const bool rescale = held < 0x1p-24;
        if (rescale) held = 1.0;
        const float up = 1.0f / (float)held;
        if (kOut) {
            // P^T tiles: waves 0, 1, 2 form (i, j) = (0, 0), (1, 1), (1, 0), the others one that is not
            // used (a branch would keep the products below from filling this chain's waits)
            const int bi = w == 0 ? 0 : 1, bj = w == 1 ? 1 : 0;
            f32x4 acc = zero4();
#pragma unroll
            for (int p = 0; p < 4; ++p)
                acc = mma32(*(const bf16x8*)(k + ((L.r8 + bj * DROWS16) ^ (64 * p))),
                            *(const bf16x8*)(q + ((L.r8 + bi * DROWS16) ^ (64 * p))), acc);
            const int i = 16 * bi + n16, j = 16 * bj + 4 * gq;
            const float hi = num(REC_GH, i), li = num(REC_GL, i);
            const f32x4 rb = num4(REC_KB, j), hj = num4(REC_GH, j), lj = num4(REC_GL, j);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = acc[e] * rb[e] * decay2(hi, li, hj[e], lj[e]);
                acc[e] = i >= j + e ? x : 0.0f;
            }
            bf16x4 hi4, lo4;
            pieces.split(acc, hi4, lo4);
            *(bf16x8*)(lds_p + w * 1024 + lane * 16) = cat8(hi4, lo4);
            // one over q's length: 2 NW lanes a row
            constexpr int PER = 64 / NW;   // channels a lane
            const bf16x2* row = (const bf16x2*)(q + (32 / NW * w + lane / (2 * NW)) * 256 + lane % (2 * NW) * (2 * PER));
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < PER / 2; ++e) s = __builtin_amdgcn_fdot2_f32_bf16(row[e], row[e], s, false);
            s = row8_sum(s);
            lds_q[32 / NW * w + lane / (2 * NW)] = A.unit ? rsqrtf(s + NORM_EPS) : 1.0f;
        }
        // S K^T and S Q^T
        f32x4 x[2][NU], y[2][NU];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            bf16x8 ak[2], aq[2];
#pragma unroll
            for (int ti = 0; ti < 2; ++ti) {
                ak[ti] = *(const bf16x8*)(k + ((L.r8 + ti * DROWS16) ^ (64 * p)));
                if (kOut) aq[ti] = *(const bf16x8*)(q + ((L.r8 + ti * DROWS16) ^ (64 * p)));
            }
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                bf16x8 pc[3];
                pieces.split(S[2 * p][u], S[2 * p + 1][u], pc);
#pragma unroll
                for (int d = 0; d < 3; ++d) {
                    const bf16x8 s = pc[d];
#pragma unroll
                    for (int ti = 0; ti < 2; ++ti) x[ti][u] = mma32(ak[ti], s, p + d == 0 ? zero4() : x[ti][u]);
                    if (kOut && d < 2) {
#pragma unroll
                        for (int ti = 0; ti < 2; ++ti) y[ti][u] = mma32(s, aq[ti], p + d == 0 ? zero4() : y[ti][u]);
                    }
                }
            }
        }
        // X = V - e^G S K^T
        f32x4 wr[2][NU];
#pragma unroll
        for (int ti = 0; ti < 2; ++ti) {
            const f32x4 cx = num4(REC_FROM_K, 16 * ti + 4 * gq) * before;
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                bf16x4 vb = tr_read(v + L.trv + 8 * u + DROWS16 * ti);
                if (kState) vb = __builtin_bit_cast(bf16x4, __builtin_bit_cast(u32x2, vb) & v_mask);
                const f32x4 vf = from_bf4(vb);
#pragma unroll
                for (int e = 0; e < 4; ++e) wr[ti][u][e] = fmaf(-cx[e], x[ti][u][e], vf[e]);
            }
        }
        const float co[2] = {kOut ? num(REC_FROM, n16) * before : 0.0f, kOut ? num(REC_FROM, 16 + n16) * before : 0.0f};
        if (rescale) {
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int u = 0; u < NU; ++u) S[t][u] *= down;
        }
        // W = X - C B X; S <- e^{G_n} S + K^T U
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            f32x4 &w0 = wr[0][u], &w1 = wr[1][u];
            {
                bf16x4 c11[3], c22[3], c21[3];
#pragma unroll
                for (int d = 0; d < 3; ++d) {
                    const char* at = rec + d * REC_TILE + n16 * 32 + gq * 8;
                    c11[d] = *(const bf16x4*)(at + REC_C11);
                    c22[d] = *(const bf16x4*)(at + REC_C22);
                    c21[d] = *(const bf16x4*)(at + REC_C21);
                }
                bf16x4 x0[3], x1[3];
                pieces.split(w0 * num4(REC_BETA, 4 * gq), x0[0], x0[1], x0[2]);
                pieces.split(w1 * num4(REC_BETA, 16 + 4 * gq), x1[0], x1[1], x1[2]);
                // pieces (a, b) with a + b <= 2; row block 0 takes two products at once
                w0 = mma32(cat8(c11[0], c11[0]), cat8(x0[0], x0[1]), w0);
                w0 = mma32(cat8(c11[1], c11[1]), cat8(x0[0], x0[1]), w0);
                w0 = mma32(cat8(c11[0], c11[2]), cat8(x0[2], x0[0]), w0);
#pragma unroll
                for (int a = 0; a < 3; ++a)
#pragma unroll
                    for (int b = 0; a + b < 3; ++b) w1 = mma32(cat8(c21[a], c22[a]), cat8(x0[b], x1[b]), w1);
            }
            bf16x8 u3[3];
            {
                const f32x4 e0 = num4(REC_TO_KB, 4 * gq) * up, e1 = num4(REC_TO_KB, 16 + 4 * gq) * up;
                bf16x4 a0[3], a1[3];
                pieces.split(w0 * e0, a0[0], a0[1], a0[2]);
                pieces.split(w1 * e1, a1[0], a1[1], a1[2]);
#pragma unroll
                for (int d = 0; d < 3; ++d) u3[d] = cat8(a0[d], a1[d]);
            }
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const char* row = k + (L.tr ^ (64 * (t >> 1))) + 8 * (t & 1);
                const bf16x8 kt = cat8(tr_read(row), tr_read(row + DROWS16));
#pragma unroll
                for (int d = 0; d < 3; ++d) S[t][u] = mma32(kt, u3[d], S[t][u]);
            }
        }
        if (kOut) {
            if (more) wait_vm<0>();
            barrier_lds();   // the next chunk is there, and P and q's lengths
            const bf16x8 p00 = *(const bf16x8*)(lds_p + lane * 16), p11 = *(const bf16x8*)(lds_p + 1024 + lane * 16),
                         p10 = *(const bf16x8*)(lds_p + 2048 + lane * 16);
            const bf16x8 p1h = __builtin_shufflevector(p10, p11, 0, 1, 2, 3, 8, 9, 10, 11),
                         p1l = __builtin_shufflevector(p10, p11, 4, 5, 6, 7, 12, 13, 14, 15);
            const float cy[2] = {A.scale * lds_q[n16], A.scale * lds_q[16 + n16]};
            u32x2 out[2][NU];
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                bf16x4 h0, l0, h1, l1;
                pieces.split(wr[0][u], h0, l0);
                pieces.split(wr[1][u], h1, l1);
                f32x4 y0 = y[0][u] * co[0], y1 = y[1][u] * co[1];
                y0 = mma32(cat8(h0, h0), p00, y0);
                y0 = mma32(cat8(l0, l0), p00, y0);
                y1 = mma32(cat8(h0, h1), p1h, y1);
                y1 = mma32(cat8(h0, h1), p1l, y1);
                y1 = mma32(cat8(l0, l1), p1h, y1);
                out[0][u] = __builtin_bit_cast(u32x2, to_bf4(y0 * cy[0]));
                out[1][u] = __builtin_bit_cast(u32x2, to_bf4(y1 * cy[1]));
            }
#pragma unroll
            for (int ti = 0; ti < 2; ++ti)
                if (kSteady || 16 * ti + n16 < rem) {
                    if constexpr (NU == 2)
                        *row_ptr<u32x4>(po + 16 * ti * sy, oy) = u32x4{out[ti][0][0], out[ti][0][1], out[ti][1][0], out[ti][1][1]};
                    else
                        *row_ptr<u32x2>(po + 16 * ti * sy, oy) = out[ti][0];
                }
            po += SC * sy;
            if (lengths != nullptr && lane < SC) lengths[lane] = lds_q[lane];   // (for a backward that is given the records)
        }
        if (kState) {
            if (more) wait_vm<0>();
            barrier_lds();
        }
        if (kRecord) {
            // the planes of this chunk's rows, and of the state when it is the next block's
            const bool edge = (c & 1) != 0 && more;
            if (more) wait_vm<0>();
            barrier_lds();
            const int64_t blk = (block0 + (c >> 1)) * Hv + it.h;
            planes.rows(wr, A.planes, blk * 2 + (c & 1));
            if (edge) planes.state(S, (float)held, A.planes, blk + Hv);
        }
    };
    wait_vm<0>();
    barrier_lds();
    if (kRecord) planes.state(S, 1.0f, A.planes, block0 * Hv + it.h);
    auto at = [&](int c, auto steady) __attribute__((always_inline)) {
        const int x = c & 1;
        chunk(c, lds + x * DSET, lds + M::R + x * REC, lds + (x ^ 1) * DSET, lds + M::R + (x ^ 1) * REC, steady);
    };
    const int chunks = (it.len + SC - 1) / SC, steady = it.len / SC - 1;
    int c = 0;
    for (; c < steady; ++c) at(c, std::true_type{});
    for (; c < chunks; ++c) at(c, std::false_type{});

    if (kState || (A.s_out != nullptr && last)) {
        const Factor decay(held);
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                f32x4 r;
#pragma unroll
                for (int e = 0; e < 4; ++e) r[e] = decay.apply(S[t][u][e]);
                if (map_job) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) seg[STATE + (L.krow(t) + e) * D + L.vrow + 4 * u] = r[e];
                    continue;
                }
                *(f32x4*)((kState ? seg : A.s_out + soff) + (L.vrow + 4 * u) * D + L.krow(t)) = r;
            }
    }
}

// The same backward in time, with Z = dS in place of S and the chunks in descending order:
//     dU = P^T do + e^{G_n - G} K Z,   Y = dU - C^T B dU,
//     Z <- e^{G_n} Z + Q^T (s e^G do) - K^T (e^G B Y),
// the pieces of P, C^T, B dU, do and Y as exact as above.
// kState: only what a segment adds to an adjoint.
template <int NU, int kParts, bool kState>
__device__ __forceinline__ void delta_adjoint(const DeltaArgs& A, int block, int grid, char* lds) {
    typedef DeltaAdjointLds M;
    constexpr int NW = 8 / NU / kParts;
    int idx = xcd_order(block, grid, A.G * kParts);
    const int part = idx % kParts;
    idx /= kParts;
    const DeltaLane<NU, kParts> L(part);
    const int w = L.w, lane = L.lane, gq = L.gq, n16 = L.n16;
    const Item it = find_item(A.map, idx);
    if (kState && it.off == 0) return;
    const bool last = it.off + it.len >= (A.map.task != nullptr ? A.map.seq_len[it.n] : A.map.len);
    const int Hv = A.map.Hv;
    const int64_t soff = ((int64_t)it.n * Hv + it.h) * (int64_t)STATE;
    float* behind = A.behind == nullptr ? nullptr : A.behind + (it.seg * Hv + it.h) * (int64_t)STATE;
    const float* s_in = !kState && behind != nullptr ? behind : A.s_in != nullptr && !(kState && !last) ? A.s_in + soff : nullptr;
    const int64_t block0 = (A.blocks.task != nullptr ? A.blocks.tape_off[it.n] + it.n
                                                     : (int64_t)it.n * ((A.blocks.len + DB - 1) / DB)) + it.off / DB;
    const int chunks = (it.len + SC - 1) / SC;

    const int64_t bk = A.sk * 2, bo = (int64_t)Hv * D * 2, bq = A.sq * 2;
    const char* pk = (const char*)((const bf16*)A.k + it.tok0 * A.sk + (it.h / A.G) * D);
    const char* pd = (const char*)((const bf16*)A.d_o + (it.tok0 * Hv + it.h) * D);
    const char* pq = (const char*)((const bf16*)A.q + it.tok0 * A.sq + (it.h / A.G) * D);
    const unsigned ok = L.offset(bk), oo = L.offset(bo), oq = L.offset(bq);
    const char* prec = A.rec + ((block0 + ((chunks - 1) >> 1)) * Hv + it.h) * (2 * REC) + ((chunks - 1) & 1) * REC;
    const int64_t over = (int64_t)(2 * Hv - 1) * REC;
    {
        const int64_t t = (int64_t)(chunks - 1) * SC;
        pk += t * bk;
        pd += t * bo;
        pq += t * bq;
    }
    // the next chunk (in walking order): all but the sequence's last are full
    auto fetch = [&](char* rows_to, char* rec_to, int rem, bool second, auto full) __attribute__((always_inline)) {
        if (decltype(full)::value || rem >= SC) {
            L.fetch(pk, bk, ok, rows_to + M::K);
            L.fetch(pd, bo, oo, rows_to + M::V);
            L.fetch(pq, bq, oq, rows_to + M::Q);
        } else {
            L.fetch(pk, bk, ok, rows_to + M::K, rem);
            L.fetch(pd, bo, oo, rows_to + M::V, rem);
            L.fetch(pq, bq, oq, rows_to + M::Q, rem);
        }
        L.fetch_record(prec, rec_to);
        pk -= SC * bk;
        pd -= SC * bo;
        pq -= SC * bq;
        prec -= second ? REC : over;
    };
    fetch(lds, lds + M::R, it.len - (chunks - 1) * SC, ((chunks - 1) & 1) != 0, std::false_type{});
    f32x4 Z[8][NU];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int u = 0; u < NU; ++u)
            Z[t][u] = s_in != nullptr ? *(const f32x4*)(s_in + (L.vrow + 4 * u) * D + L.krow(t)) : zero4();

    const Pieces pieces(lane);
    const PlaneWriter<NU, kParts> planes{L, pieces};
    double held = 1.0;   // the adjoint is `held` times Z
    auto chunk = [&](int c, const char* __restrict__ rows, const char* __restrict__ rec, char* __restrict__ rows_to,
                     char* __restrict__ rec_to, auto before) __attribute__((always_inline)) {
        auto num = [&](int array, int i) __attribute__((always_inline)) { return *(const float*)(rec + array + 4 * i); };
        auto num4 = [&](int array, int i) __attribute__((always_inline)) { return *(const f32x4*)(rec + array + 4 * i); };
        constexpr bool more = decltype(before)::value;   // (the chunks before the last are full)
        if (more) fetch(rows_to, rec_to, SC, (c & 1) == 0, before);
        const char *k = rows + M::K, *q = rows + M::Q;
        char* lds_p = lds + M::P;
        const float behind = (float)held;   // of the adjoint that the chunk meets
        held *= (double)num(REC_DECAY, 0) + (double)num(REC_DECAY, 1);
        const float down = (float)held;
        const bool rescale = held < 0x1p-24;
        if (rescale) held = 1.0;
        const float up = 1.0f / (float)held;
        {   // P tiles as their transposes' operands: lane (gq, n) rows i = 4gq + e of column j = n,
            // in waves 0, 1, 2 (i, j) = (0, 0), (1, 1), (1, 0)
            const int bi = w == 0 ? 0 : 1, bj = w == 1 ? 1 : 0;
            f32x4 acc = zero4();
#pragma unroll
            for (int p = 0; p < 4; ++p)
                acc = mma32(*(const bf16x8*)(q + ((L.r8 + bi * DROWS16) ^ (64 * p))),
                            *(const bf16x8*)(k + ((L.r8 + bj * DROWS16) ^ (64 * p))), acc);
            const int i = 16 * bi + 4 * gq, j = 16 * bj + n16;
            const float rj = A.scale * num(REC_K, j), hj = num(REC_GH, j), lj = num(REC_GL, j);
            const f32x4 ai = num4(REC_Q, i), hi = num4(REC_GH, i), li = num4(REC_GL, i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = acc[e] * (ai[e] * rj) * decay2(hi[e], li[e], hj, lj);
                acc[e] = i + e >= j ? x : 0.0f;
            }
            bf16x4 a, b, d;
            pieces.split(acc, a, b, d);
            char* to = lds_p + w * 1536 + lane * 8;
            *(bf16x4*)to = a;
            *(bf16x4*)(to + 512) = b;
            *(bf16x4*)(to + 1024) = d;
        }
        f32x4 x[2][NU];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            bf16x8 ak[2];
#pragma unroll
            for (int ti = 0; ti < 2; ++ti) ak[ti] = *(const bf16x8*)(k + ((L.r8 + ti * DROWS16) ^ (64 * p)));
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                bf16x8 pc[3];
                pieces.split(Z[2 * p][u], Z[2 * p + 1][u], pc);
#pragma unroll
                for (int d = 0; d < 3; ++d) {
                    const bf16x8 z = pc[d];
#pragma unroll
                    for (int ti = 0; ti < 2; ++ti) x[ti][u] = mma32(ak[ti], z, p + d == 0 ? zero4() : x[ti][u]);
                }
            }
        }
        bf16x4 dof[2][NU];
#pragma unroll
        for (int ti = 0; ti < 2; ++ti)
#pragma unroll
            for (int u = 0; u < NU; ++u) dof[ti][u] = tr_read(rows + M::V + L.trv + 8 * u + DROWS16 * ti);
        barrier_lds();   // P is there
        if (rescale) {
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int u = 0; u < NU; ++u) Z[t][u] *= down;
        }
        const bf16x4 none = __builtin_bit_cast(bf16x4, u32x2{0u, 0u});
        f32x4 yr[2][NU];
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            if (NU == 2) __builtin_amdgcn_sched_barrier(0);   // (as many pieces at a time as registers hold)
            f32x4 y0 = x[0][u] * (num4(REC_TO_K, 4 * gq) * behind), y1 = x[1][u] * (num4(REC_TO_K, 16 + 4 * gq) * behind);
            const bf16x4 d0 = dof[0][u], d1 = dof[1][u];
            {
                bf16x4 pt[3][3];   // tile, piece
#pragma unroll
                for (int tile = 0; tile < 3; ++tile)
#pragma unroll
                    for (int d = 0; d < 3; ++d) pt[tile][d] = *(const bf16x4*)(lds_p + tile * 1536 + d * 512 + lane * 8);
#pragma unroll
                for (int d = 0; d < 3; ++d) y0 = mma32(cat8(pt[0][d], pt[2][d]), cat8(d0, d1), y0);
                y1 = mma32(cat8(pt[1][0], pt[1][1]), cat8(d1, d1), y1);
                y1 = mma32(cat8(pt[1][2], none), cat8(d1, none), y1);
            }
            {
                bf16x4 c11[3], c22[3], c21[3];   // of -C^T: lane (gq, j) rows i = 4gq + e of column j
#pragma unroll
                for (int d = 0; d < 3; ++d) {
                    const char* at = rec + d * REC_TILE + L.trow * 32 + L.piece * 8;
                    c11[d] = tr_read(at + REC_C11);
                    c22[d] = tr_read(at + REC_C22);
                    c21[d] = tr_read(at + REC_C21);
                }
                bf16x4 q0[3], q1[3];
                pieces.split(y0 * num4(REC_BETA, 4 * gq), q0[0], q0[1], q0[2]);
                pieces.split(y1 * num4(REC_BETA, 16 + 4 * gq), q1[0], q1[1], q1[2]);
                y1 = mma32(cat8(c22[0], c22[0]), cat8(q1[0], q1[1]), y1);
                y1 = mma32(cat8(c22[1], c22[1]), cat8(q1[0], q1[1]), y1);
                y1 = mma32(cat8(c22[0], c22[2]), cat8(q1[2], q1[0]), y1);
#pragma unroll
                for (int a = 0; a < 3; ++a)
#pragma unroll
                    for (int b = 0; a + b < 3; ++b) y0 = mma32(cat8(c11[a], c21[a]), cat8(q0[b], q1[b]), y0);
            }
            yr[0][u] = y0;
            yr[1][u] = y1;
            bf16x8 y3[3], o3[3];   // what the state takes up, in pieces
            {
                bf16x4 a0[3], a1[3];
                pieces.split(y0 * (num4(REC_FROM_KB, 4 * gq) * -up), a0[0], a0[1], a0[2]);
                pieces.split(y1 * (num4(REC_FROM_KB, 16 + 4 * gq) * -up), a1[0], a1[1], a1[2]);
#pragma unroll
                for (int d = 0; d < 3; ++d) y3[d] = cat8(a0[d], a1[d]);
                const float us = up * A.scale;
                pieces.split(from_bf4(d0) * (num4(REC_FROM, 4 * gq) * num4(REC_Q, 4 * gq) * us), a0[0], a0[1], a0[2]);
                pieces.split(from_bf4(d1) * (num4(REC_FROM, 16 + 4 * gq) * num4(REC_Q, 16 + 4 * gq) * us), a1[0], a1[1], a1[2]);
#pragma unroll
                for (int d = 0; d < 3; ++d) o3[d] = cat8(a0[d], a1[d]);
            }
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const int at = (L.tr ^ (64 * (t >> 1))) + 8 * (t & 1);
                const bf16x8 kt = cat8(tr_read(k + at), tr_read(k + at + DROWS16));
                const bf16x8 qt = cat8(tr_read(q + at), tr_read(q + at + DROWS16));
#pragma unroll
                for (int d = 0; d < 3; ++d) Z[t][u] = mma32(kt, y3[d], Z[t][u]);
#pragma unroll
                for (int d = 0; d < 3; ++d) Z[t][u] = mma32(qt, o3[d], Z[t][u]);
            }
        }
        if (kState) {
            if (more) wait_vm<0>();
            barrier_lds();
            return;
        }
        // the planes of this chunk's rows, and of the adjoint when it is behind the next block
        const bool edge = (c & 1) == 0 && more;
        if (more) wait_vm<0>();
        barrier_lds();
        const int64_t blk = (block0 + (c >> 1)) * Hv + it.h;
        planes.rows(yr, A.planes, blk * 2 + (c & 1));
        if (edge) planes.state(Z, (float)held, A.planes, blk - Hv);
    };
    wait_vm<0>();
    barrier_lds();
    if (!kState) planes.state(Z, 1.0f, A.planes, (block0 + ((chunks - 1) >> 1)) * Hv + it.h);
    int x = 0;
    auto at = [&](int c, auto before) __attribute__((always_inline)) {
        chunk(c, lds + x * DSET, lds + M::R + x * REC, lds + (x ^ 1) * DSET, lds + M::R + (x ^ 1) * REC, before);
        x ^= 1;
    };
    for (int c = chunks - 1; c > 0; --c) at(c, std::true_type{});
    at(0, std::false_type{});

    if (kState || (A.s_out != nullptr && it.off == 0)) {
        const Factor decay(held);
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                f32x4 r;
#pragma unroll
                for (int e = 0; e < 4; ++e) r[e] = decay.apply(Z[t][u][e]);
                *(f32x4*)((kState ? behind : A.s_out + soff) + (L.vrow + 4 * u) * D + L.krow(t)) = r;
            }
    }
}

}  // namespace kda
