// Linear attention with a constant decay per head: training forward and
// backward, prefill, and the token-serial form for decode.
//
//     S_t = e^l S_{t-1} + v_t k_t^T   (S[v][k], FP32),      o_t = s S_t q_t
//
// with one log-decay l <= 0 per value head.  Its adjoint is
//     dS_t = s do_t q_t^T + e^l dS_{t+1},   dq_t = s S_t^T do_t,
//     dk_t = dS_t^T v_t,   dv_t = dS_t k_t,   dS_0 = e^l dS_1,
// so o, dq, dk and dv are one causal form over rows a, b, c (128 channels):
//     y_i = sum_{j<=i} e^{l(i-j)} (a_i.b_j) c_j + e^{l(i+shift)} a_i X
// with (a, b, c) = (q, k, v) and (do, v, k) forward in time (X the initial
// state, shift 1), and (v, do, q) and (k, q, do) backward in time (X the
// final state's adjoint, shift 0).  One kernel computes all four.
#include "kda_chunk.hpp"
#include "kda_common.hpp"
#include "kda_layers.h"

namespace kda {

namespace {

constexpr int SC = 32;            // tokens per chunk
constexpr int STATE = D * D;

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

struct Item {
    int64_t tok0;     // first token (flattened)
    int len;          // tokens
    int n, h;
    int64_t seg;      // segment number among all segments (segmented maps)
};

__device__ __forceinline__ int64_t uniform64(int64_t x) {
    const unsigned lo = __builtin_amdgcn_readfirstlane((int)(unsigned)x);
    const int hi = __builtin_amdgcn_readfirstlane((int)(x >> 32));
    return ((int64_t)hi << 32) | lo;
}

__device__ __forceinline__ Item find_item(const ItemMap& m, int64_t i) {
    Item it;
    const int64_t r = i / m.Hv;
    const int lead = (int)r;   // sequence, or place in the segment list
    it.h = (int)(i - r * m.Hv);
    it.seg = 0;
    int j = 0;
    if (m.task == nullptr) {
        it.n = lead;
        if (m.seg_len > 0) {
            const int per = (m.len + m.seg_len - 1) / m.seg_len;
            it.n = lead / per;
            j = lead - it.n * per;
            it.seg = lead;
        }
        it.tok0 = (int64_t)it.n * m.len;
        it.len = m.len;
    } else if (m.seg_len > 0) {
        it.n = m.seg[2 * lead];
        j = m.seg[2 * lead + 1];
        it.seg = m.tape_off[it.n] + it.n + j;
        it.tok0 = m.seq_start[it.n];
        it.len = m.seq_len[it.n];
    } else {
        const int code = m.task[i];
        it.n = code / m.Hv;
        it.h = code - it.n * m.Hv;
        it.tok0 = m.seq_start[it.n];
        it.len = m.seq_len[it.n];
    }
    if (m.seg_len > 0) {
        it.tok0 += (int64_t)j * m.seg_len;
        it.len = min(m.seg_len, it.len - j * m.seg_len);
    }
    // the same for the whole workgroup: keep it in scalar registers
    it.n = __builtin_amdgcn_readfirstlane(it.n);
    it.h = __builtin_amdgcn_readfirstlane(it.h);
    it.len = __builtin_amdgcn_readfirstlane(it.len);
    it.tok0 = uniform64(it.tok0);
    it.seg = uniform64(it.seg);
    return it;
}

// l in base 2, kept finite so that 0 * l is 0 for l = -inf (a NaN stays one).
__device__ __forceinline__ float log2_decay(float l) {
    const float x = l * LOG2E;
    return x < -1e30f ? -1e30f : x;
}
__device__ __forceinline__ double decay_power(float l, int n) {  // e^{l n}, n >= 0
    return n == 0 ? 1.0 : exp((double)l * n);
}

// A decay that a state is multiplied by over and over, by segments, tokens or calls:
// rounded to one FP32 value it would be off the same way every time, and the state
// would drift.  It is applied as the sum of two, to 2^-48 of itself.
struct Factor {
    float f, low;
    __device__ __forceinline__ explicit Factor(double x) : f((float)x), low((float)(x - (double)(float)x)) {}
    // x times the factor, plus y
    __device__ __forceinline__ float apply(float x, float y) const { return fmaf(x, f, fmaf(x, low, y)); }
    __device__ __forceinline__ float apply(float x) const { return fmaf(x, f, x * low); }
};

// LDS rows of 128 channels are 16 blocks of 8 channels; block b of row r is
// stored at block b ^ swz(r).  The 16 rows of a tile then hold one block in 16
// places, and a transposing read (4 rows of each of 4 groups, two blocks a
// row) covers all 64 banks with every 32 lanes.
__device__ __forceinline__ int swz(int r) { return ((r & 3) << 2) | ((r >> 1) & 2) | ((r >> 3) & 1); }

// Transposing read: the 16 lanes of group gq address 4 rows x 4 pieces of 4
// channels, and lane m receives the 4 rows of channel m of those 16.
__device__ __forceinline__ bf16x4 tr_read(const char* p) {
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)p));
}

// A load or store at a uniform address plus a 32-bit lane offset: the address
// is pinned to scalar registers, where it would otherwise be kept as one
// 64-bit vector per row.
template <class T>
__device__ __forceinline__ __attribute__((address_space(1))) T* row_ptr(const void* base, unsigned off) {
    uint64_t b = (uint64_t)base;
    asm volatile("" : "+s"(b));
    return (__attribute__((address_space(1))) T*)((__attribute__((address_space(1))) char*)b + off);
}

// Moves 16 bytes per lane from base + off (off per lane) to LDS at dst (uniform)
// + 16 lane; kStream: non-temporal.
template <bool kStream>
__device__ __forceinline__ void to_lds(const char* base, unsigned off, char* dst) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)row_ptr<const char>(base, off),
                                     (__attribute__((address_space(3))) void*)dst, 16, 0, kStream ? 2 : 0);
}
// Waits until at most N of this wave's vector memory operations are outstanding.
template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("" ::: "memory");   // what was issued before it stays before it
    __builtin_amdgcn_s_waitcnt((N & 15) | 0x0f70 | (N >> 4) << 14);
}
// Workgroup barrier for LDS contents: this wave's LDS operations are complete
// before it; memory operations stay on their side of it.  (__syncthreads would
// also wait for the stores to global memory.)
__device__ __forceinline__ void barrier_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// x, as a value the compiler cannot know to be the same in every loop round:
// what is formed from it is formed where it is used instead of being kept in
// registers over the loop.
__device__ __forceinline__ int fresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// Takes the leading 8 significant bits of every element off x and returns
// them as BF16 (the remainder is exact).
__device__ __forceinline__ bf16x4 take_high(f32x4& x) {
    const u32x4 u = __builtin_bit_cast(u32x4, x) & 0xffff0000u;
    x -= __builtin_bit_cast(f32x4, u);
    return __builtin_bit_cast(bf16x4, u32x2{__builtin_amdgcn_perm(u[1], u[0], 0x07060302u),
                                            __builtin_amdgcn_perm(u[3], u[2], 0x07060302u)});
}

}  // namespace

// A partial of dq or dk (value heads that share a q/k head each form one) is
// kept as quads of 8 bytes: four 15-bit floats (sign, 5 bits of exponent, 9 of
// mantissa) and 4 bits that scale the quad by a power of 2^16 so that its
// largest value is in [1/2, 2^15).  A value is rounded once, to nearest: off by at
// most 2^-10 of itself, a quarter of a BF16 rounding, or 2^-23 of the quad's
// largest.  (As FP32 the partials' way out and in took 28% of a grouped training
// step then, and BF16 partials would add as large an error again as the result's own
// rounding.)  A quad with a NaN or an infinity comes back as NaN.
__device__ __forceinline__ u32x2 pack_quad(f32x4 x) {
    const float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    const unsigned q = __float_as_uint(top) >> 27;                 // biased exponent / 16
    const float scale = __uint_as_float((253u - 16u * q) << 23);   // 2^(126 - 16q)
    // (the maxima skip NaN; 0 x is 0 for finite x only)
    const bool bad = !(x[0] * 0.0f + x[1] * 0.0f + x[2] * 0.0f + x[3] * 0.0f == 0.0f);
    unsigned m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // to 10 significant bits, or below FP16's normal values to a multiple of
        // 2^-23 (a last bit of 1.5): an FP16 value with its lowest bit clear
        const float v = x[i] * scale;
        const unsigned u = __float_as_uint(v);
        const float r = fabsf(v) < 0x1p-14f ? (v + 1.5f) - 1.5f
                                            : __uint_as_float((u + 0x1fffu + (u >> 14 & 1u)) & ~0x3fffu);
        m[i] = (unsigned)__builtin_bit_cast(unsigned short, (f16)r) >> 1;
    }
    const u32x2 w = {m[0] | m[1] << 15 | q << 30, m[2] | m[3] << 15 | (q >> 2) << 30};
    return u32x2{bad ? ~0u : w[0], bad ? ~0u : w[1]};
}
__device__ __forceinline__ f32x4 unpack_quad(u32x2 w) {
    const unsigned q = w[0] >> 30 | (w[1] >> 30) << 2;
    const float scale = __uint_as_float((1u + 16u * q) << 23);     // 2^(16q - 126)
    f32x4 x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        x[2 * i] = scale * (float)__builtin_bit_cast(f16, (unsigned short)(w[i] << 1));
        x[2 * i + 1] = scale * (float)__builtin_bit_cast(f16, (unsigned short)(w[i] >> 14 & 0xfffeu));
    }
    return x;
}

// One workgroup per item and form (kParts = 2: two, each with half of the
// state's output channels), a wave for every NU tiles of 16 channels.  Wave
// wv holds the state as MFMA accumulators: tile (t, u) is S^T[k][v] with
//     k = 32(t/2) + 8gq + 4(t%2) + e,   v = 32wv + 8(n/4) + 4u + n%4
// (NU = 1: v = 16wv + n; lane 16gq + n, element e), so that tiles t = 2p and
// 2p+1 together are, as BF16, the operand of S a over channels 32p ..
// 32p+31 in the order in which one 16-byte read takes them from a's rows, and
// the two tiles u of Y^T give a lane 8 neighbouring channels of one token to
// store (8-byte stores cost the packed forward 4%, the training step 7% then).  Per
// chunk of 32 tokens:
//     P^T = B A^T (16x16 tiles with j <= i, times s e^{l(i-j)})
//     Y^T = (S A^T) diag(e^{l(i+shift)}) + C^T P^T
//     S^T = e^{32 l} S^T + B^T (C u),   u_j = e^{l(32-shift-j)}
// The state is kept divided by the decay since it was last rescaled, so that
// most chunks only add to it (weights u_j over that decay) and y takes the
// decay as one more factor; it is rescaled when the decay falls below 2^-24.
// P, and S where it meets a, go in as two BF16 pieces, off by at most 2^-18 of
// themselves, so that the output's own rounding is the only one to be seen.
// (Rounded to BF16 each would add as large an error as that rounding: o, dq, dk
// and dv were off by 2.35e-3 of their norm instead of 1.66e-3.  P's second piece
// takes 1% of a packed training step, S's 11%, half of it in the products and
// half in taking S apart.)  The FP32 products C u go in as three BF16 pieces of 8
// significant bits each, so exactly; the state itself stays in FP32 registers.
//
// The rows of the next chunk travel from memory to the other of two LDS
// buffers, without passing through registers, while this one is computed:
//     before the first barrier   P^T (one tile in each of three waves) and the
//                                state's part of Y
//     before the second          C^T P^T, stores, the state's update
// Two buffers and at most 168 registers let three workgroups share a compute
// unit.  The forward of 8 x 1024 tokens of 96 heads takes 191 to 205 us: 907 MB, each
// row read once, at 4.4 to 4.7 TB/s, with the vector units issuing 65% and the matrix
// units busy 44% of the time, so that neither memory nor arithmetic has much room left.
// (Rows of 96 heads, 24 KB apart, put a head's b, c and a on the same few
// memory channels: with room for 97 heads a row it takes 13 us less.)  A single
// workgroup waits for itself, so with one per unit (kDeep) a chunk's LDS reads
// are issued together, ahead of the next chunk's loads, and half of the state's
// update moves before the first barrier (2048 tokens of 48 heads 98 us instead of 100,
// of 16 heads 93 instead of 97).  `reverse` walks the tokens downwards and only shifts the
// exponents.
template <int NU, int kParts, bool kOut, bool kPack, bool kStream = false>
__global__ __launch_bounds__(512 / NU / kParts, NU == 2 ? 3 : kParts == 2 ? 2 : 4) void decay_scan_kernel(ScanArgs A) {
    // LDS (bytes): the rows of b, c and a, two buffers each that differ in address
    // bit SET; the P^T tiles
    constexpr int SETS = kOut ? 3 : 2, SET = SC * D * 2, LB = 0, LC = 2 * SET, LA = 4 * SET, LPT = 1024;
    constexpr int ROWS16 = 16 * D * 2;
    __shared__ __align__(16) char lds[2 * SETS * SET];
    __shared__ __align__(16) char lds_p[kOut ? 3 * LPT : 16];

    const int tid = threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63, gq = lane >> 4, n16 = lane & 15;
    int idx = xcd_order(blockIdx.x, (int)gridDim.x, A.share * kParts);
    const int part = idx % kParts;
    idx /= kParts;
    const int wv = w + 8 / NU / kParts * part;   // this wave among the columns
    const ScanJob J = A.job[A.jobs == 1 ? 0 : idx % A.jobs];
    const Item it = find_item(A.map, idx / A.jobs);
    const int64_t slot = A.slot != nullptr ? A.slot[it.n] : it.n;
    if (slot < 0 || slot >= A.slots) return;
    const int64_t sidx = A.by_seg ? it.seg : slot;
    const int Hv = A.map.Hv;
    const int64_t soff = (sidx * Hv + it.h) * (int64_t)STATE;
    const bool rev = J.reverse != 0;
    const float l = A.log_decay[it.h];
    const float l2 = log2_decay(l);
    const int shift = rev ? 0 : 1;
    const float scale = A.scale;
    const float y_state = rev ? 1.0f : scale;     // scale of the state's part of y
    const float s_add = rev ? scale : 1.0f;       // scale of what the state takes up

    // Loads: one instruction of a wave moves 4 rows of 256 bytes (16 lanes a
    // row) to 1 KiB of LDS in lane order; a lane fetches the block that belongs
    // there.  Wave w takes rows 4w .. 4w+3 (and, with four waves, 16 more).  The address
    // is a uniform base (the chunk's lowest row) plus a 32-bit lane offset.
    const int64_t first = rev ? it.tok0 + it.len - 1 : it.tok0;
    const int64_t dir = rev ? -1 : 1;
    const int lrow = 4 * w + gq;
    constexpr int STEP = 32 / NU / kParts;   // rows that one instruction of every wave covers
    const ScanRows rows[3] = {J.b, J.c, J.a};
    const char* pr[SETS];
    int64_t bytes[SETS];
    unsigned off[SETS];
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
        bytes[i] = rows[i].stride * 2;
        pr[i] = (const char*)(rows[i].p + (it.h / rows[i].group) * D) + (first - (rev ? STEP - 1 : 0)) * bytes[i];
        off[i] = (unsigned)(rev ? STEP - 1 - lrow : lrow) * (unsigned)bytes[i] + ((n16 ^ swz(lrow)) << 4);
    }
    auto fetch = [&](char* buf, int at, int t0) __attribute__((always_inline)) {
        const int rem = it.len - t0;
#pragma unroll
        for (int j = 0; j < NU * kParts; ++j) {
            if (rem >= SC || lrow + 16 * j < rem) {
#pragma unroll
                for (int i = 0; i < SETS; ++i)
                    to_lds<kStream>(pr[i] + j * 16 * dir * bytes[i], off[i], buf + at + 2 * i * SET + (16 * j + 4 * w) * D * 2);
            } else {   // rows behind the last token are not read and count as zero
#pragma unroll
                for (int i = 0; i < SETS; ++i)
                    *(u32x4*)(buf + at + 2 * i * SET + (16 * j + 4 * w) * D * 2 + lane * 16) = u32x4{0u, 0u, 0u, 0u};
            }
        }
#pragma unroll
        for (int i = 0; i < SETS; ++i) pr[i] += SC * dir * bytes[i];
    };
    fetch(lds, 0, 0);

    // state
    f32x4 S[8][NU];
    const int vrow = NU == 2 ? 32 * wv + 8 * (n16 >> 2) + (n16 & 3) : 16 * wv + n16;   // + 4u
    auto krow = [&](int t) __attribute__((always_inline)) { return 32 * (t >> 1) + 8 * gq + 4 * (t & 1); };
    const float* s_in = J.s_in;
    if (s_in == nullptr) {
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int u = 0; u < NU; ++u) S[t][u] = zero4();
    } else if (!J.s_in_t) {
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int u = 0; u < NU; ++u)
                S[t][u] = *(const f32x4*)(s_in + soff + (vrow + 4 * u) * D + krow(t));
    } else {
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    S[t][u][e] = s_in[soff + (krow(t) + e) * D + vrow + 4 * u];
    }

    // Powers of e^l, constant over the item's full chunks; each is a product
    // of factors <= 1, so none overflows.  P^T tiles: wave 0 (i, j) = (0, 0),
    // wave 1 (1, 1), wave 2 (1, 0).
    //     P^T at i - j = 16d + n - 4gq - e:   pf[e] (d = 1 in wave 2, else 0)
    //     Y column i = 16ti + n:              y0 (times far for ti = 1)
    //     C row j = 16tj + 4gq + e:           u0[tj][e]
    const float far = __int_as_float(__builtin_amdgcn_readfirstlane(
        __float_as_int(__builtin_amdgcn_exp2f(l2 * 16.0f))));
    const float y0 = y_state * __builtin_amdgcn_exp2f(l2 * (float)(n16 + shift));
    float pf[4], u0[2][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        pf[e] = scale * __builtin_amdgcn_exp2f(l2 * (float)max((w == 2 ? 16 : 0) + n16 - 4 * gq - e, 0));
        u0[1][e] = s_add * __builtin_amdgcn_exp2f(l2 * (float)(16 - shift - 4 * gq - e));
        u0[0][e] = u0[1][e] * far;
    }
    // the state is `held` times S; a chunk's decay and its inverse
    const double lam = decay_power(l, SC), inv = 1.0 / lam;
    double held = 1.0, over = 1.0;   // over = 1 / held
    // chunks until that is below 2^-24 (at least one)
    const int every = __builtin_amdgcn_readfirstlane((int)fminf(24.0f / (SC * fabsf(l2)), 0x1p30f)) + 1;
    int left = every;

    // LDS offsets (bytes) for p = 0, where an xor of 64p gives the others: 8
    // channels (32p + 8gq) of row n, and for the transposing reads of row
    // 4gq + n/4 the piece a = n%4, channels 32p + 8a .. +3 (+ 4 for odd tiles) of b
    // and 32wv + 8a .. +3 (NU = 1: 16wv + 4a) of c
    const int r8_ = (n16 * D + ((gq ^ swz(n16)) << 3)) * 2;
    const int trow = 4 * gq + (n16 >> 2), piece = n16 & 3;
    const int tr_ = (trow * D + ((piece ^ swz(trow)) << 3)) * 2;
    const int trc_ = NU == 2 ? (trow * D + (((4 * wv + piece) ^ swz(trow)) << 3)) * 2
                             : (trow * D + (((2 * wv + (piece >> 1)) ^ swz(trow)) << 3) + 4 * (piece & 1)) * 2;
    // output rows of 16 tokens: a uniform base and a 32-bit lane offset
    const int64_t sy = (int64_t)Hv * D * 2, gy = 16 * dir * sy;
    const char* yout = (const char*)J.y;
    const bool pack = J.pack != 0;
    int64_t py = ((first - (rev ? 15 : 0)) * Hv + it.h) * D * 2;
    const unsigned oy = (unsigned)(rev ? 15 - n16 : n16) * (unsigned)sy + (16 * NU * wv + 4 * NU * gq) * 2;

    // One chunk, from `buf` + at, the next one's rows on their way into `other` +
    // (SET - at).  (Both are `lds`; as restrict pointers they show the compiler
    // that what is read through the one need not wait for what is on its way
    // into the other.)
    auto chunk = [&](int t0, int at, const char* __restrict__ buf, char* __restrict__ other,
                     auto tail_c) __attribute__((always_inline)) {
        constexpr bool kTail = decltype(tail_c)::value, kDeep = NU == 1 && kParts == 2;
        const int rem = kTail ? it.len - t0 : SC;
        const bool more = !kTail && t0 + SC < it.len;
        if (!kDeep && more) fetch(other, SET - at, t0 + SC);
        // (formed anew per chunk, rather than kept in a register each)
        const int r8 = fresh(r8_) + at, tr = fresh(tr_) + at, trc = fresh(trc_) + at;
        const float y_held = (float)held * y0;
        const double d = kTail ? decay_power(l, rem) : lam;
        held *= d;
        over = kTail ? over / d : over * inv;
        const bool rescale = --left == 0;
        const float down = (float)held;
        if (rescale) {
            held = over = 1.0;
            left = every;
        }
        const float g = (float)over;

        f32x4 y[2][NU];
        bf16x8 av[4][2], bt[8], pb[4];
        bf16x4 cf[2][NU];
        const int r8p = r8 + (w == 1 ? ROWS16 : 0);
        auto read_p = [&](int p) __attribute__((always_inline)) {
            pb[p] = *(const bf16x8*)(buf + (r8p ^ (64 * p)) + LB);
        };
        auto read_a = [&](int p) __attribute__((always_inline)) {
#pragma unroll
            for (int ti = 0; ti < 2; ++ti)
                av[p][ti] = *(const bf16x8*)(buf + (r8 ^ (64 * p)) + LA + ti * ROWS16);
        };
        auto read_b = [&](int t) __attribute__((always_inline)) {
            const char* row = buf + (tr ^ (64 * (t >> 1))) + LB + 8 * (t & 1);
            bt[t] = cat8(tr_read(row), tr_read(row + ROWS16));
        };
        auto read_c = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int u = 0; u < NU; ++u) cf[j][u] = tr_read(buf + trc + LC + 8 * u + ROWS16 * j);
        };
        if (kDeep) {   // all of the chunk's reads at once, before the next chunk's loads are issued
            if (kOut) {
#pragma unroll
                for (int p = 0; p < 4; ++p) read_a(p);
                if (w < 3) {
#pragma unroll
                    for (int p = 0; p < 4; ++p) read_p(p);
                }
            }
            read_c();
#pragma unroll
            for (int t = 0; t < 8; ++t) read_b(t);
            __builtin_amdgcn_sched_barrier(0);
            if (more) fetch(other, SET - at, t0 + SC);
        }
        if (kOut) {
            if (w < 3) {   // this wave's P^T tile
                f32x4 acc = zero4();
                if (kDeep && w == 0) {
#pragma unroll
                    for (int p = 0; p < 4; ++p) acc = mma32(pb[p], av[p][0], acc);
                } else if (kDeep) {
#pragma unroll
                    for (int p = 0; p < 4; ++p) acc = mma32(pb[p], av[p][1], acc);
                } else {
                    const int r8a = r8 + (w == 0 ? 0 : ROWS16);
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        read_p(p);
                        acc = mma32(pb[p], *(const bf16x8*)(buf + (r8a ^ (64 * p)) + LA), acc);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // a later token's row never counts, whatever it holds
                    const bool seen = (w == 2) | (n16 >= 4 * gq + e);
                    acc[e] = seen ? acc[e] * pf[e] : 0.0f;
                }
                bf16x4 hi, lo;
                split4_rne(acc, hi, lo);
                *(bf16x8*)(lds_p + w * LPT + lane * 16) = cat8(hi, lo);
            }
#pragma unroll
            for (int ti = 0; ti < 2; ++ti)
#pragma unroll
                for (int u = 0; u < NU; ++u) y[ti][u] = zero4();
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                if (!kDeep) read_a(p);
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                    bf16x4 hi[2], lo[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) split4_rne(S[2 * p + i][u], hi[i], lo[i]);
                    const bf16x8 s1 = cat8(hi[0], hi[1]), s2 = cat8(lo[0], lo[1]);
#pragma unroll
                    for (int ti = 0; ti < 2; ++ti) y[ti][u] = mma32(s1, av[p][ti], y[ti][u]);
#pragma unroll
                    for (int ti = 0; ti < 2; ++ti) y[ti][u] = mma32(s2, av[p][ti], y[ti][u]);
                }
            }
        }
        // the pieces of C u
        bf16x8 c1[NU], c2[NU], c3[NU];
        auto form_pieces = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                bf16x4 x1[2], x2[2], x3[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    f32x4 c = from_bf4(cf[j][u]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        c[e] *= g * (kTail ? s_add * __builtin_amdgcn_exp2f(
                                                         l2 * (float)max(rem - shift - 16 * j - 4 * gq - e, 0))
                                           : u0[j][e]);
                    x1[j] = take_high(c);
                    x2[j] = take_high(c);
                    x3[j] = to_bf4(c);
                }
                c1[u] = cat8(x1[0], x1[1]);
                c2[u] = cat8(x2[0], x2[1]);
                c3[u] = cat8(x3[0], x3[1]);
            }
        };
        auto update = [&](int from, int to) __attribute__((always_inline)) {
#pragma unroll
            for (int t = from; t < to; ++t) {
                if (!kDeep) read_b(t);
#pragma unroll
                for (int u = 0; u < NU; ++u) S[t][u] = mma32(bt[t], c1[u], S[t][u]);
#pragma unroll
                for (int u = 0; u < NU; ++u) S[t][u] = mma32(bt[t], c2[u], S[t][u]);
#pragma unroll
                for (int u = 0; u < NU; ++u) S[t][u] = mma32(bt[t], c3[u], S[t][u]);
            }
        };
        auto rescale_state = [&]() __attribute__((always_inline)) {
            if (rescale) {
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int u = 0; u < NU; ++u)
#pragma unroll
                        for (int e = 0; e < 4; ++e) S[t][u][e] *= down;
            }
        };
        if (kDeep) {   // half of the update beside P^T, the other half beside what follows it
            rescale_state();
            form_pieces();
            update(0, 4);
        }
        if (kOut) barrier_lds();
        if (!kDeep) {
            rescale_state();
            read_c();
        }
        if (kOut) {
            // 4 rows of a tile each, first pieces before second ones
            const bf16x8 p00 = *(const bf16x8*)(lds_p + lane * 16), p11 = *(const bf16x8*)(lds_p + LPT + lane * 16),
                         p10 = *(const bf16x8*)(lds_p + 2 * LPT + lane * 16);
            const bf16x8 p1h = __builtin_shufflevector(p10, p11, 0, 1, 2, 3, 8, 9, 10, 11),
                         p1l = __builtin_shufflevector(p10, p11, 4, 5, 6, 7, 12, 13, 14, 15);
            const float yf[2] = {y_held, y_held * far};
            const char* yb = yout + py;
#pragma unroll
            for (int u = 0; u < NU; ++u) {
#pragma unroll
                for (int ti = 0; ti < 2; ++ti)
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[ti][u][e] *= yf[ti];
                const bf16x8 c = cat8(cf[0][u], cf[1][u]);
                y[0][u] = mma32(cat8(cf[0][u], cf[0][u]), p00, y[0][u]);   // both pieces in one product
                y[1][u] = mma32(c, p1h, y[1][u]);
                y[1][u] = mma32(c, p1l, y[1][u]);
            }
#pragma unroll
            for (int ti = 0; ti < 2; ++ti) {
                u32x2 q[NU];
#pragma unroll
                for (int u = 0; u < NU; ++u)
                    q[u] = kPack && pack ? pack_quad(y[ti][u]) : __builtin_bit_cast(u32x2, to_bf4(y[ti][u]));
                if (!kTail || 16 * ti + n16 < rem) {
                    if constexpr (NU == 2)
                        *row_ptr<u32x4>(yb + ti * gy, oy) = u32x4{q[0][0], q[0][1], q[1][0], q[1][1]};
                    else
                        *row_ptr<u32x2>(yb + ti * gy, oy) = q[0];
                }
            }
            py += 2 * gy;
        }
        if (!kDeep) form_pieces();
        update(kDeep ? 4 : 0, 8);
        if (!kTail) {
            // the next chunk's rows have arrived when at most this chunk's two
            // stores, issued after them, are outstanding (they complete in order)
            if (kOut)
                wait_vm<2>();
            else
                wait_vm<0>();
            barrier_lds();
        }
    };
    wait_vm<0>();
    barrier_lds();
    int t0 = 0, at = 0;
    for (; t0 + SC <= it.len; t0 += SC) {
        chunk(t0, at, lds, lds, std::false_type{});
        at = SET - at;
    }
    if (t0 < it.len) chunk(t0, at, lds, lds, std::true_type{});

    float* s_out = J.s_out;
    if (s_out != nullptr) {
        const Factor decay(held);
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                f32x4 x;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = decay.apply(S[t][u][e]);
                *(f32x4*)(s_out + soff + (vrow + 4 * u) * D + krow(t)) = x;
            }
    }
}

template <int NU, int kParts>
static void launch_scan(const ScanArgs& a, bool states_only, bool pack, hipStream_t s) {
    const dim3 grid((unsigned)(a.map.items * a.jobs * kParts)), block(512 / NU / kParts);
    if (states_only)
        hipLaunchKernelGGL((decay_scan_kernel<NU, kParts, false, false>), grid, block, 0, s, a);
    else if (pack)
        hipLaunchKernelGGL((decay_scan_kernel<NU, kParts, true, true>), grid, block, 0, s, a);
    else if (a.stream)
        hipLaunchKernelGGL((decay_scan_kernel<NU, kParts, true, false, NU == 2>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((decay_scan_kernel<NU, kParts, true, false>), grid, block, 0, s, a);
}

// With enough workgroups to share compute units, four waves with two tiles
// each spend the least on reading the rows out of LDS.  With one workgroup per
// unit at most, eight waves shorten a chunk, and with one for every second
// unit, two workgroups of half the columns each.  Forward in us (four waves;
// eight waves; halves): 48 workgroups of 2048 tokens 137, 113, 99; 128 134, 110, 98;
// 150 135, 118, 134; 192 140, 127, 140; 256 141, 138, 155; 288 195, 202, -; 384 207, 218,
// -.  Backward, three workgroups a (sequence, head), whose walks differ: 144 of 2048
// tokens 139, 118, 126; 288 of 4096 386, 367, -; 384 of 4096 with shared heads 510, 473,
// -; 432 of 2048 212, 209, -; 504 229, 230, -; 576 286, 293, 316.
hipError_t launch_decay_scan(const ScanArgs& a, bool states_only, hipStream_t s) {
    bool pack = false;
    for (int i = 0; i < a.jobs; ++i) pack = pack || a.job[i].pack != 0;
    const int64_t groups = a.map.items * a.jobs;
    if (groups <= 128)
        launch_scan<1, 2>(a, states_only, pack, s);
    else if (groups <= (a.jobs == 3 ? 400 : 256))
        launch_scan<1, 1>(a, states_only, pack, s);
    else
        launch_scan<2, 1>(a, states_only, pack, s);
    return hipGetLastError();
}

// Chains the segments of each (sequence, value head): with R_j the own sum of
// segment j (its state from zero), the state before it in walking order is
// X_{j+1} = R_j + e^{l len_j} X_j.  Element by element: one thread per four
// elements, the sums of the next four segments on their way.  (16 heads x 32
// segments, 67 MB: 15.3 us one segment ahead, 13.6 us four ahead.)
__global__ __launch_bounds__(256) void decay_chain_kernel(ChainArgs A) {
    const ItemMap& m = A.map;
    const ChainJob& J = A.job[blockIdx.y];
    constexpr int AHEAD = 4;
    const int64_t task = blockIdx.x >> 4;   // 16 blocks of 1024 elements per state
    const int n = (int)(task / m.Hv), h = (int)(task - (int64_t)n * m.Hv);
    const int e = (int)(blockIdx.x & 15) * 1024 + threadIdx.x * 4;
    const int64_t slot = A.slot != nullptr ? A.slot[n] : n;
    if (slot < 0 || slot >= A.slots) return;
    const int64_t at = (slot * m.Hv + h) * (int64_t)STATE + e;
    const int len = m.task != nullptr ? m.seq_len[n] : m.len;
    if (len <= A.skip) return;
    const int segs = (len + m.seg_len - 1) / m.seg_len;
    const int64_t base = m.task != nullptr ? m.tape_off[n] + n : (int64_t)n * segs;
    const float l = A.log_decay[h];
    const Factor full(decay_power(l, m.seg_len)), last(decay_power(l, len - (segs - 1) * m.seg_len));
    f32x4 x = J.s_in != nullptr ? *(const f32x4*)(J.s_in + at) : zero4();
    const int64_t step = (int64_t)m.Hv * STATE;
    float* p = J.seg + (base * m.Hv + h) * STATE + e;
    auto place = [&](int i) __attribute__((always_inline)) { return J.reverse ? segs - 1 - i : i; };
    auto sum = [&](int i) __attribute__((always_inline)) { return *(const f32x4*)(p + place(min(i, segs - 1)) * step); };
    f32x4 next[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) next[u] = sum(u);
    for (int i = 0; i < segs; i += AHEAD) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (i + u >= segs) break;
            const int j = place(i + u);
            const f32x4 r = next[u];
            next[u] = sum(i + u + AHEAD);   // (behind the last: not used)
            *(f32x4*)(p + j * step) = x;
#pragma unroll
            for (int c = 0; c < 4; ++c) x[c] = (j == segs - 1 ? last : full).apply(x[c], r[c]);
        }
    }
    if (J.s_out != nullptr) *(f32x4*)(J.s_out + at) = x;
}

hipError_t launch_decay_chain(const ChainArgs& a, hipStream_t s) {
    const int64_t blocks = (int64_t)a.map.N * a.map.Hv * 16;
    hipLaunchKernelGGL(decay_chain_kernel, dim3((unsigned)blocks, a.jobs), dim3(256), 0, s, a);
    return hipGetLastError();
}

// Token-serial form on the FP32 state pool (decode, and sequences of a few
// tokens).  A workgroup takes 32 of the 128 state rows of one (sequence,
// value head): a half wave holds a row (4 channels a lane), each wave 4 pairs
// of rows, so every load and store moves 1 KiB of contiguous state, and o is
// a sum over the half wave.  No LDS, no barrier; everything FP32.  (With a decay
// rounded to one FP32 value a decode of 65536 tokens at l = -3.3e-5 would end 1.4e-3
// off.)  Bound by the
// state's way in and out; non-temporal (kStream) when that exceeds kStreamBytes:
// 128 sequences of 64 heads 205 -> 179 us, 64 of them 105 -> 91 us, 32 of them
// (268 MB) 46 us either way.
template <bool kStream>
__global__ __launch_bounds__(256) void decay_token_kernel(TokenArgs A) {
    const Item it = find_item(A.map, blockIdx.x >> 2);
    const int64_t slot = A.slot != nullptr ? A.slot[it.n] : it.n;
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
    const Factor decay(decay_power(A.log_decay[it.h], 1));
    const int hq = it.h / A.G;
    const bf16* q = (const bf16*)A.q + it.tok0 * A.sq + hq * D + ch;
    const bf16* k = (const bf16*)A.k + it.tok0 * A.sk + hq * D + ch;
    const bf16* v = (const bf16*)A.v + it.tok0 * A.sv + it.h * D + row0;
    bf16* o = (bf16*)A.o + (it.tok0 * Hv + it.h) * D + row0;
    for (int t = 0; t < it.len; ++t) {
        const f32x4 qf = from_bf4(*(const bf16x4*)(q + t * A.sq));
        const f32x4 kf = from_bf4(*(const bf16x4*)(k + t * A.sk));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float vj = (float)v[t * A.sv + 8 * j];
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[j][e] = fmaf(vj, kf[e], decay.apply(x[j][e]));
                sum += x[j][e] * qf[e];
            }
            sum = row16_sum(sum);
            sum += __shfl_xor(sum, 16, 64);
            if ((lane & 31) == 0) o[(int64_t)t * Hv * D + 8 * j] = (bf16)(A.scale * sum);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f32x4* p = (f32x4*)(S + (row0 + 8 * j) * D);
        if (kStream)
            __builtin_nontemporal_store(x[j], p);
        else
            *p = x[j];
    }
}

hipError_t launch_decay_token(const TokenArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.map.items * 4));
    if (2 * a.map.items * STATE * 4 > kStreamBytes)
        hipLaunchKernelGGL((decay_token_kernel<true>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((decay_token_kernel<false>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

// Sum over the G value heads of a q/k head, in head order, packed partials to
// BF16: 8 channels (two quads) per thread.
__global__ __launch_bounds__(256) void decay_group_sum_kernel(const bf16* src0, const bf16* src1, bf16* dst0,
                                                              bf16* dst1, int64_t vecs, int G) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;   // (token, q/k head, 8 channels)
    if (i >= vecs) return;
    const int64_t row = i >> 4;
    const int c = (int)(i & 15) * 8;
    const bf16* src = (blockIdx.y ? src1 : src0) + row * G * D + c;
    f32x4 a = zero4(), b = zero4();
    for (int g = 0; g < G; ++g) {
        const u32x4 w = *(const u32x4*)(src + g * D);
        a += unpack_quad(u32x2{w[0], w[1]});
        b += unpack_quad(u32x2{w[2], w[3]});
    }
    *(bf16x8*)((blockIdx.y ? dst1 : dst0) + row * D + c) = cat8(to_bf4(a), to_bf4(b));
}

hipError_t launch_decay_group_sum(const void* src0, const void* src1, bf16_t* dst0, bf16_t* dst1,
                                  int64_t tokens, int Hqk, int G, hipStream_t s) {
    const int64_t vecs = tokens * Hqk * (D / 8);
    hipLaunchKernelGGL(decay_group_sum_kernel, dim3((unsigned)((vecs + 255) / 256), 2), dim3(256), 0, s,
                       (const bf16*)src0, (const bf16*)src1, (bf16*)dst0, (bf16*)dst1, vecs, G);
    return hipGetLastError();
}

}  // namespace kda
