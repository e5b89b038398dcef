// Device helpers shared by the scans over token rows (kda_decay.hip, kda_delta.hip): work
// items, LDS rows and their transposing reads, loads straight to LDS, waits, and FP32
// values taken apart into BF16 pieces.
#pragma once

#include "kda_chunk.hpp"
#include "kda_common.hpp"
#include "kda_layers.h"

namespace kda {

constexpr int STATE = D * D;

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

struct Item {
    int64_t tok0;     // first token (flattened)
    int len;          // tokens
    int n, h;
    int64_t seg;      // segment number among all segments (segmented maps)
    int64_t off;      // tokens of the sequence before tok0
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
    it.off = (int64_t)j * m.seg_len;
    if (m.seg_len > 0) {
        it.tok0 += it.off;
        it.len = min(m.seg_len, it.len - j * m.seg_len);
    }
    // the same for the whole workgroup: keep it in scalar registers
    it.n = __builtin_amdgcn_readfirstlane(it.n);
    it.h = __builtin_amdgcn_readfirstlane(it.h);
    it.len = __builtin_amdgcn_readfirstlane(it.len);
    it.tok0 = uniform64(it.tok0);
    it.seg = uniform64(it.seg);
    it.off = uniform64(it.off);
    return it;
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

}  // namespace kda
