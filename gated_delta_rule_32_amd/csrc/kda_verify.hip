// Verification of drafted tokens.  With the target's probabilities p, the draft's q and
// given random numbers, draft i of a sequence stands while u_i q_i(x_i) < p_i(x_i); behind
// the last one that stands, one token is drawn from max(p - q, 0) (from p behind the last
// draft, or where p exceeds q nowhere): the first index whose running sum passes u times the total.
//
// Products and sums are formed in 64 bits, where the product of two FP32 values is exact, so
// that a token depends neither on how the row is split nor on the order of its sums (beyond
// 2^-50 of the total).  Only one row of p and q of each sequence is read, once: first the
// tiles' sums, by as many workgroups as there are tiles, then the tile that the draw falls
// into again.
#include "kda_common.hpp"
#include "kda_delta.h"

namespace kda {

namespace {

constexpr int VT = 4096;         // values of a tile
constexpr int VTHREADS = 256;
constexpr int VPER = VT / VTHREADS;

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));   // (rows of any alignment)

struct Row {
    const float* p;
    const float* q;    // null: nothing is taken off
    int point;         // the drafted token that is taken off whole; -1: none
};

// Drafts of sequence n that stand (the same in every lane of the wave).
__device__ __forceinline__ int standing(const VerifyArgs& A, int64_t n, int lens, int lane) {
    for (int base = 0; base < lens; base += 64) {
        const int i = base + lane;
        bool ok = true;
        if (i < lens) {
            const int x = A.drafts[n * A.S + i];
            ok = false;
            if (x >= 0 && x < A.V) {
                const float p = A.target[(n * (A.S + 1) + i) * A.target_stride + x];
                const float q = A.draft != nullptr ? A.draft[(n * A.S + i) * A.draft_stride + x] : 1.0f;
                ok = (double)A.uniform[n * (A.S + 1) + i] * (double)q < (double)p;
            }
        }
        const unsigned long long bad = __ballot(!ok);
        if (bad != 0) return base + __ffsll(bad) - 1;
    }
    return lens;
}
__device__ __forceinline__ int lengths(const VerifyArgs& A, int64_t n) {
    return A.lens != nullptr ? min(max(A.lens[n], 0), A.S) : A.S;
}
__device__ __forceinline__ Row draw_row(const VerifyArgs& A, int64_t n, int stand, int lens) {
    Row r;
    r.p = A.target + (n * (A.S + 1) + stand) * A.target_stride;
    const bool refused = stand < lens;
    r.q = refused && A.draft != nullptr ? A.draft + (n * A.S + stand) * A.draft_stride : nullptr;
    r.point = refused && A.draft == nullptr ? A.drafts[n * A.S + stand] : -1;
    return r;
}

// Positive parts (a NaN counts as 0) of p - q and of p.
__device__ __forceinline__ void weights(const Row& r, int i, float p, float q, double& more, double& whole) {
    const double d = r.q != nullptr ? (double)p - (double)q : i == r.point ? 0.0 : (double)p;
    more = d > 0.0 ? d : 0.0;
    whole = p > 0.0f ? (double)p : 0.0;
}
// 16 values from `at` on, zero behind the row.
__device__ __forceinline__ void load16(const float* row, int at, int V, float (&x)[VPER]) {
    if (at + VPER <= V) {
#pragma unroll
        for (int c = 0; c < VPER / 4; ++c) {
            const f32x4u y = *(const f32x4u*)(row + at + 4 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[4 * c + e] = y[e];
        }
    } else {
#pragma unroll
        for (int c = 0; c < VPER; ++c) x[c] = at + c < V ? row[at + c] : 0.0f;
    }
}

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ double wave_scan(double x, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double y = __shfl_up(x, d, 64);
        if (lane >= d) x += y;
    }
    return x;
}

}  // namespace

// Sums of a tile: [N][tiles][2], of p - q and of p.
__global__ __launch_bounds__(VTHREADS) void verify_sums_kernel(VerifyArgs A) {
    __shared__ double part[VTHREADS / 64][2];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t n = blockIdx.x / A.tiles;
    const int tile = (int)(blockIdx.x - n * A.tiles);
    const int lens = lengths(A, n), stand = standing(A, n, lens, lane);
    const Row r = draw_row(A, n, stand, lens);
    const int at = tile * VT + threadIdx.x * VPER;
    float p[VPER], q[VPER];
    load16(r.p, at, A.V, p);
    if (r.q != nullptr) load16(r.q, at, A.V, q);
    double more = 0.0, whole = 0.0;
#pragma unroll
    for (int c = 0; c < VPER; ++c) {
        double a, b;
        weights(r, at + c, p[c], q[c], a, b);
        more += a;
        whole += b;
    }
    more = __shfl(wave_scan(more, lane), 63, 64);
    whole = __shfl(wave_scan(whole, lane), 63, 64);
    if (lane == 0) {
        part[w][0] = more;
        part[w][1] = whole;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < VTHREADS / 64; ++i) s += part[i][threadIdx.x];
        A.sums[(int64_t)blockIdx.x * 2 + threadIdx.x] = s;
    }
}

// One workgroup per sequence: the tile that the draw falls into, and the token there.
__global__ __launch_bounds__(VTHREADS) void verify_draw_kernel(VerifyArgs A) {
    __shared__ double part[VTHREADS / 64];
    __shared__ int found[2];   // first index whose running sum passes; last index with a weight
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t n = blockIdx.x;
    const int lens = lengths(A, n), stand = standing(A, n, lens, lane);
    Row r = draw_row(A, n, stand, lens);
    const double* sums = A.sums + n * A.tiles * 2;
    // every wave goes through the tiles' sums by itself, in the same order
    double total = 0.0;
    int which = 0;
    for (; which < 2; ++which) {
        total = 0.0;
        for (int base = 0; base < A.tiles; base += 64) {
            const int i = base + lane;
            total += __shfl(wave_scan(i < A.tiles ? sums[2 * i + which] : 0.0, lane), 63, 64);
        }
        if (total > 0.0) break;
    }
    int token = -1;
    if (which < 2) {
        if (which == 1) {
            r.q = nullptr;
            r.point = -1;
        }
        const double u = (double)A.uniform[n * (A.S + 1) + A.S];
        const double mark = (u > 0.0 ? u : 0.0) * total;
        // the first tile whose running sum passes the mark, else the last one with a weight
        double before = 0.0, start = 0.0;
        int tile = -1, last = 0;
        double last_start = 0.0;
        for (int base = 0; base < A.tiles && tile < 0; base += 64) {
            const int i = base + lane;
            const double x = i < A.tiles ? sums[2 * i + which] : 0.0;
            const double sum = before + wave_scan(x, lane);
            const unsigned long long past = __ballot(sum > mark && x > 0.0), some = __ballot(x > 0.0);
            const double first = __shfl_up(sum, 1, 64);
            const double from = lane == 0 ? before : first;
            if (past != 0) {
                const int f = __ffsll(past) - 1;
                tile = base + f;
                start = __shfl(from, f, 64);
            } else if (some != 0) {
                const int l = 63 - __clzll(some);
                last = base + l;
                last_start = __shfl(from, l, 64);
            }
            before = __shfl(sum, 63, 64);
        }
        if (tile < 0) {
            tile = last;
            start = last_start;
        }
        if (threadIdx.x < 2) found[threadIdx.x] = threadIdx.x == 0 ? 0x7fffffff : -1;
        const int at = tile * VT + threadIdx.x * VPER;
        float p[VPER], q[VPER];
        load16(r.p, at, A.V, p);
        if (r.q != nullptr) load16(r.q, at, A.V, q);
        double x[VPER], own = 0.0;
        int mine = -1;   // this thread's last index with a weight
#pragma unroll
        for (int c = 0; c < VPER; ++c) {
            double b;
            weights(r, at + c, p[c], q[c], x[c], b);
            own += x[c];
            if (x[c] > 0.0) mine = at + c;
        }
        const double scan = wave_scan(own, lane);
        if (lane == 63) part[w] = scan;
        __syncthreads();
        double sum = start + (scan - own);
        for (int i = 0; i < w; ++i) sum += part[i];
        int first = 0x7fffffff;
#pragma unroll
        for (int c = 0; c < VPER; ++c) {
            sum += x[c];
            if (x[c] > 0.0 && sum > mark) first = min(first, at + c);
        }
        if (first != 0x7fffffff) atomicMin(&found[0], first);
        if (mine >= 0) atomicMax(&found[1], mine);
        __syncthreads();
        token = found[0] != 0x7fffffff ? found[0] : found[1];
    }
    for (int i = threadIdx.x; i <= A.S; i += VTHREADS)
        A.tokens[n * (A.S + 1) + i] = i < stand ? A.drafts[n * A.S + i] : i == stand ? token : -1;
    if (threadIdx.x == 0) A.accepted[n] = stand + 1;
}

int verify_tiles(int64_t V) { return (int)((V + VT - 1) / VT); }

hipError_t launch_verify(const VerifyArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(verify_sums_kernel, dim3((unsigned)((int64_t)a.N * a.tiles)), dim3(VTHREADS), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(verify_draw_kernel, dim3((unsigned)a.N), dim3(VTHREADS), 0, s, a);
    return hipGetLastError();
}

}  // namespace kda
