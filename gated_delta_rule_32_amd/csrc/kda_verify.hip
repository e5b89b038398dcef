// Verification of drafted tokens.  With the target's probabilities p, the draft's q and
// given random numbers, draft i of a sequence stands while u_i q_i(x_i) < p_i(x_i); behind
// the last one that stands, one token is drawn from max(p - q, 0) (from p behind the last
// draft, or where p exceeds q nowhere): the first index whose running sum passes u times the total.
//
// Products and sums are formed in 64 bits, where the product of two FP32 values is exact, so
// that a token depends neither on how the row is split nor on the order of its sums (beyond
// 2^-50 of the total).  Only one row of p and q of each sequence is read.  A row that one workgroup
// holds in registers is read once, by one kernel; of longer ones first the tiles' sums are formed, by
// as many workgroups as there are tiles, then the tile that the draw falls into is read again.
// Bound by HBM with many rows (128 of 131072: 17.8 us, 5.2 TB/s, and 9.4 us for the draws), by latency with
// few (one of 32000: 4.8 and 6.7 us).
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
// Values from `at` on, zero behind the row.
template <int kPer>
__device__ __forceinline__ void load_values(const float* row, int at, int V, float (&x)[kPer]) {
    if (at + kPer <= V) {
#pragma unroll
        for (int c = 0; c < kPer / 4; ++c) {
            const f32x4u y = *(const f32x4u*)(row + at + 4 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[4 * c + e] = y[e];
        }
    } else {
#pragma unroll
        for (int c = 0; c < kPer; ++c) x[c] = at + c < V ? row[at + c] : 0.0f;
    }
}

__device__ __forceinline__ void put_tokens(const VerifyArgs& A, int64_t n, int stand, int token, int threads) {
    for (int i = threadIdx.x; i <= A.S; i += threads)
        A.tokens[n * (A.S + 1) + i] = i < stand ? A.drafts[n * A.S + i] : i == stand ? token : -1;
    if (threadIdx.x == 0) A.accepted[n] = stand + 1;
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
    load_values(r.p, at, A.V, p);
    if (r.q != nullptr) load_values(r.q, at, A.V, q);
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
        load_values(r.p, at, A.V, p);
        if (r.q != nullptr) load_values(r.q, at, A.V, q);
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
    put_tokens(A, n, stand, token, VTHREADS);
}

// The same for a row of up to 1024 kPer values, in one go.
template <int kPer>
__global__ __launch_bounds__(1024) void verify_row_kernel(VerifyArgs A) {
    __shared__ double part[16][2];
    __shared__ int found[2];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t n = blockIdx.x;
    const int lens = lengths(A, n), stand = standing(A, n, lens, lane);
    const Row r = draw_row(A, n, stand, lens);
    const int at = threadIdx.x * kPer;
    constexpr int GROUP = kPer < 16 ? kPer : 16;
    double own[2] = {0.0, 0.0}, scan[2];
    int last[2] = {-1, -1};    // this thread's last indices with a weight
#pragma unroll
    for (int g = 0; g < kPer; g += GROUP) {
        float p[GROUP], q[GROUP];
        load_values(r.p, at + g, A.V, p);
        if (r.q != nullptr) load_values(r.q, at + g, A.V, q);
#pragma unroll
        for (int c = 0; c < GROUP; ++c) {
            double a, b;
            weights(r, at + g + c, p[c], q[c], a, b);
            own[0] += a;
            own[1] += b;
            if (a > 0.0) last[0] = at + g + c;
            if (b > 0.0) last[1] = at + g + c;
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        scan[i] = wave_scan(own[i], lane);
        if (lane == 63) part[w][i] = scan[i];
    }
    if (threadIdx.x < 2) found[threadIdx.x] = threadIdx.x == 0 ? 0x7fffffff : -1;
    __syncthreads();
    double total[2] = {0.0, 0.0}, before[2] = {0.0, 0.0};
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (j == w) before[i] = total[i];
            total[i] += part[j][i];
        }
    const bool all = !(total[0] > 0.0);   // p exceeds q nowhere
    const double u = (double)A.uniform[n * (A.S + 1) + A.S];
    const double mark = (u > 0.0 ? u : 0.0) * (all ? total[1] : total[0]);
    double sum = all ? before[1] + (scan[1] - own[1]) : before[0] + (scan[0] - own[0]);
    const double end = sum + (all ? own[1] : own[0]);
    int first = 0x7fffffff;
    const int mine = all ? last[1] : last[0];
    // only where the sum passes the mark the values are walked again (by more than the sums' rounding
    // around it, so that one of two neighbours finds it)
    if (mine >= 0 && sum <= mark * (1.0 + 0x1p-40) && end >= mark * (1.0 - 0x1p-40)) {
        for (int g = 0; g < kPer; g += GROUP) {
            float p[GROUP], q[GROUP];
            load_values(r.p, at + g, A.V, p);
            if (r.q != nullptr) load_values(r.q, at + g, A.V, q);
#pragma unroll
            for (int c = 0; c < GROUP; ++c) {
                double a, b;
                weights(r, at + g + c, p[c], q[c], a, b);
                const double x = all ? b : a;
                sum += x;
                if (x > 0.0 && sum > mark) first = min(first, at + g + c);
            }
        }
    }
    if (first != 0x7fffffff) atomicMin(&found[0], first);
    if (mine >= 0) atomicMax(&found[1], mine);
    __syncthreads();
    put_tokens(A, n, stand, found[0] != 0x7fffffff ? found[0] : found[1], 1024);
}

// Rows of up to VROW values go in one kernel.  (In us, captured, against two: 1 row of 4000 7.6 / 13.4,
// of 16000 10.1 / 13.4, 128 of 16000 11.2 / 14.7; a row of 32000 17.8 / 10.6: a thread's values then
// pass through the first cache more than once.)
constexpr int64_t VROW = 16384;
int verify_tiles(int64_t V) { return V <= VROW ? 0 : (int)((V + VT - 1) / VT); }

hipError_t launch_verify(const VerifyArgs& a, hipStream_t s) {
    if (a.tiles == 0) {
        if (a.V <= 4096)
            hipLaunchKernelGGL((verify_row_kernel<4>), dim3((unsigned)a.N), dim3(1024), 0, s, a);
        else
            hipLaunchKernelGGL((verify_row_kernel<16>), dim3((unsigned)a.N), dim3(1024), 0, s, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(verify_sums_kernel, dim3((unsigned)((int64_t)a.N * a.tiles)), dim3(VTHREADS), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(verify_draw_kernel, dim3((unsigned)a.N), dim3(VTHREADS), 0, s, a);
    return hipGetLastError();
}

}  // namespace kda
