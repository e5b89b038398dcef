// Verification of drafted tokens.  With the target's probabilities p, the draft's q and
// given random numbers, draft i of a sequence stands while u_i q_i(x_i) < p_i(x_i); behind
// the last one that stands, one token is drawn from max(p - q, 0) (from p behind the last
// draft, or where p exceeds q nowhere): the first index whose running sum passes u times the total.
//
// Products and sums are formed in 64 bits, where the product of two FP32 values is exact, so
// that a token depends neither on how the row is split nor on the order of its sums, beyond 2^-53 of the
// total for each addition that a sum takes in turn: 30 of them and one for every 64 tiles, 2^-40 in all for
// the longest rows.  Only one row of p and q of each sequence is read.  A row that one workgroup
// holds in registers is read once, by one kernel; of longer ones first the tiles' sums are formed, by
// as many workgroups as there are tiles, then the tile that the draw falls into is read again.
// Bound by HBM with many rows (128 of 131072: 17.3 us, 5.4 TB/s, and 8.8 us for the draws), by latency with
// few (one of 32000: 4.4 and 6.1 us).
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
                const float p = A.target[n * A.target_seq + i * A.target_stride + x];
                const float q = A.draft != nullptr ? A.draft[n * A.draft_seq + i * A.draft_stride + x] : 1.0f;
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
    r.p = A.target + n * A.target_seq + stand * A.target_stride;
    const bool refused = stand < lens;
    r.q = refused && A.draft != nullptr ? A.draft + n * A.draft_seq + stand * A.draft_stride : nullptr;
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

__device__ __forceinline__ double lane_of(double x, int i) {
    const u32x2 b = __builtin_bit_cast(u32x2, x);
    return __builtin_bit_cast(double, u32x2{(unsigned)__builtin_amdgcn_readlane((int)b[0], i),
                                            (unsigned)__builtin_amdgcn_readlane((int)b[1], i)});
}
// The value `kDown` lanes before this one in its row of 16, or zero.
template <int kDown>
__device__ __forceinline__ double shifted(double x) {
    const u32x2 b = __builtin_bit_cast(u32x2, x);
    return __builtin_bit_cast(double, u32x2{(unsigned)__builtin_amdgcn_update_dpp(0, (int)b[0], 0x110 + kDown, 0xF, 0xF, true),
                                            (unsigned)__builtin_amdgcn_update_dpp(0, (int)b[1], 0x110 + kDown, 0xF, 0xF, true)});
}
// Inclusive sum over the wave's lanes.
__device__ __forceinline__ double wave_scan(double x, int lane) {
    x += shifted<1>(x);
    x += shifted<2>(x);
    x += shifted<4>(x);
    x += shifted<8>(x);
    const double a = lane_of(x, 15), b = a + lane_of(x, 31), c = b + lane_of(x, 47);
    return lane < 16 ? x : x + (lane < 32 ? a : lane < 48 ? b : c);
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
    more = lane_of(wave_scan(more, lane), 63);
    whole = lane_of(wave_scan(whole, lane), 63);
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
            total += lane_of(wave_scan(i < A.tiles ? sums[2 * i + which] : 0.0, lane), 63);
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
                start = lane_of(from, f);
            } else if (some != 0) {
                const int l = 63 - __clzll(some);
                last = base + l;
                last_start = lane_of(from, l);
            }
            before = lane_of(sum, 63);
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

// The same for a row of up to 1024 kPer values, in one go.  A wave sums its 64 kPer values as
// they lie in memory; the one that the draw falls into, and the last one with a weight, take them
// again (out of a cache), kPer in a row to a lane.
template <int kPer>
__global__ __launch_bounds__(1024) void verify_row_kernel(VerifyArgs A) {
    __shared__ double part[16][2];
    __shared__ int found[2];   // first index whose running sum passes; last index with a weight
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n = blockIdx.x;
    const int lens = lengths(A, n), stand = standing(A, n, lens, lane);
    Row r = draw_row(A, n, stand, lens);
    double more = 0.0, whole = 0.0;
    {
        float p[kPer / 4][4], q[kPer / 4][4];
#pragma unroll
        for (int g = 0; g < kPer / 4; ++g) {
            const int at = w * 64 * kPer + 256 * g + 4 * lane;
            load_values(r.p, at, A.V, p[g]);
            if (r.q != nullptr) load_values(r.q, at, A.V, q[g]);
        }
#pragma unroll
        for (int g = 0; g < kPer / 4; ++g)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                double a, b;
                weights(r, w * 64 * kPer + 256 * g + 4 * lane + c, p[g][c], q[g][c], a, b);
                more += a;
                whole += b;
            }
    }
    more = wave_scan(more, lane);
    whole = wave_scan(whole, lane);
    if (lane == 63) {
        part[w][0] = more;
        part[w][1] = whole;
    }
    if (threadIdx.x < 2) found[threadIdx.x] = threadIdx.x == 0 ? 0x7fffffff : -1;
    __syncthreads();
    double total = 0.0;
#pragma unroll
    for (int j = 0; j < 16; ++j) total += part[j][0];
    const int which = total > 0.0 ? 0 : 1;   // 1: p exceeds q nowhere
    if (which == 1) {
        r.q = nullptr;
        r.point = -1;
    }
    double before = 0.0;
    int last = -1;
    total = 0.0;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        if (j == w) before = total;
        const double x = part[j][which];
        if (x > 0.0) last = j;
        total += x;
    }
    const double u = (double)A.uniform[n * (A.S + 1) + A.S];
    const double mark = (u > 0.0 ? u : 0.0) * total;
    // (by more than the sums' rounding around the mark, so that one of two neighbours finds it)
    const double end = before + part[w][which];
    if (w == last || (w < last && before <= mark * (1.0 + 0x1p-40) && end >= mark * (1.0 - 0x1p-40))) {
        const int at = (w * 64 + lane) * kPer;
        float p[kPer], q[kPer];
        load_values(r.p, at, A.V, p);
        if (r.q != nullptr) load_values(r.q, at, A.V, q);
        double own = 0.0;
        int mine = -1, first = 0x7fffffff;
#pragma unroll
        for (int c = 0; c < kPer; ++c) {
            double a, b;
            weights(r, at + c, p[c], q[c], a, b);
            own += a;
            if (a > 0.0) mine = at + c;
        }
        double sum = before + (wave_scan(own, lane) - own);
#pragma unroll
        for (int c = 0; c < kPer; ++c) {
            double a, b;
            weights(r, at + c, p[c], q[c], a, b);
            sum += a;
            if (a > 0.0 && sum > mark) first = min(first, at + c);
        }
        if (first != 0x7fffffff) atomicMin(&found[0], first);
        if (mine >= 0) atomicMax(&found[1], mine);
    }
    __syncthreads();
    put_tokens(A, n, stand, found[0] != 0x7fffffff ? found[0] : found[1], 1024);
}

// Rows of up to VROW values go in one kernel.  (In us, captured, against two: 1 row of 4000 7.3 / 10.1,
// of 16000 10.3 / 12.2, 128 of 16000 11.1 / 14.1; with 32 values a thread a row of 32000 15.5 / 11.9, 128 of
// them 18.4 / 16.0: one unit takes as long to read it as the two kernels.)
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
