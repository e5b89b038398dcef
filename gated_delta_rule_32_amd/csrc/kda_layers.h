// Launch interface of the linear-attention layer kernels: the decayed scan
// (kda_decay.hip) and the per-head row norms (kda_rownorm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_kernels.h"

namespace kda {

// A kernel that moves more than the last cache before HBM holds (256 MB) reads
// and writes without retention: nothing of it would be found there again.
constexpr int64_t kStreamBytes = (int64_t)256 << 20;

// Where a call's work items lie.  An item is (sequence n, value head h), or
// (sequence n, segment j, value head h) when the sequences are cut into
// segments of seg_len tokens (0: they are not).  With `task` null every
// sequence has `len` tokens and the items are numbered in order; otherwise
// task, seg, seq_start, seq_len and tape_off are a packed call's device
// schedule (DevPlan; tape_off[n] + n counts the segments before sequence n).
struct ItemMap {
    const int32_t* task;
    const int32_t* seg;
    const int64_t* seq_start;
    const int32_t* seq_len;
    const int64_t* tape_off;
    int N, Hv, len, seg_len;
    int64_t items;
};

// Token rows that a scan reads: the row of token t and value head h is
// p + t*stride + (h / group) * 128 (elements).
struct ScanRows {
    const bf16_t* p;
    int64_t stride;
    int group;
};
// One form of the decayed scan, y = a (b^T c) walked over the tokens
// (kda_decay.hip).
struct ScanJob {
    ScanRows b, c, a;        // (states only: no a)
    void* y;                 // [tokens][Hv][128], 2 bytes each: BF16, or packed partials
    int pack;
    int reverse;             // tokens in descending order, states shifted by one decay
    const float* s_in;       // states [.][Hv][128 v][128 k]; null: zero
    int s_in_t;              // the contraction runs over v (s_in read transposed)
    float* s_out;            // states to write, as s_in; null: none
};
struct ScanArgs {
    ItemMap map;
    ScanJob job[3];
    int jobs;                // forms in this launch, the forms of an item side by side
    int share;               // work items that read the same rows, adjacent in the item order
    int by_seg;              // states are indexed by segment, else by slot
    int stream;              // rows are read once and not found in a cache again
    const float* log_decay;  // [Hv]
    float scale;
    const int32_t* slot;     // state slot of sequence n; null: n
    int64_t slots;
};

// The segments' states chained: start states in place of the segments' own
// sums, for `jobs` sets of them.  `reverse`: from the last segment to the first.
struct ChainJob {
    float* seg;              // [segments][Hv][128][128]
    const float* s_in;       // [.][Hv][128][128], by slot; null: zero
    float* s_out;            // [.][Hv][128][128], by slot; null: none
    int reverse;
};
struct ChainArgs {
    ItemMap map;
    ChainJob job[2];
    int jobs;
    int skip;                // sequences of at most this many tokens are left out
    const float* log_decay;
    const int32_t* slot;
    int64_t slots;
};

struct TokenArgs {
    ItemMap map;             // no segments
    const bf16_t *q, *k, *v;
    int64_t sq, sk, sv;
    int G;
    bf16_t* o;
    const float* log_decay;
    float scale;
    float* pool;
    const int32_t* slot;
    int64_t slots;
};

hipError_t launch_decay_scan(const ScanArgs& a, bool states_only, hipStream_t s);
hipError_t launch_decay_chain(const ChainArgs& a, hipStream_t s);
hipError_t launch_decay_token(const TokenArgs& a, hipStream_t s);
// dst[t][hq] = sum over the G value heads of src[t][hq*G + g] (packed
// partials in, BF16 out), for both (src0, dst0) and (src1, dst1).
hipError_t launch_decay_group_sum(const void* src0, const void* src1, bf16_t* dst0, bf16_t* dst1,
                                  int64_t tokens, int Hqk, int G, hipStream_t s);

struct QkNormArgs {
    int64_t tokens;
    int T;                   // tokens per batch row (positions null: token index within its row)
    int Hq, Hk;
    int rot, interleaved;
    int per;                 // heads of a token that 16 lanes take (set by the launch)
    float eps;
    const bf16_t *q, *k;
    int64_t sq, sk;          // token strides (elements)
    const float *wq, *wk;
    const float *cos, *sin;  // [rows][rot / 2]
    int64_t rows;
    const int64_t* positions;
    bf16_t *yq, *yk;         // forward outputs
    const bf16_t *dyq, *dyk; // backward
    bf16_t *dq, *dk;
    float *dwq, *dwk;
    float* part;             // [blocks][2][128] weight-gradient partials
};
struct GNormArgs {
    int64_t tokens;
    int H;
    int silu;
    float eps;
    const bf16_t *x, *g;
    int64_t sx, sg;
    const float* w;
    bf16_t* y;
    const bf16_t* dy;
    bf16_t *dx, *dg;
    float* dw;
    float* part;             // [blocks][128]
};
int rownorm_blocks(int64_t rows);  // blocks of a backward pass (rows of its partials)
hipError_t launch_qknorm_fwd(const QkNormArgs& a, hipStream_t s);
hipError_t launch_qknorm_bwd(const QkNormArgs& a, hipStream_t s);
hipError_t launch_gnorm_fwd(const GNormArgs& a, hipStream_t s);
hipError_t launch_gnorm_bwd(const GNormArgs& a, hipStream_t s);

struct LNormArgs {
    int64_t rows;
    int C;                   // channels, a multiple of 8
    float inv;               // 1 / C
    float eps;
    const bf16_t* x;
    int64_t sx;              // row stride (elements)
    const float *w, *b;      // b: null for none
    bf16_t* y;
    const bf16_t* dy;
    bf16_t* dx;
    float *dw, *db;          // db: null for none
    float* part;             // [lnorm_part_rows][2][C]
};
constexpr int kMaxChannels = 32768;   // of a row that the widest workgroup holds
int64_t lnorm_part_rows(int64_t rows, int C);
hipError_t launch_lnorm(const LNormArgs& a, bool bwd, hipStream_t s);

}  // namespace kda
