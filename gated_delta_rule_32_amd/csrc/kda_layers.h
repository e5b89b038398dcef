// Launch interface of the linear-attention layer kernels: the decayed scan
// (kda_decay.hip) and the per-head row norms (kda_rownorm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_kernels.h"

namespace kda {

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

// One causal form  y_i = s (sum_{j<=i} e^{l(i-j)} (a_i.b_j) c_j) + ... of the
// decayed scan (kda_decay.hip).  An operand's row of token t and value head
// h is base + t*stride + (h / group) * 128 (elements).
struct ScanRole {
    const bf16_t *a, *b, *c;
    int64_t sa, sb, sc;
    int ga, gb, gc;
    void* y;                 // [tokens][Hv][128]: BF16, or FP32 partials when y_f32
    int y_f32;
    int reverse;             // tokens in descending order, state shifted by one decay
    const float* s_in;       // states [.][Hv][128 v][128 k]; null: zero
    int s_in_t;              // the contraction runs over v (s_in read transposed)
    float* s_out;            // states to write, as s_in; null: none
    int s_by_seg;            // s_in and s_out are indexed by segment, else by slot
};
struct ScanArgs {
    ItemMap map;
    ScanRole role[3];
    int roles;
    int share;               // items that read the same operand rows, adjacent in the item order
    const float* log_decay;  // [Hv]
    float scale;
    const int32_t* slot;     // state slot of sequence n; null: n
    int64_t slots;
};

// The segments' states chained: start states in place of the segments' own
// sums.  `reverse`: from the last segment to the first.
struct ChainArgs {
    ItemMap map;
    const float* log_decay;
    float* seg;              // [segments][Hv][128][128]
    const float* s_in;       // [.][Hv][128][128], by slot; null: zero
    float* s_out;            // [.][Hv][128][128], by slot; null: none
    const int32_t* slot;
    int64_t slots;
    int reverse;
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
// dst[t][hq] = sum over the G value heads of src[t][hq*G + g] (FP32 in, BF16
// out), for both (src0, dst0) and (src1, dst1).
hipError_t launch_decay_group_sum(const float* src0, const float* src1, bf16_t* dst0, bf16_t* dst1,
                                  int64_t tokens, int Hqk, int G, hipStream_t s);

struct QkNormArgs {
    int64_t tokens;
    int T;                   // tokens per batch row (positions null: token index within its row)
    int Hq, Hk;
    int rot, interleaved;
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

}  // namespace kda
