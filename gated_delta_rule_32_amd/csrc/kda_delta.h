// Launch interface of the gated delta rule's kernels (kda_delta.hip, kda_delta_grad.hip)
// and of the drafts' verification (kda_verify.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_layers.h"

namespace kda {

// What a chunk of 32 tokens needs beside its rows, per value head: a record of REC bytes.
// First -C, C being the matrix that solves the chunk's delta rule, as its strictly lower 16 x
// 16 tiles, each in three BF16 pieces of 16 rows of 16; then arrays of 32 floats over the
// tokens i, with G the running sum of the log-decays in the chunk: e^{Gi} and e^{Gn - Gi}, the
// decays from the chunk's start and to its end, beta, one over k's and q's lengths, products
// of these, G in base 2 as the sum of two floats; and the chunk's whole decay as the sum of
// two floats.
constexpr int REC_TILE = 512, REC_C11 = 0, REC_C22 = 3 * REC_TILE, REC_C21 = 6 * REC_TILE, REC_N = 9 * REC_TILE,
              REC_FROM = REC_N, REC_FROM_K = REC_N + 128, REC_FROM_KB = REC_N + 256, REC_TO_K = REC_N + 384,
              REC_TO_KB = REC_N + 512, REC_K = REC_N + 640, REC_KB = REC_N + 768, REC_BETA = REC_N + 896,
              REC_Q = REC_N + 1024, REC_GH = REC_N + 1152, REC_GL = REC_N + 1280, REC_DECAY = REC_N + 1408,
              REC = REC_N + 1536;
constexpr int DB = 64;          // tokens of a block: two chunks, whose records are adjacent

// What the backward's scans leave for the gradients.  Per block the state before it (or the adjoint
// behind it), transposed, as an operand of 8 channels v a lane needs it: what is stored times scale,
// [blocks][Hv], FP32 values rounded to their upper 24 bits (off by 2^-17 at most), the upper 16 of those as
// [blocks][Hv][v/16][128 k][16 v], and STATE_LOW bytes behind them the lower 8 likewise.  Per chunk its solution
// rows as two BF16 pieces (off by 2^-18), [blocks][Hv][2 chunks][v/32][2 pieces][32 v][32 tokens],
// tokens 16t + 4p + e at 8p + 4(t ^ (v/8)%2) + e.
constexpr int STATE_LOW = 128 * 128 * 2, PLANE_STATE = 128 * 128 * 3, PLANE_ROWS = 2 * 128 * 32 * 2;   // bytes
struct DeltaPlanes {
    char *state, *rows;
    float* scale;
};

struct DeltaArgs {
    ItemMap map;                // the scan's items: sequences, or segments of them
    ItemMap blocks;             // blocks of 64 tokens (numbered over all sequences)
    const bf16_t *q, *k, *v;
    int64_t sq, sk, sv;         // token strides (elements)
    int G;
    const bf16_t *g, *beta;     // [tokens][Hv]
    int unit;                   // q and k are taken at unit length
    float scale;
    char* rec;                  // [blocks][Hv][2][REC]
    int rq;                     // the preparation forms one over q's length too (else the scan that reads q)
    bf16_t* o;                  // [tokens][Hv][128]
    const float* s_in;          // states [.][Hv][128 v][128 k], by slot; null: zero
    float* s_out;               // null: none
    const int32_t* slot;        // state slot of sequence n; null: n
    int64_t slots;
    DeltaPlanes planes;         // what a scan leaves for the gradients
    const bf16_t* d_o;          // [tokens][Hv][128]
    // of sequences cut into segments (map), per segment and value head: what the segment adds
    // to a state, in whose place the chain puts the state before it, [128 v][128 k], and what it
    // makes of one, M transposed, [128 k][128 k']: S <- S M + Q.  Null: not cut.
    float* seg;                 // [segments][Hv][2][128][128]
    float* behind;              // of the adjoint likewise the first: [segments][Hv][128][128]
    ItemMap seqs;               // the whole sequences
};

// The gradients of a block of tokens from what the two scans left: the state before the
// block and the adjoint behind it, the rows W of the forward and Y of the backward.
struct DeltaGradArgs {
    ItemMap blocks;
    const bf16_t *q, *k;
    int64_t sq, sk;
    int G;
    int unit;
    float scale;
    const char* rec;
    const bf16_t* d_o;
    DeltaPlanes forward, backward;        // S and W, Z and Y
    void *dq, *dk;                        // [tokens][Hv][128]: BF16, or partials' upper 16 bits
    int64_t low;                          // bytes from those to their lower 8; 0: no partials
    bf16_t *dv, *dg, *dbeta;
};

// Token-serial form on the state pool.
struct DeltaTokenArgs {
    ItemMap map;                // no segments
    const bf16_t *q, *k, *v;
    int64_t sq, sk, sv;
    int G;
    const bf16_t *g, *beta;
    int unit;
    float scale;
    bf16_t* o;
    float* pool;
    const int32_t* slot;        // [N][each]; null: slot n
    int64_t slots;
    int each;                   // slots a sequence: 1, or one per token (drafted tokens)
    const int32_t* accepted;    // [N]: the state starts from slot [n][accepted - 1]; null: 1
};

hipError_t launch_delta_prepare(const DeltaArgs& a, hipStream_t s);
enum DeltaMode { kDeltaOut = 0, kDeltaRecord = 1, kDeltaState = 2 };
hipError_t launch_delta_scan(const DeltaArgs& a, hipStream_t s);   // o and the final states
hipError_t launch_delta_segments(const DeltaArgs& a, hipStream_t s);   // M and Q, and the states chained
hipError_t launch_delta_chain(const DeltaArgs& a, bool reverse, hipStream_t s);
hipError_t launch_delta_behind(const DeltaArgs& a, hipStream_t s);     // the same of the adjoint, M being there
// The backward's two scans at once: `forward` leaves its planes, `backward` its own and the
// adjoint of the initial states.
hipError_t launch_delta_both(const DeltaArgs& forward, const DeltaArgs& backward, hipStream_t s);
hipError_t launch_delta_grad(const DeltaGradArgs& a, hipStream_t s);
hipError_t launch_delta_group_sum(const void* src0, const void* src1, int64_t low, bf16_t* dst0, bf16_t* dst1, int64_t tokens,
                                  int Hqk, int G, hipStream_t s);
hipError_t launch_delta_token(const DeltaTokenArgs& a, hipStream_t s);

struct VerifyArgs {
    int N, S, V;
    const int32_t* drafts;      // [N][S]
    const int32_t* lens;        // [N] drafts of each sequence; null: S
    const float* target;        // rows [N][S+1]
    int64_t target_stride, target_seq;   // of rows and of sequences (elements)
    const float* draft;         // rows [N][S]; null: the drafts are certain
    int64_t draft_stride, draft_seq;
    const float* uniform;       // [N][S+1]
    int32_t* tokens;            // [N][S+1]
    int32_t* accepted;          // [N]
    double* sums;               // [N][tiles][2]
    int tiles;
};
int verify_tiles(int64_t V);
hipError_t launch_verify(const VerifyArgs& a, hipStream_t s);

}  // namespace kda
