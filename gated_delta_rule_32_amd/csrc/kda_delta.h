// Launch interface of the gated delta rule's kernels (kda_delta.hip, kda_delta_grad.hip)
// and of the drafts' verification (kda_verify.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_layers.h"

namespace kda {

// What a chunk of 32 tokens needs beside its rows, per value head (floats): the matrix C
// that solves the chunk's delta rule, as its strictly lower 16 x 16 tiles row by row, and
// arrays of 32 over the tokens i, with G the running sum of the log-decays in the chunk:
// the decay from the chunk's start times one over k's length, the decay to its end times
// the same, the decay from the start times the scale over q's length, beta, G in base 2 as
// the sum of two floats, the scale over q's length, one over k's length.
constexpr int REC_C11 = 0, REC_C22 = 256, REC_C21 = 512, REC_CX = 768, REC_CE = 800, REC_CO = 832, REC_BETA = 864,
              REC_GH = 896, REC_GL = 928, REC_A = 960, REC_RK = 992, REC = 1024;
constexpr int DB = 64;          // tokens of a block: two chunks, whose records are adjacent

struct DeltaArgs {
    ItemMap map;                // the scan's items: sequences, or segments of them
    ItemMap blocks;             // blocks of 64 tokens (numbered over all sequences)
    const bf16_t *q, *k, *v;
    int64_t sq, sk, sv;         // token strides (elements)
    int G;
    const bf16_t *g, *beta;     // [tokens][Hv]
    int unit;                   // q and k are taken at unit length
    float scale;
    float* rec;                 // [blocks][Hv][2][REC]
    float* fac;                 // [blocks][Hv][2][2]: the chunk's decay as the sum of two floats
    bf16_t* o;                  // [tokens][Hv][128]
    const float* s_in;          // states [.][Hv][128 v][128 k], by slot; null: zero
    float* s_out;               // null: none
    const int32_t* slot;        // state slot of sequence n; null: n
    int64_t slots;
    // for the backward: per block the state before it (or the adjoint behind it) in planes of
    // high and low BF16 parts [blocks][Hv][2][128 v][128 k], and per chunk its solution rows
    // [blocks][Hv][2 chunks][2 planes][128 v][32 tokens]
    bf16_t* state_planes;
    bf16_t* row_planes;
    const bf16_t* d_o;          // [tokens][Hv][128]
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
    const float* rec;
    const bf16_t* d_o;
    const bf16_t *s_planes, *z_planes;    // [blocks][Hv][2][128 v][128 k]
    const bf16_t *w_planes, *y_planes;    // [blocks][Hv][2 chunks][2][128 v][32 tokens]
    void *dq, *dk;                        // [tokens][Hv][128]: BF16, or packed partials
    int pack;
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
enum DeltaMode { kDeltaOut = 0, kDeltaRecord = 1 };
hipError_t launch_delta_scan(const DeltaArgs& a, DeltaMode mode, hipStream_t s);
hipError_t launch_delta_adjoint(const DeltaArgs& a, hipStream_t s);
hipError_t launch_delta_grad(const DeltaGradArgs& a, hipStream_t s);
hipError_t launch_delta_token(const DeltaTokenArgs& a, hipStream_t s);

struct VerifyArgs {
    int N, S, V;
    const int32_t* drafts;      // [N][S]
    const int32_t* lens;        // [N] drafts of each sequence; null: S
    const float* target;        // rows [N][S+1]
    int64_t target_stride;      // of rows (elements)
    const float* draft;         // rows [N][S]; null: the drafts are certain
    int64_t draft_stride;
    const float* uniform;       // [N][S+1]
    int32_t* tokens;            // [N][S+1]
    int32_t* accepted;          // [N]
    double* sums;               // [N][tiles][2]
    int tiles;
};
int verify_tiles(int64_t V);
hipError_t launch_verify(const VerifyArgs& a, hipStream_t s);

}  // namespace kda
