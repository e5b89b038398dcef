// Host services of kda_api.cpp that the other entry points' files share:
// error text, overlap checks, sequence checks and the device schedule cache.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <memory>
#include <vector>

#include "../../include/libkda.h"
#include "kda_kernels.h"

namespace kda_host {

// Records `fmt` as the calling thread's last error and returns `s`.
kda_status fail(kda_status s, const char* fmt, ...);
kda_status hip_fail(hipError_t e, const char* what);

// A byte range of a caller's buffer, with its name for error texts.
struct Span {
    const void* p;
    size_t n;
    const char* name;
};
// KDA_ERR_OVERLAP when an output overlaps another output or an input.
kda_status check_overlap(const std::vector<Span>& outs, const std::vector<Span>& ins);

// The sequences of one call (kda_problem's B, T, Hqk, Hv, N and offsets).
struct Seqs {
    int N = 0, Hqk = 0, Hv = 0, G = 0;
    int64_t tokens = 0;              // B * T
    int64_t max_len = 0;
    std::vector<int64_t> len, start; // per sequence; start is a flattened token offset
};
// kda_fwd's shape, grouping and offset checks, without its limit of 2^31
// elements per sequence (for kernels that address rows in 64 bits).
kda_status check_seqs(int B, int T, int Hqk, int Hv, int N, const int64_t* cu, const int64_t* cu_host,
                      Seqs& out);

// One call's hold on the cached device schedule of its sequence lengths, with
// `segment` tokens per segment (a multiple of 16).  Same cache, capture rules
// and errors as kda_fwd's.
struct SeqPlan {
    kda::DevPlan dev{};
    const int32_t* seg = nullptr;    // (sequence, segment) pairs, longest sequence first
    int64_t total_segs = 0;
    struct Hold;
    std::shared_ptr<Hold> hold;      // released (and its last use recorded) with the plan
};
kda_status get_seq_plan(const Seqs& s, int B, int T, bool packed, int segment, hipStream_t stream,
                        SeqPlan& out);

}  // namespace kda_host
