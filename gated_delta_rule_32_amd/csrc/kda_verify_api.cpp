// C ABI of the drafted tokens' verification (kda_verify): argument checks, workspace and
// launch.
#include <hip/hip_runtime.h>

#include "../../include/libkda.h"
#include "kda_checks.h"
#include "kda_delta.h"

namespace {

using namespace kda_host;

kda_status check_verify(const kda_verify_problem* p, kda::VerifyArgs& a) {
    if (p == nullptr) return fail(KDA_ERR_NULL_ARG, "problem is NULL");
    if (p->N < 1 || p->S < 0 || p->S > 4096 || p->V < 1 || p->V > 1 << 30)
        return fail(KDA_ERR_SHAPE, "N must be >= 1, S in [0, 4096] and V in [1, 2^30] (got %d %d %d)", p->N, p->S, p->V);
    a.N = p->N;
    a.S = p->S;
    a.V = p->V;
    a.target_stride = p->target_stride == 0 ? p->V : p->target_stride;
    a.draft_stride = p->draft_stride == 0 ? p->V : p->draft_stride;
    for (int64_t st : {a.target_stride, a.draft_stride})
        if (st < p->V || st > (int64_t)1 << 31)
            return fail(KDA_ERR_SHAPE, "a row stride must be in [V=%d, 2^31] (got %lld)", p->V, (long long)st);
    if ((int64_t)p->N * (p->S + 1) >= (int64_t)1 << 31) return fail(KDA_ERR_SHAPE, "too many rows (N x (S+1))");
    auto seq = [&](int64_t given, int rows, int64_t stride, int64_t& out) -> kda_status {
        out = given == 0 ? rows * stride : given;
        if (given != 0 && (given < (rows - 1) * stride + p->V || given > ((int64_t)1 << 60) / p->N))
            return fail(KDA_ERR_SHAPE, "a sequence stride must reach over its %d rows (got %lld)", rows, (long long)given);
        return KDA_OK;
    };
    kda_status s = seq(p->target_seq_stride, p->S + 1, a.target_stride, a.target_seq);
    if (s == KDA_OK) s = seq(p->draft_seq_stride, p->S, a.draft_stride, a.draft_seq);
    if (s != KDA_OK) return s;
    a.tiles = kda::verify_tiles(p->V);
    return a.tiles == 0 ? check_grid(p->N, 1024) : check_grid((int64_t)p->N * a.tiles);
}
size_t verify_ws(const kda::VerifyArgs& a) { return (size_t)a.N * a.tiles * 2 * sizeof(double); }

}  // namespace

extern "C" {

kda_status kda_verify_workspace_bytes(const kda_verify_problem* pp, size_t* bytes) {
    return guarded([&]() -> kda_status {
        kda::VerifyArgs a{};
        kda_status s = check_verify(pp, a);
        if (s != KDA_OK) return s;
        if (bytes == nullptr) return fail(KDA_ERR_NULL_ARG, "bytes is NULL");
        *bytes = verify_ws(a);
        return KDA_OK;
    });
}

kda_status kda_verify(const kda_verify_problem* pp, const int32_t* draft_tokens, const int32_t* draft_lens,
                      const float* target_probs, const float* draft_probs, const float* uniform, int32_t* tokens,
                      int32_t* num_accepted, void* workspace, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> kda_status {
        kda::VerifyArgs a{};
        kda_status s = check_verify(pp, a);
        if (s != KDA_OK) return s;
        if (!target_probs || !uniform || !tokens || !num_accepted || (!draft_tokens && a.S > 0))
            return fail(KDA_ERR_NULL_ARG, "a tensor argument of kda_verify is NULL");
        const size_t need = verify_ws(a);
        if ((s = check_ws(workspace, workspace_bytes, need)) != KDA_OK) return s;
        const size_t n = (size_t)a.N, rows = n * (a.S + 1), drafts = n * a.S;
        auto row_bytes = [&](int of, int64_t seq, int64_t stride) {
            return of == 0 ? 0 : (size_t)((a.N - 1) * seq + (of - 1) * stride + a.V) * sizeof(float);
        };
        s = check_overlap({{tokens, rows * 4, "tokens"}, {num_accepted, n * 4, "num_accepted"},
                           {workspace, need, "workspace"}},
                          {{draft_tokens, draft_tokens ? drafts * 4 : 0, "draft_tokens"},
                           {draft_lens, draft_lens ? n * 4 : 0, "draft_lens"},
                           {target_probs, row_bytes(a.S + 1, a.target_seq, a.target_stride), "target_probs"},
                           {draft_probs, draft_probs ? row_bytes(a.S, a.draft_seq, a.draft_stride) : 0, "draft_probs"},
                           {uniform, rows * 4, "uniform"}});
        if (s != KDA_OK) return s;
        a.drafts = draft_tokens;
        a.lens = draft_lens;
        a.target = target_probs;
        a.draft = draft_probs;
        a.uniform = uniform;
        a.tokens = tokens;
        a.accepted = num_accepted;
        a.sums = (double*)workspace;
        hipError_t e = kda::launch_verify(a, (hipStream_t)stream);
        if (e != hipSuccess) return hip_fail(e, "verification launch");
        return KDA_OK;
    });
}

}  // extern "C"
