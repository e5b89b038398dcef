// C ABI of the gated delta rule (kda_delta_*): argument checks, workspace layout and
// launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "../../include/libkda.h"
#include "kda_checks.h"
#include "kda_delta.h"

namespace {

using namespace kda_host;

constexpr int kDeltaChunk = 32;

struct Delta {
    Seqs s;
    int B = 0, T = 0;
    bool packed = false;
    float scale = 0;
    int unit = 0;
    int64_t sq = 0, sk = 0, sv = 0;
    int segment = 0;       // the caller's choice; 0: automatic
};

kda_status check_delta(const kda_delta_problem* p, Delta& d) {
    if (p == nullptr) return fail(KDA_ERR_NULL_ARG, "problem is NULL");
    kda_status s = check_seqs(p->B, p->T, p->Hqk, p->Hv, p->N, p->cu_seqlens, p->cu_seqlens_host, d.s);
    if (s != KDA_OK) return s;
    d.B = p->B;
    d.T = p->T;
    d.packed = p->cu_seqlens != nullptr;
    d.scale = p->scale == 0.0f ? 1.0f / std::sqrt(128.0f) : p->scale;
    if (!(d.scale > 0.0f) || !std::isfinite(d.scale))
        return fail(KDA_ERR_SCALE, "scale must be 0 or finite and positive (got %g)", (double)p->scale);
    if (p->use_qk_l2norm != 0 && p->use_qk_l2norm != 1)
        return fail(KDA_ERR_SHAPE, "use_qk_l2norm must be 0 or 1 (got %d)", p->use_qk_l2norm);
    d.unit = p->use_qk_l2norm;
    d.sq = p->q_stride;
    d.sk = p->k_stride;
    d.sv = p->v_stride;
    if ((s = check_stride(d.sq, p->Hqk, "q")) != KDA_OK || (s = check_stride(d.sk, p->Hqk, "k")) != KDA_OK ||
        (s = check_stride(d.sv, p->Hv, "v")) != KDA_OK)
        return s;
    if ((int64_t)p->Hv * D > kMaxStride) return fail(KDA_ERR_SHAPE, "too many value heads (%d)", p->Hv);
    if (p->segment < 0 || p->segment % 64 != 0)
        return fail(KDA_ERR_ROUTE, "segment must be 0 or a positive multiple of 64 (got %d)", p->segment);
    d.segment = p->segment;
    return KDA_OK;
}

int64_t total_blocks(const Delta& d) {
    int64_t n = 0;
    for (int64_t len : d.s.len) n += (len + kda::DB - 1) / kda::DB;
    return n;
}

int64_t total_segs(const Delta& d, int seg) {
    int64_t n = 0;
    for (int64_t len : d.s.len) n += (len + seg - 1) / seg;
    return n;
}

// Tokens of the segments that the scans walk side by side, or 0 for whole sequences:
// whichever an estimate says is faster.  A scan over whole sequences takes the longest one's
// latency, 2.4 to 2.9 us a chunk of 32 tokens, or the total's throughput, 15 ns a chunk and
// head.  Segments shorten the first, for a scan that forms each one's M and Q, and 2 to 2.4 us for
// every segment of the chain that joins them.  Both scans' chunk together takes 4.1 us with 64
// segments and heads, 4.8 with 128, 7.9 with 256 and 32 ns each with more.
// In us, forward and backward, whole sequences against the segments of this rule:
// 16 heads x 1024 tokens 93, 118 / 66, 82; 32 x 2048 171, 243 / 113, 188; 16 x 4096 322, 414 / 128,
// 198; 8 x 8192 625, 754 / 146, 211; 32 x 8192 638, 929 / 305, 620; 16 x 32768 2501, 3237 / 593, 1201;
// 64 x 16384 1413, 2353 / 1107, 2338; 4 x 65536 4866, 5699 / 437, 741; 2 sequences x 32 x 4096
// 337, 606 / 298, 622; and against segments that it does not take: 4 x 32 x 4096 397, 967 / 505, 1181 (of
// 1024 tokens), 96 x 32768 2881, 6557 / 3197, 7610 (of 8192).  Other lengths than its own, forward and backward: 16 x
// 32768 667, 1317; 577, 1227; 718, 1301 in segments of 512, 1024 and 4096 (its own 2048), 32 x 8192 307, 639; 360,
// 662 of 512 and 2048 (1024), 16 x 4096 167, 242; 130, 200; 163, 252 of 128, 256 and 1024 (512: 125, 192).
int auto_segment(const Delta& d) {
    if (d.segment != 0) return d.s.max_len > d.segment ? d.segment : 0;
    double chunks = 0;
    for (int64_t len : d.s.len) chunks += (double)((len + kDeltaChunk - 1) / kDeltaChunk);
    const double items = (double)d.s.N * d.s.Hv;
    const double whole = std::max((2.4 + 0.002 * std::min(items, 256.0)) * (double)((d.s.max_len + kDeltaChunk - 1) / kDeltaChunk),
                                  0.0151 * chunks * d.s.Hv);
    double best = 0.95 * whole;
    int seg = 0;
    for (int wanted = 64; wanted <= 512; wanted *= 2) {
        const int64_t len = (d.s.tokens * d.s.Hv / wanted + 63) / 64 * 64;
        if (len < 64 || len >= d.s.max_len) continue;
        const double n = (double)total_segs(d, (int)len) * d.s.Hv;
        const double pair = n <= 128 ? 3.4 + 0.011 * n : n <= 256 ? 7.9 : 0.032 * n;
        const double cut = pair * (double)(len / kDeltaChunk) + 2.4 * (double)((d.s.max_len + len - 1) / len) + 12.0;
        if (cut < best) {
            best = cut;
            seg = (int)len;
        }
    }
    return seg;
}

// The chunks' records, and with segments their states.  (The records first: a backward is
// given them.)
struct RecordWs {
    size_t rec = 0, seg = 0, total = 0;
};
RecordWs record_ws(const Delta& d, int seg) {
    RecordWs w;
    w.seg = align256((size_t)total_blocks(d) * d.s.Hv * 2 * kda::REC);
    w.total = align256(w.seg + (seg ? (size_t)total_segs(d, seg) * d.s.Hv * 2 * kState * sizeof(float) : 0));
    return w;
}

// The backward's workspace: records unless they are given, what the two scans leave, and
// partials of dq and dk where value heads share them.
struct PlanesWs {
    size_t state = 0, rows = 0, scale = 0;
};
struct GradWs {
    RecordWs r;
    PlanesWs forward, backward;
    size_t part_q = 0, part_k = 0, behind = 0, total = 0;
};
GradWs grad_ws(const Delta& d, int seg, bool records) {
    GradWs g;
    const int64_t blocks = total_blocks(d);
    if (!records) g.r = record_ws(d, seg);
    size_t off = g.r.total;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    const size_t items = (size_t)blocks * d.s.Hv;
    for (PlanesWs* p : {&g.forward, &g.backward}) {
        p->state = take(items * kda::PLANE_STATE);
        p->rows = take(items * 2 * kda::PLANE_ROWS);
        p->scale = take(items * sizeof(float));
    }
    const size_t part = d.s.G > 1 ? (size_t)d.s.tokens * d.s.Hv * D * 3 : 0;
    g.part_q = take(part);
    g.part_k = take(part);
    g.behind = take(seg ? (size_t)total_segs(d, seg) * d.s.Hv * kState * sizeof(float) : 0);
    g.total = off;
    return g;
}
kda::DeltaPlanes planes_at(char* ws, const PlanesWs& p) {
    return {ws + p.state, ws + p.rows, (float*)(ws + p.scale)};
}

// The item maps of a call (whole sequences, blocks of 64 tokens, and the scan's: the
// former or segments of `seg` tokens) and its hold on the device schedules (packed calls).
struct Plans {
    SeqPlan blocks, segs;
};
kda_status make_maps(const Delta& d, int seg, hipStream_t stream, Plans& plans, kda::DeltaArgs& a) {
    auto map = [&](int len, SeqPlan& plan, kda::ItemMap& m) -> kda_status {
        m = {};
        m.N = d.s.N;
        m.Hv = d.s.Hv;
        m.len = d.T;
        m.seg_len = len;
        m.items = total_segs(d, len) * d.s.Hv;
        if (!d.packed) return KDA_OK;
        kda_status s = get_seq_plan(d.s, d.B, d.T, d.packed, len, stream, plan);
        if (s != KDA_OK) return s;
        m.task = plan.dev.task;
        m.seg = plan.seg;
        m.seq_start = plan.dev.seq_start;
        m.seq_len = plan.dev.seq_len;
        m.tape_off = plan.dev.tape_off;
        return KDA_OK;
    };
    kda_status s = map(kda::DB, plans.blocks, a.blocks);
    if (s != KDA_OK) return s;
    a.seqs = a.blocks;
    a.seqs.seg_len = 0;
    a.seqs.items = (int64_t)d.s.N * d.s.Hv;
    a.map = a.seqs;
    return seg != 0 ? map(seg, plans.segs, a.map) : KDA_OK;
}

// The chunks' records and the segments' states.
kda_status run_records(const kda::DeltaArgs& a, hipStream_t stream) {
    hipError_t e = kda::launch_delta_prepare(a, stream);
    if (e != hipSuccess) return hip_fail(e, "delta prepare launch");
    if (a.seg != nullptr) {
        e = kda::launch_delta_segments(a, stream);
        if (e != hipSuccess) return hip_fail(e, "delta segment launch");
    }
    return KDA_OK;
}
kda_status run_forward(const kda::DeltaArgs& a, hipStream_t stream) {
    kda_status s = run_records(a, stream);
    if (s != KDA_OK) return s;
    hipError_t e = kda::launch_delta_scan(a, stream);
    if (e != hipSuccess) return hip_fail(e, "delta scan launch");
    return KDA_OK;
}
// The grids of these launches.
kda_status check_forward_grid(const kda::DeltaArgs& a) {
    kda_status s = check_grid(a.map.items * 4);
    if (s == KDA_OK) s = check_grid(a.blocks.items);
    if (s == KDA_OK) s = check_grid(a.seqs.items * 8, a.map.seg_len != 0 ? 512 : 256);   // (the chain's of segments)
    return s;
}

void set_inputs(const Delta& d, const void* q, const void* k, const void* v, const void* g, const void* beta,
                kda::DeltaArgs& a) {
    a.q = (const kda::bf16_t*)q;
    a.k = (const kda::bf16_t*)k;
    a.v = (const kda::bf16_t*)v;
    a.sq = d.sq;
    a.sk = d.sk;
    a.sv = d.sv;
    a.G = d.s.G;
    a.g = (const kda::bf16_t*)g;
    a.beta = (const kda::bf16_t*)beta;
    a.unit = d.unit;
    a.scale = d.scale;
}

std::vector<Span> input_spans(const kda_delta_problem* pp, const Delta& d, const void* q, const void* k, const void* v,
                              const void* g, const void* beta) {
    const size_t gates = (size_t)d.s.tokens * d.s.Hv * 2;
    return {{q, strided_bytes(d.s.tokens, d.sq, d.s.Hqk), "q"}, {k, strided_bytes(d.s.tokens, d.sk, d.s.Hqk), "k"},
            {v, strided_bytes(d.s.tokens, d.sv, d.s.Hv), "v"}, {g, gates, "g"}, {beta, gates, "beta"},
            {pp->cu_seqlens, d.packed ? (size_t)(d.s.N + 1) * 8 : 0, "cu_seqlens"}};
}

// kda_delta_infer takes sequences of up to this many tokens token by token, each by its own
// length, so that a user's tokens are computed the same way whoever else is in the batch.
// In us of 2, 4, 6, 8, 12 tokens of 32 heads, against 32 in chunks: 1 sequence 5.3, 7.8, 10.1, 12.7,
// 17.5 against 13.7; 8 of them 10.3, 14.2, 18.0, 21.8, 28.4 against 19.6; 32 of them 27, 39, 50, 62, 87
// against 41; 128 of them 97, 140, 187, 227, 315 against 132 to 142.
constexpr int64_t kTokenSerialMax = 4;

// How many sequences run in chunks (a packed call's schedule has them first), with how many
// blocks and segments of `seg` tokens (0: whole).
struct InferPlan {
    int64_t chunked = 0, blocks = 0, segs = 0;
    int seg = 0;
    RecordWs ws;
};
InferPlan infer_plan(const Delta& d, int spec) {
    InferPlan r;
    if (spec > 0 || d.s.max_len <= kTokenSerialMax) return r;
    Delta c;
    c.segment = d.segment;
    c.unit = d.unit;
    c.s.Hv = d.s.Hv;
    c.s.max_len = d.s.max_len;
    for (int64_t len : d.s.len)
        if (len > kTokenSerialMax) {
            c.s.len.push_back(len);
            c.s.tokens += len;
        }
    r.chunked = c.s.N = (int)c.s.len.size();
    r.blocks = total_blocks(c);
    r.seg = auto_segment(c);
    if (r.seg != 0) r.segs = total_segs(c, r.seg);
    r.ws = record_ws(d, r.seg);   // (blocks and segments are numbered among all sequences)
    return r;
}

}  // namespace

extern "C" {

kda_status kda_delta_fwd_workspace_bytes(const kda_delta_problem* pp, size_t* bytes) {
    return guarded([&]() -> kda_status {
        Delta d;
        kda_status s = check_delta(pp, d);
        if (s != KDA_OK) return s;
        if (bytes == nullptr) return fail(KDA_ERR_NULL_ARG, "bytes is NULL");
        *bytes = record_ws(d, auto_segment(d)).total;
        return KDA_OK;
    });
}

kda_status kda_delta_fwd(const kda_delta_problem* pp, const void* q, const void* k, const void* v, const void* g,
                         const void* beta, const float* initial_state, void* o, float* final_state,
                         void* workspace, size_t workspace_bytes, void* stream_) {
    return guarded([&]() -> kda_status {
        Delta d;
        kda_status s = check_delta(pp, d);
        if (s != KDA_OK) return s;
        if (!q || !k || !v || !g || !beta || !o)
            return fail(KDA_ERR_NULL_ARG, "a tensor argument of kda_delta_fwd is NULL");
        s = check_align({{q, "q"}, {k, "k"}, {v, "v"}, {initial_state, "initial_state"}, {o, "o"},
                         {final_state, "final_state"}});
        if (s != KDA_OK) return s;
        const int seg = auto_segment(d);
        const RecordWs w = record_ws(d, seg);
        if ((s = check_ws(workspace, workspace_bytes, w.total)) != KDA_OK) return s;
        const size_t st = (size_t)d.s.N * d.s.Hv * kState * 4;
        std::vector<Span> ins = input_spans(pp, d, q, k, v, g, beta);
        ins.push_back({initial_state, initial_state ? st : 0, "initial_state"});
        s = check_overlap({{o, (size_t)d.s.tokens * d.s.Hv * D * 2, "o"},
                           {final_state, final_state ? st : 0, "final_state"},
                           {workspace, w.total, "workspace"}}, ins);
        if (s != KDA_OK) return s;
        hipStream_t stream = (hipStream_t)stream_;
        Plans plans;
        kda::DeltaArgs a{};
        if ((s = make_maps(d, seg, stream, plans, a)) != KDA_OK || (s = check_forward_grid(a)) != KDA_OK) return s;
        set_inputs(d, q, k, v, g, beta, a);
        a.rec = (char*)workspace + w.rec;
        if (seg != 0) a.seg = (float*)((char*)workspace + w.seg);
        a.o = (kda::bf16_t*)o;
        a.s_in = initial_state;
        a.s_out = final_state;
        a.slots = d.s.N;
        return run_forward(a, stream);
    });
}

kda_status kda_delta_bwd_workspace_bytes(const kda_delta_problem* pp, int32_t records_given, size_t* bytes) {
    return guarded([&]() -> kda_status {
        Delta d;
        kda_status s = check_delta(pp, d);
        if (s != KDA_OK) return s;
        if (bytes == nullptr) return fail(KDA_ERR_NULL_ARG, "bytes is NULL");
        *bytes = grad_ws(d, auto_segment(d), records_given != 0).total;
        return KDA_OK;
    });
}

kda_status kda_delta_bwd(const kda_delta_problem* pp, const void* q, const void* k, const void* v, const void* g,
                         const void* beta, const float* initial_state, const void* records, size_t records_bytes,
                         const void* d_o, const float* dfinal_state, void* dq, void* dk, void* dv, void* dg, void* dbeta,
                         float* dinitial_state, void* workspace, size_t workspace_bytes, void* stream_) {
    return guarded([&]() -> kda_status {
        Delta d;
        kda_status s = check_delta(pp, d);
        if (s != KDA_OK) return s;
        if (!q || !k || !v || !g || !beta || !d_o || !dq || !dk || !dv || !dg || !dbeta)
            return fail(KDA_ERR_NULL_ARG, "a tensor argument of kda_delta_bwd is NULL");
        s = check_align({{q, "q"}, {k, "k"}, {v, "v"}, {initial_state, "initial_state"}, {d_o, "do"},
                         {dfinal_state, "dfinal_state"}, {dq, "dq"}, {dk, "dk"}, {dv, "dv"},
                         {dinitial_state, "dinitial_state"}});
        if (s != KDA_OK) return s;
        const int seg = auto_segment(d);
        const RecordWs given = record_ws(d, seg);
        const size_t rec = given.total;
        if (records != nullptr) {
            if (records_bytes < rec) return fail(KDA_ERR_CTX_SIZE, "records have %zu bytes, need %zu", records_bytes, rec);
            if ((s = check_align(records, "records")) != KDA_OK) return s;
        }
        const GradWs wl = grad_ws(d, seg, records != nullptr);
        if ((s = check_ws(workspace, workspace_bytes, wl.total)) != KDA_OK) return s;
        const size_t st = (size_t)d.s.N * d.s.Hv * kState * 4;
        const size_t tq = (size_t)d.s.tokens * d.s.Hqk * D * 2, tv = (size_t)d.s.tokens * d.s.Hv * D * 2,
                     tg = (size_t)d.s.tokens * d.s.Hv * 2;
        std::vector<Span> ins = input_spans(pp, d, q, k, v, g, beta);
        ins.push_back({initial_state, initial_state ? st : 0, "initial_state"});
        ins.push_back({records, records ? rec : 0, "records"});
        ins.push_back({d_o, tv, "do"});
        ins.push_back({dfinal_state, dfinal_state ? st : 0, "dfinal_state"});
        s = check_overlap({{dq, tq, "dq"}, {dk, tq, "dk"}, {dv, tv, "dv"}, {dg, tg, "dg"}, {dbeta, tg, "dbeta"},
                           {dinitial_state, dinitial_state ? st : 0, "dinitial_state"},
                           {workspace, wl.total, "workspace"}}, ins);
        if (s != KDA_OK) return s;
        hipStream_t stream = (hipStream_t)stream_;
        Plans plans;
        kda::DeltaArgs a{};
        if ((s = make_maps(d, seg, stream, plans, a)) != KDA_OK || (s = check_forward_grid(a)) != KDA_OK) return s;
        if (d.s.G > 1 && (s = check_grid((d.s.tokens * d.s.Hqk * (D / 8) + 255) / 256)) != KDA_OK) return s;
        char* ws = (char*)workspace;
        set_inputs(d, q, k, v, g, beta, a);
        a.rec = records != nullptr ? (char*)records : ws + wl.r.rec;
        if (seg != 0) a.seg = (float*)(records != nullptr ? (char*)records + given.seg : ws + wl.r.seg);
        a.rq = 1;
        a.slots = d.s.N;
        a.d_o = (const kda::bf16_t*)d_o;
        kda::DeltaArgs f = a;
        f.s_in = initial_state;
        f.planes = planes_at(ws, wl.forward);
        hipError_t e;
        if (records == nullptr && (s = run_records(f, stream)) != KDA_OK) return s;
        a.s_in = dfinal_state;
        a.s_out = dinitial_state;
        a.planes = planes_at(ws, wl.backward);
        if (seg != 0) {
            a.behind = (float*)(ws + wl.behind);
            e = kda::launch_delta_behind(a, stream);
            if (e != hipSuccess) return hip_fail(e, "delta adjoint launch");
        }
        e = kda::launch_delta_both(f, a, stream);
        if (e != hipSuccess) return hip_fail(e, "delta scans launch");
        const bool pack = d.s.G > 1;
        kda::DeltaGradArgs b{};
        b.blocks = a.blocks;
        b.q = a.q;
        b.k = a.k;
        b.sq = a.sq;
        b.sk = a.sk;
        b.G = a.G;
        b.unit = a.unit;
        b.scale = a.scale;
        b.rec = a.rec;
        b.d_o = a.d_o;
        b.forward = f.planes;
        b.backward = a.planes;
        b.dq = pack ? (void*)(ws + wl.part_q) : dq;
        b.dk = pack ? (void*)(ws + wl.part_k) : dk;
        b.low = pack ? d.s.tokens * d.s.Hv * D * 2 : 0;
        b.dv = (kda::bf16_t*)dv;
        b.dg = (kda::bf16_t*)dg;
        b.dbeta = (kda::bf16_t*)dbeta;
        e = kda::launch_delta_grad(b, stream);
        if (e != hipSuccess) return hip_fail(e, "delta gradient launch");
        if (pack) {
            e = kda::launch_delta_group_sum(ws + wl.part_q, ws + wl.part_k, b.low, (kda::bf16_t*)dq, (kda::bf16_t*)dk,
                                            d.s.tokens, d.s.Hqk, d.s.G, stream);
            if (e != hipSuccess) return hip_fail(e, "group sum launch");
        }
        return KDA_OK;
    });
}

kda_status kda_delta_infer_workspace_bytes(const kda_delta_problem* pp, int32_t num_spec_tokens, size_t* bytes) {
    return guarded([&]() -> kda_status {
        Delta d;
        kda_status s = check_delta(pp, d);
        if (s != KDA_OK) return s;
        if (bytes == nullptr) return fail(KDA_ERR_NULL_ARG, "bytes is NULL");
        if (num_spec_tokens < 0)
            return fail(KDA_ERR_SHAPE, "num_spec_tokens must be >= 0 (got %d)", num_spec_tokens);
        *bytes = infer_plan(d, num_spec_tokens).ws.total;
        return KDA_OK;
    });
}

kda_status kda_delta_infer(const kda_delta_problem* pp, const void* q, const void* k, const void* v, const void* g,
                           const void* beta, float* state_pool, int64_t pool_slots, const int32_t* state_indices,
                           const int32_t* state_indices_host, int32_t num_spec_tokens,
                           const int32_t* num_accepted_tokens, void* o, void* workspace, size_t workspace_bytes,
                           void* stream_) {
    return guarded([&]() -> kda_status {
        Delta d;
        kda_status s = check_delta(pp, d);
        if (s != KDA_OK) return s;
        if (!q || !k || !v || !g || !beta || !state_pool || !o)
            return fail(KDA_ERR_NULL_ARG, "a tensor argument of kda_delta_infer is NULL");
        s = check_align({{q, "q"}, {k, "k"}, {v, "v"}, {state_pool, "state_pool"}, {o, "o"}});
        if (s != KDA_OK) return s;
        if (pool_slots < 1 || pool_slots > ((int64_t)1 << 40) / ((int64_t)d.s.Hv * kState))
            return fail(KDA_ERR_SHAPE, "pool_slots out of range (%lld)", (long long)pool_slots);
        if ((state_indices == nullptr) != (state_indices_host == nullptr))
            return fail(KDA_ERR_NULL_ARG, "state_indices and state_indices_host go together");
        const int spec = num_spec_tokens;
        if (spec < 0) return fail(KDA_ERR_SHAPE, "num_spec_tokens must be >= 0 (got %d)", spec);
        if (spec == 0 && num_accepted_tokens != nullptr)
            return fail(KDA_ERR_SHAPE, "num_accepted_tokens needs num_spec_tokens > 0");
        if (spec > 0) {
            if (state_indices == nullptr)
                return fail(KDA_ERR_NULL_ARG, "drafted tokens need state_indices [N][1+S]");
            for (int n = 0; n < d.s.N; ++n)
                if (d.s.len[n] != 1 + (int64_t)spec)
                    return fail(KDA_ERR_SEQLENS, "sequence %d has %lld tokens; drafted tokens need 1+S=%lld", n,
                                (long long)d.s.len[n], 1 + (long long)spec);
        }
        const int64_t n_idx = (int64_t)d.s.N * (1 + (int64_t)spec);
        if (state_indices_host != nullptr) {
            std::vector<int32_t> sorted(state_indices_host, state_indices_host + n_idx);
            for (int64_t i = 0; i < n_idx; ++i)
                if (sorted[i] < 0 || sorted[i] >= pool_slots)
                    return fail(KDA_ERR_SHAPE, "state_indices[%lld] = %d is outside the pool", (long long)i, sorted[i]);
            std::sort(sorted.begin(), sorted.end());
            for (int64_t i = 1; i < n_idx; ++i)
                if (sorted[i] == sorted[i - 1])
                    return fail(KDA_ERR_SHAPE, "pool slot %d is named twice", sorted[i]);
        } else if (pool_slots < d.s.N) {
            return fail(KDA_ERR_SHAPE, "without state_indices the pool needs N=%d slots (has %lld)", d.s.N,
                        (long long)pool_slots);
        }
        const InferPlan ip = infer_plan(d, spec);
        if ((s = check_ws(workspace, workspace_bytes, ip.ws.total)) != KDA_OK) return s;
        std::vector<Span> ins = input_spans(pp, d, q, k, v, g, beta);
        ins.push_back({state_indices, state_indices ? (size_t)n_idx * 4 : 0, "state_indices"});
        ins.push_back({num_accepted_tokens, num_accepted_tokens ? (size_t)d.s.N * 4 : 0, "num_accepted_tokens"});
        s = check_overlap({{o, (size_t)d.s.tokens * d.s.Hv * D * 2, "o"},
                           {state_pool, (size_t)pool_slots * d.s.Hv * kState * 4, "state_pool"},
                           {workspace, ip.ws.total, "workspace"}}, ins);
        if (s != KDA_OK) return s;
        hipStream_t stream = (hipStream_t)stream_;
        Plans plans;
        kda::DeltaArgs a{};
        if ((s = make_maps(d, ip.seg, stream, plans, a)) != KDA_OK) return s;
        const int64_t serial = d.s.N - ip.chunked;
        a.seqs.items = ip.chunked * d.s.Hv;
        a.map.items = ip.seg != 0 ? ip.segs * d.s.Hv : a.seqs.items;
        a.blocks.items = ip.blocks * d.s.Hv;
        if ((s = check_forward_grid(a)) != KDA_OK || (s = check_grid(serial * d.s.Hv * 4)) != KDA_OK) return s;
        if (ip.chunked != 0) {
            set_inputs(d, q, k, v, g, beta, a);
            a.rec = (char*)workspace + ip.ws.rec;
            a.o = (kda::bf16_t*)o;
            a.s_in = a.s_out = state_pool;
            a.slot = state_indices;
            a.slots = pool_slots;
            if (ip.seg != 0) a.seg = (float*)((char*)workspace + ip.ws.seg);
            if ((s = run_forward(a, stream)) != KDA_OK || serial == 0) return s;
        }
        kda::DeltaTokenArgs t{};
        t.map = a.seqs;
        t.map.items = serial * d.s.Hv;
        if (d.packed) t.map.task = a.seqs.task + ip.chunked * d.s.Hv;
        t.q = (const kda::bf16_t*)q; t.sq = d.sq;
        t.k = (const kda::bf16_t*)k; t.sk = d.sk;
        t.v = (const kda::bf16_t*)v; t.sv = d.sv;
        t.G = d.s.G;
        t.g = (const kda::bf16_t*)g;
        t.beta = (const kda::bf16_t*)beta;
        t.unit = d.unit;
        t.scale = d.scale;
        t.o = (kda::bf16_t*)o;
        t.pool = state_pool;
        t.slot = state_indices;
        t.slots = pool_slots;
        t.each = 1 + spec;
        t.accepted = num_accepted_tokens;
        const hipError_t e = kda::launch_delta_token(t, stream);
        if (e != hipSuccess) return hip_fail(e, "delta decode launch");
        return KDA_OK;
    });
}

}  // extern "C"
