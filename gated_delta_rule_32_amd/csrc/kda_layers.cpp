// C ABI of the linear-attention layer operators: argument checks, workspace
// layout and launches of kda_decay_* (linear attention with a constant decay
// per head), kda_qknorm_* (query/key norm and rotary rotation) and
// kda_gnorm_* (gated norm of the heads' outputs).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <exception>
#include <vector>

#include "../../include/libkda.h"
#include "kda_host.h"
#include "kda_layers.h"

namespace {

using kda_host::check_overlap;
using kda_host::fail;
using kda_host::hip_fail;
using kda_host::SeqPlan;
using kda_host::Seqs;
using kda_host::Span;

constexpr int D = 128;
constexpr int64_t kState = (int64_t)D * D;
// Largest token stride (elements): the kernels add up to 31 of them in 32 bits.
constexpr int64_t kMaxStride = (int64_t)1 << 25;

// Most rows of a row norm: the kernels number them in 32 bits, with room for
// the last step behind them (2^31 rows are 512 GiB).
constexpr int64_t kMaxRows = (int64_t)1 << 31;

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Runs an entry point's body; an exception (host memory) becomes a status.
template <class F>
kda_status guarded(F f) {
    try {
        return f();
    } catch (const std::exception& e) {
        return fail(KDA_ERR_HIP, "host error: %s", e.what());
    }
}

// 0 means dense rows.
kda_status check_stride(int64_t& stride, int heads, const char* name) {
    if (stride == 0) stride = (int64_t)heads * D;
    if (stride < (int64_t)heads * D || stride > kMaxStride || stride % 8 != 0)
        return fail(KDA_ERR_SHAPE, "%s token stride must be a multiple of 8 in [%d, %lld] (got %lld)", name, heads * D,
                    (long long)kMaxStride, (long long)stride);
    return KDA_OK;
}

kda_status check_align(const void* p, const char* name) {
    if (((uintptr_t)p & 15) != 0) return fail(KDA_ERR_SHAPE, "%s must be 16-byte aligned", name);
    return KDA_OK;
}
kda_status check_align(std::initializer_list<std::pair<const void*, const char*>> ps) {
    for (const auto& p : ps) {
        kda_status s = check_align(p.first, p.second);
        if (s != KDA_OK) return s;
    }
    return KDA_OK;
}

// (Below the normal numbers the reciprocal square root takes eps for 0, and a row of
// zeros would come out as NaN.)
kda_status check_eps(float eps) {
    if (!(eps >= FLT_MIN) || !std::isfinite(eps))
        return fail(KDA_ERR_SHAPE, "eps must be finite and a positive normal number (got %g)", (double)eps);
    return KDA_OK;
}

// Bytes from a strided operand's first element to behind its last.
size_t strided_bytes(int64_t tokens, int64_t stride, int heads) {
    return (size_t)((tokens - 1) * stride + (int64_t)heads * D) * 2;
}

// ---------------------------------------------------------------------------
// linear attention with a constant decay per head
// ---------------------------------------------------------------------------
struct Decay {
    Seqs s;
    int B = 0, T = 0;
    bool packed = false;
    float scale = 0;
    int64_t sq = 0, sk = 0, sv = 0;
    int segment = 0;       // the caller's choice; 0: automatic
};

kda_status check_decay(const kda_decay_problem* p, Decay& d) {
    if (p == nullptr) return fail(KDA_ERR_NULL_ARG, "problem is NULL");
    kda_status s = kda_host::check_seqs(p->B, p->T, p->Hqk, p->Hv, p->N, p->cu_seqlens, p->cu_seqlens_host, d.s);
    if (s != KDA_OK) return s;
    d.B = p->B;
    d.T = p->T;
    d.packed = p->cu_seqlens != nullptr;
    d.scale = p->scale == 0.0f ? 1.0f / std::sqrt(128.0f) : p->scale;
    if (!(d.scale > 0.0f) || !std::isfinite(d.scale))
        return fail(KDA_ERR_SCALE, "scale must be 0 or finite and positive (got %g)", (double)p->scale);
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

int64_t total_segs(const Decay& d, int seg) {
    int64_t n = 0;
    for (int64_t len : d.s.len) n += (len + seg - 1) / seg;
    return n;
}

// Tokens per segment of a scan over `forms` forms (o, or dq, dk and dv), or 0
// for whole sequences: whichever an estimate says is faster.  Measured: a
// chunk of 32 tokens takes a workgroup 1.4 (few of them), 1.7 to 2.1 (up to one per
// compute unit) or 3 us (several, see launch_decay_scan), and the card gets through one
// chunk of one head every 7.3 ns.  So whole sequences take the longest one's latency or
// the total's throughput.  Segments shorten the first, for a pass that forms the
// segments' states (for the backward both ways), their way through memory (15 ns
// each) and two more launches.  That pass takes 1.2 us a chunk with few workgroups, 1.9
// with one per compute unit, 2.6 (16 heads x 32768 tokens, 5 ns a chunk in all) to 4.6 (32 x
// 8192, 9 ns) with two; the estimate takes the low ends, 1.2 us and 4.5 ns.  In us,
// whole sequences against the segments of this rule, forward: 4 heads x 512 tokens 26
// / 21, 16 x 1024 49 / 30, 64 x 1024 51 / 47, 16 x 4096 182 / 49, 32 x 8192 368 / 125, 16 x
// 32768 1420 / 223, 96 x 4096 184 / 189, 2 sequences x 32 heads x 2048 93 / 72; against
// segments of 1024, 4 x 32 x 4096 188 / 208, 8 x 32 x 2048 138 / 211; backward: 16 x 1024
// 52 / 40, 16 x 4096 182 / 86, 32 x 8192 358 / 252, 16 x 32768 1420 / 475; against segments
// of 512, 2 x 32 x 2048 112 / 127, of 576, 3 x 16 x 3000 161 / 168, of 1024, 4 x 32 x 4096 387
// / 494.
// How long the segments are, in us for those of 128, 192, 256, 384, 512, 1024 and 2048
// tokens, forward: 16 heads x 1024 tokens 29, 31, 32, 39, 47, -, -; 32 x 2048 54, 56, 45,
// 52, 52, 82, -; 32 x 8192 174, 139, 123, 115, 109, 108, 155; 16 x 32768 375, 279, 256, 237,
// 221, 205, 221; backward: 16 x 1024 41, 40, 39, 46, 50, -, -; 32 x 2048 95, 87, 79, 93, 84,
// 92, -; 32 x 8192 365, 320, 292, 278, 261, 239, 286; 16 x 32768 725, 637, 577, 530, 501, 486,
// 468.
double chunk_us(int64_t groups) {
    return groups <= 128 ? 1.4 + 0.0006 * (double)groups : groups <= 256 ? 1.25 + 0.003 * (double)groups : 3.0;
}

int auto_segment(const Decay& d, int forms) {
    if (d.segment != 0) return d.s.max_len > d.segment ? d.segment : 0;
    double chunks = 0;
    for (int64_t len : d.s.len) chunks += (double)((len + 31) / 32);
    chunks *= d.s.Hv;
    const int passes = forms == 1 ? 1 : 2;
    const double whole = 4.0 + std::max(chunk_us((int64_t)d.s.N * d.s.Hv * forms) * (double)((d.s.max_len + 31) / 32),
                                        0.0073 * forms * chunks);
    auto per_item = [&](int64_t items) { return (d.s.tokens * d.s.Hv / items + 63) / 64 * 64; };
    // backward, three forms a segment: one segment per compute unit, not below 192 tokens;
    // forward: one while that makes it at most 256 tokens long, not below 128, otherwise two
    int64_t seg = per_item(256);
    if (forms != 1)
        seg = std::max<int64_t>(seg, 192);
    else
        seg = seg <= 256 ? std::max<int64_t>(seg, 128) : std::max<int64_t>(per_item(512), 256);
    if (d.s.max_len <= seg) return 0;
    const int64_t cut_items = total_segs(d, (int)seg) * d.s.Hv;
    const double cut = std::max((chunk_us(cut_items * forms) + 1.2) * (double)(seg / 32),
                                (0.0073 * forms + 0.0045 * passes) * chunks) +
                       12.0 + 0.015 * passes * (double)cut_items;
    return cut < 0.95 * whole ? (int)seg : 0;
}

struct DecayWs {
    size_t seg_f = 0, seg_r = 0, part_q = 0, part_k = 0, total = 0;
};
DecayWs decay_ws(const Decay& d, int seg, bool backward) {
    DecayWs w;
    size_t off = 0;
    const size_t states = seg ? (size_t)total_segs(d, seg) * d.s.Hv * kState * sizeof(float) : 0;
    w.seg_f = off;
    off = align256(off + states);
    if (backward) {
        w.seg_r = off;
        off = align256(off + states);
        const size_t part = d.s.G > 1 ? (size_t)d.s.tokens * d.s.Hv * D * 2 : 0;
        w.part_q = off;
        off = align256(off + part);
        w.part_k = off;
        off = align256(off + part);
    }
    w.total = off;
    return w;
}

// The item map of a call and its hold on the device schedule (packed calls).
kda_status make_map(const Decay& d, int seg, hipStream_t stream, SeqPlan& plan, kda::ItemMap& m) {
    m = kda::ItemMap{};
    m.N = d.s.N;
    m.Hv = d.s.Hv;
    m.len = d.T;
    m.seg_len = seg;
    m.items = (seg ? total_segs(d, seg) : (int64_t)d.s.N) * d.s.Hv;
    if (d.packed) {
        kda_status s = kda_host::get_seq_plan(d.s, d.B, d.T, d.packed, seg ? seg : 256, stream, plan);
        if (s != KDA_OK) return s;
        m.task = plan.dev.task;
        m.seg = plan.seg;
        m.seq_start = plan.dev.seq_start;
        m.seq_len = plan.dev.seq_len;
        m.tape_off = plan.dev.tape_off;
    }
    return KDA_OK;
}

// A launch holds less than 2^32 threads; workgroups of 256 here.
kda_status check_grid(int64_t blocks) {
    if (blocks >= (int64_t)1 << 24) return fail(KDA_ERR_SHAPE, "too many (sequence, head) tasks or tokens");
    return KDA_OK;
}
// The scan's grid for `jobs` forms, and with segments the chain's.
kda_status check_scan_grid(const Decay& d, int seg, const kda::ItemMap& m, int jobs) {
    kda_status s = check_grid(m.items * jobs);
    if (s == KDA_OK && seg != 0) s = check_grid((int64_t)d.s.N * d.s.Hv * 16);
    return s;
}

// Work items that go to one XCD side by side (xcd_order): the value heads of a
// q/k head, whose rows they share, and about 8 heads of neighbouring rows.  Of
// single heads an odd number, so that an XCD's blocks start at different memory
// channels; but not in the backward, whose three forms share rows and lose that
// in the blocks that a window of 8 XCDs leaves over.  In us, side by side 1, 3,
// 8, 11, 16, 31: forward of 32 x 1024 tokens x 32 heads 279, 268, 279, 268, 274, 267, of 8
// x 1024 x 96 221 to 223 whichever; backward of 8 x 2048 x 32 334, 333, 331, 336, 331, 333.
// In fours, 4, 4, 8, 12, 16, 32: forward of 32 x 2048 x 16 q/k and 64 value heads 845, 843,
// 836, 842, 835, 837; 4 x 4096 x 8 and 32, both directions 710, 708, 708, 730, 706, 722.
int xcd_share(int G, bool backward) { return G == 1 && !backward ? 11 : (8 + G - 1) / G * G; }

// o's form over whole sequences or segments; the states come from `s_in` and
// go to `s_out`, both by slot.  m's items are those of the sequences longer
// than `skip` tokens.
kda_status run_forward(const Decay& d, int seg, const kda::ItemMap& m, int64_t skip, const void* q, const void* k,
                       const void* v, const float* log_decay, const float* s_in, float* s_out, const int32_t* slot,
                       int64_t slots, void* o, char* ws, hipStream_t stream) {
    const int G = d.s.G;
    kda::ScanArgs a{};
    a.map = m;
    a.jobs = 1;
    a.share = xcd_share(G, false);
    // Rows that no other head reads, more than the caches hold: non-temporal loads.
    // Forward of 8 sequences x 96 heads x 1024 tokens 202 -> 196 us, x 512 124 ->
    // 118, x 64 (50 MB) 30.0 -> 30.6; 32 sequences x 2048 tokens x 16 q/k and 64 value heads,
    // whose q and k are read four times, 838 -> 901.  (Not in the states' pass, whose rows
    // are read again; one sequence of 16384 tokens x 64 heads takes 386 us either way.)
    a.stream = G == 1 && 4 * d.s.tokens * d.s.Hv * D * 2 > kda::kStreamBytes;
    a.log_decay = log_decay;
    a.scale = d.scale;
    a.slot = slot;
    a.slots = slots;
    kda::ScanJob& j = a.job[0];
    j.b = {(const kda::bf16_t*)k, d.sk, G};
    j.c = {(const kda::bf16_t*)v, d.sv, 1};
    j.a = {(const kda::bf16_t*)q, d.sq, G};
    j.y = o;
    j.s_in = s_in;
    j.s_out = s_out;
    hipError_t e;
    if (seg != 0) {
        float* states = (float*)ws;
        kda::ScanArgs b = a;
        b.by_seg = 1;
        b.job[0].s_in = nullptr;
        b.job[0].s_out = states;
        e = kda::launch_decay_scan(b, true, stream);
        if (e != hipSuccess) return hip_fail(e, "segment state launch");
        kda::ChainArgs c{};
        c.map = m;
        c.jobs = 1;
        c.job[0] = {states, s_in, s_out, 0};
        c.skip = (int)skip;
        c.log_decay = log_decay;
        c.slot = slot;
        c.slots = slots;
        e = kda::launch_decay_chain(c, stream);
        if (e != hipSuccess) return hip_fail(e, "segment chain launch");
        j.s_in = states;
        j.s_out = nullptr;
        a.by_seg = 1;
    }
    e = kda::launch_decay_scan(a, false, stream);
    if (e != hipSuccess) return hip_fail(e, "decay scan launch");
    return KDA_OK;
}

// kda_decay_infer takes sequences of up to this many tokens token by token, each
// by its own length, so that a user's tokens are computed the same way whoever else
// is in the batch.  Token by token against one chunk, in us, for sequences of 2, 4, 8
// and 16 tokens: one sequence of 32 heads 5.6, 6.3, 9.7, 16.6 against 7.0; 8 of them 7.9,
// 10.1, 14.0, 21.7 against 11.1; 32 of them 23.7, 29.1, 41, 66 against 26.8 to 28; 128 of
// 64 heads 175, 204, 290, 469 against 212, 216, 225, 235.
constexpr int64_t kTokenSerialMax = 4;

// How a call of kda_decay_infer runs: its `chunked` longer sequences in chunks
// (segments of `seg` tokens, 0: whole), the others token by token.  A packed call's
// schedule has the longer ones first.
struct InferPlan {
    int64_t chunked = 0, segs = 0;   // segs: the chunked sequences' segments
    int seg = 0;
    size_t ws = 0;
};
InferPlan infer_plan(const Decay& d) {
    InferPlan r;
    if (d.s.max_len <= kTokenSerialMax) return r;
    Decay c;
    c.segment = d.segment;
    c.s.Hv = d.s.Hv;
    c.s.max_len = d.s.max_len;
    for (int64_t len : d.s.len)
        if (len > kTokenSerialMax) {
            c.s.len.push_back(len);
            c.s.tokens += len;
        }
    r.chunked = c.s.N = (int)c.s.len.size();
    r.seg = auto_segment(c, 1);
    if (r.seg != 0) r.segs = total_segs(c, r.seg);
    r.ws = decay_ws(d, r.seg, false).total;   // (segments are numbered among all sequences)
    return r;
}

kda_status check_ws(const void* ws, size_t bytes, size_t need) {
    if (need == 0) return KDA_OK;
    if (ws == nullptr) return fail(KDA_ERR_NULL_ARG, "workspace is NULL (needs %zu bytes)", need);
    if (bytes < need) return fail(KDA_ERR_WORKSPACE_SIZE, "workspace has %zu bytes, needs %zu", bytes, need);
    return check_align(ws, "workspace");
}

// ---------------------------------------------------------------------------
// row norms
// ---------------------------------------------------------------------------
kda_status check_qknorm(const kda_qknorm_problem* p, kda::QkNormArgs& a) {
    if (p == nullptr) return fail(KDA_ERR_NULL_ARG, "problem is NULL");
    if (p->B < 1 || p->T < 1 || p->Hq < 1 || p->Hk < 1)
        return fail(KDA_ERR_SHAPE, "B, T, Hq and Hk must be >= 1 (got %d %d %d %d)", p->B, p->T, p->Hq, p->Hk);
    if ((int64_t)p->Hq + p->Hk > kMaxStride / D)
        return fail(KDA_ERR_SHAPE, "too many heads (%d + %d)", p->Hq, p->Hk);
    if (p->rot_dim < 8 || p->rot_dim > D || p->rot_dim % 8 != 0)
        return fail(KDA_ERR_SHAPE, "rot_dim must be a multiple of 8 in [8, 128] (got %d)", p->rot_dim);
    if (p->interleaved != 0 && p->interleaved != 1)
        return fail(KDA_ERR_SHAPE, "interleaved must be 0 or 1 (got %d)", p->interleaved);
    kda_status s = check_eps(p->eps);
    if (s != KDA_OK) return s;
    if (p->table_rows < 1 || p->table_rows > ((int64_t)1 << 40))
        return fail(KDA_ERR_SHAPE, "table_rows out of range (%lld)", (long long)p->table_rows);
    a.tokens = (int64_t)p->B * p->T;
    if (a.tokens * (p->Hq + p->Hk) > kMaxRows) return fail(KDA_ERR_SHAPE, "too many rows (tokens x heads)");
    a.T = p->T;
    a.Hq = p->Hq;
    a.Hk = p->Hk;
    a.rot = p->rot_dim;
    a.interleaved = p->interleaved;
    a.eps = p->eps;
    a.rows = p->table_rows;
    a.sq = p->q_stride;
    a.sk = p->k_stride;
    if ((s = check_stride(a.sq, p->Hq, "q")) != KDA_OK || (s = check_stride(a.sk, p->Hk, "k")) != KDA_OK) return s;
    return KDA_OK;
}
kda_status qknorm_inputs(const kda_qknorm_problem* p, kda::QkNormArgs& a, const void* q, const void* k,
                         const float* wq, const float* wk, const float* cos, const float* sin,
                         const int64_t* positions, std::vector<Span>& ins) {
    if (!q || !k || !wq || !wk || !cos || !sin)
        return fail(KDA_ERR_NULL_ARG, "a tensor argument of kda_qknorm is NULL");
    if (positions == nullptr && p->table_rows < p->T)
        return fail(KDA_ERR_SHAPE, "without positions the table needs T=%d rows (has %lld)", p->T,
                    (long long)p->table_rows);
    kda_status s = check_align({{q, "q"}, {k, "k"}, {cos, "cos"}, {sin, "sin"}});
    if (s != KDA_OK) return s;
    a.q = (const kda::bf16_t*)q;
    a.k = (const kda::bf16_t*)k;
    a.wq = wq;
    a.wk = wk;
    a.cos = cos;
    a.sin = sin;
    a.positions = positions;
    const size_t table = (size_t)a.rows * (a.rot / 2) * 4;
    ins = {{q, strided_bytes(a.tokens, a.sq, a.Hq), "q"}, {k, strided_bytes(a.tokens, a.sk, a.Hk), "k"},
           {wq, D * 4, "q_weight"}, {wk, D * 4, "k_weight"}, {cos, table, "cos"}, {sin, table, "sin"},
           {positions, positions ? (size_t)a.tokens * 8 : 0, "positions"}};
    return KDA_OK;
}
size_t qknorm_ws(const kda::QkNormArgs& a) {
    return (size_t)kda::rownorm_blocks(a.tokens * (a.Hq + a.Hk)) * 2 * D * sizeof(float);
}

kda_status check_gnorm(const kda_gnorm_problem* p, kda::GNormArgs& a) {
    if (p == nullptr) return fail(KDA_ERR_NULL_ARG, "problem is NULL");
    if (p->B < 1 || p->T < 1 || p->H < 1)
        return fail(KDA_ERR_SHAPE, "B, T and H must be >= 1 (got %d %d %d)", p->B, p->T, p->H);
    if (p->activation != KDA_GATE_SIGMOID && p->activation != KDA_GATE_SILU)
        return fail(KDA_ERR_SHAPE, "unknown activation %d", p->activation);
    kda_status s = check_eps(p->eps);
    if (s != KDA_OK) return s;
    a.tokens = (int64_t)p->B * p->T;
    if (p->H > kMaxStride / D || a.tokens * p->H > kMaxRows)
        return fail(KDA_ERR_SHAPE, "too many rows (tokens x heads)");
    a.H = p->H;
    a.silu = p->activation == KDA_GATE_SILU;
    a.eps = p->eps;
    a.sx = p->x_stride;
    a.sg = p->gate_stride;
    if ((s = check_stride(a.sx, p->H, "x")) != KDA_OK || (s = check_stride(a.sg, p->H, "gate")) != KDA_OK) return s;
    return KDA_OK;
}
size_t gnorm_ws(const kda::GNormArgs& a) {
    return (size_t)kda::rownorm_blocks(a.tokens * a.H) * D * sizeof(float);
}

}  // namespace

extern "C" {

kda_status kda_decay_fwd_workspace_bytes(const kda_decay_problem* pp, size_t* bytes) {
    return guarded([&]() -> kda_status {
        Decay d;
        kda_status s = check_decay(pp, d);
        if (s != KDA_OK) return s;
        if (bytes == nullptr) return fail(KDA_ERR_NULL_ARG, "bytes is NULL");
        *bytes = decay_ws(d, auto_segment(d, 1), false).total;
        return KDA_OK;
    });
}

kda_status kda_decay_bwd_workspace_bytes(const kda_decay_problem* pp, size_t* bytes) {
    return guarded([&]() -> kda_status {
        Decay d;
        kda_status s = check_decay(pp, d);
        if (s != KDA_OK) return s;
        if (bytes == nullptr) return fail(KDA_ERR_NULL_ARG, "bytes is NULL");
        *bytes = decay_ws(d, auto_segment(d, 3), true).total;
        return KDA_OK;
    });
}

kda_status kda_decay_fwd(const kda_decay_problem* pp, const void* q, const void* k, const void* v,
                         const float* log_decay, const float* initial_state, void* o, float* final_state,
                         void* workspace, size_t workspace_bytes, void* stream_) {
    return guarded([&]() -> kda_status {
        Decay d;
        kda_status s = check_decay(pp, d);
        if (s != KDA_OK) return s;
        if (!q || !k || !v || !log_decay || !o)
            return fail(KDA_ERR_NULL_ARG, "a tensor argument of kda_decay_fwd is NULL");
        s = check_align({{q, "q"}, {k, "k"}, {v, "v"}, {initial_state, "initial_state"}, {o, "o"},
                         {final_state, "final_state"}});
        if (s != KDA_OK) return s;
        const int seg = auto_segment(d, 1);
        const size_t need = decay_ws(d, seg, false).total;
        if ((s = check_ws(workspace, workspace_bytes, need)) != KDA_OK) return s;
        const size_t st = (size_t)d.s.N * d.s.Hv * kState * 4;
        const std::vector<Span> ins = {
            {q, strided_bytes(d.s.tokens, d.sq, d.s.Hqk), "q"}, {k, strided_bytes(d.s.tokens, d.sk, d.s.Hqk), "k"},
            {v, strided_bytes(d.s.tokens, d.sv, d.s.Hv), "v"}, {log_decay, (size_t)d.s.Hv * 4, "log_decay"},
            {initial_state, initial_state ? st : 0, "initial_state"},
            {pp->cu_seqlens, d.packed ? (size_t)(d.s.N + 1) * 8 : 0, "cu_seqlens"}};
        s = check_overlap({{o, (size_t)d.s.tokens * d.s.Hv * D * 2, "o"},
                           {final_state, final_state ? st : 0, "final_state"},
                           {workspace, need, "workspace"}}, ins);
        if (s != KDA_OK) return s;
        hipStream_t stream = (hipStream_t)stream_;
        SeqPlan plan;
        kda::ItemMap m;
        if ((s = make_map(d, seg, stream, plan, m)) != KDA_OK) return s;
        if ((s = check_scan_grid(d, seg, m, 1)) != KDA_OK) return s;
        return run_forward(d, seg, m, 0, q, k, v, log_decay, initial_state, final_state, nullptr, d.s.N, o,
                           (char*)workspace, stream);
    });
}

kda_status kda_decay_bwd(const kda_decay_problem* pp, const void* q, const void* k, const void* v,
                         const float* log_decay, const float* initial_state, const void* d_o,
                         const float* dfinal_state, void* dq, void* dk, void* dv, float* dinitial_state,
                         void* workspace, size_t workspace_bytes, void* stream_) {
    return guarded([&]() -> kda_status {
        Decay d;
        kda_status s = check_decay(pp, d);
        if (s != KDA_OK) return s;
        if (!q || !k || !v || !log_decay || !d_o || !dq || !dk || !dv)
            return fail(KDA_ERR_NULL_ARG, "a tensor argument of kda_decay_bwd is NULL");
        s = check_align({{q, "q"}, {k, "k"}, {v, "v"}, {initial_state, "initial_state"}, {d_o, "do"},
                         {dfinal_state, "dfinal_state"}, {dq, "dq"}, {dk, "dk"}, {dv, "dv"},
                         {dinitial_state, "dinitial_state"}});
        if (s != KDA_OK) return s;
        const int seg = auto_segment(d, 3);
        const DecayWs wl = decay_ws(d, seg, true);
        if ((s = check_ws(workspace, workspace_bytes, wl.total)) != KDA_OK) return s;
        const size_t st = (size_t)d.s.N * d.s.Hv * kState * 4;
        const size_t tq = (size_t)d.s.tokens * d.s.Hqk * D * 2, tv = (size_t)d.s.tokens * d.s.Hv * D * 2;
        const std::vector<Span> ins = {
            {q, strided_bytes(d.s.tokens, d.sq, d.s.Hqk), "q"}, {k, strided_bytes(d.s.tokens, d.sk, d.s.Hqk), "k"},
            {v, strided_bytes(d.s.tokens, d.sv, d.s.Hv), "v"}, {log_decay, (size_t)d.s.Hv * 4, "log_decay"},
            {initial_state, initial_state ? st : 0, "initial_state"}, {d_o, tv, "do"},
            {dfinal_state, dfinal_state ? st : 0, "dfinal_state"},
            {pp->cu_seqlens, d.packed ? (size_t)(d.s.N + 1) * 8 : 0, "cu_seqlens"}};
        s = check_overlap({{dq, tq, "dq"}, {dk, tq, "dk"}, {dv, tv, "dv"},
                           {dinitial_state, dinitial_state ? st : 0, "dinitial_state"},
                           {workspace, wl.total, "workspace"}}, ins);
        if (s != KDA_OK) return s;
        hipStream_t stream = (hipStream_t)stream_;
        SeqPlan plan;
        kda::ItemMap m;
        if ((s = make_map(d, seg, stream, plan, m)) != KDA_OK) return s;
        if ((s = check_scan_grid(d, seg, m, 3)) != KDA_OK) return s;
        if (d.s.G > 1 && (s = check_grid((d.s.tokens * d.s.Hqk * (D / 8) + 255) / 256)) != KDA_OK) return s;

        char* ws = (char*)workspace;
        const int G = d.s.G;
        const kda::ScanRows rq = {(const kda::bf16_t*)q, d.sq, G}, rk = {(const kda::bf16_t*)k, d.sk, G},
                            rv = {(const kda::bf16_t*)v, d.sv, 1},
                            ro = {(const kda::bf16_t*)d_o, (int64_t)d.s.Hv * D, 1};
        const int pack = G > 1;
        kda::ScanArgs a{};
        a.map = m;
        a.jobs = 3;
        a.share = 3 * xcd_share(G, true);
        a.log_decay = log_decay;
        a.scale = d.scale;
        a.slots = d.s.N;
        // dk: (v, do, q) backward in time, the state read transposed
        kda::ScanJob& jk = a.job[0];
        jk.a = rv; jk.b = ro; jk.c = rq;
        jk.y = pack ? (void*)(ws + wl.part_k) : dk;
        jk.pack = pack;
        jk.reverse = 1;
        jk.s_in = dfinal_state;
        jk.s_in_t = 1;
        // dv: (k, q, do) backward in time; its state ends as dinitial_state
        kda::ScanJob& jv = a.job[1];
        jv.a = rk; jv.b = rq; jv.c = ro;
        jv.y = dv;
        jv.reverse = 1;
        jv.s_in = dfinal_state;
        jv.s_out = dinitial_state;
        // dq: (do, v, k) forward in time, the state read transposed
        kda::ScanJob& jq = a.job[2];
        jq.a = ro; jq.b = rv; jq.c = rk;
        jq.y = pack ? (void*)(ws + wl.part_q) : dq;
        jq.pack = pack;
        jq.s_in = initial_state;
        jq.s_in_t = 1;

        hipError_t e;
        if (seg != 0) {
            float* fwd = (float*)(ws + wl.seg_f);
            float* bwd = (float*)(ws + wl.seg_r);
            // the segments' own sums: of v k^T forward, of do q^T backward in time
            kda::ScanArgs b = a;
            b.jobs = 2;
            b.share = 2 * xcd_share(G, true);
            b.by_seg = 1;
            b.job[0] = b.job[1] = kda::ScanJob{};
            b.job[0].b = rk; b.job[0].c = rv;
            b.job[0].s_out = fwd;
            b.job[1].b = rq; b.job[1].c = ro;
            b.job[1].s_out = bwd;
            b.job[1].reverse = 1;
            e = kda::launch_decay_scan(b, true, stream);
            if (e != hipSuccess) return hip_fail(e, "segment state launch");
            kda::ChainArgs c{};
            c.map = m;
            c.jobs = 2;
            c.job[0] = {fwd, initial_state, nullptr, 0};
            c.job[1] = {bwd, dfinal_state, dinitial_state, 1};
            c.log_decay = log_decay;
            c.slots = d.s.N;
            e = kda::launch_decay_chain(c, stream);
            if (e != hipSuccess) return hip_fail(e, "segment chain launch");
            jq.s_in = fwd;
            jk.s_in = jv.s_in = bwd;
            jv.s_out = nullptr;
            a.by_seg = 1;
        }
        e = kda::launch_decay_scan(a, false, stream);
        if (e != hipSuccess) return hip_fail(e, "decay adjoint launch");
        if (G > 1) {
            e = kda::launch_decay_group_sum(ws + wl.part_q, ws + wl.part_k,
                                            (kda::bf16_t*)dq, (kda::bf16_t*)dk, d.s.tokens, d.s.Hqk, G, stream);
            if (e != hipSuccess) return hip_fail(e, "group sum launch");
        }
        return KDA_OK;
    });
}

kda_status kda_decay_infer_workspace_bytes(const kda_decay_problem* pp, size_t* bytes) {
    return guarded([&]() -> kda_status {
        Decay d;
        kda_status s = check_decay(pp, d);
        if (s != KDA_OK) return s;
        if (bytes == nullptr) return fail(KDA_ERR_NULL_ARG, "bytes is NULL");
        *bytes = infer_plan(d).ws;
        return KDA_OK;
    });
}

kda_status kda_decay_infer(const kda_decay_problem* pp, const void* q, const void* k, const void* v,
                           const float* log_decay, float* state_pool, int64_t pool_slots,
                           const int32_t* state_indices, const int32_t* state_indices_host, void* o,
                           void* workspace, size_t workspace_bytes, void* stream_) {
    return guarded([&]() -> kda_status {
        Decay d;
        kda_status s = check_decay(pp, d);
        if (s != KDA_OK) return s;
        if (!q || !k || !v || !log_decay || !state_pool || !o)
            return fail(KDA_ERR_NULL_ARG, "a tensor argument of kda_decay_infer is NULL");
        s = check_align({{q, "q"}, {k, "k"}, {v, "v"}, {state_pool, "state_pool"}, {o, "o"}});
        if (s != KDA_OK) return s;
        if (pool_slots < 1 || pool_slots > ((int64_t)1 << 40) / ((int64_t)d.s.Hv * kState))
            return fail(KDA_ERR_SHAPE, "pool_slots out of range (%lld)", (long long)pool_slots);
        if ((state_indices == nullptr) != (state_indices_host == nullptr))
            return fail(KDA_ERR_NULL_ARG, "state_indices and state_indices_host go together");
        if (state_indices_host != nullptr) {
            std::vector<int32_t> sorted(state_indices_host, state_indices_host + d.s.N);
            for (int i = 0; i < d.s.N; ++i)
                if (sorted[i] < 0 || sorted[i] >= pool_slots)
                    return fail(KDA_ERR_SHAPE, "state_indices[%d] = %d is outside the pool", i, sorted[i]);
            std::sort(sorted.begin(), sorted.end());
            for (int i = 1; i < d.s.N; ++i)
                if (sorted[i] == sorted[i - 1])
                    return fail(KDA_ERR_SHAPE, "pool slot %d is named twice", sorted[i]);
        } else if (pool_slots < d.s.N) {
            return fail(KDA_ERR_SHAPE, "without state_indices the pool needs N=%d slots (has %lld)", d.s.N,
                        (long long)pool_slots);
        }
        const InferPlan ip = infer_plan(d);
        if ((s = check_ws(workspace, workspace_bytes, ip.ws)) != KDA_OK) return s;
        const std::vector<Span> ins = {
            {q, strided_bytes(d.s.tokens, d.sq, d.s.Hqk), "q"}, {k, strided_bytes(d.s.tokens, d.sk, d.s.Hqk), "k"},
            {v, strided_bytes(d.s.tokens, d.sv, d.s.Hv), "v"}, {log_decay, (size_t)d.s.Hv * 4, "log_decay"},
            {pp->cu_seqlens, d.packed ? (size_t)(d.s.N + 1) * 8 : 0, "cu_seqlens"},
            {state_indices, state_indices ? (size_t)d.s.N * 4 : 0, "state_indices"}};
        s = check_overlap({{o, (size_t)d.s.tokens * d.s.Hv * D * 2, "o"},
                           {state_pool, (size_t)pool_slots * d.s.Hv * kState * 4, "state_pool"},
                           {workspace, ip.ws, "workspace"}}, ins);
        if (s != KDA_OK) return s;
        hipStream_t stream = (hipStream_t)stream_;
        SeqPlan plan;
        kda::ItemMap m;
        if ((s = make_map(d, ip.seg, stream, plan, m)) != KDA_OK) return s;
        m.items = (ip.seg ? ip.segs : ip.chunked) * d.s.Hv;
        const int64_t serial = d.s.N - ip.chunked;
        if ((s = check_scan_grid(d, ip.seg, m, 1)) != KDA_OK || (s = check_grid(serial * d.s.Hv * 4)) != KDA_OK)
            return s;
        if (ip.chunked != 0) {
            s = run_forward(d, ip.seg, m, kTokenSerialMax, q, k, v, log_decay, state_pool, state_pool, state_indices,
                            pool_slots, o, (char*)workspace, stream);
            if (s != KDA_OK || serial == 0) return s;
        }
        kda::TokenArgs t{};
        t.map = m;
        t.map.seg_len = 0;
        t.map.items = serial * d.s.Hv;
        if (d.packed) t.map.task = m.task + ip.chunked * d.s.Hv;
        t.q = (const kda::bf16_t*)q; t.sq = d.sq;
        t.k = (const kda::bf16_t*)k; t.sk = d.sk;
        t.v = (const kda::bf16_t*)v; t.sv = d.sv;
        t.G = d.s.G;
        t.o = (kda::bf16_t*)o;
        t.log_decay = log_decay;
        t.scale = d.scale;
        t.pool = state_pool;
        t.slot = state_indices;
        t.slots = pool_slots;
        hipError_t e = kda::launch_decay_token(t, stream);
        if (e != hipSuccess) return hip_fail(e, "decay decode launch");
        return KDA_OK;
    });
}

kda_status kda_qknorm_fwd(const kda_qknorm_problem* pp, const void* q, const void* k, const float* q_weight,
                          const float* k_weight, const float* cos, const float* sin, const int64_t* positions,
                          void* q_out, void* k_out, void* stream) {
    return guarded([&]() -> kda_status {
        kda::QkNormArgs a{};
        kda_status s = check_qknorm(pp, a);
        if (s != KDA_OK) return s;
        std::vector<Span> ins;
        if ((s = qknorm_inputs(pp, a, q, k, q_weight, k_weight, cos, sin, positions, ins)) != KDA_OK) return s;
        if (!q_out || !k_out) return fail(KDA_ERR_NULL_ARG, "an output of kda_qknorm_fwd is NULL");
        if ((s = check_align({{q_out, "q_out"}, {k_out, "k_out"}})) != KDA_OK) return s;
        s = check_overlap({{q_out, (size_t)a.tokens * a.Hq * D * 2, "q_out"},
                           {k_out, (size_t)a.tokens * a.Hk * D * 2, "k_out"}}, ins);
        if (s != KDA_OK) return s;
        a.yq = (kda::bf16_t*)q_out;
        a.yk = (kda::bf16_t*)k_out;
        hipError_t e = kda::launch_qknorm_fwd(a, (hipStream_t)stream);
        if (e != hipSuccess) return hip_fail(e, "query/key norm launch");
        return KDA_OK;
    });
}

kda_status kda_qknorm_bwd_workspace_bytes(const kda_qknorm_problem* pp, size_t* bytes) {
    return guarded([&]() -> kda_status {
        kda::QkNormArgs a{};
        kda_status s = check_qknorm(pp, a);
        if (s != KDA_OK) return s;
        if (bytes == nullptr) return fail(KDA_ERR_NULL_ARG, "bytes is NULL");
        *bytes = qknorm_ws(a);
        return KDA_OK;
    });
}

kda_status kda_qknorm_bwd(const kda_qknorm_problem* pp, const void* q, const void* k, const float* q_weight,
                          const float* k_weight, const float* cos, const float* sin, const int64_t* positions,
                          const void* dq_out, const void* dk_out, void* dq, void* dk, float* dq_weight,
                          float* dk_weight, void* workspace, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> kda_status {
        kda::QkNormArgs a{};
        kda_status s = check_qknorm(pp, a);
        if (s != KDA_OK) return s;
        std::vector<Span> ins;
        if ((s = qknorm_inputs(pp, a, q, k, q_weight, k_weight, cos, sin, positions, ins)) != KDA_OK) return s;
        if (!dq_out || !dk_out || !dq || !dk || !dq_weight || !dk_weight)
            return fail(KDA_ERR_NULL_ARG, "a gradient argument of kda_qknorm_bwd is NULL");
        if ((s = check_align({{dq_out, "dq_out"}, {dk_out, "dk_out"}, {dq, "dq"}, {dk, "dk"}})) != KDA_OK) return s;
        const size_t need = qknorm_ws(a);
        if ((s = check_ws(workspace, workspace_bytes, need)) != KDA_OK) return s;
        const size_t tq = (size_t)a.tokens * a.Hq * D * 2, tk = (size_t)a.tokens * a.Hk * D * 2;
        ins.push_back({dq_out, tq, "dq_out"});
        ins.push_back({dk_out, tk, "dk_out"});
        s = check_overlap({{dq, tq, "dq"}, {dk, tk, "dk"}, {dq_weight, D * 4, "dq_weight"},
                           {dk_weight, D * 4, "dk_weight"}, {workspace, need, "workspace"}}, ins);
        if (s != KDA_OK) return s;
        a.dyq = (const kda::bf16_t*)dq_out;
        a.dyk = (const kda::bf16_t*)dk_out;
        a.dq = (kda::bf16_t*)dq;
        a.dk = (kda::bf16_t*)dk;
        a.dwq = dq_weight;
        a.dwk = dk_weight;
        a.part = (float*)workspace;
        hipError_t e = kda::launch_qknorm_bwd(a, (hipStream_t)stream);
        if (e != hipSuccess) return hip_fail(e, "query/key norm backward launch");
        return KDA_OK;
    });
}

kda_status kda_gnorm_fwd(const kda_gnorm_problem* pp, const void* x, const void* gate, const float* weight, void* y,
                         void* stream) {
    return guarded([&]() -> kda_status {
        kda::GNormArgs a{};
        kda_status s = check_gnorm(pp, a);
        if (s != KDA_OK) return s;
        if (!x || !gate || !weight || !y) return fail(KDA_ERR_NULL_ARG, "a tensor argument of kda_gnorm_fwd is NULL");
        if ((s = check_align({{x, "x"}, {gate, "gate"}, {y, "y"}})) != KDA_OK) return s;
        s = check_overlap({{y, (size_t)a.tokens * a.H * D * 2, "y"}},
                          {{x, strided_bytes(a.tokens, a.sx, a.H), "x"},
                           {gate, strided_bytes(a.tokens, a.sg, a.H), "gate"}, {weight, D * 4, "weight"}});
        if (s != KDA_OK) return s;
        a.x = (const kda::bf16_t*)x;
        a.g = (const kda::bf16_t*)gate;
        a.w = weight;
        a.y = (kda::bf16_t*)y;
        hipError_t e = kda::launch_gnorm_fwd(a, (hipStream_t)stream);
        if (e != hipSuccess) return hip_fail(e, "gated norm launch");
        return KDA_OK;
    });
}

kda_status kda_gnorm_bwd_workspace_bytes(const kda_gnorm_problem* pp, size_t* bytes) {
    return guarded([&]() -> kda_status {
        kda::GNormArgs a{};
        kda_status s = check_gnorm(pp, a);
        if (s != KDA_OK) return s;
        if (bytes == nullptr) return fail(KDA_ERR_NULL_ARG, "bytes is NULL");
        *bytes = gnorm_ws(a);
        return KDA_OK;
    });
}

kda_status kda_gnorm_bwd(const kda_gnorm_problem* pp, const void* x, const void* gate, const float* weight,
                         const void* dy, void* dx, void* dgate, float* dweight, void* workspace,
                         size_t workspace_bytes, void* stream) {
    return guarded([&]() -> kda_status {
        kda::GNormArgs a{};
        kda_status s = check_gnorm(pp, a);
        if (s != KDA_OK) return s;
        if (!x || !gate || !weight || !dy || !dx || !dgate || !dweight)
            return fail(KDA_ERR_NULL_ARG, "a tensor argument of kda_gnorm_bwd is NULL");
        if ((s = check_align({{x, "x"}, {gate, "gate"}, {dy, "dy"}, {dx, "dx"}, {dgate, "dgate"}})) != KDA_OK) return s;
        const size_t need = gnorm_ws(a);
        if ((s = check_ws(workspace, workspace_bytes, need)) != KDA_OK) return s;
        const size_t row = (size_t)a.tokens * a.H * D * 2;
        s = check_overlap({{dx, row, "dx"}, {dgate, row, "dgate"}, {dweight, D * 4, "dweight"},
                           {workspace, need, "workspace"}},
                          {{x, strided_bytes(a.tokens, a.sx, a.H), "x"},
                           {gate, strided_bytes(a.tokens, a.sg, a.H), "gate"}, {weight, D * 4, "weight"},
                           {dy, row, "dy"}});
        if (s != KDA_OK) return s;
        a.x = (const kda::bf16_t*)x;
        a.g = (const kda::bf16_t*)gate;
        a.w = weight;
        a.dy = (const kda::bf16_t*)dy;
        a.dx = (kda::bf16_t*)dx;
        a.dg = (kda::bf16_t*)dgate;
        a.dw = dweight;
        a.part = (float*)workspace;
        hipError_t e = kda::launch_gnorm_bwd(a, (hipStream_t)stream);
        if (e != hipSuccess) return hip_fail(e, "gated norm backward launch");
        return KDA_OK;
    });
}

}  // extern "C"
