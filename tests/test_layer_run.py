"""GPU tests of the linear-attention layer operators as they are used: query/key
norm and rotation, decay attention and gated norm in one training step and in
serving, captured and on several streams; every launch variant; tensors beyond
32-bit offsets; NaN that must stay where it is.

Bars of the whole step.  u = 2^-8.  A BF16 rounding has a standard deviation of
at most u / sqrt(3) = 0.58 u of what it rounds, a scanned result one of 0.82 u
(tests/layer_util.py), and independent errors add in squares.  With decays
close to 1 no row of o is small against the others, so that its norm does not
enlarge an error.
  y: q and k rounded (0.58 u each), o (0.82 u), y itself (0.58 u): 1.3 u; bar 2 u.
  Gradients: do passes the norm's Jacobian at an o that is off by 1.2 u, which
  enters twice (its direction and its length) and is rounded: 2.4 u; the scan
  adds 0.82 u and its operands 0.58 u twice, the last stage 0.58 u: 2.8 u; bar 4 u.
Every single stage is held to its own bar besides, on the inputs it was given.
"""
import math

import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo
from tests import layer_util as lu

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128.0)
EPS = 1e-6


def rel(got, ref):
    return np.linalg.norm(lu.f64(got) - ref) / np.linalg.norm(ref)


class Layer:
    """One layer's tensors: fused token rows [q | k | v | gate]."""

    def __init__(self, lengths, Hqk, Hv, rot, seed):
        import gated_delta_rule_32_amd as kda
        g = torch.Generator().manual_seed(seed)
        T = sum(lengths)
        self.lengths, self.Hqk, self.Hv, self.rot, self.T = lengths, Hqk, Hv, rot, T
        self.rows = lu.bf(g, 1, T, 2 * Hqk + 2 * Hv, 128)
        self.wq, self.wk, self.wo = (1 + 0.2 * torch.randn(128, generator=g) for _ in range(3))
        self.l = -0.02 - 0.06 * torch.rand(Hv, generator=g)
        self.s0 = 3 * torch.randn((len(lengths), Hv, 128, 128), generator=g)
        self.dy = lu.bf(g, 1, T, Hv, 128)
        self.ds = torch.randn((len(lengths), Hv, 128, 128), generator=g)
        self.pos = torch.cat([torch.arange(L) for L in lengths])[None].contiguous()
        self.cu = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int64)
        self.cos, self.sin = kda.rotary_table(max(lengths), rot)

    def split(self, rows):
        a, b, c = self.Hqk, 2 * self.Hqk, 2 * self.Hqk + self.Hv
        return rows[:, :, :a], rows[:, :, a:b], rows[:, :, b:c], rows[:, :, c:]


def step(L, d):
    """Forward and backward of the layer; d: its tensors on the device."""
    import gated_delta_rule_32_amd as kda
    q, k, v, gate = L.split(d["rows"])
    rope = (q, k, d["wq"], d["wk"], L.cos, L.sin, d["pos"])
    qn, kn = kda.qk_norm_rope_forward(*rope)
    o, fs, ctx = kda.decay_attention_training_forward(qn, kn, v, d["l"], d["s0"], d["cu"], cu_seqlens_cpu=L.cu)
    y = kda.gated_norm_forward(o, gate, d["wo"], activation="silu")
    do, dgate, dwo = kda.gated_norm_backward(d["dy"], o, gate, d["wo"], activation="silu")
    dqn, dkn, dv, ds0 = kda.decay_attention_training_backward(ctx, do, d["ds"])
    dq, dk, dwq, dwk = kda.qk_norm_rope_backward(dqn, dkn, *rope)
    return dict(qn=qn, kn=kn, o=o, fs=fs, y=y, do=do, dgate=dgate, dwo=dwo, dqn=dqn, dkn=dkn, dv=dv, ds0=ds0, dq=dq,
                dk=dk, dwq=dwq, dwk=dwk)


def on_device(L):
    return {n: getattr(L, n).cuda() for n in ("rows", "wq", "wk", "wo", "l", "s0", "dy", "ds", "pos", "cu")}


def test_training_step_of_a_layer():
    L = Layer([130, 1, 77], 2, 4, 64, seed=1)
    got = step(L, on_device(L))
    torch.cuda.synchronize()
    q, k, v, gate = (lu.f64(x) for x in L.split(L.rows))
    c, s, pos = lu.f64(L.cos), lu.f64(L.sin), L.pos.numpy()
    wq, wk, wo, l, s0, ds = (lu.f64(x) for x in (L.wq, L.wk, L.wo, L.l, L.s0, L.ds))
    rope = lambda x, w: lo.qk_norm_rope(x, w, c, s, pos, L.rot, False, EPS)  # noqa: E731
    qn, kn = rope(q, wq), rope(k, wk)
    o, fs, _, mfinal = lo.decay_forward(qn, kn, v, l, s0, L.lengths, True, SCALE)
    y = lo.gated_norm(o, gate, wo, True, EPS)
    do, dgate, dwo = lo.gated_norm_backward(lu.f64(L.dy), o, gate, wo, True, EPS)
    dqn, dkn, dv, ds0 = lo.decay_backward(qn, kn, v, l, s0, do, ds, L.lengths, True, SCALE)
    dq, dwq = lo.qk_norm_rope_backward(dqn, q, wq, c, s, pos, L.rot, False, EPS)
    dk, dwk = lo.qk_norm_rope_backward(dkn, k, wk, c, s, pos, L.rot, False, EPS)
    for name, ref, bar in (("y", y, 2), ("dgate", dgate, 4), ("dwo", dwo, 4), ("dv", dv, 4), ("dq", dq, 4),
                           ("dk", dk, 4), ("dwq", dwq, 4), ("dwk", dwk, 4), ("ds0", ds0, 4), ("fs", fs, 2)):
        e = rel(got[name], ref)
        print(f"{name:6s} {e / lu.U:.2f} u (bar {bar} u)", flush=True)
        assert e <= bar * lu.U, name
    # every stage on the inputs it was given
    gq, gk, go, gdo = (lu.f64(got[n]) for n in ("qn", "kn", "o", "do"))
    e2 = lambda *a: tuple(x ** 2 for x in a)  # noqa: E731
    ref = lo.decay_forward(gq, gk, v, l, s0, L.lengths, True, SCALE)
    energy = lo.decay_forward(*e2(gq, gk, v), 2 * l, s0 ** 2, L.lengths, True, SCALE ** 2)[0]
    lu.check_scanned("o", got["o"], ref[0], energy)
    lu.check_state("final_state", got["fs"], ref[1], ref[3])
    refs = lo.decay_backward(gq, gk, v, l, s0, gdo, ds, L.lengths, True, SCALE)
    energies = lo.decay_backward(*e2(gq, gk, v), 2 * l, *e2(s0, gdo, ds), L.lengths, True, SCALE ** 2)
    for name, r, e in zip(("dqn", "dkn", "dv"), refs, energies):
        lu.check_scanned(name, got[name], r, e)
    y = lo.gated_norm(go, gate, wo, True, EPS)
    lu.check_bars("y", got["y"], y, lu.U * np.abs(y) * (1 + lu.U) + 2.0 ** -20 * np.abs(y))


def test_training_step_replayed():
    """The whole step in one graph, with new inputs and eager steps between the
    replays: the eager bits every time."""
    L = Layer([64, 200, 9], 1, 3, 128, seed=2)
    d = on_device(L)
    step(L, d)     # a packed call's schedule is made by one call and seen by a second
    step(L, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(L, d)
    for i in range(4):
        for x in got.values():
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = step(L, d)
        for n in got:
            assert torch.equal(got[n], want[n]), n
        d["rows"].copy_(d["rows"].roll(i + 1, 1))
        d["dy"].copy_(d["dy"].flip(1))


def serve(L, d, pool, slots, slots_cpu, out=None):
    import gated_delta_rule_32_amd as kda
    q, k, v, gate = L.split(d["rows"])
    qn, kn = kda.qk_norm_rope_forward(q, k, d["wq"], d["wk"], L.cos, L.sin, d["pos"])
    o, _ = kda.decay_attention(qn, kn, v, d["l"], pool, None, d.get("cu"), slots,
                               cu_seqlens_cpu=None if d.get("cu") is None else L.cu, ssm_state_indices_cpu=slots_cpu)
    return kda.gated_norm_forward(o, gate, d["wo"], out=out)


def test_prefill_and_captured_decode_of_a_layer():
    """Prompts in one packed call, then single tokens of all of them in a
    captured step whose rows, positions and slots change between replays; the
    bits are those of eager calls, the values those of the definition."""
    lengths, steps = [37, 70, 5], 6
    L = Layer([n + steps for n in lengths], 2, 4, 128, seed=3)
    at = L.cu.tolist()
    full = on_device(L)
    pool = torch.zeros((5, 4, 128, 128), device="cuda")
    order = [3, 0, 4]
    pool[order] = full["s0"]
    untouched = pool[[1, 2]].clone()
    pre = Layer(lengths, 2, 4, 128, seed=3)
    pick = torch.cat([torch.arange(at[n], at[n] + lengths[n]) for n in range(3)]).cuda()
    p = dict(full, rows=full["rows"][:, pick].contiguous(), pos=full["pos"][:, pick].contiguous(), cu=pre.cu.cuda())
    pre.cos, pre.sin = L.cos, L.sin
    host = torch.tensor(order, dtype=torch.int32)
    slots = host.cuda()
    outs = [serve(pre, p, pool, slots, host)]
    after_prefill = pool.clone()

    one = dict(full, rows=full["rows"][0, at[:3]][:, None].contiguous(), pos=full["pos"][0, at[:3]][:, None].contiguous())
    one.pop("cu")
    y = torch.empty((3, 1, 4, 128), dtype=torch.bfloat16, device="cuda")
    serve(L, one, pool.clone(), slots, host, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        serve(L, one, pool, slots, host, y)
    eager = after_prefill.clone()
    for t in range(steps):
        token = [at[n] + lengths[n] + t for n in range(3)]
        seqs = [0, 1, 2] if t % 2 == 0 else [2, 0, 1]    # the batch's order changes
        one["rows"].copy_(full["rows"][0, [token[n] for n in seqs]][:, None])
        one["pos"].copy_(full["pos"][0, [token[n] for n in seqs]][:, None])
        slots.copy_(torch.tensor([order[n] for n in seqs], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = serve(L, one, eager, slots, host)
        assert torch.equal(want, y) and torch.equal(pool, eager)
        outs.append(y[[seqs.index(n) for n in range(3)]].clone())
    assert torch.equal(pool[[1, 2]], untouched)
    # against the definition
    q, k, v, gate = (lu.f64(x) for x in L.split(L.rows))
    c, s, pos = lu.f64(L.cos), lu.f64(L.sin), L.pos.numpy()
    qn = lo.qk_norm_rope(q, lu.f64(L.wq), c, s, pos, 128, False, EPS)
    kn = lo.qk_norm_rope(k, lu.f64(L.wk), c, s, pos, 128, False, EPS)
    o, final, _, _ = lo.decay_forward(qn, kn, v, lu.f64(L.l), lu.f64(L.s0), L.lengths, True, SCALE)
    ref = lo.gated_norm(o, gate, lu.f64(L.wo), False, EPS)
    assert rel(outs[0][0], ref[0, pick.cpu().numpy()]) <= 2 * lu.U
    for t in range(steps):
        rows = [at[n] + lengths[n] + t for n in range(3)]
        assert rel(outs[1 + t][:, 0], ref[0, rows]) <= 2 * lu.U
    assert rel(pool[order], final) <= 2 * lu.U


def test_replayed_decode_skips_slots_outside_the_pool():
    """Padding of a captured batch: slot -1 on the device leaves its output row
    and every state as they were."""
    import gated_delta_rule_32_amd as kda
    g = torch.Generator().manual_seed(4)
    q, k, v = (lu.bf(g, 4, 1, 2, 128).cuda() for _ in range(3))
    l = torch.tensor([-0.1, -0.7], device="cuda")
    pool = torch.randn((6, 2, 128, 128), generator=g).cuda()
    host = torch.arange(4, dtype=torch.int32)
    slots, o = host.cuda(), torch.zeros((4, 1, 2, 128), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.decay_attention(q, k, v, l, pool, ssm_state_indices=slots, ssm_state_indices_cpu=host, output=o)
    for choice in ([5, 2, -1, -1], [-1, 0, 4, 7], [3, 1, 2, 0]):
        before = pool.clone()
        o.fill_(9.0)
        slots.copy_(torch.tensor(choice, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        used = [c for c in choice if 0 <= c < 6]
        for b, c in enumerate(choice):
            if c not in used:
                assert (o[b] == 9.0).all()
                continue
            S = before[c] * l.exp()[:, None, None] + v[b, 0].float()[:, :, None] * k[b, 0].float()[:, None, :]
            assert torch.allclose(pool[c], S, rtol=2.0 ** -20, atol=2.0 ** -20)
        rest = [c for c in range(6) if c not in used]
        assert torch.equal(pool[rest], before[rest])


# ---------------------------------------------------------------------------
# streams and graphs at the same time
# ---------------------------------------------------------------------------
def test_two_streams_at_once():
    """Steps of two layers on two streams, the first call of a packed shape
    included, which both streams then share."""
    a, b = Layer([41, 190, 22], 1, 2, 64, seed=5), Layer([41, 190, 22], 1, 2, 64, seed=6)
    da, db = on_device(a), on_device(b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    runs = []
    for _ in range(3):
        for L, d, s in ((a, da, streams[0]), (b, db, streams[1])):
            with torch.cuda.stream(s):
                runs.append(step(L, d))
    torch.cuda.synchronize()
    want = [step(a, da), step(b, db)]
    for i, got in enumerate(runs):
        for n in got:
            assert torch.equal(got[n], want[i % 2][n]), n


def test_two_graphs_at_once():
    """Two graphs, each with workspaces of its own, replayed on two streams."""
    layers = [Layer([300], 2, 2, 128, seed=7), Layer([300], 2, 2, 128, seed=8)]
    ds = [on_device(L) for L in layers]
    want = [step(L, d) for L, d in zip(layers, ds)]
    want = [step(L, d) for L, d in zip(layers, ds)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for L, d in zip(layers, ds):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(step(L, d))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for x in (*got[0].values(), *got[1].values()):
            x.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            for n in want[i]:
                assert torch.equal(got[i][n], want[i][n]), n


# ---------------------------------------------------------------------------
# launch variants
# ---------------------------------------------------------------------------
from tests.test_decay_attention import Inp, check_train, train  # noqa: E402

VARIANTS = {  # lengths, Hqk, Hv, segment: few, more and many workgroups, whole and cut, single and grouped heads
    "forward_150_backward_450": ([20] * 50, 3, 3, 0),
    "forward_72_backward_216_grouped": ([70, 33] * 12, 1, 3, 0),
    "forward_300_backward_900": ([5, 40, 33] * 25, 4, 4, 0),
    "forward_400_backward_1200_grouped": ([9, 34] * 50, 2, 4, 0),
    "segments_150": ([300] * 10, 3, 3, 64),
    "segments_300_grouped": ([130] * 50, 1, 2, 64),
}


@pytest.mark.parametrize("case", list(VARIANTS))
def test_every_launch_variant(case):
    lengths, Hqk, Hv, segment = VARIANTS[case]
    print(f"[variant] {case}", flush=True)
    inp = Inp(lengths, True, Hqk, Hv, seed=len(case))
    check_train(inp, train(inp, segment))


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 50])
def test_size_of_grouped_gradients(size):
    """The packed partials of shared heads keep their precision at any size."""
    inp = Inp([70, 20], True, 2, 6, seed=20)
    for name in ("do", "ds"):
        x = getattr(inp, name)
        setattr(inp, name, x * size)
    check_train(inp, train(inp))


def test_many_sequences_decode_like_few():
    """2560 states of a call (non-temporal) like the same in four calls, bit for bit."""
    import gated_delta_rule_32_amd as kda
    g = torch.Generator(device="cuda").manual_seed(21)
    q, k, v = (torch.randn((40, 1, 64, 128), generator=g, device="cuda").bfloat16() for _ in range(3))
    l = -torch.rand(64, generator=g, device="cuda")
    pool = torch.randn((40, 64, 128, 128), generator=g, device="cuda")
    parts = pool.clone()
    o, _ = kda.decay_attention(q, k, v, l, pool)
    for i in range(0, 40, 10):
        c = slice(i, i + 10)
        p, _ = kda.decay_attention(q[c], k[c], v[c], l, parts[c])
        assert torch.equal(p, o[c])
    assert torch.equal(pool, parts)


def test_large_forward_like_a_small_one():
    """A forward that exceeds the caches (non-temporal) gives the bits of one over
    the first half of every sequence."""
    import gated_delta_rule_32_amd as kda
    g = torch.Generator(device="cuda").manual_seed(28)
    q, k, v = (torch.randn((12, 1000, 24, 128), generator=g, device="cuda").bfloat16() for _ in range(3))
    assert 4 * 12 * 1000 * 24 * 256 > 2 ** 28 > 4 * 12 * 500 * 24 * 256
    l = -0.2 * torch.rand(24, generator=g, device="cuda")
    half = [x[:, :500].contiguous() for x in (q, k, v)]
    a = kda.decay_attention_training_forward(q, k, v, l, segment=65536)[0]
    b, state, _ = kda.decay_attention_training_forward(*half, l, segment=65536)
    assert torch.equal(a[:, :500], b)
    # and the second half from the state in between (in other chunks: 500 = 15 x 32 + 20)
    rest = [x[:, 500:].contiguous() for x in (q, k, v)]
    c = kda.decay_attention_training_forward(*rest, l, state, segment=65536)[0]
    assert rel(c, lu.f64(a[:, 500:])) <= 2 * lu.U


def weight_bar(rows):
    """Of the sum of absolute values: a lane adds every 16384th row (and up to 8
    in a run), 16 lanes, 1024 workgroups in runs of 32 are added up, each sum off
    by 2^-24; a term itself by 2^-20."""
    return 2.0 ** -24 * (rows / 16384 + 8 + 16 + 32 + 32) + 2.0 ** -20


def test_large_row_norms_like_small_ones():
    """A pass that exceeds the caches (non-temporal, 8 heads per unit) gives the
    rows that a small call gives; weight gradients against 64 bits."""
    import gated_delta_rule_32_amd as kda
    g = torch.Generator(device="cuda").manual_seed(22)
    T, Hq, Hk = 16400, 32, 9
    q, k, dq, dk = (torch.randn((1, T, h, 128), generator=g, device="cuda").bfloat16() for h in (Hq, Hk, Hq, Hk))
    wq, wk = (torch.randn(128, generator=g, device="cuda") for _ in range(2))
    cos, sin = kda.rotary_table(T, 96)
    pos = torch.randint(T, (1, T), generator=g, device="cuda")
    cut = slice(8000, 8030)
    small = [x[:, cut].contiguous() for x in (q, k, dq, dk, pos)]
    y = kda.qk_norm_rope_forward(q, k, wq, wk, cos, sin, pos)
    ys = kda.qk_norm_rope_forward(small[0], small[1], wq, wk, cos, sin, small[4])
    d = kda.qk_norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos)
    dsm = kda.qk_norm_rope_backward(small[2], small[3], small[0], small[1], wq, wk, cos, sin, small[4])
    for a, b in zip((*y, *d[:2]), (*ys, *dsm[:2])):
        assert torch.equal(a[:, cut], b)
    # dw = sum of (R^T dy) x^ over all rows
    c, s = (t[pos[0]].double()[:, None] for t in (cos, sin))
    for x, dy, dw in ((q, dq, d[2]), (k, dk, d[3])):
        x, dy = x[0].double(), dy[0].double()
        a, b = dy[..., :48], dy[..., 48:96]
        dn = torch.cat((c * a + s * b, c * b - s * a, dy[..., 96:]), -1)
        terms = dn * x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
        bar = weight_bar(T * (Hq + Hk)) * terms.abs().sum((0, 1))
        assert ((dw.double() - terms.sum((0, 1))).abs() <= bar).all()
    T, H = 8200, 96
    x, gate, dy = (torch.randn((1, T, H, 128), generator=g, device="cuda").bfloat16() for _ in range(3))
    small = [t[:, cut.start - 1000:cut.stop - 1000].contiguous() for t in (x, gate, dy)]
    y, ys = kda.gated_norm_forward(x, gate, wq), kda.gated_norm_forward(*small[:2], wq)
    d, dsm = kda.gated_norm_backward(dy, x, gate, wq), kda.gated_norm_backward(small[2], *small[:2], wq)
    for a, b in zip((y, *d[:2]), (ys, *dsm[:2])):
        assert torch.equal(a[:, cut.start - 1000:cut.stop - 1000], b)
    x, gate, dy = (t[0].double() for t in (x, gate, dy))
    terms = dy * x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * gate.sigmoid()
    bar = weight_bar(T * H) * terms.abs().sum((0, 1))
    assert ((d[2].double() - terms.sum((0, 1))).abs() <= bar).all()


# ---------------------------------------------------------------------------
# offsets beyond 32 bits
# ---------------------------------------------------------------------------
def test_token_strides_beyond_32_bits():
    """Rows whose last token lies behind 2^31 elements (and 2^32 bytes): the bits
    of dense calls."""
    import gated_delta_rule_32_amd as kda
    g = torch.Generator(device="cuda").manual_seed(23)
    T, H, stride = 1100, 2, 1 << 21
    wide = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda")
    at = lambda i: wide.as_strided((1, T, H, 128), (T * stride, stride, 128, 1), i * H * 128)  # noqa: E731
    dense = [torch.randn((1, T, H, 128), generator=g, device="cuda").bfloat16() for _ in range(3)]
    far = [at(i) for i in range(3)]
    for x, y in zip(far, dense):
        x.copy_(y)
    l = torch.tensor([-0.01, -0.3], device="cuda")
    w = torch.randn(128, generator=g, device="cuda")
    do = torch.randn((1, T, H, 128), generator=g, device="cuda").bfloat16()
    cos, sin = kda.rotary_table(T, 128)

    def run(q, k, v, segment):
        o, fs, ctx = kda.decay_attention_training_forward(q, k, v, l, segment=segment)
        rope = (q, k, w, w, cos, sin)
        return (o, fs, *kda.decay_attention_training_backward(ctx, do), *kda.qk_norm_rope_forward(*rope),
                *kda.qk_norm_rope_backward(do, do, *rope), kda.gated_norm_forward(q, v, w),
                *kda.gated_norm_backward(do, q, v, w), *kda.decay_attention(q, k, v, l))

    for segment in (65536, 128):
        for a, b in zip(run(*far, segment), run(*dense, segment)):
            assert torch.equal(a, b)


def test_outputs_beyond_32_bits():
    """Packed tokens, partials and pool slots behind 2^31 elements: the last
    sequence's results are the bits of a small batch of that sequence (of five,
    so that the same kernels run)."""
    import gated_delta_rule_32_amd as kda
    g = torch.Generator(device="cuda").manual_seed(24)
    Hqk, Hv = 32, 64
    lens = [1000] * 263 + [333]
    T = sum(lens)
    assert (T - 333) * Hv * 128 > 2 ** 31
    rnd = lambda h: torch.randn((1, T, h, 128), generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k, v, do = rnd(Hqk), rnd(Hqk), rnd(Hv), rnd(Hv)
    l = -torch.rand(Hv, generator=g, device="cuda")
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int64)
    last = slice(T - 333, T)
    one = [x[:, last].contiguous() for x in (q, k, v, do)]
    o, fs, ctx = kda.decay_attention_training_forward(q, k, v, l, cu_seqlens=cu.cuda(), cu_seqlens_cpu=cu, segment=65536)
    grads = kda.decay_attention_training_backward(ctx, do)
    five = [x.repeat(5, 1, 1, 1) for x in one]
    o5, fs5, ctx5 = kda.decay_attention_training_forward(*five[:3], l, segment=65536)
    grads5 = kda.decay_attention_training_backward(ctx5, five[3])
    assert torch.equal(fs[-1], fs5[4]) and torch.equal(grads[3][-1], grads5[3][4])
    for a, b in zip((o, *grads[:3]), (o5, *grads5[:3])):
        assert torch.equal(a[0, last], b[4])
    o1 = o5[4:].contiguous()
    del grads, ctx, fs
    w = torch.randn(128, generator=g, device="cuda")
    y, dx = kda.gated_norm_forward(o, v, w), kda.gated_norm_backward(do, o, v, w)
    assert torch.equal(y[:, last], kda.gated_norm_forward(o1, one[2], w))
    for a, b in zip(dx[:2], kda.gated_norm_backward(one[3], o1, one[2], w)):
        assert torch.equal(a[:, last], b)
    del y, dx
    cos, sin = kda.rotary_table(T, 64)
    pos = torch.arange(T, device="cuda")[None].contiguous()
    y = kda.qk_norm_rope_forward(v, q, w, w, cos, sin, pos)
    for a, b in zip(y, kda.qk_norm_rope_forward(one[2], one[0], w, w, cos, sin, pos[:, last].contiguous())):
        assert torch.equal(a[:, last], b)
    del q, k, v, do, o, y
    pool = torch.zeros((2100, Hv, 128, 128), device="cuda")
    assert 2098 * Hv * 128 * 128 > 2 ** 31
    start = torch.randn((Hv, 128, 128), generator=g, device="cuda")
    idx = torch.tensor([2099], dtype=torch.int32)
    for tokens in (1, 333):
        pool[2099] = start
        alone = start[None].clone()
        part = [x[:, :tokens].contiguous() for x in one[:3]]
        a, _ = kda.decay_attention(*part, l, pool, ssm_state_indices=idx.cuda(), ssm_state_indices_cpu=idx)
        b, _ = kda.decay_attention(*part, l, alone)
        assert torch.equal(a, b) and torch.equal(pool[2099:], alone) and not pool[:2099].any()


def test_context_checks_the_sequences_too():
    """The backward reads the lengths again: changed in between, it refuses."""
    import gated_delta_rule_32_amd as kda
    x = torch.zeros((1, 40, 1, 128), dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 15, 40])
    _, _, ctx = kda.decay_attention_training_forward(x, x, x, torch.zeros(1, device="cuda"), cu_seqlens=cu.cuda(),
                                                     cu_seqlens_cpu=cu)
    cu[1] = 20
    with pytest.raises(ValueError, match="changed after the forward"):
        kda.decay_attention_training_backward(ctx, x)


# ---------------------------------------------------------------------------
# NaN stays where it is
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("segment", [0, 64])
@pytest.mark.parametrize("Hqk", [2, 4])
def test_nan_stays_in_its_head(Hqk, segment):
    """A NaN in one value head's v and do reaches no other head's results, and of
    the shared heads' gradients only its own."""
    inp = Inp([150, 40], True, Hqk, 4, seed=25)
    inp.l = torch.full((4,), -0.05)
    want = train(inp, segment)
    inp.v[:, 20, 1, 3] = float("nan")
    inp.do[:, 100, 1, 7] = float("nan")
    got = train(inp, segment)
    heads, shared = [0, 2, 3], [h for h in range(Hqk) if h != 1 * Hqk // 4]
    assert torch.equal(got[0][:, :, heads], want[0][:, :, heads])
    assert torch.equal(got[1][:, heads], want[1][:, heads]) and torch.equal(got[5][:, heads], want[5][:, heads])
    assert torch.equal(got[4][:, :, heads], want[4][:, :, heads])
    for i in (2, 3):
        assert torch.equal(got[i][:, :, shared], want[i][:, :, shared])
    # it is seen where it belongs: o's channel 3 of the head from the chunk on, the
    # rows of dq and dk that its do or v enters
    assert torch.isnan(got[0][0, 32:150, 1, 3]).all() and torch.isfinite(got[0][0, 32:150, 1, 4:]).all()
    own = 1 * Hqk // 4
    assert torch.isnan(got[2][0, 100, own]).all() and torch.isnan(got[3][0, 20, own]).all()
    # the other sequence is untouched
    for i in (0, 2, 3, 4):
        assert torch.equal(got[i][:, 150:], want[i][:, 150:])


def test_nan_rows_of_the_norms_stay_alone():
    import gated_delta_rule_32_amd as kda
    g = torch.Generator().manual_seed(26)
    x, gate, dy = (lu.bf(g, 1, 40, 3, 128).cuda() for _ in range(3))
    w = torch.randn(128, generator=g).cuda()
    cos, sin = kda.rotary_table(40, 128)
    run = lambda: (kda.gated_norm_forward(x, gate, w), *kda.gated_norm_backward(dy, x, gate, w)[:2],  # noqa: E731
                   *kda.qk_norm_rope_forward(x, gate, w, w, cos, sin)[:1],
                   *kda.qk_norm_rope_backward(dy, dy, x, gate, w, w, cos, sin)[:1])
    want = run()
    x[0, 7, 1, 5] = float("nan")
    x[0, 9, 2, 0] = float("inf")
    for a, b in zip(run(), want):
        bad = torch.isnan(a).any(-1)[0]
        assert bad[7, 1] and bad[9, 2] and bad.sum() == 2
        keep = ~bad
        assert torch.equal(a[0][keep], b[0][keep])


def test_a_masked_gate():
    """Gates of minus and plus infinity and of the type's lowest and highest
    value: outputs 0 or the normed row, gradients finite."""
    import gated_delta_rule_32_amd as kda
    g = torch.Generator().manual_seed(27)
    x, dy = lu.bf(g, 1, 4, 1, 128), lu.bf(g, 1, 4, 1, 128)
    top = torch.finfo(torch.bfloat16).max
    gate = torch.tensor([-math.inf, math.inf, -top, top])[None, :, None, None].expand(1, 4, 1, 128).to(torch.bfloat16)
    w = torch.ones(128)
    y = kda.gated_norm_forward(x.cuda(), gate.contiguous().cuda(), w.cuda())
    d = kda.gated_norm_backward(dy.cuda(), x.cuda(), gate.contiguous().cuda(), w.cuda())
    normed = lo.gated_norm(lu.f64(x), np.full(x.shape, 40.0), lu.f64(w), False, EPS)
    assert not y[0, [0, 2]].any()
    for t in (1, 3):
        lu.check_bars("y", y[0, t], normed[0, t], lu.U * np.abs(normed[0, t]) * (1 + lu.U) + 2.0 ** -20)
    assert all(torch.isfinite(t).all() for t in d) and not d[1].any()
    s = kda.gated_norm_forward(x.cuda(), gate.contiguous().cuda(), w.cuda(), activation="silu")
    assert not s[0, [0, 2]].any()
