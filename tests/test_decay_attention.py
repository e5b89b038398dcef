"""GPU parity of linear attention with a constant decay per head (kda_decay_*)
against the FP64 recurrence: training forward and backward, prefill and decode
on a state pool, at the lengths, head layouts, strides and decays where the
chunked kernel can go wrong."""
import math

import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo
from tests import layer_util as lu

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128.0)

CASES = {  # lengths, packed, Hqk, Hv, segment
    "one_token": ([1], False, 1, 1, 0),
    "batch_of_one_token": ([1] * 5, False, 2, 2, 0),
    "chunk_edges": ([1, 15, 16, 17, 31, 33, 63, 64, 65], True, 1, 2, 0),
    "two_chunks": ([127, 128, 129], True, 2, 2, 0),
    "grouped": ([100] * 2, False, 2, 8, 0),
    "grouped_ragged": ([70, 3, 200], True, 1, 3, 0),
    "odd_heads": ([90, 41], True, 5, 5, 0),
    "segments_64": ([1, 64, 65, 300, 128], True, 1, 2, 64),
    "segments_128": ([130, 127, 500], True, 2, 4, 128),
    "segments_fixed": ([400] * 2, False, 1, 2, 192),
    "segments_auto": ([1500, 20, 700], True, 1, 2, 0),
    "long": ([2100], False, 2, 2, 0),
}


def decays(Hv):
    """Mild, strong, none, weak, total: the head's decay cycles through them."""
    table = [-0.05, -1.3, 0.0, -1e-4, -30.0, float("-inf"), -0.4]
    return torch.tensor([table[h % len(table)] for h in range(Hv)], dtype=torch.float32)


class Inp:
    def __init__(self, lengths, packed, Hqk, Hv, seed=0, state=True):
        g = torch.Generator().manual_seed(seed)
        B, T = (1, sum(lengths)) if packed else (len(lengths), lengths[0])
        N = len(lengths)
        self.lengths, self.packed, self.N, self.B, self.T, self.Hqk, self.Hv = lengths, packed, N, B, T, Hqk, Hv
        self.q, self.k, self.v = lu.bf(g, B, T, Hqk, 128), lu.bf(g, B, T, Hqk, 128), lu.bf(g, B, T, Hv, 128)
        self.do = lu.bf(g, B, T, Hv, 128)
        self.l = decays(Hv)
        self.s0 = torch.randn((N, Hv, 128, 128), generator=g) if state else None
        self.ds = torch.randn((N, Hv, 128, 128), generator=g) if state else None
        self.cu = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int64) if packed else None

    def dev(self, x):
        return None if x is None else x.cuda()

    def zeros(self):
        return torch.zeros(self.N, self.Hv, 128, 128)

    def reference(self, scale=SCALE):
        s0 = self.s0 if self.s0 is not None else self.zeros()
        return lo.decay_forward(lu.f64(self.q), lu.f64(self.k), lu.f64(self.v), lu.f64(self.l), lu.f64(s0),
                                self.lengths, self.packed, scale)

    def energies(self, scale=SCALE):
        """Of o, dq, dk and dv: the definitions at squared inputs."""
        s0 = self.s0 if self.s0 is not None else self.zeros()
        ds = self.ds if self.ds is not None else self.zeros()
        q, k, v, s0, do, ds = (lu.f64(x) ** 2 for x in (self.q, self.k, self.v, s0, self.do, ds))
        l = 2 * lu.f64(self.l)
        o = lo.decay_forward(q, k, v, l, s0, self.lengths, self.packed, scale ** 2)[0]
        return (o,) + lo.decay_backward(q, k, v, l, s0, do, ds, self.lengths, self.packed, scale ** 2)[:3]

    def gradients(self, scale=SCALE):
        s0 = self.s0 if self.s0 is not None else self.zeros()
        ds = self.ds if self.ds is not None else self.zeros()
        a = [lu.f64(x) for x in (self.q, self.k, self.v, self.l, s0, self.do, ds)]
        grads = lo.decay_backward(*a, self.lengths, self.packed, scale)
        # majorant of dinitial_state: the adjoint recurrence over absolute values
        a[0], a[5], a[6] = np.abs(a[0]), np.abs(a[5]), np.abs(a[6])
        return grads, lo.decay_backward(*a, self.lengths, self.packed, scale)[3]


def train(inp, segment=0, scale=None, wrap=lambda x: x):
    import gated_delta_rule_32_amd as kda
    q, k, v = (wrap(inp.dev(x)) for x in (inp.q, inp.k, inp.v))
    o, fs, ctx = kda.decay_attention_training_forward(q, k, v, inp.dev(inp.l), inp.dev(inp.s0), inp.dev(inp.cu), scale,
                                                      cu_seqlens_cpu=inp.cu, segment=segment)
    grads = kda.decay_attention_training_backward(ctx, inp.dev(inp.do), inp.dev(inp.ds))
    torch.cuda.synchronize()
    return (o, fs) + grads


def check_train(inp, got, scale=SCALE):
    o, final, major, mfinal = inp.reference(scale)
    (dq, dk, dv, dinit), minit = inp.gradients(scale)
    lu.check_bars("o, majorant", got[0], o, lu.U * np.abs(o) + 2 * lu.U * major)
    energies = inp.energies(scale)
    lu.check_scanned("o", got[0], o, energies[0])
    lu.check_state("final_state", got[1], final, mfinal)
    for name, x, ref, energy in zip(("dq", "dk", "dv"), got[2:5], (dq, dk, dv), energies[1:]):
        lu.check_scanned(name, x, ref, energy)
    lu.check_state("dinitial_state", got[5], dinit, minit)


@pytest.mark.parametrize("case", list(CASES))
def test_training_step(case):
    lengths, packed, Hqk, Hv, segment = CASES[case]
    print(f"[decay] case={case}", flush=True)
    inp = Inp(lengths, packed, Hqk, Hv, seed=len(case))
    check_train(inp, train(inp, segment))


@pytest.mark.parametrize("segment", [0, 64])
def test_no_states_given(segment):
    """initial_state and dfinal_state None count as zero."""
    inp = Inp([5, 150, 64], True, 1, 2, seed=3, state=False)
    check_train(inp, train(inp, segment))


def test_every_decay_of_the_table():
    inp = Inp([150, 1], True, 7, 7, seed=4)
    check_train(inp, train(inp))


def test_custom_scale():
    inp = Inp([80], False, 1, 1, seed=5)
    check_train(inp, train(inp, scale=0.25), scale=0.25)


@pytest.mark.parametrize("segment", [0, 64])
def test_slices_of_wider_rows(segment):
    """q, k and v as slices of one fused row, the rest of which is NaN."""
    inp = Inp([77, 130], True, 2, 4, seed=6)

    def wrap(x):
        B, T, H, _ = x.shape
        wide = torch.full((B, T, H + 3, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :, 1:H + 1] = x
        return wide[:, :, 1:H + 1]

    dense, sliced = train(inp, segment), train(inp, segment, wrap=wrap)
    for a, b in zip(dense, sliced):
        assert torch.equal(a, b)


def test_results_do_not_depend_on_the_packing():
    """A sequence's results are the same bits alone and between others, and NaN
    rows of the neighbours do not reach it."""
    inp = Inp([40, 100, 9], True, 1, 2, seed=7)
    got = train(inp)
    alone = Inp([100], False, 1, 2, seed=7)
    for name in ("q", "k", "v", "do"):
        setattr(alone, name, getattr(inp, name)[:, 40:140].contiguous())
    alone.s0, alone.ds = inp.s0[1:2].contiguous(), inp.ds[1:2].contiguous()
    ref = train(alone)
    for i in (0, 2, 3, 4):
        assert torch.equal(got[i][:, 40:140], ref[i])
    for i in (1, 5):
        assert torch.equal(got[i][1:2], ref[i])
    bad = float("nan")
    for x in (inp.q, inp.k, inp.v, inp.do):
        x[:, :40] = bad
        x[:, 140:] = bad
    got = train(inp)
    for i in (0, 2, 3, 4):
        assert torch.equal(got[i][:, 40:140], ref[i])


def test_segments_agree_with_whole_sequences():
    """The two routes differ by FP32 sums only: their states to 2^-17 of the
    majorant (2^-18 each)."""
    inp = Inp([777, 130], True, 2, 2, seed=8)
    a, b = train(inp, 0), train(inp, 64)
    _, _, _, mfinal = inp.reference()
    assert (np.abs(lu.f64(a[1]) - lu.f64(b[1])) <= 2 * lu.STATE * mfinal).all()
    lu.check_scanned("o of segments", b[0], inp.reference()[0], inp.energies()[0])


@pytest.mark.parametrize("l", [-1e-5, -1.7e-4, -0.0039])
@pytest.mark.parametrize("segment", [0, 4096, 65536])
def test_weak_decay_over_a_long_sequence(l, segment):
    """With k and v constant the state is a geometric sum, known exactly.

    Bar: with constant inputs every chunk rounds the same way.  It multiplies
    the state once and adds to it in six matrix products, each off by at most
    2^-23 of it (a matrix unit may cut instead of rounding), and a chunk's
    error lives for 1 / (1 - e^{64 l}) chunks, at most all 1024: 7 x 2^-23
    times that, plus the sums inside a chunk."""
    import gated_delta_rule_32_amd as kda
    L = 65536
    k = torch.zeros((1, L, 1, 128), dtype=torch.bfloat16, device="cuda")
    k[..., 5] = 1.0
    v = torch.zeros_like(k)
    v[..., 9] = 0.5
    _, fs, _ = kda.decay_attention_training_forward(k, k, v, torch.tensor([l], device="cuda"), segment=segment)
    l32 = float(np.float32(l))
    want = 0.5 * (1 - math.exp(l32 * L)) / (1 - math.exp(l32))
    got = float(fs[0, 0, 9, 5])
    memory = min(L / 64, 1 / (1 - math.exp(64 * l32)))
    assert abs(got - want) <= (lu.STATE + 7 * 2.0 ** -23 * memory) * want
    fs[0, 0, 9, 5] = 0
    assert not fs.any()


@pytest.mark.parametrize("l", [-1e-5, -3.3e-5, -1.7e-4])
@pytest.mark.parametrize("segment", [0, 4096, 65536])
def test_chunk_factors_do_not_drift(l, segment):
    """An initial state decays over 65536 tokens of zeros to e^{65536 l} of
    itself.  1024 roundings of the product, independent from element to
    element with standard deviation 2^-24 / sqrt(3) at most, add up to
    sqrt(1024) of one, and their mean over the 16384 elements to 1/128 of that:
    bars of 6 standard deviations for both, and for the mean 2^-24 more, the
    last rounding of the product of the factors, which all elements share.  A factor rounded the same way in
    every chunk would move the mean by up to 1024 x 2^-25 = 3e-5.  (Segment
    65536: no segments; 0: as many as the library takes.)"""
    import gated_delta_rule_32_amd as kda
    L = 65536
    x = torch.zeros((1, L, 1, 128), dtype=torch.bfloat16, device="cuda")
    s0 = torch.rand((1, 1, 128, 128), generator=torch.Generator().manual_seed(2)) + 1
    _, fs, _ = kda.decay_attention_training_forward(x, x, x, torch.tensor([l], device="cuda"), s0.cuda(),
                                                    segment=segment)
    off = lu.f64(fs) / (lu.f64(s0) * math.exp(float(np.float32(l)) * L)) - 1
    std = 32 * 2.0 ** -24 / 3 ** 0.5
    print(f"max {np.abs(off).max() / std:.2f}, mean {abs(off.mean()) / std:.4f} standard deviations", flush=True)
    assert np.abs(off).max() <= 6 * std and abs(off.mean()) <= 6 * std / 128 + 2.0 ** -24


def test_same_call_twice_gives_the_same_bits():
    inp = Inp([300, 64, 5], True, 2, 6, seed=9)
    for segment in (0, 64):
        for a, b in zip(train(inp, segment), train(inp, segment)):
            assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# state pool
# ---------------------------------------------------------------------------
def pool_call(inp, pool, slots, **kw):
    import gated_delta_rule_32_amd as kda
    idx = None if slots is None else torch.tensor(slots, dtype=torch.int32)
    out, same = kda.decay_attention(inp.dev(inp.q), inp.dev(inp.k), inp.dev(inp.v), inp.dev(inp.l), pool, None,
                                    inp.dev(inp.cu), None if idx is None else idx.cuda(), cu_seqlens_cpu=inp.cu,
                                    ssm_state_indices_cpu=idx, **kw)
    assert same is pool
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("lengths,packed,segment", [
    ([1] * 6, False, 0), ([1] * 6, True, 0), ([3] * 2, False, 0), ([8, 1, 5], True, 0),   # token by token
    ([9, 1, 70], True, 0), ([200], False, 0), ([300, 2, 64], True, 64)])                  # in chunks
def test_pool(lengths, packed, segment):
    inp = Inp(lengths, packed, 2, 4, seed=len(lengths))
    g = torch.Generator().manual_seed(1)
    slots = torch.randperm(len(lengths) + 3, generator=g)[:len(lengths)].tolist()
    pool0 = torch.randn((len(lengths) + 3, 4, 128, 128), generator=g)
    inp.s0 = pool0[slots]
    pool = pool0.cuda()
    out = pool_call(inp, pool, slots, segment=segment)
    o, final, major, mfinal = inp.reference()
    lu.check_scanned("o", out, o, inp.energies()[0])
    lu.check_state("pool", pool[slots], final, mfinal)
    rest = [i for i in range(len(lengths) + 3) if i not in slots]
    assert torch.equal(pool[rest].cpu(), pool0[rest])


def test_pool_without_indices_and_new_pool():
    import gated_delta_rule_32_amd as kda
    inp = Inp([70, 70], False, 1, 2, seed=2)
    pool = inp.s0.cuda()
    out = pool_call(inp, pool, None)
    o, final, _, mfinal = inp.reference()
    lu.check_scanned("o", out, o, inp.energies()[0])
    lu.check_state("pool", pool, final, mfinal)
    inp.s0 = None
    out, new = kda.decay_attention(inp.dev(inp.q), inp.dev(inp.k), inp.dev(inp.v), inp.dev(inp.l))
    lu.check_scanned("o from zero", out, inp.reference()[0], inp.energies()[0])
    lu.check_state("new pool", new, inp.reference()[1], inp.reference()[3])


def test_prefill_then_decode_equals_one_prefill():
    """A prompt in one call, and the same prompt split into a prefill and
    single tokens, end in the same state and outputs."""
    inp = Inp([90], False, 1, 2, seed=11)
    o, final, _, mfinal = inp.reference()
    pool = inp.s0.cuda()
    outs = []
    for a, b in [(0, 77)] + [(t, t + 1) for t in range(77, 90)]:
        part = Inp([b - a], False, 1, 2)
        part.q, part.k, part.v = (x[:, a:b].contiguous() for x in (inp.q, inp.k, inp.v))
        outs.append(pool_call(part, pool, None))
    lu.check_scanned("o", torch.cat(outs, 1), o, inp.energies()[0])
    # 13 more steps, each with a rounding of the factor and of the sum
    lu.check_bars("pool", pool, final, (lu.STATE + 26 * 2.0 ** -24) * mfinal)


def test_device_slot_outside_the_pool_is_skipped():
    """The kernels read the device copy of the indices: a sequence whose slot it
    places outside the pool is skipped, its output rows left as they were."""
    import gated_delta_rule_32_amd as kda
    for T, segment in ((1, 0), (100, 0), (100, 64)):
        inp = Inp([T] * 3, False, 1, 2, seed=12)
        pool0 = torch.randn((3, 2, 128, 128))
        pool = pool0.cuda()
        host = torch.tensor([2, 0, 1], dtype=torch.int32)
        dev = torch.tensor([2, -1, 3], dtype=torch.int32, device="cuda")
        out = torch.full((3, T, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        kda.decay_attention(inp.dev(inp.q), inp.dev(inp.k), inp.dev(inp.v), inp.dev(inp.l), pool,
                            ssm_state_indices=dev, ssm_state_indices_cpu=host, output=out, segment=segment)
        torch.cuda.synchronize()
        assert torch.equal(pool[:2].cpu(), pool0[:2])
        assert not torch.equal(pool[2].cpu(), pool0[2])
        assert (out[1:] == 7.0).all() and not (out[0] == 7.0).all(-1).any()


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------
def test_on_another_stream():
    inp = Inp([200, 31], True, 1, 2, seed=13)
    want = train(inp)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = train(inp)
    s.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("packed,segment", [(False, 0), (False, 64), (True, 0), (True, 64)])
def test_captured_step(packed, segment):
    """Forward and backward in one graph, replayed with eager calls between;
    every replay gives the eager bits, on changed inputs too.  A fixed-layout
    call needs no call before the capture."""
    import gated_delta_rule_32_amd as kda
    lengths = [150, 150] if not packed else [150, 7, 143]
    inp = Inp(lengths, packed, 1, 2, seed=14)
    d = {n: inp.dev(getattr(inp, n)) for n in ("q", "k", "v", "do", "l", "s0", "ds", "cu")}
    if packed:  # the schedule: made by one call, seen on the device by a second
        train(inp, segment)
        train(inp, segment)
    p = kda.KdaDecayProblem()
    p.B, p.T, p.Hqk, p.Hv, p.N, p.segment = inp.B, inp.T, 1, 2, inp.N, segment
    if packed:
        p.cu_seqlens, p.cu_seqlens_host = d["cu"].data_ptr(), inp.cu.data_ptr()
    outs = [torch.empty_like(d["v"]), torch.empty_like(d["s0"]), torch.empty_like(d["q"]), torch.empty_like(d["k"]),
            torch.empty_like(d["v"]), torch.empty_like(d["s0"])]
    ws = torch.empty(max(1, kda.kda_decay_fwd_workspace_bytes(p), kda.kda_decay_bwd_workspace_bytes(p)),
                     dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_decay_fwd(p, d["q"], d["k"], d["v"], d["l"], d["s0"], outs[0], outs[1], ws)
        kda.kda_decay_bwd(p, d["q"], d["k"], d["v"], d["l"], d["s0"], d["do"], d["ds"], *outs[2:], ws)
    for _ in range(3):
        for x in outs:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = train(inp, segment)
        for a, b in zip(want, outs):
            assert torch.equal(a, b)
        inp.v = inp.v.flip(1).contiguous()
        d["v"].copy_(inp.v)


def test_capture_of_a_packed_call_without_a_schedule_is_refused():
    import gated_delta_rule_32_amd as kda
    inp = Inp([11, 222, 33], True, 1, 1, seed=15)
    d = [inp.dev(x) for x in (inp.q, inp.k, inp.v, inp.l)]
    cu = inp.dev(inp.cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(kda.KdaValueError) as e:
            kda.decay_attention_training_forward(*d, cu_seqlens=cu, cu_seqlens_cpu=inp.cu)
        d[0].add_(0)  # something to capture
    assert e.value.status == kda.KDA_ERR_CAPTURE


def test_context_checks_versions():
    import gated_delta_rule_32_amd as kda
    inp = Inp([20], False, 1, 1)
    q, k, v = (inp.dev(x) for x in (inp.q, inp.k, inp.v))
    _, _, ctx = kda.decay_attention_training_forward(q, k, v, inp.dev(inp.l))
    k.add_(1)
    with pytest.raises(ValueError, match="changed after the forward"):
        kda.decay_attention_training_backward(ctx, inp.dev(inp.do))
