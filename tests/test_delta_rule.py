"""GPU parity of the gated delta rule (kda_delta_*) against the FP64 recurrence:
training forward and backward, prefill, decode and drafted tokens on a state pool, at the
lengths, head layouts, strides and gates where the chunked kernels can go wrong."""
import numpy as np
import pytest
import torch

from tests import delta_util as du
from tests import layer_util as lu
from tests.delta_util import Inp

pytestmark = pytest.mark.gpu

CASES = {  # lengths, packed, Hqk, Hv, unit, gates
    "one_token": ([1], False, 1, 1, True, "layer"),
    "batch_of_one_token": ([1] * 5, False, 2, 2, True, "mixed"),
    "chunk_edges": ([1, 15, 16, 17, 31, 32, 33, 63, 64, 65], True, 1, 2, True, "mixed"),
    "block_edges": ([127, 128, 129, 97], True, 2, 2, True, "layer"),
    "grouped": ([100] * 2, False, 2, 8, True, "layer"),
    "grouped_ragged": ([70, 3, 200], True, 1, 3, False, "mixed"),
    "odd_heads": ([90, 41], True, 5, 5, False, "strong"),
    "no_decay": ([150, 33], True, 1, 2, True, "none"),
    "long": ([1100], False, 2, 2, True, "layer"),
    "many_tasks": ([40] * 11, False, 12, 12, True, "layer"),          # eight waves a workgroup
    "more_tasks": ([40] * 10, False, 16, 32, True, "mixed"),          # four waves a workgroup
}


def call_forward(inp, scale=None, wrap=lambda x: x, **more):
    import gated_delta_rule_32_amd as kda
    q, k, v = (wrap(inp.dev(x)) for x in (inp.q, inp.k, inp.v))
    r = kda.gated_delta_rule_training_forward(q, k, v, inp.dev(inp.g), inp.dev(inp.beta), inp.dev(inp.s0), inp.dev(inp.cu),
                                              scale, use_qk_l2norm=inp.unit, cu_seqlens_cpu=inp.cu, **more)
    torch.cuda.synchronize()
    return r


def check_forward(inp, got, scale=du.SCALE):
    o, final, (wo, wfinal), _ = inp.reference(scale)
    du.check_o("o", got[0], o, wo)
    du.check_state("final_state", got[1], final, wfinal)


@pytest.mark.parametrize("case", list(CASES))
def test_forward(case):
    lengths, packed, Hqk, Hv, unit, gates = CASES[case]
    print(f"[delta] forward {case}", flush=True)
    inp = Inp(lengths, packed, Hqk, Hv, seed=len(case), unit=unit, gates=gates)
    check_forward(inp, call_forward(inp))


def test_forward_without_initial_state():
    inp = Inp([5, 150, 64], True, 1, 2, seed=3, state=False)
    check_forward(inp, call_forward(inp))


def test_forward_custom_scale():
    inp = Inp([80], False, 1, 1, seed=5)
    check_forward(inp, call_forward(inp, scale=0.25), scale=0.25)


def wide(x):
    """A slice of wider token rows, the rest of which is NaN."""
    B, T, H, _ = x.shape
    w = torch.full((B, T, H + 3, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    w[:, :, 1:H + 1] = x
    return w[:, :, 1:H + 1]


@pytest.mark.parametrize("packed", [True, False])
def test_forward_of_slices(packed):
    inp = Inp([77, 130] if packed else [77, 77], packed, 2, 4, seed=6)
    got = call_forward(inp, wrap=wide)
    want = call_forward(inp)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check_forward(inp, got)


def test_sequences_do_not_see_each_other():
    """A packed sequence gives the bits of a call of its own, whatever stands beside
    it; NaN in the others stay there."""
    inp = Inp([70, 33, 100], True, 2, 2, seed=7, gates="mixed")
    a, b = 70, 103
    alone = Inp([33], False, 2, 2, unit=True)
    alone.q, alone.k, alone.v, alone.g, alone.beta = (x[:, a:b].contiguous() for x in (inp.q, inp.k, inp.v, inp.g, inp.beta))
    alone.s0 = inp.s0[1:2].clone()
    want = call_forward(alone)
    for x in (inp.q, inp.k, inp.v, inp.g, inp.beta):
        x[:, :a] = float("nan")
        x[:, b:] = float("nan")
    got = call_forward(inp)
    assert torch.equal(got[0][:, a:b], want[0])
    assert torch.equal(got[1][1], want[1][0])


def test_zero_rows():
    """Keys and queries of zeros (padding) at unit length stay zeros."""
    inp = Inp([70], False, 1, 1, seed=8)
    inp.k[:, 20:50] = 0
    inp.q[:, 10:40] = 0
    got = call_forward(inp)
    check_forward(inp, got)
    assert not got[0][:, 10:40].any()


def test_equal_keys():
    """The same key over and over, beta 1, no decay: every token replaces what the last one
    wrote, and the chunk's matrix is all ones."""
    inp = Inp([100], False, 1, 2, seed=9, gates="none")
    inp.k[:] = inp.k[:, :1]
    inp.beta.fill_(1.0)
    check_forward(inp, call_forward(inp))


# ---------------------------------------------------------------------------
# training
# ---------------------------------------------------------------------------
def train(inp, scale=None, wrap=lambda x: x, **more):
    import gated_delta_rule_32_amd as kda
    o, fs, ctx = call_forward(inp, scale, wrap, **more)
    grads = kda.gated_delta_rule_training_backward(ctx, inp.dev(inp.do), inp.dev(inp.ds))
    torch.cuda.synchronize()
    return (o, fs) + grads


@pytest.mark.parametrize("case", list(CASES))
def test_training_step(case):
    lengths, packed, Hqk, Hv, unit, gates = CASES[case]
    print(f"[delta] training step {case}", flush=True)
    inp = Inp(lengths, packed, Hqk, Hv, seed=100 + len(case), unit=unit, gates=gates)
    got = train(inp)
    check_forward(inp, got)
    du.check_gradients(inp, got[2:])


@pytest.mark.parametrize("unit", [True, False])
def test_gradients_with_records_formed_again(unit):
    """A forward with a given workspace keeps no records: the backward forms them."""
    import gated_delta_rule_32_amd as kda
    inp = Inp([70, 33, 100], True, 1, 2, seed=21, unit=unit, gates="mixed")
    want = train(inp)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")   # (5 blocks of 2 heads need 120 KiB)
    _, _, ctx = call_forward(inp, workspace=ws)
    assert ctx.records is None
    ws.fill_(255)
    grads = kda.gated_delta_rule_training_backward(ctx, inp.dev(inp.do), inp.dev(inp.ds))
    torch.cuda.synchronize()
    du.check_gradients(inp, grads)
    # (one over q's length is summed in another order there: equal to an FP32 rounding or two, and to the gradients' own)
    for a, b in zip(want[4:7], grads[2:5]):
        assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.float().abs().max()


SEGMENTS = {  # lengths, packed, Hqk, Hv, unit, gates, segment
    "two": ([128], False, 1, 1, True, "layer", 64),
    "one_and_a_token": ([65], False, 1, 2, True, "none", 64),
    "many": ([64 * 9 + 31], False, 1, 1, True, "none", 64),
    "batch": ([260] * 3, False, 2, 4, True, "layer", 64),
    "ragged": ([1, 64, 65, 200, 3, 129, 400], True, 1, 3, False, "mixed", 64),
    "longer": ([500, 128, 129, 7, 384], True, 2, 2, True, "none", 128),
    "strong": ([300, 190], True, 1, 2, True, "strong", 64),
    "eight_waves": ([130] * 20, False, 4, 4, True, "layer", 64),       # 240 segments and heads
    "four_waves": ([190, 70, 64] * 14, True, 4, 8, True, "mixed", 64),  # 672 of them
}


@pytest.mark.parametrize("case", list(SEGMENTS))
def test_training_step_in_segments(case):
    lengths, packed, Hqk, Hv, unit, gates, segment = SEGMENTS[case]
    print(f"[delta] segments {case}", flush=True)
    inp = Inp(lengths, packed, Hqk, Hv, seed=200 + len(case), unit=unit, gates=gates)
    got = train(inp, segment=segment)
    check_forward(inp, got)
    du.check_gradients(inp, got[2:])


def test_training_step_in_segments_without_states_and_records():
    import gated_delta_rule_32_amd as kda
    inp = Inp([150, 7, 333], True, 1, 2, seed=23, state=False)
    du.check_gradients(inp, train(inp, segment=64)[2:])
    ws = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")   # (10 segments of 2 heads need 2.5 MiB, 10 blocks 240 KiB)
    _, _, ctx = call_forward(inp, workspace=ws, segment=64)
    ws.fill_(255)
    grads = kda.gated_delta_rule_training_backward(ctx, inp.dev(inp.do), None)
    torch.cuda.synchronize()
    du.check_gradients(inp, grads)


def test_a_long_sequence_on_few_heads_goes_in_segments():
    """The library's own choice of segments, and its workspace for them."""
    import gated_delta_rule_32_amd as kda
    inp = Inp([2500], False, 1, 2, seed=24, gates="none")
    p = kda.KdaDeltaProblem(1, 2500, 1, 2, 1)
    own = kda.kda_delta_fwd_workspace_bytes(p)
    p.segment = 4096
    assert own > kda.kda_delta_fwd_workspace_bytes(p)
    got = train(inp)
    check_forward(inp, got)
    du.check_gradients(inp, got[2:])


def test_training_step_without_states():
    """initial_state and dfinal_state None count as zero."""
    inp = Inp([5, 150, 64], True, 1, 2, seed=3, state=False)
    du.check_gradients(inp, train(inp)[2:])


def test_training_step_custom_scale():
    inp = Inp([80], False, 1, 1, seed=5)
    du.check_gradients(inp, train(inp, scale=0.25)[2:], scale=0.25)


def test_training_step_of_slices():
    inp = Inp([77, 130], True, 2, 4, seed=6)
    got, want = train(inp, wrap=wide), train(inp)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_training_step_of_equal_keys():
    inp = Inp([100], False, 1, 2, seed=9, gates="none")
    inp.k[:] = inp.k[:, :1]
    inp.beta.fill_(1.0)
    du.check_gradients(inp, train(inp)[2:])


def test_gradients_of_zero_rows():
    """Rows of zeros at unit length: finite gradients, the norm's slope there being 1 /
    sqrt(1e-6)."""
    inp = Inp([70], False, 1, 1, seed=8)
    inp.k[:, 20:50] = 0
    inp.q[:, 10:40] = 0
    du.check_gradients(inp, train(inp)[2:])


def test_gradients_do_not_see_other_sequences():
    inp = Inp([70, 33, 100], True, 2, 2, seed=7, gates="mixed")
    a, b = 70, 103
    names = ("q", "k", "v", "g", "beta", "do")
    alone = Inp([33], False, 2, 2, unit=True)
    for n in names:
        setattr(alone, n, getattr(inp, n)[:, a:b].contiguous())
    alone.s0, alone.ds = inp.s0[1:2].clone(), inp.ds[1:2].clone()
    want = train(alone)
    for n in names:
        getattr(inp, n)[:, :a] = float("nan")
        getattr(inp, n)[:, b:] = float("nan")
    got = train(inp)
    for i in (0, 2, 3, 4, 5, 6):
        assert torch.equal(got[i][:, a:b], want[i]), i
    assert torch.equal(got[1][1], want[1][0]) and torch.equal(got[7][1], want[7][0])


def test_gradients_behind_a_strong_decay():
    """A decay of e^-60 between two halves: what passes it is far below what does not, and
    its gate's gradient is small and right all the same."""
    inp = Inp([64], False, 1, 2, seed=10, gates="none")
    inp.g[:, 20] = -60.0
    inp.ds.zero_()
    got = train(inp)
    du.check_gradients(inp, got[2:])
    refs, weights, _ = inp.gradients()
    # (its weight has the factor e^-60 too: no other token's size may show)
    x, ref = lu.f64(got[5])[:, 20], refs[3][:, 20]
    assert np.abs(x).max() <= 2.0 ** -60 and (np.abs(x - ref) <= lu.U * np.abs(ref) + du.GRADS * weights[3][:, 20] + 2.0 ** -40 * np.abs(refs[3]).max()).all()


def test_training_step_on_another_stream_and_the_same_bits_again():
    inp = Inp([200, 31], True, 1, 2, seed=13)
    want = train(inp)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = train(inp)
    s.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("segment,packed", [(0, False), (0, True), (64, False), (64, True)])
def test_captured_training_step(segment, packed):
    """Forward and backward in one graph, replayed with eager calls between; every replay
    gives the eager bits, on changed inputs too.  A fixed-layout call needs no call before
    the capture."""
    import gated_delta_rule_32_amd as kda
    inp = Inp([150, 7, 143] if packed else [150, 150], packed, 1, 2, seed=14)
    d = {n: inp.dev(getattr(inp, n)) for n in ("q", "k", "v", "g", "beta", "do", "s0", "ds", "cu")}
    if packed:  # the schedule: made by one call, seen on the device by a second
        train(inp, segment=segment)
        train(inp, segment=segment)
    p = kda.KdaDeltaProblem(inp.B, inp.T, 1, 2, inp.N)
    p.use_qk_l2norm = 1
    p.segment = segment
    if packed:
        p.cu_seqlens, p.cu_seqlens_host = d["cu"].data_ptr(), inp.cu.data_ptr()
    outs = [torch.empty_like(d[n]) for n in ("v", "s0", "q", "k", "v", "g", "beta", "s0")]
    rec = torch.empty(kda.kda_delta_fwd_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    ws = torch.empty(kda.kda_delta_bwd_workspace_bytes(p, True), dtype=torch.uint8, device="cuda")
    ins = [d[n] for n in ("q", "k", "v", "g", "beta", "s0")]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_delta_fwd(p, *ins, outs[0], outs[1], rec)
        kda.kda_delta_bwd(p, *ins, rec, d["do"], d["ds"], *outs[2:], ws)
    for _ in range(3):
        for x in outs:
            x.zero_()
        ws.fill_(255)    # (NaN: nothing of an earlier pass may be read)
        rec.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        want = train(inp, segment=segment)
        for a, b in zip(want, outs):
            assert torch.equal(a, b)
        inp.v = inp.v.flip(1).contiguous()
        d["v"].copy_(inp.v)


def test_context_checks_versions():
    import gated_delta_rule_32_amd as kda
    inp = Inp([20], False, 1, 1)
    args = [inp.dev(x) for x in (inp.q, inp.k, inp.v, inp.g, inp.beta)]
    _, _, ctx = kda.gated_delta_rule_training_forward(*args)
    args[3].add_(0)
    with pytest.raises(ValueError, match="changed after the forward"):
        kda.gated_delta_rule_training_backward(ctx, inp.dev(inp.do))


def test_capture_of_a_packed_call_without_a_schedule_is_refused():
    import gated_delta_rule_32_amd as kda
    inp = Inp([11, 222, 35], True, 1, 1, seed=15)
    d = [inp.dev(x) for x in (inp.q, inp.k, inp.v, inp.g, inp.beta)]
    cu = inp.dev(inp.cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(kda.KdaValueError) as e:
            kda.gated_delta_rule_training_forward(*d, cu_seqlens=cu, cu_seqlens_cpu=inp.cu)
        d[0].add_(0)  # something to capture
    assert e.value.status == kda.KDA_ERR_CAPTURE


# ---------------------------------------------------------------------------
# state pool
# ---------------------------------------------------------------------------
def pool_call(inp, pool, slots, accepted=None, output=None, dev_slots=None, **more):
    import gated_delta_rule_32_amd as kda
    host = None if slots is None else torch.tensor(slots, dtype=torch.int32)
    dev = host.cuda() if dev_slots is None and host is not None else dev_slots
    spec = {} if accepted is None else dict(num_spec_tokens=host.shape[1] - 1, num_accepted_tokens=accepted)
    out, same = kda.gated_delta_rule(inp.dev(inp.q), inp.dev(inp.k), inp.dev(inp.v), inp.dev(inp.g), inp.dev(inp.beta), pool,
                                     cu_seqlens=inp.dev(inp.cu), cu_seqlens_cpu=inp.cu, ssm_state_indices=dev,
                                     ssm_state_indices_cpu=host, output=output, use_qk_l2norm=inp.unit, **spec, **more)
    torch.cuda.synchronize()
    assert same is pool
    return out


BATCHES = {  # lengths, packed, Hqk, Hv
    "decode": ([1] * 7, False, 2, 4),
    "decode_packed": ([1] * 5, True, 1, 1),
    "few_tokens": ([3] * 4, False, 2, 2),
    "prefill": ([70, 70], False, 2, 6),
    "prefill_packed": ([129, 9, 64], True, 3, 3),
    "mixed": ([8, 9, 1, 300, 5, 2], True, 2, 4),
    "last_is_long": ([4, 3, 2, 64], True, 1, 3),
    "segments": ([3, 1500, 1, 200, 9], True, 1, 2),                   # (the long one's, and the others beside them)
    "segments_of_a_batch": ([1100] * 2, False, 1, 1),
}


@pytest.mark.parametrize("case", list(BATCHES))
def test_pool(case):
    lengths, packed, Hqk, Hv = BATCHES[case]
    print(f"[delta] pool {case}", flush=True)
    n = len(lengths)
    inp = Inp(lengths, packed, Hqk, Hv, seed=31 + len(case), unit=case != "decode", gates="mixed")
    slots = torch.randperm(n + 3, generator=torch.Generator().manual_seed(4))[:n].tolist()
    pool0 = torch.randn((n + 3, Hv, 128, 128), generator=torch.Generator().manual_seed(5))
    inp.s0 = pool0[slots]
    pool = pool0.cuda()
    out = pool_call(inp, pool, slots)
    o, final, (wo, wfinal), _ = inp.reference()
    du.check_o("o", out, o, wo)
    du.check_state("pool", pool[slots], final, wfinal)
    rest = [i for i in range(n + 3) if i not in slots]
    assert torch.equal(pool[rest].cpu(), pool0[rest])
    for i, length in enumerate(lengths):     # token by token: the bits of a call of its own
        if length > 4 or not packed:
            continue
        at = int(inp.cu[i])
        one = Inp([length], False, Hqk, Hv, unit=inp.unit)
        one.q, one.k, one.v, one.g, one.beta = (x[:, at:at + length].contiguous()
                                                for x in (inp.q, inp.k, inp.v, inp.g, inp.beta))
        own = pool0.cuda()
        assert torch.equal(pool_call(one, own, [slots[i]])[0], out[0, at:at + length])
        assert torch.equal(own[slots[i]], pool[slots[i]])


def test_pool_without_indices_and_without_a_pool():
    import gated_delta_rule_32_amd as kda
    for T in (1, 40):
        inp = Inp([T] * 2, False, 1, 2, seed=9, state=False)
        o, final, (wo, wfinal), _ = inp.reference()
        pool = torch.zeros((3, 2, 128, 128), device="cuda")
        pool[2] = 5.0
        du.check_o("o", pool_call(inp, pool, None), o, wo)
        du.check_state("pool", pool[:2], final, wfinal)
        assert (pool[2] == 5.0).all()
        out, new = kda.gated_delta_rule(*(inp.dev(x) for x in (inp.q, inp.k, inp.v, inp.g, inp.beta)), use_qk_l2norm=True)
        torch.cuda.synchronize()
        du.check_o("o", out, o, wo)
        du.check_state("new pool", new, final, wfinal)


def test_pieces_of_a_prompt():
    """A prompt in pieces, by chunks and token by token, ends where the whole one does."""
    inp = Inp([200], False, 1, 2, seed=10)
    pool = inp.s0.cuda()
    outs, at = [], 0
    for length in (64, 7, 1, 100, 8, 20):
        part = Inp([length], False, 1, 2)
        part.q, part.k, part.v, part.g, part.beta = (x[:, at:at + length].contiguous()
                                                     for x in (inp.q, inp.k, inp.v, inp.g, inp.beta))
        outs.append(pool_call(part, pool, [0]))
        at += length
    o, final, (wo, wfinal), _ = inp.reference()
    du.check_o("o", torch.cat(outs, 1), o, wo)
    du.check_state("pool", pool, final, wfinal)


@pytest.mark.parametrize("S,packed", [(1, False), (4, True), (10, False)])
def test_drafted_tokens(S, packed):
    n, Hqk, Hv = 5, 1, 3
    inp = Inp([1 + S] * n, packed, Hqk, Hv, seed=11 + S, gates="mixed")
    g = torch.Generator().manual_seed(S)
    slots = torch.randperm(n * (1 + S) + 4, generator=g)[:n * (1 + S)].reshape(n, 1 + S)
    pool0 = torch.randn((n * (1 + S) + 4, Hv, 128, 128), generator=g)
    accepted = torch.tensor([1, 1 + S, 0, 99, (S + 2) // 2], dtype=torch.int32)   # 0 and 99 are clamped
    first = slots[torch.arange(n), accepted.clamp(1, 1 + S).long() - 1]
    inp.s0 = pool0[first]
    pool = pool0.cuda()
    out = pool_call(inp, pool, slots.tolist(), accepted.cuda())
    o, _, (wo, wfinal), states = inp.reference()
    du.check_o("o", out, o, wo)
    for i in range(n):
        for t in range(1 + S):
            du.check_state(f"state {i} {t}", pool[slots[i, t]][None], states[i, t][None], wfinal[i:i + 1] + 1.0 * np.abs(states[i, t]).max())
    rest = [i for i in range(pool0.shape[0]) if i not in slots.reshape(-1).tolist()]
    assert torch.equal(pool[rest].cpu(), pool0[rest])
    # without numbers of accepted tokens: from the first slot
    inp.s0 = pool0[slots[:, 0]]
    import gated_delta_rule_32_amd as kda
    pool = pool0.cuda()
    host = slots.to(torch.int32).contiguous()
    out, _ = kda.gated_delta_rule(*(inp.dev(x) for x in (inp.q, inp.k, inp.v, inp.g, inp.beta)), pool,
                                  cu_seqlens=inp.dev(inp.cu), cu_seqlens_cpu=inp.cu, ssm_state_indices=host.cuda(),
                                  ssm_state_indices_cpu=host, num_spec_tokens=S, use_qk_l2norm=True)
    torch.cuda.synchronize()
    o, _, (wo, _), _ = inp.reference()
    du.check_o("o", out, o, wo)


@pytest.mark.parametrize("T", [1, 3, 6, 100, 1500])
def test_slots_outside_the_pool(T):
    """A slot that the device copy places outside the pool is skipped, its rows left as
    they were."""
    inp = Inp([T] * 3, False, 1, 2, seed=12)
    pool0 = torch.randn((3, 2, 128, 128))
    pool = pool0.cuda()
    dev = torch.tensor([2, -1, 3], dtype=torch.int32, device="cuda")
    out = torch.full((3, T, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    pool_call(inp, pool, [2, 0, 1], output=out, dev_slots=dev)
    assert torch.equal(pool[:2].cpu(), pool0[:2])
    assert not torch.equal(pool[2].cpu(), pool0[2])
    assert (out[1:] == 7.0).all() and not (out[0] == 7.0).all(-1).any()


def test_drafted_slots_outside_the_pool():
    """A token's slot outside the pool is not stored; a sequence whose first slot is outside is
    skipped."""
    inp = Inp([3, 3], False, 1, 1, seed=13)
    pool0 = torch.randn((8, 1, 128, 128))
    inp.s0 = pool0[[0, 3]]
    dev = torch.tensor([[0, -1, 2], [8, 4, 5]], dtype=torch.int32, device="cuda")
    out = torch.full((2, 3, 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    pool = pool0.cuda()
    ones = torch.ones(2, dtype=torch.int32, device="cuda")
    pool_call(inp, pool, [[0, 1, 2], [3, 4, 5]], ones, output=out, dev_slots=dev)
    _, _, (_, wfinal), states = inp.reference()
    for t, slot in ((0, 0), (2, 2)):
        du.check_state("state", pool[slot:slot + 1], states[0, t][None], wfinal[:1] + np.abs(states[0, t]).max())
    keep = [1, 3, 4, 5, 6, 7]
    assert torch.equal(pool[keep].cpu(), pool0[keep])
    assert (out[1] == 7.0).all()


@pytest.mark.parametrize("T", [1, 4, 8])
def test_weak_decays_over_many_tokens(T):
    """2^13 tokens in calls of a few at a decay of 2^-15 a token: the state keeps to the exact
    powers (a decay rounded to FP32 would drift by 2^-24 a token, one way)."""
    import gated_delta_rule_32_amd as kda
    steps = 8192 // T
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    g = torch.full((1, T, 1), -2.0 ** -15, dtype=torch.bfloat16, device="cuda")
    s0 = torch.rand((1, 1, 128, 128), generator=torch.Generator().manual_seed(1)) + 1.0
    pool = s0.cuda()
    for _ in range(steps):
        kda.gated_delta_rule(z(1, T, 1, 128), z(1, T, 1, 128), z(1, T, 1, 128), g, z(1, T, 1), pool)
    torch.cuda.synchronize()
    want = s0.double().numpy() * np.exp(-2.0 ** -15 * T * steps)
    # one rounding a token, of either sign: 2^-24 sqrt(tokens) = 2^-17.5, and as much again
    assert (np.abs(lu.f64(pool) - want) / want).max() <= 2.0 ** -16.5


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------
def test_forward_on_another_stream():
    inp = Inp([200, 31], True, 1, 2, seed=13)
    want = call_forward(inp)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = call_forward(inp)
    s.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_captured_decode_and_prefill():
    """A decode and a prefill call in one graph, replayed with eager work between: every
    replay gives the eager bits; a slot of -1 put in later is skipped."""
    import gated_delta_rule_32_amd as kda
    one, many = Inp([1] * 3, False, 1, 2, seed=14), Inp([70] * 2, False, 1, 2, seed=15)
    pool0 = torch.randn((6, 2, 128, 128), generator=torch.Generator().manual_seed(3))
    pool = pool0.cuda()
    slots = [torch.tensor(x, dtype=torch.int32) for x in ([4, 0, 2], [1, 3])]
    dev = [x.cuda() for x in slots]
    args = [[i.dev(x) for x in (i.q, i.k, i.v, i.g, i.beta)] for i in (one, many)]
    outs = [torch.empty_like(a[2]) for a in args]
    p = kda.KdaDeltaProblem(2, 70, 1, 2, 2)
    p.use_qk_l2norm = 1
    ws = torch.empty(kda.kda_delta_infer_workspace_bytes(p), dtype=torch.uint8, device="cuda")

    def run(pool, outs):
        for a, o, d, h in zip(args, outs, dev, slots):
            kda.gated_delta_rule(*a, pool, ssm_state_indices=d, ssm_state_indices_cpu=h, output=o, use_qk_l2norm=True,
                                 workspace=ws)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(pool, outs)
    eager, eager_outs = pool0.cuda(), [torch.empty_like(o) for o in outs]
    pool.copy_(pool0)
    for i in range(4):
        if i == 2:
            dev[0][1] = -1
        for o in outs + eager_outs:
            o.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        run(eager, eager_outs)
        torch.cuda.synchronize()
        assert torch.equal(pool, eager)
        for a, b in zip(outs, eager_outs):
            assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# far rows and far apart values
# ---------------------------------------------------------------------------
def test_rows_behind_2_31_elements():
    """Token rows as far apart as a call takes: q's, k's and v's last ones lie behind 2^31 elements."""
    import gated_delta_rule_32_amd as kda
    T, stride = 70, 1 << 25
    inp = Inp([T], False, 1, 2, seed=61)
    wide = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda").view(1, T, stride)
    d = []
    for at, x in ((0, inp.q), (256, inp.k), (stride - 256, inp.v)):
        n = x.shape[2] * 128
        wide[:, :, at:at + n] = x.view(1, T, n).cuda()
        d.append(wide[:, :, at:at + n].unflatten(-1, (-1, 128)))
    rest = [inp.dev(x) for x in (inp.g, inp.beta, inp.s0)]
    o, fs, ctx = kda.gated_delta_rule_training_forward(*d, *rest, use_qk_l2norm=True)
    grads = kda.gated_delta_rule_training_backward(ctx, inp.dev(inp.do), inp.dev(inp.ds))
    pool = inp.dev(inp.s0)
    served, _ = kda.gated_delta_rule(*d, *rest[:2], pool, use_qk_l2norm=True)
    torch.cuda.synchronize()
    for a, b in zip(train(inp), (o, fs) + grads):
        assert torch.equal(a, b)
    assert torch.equal(served, o) and torch.equal(pool, fs)


@pytest.mark.parametrize("T", [1, 3, 40])
def test_slots_behind_2_31_elements(T):
    Hv, slots = 64, [2099, 7]
    inp = Inp([T] * 2, False, 16, Hv, seed=62)
    pool = torch.empty((2100, Hv, 128, 128), device="cuda")     # 2.2e9 values
    pool[slots] = inp.s0.cuda()
    out = pool_call(inp, pool, slots)
    near = inp.s0.cuda()
    assert torch.equal(out, pool_call(inp, near, [0, 1]))
    assert torch.equal(pool[slots], near)


@pytest.mark.parametrize("segment", [0, 64])
def test_values_far_apart(segment):
    """Tokens, output channels and states of sizes from 2^-12 to 2^12 side by side: every result is
    held to the sizes of its own terms.  (The backward keeps 32 channels' states and rows to a part
    of their largest value in FP16: 2^-39 of it, far below the bars at a ratio of 2^24.)"""
    inp = Inp([190, 70], True, 1, 2, seed=63, gates="layer")
    g = torch.Generator().manual_seed(64)

    def spread(x, *dims):
        shape = [n if i in dims else 1 for i, n in enumerate(x.shape)]
        return (x.float() * 2.0 ** torch.randint(-6, 7, shape, generator=g)).to(x.dtype)
    inp.v, inp.do = spread(spread(inp.v, 1), 2, 3), spread(spread(inp.do, 1), 2, 3)
    inp.s0, inp.ds = spread(spread(inp.s0, 1, 2), 0), spread(spread(inp.ds, 1, 2), 0)
    got = train(inp, segment=segment)
    check_forward(inp, got)
    du.check_gradients(inp, got[2:])


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** -40, 2.0 ** 40])
def test_small_and_large_values(scale):
    """The rule is linear in v and the states, its gradients in do: a power of two goes through all of
    it exactly, while the numbers stay normal.  At 2^-60 the gradients of q and k are of the size of 2^-120 and the
    pieces of their factors end at 2^-126, BF16's least normal number: of each of a token's 64 elements
    of the three matrices e, f and f^T less than 2^-126 is lost twice, times a key's or query's channel, at
    most 1; and as much of each of 128 products with a state.  That is below 2^-116; a gate's gradient sums
    128 channels of those, at most 1 in all, over up to 100 tokens of two gradients: 2^-108."""
    inp = Inp([100], False, 1, 2, seed=65)
    want = train(inp)
    for n in ("v", "s0", "do", "ds"):
        x = getattr(inp, n)
        setattr(inp, n, (x.float() * scale).to(x.dtype))
    got = train(inp)
    for name, a, b, power in zip("o final dq dk dv dg dbeta ds0".split(), want, got, (1, 1, 2, 2, 1, 2, 2, 1)):
        if power == 2 and scale < 2.0 ** -50:
            bar = 2.0 ** -108 if name in ("dg", "dbeta") else 2.0 ** -116
            assert (a.double() * scale ** power - b.double()).abs().max() <= bar, name
        else:
            assert torch.equal((a.double() * scale ** power).to(a.dtype), b), name
