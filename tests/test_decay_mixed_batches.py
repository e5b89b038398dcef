"""GPU tests of kda_decay_infer on batches that hold prompts and single tokens: each
sequence runs by its own length, so that a user's next token has the same bits
whoever else is in the batch."""
import numpy as np
import pytest
import torch

from tests import layer_util as lu
from tests.test_decay_attention import Inp, pool_call

pytestmark = pytest.mark.gpu

BATCHES = {  # lengths, Hqk, Hv, segment
    "one_prompt": ([1, 1, 70, 1], 2, 2, 0),
    "edges": ([4, 9, 1, 300, 5, 2], 2, 4, 0),
    "segments": ([4, 9, 1, 300, 5, 2], 2, 4, 64),
    "segments_auto": ([1, 2000, 1], 1, 2, 0),
    "many": ([1, 40, 3] * 30, 4, 4, 0),
    "last_is_long": ([4, 3, 2, 64], 1, 3, 64),
}


def alone(inp, slots, pool0, n):
    """The call of sequence n by itself."""
    at = int(inp.cu[n])
    one = Inp([inp.lengths[n]], False, inp.Hqk, inp.Hv)
    one.q, one.k, one.v = (x[:, at:at + inp.lengths[n]].contiguous() for x in (inp.q, inp.k, inp.v))
    one.l = inp.l
    pool = pool0.cuda()
    return pool_call(one, pool, [slots[n]]), pool[slots[n]]


def batch(case):
    lengths, Hqk, Hv, segment = BATCHES[case]
    inp = Inp(lengths, True, Hqk, Hv, seed=51 + len(case))
    g = torch.Generator().manual_seed(5)
    slots = torch.randperm(len(lengths) + 2, generator=g)[:len(lengths)].tolist()
    pool0 = torch.randn((len(lengths) + 2, Hv, 128, 128), generator=g)
    inp.s0 = pool0[slots]
    return inp, slots, pool0, segment


@pytest.mark.parametrize("case", list(BATCHES))
def test_short_sequences_do_not_see_the_batch(case):
    print(f"[mixed] {case}", flush=True)
    inp, slots, pool0, segment = batch(case)
    pool = pool0.cuda()
    out = pool_call(inp, pool, slots, segment=segment)
    o, final, _, mfinal = inp.reference()
    lu.check_scanned("o", out, o, inp.energies()[0])
    lu.check_state("pool", pool[slots], final, mfinal)
    rest = [i for i in range(pool0.shape[0]) if i not in slots]
    assert torch.equal(pool[rest].cpu(), pool0[rest])
    for n, length in enumerate(inp.lengths):
        if length > 4:
            continue
        want, state = alone(inp, slots, pool0, n)
        at = int(inp.cu[n])
        assert torch.equal(out[0, at:at + length], want[0]), n
        assert torch.equal(pool[slots[n]], state), n


@pytest.mark.parametrize("segment", [0, 64])
def test_prompts_do_not_see_the_short_sequences(segment):
    inp, slots, pool0, _ = batch("edges")
    pool = pool0.cuda()
    out = pool_call(inp, pool, slots, segment=segment)
    long = [n for n, length in enumerate(inp.lengths) if length > 4]
    part = Inp([inp.lengths[n] for n in long], True, inp.Hqk, inp.Hv)
    rows = torch.cat([torch.arange(int(inp.cu[n]), int(inp.cu[n + 1])) for n in long])
    part.q, part.k, part.v = (x[:, rows].contiguous() for x in (inp.q, inp.k, inp.v))
    part.l = inp.l
    other = pool0.cuda()
    want = pool_call(part, other, [slots[n] for n in long], segment=segment)
    assert torch.equal(out[:, rows.cuda()], want)
    for n in long:
        assert torch.equal(pool[slots[n]], other[slots[n]])


@pytest.mark.parametrize("segment", [0, 64])
def test_slots_outside_the_pool_in_a_mixed_batch(segment):
    """A single token and a prompt whose slot the device copy places outside the pool
    are skipped, their rows left as they were; the others run."""
    import gated_delta_rule_32_amd as kda
    inp, slots, pool0, _ = batch("edges")
    pool = pool0.cuda()
    host = torch.tensor(slots, dtype=torch.int32)
    dev = host.clone()
    dev[2], dev[3] = -1, pool0.shape[0]          # 1 token, 300 tokens
    out = torch.full(inp.v.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    kda.decay_attention(inp.dev(inp.q), inp.dev(inp.k), inp.dev(inp.v), inp.dev(inp.l), pool, None, inp.dev(inp.cu),
                        dev.cuda(), out, cu_seqlens_cpu=inp.cu, ssm_state_indices_cpu=host, segment=segment)
    torch.cuda.synchronize()
    o, final, _, mfinal = inp.reference()
    for n in range(6):
        a, b = int(inp.cu[n]), int(inp.cu[n + 1])
        if n in (2, 3):
            assert (out[0, a:b] == 7.0).all() and torch.equal(pool[slots[n]].cpu(), pool0[slots[n]])
        else:
            lu.check_scanned("o", out[:, a:b], o[:, a:b], inp.energies()[0][:, a:b])
            lu.check_state("pool", pool[slots[n]], final[n], mfinal[n])


def test_captured_mixed_batch():
    """Replayed with eager calls between, on changed inputs: the eager bits."""
    import gated_delta_rule_32_amd as kda
    inp, slots, pool0, _ = batch("segments")
    q, k, v, l, cu = (inp.dev(x) for x in (inp.q, inp.k, inp.v, inp.l, inp.cu))
    host = torch.tensor(slots, dtype=torch.int32)
    idx, pool, out = host.cuda(), pool0.cuda(), torch.empty_like(v)

    def call(pool, out):
        kda.decay_attention(q, k, v, l, pool, None, cu, idx, out, cu_seqlens_cpu=inp.cu, ssm_state_indices_cpu=host,
                            segment=64)

    eager = pool.clone()
    for _ in range(2):   # the schedule: made by one call, seen on the device by a second
        call(eager.clone(), out)
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(pool, out)
    pool.copy_(eager)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(out)
        call(eager, want)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(pool, eager)
        v.copy_(v.flip(1))
