"""GPU tests of the gated delta rule's calls across streams: a context that is dropped while its
backward still runs."""
import pytest
import torch

from tests.delta_util import Inp
from tests.test_delta_rule import call_forward

pytestmark = pytest.mark.gpu


def test_context_dropped_while_its_backward_waits_on_another_stream():
    """The records' and inputs' memory is not handed out on the forward's stream before the other
    stream's backward has read it."""
    import gated_delta_rule_32_amd as kda
    inp = Inp([130, 70], True, 1, 2, seed=351)
    do, ds = inp.dev(inp.do), inp.dev(inp.ds)
    _, _, ctx = call_forward(inp)
    want = kda.gated_delta_rule_training_backward(ctx, do, ds)
    torch.cuda.synchronize()
    _, _, ctx = call_forward(inp)
    held = [t for t in (*ctx.inputs[:7], ctx.records) if t is not None]
    sizes, places = [t.untyped_storage().nbytes() for t in held], {t.data_ptr() for t in held}
    del held
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(500_000_000)
        got = kda.gated_delta_rule_training_backward(ctx, do, ds)
    del ctx
    new = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
    places &= {t.data_ptr() for t in new}
    waits = not side.query()
    side.synchronize()
    assert waits and not places
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_backward_on_the_forwards_stream_gives_its_memory_back():
    """No other stream: the records' memory is there again for the next step."""
    import gated_delta_rule_32_amd as kda
    inp = Inp([130, 70], True, 1, 2, seed=352)
    do = inp.dev(inp.do)
    args = [inp.dev(x) for x in (inp.q, inp.k, inp.v, inp.g, inp.beta)]
    cu = inp.dev(inp.cu)
    used = []
    for _ in range(4):
        _, _, ctx = kda.gated_delta_rule_training_forward(*args, cu_seqlens=cu, cu_seqlens_cpu=inp.cu)
        kda.gated_delta_rule_training_backward(ctx, do)
        del ctx
        used.append(torch.cuda.memory_allocated())
    assert used[1] == used[3]


@pytest.mark.parametrize("packed", [False, True])
def test_captured_backward_of_an_eager_forward(packed):
    """A graph of the backward alone, replayed with eager steps between: the eager bits."""
    import gated_delta_rule_32_amd as kda
    inp = Inp([130, 70] if packed else [130, 130], packed, 1, 2, seed=353)
    do, ds = inp.dev(inp.do), inp.dev(inp.ds)
    call_forward(inp)
    _, _, ctx = call_forward(inp)
    want = kda.gated_delta_rule_training_backward(ctx, do, ds)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kda.gated_delta_rule_training_backward(ctx, do, ds)
    for _ in range(3):
        for x in got:
            x.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        again = kda.gated_delta_rule_training_backward(ctx, do, ds)
        torch.cuda.synchronize()
        for a, b, c in zip(got, want, again):
            assert torch.equal(a, b) and torch.equal(c, b)
