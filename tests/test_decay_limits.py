"""GPU tests of the decayed attention at the edges of what its header allows: outputs
that are not wanted, and states near the largest magnitude."""
import pytest
import torch

from tests import layer_util as lu
from tests.test_decay_attention import Inp, train

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("segment", [0, 64])
def test_states_that_are_not_wanted(segment):
    """final_state and dinitial_state may be NULL: the other results keep their bits."""
    import gated_delta_rule_32_amd as kda
    inp = Inp([150, 9, 70], True, 2, 4, seed=61)
    want = train(inp, segment)
    p = kda.KdaDecayProblem(1, 229, 2, 4, 3, inp.dev(inp.cu).data_ptr(), inp.cu.data_ptr(), 0.0, segment)
    d = {n: inp.dev(getattr(inp, n)) for n in ("q", "k", "v", "do", "l", "s0", "ds")}
    ws = torch.empty(max(1, kda.kda_decay_fwd_workspace_bytes(p), kda.kda_decay_bwd_workspace_bytes(p)),
                     dtype=torch.uint8, device="cuda")
    o, dq, dk, dv = (torch.empty_like(d[n]) for n in ("v", "q", "k", "v"))
    kda.kda_decay_fwd(p, d["q"], d["k"], d["v"], d["l"], d["s0"], o, None, ws)
    kda.kda_decay_bwd(p, d["q"], d["k"], d["v"], d["l"], d["s0"], d["do"], d["ds"], dq, dk, dv, None, ws)
    torch.cuda.synchronize()
    for a, b in zip((o, dq, dk, dv), (want[0], *want[2:5])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("segment", [0, 64])
@pytest.mark.parametrize("size", [2.0 ** 90, 2.0 ** -90])
def test_large_and_small_values(size, segment):
    """Values of v and states of about 2^90 (sums up to 2^99) or 2^-90, in heads of every
    decay: the state is kept divided by up to 2^-24 of itself, which must not overflow."""
    inp = Inp([400, 33], True, 1, 7, seed=62)
    inp.v, inp.s0 = (inp.v.float() * size).bfloat16(), inp.s0 * size
    got = train(inp, segment)
    o, final, _, mfinal = inp.reference()
    lu.check_scanned("o", got[0], o, inp.energies()[0])
    lu.check_state("final_state", got[1], final, mfinal)
