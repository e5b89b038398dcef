"""GPU tests of the drafted tokens' verification: rows of both operands far apart, outputs that the
caller gives, and NaN in what a draft is compared by."""
import numpy as np
import pytest
import torch

from tests.test_verify_drafts import Drafts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [3000, 20000])
@pytest.mark.parametrize("last_stands", [False, True])
def test_rows_of_both_operands_behind_2_31_values(V, last_stands):
    """Rows of 2 GiB: the target's last two and the drafts' last one begin behind 2^31 values.  Every draft but
    the last stands by a random number close below its border; the last is refused, so that p and q are read whole
    there, or stands."""
    import gated_delta_rule_32_amd as kda
    S, stride = 6, 1 << 29
    d = Drafts(1, S, V, 22)
    x = d.drafts.long()[..., None]
    p, q = d.target[:, :S].gather(2, x)[..., 0], d.draft.gather(2, x)[..., 0]
    border = (p / q).clamp(max=0.999)
    d.uniform[:, :S] = 0.97 * border
    if not last_stands:
        d.draft[0, S - 1] = 0.5 * d.draft[0, S - 1]
        d.draft[0, S - 1, x[0, S - 1, 0]] = 2 * d.target[0, S - 1, x[0, S - 1, 0]] + 0.25
        d.uniform[:, S - 1] = 0.75

    def far(t):
        w = torch.empty(t.shape[1] * stride, device="cuda").view(1, t.shape[1], stride)[..., :V]
        w.copy_(t)
        return w
    target, draft = far(d.target), far(d.draft)
    assert (S - 2) * stride >= 1 << 31
    tokens, accepted = kda.verify_drafts(d.drafts.cuda(), target, d.uniform.cuda(), draft)
    want, count = d.reference()
    assert count[0] == (S + 1 if last_stands else S)
    assert np.array_equal(accepted.cpu().numpy(), count) and np.array_equal(tokens.cpu().numpy(), want)


@pytest.mark.parametrize("V", [700, 40000])
def test_given_outputs_are_filled(V):
    import gated_delta_rule_32_amd as kda
    d = Drafts(5, 3, V, 23)
    out = (torch.full((5, 4), -77, dtype=torch.int32, device="cuda"), torch.full((5,), -77, dtype=torch.int32, device="cuda"))
    ws = torch.full((kda.kda_verify_workspace_bytes(kda.KdaVerifyProblem(5, 3, V)),), 255, dtype=torch.uint8, device="cuda")
    got = d.call(out=out, workspace=ws)
    want, count = d.reference()
    assert got[0] is out[0] and got[1] is out[1]
    assert np.array_equal(out[0].cpu().numpy(), want) and np.array_equal(out[1].cpu().numpy(), count)


@pytest.mark.parametrize("V", [700, 40000])
def test_a_draft_compared_by_nan_does_not_stand(V):
    """NaN as the random number, as the target's or as the draft's probability of the token, which has no
    weight in the draw then."""
    d = Drafts(4, 2, V, 24)
    d.uniform[:, :2] = 0.0
    x = d.drafts[:, 0].long()
    d.uniform[0, 0] = float("nan")
    d.target[1, 0, x[1]] = float("nan")
    d.draft[2, 0, x[2]] = float("nan")
    assert d.call()[1].tolist() == [1, 1, 1, 3]
    d.check()


@pytest.mark.parametrize("V", [1, 700, 20000])
def test_first_rows_of_buffers_with_more(V):
    """Drafts' and target's probabilities as the first rows of one shape of buffer, of sequences that lie
    apart, of wider rows too; what lies between is NaN."""
    for n, S, pad in ((5, 3, 0), (4, 1, 3), (1, 4, 0), (3, 0, 0)):
        def wrap(x):
            w = torch.full((2 * n, S + 3, V + pad), float("nan"), device="cuda")[::2, :x.shape[1], :V]
            w.copy_(x)
            return w
        d = Drafts(n, S, V, 25 + S)
        tokens, accepted = d.call(wrap=wrap)
        want, count = d.reference()
        assert np.array_equal(tokens.cpu().numpy(), want) and np.array_equal(accepted.cpu().numpy(), count)
