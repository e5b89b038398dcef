"""GPU tests of the drafted tokens' verification (kda_verify) against the FP64 oracle.

Tokens are whole numbers and have to be equal: products of two FP32 values are exact in
64 bits, and sums of up to 2^17 of them there are off by 2^-40 at most, so that the chance of a draw
within a border is far below one in a million."""
import numpy as np
import pytest
import torch

from oracle import delta_oracle as do_

pytestmark = pytest.mark.gpu


class Drafts:
    def __init__(self, N, S, V, seed, point=False, lens=None, sharp=3.0):
        g = torch.Generator().manual_seed(seed)
        logits = sharp * torch.randn((N, S + 1, V), generator=g)
        self.target = torch.softmax(logits, -1)
        self.draft = None if point else torch.softmax(0.9 * logits[:, :S] + 0.3 * torch.randn((N, S, V), generator=g), -1)
        drawn = self.target[:, :S] if point else self.draft
        race = -torch.log(torch.rand((N, S, V), generator=g).clamp_min(1e-30))
        self.drafts = (drawn / race).argmax(-1).to(torch.int32) if S else torch.zeros((N, 0), dtype=torch.int32)
        self.lens = None if lens is None else torch.tensor([lens[i % len(lens)] for i in range(N)], dtype=torch.int32)
        self.uniform = torch.rand((N, S + 1), generator=g)

    def reference(self):
        n = lambda x: None if x is None else x.numpy()  # noqa: E731
        return do_.verify(n(self.drafts), n(self.lens), n(self.target), n(self.draft), n(self.uniform))

    def call(self, wrap=lambda x: x, **more):
        import gated_delta_rule_32_amd as kda
        c = lambda x: None if x is None else x.cuda()  # noqa: E731
        w = lambda x: None if x is None else wrap(x.cuda())  # noqa: E731
        r = kda.verify_drafts(c(self.drafts), w(self.target), c(self.uniform), w(self.draft), c(self.lens), **more)
        torch.cuda.synchronize()
        return r

    def check(self, **more):
        tokens, accepted = self.call(**more)
        want, count = self.reference()
        assert np.array_equal(accepted.cpu().numpy(), count)
        assert np.array_equal(tokens.cpu().numpy(), want)


@pytest.mark.parametrize("point", [False, True])
@pytest.mark.parametrize("N,S,V", [(1, 1, 1), (3, 2, 2), (9, 4, 17), (5, 3, 4095), (5, 3, 4096), (5, 3, 4097), (4, 5, 9000),
                                   (2, 1, 40001), (2, 70, 33), (3, 0, 5000), (3, 2, 16384), (3, 2, 16385), (4, 3, 32767),
                                   (4, 3, 32768), (4, 3, 32769), (2, 2, 300007)])
def test_parity(N, S, V, point):
    print(f"[verify] {N} {S} {V} {point}", flush=True)
    for seed in range(3):
        Drafts(N, S, V, seed, point).check()


def test_given_numbers_of_drafts():
    Drafts(12, 4, 300, 5, lens=[0, 1, 2, 3, 4, -3, 9]).check()
    Drafts(12, 4, 300, 6, point=True, lens=[0, 4, 1]).check()


def test_every_draft_stands_and_none_does():
    d = Drafts(4, 3, 500, 7)
    d.uniform[:, :3] = 0.0
    assert (d.call()[1] == 4).all()
    d.check()
    d.uniform[:, :3] = 0.999999
    d.draft = torch.zeros_like(d.draft).scatter_(2, d.drafts.long()[..., None], 1.0)
    assert (d.call()[1] == 1).all()
    d.check()


def test_drafts_outside_the_vocabulary_never_stand():
    for point in (False, True):
        d = Drafts(3, 2, 100, 8, point)
        d.uniform[:, 0] = 0.0
        d.drafts[0, 0], d.drafts[1, 0], d.drafts[2, 1] = -1, 100, 2 ** 31 - 1
        d.check()


@pytest.mark.parametrize("V", [5000, 50000])
def test_equal_probabilities_fall_back_to_the_targets(V):
    """Where p exceeds q nowhere, the token is drawn from p."""
    d = Drafts(3, 2, V, 9)
    d.target[:, :2] = 0.5 * d.draft
    d.uniform[:, 0] = 0.75
    assert (d.call()[1] == 1).all()
    d.check()


@pytest.mark.parametrize("V", [100, 40000])
def test_rows_without_a_probability(V):
    d = Drafts(3, 1, V, 10)
    d.target[1] = 0.0
    tokens, accepted = d.call()
    assert accepted[1] == 1 and tokens[1].tolist() == [-1, -1]
    d.check()


@pytest.mark.parametrize("V", [9000, 39000])
def test_draws_at_the_ends(V):
    """A random number of 0 (or below, or NaN) draws the first index with a weight, one of
    1 and above the last."""
    d = Drafts(5, 0, V, 11)
    d.target[:, :, :5] = 0.0
    d.target[:, :, V - 10:] = 0.0
    d.uniform[:, 0] = torch.tensor([0.0, -1.0, float("nan"), 1.0, 7.0])
    tokens, _ = d.call()
    assert tokens[:, 0].tolist() == [5, 5, 5, V - 11, V - 11]
    d.check()


@pytest.mark.parametrize("V", [8192, 65536])
def test_ties_go_to_the_lowest_index(V):
    """Equal weights: u V falls on a border, which belongs to the index above it."""
    d = Drafts(4, 0, V, 12)
    d.target[:] = 1.0 / V
    d.uniform[:, 0] = torch.tensor([0.0, 0.5, 0.25, 4095 / V])
    assert d.call()[0][:, 0].tolist() == [0, V // 2, V // 4, 4095]


@pytest.mark.parametrize("V", [600, 40000])
def test_nan_counts_as_nothing(V):
    d = Drafts(2, 1, V, 13)
    d.uniform[:, 0] = 0.9999999
    d.target[0, 0, 7] = float("nan")
    d.draft[1, 0, 5] = float("nan")
    d.check()


@pytest.mark.parametrize("V", [1000, 1001])
def test_slices_of_wider_rows(V):
    """A padded vocabulary, the padding NaN."""
    def wrap(x):
        w = torch.full((*x.shape[:2], V + 7), float("nan"), device="cuda")
        w[..., :V] = x
        return w[..., :V]
    Drafts(5, 3, V, 14).check(wrap=wrap)


@pytest.mark.parametrize("V", [700, 40000])
def test_given_outputs_and_workspace(V):
    import gated_delta_rule_32_amd as kda
    d = Drafts(5, 3, V, 15)
    out = (torch.empty((5, 4), dtype=torch.int32, device="cuda"), torch.empty(5, dtype=torch.int32, device="cuda"))
    ws = torch.empty(kda.kda_verify_workspace_bytes(kda.KdaVerifyProblem(5, 3, V)), dtype=torch.uint8, device="cuda")
    got = d.call(out=out, workspace=ws)
    assert got[0] is out[0] and got[1] is out[1]
    d.check()


@pytest.mark.parametrize("V", [5000, 40000])
def test_captured(V):
    """One graph, replayed on changed inputs with eager calls between."""
    import gated_delta_rule_32_amd as kda
    a, b = Drafts(6, 3, V, 16), Drafts(6, 3, V, 17)
    dev = [x.cuda() for x in (a.drafts, a.target, a.uniform, a.draft)]
    out = (torch.empty((6, 4), dtype=torch.int32, device="cuda"), torch.empty(6, dtype=torch.int32, device="cuda"))
    ws = torch.empty(kda.kda_verify_workspace_bytes(kda.KdaVerifyProblem(6, 3, V)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.verify_drafts(*dev, out=out, workspace=ws)
    for d in (a, b, a, b):
        for x, y in zip(dev, (d.drafts, d.target, d.uniform, d.draft)):
            x.copy_(y)
        for x in out:
            x.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        want = d.call()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_one_sequence_does_not_see_the_others():
    d = Drafts(7, 3, 9000, 18)
    tokens, accepted = d.call()
    for n in range(7):
        one = Drafts(1, 3, 9, 0)
        one.drafts, one.target, one.draft, one.uniform = (x[n:n + 1].contiguous() for x in (d.drafts, d.target, d.draft, d.uniform))
        t, a = one.call()
        assert torch.equal(t[0], tokens[n]) and a[0] == accepted[n]


@pytest.mark.parametrize("V", [3000, 20000])
def test_rows_behind_2_31_values(V):
    stride = 1 << 29                       # five rows of 2 GiB: the last begins behind 2^31 values
    space = torch.empty(5 * stride, device="cuda")

    def wrap(x):
        w = space[:x.shape[0] * x.shape[1] * stride].view(*x.shape[:2], stride)[..., :V]
        w.copy_(x)
        return w
    d = Drafts(1, 4, V, 21)
    d.uniform[:, :4] = 0.0                 # (all stand: the draw is from the last row)
    d.draft = d.draft.clamp_min(1e-9)
    import gated_delta_rule_32_amd as kda
    tokens, accepted = kda.verify_drafts(d.drafts.cuda(), wrap(d.target.cuda()), d.uniform.cuda(), d.draft.cuda())
    want, count = d.reference()
    assert np.array_equal(accepted.cpu().numpy(), count) and np.array_equal(tokens.cpu().numpy(), want)
