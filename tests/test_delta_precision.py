"""GPU tests of how far the gated delta rule's results may be off: each BF16 result by one rounding
of what 32-bit arithmetic gives.  (The bars of delta_util leave room for what the gradients are formed from in
11 bits, and for partials of 10; it has 16 to 18, and the partials 16.)

Bars.  u = 2^-8 is half a BF16 step relative to the value.
  - One element: u |ref| (and u of that, where the value crosses into the next binade), and what came
    before the rounding.  Written rows and states are off by 2^-18 of their terms' sizes (delta_util), and as two BF16
    pieces by 2^-18 more (a piece is off by 2^-9 of itself at most, the second by that of the first's
    rest); where two of them are multiplied that is 2^-16, the block's matrices as pieces and the sums of 128
    + 64 products in FP32 add 2^-18 each: below 2^-15 of the oracle's weights.
  - The norm: that of the exact values' own roundings, r.  Errors d before the rounding, independent of it,
    make it sqrt(r^2 + d^2).  Of random sign they are about 2^-17 of the result, and 2^-13 with
    terms 16 times as large as their sums; r is 2^-9.2 of it, so that this adds 2^-8.6 of r at most: bar
    (1 + 2^-8) r.  (A part of 11 bits, 2^-12.8 in the mean square, would add 2^-8.2 of r for
    each factor that it enters in.)
"""
import numpy as np
import pytest
import torch

from tests import delta_util as du
from tests import layer_util as lu
from tests.delta_util import Inp
from tests.test_delta_rule import train

pytestmark = pytest.mark.gpu

FINE = 2.0 ** -15


def check_one_rounding(name, got, ref, weights):
    got = lu.f64(got)
    assert np.isfinite(got).all(), f"{name}: not finite"
    err = np.abs(got - ref)
    worst = (err / np.maximum(lu.U * np.abs(ref) * (1 + lu.U) + FINE * weights, 1e-30)).max()
    once = np.linalg.norm(lu.f64(torch.from_numpy(ref).bfloat16()) - ref)
    ratio = np.linalg.norm(err) / once
    print(f"{name:5s} norm {ratio:.5f} of one rounding's (bar {1 + lu.U:.5f})  elementwise {worst:.3f} of the bar", flush=True)
    assert worst <= 1.0 and ratio <= 1 + lu.U, name


CASES = {  # lengths, packed, Hqk, Hv, unit, gates, segment: every launch variant, whole and cut
    "few_workgroups": ([70, 200, 33], True, 3, 3, True, "layer", 0),
    "many_workgroups": ([96, 65] * 13, True, 6, 6, True, "layer", 0),
    "given_lengths": ([150, 190], True, 2, 2, False, "layer", 0),
    "no_decay": ([300], False, 2, 2, True, "none", 0),
    "segments": ([300, 130], True, 2, 2, True, "layer", 64),
    "many_segments": ([500, 700], True, 8, 8, True, "layer", 64),
    "grouped": ([150, 31], True, 2, 8, True, "layer", 0),
}


@pytest.mark.parametrize("case", list(CASES))
def test_results_are_rounded_once(case):
    lengths, packed, Hqk, Hv, unit, gates, segment = CASES[case]
    print(f"[delta precision] {case}", flush=True)
    inp = Inp(lengths, packed, Hqk, Hv, seed=300 + len(case), unit=unit, gates=gates)
    got = train(inp, segment=segment)
    o, _, (wo, _), _ = inp.reference()
    refs, weights, _ = inp.gradients()
    check_one_rounding("o", got[0], o, wo)
    for i, name in enumerate(("dq", "dk", "dv", "dg", "dbeta")):
        if i > 1 or Hqk == Hv:
            check_one_rounding(name, got[2 + i], refs[i], weights[i])


SHARED = {  # lengths, packed, Hqk, Hv, unit, segment
    "two": ([150, 31], True, 2, 4, True, 0),
    "four": ([200], False, 2, 8, True, 0),
    "three_of_given_length": ([70, 3, 130], True, 1, 3, False, 0),
    "segments": ([260] * 2, False, 2, 4, True, 64),
}


@pytest.mark.parametrize("case", list(SHARED))
def test_gradients_of_shared_heads_are_rounded_once(case):
    """dq and dk that sum over value heads: a head's partial is off by 2^-17 of itself, which the bars
    above leave room for (2^-17 of the partials' sizes for one element)."""
    lengths, packed, Hqk, Hv, unit, segment = SHARED[case]
    print(f"[delta precision] shared {case}", flush=True)
    inp = Inp(lengths, packed, Hqk, Hv, seed=320 + len(case), unit=unit)
    got = train(inp, segment=segment)
    refs, weights, parts = inp.gradients()
    for i, name in enumerate(("dq", "dk")):
        check_one_rounding(name, got[2 + i], refs[i], weights[i] + 2.0 ** -17 / FINE * parts[i])


def test_a_shared_heads_nan_and_infinity_stay_in_their_sequence():
    """A NaN of any bits in one value head's adjoint: its sequence's dq and dk are NaN where the heads
    are summed, the other sequence's what they are without."""
    inp = Inp([70, 40], True, 1, 2, seed=340)
    want = train(inp)
    inp.do[:, 10, 1] = torch.tensor([0x7fff], dtype=torch.int16).view(torch.bfloat16)
    got = train(inp)
    assert got[2][:, 10].isnan().all()
    for a, b in zip(got[2:7], want[2:7]):
        assert torch.equal(a[:, 70:], b[:, 70:])


@pytest.mark.parametrize("bits", [0x7fc00000, 0x7fffffff, -1, 0x7f800001, 0x7f800000])
@pytest.mark.parametrize("Hqk", [1, 2])
def test_a_states_nan_is_not_lost(bits, Hqk):
    """A NaN of any bits, or an infinity, in an initial state's or final adjoint's element [v, k]: the gradients that
    take it up are NaN or infinite (dq's channel k of every token that sees the state; every token's dk)."""
    inp = Inp([70, 40], True, Hqk, 2, seed=341, unit=False)
    bad = torch.tensor([bits], dtype=torch.int32).view(torch.float32)
    inp.s0[0, 1, 5, 7] = bad
    got = train(inp)
    assert not got[2][:, :64, Hqk - 1, 7].isfinite().any()
    assert all(t[:, 70:].isfinite().all() for t in got[2:7])
    inp = Inp([70, 40], True, Hqk, 2, seed=341, unit=False)
    inp.ds[0, 1, 5, 7] = bad
    got = train(inp)
    assert not got[3][:, :70, Hqk - 1, 7].isfinite().any()
    assert all(t[:, 70:].isfinite().all() for t in got[2:7])


def test_tokens_of_sizes_far_apart_in_one_block():
    """do and v of neighbouring tokens 2^30 apart: a small token's gradients are as exact as a large
    one's wherever its own terms make them up (its dq of the state before the block, by the state alone; its dv
    behind which nothing comes)."""
    inp = Inp([64], False, 1, 1, seed=342, unit=False)
    inp.ds.zero_()
    size = 2.0 ** -30 * torch.ones(64)
    size[::2] = 1.0
    size[63] = 2.0 ** -30
    inp.do = (inp.do.float() * size[None, :, None, None]).bfloat16()
    got = train(inp)
    refs, _, _ = inp.gradients()
    # dq_i is do_i times the state behind token i: all of a token's terms have do_i's size
    small = size < 1.0
    for name, x, ref in (("dq", got[2][:, small], refs[0][:, small]), ("dv", got[4][:, 63:], refs[2][:, 63:])):
        x = lu.f64(x)
        once = np.linalg.norm(lu.f64(torch.from_numpy(ref).bfloat16()) - ref)
        ratio = np.linalg.norm(x - ref) / once
        print(f"{name} norm {ratio:.5f} of one rounding's", flush=True)
        assert ratio <= 1 + lu.U, name
