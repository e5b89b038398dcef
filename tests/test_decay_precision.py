"""GPU tests of how far the decayed scan's results may be off: o, dq, dk and dv by
one BF16 rounding, the sums of shared heads by what their packed partials lose,
the states of long decodes by random roundings only.

Bars.  u = 2^-8 is half a BF16 step relative to the value.
  - One element with one rounding: u |ref| (and u of that, where the value crosses
    into the next binade), plus what came before the rounding.  The products P and
    the state go into their products as two BF16 pieces, off by at most 2^-18 of
    themselves: independent errors of standard deviation 2^-18 / sqrt(3), which for
    P and the state together add up to 2^-18 sqrt(2/3) sqrt(energy) (energy: the
    definition at squared inputs, tests/layer_util.py); 8 of those are 2^-15.3 of
    it.  The factors e^{l(i-j)} are off by about 2^-23 (an exponential of 2^-23,
    an exponent of 2^-24 of itself, which the factor's own size outweighs), sums of
    160 products in FP32 by 8 sqrt(160) 2^-24 = 2^-17.3: 2^-14 of sqrt(energy) in all.
  - The norm of the error: a rounding's is 2^-8 / sqrt(3) = 0.58 u of values with
    mantissas of 1, and 0.42 u of mantissas spread evenly over their logarithm; the
    bar is 0.5 u.
"""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo
from tests import layer_util as lu
from tests.test_decay_attention import SCALE, Inp, train

pytestmark = pytest.mark.gpu

FINE = 2.0 ** -14


def check_one_rounding(name, got, ref, energy, extra=0.0):
    got = lu.f64(got)
    assert np.isfinite(got).all(), f"{name}: not finite"
    err = np.abs(got - ref)
    rel = np.linalg.norm(err) / np.linalg.norm(ref)
    worst = (err / np.maximum(lu.U * np.abs(ref) * (1 + lu.U) + FINE * np.sqrt(energy) + extra, 1e-30)).max()
    print(f"{name:4s} rel {rel / lu.U:.3f} u (bar 0.5 u)  elementwise {worst:.2f} of the bar", flush=True)
    assert worst <= 1.0 and rel <= 0.5 * lu.U, name


CASES = {  # lengths, packed, Hqk, Hv, segment: every launch variant, whole and cut
    "few_workgroups": ([70, 200, 33], True, 3, 3, 0),
    "eight_waves": ([96] * 25, False, 6, 6, 0),
    "many_workgroups": ([40, 65] * 20, True, 8, 8, 0),
    "grouped": ([150, 31], True, 2, 8, 0),
    "segments": ([300, 130], True, 2, 2, 64),
    "long": ([2100], False, 4, 4, 0),
}


@pytest.mark.parametrize("case", list(CASES))
def test_results_are_rounded_once(case):
    lengths, packed, Hqk, Hv, segment = CASES[case]
    print(f"[precision] {case}", flush=True)
    inp = Inp(lengths, packed, Hqk, Hv, seed=31 + len(case))
    got = train(inp, segment)
    (dq, dk, dv, _), _ = inp.gradients()
    energies = inp.energies()
    check_one_rounding("o", got[0], inp.reference()[0], energies[0])
    check_one_rounding("dv", got[4], dv, energies[3])
    if Hqk == Hv:
        check_one_rounding("dq", got[2], dq, energies[1])
        check_one_rounding("dk", got[3], dk, energies[2])


def test_prefill_is_rounded_once():
    import gated_delta_rule_32_amd as kda
    inp = Inp([90, 257], True, 2, 4, seed=32)
    out, _ = kda.decay_attention(*(inp.dev(x) for x in (inp.q, inp.k, inp.v, inp.l)), inp.s0.cuda(),
                                 cu_seqlens=inp.dev(inp.cu), cu_seqlens_cpu=inp.cu)
    check_one_rounding("o", out, inp.reference()[0], inp.energies()[0])
