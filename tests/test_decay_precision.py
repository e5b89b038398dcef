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


# ---------------------------------------------------------------------------
# packed partials of shared heads
# ---------------------------------------------------------------------------
# A partial keeps 10 significant bits, rounded once: off by at most 2^-10 of
# itself, or, far below the largest of its quad of channels, 2^-23 of that one.
PACK, PACK_SMALL = 2.0 ** -10, 2.0 ** -23


def shared_sum(x, y):
    """dq and dk as the sums of two given partials each: one token per sequence,
    two value heads on one q/k head, no decay, q = k = 0, and do and v that pick
    row 0 of the states, so that dq is x[:, 0] + y[:, 0] (the initial state's
    rows) and dk is x[:, 1] + y[:, 1] (the final state's adjoint's)."""
    import gated_delta_rule_32_amd as kda
    n = x.shape[0]
    zero = torch.zeros((n, 1, 1, 128), dtype=torch.bfloat16, device="cuda")
    pick = torch.zeros((n, 1, 2, 128), dtype=torch.bfloat16, device="cuda")
    pick[..., 0] = 1.0
    states = [torch.zeros((n, 2, 128, 128), device="cuda") for _ in range(2)]
    for i in range(2):
        states[i][:, 0, 0], states[i][:, 1, 0] = x[:, i].cuda(), y[:, i].cuda()
    _, _, ctx = kda.decay_attention_training_forward(zero, zero, pick, torch.zeros(2, device="cuda"), states[0], scale=1.0)
    dq, dk, _, _ = kda.decay_attention_training_backward(ctx, pick, states[1])
    return torch.stack((dq[:, 0, 0], dk[:, 0, 0]), 1).double().cpu()


def test_partials_of_shared_heads_are_rounded_once():
    """x has 16 significant bits, which the two BF16 pieces of a state hold, and
    the other head's partial is -bf16(x), which no rounding touches, so that the
    sum (a few last bits, exact in BF16) shows what became of x.  Rounded to nearest,
    the deviations of 131072 values have a standard deviation of at most 2^-10 /
    sqrt(3) of themselves and a mean of nothing: bar 6 standard deviations of the
    mean, 6 x 2^-10 / sqrt(3) / sqrt(131072) = 9.3e-6.  (Rounded twice, with all ties away from zero,
    they had a mean of 3.5e-4 and a worst value of 1.5 x 2^-10.)"""
    g = torch.Generator().manual_seed(33)
    n = 512
    x = (1 + torch.randint(2 ** 15, (n, 2, 128), generator=g) * 2.0 ** -15).float()
    x = x * torch.exp2(torch.randint(-3, 4, (n, 2, 128), generator=g).float())
    x = x * torch.where(torch.rand((n, 2, 128), generator=g) < 0.5, -1.0, 1.0)
    near = x.bfloat16().float()
    kept = shared_sum(x, -near) + near.double()
    off = (kept / x.double() - 1).numpy()
    bar = 6 * PACK / 3 ** 0.5 / off.size ** 0.5
    print(f"worst {np.abs(off).max() / PACK:.3f} x 2^-10, mean {off.mean():.2e} (bar {bar:.1e})", flush=True)
    assert np.abs(off).max() <= PACK and abs(off.mean()) <= bar


def test_small_partials_beside_large_ones():
    """Channels of a quad 2^0 to 2^40 apart, at several sizes of the whole."""
    g = torch.Generator().manual_seed(34)
    n = 64
    x = torch.randn((n, 2, 128), generator=g) * torch.exp2(-40 * torch.rand((n, 2, 128), generator=g))
    x = x * torch.exp2(torch.randint(-60, 61, (n, 1, 1), generator=g).float())
    got, ref = shared_sum(x, torch.zeros_like(x)), x.double()
    top = ref.abs().unflatten(-1, (-1, 4)).amax(-1, keepdim=True).expand(-1, -1, -1, 4).flatten(-2)
    bar = (lu.U * (1 + PACK) + PACK + 2.0 ** -17) * ref.abs() + PACK_SMALL * top
    worst = ((got - ref).abs() / bar).max()
    print(f"{worst:.3f} of the bar", flush=True)
    assert worst <= 1.0


@pytest.mark.parametrize("segment", [0, 64])
def test_gradients_of_shared_heads(segment):
    """Against the sum of the single heads' gradients, whose absolute values say
    what the partials lose."""
    inp = Inp([150, 31, 64], True, 2, 6, seed=35)
    got = train(inp, segment)
    alone = Inp([150, 31, 64], True, 6, 6, seed=35)
    for name in ("q", "k"):
        setattr(alone, name, getattr(inp, name).repeat_interleave(3, 2))
    for name in ("v", "do", "s0", "ds"):
        setattr(alone, name, getattr(inp, name))
    (dq, dk, _, _), _ = alone.gradients()
    energies = inp.energies()
    for name, x, heads, energy in (("dq", got[2], dq, energies[1]), ("dk", got[3], dk, energies[2])):
        heads = heads.reshape(1, 245, 2, 3, 128)
        top = np.abs(heads).reshape(1, 245, 2, 3, 32, 4).max(-1, keepdims=True).repeat(4, -1).reshape(heads.shape)
        check_one_rounding(name, x, heads.sum(3), energy, PACK * np.abs(heads).sum(3) + PACK_SMALL * top.sum(3))


# ---------------------------------------------------------------------------
# long decodes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("l", [-1e-5, -3.3e-5, -1.7e-4, -0.25])
@pytest.mark.parametrize("tokens", [1, 8])
def test_decode_does_not_drift(l, tokens):
    """A state decays over 16384 decoded tokens of zeros to e^{16384 l} of itself.
    Each token rounds it once (and a far smaller product), to nearest: standard
    deviation at most 2^-24 / sqrt(3) of the state, sqrt(16384) of it in the end if
    the roundings are independent, and of the mean over 16384 elements 1/128 of
    that; bars of 6 standard deviations.  A factor rounded to FP32 would move the
    mean by up to 16384 x 2^-25 = 4.9e-4.

    Under a weak decay the roundings of neighbouring tokens are alike, also of exact
    products.  A token takes d = (1 - e^l) x off x, D = d / ulp is between 2^23
    (1 - e^l) and twice that, and the rounding is that of D to a whole number.  D
    shrinks by (1 - e^l) D a token, so that it takes p = 1 / ((1 - e^l) D) <= 1 /
    ((1 - e^l)^2 2^23) tokens from one whole number to the next.  Over such a period
    the roundings go evenly through -1/2 .. 1/2 ulp and cancel; a part of one leaves
    at most the sum over a half's tokens with one sign, p / 8 ulp, where an ulp is
    at most 2^-23 of x.  Every binade that the state passes through starts anew:
    (1 + binades) p / 8 x 2^-23 more, for the mean as well (l = -1e-5: p = 1192,
    1.8e-5 a binade)."""
    import gated_delta_rule_32_amd as kda
    L = 16384 if l > -0.1 else 64
    x = torch.zeros((1, tokens, 1, 128), dtype=torch.bfloat16, device="cuda")
    s0 = torch.rand((1, 1, 128, 128), generator=torch.Generator().manual_seed(36)) + 1
    decay = torch.tensor([l], device="cuda")
    pool, out = s0.cuda(), torch.empty_like(x)
    for _ in range(L // tokens):
        kda.decay_attention(x, x, x, decay, pool, output=out)
    off = lu.f64(pool) / (lu.f64(s0) * np.exp(float(np.float32(l)) * L)) - 1
    std = L ** 0.5 * 2.0 ** -24 / 3 ** 0.5
    alike = (1 + np.ceil(-l * L / np.log(2))) / (8 * np.expm1(l) ** 2 * 2.0 ** 23) * 2.0 ** -23
    print(f"max {np.abs(off).max():.2e} (bar {6 * std + alike:.2e}), mean {abs(off.mean()):.2e} "
          f"(bar {6 * std / 128 + alike:.2e})", flush=True)
    assert np.abs(off).max() <= 6 * std + alike and abs(off.mean()) <= 6 * std / 128 + alike


# ---------------------------------------------------------------------------
# segments
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("segment", [0, 64, 256])
def test_segments_agree_with_one_walk(segment):
    """All results in segments against those of whole sequences (segments of 65536
    tokens, which take no workspace).  States: a chunk of 32 tokens adds to them in
    three products, a rescaling and a segment's end round once more, each off by at
    most 2^-23 of the sum of absolute values; 25 chunks, 4 roundings each, both
    routes.  The others: one BF16 rounding each, which may fall to either side."""
    import gated_delta_rule_32_amd as kda
    inp = Inp([777, 130], True, 2, 2, seed=37)
    p = kda.KdaDecayProblem(1, 907, 2, 2, 2, inp.cu.data_ptr(), inp.cu.data_ptr(), 0.0, 65536)
    assert kda.kda_decay_fwd_workspace_bytes(p) == kda.kda_decay_bwd_workspace_bytes(p) == 0
    p.segment = segment
    # (0: whatever the library takes)
    assert segment == 0 or min(kda.kda_decay_fwd_workspace_bytes(p), kda.kda_decay_bwd_workspace_bytes(p)) > 0
    whole, cut = train(inp, 65536), train(inp, segment)
    (dq, dk, dv, dinit), minit = inp.gradients()
    o, final, _, mfinal = inp.reference()
    bar = 25 * 4 * 2.0 ** -23
    for name, i, ref, major in (("final_state", 1, final, mfinal), ("dinitial_state", 5, dinit, minit)):
        lu.check_bars(name, whole[i], ref, bar * major)
        lu.check_bars(name, cut[i], lu.f64(whole[i]), 2 * bar * major)
    for name, i, ref, energy in zip(("o", "dq", "dk", "dv"), (0, 2, 3, 4), (o, dq, dk, dv), inp.energies()):
        check_one_rounding(name, cut[i], ref, energy)
        lu.check_bars(name, cut[i], lu.f64(whole[i]),
                      2 * (lu.U * (1 + lu.U) * np.abs(ref) + FINE * np.sqrt(energy)))


@pytest.mark.parametrize("l", [-1e-5, -3.3e-5, -1.7e-4])
@pytest.mark.parametrize("tokens", [9, 33, 100])
def test_prefill_in_pieces_does_not_drift(l, tokens):
    """The same for a prompt that comes in 2048 pieces of a few chunks: a piece decays
    the state by e^{tokens l} and rounds it once.  That sequence of exact products,
    each rounded to nearest, is followed in 64 bits; the kernel's product is off by
    2^-47 before its rounding, which so goes the other way about once in 2^-24 / 2^-47
    = 2^23 cases, 4 times among 2048 x 16384, and mostly in different elements: bar
    4 last bits of one element, 2^-23 each, and 4 x 2^-23 / 16384 x 4 for the mean.  A
    factor rounded to FP32 would move the mean by up to 2048 x 2^-25 = 6.1e-5.  (The
    sequence itself is up to 1.2e-7 off on average where e^{tokens l} makes the
    roundings of neighbouring values alike.)"""
    import gated_delta_rule_32_amd as kda
    calls = 2048
    x = torch.zeros((1, tokens, 1, 128), dtype=torch.bfloat16, device="cuda")
    s0 = torch.rand((1, 1, 128, 128), generator=torch.Generator().manual_seed(38)) + 1
    decay = torch.tensor([l], device="cuda")
    pool, out = s0.cuda(), torch.empty_like(x)
    for _ in range(calls):
        kda.decay_attention(x, x, x, decay, pool, output=out)
    factor, ideal = np.exp(float(np.float32(l)) * tokens), s0.numpy()
    for _ in range(calls):
        ideal = (ideal.astype(np.float64) * factor).astype(np.float32)
    off = lu.f64(pool) / ideal.astype(np.float64) - 1
    print(f"max {np.abs(off).max():.2e} (bar {4 * 2.0 ** -23:.2e}), mean {abs(off.mean()):.2e} (bar {2.0 ** -33:.2e})",
          flush=True)
    assert np.abs(off).max() <= 4 * 2.0 ** -23 and abs(off.mean()) <= 2.0 ** -33


@pytest.mark.parametrize("l", [-1e-5, -3.3e-5, -1.7e-4])
def test_prefill_in_segmented_pieces_does_not_drift(l):
    """Pieces of 200 tokens in segments of 64, 64, 64 and 8, each of which decays the
    state and rounds it once: bars as above for 4 x 512 roundings."""
    import gated_delta_rule_32_amd as kda
    x = torch.zeros((1, 200, 1, 128), dtype=torch.bfloat16, device="cuda")
    s0 = torch.rand((1, 1, 128, 128), generator=torch.Generator().manual_seed(39)) + 1
    decay = torch.tensor([l], device="cuda")
    pool, out = s0.cuda(), torch.empty_like(x)
    for _ in range(512):
        kda.decay_attention(x, x, x, decay, pool, output=out, segment=64)
    ideal = s0.numpy()
    for n in [64, 64, 64, 8] * 512:
        ideal = (ideal.astype(np.float64) * np.exp(float(np.float32(l)) * n)).astype(np.float32)
    off = lu.f64(pool) / ideal.astype(np.float64) - 1
    print(f"max {np.abs(off).max():.2e} (bar {4 * 2.0 ** -23:.2e}), mean {abs(off.mean()):.2e} (bar {2.0 ** -33:.2e})",
          flush=True)
    assert np.abs(off).max() <= 4 * 2.0 ** -23 and abs(off.mean()) <= 2.0 ** -33
