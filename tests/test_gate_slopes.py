"""GPU tests of the gated norm's gate gradient at open, closed and infinite gates.

Bar: dgate = dy w x^ slope is rounded once (u |ref|, u = 2^-8, and u of that).  Before it, about
ten FP32 operations, and the exponential of the gate: its argument g log2(e) is
rounded to 2^-24 of itself, and so is the product, which moves e^g by up to
|g| 2^-23 of itself, for |g| <= 80 by 2^-16.7.  Hardware exponential,
reciprocal and square root: 2^-22 each.  2^-16 in all.
"""
import math

import numpy as np
import pytest
import torch

from tests import layer_util as lu

pytestmark = pytest.mark.gpu

EPS = 1e-6
FINE = 2.0 ** -16


def slopes(g, silu):
    """The slope without cancellation, in 64 bits: sigmoid(-g) in place of 1 - sigmoid(g)."""
    with np.errstate(over="ignore"):
        s, t = 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))
    return s * (1 + g * t) if silu else s * t


def gate_gradient(gate, act, seed):
    import gated_delta_rule_32_amd as kda
    gen = torch.Generator().manual_seed(seed)
    x, dy = (lu.bf(gen, *gate.shape) for _ in range(2))
    w = torch.randn(128, generator=gen)
    dx, dg, dw = kda.gated_norm_backward(dy.cuda(), x.cuda(), gate.cuda(), w.cuda(), activation=act)
    xn = lu.f64(x) / np.sqrt((lu.f64(x) ** 2).mean(-1, keepdims=True) + EPS)
    return dx, dg, dw, lu.f64(dy) * lu.f64(w) * xn


def test_sigmoid_slope_of_open_and_closed_gates():
    """Relative to the slope itself, at either sign."""
    values = [0.0, 0.5, 3.0, 6.0, 9.0, 12.0, 14.0, 16.0, 17.0, 20.0, 30.0, 50.0, 80.0]
    gate = torch.tensor(values + [-v for v in values]).bfloat16()[None, :, None, None].expand(1, -1, 3, 128).contiguous()
    _, dg, _, terms = gate_gradient(gate, "sigmoid", 41)
    ref = terms * slopes(lu.f64(gate), False)
    lu.check_bars("dgate", dg, ref, (lu.U * (1 + lu.U) + FINE) * np.abs(ref))


def test_silu_slope_of_open_and_closed_gates():
    """Where the slope's two terms cancel (g = -1.28), relative to those; elsewhere they do not."""
    values = [0.0, 0.5, 1.25, 1.28, 1.3, 3.0, 6.0, 12.0, 16.0, 20.0, 50.0, 80.0]
    gate = torch.tensor(values + [-v for v in values]).bfloat16()[None, :, None, None].expand(1, -1, 3, 128).contiguous()
    _, dg, _, terms = gate_gradient(gate, "silu", 42)
    g = lu.f64(gate)
    s, t = 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))
    ref = terms * slopes(g, True)
    lu.check_bars("dgate", dg, ref, lu.U * (1 + lu.U) * np.abs(ref) + FINE * np.abs(terms) * s * (1 + np.abs(g) * t))


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_slopes_of_infinite_gates(act):
    """Gates of minus and plus infinity and of the type's lowest and highest value:
    the slope is 0, but 1 for an open SiLU gate; a closed gate's dx is 0 too."""
    top = torch.finfo(torch.bfloat16).max
    gate = torch.tensor([-math.inf, -top, math.inf, top])[None, :, None, None].expand(1, 4, 2, 128)
    dx, dg, _, terms = gate_gradient(gate.to(torch.bfloat16).contiguous(), act, 43)
    assert not dg[0, :2].any() and not dx[0, :2].any()
    ref = terms[0, 2:] if act == "silu" else np.zeros_like(terms[0, 2:])
    lu.check_bars("dgate", dg[0, 2:], ref, (lu.U * (1 + lu.U) + FINE) * np.abs(ref))


def test_a_nan_gate_is_seen():
    gate = torch.zeros((1, 1, 1, 128), dtype=torch.bfloat16)
    gate[0, 0, 0, 5] = math.nan
    for act in ("sigmoid", "silu"):
        dg = gate_gradient(gate, act, 44)[1]
        assert torch.isnan(dg[0, 0, 0, 5]) and torch.isfinite(dg[0, 0, 0, :5]).all() and torch.isfinite(dg[0, 0, 0, 6:]).all()


def test_rows_of_zeros_at_the_smallest_eps():
    import gated_delta_rule_32_amd as kda
    x = torch.zeros((1, 2, 1, 128), dtype=torch.bfloat16)
    x[0, 1] = 3.0
    one, w = torch.ones_like(x).cuda(), torch.ones(128, device="cuda")
    eps = 2.0 ** -126
    y = kda.gated_norm_forward(x.cuda(), one, w, eps=eps)
    d = kda.gated_norm_backward(one, x.cuda(), one, w, eps=eps)
    cos, sin = kda.rotary_table(2, 128)
    q = kda.qk_norm_rope_forward(x.cuda(), x.cuda(), w, w, cos, sin, eps=eps)
    assert not y[0, 0].any() and not q[0][0, 0].any() and all(torch.isfinite(t).all() for t in (y, *d, *q))
    lu.check_bars("y", y[0, 1], np.full((1, 128), 1 / (1 + math.exp(-1))), lu.U)
