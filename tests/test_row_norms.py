"""GPU parity of the per-head row norms (kda_qknorm_*, kda_gnorm_*) against
their FP64 definitions.

Bars: an output is rounded once (u |ref|); before it, FP32 arithmetic of about
16 operations on values no larger than a few times the row's largest term adds
2^-20 of that: u |ref| + 2^-20 times the row's (for the rotation: the pair's)
scale.  A weight gradient adds up N terms in FP32, in runs of at most N / 16
per lane: bounded by 2^-24 N of the sum of absolute values for small N; the bar
is 2^-24 (N / 16 + 64) of it.
"""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo
from tests import layer_util as lu

pytestmark = pytest.mark.gpu

FINE = 2.0 ** -20


def bar(ref, scale):
    return lu.U * np.abs(ref) * (1 + lu.U) + FINE * scale


def row_scale(ref):
    return np.abs(ref).max(-1, keepdims=True) + 1e-30


def weight_bar(terms, n):
    return 2.0 ** -24 * (n / 16 + 64) * terms


CASES = {  # B, T, Hq, Hk, rot, pairs, positions
    "one_token": (1, 1, 1, 1, 128, False, True),
    "decode_batch": (5, 1, 8, 2, 128, False, True),
    "odd": (2, 37, 3, 1, 64, False, True),
    "pairs": (1, 29, 4, 4, 128, True, True),
    "pairs_partial": (1, 41, 2, 1, 24, True, True),
    "smallest_rotation": (1, 17, 2, 2, 8, False, True),
    "largest_odd_rotation": (1, 17, 2, 2, 120, False, True),
    "no_positions": (3, 50, 2, 1, 96, False, False),
    "many_rows": (1, 1500, 12, 4, 128, False, True),
}


def tables(rows, rot):
    import gated_delta_rule_32_amd as kda
    return kda.rotary_table(rows, rot)


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("case", list(CASES))
def test_qk_norm_rope(case, fused):
    import gated_delta_rule_32_amd as kda
    B, T, Hq, Hk, rot, pairs, given = CASES[case]
    print(f"[qknorm] case={case} fused={fused}", flush=True)
    g = torch.Generator().manual_seed(len(case))
    qkv = lu.bf(g, B, T, Hq + Hk + 2, 128)
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    dyq, dyk = lu.bf(g, B, T, Hq, 128), lu.bf(g, B, T, Hk, 128)
    wq, wk = torch.randn(128, generator=g), torch.randn(128, generator=g)
    rows = 5000
    cos, sin = tables(rows, rot)
    pos = torch.randint(rows, (B, T), generator=g)
    if given:
        pos[0, 0], pos[-1, -1] = 0, rows - 1
    else:
        pos = torch.arange(T).expand(B, T)
    dqkv = qkv.cuda()
    dev = (dqkv[:, :, :Hq], dqkv[:, :, Hq:Hq + Hk])
    if not fused:
        dev = tuple(x.contiguous() for x in dev)
    args = (*dev, wq.cuda(), wk.cuda(), cos, sin, pos.contiguous().cuda() if given else None)
    y = kda.qk_norm_rope_forward(*args, eps=1e-5, interleaved=pairs)
    grads = kda.qk_norm_rope_backward(dyq.cuda(), dyk.cuda(), *args, eps=1e-5, interleaved=pairs)
    torch.cuda.synchronize()
    c, s = lu.f64(cos), lu.f64(sin)
    for i, (x, w, dy, name) in enumerate(((q, wq, dyq, "q"), (k, wk, dyk, "k"))):
        ref = lo.qk_norm_rope(lu.f64(x), lu.f64(w), c, s, pos.numpy(), rot, pairs, 1e-5)
        dx, dw = lo.qk_norm_rope_backward(lu.f64(dy), lu.f64(x), lu.f64(w), c, s, pos.numpy(), rot, pairs, 1e-5)
        lu.check_bars(name, y[i], ref, bar(ref, row_scale(ref)))
        # the terms of dx, before they cancel: |w dn| r and |x^| mean|w dn x^| r
        r = 1 / np.sqrt((lu.f64(x) ** 2).mean(-1, keepdims=True) + 1e-5)
        terms = r * np.abs(lu.f64(w)).max() * row_scale(lu.f64(dy)) * (1 + 4 * row_scale(lu.f64(x)) * r)
        lu.check_bars("d" + name, grads[i], dx, bar(dx, terms))
        mass = (np.abs(lu.f64(dy)).max(-1, keepdims=True) * 1.5 * np.abs(lu.f64(x)) * r).sum((0, 1, 2))
        lu.check_bars(f"d{name}_weight", grads[2 + i], dw, weight_bar(mass, B * T * (Hq + Hk)) + FINE * mass)


def test_position_outside_the_table_is_nan():
    import gated_delta_rule_32_amd as kda
    g = torch.Generator().manual_seed(1)
    q, k = lu.bf(g, 1, 4, 2, 128).cuda(), lu.bf(g, 1, 4, 1, 128).cuda()
    w = torch.ones(128, device="cuda")
    cos, sin = tables(10, 64)
    pos = torch.tensor([[3, -1, 10, 9]], device="cuda")
    yq, yk = kda.qk_norm_rope_forward(q, k, w, w, cos, sin, pos)
    for y in (yq, yk):
        assert torch.isnan(y[0, 1:3]).all() and torch.isfinite(y[0, 0]).all() and torch.isfinite(y[0, 3]).all()


def test_rows_of_zeros_and_large_values():
    """A zero row stays zero (eps keeps its norm finite), a row of large values
    is normed like any other, and a row far below eps is scaled by eps alone."""
    import gated_delta_rule_32_amd as kda
    x = torch.zeros((1, 3, 1, 128), dtype=torch.bfloat16)
    x[0, 1] = 1e15
    x[0, 2, 0, 7] = 1e-20
    g = torch.zeros_like(x)
    w = torch.ones(128)
    y = kda.gated_norm_forward(x.cuda(), g.cuda(), w.cuda(), eps=1e-6)
    ref = lo.gated_norm(lu.f64(x), lu.f64(g), lu.f64(w), False, 1e-6)
    lu.check_bars("y", y, ref, bar(ref, row_scale(ref)))


GCASES = {"one": (1, 1, 1), "odd": (2, 33, 3), "batch": (6, 1, 5), "many": (1, 2000, 16)}


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("case", list(GCASES))
def test_gated_norm(case, fused, act):
    import gated_delta_rule_32_amd as kda
    B, T, H = GCASES[case]
    print(f"[gnorm] case={case} fused={fused} act={act}", flush=True)
    gen = torch.Generator().manual_seed(7)
    wide = lu.bf(gen, B, T, 2 * H + 1, 128)
    x, g = wide[:, :, :H], wide[:, :, H:2 * H] * 4
    dy, w = lu.bf(gen, B, T, H, 128), torch.randn(128, generator=gen)
    if fused:
        buf = torch.cat((x, g, wide[:, :, 2 * H:]), 2).cuda()
        dev = (buf[:, :, :H], buf[:, :, H:2 * H])
    else:
        dev = (x.contiguous().cuda(), g.contiguous().cuda())
    y = kda.gated_norm_forward(*dev, w.cuda(), activation=act)
    dx, dg, dw = kda.gated_norm_backward(dy.cuda(), *dev, w.cuda(), activation=act)
    torch.cuda.synchronize()
    a = [lu.f64(t) for t in (x, g, w)]
    silu = act == "silu"
    ref = lo.gated_norm(*a, silu, 1e-6)
    lu.check_bars("y", y, ref, bar(ref, np.abs(ref)))
    rdx, rdg, rdw = lo.gated_norm_backward(lu.f64(dy), *a, silu, 1e-6)
    r = 1 / np.sqrt((a[0] ** 2).mean(-1, keepdims=True) + 1e-6)
    actv, slope = lo._act(a[1], silu)
    t = np.abs(lu.f64(dy) * a[2] * actv) * r
    xh = np.abs(a[0]) * r
    lu.check_bars("dx", dx, rdx, bar(rdx, t + xh * (t * xh).mean(-1, keepdims=True)))
    # the slope's own terms: s (1 + |g| (1 - s)); 1 - s loses up to 2^-23 absolutely
    loss = np.abs(lu.f64(dy) * a[2]) * xh * (2.0 ** -20 * (1 + np.abs(a[1])))
    lu.check_bars("dgate", dg, rdg, bar(rdg, np.abs(rdg)) + loss)
    mass = np.abs(lu.f64(dy) * actv * a[0] * r).sum((0, 1, 2))
    lu.check_bars("dweight", dw, rdw, weight_bar(mass, B * T * H) + FINE * mass)


def test_deterministic_and_captured():
    """The weight gradients are the same bits every time, and in a replayed graph."""
    import gated_delta_rule_32_amd as kda
    gen = torch.Generator().manual_seed(3)
    x, g, dy = (lu.bf(gen, 1, 700, 6, 128).cuda() for _ in range(3))
    w = torch.randn(128, generator=gen).cuda()
    cos, sin = tables(700, 64)
    qa = (x[:, :, :4], x[:, :, 4:], w, w, cos, sin)
    da = (dy[:, :, :4].contiguous(), dy[:, :, 4:].contiguous())

    def step():
        return (kda.gated_norm_forward(x, g, w), *kda.gated_norm_backward(dy, x, g, w),
                *kda.qk_norm_rope_forward(*qa), *kda.qk_norm_rope_backward(*da, *qa))

    want = step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        again = step()
        for a, b, c in zip(want, got, again):
            assert torch.equal(a, b) and torch.equal(a, c)
