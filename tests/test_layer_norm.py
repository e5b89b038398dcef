"""GPU tests of the layer norm (kda_lnorm_*) against the FP64 oracle.

Bars.  u = 2^-8, one BF16 rounding.  In FP32 the mean of C values is off by at most
2^-24 log2(C) of their mean size (sums go in trees, of at most 12 values a thread in turn), which
moves every x - m alike, and 1 / sqrt by a few of 2^-24: 2^-19 of max|x| r |w| for y, beside the
rounding.  dx adds two more such means: 2^-18 of the sizes of d r, and of h mean|d h| r.  dw and db: each
of the workgroup's sums takes its rows in turn, then the workgroups' sums in fours: with n
rows 2^-24 (n / workgroups + workgroups / 16 + 4) of the terms' sizes at most, and 2^-18 of them for h."""
import numpy as np
import pytest
import torch

from oracle import delta_oracle as do_
from tests import layer_util as lu

pytestmark = pytest.mark.gpu

SHAPES = [(1, 8), (3, 16), (5, 504), (70, 512), (9, 520), (13, 1024), (6, 1032), (700, 2048), (33, 4096), (7, 6144 + 8),
          (5, 8192), (3, 12288), (4, 12296), (3, 16384), (2, 16392), (3, 32760), (2, 32768),
          (20001, 96), (9000, 128), (2500, 136), (2100, 1000), (1300, 4096), (700, 12288), (300, 16384), (270, 24000),
          (260, 32768)]    # (more rows than workgroups take at once)


def make(T, C, seed, shift=0.5):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((T, C), generator=g) + shift * torch.randn((T, 1), generator=g)).bfloat16()
    return x, 1 + 0.2 * torch.randn(C, generator=g), 0.3 * torch.randn(C, generator=g), lu.bf(g, T, C)


def check_forward(y, x, w, b, eps):
    ref, hat = do_.layer_norm(lu.f64(x), lu.f64(w), None if b is None else lu.f64(b), eps)
    x64 = lu.f64(x)
    size = np.sqrt(x64.var(-1, keepdims=True) + eps)
    top = np.abs(x64).max(-1, keepdims=True) / size
    bar = (top + np.abs(hat)) * np.abs(lu.f64(w)) + (0.0 if b is None else np.abs(lu.f64(b)))
    lu.check_bars("y", y, ref, lu.U * np.abs(ref) + 2.0 ** -19 * bar)


def check_backward(got, dy, x, w, eps):
    dx, dw, db = do_.layer_norm_backward(*(lu.f64(t) for t in (dy, x, w)), eps)
    x64, d = lu.f64(x), np.abs(lu.f64(dy) * lu.f64(w))
    size = np.sqrt(x64.var(-1, keepdims=True) + eps)
    _, hat = do_.layer_norm(x64, np.ones(x.shape[1]), None, eps)
    top = np.abs(x64).max(-1, keepdims=True) / size + np.abs(hat)
    bar = (d + d.mean(-1, keepdims=True) + top * (d * np.abs(hat)).mean(-1, keepdims=True) + top * d.mean(-1, keepdims=True)) / size
    lu.check_bars("dx", got[0], dx, lu.U * np.abs(dx) + 2.0 ** -18 * bar)
    sums = 2.0 ** -24 * (x.shape[0] / 256 + 36)
    terms = (np.abs(lu.f64(dy)) * np.abs(hat)).sum(0)
    lu.check_bars("dw", got[1], dw, sums * terms + 2.0 ** -18 * (np.abs(lu.f64(dy)) * top).sum(0))
    if got[2] is not None:
        lu.check_bars("db", got[2], db, sums * np.abs(lu.f64(dy)).sum(0))


@pytest.mark.parametrize("T,C", SHAPES)
def test_parity(T, C):
    import gated_delta_rule_32_amd as kda
    print(f"[lnorm] {T} {C}", flush=True)
    x, w, b, dy = make(T, C, T + C)
    y = kda.layer_norm_forward(x.cuda(), w.cuda(), b.cuda())
    got = kda.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda())
    torch.cuda.synchronize()
    check_forward(y, x, w, b, 1e-5)
    check_backward(got, dy, x, w, 1e-5)


@pytest.mark.parametrize("T,C", [(66000, 1024), (5500, 12288)])
def test_more_than_a_cache_holds(T, C):
    """Rows that go past the caches: the same bits as of the rows by themselves, and the sums over
    all of them."""
    import gated_delta_rule_32_amd as kda
    g = torch.Generator(device="cuda").manual_seed(5)
    x, dy = (torch.randn((T, C), generator=g, device="cuda").bfloat16() for _ in range(2))
    w, b = (torch.randn(C, generator=g, device="cuda") for _ in range(2))
    y, (dx, dw, db) = kda.layer_norm_forward(x, w, b), kda.layer_norm_backward(dy, x, w)
    for r in (slice(0, 40), slice(T // 2, T // 2 + 40), slice(T - 40, T)):
        assert torch.equal(kda.layer_norm_forward(x[r], w, b), y[r])
        assert torch.equal(kda.layer_norm_backward(dy[r], x[r], w)[0], dx[r])
    sum_w, sum_b, terms_w, terms_b = (torch.zeros(C, dtype=torch.float64, device="cuda") for _ in range(4))
    for i in range(0, T, 4096):
        x64, d64 = x[i:i + 4096].double(), dy[i:i + 4096].double()
        c = x64 - x64.mean(-1, keepdim=True)
        h = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5)
        sum_w += (d64 * h).sum(0)
        sum_b += d64.sum(0)
        terms_w += (d64 * h).abs().sum(0)
        terms_b += d64.abs().sum(0)
    # a thread adds T / 256 rows in turn at most, the second kernel 8 and 16 partial sums: 2^-24 each; h 2^-20
    bar = 2.0 ** -24 * (T / 256 + 24)
    assert ((dw - sum_w).abs() <= (bar + 2.0 ** -20) * terms_w).all()
    assert ((db - sum_b).abs() <= bar * terms_b).all()


def test_without_a_bias_and_with_another_eps():
    import gated_delta_rule_32_amd as kda
    x, w, _, dy = make(17, 264, 1)
    check_forward(kda.layer_norm_forward(x.cuda(), w.cuda(), eps=0.25), x, w, None, 0.25)
    check_backward(kda.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), eps=0.25), dy, x, w, 0.25)
    p = kda.KdaLNormProblem(17, 264, 0.25, 0)
    dx, dw = torch.empty_like(x, device="cuda"), torch.empty_like(w, device="cuda")
    ws = torch.empty(kda.kda_lnorm_bwd_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    kda.kda_lnorm_bwd(p, x.cuda(), w.cuda(), dy.cuda(), dx, dw, None, ws)   # no gradient of a bias
    torch.cuda.synchronize()
    check_backward((dx, dw, None), dy, x, w, 0.25)


def test_rows_far_from_zero():
    """A mean a hundred times the spread: the squares are summed around it."""
    import gated_delta_rule_32_amd as kda
    g = torch.Generator().manual_seed(2)
    x = (100.0 + torch.randn((6, 1000), generator=g)).bfloat16()
    _, w, b, dy = make(6, 1000, 3)
    check_forward(kda.layer_norm_forward(x.cuda(), w.cuda(), b.cuda()), x, w, b, 1e-5)
    check_backward(kda.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda()), dy, x, w, 1e-5)


def test_rows_of_one_value():
    import gated_delta_rule_32_amd as kda
    x = torch.full((4, 512), 3.0, dtype=torch.bfloat16)
    x[1] = 0.0
    _, w, b, dy = make(4, 512, 4)
    y = kda.layer_norm_forward(x.cuda(), w.cuda(), b.cuda())
    assert torch.equal(y.cpu(), b.bfloat16().expand(4, 512))
    check_backward(kda.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda()), dy, x, w, 1e-5)


@pytest.mark.parametrize("C", [256, 4096])
def test_slices_and_leading_dimensions(C):
    """A slice of wider rows, the rest of which is NaN; a NaN row stays in its row and the
    weights' gradients."""
    import gated_delta_rule_32_amd as kda
    x, w, b, dy = make(12, C, 5)
    wide = torch.full((3, 4, C + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[..., 8:8 + C] = x.reshape(3, 4, C).cuda()
    part = wide[..., 8:8 + C]
    y = kda.layer_norm_forward(part, w.cuda(), b.cuda())
    assert y.shape == (3, 4, C)
    check_forward(y.reshape(12, C), x, w, b, 1e-5)
    got = kda.layer_norm_backward(dy.reshape(3, 4, C).cuda(), part, w.cuda())
    check_backward((got[0].reshape(12, C), *got[1:]), dy, x, w, 1e-5)
    # every second row
    y = kda.layer_norm_forward(x.cuda()[::2], w.cuda(), b.cuda())
    check_forward(y, x[::2], w, b, 1e-5)
    bad = x.clone()
    bad[5, 3] = float("nan")
    y = kda.layer_norm_forward(bad.cuda(), w.cuda(), b.cuda())
    assert y[5].isnan().all() and not y[[i for i in range(12) if i != 5]].isnan().any()


def test_more_rows_than_workgroups():
    import gated_delta_rule_32_amd as kda
    for T, C in ((3001, 64), (1500, 1040)):
        x, w, b, dy = make(T, C, 6)
        check_forward(kda.layer_norm_forward(x.cuda(), w.cuda(), b.cuda()), x, w, b, 1e-5)
        check_backward(kda.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda()), dy, x, w, 1e-5)


def test_the_same_bits_again_and_captured():
    import gated_delta_rule_32_amd as kda
    x, w, b, dy = (t.cuda() for t in make(900, 1200, 7))
    p = kda.KdaLNormProblem(900, 1200, 1e-5, 0)
    ws = torch.empty(kda.kda_lnorm_bwd_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.layer_norm_forward(x, w, b, out=outs[0])
        kda.layer_norm_backward(dy, x, w, out=outs[1:], workspace=ws)
    for _ in range(3):
        for o in outs:
            o.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        want = [kda.layer_norm_forward(x, w, b), *kda.layer_norm_backward(dy, x, w)]
        torch.cuda.synchronize()
        for a, c in zip(outs, want):
            assert torch.equal(a, c)
        x.copy_(x.flip(0))


@pytest.mark.parametrize("C", [64, 2000])
def test_rows_behind_2_31_elements(C):
    import gated_delta_rule_32_amd as kda
    T, stride = 70, 1 << 25
    x, w, b, dy = make(T, C, 31)
    wide = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda").view(T, stride)[:, 8:8 + C]
    wide.copy_(x)
    args = [t.cuda() for t in (w, b, dy)]
    y, grads = kda.layer_norm_forward(wide, *args[:2]), kda.layer_norm_backward(args[2], wide, args[0])
    assert torch.equal(y, kda.layer_norm_forward(x.cuda(), *args[:2]))
    assert all(torch.equal(a, e) for a, e in zip(grads, kda.layer_norm_backward(args[2], x.cuda(), args[0])))
