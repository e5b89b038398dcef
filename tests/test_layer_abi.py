"""CPU tests of the linear-attention layer operators: host-side refusals of the
C ABI (nothing is launched: the pointers are never dereferenced), workspace
sizes, the binding's argument checks, and the pins of their FP64 oracle."""
import ctypes
import math

import numpy as np
import pytest
import torch

import gated_delta_rule_32_amd as kda
from oracle import layer_oracle as lo

OK, NULL, SHAPE, GROUPING, SEQLENS, SCALE, OVERLAP, WS, ROUTE = 0, 1, 2, 3, 4, 5, 7, 10, 11
GAP = 1 << 32


def ptrs(n):
    return [(i + 1) * GAP for i in range(n)]


def decay(**kw):
    p = kda.KdaDecayProblem()
    for k, v in dict(dict(B=1, T=40, Hqk=2, Hv=4, N=1), **kw).items():
        setattr(p, k, v)
    return p


def fwd(p, ws=0, ws_bytes=0, **replace):
    a = dict(zip("q k v l s0 o fs".split(), ptrs(7)))
    a.update(replace)
    return kda._lib.kda_decay_fwd(ctypes.byref(p), *a.values(), ws, ws_bytes, None)


def bwd(p, ws=90 * GAP, ws_bytes=1 << 40, **replace):
    a = dict(zip("q k v l s0 do ds dq dk dv di".split(), ptrs(11)))
    a.update(replace)
    return kda._lib.kda_decay_bwd(ctypes.byref(p), *a.values(), ws, ws_bytes, None)


def infer(p, slots=4, idx=None, ws=0, **replace):
    a = dict(zip("q k v l pool".split(), ptrs(5)))
    a["o"] = 6 * GAP
    a.update(replace)
    host = None if idx is None else (ctypes.c_int32 * len(idx))(*idx)
    return kda._lib.kda_decay_infer(ctypes.byref(p), a["q"], a["k"], a["v"], a["l"], a["pool"], slots,
                                    None if idx is None else 8 * GAP, host, a["o"], ws, 0, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), SHAPE), (dict(T=0), SHAPE), (dict(N=2), SHAPE), (dict(Hv=3), GROUPING), (dict(scale=-1.0), SCALE),
    (dict(scale=math.inf), SCALE), (dict(scale=math.nan), SCALE), (dict(segment=-64), ROUTE), (dict(segment=65), ROUTE),
    (dict(q_stride=248), SHAPE), (dict(k_stride=260), SHAPE), (dict(v_stride=-512), SHAPE),
    (dict(v_stride=1 << 26), SHAPE), (dict(Hqk=1 << 19, Hv=1 << 19), SHAPE), (dict(cu_seqlens=GAP), NULL)])
def test_decay_refuses_problems(kw, status):
    for call in (fwd, bwd, infer):
        assert call(decay(**kw)) == status
    n = ctypes.c_size_t()
    for name in ("fwd", "bwd", "infer"):
        assert getattr(kda._lib, f"kda_decay_{name}_workspace_bytes")(ctypes.byref(decay(**kw)), ctypes.byref(n)) == status


def test_decay_refuses_sequences():
    for cu, status in (([1, 40], SEQLENS), ([0, 20, 20, 40], SEQLENS), ([0, 30, 20, 40], SEQLENS), ([0, 39], SEQLENS)):
        host = (ctypes.c_int64 * len(cu))(*cu)
        p = decay(N=len(cu) - 1, cu_seqlens=GAP, cu_seqlens_host=ctypes.addressof(host))
        assert fwd(p) == status
    host = (ctypes.c_int64 * 2)(0, 40)
    assert fwd(decay(B=2, cu_seqlens=GAP, cu_seqlens_host=ctypes.addressof(host))) == SHAPE


def test_decay_refuses_arguments():
    p = decay()
    for name in "q k v l o".split():
        assert fwd(p, **{name: None}) == NULL
    for name in "q k v l do dq dk dv".split():
        assert bwd(p, **{name: None}) == NULL
    for name in "q k v l pool o".split():
        assert infer(p, **{name: None}) == NULL
    for name in "q k v s0 o fs".split():
        assert fwd(p, **{name: 20 * GAP + 8}) == SHAPE        # not 16-byte aligned
    for name in "q k v s0 do ds dq dk dv di".split():
        assert bwd(p, **{name: 20 * GAP + 8}) == SHAPE
    assert fwd(p, o=GAP + 64) == OVERLAP                       # o over q
    assert fwd(p, fs=5 * GAP) == OVERLAP                       # final over initial state
    assert fwd(decay(v_stride=4096), o=3 * GAP + 39 * 8192) == OVERLAP   # o over v's last strided row
    assert bwd(p, dk=8 * GAP) == OVERLAP                       # dk over dq
    assert bwd(p, dq=6 * GAP) == OVERLAP                       # dq over do
    assert infer(p, o=5 * GAP) == OVERLAP
    assert infer(p, slots=0) == SHAPE
    assert infer(decay(B=3, N=3), slots=2) == SHAPE            # slots for every sequence
    assert infer(decay(B=2, N=2), idx=[0, 4]) == SHAPE
    assert infer(decay(B=2, N=2), idx=[0, -1]) == SHAPE
    assert infer(decay(B=2, N=2), idx=[3, 3]) == SHAPE


def test_decay_refuses_more_than_a_launch():
    """2^24 workgroups of 256 threads are more than one launch holds."""
    far = lambda names: {n: (i + 1) << 46 for i, n in enumerate(names.split())}  # noqa: E731
    p = decay(B=1 << 18, N=1 << 18, T=1, Hqk=64, Hv=64)
    assert fwd(p, **far("q k v l s0 o fs")) == SHAPE
    assert bwd(p, **far("q k v l s0 do ds dq dk dv di")) == SHAPE
    p = decay(B=1 << 16, N=1 << 16, T=1, Hqk=64, Hv=64)
    assert infer(p, slots=1 << 16, **far("q k v l pool o")) == SHAPE


def test_decay_workspace_sizes():
    state = 128 * 128 * 4
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    # whole sequences, no shared heads: nothing
    p = decay(Hqk=4, segment=64, T=64)
    assert kda.kda_decay_fwd_workspace_bytes(p) == 0 and kda.kda_decay_bwd_workspace_bytes(p) == 0
    # shared heads: partials of dq and dk, 2 bytes a value
    p = decay(segment=64, T=64)
    assert kda.kda_decay_bwd_workspace_bytes(p) == 2 * up(64 * 4 * 128 * 2)
    # segments: a state each, both ways in the backward
    p = decay(segment=64, T=200)
    assert kda.kda_decay_fwd_workspace_bytes(p) == 4 * 4 * state
    assert kda.kda_decay_bwd_workspace_bytes(p) == 2 * 4 * 4 * state + 2 * up(200 * 4 * 128 * 2)
    assert kda.kda_decay_infer_workspace_bytes(p) == 4 * 4 * state
    assert fwd(p) == NULL
    assert fwd(p, ws=90 * GAP, ws_bytes=4 * 4 * state - 1) == WS
    assert bwd(p, ws_bytes=100) == WS
    assert fwd(p, ws=90 * GAP + 4, ws_bytes=1 << 30) == SHAPE
    assert fwd(p, ws=GAP, ws_bytes=1 << 30) == OVERLAP
    # a few tokens run token by token
    assert kda.kda_decay_infer_workspace_bytes(decay(T=8)) == 0


def qk(**kw):
    p = kda.KdaQkNormProblem()
    for k, v in dict(dict(B=1, T=10, Hq=4, Hk=2, rot_dim=64, eps=1e-6, table_rows=100), **kw).items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), SHAPE), (dict(T=0), SHAPE), (dict(Hq=0), SHAPE), (dict(Hk=0), SHAPE), (dict(rot_dim=0), SHAPE),
    (dict(rot_dim=4), SHAPE), (dict(rot_dim=136), SHAPE), (dict(rot_dim=60), SHAPE), (dict(interleaved=2), SHAPE),
    (dict(eps=0.0), SHAPE), (dict(eps=math.nan), SHAPE), (dict(table_rows=0), SHAPE), (dict(q_stride=504), SHAPE),
    (dict(k_stride=258), SHAPE), (dict(Hq=1 << 30, Hk=1 << 30), SHAPE)])
def test_qknorm_refuses_problems(kw, status):
    a = ptrs(16)
    assert kda._lib.kda_qknorm_fwd(ctypes.byref(qk(**kw)), *a[:9], None) == status
    assert kda._lib.kda_qknorm_bwd(ctypes.byref(qk(**kw)), *a[:13], a[13], 1 << 30, None) == status


def test_qknorm_refuses_arguments():
    a, b = ptrs(9), ptrs(14)
    for i in (0, 1, 2, 3, 4, 5, 7, 8):
        assert kda._lib.kda_qknorm_fwd(ctypes.byref(qk()), *a[:i], None, *a[i + 1:], None) == NULL
    for i in (0, 1, 2, 3, 4, 5, 7, 8, 9, 10, 11, 12, 13):
        assert kda._lib.kda_qknorm_bwd(ctypes.byref(qk()), *b[:i], None, *b[i + 1:], 1 << 30, None) == NULL
    for i in (0, 1, 4, 5, 7, 8):
        assert kda._lib.kda_qknorm_fwd(ctypes.byref(qk()), *a[:i], 50 * GAP + 8, *a[i + 1:], None) == SHAPE
    assert kda._lib.kda_qknorm_fwd(ctypes.byref(qk(table_rows=9)), *a[:6], None, *a[7:], None) == SHAPE
    assert kda._lib.kda_qknorm_fwd(ctypes.byref(qk()), *a[:7], a[0], a[8], None) == OVERLAP     # in place
    assert kda._lib.kda_qknorm_bwd(ctypes.byref(qk()), *b, 16, None) == WS
    need = kda.kda_qknorm_bwd_workspace_bytes(qk())
    assert need == 4 * 2 * 128 * 4     # 60 rows, 16 to a workgroup
    assert kda.kda_qknorm_bwd_workspace_bytes(qk(T=1 << 20)) == 1024 * 2 * 128 * 4


def gn(**kw):
    p = kda.KdaGNormProblem()
    for k, v in dict(dict(B=1, T=10, H=4, eps=1e-6), **kw).items():
        setattr(p, k, v)
    return p


def test_gnorm_refusals():
    a, b = ptrs(4), ptrs(8)
    for kw in (dict(B=0), dict(T=0), dict(H=0), dict(activation=2), dict(eps=-1.0), dict(x_stride=500),
               dict(gate_stride=516)):
        assert kda._lib.kda_gnorm_fwd(ctypes.byref(gn(**kw)), *a, None) == SHAPE
        assert kda._lib.kda_gnorm_bwd(ctypes.byref(gn(**kw)), *b, 1 << 30, None) == SHAPE
    for i in range(4):
        assert kda._lib.kda_gnorm_fwd(ctypes.byref(gn()), *a[:i], None, *a[i + 1:], None) == NULL
    for i in range(8):
        assert kda._lib.kda_gnorm_bwd(ctypes.byref(gn()), *b[:i], None, *b[i + 1:], 1 << 30, None) == NULL
    assert kda._lib.kda_gnorm_fwd(ctypes.byref(gn()), *a[:3], a[0], None) == OVERLAP
    assert kda._lib.kda_gnorm_fwd(ctypes.byref(gn()), *a[:3], 50 * GAP + 2, None) == SHAPE
    assert kda._lib.kda_gnorm_bwd(ctypes.byref(gn()), *b, 16, None) == WS


def test_binding_refuses_tensors():
    x = torch.zeros((1, 4, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        kda.decay_attention(x, x, x, torch.zeros(2))
    with pytest.raises(ValueError, match="B, T, H, 128"):
        kda.gated_norm_forward(x[0], x, torch.ones(128))
    layers = kda._layers
    cpu = torch.device("cpu")
    wide = torch.zeros((2, 4, 6, 128), dtype=torch.bfloat16)
    assert layers._rows("x", wide[:, :, 1:3], (2, 4, 2, 128), cpu) == 6 * 128
    assert layers._rows("x", wide[:, :1, 1:3].contiguous()[:, :, :1], (2, 1, 1, 128), cpu) == 2 * 128
    assert layers._rows("x", wide[:, :1, 1:3], (2, 1, 2, 128), cpu) == 4 * 6 * 128   # batch rows as tokens
    assert layers._rows("x", wide[1:, 2:3], (1, 1, 6, 128), cpu) == 6 * 128
    for bad in (wide[:, :3], wide[..., ::2, :][:, :, :2], wide.transpose(1, 2)):
        with pytest.raises(ValueError):
            layers._rows("x", bad, tuple(bad.shape), cpu)
    with pytest.raises(ValueError, match="bfloat16"):
        layers._rows("x", wide.float(), (2, 4, 6, 128), cpu)


def test_binding_refuses_expanded_rows():
    """A token stride of 0 must not reach the library, where it means dense rows."""
    one = torch.zeros((1, 1, 2, 128), dtype=torch.bfloat16)
    long = torch.zeros(4000, dtype=torch.bfloat16)
    for x in (one.expand(1, 5, 2, 128), one.expand(5, 1, 2, 128), one.expand(3, 5, 2, 128),
              long.as_strided((1, 5, 2, 128), (640, 128, 128, 1))):
        with pytest.raises(ValueError, match="token"):
            kda._layers._rows("x", x, tuple(x.shape), torch.device("cpu"))


def test_rotary_table():
    cos, sin = kda.rotary_table(100000, 64, theta=500000.0, device="cpu")
    assert cos.shape == sin.shape == (100000, 32) and cos.dtype == torch.float32
    for pos, i in ((0, 0), (1, 0), (99999, 0), (99999, 31), (54321, 7)):
        angle = pos * 500000.0 ** (-2 * i / 64)
        assert float(cos[pos, i]) == pytest.approx(math.cos(angle), abs=2.0 ** -24)
        assert float(sin[pos, i]) == pytest.approx(math.sin(angle), abs=2.0 ** -24)


# ---------------------------------------------------------------------------
# pins of the oracle
# ---------------------------------------------------------------------------
def test_oracle_decay_closed_form():
    """o_t = scale sum_j e^{l(t-j)} (q_t.k_j) v_j + scale e^{l(t+1)} S_0 q_t."""
    r = np.random.RandomState(0)
    q, k, v = (r.randn(1, 9, h, 128) for h in (1, 1, 2))
    s0, l = r.randn(2, 2, 128, 128), np.array([-0.3, 0.0])
    o, final, _, _ = lo.decay_forward(q, k, v, l, s0, [4, 5], True, 0.1)
    for n, (t0, L) in enumerate(((0, 4), (4, 5))):
        for h in range(2):
            for t in range(L):
                want = math.exp(l[h] * (t + 1)) * s0[n, h] @ q[0, t0 + t, 0]
                for j in range(t + 1):
                    want = want + math.exp(l[h] * (t - j)) * (q[0, t0 + t, 0] @ k[0, t0 + j, 0]) * v[0, t0 + j, h]
                np.testing.assert_allclose(o[0, t0 + t, h], 0.1 * want, rtol=1e-12, atol=1e-12)


def _difference(f, x, dx, eps=1e-6):
    return (f(x + eps * dx) - f(x - eps * dx)) / (2 * eps)


def test_oracle_decay_gradients_by_differences():
    r = np.random.RandomState(1)
    x = dict(q=r.randn(1, 7, 1, 128), k=r.randn(1, 7, 1, 128), v=r.randn(1, 7, 2, 128), s0=r.randn(2, 2, 128, 128))
    l, do, ds = np.array([-0.2, -1.0]), r.randn(1, 7, 2, 128), r.randn(2, 2, 128, 128)

    def loss(y):
        o, final, _, _ = lo.decay_forward(y["q"], y["k"], y["v"], l, y["s0"], [3, 4], True, 0.3)
        return (o * do).sum() + (final * ds).sum()

    grads = dict(zip(("q", "k", "v", "s0"),
                     lo.decay_backward(x["q"], x["k"], x["v"], l, x["s0"], do, ds, [3, 4], True, 0.3)))
    for name in x:
        d = r.randn(*x[name].shape)
        got = _difference(lambda y: loss(dict(x, **{name: y})), x[name], d)
        assert got == pytest.approx((grads[name] * d).sum(), rel=1e-6)


@pytest.mark.parametrize("pairs", [False, True])
def test_oracle_qk_norm_rope_gradients_by_differences(pairs):
    r = np.random.RandomState(2)
    x, w, dy = r.randn(2, 3, 2, 128), r.randn(128), r.randn(2, 3, 2, 128)
    angle = r.rand(10, 16) * 6
    cos, sin, pos = np.cos(angle), np.sin(angle), r.randint(10, size=(2, 3))
    f = lambda a, b: (lo.qk_norm_rope(a, b, cos, sin, pos, 32, pairs, 1e-3) * dy).sum()  # noqa: E731
    dx, dw = lo.qk_norm_rope_backward(dy, x, w, cos, sin, pos, 32, pairs, 1e-3)
    d, e = r.randn(*x.shape), r.randn(128)
    assert _difference(lambda a: f(a, w), x, d) == pytest.approx((dx * d).sum(), rel=1e-6)
    assert _difference(lambda b: f(x, b), w, e) == pytest.approx((dw * e).sum(), rel=1e-6)
    # a rotation keeps each pair's length
    n = lo.qk_norm_rope(x, w, np.ones_like(cos), np.zeros_like(cos), pos, 32, pairs, 1e-3)
    y = lo.qk_norm_rope(x, w, cos, sin, pos, 32, pairs, 1e-3)
    u, v = (slice(0, 32, 2), slice(1, 32, 2)) if pairs else (slice(0, 16), slice(16, 32))
    np.testing.assert_allclose(y[..., u] ** 2 + y[..., v] ** 2, n[..., u] ** 2 + n[..., v] ** 2, rtol=1e-12)
    np.testing.assert_array_equal(y[..., 32:], n[..., 32:])


@pytest.mark.parametrize("silu", [False, True])
def test_oracle_gated_norm_gradients_by_differences(silu):
    r = np.random.RandomState(3)
    a = [r.randn(1, 3, 2, 128), r.randn(1, 3, 2, 128) * 3, r.randn(128)]
    dy = r.randn(1, 3, 2, 128)
    grads = lo.gated_norm_backward(dy, *a, silu, 1e-3)
    for i in range(3):
        d = r.randn(*a[i].shape)
        f = lambda y: (lo.gated_norm(*[y if j == i else a[j] for j in range(3)], silu, 1e-3) * dy).sum()  # noqa: E731
        assert _difference(f, a[i], d) == pytest.approx((grads[i] * d).sum(), rel=1e-6)


def test_package_imports_with_a_torch_without_gpu_support():
    """The package's host-only calls need nothing of torch's GPU bindings, which
    such a build lacks."""
    import subprocess
    import sys
    code = ("import torch\n"
            "del torch._C._cuda_getCurrentRawStream\n"
            "import gated_delta_rule_32_amd as kda\n"
            "assert kda.kda_version() > 0 and kda.kda_gnorm_bwd_workspace_bytes(kda.KdaGNormProblem(1, 1, 1, 0, 1e-6)) > 0\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("eps,status", [(1e-40, SHAPE), (1.1e-38, SHAPE), (2.0 ** -126, OK), (1e-30, OK)])
def test_row_norms_refuse_an_eps_below_the_normal_numbers(eps, status):
    """The kernels would take it for 0, and turn a row of zeros into NaN."""
    n = ctypes.c_size_t()
    assert kda._lib.kda_qknorm_bwd_workspace_bytes(ctypes.byref(qk(eps=eps)), ctypes.byref(n)) == status
    assert kda._lib.kda_gnorm_bwd_workspace_bytes(ctypes.byref(gn(eps=eps)), ctypes.byref(n)) == status
    if status != OK:
        a, b = ptrs(14), ptrs(8)
        assert kda._lib.kda_qknorm_fwd(ctypes.byref(qk(eps=eps)), *a[:9], None) == status
        assert kda._lib.kda_gnorm_fwd(ctypes.byref(gn(eps=eps)), *b[:4], None) == status
