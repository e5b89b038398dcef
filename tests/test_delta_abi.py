"""CPU tests of the gated delta rule, the drafts' verification and the layer norm:
host-side refusals of the C ABI (nothing is launched: the pointers are never
dereferenced), workspace sizes, the binding's argument checks, and the pins of their FP64
oracle."""
import ctypes
import math

import numpy as np
import pytest
import torch

import gated_delta_rule_32_amd as kda
from oracle import delta_oracle as do_

OK, NULL, SHAPE, GROUPING, SEQLENS, SCALE, OVERLAP, CTX_SIZE, WS, ROUTE = 0, 1, 2, 3, 4, 5, 7, 8, 10, 11
GAP = 1 << 36
BIG = 1 << 35


def ptrs(names):
    return {n: (i + 1) * GAP for i, n in enumerate(names.split())}


def delta(**kw):
    p = kda.KdaDeltaProblem()
    for k, v in dict(dict(B=1, T=40, Hqk=2, Hv=4, N=1), **kw).items():
        setattr(p, k, v)
    return p


def fwd(p, ws=90 * GAP, ws_bytes=BIG, **replace):
    a = ptrs("q k v g beta s0 o fs")
    a.update(replace)
    return kda._lib.kda_delta_fwd(ctypes.byref(p), *a.values(), ws, ws_bytes, None)


def bwd(p, ws=90 * GAP, ws_bytes=BIG, rec=None, rec_bytes=BIG, **replace):
    a = ptrs("q k v g beta s0 do ds dq dk dv dg db di")
    a.update(replace)
    a = list(a.values())
    return kda._lib.kda_delta_bwd(ctypes.byref(p), *a[:6], rec, rec_bytes, *a[6:], ws, ws_bytes, None)


def infer(p, slots=40, idx=None, spec=0, acc=None, ws=90 * GAP, ws_bytes=BIG, **replace):
    a = ptrs("q k v g beta pool")
    a["o"] = 7 * GAP
    a.update(replace)
    host = None if idx is None else (ctypes.c_int32 * len(idx))(*idx)
    o = a.pop("o")
    return kda._lib.kda_delta_infer(ctypes.byref(p), *a.values(), slots, None if idx is None else 8 * GAP, host, spec, acc, o,
                                    ws, ws_bytes, None)


def sizes(p):
    n = ctypes.c_size_t()
    out = [kda._lib.kda_delta_fwd_workspace_bytes(ctypes.byref(p), ctypes.byref(n)),
           kda._lib.kda_delta_bwd_workspace_bytes(ctypes.byref(p), 0, ctypes.byref(n))]
    out.append(kda._lib.kda_delta_infer_workspace_bytes(ctypes.byref(p), 0, ctypes.byref(n)))
    return out


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), SHAPE), (dict(T=0), SHAPE), (dict(N=2), SHAPE), (dict(Hv=3), GROUPING), (dict(scale=-1.0), SCALE),
    (dict(scale=math.inf), SCALE), (dict(scale=math.nan), SCALE), (dict(segment=-64), ROUTE), (dict(segment=65), ROUTE),
    (dict(q_stride=248), SHAPE), (dict(k_stride=260), SHAPE), (dict(v_stride=-512), SHAPE), (dict(use_qk_l2norm=2), SHAPE),
    (dict(use_qk_l2norm=-1), SHAPE), (dict(v_stride=1 << 26), SHAPE), (dict(Hqk=1 << 19, Hv=1 << 19), SHAPE),
    (dict(cu_seqlens=GAP), NULL)])
def test_refuses_problems(kw, status):
    for call in (fwd, bwd, infer):
        assert call(delta(**kw)) == status
    assert sizes(delta(**kw)) == [status] * 3


def test_refuses_sequences():
    for cu, status in (([1, 40], SEQLENS), ([0, 20, 20, 40], SEQLENS), ([0, 30, 20, 40], SEQLENS), ([0, 39], SEQLENS)):
        host = (ctypes.c_int64 * len(cu))(*cu)
        p = delta(N=len(cu) - 1, cu_seqlens=GAP, cu_seqlens_host=ctypes.addressof(host))
        assert fwd(p) == bwd(p) == infer(p) == status


def test_refuses_arguments():
    p = delta()
    for name in "q k v g beta o".split():
        assert fwd(p, **{name: None}) == NULL
    for name in "q k v g beta do dq dk dv dg db".split():
        assert bwd(p, **{name: None}) == NULL
    for name in "q k v g beta pool o".split():
        assert infer(p, **{name: None}) == NULL
    for name in "q k v s0 o fs".split():
        assert fwd(p, **{name: 20 * GAP + 8}) == SHAPE        # not 16-byte aligned
    for name in "q k v s0 do ds dq dk dv di".split():
        assert bwd(p, **{name: 20 * GAP + 8}) == SHAPE
    for name in "q k v pool o".split():
        assert infer(p, **{name: 20 * GAP + 8}) == SHAPE
    assert fwd(p, ws=None) == NULL and bwd(p, ws=None) == NULL and infer(p, ws=None) == NULL
    assert fwd(p, ws=90 * GAP + 4) == SHAPE
    n = ctypes.c_size_t()
    assert kda._lib.kda_delta_fwd_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == OK
    assert fwd(p, ws_bytes=n.value - 1) == WS
    for rec in (None, 80 * GAP):
        assert kda._lib.kda_delta_bwd_workspace_bytes(ctypes.byref(p), rec is not None, ctypes.byref(n)) == OK
        assert bwd(p, ws_bytes=n.value - 1, rec=rec) == WS
    assert bwd(p, rec=80 * GAP, rec_bytes=4 * 2 * 6144 - 1) == CTX_SIZE
    assert bwd(p, rec=80 * GAP + 8) == SHAPE


def test_refuses_overlaps():
    p = delta()
    assert fwd(p, o=GAP + 64) == OVERLAP                       # o over q
    assert fwd(p, o=4 * GAP) == OVERLAP                        # o over g
    assert fwd(p, fs=6 * GAP) == OVERLAP                       # final over initial state
    assert fwd(p, ws=5 * GAP) == OVERLAP                       # workspace over beta
    assert fwd(delta(v_stride=4096), o=3 * GAP + 39 * 8192) == OVERLAP   # o over v's last strided row
    assert bwd(p, dk=9 * GAP) == OVERLAP                       # dk over dq
    assert bwd(p, dq=7 * GAP) == OVERLAP                       # dq over do
    assert bwd(p, dg=13 * GAP) == OVERLAP                      # dg over dbeta
    assert bwd(p, di=8 * GAP) == OVERLAP                       # dinitial over dfinal
    assert bwd(p, rec=12 * GAP - 64) == OVERLAP                # records into dv's space
    assert bwd(p, rec=90 * GAP) == OVERLAP                     # records in the workspace
    assert infer(p, o=6 * GAP) == OVERLAP
    assert infer(delta(B=2, T=1, N=2), idx=[0, 1], o=8 * GAP) == OVERLAP


def test_refuses_slots():
    assert infer(delta(), slots=0) == SHAPE
    assert infer(delta(B=3, N=3), slots=2) == SHAPE            # slots for every sequence
    assert infer(delta(B=2, N=2), slots=4, idx=[0, 4]) == SHAPE
    assert infer(delta(B=2, N=2), idx=[0, -1]) == SHAPE
    assert infer(delta(B=2, N=2), idx=[3, 3]) == SHAPE


def test_refuses_drafted_tokens():
    p = delta(B=2, T=3, N=2)
    assert infer(p, spec=-1) == SHAPE
    assert infer(p, acc=20 * GAP) == SHAPE                     # accepted tokens without drafted ones
    assert infer(p, spec=2) == NULL                            # no slots
    assert infer(p, spec=3, idx=list(range(8))) == SEQLENS     # 3 tokens, not 4
    assert infer(p, spec=2, idx=[0, 1, 2, 3, 4, 2]) == SHAPE   # a slot twice
    assert infer(p, spec=2, idx=[0, 1, 2, 3, 4, 40]) == SHAPE
    assert infer(p, spec=2, idx=list(range(6)), acc=7 * GAP) == OVERLAP   # accepted tokens inside o
    n = ctypes.c_size_t()
    assert kda._lib.kda_delta_infer_workspace_bytes(ctypes.byref(p), -1, ctypes.byref(n)) == SHAPE


def test_refuses_more_than_a_launch():
    far = lambda names: {n: (i + 1) << 52 for i, n in enumerate(names.split())}  # noqa: E731
    p = delta(B=1 << 19, N=1 << 19, T=1, Hqk=64, Hv=64)
    assert fwd(p, ws=60 << 52, ws_bytes=1 << 60, **far("q k v g beta s0 o fs")) == SHAPE
    assert bwd(p, ws=60 << 52, ws_bytes=1 << 60, **far("q k v g beta s0 do ds dq dk dv dg db di")) == SHAPE
    p = delta(B=1 << 16, N=1 << 16, T=1, Hqk=64, Hv=64)
    assert infer(p, slots=1 << 16, **far("q k v g beta pool o")) == SHAPE


def test_workspace_sizes():
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731

    def need(name, p, *a):
        n = ctypes.c_size_t()
        assert getattr(kda._lib, f"kda_delta_{name}_workspace_bytes")(ctypes.byref(p), *a, ctypes.byref(n)) == OK
        return n.value
    p = delta(T=65, B=2, N=2)                                  # two blocks a sequence
    records = up(4 * 4 * 2 * 6144)
    assert need("fwd", p) >= records
    assert need("infer", p, 0) >= records
    assert need("infer", delta(T=4), 0) == 0                   # token by token
    assert need("infer", delta(T=40), 39) == 0
    assert need("bwd", p, 0) == records + need("bwd", p, 1) >= records + 2 * 4 * 4 * (32768 + 16384)
    cut = delta(T=65, B=2, N=2, segment=64)                    # two segments a sequence, two matrices each
    states = 4 * 4 * 65536
    assert need("fwd", cut) == need("infer", cut, 0) == need("fwd", p) + 2 * states
    assert need("bwd", cut, 1) == need("bwd", p, 1) + states
    assert need("bwd", cut, 0) == need("bwd", p, 0) + 3 * states
    assert need("fwd", delta(T=64, B=2, N=2, segment=64)) == need("fwd", delta(T=64, B=2, N=2))
    n = ctypes.c_size_t()
    assert kda._lib.kda_delta_fwd_workspace_bytes(ctypes.byref(p), None) == NULL
    assert kda._lib.kda_delta_bwd_workspace_bytes(ctypes.byref(p), 0, None) == NULL
    assert kda._lib.kda_delta_infer_workspace_bytes(None, 0, ctypes.byref(n)) == NULL


# ---------------------------------------------------------------------------
# verification
# ---------------------------------------------------------------------------
def verify(p, ws=90 * GAP, ws_bytes=BIG, **replace):
    a = ptrs("drafts lens target draft uniform tokens accepted")
    a.update(replace)
    return kda._lib.kda_verify(ctypes.byref(p), *a.values(), ws, ws_bytes, None)


@pytest.mark.parametrize("N,S,V,ts,ds", [
    (0, 1, 8, 0, 0), (1, -1, 8, 0, 0), (1, 4097, 8, 0, 0), (1, 1, 0, 0, 0), (1, 1, (1 << 30) + 1, 0, 0), (1, 1, 8, 7, 0),
    (1, 1, 8, 0, 7), (1, 1, 8, -8, 0), (1, 1, 8, (1 << 31) + 1, 0), (1 << 30, 4, 8, 0, 0), (1 << 24, 1, 8, 0, 0)])
def test_verify_refuses_problems(N, S, V, ts, ds):
    p = kda.KdaVerifyProblem(N, S, V, ts, ds)
    assert verify(p) == SHAPE
    n = ctypes.c_size_t()
    assert kda._lib.kda_verify_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == SHAPE


def test_verify_refuses_arguments():
    p = kda.KdaVerifyProblem(3, 2, 100)
    for name in "drafts target uniform tokens accepted".split():
        assert verify(p, **{name: None}) == NULL
    long = kda.KdaVerifyProblem(3, 2, 40000)                   # (the sums of ten tiles of each row)
    n = ctypes.c_size_t()
    for q, need in ((p, 0), (kda.KdaVerifyProblem(3, 2, 16384), 0), (long, 3 * 10 * 16)):
        assert kda._lib.kda_verify_workspace_bytes(ctypes.byref(q), ctypes.byref(n)) == OK and n.value == need
    assert verify(long, ws=None) == NULL
    assert verify(long, ws_bytes=3 * 10 * 16 - 1) == WS
    assert verify(long, ws=90 * GAP + 8) == SHAPE
    assert verify(long, ws=4 * GAP) == OVERLAP
    assert verify(p, tokens=GAP) == OVERLAP                    # tokens over the drafts
    assert verify(p, accepted=2 * GAP) == OVERLAP              # over draft_lens
    assert verify(p, tokens=3 * GAP + 8 * 400) == OVERLAP      # over target's last row
    assert verify(p, accepted=6 * GAP + 4) == OVERLAP          # over the tokens
    assert kda._lib.kda_verify_workspace_bytes(ctypes.byref(p), None) == NULL


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
def lnorm_fwd(p, **replace):
    a = ptrs("x w b y")
    a.update(replace)
    return kda._lib.kda_lnorm_fwd(ctypes.byref(p), *a.values(), None)


def lnorm_bwd(p, ws=90 * GAP, ws_bytes=BIG, **replace):
    a = ptrs("x w dy dx dw db")
    a.update(replace)
    return kda._lib.kda_lnorm_bwd(ctypes.byref(p), *a.values(), ws, ws_bytes, None)


@pytest.mark.parametrize("rows,C,eps,stride", [
    (0, 64, 1e-5, 0), (-1, 64, 1e-5, 0), (1 << 31, 64, 1e-5, 0), (4, 0, 1e-5, 0), (4, 60, 1e-5, 0), (4, 32776, 1e-5, 0),
    (4, 64, 0.0, 0), (4, 64, -1.0, 0), (4, 64, math.nan, 0), (4, 64, math.inf, 0), (4, 64, 1e-40, 0), (4, 64, 1e-5, 56),
    (4, 64, 1e-5, 68), (4, 64, 1e-5, -64), (4, 64, 1e-5, (1 << 40) + 8)])
def test_lnorm_refuses_problems(rows, C, eps, stride):
    p = kda.KdaLNormProblem(rows, C, eps, stride)
    assert lnorm_fwd(p) == SHAPE and lnorm_bwd(p) == SHAPE
    n = ctypes.c_size_t()
    assert kda._lib.kda_lnorm_bwd_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == SHAPE


def test_lnorm_refuses_arguments():
    p = kda.KdaLNormProblem(10, 64, 1e-5, 0)
    for name in "x w y".split():
        assert lnorm_fwd(p, **{name: None}) == NULL
    for name in "x w dy dx dw".split():
        assert lnorm_bwd(p, **{name: None}) == NULL
    for name in "x w b y".split():
        assert lnorm_fwd(p, **{name: 20 * GAP + 8}) == SHAPE
    for name in "x w dy dx".split():
        assert lnorm_bwd(p, **{name: 20 * GAP + 8}) == SHAPE
    assert lnorm_fwd(p, y=GAP) == OVERLAP
    assert lnorm_fwd(kda.KdaLNormProblem(10, 64, 1e-5, 128), y=GAP + 9 * 256) == OVERLAP
    assert lnorm_bwd(p, dx=3 * GAP) == OVERLAP
    assert lnorm_bwd(p, db=5 * GAP) == OVERLAP                 # dbias over dweight
    assert lnorm_bwd(p, ws=None) == NULL and lnorm_bwd(p, ws_bytes=16) == WS


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
def test_binding_refuses_cpu_tensors_and_wrong_types():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    q, v, g = bf(1, 4, 2, 128), bf(1, 4, 4, 128), bf(1, 4, 4)
    with pytest.raises(ValueError, match="GPU"):
        kda.gated_delta_rule_training_forward(q, q, v, g, g)
    with pytest.raises(ValueError, match="GPU"):
        kda.gated_delta_rule(q, q, v, g, g)
    with pytest.raises(ValueError, match="GPU"):
        kda.verify_drafts(torch.zeros((1, 1), dtype=torch.int32), torch.zeros((1, 2, 8)), torch.zeros((1, 2)))
    with pytest.raises(ValueError, match="1\\+S"):
        kda.verify_drafts(torch.zeros((1, 1), dtype=torch.int32), torch.zeros((2, 8)), torch.zeros((1, 2)))
    with pytest.raises(ValueError, match="GPU"):
        kda.layer_norm_forward(bf(4, 64), torch.ones(64))
    with pytest.raises(ValueError, match="bfloat16"):
        kda.layer_norm_forward(torch.zeros(4, 64), torch.ones(64))
    with pytest.raises(ValueError, match="context"):
        kda.gated_delta_rule_training_backward(None, v)


def test_everything_is_exported():
    for name in ("kda_delta_fwd", "kda_delta_bwd", "kda_delta_infer", "kda_verify", "kda_lnorm_fwd", "kda_lnorm_bwd"):
        assert name in kda.EXPORTED and callable(getattr(kda, name))


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------
def case(seed, lengths=(3, 5), Hqk=1, Hv=2):
    r = np.random.default_rng(seed)
    T, N = sum(lengths), len(lengths)
    return dict(q=r.standard_normal((1, T, Hqk, 128)), k=r.standard_normal((1, T, Hqk, 128)),
                v=r.standard_normal((1, T, Hv, 128)), g=-r.random((1, T, Hv)), beta=r.random((1, T, Hv)),
                state=0.3 * r.standard_normal((N, Hv, 128, 128))), list(lengths), r


@pytest.mark.parametrize("unit", [True, False])
def test_oracle_gradients_against_differences(unit):
    x, lengths, r = case(1)
    if not unit:
        x["k"] /= np.linalg.norm(x["k"], axis=-1, keepdims=True)
    do, ds = r.standard_normal(x["v"].shape), r.standard_normal(x["state"].shape)

    def loss(y):
        o, final, _, _ = do_.delta_forward(**y, lengths=lengths, packed=True, scale=0.1, unit=unit)
        return (do * o).sum() + (ds * final).sum()
    grads, _, _ = do_.delta_backward(**x, do=do, dfinal=ds, lengths=lengths, packed=True, scale=0.1, unit=unit)
    for name, grad in zip(("q", "k", "v", "g", "beta", "state"), grads):
        d = r.standard_normal(x[name].shape)
        h = 1e-5
        up, down = dict(x, **{name: x[name] + h * d}), dict(x, **{name: x[name] - h * d})
        got = (loss(up) - loss(down)) / (2 * h)
        want = (grad * d).sum()
        # third derivatives are of the size of the first: h^2 of them, and 1e-16 / h of the loss
        assert abs(got - want) <= 1e-7 * (np.abs(grad * d).sum() + abs(loss(x))), name


def test_oracle_closed_forms():
    """One token: S = e^g S0 + beta (v - e^g S0 k) k^T; beta 1 and a unit key make S k = v."""
    x, _, _ = case(2, lengths=(1,), Hv=1)
    x["beta"][:] = 1.0
    o, final, _, _ = do_.delta_forward(**x, lengths=[1], packed=False, scale=1.0, unit=True)
    k = x["k"][0, 0, 0] / np.sqrt((x["k"][0, 0, 0] ** 2).sum() + 1e-6)
    a = np.exp(x["g"][0, 0, 0])
    S = a * x["state"][0, 0]
    assert np.allclose(final[0, 0], S + np.outer(x["v"][0, 0, 0] - S @ k, k), atol=1e-12)
    assert np.allclose(final[0, 0] @ k, x["v"][0, 0, 0], atol=1e-6)   # |k|^2 is 1 - 1e-6 / |k|^2
    x["beta"][:] = 0.0
    _, final, _, _ = do_.delta_forward(**x, lengths=[1], packed=False, scale=1.0, unit=True)
    assert np.allclose(final[0, 0], S)


def test_oracle_weights_bound_their_sums():
    x, lengths, r = case(3, lengths=(20,), Hv=1)
    o, final, (wo, wfinal), _ = do_.delta_forward(**x, lengths=lengths, packed=False, scale=0.1, unit=True)
    assert (np.abs(o) <= wo * (1 + 1e-9)).all()
    assert (np.linalg.norm(final, axis=-1) <= wfinal * (1 + 1e-9)).all()
    do, ds = r.standard_normal(x["v"].shape), r.standard_normal(x["state"].shape)
    grads, weights, _ = do_.delta_backward(**x, do=do, dfinal=ds, lengths=lengths, packed=False, scale=0.1, unit=True)
    for got, w in zip(grads[2:5], weights[2:5]):
        assert (np.abs(got) <= w * (1 + 1e-9)).all()
    assert (np.linalg.norm(grads[5], axis=-1) <= weights[5] * (1 + 1e-9)).all()


def test_oracle_verification_keeps_the_targets_distribution():
    """Whatever the drafts are drawn from, the first token is distributed as the target:
    the mean over a fine grid of random numbers."""
    p, q = np.array([0.5, 0.3, 0.2, 0.0]), np.array([0.25, 0.25, 0.4, 0.1])
    m = 40
    u = (np.arange(m) + 0.5) / m
    mass = np.zeros(4)
    for x in range(4):
        uniform = np.stack(np.meshgrid(u, u, indexing="ij"), -1).reshape(-1, 2)
        n = len(uniform)
        tokens, _ = do_.verify(np.full((n, 1), x), None, np.tile(np.stack([p, p]), (n, 1, 1)), np.tile(q, (n, 1, 1)), uniform)
        mass += q[x] * np.bincount(tokens[:, 0], minlength=4) / n
    assert np.abs(mass - p).max() <= 2.0 / m


def test_oracle_layer_norm_gradients_against_differences():
    r = np.random.default_rng(4)
    x, w, b, dy, d = r.standard_normal((3, 16)), r.standard_normal(16), r.standard_normal(16), r.standard_normal((3, 16)), r.standard_normal((3, 16))
    dx, dw, db = do_.layer_norm_backward(dy, x, w, 1e-5)
    f = lambda x, w: (dy * do_.layer_norm(x, w, b, 1e-5)[0]).sum()  # noqa: E731
    h = 1e-6
    assert abs((f(x + h * d, w) - f(x - h * d, w)) / (2 * h) - (dx * d).sum()) <= 1e-7
    assert abs((f(x, w + h * d[0]) - f(x, w - h * d[0])) / (2 * h) - (dw * d[0]).sum()) <= 1e-7
    assert np.allclose(db, dy.sum(0))
