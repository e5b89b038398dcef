"""Python binding of libkda's linear-attention layer operators: linear
attention with a constant decay per head (training forward and backward,
decode and prefill), the query/key norm with rotary rotation in front of it,
the gated norm of the heads' outputs behind it, and the layer norm of token rows.

Argument marshalling only, as in the package itself: the low-level functions
carry the C names (include/libkda.h), the others take and return tensors.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

from . import HEAD_DIM, _check, _lib, _ptr, _require

GATE_SIGMOID, GATE_SILU = 0, 1
_ACTIVATIONS = {"sigmoid": GATE_SIGMOID, "silu": GATE_SILU}
_BF, _F32 = torch.bfloat16, torch.float32
_vp = ctypes.c_void_p
_size = ctypes.c_size_t
_byref = ctypes.byref
# (a torch built without GPU support has none; it makes no GPU tensors either)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class KdaDecayProblem(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("Hqk", ctypes.c_int32),
        ("Hv", ctypes.c_int32), ("N", ctypes.c_int32),
        ("cu_seqlens", _vp), ("cu_seqlens_host", _vp),
        ("scale", ctypes.c_float), ("segment", ctypes.c_int32),
        ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
    ]


class KdaQkNormProblem(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hk", ctypes.c_int32),
        ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float),
        ("table_rows", ctypes.c_int64), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
    ]


class KdaGNormProblem(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
        ("activation", ctypes.c_int32), ("eps", ctypes.c_float),
        ("x_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64),
    ]


class KdaLNormProblem(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("C", ctypes.c_int32), ("eps", ctypes.c_float), ("x_stride", ctypes.c_int64),
    ]


def _declare(name, problem, *args):
    f = getattr(_lib, name)
    f.restype = ctypes.c_int
    f.argtypes = [ctypes.POINTER(problem), *args]


for _name in ("kda_decay_fwd_workspace_bytes", "kda_decay_bwd_workspace_bytes", "kda_decay_infer_workspace_bytes"):
    _declare(_name, KdaDecayProblem, ctypes.POINTER(_size))
_declare("kda_decay_fwd", KdaDecayProblem, *[_vp] * 8, _size, _vp)
_declare("kda_decay_bwd", KdaDecayProblem, *[_vp] * 12, _size, _vp)
_declare("kda_decay_infer", KdaDecayProblem, *[_vp] * 5, ctypes.c_int64, *[_vp] * 4, _size, _vp)
_declare("kda_qknorm_fwd", KdaQkNormProblem, *[_vp] * 10)
_declare("kda_qknorm_bwd_workspace_bytes", KdaQkNormProblem, ctypes.POINTER(_size))
_declare("kda_qknorm_bwd", KdaQkNormProblem, *[_vp] * 14, _size, _vp)
_declare("kda_gnorm_fwd", KdaGNormProblem, *[_vp] * 5)
_declare("kda_gnorm_bwd_workspace_bytes", KdaGNormProblem, ctypes.POINTER(_size))
_declare("kda_gnorm_bwd", KdaGNormProblem, *[_vp] * 8, _size, _vp)
_declare("kda_lnorm_fwd", KdaLNormProblem, *[_vp] * 5)
_declare("kda_lnorm_bwd_workspace_bytes", KdaLNormProblem, ctypes.POINTER(_size))
_declare("kda_lnorm_bwd", KdaLNormProblem, *[_vp] * 7, _size, _vp)

EXPORTED = ("kda_decay_fwd_workspace_bytes", "kda_decay_bwd_workspace_bytes", "kda_decay_infer_workspace_bytes",
            "kda_decay_fwd", "kda_decay_bwd", "kda_decay_infer", "kda_qknorm_fwd",
            "kda_qknorm_bwd_workspace_bytes", "kda_qknorm_bwd", "kda_gnorm_fwd",
            "kda_gnorm_bwd_workspace_bytes", "kda_gnorm_bwd", "kda_lnorm_fwd", "kda_lnorm_bwd_workspace_bytes",
            "kda_lnorm_bwd")


# ---------------------------------------------------------------------------
# C names
# ---------------------------------------------------------------------------
def _bytes(name, p) -> int:
    n = _size(0)
    _check(getattr(_lib, name)(ctypes.byref(p), ctypes.byref(n)))
    return int(n.value)


def kda_decay_fwd_workspace_bytes(p: KdaDecayProblem) -> int:
    return _bytes("kda_decay_fwd_workspace_bytes", p)


def kda_decay_bwd_workspace_bytes(p: KdaDecayProblem) -> int:
    return _bytes("kda_decay_bwd_workspace_bytes", p)


def kda_decay_infer_workspace_bytes(p: KdaDecayProblem) -> int:
    return _bytes("kda_decay_infer_workspace_bytes", p)


def kda_qknorm_bwd_workspace_bytes(p: KdaQkNormProblem) -> int:
    return _bytes("kda_qknorm_bwd_workspace_bytes", p)


def kda_gnorm_bwd_workspace_bytes(p: KdaGNormProblem) -> int:
    return _bytes("kda_gnorm_bwd_workspace_bytes", p)


def kda_lnorm_bwd_workspace_bytes(p: KdaLNormProblem) -> int:
    return _bytes("kda_lnorm_bwd_workspace_bytes", p)


def _ws(t: Optional[torch.Tensor]):
    return (None, 0) if t is None else (t.data_ptr(), t.numel() * t.element_size())


def _call(f, stream, t, *args) -> None:
    """f(*args, stream), by default on the current stream of t's device, which is
    the current one for the call."""
    i = t.get_device()
    _require(i >= 0, "tensors must be on a GPU")
    if stream is None:
        stream = _raw_stream(i)  # (current_stream builds an object: 2 us)
    if i == torch.cuda.current_device():
        _check(f(*args, stream))
    else:
        with torch.cuda.device(i):
            _check(f(*args, stream))


def kda_decay_fwd(p: KdaDecayProblem, q, k, v, log_decay, initial_state, o, final_state,
                  workspace: Optional[torch.Tensor] = None, stream: Optional[int] = None) -> None:
    """C kda_decay_fwd on torch tensors (no shape checks beyond the library's)."""
    _call(_lib.kda_decay_fwd, stream, q, _byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(initial_state),
          _ptr(o), _ptr(final_state), *_ws(workspace))


def kda_decay_bwd(p: KdaDecayProblem, q, k, v, log_decay, initial_state, d_o, dfinal_state, dq, dk, dv,
                  dinitial_state, workspace: Optional[torch.Tensor] = None, stream: Optional[int] = None) -> None:
    """C kda_decay_bwd on torch tensors."""
    _call(_lib.kda_decay_bwd, stream, q, _byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(initial_state),
          _ptr(d_o), _ptr(dfinal_state), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dinitial_state), *_ws(workspace))


def kda_decay_infer(p: KdaDecayProblem, q, k, v, log_decay, state_pool, state_indices, state_indices_cpu, o,
                    workspace: Optional[torch.Tensor] = None, stream: Optional[int] = None) -> None:
    """C kda_decay_infer on torch tensors."""
    _call(_lib.kda_decay_infer, stream, q, _byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(state_pool),
          state_pool.shape[0], _ptr(state_indices), _ptr(state_indices_cpu), _ptr(o), *_ws(workspace))


def kda_qknorm_fwd(p: KdaQkNormProblem, q, k, q_weight, k_weight, cos, sin, positions, q_out, k_out,
                   stream: Optional[int] = None) -> None:
    """C kda_qknorm_fwd on torch tensors."""
    _call(_lib.kda_qknorm_fwd, stream, q, _byref(p), _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(cos),
          _ptr(sin), _ptr(positions), _ptr(q_out), _ptr(k_out))


def kda_qknorm_bwd(p: KdaQkNormProblem, q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out, dq, dk,
                   dq_weight, dk_weight, workspace: torch.Tensor, stream: Optional[int] = None) -> None:
    """C kda_qknorm_bwd on torch tensors."""
    _call(_lib.kda_qknorm_bwd, stream, q, _byref(p), _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(cos),
          _ptr(sin), _ptr(positions), _ptr(dq_out), _ptr(dk_out), _ptr(dq), _ptr(dk), _ptr(dq_weight),
          _ptr(dk_weight), *_ws(workspace))


def kda_gnorm_fwd(p: KdaGNormProblem, x, gate, weight, y, stream: Optional[int] = None) -> None:
    """C kda_gnorm_fwd on torch tensors."""
    _call(_lib.kda_gnorm_fwd, stream, x, _byref(p), _ptr(x), _ptr(gate), _ptr(weight), _ptr(y))


def kda_gnorm_bwd(p: KdaGNormProblem, x, gate, weight, dy, dx, dgate, dweight, workspace: torch.Tensor,
                  stream: Optional[int] = None) -> None:
    """C kda_gnorm_bwd on torch tensors."""
    _call(_lib.kda_gnorm_bwd, stream, x, _byref(p), _ptr(x), _ptr(gate), _ptr(weight), _ptr(dy), _ptr(dx),
          _ptr(dgate), _ptr(dweight), *_ws(workspace))


def kda_lnorm_fwd(p: KdaLNormProblem, x, weight, bias, y, stream: Optional[int] = None) -> None:
    """C kda_lnorm_fwd on torch tensors."""
    _call(_lib.kda_lnorm_fwd, stream, x, _byref(p), _ptr(x), _ptr(weight), _ptr(bias), _ptr(y))


def kda_lnorm_bwd(p: KdaLNormProblem, x, weight, dy, dx, dweight, dbias, workspace: torch.Tensor,
                  stream: Optional[int] = None) -> None:
    """C kda_lnorm_bwd on torch tensors."""
    _call(_lib.kda_lnorm_bwd, stream, x, _byref(p), _ptr(x), _ptr(weight), _ptr(dy), _ptr(dx), _ptr(dweight),
          _ptr(dbias), *_ws(workspace))


# ---------------------------------------------------------------------------
# argument checks
# ---------------------------------------------------------------------------
def _dense(name, t, dtype, shape, device):
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        _require(isinstance(t, torch.Tensor), f"{name} must be a tensor")
        _require(t.dtype == dtype, f"{name} must be {dtype}, got {t.dtype}")
        _require(t.shape == shape, f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        _require(t.device == device, f"{name} must be on {device}, got {t.device}")
        _require(False, f"{name} must be contiguous")


def _rows(name, t, shape, device) -> int:
    """The token stride of a BF16 [B, T, H, 128] operand: dense, or a slice of
    wider token rows."""
    if not (isinstance(t, torch.Tensor) and t.dtype is _BF and t.shape == shape and t.device == device):
        _require(isinstance(t, torch.Tensor) and t.dtype is _BF, f"{name} must be a bfloat16 tensor")
        _require(t.shape == shape, f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        _require(False, f"{name} must be on {device}, got {t.device}")
    B, T, H, D = shape
    if t.is_contiguous():
        return H * D
    sb, st, sh, sd = t.stride()
    _require(sd == 1 and (H == 1 or sh == D), f"{name} must have dense heads and channels")
    if T == 1:  # the token stride is free; the rows are the batch's
        st = sb if B > 1 else H * D
    _require(B == 1 or sb == T * st, f"{name}'s batch rows must be T token strides apart")
    # (0, an expanded tensor's, would mean dense rows to the library)
    _require(st >= H * D, f"{name}'s token rows must not overlap")
    return st


def _cuda(t) -> torch.device:
    if not (isinstance(t, torch.Tensor) and t.dim() == 4 and t.is_cuda):
        _require(isinstance(t, torch.Tensor) and t.dim() == 4, "token tensors must be [B, T, H, 128]")
        _require(False, f"tensors must be on a GPU, got {t.device}")
    return t.device


def _new(t: torch.Tensor) -> torch.Tensor:
    """A dense tensor of t's shape and type."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _decay_problem(q, k, v, log_decay, scale, cu_seqlens, cu_seqlens_cpu, segment) -> KdaDecayProblem:
    dev = _cuda(q)
    _cuda(v)
    B, T, Hqk, _ = q.shape
    Hv = v.shape[2]
    qk = (B, T, Hqk, HEAD_DIM)
    p = KdaDecayProblem(B, T, Hqk, Hv, B, None, None, 0.0, 0, _rows("q", q, qk, dev), _rows("k", k, qk, dev),
                        _rows("v", v, (B, T, Hv, HEAD_DIM), dev))
    _dense("log_decay", log_decay, _F32, (Hv,), dev)
    if cu_seqlens is not None:
        _require(cu_seqlens_cpu is not None, "packed calls need cu_seqlens_cpu")
        _require(cu_seqlens.dtype == torch.int64 and cu_seqlens_cpu.dtype == torch.int64, "cu_seqlens must be int64")
        _require(cu_seqlens.is_contiguous() and cu_seqlens.device == dev,
                 "cu_seqlens must be contiguous on the device of q")
        _require(cu_seqlens_cpu.device.type == "cpu" and cu_seqlens_cpu.is_contiguous(),
                 "cu_seqlens_cpu must be a contiguous CPU tensor")
        _require(cu_seqlens.dim() == 1 and cu_seqlens.shape == cu_seqlens_cpu.shape and cu_seqlens.numel() >= 2,
                 "cu_seqlens and cu_seqlens_cpu must be [N+1]")
        p.N = cu_seqlens.numel() - 1
        p.cu_seqlens = cu_seqlens.data_ptr()
        p.cu_seqlens_host = cu_seqlens_cpu.data_ptr()
        # the struct holds raw pointers: keep the tensors alive with it
        p._keep = (cu_seqlens, cu_seqlens_cpu)
    else:
        _require(cu_seqlens_cpu is None, "cu_seqlens_cpu must be omitted for fixed layout")
    if scale is not None:
        p.scale = float(scale)
        if not p.scale > 0.0:
            _require(False, f"scale must be positive, got {scale}")
    if segment != 0:
        p.segment = int(segment)
    return p


def _workspace(need, given, device):
    if need == 0:
        return None
    if given is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    _require(given.device == device and given.is_contiguous(), f"workspace must be contiguous on {device}")
    _require(given.numel() * given.element_size() >= need, f"workspace must have at least {need} bytes")
    return given


# ---------------------------------------------------------------------------
# linear attention with a constant decay per head
# ---------------------------------------------------------------------------
@dataclass
class DecayAttentionTrainingContext:
    """What the backward needs of the forward: its problem and its inputs
    (cu_seqlens and its CPU mirror among them) with their versions (no device
    memory of its own)."""
    problem: KdaDecayProblem
    inputs: tuple
    versions: tuple


def decay_attention_training_forward(q, k, v, log_decay, initial_state=None, cu_seqlens=None, scale=None, out=None,
                                     final_state_out=None, *, cu_seqlens_cpu=None, segment: int = 0,
                                     workspace: Optional[torch.Tensor] = None):
    """Linear attention with a constant decay per value head, training forward:
    returns (o, final_state, ctx).

    Per sequence and value head, S <- exp(log_decay) S + v k^T and o = scale S q
    (scale 1/sqrt(128) by default), from initial_state (FP32 [N, Hv, 128, 128],
    value-first; None: zero).  q, k: BF16 [B, T, Hqk, 128], v: [B, T, Hv, 128],
    dense or slices of wider token rows; value head h uses q/k head
    h // (Hv // Hqk).  log_decay: FP32 [Hv], at most 0, a constant (no
    gradient).  Packed calls pass cu_seqlens (int64 [N+1]) with its CPU mirror
    and B = 1."""
    dev = _cuda(q)
    p = _decay_problem(q, k, v, log_decay, scale, cu_seqlens, cu_seqlens_cpu, segment)
    states = (p.N, p.Hv, HEAD_DIM, HEAD_DIM)
    if initial_state is not None:
        _dense("initial_state", initial_state, _F32, states, dev)
    o = _new(v) if out is None else out
    if out is not None:
        _dense("out", o, _BF, (p.B, p.T, p.Hv, HEAD_DIM), dev)
    fs = torch.empty(states, dtype=_F32, device=dev) if final_state_out is None else final_state_out
    if final_state_out is not None:
        _dense("final_state_out", fs, _F32, states, dev)
    ws = _workspace(kda_decay_fwd_workspace_bytes(p), workspace, dev)
    kda_decay_fwd(p, q, k, v, log_decay, initial_state, o, fs, ws)
    inputs = (q, k, v, log_decay, initial_state, cu_seqlens, cu_seqlens_cpu)
    versions = tuple(None if t is None else t._version for t in inputs)
    return o, fs, DecayAttentionTrainingContext(p, inputs, versions)


def decay_attention_training_backward(context: DecayAttentionTrainingContext, do, dfinal_state=None,
                                      out: Optional[Sequence[torch.Tensor]] = None,
                                      workspace: Optional[torch.Tensor] = None):
    """Gradients (dq, dk, dv, dinitial_state) of <do, o> + <dfinal_state,
    final_state> (dfinal_state None: zero)."""
    _require(context is not None, "context is required")
    p, inputs = context.problem, context.inputs
    now = tuple(None if t is None else t._version for t in inputs)
    _require(now == context.versions, "an input changed after the forward (tensor version)")
    q, k, v, log_decay, s0, _, _ = inputs
    dev = q.device
    states = (p.N, p.Hv, HEAD_DIM, HEAD_DIM)
    _dense("do", do, _BF, v.shape, dev)
    if dfinal_state is not None:
        _dense("dfinal_state", dfinal_state, _F32, states, dev)
    if out is None:
        out = (_new(q), _new(k), _new(v), torch.empty(states, dtype=_F32, device=dev))
    else:
        _require(len(out) == 4, "out must hold four tensors")
        for name, t, dtype, shape in zip(("dq", "dk", "dv", "dinitial_state"), out, (_BF, _BF, _BF, _F32),
                                         (q.shape, k.shape, v.shape, states)):
            _dense(name, t, dtype, shape, dev)
    ws = _workspace(kda_decay_bwd_workspace_bytes(p), workspace, dev)
    kda_decay_bwd(p, q, k, v, log_decay, s0, do, dfinal_state, *out, ws)
    return tuple(out)


def decay_attention(q, k, v, log_decay, initial_state=None, scale=None, cu_seqlens=None, ssm_state_indices=None,
                    output=None, *, cu_seqlens_cpu=None, ssm_state_indices_cpu=None, segment: int = 0,
                    workspace: Optional[torch.Tensor] = None):
    """Decode and prefill of the same recurrence on an FP32 state pool: returns
    (output, pool).  initial_state is the pool [P, Hv, 128, 128], updated in
    place: sequence n reads and writes slot ssm_state_indices[n] (int32, with
    its CPU mirror), or slot n.  None starts every sequence from zero in a new
    pool of N slots.  Sequences of up to 4 tokens run token by token, longer ones
    in chunks, whatever else is in the call."""
    dev = _cuda(q)
    p = _decay_problem(q, k, v, log_decay, scale, cu_seqlens, cu_seqlens_cpu, segment)
    if initial_state is None:
        _require(ssm_state_indices is None, "ssm_state_indices need an initial_state pool")
        initial_state = torch.zeros((p.N, p.Hv, HEAD_DIM, HEAD_DIM), dtype=_F32, device=dev)
    else:
        _require(isinstance(initial_state, torch.Tensor) and initial_state.dim() == 4,
                 "initial_state must be [P, Hv, 128, 128]")
        _dense("initial_state", initial_state, _F32, (initial_state.shape[0], p.Hv, HEAD_DIM, HEAD_DIM), dev)
    if ssm_state_indices is not None:
        _require(ssm_state_indices_cpu is not None, "ssm_state_indices needs its CPU mirror")
        _dense("ssm_state_indices", ssm_state_indices, torch.int32, (p.N,), dev)
        _dense("ssm_state_indices_cpu", ssm_state_indices_cpu, torch.int32, (p.N,), torch.device("cpu"))
    else:
        _require(ssm_state_indices_cpu is None, "ssm_state_indices_cpu needs ssm_state_indices")
    o = _new(v) if output is None else output
    if output is not None:
        _dense("output", o, _BF, (p.B, p.T, p.Hv, HEAD_DIM), dev)
    ws = None if p.T == 1 else _workspace(kda_decay_infer_workspace_bytes(p), workspace, dev)
    kda_decay_infer(p, q, k, v, log_decay, initial_state, ssm_state_indices, ssm_state_indices_cpu, o, ws)
    return o, initial_state


# ---------------------------------------------------------------------------
# query/key norm with rotary rotation
# ---------------------------------------------------------------------------
def rotary_table(rows: int, rot_dim: int, theta: float = 10000.0, device="cuda"):
    """(cos, sin), FP32 [rows, rot_dim/2]: the angles position * theta^(-2p/rot_dim),
    formed in 64 bits and rounded once."""
    _require(rows >= 1 and rot_dim >= 2 and rot_dim % 2 == 0, "rows must be >= 1 and rot_dim even")
    freq = theta ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * freq
    return angle.cos().float().to(device), angle.sin().float().to(device)


def _qknorm_problem(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved) -> KdaQkNormProblem:
    dev = _cuda(q)
    _cuda(k)
    B, T, Hq, _ = q.shape
    Hk = k.shape[2]
    q_stride, k_stride = _rows("q", q, (B, T, Hq, HEAD_DIM), dev), _rows("k", k, (B, T, Hk, HEAD_DIM), dev)
    _dense("q_weight", q_weight, _F32, (HEAD_DIM,), dev)
    _dense("k_weight", k_weight, _F32, (HEAD_DIM,), dev)
    _require(isinstance(cos, torch.Tensor) and cos.dim() == 2, "cos must be [rows, rot_dim/2]")
    rows, half = angles = cos.shape
    _dense("cos", cos, _F32, angles, dev)
    _dense("sin", sin, _F32, angles, dev)
    if positions is not None:
        _dense("positions", positions, torch.int64, (B, T), dev)
    return KdaQkNormProblem(B, T, Hq, Hk, 2 * half, bool(interleaved), float(eps), rows, q_stride, k_stride)


def qk_norm_rope_forward(q, k, q_weight, k_weight, cos, sin, positions=None, *, eps: float = 1e-6,
                         interleaved: bool = False, out: Optional[Sequence[torch.Tensor]] = None):
    """RMS norm of every query and key head and the rotary rotation, in one pass:
    returns (q_out, k_out).  q: BF16 [B, T, Hq, 128], k: [B, T, Hk, 128], dense
    or slices of wider token rows; weights FP32 [128]; cos, sin: FP32 [rows,
    rot_dim/2] (rotary_table), row `position` for a token; positions: int64
    [B, T], None for the token's index in its row.  Rotates the first rot_dim
    channels: pairs (p, p + rot_dim/2), or (2p, 2p+1) when interleaved."""
    p = _qknorm_problem(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)
    if out is None:
        out = (_new(q), _new(k))
    else:
        _require(len(out) == 2, "out must hold two tensors")
        _dense("q_out", out[0], _BF, q.shape, q.device)
        _dense("k_out", out[1], _BF, k.shape, q.device)
    kda_qknorm_fwd(p, q, k, q_weight, k_weight, cos, sin, positions, *out)
    return tuple(out)


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, cos, sin, positions=None, *, eps: float = 1e-6,
                          interleaved: bool = False, out: Optional[Sequence[torch.Tensor]] = None,
                          workspace: Optional[torch.Tensor] = None):
    """Gradients (dq, dk, dq_weight, dk_weight) from the adjoints of
    qk_norm_rope_forward's outputs and its inputs."""
    p = _qknorm_problem(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)
    dev = q.device
    _dense("dq_out", dq_out, _BF, q.shape, dev)
    _dense("dk_out", dk_out, _BF, k.shape, dev)
    if out is None:
        out = (_new(q), _new(k), _new(q_weight), _new(k_weight))
    else:
        _require(len(out) == 4, "out must hold four tensors")
        for name, t, dtype, shape in zip(("dq", "dk", "dq_weight", "dk_weight"), out, (_BF, _BF, _F32, _F32),
                                         (q.shape, k.shape, (HEAD_DIM,), (HEAD_DIM,))):
            _dense(name, t, dtype, shape, dev)
    ws = _workspace(kda_qknorm_bwd_workspace_bytes(p), workspace, dev)
    kda_qknorm_bwd(p, q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out, *out, ws)
    return tuple(out)


# ---------------------------------------------------------------------------
# gated norm of the heads' outputs
# ---------------------------------------------------------------------------
def _gnorm_problem(x, gate, weight, eps, activation) -> KdaGNormProblem:
    dev = _cuda(x)
    B, T, H, _ = x.shape
    if activation not in _ACTIVATIONS:
        _require(False, f"activation must be one of {tuple(_ACTIVATIONS)}, got {activation!r}")
    shape = (B, T, H, HEAD_DIM)
    _dense("weight", weight, _F32, (HEAD_DIM,), dev)
    return KdaGNormProblem(B, T, H, _ACTIVATIONS[activation], float(eps), _rows("x", x, shape, dev),
                           _rows("gate", gate, shape, dev))


def gated_norm_forward(x, gate, weight, *, eps: float = 1e-6, activation: str = "sigmoid",
                       out: Optional[torch.Tensor] = None):
    """weight * x / sqrt(mean(x^2) + eps) * act(gate) per head, act "sigmoid" or
    "silu".  x, gate: BF16 [B, T, H, 128], dense or slices of wider token rows;
    weight: FP32 [128]."""
    p = _gnorm_problem(x, gate, weight, eps, activation)
    if out is None:
        out = _new(x)
    else:
        _dense("out", out, _BF, x.shape, x.device)
    kda_gnorm_fwd(p, x, gate, weight, out)
    return out


def gated_norm_backward(dy, x, gate, weight, *, eps: float = 1e-6, activation: str = "sigmoid",
                        out: Optional[Sequence[torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None):
    """Gradients (dx, dgate, dweight) from gated_norm_forward's adjoint and inputs."""
    p = _gnorm_problem(x, gate, weight, eps, activation)
    dev = x.device
    _dense("dy", dy, _BF, x.shape, dev)
    if out is None:
        out = (_new(x), _new(x), _new(weight))
    else:
        _require(len(out) == 3, "out must hold three tensors")
        for name, t, dtype, shape in zip(("dx", "dgate", "dweight"), out, (_BF, _BF, _F32),
                                         (x.shape, x.shape, (HEAD_DIM,))):
            _dense(name, t, dtype, shape, dev)
    ws = _workspace(kda_gnorm_bwd_workspace_bytes(p), workspace, dev)
    kda_gnorm_bwd(p, x, gate, weight, dy, *out, ws)
    return tuple(out)


# ---------------------------------------------------------------------------
# layer norm of token rows
# ---------------------------------------------------------------------------
def _lnorm_problem(x, weight, eps) -> KdaLNormProblem:
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype is _BF and x.dim() >= 1 and x.numel() > 0):
        _require(isinstance(x, torch.Tensor) and x.dtype is _BF, "x must be a bfloat16 tensor")
        _require(x.dim() >= 1 and x.numel() > 0, "x must be [..., C] and not empty")
        _require(False, f"tensors must be on a GPU, got {x.device}")
    C = x.shape[-1]
    _dense("weight", weight, _F32, (C,), x.device)
    rows = x.numel() // C
    stride = C
    if not x.is_contiguous():
        _require(x.stride(-1) == 1 or C == 1, "x must have dense channels")
        # rows a fixed distance apart, whatever the leading dimensions
        at = [(n, st) for n, st in zip(x.shape[:-1], x.stride()[:-1]) if n > 1]
        if at:
            stride = at[-1][1]
            _require(stride >= C, "x's rows must not overlap")
            _require(all(a[1] == b[0] * b[1] for a, b in zip(at, at[1:])), "x's rows must be a fixed distance apart")
    return KdaLNormProblem(rows, C, float(eps), stride)


def layer_norm_forward(x, weight, bias=None, *, eps: float = 1e-5, out: Optional[torch.Tensor] = None):
    """weight * (x - mean) / sqrt(mean((x - mean)^2) + eps) + bias over the last
    dimension.  x: BF16 [..., C], C a multiple of 8 up to 32768, dense or a slice of
    wider rows; weight, bias: FP32 [C] (bias None: none)."""
    p = _lnorm_problem(x, weight, eps)
    if bias is not None:
        _dense("bias", bias, _F32, weight.shape, x.device)
    if out is None:
        out = _new(x)
    else:
        _dense("out", out, _BF, x.shape, x.device)
    kda_lnorm_fwd(p, x, weight, bias, out)
    return out


def layer_norm_backward(dy, x, weight, *, eps: float = 1e-5, out: Optional[Sequence[torch.Tensor]] = None,
                        workspace: Optional[torch.Tensor] = None):
    """Gradients (dx, dweight, dbias) from layer_norm_forward's adjoint and inputs
    (none depends on the bias)."""
    p = _lnorm_problem(x, weight, eps)
    dev = x.device
    _dense("dy", dy, _BF, x.shape, dev)
    if out is None:
        out = (_new(x), _new(weight), _new(weight))
    else:
        _require(len(out) == 3, "out must hold three tensors")
        for name, t, dtype, shape in zip(("dx", "dweight", "dbias"), out, (_BF, _F32, _F32),
                                         (x.shape, weight.shape, weight.shape)):
            _dense(name, t, dtype, shape, dev)
    ws = _workspace(kda_lnorm_bwd_workspace_bytes(p), workspace, dev)
    kda_lnorm_bwd(p, x, weight, dy, *out, ws)
    return tuple(out)
