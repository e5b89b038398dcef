"""Python binding of libkda's gated delta rule with one decay per value head and
token: training forward and backward, decode, decode of drafted tokens and
prefill.

Argument marshalling only, as in the package itself: the low-level functions
carry the C names (include/libkda.h), the others take and return tensors.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

from . import HEAD_DIM, _check, _lib, _ptr, _require
from .layers import (_bytes, _byref, _call, _cuda, _declare, _dense, _new, _raw_stream, _rows, _size, _vp, _workspace,
                     _ws)

_BF, _F32 = torch.bfloat16, torch.float32


class KdaDeltaProblem(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("Hqk", ctypes.c_int32),
        ("Hv", ctypes.c_int32), ("N", ctypes.c_int32),
        ("cu_seqlens", _vp), ("cu_seqlens_host", _vp),
        ("scale", ctypes.c_float), ("use_qk_l2norm", ctypes.c_int32), ("segment", ctypes.c_int32),
        ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
    ]


_declare("kda_delta_fwd_workspace_bytes", KdaDeltaProblem, ctypes.POINTER(_size))
_declare("kda_delta_fwd", KdaDeltaProblem, *[_vp] * 9, _size, _vp)
_declare("kda_delta_bwd_workspace_bytes", KdaDeltaProblem, ctypes.c_int32, ctypes.POINTER(_size))
_declare("kda_delta_bwd", KdaDeltaProblem, *[_vp] * 7, _size, *[_vp] * 9, _size, _vp)
_declare("kda_delta_infer_workspace_bytes", KdaDeltaProblem, ctypes.c_int32, ctypes.POINTER(_size))
_declare("kda_delta_infer", KdaDeltaProblem, *[_vp] * 6, ctypes.c_int64, *[_vp] * 2, ctypes.c_int32, *[_vp] * 3, _size,
         _vp)

EXPORTED = ("kda_delta_fwd_workspace_bytes", "kda_delta_fwd", "kda_delta_bwd_workspace_bytes", "kda_delta_bwd",
            "kda_delta_infer_workspace_bytes", "kda_delta_infer")


def kda_delta_fwd_workspace_bytes(p: KdaDeltaProblem) -> int:
    return _bytes("kda_delta_fwd_workspace_bytes", p)


def kda_delta_fwd(p: KdaDeltaProblem, q, k, v, g, beta, initial_state, o, final_state,
                  workspace: Optional[torch.Tensor] = None, stream: Optional[int] = None) -> None:
    """C kda_delta_fwd on torch tensors (no shape checks beyond the library's)."""
    _call(_lib.kda_delta_fwd, stream, q, _byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
          _ptr(initial_state), _ptr(o), _ptr(final_state), *_ws(workspace))


def kda_delta_bwd_workspace_bytes(p: KdaDeltaProblem, records_given: bool = False) -> int:
    n = _size(0)
    _check(_lib.kda_delta_bwd_workspace_bytes(_byref(p), bool(records_given), _byref(n)))
    return int(n.value)


def kda_delta_bwd(p: KdaDeltaProblem, q, k, v, g, beta, initial_state, records, d_o, dfinal_state, dq, dk, dv, dg, dbeta,
                  dinitial_state, workspace: torch.Tensor, stream: Optional[int] = None) -> None:
    """C kda_delta_bwd on torch tensors (records: kda_delta_fwd's workspace, or None)."""
    _call(_lib.kda_delta_bwd, stream, q, _byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
          _ptr(initial_state), *_ws(records), _ptr(d_o), _ptr(dfinal_state), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta),
          _ptr(dinitial_state), *_ws(workspace))


def kda_delta_infer_workspace_bytes(p: KdaDeltaProblem, num_spec_tokens: int = 0) -> int:
    n = _size(0)
    _check(_lib.kda_delta_infer_workspace_bytes(_byref(p), num_spec_tokens, _byref(n)))
    return int(n.value)


def kda_delta_infer(p: KdaDeltaProblem, q, k, v, g, beta, state_pool, state_indices, state_indices_cpu,
                    num_spec_tokens, num_accepted_tokens, o, workspace: Optional[torch.Tensor] = None,
                    stream: Optional[int] = None) -> None:
    """C kda_delta_infer on torch tensors."""
    _call(_lib.kda_delta_infer, stream, q, _byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
          _ptr(state_pool), state_pool.shape[0], _ptr(state_indices), _ptr(state_indices_cpu), num_spec_tokens,
          _ptr(num_accepted_tokens), _ptr(o), *_ws(workspace))


def _problem(q, k, v, g, beta, scale, use_qk_l2norm, cu_seqlens, cu_seqlens_cpu, segment) -> KdaDeltaProblem:
    dev = _cuda(q)
    _cuda(v)
    B, T, Hqk, _ = q.shape
    Hv = v.shape[2]
    qk = (B, T, Hqk, HEAD_DIM)
    p = KdaDeltaProblem(B, T, Hqk, Hv, B, None, None, 0.0, bool(use_qk_l2norm), 0, _rows("q", q, qk, dev),
                        _rows("k", k, qk, dev), _rows("v", v, (B, T, Hv, HEAD_DIM), dev))
    _dense("g", g, _BF, (B, T, Hv), dev)
    _dense("beta", beta, _BF, (B, T, Hv), dev)
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


@dataclass
class GatedDeltaRuleTrainingContext:
    """What the backward needs of the forward: its problem, its inputs (cu_seqlens
    and its CPU mirror among them) with their versions, and its chunks' records
    (about 200 bytes a token and value head, and 128 KiB for each segment of a long
    sequence on few heads; None where the forward was given a
    workspace, which the caller may have used again since).  A backward on another stream than
    the forward's is the caller's to order behind it; the context may be dropped as soon as it is
    called."""
    problem: KdaDeltaProblem
    inputs: tuple
    versions: tuple
    records: Optional[torch.Tensor] = None
    stream: Optional[int] = None   # of the forward


def gated_delta_rule_training_forward(q, k, v, g, beta, initial_state=None, cu_seqlens=None, scale=None, out=None,
                                      final_state_out=None, *, use_qk_l2norm: bool = False, cu_seqlens_cpu=None,
                                      segment: int = 0, workspace: Optional[torch.Tensor] = None):
    """The gated delta rule, training forward: returns (o, final_state, ctx).

    Per sequence and value head, S <- exp(g) S, S <- S + beta (v - S k) k^T and
    o = scale S q (scale 1/sqrt(128) by default), from initial_state (FP32
    [N, Hv, 128, 128], value-first; None: zero).  q, k: BF16 [B, T, Hqk, 128],
    v: [B, T, Hv, 128], dense or slices of wider token rows; value head h uses
    q/k head h // (Hv // Hqk); with use_qk_l2norm q and k are taken at unit
    length.  g (the decay's logarithm, at most 0) and beta: BF16 [B, T, Hv].
    Packed calls pass cu_seqlens (int64 [N+1]) with its CPU mirror and B = 1.
    segment: tokens of the segments that a sequence is walked in (a multiple of 64;
    0: the library's choice)."""
    dev = _cuda(q)
    p = _problem(q, k, v, g, beta, scale, use_qk_l2norm, cu_seqlens, cu_seqlens_cpu, segment)
    states = (p.N, p.Hv, HEAD_DIM, HEAD_DIM)
    if initial_state is not None:
        _dense("initial_state", initial_state, _F32, states, dev)
    o = _new(v) if out is None else out
    if out is not None:
        _dense("out", o, _BF, (p.B, p.T, p.Hv, HEAD_DIM), dev)
    fs = torch.empty(states, dtype=_F32, device=dev) if final_state_out is None else final_state_out
    if final_state_out is not None:
        _dense("final_state_out", fs, _F32, states, dev)
    ws = _workspace(kda_delta_fwd_workspace_bytes(p), workspace, dev)
    kda_delta_fwd(p, q, k, v, g, beta, initial_state, o, fs, ws)
    inputs = (q, k, v, g, beta, initial_state, cu_seqlens, cu_seqlens_cpu)
    versions = tuple(None if t is None else t._version for t in inputs)
    return o, fs, GatedDeltaRuleTrainingContext(p, inputs, versions, ws if workspace is None else None,
                                                _raw_stream(q.get_device()))


def gated_delta_rule_training_backward(context: GatedDeltaRuleTrainingContext, do, dfinal_state=None,
                                       out: Optional[Sequence[torch.Tensor]] = None,
                                       workspace: Optional[torch.Tensor] = None):
    """Gradients (dq, dk, dv, dg, dbeta, dinitial_state) of <do, o> +
    <dfinal_state, final_state> (dfinal_state None: zero)."""
    _require(context is not None, "context is required")
    p, inputs = context.problem, context.inputs
    now = tuple(None if t is None else t._version for t in inputs)
    _require(now == context.versions, "an input changed after the forward (tensor version)")
    q, k, v, g, beta, s0, _, _ = inputs
    dev = q.device
    states = (p.N, p.Hv, HEAD_DIM, HEAD_DIM)
    _dense("do", do, _BF, v.shape, dev)
    if dfinal_state is not None:
        _dense("dfinal_state", dfinal_state, _F32, states, dev)
    if out is None:
        out = (_new(q), _new(k), _new(v), _new(g), _new(beta), torch.empty(states, dtype=_F32, device=dev))
    else:
        _require(len(out) == 6, "out must hold six tensors")
        for name, t, dtype, shape in zip(("dq", "dk", "dv", "dg", "dbeta", "dinitial_state"), out,
                                         (_BF, _BF, _BF, _BF, _BF, _F32),
                                         (q.shape, k.shape, v.shape, g.shape, beta.shape, states)):
            _dense(name, t, dtype, shape, dev)
    records = context.records
    ws = _workspace(kda_delta_bwd_workspace_bytes(p, records is not None), workspace, dev)
    kda_delta_bwd(p, q, k, v, g, beta, s0, records, do, dfinal_state, *out, ws)
    if _raw_stream(q.get_device()) != context.stream:
        # once the context is dropped, its memory waits for this stream too
        other = torch.cuda.current_stream(dev)
        for t in (*inputs[:7], records):
            if t is not None:
                t.record_stream(other)
    return tuple(out)


def gated_delta_rule(q, k, v, g, beta, initial_state=None, scale=None, cu_seqlens=None, ssm_state_indices=None,
                     output=None, *, use_qk_l2norm: bool = False, num_spec_tokens: int = 0, num_accepted_tokens=None,
                     cu_seqlens_cpu=None, ssm_state_indices_cpu=None, workspace: Optional[torch.Tensor] = None):
    """Decode and prefill of the same recurrence on an FP32 state pool: returns
    (output, pool).  initial_state is the pool [P, Hv, 128, 128], updated in
    place: sequence n reads and writes slot ssm_state_indices[n] (int32, with
    its CPU mirror), or slot n.  None starts every sequence from zero in a new
    pool of N slots.  Sequences of up to 4 tokens run token by token, longer ones
    in chunks, whatever else is in the call.  Drafted tokens (num_spec_tokens =
    S): every sequence has 1+S tokens, ssm_state_indices is [N, 1+S]; the state
    starts from slot [n, a-1] with a = num_accepted_tokens[n] (int32; verify_drafts
    gives it) clamped to [1, 1+S], 1 when omitted, and the state after token s goes
    to slot [n, s]."""
    dev = _cuda(q)
    p = _problem(q, k, v, g, beta, scale, use_qk_l2norm, cu_seqlens, cu_seqlens_cpu, 0)
    spec = int(num_spec_tokens or 0)
    _require(spec >= 0, f"num_spec_tokens must be >= 0, got {num_spec_tokens}")
    if initial_state is None:
        _require(ssm_state_indices is None and spec == 0,
                 "ssm_state_indices and drafted tokens need an initial_state pool")
        initial_state = torch.zeros((p.N, p.Hv, HEAD_DIM, HEAD_DIM), dtype=_F32, device=dev)
    else:
        _require(isinstance(initial_state, torch.Tensor) and initial_state.dim() == 4,
                 "initial_state must be [P, Hv, 128, 128]")
        _dense("initial_state", initial_state, _F32, (initial_state.shape[0], p.Hv, HEAD_DIM, HEAD_DIM), dev)
    if ssm_state_indices is not None:
        _require(ssm_state_indices_cpu is not None, "ssm_state_indices needs its CPU mirror")
        shape = (p.N, 1 + spec) if spec else (p.N,)
        _dense("ssm_state_indices", ssm_state_indices, torch.int32, shape, dev)
        _dense("ssm_state_indices_cpu", ssm_state_indices_cpu, torch.int32, shape, torch.device("cpu"))
    else:
        _require(ssm_state_indices_cpu is None, "ssm_state_indices_cpu needs ssm_state_indices")
    if num_accepted_tokens is not None:
        _dense("num_accepted_tokens", num_accepted_tokens, torch.int32, (p.N,), dev)
    o = _new(v) if output is None else output
    if output is not None:
        _dense("output", o, _BF, (p.B, p.T, p.Hv, HEAD_DIM), dev)
    ws = None if p.T == 1 else _workspace(kda_delta_infer_workspace_bytes(p, spec), workspace, dev)
    kda_delta_infer(p, q, k, v, g, beta, initial_state, ssm_state_indices, ssm_state_indices_cpu, spec,
                    num_accepted_tokens, o, ws)
    return o, initial_state
