"""Python binding of libkda's verification of drafted tokens.

Argument marshalling only, as in the package itself: the low-level functions
carry the C names (include/libkda.h), verify_drafts takes and returns tensors.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _lib, _ptr, _require
from .layers import _bytes, _byref, _call, _declare, _dense, _size, _vp, _workspace, _ws

_I32, _F32 = torch.int32, torch.float32


class KdaVerifyProblem(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int32), ("S", ctypes.c_int32), ("V", ctypes.c_int32),
        ("target_stride", ctypes.c_int64), ("draft_stride", ctypes.c_int64),
        ("target_seq_stride", ctypes.c_int64), ("draft_seq_stride", ctypes.c_int64),
    ]


_declare("kda_verify_workspace_bytes", KdaVerifyProblem, ctypes.POINTER(_size))
_declare("kda_verify", KdaVerifyProblem, *[_vp] * 8, _size, _vp)

EXPORTED = ("kda_verify_workspace_bytes", "kda_verify")


def kda_verify_workspace_bytes(p: KdaVerifyProblem) -> int:
    return _bytes("kda_verify_workspace_bytes", p)


def kda_verify(p: KdaVerifyProblem, draft_tokens, draft_lens, target_probs, draft_probs, uniform, tokens, num_accepted,
               workspace: Optional[torch.Tensor] = None, stream: Optional[int] = None) -> None:
    """C kda_verify on torch tensors (no shape checks beyond the library's)."""
    _call(_lib.kda_verify, stream, target_probs, _byref(p), _ptr(draft_tokens), _ptr(draft_lens), _ptr(target_probs),
          _ptr(draft_probs), _ptr(uniform), _ptr(tokens), _ptr(num_accepted), *_ws(workspace))


def _prob_rows(name, t, shape, device):
    """The strides of rows and of sequences of FP32 [N, rows, V] probabilities (the latter 0: as
    many rows): dense, or a slice of wider rows, or of more of them."""
    if not (isinstance(t, torch.Tensor) and t.dtype is _F32 and t.shape == shape and t.device == device):
        _require(isinstance(t, torch.Tensor) and t.dtype is _F32, f"{name} must be a float32 tensor")
        _require(t.shape == shape, f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        _require(False, f"{name} must be on {device}, got {t.device}")
    N, R, V = shape
    if t.is_contiguous():
        return V, 0
    sn, sr, sv = t.stride()
    _require(sv == 1 or V == 1, f"{name} must have dense rows")
    if R <= 1:
        sr = V
    _require(sr >= V and (N == 1 or sn >= (R - 1) * sr + V), f"{name}'s rows must not overlap")
    return sr, sn if N > 1 else 0


def verify_drafts(draft_tokens, target_probs, uniform, draft_probs=None, draft_lens=None, *,
                  out: Optional[Sequence[torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None):
    """Which drafted tokens stand against the target's probabilities, and the token
    behind them: returns (tokens, num_accepted), int32 [N, 1+S] and [N].

    draft_tokens: int32 [N, S], the drafts x of every sequence (draft_lens: int32
    [N], how many of them there are; None: S each).  target_probs: float32 [N, 1+S,
    V], the target's probabilities p at each draft's place and behind the last one.
    draft_probs: float32 [N, S, V], those q that the drafts were drawn from; None
    for drafts that are certain.  Both may be slices of wider rows, or the first rows of buffers with
    more of them.  uniform: float32 [N, 1+S], random numbers in [0, 1).
    Draft i stands while those before it do and uniform[:, i] q(x) < p(x); then one
    token is drawn from the positive part of p - q (behind the last draft from p) by
    uniform[:, S].  tokens holds the drafts that stand, the drawn token, then -1;
    num_accepted is one more than the drafts that stand, as gated_delta_rule and
    recurrent_kda take it for the call that follows."""
    if not (isinstance(target_probs, torch.Tensor) and target_probs.dim() == 3 and target_probs.is_cuda):
        _require(isinstance(target_probs, torch.Tensor) and target_probs.dim() == 3, "target_probs must be [N, 1+S, V]")
        _require(False, f"tensors must be on a GPU, got {target_probs.device}")
    dev = target_probs.device
    N, S, V = target_probs.shape
    S -= 1
    _require(N >= 1 and S >= 0 and V >= 1, "target_probs must not be empty")
    p = KdaVerifyProblem(N, S, V)
    p.target_stride, p.target_seq_stride = _prob_rows("target_probs", target_probs, (N, S + 1, V), dev)
    _dense("draft_tokens", draft_tokens, _I32, (N, S), dev)
    _dense("uniform", uniform, _F32, (N, S + 1), dev)
    if draft_probs is not None:
        p.draft_stride, p.draft_seq_stride = _prob_rows("draft_probs", draft_probs, (N, S, V), dev)
    if draft_lens is not None:
        _dense("draft_lens", draft_lens, _I32, (N,), dev)
    if out is None:
        out = (draft_tokens.new_empty((N, S + 1)), draft_tokens.new_empty((N,)))
    else:
        _require(len(out) == 2, "out must hold two tensors")
        _dense("tokens", out[0], _I32, (N, S + 1), dev)
        _dense("num_accepted", out[1], _I32, (N,), dev)
    ws = _workspace(kda_verify_workspace_bytes(p), workspace, dev)
    kda_verify(p, draft_tokens, draft_lens, target_probs, draft_probs, uniform, *out, ws)
    return tuple(out)
