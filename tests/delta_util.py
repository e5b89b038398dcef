"""Inputs and bars shared by the tests of the gated delta rule.

Bars.  u = 2^-8 is half a BF16 step relative to the value, the most that one
rounding is off.
  - What the rule adds up.  For |beta| |k|^2 <= 2 the rule's factor 1 - beta k k^T does
    not enlarge a row of the state, so an error made in a token's written row is
    carried on at its size and decays with the state.  A written row w = v - S k is
    formed in FP32 from a chunk's sums of up to 128 + 64 terms, and C, which solves the chunk's rule, adds as
    many again: 2^-24 for each of 2^6 of them (their errors are of random sign),
    2^-18 of the terms' sizes.  The oracle's weights M add up these sizes for each row of the
    state; a final state's element is off by at most 2^-18 M.
  - o = scale S q takes S in two pieces of 8 bits (off by 2^-16) and the chunk's
    products and written rows in two (2^-17 each): 2^-14 of the weights, and its own rounding, u |o|.
  - The norm of a BF16 result's error: one rounding's errors are spread evenly, u/sqrt(3) of the value in
    the mean square at most; 3/4 u leaves 30% for the parts above.
  - A gradient's sums take the states before and behind a block and the rows W and Y in FP16, off by
    2^-11 at most and 2^-12.3 in the mean square; over 128 terms that is 2^-12.3 sqrt(2) / sqrt(128)
    of the weights, 2^-14 with terms of uneven sizes, in the mean square.  The block's matrices go as two BF16 pieces
    (2^-17).  2^-13 of the weights covers twice that, and u |ref| beside it leaves room for more.  dq and dk of shared heads are
    sums of partials that are rounded to 10 bits: 2^-10 of the partials' sizes.  dinitial_state is as exact
    as a final state.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import delta_oracle as do_
from tests import layer_util as lu

SCALE = 1.0 / math.sqrt(128.0)
STATE = 2.0 ** -18
PARTS = 2.0 ** -14
GRADS = 2.0 ** -13


class Inp:
    """A call's inputs on the CPU.  `gates`: "layer" (as a layer starts out with), "strong", "none" or
    "mixed" (none, strong, total and ordinary decays side by side, beta of 0 and 1 among them)."""

    def __init__(self, lengths, packed, Hqk, Hv, seed=0, state=True, unit=True, gates="layer"):
        g = torch.Generator().manual_seed(seed)
        B, T = (1, sum(lengths)) if packed else (len(lengths), lengths[0])
        N = len(lengths)
        self.lengths, self.packed, self.N, self.B, self.T, self.Hqk, self.Hv = lengths, packed, N, B, T, Hqk, Hv
        self.unit = unit
        self.q, self.k, self.v = lu.bf(g, B, T, Hqk, 128), lu.bf(g, B, T, Hqk, 128), lu.bf(g, B, T, Hv, 128)
        if not unit:   # (a rounded row's length is within 2^-8 of 1: beta |k|^2 stays below 2)
            self.q, self.k = ((x.float() / x.float().norm(dim=-1, keepdim=True)).bfloat16() for x in (self.q, self.k))
        self.do = lu.bf(g, B, T, Hv, 128)
        x = torch.rand((B, T, Hv), generator=g)
        beta = torch.sigmoid(torch.randn((B, T, Hv), generator=g))
        if gates == "layer":
            gate = -(1 + 15 * torch.rand((Hv,), generator=g)) * 0.001 * 100.0 ** x
        elif gates == "strong":
            gate = -30.0 * x
        elif gates == "none":
            gate = torch.zeros_like(x)
        else:
            kind = torch.randint(0, 6, (B, T, Hv), generator=g)
            gate = torch.where(kind == 0, 0.0, torch.where(kind == 1, -40.0 * x, torch.where(kind == 2, -float("inf"), -0.1 * x)))
            pick = torch.randint(0, 5, (B, T, Hv), generator=g)
            beta = torch.where(pick == 0, 0.0, torch.where(pick == 1, 1.0, beta))
        self.g, self.beta = gate.bfloat16(), beta.bfloat16()
        self.s0 = torch.randn((N, Hv, 128, 128), generator=g) if state else None
        self.ds = torch.randn((N, Hv, 128, 128), generator=g) if state else None
        self.cu = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int64) if packed else None

    def dev(self, x):
        return None if x is None else x.cuda()

    def zeros(self):
        return torch.zeros(self.N, self.Hv, 128, 128)

    def rows(self):
        return [lu.f64(x) for x in (self.q, self.k, self.v, self.g, self.beta)]

    def reference(self, scale=SCALE):
        s0 = self.s0 if self.s0 is not None else self.zeros()
        return do_.delta_forward(*self.rows(), lu.f64(s0), self.lengths, self.packed, scale, self.unit)

    def gradients(self, scale=SCALE):
        s0 = self.s0 if self.s0 is not None else self.zeros()
        ds = self.ds if self.ds is not None else self.zeros()
        return do_.delta_backward(*self.rows(), lu.f64(s0), lu.f64(self.do), lu.f64(ds), self.lengths, self.packed, scale,
                                  self.unit)


def check_o(name, got, ref, weights):
    got = lu.f64(got)
    norm = np.linalg.norm(ref)
    lu.check_bars(name, torch.from_numpy(got), ref, lu.U * np.abs(ref) + PARTS * weights)
    if norm:
        rel = np.linalg.norm(got - ref) / norm
        print(f"{name:14s} rel {rel:.2e} (bar {0.75 * lu.U:.2e})", flush=True)
        assert rel <= 0.75 * lu.U, name


def check_state(name, got, ref, weights):
    """`weights`: of the state's rows."""
    lu.check_bars(name, got, ref, STATE * weights[..., None] * np.ones_like(ref))


def check_gradients(inp, got, scale=SCALE):
    """got: dq, dk, dv, dg, dbeta, dinitial_state."""
    refs, weights, parts = inp.gradients(scale)
    for i, name in enumerate(("dq", "dk", "dv", "dg", "dbeta")):
        x, ref = lu.f64(got[i]), refs[i]
        extra = 2.0 ** -10 * parts[i] if i < 2 and inp.Hv > inp.Hqk else 0.0
        lu.check_bars(name, torch.from_numpy(x), ref, lu.U * np.abs(ref) + GRADS * weights[i] + extra)
        rel = np.linalg.norm(x - ref) / max(np.linalg.norm(ref), 1e-30)
        # (a few values' norm is no mean square: two tokens' gates are held to their own roundings)
        print(f"{name:14s} rel {rel:.2e} (bar {0.75 * lu.U:.2e})", flush=True)
        if ref.size >= 64 and np.linalg.norm(ref) > 2.0 ** -10 * np.linalg.norm(weights[i]):
            assert rel <= 0.75 * lu.U, name
    check_state("dinitial_state", got[5], refs[5], weights[5])
