"""Inputs and bars shared by the tests of the linear-attention layer operators.

Bars.  u = 2^-8 is half a BF16 step relative to the value, the most that one
rounding is off.
  - A BF16 result with one rounding (row norms): elementwise u |ref|, plus what
    its FP32 arithmetic adds (stated where it is used).
  - A scanned BF16 result (o, dq, dk, dv) has three: the products P, the state
    as an operand, and the result.  Their errors are independent with standard
    deviation at most u/sqrt(3) of what they round, and the parts that P and
    the state feed add up to the result, so the error's norm is about
    u sqrt(2/3) = 0.82 u of the result's; the bar is u.  One element: its own
    rounding, u |ref|, and a sum of many errors.  The state's are those of
    s sum_k S[v][k] q_k, of variance u^2/3 s^2 sum_k S[v][k]^2 q_k^2, and S^2
    is about E, the same recurrence over squares (E <- e^{2l} E + v^2 k^2):
    what a row's terms weigh does not shrink where the terms cancel.  Those of
    P are as large.  So the bar is u |ref| + 8 u sqrt(2/3) sqrt(energy), with
    energy = s^2 sum_k E[v][k] q_k^2: the definition at squared inputs.
  - An FP32 state adds up exact products over a chunk of 64 tokens in FP32:
    2^-24 for each of 64 sums, 2^-18 of the sum of absolute values.
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -8
ELEMENT = 8 * U * (2.0 / 3.0) ** 0.5
STATE = 2.0 ** -18


def bf(gen, *shape):
    return torch.randn(shape, generator=gen, dtype=torch.float32).to(torch.bfloat16)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def check_scanned(name, got, ref, energy):
    got = f64(got)
    assert np.isfinite(got).all(), f"{name}: not finite"
    err = np.abs(got - ref)
    norm = np.linalg.norm(ref)
    rel = np.linalg.norm(err) / norm if norm else np.linalg.norm(err)
    worst = (err / np.maximum(U * np.abs(ref) + ELEMENT * np.sqrt(energy), 1e-30)).max()
    print(f"{name:14s} rel {rel:.2e} (bar {U:.2e})  elementwise {worst:.2f} of the bar", flush=True)
    assert rel <= U and worst <= 1.0, name


def check_state(name, got, ref, majorant):
    got = f64(got)
    assert np.isfinite(got).all(), f"{name}: not finite"
    worst = (np.abs(got - ref) / np.maximum(STATE * majorant, 1e-30)).max()
    print(f"{name:14s} elementwise {worst:.2f} of the bar", flush=True)
    assert worst <= 1.0, name


def check_bars(name, got, ref, bar):
    """|got - ref| <= bar, elementwise."""
    got = f64(got)
    assert np.isfinite(got).all(), f"{name}: not finite"
    worst = (np.abs(got - ref) / np.maximum(bar, 1e-30)).max()
    print(f"{name:14s} elementwise {worst:.2f} of the bar", flush=True)
    assert worst <= 1.0, name
