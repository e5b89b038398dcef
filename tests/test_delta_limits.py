"""CPU tests of limits: a launch holds less than 2^32 threads, and what would take more is refused before
it, by the number of threads that the kernel's workgroups have; distances between the verification's sequences."""
import ctypes

import pytest

import gated_delta_rule_32_amd as kda
from tests.test_delta_abi import GAP, OK, OVERLAP, SHAPE, bwd, delta, fwd, verify

FAR = 1 << 52


@pytest.mark.parametrize("V,most", [(1, (1 << 22) - 1), (16384, (1 << 22) - 1), (16385, ((1 << 24) - 1) // 5), (1 << 20, (1 << 16) - 1)])
def test_verification_refuses_more_than_a_launch(V, most):
    """Rows of up to 16384 values take a workgroup of 1024 threads a sequence, longer ones one of 256 for
    every 4096 values."""
    n = ctypes.c_size_t()
    for S in (0, 1):
        p = kda.KdaVerifyProblem(most, S, V)
        assert kda._lib.kda_verify_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == OK
        p.N += 1
        assert kda._lib.kda_verify_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == SHAPE
        assert verify(p) == SHAPE


def test_segments_refuse_more_than_a_chains_launch():
    """The chain of segments takes eight workgroups of 512 threads a sequence and value head: 2^20 of them
    are too many."""
    p = delta(B=1 << 14, T=100, Hqk=64, Hv=64, N=1 << 14, segment=64)
    names = {"fwd": "q k v g beta s0 o fs", "bwd": "q k v g beta s0 do ds dq dk dv dg db di"}
    for call, ws in ((fwd, "fwd"), (bwd, "bwd")):
        a = {n: (i + 1) * FAR for i, n in enumerate(names[ws].split())}
        assert call(p, ws=60 * FAR, ws_bytes=1 << 60, **a) == SHAPE


@pytest.mark.parametrize("which", ["target_seq_stride", "draft_seq_stride"])
def test_verification_refuses_sequence_strides(which):
    """Sequences that overlap, and ones so far apart that an offset passes 63 bits."""
    n = ctypes.c_size_t()
    rows = 4 if which == "target_seq_stride" else 3
    for stride, status in ((0, OK), ((rows - 1) * 9 + 8, OK), ((rows - 1) * 9 + 7, SHAPE), (-64, SHAPE), ((1 << 60) // 5, OK),
                           ((1 << 60) // 5 + 1, SHAPE)):
        p = kda.KdaVerifyProblem(5, 3, 8, 9, 9)
        setattr(p, which, stride)
        assert kda._lib.kda_verify_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == status
    p = kda.KdaVerifyProblem(2, 3, 8, 0, 0, 1 << 20, 1 << 20)
    assert verify(p, tokens=3 * GAP + (1 << 22) + 96) == OVERLAP        # over the last row of the second sequence
    assert verify(p, tokens=4 * GAP + (1 << 22) + 64) == OVERLAP
