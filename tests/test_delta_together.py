"""The gated delta rule, the drafted tokens' verification and the layer norm as a model uses them
together: a training layer, and a serving loop of drafted tokens.  Every stage is held to its own
bars against the FP64 oracle, on the inputs that the stage before it gave."""
import numpy as np
import pytest
import torch

from oracle import delta_oracle as do_
from tests import delta_util as du
from tests import layer_util as lu
from tests import test_layer_norm as ln
from tests.delta_util import Inp
from tests.test_verify_drafts import Drafts

pytestmark = pytest.mark.gpu

SPLIT = [128, 128, 256]     # q, k and two heads of v in a normalised row
C = sum(SPLIT)


def rows(y, B, T):
    """q, k, v [B, T, heads, 128] as slices of y's rows."""
    return [x.unflatten(-1, (-1, 128)) for x in y.view(B, T, C).split(SPLIT, -1)]


@pytest.mark.parametrize("lengths,packed", [([70, 70], False), ([65, 3, 130], True)])
def test_training_layer(lengths, packed):
    """Normalised rows are the rule's q, k and v; their gradients go back through the norm."""
    import gated_delta_rule_32_amd as kda
    inp = Inp(lengths, packed, 1, 2, seed=71)
    tokens = inp.B * inp.T
    x, w, b, _ = ln.make(tokens, C, 72)
    dev = [t.cuda() for t in (x, w, b)]

    def step(x, w, b):
        y = kda.layer_norm_forward(x, w, b)
        o, final, ctx = kda.gated_delta_rule_training_forward(*rows(y, inp.B, inp.T), d["g"], d["beta"], d["s0"], d["cu"],
                                                              use_qk_l2norm=True, cu_seqlens_cpu=inp.cu)
        grads = kda.gated_delta_rule_training_backward(ctx, d["do"], d["ds"])
        dy = torch.cat([t.flatten(2) for t in grads[:3]], -1).view(tokens, C)
        return (y, o, final, dy, *grads, *kda.layer_norm_backward(dy, x, w))

    d = {n: inp.dev(getattr(inp, n)) for n in ("g", "beta", "s0", "do", "ds", "cu")}
    y, o, final, dy, *rest = step(*dev)
    torch.cuda.synchronize()
    ln.check_forward(y, x, w, b, 1e-5)
    inp.q, inp.k, inp.v = (t.contiguous() for t in rows(y.cpu(), inp.B, inp.T))
    ref_o, ref_final, (wo, wfinal), _ = inp.reference()
    du.check_o("o", o, ref_o, wo)
    du.check_state("final_state", final, ref_final, wfinal)
    du.check_gradients(inp, rest[:6])
    ln.check_backward(rest[6:], dy.cpu(), x, w, 1e-5)
    # in a graph, on other rows, with eager work between (the packed schedule is there by now)
    graph = torch.cuda.CUDAGraph()
    step(*dev)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step(*dev)
    for _ in range(3):
        dev[0].copy_(dev[0].flip(0))
        graph.replay()
        torch.cuda.synchronize()
        for name, a, e in zip("y o final dy dq dk dv dg dbeta ds0 dx dw db".split(), got, step(*dev)):
            assert torch.equal(a, e), name


def test_serving_loop():
    """Prompts, then drafted tokens whose verification says, on the device, where the next
    call's states start: the recurrence over the prompt and the tokens that stood."""
    import gated_delta_rule_32_amd as kda
    N, S, V, prompts = 5, 3, 700, [40, 7, 1, 3, 90]
    slots = torch.randperm(N * (S + 1) + 2, generator=torch.Generator().manual_seed(1))[:N * (S + 1)].view(N, S + 1).to(torch.int32)
    pool = torch.randn((N * (S + 1) + 2, 2, 128, 128), generator=torch.Generator().manual_seed(2)).cuda()
    start = pool[slots[:, 0].long().cuda()].cpu()
    prompt = Inp(prompts, True, 1, 2, seed=81)
    first = slots[:, 0].contiguous()
    kda.gated_delta_rule(*(prompt.dev(t) for t in (prompt.q, prompt.k, prompt.v, prompt.g, prompt.beta)), pool,
                         cu_seqlens=prompt.dev(prompt.cu), cu_seqlens_cpu=prompt.cu, ssm_state_indices=first.cuda(),
                         ssm_state_indices_cpu=first, use_qk_l2norm=True)
    torch.cuda.synchronize()
    kept = pool.clone()
    rounds = []
    for i in range(3):
        inp = Inp([S + 1] * N, False, 1, 2, seed=90 + i)
        x, w, b, _ = ln.make(N * (S + 1), C, 95 + i)
        rounds.append((inp, [t.cuda() for t in (x, w, b)], [inp.dev(inp.g), inp.dev(inp.beta)], Drafts(N, S, V, 20 + i)))
    draws = [[t.cuda() for t in (r[3].drafts, r[3].target, r[3].uniform, r[3].draft)] for r in rounds]
    dev_slots = slots.cuda()

    def loop():
        out, accepted = [], torch.ones(N, dtype=torch.int32, device="cuda")
        for (inp, norm, gates, _), draw in zip(rounds, draws):
            y = kda.layer_norm_forward(*norm)
            o, _ = kda.gated_delta_rule(*rows(y, N, S + 1), *gates, pool, ssm_state_indices=dev_slots,
                                        ssm_state_indices_cpu=slots, use_qk_l2norm=True, num_spec_tokens=S,
                                        num_accepted_tokens=accepted)
            tokens, accepted = kda.verify_drafts(*draw)
            out += [y, o, tokens, accepted]
        return out

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = loop()
    pool.copy_(kept)
    got = loop()
    torch.cuda.synchronize()
    end = pool.clone()
    for _ in range(3):
        pool.copy_(kept)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, e) for a, e in zip(captured, got)) and torch.equal(pool, end)
        draws[0][2].add_(0.0)
    # against the oracle: user n's tokens so far, from the start of the prompt
    so_far = [[t[:, prompt.cu[n]:prompt.cu[n + 1]] for t in (prompt.q, prompt.k, prompt.v, prompt.g, prompt.beta)] for n in range(N)]
    stood = set()
    for i, (inp, _, _, drafts) in enumerate(rounds):
        y, o, tokens, accepted = (t.cpu() for t in got[4 * i:4 * i + 4])
        want, count = drafts.reference()
        assert np.array_equal(tokens.numpy(), want) and np.array_equal(accepted.numpy(), count)
        q, k, v = rows(y, N, S + 1)
        for n in range(N):
            new = [t[n:n + 1] for t in (q, k, v, inp.g, inp.beta)]
            seq = [torch.cat([a, c], 1) for a, c in zip(so_far[n], new)]
            T = seq[0].shape[1]
            ref, _, (weights, _), _ = do_.delta_forward(*(lu.f64(t) for t in seq), lu.f64(start[n:n + 1]), [T], False, du.SCALE, True)
            lu.check_bars(f"o {i} {n}", o[n:n + 1], ref[:, T - S - 1:],
                          lu.U * np.abs(ref[:, T - S - 1:]) + du.PARTS * weights[:, T - S - 1:])
            a = int(accepted[n])
            stood.add(a)
            so_far[n] = [torch.cat([t, c[:, :a]], 1) for t, c in zip(so_far[n], new)]
    assert len(stood) > 1     # (drafts stood and did not)


def test_calls_on_two_streams_at_once():
    """Training steps, prompts and drafted tokens on two streams, each with its own tensors and both
    with the same cached schedules: the bits of the calls by themselves, again and again."""
    import gated_delta_rule_32_amd as kda
    inps = [Inp([200, 64, 1, 130], True, 1, 2, seed=s) for s in (101, 102)]
    dev = [{n: i.dev(getattr(i, n)) for n in ("q", "k", "v", "g", "beta", "s0", "do", "ds", "cu")} for i in inps]
    rows_ = [ln.make(300, 1024, s) for s in (103, 104)]
    rows_ = [[t.cuda() for t in r] for r in rows_]

    def work(j):
        d, (x, w, b, dy) = dev[j], rows_[j]
        ins = [d[n] for n in ("q", "k", "v", "g", "beta")]
        more = dict(use_qk_l2norm=True, cu_seqlens_cpu=inps[j].cu)
        out = []
        for segment in (0, 64):
            o, final, ctx = kda.gated_delta_rule_training_forward(*ins, d["s0"], d["cu"], segment=segment, **more)
            out += [o, final, *kda.gated_delta_rule_training_backward(ctx, d["do"], d["ds"])]
        pool = d["s0"].clone()
        out += [kda.gated_delta_rule(*ins, pool, cu_seqlens=d["cu"], **more)[0], pool]
        out += [kda.layer_norm_forward(x, w, b), *kda.layer_norm_backward(dy, x, w)]
        return out
    want = [work(0), work(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for j in (0, 1):
            with torch.cuda.stream(streams[j]):
                got[j].append(work(j))
    torch.cuda.synchronize()
    for j in (0, 1):
        for again in got[j]:
            assert all(torch.equal(a, e) for a, e in zip(again, want[j]))
