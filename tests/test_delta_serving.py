"""GPU tests of the gated delta rule's serving forms: state pools that no cache holds, and a captured
loop of drafted tokens whose inputs change from replay to replay."""
import pytest
import torch

from tests.delta_util import Inp
from tests.test_verify_drafts import Drafts

pytestmark = pytest.mark.gpu


def parts(inp, rows):
    return [x[rows].contiguous().cuda() for x in (inp.q, inp.k, inp.v, inp.g, inp.beta)]


def test_decode_of_states_past_the_caches():
    """48 x 64 states go past the caches (2 x 192 MiB); the bits of the same sequences a few at a time."""
    import gated_delta_rule_32_amd as kda
    N, Hv = 48, 64
    inp = Inp([1] * N, False, 16, Hv, seed=361, state=False, gates="mixed")
    slots = torch.randperm(N + 3, generator=torch.Generator().manual_seed(1))[:N].to(torch.int32)
    pool = torch.randn((N + 3, Hv, 128, 128), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    near = pool.clone()
    out, _ = kda.gated_delta_rule(*parts(inp, slice(None)), pool, ssm_state_indices=slots.cuda(), ssm_state_indices_cpu=slots,
                                  use_qk_l2norm=True)
    for i in range(0, N, 6):
        some = slots[i:i + 6].contiguous()
        few, _ = kda.gated_delta_rule(*parts(inp, slice(i, i + 6)), near, ssm_state_indices=some.cuda(),
                                      ssm_state_indices_cpu=some, use_qk_l2norm=True)
        assert torch.equal(few, out[i:i + 6])
    assert torch.equal(near, pool)


def test_drafted_tokens_of_states_past_the_caches():
    import gated_delta_rule_32_amd as kda
    N, Hv, S = 32, 32, 4
    inp = Inp([S + 1] * N, False, 16, Hv, seed=362, state=False, gates="mixed")
    g = torch.Generator().manual_seed(3)
    slots = torch.randperm(N * (S + 1) + 2, generator=g)[:N * (S + 1)].view(N, S + 1).to(torch.int32)
    accepted = torch.randint(1, S + 2, (N,), generator=g, dtype=torch.int32)
    pool = torch.randn((N * (S + 1) + 2, Hv, 128, 128), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    near = pool.clone()
    more = dict(use_qk_l2norm=True, num_spec_tokens=S)
    out, _ = kda.gated_delta_rule(*parts(inp, slice(None)), pool, ssm_state_indices=slots.cuda(), ssm_state_indices_cpu=slots,
                                  num_accepted_tokens=accepted.cuda(), **more)
    for i in range(0, N, 8):
        some = slots[i:i + 8].contiguous()
        few, _ = kda.gated_delta_rule(*parts(inp, slice(i, i + 8)), near, ssm_state_indices=some.cuda(),
                                      ssm_state_indices_cpu=some, num_accepted_tokens=accepted[i:i + 8].cuda(), **more)
        assert torch.equal(few, out[i:i + 8])
    assert torch.equal(near, pool)


def test_captured_loop_of_drafted_tokens_on_other_inputs():
    """Two rounds of drafted tokens and their verification in one graph, replayed on other tokens, drafts and random numbers
    each time: the eager loop's bits, other numbers of accepted tokens among them."""
    import gated_delta_rule_32_amd as kda
    N, S, V, seeds = 5, 3, 700, (371, 372, 373, 371)
    slots = torch.randperm(N * (S + 1), generator=torch.Generator().manual_seed(5)).view(N, S + 1).to(torch.int32)
    dev_slots = slots.cuda()
    kept = torch.randn((N * (S + 1), 2, 128, 128), generator=torch.Generator().manual_seed(6)).cuda()
    pool = kept.clone()

    def inputs(seed):
        rounds = []
        for i in range(2):
            inp, d = Inp([S + 1] * N, False, 1, 2, seed=seed + 10 * i, state=False), Drafts(N, S, V, seed + 10 * i)
            if seed % 2:   # (more of the drafts stand)
                d.uniform[:, :S] *= 0.25
            rounds.append(parts(inp, slice(None)) + [t.cuda() for t in (d.drafts, d.target, d.uniform, d.draft)])
        return rounds

    def loop(rounds, pool):
        out, accepted = [], None
        for r in rounds:
            o, _ = kda.gated_delta_rule(*r[:5], pool, ssm_state_indices=dev_slots, ssm_state_indices_cpu=slots,
                                        use_qk_l2norm=True, num_spec_tokens=S, num_accepted_tokens=accepted)
            tokens, accepted = kda.verify_drafts(*r[5:])
            out += [o, tokens, accepted]
        return out
    held = inputs(seeds[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = loop(held, pool)
    seen = set()
    for seed in seeds:
        now = inputs(seed)
        for a, b in zip(held, now):
            for x, y in zip(a, b):
                x.copy_(y)
        for x in captured:
            x.fill_(-9)
        pool.copy_(kept)
        graph.replay()
        torch.cuda.synchronize()
        eager = kept.clone()
        want = loop(now, eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, e) for a, e in zip(captured, want)) and torch.equal(pool, eager)
        seen.add(tuple(want[2].tolist() + want[5].tolist()))
    assert len(seen) > 1      # (other numbers of accepted tokens)
