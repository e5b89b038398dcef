"""GPU tests of the layer norm's forms for rows that go past the caches: every number of threads a row,
with rows that end a walk unevenly."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def rows_of(T, C, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, dy = (torch.randn((T, C), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w, b = (torch.randn(C, generator=g, device="cuda") for _ in range(2))
    return x, w, b, dy


def test_more_rows_than_a_launch_of_wide_workgroups_takes_at_once():
    """Workgroups of 1024 threads walk over the rows behind the first 2^16."""
    import gated_delta_rule_32_amd as kda
    T, C = 2 ** 16 + 301, 12296
    x, w, b, _ = rows_of(T, C, 5)
    y = kda.layer_norm_forward(x, w, b)
    for at in (0, 250, 2 ** 16 - 40, T - 40):
        assert torch.equal(kda.layer_norm_forward(x[at:at + 40], w, b), y[at:at + 40])
