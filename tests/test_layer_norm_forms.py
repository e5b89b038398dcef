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


@pytest.mark.parametrize("T,C", [(700013, 96), (131101, 512), (67211, 1000), (33001, 2048), (16411, 4096), (11003, 6144),
                                 (8209, 8192), (5501, 12288), (4099, 16384), (2803, 24000), (2051, 32768)])
def test_rows_past_the_caches(T, C):
    """The bits of a few of the rows by themselves, whose values a cache holds, and the sums over all of them
    against 64 bits (a thread adds T / 256 rows in turn at most, the second kernel and the rows of a workgroup 24
    more: 2^-24 of the terms' sizes each, and 2^-20 for h)."""
    import gated_delta_rule_32_amd as kda
    print(f"[lnorm] {T} {C}", flush=True)
    x, w, b, dy = rows_of(T, C, C)
    assert T * C * 4 > 2 ** 28
    y, (dx, dw, db) = kda.layer_norm_forward(x, w, b), kda.layer_norm_backward(dy, x, w)
    for r in (slice(0, 37), slice(T // 2, T // 2 + 37), slice(T - 37, T)):
        assert torch.equal(kda.layer_norm_forward(x[r], w, b), y[r])
        assert torch.equal(kda.layer_norm_backward(dy[r], x[r], w)[0], dx[r])
    sum_w, sum_b, terms_w, terms_b = (torch.zeros(C, dtype=torch.float64, device="cuda") for _ in range(4))
    step = 2 ** 24 // C
    for i in range(0, T, step):
        x64, d64 = x[i:i + step].double(), dy[i:i + step].double()
        c = x64 - x64.mean(-1, keepdim=True)
        r = torch.rsqrt((c * c).mean(-1, keepdim=True) + 1e-5)
        h = c * r
        sum_w += (d64 * h).sum(0)
        sum_b += d64.sum(0)
        terms_w += (d64 * h).abs().sum(0)
        terms_b += d64.abs().sum(0)
        # every row's result: one rounding, and 2^-19 and 2^-18 of its terms' sizes (a normal row's are below 6)
        ref = h * w + b
        assert ((y[i:i + step].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -19 * 12 * (w.abs() + b.abs())).all()
        d = d64 * w
        ref = r * (d - d.mean(-1, keepdim=True) - h * (d * h).mean(-1, keepdim=True))
        bar = 2.0 ** -8 * ref.abs() + 2.0 ** -18 * r * (d.abs() + 8 * w.abs().mean())
        assert ((dx[i:i + step].double() - ref).abs() <= bar).all()
    bar = 2.0 ** -24 * (T / 256 + 24)
    assert ((dw - sum_w).abs() <= (bar + 2.0 ** -20) * terms_w).all()
    assert ((db - sum_b).abs() <= bar * terms_b).all()


def test_more_rows_than_a_launch_of_wide_workgroups_takes_at_once():
    """Workgroups of 1024 threads walk over the rows behind the first 2^16."""
    import gated_delta_rule_32_amd as kda
    T, C = 2 ** 16 + 301, 12296
    x, w, b, _ = rows_of(T, C, 5)
    y = kda.layer_norm_forward(x, w, b)
    for at in (0, 250, 2 ** 16 - 40, T - 40):
        assert torch.equal(kda.layer_norm_forward(x[at:at + 40], w, b), y[at:at + 40])
