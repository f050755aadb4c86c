"""Calls of more work than one launch holds (2^32 threads in a dimension)."""
import pytest
import torch

import shared_matrix_expert_amd as em
from gpu_helpers import DEV, say
from test_gpu_norm import U, half

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.mark.parametrize("T,d", [(1 << 25, 1032), ((1 << 22) + 5, 8200)])
def test_norm_of_more_rows_than_a_launch_holds(T, d):
    """61 different rows again and again: each of them has its rstd and its y."""
    say(f"case: norm of {T} x {d}")
    g = torch.Generator(device=DEV).manual_seed(d)
    rows = torch.randn(61, d, generator=g, device=DEV).to(torch.bfloat16)
    n = T // 61
    x = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    x[:n * 61].view(n, 61, d).copy_(rows.expand(n, 61, d))
    x[n * 61:] = rows[:T - n * 61]
    y, rstd = torch.empty_like(x), torch.empty(T, device=DEV)
    gain = torch.ones(d, device=DEV)
    em.edge_moe_norm(x, gain, 1e-5, y=y, rstd=rstd)
    want = 1 / torch.sqrt(rows.double().square().mean(1) + 1e-5)
    every = want.expand(n + 1, 61).reshape(-1)[:T]
    assert bool(((rstd.double() - every).abs() <= 1.01 * U * every).all())
    del x
    ys = rows.double() * want[:, None]
    seen = [y[:n * 61].view(n, 61, d)[i] for i in range(0, n, n // 400)] + [y[(n - 1) * 61:n * 61]]
    for got in seen:
        assert bool(((got.double() - ys).abs() <= (half(torch.bfloat16) + 4 * U) * ys.abs() + 2.0 ** -134).all())
    assert torch.equal(y[n * 61:], y[:T - n * 61])
