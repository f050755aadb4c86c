"""The norm's sums where they are long or not finite: dgain of many rows, whose error may
not grow with their number, and rows that hold an infinity."""
import pytest
import torch

import shared_matrix_expert_amd as em
from gpu_helpers import DEV, say
from test_gpu_norm import TYPES, run_backward

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

U = 2.0 ** -24
# Roundings of a term of dgain: v's and the product's, two of the sum over a workgroup's
# rows, one of the workgroup's sum, one of dgain.
TERM = 6 * U


@pytest.mark.parametrize("T,d", [(1 << 20, 8), (1 << 18, 512), (1 << 17, 1024), (1 << 17, 2048), (1 << 16, 4096), (1 << 15, 8192),
                                 (1 << 14, 16384), (1 << 13, 32768)])
def test_dgain_of_equal_rows(T, d):
    """Equal terms, whose float32 sum loses the same part of each row again and again: one
    part for every length of the sum, by column."""
    say(f"case: dgain of {T} equal rows of {d}")
    x, gain, rstd = torch.ones(T, d, dtype=torch.bfloat16, device=DEV), torch.ones(d, device=DEV), torch.ones(T, device=DEV)
    part = 0.4 * torch.exp2(-(torch.arange(d, device=DEV) % 8 + 13).float())
    dy = (1 + part).expand(T, d).contiguous()
    dgain = torch.empty(d, device=DEV)
    run_backward(x, gain, rstd, dy, dgain=dgain)
    want = T * (1 + part).double()
    assert bool(((dgain.double() - want).abs() <= TERM * want).all())


@pytest.mark.parametrize("grad", list(TYPES))
@pytest.mark.parametrize("T,d", [(262147, 64), (100003, 1000), (65539, 2056), (16385, 8200), (9001, 16392)])
def test_dgain_of_many_rows(T, d, grad):
    say(f"case: dgain of {T} rows of {d}, {grad}")
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
    dy = (1 + torch.rand(T, d, generator=g, device=DEV)).to(TYPES[grad]) * x.sign().to(TYPES[grad])      # terms of one sign
    gain, rstd, dgain = torch.ones(d, device=DEV), torch.rand(T, generator=g, device=DEV) + 0.5, torch.empty(d, device=DEV)
    run_backward(x, gain, rstd, dy, dgain=dgain)
    want = torch.zeros(d, dtype=torch.float64, device=DEV)
    for i in range(0, T, 8192):
        want += (dy[i:i + 8192].double() * x[i:i + 8192].double() * rstd[i:i + 8192, None].double()).sum(0)
    assert bool(((dgain.double() - want).abs() <= TERM * want).all())
