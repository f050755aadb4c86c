"""The norm's sums where they are not finite: rows that hold an infinity."""
import pytest
import torch

import shared_matrix_expert_amd as em
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.mark.parametrize("d", [128, 1024, 4096, 16384, 32768])
def test_rows_with_an_infinity(d):
    """1 / sqrt(infinity) is zero: NaN where the infinity is, zeros beside it."""
    g = torch.Generator(device=DEV).manual_seed(d)
    x = torch.randn(9, d, generator=g, device=DEV).to(torch.bfloat16)
    x[2, 5], x[4, d - 1], x[6, 1], x[6, 2] = float("inf"), float("-inf"), float("inf"), float("nan")
    add = torch.zeros(9, d, device=DEV)
    add[7, 3] = float("inf")
    y, rstd = torch.empty_like(x), torch.empty(9, device=DEV)
    codes, scales = torch.empty(9, d, dtype=torch.uint8, device=DEV), torch.empty(d // 128, 9, 4, dtype=torch.uint8, device=DEV)
    em.edge_moe_norm(x, torch.ones(d, device=DEV), 1e-5, add=add, y=y, codes=codes, scales=scales, rstd=rstd)
    back = torch.empty(9, d, device=DEV)
    em.edge_moe_mx_dequantize(em.MX_FP8, codes, scales, back)
    for row, at in ((2, 5), (4, d - 1), (7, 3)):
        assert float(rstd[row]) == 0
        here = torch.arange(d, device=DEV) == at
        assert bool(y[row, here].isnan().all()) and bool((y[row, ~here] == 0).all())
        block = torch.arange(d, device=DEV) // 32 == at // 32
        assert bool(back[row, block].isnan().all()) and bool((back[row, ~block] == 0).all())
    assert bool(rstd[6].isnan()) and bool(y[6].isnan().all())
    ok = [0, 1, 3, 5, 8]
    assert bool(rstd[ok].isfinite().all()) and bool(y[ok].isfinite().all())
