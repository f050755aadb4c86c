"""The MX-matrix and router-training operators at the smallest and largest sizes of
each dimension that they take."""
import numpy as np
import pytest
import torch

import shared_matrix_expert_amd as em
from oracle import operators as ops
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from test_gpu_mx_matrices import check_quantize, fmt_of, i32, matrices, product, rows_of, within  # noqa: E402
from test_gpu_router_train import case, check_backward, check_balance, dims  # noqa: E402


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (33, 1, 1), (1, 2, 2), (40, 3, 3), (9, 5, 4), (2100, 2, 1), (2500, 40, 32),
                                   (4200, 1, 1), (4200, 3, 2), (4500, 1024, 32), (1, 1024, 32)])
def test_router_experts_and_picks(T, E, k):
    say(f"case: router {T} x {E}, top {k}")
    z, idx, *_ = case(T, E, k, T)
    check_balance(dims(T, E, k), z, idx)
    check_backward(T, E, k, 128)


@pytest.mark.parametrize("T,E,d", [(5, 9, 32768), (300, 64, 32768), (1, 1024, 8192)])
def test_router_widths(T, E, d):
    say(f"case: backward {T} x {E} x {d}")
    check_backward(T, E, 2, d)


@fmt_of
@pytest.mark.parametrize("M,R", [(513, 40), (1024, 1500), (1024, 9000), (700, 60000)])
def test_product_matrices(fmt, M, R):
    """Up to 1024 matrices, empty ones among them, by both kernels; rows of none kept."""
    N, K = 24, 128
    say(f"case: {M} matrices, {R} rows")
    rng = np.random.default_rng(R)
    off = np.sort(rng.integers(1, R, M + 1))
    T = 300
    src = rng.integers(0, T, R)
    q, e, W = matrices(M, N, K, M)
    x = rows_of(T, K, 5)
    y = torch.full((R, N), 3.25, dtype=torch.bfloat16, device=DEV)
    product(fmt, x.to(DEV), q, e, y, offsets=i32(off), row_src=i32(src))
    within(y, *ops.product(x.double().numpy(), fmt, W, off, src), K)
    assert bool((y[:off[0]] == 3.25).all()) and bool((y[off[-1]:] == 3.25).all())


@fmt_of
@pytest.mark.parametrize("T,N,K", [(1, 24, 32768), (20, 40, 32768), (70, 24, 32768), (300, 24, 32768), (3, 32768, 128),
                                   (100, 32768, 128), (600, 32767, 128)])
def test_product_widths(fmt, T, N, K):
    say(f"case: {T} x {N} x {K}")
    q, e, W = matrices(1, N, K, T)
    x = rows_of(T, K, N)
    y = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    product(fmt, x.to(DEV), q, e, y)
    within(y, *ops.product(x.double().numpy(), fmt, W), K)


@fmt_of
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rounding_widths(fmt, dtype):
    src = torch.randn(2, 3, 32768, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(dtype)
    codes, scales = check_quantize(fmt, src)
    dst = torch.empty_like(src)
    em.edge_moe_mx_dequantize(fmt, codes, scales, dst)
    want = torch.from_numpy(ops.rounded(src.float().cpu().numpy().astype(np.float64), fmt)).to(dtype)
    assert torch.equal(dst.cpu(), want)


@fmt_of
def test_no_rows(fmt):
    """R = 0: nothing is written, with and without groups."""
    q, e, _ = matrices(2, 40, 256, 1)
    x = rows_of(4, 256, 1).to(DEV)
    y = torch.empty(0, 40, dtype=torch.bfloat16, device=DEV)
    product(fmt, x, q, e, y, offsets=i32([0, 0, 0]))
    product(fmt, x, q[:1].contiguous(), e[:1].contiguous(), y, row_src=i32([]))
