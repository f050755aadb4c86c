"""Calls of more work than one launch holds (2^32 threads in a dimension, 65536 workgroups
in the second one)."""
import pytest
import torch

import shared_matrix_expert_amd as em
from gpu_helpers import DEV, say
from test_gpu_dense_product import GUARD, product, same, whole, workspace
from test_gpu_norm import U, half
from test_gpu_packed_product import matrices

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


def test_few_rows_of_more_tokens_than_a_launch_holds():
    """2^20 tokens' dx of 16384 columns, 2^32 threads in one launch, from 2000 rows."""
    g = torch.Generator(device=DEV).manual_seed(3)
    T, R, M, N, K = 1 << 20, 2000, 3, 408, 16384
    off = [0, 700, 1300, R]
    w, dy = whole(g, M, N, K), whole(g, R, N)
    token_rows = torch.full((T, 2), -1, dtype=torch.int32, device=DEV)
    tokens = torch.randperm(T, generator=g, device=DEV)[:R]
    tokens[0], tokens[1] = T - 1, tokens[2]                      # the last token; one with two rows
    token_rows[tokens, torch.arange(R, device=DEV) % 2] = torch.arange(R, dtype=torch.int32, device=DEV)
    rows = torch.cat([dy[a:b].double() @ w[m].double() for m, (a, b) in enumerate(zip(off, off[1:]))])
    dx = torch.full((T, K), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = workspace(em.edge_moe_dense_product_backward_ws_bytes(T, R, M, N, K))
    em.edge_moe_dense_product_backward(dy, ws[:-GUARD], w=w, dx=dx, offsets=torch.tensor(off, dtype=torch.int32, device=DEV),
                                       token_rows=token_rows)
    assert bool((ws[-GUARD:] == 0xA5).all())
    live = (token_rows >= 0).any(1)
    named = token_rows[live].long()
    want = (rows[named.clamp(min=0)] * (named >= 0).unsqueeze(-1)).sum(1)
    same(dx[live], want)
    for i in range(0, T, 1 << 16):
        assert not bool(dx[i:i + (1 << 16)][~live[i:i + (1 << 16)]].any())


def test_int4_rows_past_a_grids_second_dimension():
    """More than 65536 tiles of 16 and of 64 rows, in a matrix and in three of them."""
    g = torch.Generator(device=DEV).manual_seed(4)
    T, K = 4096, 64
    x = whole(g, T, K)
    for R, N, q in (((1 << 22) + 77, 8, 32), ((1 << 22) + 77, 3, 64)):
        src = torch.randint(-1, T, (R,), generator=g, device=DEV, dtype=torch.int32)
        for off in ([0, R], [5, 17, R // 2 + 3, R - 2]):
            M = len(off) - 1
            codes, scales, w = matrices(g, M, N, K, q)
            y = torch.full((R, N), 7.0, device=DEV)
            ws = workspace(em.edge_moe_packed_product_ws_bytes(T, R, M, N, K, q))
            em.edge_moe_packed_product(q, x, codes, scales, y, ws[:-GUARD], offsets=torch.tensor(off, dtype=torch.int32, device=DEV),
                                       row_src=src)
            assert bool((ws[-GUARD:] == 0xA5).all())
            same(y, product(x, w, off, src, R), (off[0], off[-1]))
