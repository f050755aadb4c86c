"""Workspace of the dense product's gradients (no GPU needed): the size that a caller asks
for with the tokens of its batch also holds a call for dx by rows, which names no tokens
(the binding passes one)."""
import shared_matrix_expert_amd as em


def test_rows_need_no_more_than_tokens_do():
    less = []
    for M in (1, 2, 8, 64, 128, 129, 512):
        for N in (8, 16, 128, 1024, 8192):
            for K in (8, 64, 520, 4096, 16384, 32768):
                for R in (0, 1, 20, 300, 2000, 50000, 1 << 20):
                    one = em.edge_moe_dense_product_backward_ws_bytes(1, R, M, N, K)
                    for T in (1, 17, 1000, 4096, 1 << 18, 1 << 20):
                        if em.edge_moe_dense_product_backward_ws_bytes(T, R, M, N, K) < one:
                            less.append((T, R, M, N, K))
    assert not less, f"{len(less)}: {less[:8]}"
