"""The MX-matrix and router-training operators on buffers past 2^31 elements or
2^32 bytes: the last rows are those of the same call on these rows alone (each
row's arithmetic is the same), or the float64 oracle's.
"""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import shared_matrix_expert_amd as em
from oracle import operators as ops
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from test_gpu_mx_matrices import matrices, product, within  # noqa: E402  (skipped there too without a GPU)

U = 2.0 ** -24
TAIL = 45


def filled(rows, K, tail, seed):
    """bf16 [rows][K], zeros but for the last rows."""
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    x[-tail:] = torch.randn(tail, K, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(torch.bfloat16)
    return x


@pytest.mark.parametrize("fmt", [em.MX_FP4, em.MX_FP8], ids=["fp4", "fp8"])
def test_round(fmt):
    N, K = (1 << 20) + 21, 4224                       # 2^32.04 elements
    say(f"case: round {N} x {K}")
    x = filled(N, K, TAIL, 1)
    per = K // 2 if fmt == em.MX_FP4 else K
    codes = torch.full((N, per), 0x55, dtype=torch.uint8, device=DEV)
    scales = torch.full((K // 128, N, 4), 0x55, dtype=torch.uint8, device=DEV)
    em.edge_moe_mx_quantize(fmt, x, codes, scales)
    q = torch.empty(TAIL, per, dtype=torch.uint8, device=DEV)
    e = torch.empty(K // 128, TAIL, 4, dtype=torch.uint8, device=DEV)
    em.edge_moe_mx_quantize(fmt, x[-TAIL:], q, e)
    assert torch.equal(codes[-TAIL:], q) and torch.equal(scales[:, -TAIL:], e)
    assert not bool(codes[:-TAIL].any()) and not bool(scales[:, :-TAIL].any())
    back = torch.full((N, K), 3.0, dtype=torch.bfloat16, device=DEV)
    em.edge_moe_mx_dequantize(fmt, codes, scales, back)
    one = torch.empty(TAIL, K, dtype=torch.bfloat16, device=DEV)
    em.edge_moe_mx_dequantize(fmt, q, e, one)
    assert torch.equal(back[-TAIL:], one) and not bool(back[:-TAIL].any())


@pytest.mark.parametrize("T,N,K,R", [(300000, 8192, 128, 300000), (1 << 20, 256, 4224, 1 << 20), (1 << 20, 256, 4224, TAIL)])
def test_product(T, N, K, R):
    """Long y, long x, and a few gathered rows of a long x."""
    say(f"case: product {R} rows of {T} x {N} x {K}")
    q, e, W = matrices(1, N, K, 2)
    x = filled(T, K, TAIL, 3)
    y = torch.full((R, N), 3.0, dtype=torch.bfloat16, device=DEV)
    src = torch.arange(T - TAIL, T, dtype=torch.int32, device=DEV) if R == TAIL else None
    product(em.MX_FP8, x, q, e, y, row_src=src)
    within(y[-TAIL:], *ops.product(x[-TAIL:].double().cpu().numpy(), em.MX_FP8, W), K)
    assert not bool(y[:-TAIL].any())


def test_router():
    T, E, k, d = 1 << 20, 1024, 4, 1024               # logits, dlogits and dx of 2^32 bytes
    D = SimpleNamespace(T=T, d=d, h=128, n_experts=E, experts_per_group=E, top_k=k, delta_rank=8, lora_rank=2,
                        quant_group=32)
    say(f"case: router {T} x {E} x {d}")
    g = torch.Generator(device=DEV).manual_seed(4)
    z = torch.zeros(T, E, device=DEV)
    z[-TAIL:] = 2 * torch.randn(TAIL, E, generator=g, device=DEV)
    idx = torch.zeros(T, k, dtype=torch.int32, device=DEV)
    idx[-TAIL:] = z[-TAIL:].topk(k, 1).indices.int()
    off = torch.tensor([T - TAIL, T], dtype=torch.int32, device=DEV)
    counts = torch.empty(1, E, dtype=torch.int32, device=DEV)
    probs, loss = torch.empty(1, E, device=DEV), torch.empty(2, device=DEV)
    ws = torch.empty(max(em.edge_moe_balance_ws_bytes(D, 1), em.edge_moe_route_backward_ws_bytes(D)), dtype=torch.uint8,
                     device=DEV)
    em.edge_moe_balance(D, z, idx, counts, probs, loss, ws, seq_offsets=off)
    zt, it = z[-TAIL:].cpu().numpy(), idx[-TAIL:].cpu().numpy()
    c, p, L = ops.balance(zt, it)
    assert np.array_equal(counts.cpu().numpy(), c)
    assert np.all(np.abs(probs.cpu().numpy() - p) <= 100 * U * p)
    x = filled(T, d, TAIL, 5)
    wr = torch.randn(E, d, generator=g, device=DEV).to(torch.bfloat16)
    out = {n: torch.full(s, float("nan"), device=DEV) for n, s in
           (("dlogits", (T, E)), ("dx", (T, d)), ("dw_router", (E, d)), ("dbias", (E,)))}
    dl = torch.tensor([0.6, -0.2], device=DEV)
    em.edge_moe_route_backward(D, z, idx, ws, d_loss=dl, counts=counts, seq_offsets=off, x=x, w_router=wr, **out)
    dz, mag = ops.route_backward(zt, it, d_loss=np.array([0.6, -0.2], np.float32), counts=c)
    tz = 250 * U * mag + 1e-40                        # the bounds of the small shapes' tests
    assert np.all(np.abs(out["dlogits"][-TAIL:].cpu().numpy() - dz) <= tz)
    xs, w = x[-TAIL:].double().cpu().numpy(), wr.double().cpu().numpy()
    for got, a, b, ta, K in ((out["dx"][-TAIL:], dz, w, tz, E), (out["dw_router"], dz.T, xs, tz.T, T)):
        # T - TAIL of dW_r's terms are zeros: only their sums' additions count, and those are exact
        n = 3 * (min(K, 2048) // 32 + 1)
        tol = ta @ np.abs(b) + (2 * n + 8) * U * (np.abs(a) @ np.abs(b)) + 1e-40
        assert np.all(np.abs(got.cpu().numpy() - a @ b) <= tol)
    assert not bool(out["dlogits"][:-TAIL].any()) and not bool(out["dx"][:-TAIL].any())
