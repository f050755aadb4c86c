"""The MX-matrix and router-training operators at the edges of their ranges: block
scales far from 1 on both sides of a product, results down to bf16's subnormals;
two calls at once; a padded batch."""
import numpy as np
import pytest
import torch

import shared_matrix_expert_amd as em
from oracle import operators as ops
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from test_gpu_mx_matrices import fmt_of, i32, matrices, product, rows_of, within  # noqa: E402
from test_gpu_router_train import ALL, LOAD, U, case, dev, dims, run_backward  # noqa: E402


@fmt_of
@pytest.mark.parametrize("T", [3, 70, 400])
@pytest.mark.parametrize("x_exp,w_exp", [(100, -100), (-118, 60), (-126, 20), (120, -120), (-110, -27), (0, -127), (20, 93)])
def test_product_scales(fmt, T, x_exp, w_exp):
    """x about 2^x_exp, W's blocks 2^(w_exp - 2) to 2^(w_exp + 2) (limited to the
    format's): only the sum of the exponents shows in y."""
    N, K = 40, 256
    rng = np.random.default_rng(T)
    codes = rng.integers(0, 16, (1, N, K), dtype=np.uint8)
    x8 = np.clip(rng.integers(w_exp + 125, w_exp + 130, (1, N, K // 32)), 0, 254).astype(np.uint8)
    q, e = torch.from_numpy(ops.pack(codes, ops.FP4)).to(DEV), torch.from_numpy(ops.by_step(x8)).to(DEV)
    x = (rows_of(T, K, T).double() * 2.0 ** x_exp).to(torch.bfloat16)
    y = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    say(f"case: {T} rows, x 2^{x_exp}, W 2^{w_exp}")
    product(fmt, x.to(DEV), q, e, y)
    within(y, *ops.product(x.double().numpy(), fmt, ops.values(codes, x8, ops.FP4)), K)


def test_two_calls_at_once():
    """Each of two streams has its workspace and outputs: the bits of a call alone."""
    T, E, k, d = 1500, 128, 4, 1024
    z, idx, w, dw, x, wr = case(T, E, k, 2, d)
    D = dims(T, E, k, d)
    q, e, _ = matrices(3, 1024, d, 3)
    off, src = i32([0, 500, 510, 1500]), i32(np.random.default_rng(0).integers(0, T, T))
    zd, idxd, wd, dwd, xd, wrd, g = dev(z), dev(idx), dev(w), dev(dw), x.to(DEV), wr.to(DEV), dev(np.array([0.5, 0.1], np.float32))

    def buffers():
        b = {n: torch.zeros(s, device=DEV) for n, s in
             (("probs", (1, E)), ("loss", (2,)), ("dlogits", (T, E)), ("dx", (T, d)), ("dw_router", (E, d)), ("dbias", (E,)))}
        b["counts"] = torch.zeros(1, E, dtype=torch.int32, device=DEV)
        b["y"] = torch.zeros(T, 1024, dtype=torch.bfloat16, device=DEV)
        b["ws"] = torch.empty(max(em.edge_moe_balance_ws_bytes(D, 1), em.edge_moe_route_backward_ws_bytes(D),
                                  em.edge_moe_mx_product_ws_bytes(T, T, 3, 1024, d, em.MX_FP8)), dtype=torch.uint8, device=DEV)
        return b

    def step(b, stream=None):
        em.edge_moe_balance(D, zd, idxd, b["counts"], b["probs"], b["loss"], b["ws"], stream=stream)
        em.edge_moe_mx_product(em.MX_FP8, xd, q, e, b["y"], b["ws"], offsets=off, row_src=src, stream=stream)
        em.edge_moe_route_backward(D, zd, idxd, b["ws"], topk_w=wd, d_topk_w=dwd, d_loss=g, counts=b["counts"], x=xd,
                                   w_router=wrd, stream=stream, **{n: b[n] for n in ALL})
    alone, both, streams = buffers(), [buffers(), buffers()], [torch.cuda.Stream(), torch.cuda.Stream()]
    step(alone)
    torch.cuda.synchronize()
    for _ in range(10):
        for b, s in zip(both, streams):
            step(b, s)
    torch.cuda.synchronize()
    for b in both:
        assert all(torch.equal(b[n], alone[n]) for n in alone if n != "ws")


@pytest.mark.parametrize("T,E", [(60, 30), (4700, 64)])
def test_padded_batch(T, E):
    """Tokens behind the last sequence (NaN logits, out-of-range picks, no gradient
    at their weights) leave losses and gradients as they are without them."""
    k, d, live = 3, 128, T - 13
    z, idx, w, dw, x, wr = case(T, E, k, 9, d)
    off = [0, live // 3, live]
    z[live:], idx[live:], dw[live:] = np.nan, -1, 0
    g = np.array([0.6, -0.2], np.float32)
    counts, probs, loss = torch.empty(2, E, dtype=torch.int32, device=DEV), torch.empty(2, E, device=DEV), torch.empty(2, device=DEV)
    D = dims(T, E, k, d)
    ws = torch.empty(em.edge_moe_balance_ws_bytes(D, 2), dtype=torch.uint8, device=DEV)
    em.edge_moe_balance(D, dev(z), dev(idx), counts, probs, loss, ws, seq_offsets=i32(off))
    c, p, L = ops.balance(z[:live], idx[:live], off)
    assert np.array_equal(counts.cpu().numpy(), c)
    assert np.all(np.abs(probs.cpu().numpy() - p) <= LOAD * p + 1e-40)
    assert np.all(np.abs(loss.cpu().numpy() - L) <= LOAD * L + 1e-40)
    out = run_backward(D, z, idx, want=ALL, dirty=True, topk_w=dev(w), d_topk_w=dev(dw), d_loss=dev(g), counts=counts,
                       seq_offsets=i32(off), x=x.to(DEV), w_router=wr.to(DEV))
    dz, mag = ops.route_backward(z[:live], idx[:live], w[:live], dw[:live], g, c, off)
    tz = 2.5 * LOAD * mag + 1e-40
    assert np.all(np.abs(out["dlogits"][:live].cpu().numpy() - dz) <= tz)
    assert not bool(out["dlogits"][live:].any()) and not bool(out["dx"][live:].any())
    xs = x[:live].double().numpy()
    tol = tz.T @ np.abs(xs) + (6 * (T // 32 + 1) + 8) * U * (np.abs(dz.T) @ np.abs(xs)) + 1e-40
    assert np.all(np.abs(out["dw_router"].cpu().numpy() - dz.T @ xs) <= tol)
    assert np.all(np.abs(out["dbias"].cpu().numpy() - dz.sum(0)) <= tz.sum(0) + 8 * U * np.abs(dz).sum(0) + 1e-40)
