"""The MX-matrix and router-training operators in one run beside the layer they
serve, on one side stream and one workspace: dense weights are quantised, a batch
is routed and run through edge_moe_forward_mx, the routed rows go through the
experts' MX product with the layer's own permutation, and the router is
differentiated through its weights (from the layer's expert outputs), its balance
and its z loss.  Each step is held to the float64 oracle on that step's inputs."""
import numpy as np
import pytest
import torch

import shared_matrix_expert_amd as em
import synth
from oracle import operators as ops
from oracle.codecs import bf16_to_f64
from gpu_helpers import DEV, bits_to_dev, say
from test_gpu_mx_matrices import within
from test_gpu_router_train import LOAD, U

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.mark.parametrize("T", [96, 1, 200])
def test_quantise_route_forward_product_and_gradients(T):
    D = synth.config(5).dims.with_T(T)
    E, k, d, r = D.n_experts, D.top_k, D.d, D.delta_rank
    g = torch.Generator(device=DEV).manual_seed(11)
    dense = {n: (torch.randn(*s, generator=g, device=DEV) * synth.WEIGHT_STD).to(torch.bfloat16) for n, s in
             (("s_up", (D.n_groups, D.h, d)), ("s_dn", (D.n_groups, d, D.h)), ("a_up", (E, r, d)), ("b_up", (E, D.h, r)),
              ("a_dn", (E, r, D.h)), ("b_dn", (E, d, r)), ("lora_up_u", (D.n_groups, D.lora_rank, d)),
              ("lora_up_v", (D.n_groups, D.h, D.lora_rank)), ("lora_dn_u", (D.n_groups, D.lora_rank, D.h)),
              ("lora_dn_v", (D.n_groups, d, D.lora_rank)))}
    x = bits_to_dev(synth.make_activations(5, 3, T=T))
    wr = bits_to_dev(synth.make_router(5, 3)[0])
    R, S = T * k, 3
    off = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32, device=DEV)       # an empty sequence
    ws = torch.empty(max(em.edge_moe_workspace_bytes(D), em.edge_moe_workspace_bytes_mx(D),
                         em.edge_moe_mx_product_ws_bytes(T, R, E, r, d, em.MX_FP8), em.edge_moe_balance_ws_bytes(D, S),
                         em.edge_moe_route_backward_ws_bytes(D)), dtype=torch.uint8, device=DEV)

    def f32(*s):
        return torch.full(s, float("nan"), device=DEV)

    def i32(*s):
        return torch.full(s, -1, dtype=torch.int32, device=DEV)
    idx, w, logits, y = i32(T, k), f32(T, k), f32(T, E), f32(T, d)
    tr = {"expert_offsets": i32(E + 1), "row_token": i32(R), "row_slot": i32(R), "expert_out": f32(R, d)}
    z1 = torch.full((R, r), float("nan"), dtype=torch.bfloat16, device=DEV)
    counts, probs, loss = i32(S, E), f32(S, E), f32(2)
    dlogits, dx, dwr, dbias = f32(T, E), f32(T, d), f32(E, d), f32(E)
    dy = torch.randn(T, d, generator=g, device=DEV)
    d_loss = torch.tensor([0.5, 0.1], device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        W = em.mx_weights(dense)
        em.edge_moe_route(D, x, wr, None, idx, w, logits, ws)
        em.edge_moe_forward_mx(D, x, idx, w, W, y, ws, trace=tr)
        em.edge_moe_mx_product(em.MX_FP8, x, W["a_up"], W["a_up_scale"], z1, ws, offsets=tr["expert_offsets"],
                               row_src=tr["row_token"])
        dw = (dy.unsqueeze(1) * tr["expert_out"].view(T, k, d)).sum(-1)              # y = sum_j w_j o_j
        em.edge_moe_balance(D, logits, idx, counts, probs, loss, ws, seq_offsets=off)
        em.edge_moe_route_backward(D, logits, idx, ws, topk_w=w, d_topk_w=dw, d_loss=d_loss, counts=counts, seq_offsets=off,
                                   x=x, w_router=wr, dlogits=dlogits, dx=dx, dw_router=dwr, dbias=dbias)
    s.synchronize()

    def host(t):
        return t.cpu().numpy().astype(np.float64)
    # the product, on the layer's own permutation and the quantised matrices' values
    a_up = ops.rounded(dense["a_up"].float().cpu().numpy().astype(np.float64), ops.FP4)
    xv = bf16_to_f64(x.cpu().numpy().view(np.uint16))
    within(z1, *ops.product(xv, ops.FP8, a_up, tr["expert_offsets"].cpu().numpy(), tr["row_token"].cpu().numpy()), d)
    # load and losses
    zc, ic, oc = host(logits), idx.cpu().numpy(), off.cpu().numpy()
    cr, pr, lr = ops.balance(zc, ic, oc)
    assert np.array_equal(counts.cpu().numpy(), cr) and cr.sum() == R
    assert np.all(np.abs(host(probs) - pr) <= LOAD * pr + 1e-40)
    assert np.all(np.abs(host(loss) - lr) <= LOAD * np.abs(lr) + 1e-40)
    # gradients
    dz, mag = ops.route_backward(zc, ic, host(w), host(dw), [0.5, 0.1], cr, oc)
    tz = 2.5 * LOAD * mag + 1e-40
    assert np.all(np.abs(host(dlogits) - dz) <= tz)
    wv = bf16_to_f64(wr.cpu().numpy().view(np.uint16))
    for got, a, b, ta, K in ((dx, dz, wv, tz, E), (dwr, dz.T, xv, tz.T, T)):
        tol = ta @ np.abs(b) + (2 * 3 * (K // 32 + 1) + 8) * U * (np.abs(a) @ np.abs(b)) + 1e-40
        assert np.all(np.abs(host(got) - a @ b) <= tol)
    assert np.all(np.abs(host(dbias) - dz.sum(0)) <= tz.sum(0) + 8 * U * np.abs(dz).sum(0) + 1e-40)
    say(f"  {T} tokens: balance {lr[0]:.4f}, z {lr[1]:.3f}, |dx| {np.abs(dz @ wv).max():.3g}")
