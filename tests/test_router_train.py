"""Host-side checks of the router-training operators (no GPU needed): the
oracle's gradient against differences of its own losses and weights, closed
forms, the library's refusals before any device call, the binding's checks."""
import ctypes
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import shared_matrix_expert_amd as em
from oracle import operators as ops

BASE = 1 << 40                                  # never dereferenced


def dims(T, E, k, d=128):
    return SimpleNamespace(T=T, d=d, h=128, n_experts=E, experts_per_group=E, top_k=k, delta_rank=8, lora_rank=2,
                           quant_group=32)


# ------------------------------------------------------------------ the oracle ----

def test_balance_closed_forms():
    # uniform logits, every expert picked equally often: loss 1, z = log(E)^2
    idx = np.array([[0, 1], [2, 3]])
    c, p, loss = ops.balance(np.zeros((2, 4)), idx)
    assert c.tolist() == [[1, 1, 1, 1]] and np.allclose(p, 0.25)
    assert np.isclose(loss[0], 1.0) and np.isclose(loss[1], np.log(4) ** 2)
    # all the weight and all the picks on one expert: E
    z = np.full((3, 4), -np.inf)
    z[:, 2] = 1.5
    c, p, loss = ops.balance(z, np.full((3, 1), 2))
    assert np.isclose(loss[0], 4.0) and np.isclose(loss[1], 2.25)
    # dropped slots, an empty sequence, tokens in no sequence, a token without a distribution
    z = np.zeros((4, 4))
    z[1] = -np.inf
    c, p, loss = ops.balance(z, np.array([[0], [-1], [9], [1]]), [0, 0, 2])
    assert c.tolist() == [[0] * 4, [1, 0, 0, 0]] and np.allclose(p[1], 0.125)
    assert np.isclose(loss[0], 4 / 2 * 0.125) and np.isclose(loss[1], np.log(4) ** 2 / 2)
    assert ops.balance(np.zeros((2, 4)), np.zeros((2, 1), int), [1, 1])[2].tolist() == [0, 0]


def test_gradient_against_differences():
    rng = np.random.default_rng(0)
    T, E, k, off = 7, 6, 2, [0, 3, 3, 6]                       # an empty sequence, a token in none
    z = rng.standard_normal((T, E))
    idx = np.argsort(-z, 1)[:, :k]
    dw, g = rng.standard_normal((T, k)), np.array([0.7, -0.3])
    counts = ops.balance(z, idx, off)[0]

    def weights(z):
        s = np.take_along_axis(z, idx, 1)
        e = np.exp(s - s.max(1, keepdims=True))
        return e / e.sum(1, keepdims=True)

    def objective(z):                                          # the counts and the selection are constants
        return (weights(z) * dw).sum() + g @ ops.balance(z, idx, off)[2]
    dz, mag = ops.route_backward(z, idx, weights(z), dw, g, counts, off)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            up, dn = z.copy(), z.copy()
            up[t, e] += h
            dn[t, e] -= h
            assert abs((objective(up) - objective(dn)) / (2 * h) - dz[t, e]) < 1e-8 + 1e-8 * mag[t, e]
    assert np.all(np.abs(dz) <= mag + 1e-15)


# ------------------------------------------------------------------ refusals ------

def test_balance_validation_before_any_device_call():
    lib = em.load()
    D = em.cdims(dims(100, 64, 4))
    need = em.edge_moe_balance_ws_bytes(dims(100, 64, 4), 3)
    ok = dict(z=BASE, idx=BASE, off=BASE, S=3, c=BASE, p=BASE, loss=BASE, ws=BASE, nb=need)

    def call(D=D, **kw):
        a = {**ok, **kw}
        return lib.edge_moe_balance(ctypes.byref(D), a["z"], a["idx"], a["off"], a["S"], a["c"], a["p"], a["loss"],
                                    a["ws"], a["nb"], None)
    for bad in (dict(z=None), dict(z=BASE + 2), dict(idx=None), dict(idx=BASE + 1), dict(off=BASE + 2), dict(S=0),
                dict(S=-1), dict(off=None), dict(c=None), dict(p=None), dict(p=BASE + 2), dict(loss=None),
                dict(ws=BASE + 4)):
        assert call(**bad) == em.EDGE_MOE_EINVAL, bad
    assert call(S=4096) == em.EDGE_MOE_EUNSUPPORTED
    assert call(ws=None) == em.EDGE_MOE_EWORKSPACE and call(nb=need - 1) == em.EDGE_MOE_EWORKSPACE
    assert call(D=em.cdims(dims(0, 64, 4))) == em.EDGE_MOE_EINVAL
    assert call(D=em.cdims(dims(8, 1025, 4))) == em.EDGE_MOE_EUNSUPPORTED
    assert em.edge_moe_balance_ws_bytes(dims(8, 64, 65), 1) == 0 and em.edge_moe_balance_ws_bytes(dims(8, 64, 4), 0) == 0


def test_backward_validation_before_any_device_call():
    lib = em.load()
    D = em.cdims(dims(100, 64, 4))
    need = em.edge_moe_route_backward_ws_bytes(dims(100, 64, 4))
    full = {n: BASE for n, _ in em.CRouteGrad._fields_}
    full["n_seq"] = 2

    def call(D=D, ws=BASE, nb=need, **kw):
        return lib.edge_moe_route_backward(ctypes.byref(D), ctypes.byref(em.CRouteGrad(**{**full, **kw})), ws, nb, None)
    none = dict(dlogits=None, dx=None, dw_router=None, dbias=None)
    for bad in (dict(logits=None), dict(logits=BASE + 2), dict(topk_idx=None), dict(topk_w=None), dict(d_topk_w=BASE + 2),
                dict(d_topk_w=None, d_loss=None), dict(d_loss=BASE + 2), dict(counts=None), dict(n_seq=0),
                dict(seq_offsets=None), dict(x=None), dict(x=BASE + 8), dict(w_router=None), dict(w_router=BASE + 4),
                none, dict(dlogits=BASE + 2), dict(dx=BASE + 8), dict(dw_router=BASE + 4), dict(dbias=BASE + 1),
                dict(ws=BASE + 8)):
        assert call(**bad) == em.EDGE_MOE_EINVAL, bad
    assert call(n_seq=4096) == em.EDGE_MOE_EUNSUPPORTED
    assert call(ws=None) == em.EDGE_MOE_EWORKSPACE and call(nb=need - 1) == em.EDGE_MOE_EWORKSPACE
    assert lib.edge_moe_route_backward(ctypes.byref(D), None, BASE, need, None) == em.EDGE_MOE_EINVAL
    assert call(D=em.cdims(dims(100, 64, 0))) == em.EDGE_MOE_EINVAL
    assert em.edge_moe_route_backward_ws_bytes(dims(100, 64, 4, d=100)) == 0


def test_binding_checks():
    D = dims(4, 8, 2)
    z, idx = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    c, p, loss, ws = torch.zeros(1, 8, dtype=torch.int32), torch.zeros(1, 8), torch.zeros(2), torch.zeros(1 << 16, dtype=torch.uint8)
    for args in ((z[:3], idx, c, p, loss), (z.double(), idx, c, p, loss), (z, idx.long(), c, p, loss),
                 (z, idx, c.float(), p, loss), (z, idx, c, p[:, :4], loss), (z, idx, c, p, loss[:1]), (z, idx, c, p, loss)):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):     # the last: host tensors
            em.edge_moe_balance(D, *args, ws)
    for kw in (dict(d_loss=loss, counts=p, dlogits=z), dict(d_topk_w=z, topk_w=z, dlogits=z),
               dict(d_loss=loss, counts=c, dx=z), dict(d_loss=loss, counts=c, dbias=z[0], x=z)):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            em.edge_moe_route_backward(D, z, idx, ws, **kw)
