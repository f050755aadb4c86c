"""The router operators write nothing past the workspace they ask for, whatever
tiles and slices their plan takes, and every plan's products are right."""
import numpy as np
import pytest
import torch

import shared_matrix_expert_amd as em
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from test_gpu_router_train import ALL, case, dev, dims  # noqa: E402

TAIL = 1 << 16


def guarded(n):
    ws = torch.full((n + TAIL,), 0xA5, dtype=torch.uint8, device=DEV)
    return ws[:n], ws[n:]


@pytest.mark.parametrize("T,E,k,d,S", [(1, 8, 1, 128, 1), (31, 64, 4, 512, 3), (200, 30, 3, 128, 4095), (2049, 33, 2, 128, 70),
                                       (4099, 1001, 3, 128, 9), (5, 1024, 2, 128, 2)])
def test_load(T, E, k, d, S):
    say(f"case: load {T} x {E}, {S} sequences")
    z, idx, *_ = case(T, E, k, T)
    D = dims(T, E, k, d)
    off = np.sort(np.random.default_rng(T).integers(0, T + 1, S + 1)).astype(np.int32)
    ws, tail = guarded(em.edge_moe_balance_ws_bytes(D, S))
    em.edge_moe_balance(D, dev(z), dev(idx), torch.empty(S, E, dtype=torch.int32, device=DEV), torch.empty(S, E, device=DEV),
                        torch.empty(2, device=DEV), ws, seq_offsets=dev(off))
    assert bool((tail == 0xA5).all())


# A shape of every plan (64 or 128 tile rows, 1 to 32 token slices, 1 to 8 expert slices).
PLANS = [(11, 88, 640), (1, 461, 640), (3, 488, 2176), (56, 1017, 2432), (559, 181, 4224), (338, 473, 384), (188, 519, 256),
         (150, 1009, 384), (316, 54, 128), (557, 367, 128), (993, 752, 512), (379, 1000, 384), (695, 49, 640), (2096, 445, 384),
         (960, 578, 128), (838, 1000, 128), (1631, 8, 640), (2723, 425, 128), (1989, 482, 128), (6294, 9, 128), (695, 465, 4096),
         (351, 820, 3456), (230, 651, 3968), (77, 1006, 3840), (1237, 623, 2048), (1022, 908, 1152), (456, 883, 1408),
         (2718, 860, 1152), (2006, 828, 1024), (631, 812, 640), (902, 107, 3584), (2641, 604, 384), (1043, 564, 384),
         (2570, 99, 1024), (4713, 629, 128), (3388, 801, 128), (14605, 61, 128)]


@pytest.mark.parametrize("T,E,d", PLANS)
def test_backward(T, E, d):
    """The tail stays, and dx and dW_r are the products of dlogits to the float32
    sums' bound (2 u for each of an instruction's additions, 8 u within it)."""
    say(f"case: backward {T} x {E} x {d}")
    k = 3
    z, idx, w, dw, x, wr = case(T, E, k, T, d)
    D = dims(T, E, k, d)
    counts = torch.ones(1, E, dtype=torch.int32, device=DEV)
    shapes = dict(zip(ALL, ((T, E), (T, d), (E, d), (E,))))
    zd, idxd, wd, dwd, xd, wrd = dev(z), dev(idx), dev(w), dev(dw), x.to(DEV), wr.to(DEV)
    full = {}
    for want in (ALL, ("dx",), ("dw_router", "dbias")):
        ws, tail = guarded(em.edge_moe_route_backward_ws_bytes(D))
        out = {n: torch.full(shapes[n], float("nan"), device=DEV) for n in want}
        em.edge_moe_route_backward(D, zd, idxd, ws, topk_w=wd, d_topk_w=dwd, d_loss=torch.ones(2, device=DEV), counts=counts,
                                   x=xd, w_router=wrd, **out)
        assert bool((tail == 0xA5).all()), want
        full = full or out
        assert all(torch.equal(out[n], full[n]) for n in want)
    dz = full["dlogits"].double()
    for name, a, b, n in (("dx", dz, wrd.double(), E), ("dw_router", dz.t().contiguous(), xd.double(), T)):
        tol = (6 * (n // 32 + 1) + 8) * 2.0 ** -24 * (a.abs() @ b.abs()) + 1e-40
        assert bool(((full[name].double() - a @ b).abs() <= tol).all()), name
    assert bool(((full["dbias"].double() - dz.sum(0)).abs() <= 8 * 2.0 ** -24 * dz.abs().sum(0) + 1e-40).all())
