"""Load and gradients of the router where a wave holds four tokens (batches past
2048 tokens in the load, past 4096 in the gradient): sequence boundaries inside
a wave's run, many sequences in one workgroup's tokens, tokens in none; expert
counts on both sides of every row width, rows that are not 16-byte aligned."""
import numpy as np
import pytest
import torch

import shared_matrix_expert_amd as em
from oracle import operators as ops
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from test_gpu_router_train import LOAD, case, check_backward, check_balance, dev, dims  # noqa: E402

T, K = 4700, 3
# several sequences in the first 16 tokens, empty ones, single tokens, boundaries inside
# and at the ends of runs of 4 and 16, tokens before the first and behind the last
RAGGED = [3, 5, 5, 9, 12, 20, 32, 33, 34, 35, 36, 2048, 2064, 2101, 2102, 4096, 4099, 4099, 4500, 4613]
EXPERTS = [30, 64, 399, 512, 1001, 1024]


def offsets(kind):
    if kind == "ragged":
        return RAGGED
    n = 1600 if kind == "three tokens each" else 4095
    off = np.sort(np.random.default_rng(n).integers(0, T + 1, n + 1))
    return off.tolist()


@pytest.mark.parametrize("kind", ["ragged", "three tokens each", "4095 sequences"])
@pytest.mark.parametrize("E", EXPERTS)
def test_balance(E, kind):
    say(f"case: balance {T} x {E}, {kind}")
    z, idx, *_ = case(T, E, K, E)
    check_balance(dims(T, E, K), z, idx, offsets(kind))


@pytest.mark.parametrize("E", EXPERTS)
def test_backward(E):
    say(f"case: backward {T} x {E}")
    check_backward(T, E, K, 128, RAGGED)


@pytest.mark.parametrize("kind", ["three tokens each", "4095 sequences"])
@pytest.mark.parametrize("E", [64, 399])
def test_backward_of_short_sequences(E, kind):
    say(f"case: backward {T} x {E}, {kind}")
    check_backward(T, E, K, 128, offsets(kind), weights=False)


@pytest.mark.parametrize("t,off", [(40, [3, 5, 5, 9, 30]), (2500, [1, 2, 2, 7, 2047, 2300]), (T, RAGGED)])
@pytest.mark.parametrize("E", [64, 512, 1000])
def test_rows_at_four_bytes(t, off, E):
    """E a multiple of 4 with logits, then dlogits too, at an address that is not
    16-byte aligned."""
    say(f"case: {t} x {E} at 4 bytes")
    z, idx, w, dw, *_ = case(t, E, K, E)
    D = dims(t, E, K)
    offd, idxd = dev(np.asarray(off, np.int32)), dev(idx)

    def at_four(values=None):
        buf = torch.full((t * E + 8,), 7.0, device=DEV)
        part = buf[1:1 + t * E].view(t, E)
        assert part.data_ptr() % 16 == 4
        if values is not None:
            part.copy_(values)
        return buf, part
    _, zd = at_four(dev(z))
    S = len(off) - 1
    counts, probs, loss = torch.empty(S, E, dtype=torch.int32, device=DEV), torch.empty(S, E, device=DEV), torch.empty(2, device=DEV)
    ws = torch.empty(max(em.edge_moe_balance_ws_bytes(D, S), em.edge_moe_route_backward_ws_bytes(D)), dtype=torch.uint8, device=DEV)
    em.edge_moe_balance(D, zd, idxd, counts, probs, loss, ws, seq_offsets=offd)
    c, p, _ = ops.balance(z, idx, off)
    assert np.array_equal(counts.cpu().numpy(), c)
    assert np.all(np.abs(probs.cpu().numpy() - p) <= LOAD * p + 1e-40)
    g = np.array([0.6, -0.2], np.float32)
    dz, mag = ops.route_backward(z, idx, w, dw, g, c, off)
    for logits, (buf, out) in ((zd, at_four()), (dev(z), at_four()), (zd, (None, torch.empty(t, E, device=DEV)))):
        dbias = torch.empty(E, device=DEV)
        em.edge_moe_route_backward(D, logits, idxd, ws, topk_w=dev(w), d_topk_w=dev(dw), d_loss=dev(g), counts=counts,
                                   seq_offsets=offd, dlogits=out, dbias=dbias)
        tz = 2.5 * LOAD * mag + 1e-40                        # the bounds of the aligned rows' tests
        assert np.all(np.abs(out.cpu().numpy() - dz) <= tz)
        assert np.all(np.abs(dbias.cpu().numpy() - dz.sum(0)) <= tz.sum(0) + 8 * 2.0 ** -24 * np.abs(dz).sum(0) + 1e-40)
        if buf is not None:
            assert float(buf[0]) == 7 and bool((buf[1 + t * E:] == 7).all())
