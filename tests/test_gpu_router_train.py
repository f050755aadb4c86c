"""The router-training operators on the GPU against the float64 oracle.

Tolerances, in units u = 2^-24 (half a float32 step): a probability carries the
rounding of z - max (|z - max| u), the exponential and the reciprocal (4 u), and
the sum of E terms (each lane's E / 64, then six steps across the lanes); the
column sums add at most the roundings of 16 tokens' sums (four a wave, then four
waves) before float64.  LOAD below bounds their sum for
|z - max| <= 40 and E <= 1024: 40 + 4 + 22 + 10 < 100.
"""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import shared_matrix_expert_amd as em
import synth
from oracle import mx
from oracle import operators as ops
from oracle.codecs import bf16_to_f64
from gpu_helpers import DEV, bits_to_dev, say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

U = 2.0 ** -24
LOAD = 100 * U


def dims(T, E, k, d=128):
    return SimpleNamespace(T=T, d=d, h=128, n_experts=E, experts_per_group=E, top_k=k, delta_rank=8, lora_rank=2,
                           quant_group=32)


def case(T, E, k, seed, d=128):
    rng = np.random.default_rng(seed)
    z = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    idx = np.argsort(-z, 1, kind="stable")[:, :k].astype(np.int32)
    s = np.take_along_axis(z, idx, 1).astype(np.float64)
    w = np.exp(s - s.max(1, keepdims=True))
    w = (w / w.sum(1, keepdims=True)).astype(np.float32)
    dw = (0.02 * rng.standard_normal((T, k))).astype(np.float32)
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).to(torch.bfloat16)
    wr = torch.from_numpy((rng.standard_normal((E, d)) / np.sqrt(d)).astype(np.float32)).to(torch.bfloat16)
    return z, idx, w, dw, x, wr


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def run_balance(D, z, idx, off=None, ws=None, stream=None):
    S = 1 if off is None else len(off) - 1
    c = torch.full((S, D.n_experts), -7, dtype=torch.int32, device=DEV)
    p = torch.full((S, D.n_experts), -7.0, device=DEV)
    loss = torch.full((2,), -7.0, device=DEV)
    if ws is None:
        ws = torch.empty(em.edge_moe_balance_ws_bytes(D, S), dtype=torch.uint8, device=DEV)
    em.edge_moe_balance(D, dev(z), dev(idx), c, p, loss, ws, seq_offsets=dev(None if off is None else np.asarray(off, np.int32)),
                        stream=stream)
    return c, p, loss


def check_balance(D, z, idx, off=None):
    c, p, loss = run_balance(D, z, idx, off)
    cr, pr, lr = ops.balance(z, idx, off)
    assert np.array_equal(c.cpu().numpy(), cr), "counts differ"
    got = p.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - pr) <= LOAD * pr + 1e-40), f"probs off by {np.max(np.abs(got - pr) / (pr + 1e-40)) / U:.3g} u"
    # the balance loss is a sum of non-negative terms: the probabilities' bound;
    # lse^2: twice lse's, an absolute 30 u (the sum's relative error, the logarithm) + |lse| u
    lse = np.sqrt(lr[1]) if lr[1] else 0.0
    tol = np.array([LOAD * lr[0], 2 * (lse + 1) * (30 + 2 * (lse + 1)) * U + 4 * U * lr[1]])
    assert np.all(np.abs(loss.cpu().numpy() - lr) <= tol + 1e-40), (loss.cpu().numpy(), lr)
    return cr


SHAPES = [(1, 8, 1), (2, 10, 3), (31, 64, 4), (33, 130, 2), (64, 257, 8), (130, 512, 10), (300, 1000, 6), (700, 33, 32),
          (1025, 1024, 5), (2100, 128, 3)]


@pytest.mark.parametrize("T,E,k", SHAPES)
def test_balance_one_sequence(T, E, k):
    say(f"case: balance {T} x {E}, top {k}")
    z, idx, *_ = case(T, E, k, T)
    check_balance(dims(T, E, k), z, idx)
    check_balance(dims(T, E, k), z, idx, [0, T])


@pytest.mark.parametrize("off", [[0, 10, 10, 11, 96, 200], [5, 37, 130], [0, 0, 0], [200, 200], [0, 200, 200],
                                 "seventy", "four thousand"])
@pytest.mark.parametrize("E", [64, 30])
def test_balance_ragged_sequences(off, E):
    """Empty sequences, tokens before the first and behind the last, more
    sequences than lanes, more than tokens."""
    T, k = 200, 3
    rng = np.random.default_rng(1)
    if off == "seventy":
        off = np.sort(rng.integers(0, T + 1, 71)).tolist()
    elif off == "four thousand":
        off = np.sort(rng.integers(0, T + 1, 4096)).tolist()
    z, idx, *_ = case(T, E, k, 3)
    check_balance(dims(T, E, k), z, idx, off)


def test_balance_masked_experts_and_dropped_slots():
    T, E, k = 90, 64, 4
    z, idx, *_ = case(T, E, k, 5)
    z[:, 40:] = -np.inf                           # experts masked for every token
    z[7] = -np.inf                                # a token with every expert masked
    z[8] = -np.inf
    z[8, 3] = 2.0                                 # one expert left
    z[9] = np.finfo(np.float32).min               # masked by the type's lowest value: uniform
    z[10, 1:] = np.finfo(np.float32).min
    idx[11, 2], idx[12, 0], idx[13] = -1, E, 2 ** 31 - 1
    idx[14] = 5                                   # one expert four times
    keep = np.r_[0:9, 10:T]                       # token 9's lse^2 is past float32
    check_balance(dims(T, E, k), z, idx, [0, 9])
    check_balance(dims(T - 1, E, k), z[keep], idx[keep])
    c, p, loss = run_balance(dims(T, E, k), z, idx)
    assert np.isinf(float(loss[1])) and np.isfinite(float(loss[0]))
    z[20, 3] = np.nan
    assert np.isnan(run_balance(dims(T, E, k), z, idx)[2].cpu().numpy()).all()


@pytest.mark.parametrize("rest", [float("nan"), -float("inf")])
def test_balance_rows_of_nan(rest):
    """A row of NaN alone, or of NaN among masked experts, is no masked token."""
    T, E, k = 20, 300, 2
    z, idx, *_ = case(T, E, k, 5)
    z[7] = rest
    z[7, 11] = np.nan
    _, p, loss = run_balance(dims(T, E, k), z, idx)
    assert bool(torch.isnan(p).all()) and bool(torch.isnan(loss).all())


def run_backward(D, z, idx, **kw):
    T, E, d = D.T, D.n_experts, D.d
    want = kw.pop("want")
    out = {n: torch.full(s, float("nan"), device=DEV) for n, s in
           (("dlogits", (T, E)), ("dx", (T, d)), ("dw_router", (E, d)), ("dbias", (E,))) if n in want}
    ws = torch.empty(em.edge_moe_route_backward_ws_bytes(D), dtype=torch.uint8, device=DEV)
    if kw.pop("dirty", False):
        ws.fill_(255)
    em.edge_moe_route_backward(D, dev(z), dev(idx), ws, **kw, **out)
    return out


ALL = ("dlogits", "dx", "dw_router", "dbias")


def check_backward(T, E, k, d, off=None, weights=True, losses=True, edit=None, seed=0):
    z, idx, w, dw, x, wr = case(T, E, k, seed + T, d)
    if edit:
        edit(z, idx)
    D = dims(T, E, k, d)
    g = np.array([0.6, -0.2], np.float32) if losses else None
    counts = ops.balance(z, idx, off)[0].astype(np.int32) if losses else None
    out = run_backward(D, z, idx, want=ALL, dirty=True, topk_w=dev(w) if weights else None,
                       d_topk_w=dev(dw) if weights else None, d_loss=dev(g), counts=dev(counts),
                       seq_offsets=dev(np.asarray(off, np.int32)) if off is not None and losses else None,
                       x=x.to(DEV), w_router=wr.to(DEV))
    dz, mag = ops.route_backward(z, idx, w if weights else None, dw if weights else None, g, counts, off)
    got = {n: v.cpu().numpy().astype(np.float64) for n, v in out.items()}
    # each term of dz: the probabilities' bound, the same again for the mean that
    # is subtracted, and the lse's 30 u
    tz = 2.5 * LOAD * mag + 1e-40
    err = np.abs(got["dlogits"] - dz)
    say(f"  dlogits: worst error {np.max(err / tz):.3g} of the bound")
    assert np.all(err <= tz)
    # products: the terms' errors, then float32 sums of 3 K / 32 instructions of 32
    # exact products each (2 u each, and 8 u for the sum inside an instruction)
    for name, a, b, ta, K in (("dx", dz, wr.double().numpy(), tz, E), ("dw_router", dz.T, x.double().numpy(), tz.T, T)):
        n = 3 * (K // 32 + 1)
        tol = ta @ np.abs(b) + (2 * n + 8) * U * (np.abs(a) @ np.abs(b)) + 1e-40
        err = np.abs(got[name] - a @ b)
        norm = np.linalg.norm(a @ b)
        say(f"  {name}: worst error {np.max(err / tol):.3g} of the bound, relative 2-norm {np.linalg.norm(err) / max(norm, 1e-300):.3g}")
        assert np.all(err <= tol)
    tol = tz.sum(0) + 8 * U * np.abs(dz).sum(0) + 1e-40
    assert np.all(np.abs(got["dbias"] - dz.sum(0)) <= tol)
    return out, (D, z, idx, w, dw, x, wr, g, counts)


@pytest.mark.parametrize("T,E,k,d", [(1, 8, 1, 128), (2, 10, 3, 384), (31, 64, 4, 512), (65, 130, 2, 128), (96, 64, 4, 512),
                                     (130, 512, 10, 640), (257, 1000, 6, 256), (300, 257, 5, 1024), (1025, 128, 2, 128),
                                     (1501, 512, 10, 512), (5, 913, 6, 640), (751, 480, 7, 1280), (2273, 80, 4, 128),
                                     (1531, 10, 2, 3200), (7181, 16, 3, 384), (11764, 48, 4, 128)])
def test_backward_shapes(T, E, k, d):
    say(f"case: backward {T} x {E} x {d}, top {k}")
    check_backward(T, E, k, d)


@pytest.mark.parametrize("off", [[0, 10, 10, 11, 96, 200], [5, 37, 130], [0, 0, 0], "seventy", "four thousand"])
def test_backward_ragged_sequences(off):
    rng = np.random.default_rng(2)
    if off == "seventy":
        off = np.sort(rng.integers(0, 201, 71)).tolist()
    elif off == "four thousand":
        off = np.sort(rng.integers(0, 201, 4096)).tolist()
    check_backward(200, 64, 3, 128, off)


@pytest.mark.parametrize("weights,losses", [(True, False), (False, True)])
def test_backward_one_source(weights, losses):
    check_backward(77, 40, 4, 256, weights=weights, losses=losses)


def test_backward_masked_experts_and_odd_picks():
    def edit(z, idx):
        z[:, 40:] = -np.inf
        z[7] = -np.inf
        z[8, 1:] = np.finfo(np.float32).min
        idx[11, 2], idx[12, 0], idx[13] = -1, 64, 2 ** 31 - 1
        idx[14] = 5
    check_backward(90, 64, 4, 128, [0, 8, 90], edit=edit)


@pytest.mark.parametrize("T,E,d", [(40, 64, 128), (600, 512, 256)])
def test_backward_keeps_24_bits(T, E, d):
    """With one-hot rows of W_r and x the products pick single values of dz: the
    same bits as dlogits."""
    z, idx, w, dw, x, wr = case(T, E, 4, 1, d)
    e_of, t_of = np.arange(d) % E, (np.arange(d) * 7) % T
    hot = torch.zeros(E, d)
    hot[e_of, np.arange(d)] = 1
    xh = torch.zeros(T, d)
    xh[t_of, np.arange(d)] = 1
    D = dims(T, E, 4, d)
    counts = ops.balance(z, idx)[0].astype(np.int32)
    out = run_backward(D, z, idx, want=ALL, topk_w=dev(w), d_topk_w=dev(dw), d_loss=dev(np.array([1.0, 0.5], np.float32)),
                       counts=dev(counts), x=xh.to(torch.bfloat16).to(DEV), w_router=hot.to(torch.bfloat16).to(DEV))
    dz = out["dlogits"]
    assert torch.equal(out["dx"], dz[:, torch.from_numpy(e_of).to(DEV)])
    assert torch.equal(out["dw_router"], dz[torch.from_numpy(t_of).to(DEV)].t())


@pytest.mark.parametrize("want", [("dlogits",), ("dx",), ("dw_router",), ("dbias",), ("dx", "dbias")])
def test_backward_outputs_on_their_own(want):
    """Each output alone has the bits it has among all of them."""
    full, (D, z, idx, w, dw, x, wr, g, counts) = check_backward(150, 96, 3, 256)
    out = run_backward(D, z, idx, want=want, dirty=True, topk_w=dev(w), d_topk_w=dev(dw), d_loss=dev(g), counts=dev(counts),
                       x=x.to(DEV), w_router=wr.to(DEV))
    assert set(out) == set(want)
    for n in want:
        assert torch.equal(out[n], full[n]), n


def test_repeats_streams_and_graphs():
    """Load and backward as one training step's tail: the same bits on another
    stream and in every replay of a graph, with eager work between replays."""
    T, E, k, d = 333, 64, 4, 512
    z, idx, w, dw, x, wr = case(T, E, k, 8, d)
    D = dims(T, E, k, d)
    off = dev(np.array([0, 100, 100, 320], np.int32))
    zd, idxd, wd, dwd, xd, wrd = dev(z), dev(idx), dev(w), dev(dw), x.to(DEV), wr.to(DEV)
    g = dev(np.array([0.01, 0.001], np.float32))

    def buffers():
        b = {n: torch.full(s, float("nan"), device=DEV) for n, s in
             (("probs", (3, E)), ("loss", (2,)), ("dlogits", (T, E)), ("dx", (T, d)), ("dw_router", (E, d)), ("dbias", (E,)))}
        b["counts"] = torch.full((3, E), -1, dtype=torch.int32, device=DEV)
        b["ws"] = torch.empty(max(em.edge_moe_balance_ws_bytes(D, 3), em.edge_moe_route_backward_ws_bytes(D)),
                              dtype=torch.uint8, device=DEV)
        return b

    def step(b, stream=None):
        em.edge_moe_balance(D, zd, idxd, b["counts"], b["probs"], b["loss"], b["ws"], seq_offsets=off, stream=stream)
        em.edge_moe_route_backward(D, zd, idxd, b["ws"], topk_w=wd, d_topk_w=dwd, d_loss=g, counts=b["counts"],
                                   seq_offsets=off, x=xd, w_router=wrd, stream=stream, **{n: b[n] for n in ALL})
    names = ("counts", "probs", "loss") + ALL
    a, b = buffers(), buffers()
    step(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(b, s)
    s.synchronize()
    assert all(torch.equal(a[n], b[n]) for n in names)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for i in range(4):
        zd.copy_(dev(case(T, E, k, 30 + i, d)[0]))
        for n in names:
            b[n].fill_(3)
        b["ws"].fill_(i * 85)
        graph.replay()
        torch.cuda.synchronize()
        step(a)
        assert all(torch.equal(a[n], b[n]) for n in names), f"replay {i}"
