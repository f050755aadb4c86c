"""Workloads of the layer's MX-matrix and router-training operators.

Four kinds of pass:

* ``mx_round``: matrices or token rows to the microscaling format and back
  (edge_moe_mx_quantize, edge_moe_mx_dequantize);
* ``mx_product``: the product of token rows with MXFP4 matrices, one matrix or
  one per expert (edge_moe_mx_product);
* ``balance``: the router's load: counts, mean probabilities, balance and z
  losses, and their gradient at the logits (edge_moe_balance,
  edge_moe_route_backward);
* ``route_backward``: the router's whole backward pass, from the gradients of
  the selection weights and of the losses to those of x, W_r and the bias
  (edge_moe_route_backward).

``run`` computes a pass in plain torch operations, or through the library
where ``own`` is true; ``exact`` gives the definition in float64.
"""
import math
from types import SimpleNamespace

import numpy as np
import torch

own = False

DEV = "cuda"
FULL = dict(d=4096, h=8192, E=512, k=10)          # the layer's full shapes


def listed():
    return [
        # one expert's A_up (128 x 4096) from float32 master weights: a tensor of a streamed expert
        dict(name="round one expert", kind="mx_round", fmt="fp4", src="fp32", M=1, N=128, K=4096),
        # a prompt's token rows as the input of an MX product
        dict(name="round prompt rows", kind="mx_round", fmt="fp8", src="bf16", M=1, N=16384, K=4096),
        # a layer's shared up matrices, eight groups, from bf16
        dict(name="round shared up", kind="mx_round", fmt="fp4", src="bf16", M=8, N=8192, K=4096),
        # one token through one group's shared up matrix
        dict(name="product one token", kind="mx_product", xfmt="fp8", T=1, M=1, N=8192, K=4096, k=0),
        # a verify batch through its experts' rank-128 inputs: 8 tokens, ten of 512 experts each
        dict(name="product verify experts", kind="mx_product", xfmt="fp8", T=8, M=512, N=128, K=4096, k=10),
        # a ragged batch sorted by group through the groups' shared down matrices, both sides in 4 bits
        dict(name="product ragged groups", kind="mx_product", xfmt="fp4", T=5001, M=8, N=4096, K=8192, k=0),
        # a prompt through one shared up matrix
        dict(name="product prompt", kind="mx_product", xfmt="fp8", T=16384, M=1, N=8192, K=4096, k=0),
        # the load of a small batch of ragged sequences
        dict(name="balance small", kind="balance", T=333, E=64, k=4, S=3),
        # the load of a training batch: 16 ragged sequences
        dict(name="balance batch", kind="balance", T=16384, E=512, k=10, S=16),
        # the small MX test layer's router
        dict(name="backward small", kind="route_backward", T=96, E=64, k=4, S=1, d=512),
        # an odd batch of short sequences through the full router
        dict(name="backward ragged", kind="route_backward", T=1501, E=512, k=10, S=7, d=4096),
        # a training batch through the full router
        dict(name="backward batch", kind="route_backward", T=16384, E=512, k=10, S=16, d=4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    kind = rng.choice(["mx_round", "mx_product", "balance", "route_backward"])
    if kind == "mx_round":
        while True:
            c = dict(kind=kind, fmt=rng.choice(["fp4", "fp8"]), src=rng.choice(["bf16", "fp32"]),
                     M=_log(rng, 1, 64), N=_log(rng, 16, 16384), K=128 * _log(rng, 1, 64))
            if 1 << 12 <= c["M"] * c["N"] * c["K"] <= 1 << 27:
                return c
    if kind == "mx_product":
        while True:
            M = 1 if rng.random() < 0.4 else _log(rng, 2, 512)
            k = rng.choice([0, rng.randint(2, 10)]) if M > 1 else 0
            k = min(k, M)
            c = dict(kind=kind, xfmt=rng.choice(["fp8", "fp4"]), T=_log(rng, 1, 16384), M=M,
                     N=_log(rng, 16, 8192), K=128 * _log(rng, 1, 64), k=k)
            R = c["T"] * max(1, k)
            if M * c["N"] * c["K"] <= 1 << 28 and R <= 65536 and R * c["K"] <= 1 << 27 and R * c["N"] * c["K"] <= 1 << 38:
                return c
    E = rng.choice([_log(rng, 8, 1024), 8 * _log(rng, 1, 128)])
    k = rng.randint(1, min(E, 16))
    if kind == "balance":
        T = _log(rng, 1, min(16384, (1 << 23) // E))
        return dict(kind=kind, T=T, E=E, k=k, S=min(T, _log(rng, 1, 32)))
    while True:
        T, d = _log(rng, 1, 16384), 128 * _log(rng, 1, 64)
        if T * E * d <= 1 << 35 and T * E <= 1 << 23 and T * d <= 1 << 26:
            return dict(kind=kind, T=T, E=E, k=k, S=min(T, _log(rng, 1, 32)), d=d)


# ------------------------------------------------------------------ inputs ---------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)


def _cuts(total, parts, seed):
    """parts + 1 offsets from 0 to total, ragged."""
    rng = np.random.default_rng(seed)
    share = rng.dirichlet(np.full(parts, 4.0))
    cut = np.floor(np.cumsum(share)[:-1] * total).astype(np.int64)
    return np.concatenate([[0], cut, [total]])


def _router_inputs(case, seed):
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    g = _gen(seed)
    s = {"T": T, "E": E, "k": k, "S": S}
    if case["kind"] == "route_backward":
        d = case["d"]
        s["x"] = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
        s["w_router"] = (torch.randn(E, d, generator=g, device=DEV) / math.sqrt(d)).to(torch.bfloat16)
        s["logits"] = s["x"].float() @ s["w_router"].float().t()
        s["dx"] = torch.empty(T, d, device=DEV)
        s["dw_router"] = torch.empty(E, d, device=DEV)
        s["dbias"] = torch.empty(E, device=DEV)
    else:
        d = 128
        s["logits"] = torch.randn(T, E, generator=g, device=DEV)
        s["dlogits"] = torch.empty(T, E, device=DEV)
    top, idx = s["logits"].topk(k, dim=1)
    s["topk_idx"] = idx.to(torch.int32).contiguous()
    s["topk_w"] = torch.softmax(top, 1).contiguous()
    s["d_topk_w"] = 0.02 * torch.randn(T, k, generator=g, device=DEV)
    s["d_loss"] = torch.tensor([0.01, 0.001], device=DEV)          # the losses' weights in the objective
    s["seq_offsets"] = torch.from_numpy(_cuts(T, S, seed).astype(np.int32)).to(DEV)
    s["counts"] = torch.empty(S, E, dtype=torch.int32, device=DEV)
    s["probs"] = torch.empty(S, E, device=DEV)
    s["loss"] = torch.empty(2, device=DEV)
    if case["kind"] == "route_backward":                            # the forward pass left the counts
        s["counts"].copy_(_counts(s))
    s["dims"] = SimpleNamespace(T=T, d=d, h=128, n_experts=E, experts_per_group=E, top_k=k, delta_rank=8,
                                lora_rank=2, quant_group=32)
    return s


def prepare(case, seed):
    kind = case["kind"]
    g = _gen(seed)
    if kind == "mx_round":
        M, N, K, fp4 = case["M"], case["N"], case["K"], case["fmt"] == "fp4"
        src = torch.randn(M, N, K, generator=g, device=DEV)
        src = src * 0.02 if fp4 else src
        src = src if case["src"] == "fp32" else src.to(torch.bfloat16)
        return {"kind": kind, "fp4": fp4, "src": src, "out": torch.empty(M, N, K, dtype=src.dtype, device=DEV),
                "codes": torch.empty(M, N, K // 2 if fp4 else K, dtype=torch.uint8, device=DEV),
                "scales": torch.empty(M, K // 128, N, 4, dtype=torch.uint8, device=DEV)}
    if kind == "mx_product":
        T, M, N, K, k = (case[n] for n in ("T", "M", "N", "K", "k"))
        R = T * max(1, k)
        s = {"kind": kind, "fp4": case["xfmt"] == "fp4",
             "x": torch.randn(T, K, generator=g, device=DEV).to(torch.bfloat16),
             # codes uniform over the format, block scales about 2^-9 .. 2^-6: weights near N(0, 0.02^2)
             "codes": torch.randint(0, 256, (M, N, K // 2), generator=g, device=DEV, dtype=torch.uint8),
             "scales": torch.randint(118, 122, (M, K // 128, N, 4), generator=g, device=DEV, dtype=torch.uint8),
             "y": torch.empty(R, N, dtype=torch.bfloat16, device=DEV), "offsets": None, "row_src": None}
        if M > 1:
            if k:                                                    # k distinct matrices a token, rows sorted by matrix
                pick = torch.rand(T, M, generator=g, device=DEV).topk(k, dim=1).indices
                order = torch.argsort(pick.reshape(-1) * T + torch.arange(T, device=DEV).repeat_interleave(k))
                s["row_src"] = (order // k).to(torch.int32)
                cnt = np.bincount(pick.cpu().numpy().reshape(-1), minlength=M)
                off = np.concatenate([[0], np.cumsum(cnt)])
            else:
                off = _cuts(T, M, seed)
            s["offsets"] = torch.from_numpy(off.astype(np.int32)).to(DEV)
            # the plain form's plan: the matrices that have rows, and each one's rows padded to the longest
            act = np.nonzero(np.diff(off))[0]
            n = np.diff(off)[act]
            rows = off[act][:, None] + np.minimum(np.arange(n.max())[None, :], n[:, None] - 1)
            keep = np.arange(n.max())[None, :] < n[:, None]
            s["active"] = torch.from_numpy(act).to(DEV)
            s["rows"] = torch.from_numpy(rows).to(DEV)
            s["keep"] = torch.from_numpy(keep).to(DEV)
        return s
    return dict(_router_inputs(case, seed), kind=kind)


# ------------------------------------------------------------------ plain forms ----

def _pow2(n):
    """2^n as float32 for whole n in -126 .. 127, by its bits."""
    return ((n + 127) << 23).view(torch.float32)


def _quantised(v, fp4):
    """The float32 values that v's blocks of 32 along the last axis take in MXFP4 / MXFP8."""
    emax, mant, least, top = (2, 1, 0, 6.0) if fp4 else (8, 3, -6, 448.0)
    b = v.float().reshape(*v.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    x = torch.where(amax > 0, (torch.frexp(amax)[1] - 1 - emax).clamp(-127, 127), -127).clamp(min=-126)
    a = b * _pow2(-x)
    e = (torch.frexp(a)[1] - 1).clamp(min=least)
    a = (torch.round(a * _pow2(mant - e)) * _pow2(e - mant)).clamp(-top, top)
    return (a * _pow2(x)).reshape(v.shape)


def _weights(codes, scales):
    """float32 values of MXFP4 matrices [..., N, K/2] with scales [..., K/128, N, 4]."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=DEV)
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1)
    sc = _pow2(scales.transpose(-3, -2).flatten(-2).int() - 127)     # [..., N, K/32]
    return (v.reshape(*sc.shape, 32) * sc.unsqueeze(-1)).flatten(-2)


def _counts(s):
    """Picks of every expert by sequence: [S][E]."""
    t = torch.arange(s["T"], device=DEV)
    seq = (t.unsqueeze(1) >= s["seq_offsets"][1:-1].unsqueeze(0)).sum(1)
    flat = (seq.unsqueeze(1) * s["E"] + s["topk_idx"]).reshape(-1)
    return torch.bincount(flat, minlength=s["S"] * s["E"]).reshape(s["S"], s["E"]).int()


def _member(s, dtype):
    """[S][T]: one where the token belongs to the sequence."""
    t = torch.arange(s["T"], device=DEV).unsqueeze(0)
    return ((t >= s["seq_offsets"][:-1].unsqueeze(1)) & (t < s["seq_offsets"][1:].unsqueeze(1))).to(dtype)


def _softmax(z):
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    n = e.sum(1, keepdim=True)
    return e / n, (m + torch.log(n)).squeeze(1)


def _dlogits(s, with_weights):
    """The gradient at the logits, float32."""
    p, lse = _softmax(s["logits"])
    n = (s["seq_offsets"][1:] - s["seq_offsets"][:-1]).float()
    f = s["counts"].float() * (s["E"] / s["k"]) / n.clamp(min=1).unsqueeze(1)
    live = (n > 0).sum()
    seq = (torch.arange(s["T"], device=DEV).unsqueeze(1) >= s["seq_offsets"][1:-1].unsqueeze(0)).sum(1)
    ft = f[seq]
    gb = s["d_loss"][0] / live / n[seq]
    dz = gb.unsqueeze(1) * p * (ft - (p * ft).sum(1, keepdim=True))
    dz += (2 * s["d_loss"][1] / n.sum() * lse).unsqueeze(1) * p
    if with_weights:
        w, dw = s["topk_w"], s["d_topk_w"]
        dz.scatter_add_(1, s["topk_idx"].long(), w * (dw - (w * dw).sum(1, keepdim=True)))
    return dz


def _plain(s):
    kind = s["kind"]
    if kind == "mx_round":
        return _quantised(s["src"], s["fp4"]).to(s["src"].dtype)
    if kind == "mx_product":
        x = _quantised(s["x"], s["fp4"])
        if s["offsets"] is None:
            return (x @ _weights(s["codes"][0], s["scales"][0]).t()).to(torch.bfloat16)
        w = _weights(s["codes"][s["active"]], s["scales"][s["active"]])
        src = s["rows"] if s["row_src"] is None else s["row_src"].long()[s["rows"]]
        return torch.bmm(x[src], w.transpose(1, 2).contiguous())[s["keep"]].to(torch.bfloat16)
    if kind == "balance":
        p, lse = _softmax(s["logits"])
        n = (s["seq_offsets"][1:] - s["seq_offsets"][:-1]).double()
        c = _counts(s)
        mean = (_member(s, torch.float64) @ p.double()) / n.clamp(min=1).unsqueeze(1)
        f = c.double() * (s["E"] / s["k"]) / n.clamp(min=1).unsqueeze(1)
        loss = torch.stack([(f * mean).sum() / (n > 0).sum(), (lse.double() ** 2).mean()])
        s["counts"].copy_(c)
        return {"counts": c, "probs": mean.float(), "loss": loss.float(), "dlogits": _dlogits(s, False)}
    dz = _dlogits(s, True)
    return {"dx": dz @ s["w_router"].float(), "dw_router": dz.t() @ s["x"].float(), "dbias": dz.double().sum(0).float()}


# ------------------------------------------------------------------ one pass -------

def _own(s):
    import shared_matrix_expert_amd as em
    kind = s["kind"]
    if kind == "mx_round":
        fmt = em.MX_FP4 if s["fp4"] else em.MX_FP8
        em.edge_moe_mx_quantize(fmt, s["src"], s["codes"], s["scales"])
        em.edge_moe_mx_dequantize(fmt, s["codes"], s["scales"], s["out"])
        return s["out"]
    if kind == "mx_product":
        fmt = em.MX_FP4 if s["fp4"] else em.MX_FP8
        if "ws" not in s:
            (T, K), (M, N, _) = s["x"].shape, s["codes"].shape
            s["ws"] = torch.empty(em.edge_moe_mx_product_ws_bytes(T, s["y"].shape[0], M, N, K, fmt),
                                  dtype=torch.uint8, device=DEV)
        em.edge_moe_mx_product(fmt, s["x"], s["codes"], s["scales"], s["y"], s["ws"], offsets=s["offsets"],
                               row_src=s["row_src"])
        return s["y"]
    if "ws" not in s:
        s["ws"] = torch.empty(max(em.edge_moe_balance_ws_bytes(s["dims"], s["S"]),
                                  em.edge_moe_route_backward_ws_bytes(s["dims"])), dtype=torch.uint8, device=DEV)
    if kind == "balance":
        em.edge_moe_balance(s["dims"], s["logits"], s["topk_idx"], s["counts"], s["probs"], s["loss"], s["ws"],
                            seq_offsets=s["seq_offsets"])
        em.edge_moe_route_backward(s["dims"], s["logits"], s["topk_idx"], s["ws"], d_loss=s["d_loss"],
                                   counts=s["counts"], seq_offsets=s["seq_offsets"], dlogits=s["dlogits"])
        return {n: s[n] for n in ("counts", "probs", "loss", "dlogits")}
    em.edge_moe_route_backward(s["dims"], s["logits"], s["topk_idx"], s["ws"], topk_w=s["topk_w"],
                               d_topk_w=s["d_topk_w"], d_loss=s["d_loss"], counts=s["counts"],
                               seq_offsets=s["seq_offsets"], x=s["x"], w_router=s["w_router"], dx=s["dx"],
                               dw_router=s["dw_router"], dbias=s["dbias"])
    return {n: s[n] for n in ("dx", "dw_router", "dbias")}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    kind = case["kind"]
    if kind == "mx_round":
        n = case["M"] * case["N"] * case["K"]
        wide = 2 if case["src"] == "bf16" else 4
        packed = (0.5 if case["fmt"] == "fp4" else 1.0) + 1 / 32
        return {"bytes": n * (2 * wide + 2 * packed), "flops": 4 * n}
    if kind == "mx_product":
        T, M, N, K, k = (case[n] for n in ("T", "M", "N", "K", "k"))
        R = T * max(1, k)
        live = M * (1 - (1 - 1 / M) ** R) if k else min(M, R)      # matrices that have rows
        return {"bytes": 2 * T * K + live * N * K * (0.5 + 1 / 32) + 2 * R * N, "flops": 2 * R * N * K}
    T, E, k, S = (case[n] for n in ("T", "E", "k", "S"))
    if kind == "balance":
        return {"bytes": 8 * T * E + 4 * T * k + 8 * S * E, "flops": 12 * T * E}
    d = case["d"]
    return {"bytes": 4 * T * E + 12 * T * k + 4 * S * E + 6 * T * d + 6 * E * d, "flops": 4 * T * E * d + 12 * T * E}


# ------------------------------------------------------------------ in 64 bits -----

def _exact_quantised(v, fp4):
    """float64 values of the round trip: every element against the format's sorted
    magnitudes, the nearer one, at equal distance the one with the even code."""
    if fp4:
        mags = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    else:
        mags = [m / 512 for m in range(8)] + [(8 + m) / 8 * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
        mags = mags[:127]                                            # the last code is NaN
    grid = torch.tensor(mags, dtype=torch.float64, device=DEV)
    b = v.double().unflatten(-1, (-1, 32))
    amax = b.abs().max(-1, keepdim=True).values
    bits = amax.view(torch.int64) >> 52                              # biased exponent of the float64
    x = (bits - 1023 - (2 if fp4 else 8)).clamp(-127, 127)
    step = ((torch.where(amax > 0, x, 0) + 1023) << 52).view(torch.float64)
    a = b.abs() / step
    mid = (grid[1:] + grid[:-1]) / 2
    low = torch.bucketize(a, mid)                                    # at a midpoint: the lower code
    up = low + ((low % 2 == 1) & (a == mid[low.clamp(max=len(mags) - 2)])).long()
    return (torch.where(b < 0, -1.0, 1.0) * grid[up] * step).flatten(-2)


def _exact_weights(codes, scales):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    e, m = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1))
    sc = torch.exp2(scales.movedim(-3, -2).flatten(-2).double() - 127)
    return torch.where(c > 7, -mag, mag) * sc.repeat_interleave(32, dim=-1)


def _exact_product(s):
    x = _exact_quantised(s["x"], s["fp4"])
    if s["row_src"] is not None:
        x = x[s["row_src"].long()]
    y = torch.empty(s["y"].shape, dtype=torch.float64, device=DEV)
    off = [0, x.shape[0]] if s["offsets"] is None else s["offsets"].tolist()
    for m in range(len(off) - 1):
        if off[m + 1] > off[m]:
            y[off[m]:off[m + 1]] = x[off[m]:off[m + 1]] @ _exact_weights(s["codes"][m], s["scales"][m]).t()
    return y


def _exact_router(s, kind):
    z = s["logits"].double()
    T, E, S = s["T"], s["E"], s["S"]
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    off = s["seq_offsets"].tolist()
    live = sum(off[i + 1] > off[i] for i in range(S))
    idx = s["topk_idx"].long()
    picks = torch.zeros(T, E, dtype=torch.float64, device=DEV).scatter_add_(1, idx, torch.ones(idx.shape, dtype=torch.float64, device=DEV))
    gb, gz = (float(v) for v in s["d_loss"].double())
    counts = torch.zeros(S, E, dtype=torch.float64, device=DEV)
    mean = torch.zeros(S, E, dtype=torch.float64, device=DEV)
    dz = 2 * gz / T * lse[:, None] * p
    bal = 0.0
    for i in range(S):
        lo, hi = off[i], off[i + 1]
        if hi == lo:
            continue
        counts[i] = picks[lo:hi].sum(0)
        mean[i] = p[lo:hi].mean(0)
        f = counts[i] * E / (s["k"] * (hi - lo))
        bal = bal + (f * mean[i]).sum() / live
        dz[lo:hi] += gb / live / (hi - lo) * p[lo:hi] * (f - (p[lo:hi] @ f)[:, None])
    if kind == "balance":
        return {"counts": None, "probs": mean, "loss": torch.stack([bal, lse.square().mean()]), "dlogits": dz}
    w, dw = s["topk_w"].double(), s["d_topk_w"].double()
    dz.scatter_add_(1, idx, w * dw - w * (w * dw).sum(1, keepdim=True))
    return {"dx": dz @ s["w_router"].double(), "dw_router": dz.t() @ s["x"].double(), "dbias": dz.sum(0)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "mx_round":
        return torch.cat([_exact_quantised(m, s["fp4"]).unsqueeze(0) for m in s["src"]])
    if case["kind"] == "mx_product":
        return _exact_product(s)
    return _exact_router(s, case["kind"])
