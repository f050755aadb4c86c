"""Workloads of the operators around the expert layer: the norm between layers,
dense expert matrices and their training, and products with int4 matrices.

Five kinds of pass:

* ``norm``: the residual's addition, the root-mean-square norm and its output in
  bf16 or in MXFP8 (edge_moe_norm);
* ``norm_backward``: its gradients at the residual stream and the gain
  (edge_moe_norm_backward);
* ``dense``: the product of token rows with bf16 matrices, one matrix or one per
  expert with ragged rows (edge_moe_dense_product);
* ``dense_backward``: its gradients at x and at the matrices
  (edge_moe_dense_product_backward);
* ``int4``: the product of token rows with int4 matrices in the layer's own
  storage (edge_moe_packed_product).

``run`` computes a pass in plain torch operations, or through the library
where ``own`` is true; ``exact`` gives the definition in float64.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-5


def listed():
    return [
        # the residual and norm in front of a layer in decoding: one token, MXFP8 out for the products behind it
        dict(name="norm one token", kind="norm", T=1, d=4096, add="fp32", gain="bf16", out="codes"),
        # the same over a 16K prompt
        dict(name="norm prompt", kind="norm", T=16384, d=4096, add="fp32", gain="bf16", out="codes"),
        # a first norm of a small odd width: nothing to add, bf16 out, float32 gain
        dict(name="norm odd width", kind="norm", T=777, d=1000, add="none", gain="fp32", out="bf16"),
        # training: an odd batch of the small test layer's width
        dict(name="norm backward small", kind="norm_backward", T=333, d=512, grad="fp32", gain="fp32"),
        # training: a batch at full width, gradients kept in bf16
        dict(name="norm backward batch", kind="norm_backward", T=16384, d=4096, grad="bf16", gain="bf16"),
        # a verify batch through its experts' rank-128 inputs before they are quantised: 8 tokens, ten of 512 experts each
        dict(name="dense verify experts", kind="dense", T=8, M=512, N=128, K=4096, k=10, out="bf16"),
        # a training batch sorted by group through the groups' shared up matrices
        dict(name="dense batch groups", kind="dense", T=16384, M=8, N=8192, K=4096, k=0, out="bf16"),
        # training of the LoRA inputs, rank 16: an odd batch, three of eight groups a token
        dict(name="dense backward lora", kind="dense_backward", T=1501, M=8, N=16, K=4096, k=3, out="fp32"),
        # training of the groups' shared down matrices: an odd batch sorted by group, gradients in bf16
        dict(name="dense backward groups", kind="dense_backward", T=5001, M=8, N=4096, K=8192, k=0, out="bf16"),
        # one token through one group's shared up matrix
        dict(name="int4 one token", kind="int4", T=1, M=1, N=8192, K=4096, k=0, gq=128, out="fp32"),
        # a verify batch through its experts' rank-128 inputs: 8 tokens, ten of 512 experts each
        dict(name="int4 verify experts", kind="int4", T=8, M=512, N=128, K=4096, k=10, gq=128, out="bf16"),
        # a short ragged prompt sorted by group through the groups' shared down matrices
        dict(name="int4 ragged groups", kind="int4", T=1001, M=8, N=4096, K=8192, k=0, gq=128, out="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def _grouped(rng, most_rows, k_step):
    """T rows (or T tokens' picks of k of M matrices) and matrices of N x K."""
    while True:
        M = 1 if rng.random() < 0.3 else _log(rng, 2, 512)
        k = min(M, rng.choice([0, rng.randint(2, 10)])) if M > 1 else 0
        c = dict(T=_log(rng, 1, most_rows), M=M, N=8 * _log(rng, 1, 1024), K=k_step * _log(rng, 1, 8192 // k_step), k=k)
        R = c["T"] * max(1, k)
        if M * c["N"] * c["K"] <= 1 << 28 and R * max(c["N"], c["K"]) <= 1 << 27 and R * c["N"] * c["K"] <= 1 << 38:
            return c


def draw(rng):
    kind = rng.choice(["norm", "norm_backward", "dense", "dense_backward", "int4"])
    if kind.startswith("norm"):
        while True:
            d = 128 * _log(rng, 1, 64) if rng.random() < 0.5 else 8 * _log(rng, 8, 1024)
            c = dict(kind=kind, T=_log(rng, 1, 16384), d=d, gain=rng.choice(["bf16", "fp32"]))
            if c["T"] * d > 1 << 26:
                continue
            if kind == "norm":
                return dict(c, add=rng.choice(["none", "bf16", "fp32"]), out=rng.choice(["bf16", "codes"]) if d % 128 == 0 else "bf16")
            return dict(c, grad=rng.choice(["bf16", "fp32"]))
    if kind == "int4":
        c = dict(_grouped(rng, 4096, 32), kind=kind, out=rng.choice(["bf16", "fp32"]))
        return dict(c, gq=rng.choice([g for g in (32, 64, 128, 256) if c["K"] % min(g, c["K"]) == 0]))
    return dict(_grouped(rng, 16384, 8), kind=kind, out=rng.choice(["bf16", "fp32"]))


# ------------------------------------------------------------------ inputs ---------

_TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _cuts(total, parts, seed):
    """parts + 1 offsets from 0 to total, ragged."""
    rng = np.random.default_rng(seed)
    share = rng.dirichlet(np.full(parts, 4.0))
    cut = np.floor(np.cumsum(share)[:-1] * total).astype(np.int64)
    return np.concatenate([[0], cut, [total]])


def _plan(s, case, g, seed):
    """A batch's rows sorted by matrix: offsets, the token of each row, the rows of each token."""
    T, M, k = case["T"], case["M"], case["k"]
    s.update(offsets=None, row_src=None, token_rows=None)
    if M == 1:
        return
    if k:                                                            # k distinct matrices a token
        pick = torch.rand(T, M, generator=g, device=DEV).topk(k, dim=1).indices
        order = torch.argsort(pick.reshape(-1) * T + torch.arange(T, device=DEV).repeat_interleave(k))
        s["row_src"] = (order // k).to(torch.int32)
        s["token_rows"] = torch.argsort(order).reshape(T, k).to(torch.int32)
        off = np.concatenate([[0], np.cumsum(np.bincount(pick.cpu().numpy().reshape(-1), minlength=M))])
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


def prepare(case, seed):
    kind = case["kind"]
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 29)
    s = dict(case)
    if kind.startswith("norm"):
        T, d = case["T"], case["d"]
        s["gain"] = (1 + 0.1 * _randn(g, d)).to(_TYPE[case["gain"]])
        scale = torch.exp(0.5 * _randn(g, T, 1))                     # tokens of different sizes
        if kind == "norm":
            s["x"] = (scale * _randn(g, T, d)).to(torch.bfloat16)
            s["add"] = None if case["add"] == "none" else (0.2 * scale * _randn(g, T, d)).to(_TYPE[case["add"]])
            s["x_out"] = None if s["add"] is None else torch.empty_like(s["x"])
            s["rstd"] = torch.empty(T, device=DEV)
            s["y"] = s["codes"] = s["scales"] = None
            if case["out"] == "bf16":
                s["y"] = torch.empty_like(s["x"])
            else:
                s["codes"] = torch.empty(T, d, dtype=torch.uint8, device=DEV)
                s["scales"] = torch.empty(d // 128, T, 4, dtype=torch.uint8, device=DEV)
            return s
        t = _TYPE[case["grad"]]
        s["x"] = (scale * _randn(g, T, d)).to(torch.bfloat16)
        s["rstd"] = torch.rsqrt(s["x"].double().square().mean(1) + EPS).float()       # the forward pass left it
        s["dy"] = (0.01 * _randn(g, T, d)).to(t)
        s["dres"] = (0.01 * _randn(g, T, d)).to(t)
        s["dx"] = torch.empty(T, d, dtype=t, device=DEV)
        s["dgain"] = torch.empty(d, device=DEV)
        return s
    T, M, N, K, k = (case[n] for n in ("T", "M", "N", "K", "k"))
    R, t = T * max(1, k), _TYPE[case["out"]]
    s["x"] = _randn(g, T, K).to(torch.bfloat16)
    _plan(s, case, g, seed)
    if kind == "int4":
        s["codes"] = torch.randint(0, 256, (M, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
        s["scales"] = (0.002 + 0.004 * torch.rand(M, N, K // min(case["gq"], K), generator=g, device=DEV)).to(torch.float16)
    else:
        s["w"] = (0.02 * _randn(g, M, N, K)).to(torch.bfloat16)
    if kind == "dense_backward":
        s["dy"] = _randn(g, R, N).to(torch.bfloat16)
        s["dx"] = torch.empty(T, K, dtype=t, device=DEV)
        s["dw"] = torch.empty(M, N, K, dtype=t, device=DEV)
    else:
        s["y"] = torch.empty(R, N, dtype=t, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms ----

def _sum_bf16(x, add):
    """bf16 of the exact sum: where float32 lands on the middle of two bf16 values,
    what it lost decides."""
    exact = x.double() + add.double()
    f = exact.float()
    bits = f.view(torch.int32)
    lost = torch.sign(exact - f.double()) * torch.sign(f)
    bits = torch.where((bits & 0xFFFF) == 0x8000, bits + lost.int(), bits)
    return bits.view(torch.float32).to(torch.bfloat16)


def _pow2(n):
    """2^n as float32 for whole n in -126 .. 127, by its bits."""
    return ((n + 127) << 23).view(torch.float32)


def _mxfp8(y):
    """E4M3 codes [T][d] and E8M0 scales [d/128][T][4] of bf16 rows, each as its own type."""
    b = y.float().unflatten(1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, (torch.frexp(amax)[1] - 9).clamp(-126, 127), -126)
    a = b * _pow2(-e)
    m = (torch.frexp(a)[1] - 1).clamp(min=-6)
    a = (torch.round(a * _pow2(3 - m)) * _pow2(m - 3)).clamp(-448, 448)
    scales = (e + 127).to(torch.uint8).reshape(len(y), -1, 4).transpose(0, 1).contiguous()
    return a.flatten(1).to(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def _int4(s):
    """float32 values of int4 matrices, the low nibble first."""
    q = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).flatten(-2).float()
    q = torch.where(q > 7, q - 16, q)
    sc = s["scales"].float()
    return (q.unflatten(-1, (sc.shape[-1], -1)) * sc.unsqueeze(-1)).flatten(-2)


def _plain(s):
    kind = s["kind"]
    if kind == "norm":
        r = s["x"] if s["add"] is None else _sum_bf16(s["x"], s["add"])
        rstd = torch.rsqrt(r.float().square().mean(1, keepdim=True) + EPS)
        y = (r.float() * rstd * s["gain"].float()).to(torch.bfloat16)
        out = {"rstd": rstd.squeeze(1)}
        if s["add"] is not None:
            out["x_out"] = r
        if s["out"] == "bf16":
            out["y"] = y
        else:
            out["codes"], out["scales"] = _mxfp8(y)
        return out
    if kind == "norm_backward":
        v = s["x"].float() * s["rstd"].unsqueeze(1)
        dy = s["dy"].float()
        dv = dy * s["gain"].float()
        dx = s["dres"].float() + s["rstd"].unsqueeze(1) * (dv - v * (dv * v).mean(1, keepdim=True))
        return {"dx": dx.to(s["dx"].dtype), "dgain": (dy * v).double().sum(0).float()}
    x, one = s["x"].float(), s["offsets"] is None
    w = _int4(s) if kind == "int4" else s["w"].float()
    src = None if one else s["rows"] if s["row_src"] is None else s["row_src"].long()[s["rows"]]
    if kind != "dense_backward":
        y = x @ w[0].t() if one else torch.bmm(x[src], w[s["active"]].transpose(1, 2).contiguous())[s["keep"]]
        return y.to(s["y"].dtype)
    dy, dw = s["dy"].float(), torch.zeros(s["dw"].shape, device=DEV)
    if one:
        dx = dy @ w[0]
        dw[0] = dy.t() @ x
    else:
        dyp = dy[s["rows"]] * s["keep"].unsqueeze(-1)
        dx = torch.bmm(dyp, w[s["active"]])[s["keep"]]
        dw[s["active"]] = torch.bmm(dyp.transpose(1, 2).contiguous(), x[src])
        if s["token_rows"] is not None:
            dx = dx[s["token_rows"].long()].sum(1)
    return {"dx": dx.to(s["dx"].dtype), "dw": dw.to(s["dw"].dtype)}


# ------------------------------------------------------------------ one pass -------

def _ws(s, nbytes):
    """The workspace, allocated once, as a user's program keeps it."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(1, nbytes()), dtype=torch.uint8, device=DEV)
    return s["ws"]


def _own(s):
    import shared_matrix_expert_amd as em
    kind = s["kind"]
    if kind == "norm":
        em.edge_moe_norm(s["x"], s["gain"], EPS, add=s["add"], x_out=s["x_out"], y=s["y"], codes=s["codes"],
                         scales=s["scales"], rstd=s["rstd"])
        out = {"rstd": s["rstd"]}
        if s["add"] is not None:
            out["x_out"] = s["x_out"]
        if s["out"] == "bf16":
            out["y"] = s["y"]
        else:
            out["codes"], out["scales"] = s["codes"].view(torch.float8_e4m3fn), s["scales"].view(torch.float8_e8m0fnu)
        return out
    if kind == "norm_backward":
        em.edge_moe_norm_backward(s["x"], s["gain"], s["rstd"], s["dy"],
                                  _ws(s, lambda: em.edge_moe_norm_backward_ws_bytes(s["T"], s["d"])), dres=s["dres"],
                                  dx=s["dx"], dgain=s["dgain"])
        return {"dx": s["dx"], "dgain": s["dgain"]}
    T, M, N, K = (s[n] for n in ("T", "M", "N", "K"))
    R = T * max(1, s["k"])
    if kind == "int4":
        ws = _ws(s, lambda: em.edge_moe_packed_product_ws_bytes(T, R, M, N, K, s["gq"]))
        em.edge_moe_packed_product(s["gq"], s["x"], s["codes"], s["scales"], s["y"], ws, offsets=s["offsets"], row_src=s["row_src"])
        return s["y"]
    if kind == "dense":
        ws = _ws(s, lambda: em.edge_moe_dense_product_ws_bytes(T, R, M, N, K))
        em.edge_moe_dense_product(s["x"], s["w"], s["y"], ws, offsets=s["offsets"], row_src=s["row_src"])
        return s["y"]
    ws = _ws(s, lambda: em.edge_moe_dense_product_backward_ws_bytes(T, R, M, N, K))
    em.edge_moe_dense_product_backward(s["dy"], ws, x=s["x"], w=s["w"], dx=s["dx"], dw=s["dw"], offsets=s["offsets"],
                                       row_src=s["row_src"], token_rows=s["token_rows"])
    return {"dx": s["dx"], "dw": s["dw"]}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    kind = case["kind"]
    wide = {"bf16": 2, "fp32": 4, "none": 0}
    if kind == "norm":
        n = case["T"] * case["d"]
        out = 2 if case["out"] == "bf16" else 1 + 1 / 32
        return {"bytes": n * (2 + wide[case["add"]] + (0 if case["add"] == "none" else 2) + out), "flops": 6 * n}
    if kind == "norm_backward":
        n = case["T"] * case["d"]
        return {"bytes": n * (2 + 3 * wide[case["grad"]]), "flops": 12 * n}
    T, M, N, K, k = (case[n] for n in ("T", "M", "N", "K", "k"))
    R, out = T * max(1, k), wide[case["out"]]
    live = M * (1 - (1 - 1 / M) ** R) if k else min(M, R)              # matrices that have rows
    if kind == "dense_backward":
        return {"bytes": 2 * R * N + 2 * T * K + 2 * live * N * K + out * (T * K + M * N * K), "flops": 4 * R * N * K}
    w = 2 if kind == "dense" else 0.5 + 2 / min(case["gq"], K)
    return {"bytes": 2 * T * K + live * N * K * w + out * R * N, "flops": 2 * R * N * K}


# ------------------------------------------------------------------ in 64 bits -----

def _nearest(v, digits, least):
    """float64 values to `digits` significant bits, ties to even, no finer than 2^least."""
    e = torch.frexp(v)[1].double() - digits
    step = torch.exp2(e.clamp(min=least))
    return torch.round(v / step) * step


def _exact_norm(s):
    r = s["x"].double()
    if s["add"] is not None:
        r = _nearest(r + s["add"].double(), 8, -133)
    rstd = 1 / torch.sqrt((r * r).sum(1) / s["d"] + EPS)
    y = r * rstd[:, None] * s["gain"].double()
    out = {"rstd": rstd}
    if s["add"] is not None:
        out["x_out"] = r
    if s["out"] == "bf16":
        out["y"] = y
        return out
    b = _nearest(y, 8, -133).reshape(s["T"], s["d"] // 32, 32)
    big = b.abs().max(-1).values
    scale = torch.exp2(torch.where(big > 0, torch.frexp(big)[1].double() - 9, -127.0).clamp(min=-127))
    a = _nearest(b / scale[..., None], 4, -9)
    out["codes"] = torch.clamp(a, -448, 448).reshape(s["T"], s["d"])
    out["scales"] = scale.reshape(s["T"], -1, 4).permute(1, 0, 2).contiguous()
    return out


def _exact_int4(codes, scales):
    c = codes.long()
    lo, hi = c % 16, c // 16
    q = torch.stack([lo - 16 * (lo >= 8), hi - 16 * (hi >= 8)], -1).flatten(-2).double()
    return q * scales.double().repeat_interleave(q.shape[-1] // scales.shape[-1], -1)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        return _exact_norm(s)
    if kind == "norm_backward":
        x, g, rstd, dy = (s[n].double() for n in ("x", "gain", "rstd", "dy"))
        h = dy * g
        dot = (h * x).sum(1)
        dx = s["dres"].double() + rstd[:, None] * h - x * (rstd ** 3 * dot / s["d"])[:, None]
        return {"dx": dx, "dgain": (dy * x * rstd[:, None]).sum(0)}
    x = s["x"].double()
    xr = x if s["row_src"] is None else x[s["row_src"].long()]
    off = [0, xr.shape[0]] if s["offsets"] is None else s["offsets"].tolist()
    parts = [(m, off[m], off[m + 1]) for m in range(len(off) - 1) if off[m + 1] > off[m]]
    if kind == "dense_backward":
        dxr, dw = torch.empty(xr.shape, dtype=torch.float64, device=DEV), torch.zeros(s["dw"].shape, dtype=torch.float64, device=DEV)
        for m, a, b in parts:
            dy = s["dy"][a:b].double()
            dxr[a:b] = dy @ s["w"][m].double()
            dw[m] = dy.t() @ xr[a:b]
        if s["row_src"] is None:
            return {"dx": dxr, "dw": dw}
        return {"dx": torch.zeros_like(x).index_add_(0, s["row_src"].long(), dxr), "dw": dw}
    y = torch.empty(s["y"].shape, dtype=torch.float64, device=DEV)
    for m, a, b in parts:
        w = _exact_int4(s["codes"][m], s["scales"][m]) if kind == "int4" else s["w"][m].double()
        y[a:b] = xr[a:b] @ w.t()
    return y
