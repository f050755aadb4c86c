"""What the binding of the MX-matrix and router-training operators checks before
the library is called (its kernels trust these sizes), one argument at a time:
each case is the valid call with one tensor changed, and the error names it.
Tensors and the library are stand-ins that say they are on the GPU, so that no
other check can answer in place of the one meant."""
from types import SimpleNamespace

import pytest
import torch

import shared_matrix_expert_amd as em
from fakes import OnGpu, Recorder, fake, on_device

U8, I32, BF16, F32 = torch.uint8, torch.int32, torch.bfloat16, torch.float32
T, E, K, D, S = 5, 8, 2, 128, 3
DIMS = SimpleNamespace(T=T, d=D, h=128, n_experts=E, experts_per_group=E, top_k=K, delta_rank=8, lora_rank=2, quant_group=32)
M, N, C, R = 2, 16, 256, 6                                  # matrices of N x C, R rows of y

# argument -> (shape, type) of each call, all of them given
ROUTER = dict(logits=((T, E), F32), topk_idx=((T, K), I32), seq_offsets=((S + 1,), I32), counts=((S, E), I32))
CALLS = {
    "balance": dict(ROUTER, probs=((S, E), F32), loss=((2,), F32)),
    "route_backward": dict(ROUTER, topk_w=((T, K), F32), d_topk_w=((T, K), F32), d_loss=((2,), F32), x=((T, D), BF16),
                           w_router=((E, D), BF16), dlogits=((T, E), F32), dx=((T, D), F32), dw_router=((E, D), F32),
                           dbias=((E,), F32)),
    "mx_quantize": dict(src=((M, N, C), BF16), codes=((M, N, C // 2), U8), scales=((M, C // 128, N, 4), U8)),
    "mx_dequantize": dict(dst=((M, N, C), BF16), codes=((M, N, C // 2), U8), scales=((M, C // 128, N, 4), U8)),
    "mx_product": dict(x=((T, C), BF16), y=((R, N), BF16), codes=((M, N, C // 2), U8), scales=((M, C // 128, N, 4), U8),
                       offsets=((M + 1,), I32), row_src=((R,), I32)),
}
WITH_WS = ("balance", "route_backward", "mx_product")
ROWS = {"src", "dst", "x", "y"}                             # taken at a row stride (x of the router's calls is not)


@pytest.fixture
def lib(monkeypatch):
    on_device(monkeypatch, 0, stream=0x99)
    r = Recorder()
    monkeypatch.setattr(em, "_lib", r)
    return r


def tensors(name):
    a = {k: fake(*shape, dtype=t, address=(1 << 40) + (i << 32)) for i, (k, (shape, t)) in enumerate(CALLS[name].items())}
    if name in WITH_WS:
        a["ws"] = fake(999, dtype=U8, address=1 << 50)
    return a


def call(name, a):
    a = dict(a)
    if name == "balance":
        return em.edge_moe_balance(DIMS, *(a.pop(n) for n in ("logits", "topk_idx", "counts", "probs", "loss", "ws")), **a)
    if name == "route_backward":
        return em.edge_moe_route_backward(DIMS, a.pop("logits"), a.pop("topk_idx"), a.pop("ws"), **a)
    if name == "mx_product":
        return em.edge_moe_mx_product(em.MX_FP8, *(a.pop(n) for n in ("x", "codes", "scales", "y", "ws")), **a)
    order = ("src", "codes", "scales") if name == "mx_quantize" else ("codes", "scales", "dst")
    return getattr(em, "edge_moe_" + name)(em.MX_FP4, *(a[n] for n in order))


def meta(t):
    return t._t


def other_type(t):
    return torch.float64 if t.dtype != torch.float64 else F32


ARGS = [(c, a) for c in CALLS for a in CALLS[c]]
args = pytest.mark.parametrize("name,arg", ARGS, ids=[f"{c}-{a}" for c, a in ARGS])


def test_valid_calls_reach_the_library(lib):
    """Every address, size and stream in its place."""
    for name in CALLS:
        a = tensors(name)
        call(name, a)
        (fn, got), = lib.calls
        lib.calls.clear()
        assert fn == "edge_moe_" + name
        p = {k: v.data_ptr() for k, v in a.items()}
        if name == "balance":
            assert list(got[1:]) == [p["logits"], p["topk_idx"], p["seq_offsets"], S, p["counts"], p["probs"], p["loss"],
                                     p["ws"], 999, 0x99]
        elif name == "route_backward":
            g = got[1]
            assert {n: getattr(g, n) for n, _ in g._fields_} == {**{k: v for k, v in p.items() if k != "ws"}, "n_seq": S}
            assert list(got[2:]) == [p["ws"], 999, 0x99]
        elif name == "mx_product":
            assert [getattr(got[0], n) for n, _ in got[0]._fields_] == [T, R, M, N, C, em.MX_FP8]
            assert list(got[1:]) == [p["x"], C, p["row_src"], p["offsets"], p["codes"], p["scales"], p["y"], N, p["ws"], 999, 0x99]
        else:
            dense = [p["src" if name == "mx_quantize" else "dst"], C]
            packed = [p["codes"], p["scales"]]
            assert list(got) == [M, N, C, em.MX_FP4, 0, *(dense + packed if name == "mx_quantize" else packed + dense), 0x99]
        if name in ("balance", "route_backward"):
            assert [getattr(got[0], n) for n in ("T", "d", "n_experts", "top_k")] == [T, D, E, K]


def refuses(lib, name, match, **changed):
    with pytest.raises(ValueError, match=match):
        call(name, {**tensors(name), **changed})
    assert not lib.calls


@args
def test_counts(lib, name, arg):
    t = meta(tensors(name)[arg])
    for n in {0, t.numel() - 1, t.numel() + 1, 2 * t.numel()}:
        bad = OnGpu(torch.empty(n, dtype=t.dtype, device="meta"))
        if name.startswith("mx_") and arg in ROWS:           # rows set the sizes: then the others do not fit them
            bad = OnGpu(torch.empty(t.shape[-2], n + 128, dtype=t.dtype, device="meta"))
            refuses(lib, name, "^(codes|scales):", **{arg: bad})
        elif name == "mx_product" and arg == "codes":        # the first dimension sets the number of matrices
            for width in (0, C // 2 - 1, C // 2 + 1, C):
                refuses(lib, name, "^codes: expected", codes=fake(M, N, width, dtype=U8))
        elif arg == "seq_offsets":                           # sets the number of sequences
            refuses(lib, name, "^(counts|seq_offsets):", **{arg: bad})
        else:
            refuses(lib, name, f"^{arg}: expected", **{arg: bad})


@args
def test_types(lib, name, arg):
    t = meta(tensors(name)[arg])
    match = "bfloat16" if t.dtype == BF16 else f"^{arg}: expected"
    refuses(lib, name, match, **{arg: OnGpu(t.to(other_type(t)))})
    if t.dtype == I32:
        refuses(lib, name, match, **{arg: OnGpu(t.to(torch.int64))})


@args
def test_contiguity(lib, name, arg):
    t = meta(tensors(name)[arg])
    apart = torch.empty(*t.shape, 2, dtype=t.dtype, device="meta")[..., 0]
    match = "contiguous" if name.startswith("mx_") and arg in ROWS else f"^{arg}: expected"
    refuses(lib, name, match, **{arg: OnGpu(apart)})


@args
def test_devices(lib, name, arg):
    t = meta(tensors(name)[arg])
    for device in (1, -1):
        refuses(lib, name, "must be on (one|the current) GPU", **{arg: OnGpu(t, device=device)})


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("device", [1, -1])
def test_current_device(lib, name, device):
    moved = {k: OnGpu(meta(v), device=device) for k, v in tensors(name).items()}
    refuses(lib, name, "must be on the current GPU", **moved)


@pytest.mark.parametrize("name", WITH_WS)
def test_workspaces(lib, name):
    refuses(lib, name, "must be on one GPU", ws=fake(999, dtype=U8, device=1))
    refuses(lib, name, "contiguous", ws=OnGpu(torch.empty(999, 2, dtype=U8, device="meta")[:, 0]))
    call(name, {**tensors(name), "ws": fake(999, dtype=torch.int32, address=1 << 50)})
    assert 4 * 999 in lib.calls[0][1]                        # bytes, whatever the type


@pytest.mark.parametrize("name", ["mx_quantize", "mx_dequantize"])
def test_formats(lib, name):
    a = tensors(name)
    for fmt in (2, -1, None):
        with pytest.raises(ValueError, match="format"):
            order = ("src", "codes", "scales") if name == "mx_quantize" else ("codes", "scales", "dst")
            getattr(em, "edge_moe_" + name)(fmt, *(a[n] for n in order))
    refuses(lib, name, "^codes:", codes=fake(M, N, C, dtype=U8))         # FP8's codes
    dense = "src" if name == "mx_quantize" else "dst"
    refuses(lib, name, "two dimensions", **{dense: fake(C, dtype=BF16)})


def test_product_matrices(lib):
    """One matrix without its leading dimension; x and y of rows."""
    a = tensors("mx_product")
    call("mx_product", {**a, "codes": fake(N, C // 2, dtype=U8), "scales": fake(C // 128, N, 4, dtype=U8),
                        "offsets": fake(2, dtype=I32)})
    assert lib.calls.pop()[1][0].M == 1
    for arg in ("x", "y"):
        refuses(lib, "mx_product", "rows", **{arg: fake(3, *a[arg].shape, dtype=BF16)})


@pytest.mark.parametrize("name,dense", [("mx_quantize", "src"), ("mx_dequantize", "dst"), ("mx_product", "x"), ("mx_product", "y")])
def test_row_strides(lib, name, dense):
    """Rows of a wider buffer pass their stride on; rows at several strides are refused."""
    t = meta(tensors(name)[dense])
    wide = torch.empty(*t.shape[:-1], t.shape[-1] + 128, dtype=t.dtype, device="meta")[..., :t.shape[-1]]
    call(name, {**tensors(name), dense: OnGpu(wide)})
    assert t.shape[-1] + 128 in lib.calls.pop()[1]
    if t.dim() == 3:
        refuses(lib, name, "one stride", **{dense: OnGpu(torch.empty(M, N + 1, C, dtype=BF16, device="meta")[:, :N])})
