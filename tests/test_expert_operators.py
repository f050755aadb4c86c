"""Host-side checks of the norm and of the products with dense and int4 matrices (no
GPU needed): the library's refusals before any device call (fake addresses that are
never dereferenced), and what the binding checks, one argument at a time, with
stand-ins that say they are on the GPU."""
import ctypes

import pytest
import torch

import shared_matrix_expert_amd as em
from fakes import OnGpu, Recorder, fake, on_device

BASE = 1 << 40                                  # never dereferenced
BF16, F32, I32, U8, F16 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.float16
INVALID, UNSUPPORTED, WORKSPACE = em.EDGE_MOE_EINVAL, em.EDGE_MOE_EUNSUPPORTED, em.EDGE_MOE_EWORKSPACE


# ------------------------------------------------------------------ refusals ------

def refused(call, cases):
    for status, bad in cases:
        for b in bad:
            assert call(**b) == status, b


def test_norm_validation_before_any_device_call():
    ok = dict(T=4, d=256, eps=1e-5, add_type=1, gain_type=0, x=BASE, x_stride=256, add=BASE, add_stride=256, gain=BASE, x_out=BASE,
              x_out_stride=256, y=BASE, y_stride=256, codes=BASE, scales=BASE, rstd=BASE)

    def call(**kw):
        return em.load().edge_moe_norm(ctypes.byref(em.CNormArgs(**{**ok, **kw})), None)
    none = dict(x_out=None, y=None, codes=None, scales=None, rstd=None)
    refused(call, [
        (INVALID, [dict(T=-1), dict(d=0), dict(d=4), dict(d=252), dict(d=-8), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                   dict(eps=float("inf")), dict(add_type=2), dict(gain_type=-1), dict(x=None), dict(x=BASE + 8), dict(x_stride=248),
                   dict(x_stride=260), dict(x_stride=(1 << 32) + 8), dict(add=BASE + 8), dict(add_stride=258), dict(add_stride=8),
                   dict(add_type=0, add_stride=260), dict(gain=None), dict(gain=BASE + 4), dict(x_out=BASE + 2), dict(x_out_stride=255),
                   dict(y=BASE + 8), dict(y_stride=0), dict(codes=None), dict(scales=None), dict(codes=BASE + 8), dict(scales=BASE + 2),
                   dict(rstd=BASE + 2), none]),
        (UNSUPPORTED, [dict(T=(1 << 25) + 1), dict(d=32776, x_stride=32776), dict(d=248)])])
    assert em.load().edge_moe_norm(None, None) == INVALID


def test_norm_backward_validation_before_any_device_call():
    ok = dict(T=4, d=256, gain_type=0, grad_type=1, x=BASE, x_stride=256, gain=BASE, rstd=BASE, dy=BASE, dy_stride=256, dres=BASE,
              dres_stride=256, dx=BASE, dx_stride=256, dgain=BASE)
    need = em.edge_moe_norm_backward_ws_bytes(4, 256)

    def call(ws=BASE, nb=need, **kw):
        return em.load().edge_moe_norm_backward(ctypes.byref(em.CNormGrad(**{**ok, **kw})), ws, nb, None)
    refused(call, [
        (INVALID, [dict(T=-1), dict(d=12), dict(gain_type=2), dict(grad_type=2), dict(x=None), dict(x=BASE + 8), dict(x_stride=128),
                   dict(gain=None), dict(rstd=None), dict(rstd=BASE + 2), dict(dy=None), dict(dy_stride=254), dict(dres=BASE + 8),
                   dict(dres_stride=8), dict(dx=BASE + 4), dict(dx_stride=258), dict(grad_type=0, dx_stride=260), dict(dgain=BASE + 1),
                   dict(dx=None, dgain=None), dict(ws=BASE + 16)]),
        (UNSUPPORTED, [dict(T=(1 << 25) + 1), dict(d=32776, x_stride=32776)]),
        (WORKSPACE, [dict(ws=None), dict(nb=need - 1)])])
    assert em.load().edge_moe_norm_backward(None, BASE, 1 << 30, None) == INVALID
    assert need >= 256 * 4 and em.edge_moe_norm_backward_ws_bytes(0, 8) > 0
    for bad in ((-1, 256), (4, 4), (4, 32776), ((1 << 25) + 1, 8), ((1 << 32) + 4, 8)):
        assert em.edge_moe_norm_backward_ws_bytes(*bad) == 0


def test_dense_validation_before_any_device_call():
    ok = dict(T=8, R=8, M=1, N=64, K=256, x=BASE, xs=256, src=None, off=None, w=BASE, yt=0, y=BASE, ys=64, ws=BASE, nb=1 << 40)

    def call(**kw):
        a = {**ok, **kw}
        d = em.CDenseDims(*(a[n] for n in ("T", "R", "M", "N", "K")))
        return em.load().edge_moe_dense_product(ctypes.byref(d), *(a[n] for n in ("x", "xs", "src", "off", "w", "yt", "y", "ys", "ws", "nb")), None)
    refused(call, [
        (INVALID, [dict(T=0), dict(R=-1), dict(M=0), dict(N=0), dict(N=4), dict(N=60), dict(K=0), dict(K=252), dict(x=None),
                   dict(x=BASE + 8), dict(xs=248), dict(xs=260), dict(xs=(1 << 32) + 8), dict(src=BASE + 2), dict(off=BASE + 1),
                   dict(w=None), dict(w=BASE + 8), dict(yt=2), dict(y=None), dict(y=BASE + 8), dict(ys=56), dict(ys=68),
                   dict(yt=1, ys=66), dict(M=2), dict(R=9), dict(ws=BASE + 16)]),
        (UNSUPPORTED, [dict(T=(1 << 20) + 1), dict(R=(1 << 25) + 1, src=BASE), dict(M=1025, off=BASE), dict(N=32776, ys=32776),
                       dict(K=32776, xs=32776)]),
        (WORKSPACE, [dict(ws=None), dict(nb=em.edge_moe_dense_product_ws_bytes(8, 8, 1, 64, 256) - 1)])])
    assert em.load().edge_moe_dense_product(None, BASE, 256, None, None, BASE, 0, BASE, 64, BASE, 1 << 30, None) == INVALID
    for bad in ((0, 8, 1, 64, 256), (8, 8, 1, 60, 256), (8, 8, 1, 64, 32776), (8, 8, 1025, 64, 256), (8, 1 << 33, 1, 64, 256)):
        assert em.edge_moe_dense_product_ws_bytes(*bad) == 0 and em.edge_moe_dense_product_backward_ws_bytes(*bad) == 0


def test_dense_backward_validation_before_any_device_call():
    ok = dict(dy=BASE, dy_stride=64, x=BASE, x_stride=256, row_src=BASE, offsets=BASE, token_rows=BASE, per_token=2, w=BASE, dx=BASE,
              dx_stride=256, dx_type=1, dw_type=1, dw=BASE)
    dims = (8, 16, 2, 64, 256)
    need = em.edge_moe_dense_product_backward_ws_bytes(*dims)

    def call(dims=dims, ws=BASE, nb=1 << 40, **kw):
        return em.load().edge_moe_dense_product_backward(ctypes.byref(em.CDenseDims(*dims)), ctypes.byref(em.CDenseGrad(**{**ok, **kw})), ws, nb, None)
    refused(call, [
        (INVALID, [dict(dims=(0, 16, 2, 64, 256)), dict(dims=(8, 16, 2, 12, 256)), dict(dy=None), dict(dy=BASE + 8), dict(dy_stride=56),
                   dict(dy_stride=68), dict(x=None), dict(x=BASE + 8), dict(x_stride=252), dict(row_src=BASE + 2), dict(row_src=None),
                   dict(offsets=None), dict(offsets=BASE + 2), dict(token_rows=BASE + 1), dict(per_token=0), dict(per_token=-1),
                   dict(w=None), dict(w=BASE + 8), dict(dx=BASE + 8), dict(dx_stride=248), dict(dx_stride=258), dict(dx_type=2),
                   dict(dw_type=-1), dict(dw=BASE + 8), dict(dx=None, dw=None), dict(ws=BASE + 8)]),
        (UNSUPPORTED, [dict(dims=(8, 16, 1025, 64, 256)), dict(per_token=1025)]),
        (WORKSPACE, [dict(ws=None), dict(nb=need - 1)])])
    assert em.load().edge_moe_dense_product_backward(ctypes.byref(em.CDenseDims(*dims)), None, BASE, 1 << 40, None) == INVALID
    assert need >= 16 * 256 * 4                                  # dx's rows, added up by token


def test_packed_validation_before_any_device_call():
    ok = dict(T=8, R=8, M=1, N=65, K=256, q=64, x=BASE, xs=256, src=None, off=None, c=BASE, s=BASE, yt=0, y=BASE, ys=65, ws=BASE, nb=1 << 40)

    def call(**kw):
        a = {**ok, **kw}
        d = em.CPackedDims(*(a[n] for n in ("T", "R", "M", "N", "K", "q")))
        return em.load().edge_moe_packed_product(ctypes.byref(d), *(a[n] for n in ("x", "xs", "src", "off", "c", "s", "yt", "y", "ys", "ws", "nb")), None)
    refused(call, [
        (INVALID, [dict(T=0), dict(R=-1), dict(M=0), dict(N=0), dict(K=0), dict(K=16), dict(K=248), dict(q=0), dict(q=16), dict(q=48),
                   dict(q=8192), dict(K=96, q=64, xs=96), dict(x=None), dict(x=BASE + 8), dict(xs=248), dict(xs=260), dict(src=BASE + 2),
                   dict(off=BASE + 1), dict(c=None), dict(c=BASE + 8), dict(s=None), dict(s=BASE + 2), dict(yt=2), dict(y=None),
                   dict(y=BASE + 1), dict(yt=1, y=BASE + 2), dict(ys=64), dict(M=2), dict(R=9), dict(ws=BASE + 16)]),
        (UNSUPPORTED, [dict(T=(1 << 20) + 1), dict(R=(1 << 25) + 1, src=BASE), dict(M=1025, off=BASE), dict(N=32769, ys=32769),
                       dict(K=32768 + 64, xs=40000)]),
        (WORKSPACE, [dict(ws=None), dict(nb=em.edge_moe_packed_product_ws_bytes(8, 8, 1, 65, 256, 64) - 1)])])
    assert em.load().edge_moe_packed_product(None, BASE, 256, None, None, BASE, BASE, 0, BASE, 65, BASE, 1 << 30, None) == INVALID
    for bad in ((0, 8, 1, 64, 256, 64), (8, 8, 1, 64, 200, 64), (8, 8, 1, 64, 256, 33), (8, 8, 1, 1 << 33, 256, 64)):
        assert em.edge_moe_packed_product_ws_bytes(*bad) == 0


def test_coded_product_validation_before_any_device_call():
    ok = dict(T=8, R=8, M=1, N=64, K=256, fmt=em.MX_FP8, x=BASE, xs=BASE, src=None, off=None, q=BASE, e=BASE, y=BASE, ys=64)

    def call(**kw):
        a = {**ok, **kw}
        d = em.CMxDims(*(a[n] for n in ("T", "R", "M", "N", "K", "fmt")))
        return em.load().edge_moe_mx_product_coded(ctypes.byref(d), *(a[n] for n in ("x", "xs", "src", "off", "q", "e", "y", "ys")), None)
    refused(call, [
        (INVALID, [dict(T=0), dict(R=-1), dict(M=0), dict(N=0), dict(K=0), dict(fmt=2), dict(x=None), dict(x=BASE + 8), dict(xs=None),
                   dict(xs=BASE + 2), dict(src=BASE + 2), dict(off=BASE + 1), dict(q=None), dict(q=BASE + 8), dict(e=BASE + 2), dict(y=None),
                   dict(y=BASE + 1), dict(ys=63), dict(ys=(1 << 32) + 1), dict(M=2), dict(R=9)]),
        (UNSUPPORTED, [dict(K=192), dict(T=(1 << 20) + 1), dict(R=(1 << 25) + 1, src=BASE), dict(M=1025, off=BASE),
                       dict(N=32769, ys=32769), dict(K=32896)])])
    assert em.load().edge_moe_mx_product_coded(None, BASE, BASE, None, None, BASE, BASE, BASE, 64, None) == INVALID


# ------------------------------------------------------------------ the binding ---

T, D, M, N, K, R, PER, Q = 5, 256, 2, 64, 256, 6, 3, 64
CALLS = {
    "norm": dict(x=((T, D), BF16), gain=((D,), F32), add=((T, D), F32), x_out=((T, D), BF16), y=((T, D), BF16), codes=((T, D), U8),
                 scales=((D // 128, T, 4), U8), rstd=((T,), F32)),
    "norm_backward": dict(x=((T, D), BF16), gain=((D,), BF16), rstd=((T,), F32), dy=((T, D), F32), dres=((T, D), F32), dx=((T, D), F32),
                          dgain=((D,), F32)),
    "dense_product": dict(x=((T, K), BF16), w=((M, N, K), BF16), y=((R, N), F32), offsets=((M + 1,), I32), row_src=((R,), I32)),
    "dense_product_backward": dict(dy=((R, N), BF16), x=((T, K), BF16), w=((M, N, K), BF16), dx=((T, K), F32), dw=((M, N, K), F32),
                                   offsets=((M + 1,), I32), row_src=((R,), I32), token_rows=((T, PER), I32)),
    "mx_product_coded": dict(x_codes=((T, K), U8), x_scales=((K // 128, T, 4), U8), codes=((M, N, K // 2), U8),
                             scales=((M, K // 128, N, 4), U8), y=((R, N), BF16), offsets=((M + 1,), I32), row_src=((R,), I32)),
    "packed_product": dict(x=((T, K), BF16), codes=((M, N, K // 2), U8), scales=((M, N, K // Q), F16), y=((R, N), F32),
                           offsets=((M + 1,), I32), row_src=((R,), I32)),
}
WITH_WS = [n for n in CALLS if n not in ("norm", "mx_product_coded")]
ARGS = [(c, a) for c in CALLS for a in CALLS[c]]
args = pytest.mark.parametrize("name,arg", ARGS, ids=[f"{c}-{a}" for c, a in ARGS])


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
    first = {"norm": ("x", "gain"), "norm_backward": ("x", "gain", "rstd", "dy", "ws"), "dense_product": ("x", "w", "y", "ws"),
             "dense_product_backward": ("dy", "ws"), "packed_product": ("x", "codes", "scales", "y", "ws"),
             "mx_product_coded": ("x_codes", "x_scales", "codes", "scales", "y")}[name]
    lead = [a.pop(n) for n in first]
    if name == "norm":
        lead.append(1e-5)
    if name in ("packed_product", "mx_product_coded"):
        lead.insert(0, Q if name == "packed_product" else em.MX_FP8)
    return getattr(em, "edge_moe_" + name)(*lead, **a)


def values(struct):
    return {n: getattr(struct, n) for n, _ in struct._fields_}


def test_valid_calls_reach_the_library(lib):
    """Every address, size, stride, type and stream in its place."""
    for name in CALLS:
        a = tensors(name)
        call(name, a)
        (fn, got), = lib.calls
        lib.calls.clear()
        assert fn == "edge_moe_" + name
        p = {k: v.data_ptr() for k, v in a.items()}
        if name == "norm":
            v = values(got[0])
            assert abs(v.pop("eps") - 1e-5) < 1e-12
            assert v == {**p, "T": T, "d": D, "add_type": 1, "gain_type": 1, "x_stride": D, "add_stride": D, "x_out_stride": D, "y_stride": D}
            assert got[1] == 0x99
        elif name == "norm_backward":
            assert values(got[0]) == {**{k: v for k, v in p.items() if k != "ws"}, "T": T, "d": D, "gain_type": 0, "grad_type": 1,
                                      "x_stride": D, "dy_stride": D, "dres_stride": D, "dx_stride": D}
            assert list(got[1:]) == [p["ws"], 999, 0x99]
        elif name == "dense_product_backward":
            assert list(values(got[0]).values()) == [T, R, M, N, K]
            assert values(got[1]) == {**{k: v for k, v in p.items() if k != "ws"}, "dy_stride": N, "x_stride": K, "dx_stride": K,
                                      "per_token": PER, "dx_type": 1, "dw_type": 1}
            assert list(got[2:]) == [p["ws"], 999, 0x99]
        elif name == "dense_product":
            assert list(values(got[0]).values()) == [T, R, M, N, K]
            assert list(got[1:]) == [p["x"], K, p["row_src"], p["offsets"], p["w"], 1, p["y"], N, p["ws"], 999, 0x99]
        elif name == "mx_product_coded":
            assert list(values(got[0]).values()) == [T, R, M, N, K, em.MX_FP8]
            assert list(got[1:]) == [p["x_codes"], p["x_scales"], p["row_src"], p["offsets"], p["codes"], p["scales"], p["y"], N, 0x99]
        else:
            assert list(values(got[0]).values()) == [T, R, M, N, K, Q]
            assert list(got[1:]) == [p["x"], K, p["row_src"], p["offsets"], p["codes"], p["scales"], 1, p["y"], N, p["ws"], 999, 0x99]


def test_outputs_that_are_not_asked_for(lib):
    """Only what is given is passed on; dx by rows without token_rows."""
    a = tensors("norm")
    call("norm", {n: a[n] for n in ("x", "gain", "y")})
    v = values(lib.calls.pop()[1][0])
    assert [v[n] for n in ("add", "x_out", "codes", "scales", "rstd")] == [None] * 5 and v["y"] == a["y"].data_ptr()
    a = tensors("dense_product_backward")
    call("dense_product_backward", {"dy": a["dy"], "ws": a["ws"], "w": a["w"], "offsets": a["offsets"], "dx": fake(R, K, dtype=BF16)})
    dims, g = lib.calls.pop()[1][:2]
    assert values(dims)["R"] == R and g.dw is None and g.dx_type == 0 and g.token_rows is None
    call("dense_product_backward", {n: a[n] for n in ("dy", "ws", "x", "dw", "offsets", "row_src")})
    g = lib.calls.pop()[1][1]
    assert g.dx is None and g.w is None and g.dw == a["dw"].data_ptr()
    for bad in (dict(dy=a["dy"], ws=a["ws"]), dict(dy=a["dy"], ws=a["ws"], dx=a["dx"]), dict(dy=a["dy"], ws=a["ws"], dw=a["dw"])):
        with pytest.raises(ValueError):
            call("dense_product_backward", bad)


@pytest.mark.parametrize("rows", [T, R])
def test_token_rows_without_a_row_are_not_dx_by_rows(lib, rows):
    """[T][0] names no rows of any token: refused, whatever rows dx has."""
    for extra in ({}, dict(x=None, dw=None)):
        refuses(lib, "dense_product_backward", token_rows=fake(rows, 0, dtype=I32), dx=fake(R, K, dtype=F32), **extra)


def refuses(lib, name, **changed):
    with pytest.raises((ValueError, em.EdgeMoeError)):
        call(name, {**tensors(name), **changed})
    assert not lib.calls


@args
def test_shapes(lib, name, arg):
    t = tensors(name)[arg]._t
    if t.dim() == 1:
        wrong = [torch.empty(t.shape[0] + 1, dtype=t.dtype, device="meta"), torch.empty(0, dtype=t.dtype, device="meta")]
    else:
        wrong = [torch.empty(*t.shape[:-1], t.shape[-1] + 8, dtype=t.dtype, device="meta"),
                 torch.empty(*t.shape[:-2], t.shape[-2] + 1, t.shape[-1], dtype=t.dtype, device="meta")]
        if (name, arg) == ("dense_product_backward", "token_rows"):
            wrong = wrong[1:]                                    # the second dimension is the caller's
        if (name, arg) in (("dense_product", "x"), ("packed_product", "x")):
            wrong = wrong[:1]                                    # x's rows set T
    for w in wrong:
        refuses(lib, name, **{arg: OnGpu(w)})
    refuses(lib, name, **{arg: OnGpu(t.flatten()[:0])})


@args
def test_types(lib, name, arg):
    t = tensors(name)[arg]._t
    refuses(lib, name, **{arg: OnGpu(t.to(torch.float64))})
    if t.dtype == I32:
        refuses(lib, name, **{arg: OnGpu(t.to(torch.int64))})


@args
def test_contiguity(lib, name, arg):
    t = tensors(name)[arg]._t
    refuses(lib, name, **{arg: OnGpu(torch.empty(*t.shape, 2, dtype=t.dtype, device="meta")[..., 0])})


@args
def test_devices(lib, name, arg):
    for device in (1, -1):
        refuses(lib, name, **{arg: OnGpu(tensors(name)[arg]._t, device=device)})


@pytest.mark.parametrize("name", list(CALLS))
def test_current_device_and_streams(lib, name):
    refuses(lib, name, **{k: OnGpu(v._t, device=1) for k, v in tensors(name).items()})

    class Stream:
        device_index, cuda_stream = 1, 0x77
    refuses(lib, name, stream=Stream())
    Stream.device_index = 0
    call(name, {**tensors(name), "stream": Stream()})
    assert lib.calls[0][1][-1] == 0x77


@pytest.mark.parametrize("name", WITH_WS)
def test_workspaces(lib, name):
    refuses(lib, name, ws=fake(999, dtype=U8, device=1))
    refuses(lib, name, ws=OnGpu(torch.empty(999, 2, dtype=U8, device="meta")[:, 0]))
    call(name, {**tensors(name), "ws": fake(999, dtype=torch.int32, address=1 << 50)})
    assert 4 * 999 in lib.calls[0][1]                            # bytes, whatever the type


ROWS = [("norm", "x"), ("norm", "add"), ("norm", "x_out"), ("norm", "y"), ("norm_backward", "x"), ("norm_backward", "dy"),
        ("norm_backward", "dres"), ("norm_backward", "dx"), ("dense_product", "x"), ("dense_product", "y"),
        ("dense_product_backward", "dy"), ("dense_product_backward", "x"), ("dense_product_backward", "dx"),
        ("packed_product", "x"), ("packed_product", "y")]


@pytest.mark.parametrize("name,arg", ROWS, ids=[f"{a}-{b}" for a, b in ROWS])
def test_row_strides(lib, name, arg):
    """Rows of a wider buffer pass their stride on; rows at several strides are refused."""
    t = tensors(name)[arg]._t
    wide = torch.empty(t.shape[0], t.shape[1] + 136, dtype=t.dtype, device="meta")[:, :t.shape[1]]
    call(name, {**tensors(name), arg: OnGpu(wide)})
    got = lib.calls.pop()[1]
    seen = [v for g in got for v in (values(g).values() if hasattr(g, "_fields_") else [g])]
    assert t.shape[1] + 136 in seen
    if name.startswith("norm") and arg == "x":
        deep = torch.empty(3, 4, D, dtype=BF16, device="meta")[:, :2]
        with pytest.raises(ValueError, match="one stride"):
            call(name, {**{k: OnGpu(torch.empty(6, *v._t.shape[1:], dtype=v._t.dtype, device="meta")) if v._t.shape[:1] == (T,) else v
                           for k, v in tensors(name).items()}, arg: OnGpu(deep)})


def test_one_matrix_without_its_leading_dimension(lib):
    call("dense_product", {**tensors("dense_product"), "w": fake(N, K, dtype=BF16), "offsets": fake(2, dtype=I32)})
    assert lib.calls.pop()[1][0].M == 1
    call("packed_product", {**tensors("packed_product"), "codes": fake(N, K // 2, dtype=U8), "scales": fake(N, K // Q, dtype=F16),
                            "offsets": fake(2, dtype=I32)})
    assert lib.calls.pop()[1][0].M == 1
    call("dense_product_backward", {**tensors("dense_product_backward"), "w": fake(N, K, dtype=BF16), "dw": fake(N, K),
                                    "offsets": fake(2, dtype=I32)})
    assert lib.calls.pop()[1][0].M == 1
    refuses(lib, "dense_product_backward", dw=fake(M + 1, N, K))


def test_bit_patterns_pass_for_their_types(lib):
    a = tensors("packed_product")
    call("packed_product", {**a, "x": fake(T, K, dtype=torch.int16), "scales": fake(M, N, K // Q, dtype=torch.int16),
                            "y": fake(R, N, dtype=torch.int16)})
    assert lib.calls.pop()[1][7] == 0
