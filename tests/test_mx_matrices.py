"""Host-side checks of the MX matrix operators (no GPU needed): the oracle's
own pins, the library's refusals before any device call (fake addresses that
are never dereferenced), and the binding's checks of what it is given."""
import ctypes

import numpy as np
import pytest
import torch

import shared_matrix_expert_amd as em
from oracle import mx
from oracle import operators as ops

BASE = 1 << 40                                  # never dereferenced


# ------------------------------------------------------------------ the oracle ----

def test_e2m1_encoder_against_brute_force():
    rng = np.random.default_rng(0)
    grid = mx.e2m1_to_f64(np.arange(8))
    mids = (grid[1:] + grid[:-1]) / 2
    v = np.concatenate([grid, mids, np.nextafter(mids, 0), np.nextafter(mids, 9), rng.uniform(0, 9, 2000)])
    for sign in (1.0, -1.0):
        got = ops.e2m1_encode(sign * v)
        assert np.all((got >> 3) == (sign < 0))
        for a, c in zip(v, got & 7):
            d = np.abs(grid - a)
            best = np.nonzero(d == d.min())[0]
            want = best[0] if best.size == 1 else best[best % 2 == 0][0]
            assert c == want, (a, c, want)
    assert ops.e2m1_encode(np.array([-0.0]))[0] == 8


def test_quantize_agrees_with_the_layers_rounding():
    v = np.random.default_rng(1).standard_normal((5, 256)) * np.exp2(np.arange(-2, 3))[:, None] * 7
    v[2, :32] = 0
    codes, x = ops.quantize(v, ops.FP8)
    want, xw = mx.quant_mxfp8(v)
    assert np.array_equal(codes, want) and np.array_equal(x, xw)


def test_quantize_non_finite_blocks_and_zero_blocks():
    v = np.ones((1, 128))
    v[0, 3] = np.nan
    v[0, 40] = -np.inf
    v[0, 64:96] = 0
    for fmt in (ops.FP4, ops.FP8):
        codes, x = ops.quantize(v, fmt)
        assert x[0].tolist() == [255, 255, 0, 127 - (2 if fmt == ops.FP4 else 8)]
        assert not codes[0, :96].any()
        back = ops.values(codes, x, fmt)
        assert np.isnan(back[0, :64]).all() and not back[0, 64:96].any() and (back[0, 96:] == 1).all()


# ------------------------------------------------------------------ refusals ------

@pytest.mark.parametrize("name", ["edge_moe_mx_quantize", "edge_moe_mx_dequantize"])
def test_round_validation_before_any_device_call(name):
    ok = dict(M=2, N=3, K=256, fmt=em.MX_FP4, type=0, dense=BASE, stride=256, codes=BASE, scales=BASE)

    def call(**kw):
        a = {**ok, **kw}
        dense = (a["dense"], a["stride"])
        packed = (a["codes"], a["scales"])
        args = dense + packed if name.endswith("_quantize") else packed + dense
        return getattr(em.load(), name)(a["M"], a["N"], a["K"], a["fmt"], a["type"], *args, None)
    for bad in (dict(M=0), dict(N=0), dict(N=-1), dict(K=0), dict(fmt=2), dict(fmt=-1), dict(type=2),
                dict(dense=None), dict(dense=BASE + 8), dict(codes=None), dict(codes=BASE + 4), dict(scales=None),
                dict(scales=BASE + 2), dict(stride=255), dict(stride=260), dict(stride=-256),
                dict(type=1, stride=258)):
        assert call(**bad) == em.EDGE_MOE_EINVAL, bad
    for bad in (dict(K=96, stride=96), dict(K=32896, stride=32896), dict(M=1 << 20, N=1 << 20),
                dict(M=1 << 9, N=(1 << 18) + 1, K=128, stride=128)):       # more rows than a launch holds
        assert call(**bad) == em.EDGE_MOE_EUNSUPPORTED, bad


def test_binding_checks_shapes_types_and_devices():
    src = torch.zeros(2, 3, 256, dtype=torch.bfloat16)
    codes, scales = torch.zeros(2, 3, 128, dtype=torch.uint8), torch.zeros(2, 2, 3, 4, dtype=torch.uint8)
    for bad in (dict(codes=codes[:1]), dict(scales=scales[:1]), dict(codes=codes.to(torch.int8)),
                dict(src=src[0, 0]), dict(fmt=7), dict(fmt=em.MX_FP8)):
        a = {**dict(fmt=em.MX_FP4, src=src, codes=codes, scales=scales), **bad}
        with pytest.raises(ValueError):
            em.edge_moe_mx_quantize(a["fmt"], a["src"], a["codes"], a["scales"])
    assert em._row_stride(src) == 256
    assert em._row_stride(torch.zeros(2, 3, 512)[..., :256]) == 512
    assert em._row_stride(torch.zeros(1, 1, 128)) == 128
    assert em._row_stride(torch.zeros(4, 6, 128)[:, :1]) == 768
    for t in (torch.zeros(4, 6, 128)[:, :3], torch.zeros(128, 4).t(), torch.zeros(128)):
        with pytest.raises(ValueError):
            em._row_stride(t)
    with pytest.raises(ValueError):
        em._dense_type(src.half())


def test_product_validation_before_any_device_call():
    lib = em.load()
    ok = dict(T=8, R=8, M=1, N=64, K=256, fmt=em.MX_FP8, x=BASE, xs=256, src=None, off=None, q=BASE, e=BASE, y=BASE,
              ys=64, ws=BASE, nb=1 << 30)

    def call(**kw):
        a = {**ok, **kw}
        d = em.CMxDims(a["T"], a["R"], a["M"], a["N"], a["K"], a["fmt"])
        return lib.edge_moe_mx_product(ctypes.byref(d), a["x"], a["xs"], a["src"], a["off"], a["q"], a["e"], a["y"],
                                       a["ys"], a["ws"], a["nb"], None)
    for bad in (dict(T=0), dict(R=-1), dict(M=0), dict(N=0), dict(K=0), dict(fmt=2), dict(x=None), dict(x=BASE + 8),
                dict(xs=248), dict(xs=260), dict(src=BASE + 2), dict(off=BASE + 1), dict(q=None), dict(q=BASE + 8),
                dict(e=BASE + 2), dict(y=None), dict(y=BASE + 1), dict(ys=63), dict(M=2), dict(R=9), dict(ws=BASE + 16)):
        assert call(**bad) == em.EDGE_MOE_EINVAL, bad
    for bad in (dict(K=192, xs=192), dict(T=(1 << 20) + 1), dict(R=(1 << 25) + 1, src=BASE), dict(M=1025, off=BASE),
                dict(N=32769, ys=32769), dict(K=32896, xs=32896)):
        assert call(**bad) == em.EDGE_MOE_EUNSUPPORTED, bad
    assert call(ws=None) == em.EDGE_MOE_EWORKSPACE
    need = em.edge_moe_mx_product_ws_bytes(8, 8, 1, 64, 256, em.MX_FP8)
    assert need >= 8 * (256 + 8) and call(nb=need - 1) == em.EDGE_MOE_EWORKSPACE
    assert lib.edge_moe_mx_product(None, BASE, 256, None, None, BASE, BASE, BASE, 64, BASE, 1 << 30, None) == em.EDGE_MOE_EINVAL
    assert em.edge_moe_mx_product_ws_bytes(8, 8, 1, 64, 200, em.MX_FP8) == 0


def test_product_binding_checks():
    x, y = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.bfloat16)
    q, e = torch.zeros(1, 64, 128, dtype=torch.uint8), torch.zeros(1, 2, 64, 4, dtype=torch.uint8)
    ws = torch.zeros(4096, dtype=torch.uint8)
    ok = dict(x=x, codes=q, scales=e, y=y)
    for bad in (dict(x=x.float()), dict(x=x[0]), dict(codes=q[..., :64]), dict(scales=e[..., :2]), dict(y=y.float()),
                dict(y=y[:, :32]), dict(offsets=torch.zeros(3, dtype=torch.int32)), dict(offsets=torch.zeros(2)),
                dict(row_src=torch.zeros(5, dtype=torch.int32)), dict(row_src=torch.zeros(4, dtype=torch.int64)), {}):
        a = {**ok, **bad}
        with pytest.raises((ValueError, RuntimeError, AssertionError)):     # the last: host tensors
            em.edge_moe_mx_product(em.MX_FP8, a.pop("x"), a.pop("codes"), a.pop("scales"), a.pop("y"), ws, **a)


def test_product_refuses_rows_past_32_bits():
    y = torch.empty((1 << 32) + 4, 1, dtype=torch.bfloat16, device="meta")
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    q, e = torch.zeros(1, 1, 64, dtype=torch.uint8), torch.zeros(1, 1, 1, 4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="too many rows"):
        em.edge_moe_mx_product(em.MX_FP8, x, q, e, y, torch.zeros(4096, dtype=torch.uint8))


def test_tensors_must_be_on_the_current_gpu(monkeypatch):
    class On:
        def __init__(self, dev):
            self.dev, self.device = dev, f"cuda:{dev}"

        def get_device(self):
            return self.dev
    em.load()
    monkeypatch.setattr(em._cuda, "getDevice", lambda: 1)
    assert em._same_device(On(1), None, On(1)) == 1
    for bad in ((On(0), On(0)), (On(1), On(0)), (On(-1), On(-1)), (On(1), None, On(-1))):
        with pytest.raises(ValueError):
            em._same_device(*bad)
