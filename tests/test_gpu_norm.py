"""The norm and its backward pass on the GPU against the formulas in float64.

The residual's sum and the MXFP8 codes are whole choices of their formats and
compared bit for bit; the rest to bounds that count float32 roundings (u = 2^-24
each) and the output's half step."""
import math

import numpy as np
import pytest
import torch

import shared_matrix_expert_amd as em
from oracle import operators as ops
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
# widths of one run of eight to the largest, on both sides of every number of waves a row
SHAPES = [(1, 8), (3, 64), (5, 504), (1, 512), (257, 520), (70, 1000), (4, 1024), (9, 1032), (333, 2048), (5, 2056), (1, 4096),
          (2100, 4096), (6, 4104), (37, 8192), (3, 8200), (2, 16384), (2, 16392), (3, 32768)]


def half(t):
    return torch.finfo(t).eps / 2


def rows(T, d, dtype, g, stride=None, scale=1.0):
    """T rows of d values; with a stride, of a wider buffer of NaN."""
    v = (scale * torch.randn(T, d, generator=g, device=DEV)).to(dtype)
    if stride is None:
        return v
    wide = torch.full((T, stride), float("nan"), dtype=dtype, device=DEV)
    wide[:, 8:8 + d] = v
    return wide[:, 8:8 + d]


def pow2(n):
    """2^n as float64, by its bits (torch's powers on the GPU are not exact)."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def to_bf16(v):
    """float64 to bf16, rounded once, as float64."""
    e = torch.frexp(v)[1].clamp(min=-125) - 8
    return torch.round(v * pow2(-e)) * pow2(e)


def forward(x, gain, eps, add):
    r = x.double() if add is None else to_bf16(x.double() + add.double())
    rstd = 1 / torch.sqrt((r * r).mean(1) + eps)
    return r, rstd, r * rstd[:, None] * gain.double()


def check_forward(x, gain, eps, add, strided=False):
    T, d = x.shape
    w = d + 24 if strided else d
    x_out = torch.full((T, w), 7.0, dtype=torch.bfloat16, device=DEV)[:, :d]
    y = torch.full((T, w), 7.0, dtype=torch.bfloat16, device=DEV)[:, :d]
    rstd = torch.full((T,), 7.0, device=DEV)
    codes = scales = None
    if d % 128 == 0:
        codes = torch.full((T, d), 0xEE, dtype=torch.uint8, device=DEV)
        scales = torch.full((d // 128, T, 4), 0xEE, dtype=torch.uint8, device=DEV)
    em.edge_moe_norm(x, gain, eps, add=add, x_out=x_out, y=y, codes=codes, scales=scales, rstd=rstd)
    torch.cuda.synchronize()
    r, s, yy = forward(x, gain, eps, add)
    assert torch.equal(x_out.double(), r), "the residual's sum differs"
    assert bool(((rstd.double() - s).abs() <= 1.01 * U * s).all())
    # rstd's rounding and two products, then bf16's half step (of a subnormal: 2^-134)
    tol = (half(torch.bfloat16) + 4 * U) * yy.abs() + 2.0 ** -134
    assert bool(((y.double() - yy).abs() <= tol).all())
    if codes is not None:
        q, e = ops.quantize(y.float().cpu().numpy().astype(np.float64), ops.FP8)
        assert np.array_equal(scales.cpu().numpy(), ops.by_step(e[None])[0]), "block scales differ"
        assert np.array_equal(codes.cpu().numpy(), q), "codes differ"
    if strided:
        for t in (x_out, y):
            assert bool((t._base[:, d:] == 7).all())
    return y, codes, scales


@pytest.mark.parametrize("add", [None, "bf16", "fp32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward_shapes(T, d, add):
    g = torch.Generator(device=DEV).manual_seed(T * 8191 + d)
    say(f"case: norm {T} x {d}, add {add}")
    gain = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(TYPES["fp32" if d % 3 else "bf16"])
    check_forward(rows(T, d, torch.bfloat16, g), gain, 1e-5, None if add is None else rows(T, d, TYPES[add], g))


@pytest.mark.parametrize("add", ["bf16", "fp32"])
def test_forward_rows_at_a_stride(add):
    g = torch.Generator(device=DEV).manual_seed(4)
    x, a = rows(33, 640, torch.bfloat16, g, 664), rows(33, 640, TYPES[add], g, 680)
    check_forward(x, torch.ones(640, device=DEV), 1e-6, a, strided=True)


def test_sum_is_rounded_once():
    """Sums on and one float32 step beside the middle of two bf16 values, where a sum
    rounded through float32 goes wrong; equal to edge_moe_residual's."""
    x = torch.tensor([1.0, 257 / 256 * 2, 3.0, -1.0, -5.0, 2.0 ** 100, 2.0 ** -100, 1.0], device=DEV).to(torch.bfloat16)
    mid = pow2(torch.frexp(x.double())[1] - 9)
    cases = []
    for sign in (1, -1):
        for tiny in (0.0, 2.0 ** -30, -2.0 ** -30, 2.0 ** -20, -2.0 ** -20):
            cases.append(sign * mid * (1 + tiny))
    a = torch.stack(cases).float()
    xs = x.expand(len(cases), 8).contiguous()
    check_forward(xs, torch.ones(8, device=DEV), 1e-5, a)
    out = torch.empty_like(xs)
    em.edge_moe_residual(xs, a, out)
    again = torch.empty_like(xs)
    em.edge_moe_norm(xs, torch.ones(8, device=DEV), 1e-5, add=a, x_out=again)
    assert torch.equal(out, again)


def test_rows_of_every_size_and_in_place():
    """Rows of 2^-120 to 2^120, of zeros, and of one value that outweighs all others."""
    g = torch.Generator(device=DEV).manual_seed(9)
    e = torch.arange(-120, 121, 16, device=DEV).double()
    x = (torch.randn(len(e), 256, generator=g, device=DEV).double() * pow2(e)[:, None]).to(torch.bfloat16)
    x[3] = 0
    x[5, 7] = 2.0 ** 127
    y, _, _ = check_forward(x, torch.ones(256, device=DEV), 1e-30, None)
    assert bool((y[3] == 0).all())
    a = torch.randn(len(e), 256, generator=g, device=DEV)
    want, _, _ = forward(x, torch.ones(256, device=DEV), 1e-5, a)
    em.edge_moe_norm(x, torch.ones(256, device=DEV), 1e-5, add=a, x_out=x)
    assert torch.equal(x.double(), want)


def test_rows_that_are_not_finite_stay_alone():
    g = torch.Generator(device=DEV).manual_seed(2)
    x = rows(9, 512, torch.bfloat16, g)
    x[2, 5], x[4, 9], x[6, 1] = float("nan"), float("inf"), float("-inf")
    y = torch.empty_like(x)
    codes, scales = torch.empty(9, 512, dtype=torch.uint8, device=DEV), torch.empty(4, 9, 4, dtype=torch.uint8, device=DEV)
    em.edge_moe_norm(x, torch.ones(512, device=DEV), 1e-5, y=y, codes=codes, scales=scales)
    ok = [0, 1, 3, 5, 7, 8]
    _, _, want = forward(x[ok], torch.ones(512, device=DEV), 1e-5, None)
    assert bool(((y[ok].double() - want).abs() <= (half(torch.bfloat16) + 4 * U) * want.abs()).all())
    assert bool(y[2].isnan().all()) and bool(y[4, 9].isnan()) and bool(y[6, 1].isnan())
    back = torch.empty(9, 512, dtype=torch.bfloat16, device=DEV)
    em.edge_moe_mx_dequantize(em.MX_FP8, codes, scales, back)
    assert bool(back[ok].isfinite().all()) and bool(back[2].isnan().all())


def backward(x, gain, rstd, dy, dres):
    x, gain, rstd, dy = x.double(), gain.double(), rstd.double()[:, None], dy.double()
    v, dv = x * rstd, dy * gain
    dx = rstd * (dv - v * (dv * v).mean(1, keepdim=True))
    mag = rstd * (dv.abs() + v.abs() * (dv * v).abs().mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
        mag = mag + dres.double().abs()
    return dx, mag, (dy * v).sum(0), (dy * v).abs().sum(0)


def check_backward(x, gain, rstd, dy, dres, dx, dgain):
    T, d = x.shape
    want, mag, wg, mg = backward(x, gain, rstd, dy, dres)
    # at most 32 products a lane are added in float32; v, dv, the mean and dr a rounding each
    if dx is not None:
        assert bool(((dx.double() - want).abs() <= 40 * U * mag + half(dx.dtype) * want.abs() + 2.0 ** -134).all())
    # a lane adds at most T / 256 rows (and one) in float32, four waves' sums follow
    if dgain is not None:
        assert bool(((dgain.double() - wg).abs() <= (T / 256 + 8) * U * mg + 1e-40).all())


def run_backward(x, gain, rstd, dy, dres=None, dx=None, dgain=None):
    T, d = x.shape
    ws = torch.full((em.edge_moe_norm_backward_ws_bytes(T, d) + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    em.edge_moe_norm_backward(x, gain, rstd, dy, ws[:-512], dres=dres, dx=dx, dgain=dgain)
    torch.cuda.synchronize()
    assert bool((ws[-512:] == 0xA5).all()), "wrote past the workspace"


@pytest.mark.parametrize("grad", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_backward_shapes(T, d, grad):
    g = torch.Generator(device=DEV).manual_seed(T * 8191 + d)
    say(f"case: norm backward {T} x {d}, {grad}")
    t = TYPES[grad]
    x, gain = rows(T, d, torch.bfloat16, g), (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(TYPES["bf16" if d % 3 else "fp32"])
    rstd = torch.empty(T, device=DEV)
    em.edge_moe_norm(x, gain, 1e-5, rstd=rstd)
    dy, dres = rows(T, d, t, g), rows(T, d, t, g) if T % 2 else None
    dx, dgain = torch.full((T, d), 7.0, dtype=t, device=DEV), torch.full((d,), 7.0, device=DEV)
    run_backward(x, gain, rstd, dy, dres, dx, dgain)
    check_backward(x, gain, rstd, dy, dres, dx, dgain)
    # each output alone has the bits it has with the other; dx over dres
    alone, galone = torch.empty_like(dx), torch.empty_like(dgain)
    run_backward(x, gain, rstd, dy, dres, dx=alone)
    run_backward(x, gain, rstd, dy, dres, dgain=galone)
    assert torch.equal(alone, dx) and torch.equal(galone, dgain)
    if dres is not None:
        run_backward(x, gain, rstd, dy, dres, dx=dres)
        assert torch.equal(dres, dx)


@pytest.mark.parametrize("grad", ["bf16", "fp32"])
def test_backward_rows_at_a_stride(grad):
    g = torch.Generator(device=DEV).manual_seed(6)
    t = TYPES[grad]
    x, dy, dres = rows(41, 1000, torch.bfloat16, g, 1024), rows(41, 1000, t, g, 1016), rows(41, 1000, t, g, 1032)
    gain, rstd = torch.randn(1000, generator=g, device=DEV), torch.rand(41, generator=g, device=DEV) + 0.5
    wide = torch.full((41, 1040), 3.0, dtype=t, device=DEV)
    dgain = torch.empty(1000, device=DEV)
    run_backward(x, gain, rstd, dy, dres, wide[:, 16:1016], dgain)
    check_backward(x, gain, rstd, dy, dres, wide[:, 16:1016], dgain)
    assert bool((wide[:, :16] == 3).all()) and bool((wide[:, 1016:] == 3).all())


def test_backward_against_differences():
    """Gradients against central differences of the forward formula in float64."""
    g = torch.Generator(device=DEV).manual_seed(8)
    x, a = rows(6, 64, torch.bfloat16, g), None
    gain, dy = 1 + 0.3 * torch.randn(64, generator=g, device=DEV), torch.randn(6, 64, generator=g, device=DEV)
    rstd, dx, dgain = torch.empty(6, device=DEV), torch.empty(6, 64, device=DEV), torch.empty(64, device=DEV)
    em.edge_moe_norm(x, gain, 1e-5, rstd=rstd)
    run_backward(x, gain, rstd, dy, None, dx, dgain)

    def loss(xv, gv):
        return (dy.double() * xv * gv / torch.sqrt((xv * xv).mean(1, keepdim=True) + 1e-5)).sum()
    h = 1e-5
    for t, i in ((0, 0), (2, 17), (5, 63)):
        e = torch.zeros(6, 64, dtype=torch.float64, device=DEV)
        e[t, i] = h
        num = (loss(x.double() + e, gain.double()) - loss(x.double() - e, gain.double())) / (2 * h)
        assert abs(float(num) - float(dx[t, i])) <= 1e-5 * max(1.0, abs(float(num)))
        num = (loss(x.double(), gain.double() + e[t]) - loss(x.double(), gain.double() - e[t])) / (2 * h)
        assert abs(float(num) - float(dgain[i])) <= 1e-5 * max(1.0, abs(float(num)))


def test_no_rows():
    gain = torch.ones(64, device=DEV)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    em.edge_moe_norm(x, gain, 1e-5, y=torch.empty_like(x))
    dgain = torch.full((64,), 7.0, device=DEV)
    run_backward(x, gain, torch.empty(0, device=DEV), torch.empty(0, 64, device=DEV), dgain=dgain)
    assert bool((dgain == 0).all())


def test_side_stream_and_graph_replays():
    g = torch.Generator(device=DEV).manual_seed(1)
    T, d = 700, 1024
    gain = torch.ones(d, device=DEV)
    x, a, dy = rows(T, d, torch.bfloat16, g), rows(T, d, torch.float32, g), rows(T, d, torch.float32, g)
    x_out, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device=DEV)
    dx, dgain = torch.empty(T, d, device=DEV), torch.empty(d, device=DEV)
    ws = torch.empty(em.edge_moe_norm_backward_ws_bytes(T, d), dtype=torch.uint8, device=DEV)

    def step():
        em.edge_moe_norm(x, gain, 1e-5, add=a, x_out=x_out, y=y, rstd=rstd)
        em.edge_moe_norm_backward(x_out, gain, rstd, dy, ws, dx=dx, dgain=dgain)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        x.copy_(rows(T, d, torch.bfloat16, g))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (x_out, y, rstd, dx, dgain)]
        for t in (x_out, y, rstd, dx, dgain):
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(want, (x_out, y, rstd, dx, dgain))), seed
