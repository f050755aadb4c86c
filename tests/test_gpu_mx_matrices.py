"""The MX matrix operators on the GPU against the float64 oracle.

Quantiser and dequantiser: codes, scales and values are whole choices of the
format, so they are compared bit for bit.
"""
import numpy as np
import pytest
import torch

import shared_matrix_expert_amd as em
import synth
from oracle import operators as ops
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

FORMATS = [(em.MX_FP4, "fp4"), (em.MX_FP8, "fp8")]
fmt_of = pytest.mark.parametrize("fmt", [f for f, _ in FORMATS], ids=[n for _, n in FORMATS])


def quantize(fmt, src):
    """src [M][N][K] device tensor -> (codes, scales) as host arrays."""
    M, N, K = src.shape
    codes = torch.full((M, N, K // 2 if fmt == em.MX_FP4 else K), 0xEE, dtype=torch.uint8, device=DEV)
    scales = torch.full((M, K // 128, N, 4), 0xEE, dtype=torch.uint8, device=DEV)
    em.edge_moe_mx_quantize(fmt, src, codes, scales)
    torch.cuda.synchronize()
    return codes, scales


def check_quantize(fmt, src):
    codes, scales = quantize(fmt, src)
    want, x = ops.quantize(src.float().cpu().numpy().astype(np.float64), fmt)
    assert np.array_equal(scales.cpu().numpy(), ops.by_step(x)), "block scales differ"
    got, want = codes.cpu().numpy(), ops.pack(want, fmt)
    assert np.array_equal(got, want), f"{(got != want).sum()} of {want.size} code bytes differ"
    return codes, scales


def all_bf16():
    """Every finite bf16, both signs, ascending magnitude."""
    bits = np.arange(0x7F80, dtype=np.uint16)
    return np.stack([bits, bits | 0x8000], 1).reshape(-1)


@fmt_of
@pytest.mark.parametrize("order", ["neighbours", "one binade up", "shuffled"])
def test_quantize_every_bf16(fmt, order):
    bits = all_bf16()
    if order == "shuffled":
        bits = np.random.default_rng(3).permutation(bits)
    bits = bits.reshape(-1, 32).copy()
    if order == "one binade up":                 # a block's maximum up to 2^8 above its other elements
        top = bits.max(1) & 0x7FFF
        bits[:, 31] = np.minimum(top.astype(np.int64) + 128 * (1 + np.arange(len(bits)) % 8), 0x7F7F)
    bits = bits[:len(bits) // 4 * 4].reshape(1, -1, 128)
    src = torch.from_numpy(bits.view(np.int16)).to(DEV).view(torch.bfloat16)
    say(f"case: every bf16, {order}, {src.shape[1]} rows")
    check_quantize(fmt, src)


@fmt_of
def test_quantize_float32_ties_and_subnormals(fmt):
    """float32 values on and one step beside every rounding boundary of the
    format, at scales through the whole exponent range."""
    grid = np.sort(np.unique(np.abs(ops.values(np.arange(16 if fmt == em.MX_FP4 else 256) & (0xF if fmt == em.MX_FP4 else 0x7E),
                                               np.full(1 if fmt == em.MX_FP4 else 8, 127), fmt)
                                    if fmt == em.MX_FP8 else ops.mx.e2m1_to_f64(np.arange(8)))))
    mids = ((grid[1:] + grid[:-1]) / 2).astype(np.float32)
    pts = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(1e9)), grid.astype(np.float32)])
    pts = np.concatenate([pts, -pts])
    pts = np.pad(pts, (0, -len(pts) % 31))
    blocks = []
    for e in (-149, -140, -127, -126, -60, -3, 0, 1, 40, 110):
        b = np.zeros((len(pts) // 31, 32), np.float32)
        b[:, :31] = pts.reshape(-1, 31)
        b[:, 31] = grid[-1]                       # the block's largest magnitude: the format's own
        with np.errstate(over="ignore", under="ignore"):
            blocks.append(np.ldexp(b, e))
    v = np.concatenate(blocks)
    v = v[np.isfinite(v).all(1)]
    v = np.pad(v, ((0, -len(v) % 4), (0, 0))).reshape(1, -1, 128)
    check_quantize(fmt, torch.from_numpy(v.copy()).to(DEV))


@fmt_of
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 1, 128), (1, 17, 640), (3, 5, 512), (2, 33, 4096), (7, 1, 256)])
def test_quantize_shapes_and_back(fmt, dtype, shape):
    g = torch.Generator(device=DEV).manual_seed(5)
    src = (torch.randn(*shape, generator=g, device=DEV) * torch.exp2(torch.randint(-30, 30, (*shape[:-1], 1), generator=g, device=DEV).float())).to(dtype)
    codes, scales = check_quantize(fmt, src)
    for out_t in (torch.float32, torch.bfloat16):
        dst = torch.full(shape, 7.0, dtype=out_t, device=DEV)
        em.edge_moe_mx_dequantize(fmt, codes, scales, dst)
        want = torch.from_numpy(ops.rounded(src.float().cpu().numpy().astype(np.float64), fmt)).to(out_t)
        assert torch.equal(dst.cpu(), want)


@fmt_of
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_at_a_stride(fmt, dtype):
    """Rows of a wider buffer on both sides; what lies between the rows is neither
    read into a result nor written."""
    wide = torch.full((2, 9, 512), float("nan"), dtype=dtype, device=DEV)
    src = wide[..., 128:384]
    src.copy_(torch.randn(2, 9, 256, device=DEV))
    codes, scales = check_quantize(fmt, src)
    out = torch.full((2, 9, 512), 3.0, dtype=dtype, device=DEV)
    em.edge_moe_mx_dequantize(fmt, codes, scales, out[..., 128:384])
    want = torch.from_numpy(ops.rounded(src.float().cpu().numpy().astype(np.float64), fmt)).to(dtype)
    assert torch.equal(out[..., 128:384].cpu(), want)
    assert bool((out[..., :128] == 3).all()) and bool((out[..., 384:] == 3).all())


@fmt_of
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_non_finite_blocks(fmt, dtype):
    src = torch.randn(1, 4, 256, device=DEV).to(dtype)
    src[0, 0, 5] = float("nan")
    src[0, 1, 37] = float("inf")
    src[0, 1, 200] = float("-inf")
    src[0, 2, 64:96] = 0
    src[0, 3, :32] = -0.0
    codes, scales = check_quantize(fmt, src)
    dst = torch.empty(1, 4, 256, dtype=dtype, device=DEV)
    em.edge_moe_mx_dequantize(fmt, codes, scales, dst)
    want = torch.from_numpy(ops.rounded(src.float().cpu().numpy().astype(np.float64), fmt)).to(dtype)
    assert torch.equal(torch.isnan(dst).cpu(), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(dst).cpu(), torch.nan_to_num(want))


@fmt_of
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dequantize_every_code_at_every_scale(fmt, dtype):
    n = 16 if fmt == em.MX_FP4 else 256
    codes = np.tile(np.arange(n, dtype=np.uint8), (256, 512 // n))[None]           # row X: every code
    x = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)[None]
    cd = torch.from_numpy(np.ascontiguousarray(ops.pack(codes, fmt))).to(DEV)
    xd = torch.from_numpy(ops.by_step(x)).to(DEV)
    dst = torch.empty(1, 256, 512, dtype=dtype, device=DEV)
    em.edge_moe_mx_dequantize(fmt, cd, xd, dst)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(ops.values(codes, x, fmt)).to(torch.float32).to(dtype)
    got = dst.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


def test_weights_of_the_layer():
    """mx_weights on a layer's dense matrices: the stored weights that the
    layer's tests draw, and edge_moe_forward_mx runs on them to the same bits."""
    D = synth.config(5).dims
    want = synth.make_weights_mx(5, 0, device=DEV)
    dense = dict(want)
    for key, shape in (("s_up", (D.n_groups, D.h, D.d)), ("s_dn", (D.n_groups, D.d, D.h)),
                       ("a_up", (D.n_experts, D.delta_rank, D.d)), ("b_up", (D.n_experts, D.h, D.delta_rank)),
                       ("a_dn", (D.n_experts, D.delta_rank, D.h)), ("b_dn", (D.n_experts, D.d, D.delta_rank))):
        g = torch.Generator(device=DEV).manual_seed(synth._torch_seed(5, 0, key, 0))
        dense[key] = torch.stack([torch.randn(*shape[1:], generator=g, device=DEV) * synth.WEIGHT_STD
                                  for _ in range(shape[0])])
    W = em.mx_weights(dense)
    for key in em._WEIGHT_KEYS[:12]:
        assert torch.equal(W[key], want[key]), key
    x = torch.from_numpy(synth.make_activations(5, 0).view(np.int16)).to(DEV)
    wr, _ = synth.make_router(5, 0)
    ws = torch.empty(max(em.edge_moe_workspace_bytes(D), em.edge_moe_workspace_bytes_mx(D)), dtype=torch.uint8, device=DEV)
    idx = torch.empty(D.T, D.top_k, dtype=torch.int32, device=DEV)
    w = torch.empty(D.T, D.top_k, dtype=torch.float32, device=DEV)
    em.edge_moe_route(D, x, torch.from_numpy(wr.view(np.int16)).to(DEV), None, idx, w, None, ws)
    ys = []
    for weights in (W, want):
        y = torch.empty(D.T, D.d, device=DEV)
        em.edge_moe_forward_mx(D, x, idx, w, weights, y, ws)
        ys.append(y)
    assert torch.equal(*ys)
