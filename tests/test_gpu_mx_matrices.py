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


# ------------------------------------------------------------------ the product ---

def matrices(M, N, K, seed):
    """Random MXFP4 matrices, weights near N(0, 0.02^2): device codes and scales, float64 values."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (M, N, K), dtype=np.uint8)
    x = rng.integers(118, 122, (M, N, K // 32), dtype=np.uint8)
    return (torch.from_numpy(ops.pack(codes, ops.FP4)).to(DEV), torch.from_numpy(ops.by_step(x)).to(DEV),
            ops.values(codes, x, ops.FP4))


def rows_of(T, K, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, K, generator=g).to(torch.bfloat16)


def within(y, ref, mag, K):
    """|dy| <= 2^-8 |y| (one rounding to bf16) + 2^-13 times the products'
    magnitude sum (an instruction's sum of 128 products is good to about 2^-13.5
    of theirs) + K / 128 float32 additions of partial sums no larger than it."""
    got = y.float().cpu().numpy().astype(np.float64)
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -13 + K / 128 * 2.0 ** -24) * (1 + 2.0 ** -8) * mag + 2.0 ** -133
    live = np.isfinite(ref)
    worst = float(np.max(np.abs(got - ref)[live] / tol[live], initial=0.0))
    say(f"  worst |dy| / tolerance = {worst:.3g}")
    assert np.isfinite(got[live]).all() and worst <= 1.0


def product(fmt, x, codes, scales, y, offsets=None, row_src=None, stream=None):
    (T, K), (R, N) = x.shape, y.shape
    ws = torch.empty(em.edge_moe_mx_product_ws_bytes(T, R, codes.shape[0], N, K, fmt), dtype=torch.uint8, device=DEV)
    em.edge_moe_mx_product(fmt, x, codes, scales, y, ws, offsets=offsets, row_src=row_src, stream=stream)
    return ws


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


@fmt_of
@pytest.mark.parametrize("T,N,K", [(1, 16, 128), (1, 2048, 4096), (2, 1, 256), (3, 37, 384), (16, 64, 640),
                                   (17, 100, 512), (33, 50, 1024), (64, 96, 128), (65, 257, 256), (127, 33, 384),
                                   (191, 512, 512), (192, 256, 128), (257, 300, 1152), (700, 1030, 256),
                                   (20, 4096, 256), (50, 2080, 256), (40, 8192, 128), (3000, 4608, 256), (2800, 5000, 128),
                                   (1000, 7937, 128), (997, 7920, 384), (1530, 8000, 256), (1400, 8191, 128)])
def test_product_dense(fmt, T, N, K):
    say(f"case: product {T} x {N} x {K}")
    q, e, W = matrices(1, N, K, T + N)
    x = rows_of(T, K, T)
    y = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    product(fmt, x.to(DEV), q, e, y)
    within(y, *ops.product(x.double().numpy(), fmt, W), K)


@fmt_of
@pytest.mark.parametrize("sizes,T", [([5], 5), ([0, 7, 0, 0, 20, 1, 0], 28), ([0, 0, 0], 4), ([90, 0, 300, 10, 0], 400),
                                     ([500, 3, 0, 260], 763), ("many", 130), ("many routed", 40)])
def test_product_grouped(fmt, sizes, T):
    """Ragged groups, empty ones among them, up to hundreds of matrices; rows
    before the first and behind the last group keep what they held."""
    rng = np.random.default_rng(9)
    N, K = 72, 256
    src = None
    if sizes == "many":
        sizes = np.bincount(rng.integers(0, 200, 130), minlength=200)
    elif sizes == "many routed":
        sizes = np.bincount(rng.choice(512, 400), minlength=512)
        src = rng.integers(0, T, 400)
    n = int(np.sum(sizes))
    head, tail = (0, 0) if src is not None else (2, 3)
    R = head + n + tail
    off = head + np.concatenate([[0], np.cumsum(sizes)])
    q, e, W = matrices(len(sizes), N, K, 4)
    x = rows_of(max(T, R) if src is None else T, K, 6)
    y = torch.full((R, N), 3.25, dtype=torch.bfloat16, device=DEV)
    say(f"case: {len(sizes)} groups, {R} rows")
    product(fmt, x.to(DEV), q, e, y, offsets=i32(off), row_src=None if src is None else i32(src))
    ref, mag = ops.product(x.double().numpy(), fmt, W, off, src, R)
    within(y, ref, mag, K)
    assert bool((y[:head] == 3.25).all()) and bool((y[head + n:] == 3.25).all())


@fmt_of
@pytest.mark.parametrize("sizes", [[600, 0, 700, 65], [1500, 3, 0, 700, 129], [2050, 0, 1, 1300], [90] * 12])
def test_product_grouped_tiles(fmt, sizes):
    """Groups that the tiled kernel takes by 64 to 256 rows, odd columns."""
    N, K, R = 4101, 256, sum(sizes)
    q, e, W = matrices(len(sizes), N, K, 11)
    x = rows_of(R, K, 12)
    y = torch.full((R + 2, N), 3.25, dtype=torch.bfloat16, device=DEV)
    say(f"case: groups of {sizes}")
    off = np.concatenate([[0], np.cumsum(sizes)])
    product(fmt, x.to(DEV), q, e, y[:R], offsets=i32(off))
    within(y[:R], *ops.product(x.double().numpy(), fmt, W, off), K)
    assert bool((y[R:] == 3.25).all())


@fmt_of
@pytest.mark.parametrize("M,N,K,R", [(40, 128, 384, 3000), (20, 123, 128, 9000), (3, 100, 512, 20000), (1, 128, 256, 9000),
                                     (1, 77, 128, 40000), (1, 2, 384, 50000)])
def test_product_narrow_matrices(fmt, M, N, K, R):
    """Many rows through matrices of at most 128 columns, sharing x rows, some rows of no x."""
    rng = np.random.default_rng(M)
    off = np.sort(np.concatenate([[0, R], rng.integers(0, R + 1, M - 1)]))
    T = 500
    src = rng.integers(-1, T, R)
    q, e, W = matrices(M, N, K, 13)
    x = rows_of(T, K, 14)
    y = torch.full((R + 1, N), 3.25, dtype=torch.bfloat16, device=DEV)
    say(f"case: {R} rows, {M} x {N} x {K}")
    product(fmt, x.to(DEV), q, e, y[:R], offsets=i32(off), row_src=i32(src))
    within(y[:R], *ops.product(x.double().numpy(), fmt, W, off, src), K)
    assert bool((y[R:] == 3.25).all()) and bool((y[:R][i32(src) < 0] == 0).all())


@fmt_of
@pytest.mark.parametrize("R,T,N", [(40, 7, 48), (500, 60, 48), (90, 17, 640), (900, 300, 512), (1400, 200, 8192)])
def test_product_gathered_rows(fmt, R, T, N):
    """Shared x rows, and entries that name no row: zeros."""
    rng = np.random.default_rng(2)
    src = rng.integers(0, T, R)
    src[[0, 5, R - 1]] = [-1, T, 2 ** 31 - 1]
    q, e, W = matrices(2, N, 384, 1)
    off = [0, R // 3, R]
    x = rows_of(T, 384, 3)
    y = torch.full((R, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    product(fmt, x.to(DEV), q, e, y, offsets=i32(off), row_src=i32(src))
    within(y, *ops.product(x.double().numpy(), fmt, W, off, src), 384)
    assert bool((y[[0, 5, R - 1]] == 0).all())


@fmt_of
@pytest.mark.parametrize("R,T,N", [(1, 400, 64), (3, 17, 40), (40, 700, 48), (60, 900, 640), (300, 2000, 512), (700, 1501, 8192)])
@pytest.mark.parametrize("gather", [True, False])
def test_product_of_few_rows_of_a_long_x(fmt, R, T, N, gather):
    """Fewer y rows than x rows: gathered ones (two the same, one that names no
    row), or x's first; the workspace is that of R rows."""
    rng = np.random.default_rng(R)
    src = rng.integers(0, T, R) if gather else None
    if gather and R > 2:
        src[0], src[1], src[R - 1] = src[2], T, T - 1
    q, e, W = matrices(2, N, 384, 1)
    off = [0, R // 3, R]
    x = rows_of(T, 384, 3)
    y = torch.full((R, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = torch.full((em.edge_moe_mx_product_ws_bytes(T, R, 2, N, 384, fmt) + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    assert ws.numel() <= 4096 + 512 + R * (384 + 12)
    em.edge_moe_mx_product(fmt, x.to(DEV), q, e, y, ws[:-4096], offsets=i32(off), row_src=None if src is None else i32(src))
    ref = ops.product(x[:R].double().numpy(), fmt, W, off) if src is None else ops.product(x.double().numpy(), fmt, W, off, src)
    within(y, *ref, 384)
    assert bool((ws[-4096:] == 0xA5).all())


@fmt_of
@pytest.mark.parametrize("T", [5, 90, 230])
def test_product_strided_rows(fmt, T):
    q, e, W = matrices(1, 44, 256, 8)
    x = rows_of(T, 512, 1)
    y = torch.full((T, 100), 2.5, dtype=torch.bfloat16, device=DEV)
    for shift in (8, 5):                          # aligned and odd columns of a wider buffer
        out = y[:, shift:shift + 44]
        product(fmt, x.to(DEV)[:, 128:384], q, e, out)
        within(out, *ops.product(x[:, 128:384].double().numpy(), fmt, W), 256)
        assert bool((y[:, :shift] == 2.5).all()) and bool((y[:, shift + 44:] == 2.5).all())
        y.fill_(2.5)


@fmt_of
@pytest.mark.parametrize("T", [4, 100, 300])
def test_product_non_finite(fmt, T):
    """NaN and infinities of x and NaN scales of W stay in the rows and columns they enter."""
    q, e, W = matrices(1, 40, 256, 2)
    e[0, 1, 7, 2] = 255                           # row 7 of W, block 6
    x = rows_of(T, 256, 4)
    x[1, 200] = float("nan")
    x[3, 0] = float("-inf")
    y = torch.zeros(T, 40, dtype=torch.bfloat16, device=DEV)
    product(fmt, x.to(DEV), q, e, y)
    bad = torch.zeros(T, 40, dtype=torch.bool)
    bad[[1, 3]] = True
    bad[:, 7] = True
    assert torch.equal(torch.isnan(y).cpu(), bad)
    ref, mag = ops.product(np.nan_to_num(x.double().numpy(), nan=0.0, posinf=0.0, neginf=0.0), fmt, W)
    ref[bad.numpy()] = np.nan
    within(y, ref, mag, 256)


@fmt_of
@pytest.mark.parametrize("off", [[0, 30, 10, 40], [-5, 20, 90, 40], [40, 0, 0, 40], [7, 7, 7, 7]])
@pytest.mark.parametrize("R", [40, 500])
def test_product_bad_offsets_stay_inside(fmt, off, R):
    """Descending or out-of-range offsets: nothing outside y's rows is written."""
    q, e, _ = matrices(3, 32, 128, 2)
    off = [o * R // 40 for o in off]
    buf = torch.full((R + 64, 32), 1.5, dtype=torch.bfloat16, device=DEV)
    product(fmt, rows_of(R, 128, 4).to(DEV), q, e, buf[32:32 + R], offsets=i32(off))
    assert bool((buf[:32] == 1.5).all()) and bool((buf[32 + R:] == 1.5).all())


@pytest.mark.parametrize("T", [3, 70, 260])
def test_product_repeats_streams_and_graphs(T):
    """Bitwise the same again, on another stream, and in every replay of a
    captured graph with eager work on the workspace's memory between replays."""
    q, e, W = matrices(1, 300, 512, 5)
    x = rows_of(T, 512, 7).to(DEV)
    y0, y1 = (torch.zeros(T, 300, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    product(em.MX_FP8, x, q, e, y0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = product(em.MX_FP8, x, q, e, y1, stream=s)
    s.synchronize()
    assert torch.equal(y0, y1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        em.edge_moe_mx_product(em.MX_FP8, x, q, e, y1, ws)
    for i in range(4):
        x.copy_(rows_of(T, 512, 20 + i))
        y1.fill_(9)
        ws.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        product(em.MX_FP8, x, q, e, y0)
        assert torch.equal(y0, y1), f"replay {i}"
