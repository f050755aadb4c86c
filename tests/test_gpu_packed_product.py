"""Products with int4 matrices on the GPU against float64.

Whole-number x and scales that are powers of two make every sum exact in float32:
the result must then be the formula's, rounded once, bit for bit.  Scales of any
kind are held to a bound that counts roundings: an instruction sums its 32 products
and its accumulator to within two float32 roundings of their magnitudes, a group's
sum is scaled and added with one."""
import numpy as np
import pytest
import torch

import shared_matrix_expert_amd as em
from gpu_helpers import DEV, say
from test_gpu_dense_product import GUARD, TYPES, U, gathered, plan, product, same, whole, workspace

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

# T, M, N, K, k, quant_group
CASES = [
    (1, 1, 8, 32, 0, 32), (1, 1, 1, 96, 0, 128), (3, 1, 17, 64, 0, 32), (2, 1, 33, 160, 0, 32), (5, 1, 100, 192, 0, 64),
    (1, 1, 8192, 4096, 0, 128), (1, 1, 4096, 8192, 0, 128), (7, 1, 1000, 2048, 0, 256), (16, 1, 512, 3200, 0, 4096),
    (17, 1, 520, 1024, 0, 32), (33, 1, 257, 1024, 0, 64), (70, 1, 1001, 512, 0, 128), (200, 1, 264, 2048, 0, 32),
    (1000, 1, 1024, 1024, 0, 128), (300, 1, 72, 96, 0, 32), (500, 1, 129, 224, 0, 32),
    (1, 64, 128, 512, 8, 128), (8, 512, 128, 1024, 10, 128), (96, 64, 128, 512, 4, 32), (300, 8, 65, 256, 3, 64),
    (777, 5, 520, 768, 0, 256), (1001, 8, 512, 1024, 0, 128), (900, 200, 40, 96, 7, 32), (600, 1024, 9, 64, 5, 64),
    (9, 1, 300, 4096, 0, 128), (13, 1, 96, 8192, 0, 128), (40, 1, 256, 4096, 0, 32), (500, 2, 300, 4096, 0, 64), (1200, 1, 130, 416, 0, 32),
    (90, 3, 1000, 2080, 0, 32), (700, 1, 1024, 4096, 0, 128), (5000, 2, 2048, 512, 0, 32), (4000, 1, 1000, 288, 0, 32),
    (300, 64, 128, 1024, 8, 64), (77, 1, 130, 1152, 0, 128), (41, 1, 128, 96, 0, 128),
]


def matrices(g, M, N, K, quant_group, exact=True):
    """codes, scales and the float64 values of int4 matrices."""
    q = min(quant_group, K)
    codes = torch.randint(0, 256, (M, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    if exact:
        scales = (2.0 ** torch.randint(-2, 2, (M, N, K // q), generator=g, device=DEV).float()).round(decimals=2).to(torch.float16)
    else:
        scales = (torch.randn(M, N, K // q, generator=g, device=DEV) * 0.01).to(torch.float16)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    c = torch.where(c > 7, c - 16, c).double()
    return codes, scales, c * scales.double().repeat_interleave(q, -1)


def run(quant_group, x, codes, scales, R, N, out, offsets, src, y=None):
    T, K = x.shape
    y = torch.full((R, N), 7.0, dtype=out, device=DEV) if y is None else y
    ws = workspace(em.edge_moe_packed_product_ws_bytes(T, R, codes.shape[0], N, K, quant_group))
    em.edge_moe_packed_product(quant_group, x, codes, scales, y, ws[:-GUARD], offsets=offsets, row_src=src)
    torch.cuda.synchronize()
    assert bool((ws[-GUARD:] == 0xA5).all()), "wrote past the workspace"
    return y


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("T,M,N,K,k,q", CASES)
def test_product_of_whole_numbers(T, M, N, K, k, q, out):
    say(f"case: int4, {T} tokens, {M} x {N} x {K}, k = {k}, groups of {q}, {out}")
    g = torch.Generator(device=DEV).manual_seed(T + K)
    R, off, offsets, src, _ = plan(T, M, k, T + N, gap=3 if M > 1 else 0)
    x = whole(g, max(T, R if src is None else 1), K)
    codes, scales, w = matrices(g, M, N, K, q)
    assert set(scales.unique().tolist()) <= {0.25, 0.5, 1.0, 2.0}
    y = run(q, x, codes, scales, R, N, TYPES[out], offsets if M > 1 else None, src)
    same(y, product(x, w, off, src, R), (int(off[0]), int(off[-1])))


@pytest.mark.parametrize("T,M,N,K,k,q", [(1, 1, 1000, 4096, 0, 128), (40, 3, 65, 512, 2, 32), (500, 4, 264, 1024, 0, 64), (777, 5, 520, 768, 0, 256)])
def test_values_of_any_kind(T, M, N, K, k, q):
    g = torch.Generator(device=DEV).manual_seed(3)
    R, off, offsets, src, _ = plan(T, M, k, 5)
    x = (torch.randn(T, K, generator=g, device=DEV) * torch.exp2(torch.randint(-20, 20, (T, 1), generator=g, device=DEV).float())).to(torch.bfloat16)
    codes, scales, w = matrices(g, M, N, K, q, exact=False)
    want, mag = product(x, w, off, src, R), product(x.abs(), w.abs(), off, src, R)
    for out in TYPES.values():
        got = run(q, x, codes, scales, R, N, out, offsets if M > 1 else None, src)
        tol = (2 * (K // 32 + 1) + K // min(q, K) + 20) * U * mag + torch.finfo(out).eps / 2 * want.abs()
        assert bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("q", [32, 128])
def test_rows_at_a_stride_and_shared_tokens(q):
    g = torch.Generator(device=DEV).manual_seed(7)
    M, N, K, T, R = 4, 133, 256, 90, 400
    src = torch.randint(0, T, (R,), generator=g, device=DEV, dtype=torch.int32)
    src[5], src[100], src[399] = -1, T, 2 ** 31 - 1
    off = np.array([2, 2, 77, 300, 398])
    offsets = torch.from_numpy(off.astype(np.int32)).to(DEV)
    codes, scales, w = matrices(g, M, N, K, q)
    xw = torch.full((T, K + 48), float("nan"), dtype=torch.bfloat16, device=DEV)
    xw[:, 16:-32] = whole(g, T, K)
    x = xw[:, 16:-32]
    for out in TYPES.values():
        for odd in (1, 8):
            yw = torch.full((R, N + 2 * odd + 1), 7.0, dtype=out, device=DEV)
            y = yw[:, odd:odd + N]
            run(q, x, codes, scales, R, N, out, offsets, src, y=y)
            same(y, product(x, w, off, src, R), (2, 398))
            assert bool((yw[:, :odd] == 7).all()) and bool((yw[:, odd + N:] == 7).all())


def test_what_is_not_finite_reaches_only_its_own_sums():
    g = torch.Generator(device=DEV).manual_seed(12)
    for K, q, R in ((160, 32, 20), (160, 32, 300), (256, 128, 20), (256, 128, 300)):
        x = whole(g, R, K)
        codes, scales, w = matrices(g, 1, 72, K, q)
        clean = product(x, w, [0, R], None, R)
        x[3, 5], x[9, K - 1] = float("inf"), float("nan")
        scales[0, 7, 0] = float("nan")
        y = run(q, x, codes, scales, R, 72, torch.float32, None, None)
        ok = torch.ones(R, 72, dtype=torch.bool, device=DEV)
        ok[3] = ok[9] = False
        ok[:, 7] = False
        assert torch.equal(y[ok].double(), clean[ok])
        assert bool(y[9].isnan().all()) and bool(y[:, 7].isnan().all())


def test_offsets_that_are_no_offsets_stay_inside():
    g = torch.Generator(device=DEV).manual_seed(13)
    M, N, K, R = 6, 64, 64, 200
    x = whole(g, R, K)
    codes, scales, _ = matrices(g, M, N, K, 32)
    for bad in ([0, 150, 20, 180, 90, 10, 200], [-5, 30, 2 ** 31 - 1, 7, -2 ** 31, 90, 1000], [200] * 7):
        y = torch.full((R + 64, N), 7.0, device=DEV)
        run(32, x, codes, scales, R, N, torch.float32, torch.tensor(bad, dtype=torch.int32, device=DEV), None, y=y[:R])
        assert bool((y[R:] == 7).all())


@pytest.mark.parametrize("T,M,N,K,k", [(8, 64, 128, 1024, 4), (600, 4, 256, 1024, 2)])
def test_side_stream_graph_replays_and_two_calls_at_once(T, M, N, K, k):
    g = torch.Generator(device=DEV).manual_seed(15)
    R, off, offsets, src, _ = plan(T, M, k, 6)
    x = whole(g, T, K)
    codes, scales, w = matrices(g, M, N, K, 128)
    nbytes = em.edge_moe_packed_product_ws_bytes(T, R, M, N, K, 128)
    outs = [(torch.empty(R, N, device=DEV), torch.empty(nbytes, dtype=torch.uint8, device=DEV)) for _ in range(2)]
    torch.cuda.synchronize()
    for y, ws in outs:
        s = torch.cuda.Stream()
        em.edge_moe_packed_product(128, x, codes, scales, y, ws, offsets=offsets, row_src=src, stream=s)
    torch.cuda.synchronize()
    for y, _ in outs:
        same(y, product(x, w, off, src, R))
    y, ws = outs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        em.edge_moe_packed_product(128, x, codes, scales, y, ws, offsets=offsets, row_src=src)
    for _ in range(3):
        x.copy_(whole(g, T, K))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same(y, product(x, w, off, src, R))
