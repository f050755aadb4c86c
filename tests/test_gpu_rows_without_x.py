"""Rows of the products with int4 and bf16 matrices whose row_src entry is no row of x:
rows of zeros, whatever kernel, tile and number of slices the sizes choose, that add
nothing to dW.

Whole-number x and scales that are powers of two make every sum exact in float32: the
result must be the formula's, rounded once, bit for bit."""
import numpy as np
import pytest
import torch

import shared_matrix_expert_amd as em
from gpu_helpers import DEV, say
from test_gpu_dense_product import TYPES, gradients, product, run, run_backward, same, whole
from test_gpu_packed_product import matrices
from test_gpu_packed_product import run as run_packed

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

# R, M, N, K, quant_group: few rows (16 at once, with eight and four waves and 16 and 32
# columns a workgroup; 32; 64), then tiles of 64 x 128, 64 x 256 and 128 x 256 with K whole
# and in 2, 4 and 8 slices, each with one, two and four groups in 128 of K where it occurs
PACKED = [
    (4, 1, 8, 32, 32), (5, 1, 8, 128, 64), (4, 1, 8, 64, 32), (2161, 1, 8, 32, 128), (2085, 1, 8, 128, 64), (2255, 1, 8, 64, 32),
    (4133, 1, 8, 64, 128), (4102, 2, 8, 192, 64), (4106, 5, 8, 96, 32), (12, 1, 4096, 512, 128), (13, 1, 8192, 512, 64),
    (5450, 64, 8, 32, 128), (5576, 64, 8, 128, 64), (5761, 8, 10, 288, 32), (70, 1, 9, 32, 128), (94, 1, 9, 192, 64), (70, 1, 9, 96, 32),
    (5522, 1, 144, 896, 128), (4529, 1, 199, 1408, 64), (5647, 2, 198, 768, 32),
    (4572, 1, 132, 2560, 128), (5242, 1, 129, 2048, 64), (4996, 1, 138, 2816, 32), (640, 512, 128, 4096, 128),
    (4837, 1, 67, 2816, 128), (3849, 1, 100, 3392, 64), (5414, 1, 80, 3808, 32), (4100, 64, 128, 4096, 128),
    (3295, 1, 101, 3840, 128), (650, 2, 622, 3840, 64), (1711, 1, 239, 4032, 32),
    (3231, 1, 1168, 96, 128), (1104, 1, 3475, 128, 64), (5186, 2, 670, 416, 32),
    (1126, 64, 394, 2816, 128), (4823, 64, 152, 2304, 64), (3999, 1, 436, 3104, 32),
    (4093, 1, 167, 2048, 128), (3961, 1, 198, 2176, 64), (3913, 1, 204, 3520, 32), (256, 1, 4096, 4096, 128),
    (3053, 1, 1286, 128, 128), (3587, 1, 1112, 192, 64), (5586, 1, 656, 672, 32),
    (1725, 200, 368, 1408, 128), (1718, 200, 277, 1024, 64), (523, 64, 1142, 768, 32),
    (1325, 200, 230, 1536, 128), (588, 64, 569, 1536, 64), (2586, 1, 644, 3968, 32),
    (59, 5, 4400, 2048, 128), (93, 8, 2185, 3968, 64), (61, 5, 3692, 3904, 32),
]
T = 50


def rows(R, M, seed):
    """row_src with an entry that is no row among every seven (and the first and last live
    row's), and offsets of ragged groups that leave a row in front and one behind."""
    rng = np.random.default_rng(seed)
    src = rng.integers(0, T, R)
    none = rng.random(R) < 1 / 7
    none[[0, 1, R - 2, R - 1]] = True
    src[none] = rng.choice([-1, T, 2 ** 31 - 1, -2 ** 31], none.sum())
    off = np.array([0, R]) if M == 1 else np.concatenate([[1], np.sort(rng.integers(1, R, M - 1)), [R - 1]])
    src, offsets = (torch.from_numpy(a.astype(np.int32)).to(DEV) for a in (src, off))
    return src, off, offsets if M > 1 else None, torch.from_numpy(none).to(DEV)


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("R,M,N,K,q", PACKED)
def test_int4_rows_without_x_are_zeros(R, M, N, K, q, out):
    say(f"case: int4 rows without x, {R} through {M} x {N} x {K}, groups of {q}, {out}")
    g = torch.Generator(device=DEV).manual_seed(R + K)
    src, off, offsets, _ = rows(R, M, R)
    x = whole(g, T, K) + 1                                        # (row 0 is not zero)
    codes, scales, w = matrices(g, M, N, K, q)
    y = run_packed(q, x, codes, scales, R, N, TYPES[out], offsets, src)
    same(y, product(x, w, off, src, R), (int(off[0]), int(off[-1])))


@pytest.mark.parametrize("R,M,N,K,q", PACKED)
def test_int4_rows_without_x_are_zeros_beside_scales_that_are_not_finite(R, M, N, K, q):
    """Infinite and NaN scales, and a row 0 of x that is NaN: the rows without x stay zeros,
    the other rows of the other columns exact."""
    say(f"case: int4 rows without x, scales not finite, {R} through {M} x {N} x {K}, groups of {q}")
    g = torch.Generator(device=DEV).manual_seed(R + K)
    src, off, offsets, none = rows(R, M, R)
    src[src == 0] = 1
    x = whole(g, T, K)
    codes, scales, w = matrices(g, M, N, K, q)
    want = product(x, w, off, src, R)
    x[0] = float("nan")
    scales[:, 3, 0], scales[:, 5, -1] = float("inf"), float("nan")
    y = run_packed(q, x, codes, scales, R, N, torch.float32, offsets, src)
    live = torch.zeros(R, dtype=torch.bool, device=DEV)
    live[int(off[0]):int(off[-1])] = True
    assert bool((y[live & none] == 0).all())
    keep = [n for n in range(N) if n not in (3, 5)]
    assert torch.equal(y[live][:, keep].double(), want[live][:, keep])
    assert bool((y[~live] == 7).all())


# R, M, N, K
DENSE = [(4, 1, 8, 8), (7, 64, 128, 512), (300, 64, 128, 512), (4503, 8, 16, 1024), (6300, 200, 40, 72), (700, 1, 264, 520),
         (5000, 3, 768, 1544), (6000, 16, 8, 2056), (3000, 2, 72, 104), (2000, 1, 4096, 264), (9000, 12, 80, 1000)]


@pytest.mark.parametrize("far", [False, True], ids=["", "rows far apart"])
@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("R,M,N,K", DENSE)
def test_dense_rows_without_x_add_nothing(R, M, N, K, out, far):
    """Such a row is zeros in y and adds nothing to dW, whatever its dy and the first row
    of x hold."""
    say(f"case: dense rows without x, {R} through {M} x {N} x {K}, {out}{', far apart' if far else ''}")
    g = torch.Generator(device=DEV).manual_seed(R + K)
    R = min(R, 300) if far else R
    src, off, offsets, none = rows(R, M, R)
    src[src == 0] = 1
    x, w, dy = whole(g, T, K), whole(g, M, N, K), whole(g, R, N)
    live = (int(off[0]), int(off[-1]))
    want_y = product(x, w, off, src, R)
    want_dx, want_dw = gradients(x, w, dy, off, src, None)
    x[0] = float("nan")
    bad = dy.clone()
    bad[none], bad[none, ::3] = float("nan"), float("inf")
    bad[:live[0]], bad[live[1]:] = float("nan"), float("nan")
    if far:                                                      # lane offsets within a tile pass 32 bits
        wide = torch.empty(R << 23, dtype=torch.bfloat16, device=DEV).as_strided((R, N), (1 << 23, 1), 0)
        bad = wide.copy_(bad)
    same(run(x, w, R, TYPES[out], offsets, src), want_y, live)
    dx, dw = run_backward(x, w, bad, offsets, src, None, TYPES[out])
    same(dw, want_dw)
    named = ~none
    named[:live[0]], named[live[1]:] = False, False
    same(dx[named], want_dx[named])


def test_rows_that_lose_their_x_between_replays():
    """A captured step of products with int4 and bf16 matrices and dW; other rows are without
    x, beside a dy that is not finite, in each replay."""
    g = torch.Generator(device=DEV).manual_seed(2)
    R, M, N, K = 4100, 8, 128, 1024
    x, w, dy = whole(g, T, K), whole(g, M, N, K), whole(g, R, N)
    codes, scales, w4 = matrices(g, M, N, K, 128)
    src, off, offsets, _ = rows(R, M, 0)
    live = (int(off[0]), int(off[-1]))
    y, y4, dw = (torch.full(s, 7.0, device=DEV) for s in ((R, N), (R, N), (M, N, K)))
    ws = torch.empty(max(em.edge_moe_dense_product_ws_bytes(T, R, M, N, K), em.edge_moe_packed_product_ws_bytes(T, R, M, N, K, 128),
                         em.edge_moe_dense_product_backward_ws_bytes(T, R, M, N, K)), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        em.edge_moe_dense_product(x, w, y, ws, offsets=offsets, row_src=src)
        em.edge_moe_packed_product(128, x, codes, scales, y4, ws, offsets=offsets, row_src=src)
        em.edge_moe_dense_product_backward(dy, ws, x=x, dw=dw, offsets=offsets, row_src=src)
    for seed in range(1, 4):
        other, off, o, none = rows(R, M, seed)
        src.copy_(other)
        offsets.copy_(o)
        dy.copy_(whole(g, R, N))
        want = gradients(x, w, dy, off, src, None)[1]
        dy[none] = float("nan")
        y.fill_(7.0)
        y4.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        same(y, product(x, w, off, src, R), live)
        same(y4, product(x, w4, off, src, R), live)
        same(dw, want)
