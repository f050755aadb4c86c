"""The norm and the products with dense and int4 matrices at their largest extents on the
GPU: rows whose offsets pass 32 bits, the most rows, the widest matrices.

Whole numbers make every sum exact in float32, so that results are the formula's, rounded
once, bit for bit; the norm's are held to the roundings they make: a product of three
factors with a float32 rstd, and the output's own."""
import numpy as np
import pytest
import torch

import shared_matrix_expert_amd as em
from gpu_helpers import DEV
from test_gpu_dense_product import GUARD, U, gradients, plan, product, run, run_backward, same, whole, workspace
from test_gpu_packed_product import matrices
from test_gpu_packed_product import run as run_packed

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

FAR = 1 << 24                                                     # elements between rows: 300 rows pass 2^32 of them
ROWS = 300


@pytest.fixture(scope="module")
def far():
    """bf16 rows FAR elements apart, as views of one buffer at different columns."""
    buf = torch.zeros(ROWS * FAR, dtype=torch.bfloat16, device=DEV)

    def rows(T, cols, at, dtype=torch.bfloat16):
        b = buf if dtype == torch.bfloat16 else buf.view(dtype)
        return b.as_strided((T, cols), (FAR * 2 // dtype.itemsize, 1), at)
    yield rows
    del buf
    torch.cuda.empty_cache()


def put(view, values):
    view.copy_(values)
    return view


@pytest.mark.parametrize("d,kind", [(512, torch.bfloat16), (4096, torch.float32)])
def test_norm_of_rows_far_apart(far, d, kind):
    g = torch.Generator(device=DEV).manual_seed(1)
    r = whole(g, ROWS, d)
    x, y, dx = put(far(ROWS, d, 0), r), far(ROWS, d, 65536), far(ROWS, d, 131072, kind)
    dy = put(far(ROWS, d, 262144, kind), whole(g, ROWS, d).to(kind))
    gain = (whole(g, d) + 3).float()
    rstd, dgain = torch.empty(ROWS, device=DEV), torch.empty(d, device=DEV)
    em.edge_moe_norm(x, gain, 1e-5, y=y, rstd=rstd)
    ws = workspace(em.edge_moe_norm_backward_ws_bytes(ROWS, d))
    em.edge_moe_norm_backward(x, gain, rstd, dy, ws[:-GUARD], dx=dx, dgain=dgain)
    want_rstd = (r.double().square().mean(1, keepdim=True) + float(np.float32(1e-5))).rsqrt()
    v = r.double() * want_rstd
    assert bool(((rstd.double() - want_rstd[:, 0]).abs() <= 2 * U * want_rstd[:, 0]).all())
    want = v * gain.double()
    assert bool(((y.double() - want).abs() <= (2.0 ** -8 + 4 * U) * want.abs()).all())
    dv = dy.double() * gain.double()
    dr = want_rstd * (dv - v * (dv * v).mean(1, keepdim=True))
    # rstd's, v's, dv's, the mean's (d terms in float32) and the result's roundings
    size = want_rstd * (dv.abs() + v.abs() * (dv * v).abs().mean(1, keepdim=True))
    half = 2.0 ** -8 if kind == torch.bfloat16 else U
    assert bool(((dx.double() - dr).abs() <= half * dr.abs() + (d / 512 + 16) * U * size).all())
    terms = dy.double() * v
    assert bool(((dgain.double() - terms.sum(0)).abs() <= (ROWS + 8) * U * terms.abs().sum(0)).all())


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,M,N,K,k", [(ROWS, 1, 264, 520, 0), (ROWS, 3, 264, 520, 2), (ROWS, 40, 72, 136, 2), (9, 8, 72, 136, 1)])
def test_dense_products_of_rows_far_apart(far, T, M, N, K, k, out):
    g = torch.Generator(device=DEV).manual_seed(2)
    R, off, offsets, src, token_rows = plan(T, M, k, 3)
    n = min(R, ROWS)                                              # rows that fit the buffer
    if R > n:
        off = np.minimum(off, n)
        offsets, src, R = offsets.clamp(max=n), src[:n].contiguous(), n
    x, w = put(far(T, K, 0), whole(g, T, K)), whole(g, M, N, K)
    dy, y = put(far(R, N, 65536), whole(g, R, N)), far(R, N, 131072, out)
    y.fill_(7.0)
    same(run(x, w, R, out, offsets, src, y=y), product(x, w, off, src, R), (int(off[0]), int(off[-1])))
    for tr in (None, token_rows) if k else (None,):
        dx = far(T if tr is not None else R, K, 262144, out)
        dx.fill_(7.0)
        dx, dw = run_backward(x, w, dy, offsets, src, tr, out, dx=dx)
        want_dx, want_dw = gradients(x, w, dy, off, src, tr)
        same(dx, want_dx, None if tr is not None else (int(off[0]), int(off[-1])))
        same(dw, want_dw)


@pytest.mark.parametrize("q", [32, 128])
@pytest.mark.parametrize("T,M,N,K,k", [(ROWS, 1, 264, 1024, 0), (ROWS, 3, 264, 512, 1), (5, 1, 264, 1024, 0), (25, 1, 40, 256, 0)])
def test_packed_products_of_rows_far_apart(far, T, M, N, K, k, q):
    g = torch.Generator(device=DEV).manual_seed(3)
    R, off, offsets, src, _ = plan(T, M, k, 5)
    codes, scales, w = matrices(g, M, N, K, q)
    x, y = put(far(T, K, 0), whole(g, T, K)), far(R, N, 65536, torch.float32)
    y.fill_(7.0)
    same(run_packed(q, x, codes, scales, R, N, torch.float32, offsets, src, y=y), product(x, w, off, src, R),
         (int(off[0]), int(off[-1])))


def test_the_most_rows():
    """2^25 rows of 2^20 tokens through all of the operators: each is the exact result."""
    g = torch.Generator(device=DEV).manual_seed(4)
    T, R, k = 1 << 20, 1 << 25, 32
    src = torch.randint(0, T, (R,), generator=g, device=DEV, dtype=torch.int32)
    x, w, dy = whole(g, T, 32, span=1), whole(g, 1, 8, 32), whole(g, R, 8, span=1)
    y = torch.empty(R, 8, dtype=torch.bfloat16, device=DEV)
    ws = workspace(em.edge_moe_dense_product_ws_bytes(T, R, 1, 8, 32))
    em.edge_moe_dense_product(x, w, y, ws[:-GUARD], row_src=src)
    per_token = x.float() @ w[0].float().t()                       # (whole numbers: exact)
    assert torch.equal(y, per_token[src.long()].to(torch.bfloat16))
    token_rows = torch.randint(0, R, (T, k), generator=g, device=DEV, dtype=torch.int32)
    dx, dw = torch.empty(T, 32, device=DEV), torch.empty(1, 8, 32, device=DEV)
    ws = workspace(em.edge_moe_dense_product_backward_ws_bytes(T, R, 1, 8, 32))
    em.edge_moe_dense_product_backward(dy, ws[:-GUARD], x=x, w=w, dx=dx, dw=dw, row_src=src, token_rows=token_rows)
    per_row = dy.float() @ w[0].float()
    want = torch.zeros(T, 32, device=DEV)
    for j in range(k):
        want += per_row[token_rows[:, j].long()]
    assert torch.equal(dx, want)
    want = sum(dy[i:i + (1 << 22)].float().t().double() @ x[src[i:i + (1 << 22)].long()].double() for i in range(0, R, 1 << 22))
    assert torch.equal(dw[0].double(), want)
    del dy, y, per_row, dx
    for N in (1, 8):                                              # (of one column the scales are an odd number)
        codes, scales, values = matrices(g, 1, N, 32, 32)
        y = torch.empty(R, N, device=DEV)
        ws = workspace(em.edge_moe_packed_product_ws_bytes(T, R, 1, N, 32, 32))
        em.edge_moe_packed_product(32, x, codes, scales, y, ws[:-GUARD], row_src=src)
        assert torch.equal(y, (x.double() @ values[0].t()).float()[src.long()])
    del y, src, token_rows
    r = whole(g, R, 8)
    out, rstd = torch.empty_like(r), torch.empty(R, device=DEV)
    gain, dgain = torch.ones(8, device=DEV), torch.empty(8, device=DEV)
    em.edge_moe_norm(r, gain, 1.0, y=out, rstd=rstd)
    v = r.double() * (r.double().square().mean(1, keepdim=True) + 1.0).rsqrt()
    assert bool(((out.double() - v).abs() <= (2.0 ** -8 + 4 * U) * v.abs()).all())
    ws = workspace(em.edge_moe_norm_backward_ws_bytes(R, 8))
    em.edge_moe_norm_backward(r, gain, rstd, r, ws[:-GUARD], dgain=dgain)
    want = (r.double() * v).sum(0)                                # (all terms positive; a lane sums R / 2048 of them)
    assert bool(((dgain.double() - want).abs() <= (R / 2048 + 16) * U * want).all())


@pytest.mark.parametrize("T", [1, 20, 70])
def test_the_widest_matrices(T):
    g = torch.Generator(device=DEV).manual_seed(5)
    S = 32768
    x, w, dy = whole(g, T, S, span=1), whole(g, 1, S, S, span=1), whole(g, T, S, span=1)
    off = np.array([0, T])
    rows = [slice(i, i + 4096) for i in range(0, S, 4096)]
    y = run(x, w, T, torch.float32, None, None)
    dx, dw = run_backward(x, w, dy, None, None, None, torch.float32)
    want_dx = torch.zeros(T, S, dtype=torch.float64, device=DEV)
    for r in rows:
        part = w[0, r].double()
        same(y[:, r].contiguous(), x.double() @ part.t())
        want_dx += dy[:, r].double() @ part
        same(dw[0, r], dy[:, r].double().t() @ x.double())
    same(dx, want_dx)
    del w, dw
    codes = torch.randint(0, 256, (1, S, S // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.ones(1, S, S // 128, dtype=torch.float16, device=DEV)
    y = run_packed(128, x, codes, scales, T, S, torch.float32, None, None)
    for r in rows:
        c = torch.stack([codes[0, r] & 15, codes[0, r] >> 4], -1).flatten(-2).double()
        same(y[:, r].contiguous(), x.double() @ torch.where(c > 7, c - 16, c).t())


def test_more_rows_of_a_token_than_its_map_holds():
    """Few matrices of few rows, where dx of tokens is otherwise one sum over all matrices."""
    g = torch.Generator(device=DEV).manual_seed(6)
    T, M, N, K = 1500, 8, 16, 2056
    R, off, offsets, src, _ = plan(T, M, 3, 7)
    x, w, dy = whole(g, T, K), whole(g, M, N, K), whole(g, R, N)
    for k in (32, 33, 100):
        token_rows = torch.randint(-1, R, (T, k), generator=g, device=DEV, dtype=torch.int32)
        token_rows[5] = token_rows[5, 0]                          # one row k times
        dx, _ = run_backward(x, w, dy, offsets, src, token_rows, torch.float32, want=("dx",))
        same(dx, gradients(x, w, dy, off, src, token_rows)[0])


@pytest.mark.parametrize("dx_type,dw_type", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("T,M,N,K,k", [(1500, 8, 16, 2056, 3), (700, 6, 264, 520, 2)])
def test_gradients_of_two_types_replayed_and_two_at_once(T, M, N, K, k, dx_type, dw_type):
    """Tokens' dx in one sum and by rows: captured, replayed with new inputs between eager
    calls, and on two streams with a workspace each."""
    g = torch.Generator(device=DEV).manual_seed(8)
    R, off, offsets, src, token_rows = plan(T, M, k, 9)
    x, w, dy = whole(g, T, K), whole(g, M, N, K), whole(g, R, N)
    nbytes = em.edge_moe_dense_product_backward_ws_bytes(T, R, M, N, K)
    out = [(torch.empty(T, K, dtype=dx_type, device=DEV), torch.empty(M, N, K, dtype=dw_type, device=DEV), workspace(nbytes))
           for _ in range(2)]

    def call(i, dy):
        dx, dw, ws = out[i]
        em.edge_moe_dense_product_backward(dy, ws[:-GUARD], x=x, w=w, dx=dx, dw=dw, offsets=offsets, row_src=src, token_rows=token_rows)

    def check(i, dy):
        torch.cuda.synchronize()
        dx, dw = gradients(x, w, dy, off, src, token_rows)
        same(out[i][0], dx)
        same(out[i][1], dw)
        assert bool((out[i][2][-GUARD:] == 0xA5).all())
    call(0, dy)
    check(0, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(0, dy)
    for _ in range(3):
        dy.copy_(whole(g, R, N))
        call(1, dy)
        graph.replay()
        check(0, dy)
        check(1, dy)
    other = whole(g, R, N)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call(0, dy)
    call(1, other)
    check(0, dy)
    check(1, other)
