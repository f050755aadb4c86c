"""Products with bf16 matrices and their gradients on the GPU against float64.

Most cases hold whole numbers so small that every sum is exact in float32: the
result must then be the formula's, rounded once, bit for bit.  Values of any kind
are held to a bound that counts roundings: an instruction sums its 32 products and
its accumulator to within two float32 roundings of their magnitudes."""
import numpy as np
import pytest
import torch

import shared_matrix_expert_amd as em
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
GUARD = 512

# T, M, N, K, k (0: rows in order), as names of what they reach
CASES = [
    (1, 1, 8, 8, 0), (1, 1, 64, 32, 0), (3, 1, 24, 40, 0), (17, 1, 8, 4096, 0), (5, 1, 4096, 16, 0),
    (1, 1, 8192, 4096, 0), (8, 1, 1000, 2008, 0), (33, 2, 72, 104, 0), (64, 1, 4096, 1024, 0), (200, 1, 256, 8192, 0),
    (70, 1, 520, 264, 0), (129, 1, 136, 1000, 0), (257, 1, 264, 520, 0), (1000, 1, 2048, 1024, 0), (3000, 1, 16, 2048, 0),
    (2500, 1, 2048, 16, 0), (1, 64, 128, 512, 8), (8, 512, 128, 1024, 10), (96, 64, 128, 512, 4), (300, 8, 64, 264, 3),
    (1501, 8, 16, 1024, 3), (777, 5, 520, 776, 0), (2000, 8, 1024, 512, 0), (900, 200, 40, 72, 7), (600, 1024, 8, 64, 5),
    (1000, 16, 8, 2056, 6), (3000, 12, 80, 1000, 4), (20000, 40, 16, 520, 5), (4096, 3, 768, 1544, 2), (5300, 1, 4104, 264, 0), (5000, 3, 4096, 328, 0), (300, 2, 4360, 4360, 0),
]


def plan(T, M, k, seed, gap=0):
    """Rows of a batch sorted by matrix, with empty matrices; `gap` rows before the
    first and behind the last matrix."""
    rng = np.random.default_rng(seed)
    if k:
        pick = np.argsort(rng.random((T, M)), axis=1)[:, :min(k, M)] if M > 1 else np.zeros((T, 1), np.int64)
        e, t = pick.reshape(-1), np.repeat(np.arange(T), pick.shape[1])
        order = np.lexsort((t, e))
        src = t[order]
        cnt = np.bincount(e, minlength=M)
        slot = np.empty(len(order), np.int64)
        slot[order] = np.arange(len(order))
        token_rows = slot.reshape(T, -1) + gap
    else:
        cnt = rng.multinomial(T, rng.dirichlet(np.full(M, 0.7))) if M > 1 else np.array([T])
        src = token_rows = None
    off = np.concatenate([[0], np.cumsum(cnt)]) + gap
    R = int(off[-1]) + gap
    if src is not None:
        src = np.concatenate([rng.integers(0, T, gap), src, rng.integers(0, T, gap)])

    def dev(a):
        return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)
    return R, off, dev(off), dev(src), dev(token_rows)


def whole(g, *shape, span=2):
    """Whole numbers of -span .. span in bf16."""
    return torch.randint(-span, span + 1, shape, generator=g, device=DEV).to(torch.bfloat16)


def gathered(x, src):
    if src is None:
        return x.double()
    ok = (src >= 0) & (src < len(x))
    return x.double()[src.long().clamp(0, len(x) - 1)] * ok[:, None]


def product(x, w, off, src, R):
    """y in float64, and the rows that matrices have."""
    xr = gathered(x, src)
    y = torch.zeros(R, w.shape[1], dtype=torch.float64, device=DEV)
    for m in range(len(off) - 1):
        a, b = off[m], off[m + 1]
        if b > a:
            y[a:b] = xr[a:b] @ w[m].double().t()
    return y


def gradients(x, w, dy, off, src, token_rows):
    R, (M, N, K) = dy.shape[0], w.shape
    xr = gathered(x, src)
    dxr, dw = torch.zeros(R, K, dtype=torch.float64, device=DEV), torch.zeros(M, N, K, dtype=torch.float64, device=DEV)
    for m in range(M):
        a, b = off[m], off[m + 1]
        if b > a:
            d = dy[a:b].double()
            dxr[a:b] = d @ w[m].double()
            dw[m] = d.t() @ xr[a:b]
    if token_rows is None:
        return dxr, dw
    live = (token_rows >= int(off[0])) & (token_rows < int(off[-1]))
    return (dxr[token_rows.long().clamp(0, R - 1)] * live.unsqueeze(-1)).sum(1), dw


def workspace(nbytes):
    return torch.full((nbytes + GUARD,), 0xA5, dtype=torch.uint8, device=DEV)


def run(x, w, R, out, offsets, src, y=None):
    T, (M, N, K) = x.shape[0], w.shape
    y = torch.full((R, N), 7.0, dtype=out, device=DEV) if y is None else y
    ws = workspace(em.edge_moe_dense_product_ws_bytes(T, R, M, N, K))
    em.edge_moe_dense_product(x, w, y, ws[:-GUARD], offsets=offsets, row_src=src)
    torch.cuda.synchronize()
    assert bool((ws[-GUARD:] == 0xA5).all()), "wrote past the workspace"
    return y


def run_backward(x, w, dy, offsets, src, token_rows, out, want=("dx", "dw"), dx=None):
    T, R, (M, N, K) = x.shape[0], dy.shape[0], w.shape
    if "dx" in want and dx is None:
        dx = torch.full((R if token_rows is None else T, K), 7.0, dtype=out, device=DEV)
    dw = torch.full((M, N, K), 7.0, dtype=out, device=DEV) if "dw" in want else None
    ws = workspace(em.edge_moe_dense_product_backward_ws_bytes(T, R, M, N, K))
    em.edge_moe_dense_product_backward(dy, ws[:-GUARD], x=x, w=w, dx=dx, dw=dw, offsets=offsets, row_src=src,
                                       token_rows=token_rows)
    torch.cuda.synchronize()
    assert bool((ws[-GUARD:] == 0xA5).all()), "wrote past the workspace"
    return dx, dw


def same(got, want64, rows=None):
    """Bit for bit the exact result rounded once; rows of no matrix as they were."""
    want = want64.float().to(got.dtype)                       # whole numbers below 2^24: float32 holds them
    if rows is not None:
        keep = torch.full_like(want, 7.0)
        keep[rows[0]:rows[1]] = want[rows[0]:rows[1]]
        want = keep
    assert torch.equal(got, want), f"{int((got != want).sum())} of {got.numel()} values differ"


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("T,M,N,K,k", CASES)
def test_product_of_whole_numbers(T, M, N, K, k, out):
    say(f"case: y, {T} tokens, {M} x {N} x {K}, k = {k}, {out}")
    g = torch.Generator(device=DEV).manual_seed(T + K)
    R, off, offsets, src, _ = plan(T, M, k, T + N, gap=3 if M > 1 else 0)
    x, w = whole(g, max(T, R if src is None else 1), K), whole(g, M, N, K)
    y = run(x, w, R, TYPES[out], offsets if M > 1 else None, src)
    same(y, product(x, w, off, src, R), (int(off[0]), int(off[-1])))


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("T,M,N,K,k", CASES)
def test_gradients_of_whole_numbers(T, M, N, K, k, out):
    say(f"case: gradients, {T} tokens, {M} x {N} x {K}, k = {k}, {out}")
    g = torch.Generator(device=DEV).manual_seed(T + K + 1)
    R, off, offsets, src, token_rows = plan(T, M, k, T + N, gap=3 if M > 1 else 0)
    x, w, dy = whole(g, max(T, R if src is None else 1), K), whole(g, M, N, K), whole(g, R, N)
    offsets = offsets if M > 1 else None
    live = (int(off[0]), int(off[-1]))
    dx, dw = run_backward(x, w, dy, offsets, src, token_rows, TYPES[out])
    wx, ww = gradients(x, w, dy, off, src, token_rows)
    same(dx, wx, live if token_rows is None else None)
    same(dw, ww)
    # each alone has the bits it has with the other; dx by rows where tokens were asked
    ax, _ = run_backward(x, w, dy, offsets, src, token_rows, TYPES[out], ("dx",))
    _, aw = run_backward(x, w, dy, offsets, src, token_rows, TYPES[out], ("dw",))
    assert torch.equal(ax, dx) and torch.equal(aw, dw)
    if token_rows is not None:
        rx, _ = run_backward(x, w, dy, offsets, src, None, TYPES[out], ("dx",))
        same(rx, gradients(x, w, dy, off, src, None)[0], live)


@pytest.mark.parametrize("T,M,N,K,k", [(8, 512, 128, 1024, 10), (777, 5, 520, 776, 0), (129, 1, 136, 1000, 0), (1501, 8, 16, 1024, 3)])
def test_values_of_any_kind(T, M, N, K, k):
    g = torch.Generator(device=DEV).manual_seed(3)
    R, off, offsets, src, token_rows = plan(T, M, k, 5)
    x = (torch.randn(T, K, generator=g, device=DEV) * torch.exp2(torch.randint(-20, 20, (T, 1), generator=g, device=DEV).float())).to(torch.bfloat16)
    w, dy = torch.randn(M, N, K, generator=g, device=DEV).to(torch.bfloat16), torch.randn(R, N, generator=g, device=DEV).to(torch.bfloat16)
    offsets = offsets if M > 1 else None

    def within(got, want, mag, n, more=0):
        tol = (2 * (n // 32 + 1) + 20 + more) * U * mag + torch.finfo(got.dtype).eps / 2 * want.abs()
        assert bool(((got.double() - want).abs() <= tol).all())
    for out in TYPES.values():
        within(run(x, w, R, out, offsets, src), product(x, w, off, src, R), product(x.abs(), w.abs(), off, src, R), K)
        dx, dw = run_backward(x, w, dy, offsets, src, token_rows, out)
        wx, ww = gradients(x, w, dy, off, src, token_rows)
        mx, mw = gradients(x.abs(), w.abs(), dy.abs(), off, src, token_rows)
        within(dx, wx, mx, N, k)
        within(dw, ww, mw, int(np.diff(off).max()))


def test_rows_at_a_stride_and_shared_tokens():
    """x, y, dy and dx rows of wider buffers whose other columns are NaN and stay;
    tokens named twice, and row_src entries that are no row."""
    g = torch.Generator(device=DEV).manual_seed(7)
    M, N, K, T, R = 4, 136, 264, 90, 400
    src = torch.randint(0, T, (R,), generator=g, device=DEV, dtype=torch.int32)
    src[5], src[100], src[399] = -1, T, 2 ** 31 - 1
    off = np.array([2, 2, 77, 300, 398])
    offsets = torch.from_numpy(off.astype(np.int32)).to(DEV)
    token_rows = torch.randint(0, R, (T, 5), generator=g, device=DEV, dtype=torch.int32)
    token_rows[0] = -1
    token_rows[1, 2], token_rows[2, 0], token_rows[3] = R, -2 ** 31, 9           # one row five times

    def wide(v, dtype=torch.bfloat16):
        b = torch.full((v.shape[0], v.shape[1] + 48), float("nan"), dtype=dtype, device=DEV)
        b[:, 16:-32] = v
        return b[:, 16:-32]
    x, dy, w = wide(whole(g, T, K)), wide(whole(g, R, N)), whole(g, M, N, K)
    for out in TYPES.values():
        y = wide(torch.full((R, N), 7.0, device=DEV), out)
        run(x, w, R, out, offsets, src, y=y)
        same(y, product(x, w, off, src, R), (2, 398))
        for tr in (token_rows, None):
            dx = wide(torch.full((T if tr is not None else R, K), 7.0, device=DEV), out)
            _, dw = run_backward(x, w, dy, offsets, src, tr, out, dx=dx)
            wx, ww = gradients(x, w, dy, off, src, tr)
            same(dx, wx, None if tr is not None else (2, 398))
            same(dw, ww)
            for b in (y, dx):
                assert bool(b._base[:, :16].isnan().all()) and bool(b._base[:, -32:].isnan().all())


def test_what_is_not_finite_reaches_only_its_own_sums():
    """NaN and infinities in rows and columns beside a tile's, in padded rows and in
    other matrices' rows stay there."""
    g = torch.Generator(device=DEV).manual_seed(12)
    M, N, K = 3, 72, 104
    off = np.array([4, 41, 41, 90])
    offsets = torch.from_numpy(off.astype(np.int32)).to(DEV)
    R = 130
    x, w, dy = whole(g, R, K), whole(g, M, N, K), whole(g, R, N)
    for t in (x, dy):
        t[:4], t[90:] = float("nan"), float("inf")               # rows of no matrix
    w[1] = float("nan")                                           # a matrix without rows
    cx, cw, cd = x.clone(), w.clone(), dy.clone()
    for t in (cx, cd):
        t[:4] = t[90:] = 0
    cw[1] = 0
    y = run(x, w, R, torch.float32, offsets, None)
    same(y, product(cx, cw, off, None, R), (4, 90))
    dx, dw = run_backward(x, w, dy, offsets, None, None, torch.float32)
    wx, ww = gradients(cx, cw, cd, off, None, None)
    same(dx, wx, (4, 90))
    same(dw, ww)
    x[50, 7] = float("inf")                                       # one x value: its row of y, its column of one dW
    y = run(x, w, R, torch.float32, offsets, None)
    assert bool(y[4:50].isfinite().all()) and bool(y[51:90].isfinite().all())
    _, dw = run_backward(x, w, dy, offsets, None, None, torch.float32, ("dw",))
    bad = ~dw.isfinite()
    assert not bool(bad[:2].any()) and not bool(bad[2, :, :7].any()) and not bool(bad[2, :, 8:].any()) and bool(bad[2, :, 7].any())
    w[0, 5, 3] = float("-inf")                                    # one weight: its column of y, its column of dx
    y = run(x, w, R, torch.float32, offsets, None)
    bad = ~y[4:41].isfinite()
    assert not bool(bad[:, :5].any()) and not bool(bad[:, 6:].any())


@pytest.mark.parametrize("T,M,N,K,k", [(150, 8, 16, 264, 3), (600, 8, 16, 2056, 4), (2500, 8, 24, 1160, 3), (250, 16, 64, 8200, 6), (5000, 40, 16, 520, 5)])
def test_tokens_see_only_their_own_matrices(T, M, N, K, k):
    """dx by tokens where one matrix is NaN and one infinite: the tokens that have no row
    of them have their exact sums; tokens with several rows of one matrix."""
    g = torch.Generator(device=DEV).manual_seed(16)
    R, off, offsets, src, token_rows = plan(T, M, k, 9)
    token_rows[1] = token_rows[0]                                 # rows of two tokens
    token_rows[2] = token_rows[2, 0]                              # one row k times
    token_rows[3, 0] = -1
    w, dy = whole(g, M, N, K), whole(g, R, N)
    want = gradients(torch.zeros(T, K, device=DEV), w, dy, off, None if src is None else src, token_rows)[0]
    w[1], w[3, :, ::2] = float("nan"), float("inf")
    dx = torch.full((T, K), 7.0, device=DEV)
    ws = workspace(em.edge_moe_dense_product_backward_ws_bytes(T, R, M, N, K))
    em.edge_moe_dense_product_backward(dy, ws[:-GUARD], w=w, dx=dx, offsets=offsets, token_rows=token_rows)
    assert bool((ws[-GUARD:] == 0xA5).all())
    tr = token_rows.cpu().numpy()
    mats = [set(np.searchsorted(off, r, side="right") - 1 for r in row if r >= 0) for row in tr]
    clean = torch.tensor([not ms & {1, 3} for ms in mats], device=DEV)
    assert torch.equal(dx[clean].double(), want[clean]) and bool(clean.any())
    nans = torch.tensor([1 in ms for ms in mats], device=DEV)
    assert bool(dx[nans].isnan().all()) and bool(nans.any())


def test_offsets_that_are_no_offsets_stay_inside():
    """Descending offsets and ones outside 0..R: other results, no write outside y, dx or dW."""
    g = torch.Generator(device=DEV).manual_seed(13)
    M, N, K, R = 6, 64, 64, 200
    x, w, dy = whole(g, R, K), whole(g, M, N, K), whole(g, R, N)
    for bad in ([0, 150, 20, 180, 90, 10, 200], [-5, 30, 2 ** 31 - 1, 7, -2 ** 31, 90, 1000], [200] * 7):
        offsets = torch.tensor(bad, dtype=torch.int32, device=DEV)
        y = torch.full((R + 64, N), 7.0, device=DEV)
        run(x, w, R, torch.float32, offsets, None, y=y[:R])
        assert bool((y[R:] == 7).all())
        dx = torch.full((R + 64, K), 7.0, device=DEV)
        run_backward(x, w, dy, offsets, None, None, torch.float32, dx=dx[:R])
        assert bool((dx[R:] == 7).all())


def test_no_rows():
    g = torch.Generator(device=DEV).manual_seed(14)
    x, w = whole(g, 3, 64), whole(g, 4, 32, 64)
    offsets = torch.zeros(5, dtype=torch.int32, device=DEV)
    empty = torch.empty(0, dtype=torch.int32, device=DEV)
    run(x, w, 0, torch.float32, offsets, empty)
    token_rows = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    dx, dw = run_backward(x, w, torch.empty(0, 32, dtype=torch.bfloat16, device=DEV), offsets, empty, token_rows, torch.float32)
    assert bool((dw == 0).all()) and bool((dx == 0).all())


@pytest.mark.parametrize("T,M,N,K,k", [(8, 64, 128, 1024, 4), (600, 4, 256, 1024, 2)])
def test_side_stream_graph_replays_and_two_calls_at_once(T, M, N, K, k):
    g = torch.Generator(device=DEV).manual_seed(15)
    R, off, offsets, src, token_rows = plan(T, M, k, 6)
    x, w, dy = whole(g, T, K), whole(g, M, N, K), whole(g, R, N)
    nbytes = max(em.edge_moe_dense_product_ws_bytes(T, R, M, N, K), em.edge_moe_dense_product_backward_ws_bytes(T, R, M, N, K))

    def outputs():
        return (torch.empty(R, N, device=DEV), torch.empty(T, K, device=DEV), torch.empty(M, N, K, device=DEV),
                torch.empty(nbytes, dtype=torch.uint8, device=DEV))

    def step(y, dx, dw, ws):
        em.edge_moe_dense_product(x, w, y, ws, offsets=offsets, row_src=src)
        em.edge_moe_dense_product_backward(dy, ws, x=x, w=w, dx=dx, dw=dw, offsets=offsets, row_src=src, token_rows=token_rows)
    a, b = outputs(), outputs()
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        step(*a)
    with torch.cuda.stream(t):
        step(*b)
    torch.cuda.synchronize()
    want = product(x, w, off, src, R), *gradients(x, w, dy, off, src, token_rows)
    for o in (a, b):
        for got, ref in zip(o, want):
            same(got, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*a)
    for _ in range(3):
        x.copy_(whole(g, T, K))
        dy.copy_(whole(g, R, N))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip(a, (product(x, w, off, src, R), *gradients(x, w, dy, off, src, token_rows))):
            same(got, ref)
