"""The norm and the products on bases that lie no better than documented: rows at 16 bytes,
lists, scales and statistics at 4, the int4 product's y at its element."""
import pytest
import torch

import shared_matrix_expert_amd as em
from gpu_helpers import DEV, say
from test_gpu_dense_product import TYPES, gradients, plan, product, same, whole
from test_gpu_packed_product import matrices

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)


def at(t, nbytes):
    """A contiguous copy of t whose address is `nbytes` past a multiple of 256."""
    b = torch.full((t.numel() * t.element_size() + 512,), 0x55, dtype=torch.uint8, device=DEV)
    return b[nbytes:nbytes + t.numel() * t.element_size()].view(t.dtype).view(t.shape).copy_(t)


@pytest.mark.parametrize("T,M,N,K,k,q", [(1, 1, 512, 4096, 0, 128), (9, 1, 300, 8192, 0, 128), (40, 1, 256, 4096, 0, 32),
                                         (300, 64, 128, 1024, 8, 64), (1200, 1, 130, 416, 0, 32), (1001, 8, 512, 1024, 0, 128),
                                         (256, 1, 4096, 4096, 0, 128), (70, 1, 9, 96, 0, 32)])
def test_int4_product(T, M, N, K, k, q):
    say(f"case: int4 product at its alignments, {T} tokens, {M} x {N} x {K}, groups of {q}")
    g = torch.Generator(device=DEV).manual_seed(K)
    R, off, offsets, src, _ = plan(T, M, k, 5)
    x = whole(g, T, K)
    codes, scales, w = matrices(g, M, N, K, q)
    want = product(x, w, off, src, R)
    ws = torch.empty(em.edge_moe_packed_product_ws_bytes(T, R, M, N, K, q), dtype=torch.uint8, device=DEV)
    for out in TYPES.values():
        y = at(torch.full((R, N), 7.0, dtype=out, device=DEV), out.itemsize)
        em.edge_moe_packed_product(q, at(x, 16), at(codes, 48), at(scales, 4), y, ws, offsets=at(offsets, 4) if M > 1 else None,
                                   row_src=None if src is None else at(src, 12))
        same(y, want)


@pytest.mark.parametrize("T,M,N,K,k", [(8, 64, 128, 512, 4), (1501, 8, 16, 1024, 3), (600, 4, 256, 1024, 2), (96, 1, 264, 520, 0)])
def test_dense_product(T, M, N, K, k):
    say(f"case: dense product at its alignments, {T} tokens, {M} x {N} x {K}")
    g = torch.Generator(device=DEV).manual_seed(K)
    R, off, offsets, src, token_rows = plan(T, M, k, 5)
    x, w, dy = whole(g, T, K), whole(g, M, N, K), whole(g, R, N)
    lists = dict(offsets=at(offsets, 4) if M > 1 else None, row_src=None if src is None else at(src, 12))
    ws = torch.empty(max(em.edge_moe_dense_product_ws_bytes(T, R, M, N, K), em.edge_moe_dense_product_backward_ws_bytes(T, R, M, N, K)),
                     dtype=torch.uint8, device=DEV)
    want_dx, want_dw = gradients(x, w, dy, off, src, token_rows)
    for out in TYPES.values():
        y, dx, dw = (at(torch.full(s, 7.0, dtype=out, device=DEV), 16) for s in ((R, N), (T, K), (M, N, K)))
        em.edge_moe_dense_product(at(x, 16), at(w, 48), y, ws, **lists)
        em.edge_moe_dense_product_backward(at(dy, 80), ws, x=at(x, 16), w=at(w, 48), dx=dx, dw=dw,
                                           token_rows=None if token_rows is None else at(token_rows, 4), **lists)
        same(y, product(x, w, off, src, R))
        same(dx, want_dx)
        same(dw, want_dw)


@pytest.mark.parametrize("T,d", [(5, 128), (300, 1000), (77, 4096), (9, 16384)])
def test_norm(T, d):
    say(f"case: norm at its alignments, {T} x {d}")
    g = torch.Generator(device=DEV).manual_seed(d)
    x, add, dy = (torch.randn(T, d, generator=g, device=DEV).to(t) for t in (torch.bfloat16, torch.float32, torch.float32))
    gain = torch.randn(d, generator=g, device=DEV)
    ws = torch.empty(em.edge_moe_norm_backward_ws_bytes(T, d), dtype=torch.uint8, device=DEV)
    results = []
    for far in (0, 16):                                           # bases at 256 bytes, and no better than asked for
        def new(*s, dtype=torch.bfloat16):
            return at(torch.zeros(*s, dtype=dtype, device=DEV), far)
        x_out, y, codes = new(T, d), new(T, d), new(T, d, dtype=torch.uint8)
        scales = at(torch.zeros(d // 128, T, 4, dtype=torch.uint8, device=DEV), far // 4) if d % 128 == 0 else None
        rstd, dgain = (at(torch.zeros(n, device=DEV), far // 4) for n in (T, d))
        dx = new(T, d, dtype=torch.float32)
        em.edge_moe_norm(at(x, far), at(gain, far), 1e-5, add=at(add, far), x_out=x_out, y=y, codes=codes if d % 128 == 0 else None,
                         scales=scales, rstd=rstd)
        em.edge_moe_norm_backward(x_out, at(gain, far), rstd, at(dy, far), ws, dres=at(add, far), dx=dx, dgain=dgain)
        results.append([t for t in (x_out, y, codes, scales, rstd, dx, dgain) if t is not None])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert bool(results[0][0].any()) and bool(results[0][-1].any())


@pytest.mark.parametrize("T,M,N,K,k", [(1, 1, 256, 512, 0), (300, 6, 129, 256, 2), (2000, 4, 512, 512, 2)])
def test_product_of_codes(T, M, N, K, k):
    say(f"case: product of codes at its alignments, {T} tokens, {M} x {N} x {K}")
    g = torch.Generator(device=DEV).manual_seed(N)
    R, off, offsets, src, _ = plan(T, M, k, 5)
    codes = torch.randint(0, 256, (M, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(118, 122, (M, K // 128, N, 4), generator=g, device=DEV, dtype=torch.uint8)
    xc, xs = torch.empty(T, K, dtype=torch.uint8, device=DEV), torch.empty(K // 128, T, 4, dtype=torch.uint8, device=DEV)
    em.edge_moe_mx_quantize(em.MX_FP8, torch.randn(T, K, generator=g, device=DEV).to(torch.bfloat16), xc, xs)
    ys = []
    for far, near, by_element in ((0, 0, 0), (16, 4, 2)):
        y = at(torch.zeros(R, N, dtype=torch.bfloat16, device=DEV), by_element)
        em.edge_moe_mx_product_coded(em.MX_FP8, at(xc, far), at(xs, near), at(codes, far), at(scales, near), y,
                                     offsets=at(offsets, near) if M > 1 else None, row_src=None if src is None else at(src, near))
        ys.append(y)
    assert torch.equal(*ys) and bool(ys[0].any())
