"""The norm and the products with dense, int4 and MX matrices in one run beside the
layer, on one side stream and one workspace: a training step of dense experts between
two layers, and a serving step from the norm's codes.  Each step is held to float64 on
that step's inputs."""
import pytest
import torch

import shared_matrix_expert_amd as em
import synth
from gpu_helpers import DEV, bits_to_dev, say
from test_gpu_dense_product import U, gathered, gradients, product
from test_gpu_norm import check_backward, forward, half

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)


def within(got, want, mag, n):
    tol = (2 * (n // 32 + 1) + 40) * U * mag + torch.finfo(got.dtype).eps / 2 * want.abs() + 2.0 ** -134
    assert bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("T", [1, 96, 500])
def test_training_and_serving_step(T):
    D = synth.config(5).dims.with_T(T)
    E, k, d, r = D.n_experts, D.top_k, D.d, D.delta_rank
    R = T * k
    g = torch.Generator(device=DEV).manual_seed(21)

    def randn(*s, scale=1.0, dtype=torch.bfloat16):
        return (scale * torch.randn(*s, generator=g, device=DEV)).to(dtype)
    x, add, gain = randn(T, d), randn(T, d, dtype=torch.float32), randn(d, scale=0.2) + 1
    wr = bits_to_dev(synth.make_router(5, 3)[0])
    up, down = randn(E, r, d, scale=0.05), randn(E, d, r, scale=0.1)
    d_out = randn(T, d, scale=0.1, dtype=torch.float32)
    W4 = synth.make_weights(5, 0, device=DEV)
    ws = torch.empty(max(em.edge_moe_workspace_bytes(D), em.edge_moe_norm_backward_ws_bytes(T, d),
                         em.edge_moe_dense_product_ws_bytes(T, R, E, r, d), em.edge_moe_dense_product_ws_bytes(R, R, E, d, r),
                         em.edge_moe_dense_product_backward_ws_bytes(T, R, E, r, d),
                         em.edge_moe_dense_product_backward_ws_bytes(R, R, E, d, r),
                         em.edge_moe_packed_product_ws_bytes(T, R, E, r, d, D.quant_group)), dtype=torch.uint8, device=DEV)

    def new(*s, dtype=torch.bfloat16):
        return torch.empty(*s, dtype=dtype, device=DEV)
    f = torch.float32
    x_out, y, rstd = new(T, d), new(T, d), new(T, dtype=f)
    codes, scales = new(T, d, dtype=torch.uint8), new(d // 128, T, 4, dtype=torch.uint8)
    idx, w = new(T, k, dtype=torch.int32), new(T, k, dtype=f)
    h, o = new(R, r), new(R, d)
    do, da, dh = new(R, d), new(R, r, dtype=f), new(R, r)
    d_up, d_down, dy = new(E, r, d, dtype=f), new(E, d, r), new(T, d, dtype=f)
    dx, dgain = new(T, d, dtype=f), new(d, dtype=f)
    q_up, e_up = new(E, r, d // 2, dtype=torch.uint8), new(E, d // 128, r, 4, dtype=torch.uint8)
    z, z2, z4 = new(R, r), new(R, r), new(R, r, dtype=f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        em.edge_moe_norm(x, gain, 1e-5, add=add, x_out=x_out, y=y, codes=codes, scales=scales, rstd=rstd)
        em.edge_moe_route(D, y, wr, None, idx, w, None, ws)
        order = torch.argsort(idx.reshape(-1).long() * T + torch.arange(T, device=DEV).repeat_interleave(k))
        src = (order // k).int()
        token_rows = torch.argsort(order).view(T, k).int()
        offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.bincount(idx.reshape(-1), minlength=E).cumsum(0)]).int()
        # forward and backward through the experts
        em.edge_moe_dense_product(y, up, h, ws, offsets=offsets, row_src=src)
        a = torch.nn.functional.silu(h.float()).to(torch.bfloat16)
        em.edge_moe_dense_product(a, down, o, ws, offsets=offsets)
        do.copy_(w.reshape(-1)[order].unsqueeze(1) * d_out[src.long()])
        em.edge_moe_dense_product_backward(do, ws, x=a, w=down, dx=da, dw=d_down, offsets=offsets)
        sg = torch.sigmoid(h.float())
        dh.copy_(da * sg * (1 + h.float() * (1 - sg)))
        em.edge_moe_dense_product_backward(dh, ws, x=y, w=up, dx=dy, dw=d_up, offsets=offsets, row_src=src, token_rows=token_rows)
        em.edge_moe_norm_backward(x_out, gain, rstd, dy, ws, dres=d_out, dx=dx, dgain=dgain)
        # serving: the same experts in MXFP4 from the norm's codes, and the layer's own int4 ones
        em.edge_moe_mx_quantize(em.MX_FP4, up, q_up, e_up)
        em.edge_moe_mx_product_coded(em.MX_FP8, codes, scales, q_up, e_up, z, offsets=offsets, row_src=src)
        em.edge_moe_mx_product(em.MX_FP8, y, q_up, e_up, z2, torch.empty(em.edge_moe_mx_product_ws_bytes(T, R, E, r, d, em.MX_FP8),
                                                                        dtype=torch.uint8, device=DEV), offsets=offsets, row_src=src)
        em.edge_moe_packed_product(D.quant_group, y, W4["a_up"], W4["a_up_scale"], z4, ws, offsets=offsets, row_src=src)
    s.synchronize()
    off = offsets.tolist()
    rr, _, yy = forward(x, gain, 1e-5, add)
    assert torch.equal(x_out.double(), rr)
    assert bool(((y.double() - yy).abs() <= (half(torch.bfloat16) + 4 * U) * yy.abs() + 2.0 ** -134).all())
    within(h, product(y, up, off, src, R), product(y.abs(), up.abs(), off, src, R), d)
    within(o, product(a, down, off, None, R), product(a.abs(), down.abs(), off, None, R), r)
    for got, args in (((da, d_down), (a, down, do, off, None, None)), ((dy, d_up), (y, up, dh, off, src, token_rows))):
        want, mag = gradients(*args), gradients(*(t.abs() if torch.is_tensor(t) and t.is_floating_point() else t for t in args))
        within(got[0], want[0], mag[0], args[2].shape[1] + 32 * k)
        within(got[1], want[1], mag[1], R)
    check_backward(x_out, gain, rstd, dy, d_out, dx, dgain)
    assert torch.equal(z, z2), "from the norm's codes the product has other bits"
    c = torch.stack([W4["a_up"] & 15, W4["a_up"] >> 4], -1).flatten(-2).long()
    w4 = torch.where(c > 7, c - 16, c).double() * W4["a_up_scale"].view(torch.float16).double().repeat_interleave(D.quant_group, -1)
    within(z4, product(y, w4, off, src, R), product(y.abs(), w4.abs(), off, src, R), 2 * d)
    say(f"  {T} tokens: |dx| {float(dx.abs().max()):.3g}, |d_up| {float(d_up.abs().max()):.3g}")


@pytest.mark.parametrize("fmt", [em.MX_FP4, em.MX_FP8], ids=["fp4", "fp8"])
@pytest.mark.parametrize("T,M,N,K,k", [(1, 1, 256, 512, 0), (20, 1, 1000, 256, 0), (700, 1, 264, 384, 0), (8, 64, 128, 512, 4),
                                       (300, 6, 129, 256, 2), (2000, 4, 512, 512, 2)])
def test_product_of_codes_has_the_products_bits(fmt, T, M, N, K, k):
    """Against edge_moe_mx_product on the rows that were coded; rows of no matrix stay,
    row_src entries that are no row give zeros."""
    g = torch.Generator(device=DEV).manual_seed(T + N)
    R = T * max(1, k)
    x = torch.randn(T, K, generator=g, device=DEV).to(torch.bfloat16)
    codes = torch.randint(0, 256, (M, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(118, 122, (M, K // 128, N, 4), generator=g, device=DEV, dtype=torch.uint8)
    offsets = src = None
    if k:
        src = torch.randint(0, T, (R,), generator=g, device=DEV, dtype=torch.int32)
        src[R // 2] = -1
    if M > 1:
        cut = torch.sort(torch.randint(0, R, (M - 1,), generator=g, device=DEV)).values
        offsets = torch.cat([torch.ones(1, dtype=torch.long, device=DEV), cut.clamp(min=1), torch.full((1,), R - 1, device=DEV)]).int()
    xc = torch.empty(T, K // 2 if fmt == em.MX_FP4 else K, dtype=torch.uint8, device=DEV)
    xs = torch.empty(K // 128, T, 4, dtype=torch.uint8, device=DEV)
    em.edge_moe_mx_quantize(fmt, x, xc, xs)
    y, want = (torch.full((R, N), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws = torch.empty(em.edge_moe_mx_product_ws_bytes(T, R, M, N, K, fmt), dtype=torch.uint8, device=DEV)
    em.edge_moe_mx_product(fmt, x, codes, scales, want, ws, offsets=offsets, row_src=src)
    em.edge_moe_mx_product_coded(fmt, xc, xs, codes, scales, y, offsets=offsets, row_src=src)
    assert torch.equal(y, want)
