"""The norm's sums where they are long or not finite: dgain of many rows, whose error may
not grow with their number, and rows that hold an infinity."""
import pytest
import torch

import shared_matrix_expert_amd as em
from gpu_helpers import DEV, say
from test_gpu_norm import TYPES, check_backward, run_backward

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.mark.parametrize("d", [128, 1024, 4096, 16384, 32768])
def test_rows_with_an_infinity(d):
    """1 / sqrt(infinity) is zero: NaN where the infinity is, zeros beside it."""
    g = torch.Generator(device=DEV).manual_seed(d)
    x = torch.randn(9, d, generator=g, device=DEV).to(torch.bfloat16)
    x[2, 5], x[4, d - 1], x[6, 1], x[6, 2] = float("inf"), float("-inf"), float("inf"), float("nan")
    add = torch.zeros(9, d, device=DEV)
    add[7, 3] = float("inf")
    y, rstd = torch.empty_like(x), torch.empty(9, device=DEV)
    codes, scales = torch.empty(9, d, dtype=torch.uint8, device=DEV), torch.empty(d // 128, 9, 4, dtype=torch.uint8, device=DEV)
    em.edge_moe_norm(x, torch.ones(d, device=DEV), 1e-5, add=add, y=y, codes=codes, scales=scales, rstd=rstd)
    back = torch.empty(9, d, device=DEV)
    em.edge_moe_mx_dequantize(em.MX_FP8, codes, scales, back)
    for row, at in ((2, 5), (4, d - 1), (7, 3)):
        assert float(rstd[row]) == 0
        here = torch.arange(d, device=DEV) == at
        assert bool(y[row, here].isnan().all()) and bool((y[row, ~here] == 0).all())
        block = torch.arange(d, device=DEV) // 32 == at // 32
        assert bool(back[row, block].isnan().all()) and bool((back[row, ~block] == 0).all())
    assert bool(rstd[6].isnan()) and bool(y[6].isnan().all())
    ok = [0, 1, 3, 5, 8]
    assert bool(rstd[ok].isfinite().all()) and bool(y[ok].isfinite().all())


U = 2.0 ** -24
# Roundings of a term of dgain: v's, that of a workgroup's sum over its rows, and dgain's own.
TERM = 3.01 * U


@pytest.mark.parametrize("T,d", [(1 << 20, 8), (1 << 18, 512), (1 << 17, 1024), (1 << 17, 2048), (1 << 16, 4096), (1 << 15, 8192),
                                 (1 << 14, 16384), (1 << 13, 32768)])
def test_dgain_of_equal_rows(T, d):
    """Equal terms, whose float32 sum loses the same part of each row again and again: one
    part for every length of the sum, by column."""
    say(f"case: dgain of {T} equal rows of {d}")
    x, gain, rstd = torch.ones(T, d, dtype=torch.bfloat16, device=DEV), torch.ones(d, device=DEV), torch.ones(T, device=DEV)
    part = 0.4 * torch.exp2(-(torch.arange(d, device=DEV) % 8 + 13).float())
    dy = (1 + part).expand(T, d).contiguous()
    dgain = torch.empty(d, device=DEV)
    run_backward(x, gain, rstd, dy, dgain=dgain)
    want = T * (1 + part).double()
    assert bool(((dgain.double() - want).abs() <= TERM * want).all())


@pytest.mark.parametrize("grad", list(TYPES))
@pytest.mark.parametrize("T,d", [(262147, 64), (100003, 1000), (65539, 2056), (16385, 8200), (9001, 16392)])
def test_dgain_of_many_rows(T, d, grad):
    say(f"case: dgain of {T} rows of {d}, {grad}")
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
    dy = (1 + torch.rand(T, d, generator=g, device=DEV)).to(TYPES[grad]) * x.sign().to(TYPES[grad])      # terms of one sign
    gain, rstd, dgain = torch.ones(d, device=DEV), torch.rand(T, generator=g, device=DEV) + 0.5, torch.empty(d, device=DEV)
    run_backward(x, gain, rstd, dy, dgain=dgain)
    want = torch.zeros(d, dtype=torch.float64, device=DEV)
    for i in range(0, T, 8192):
        want += (dy[i:i + 8192].double() * x[i:i + 8192].double() * rstd[i:i + 8192, None].double()).sum(0)
    assert bool(((dgain.double() - want).abs() <= TERM * want).all())


@pytest.mark.parametrize("grad", list(TYPES))
@pytest.mark.parametrize("T,d", [(41, 1000), (300, 4096), (700, 8200), (257, 16384), (300, 32768)])
def test_gradients_over_the_ones_they_come_from(T, d, grad):
    """dx over dy, and over dres, with dgain: the bits of a call with rows of its own."""
    g = torch.Generator(device=DEV).manual_seed(T)
    x, rstd = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16), torch.rand(T, generator=g, device=DEV) + 0.5
    dy, dres = (torch.randn(T, d, generator=g, device=DEV).to(TYPES[grad]) for _ in range(2))
    gain = torch.randn(d, generator=g, device=DEV)
    dx, dgain, again = torch.empty_like(dy), torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    run_backward(x, gain, rstd, dy, dres, dx, dgain)
    check_backward(x, gain, rstd, dy, dres, dx, dgain)
    for over in ("dy", "dres"):
        a = dict(dy=dy.clone(), dres=dres.clone())
        run_backward(x, gain, rstd, a["dy"], a["dres"], a[over], again)
        assert torch.equal(a[over], dx) and torch.equal(again, dgain)


def test_wide_rows_on_two_streams_and_replayed():
    """Rows whose dgain is a pass of its own: two calls at once with a workspace each, and a
    captured one replayed over new gradients between eager calls."""
    g = torch.Generator(device=DEV).manual_seed(12)
    T, d = 700, 16384
    x, rstd = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16), torch.rand(T, generator=g, device=DEV) + 0.5
    gain, dres = torch.randn(d, generator=g, device=DEV), torch.randn(T, d, generator=g, device=DEV)
    dys = [torch.randn(T, d, generator=g, device=DEV) for _ in range(2)]
    out = [(torch.empty(T, d, device=DEV), torch.empty(d, device=DEV),
            torch.empty(em.edge_moe_norm_backward_ws_bytes(T, d), dtype=torch.uint8, device=DEV)) for _ in range(2)]

    def call(i):
        em.edge_moe_norm_backward(x, gain, rstd, dys[i], out[i][2], dres=dres, dx=out[i][0], dgain=out[i][1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(0)
    call(1)
    torch.cuda.synchronize()
    for i in range(2):
        check_backward(x, gain, rstd, dys[i], dres, out[i][0], out[i][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0)
    for _ in range(3):
        dys[0].copy_(torch.randn(T, d, generator=g, device=DEV))
        call(1)
        graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            check_backward(x, gain, rstd, dys[i], dres, out[i][0], out[i][1])
