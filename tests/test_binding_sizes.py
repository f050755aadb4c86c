"""Sizes past 32 bits reach the library as sizes that it refuses, not with their
upper bits cut off (a batch of 2^32 + 4 tokens is no batch of 4)."""
from types import SimpleNamespace

import pytest
import torch

import shared_matrix_expert_amd as em
from fakes import fake, on_device

BIG = 1 << 32
U8, I32, BF16 = torch.uint8, torch.int32, torch.bfloat16


def dims(T, E=1, k=1, d=128):
    return SimpleNamespace(T=T, d=d, h=128, n_experts=E, experts_per_group=E, top_k=k, delta_rank=8, lora_rank=2,
                           quant_group=32)


def test_structs_keep_whole_sizes():
    D = em.cdims(dims(7, 64, 4, 512))
    assert [getattr(D, n) for n, _ in em.CDims._fields_] == [7, 512, 128, 64, 64, 4, 8, 2, 32]
    assert em.cdims(dims(BIG + 4)).T == (1 << 31) - 1 and em.cdims(dims(-BIG + 4)).T == -(1 << 31)
    assert em.cdims(dims((1 << 31) - 1)).T == (1 << 31) - 1 and em.cdims(dims(4.0)).T == 4
    assert em.cdims(dims(4, d=BIG + 128)).d == (1 << 31) - 1


def test_workspace_sizes():
    assert em.edge_moe_workspace_bytes(dims(BIG + 4)) == 0
    assert em.edge_moe_balance_ws_bytes(dims(BIG + 4), 1) == 0 and em.edge_moe_balance_ws_bytes(dims(4), BIG + 1) == 0
    assert em.edge_moe_route_backward_ws_bytes(dims(BIG + 4)) == 0
    ok = (8, 8, 1, 64, 256, em.MX_FP8)
    assert em.edge_moe_mx_product_ws_bytes(*ok) > 0
    for i in range(6):
        bad = list(ok)
        bad[i] += BIG
        assert em.edge_moe_mx_product_ws_bytes(*bad) == 0, bad


def refused(call, *args, **kw):
    with pytest.raises(em.EdgeMoeError) as e:
        call(*args, **kw)
    return e.value.status


def test_rounding(monkeypatch):
    on_device(monkeypatch)
    for N, K in ((1, BIG + 128), (BIG + 1, 128)):
        for fmt, per in ((em.MX_FP4, K // 2), (em.MX_FP8, K)):
            a = fake(N, K, dtype=BF16), fake(N, per, dtype=U8), fake(K // 128, N, 4, dtype=U8)
            assert refused(em.edge_moe_mx_quantize, fmt, *a) == em.EDGE_MOE_EUNSUPPORTED
            assert refused(em.edge_moe_mx_dequantize, fmt, *a[1:], a[0]) == em.EDGE_MOE_EUNSUPPORTED


def test_product(monkeypatch):
    on_device(monkeypatch)
    ws = fake(1 << 30, dtype=U8)
    for N, K in ((16, BIG + 128), (BIG + 16, 128)):
        a = (fake(4, K, dtype=BF16), fake(1, N, K // 2, dtype=U8), fake(1, K // 128, N, 4, dtype=U8), fake(4, N, dtype=BF16))
        assert refused(em.edge_moe_mx_product, em.MX_FP8, *a, ws) == em.EDGE_MOE_EUNSUPPORTED


def test_router(monkeypatch):
    on_device(monkeypatch)
    T, ws = BIG + 4, fake(1 << 30, dtype=U8)
    z, idx = fake(T, 1), fake(T, 1, dtype=I32)
    assert refused(em.edge_moe_balance, dims(T), z, idx, fake(1, 1, dtype=I32), fake(1, 1), fake(2), ws) == em.EDGE_MOE_EUNSUPPORTED
    assert refused(em.edge_moe_route_backward, dims(T), z, idx, ws, topk_w=z, d_topk_w=z, dbias=fake(1)) == em.EDGE_MOE_EUNSUPPORTED
    S = BIG + 1
    load = dict(seq_offsets=fake(S + 1, dtype=I32))
    counts = fake(S, 1, dtype=I32)
    assert refused(em.edge_moe_balance, dims(4), fake(4, 1), fake(4, 1, dtype=I32), counts, fake(S, 1), fake(2), ws,
                   **load) == em.EDGE_MOE_EUNSUPPORTED
    assert refused(em.edge_moe_route_backward, dims(4), fake(4, 1), fake(4, 1, dtype=I32), ws, d_loss=fake(2), counts=counts,
                   dbias=fake(1), **load) == em.EDGE_MOE_EUNSUPPORTED
