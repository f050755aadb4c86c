"""The MX-matrix and router-training calls take streams of the tensors' GPU only
(no GPU needed: stand-ins for tensors, streams and the library)."""
from types import SimpleNamespace

import pytest
import torch

import shared_matrix_expert_amd as em
from fakes import Recorder, fake, on_device

U8, I32, BF16 = torch.uint8, torch.int32, torch.bfloat16
D = SimpleNamespace(T=4, d=128, h=128, n_experts=8, experts_per_group=8, top_k=2, delta_rank=8, lora_rank=2, quant_group=32)


def g(*shape, dtype=torch.float32):
    return fake(*shape, dtype=dtype, device=1)


def calls():
    ws = g(4096, dtype=U8)
    m = g(1, 16, 128, dtype=BF16), g(1, 16, 64, dtype=U8), g(1, 1, 16, 4, dtype=U8)
    z, idx, counts = g(4, 8), g(4, 2, dtype=I32), g(1, 8, dtype=I32)
    return {
        "quantize": lambda s: em.edge_moe_mx_quantize(em.MX_FP4, *m, stream=s),
        "dequantize": lambda s: em.edge_moe_mx_dequantize(em.MX_FP4, *m[1:], m[0], stream=s),
        "product": lambda s: em.edge_moe_mx_product(em.MX_FP8, g(4, 128, dtype=BF16), *m[1:], g(4, 16, dtype=BF16), ws, stream=s),
        "balance": lambda s: em.edge_moe_balance(D, z, idx, counts, g(1, 8), g(2), ws, stream=s),
        "backward": lambda s: em.edge_moe_route_backward(D, z, idx, ws, d_loss=g(2), counts=counts, dbias=g(8), stream=s),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_streams(monkeypatch, name):
    on_device(monkeypatch, 1, stream=0x99)
    lib = Recorder()
    monkeypatch.setattr(em, "_lib", lib)
    call = calls()[name]
    with pytest.raises(ValueError, match="stream must be of the tensors' GPU 1, got one of GPU 0"):
        call(SimpleNamespace(cuda_stream=0x77, device_index=0))
    assert not lib.calls
    for stream, handle in ((None, 0x99), (SimpleNamespace(cuda_stream=0x77, device_index=1), 0x77), (0x55, 0x55),
                           (SimpleNamespace(cuda_stream=0x66), 0x66)):
        call(stream)
        assert lib.calls.pop()[1][-1] == handle
