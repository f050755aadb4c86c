"""load() and the host-only calls need no more of torch than that it imports: a
build without GPU support, or an older one, has neither the private device
calls nor every type."""
import pytest
import torch

import shared_matrix_expert_amd as em
import synth


@pytest.fixture
def plain_torch(monkeypatch):
    for where, name in ((torch._C, "_cuda_getDevice"), (torch._C, "_cuda_getCurrentRawStream"), (torch, "uint16")):
        monkeypatch.delattr(where, name, raising=False)
    monkeypatch.setattr(em, "_lib", None)
    for table in (em._dtypes, em._dense_types):
        monkeypatch.setattr(em, "_dtypes" if table is em._dtypes else "_dense_types", {})
    monkeypatch.setattr(em._cuda, "getDevice", None)
    monkeypatch.setattr(em._cuda, "getRawStream", None)
    return monkeypatch


def test_host_only_calls(plain_torch):
    D = synth.config(2).dims
    assert em.edge_moe_workspace_bytes(D) > 0
    assert em.edge_moe_mx_product_ws_bytes(8, 8, 1, 64, 256, em.MX_FP8) > 0
    assert em.edge_moe_abi_version() > 0
    assert em._dense_type(torch.zeros(1, dtype=torch.bfloat16)) == 0


def test_public_calls_stand_in(plain_torch):
    em.load()

    class Stream:
        cuda_stream = 77
    plain_torch.setattr(torch.cuda, "current_device", lambda: 3)
    plain_torch.setattr(torch.cuda, "current_stream", lambda device=None: Stream() if device == 3 else None)
    assert em._stream(None) == 77
    assert em._stream_on(3, None) == 77


def test_the_current_device_by_the_public_call(plain_torch):
    plain_torch.setattr(torch.cuda, "current_device", lambda: 3)
    em.load()
    assert em._cuda.getDevice() == 3
