"""Stand-ins for the binding's tests without a GPU: tensors that say they are on
one, and a library that records what it is called with."""
import torch

import shared_matrix_expert_amd as em


class OnGpu:
    """A tensor's type, shape and strides (of a meta tensor: no memory) with a
    GPU's index and an address that is never dereferenced."""

    def __init__(self, t, device=0, address=1 << 40):
        self._t, self._device, self._address = t.to("meta"), device, address
        self.is_cuda, self.device = device >= 0, f"cuda:{device}"

    def __getattr__(self, name):
        return getattr(self._t, name)

    def get_device(self):
        return self._device

    def data_ptr(self):
        return self._address


def fake(*shape, dtype=torch.float32, **kw):
    return OnGpu(torch.empty(*shape, dtype=dtype, device="meta"), **kw)


class Recorder:
    """Library whose calls all succeed; `calls` lists (name, arguments)."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return em.EDGE_MOE_OK
        return call


def on_device(monkeypatch, index=0, stream=0x55):
    """GPU `index` is the current one, with this current stream."""
    em.load()
    monkeypatch.setattr(em._cuda, "getDevice", lambda: index)
    monkeypatch.setattr(em._cuda, "getRawStream", lambda device: stream)
