"""mx_weights and tile_weights make tensors and fill them on a stream the caller
names.  Torch hands out memory in the order of the stream it was asked on, so
the tensors have to be asked for on the stream that fills them (no GPU needed
here: streams and launches are stand-ins)."""
import contextlib

import pytest
import torch

import shared_matrix_expert_amd as em
import synth


class Stream:
    cuda_stream = 0x1234


@pytest.fixture
def asked(monkeypatch):
    """The stream each tensor was asked for on (None: the current one)."""
    now, seen = [None], []

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    def spy(make):
        def made(*a, **kw):
            seen.append(now[-1])
            return make(*a, **kw)
        return made
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    monkeypatch.setattr(torch, "empty", spy(torch.empty))
    monkeypatch.setattr(torch, "empty_like", spy(torch.empty_like))
    return seen


S = Stream()
STREAMS = [(None, None), (S, S), (0x77, ("external", 0x77)), (0, "default")]


@pytest.mark.parametrize("stream,owner", STREAMS)
def test_mx_weights_belong_to_the_stream_that_fills_them(monkeypatch, asked, stream, owner):
    filled = []
    monkeypatch.setattr(em, "edge_moe_mx_quantize", lambda fmt, src, codes, scales, s: filled.append(s))
    dense = {k: torch.zeros(1, 1, 128) for k in em._WEIGHT_KEYS[:16]}
    asked.clear()
    em.mx_weights(dense, stream)
    assert filled == [stream] * 6
    assert asked == [owner] * 12


@pytest.mark.parametrize("stream,owner", STREAMS)
def test_tiled_weights_belong_to_the_stream_that_fills_them(monkeypatch, asked, stream, owner):
    filled = []
    monkeypatch.setattr(em, "edge_moe_tile_shared", lambda dims, which, src, dst, s: filled.append(s))
    D = synth.config(2).dims
    em.tile_weights(D, {k: torch.zeros(2) for k in em._WEIGHT_KEYS[:16]}, stream)
    assert filled == [stream] * 4
    assert asked == [owner] * 4
