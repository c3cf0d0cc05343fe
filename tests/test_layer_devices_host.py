"""Tensors on another GPU than the current one, on the host (no GPU): the layer objects make the tensors' GPU current
before they call the library, whose older calls go to the current one."""
import contextlib

import pytest
import torch

from mixed_precision_decode_b200 import layer as L


class At:
    """A tensor that says which GPU it is on, and nothing else."""

    def __init__(self, dev):
        self.dev = dev

    def get_device(self):
        return self.dev


@pytest.fixture
def current(monkeypatch):
    """Stands in for torch's current GPU and stream: [GPU, stream handle or None]."""
    now = [0, None]

    @contextlib.contextmanager
    def entered(dev, stream):
        before = list(now)
        now[:] = [dev, stream]
        yield
        now[:] = before

    monkeypatch.setattr(L, "_current_gpu", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", lambda dev: entered(int(dev), None))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: (0 if device is None else device, h))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: entered(*s))
    return now


@pytest.mark.parametrize("dev", [0, 1, 3])
@pytest.mark.parametrize("stream", [None, 0x5eed])
def test_the_tensors_gpu_is_current(current, dev, stream):
    with L._on(stream, At(dev)):
        assert current == [dev, stream]
    assert current == [0, None]


def test_host_tensors_change_nothing(current):
    with L._on(None, At(-1)):
        assert current == [0, None]


def test_block_calls_run_where_the_tensors_are(current, monkeypatch):
    """A block on GPU 1 while GPU 0 is current: its norm, router product, routing and FFN all run with GPU 1 current."""
    E, K, D, F = 4, 2, 16, 8
    at = []
    for name in ("norm_residual", "shared_proj", "topk_route", "dense_ffn_forward"):
        monkeypatch.setattr(L.B, name, lambda *a, name=name, **k: at.append((name, current[0])))
    w = torch.randn(E, F, D).half()
    blk = L.MoEBlock(L.DenseMoEFFN(w, w, torch.randn(E, D, F).half(), K), torch.rand(D), torch.randn(E, D).half())
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)
    blk.forward(torch.randn(3, D))
    assert at == [(n, 1) for n in ("norm_residual", "shared_proj", "topk_route", "dense_ffn_forward")]
