"""What the layer objects allocate for themselves on a given stream, on the host (no GPU): every allocation, fill and
library call of a call with stream= is made while that stream is current.  The library's calls are left out."""
import contextlib

import pytest
import torch

from mixed_precision_decode_b200 import bitsmoe as B
from mixed_precision_decode_b200 import layer as L

STREAM = 0x5eed
E, K, D, F, R = 4, 2, 16, 8, 6


@pytest.fixture
def watch(monkeypatch):
    """Names of the allocations and calls made, each with whether STREAM was current."""
    seen, depth = [], [0]

    @contextlib.contextmanager
    def on(stream, *like):
        depth[0] += stream == STREAM
        yield
        depth[0] -= stream == STREAM

    def noted(name, f):
        def call(*a, **k):
            seen.append((name, depth[0] > 0))
            return f(*a, **k)
        return call

    monkeypatch.setattr(L, "_on", on)
    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, noted("torch." + name, getattr(torch, name)))
    for name in ("contiguous", "cpu"):
        monkeypatch.setattr(torch.Tensor, name, noted(name, getattr(torch.Tensor, name)))
    for name in ("compute_scales", "pack", "layer_forward", "layer_forward_chained", "ffn_forward", "ffn_down_q4", "q4_pack",
                 "q4_unpack", "topk_route", "dense_ffn_forward", "norm_residual", "shared_proj", "ssd_decompose"):
        monkeypatch.setattr(L.B, name, noted(name, lambda *a, **k: None))
    monkeypatch.setattr(L.B, "ssd_workspace_bytes", lambda *a: 64)

    def check(*calls):
        made = [n for n, _ in seen]
        assert all(c in made for c in calls), made
        assert all(inside for _, inside in seen), [n for n, inside in seen if not inside]
        seen.clear()

    check.clear = seen.clear
    return check


def _projection():
    widths = torch.full((E, R), 4, dtype=torch.uint8)
    return L.PackedProjection.from_factors(torch.randn(R, D).half(), torch.rand(E, R), torch.randn(E, R, F), widths, K,
                                           stream=STREAM)


def _layer():
    return L.SpectralMoELayer(_projection(), _projection())


def _tokens(T):
    return torch.randn(T, D).half(), torch.zeros(T, K, dtype=torch.int32), torch.rand(T, K)


def test_packing_and_decomposition(watch):
    _projection()
    watch("torch.empty", "compute_scales", "pack")
    W = torch.randn(E, F, D)
    watch.clear()
    _, dec = L.decompose_and_pack(W, R, [4, 2], [2, R - 2], K, stream=STREAM)
    watch("torch.empty", "ssd_decompose", "pack")
    x, ids, gw = _tokens(3)
    dec["amps"], dec["comps"] = torch.rand(E, R), torch.randn(E, R, F)
    watch.clear()
    L.fqcm_widths(dec, x, ids, gw, 3.0, stream=STREAM)
    watch("torch.empty", "shared_proj")


@pytest.mark.parametrize("T", [1, 3])
def test_spectral_layer(watch, T):
    layer = _layer()
    tokens = _tokens(T)
    watch.clear()
    layer.forward(*tokens, want_experts=True, want_z=True, stream=STREAM)
    watch("torch.empty", "layer_forward")
    layer.forward(*tokens, stream=STREAM, next_layer=layer)
    watch("torch.empty", "layer_forward_chained")


@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("kind", ["fp16", "q4"])
def test_spectral_ffn(watch, kind, T):
    layer = _layer()
    wd = torch.randn(E, D, F).half()
    ffn = L.SpectralMoEFFN(layer, L.Q4Down.pack(wd, 32, stream=STREAM) if kind == "q4" else wd)
    tokens = _tokens(T)
    watch.clear()
    ffn.forward(*tokens, stream=STREAM)
    watch("torch.empty", *(["layer_forward", "ffn_down_q4"] if kind == "q4" else ["ffn_forward"]))


def test_routing_dense_ffn_and_block(watch):
    w = torch.randn(E, F, D).half()
    ffn = L.DenseMoEFFN(w, w, torch.randn(E, D, F).half(), K)
    blk = L.MoEBlock(ffn, torch.rand(D), torch.randn(E, D).half())
    h, logits = torch.randn(3, D), torch.randn(3, E)
    watch.clear()
    r = L.route(logits, K, stream=STREAM)
    watch("torch.empty", "topk_route")
    ffn.forward(h.half(), r, stream=STREAM)
    watch("torch.empty", "dense_ffn_forward")
    blk.forward(h, stream=STREAM)
    watch("torch.empty", "norm_residual", "shared_proj", "topk_route", "dense_ffn_forward")
