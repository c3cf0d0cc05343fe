"""What the layer objects keep between calls, on the host (no GPU): one token's state, and nothing that grows with the
batch sizes they have seen or that two calls of several tokens would share.  The library's calls only note their
workspace."""
import pytest
import torch

from mixed_precision_decode_b200 import layer as L

E, K, D, F, R = 4, 2, 16, 8, 6


@pytest.fixture
def used(monkeypatch):
    """The workspaces that the calls were given, held so that no memory is used twice."""
    got = []
    monkeypatch.setattr(L.B, "layer_forward", lambda g, u, x, i, w, T, ws, n, *a: got.append(("layer", ws, n)))
    monkeypatch.setattr(L.B, "ffn_forward", lambda g, u, wd, x, i, w, T, out, ws, n, *a: got.append(("ffn", ws, n)))
    monkeypatch.setattr(L.B, "ffn_down_q4", lambda d, b, g, yg, yu, i, w, T, out, ws, n, *a: got.append(("q4", ws, n)))
    for name in ("compute_scales", "pack", "q4_pack"):
        monkeypatch.setattr(L.B, name, lambda *a, **k: None)
    return got


def _object(kind):
    widths = torch.full((E, R), 4, dtype=torch.uint8)
    p = [L.PackedProjection.from_factors(torch.randn(R, D).half(), torch.rand(E, R), torch.randn(E, R, F), widths, K)
         for _ in range(2)]
    layer, wd = L.SpectralMoELayer(*p), torch.randn(E, D, F).half()
    return layer if kind == "layer" else L.SpectralMoEFFN(layer, L.Q4Down.pack(wd, 32) if kind == "q4" else wd)


def _call(obj, T):
    obj.forward(torch.randn(T, D).half(), torch.zeros(T, K, dtype=torch.int32), torch.rand(T, K))


def _bytes(obj):
    kept = (o._ws.one for o in (obj, getattr(obj, "layer", None)) if o is not None)
    return sum(t.nbytes for t in kept if t is not None)


@pytest.mark.parametrize("kind", ["layer", "fp16", "q4"])
def test_nothing_is_kept_for_the_batch_sizes_seen(used, kind):
    obj = _object(kind)
    _call(obj, 1)
    one = _bytes(obj)
    for T in (2, 3, 50, 200, 3):
        _call(obj, T)
    assert _bytes(obj) == one
    for _, ws, n in used:
        assert (0 if ws is None else ws.nbytes) >= n


@pytest.mark.parametrize("kind", ["layer", "fp16", "q4"])
def test_calls_of_several_tokens_share_nothing(used, kind):
    obj = _object(kind)
    for _ in range(2):
        _call(obj, 5)
    names = {name for name, _, _ in used}
    for name in names:
        a, b = (ws for n, ws, _ in used if n == name)
        assert a.data_ptr() != b.data_ptr()


@pytest.mark.parametrize("kind", ["layer", "fp16"])
def test_one_tokens_state_made_in_a_capture_is_the_graphs(used, kind, monkeypatch):
    """Zeros that are filled in when a graph is replayed must not serve a call outside it."""
    obj = _object(kind)
    monkeypatch.setattr(L, "_capturing", lambda t: True)
    _call(obj, 1)
    monkeypatch.setattr(L, "_capturing", lambda t: False)
    _call(obj, 1)
    _call(obj, 1)
    (_, a, _), (_, b, _), (_, c, _) = used
    assert a is not b and b is c


@pytest.mark.parametrize("kind", ["layer", "fp16"])
def test_one_tokens_state_is_kept_and_begins_as_zeros(used, kind):
    obj = _object(kind)
    for _ in range(2):
        _call(obj, 1)
    (_, a, _), (_, b, _) = used
    assert a is b and not a.any()
