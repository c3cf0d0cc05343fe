"""The layer objects' composition on the host (no GPU): which parameters a block hands to the operators.  The
operators are replaced by plain ones on the CPU."""
import warnings

import pytest
import torch

from mixed_precision_decode_b200 import bitsmoe as B
from mixed_precision_decode_b200 import layer as L


class PlainFFN:
    """A routed FFN whose output is one matrix times its input."""

    def __init__(self, m, E):
        self.m, self.dims = m, B.ffn_dims(m.shape[0], 8, E, 1)

    def forward(self, x, ids, gw, status=None, stream=None):
        return x.double() @ self.m.T


def _rms(v, w, eps):
    return v / torch.sqrt(v.square().mean(1, keepdim=True) + eps) * w


@pytest.fixture
def plain(monkeypatch):
    """norm_residual by its formula in 64 bits; routing, which PlainFFN does not look at, left out."""
    def norm(h, y=None, w_pre=None, x=None, *, w_post=None, gate=None, alpha=1.0, eps=1e-6, h_out=None, stream=None):
        v = h.double()
        if y is None:
            assert w_post is None and gate is None
        else:
            u = y.double() if w_post is None else _rms(y.double(), w_post, eps)
            v = v + alpha * u * (1.0 if gate is None else gate)
            h.copy_(v)
        if x is not None:
            x.copy_(_rms(v, w_pre, eps))

    monkeypatch.setattr(L.B, "norm_residual", norm)
    monkeypatch.setattr(L.B, "shared_proj", lambda *a, **k: None)
    monkeypatch.setattr(L, "route", lambda *a, **k: L.Routing(None, None, None, None))


def _blocks(n, d, E, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    return [L.MoEBlock(PlainFFN(r(d, d), E), 1 + 0.3 * r(d), r(E, d).half(), w_post=(1 + 0.3 * r(d)) if i % 3 else None,
                       alpha=0.5 + 0.25 * i) for i in range(n)], r(3, d)


def test_post_norm_and_alpha_belong_to_the_block_that_made_y(plain):
    """A stack whose blocks all have another w_post and alpha, against h <- h + alpha_b gate rmsnorm(y_b) w_post_b
    block by block.  x is fp16 between the norm and the FFN on both sides, so the two differ by 64-bit roundings only."""
    d, E = 24, 4
    blocks, h = _blocks(4, d, E, 7)
    gates = [torch.rand((3, 1), generator=torch.Generator().manual_seed(i), dtype=torch.float64) for i in range(4)]
    want = h.clone()
    for b, gate in zip(blocks, gates):
        y = _rms(want, b.w_norm, b.eps).half().double() @ b.ffn.m.T
        want += b.alpha * gate * (y if b.w_post is None else _rms(y, b.w_post, b.eps))
    y = before = gate = None
    for b, own in zip(blocks, gates):
        y = b.forward(h, y, gate=gate, made_by=before)
        before, gate = b, own
    blocks[-1].finish(h, y, gate=gate)
    assert float((h - want).abs().max()) <= 1e-9 * float(want.abs().max())


def test_made_by_as_a_pair_and_left_out(plain):
    d, E = 16, 4
    (a, b), h0 = _blocks(2, d, E, 8)
    h = h0.clone()
    y = a.forward(h)
    y_of_a, h1, h2 = y.clone(), h.clone(), h.clone()
    b.forward(h1, y, made_by=a)
    b.forward(h2, y, made_by=(a.w_post, a.alpha))
    assert torch.equal(h1, h2) and torch.equal(y, y_of_a)
    h3 = h.clone()
    with pytest.warns(UserWarning, match="made_by"):  # a stack whose blocks share them may leave it out
        b.forward(h3, y)
    assert torch.equal(h3, h + b.alpha * _rms(y, b.w_post, b.eps)) and not torch.equal(h3, h1)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        plain_block = L.MoEBlock(a.ffn, a.w_norm, a.w_router)
        plain_block.forward(h.clone(), y)  # nothing to be told
        b.forward(h.clone())
