"""Offsets of a grouped product that fall: no row belongs to two experts, and the others keep their results."""
import pytest
import torch

from mixed_precision_decode_b200 import bitsmoe as B

pytestmark = pytest.mark.gpu

U23, U24 = 2.0 ** -23, 2.0 ** -24


def _offsets(kind, E, n):
    off = [round(n * e / E) for e in range(E + 1)]
    if kind == "one":        # below the one before, and then the group after it would start among earlier rows
        off[2 * E // 3] = off[E // 4]
    elif kind == "early":    # a high one near the front, above many after it (more than a warp's 32 experts)
        off[1] = off[4 * E // 5]
    elif kind == "beyond":   # one past the rows, one below zero
        off[E // 2], off[E // 2 + 1] = n + 100, -7
    elif kind == "zigzag":
        off = [n if e % 2 else 0 for e in range(E + 1)]
    return off


@pytest.mark.parametrize("kind", ["one", "early", "beyond", "zigzag"])
@pytest.mark.parametrize("E, n, N, K", [(3, 12, 48, 64), (3, 480, 480, 64), (70, 140, 48, 64), (70, 700, 264, 64),
                                        (3, 480, 480, 1032)])
@pytest.mark.parametrize("form", ["sorted", "scatter", "gated", "gated_gather"])
def test_falling_offsets(E, n, N, K, kind, form):
    """An offset counts as the largest up to it, inside the rows (480 and 700 rows: the kernel for many rows).

    K products and sums of fp16 values in fp32, truncated at most twice in each step of 16: (K / 16 + 24) units of 2^-23
    of the terms' absolute sum, as in test_gpu_block_ops.py, or K + 24 units of 2^-24 one after the other; the gate's SiLU
    has slope 1.1 at most."""
    g = torch.Generator(device="cuda")
    g.manual_seed(E * n + N)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    a, W, U = r(n, K).half(), r(E, N, K).half(), r(E, N, K).half()
    rows = torch.randperm(n, generator=g, device="cuda").to(torch.int32) if form in ("scatter", "gated_gather") else None
    off = _offsets(kind, E, n)
    flat, most = [], 0
    for o in off:
        most = min(max(most, o), n)
        flat.append(most)
    out = torch.full((n, N), 7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.grouped_matmul(a, W, torch.tensor(off, dtype=torch.int32, device="cuda"), out, rows=rows, scatter=form == "scatter",
                     W_up=U if "gated" in form else None, status=st)
    assert B.read_status(st) == (0 if flat == off else B.ST_BADGROUP)  # "early" of 3 experts does not fall
    ref, tol = torch.full((n, N), 7.0, dtype=torch.float64, device="cuda"), torch.zeros(n, N, dtype=torch.float64, device="cuda")
    units = max((K // 16 + 24) * U23, (K + 24) * U24)
    for e in range(E):
        at = torch.arange(flat[e], flat[e + 1], device="cuda")
        src = at if rows is None else rows[at].long()
        at = src if form == "scatter" else at
        x, w, u = a[src].double(), W[e].double().T, U[e].double().T
        y, t = x @ w, units * (x.abs() @ w.abs())
        if "gated" in form:
            s, up = y * torch.sigmoid(y), x @ u
            t = 1.1 * t * up.abs() + s.abs() * units * (x.abs() @ u.abs()) + (s * up).abs() * 16 * U24
            y = s * up
        ref[at], tol[at] = y, 1.01 * t + U24 * y.abs() + 1e-30
    assert bool(((out.double() - ref).abs() <= tol).all())
