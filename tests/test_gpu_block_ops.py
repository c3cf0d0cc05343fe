"""The operators around the routed experts -- the norms with the gated residual, the
router with its grouped pairs, the 4-bit down projection and the products grouped by
expert -- against plain implementations in 64 bits.

Tolerances count roundings.  eps(t) / 2 of the value for one rounding to type t;
2^-24 relative for an fp32 operation, 2^-23 for an addition inside a tensor-core
instruction (it may truncate).  A sum of n terms v taken in N sequential additions is
off by at most N 2^-23 sum|v|."""
import numpy as np
import pytest
import torch

from mixed_precision_decode_b200 import bitsmoe as B

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U24, U23 = 2.0 ** -24, 2.0 ** -23
TINY = {F32: 2.0 ** -149, F16: 2.0 ** -24, BF16: 2.0 ** -133}  # smallest subnormals


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rounding(ref, dtype):
    """Bound of one rounding of ref to dtype."""
    return ref.abs() * (torch.finfo(dtype).eps / 2) + TINY[dtype]


def _within(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((err / tol).nan_to_num(nan=np.inf).max()))


# ---------------------------------------------------------------------------
# norms and residual
# ---------------------------------------------------------------------------
def _norm_ref(h, y, w_pre, w_post, gate, alpha, eps):
    """(h', x, bound of h' before rounding, bound of x before rounding), float64.  A row's sum of squares is
    taken in at most 60 sequential additions, so its inverse root is off by 32 units, the factors by one each."""
    c = 64 * U24
    h = h.double()
    v, size = h, h.abs()
    if y is not None:
        u = y.double()
        if w_post is not None:
            u = u / torch.sqrt(u.square().mean(1, keepdim=True) + eps) * w_post.double()
        u = alpha * u * (gate.double() if gate is not None else 1.0)
        v, size = h + u, h.abs() + u.abs()
    x = None
    if w_pre is not None:
        r = 1.0 / torch.sqrt(v.square().mean(1, keepdim=True) + eps)
        x = v * r * w_pre.double()
        # the error of h' and that of the root
        tx = c * (size * r * w_pre.double().abs() + x.abs() * (1 + (size.square().mean(1, keepdim=True)).sqrt() * r))
        return v, x, c * size, tx
    return v, x, c * size, None


NORM_CASES = [
    # T, d, h, y, x, post, gate
    (1, 2048, F32, F32, F16, False, None),
    (1, 1, F32, F32, F32, True, None),
    (3, 7, F16, BF16, F32, True, "token"),
    (5, 8, BF16, F32, BF16, False, "channel"),
    (333, 1001, F16, F32, F16, False, "token"),
    (131, 1999, BF16, BF16, BF16, True, "both"),
    (128, 4090, F16, F16, F32, True, "token"),
    (129, 1025, F32, F32, F32, False, "channel"),
    (150, 3251, F32, BF16, F16, True, "channel"),
    (9, 13, F32, F16, F16, True, "channel"),
    (6, 4090, F16, F16, F32, True, "token"),
    (6, 4091, F32, BF16, F32, False, "channel"),
    (1, 3251, F32, F32, BF16, True, "channel"),
    (50, 130, F32, F32, F32, True, None),
    (17, 256, BF16, F16, F16, True, "both"),
    (9, 520, F32, F32, BF16, True, "one"),
    (65, 1024, F16, F16, F16, True, "channel"),
    (4, 1032, F32, F32, F16, False, "both"),
    (7, 4096, BF16, F32, BF16, True, "channel"),
    (2, 8192, F32, BF16, F32, True, "token"),
    (2, 16384, F16, F16, F16, False, None),
    (2, 40000, F32, F32, F16, True, "channel"),   # wider than registers, 16-byte rows
    (2, 20001, BF16, F32, F16, True, "both"),     # wider than registers, any alignment
    (2, 5003, F16, F32, F32, True, "token"),
]


def _gate(g, kind, T, d):
    shape = {None: None, "token": (T, 1), "channel": (1, d), "both": (T, d), "one": (1, 1)}[kind]
    return None if shape is None else torch.sigmoid(_randn(g, *shape))


@pytest.mark.parametrize("case", NORM_CASES, ids=[f"{c[0]}x{c[1]}" for c in NORM_CASES])
@pytest.mark.parametrize("place", ["dense", "strided", "in_place"])
def test_norm_residual(case, place):
    T, d, ht, yt, xt, post, kind = case
    g = _gen(T * 10007 + d)
    pad = 0 if place != "strided" else 5

    def make(t, scale):
        buf = (scale * _randn(g, T, d + pad)).to(t)
        return buf[:, pad:] if pad else buf

    h, y = make(ht, 2.0), make(yt, 0.5)
    h_in = h.clone()
    x = torch.full((T, d + pad), float("nan"), dtype=xt, device="cuda")[:, :d]
    w_pre = 1 + 0.1 * _randn(g, d)
    w_post = 1 + 0.1 * _randn(g, d) if post else None
    gate = _gate(g, kind, T, d)
    out = None if place == "in_place" else torch.full((T, d + pad), float("nan"), dtype=ht, device="cuda")[:, :d]
    B.norm_residual(h, y, w_pre, x, w_post=w_post, gate=gate, alpha=0.7, eps=1e-5, h_out=out)
    rh, rx, th, tx = _norm_ref(h_in, y, w_pre, w_post, gate, 0.7, 1e-5)
    got = h if out is None else out
    _within(got, rh, th + _rounding(rh, ht), "h'")
    _within(x, rx, tx + _rounding(rx, xt), "x")
    if out is not None:
        assert torch.equal(h, h_in)


def test_norm_residual_parts():
    """The norm alone, the residual alone, and nothing written beside them."""
    g = _gen(3)
    h, y, w = _randn(g, 6, 96), _randn(g, 6, 96), _randn(g, 96)
    x = torch.empty(6, 96, device="cuda", dtype=F16)
    h0 = h.clone()
    B.norm_residual(h, w_pre=w, x=x)
    rh, rx, th, tx = _norm_ref(h, None, w, None, None, 1.0, 1e-6)
    _within(x, rx, tx + _rounding(rx, F16), "norm alone")
    assert torch.equal(h, h0)
    B.norm_residual(h, y, alpha=-0.5)
    rh, _, th, _ = _norm_ref(h0, y, None, None, None, -0.5, 1e-6)
    _within(h, rh, th + _rounding(rh, F32), "residual alone")
    B.norm_residual(h[:0], y[:0], w, x[:0])  # no rows


@pytest.mark.parametrize("d", [64, 2048, 40000])
def test_norm_residual_special_rows(d):
    """A row of zeros gives zeros; a NaN stays in its row."""
    g = _gen(4)
    h, w = _randn(g, 4, d), torch.ones(d, device="cuda")
    y = torch.zeros(4, d, device="cuda")
    h[1] = 0
    h[2, d // 2] = float("nan")
    x = torch.empty(4, d, device="cuda")
    B.norm_residual(h, y, w, x, w_post=w)
    assert bool((x[1] == 0).all()) and bool(torch.isnan(x[2]).all())
    assert bool(torch.isfinite(x[0]).all()) and bool(torch.isfinite(x[3]).all())


@pytest.mark.parametrize("T, d", [(9, 8), (9, 61), (9, 1001), (130, 61), (130, 1025), (130, 1026), (130, 1027), (130, 2050),
                                  (130, 4089), (130, 4090)])
@pytest.mark.parametrize("types", [(F16, F16, F16), (F32, BF16, F16), (BF16, F32, F32)])
def test_norm_residual_between_gaps(T, d, types):
    """Rows that start at any element, with gaps that agree modulo 4 between them: the results are those of dense
    rows, and what lies in the gaps, NaN, is neither read nor written."""
    ht, yt, xt = types
    g = _gen(d)
    nan = float("nan")

    def rows(t, ld, value=None):
        buf = torch.full((T, ld), nan, dtype=t, device="cuda")
        v = buf[:, :d]
        if value is not None:
            v.copy_(value)
        return buf, v

    h, y = _randn(g, T, d).to(ht), _randn(g, T, d).to(yt)
    w, wp, gate = 1 + 0.1 * _randn(g, d), 1 + 0.1 * _randn(g, d), _randn(g, T, d)
    for w_post in (None, wp):
        hb, hv = rows(ht, d + 4, h)
        yb, yv = rows(yt, d, y)
        ob, ov = rows(ht, d + 8)
        xb, xv = rows(xt, d + 12)
        B.norm_residual(hv, yv, w, xv, w_post=w_post, gate=gate, alpha=0.5, h_out=ov)
        rh, rx, th, tx = _norm_ref(h, y, w, w_post, gate, 0.5, 1e-6)
        _within(ov, rh, th + _rounding(rh, ht), "h'")
        _within(xv, rx, tx + _rounding(rx, xt), "x")
        B.norm_residual(hv, yv, w, xv, w_post=w_post, gate=gate, alpha=0.5)  # in place
        assert torch.equal(hv, ov)
        for b in (hb, ob, xb):
            assert bool(torch.isnan(b[:, d:]).all())


@pytest.mark.parametrize("T", [1, 2050])
@pytest.mark.parametrize("d", [1, 8, 64, 300, 520, 1000, 1001, 1026, 2000, 3999, 4090, 4104, 6000, 9000])
def test_norm_residual_infinity_in_the_last_place(d, T):
    """mean(h^2) is infinite, 1 / sqrt of it 0: the row's other elements become 0, the infinite one NaN (infinity
    times 0), and no other row notices; the same through the norm on y."""
    g = _gen(5)
    h, w = _randn(g, T, d).half(), torch.ones(d, device="cuda")
    h[-1, -1] = float("inf")
    y = torch.zeros(T, d, device="cuda")
    x = torch.empty(T, d, device="cuda")
    B.norm_residual(h.clone(), y, w, x, w_post=w)
    assert bool((x[-1, :-1] == 0).all()) and bool(torch.isnan(x[-1, -1])) and bool(torch.isfinite(x[:-1]).all())
    h_out = torch.empty_like(h)
    B.norm_residual(y.half(), h, w, x, w_post=w, h_out=h_out)
    assert bool((h_out[-1, :-1] == 0).all()) and bool(torch.isnan(h_out[-1, -1])) and bool(torch.isfinite(x[:-1]).all())


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------
def _route_ref(logits, K, scoring, renorm, scale):
    """ids, weights (float64), offsets, order on the CPU; rows with a NaN or +inf give -1 and 0."""
    l = logits.cpu().double()
    T, E = l.shape
    v, i = torch.sort(l, dim=1, descending=True, stable=True)
    ok = v[:, :K] > -np.inf
    ok &= (l < np.inf).all(1, keepdim=True)  # false for NaN too
    if scoring == "softmax":
        w = torch.exp(v[:, :K] - v[:, :1].clamp_min(-1e300))
        tot = torch.exp(l - v[:, :1].clamp_min(-1e300)).sum(1, keepdim=True)
    else:
        w, tot = 1 / (1 + torch.exp(-v[:, :K])), torch.ones(T, 1, dtype=torch.float64)
    w = torch.where(ok, w, torch.zeros_like(w))
    if renorm:
        tot = w.sum(1, keepdim=True)
    w = torch.where(ok, scale * w / tot, torch.zeros_like(w))
    ids = torch.where(ok, i[:, :K], -1)
    key = torch.where(ids < 0, E, ids).reshape(-1)
    order = torch.sort(key, stable=True).indices
    n = int((key < E).sum())
    order[n:] = -1
    offsets = torch.zeros(E + 1, dtype=torch.long)
    offsets[1:] = torch.bincount(key, minlength=E + 1)[:E].cumsum(0)
    return ids, w, offsets, order


def _route(logits, K, groups=True, **kw):
    T, E = logits.shape
    i32 = {"dtype": torch.int32, "device": "cuda"}
    ids, gw = torch.full((T, K), -7, **i32), torch.full((T, K), float("nan"), device="cuda")
    off, order = (torch.full((E + 1,), -7, **i32), torch.full((T * K,), -7, **i32)) if groups else (None, None)
    st = torch.zeros(1, **i32)
    n = B.topk_route_workspace_bytes(T, E, K)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    B.topk_route(logits, ids, gw, off, order, workspace=ws, status=st, **kw)
    return ids, gw, off, order, B.read_status(st)


def _check_route(logits, K, scoring, renorm, scale=1.0, status=0):
    ids, gw, off, order, st = _route(logits, K, scoring=scoring, renormalise=renorm, scale=scale)
    rids, rw, roff, rorder = _route_ref(logits, K, scoring, renorm, scale)
    assert st == status
    assert torch.equal(ids.cpu().long(), rids)
    assert torch.equal(off.cpu().long(), roff)
    assert torch.equal(order.cpu().long(), rorder)
    # the exponent's argument is off by one unit of |l - m| (up to ~30 here), exp by two, the sum by its additions
    _within(gw.cpu(), rw, 128 * U24 * rw.abs() + TINY[F32], "weights")


ROUTE_CASES = [
    (1, 1, 1), (1, 128, 8), (2, 5, 5), (31, 33, 3), (64, 128, 8), (128, 64, 6), (129, 128, 8), (1000, 200, 7),
    (5000, 128, 8), (300, 512, 16), (40, 513, 9), (500, 2000, 40), (3, 300, 64), (700, 32, 32), (260, 8192, 2),
]


@pytest.mark.parametrize("case", ROUTE_CASES, ids=["x".join(map(str, c)) for c in ROUTE_CASES])
@pytest.mark.parametrize("mode", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)],
                         ids=lambda m: m[0] + ("_renorm" if m[1] else ""))
def test_topk_route(case, mode):
    T, E, K = case
    g = _gen(T + 31 * E + K)
    dtype = (F32, F16, BF16)[(T + E) % 3]  # 16-bit logits have many equal values
    logits = (1.5 * _randn(g, T, E)).to(dtype)
    _check_route(logits, K, *mode, scale=2.5)


@pytest.mark.parametrize("T", [40, 400])
def test_topk_route_closed_and_bad_rows(T):
    """Closed experts, rows without any open one, ties of integers and of signed zeros, a strided operand,
    rows with NaN and +inf."""
    g = _gen(T)
    buf = torch.round(2 * _randn(g, T, 70))
    buf[buf == 0] *= -1.0
    logits = buf[:, 3:63]
    shut = torch.rand((T, 60), generator=g, device="cuda") < 0.7
    logits.masked_fill_(shut, float("-inf"))
    logits[5] = float("-inf")
    logits[T - 1, 1:] = float("-inf")
    for mode in (("softmax", True), ("softmax", False), ("sigmoid", True)):
        _check_route(logits, 9, *mode)
    logits[2, 7] = float("nan")
    logits[3, 59] = float("inf")
    _check_route(logits, 9, "softmax", True, status=B.ST_NONFINITE)
    _check_route(logits[:, :4], 4, "softmax", True)


def test_topk_route_extremes():
    """Logits whose exponentials leave fp32's range; every token on one expert; nothing but the ids."""
    l = torch.tensor([[3e38, -3e38, 0.0], [-200.0, -210.0, -3e38], [88.0, 89.0, 200.0]], device="cuda")
    for mode in (("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)):
        ids, gw, _, _, st = _route(l, 2, scoring=mode[0], renormalise=mode[1])
        rids, rw, _, _ = _route_ref(l, 2, mode[0], mode[1], 1.0)
        assert st == 0 and torch.equal(ids.cpu().long(), rids)
        # arguments up to 210 here: one unit of them in the exponent
        _within(gw.cpu(), rw, 512 * U24 * rw.abs() + 2.0 ** -125, mode)
    one = torch.zeros(300, 16, device="cuda")
    one[:, 11] = 1.0
    _check_route(one, 1, "softmax", True)
    ids, _, _, _, _ = _route(one, 1, groups=False)
    assert bool((ids == 11).all())
    off = torch.full((17,), -1, dtype=torch.int32, device="cuda")
    z = torch.empty(0, 1, dtype=torch.int32, device="cuda")
    B.topk_route(one[:0], z, z.float(), off)
    assert bool((off == 0).all())


# ---------------------------------------------------------------------------
# 4-bit matrices
# ---------------------------------------------------------------------------
def _q4_ref(W, G):
    """Codes and fp16 scales of W [E][rows][cols] by the stated quantiser (fp32 operations, as stated)."""
    W = W.float().cpu().numpy()
    E, R, C = W.shape
    Cp = -(-C // G) * G
    w = np.zeros((E, R, Cp), np.float32)
    w[:, :, :C] = W
    w = w.reshape(E, R, Cp // G, G)
    s = (np.float32(2) * np.abs(w).max(3) / np.float32(15)).astype(np.float16)
    sf = s.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(sf > 0, np.clip(np.floor(w / sf + np.float32(8)), 0, 15), 0)
    return q.reshape(E, R, Cp)[:, :, :C].astype(np.int64), s


def _q4_blob(W, G):
    blob = torch.full((B.q4_bytes(*W.shape, G),), 0xAB, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.q4_pack(W, G, blob, st)
    return blob, B.read_status(st)


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 37, 24), (3, 16, 64), (2, 50, 200), (1, 130, 328)])
def test_q4_pack_format(shape, G):
    """The packed bytes, decoded by the format's text, hold the quantiser's codes and scales; padding is zero;
    unpacking gives s (q - 7.5)."""
    E, R, C = shape
    g = _gen(R * C + G)
    W = _randn(g, E, R, C).to((F32, F16, BF16)[(R + G // 32) % 3])
    W[0, 0, : min(C, G)] = 0  # a group of zeros
    blob, st = _q4_blob(W, G)
    assert st == 0
    q, s = _q4_ref(W, G)
    Cp, nb = -(-C // max(64, G)) * max(64, G), -(-R // 16)
    blocks = blob.cpu().numpy().reshape(E, nb, -1)
    words = blocks[:, :, : 8 * Cp].copy().view(np.uint32).reshape(E, nb, Cp // 64, 32, 4)
    scales = blocks[:, :, 8 * Cp:].copy().view(np.float16).reshape(E, nb, Cp // G, 16)
    want_q = np.zeros((E, nb * 16, Cp), np.int64)
    want_q[:, :R, :C] = q
    got_q = np.zeros_like(want_q)
    for lane in range(32):
        a, b = lane // 4, lane % 4
        for t in range(4):
            for p in range(2):
                for u in range(2):
                    for v in range(2):
                        n = 4 * p + 2 * u + v
                        got_q[:, a + 8 * v::16, 16 * t + 8 * u + 2 * b + p::64] = words[:, :, :, lane, t] >> (4 * n) & 15
    assert np.array_equal(got_q, want_q)
    want_s = np.zeros((E, nb * 16, Cp // G), np.float16)
    want_s[:, :R, : s.shape[2]] = s
    got_s = scales.transpose(0, 1, 3, 2).reshape(E, nb * 16, Cp // G)
    assert np.array_equal(got_s.view(np.uint16), want_s.view(np.uint16))
    out = torch.empty(E, R, C, device="cuda")
    B.q4_unpack(blob, G, out)
    ref = (want_q[:, :R, :C] - 7.5) * np.repeat(want_s[:, :R].astype(np.float64), G, 2)[:, :, :C]
    assert np.array_equal(out.cpu().numpy(), ref.astype(np.float32))


def test_q4_pack_bad_groups():
    """A NaN, an infinity and a scale beyond fp16 store their group as zeros and set the status; others stay."""
    W = torch.ones(1, 4, 128, device="cuda")
    W[0, 1, 5] = float("nan")
    W[0, 2, 70] = float("inf")
    W[0, 3, 0] = 1e6
    blob, st = _q4_blob(W, 64)
    assert st == B.ST_NONFINITE | B.ST_BADSCALE
    out = torch.empty(1, 4, 128, device="cuda")
    B.q4_unpack(blob, 64, out)
    zero = torch.zeros(4, 2, dtype=torch.bool)
    zero[1, 0] = zero[2, 1] = zero[3, 0] = True
    got = (out.view(4, 2, 64) == 0).all(2).cpu()
    assert torch.equal(got, zero)


Q4_CASES = [
    # d_model, d_ff, E, K, T's
    (64, 32, 4, 2, (1, 4)),
    (37, 24, 6, 3, (1, 5, 40)),
    (16, 8, 3, 2, (1, 3)),
    (300, 136, 5, 5, (1, 2, 21)),
    (256, 64, 4, 2, (48, 130)),
    (2048, 768, 128, 8, (1, 2, 16, 64)),
    (1000, 4104, 8, 2, (1, 7)),
    (96, 14336, 8, 2, (1, 5)),
    (33, 520, 1, 1, (1, 100)),
    (64, 4096, 40, 24, (1, 3)),
]


def _q4_inputs(d_model, d_ff, E, K, T, seed, up=True):
    g = _gen(seed)
    W = _randn(g, E, d_model, d_ff) * d_ff ** -0.5
    yg, yu = 2 * _randn(g, T, K, d_ff), _randn(g, T, K, d_ff) if up else None
    ids = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :K].to(torch.int32).contiguous()
    return W, yg, yu, ids, torch.softmax(_randn(g, T, K), 1)


def _q4_run(dims, blob, G, yg, yu, ids, gw, out=None, stream=None):
    T = ids.shape[0]
    out = torch.full((T, dims.d_model), float("nan"), device="cuda") if out is None else out
    n = B.ffn_down_q4_workspace_bytes(dims, G, T)
    ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.ffn_down_q4(dims, blob, G, yg, yu, ids, gw, T, out, ws, n, st)
    return out, B.read_status(st)


def _q4_down_ref(blob, shape, G, yg, yu, ids, gw):
    """(out, bound), float64 on the GPU, expert by expert, from the unpacked values."""
    E, R, C = shape
    W = torch.empty(shape, device="cuda")
    B.q4_unpack(blob, G, W)
    T, K = ids.shape
    h = yg.double().view(T * K, C)
    if yu is not None:
        h = h * torch.sigmoid(h) * yu.double().view(T * K, C)
    y, size = torch.zeros(T * K, R, dtype=torch.float64, device="cuda"), torch.zeros(T * K, R, dtype=torch.float64, device="cuda")
    fixed = torch.zeros_like(y)
    flat = ids.view(-1)
    for e in range(E):
        at = (flat == e).nonzero().view(-1)
        if at.numel():
            y[at] = h[at] @ W[e].double().T
            a = W[e].double().abs().T
            size[at] = h[at].abs() @ a
            fixed[at] = h[at].abs().amax(1, keepdim=True) * a.sum(0)
    g = gw.double().view(T, K, 1)
    # h: a few units of fp32 (exp, division, product), then half a fixed-point unit, 2^-31 of a power of two that is at
    # most twice the row's largest |h|; the integer sums of a group are exact; the sum: G / 16 steps for a group's
    # conversions and scale, the groups, at most 8 column ranges, the slots
    n = G // 16 + C // G + 8 + K + 4
    tol = (n * U23 + 8 * U24) * size + 2.0 ** -30 * fixed
    return (y.view(T, K, R) * g).sum(1), (tol.view(T, K, R) * g.abs()).sum(1) + 1e-37


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("case", Q4_CASES, ids=["x".join(map(str, c[:4])) for c in Q4_CASES])
def test_ffn_down_q4(case, G):
    d_model, d_ff, E, K, tokens = case
    dims = B.ffn_dims(d_model, d_ff, E, K)
    for T in tokens:
        W, yg, yu, ids, gw = _q4_inputs(d_model, d_ff, E, K, T, 17 * T + d_ff)
        blob, st = _q4_blob(W, G)
        assert st == 0
        for up in (yu, None):
            out, st = _q4_run(dims, blob, G, yg, up, ids, gw)
            assert st == 0
            ref, tol = _q4_down_ref(blob, W.shape, G, yg, up, ids, gw)
            _within(out, ref, tol, (T, up is None))


@pytest.mark.parametrize("T", [1, 6])
def test_ffn_down_q4_ids(T):
    """Ids outside [0, E) are left out and reported; the same expert in two slots; every token on one expert; a
    token without any expert."""
    W, yg, yu, ids, gw = _q4_inputs(80, 96, 5, 3, T, 5 + T)
    dims = B.ffn_dims(80, 96, 5, 3)
    blob, _ = _q4_blob(W, 32)
    for edit, bad in ((lambda i: i.__setitem__((0, 1), -1), True), (lambda i: i.__setitem__((T - 1, 0), 5), True),
                      (lambda i: i.fill_(3), False), (lambda i: i[0].fill_(-1), True), (lambda i: i.fill_(99), True)):
        j = ids.clone()
        edit(j)
        out, st = _q4_run(dims, blob, 32, yg, yu, j, gw)
        assert st == (B.ST_BADEXPERT if bad else 0)
        ref, tol = _q4_down_ref(blob, W.shape, 32, yg, yu, j, gw)
        _within(out, ref, tol, "ids")


@pytest.mark.parametrize("T", [1, 5])
def test_ffn_down_q4_range(T):
    """|h| far beyond fp16's range and far below it: a power of two brings each row into range."""
    W, yg, yu, ids, gw = _q4_inputs(64, 128, 4, 2, T, 77)
    dims = B.ffn_dims(64, 128, 4, 2)
    blob, _ = _q4_blob(W, 64)
    for s in (1e8, 1e-12, 0.0):
        out, st = _q4_run(dims, blob, 64, s * yg, None, ids, gw)
        ref, tol = _q4_down_ref(blob, W.shape, 64, s * yg, None, ids, gw)
        assert st == 0
        _within(out, ref, tol, s)


# ---------------------------------------------------------------------------
# products grouped by expert
# ---------------------------------------------------------------------------
def _offsets(sizes):
    return torch.tensor([0] + list(np.cumsum(sizes)), dtype=torch.int32, device="cuda")


def _gmm_ref(a, W, W_up, offsets, rows, div, scatter, out, K):
    """(out, bound before rounding): float64 on the GPU; rows that no group names keep out's values."""
    ref = out.double().clone()
    tol = torch.zeros_like(ref)
    off = offsets.tolist()
    n = (K // 16 + 24) * U23
    for e in range(W.shape[0]):
        at = torch.arange(off[e], off[e + 1], device="cuda")
        if not at.numel():
            continue
        src = at if rows is None else rows[at].long() // div
        dst = rows[at].long() if scatter else at
        x = a[src].double()
        y, s = x @ W[e].double().T, x.abs() @ W[e].double().abs().T
        t = n * s
        if W_up is not None:
            u, su = x @ W_up[e].double().T, x.abs() @ W_up[e].double().abs().T
            sig = torch.sigmoid(y)
            # |SiLU'| <= 1.1; exp and division: the argument's rounding and a few units
            t = 1.1 * t * u.abs() + (y * sig).abs() * n * su + (y * sig * u).abs() * (8 + y.abs()) * U24
            t = t + 1.1 * n * s * n * su
            y = y * sig * u
        ref[dst], tol[dst] = y, t
    return ref, tol


def _check_gmm(sizes, N, K, dtype, out_dtype, form, seed=0, lda=0, spare=0):
    g = _gen(seed + N + 7 * K + sum(sizes))
    E, P = len(sizes), sum(sizes)
    W = (_randn(g, E, N, K) * K ** -0.5).to(dtype)
    W_up = (_randn(g, E, N, K) * K ** -0.5).to(dtype) if form.startswith("gated") else None
    n = P + spare
    rows, div, scatter = None, 1, False
    if form in ("gated_gather", "gather"):
        div = 3
        rows = torch.randint(0, max(1, n), (n,), generator=g, device="cuda", dtype=torch.int32)
        n_a = -(-n // div)
    else:
        n_a = n
        if form == "scatter":
            rows = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
            scatter = True
    a = _randn(g, n_a, K + lda).to(dtype)[:, :K]
    out = torch.full((n, N), 7.0, dtype=out_dtype, device="cuda")
    ref, tol = _gmm_ref(a, W, W_up, _offsets(sizes), rows, div, scatter, out, K)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.grouped_matmul(a, W, _offsets(sizes), out, W_up=W_up, rows=rows, rows_per_a=div, scatter=scatter, status=st)
    assert B.read_status(st) == 0
    _within(out, ref, torch.where(tol > 0, tol + _rounding(ref, out_dtype), tol), (form, N, K))


GMM_SIZES = [
    ([1], 16, 8), ([1, 0, 2], 5, 24), ([0, 7, 1, 0, 9], 130, 64), ([33, 1, 64, 0], 257, 136), ([3] * 40, 96, 256),
    ([8, 8, 8, 8, 8, 8, 8, 8], 768, 2048), ([300], 64, 72), ([129, 511, 2], 300, 520), ([257, 1, 0, 96, 40], 512, 1024),
    ([0, 0, 0, 5], 384, 4096), ([1000, 24], 128, 768), ([17] * 130, 264, 320),
    ([700], 257, 72), ([400, 3, 0, 200], 333, 8), ([2] * 200, 700, 40), ([1] * 129 + [0], 1030, 136),
]


@pytest.mark.parametrize("form", ["sorted", "gather", "scatter", "gated", "gated_gather"])
@pytest.mark.parametrize("case", GMM_SIZES, ids=[f"{len(s)}x{sum(s)}x{n}x{k}" for s, n, k in GMM_SIZES])
def test_grouped_matmul(case, form):
    sizes, N, K = case
    for dtype, out_dtype in ((F16, F16), (BF16, BF16), (F16, F32), (BF16, F32)):
        _check_gmm(sizes, N, K, dtype, out_dtype, form)


def test_grouped_matmul_strided_and_spare_rows():
    """Rows of A further apart than K; places behind the last group and rows without a pair stay as they were."""
    for form in ("sorted", "gated_gather", "scatter"):
        _check_gmm([5, 0, 40, 300], 136, 72, F16, F16, form, lda=16, spare=37)
        _check_gmm([5, 0, 40, 700], 264, 72, F16, F16, form, lda=16, spare=37)
        _check_gmm([5, 0, 40, 700], 268, 72, BF16, F32, form, lda=8, spare=37)
        _check_gmm([2, 1], 40, 64, BF16, F32, form, lda=8, spare=3)
        _check_gmm([0, 0], 40, 64, BF16, F32, form, spare=3)


@pytest.mark.parametrize("scale, N", [(1, 48), (40, 48), (40, 480)])
def test_grouped_matmul_bad_indexes(scale, N):
    """Offsets outside the rows are clamped, row indexes outside A or out are left out; both are reported and
    every other row is right.  40 x 480: the tensor-core kernel."""
    g = _gen(9)
    n, K = 12 * scale, 64
    a, W = _randn(g, n, K).half(), _randn(g, 3, N, K).half()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(offsets, rows=None, scatter=False):
        out = torch.full((n, N), 7.0, device="cuda")
        st.zero_()
        B.grouped_matmul(a, W, torch.tensor(offsets, dtype=torch.int32, device="cuda"), out, rows=rows, scatter=scatter,
                         status=st)
        return out, B.read_status(st)

    def want(offsets, rows=None, scatter=False):
        out = torch.full((n, N), 7.0, device="cuda")
        o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        return _gmm_ref(a, W, None, o, rows, 1, scatter, out, K)

    for off, clamped in (([0, 4 * scale, 4 * scale, 99 * scale], [0, 4 * scale, 4 * scale, n]),
                         ([-5, 3 * scale, 2 * scale, 2 * scale], [0, 3 * scale, 3 * scale, 3 * scale])):
        out, bits = run(off)
        assert bits == B.ST_BADGROUP
        ref, tol = want(clamped)
        _within(out, ref, tol + _rounding(ref, F32), off)
    rows = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    bad = rows.clone()
    bad[3], bad[7 * scale] = -1, n
    for scatter in (False, True):
        out, bits = run([0, 4 * scale, 9 * scale, n], bad, scatter)
        assert bits == B.ST_BADGROUP
        ref, tol = want([0, 4 * scale, 9 * scale, n], rows, scatter)
        for i in (3, 7 * scale):
            at = int(rows[i]) if scatter else i
            ref[at], tol[at] = 7.0, 0.0
        _within(out, ref, tol + _rounding(ref, F32) * (tol > 0), scatter)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("form", ["few", "many", "gated"])
@pytest.mark.parametrize("K", [760, 776, 4096])
def test_grouped_matmul_sums_of_one_sign(K, form, gather):
    """fp32 results of long sums whose terms have one sign, where an accumulator that cuts toward zero drifts with the
    length.  At most 48 steps of 16 k's go into one such accumulator.  A step aligns 16 products and the partial sum to
    the largest of them, with two bits or more below fp32's 24, cuts them there and cuts their sum to 24 bits: up to
    17 / 4 + 1 = 5.25 units (2^-23) of the partial sum, half of that on average, and the partial sums of equally
    distributed terms are half of the last one on average.  So: 48 x 5.25 = 252 units at most, 48 x 5.25 / 4 = 63 on
    average, and the few of the other additions.  (A single accumulator's average at K = 4096 would be 336.)
    (The first form of this bound counted the cut of the sum alone, 48 and 24 units, and failed with 34 on average.)
    Gated: every gate is 40, whose SiLU is 40 in fp32."""
    g = _gen(K)
    E, N, per = 3, 96 if form == "few" else 640, 6 if form == "few" else 70
    P = E * per
    a = torch.rand((P, K), generator=g, device="cuda").half() + 0.5
    W = (torch.rand((E, N, K), generator=g, device="cuda") + 0.5).half()
    gate = None
    if form == "gated":
        gate = torch.zeros_like(W)
        gate[:, :, 0] = 40.0
        a[:, 0] = 1.0
    rows = torch.randperm(P, generator=g, device="cuda").to(torch.int32) if gather else None
    out = torch.zeros((P, N), device="cuda")
    off = _offsets([per] * E)
    B.grouped_matmul(a, W if gate is None else gate, off, out, W_up=None if gate is None else W, rows=rows)
    x = (a if rows is None else a[rows.long()]).double().view(E, per, K)
    ref = torch.einsum("epk,enk->epn", x, W.double()).reshape(P, N) * (1.0 if gate is None else 40.0)
    err = (out.double() - ref).abs() / ref
    extra = 8 + (K + 767) // 768  # the joins, the gate's SiLU and product
    assert float(err.max()) <= (252 + extra) * U23
    assert float(err.mean()) <= 63 * U23 + 4 * U24


def test_grouped_matmul_non_finite_rows_stay_apart():
    """NaN and infinities in one row of A, or in another expert's rows and matrix, reach no other row."""
    g = _gen(11)
    for sizes, N in (([3, 4, 2], 40), ([150, 90, 200], 40), ([150, 90, 200], 400)):
        P = sum(sizes)
        a, W = _randn(g, P, 72).half(), _randn(g, 3, N, 72).half()
        a[1], a[sizes[0]] = float("nan"), float("inf")
        W[2] = float("nan")
        out = torch.zeros(P, N, device="cuda")
        B.grouped_matmul(a, W, _offsets(sizes), out)
        fin = torch.isfinite(out).all(1).cpu()
        want = torch.ones(P, dtype=torch.bool)
        want[1] = want[sizes[0]] = False
        want[sizes[0] + sizes[1]:] = False
        assert torch.equal(fin, want)


# ---------------------------------------------------------------------------
# as they are used: other streams, graphs, shared workspaces, a block
# ---------------------------------------------------------------------------
def _rel(got, ref):
    """Largest error of a row over the row's largest value."""
    got, ref = got.double(), ref.double()
    return float(((got - ref).abs().amax(-1) / ref.abs().amax(-1).clamp_min(1e-30)).max())


@pytest.mark.parametrize("T", [1, 40, 400])
def test_operators_on_another_stream_and_in_a_graph(T):
    """Each operator on a side stream and in a replayed graph whose inputs change between replays equals its
    plain call bit for bit (no operator's result depends on timing)."""
    g = _gen(T)
    E, K, d, d_ff = 16, 3, 256, 192
    i32 = {"dtype": torch.int32, "device": "cuda"}
    h, y, w = _randn(g, T, d), _randn(g, T, d), 1 + 0.1 * _randn(g, d)
    w_router = _randn(g, T, E)
    blob, _ = _q4_blob(_randn(g, E, d, d_ff), 64)
    wg, wu = _randn(g, E, d_ff, d).half() * 0.1, _randn(g, E, d_ff, d).half() * 0.1
    yg, yu = _randn(g, T, K, d_ff), _randn(g, T, K, d_ff)
    dims = B.ffn_dims(d, d_ff, E, K)
    bufs = {"h_out": torch.empty_like(h), "x": torch.empty(T, d, dtype=F16, device="cuda"),
            "ids": torch.empty(T, K, **i32), "gw": torch.empty(T, K, device="cuda"), "off": torch.empty(E + 1, **i32),
            "order": torch.empty(T * K, **i32), "act": torch.zeros(T * K, d_ff, dtype=F16, device="cuda"),
            "out": torch.empty(T, d, device="cuda")}
    nr, nq = B.topk_route_workspace_bytes(T, E, K), B.ffn_down_q4_workspace_bytes(dims, 64, T)
    ws_r = torch.empty(max(nr, 256), dtype=torch.uint8, device="cuda")
    ws_q = torch.empty(max(nq, 256), dtype=torch.uint8, device="cuda")

    def run():
        B.norm_residual(h, y, w, bufs["x"], h_out=bufs["h_out"])
        B.topk_route(w_router, bufs["ids"], bufs["gw"], bufs["off"], bufs["order"], workspace=ws_r)
        B.grouped_matmul(bufs["x"], wg, bufs["off"], bufs["act"], W_up=wu, rows=bufs["order"], rows_per_a=K, scatter=True)
        B.ffn_down_q4(dims, blob, 64, yg, yu, bufs["ids"], bufs["gw"], T, bufs["out"], ws_q, nq)

    def snap():
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in bufs.items()}
        for v in bufs.values():
            v.zero_()
        torch.cuda.synchronize()
        return got

    run()
    first = snap()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run()
    other = snap()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    graph.replay()
    replay = snap()
    for k, v in first.items():
        assert torch.equal(v, other[k]) and torch.equal(v, replay[k]), k
    keep = [t.clone() for t in (y, w_router, yg)]
    for t in (y, w_router, yg):
        t.copy_(torch.flip(t, [-1]) * 1.5)
    graph.replay()
    changed = snap()
    run()
    plain = snap()
    for k, v in plain.items():
        assert torch.equal(v, changed[k]), k
    assert not torch.equal(changed["x"], first["x"]) and not torch.equal(changed["out"], first["out"])
    for t, v in zip((y, w_router, yg), keep):
        t.copy_(v)
    graph.replay()
    again = snap()
    for k, v in first.items():
        assert torch.equal(v, again[k]), k


def test_concurrent_calls_with_their_own_workspaces():
    """Two streams at once, each with its own buffers: the same results as alone."""
    E, K, d, d_ff = 24, 4, 512, 256
    g = _gen(8)
    blob, _ = _q4_blob(_randn(g, E, d, d_ff), 32)
    W = _randn(g, E, d, d_ff).half()
    dims = B.ffn_dims(d, d_ff, E, K)
    sets = []
    for k in range(2):
        T = 300 + 33 * k
        ids = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :K].to(torch.int32).contiguous()
        logits = _randn(g, T, E)
        i32 = {"dtype": torch.int32, "device": "cuda"}
        n = B.ffn_down_q4_workspace_bytes(dims, 32, T)
        sets.append({"T": T, "logits": logits, "yg": _randn(g, T, K, d_ff), "a": _randn(g, T * K, d_ff).half(),
                     "ids": torch.empty(T, K, **i32), "gw": torch.empty(T, K, device="cuda"), "off": torch.empty(E + 1, **i32),
                     "order": torch.empty(T * K, **i32), "out": torch.empty(T, d, device="cuda"),
                     "y": torch.zeros(T * K, d, device="cuda"), "n": n, "ws": torch.empty(n, dtype=torch.uint8, device="cuda"),
                     "wr": torch.empty(B.topk_route_workspace_bytes(T, E, K), dtype=torch.uint8, device="cuda")})

    def run(s):
        B.topk_route(s["logits"], s["ids"], s["gw"], s["off"], s["order"], workspace=s["wr"])
        B.grouped_matmul(s["a"], W, s["off"], s["y"], rows=s["order"], scatter=True)
        B.ffn_down_q4(dims, blob, 32, s["yg"], None, s["ids"], s["gw"], s["T"], s["out"], s["ws"], s["n"])

    alone = []
    for s in sets:
        run(s)
        torch.cuda.synchronize()
        alone.append({k: s[k].clone() for k in ("ids", "gw", "off", "order", "out", "y")})
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                run(s)
    torch.cuda.synchronize()
    for s, want in zip(sets, alone):
        for k, v in want.items():
            assert torch.equal(s[k], v), k


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [1, 7, 260])
def test_dense_ffn(T, dtype):
    """The routed FFN of dense experts against 64 bits, one expert closed to every token and one token without any.

    h is rounded to the matrices' type once (eps / 2 of itself, which the down product turns into at most eps / 2
    sum|w h|); the rest as for the products themselves."""
    from mixed_precision_decode_b200.layer import DenseMoEFFN, route
    E, K, d, d_ff = 6, 2, 136, 200
    g = _gen(50 + T)
    ffn = DenseMoEFFN((_randn(g, E, d_ff, d) * d ** -0.5).to(dtype), (_randn(g, E, d_ff, d) * d ** -0.5).to(dtype),
                      (_randn(g, E, d, d_ff) * d_ff ** -0.5).to(dtype), K)
    x = _randn(g, T, d).to(dtype)
    logits = _randn(g, T, E)
    logits[:, 4] = float("-inf")
    if T > 1:
        logits[T // 2] = float("-inf")
    r = route(logits, K)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ffn.forward(x, r, status=st)
    assert B.read_status(st) == 0
    ref, tol = torch.zeros(T, d, dtype=torch.float64, device="cuda"), torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(K):
            e, w = int(r.topk_ids[t, j]), float(r.gate_w[t, j])
            assert e != 4
            if e < 0:
                continue
            a, b = ffn.w_gate[e].double(), ffn.w_up[e].double()
            v = x[t].double()
            n = (d // 16 + 24) * U23
            gate, up = a @ v, b @ v
            eg, eu = n * (a.abs() @ v.abs()), n * (b.abs() @ v.abs())
            h = gate * torch.sigmoid(gate) * up
            eh = 1.1 * eg * up.abs() + (gate * torch.sigmoid(gate)).abs() * eu + h.abs() * (16 * U24)
            eh = eh + _rounding(h, dtype)
            wd = ffn.w_down[e].double()
            ref[t] += w * (wd @ h)
            tol[t] += abs(w) * (wd.abs() @ eh + (d_ff // 16 + 24) * U23 * (wd.abs() @ h.abs()))
    _within(out, ref, tol * 1.01 + 4 * U24 * ref.abs() + 1e-30, "dense ffn")
    if T > 1:
        assert bool((out[T // 2] == 0).all())


@pytest.mark.parametrize("T", [1, 12])
@pytest.mark.parametrize("kind", ["spectral", "spectral_q4", "dense"])
def test_moe_block_stack(kind, T):
    """Three blocks as a decoder runs them -- norm, router, routed FFN, the residual added by the next block's norm --
    against the same steps from the operators' plain forms on the routing that the block chose: every output of the
    chain within the outputs' 2e-3 bound, every choice of experts one that the logits allow."""
    from cases import SMALL, get_case
    from mixed_precision_decode_b200 import synth
    from mixed_precision_decode_b200.layer import DenseMoEFFN, MoEBlock, Q4Down, SpectralMoEFFN, route
    case = get_case("tiny")
    cfg = SMALL["tiny"]
    E, K, d = cfg.n_experts, cfg.top_k, cfg.d_in
    g = _gen(60 + T)
    h = _randn(g, T, d)
    blocks, downs = [], []
    for b in range(3):
        wd = synth.make_down(cfg, synth.make_generator(70 + b, torch.device("cuda")), torch.device("cuda"))
        if kind == "dense":
            wg, wu = ((_randn(g, E, cfg.d_out, d) * d ** -0.5).half() for _ in range(2))
            ffn = DenseMoEFFN(wg, wu, wd, K)
        else:
            ffn = SpectralMoEFFN(case.layer, Q4Down.pack(wd, 32) if kind == "spectral_q4" else wd)
        w_down = ffn.q4.unpack().double() if kind == "spectral_q4" else wd.double()
        downs.append(w_down)
        blocks.append(MoEBlock(ffn, 1 + 0.1 * _randn(g, d), _randn(g, E, d).half(), w_post=1 + 0.1 * _randn(g, d), alpha=0.5))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, hr, yr = None, h.double(), None
    for blk, w_down in zip(blocks, downs):
        y_in = y
        y = blk.forward(h, y, status=st)
        # the plain steps, from the block's own h (its roundings are bounded by the operators' tests)
        if y_in is not None:
            u = y_in.double()
            hr = hr + 0.5 * u / torch.sqrt(u.square().mean(1, keepdim=True) + 1e-6) * blk.w_post.double()
        assert _rel(h, hr) <= 1e-5
        hr = h.double()
        x = (hr / torch.sqrt(hr.square().mean(1, keepdim=True) + 1e-6) * blk.w_norm.double()).half()
        logits = torch.empty(T, E, device="cuda")
        B.shared_proj(blk.w_router, x, logits, T, d, E)
        r = route(logits, K)
        if kind == "dense":
            a = x.double()
            want = torch.zeros(T, d, dtype=torch.float64, device="cuda")
            for t in range(T):
                for j in range(K):
                    e = int(r.topk_ids[t, j])
                    gate, up = blk.ffn.w_gate[e].double() @ a[t], blk.ffn.w_up[e].double() @ a[t]
                    want[t] += float(r.gate_w[t, j]) * (w_down[e] @ (gate * torch.sigmoid(gate) * up))
        else:
            o = case.layer.forward(x, r.topk_ids, r.gate_w, want_experts=True)
            gate, up = o["Y_experts_gate"].double(), o["Y_experts_up"].double()
            hh = gate * torch.sigmoid(gate) * up
            want = torch.einsum("tk,tkdf,tkf->td", r.gate_w.double(), w_down[r.topk_ids.long()], hh)
        assert _rel(y, want) <= 4e-3  # x may round the other way in the last bit of fp16, 2e-3 on either side
    blocks[-1].finish(h, y)
    assert bool(torch.isfinite(h).all()) and B.read_status(st) == 0


def test_empty_batch():
    from mixed_precision_decode_b200.layer import DenseMoEFFN, MoEBlock
    g = _gen(3)
    E, K, d, d_ff = 4, 2, 64, 32
    ffn = DenseMoEFFN(_randn(g, E, d_ff, d).half(), _randn(g, E, d_ff, d).half(), _randn(g, E, d, d_ff).half(), K)
    blk = MoEBlock(ffn, _randn(g, d), _randn(g, E, d).half())
    h = _randn(g, 0, d)
    y = blk.forward(h)
    assert y.shape == (0, d) and blk.finish(h, y).shape == (0, d)


def test_moe_block_on_a_given_stream():
    """stream=, as a torch stream and as a raw handle, while the current stream allocates and overwrites memory: a
    tensor that a call keeps for itself must not be handed to the current stream while the kernels run."""
    from mixed_precision_decode_b200.layer import DenseMoEFFN, MoEBlock
    g = _gen(77)
    E, K, d, d_ff, T = 8, 2, 512, 768, 300
    ffn = DenseMoEFFN((_randn(g, E, d_ff, d) * d ** -0.5).half(), (_randn(g, E, d_ff, d) * d ** -0.5).half(),
                      (_randn(g, E, d, d_ff) * d_ff ** -0.5).half(), K)
    blocks = [MoEBlock(ffn, 1 + 0.1 * _randn(g, d), _randn(g, E, d).half()) for _ in range(4)]
    h0 = _randn(g, T, d)

    def run(stream, noise):
        h, y = h0.clone(), None
        torch.cuda.synchronize()
        for blk in blocks:
            y = blk.forward(h, y, stream=stream)
            if noise:
                for n in (T * d, 4 * T * K, T * E, B.dense_ffn_workspace_bytes(ffn.dims, T) // 4):
                    for _ in range(4):
                        torch.full((n,), float("nan"), device="cuda")
        blocks[-1].finish(h, y, stream=stream)
        torch.cuda.synchronize()
        return h

    want = run(None, False)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        assert torch.equal(run(stream, True), want)


def test_two_graphs_share_workspaces():
    """Two captured graphs of different batches on the same workspaces, replayed in turn: no call leaves anything in a
    workspace that the next one reads."""
    E, K, d, d_ff = 20, 3, 384, 256
    g = _gen(31)
    blob, _ = _q4_blob(_randn(g, E, d, d_ff), 64)
    wg, wu, wd = _randn(g, E, d_ff, d).half() * 0.1, _randn(g, E, d_ff, d).half() * 0.1, _randn(g, E, d, d_ff).half() * 0.1
    dims = B.ffn_dims(d, d_ff, E, K)
    Ts = (150, 37)
    n = max(max(B.topk_route_workspace_bytes(T, E, K), B.ffn_down_q4_workspace_bytes(dims, 64, T),
                B.dense_ffn_workspace_bytes(dims, T)) for T in Ts)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")  # one for all three operators
    sets = []
    for T in Ts:
        i32 = {"dtype": torch.int32, "device": "cuda"}
        s = {"logits": _randn(g, T, E), "yg": _randn(g, T, K, d_ff), "yu": _randn(g, T, K, d_ff), "x": _randn(g, T, d).half(),
             "ids": torch.empty(T, K, **i32), "gw": torch.empty(T, K, device="cuda"), "off": torch.empty(E + 1, **i32),
             "order": torch.empty(T * K, **i32), "q4": torch.empty(T, d, device="cuda"),
             "dense": torch.empty(T, d, device="cuda")}

        def run(s=s, T=T):
            B.topk_route(s["logits"], s["ids"], s["gw"], s["off"], s["order"], workspace=ws)
            B.ffn_down_q4(dims, blob, 64, s["yg"], s["yu"], s["ids"], s["gw"], T, s["q4"], ws, n)
            B.dense_ffn_forward(dims, wg, wu, wd, s["x"], s["ids"], s["gw"], s["off"], s["order"], s["dense"], ws)

        run()
        torch.cuda.synchronize()
        s["want"] = {k: s[k].clone() for k in ("ids", "gw", "off", "order", "q4", "dense")}
        s["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(s["graph"]):
            run()
        sets.append(s)
    for k in (0, 1, 0, 0, 1):
        for key in ("q4", "dense", "ids"):
            sets[k][key].zero_()
        sets[k]["graph"].replay()
        torch.cuda.synchronize()
        for key, want in sets[k]["want"].items():
            assert torch.equal(sets[k][key], want), key


def test_routing_right_before_the_single_token_step():
    """The single-token 4-bit step looks at the ids before the routing that writes them has ended: what it computes goes
    by the ids written, in a chain of 40 routings and steps whose choices all differ."""
    E, K, d, d_ff, n = 64, 4, 256, 128, 40
    g = _gen(91)
    blob, _ = _q4_blob(_randn(g, E, d, d_ff), 64)
    dims = B.ffn_dims(d, d_ff, E, K)
    yg = _randn(g, 1, K, d_ff)
    logits = _randn(g, n, E)
    ids, gw = torch.empty(1, K, dtype=torch.int32, device="cuda"), torch.empty(1, K, device="cuda")
    out, want = torch.empty(n, 1, d, device="cuda"), torch.empty(n, 1, d, device="cuda")

    def chain():
        for i in range(n):
            B.topk_route(logits[i:i + 1], ids, gw)
            B.ffn_down_q4(dims, blob, 64, yg, None, ids, gw, 1, out[i], None, 0)

    for i in range(n):
        B.topk_route(logits[i:i + 1], ids, gw)
        torch.cuda.synchronize()
        B.ffn_down_q4(dims, blob, 64, yg, None, ids, gw, 1, want[i], None, 0)
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    chain()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    with torch.cuda.graph(graph):
        chain()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
