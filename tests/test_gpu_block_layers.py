"""The layer objects around the routed experts as a stack uses them, on the GPU: whose parameters add an output, streams
and workspaces, and the calls next to one another.  Tolerances count roundings, as in test_gpu_block_ops.py."""
import pytest
import torch

from mixed_precision_decode_b200 import bitsmoe as B

pytestmark = pytest.mark.gpu

U24 = 2.0 ** -24


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _dense(g, E, K, d, d_ff):
    from mixed_precision_decode_b200.layer import DenseMoEFFN
    return DenseMoEFFN((_randn(g, E, d_ff, d) * d ** -0.5).half(), (_randn(g, E, d_ff, d) * d ** -0.5).half(),
                       (_randn(g, E, d, d_ff) * d_ff ** -0.5).half(), K)


def _spectral(kind, seed):
    """A SpectralMoEFFN of the small test layer, with fp16 or 4-bit down matrices."""
    from cases import SMALL, get_case
    from mixed_precision_decode_b200 import synth
    from mixed_precision_decode_b200.layer import Q4Down, SpectralMoEFFN
    cfg = SMALL["tiny"]
    wd = synth.make_down(cfg, synth.make_generator(seed, torch.device("cuda")), torch.device("cuda"))
    return SpectralMoEFFN(get_case("tiny").layer, Q4Down.pack(wd, 32) if kind == "q4" else wd)


@pytest.mark.parametrize("T", [1, 9, 140])
@pytest.mark.parametrize("kind", ["dense", "fp16", "q4"])
def test_stack_adds_each_output_with_its_makers_parameters(kind, T):
    """Every block has its own w_post and alpha, two have no w_post: h after each forward and after finish is the h
    before it plus alpha gate rmsnorm(y) w_post of the block that made y.  A row's sum of squares is taken in at most 60
    sequential additions: its inverse root is off by 32 units of 2^-24, the factors by one each."""
    from mixed_precision_decode_b200.layer import MoEBlock
    g = _gen(T + len(kind))
    ffns = [_dense(g, 6, 2, 136, 200) if kind == "dense" else _spectral(kind, 40 + b) for b in range(4)]
    d, E = ffns[0].dims.d_model, ffns[0].dims.n_experts
    blocks = [MoEBlock(f, 1 + 0.1 * _randn(g, d), _randn(g, E, d).half(), w_post=1 + 0.3 * _randn(g, d) if b % 3 else None,
                       alpha=0.5 + 0.25 * b) for b, f in enumerate(ffns)]
    gates = [torch.sigmoid(_randn(g, T, 1)) for _ in blocks]
    h = _randn(g, T, d)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def check(before, y, made_by, gate):
        u = y.double()
        if made_by.w_post is not None:
            u = u / torch.sqrt(u.square().mean(1, keepdim=True) + made_by.eps) * made_by.w_post.double()
        u = made_by.alpha * gate.double() * u
        tol = 64 * U24 * (before.abs() + u.abs()) + 2.0 ** -149
        assert bool(((h.double() - before - u).abs() <= tol).all())

    y = before = gate = None
    for b, own in zip(blocks, gates):
        h0, y0 = h.double(), y
        y = b.forward(h, y, gate=gate, status=st, made_by=before)
        if y0 is not None:
            check(h0, y0, before, gate)
        before, gate = b, own
    h0 = h.double()
    assert blocks[-1].finish(h, y, gate=gate) is h
    check(h0, y, blocks[-1], gate)
    assert B.read_status(st) == 0


@pytest.mark.parametrize("T", [1, 9, 140])
@pytest.mark.parametrize("kind", ["fp16", "q4", "layer"])
def test_spectral_calls_on_a_given_stream(kind, T):
    """stream=, as a torch stream and as a raw handle, on a new object each time (its first call makes the workspace),
    while the current stream allocates and overwrites memory: the results are those of the current stream's calls.  One
    token's partial rows are added by atomics, in any order: there within the outputs' 2e-3 bound."""
    from cases import get_case
    from mixed_precision_decode_b200.layer import SpectralMoELayer
    g = _gen(5 * T)
    ffn = _spectral("q4" if kind == "q4" else "fp16", 91)
    d, E, K = ffn.dims.d_model, ffn.dims.n_experts, ffn.dims.top_k
    x, gw = _randn(g, T, d).half(), torch.rand((T, K), generator=g, device="cuda")
    ids = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :K].to(torch.int32).contiguous()
    layer = get_case("tiny").layer

    def run(stream, noise):
        new = SpectralMoELayer(layer.gate, layer.up)
        if kind != "layer":
            new = type(ffn)(new, ffn.q4 or ffn.w_down)
        torch.cuda.synchronize()
        sizes = (T * d, 2 * T * d, T * K * ffn.dims.d_ff, new.workspace(T).numel() // 4)
        new._ws.one = None
        torch.cuda.synchronize()
        got = []
        for _ in range(4):
            got.append(new.forward(x, ids, gw, stream=stream))
            if noise:
                for n in sizes:
                    for _ in range(4):
                        torch.full((max(n, 64),), float("nan"), device="cuda")
        torch.cuda.synchronize()
        return torch.stack([y if kind != "layer" else torch.cat((y["Y_sum_gate"], y["Y_sum_up"]), 1) for y in got])

    want = run(None, False)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = run(stream, True)
        if T > 1:
            assert torch.equal(got, want)
        else:
            assert bool(((got - want).abs() <= 2e-3 * want.abs().amax(-1, keepdim=True)).all())


@pytest.mark.parametrize("kind", ["fp16", "q4"])
def test_single_token_step_right_behind_its_routing(kind):
    """The single-token steps look at the ids before the routing that writes them has ended: what they compute goes by
    the ids written, in a chain of 40 routings and steps whose choices all differ, run at once and as a replayed graph."""
    E, K, d, d_ff, n = 64, 4, 256, 128, 40
    g = _gen(92)
    w = _randn(g, E, d, d_ff).half()
    dims = B.ffn_dims(d, d_ff, E, K)
    blob = torch.empty(B.q4_bytes(E, d, d_ff, 64), dtype=torch.uint8, device="cuda")
    B.q4_pack(w, 64, blob)
    yg, yu = _randn(g, 1, K, d_ff), _randn(g, 1, K, d_ff)
    logits = _randn(g, n, E)
    ids, gw = torch.empty(1, K, dtype=torch.int32, device="cuda"), torch.empty(1, K, device="cuda")
    out, want = torch.empty(n, 1, d, device="cuda"), torch.empty(n, 1, d, device="cuda")
    assert B.ffn_down_workspace_bytes(dims, 1) == 0 and B.ffn_down_q4_workspace_bytes(dims, 64, 1) == 0

    def step(to):
        if kind == "fp16":
            B.ffn_down(dims, w, yg, yu, ids, gw, 1, to)
        else:
            B.ffn_down_q4(dims, blob, 64, yg, yu, ids, gw, 1, to)

    def chain():
        for i in range(n):
            B.topk_route(logits[i:i + 1], ids, gw)
            step(out[i])

    for i in range(n):
        B.topk_route(logits[i:i + 1], ids, gw)
        torch.cuda.synchronize()
        step(want[i])
        torch.cuda.synchronize()
    chain()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("T", [2, 33, 150])
@pytest.mark.parametrize("kind", ["fp16", "q4", "layer"])
def test_overlapping_calls_of_one_object(kind, T):
    """Two streams call one object at the same T, again and again, with other inputs: each gets what it gets alone."""
    ffn = _spectral("q4" if kind == "q4" else "fp16", 92)
    obj = ffn.layer if kind == "layer" else ffn
    d, E, K = ffn.dims.d_model, ffn.dims.n_experts, ffn.dims.top_k
    sets = []
    for i in range(2):
        g = _gen(7 * T + i)
        x, gw = _randn(g, T, d).half(), torch.rand((T, K), generator=g, device="cuda")
        ids = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :K].to(torch.int32).contiguous()
        sets.append((x, ids, gw))
    leaf = (lambda y: y["Y_sum_gate"]) if kind == "layer" else (lambda y: y)
    want = [leaf(obj.forward(*s)).clone() for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(sets):
            got[i].append(leaf(obj.forward(*s, stream=streams[i])))
    torch.cuda.synchronize()
    for w, ys in zip(want, got):
        for y in ys:
            assert torch.equal(y, w)


@pytest.mark.parametrize("T", [1, 9])
@pytest.mark.parametrize("kind", ["dense", "fp16", "q4"])
def test_stack_captured_before_its_first_call(kind, T):
    """A stack of new blocks captured into a graph and replayed, an eager pass before its first replay and another after:
    all of them give the same residual stream (one token over the spectral layer: within the outputs' 2e-3 bound, the
    order of its atomics being open)."""
    from mixed_precision_decode_b200.layer import MoEBlock, SpectralMoEFFN, SpectralMoELayer
    g = _gen(3 * T + len(kind))
    ffns = [_dense(g, 6, 2, 136, 200) if kind == "dense" else _spectral(kind, 60 + b) for b in range(3)]
    if kind != "dense":
        ffns = [SpectralMoEFFN(SpectralMoELayer(f.layer.gate, f.layer.up), f.q4 or f.w_down) for f in ffns]
    d, E = ffns[0].dims.d_model, ffns[0].dims.n_experts
    blocks = [MoEBlock(f, 1 + 0.1 * _randn(g, d), _randn(g, E, d).half(), w_post=1 + 0.1 * _randn(g, d), alpha=0.5)
              for f in ffns]
    h0 = _randn(g, T, d)
    h = h0.clone()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run():
        h.copy_(h0)
        y = before = None
        for b in blocks:
            y = b.forward(h, y, status=st, made_by=before)
            before = b
        blocks[-1].finish(h, y)

    torch.empty(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run()
    got = []
    for step in (run, graph.replay, graph.replay, run, graph.replay):
        h.zero_()
        step()
        torch.cuda.synchronize()
        got.append(h.clone())
    assert B.read_status(st) == 0 and bool(torch.isfinite(got[0]).all())
    for other in got[1:]:
        if T > 1 or kind == "dense":
            assert torch.equal(other, got[0])
        else:
            assert float((other - got[0]).abs().max() / got[0].abs().max()) <= 2e-3


@pytest.mark.parametrize("kind", ["dense", "fp16", "q4"])
def test_empty_batches(kind):
    from mixed_precision_decode_b200.layer import MoEBlock
    g = _gen(4)
    ffn = _dense(g, 6, 2, 136, 200) if kind == "dense" else _spectral(kind, 66)
    d, E = ffn.dims.d_model, ffn.dims.n_experts
    blk = MoEBlock(ffn, _randn(g, d), _randn(g, E, d).half())
    h = _randn(g, 0, d)
    y = blk.forward(h)
    assert y.shape == (0, d) and blk.finish(h, blk.forward(h, y, made_by=blk)).shape == (0, d)
