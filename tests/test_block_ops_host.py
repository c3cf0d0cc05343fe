"""The block operators' argument checks on the host (no GPU): the C calls refuse bad
dimensions, types, alignments and sizes before any launch, and the binding refuses
tensors of another shape, type or device."""
import os
import re
import struct
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    from mixed_precision_decode_b200 import build
    build.build()
    from mixed_precision_decode_b200 import bitsmoe
    return bitsmoe


def _call(f, fmt, args):
    return f(struct.pack(fmt, *[0 if v is None else v for v in args.values()]), None)


NORM = dict(h=256, y=512, w_post=None, gate=None, h_out=256, w_pre=1024, x=2048, h_stride=16, y_stride=16, gate_stride=0,
            ho_stride=16, x_stride=16, rows=2, d=16, h_type=0, y_type=0, x_type=1, per_channel=0, alpha=1.0, eps=1e-6)


def _norm(B, **kw):
    return _call(B.lib().bitsmoe_norm_residual, "@7P5q6i2f", {**NORM, **kw})


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(d=0), dict(h_type=3), dict(y_type=-1), dict(x_type=7), dict(h=None), dict(h_out=None, x=None),
    dict(w_pre=None), dict(y=None, w_post=1024), dict(y=None, gate=1024), dict(h_stride=-1), dict(gate_stride=-1),
    dict(x_stride=8), dict(ho_stride=15), dict(h=258), dict(y=514), dict(x=2049), dict(w_pre=1026), dict(eps=-1.0),
    dict(eps=float("nan")), dict(ho_stride=32),
])
def test_norm_residual_refusals(B, bad):
    assert _norm(B, **bad) == B.EINVAL


def test_norm_residual_empty(B):
    assert _norm(B, rows=0, h=None) == B.OK
    assert B.lib().bitsmoe_norm_residual(None, None) == B.EINVAL


ROUTE = dict(logits=256, ids=512, gw=1024, offsets=None, order=None, ws=None, status=None, ws_bytes=0, stride=8, tokens=3,
             E=8, K=2, type=0, scoring=0, renorm=1, scale=1.0, reserved=0)


def _route(B, **kw):
    return _call(B.lib().bitsmoe_topk_route, "@7PQq6ifi", {**ROUTE, **kw})


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(E=0), dict(E=8193), dict(K=0), dict(K=9), dict(type=5), dict(scoring=2), dict(logits=None),
    dict(ids=None), dict(gw=None), dict(stride=-8), dict(logits=258), dict(ids=514), dict(offsets=3), dict(order=2),
    dict(E=2000, K=1025, stride=2000), dict(tokens=2 ** 30, K=8), dict(reserved=1),
    dict(tokens=4096, offsets=2048),  # the two-launch path without a workspace
    dict(tokens=4096, order=2048, ws=1000, ws_bytes=1 << 20),  # misaligned workspace
])
def test_topk_route_refusals(B, bad):
    assert _route(B, **bad) == B.EINVAL


def test_topk_route_workspace(B):
    assert B.topk_route_workspace_bytes(1, 128, 8) == 0 and B.topk_route_workspace_bytes(0, 128, 8) == 0
    n = B.topk_route_workspace_bytes(4096, 128, 8)
    assert n > 0 and n % (4 * 128) == 0
    assert _route(B, tokens=4096, E=128, stride=128, order=2048, ws=512, ws_bytes=n - 1) == B.ESIZE
    assert _route(B, tokens=0, logits=None) == B.OK
    assert B.lib().bitsmoe_topk_route(None, None) == B.EINVAL


def test_q4_sizes_and_refusals(B):
    L = B.lib()
    # one block of 16 rows: 8 bytes a padded column, 32 a group
    assert B.q4_bytes(1, 1, 1, 32) == 64 * 8 + 2 * 32
    assert B.q4_bytes(3, 17, 65, 128) == 3 * 2 * (128 * 8 + 32)
    assert B.q4_bytes(128, 2048, 768, 64) == 128 * 128 * (768 * 8 + 12 * 32)
    for bad in ((0, 1, 1, 32), (1, 0, 1, 32), (1, 1, 0, 32), (1, 1, 1, 16), (1, 1, 1, 0)):
        assert B.q4_bytes(*bad) == 0
    assert L.bitsmoe_q4_pack(256, 0, 1, 4, 8, 48, 512, None, None) == B.EINVAL
    assert L.bitsmoe_q4_pack(256, 4, 1, 4, 8, 64, 512, None, None) == B.EINVAL
    assert L.bitsmoe_q4_pack(None, 0, 1, 4, 8, 64, 512, None, None) == B.EINVAL
    assert L.bitsmoe_q4_pack(258, 0, 1, 4, 8, 64, 512, None, None) == B.EINVAL
    assert L.bitsmoe_q4_pack(256, 0, 1, 4, 8, 64, 520, None, None) == B.EINVAL
    assert L.bitsmoe_q4_unpack(256, 1, 4, 8, 64, None, None) == B.EINVAL
    assert L.bitsmoe_q4_unpack(264, 1, 4, 8, 64, 512, None) == B.EINVAL


def test_ffn_down_q4_refusals(B):
    d = B.ffn_dims(2048, 768, 128, 8)
    n = B.ffn_down_q4_workspace_bytes(d, 64, 64)
    assert n >= 64 * 8 * (2048 + 768) * 4
    ok = dict(d_model=2048, d_ff=768, E=128, K=8, group=64, tokens=64, blob=256, yg=256, yu=256, ids=256, gw=256, out=256,
              ws=512, st=None, nb=n)

    def call(**kw):
        return _call(B.lib().bitsmoe_ffn_down_q4, "@6i8PQ", {**ok, **kw})

    for bad in (dict(group=16), dict(tokens=-1), dict(blob=None), dict(yg=None), dict(ids=None), dict(gw=None),
                dict(out=None), dict(blob=264), dict(yg=260), dict(yu=260), dict(ws=None), dict(ws=520), dict(d_ff=12),
                dict(d_model=0), dict(E=0), dict(E=4097 * 4), dict(K=0), dict(tokens=1 << 28)):
        assert call(**bad) == B.EINVAL, bad
    assert call(nb=n - 1) == B.ESIZE
    assert call(tokens=0, blob=None) == B.OK
    assert B.lib().bitsmoe_ffn_down_q4(None, None) == B.EINVAL
    assert B.ffn_down_q4_launches(d, 64, 0) == 0 and B.ffn_down_q4_launches(d, 64, 64) >= 1
    with pytest.raises(B.BitsMoEError):
        B.ffn_down_q4_launches(d, 60, 1)


def test_grouped_matmul_refusals(B):
    ok = dict(A=256, W=512, W_up=None, offsets=1024, rows=None, out=2048, st=None, lda=16, n_rows=4, n_a_rows=4, n_out=8,
              n_in=16, n_experts=2, in_type=1, out_type=1, per=1, scatter=0, reserved=0)

    def call(**kw):
        return _call(B.lib().bitsmoe_grouped_matmul, "@7Pq10i", {**ok, **kw})

    for bad in (dict(n_rows=-1), dict(n_a_rows=-1), dict(n_out=0), dict(n_in=12), dict(n_in=0), dict(n_experts=0),
                dict(n_experts=4097), dict(in_type=0), dict(out_type=2), dict(n_a_rows=3),
                dict(n_experts=4096, n_out=1 << 20), dict(A=None), dict(W=None), dict(offsets=None), dict(out=None),
                dict(A=264), dict(W=520), dict(W_up=8), dict(lda=8), dict(lda=20), dict(scatter=1), dict(per=2), dict(per=0),
                dict(offsets=1026), dict(rows=3), dict(out=2049), dict(reserved=1)):
        assert call(**bad) == B.EINVAL, bad
    assert call(n_rows=0, A=None) == B.OK
    assert B.lib().bitsmoe_grouped_matmul(None, None) == B.EINVAL


def test_dense_ffn_refusals(B):
    d = B.ffn_dims(64, 32, 4, 2)
    n = B.dense_ffn_workspace_bytes(d, 3)
    assert n >= 3 * 2 * (32 * 2 + 64 * 4) and B.dense_ffn_workspace_bytes(d, 0) == 0
    assert B.dense_ffn_workspace_bytes(B.ffn_dims(60, 32, 4, 2), 3) == 0
    ok = dict(d_model=64, d_ff=32, E=4, K=2, tokens=3, type=1, x=256, wg=256, wu=256, wd=256, ids=256, gw=256, off=256, od=256,
              out=256, ws=512, st=None, nb=n, xs=64)

    def call(**kw):
        return _call(B.lib().bitsmoe_dense_ffn_forward, "@6i11PQq", {**ok, **kw})

    for bad in (dict(d_model=60), dict(d_ff=4), dict(E=0), dict(E=4097), dict(K=0), dict(tokens=-1), dict(type=0), dict(x=None),
                dict(wg=None), dict(wu=None), dict(wd=None), dict(ids=None), dict(gw=None), dict(off=None), dict(od=None),
                dict(out=None), dict(ws=None), dict(ws=520), dict(xs=56), dict(x=264)):
        assert call(**bad) == B.EINVAL, bad
    assert call(nb=n - 1) == B.ESIZE and call(tokens=0, x=None) == B.OK
    assert B.lib().bitsmoe_dense_ffn_forward(None, None) == B.EINVAL


def test_packed_structures_match_the_header(tmp_path, B):
    """The binding's packed layouts have the sizes and field offsets of the header's structures."""
    fields = {
        "bitsmoe_norm_args": (B._NORM, ["h", "y", "w_post", "gate", "h_out", "w_pre", "x", "h_stride", "y_stride",
                                        "gate_stride", "h_out_stride", "x_stride", "rows", "d", "h_type", "y_type", "x_type",
                                        "gate_per_channel", "alpha", "eps"]),
        "bitsmoe_route_args": (B._ROUTE, ["logits", "topk_ids", "gate_w", "offsets", "order", "workspace", "status",
                                          "workspace_bytes", "logits_stride", "tokens", "n_experts", "top_k", "logits_type",
                                          "scoring", "renormalise", "scale", "reserved"]),
        "bitsmoe_q4_args": (B._Q4, ["dims.d_model", "dims.d_ff", "dims.n_experts", "dims.top_k", "group", "tokens", "blob",
                                    "Y_gate", "Y_up", "topk_ids", "gate_w", "out", "workspace", "status",
                                    "workspace_bytes"]),
        "bitsmoe_dense_ffn_args": (B._DENSE, ["dims.d_model", "dims.d_ff", "dims.n_experts", "dims.top_k", "tokens", "type",
                                              "x", "W_gate", "W_up", "W_down", "topk_ids", "gate_w", "offsets", "order",
                                              "out", "workspace", "status", "workspace_bytes", "x_stride"]),
        "bitsmoe_gmm_args": (B._GMM, ["A", "W", "W_up", "offsets", "rows", "out", "status", "a_stride", "n_rows", "n_a_rows",
                                      "n_out", "n_in", "n_experts", "in_type", "out_type", "rows_per_a", "scatter",
                                      "reserved"]),
    }
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "bitsmoe.h"\nint main(void) {\n'
    for name, (_, fs) in fields.items():
        src += f'printf("%zu", sizeof({name}));\n'
        src += "".join(f'printf(" %zu", offsetof({name}, {f}));\n' for f in fs) + 'printf("\\n");\n'
    c = tmp_path / "layout.c"
    c.write_text(src + "return 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(tmp_path / "layout")], check=True)
    lines = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.splitlines()
    for (name, (st, fs)), line in zip(fields.items(), lines):
        size, *offs = map(int, line.split())
        assert st.size == size, name
        codes = "".join(ch * int(n or 1) for n, ch in re.findall(r"(\d*)([a-zA-Z])", st.format))
        assert len(codes) == len(fs)
        got = [struct.calcsize("@" + codes[:i] + "0" + codes[i]) for i in range(len(codes))]
        assert got == offs, name


def _refused(B, f, *a, **kw):
    with pytest.raises(B.BitsMoEError) as ei:
        f(*a, **kw)
    return ei.value.code


def test_binding_refuses_other_tensors(B):
    """Shapes, types and devices are looked at before the library is called."""
    z = torch.zeros
    h = z(4, 16)
    w = z(16)
    for kw in (dict(y=z(4, 8)), dict(y=z(4, 16, dtype=torch.float64)), dict(h_out=z(4, 16, dtype=torch.float16)),
               dict(x=z(4, 16)), dict(x=z(4, 16), w_pre=z(8)), dict(x=z(4, 16), w_pre=w.half()),
               dict(y=z(4, 16), gate=z(4)), dict(y=z(4, 16), gate=z(3, 1)), dict(y=z(4, 16), gate=z(4, 1).half()),
               dict(y=z(16, 4).T), dict(x=z(4, 16), w_pre=w)):  # the last one: not on a GPU
        assert _refused(B, B.norm_residual, h, **kw) == B.EINVAL, kw
    i = z(4, 2, dtype=torch.int32)
    g = z(4, 2)
    for a, kw in (((h, i, z(4, 3)), {}), ((h, i.long(), g), {}), ((h.double(), i, g), {}),
                  ((h, i, g), dict(scoring="relu")), ((h, i, g, z(16, dtype=torch.int32)), {}), ((h, i, g), {}),
                  ((h, i, g), dict(order=z(9, dtype=torch.int32))), ((h[0], i, g), {})):
        assert _refused(B, B.topk_route, *a, **kw) == B.EINVAL
    a, W, off = z(4, 16).half(), z(2, 8, 16).half(), z(3, dtype=torch.int32)
    out = z(4, 8).half()
    for x, kw in (((a, W.bfloat16(), off, out), {}), ((a, W, off[:2], out), {}), ((a, W, off, z(4, 7).half()), {}),
                  ((a, W, off, out), dict(W_up=z(2, 8, 8).half())), ((a, W, off, out), dict(rows=z(3, dtype=torch.int32))),
                  ((a.double(), W, off, out), {}), ((a, W, off, out), {}), ((z(4, 8).half(), W, off, out), {})):
        assert _refused(B, B.grouped_matmul, *x, **kw) == B.EINVAL
    blob = z(B.q4_bytes(2, 8, 16, 32), dtype=torch.uint8)
    assert _refused(B, B.q4_pack, z(2, 8, 16), 48, blob) == B.EINVAL
    assert _refused(B, B.q4_pack, z(2, 8, 16), 32, blob[:-1]) == B.ESIZE
    assert _refused(B, B.q4_pack, z(2, 8, 16), 32, blob) == B.EINVAL  # not on a GPU
    assert _refused(B, B.q4_unpack, blob[:-1], 32, z(2, 8, 16)) == B.ESIZE
    d = B.ffn_dims(8, 16, 2, 2)
    y = z(4, 2, 16)
    assert _refused(B, B.ffn_down_q4, d, blob, 32, y, z(4, 2, 8), i, g, 4, z(4, 8)) == B.EINVAL
    assert _refused(B, B.ffn_down_q4, d, blob[:-1], 32, y, y, i, g, 4, z(4, 8)) == B.ESIZE
    assert _refused(B, B.ffn_down_q4, d, blob, 32, y, y, i, g, 4, z(4, 8)) == B.EINVAL
