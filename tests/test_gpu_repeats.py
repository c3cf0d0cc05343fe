"""The block operators repeat themselves bit for bit, whatever ran between: no result depends on timing, on what a
workspace holds or on a call before."""
import pytest
import torch

from mixed_precision_decode_b200 import bitsmoe as B

pytestmark = pytest.mark.gpu


def _inputs(seed, T, E, K, d, d_ff, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    i32 = {"dtype": torch.int32, "device": "cuda"}
    s = {"logits": r(T, E).to(dtype), "ids": torch.empty(T, K, **i32), "gw": torch.empty(T, K, device="cuda"),
         "off": torch.empty(E + 1, **i32), "order": torch.empty(T * K, **i32), "h": r(T, d).to(dtype), "y": r(T, d),
         "x": torch.empty(T, d, dtype=dtype, device="cuda"), "h_out": torch.empty(T, d, dtype=dtype, device="cuda"),
         "w": 1 + 0.1 * r(d), "gate": r(T, 1), "yg": r(T, K, d_ff), "yu": r(T, K, d_ff),
         "q4": torch.empty(T, d, device="cuda"), "hh": torch.empty(T * K, d_ff, dtype=dtype, device="cuda"),
         "down": torch.empty(T * K, d, device="cuda"), "dense": torch.empty(T, d, device="cuda")}
    return s


OUT = ("ids", "gw", "off", "order", "x", "h_out", "q4", "hh", "down", "dense")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T, E, K, d, d_ff", [(1, 16, 4, 256, 128), (40, 16, 4, 256, 128), (700, 8, 2, 1024, 384),
                                              (300, 32, 8, 520, 1032)])
def test_operators_repeat_themselves(T, E, K, d, d_ff, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    wg, wu, wd = (r(E, d_ff, d) * d ** -0.5).to(dtype), (r(E, d_ff, d) * d ** -0.5).to(dtype), (r(E, d, d_ff) * 0.05).to(dtype)
    blob = torch.empty(B.q4_bytes(E, d, d_ff, 64), dtype=torch.uint8, device="cuda")
    B.q4_pack(wd, 64, blob)
    dims = B.ffn_dims(d, d_ff, E, K)
    n = max(B.topk_route_workspace_bytes(T, E, K), B.ffn_down_q4_workspace_bytes(dims, 64, T), B.dense_ffn_workspace_bytes(dims, T))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def run(s):
        B.norm_residual(s["h"], s["y"], s["w"], s["x"], w_post=s["w"], gate=s["gate"], h_out=s["h_out"])
        B.topk_route(s["logits"], s["ids"], s["gw"], s["off"], s["order"], workspace=ws)
        B.ffn_down_q4(dims, blob, 64, s["yg"], s["yu"], s["ids"], s["gw"], T, s["q4"], ws, n)
        B.grouped_matmul(s["x"], wg, s["off"], s["hh"], W_up=wu, rows=s["order"], rows_per_a=K, scatter=True)
        B.grouped_matmul(s["hh"], wd, s["off"], s["down"], rows=s["order"], scatter=True)
        B.dense_ffn_forward(dims, wg, wu, wd, s["x"], s["ids"], s["gw"], s["off"], s["order"], s["dense"], ws)

    a, b = _inputs(1, T, E, K, d, d_ff, dtype), _inputs(2, T, E, K, d, d_ff, dtype)
    run(a)
    first = {k: a[k].clone() for k in OUT}
    for i in range(12):
        if i % 3 == 0:
            run(b)
        if i % 4 == 0:
            ws.fill_(0xFF)
        run(a)
        for k in OUT:
            assert torch.equal(a[k], first[k]), (k, i)
