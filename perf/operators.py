"""The operators of a mixture-of-experts block around the spectral experts, as measured cases.

Four operators: the norms and the gated residual around a block (``norm``), the top-k
router with its pairs grouped by expert (``route``), the experts' down projection with
4-bit weights and group scales (``q4``) and matrix products grouped by expert with
ragged sizes (``gmm``).  ``run`` computes them in plain torch operations, or with
``own`` through the library's calls.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token between two blocks of a decode step: fp32 residual stream, the FFN's fp32 output, fp16 input of the next layer
        _norm("norm_decode", 1, 2048, "f32", "f32", "f16", False, "none"),
        # a ragged batch of an odd width, each token's output scaled by its own gate
        _norm("norm_ragged", 333, 1001, "f16", "f32", "f16", False, "token"),
        # a long prompt: bf16 residual, a norm on the block's output as well and a learned gate per channel
        _norm("norm_prefill", 8192, 4096, "bf16", "f32", "bf16", True, "channel"),
        # one token's routing in a decode step (Qwen-shaped layer)
        _route("route_decode", 1, 128, 8, "f32", "softmax", True, 0.0),
        # a long prompt's routing, some experts closed to some tokens
        _route("route_prefill", 16384, 128, 8, "f32", "softmax", True, 0.05),
        # the down step of one decode token (Qwen-shaped layer)
        _q4("q4_decode", 1, 2048, 768, 128, 8, 64, "uniform"),
        # a decode batch: nearly every expert is touched by a few tokens
        _q4("q4_batch", 64, 2048, 768, 128, 8, 64, "uniform"),
        # a small batch on few wide experts with skewed routing (Mixtral-shaped layer)
        _q4("q4_wide", 5, 4096, 14336, 8, 2, 128, "zipf"),
        # gate and up products of a small decode batch, x gathered by the routing
        _gmm("gmm_decode", "gated", 8, 768, 2048, 128, 8, "f16", "f16", "uniform", 0),
        # gate and up products of a prompt, x gathered by the routing
        _gmm("gmm_prompt", "gated", 2048, 768, 2048, 128, 8, "bf16", "bf16", "uniform", 0),
        # the down product of the same prompt, fp32 rows scattered back to (token, slot) order, the tail of the batch padding
        _gmm("gmm_down", "scatter", 2048, 2048, 768, 128, 8, "bf16", "f32", "uniform", 37),
        # rows already sorted by expert on few wide experts with skewed sizes
        _gmm("gmm_wide", "sorted", 1025, 14336, 4096, 8, 2, "f16", "f16", "zipf", 0),
    ]


def _norm(name, T, d, h, y, x, post, gate):
    return {"name": name, "op": "norm", "T": T, "d": d, "h": h, "y": y, "x": x, "post": post, "gate": gate}


def _route(name, T, E, K, type, scoring, renormalise, closed):
    return {"name": name, "op": "route", "T": T, "E": E, "K": K, "type": type, "scoring": scoring,
            "renormalise": renormalise, "closed": closed}


def _q4(name, T, d_model, d_ff, E, K, group, routing):
    return {"name": name, "op": "q4", "T": T, "d_model": d_model, "d_ff": d_ff, "E": E, "K": K, "group": group,
            "routing": routing}


def _gmm(name, form, T, N, D, E, K, type, out, routing, padding):
    return {"name": name, "op": "gmm", "form": form, "T": T, "N": N, "D": D, "E": E, "K": K, "type": type, "out": out,
            "routing": routing, "padding": padding}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "route", "q4", "gmm"))
    if op == "norm":
        d = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            d = max(8, d // 8 * 8)
        T = _log(rng, 1, min(8192, 8192 * 4096 // d))
        c = _norm("", T, d, rng.choice(("f32", "f16", "bf16")), rng.choice(("f32", "f16", "bf16")),
                  rng.choice(("f16", "bf16", "f32")), rng.random() < 0.5, rng.choice(("none", "token", "channel")))
    elif op == "route":
        E = _log(rng, 4, 512)
        c = _route("", _log(rng, 1, min(16384, 16384 * 128 // E)), E, _log(rng, 1, min(E, 16)),
                   rng.choice(("f32", "f16", "bf16")), rng.choice(("softmax", "sigmoid")), rng.random() < 0.6,
                   rng.choice((0.0, 0.1, 0.5)))
    elif op == "q4":
        E, d_ff = _log(rng, 2, 128), 8 * _log(rng, 8, 512)
        c = _q4("", _log(rng, 1, 256), _log(rng, 64, min(4096, 2048 * 768 * 128 // (E * d_ff))), d_ff, E,
                _log(rng, 1, min(E, 8)), rng.choice((32, 64, 128)), rng.choice(("uniform", "zipf")))
    else:
        E, D = _log(rng, 2, 128), 8 * _log(rng, 8, 512)
        form = rng.choice(("gated", "scatter", "sorted"))
        type = rng.choice(("f16", "bf16"))
        c = _gmm("", form, _log(rng, 1, 2048), _log(rng, 64, min(8192, 2048 * 768 * 128 // (E * D))), D, E,
                 _log(rng, 1, min(E, 8)), type, rng.choice((type, "f32")), rng.choice(("uniform", "zipf")),
                 rng.choice((0, 0, 5)))
    del c["name"]
    return c


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["d"]
        b = n * (2 * BYTES[c["h"]] + BYTES[c["y"]] + BYTES[c["x"]]) + 4 * c["d"] * (1 + c["post"])
        b += {"none": 0, "token": 4 * c["T"], "channel": 4 * c["d"]}[c["gate"]]
        return {"bytes": b, "flops": n * (6 + 4 * c["post"])}
    if c["op"] == "route":
        return {"bytes": c["T"] * c["E"] * BYTES[c["type"]] + 12 * c["T"] * c["K"] + 4 * (c["E"] + 1),
                "flops": 3 * c["T"] * c["E"]}
    touched = _touched(c["T"], c["E"], c["K"])
    pairs = c["T"] * c["K"]
    if c["op"] == "q4":
        per = c["d_model"] * c["d_ff"]
        return {"bytes": touched * per * (0.5 + 2.0 / c["group"]) + pairs * (8 * c["d_ff"] + 8) + 4 * c["T"] * c["d_model"],
                "flops": 2.0 * pairs * per}
    n = 2 if c["form"] == "gated" else 1
    a = c["T"] if c["form"] == "gated" else pairs
    return {"bytes": 2.0 * n * touched * c["N"] * c["D"] + 2 * a * c["D"] + pairs * c["N"] * BYTES[c["out"]] + 4 * pairs,
            "flops": 2.0 * n * pairs * c["N"] * c["D"]}


def _touched(T, E, K):
    """Experts that T tokens are expected to touch (uniform routing)."""
    return min(E, T * K, E * (1.0 - (1.0 - K / E) ** T) if K < E else E)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"case": c, **{"norm": _prepare_norm, "route": _prepare_route, "q4": _prepare_q4, "gmm": _prepare_gmm}[c["op"]](c, g)}


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _prepare_norm(c, g):
    T, d = c["T"], c["d"]
    s = {"h": (2.0 * _randn(g, T, d)).to(TYPES[c["h"]]), "y": (0.5 * _randn(g, T, d)).to(TYPES[c["y"]]),
         "w_pre": 1.0 + 0.1 * _randn(g, d), "w_post": 1.0 + 0.1 * _randn(g, d) if c["post"] else None, "gate": None,
         "alpha": 0.7, "eps": 1e-6}
    if c["gate"] != "none":
        s["gate"] = torch.sigmoid(_randn(g, *((T, 1) if c["gate"] == "token" else (1, d))))
    s["h_out"] = torch.empty_like(s["h"])
    s["x"] = torch.empty((T, d), dtype=TYPES[c["x"]], device="cuda")
    return s


def _prepare_route(c, g):
    T, E, K = c["T"], c["E"], c["K"]
    logits = (1.5 * _randn(g, T, E)).to(TYPES[c["type"]])
    if c["closed"] > 0:  # experts that a token may not use, and now and then a token without any
        shut = torch.rand((T, E), generator=g, device="cuda") < c["closed"]
        shut |= torch.rand((T, 1), generator=g, device="cuda") < 0.02
        logits = logits.masked_fill(shut, float("-inf"))
    i32 = {"dtype": torch.int32, "device": "cuda"}
    s = {"logits": logits, "ids": torch.empty((T, K), **i32), "gate_w": torch.empty((T, K), device="cuda"),
         "offsets": torch.empty(E + 1, **i32), "order": torch.empty(T * K, **i32)}
    s["scratch"] = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    return s


def _routing(c, g):
    """ids [T][K] int32, gate weights [T][K] f32 and the longest group's length."""
    T, E, K = c["T"], c["E"], c["K"]
    score = torch.rand((T, E), generator=g, device="cuda")
    if c["routing"] == "zipf":  # without replacement, expert e with weight (e + 1)^-1.2
        score = score.log() * torch.arange(1, E + 1, device="cuda", dtype=torch.float32) ** 1.2
    ids = score.argsort(dim=1, descending=True)[:, :K].to(torch.int32).contiguous()
    gate_w = torch.softmax(_randn(g, T, K), dim=1)
    return ids, gate_w, int(torch.bincount(ids.reshape(-1).long(), minlength=E).max())


def _prepare_q4(c, g):
    ids, gate_w, most = _routing(c, g)
    T, K, E, N, D, G = c["T"], c["K"], c["E"], c["d_model"], c["d_ff"], c["group"]
    s = {"ids": ids, "gate_w": gate_w, "most": most, "y_gate": 2.0 * _randn(g, T, K, D), "y_up": _randn(g, T, K, D),
         "out": torch.empty((T, N), device="cuda")}
    # The packed weights as a checkpoint holds them.  Per expert and block of 16 rows: the codes of 16 x 64 tiles
    # as [tile][lane][4] 32-bit words, then the group scales [group][16] in fp16; rows padded to 16, columns to a
    # multiple of 64 and of the group; w = scale (q - 7.5).  Lane 4 a + b of word t of a tile: rows a and a + 8,
    # columns 16 t + 2 b + {0, 1, 8, 9}; nibble 4 p + 2 u + v is row a + 8 v, column 16 t + 8 u + 2 b + p.
    Np, Dp = -(-N // 16) * 16, -(-D // max(64, G)) * max(64, G)
    blob = torch.empty((E, Np // 16, 2 * Dp + 8 * (Dp // G)), dtype=torch.int32, device="cuda")
    step = max(1, (1 << 26) // (Np * Dp))
    for e in range(0, E, step):
        n = min(step, E - e)
        w = torch.zeros((n, Np, Dp), device="cuda")
        w[:, :N, :D] = _randn(g, n, N, D) * D ** -0.5
        w = w.view(n, Np, Dp // G, G)
        scale = (2.0 * w.abs().amax(dim=3) / 15.0).half()
        f = scale.float().unsqueeze(3)
        q = torch.where(f > 0, torch.floor(w / f + 8.0), torch.zeros_like(w)).clamp_(0, 15).to(torch.int32)
        q = q.view(n, Np // 16, 2, 8, Dp // 64, 4, 2, 4, 2)  # block, v, a, tile, t, u, b, p
        q = q.permute(0, 1, 4, 3, 7, 5, 8, 6, 2).reshape(n, Np // 16, 2 * Dp, 8)
        shift = 4 * torch.arange(8, device="cuda", dtype=torch.int32)
        blob[e:e + n, :, :2 * Dp] = (q << shift).sum(dim=3, dtype=torch.int64).to(torch.int32)
        scale = scale.view(n, Np // 16, 16, Dp // G).permute(0, 1, 3, 2).contiguous()
        blob[e:e + n, :, 2 * Dp:] = scale.view(n, Np // 16, -1).view(torch.int32)
        del w, f, q, scale
    s["blob"] = blob.view(-1).view(torch.uint8)
    s["scratch"] = torch.empty((1 << 20) + 4 * T * K * (N + 2 * D + 64), dtype=torch.uint8, device="cuda")
    return s


def _prepare_gmm(c, g):
    ids, _, most = _routing(c, g)
    T, K, E, N, D, type = c["T"], c["K"], c["E"], c["N"], c["D"], TYPES[c["type"]]
    pairs = T * K
    real = (T - min(c["padding"], T - 1)) * K  # the tail of the batch holds no tokens
    flat = ids.view(-1).long().clone()
    flat[real:] = E
    order = torch.sort(flat, stable=True).indices.to(torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(flat[:real], minlength=E).cumsum(0).to(torch.int32)
    s = {"offsets": offsets, "order": order, "most": most, "rows": real}
    s["a"] = _randn(g, T if c["form"] == "gated" else pairs, D).to(type)
    for name in ("w", "w_up") if c["form"] == "gated" else ("w",):
        s[name] = torch.empty((E, N, D), dtype=type, device="cuda")
        for e in range(E):
            s[name][e] = _randn(g, N, D) * D ** -0.5
    s["out"] = torch.zeros((pairs, N), dtype=TYPES[c["out"]], device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "route": _own_route, "q4": _own_q4, "gmm": _own_gmm}[op](state)
    return {"norm": _plain_norm, "route": _plain_route, "q4": _plain_q4, "gmm": _plain_gmm}[op](state)


def _own_norm(s):
    from mixed_precision_decode_b200 import bitsmoe as B

    B.norm_residual(s["h"], s["y"], s["w_pre"], s["x"], w_post=s["w_post"], gate=s["gate"], alpha=s["alpha"],
                    eps=s["eps"], h_out=s["h_out"])
    return s["h_out"], s["x"]


def _plain_norm(s):
    u = s["y"].float()
    if s["w_post"] is not None:
        u = u * torch.rsqrt((u * u).mean(dim=1, keepdim=True) + s["eps"]) * s["w_post"]
    if s["gate"] is not None:
        u = u * s["gate"]
    h = s["h"].float() + s["alpha"] * u
    x = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + s["eps"]) * s["w_pre"]
    return h.to(s["h"].dtype), x.to(s["x"].dtype)


def _own_route(s):
    from mixed_precision_decode_b200 import bitsmoe as B

    B.topk_route(s["logits"], s["ids"], s["gate_w"], s["offsets"], s["order"], scoring=s["case"]["scoring"],
                 renormalise=s["case"]["renormalise"], workspace=s["scratch"])
    return s["ids"], s["gate_w"], s["offsets"], s["order"]


def _plain_route(s):
    c = s["case"]
    K, E = c["K"], c["E"]
    l = s["logits"].float()
    v, i = torch.sort(l, dim=1, descending=True, stable=True)
    top, is_open = v[:, :K], v[:, :K] > float("-inf")
    if c["scoring"] == "softmax":
        m = torch.where(is_open[:, :1], top[:, :1], torch.zeros_like(top[:, :1]))
        w, total = torch.exp(top - m), torch.exp(l - m).sum(dim=1, keepdim=True)
    else:
        w, total = 1.0 / (1.0 + torch.exp(-top)), torch.ones_like(top[:, :1])
    if c["renormalise"]:
        total = w.sum(dim=1, keepdim=True)
    gate_w = torch.where(is_open, w / total, torch.zeros_like(w))
    ids = torch.where(is_open, i[:, :K], -1).to(torch.int32)
    key = torch.where(is_open, i[:, :K], E).reshape(-1)
    sorted_key, order = torch.sort(key, stable=True)
    offsets = (key.unsqueeze(1) < torch.arange(E + 1, device=key.device)).sum(dim=0).to(torch.int32)
    return ids, gate_w, offsets, torch.where(sorted_key < E, order, -1).to(torch.int32)


def _own_q4(s):
    from mixed_precision_decode_b200 import bitsmoe as B

    c = s["case"]
    dims = B.ffn_dims(c["d_model"], c["d_ff"], c["E"], c["K"])
    B.ffn_down_q4(dims, s["blob"], c["group"], s["y_gate"], s["y_up"], s["ids"], s["gate_w"], c["T"], s["out"],
                  s["scratch"], s["scratch"].numel())
    return s["out"]


def _padded(key, E, most):
    """Row of every pair in [E][most] padded groups (key: each pair's expert, E for none)."""
    n = key.numel()
    sorted_key, order = torch.sort(key, stable=True)
    first = (key.unsqueeze(1) < torch.arange(E + 1, device=key.device)).sum(dim=0)
    row = torch.empty_like(order)
    row[order] = sorted_key * most + torch.arange(n, device=key.device) - first[sorted_key]
    return row


def _q4_weights(blob, N, D, G):
    """fp32 weights [..][N][D] of packed experts."""
    Dp = -(-D // max(64, G)) * max(64, G)
    E, R = blob.shape[:2]
    q = blob[:, :, :2 * Dp].reshape(E, R, Dp // 64, 8, 4, 4, 1)
    q = (q >> (4 * torch.arange(8, device=q.device, dtype=torch.int32))) & 15
    q = q.view(E, R, Dp // 64, 8, 4, 4, 2, 2, 2).permute(0, 1, 8, 3, 2, 5, 7, 4, 6).reshape(E, R * 16, Dp // G, G)
    scale = blob[:, :, 2 * Dp:].contiguous().view(torch.float16).view(E, R, Dp // G, 16).permute(0, 1, 3, 2)
    w = (q.float() - 7.5) * scale.reshape(E, R * 16, Dp // G, 1).float()
    return w.view(E, R * 16, Dp)[:, :N, :D]


def _plain_q4(s):
    c = s["case"]
    T, K, E, N, D = c["T"], c["K"], c["E"], c["d_model"], c["d_ff"]
    blob = s["blob"].view(torch.int32).view(E, -(-N // 16), -1)
    h = (s["y_gate"] / (1.0 + torch.exp(-s["y_gate"])) * s["y_up"]).view(T * K, D)
    key = s["ids"].view(-1).long()
    if T * K <= E:
        y = torch.matmul(_q4_weights(blob[key], N, D, c["group"]), h.unsqueeze(2)).squeeze(2)
    else:
        row = _padded(key, E, s["most"])
        hp = torch.zeros((E * s["most"], D), device=h.device)
        hp[row] = h
        y = torch.bmm(hp.view(E, -1, D), _q4_weights(blob, N, D, c["group"]).transpose(1, 2)).view(-1, N)[row]
    return (y.view(T, K, N) * s["gate_w"].unsqueeze(2)).sum(dim=1)


def _own_gmm(s):
    from mixed_precision_decode_b200 import bitsmoe as B

    c = s["case"]
    if c["form"] == "gated":
        B.grouped_matmul(s["a"], s["w"], s["offsets"], s["out"], W_up=s["w_up"], rows=s["order"], rows_per_a=c["K"])
    elif c["form"] == "scatter":
        B.grouped_matmul(s["a"], s["w"], s["offsets"], s["out"], rows=s["order"], scatter=True)
    else:
        B.grouped_matmul(s["a"], s["w"], s["offsets"], s["out"])
    return s["out"]


def _plain_gmm(s):
    c = s["case"]
    E, N, D, most, real = c["E"], c["N"], c["D"], s["most"], s["rows"]
    place = torch.arange(real, device="cuda")
    key = (place.unsqueeze(1) >= s["offsets"][1:]).sum(dim=1)
    slot = key * most + place - s["offsets"].long()[key]
    pair = s["order"][:real].long()
    source = pair // c["K"] if c["form"] == "gated" else pair if c["form"] == "scatter" else place
    a = torch.zeros((E * most, D), device="cuda")
    a[slot] = s["a"][source].float()
    a = a.view(E, most, D)
    y = torch.bmm(a, s["w"].float().transpose(1, 2)).view(-1, N)[slot]
    if c["form"] == "gated":
        y = y / (1.0 + torch.exp(-y)) * torch.bmm(a, s["w_up"].float().transpose(1, 2)).view(-1, N)[slot]
    out = torch.zeros_like(s["out"])
    out[pair if c["form"] == "scatter" else place] = y.to(out.dtype)
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "q4": _exact_q4, "gmm": _exact_gmm}[case["op"]](s)


def _exact_norm(s):
    def rms(v):
        return torch.sqrt(v.square().sum(1, keepdim=True) / v.shape[1] + s["eps"])

    h, x = [], []
    for t in range(0, s["h"].shape[0], 1024):
        b = slice(t, t + 1024)
        u = s["y"][b].double()
        if s["w_post"] is not None:
            u = u / rms(u) * s["w_post"].double()
        if s["gate"] is not None:
            gate = s["gate"].double()
            u = u * (gate[b] if gate.shape[1] == 1 and gate.shape[0] > 1 else gate)
        v = s["h"][b].double() + s["alpha"] * u
        h.append(v)
        x.append(v / rms(v) * s["w_pre"].double())
    return torch.cat(h), torch.cat(x)


def _exact_route(s):
    c = s["case"]
    l = s["logits"].double()
    left, rows, score = l.clone(), torch.arange(c["T"], device="cuda"), []
    if c["scoring"] == "softmax":
        p = torch.softmax(l, dim=1)
    else:
        p = torch.sigmoid(l)
    for _ in range(c["K"]):  # the largest that is left, the first of equal ones
        most = left.max(dim=1, keepdim=True).values
        pick = (left == most).long().argmax(dim=1)
        shut = most.squeeze(1) == float("-inf")
        score.append(torch.where(shut, torch.zeros_like(p[:, 0]), p[rows, pick]))
        left[rows, pick] = float("-inf")
    w = torch.stack(score, dim=1)
    if c["renormalise"]:
        w = torch.where(w > 0, w / w.sum(dim=1, keepdim=True).clamp_min(1e-300), w)
    return None, w, None, None


def _exact_q4(s):
    c = s["case"]
    T, K, N, D, G = c["T"], c["K"], c["d_model"], c["d_ff"], c["group"]
    Dp, R = -(-D // max(64, G)) * max(64, G), -(-N // 16)
    words = s["blob"].view(torch.int32).view(c["E"], R, -1)
    r, k = torch.arange(N, device="cuda").unsqueeze(1), torch.arange(D, device="cuda").unsqueeze(0)
    lane = r % 8 * 4 + k % 8 // 2
    word = k // 64 * 128 + lane * 4 + k % 64 // 16
    shift = 4 * (k % 2 * 4 + k % 16 // 8 * 2 + r % 16 // 8)
    ids = s["ids"].view(-1).tolist()
    g, u = s["y_gate"].double().view(T * K, D), s["y_up"].double().view(T * K, D)
    h = g * torch.sigmoid(g) * u
    y = torch.zeros((T * K, N), dtype=torch.float64, device="cuda")
    for e in sorted(set(ids)):
        q = (words[e][r // 16, word] >> shift) & 15
        scales = words[e][:, 2 * Dp:].contiguous().view(torch.float16).view(R, Dp // G, 16)
        w = (q.double() - 7.5) * scales[r // 16, k // G, r % 16].double()
        at = torch.tensor([j for j, v in enumerate(ids) if v == e], device="cuda")
        y[at] = h[at] @ w.T
    return (y.view(T, K, N) * s["gate_w"].double().unsqueeze(2)).sum(1)


def _exact_gmm(s):
    c = s["case"]
    bounds, order = s["offsets"].tolist(), s["order"].long()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        at = torch.arange(bounds[e], bounds[e + 1], device="cuda")
        if not at.numel():
            continue
        to = order[at] if c["form"] == "scatter" else at
        a = s["a"][order[at] // c["K"] if c["form"] == "gated" else to].double()
        y = a @ s["w"][e].double().T
        if c["form"] == "gated":
            y = y * torch.sigmoid(y) * (a @ s["w_up"][e].double().T)
        out[to] = y
    return out
