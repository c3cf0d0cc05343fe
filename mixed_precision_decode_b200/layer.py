"""User-facing objects over the C ABI: a packed projection, a spectral MoE gate/up
layer, expert FFNs, routing and the block around them.  torch provides device memory
and streams; every computation is a libbitsmoe kernel."""
from __future__ import annotations

import contextlib
import functools
import warnings

import torch

from . import bitsmoe as B

_HERE = contextlib.nullcontext()
_current_gpu = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else lambda: -1


def _on(stream, like: torch.Tensor):
    """Makes like's GPU and the given stream (torch's current one there, when None) current.  Tensors that a call
    allocates, fills or copies for itself then belong to the stream that its kernels run on: ordered with them, and,
    freed on return, their memory goes to later work of that stream alone."""
    if isinstance(stream, torch.cuda.Stream):
        return torch.cuda.stream(stream)
    dev = like.get_device()
    if stream is not None:
        return torch.cuda.stream(torch.cuda.ExternalStream(int(stream), device=dev))
    return _HERE if dev < 0 or dev == _current_gpu() else torch.cuda.device(dev)


def _capturing(t: torch.Tensor) -> bool:
    return t.is_cuda and torch.cuda.is_current_stream_capturing()


class _Workspaces:
    """Workspaces of size(T) bytes for an object's calls of T tokens."""

    def __init__(self, size, device, keep_one: bool):
        self._size, self._device, self._keep_one = size, device, keep_one
        self._bytes = {}   # of the last T's: asking the library costs a microsecond
        self.one = None    # one token's, when it is kept

    def get(self, T: int) -> torch.Tensor:
        if T == 1 and self.one is not None:
            return self.one
        n = self._bytes.get(T)
        if n is None:
            if len(self._bytes) >= 64:
                self._bytes.clear()
            n = self._bytes[T] = max(self._size(T), 256)
        if T != 1 or not self._keep_one:
            return torch.empty(n, dtype=torch.uint8, device=self._device)
        ws = torch.zeros(n, dtype=torch.uint8, device=self._device)
        if not _capturing(ws):  # else the zeros are the graph's, filled in at its replays alone
            self.one = ws
        return ws


class PackedProjection:
    """One projection (gate or up) of a spectral MoE layer, packed on the GPU.

    phi_t [r][d_in] fp16 (rows phi_k, kept unquantised), blob = the format-v2
    bit-plane blob of the expert directions, plan = its host descriptor."""

    def __init__(self, plan: B.Plan, blob: torch.Tensor, phi_t: torch.Tensor):
        self.plan, self.blob, self.phi_t = plan, blob, phi_t
        d = plan.dims
        self.d_in, self.d_out, self.n_experts, self.rank, self.top_k = d.d_in, d.d_out, d.n_experts, d.rank, d.top_k

    @classmethod
    def from_factors(cls, phi_t: torch.Tensor, amps: torch.Tensor, comps: torch.Tensor, widths: torch.Tensor,
                     top_k: int, scales: torch.Tensor | None = None, status: torch.Tensor | None = None,
                     stream=None) -> "PackedProjection":
        """Quantise and pack unit directions comps [E][r][d_out] (f32, on the GPU) at
        widths [E][r] (u8) with amplitudes amps [E][r] (f32)."""
        E, r, d_out = comps.shape
        d_in = phi_t.shape[1]
        dev = comps.device
        with _on(stream, comps):
            plan = B.pack_plan(d_in, d_out, E, r, top_k, widths.cpu())
            w_dev = widths.to(dev, torch.uint8).contiguous()
            if scales is None:
                scales = torch.empty((E, r), dtype=torch.int16, device=dev)
                B.compute_scales(plan, comps, w_dev, scales, status, stream)
            blob = torch.empty(plan.blob_bytes, dtype=torch.uint8, device=dev)
            B.pack(plan, comps.contiguous(), w_dev, scales.contiguous(), amps.contiguous(), blob, status, stream)
            return cls(plan, blob, phi_t.contiguous())

    def expert_bytes_touched(self, experts) -> int:
        """Packed bytes (planes + per-component metadata, padding included) of the given experts."""
        h = self.plan.header()
        tot = 0
        for e in experts:
            d = h[64 + 64 * int(e): 128 + 64 * int(e)]
            tot += int(d[8:16].view("uint64")[0])
        return tot


def decompose_and_pack(W: torch.Tensor, rank: int, widths_in_order, counts, top_k: int, status=None,
                       stream=None) -> tuple["PackedProjection", dict]:
    """The offline step before the decode path, on the GPU: the shared-basis spectral
    decomposition of one projection's expert matrices W [E][d_out][d_in] (f32),
    widths by descending amplitude (counts[j] components of each expert at
    widths_in_order[j]), then quantisation and packing.  Returns the packed
    projection and the decomposition (phi_t, sigma, amps, comps, widths)."""
    E, d_out, d_in = W.shape
    dev = W.device
    with _on(stream, W):
        n = B.ssd_workspace_bytes(E, d_out, d_in, rank)
        if n == 0:
            raise B.BitsMoEError(B.ECUDA, "ssd_workspace_bytes")
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        phi_t = torch.empty((rank, d_in), dtype=torch.float16, device=dev)
        phi_t32 = torch.empty((rank, d_in), dtype=torch.float32, device=dev)
        sigma = torch.empty(rank, dtype=torch.float32, device=dev)
        amps = torch.empty((E, rank), dtype=torch.float32, device=dev)
        comps = torch.empty((E, rank, d_out), dtype=torch.float32, device=dev)
        B.ssd_decompose(W.contiguous(), rank, phi_t, amps, comps, ws, n, sigma=sigma, phi_t32=phi_t32, status=status,
                        stream=stream)
        del ws
        widths = torch.from_numpy(B.assign_widths(amps.cpu().numpy(), widths_in_order, counts))
        pk = PackedProjection.from_factors(phi_t, amps, comps, widths, top_k, status=status, stream=stream)
        return pk, {"phi_t": phi_t, "phi_t32": phi_t32, "sigma": sigma, "amps": amps, "comps": comps, "widths": widths}


def fqcm_widths(dec: dict, x_calib: torch.Tensor, ids_calib: torch.Tensor, gw_calib: torch.Tensor,
                avg_bits: float, stream=None) -> tuple[torch.Tensor, float, dict]:
    """Widths of one decomposed projection (decompose_and_pack's second result) by the
    FQCM cost under a budget of avg_bits per element: z = Phi^T x of the calibration
    tokens x_calib [T][d_in] fp16 on the GPU, then on the host the activation
    importance beta from z and the routing (ids_calib, gw_calib [T][top_k]), the
    distortion of every component at every width, and the allocation.
    Returns (widths [E][r] u8, total cost, {"beta", "eps"})."""
    phi_t = dec["phi_t"]
    r, d_in = phi_t.shape
    E, _, d_out = dec["comps"].shape
    T = x_calib.shape[0]
    with _on(stream, phi_t):
        Z = torch.empty((T, r), dtype=torch.float32, device=phi_t.device)
        B.shared_proj(phi_t, x_calib.contiguous(), Z, T, d_in, r, stream)
        beta = B.fqcm_beta(Z.cpu().numpy(), ids_calib.cpu().numpy(), gw_calib.cpu().numpy(), E)
        eps = B.fqcm_eps(dec["comps"].cpu().numpy())
        amps = dec["amps"].cpu().numpy()
    budget = int(avg_bits * E * r * d_out)
    widths, loss = B.allocate_widths(amps, beta, eps, d_out, budget)
    return torch.from_numpy(widths), loss, {"beta": beta, "eps": eps}


class SpectralMoELayer:
    """Gate and up projections of one MoE layer in shared-spectral form.

    Calls for one token keep state in the object between them: they must not overlap on
    the GPU, whatever their streams, nor may replays of graphs captured from them."""

    def __init__(self, gate: PackedProjection, up: PackedProjection):
        assert gate.d_in == up.d_in and gate.top_k == up.top_k and gate.n_experts == up.n_experts
        self.gate, self.up = gate, up
        self._ws = _Workspaces(lambda T: B.layer_workspace_bytes(gate.plan, up.plan, T), gate.blob.device, True)
        self._ios = {}

    def workspace(self, T: int) -> torch.Tensor:
        """A workspace for a call of T tokens.  One token's is the layer's own, made and
        zero-filled on first use: its head keeps the fused path's counters between calls.
        (First use in a stream capture: a call's own, zero-filled at every replay.)
        Any other T uses nothing that an earlier call left and gets a new one."""
        return self._ws.get(T)

    def _proj_ios(self, out: dict) -> tuple:
        """The two projections' I/O descriptors for these output buffers, reused
        while a caller keeps passing the same buffers (a decode loop)."""
        zg, zu, yg, yu = out.get("Z_gate"), out.get("Z_up"), out.get("Y_experts_gate"), out.get("Y_experts_up")
        key = (out["Y_sum_gate"].data_ptr(), out["Y_sum_up"].data_ptr(), zg is not None and zg.data_ptr(),
               zu is not None and zu.data_ptr(), yg is not None and yg.data_ptr(), yu is not None and yu.data_ptr())
        ios = self._ios.get(key)
        if ios is None:
            ios = tuple(B.proj_io(p.plan, p.blob, p.phi_t, out[f"Y_sum_{name}"], out.get(f"Z_{name}"),
                                  out.get(f"Y_experts_{name}"))
                        for name, p in (("gate", self.gate), ("up", self.up)))
            if len(self._ios) >= 64:
                self._ios.clear()
            self._ios[key] = ios
        return ios

    def forward(self, x: torch.Tensor, topk_ids: torch.Tensor, gate_w: torch.Tensor, out: dict | None = None,
                want_experts: bool = False, want_z: bool = False, status: torch.Tensor | None = None,
                stream=None, next_layer: "SpectralMoELayer | None" = None) -> dict:
        """x [T][d_in] fp16, topk_ids [T][top_k] int32, gate_w [T][top_k] f32 (all on the GPU).
        Returns Y_sum_gate / Y_sum_up [T][d_out] f32 (and Y_experts_* / Z_* on request).
        next_layer: the layer a decode loop runs next; its Phi^T are prefetched into
        L2 while this call evaluates its experts (single-token path)."""
        T = x.shape[0]
        dev = x.device
        with _on(stream, x):
            if out is None:
                out = {}
                for name, p in (("gate", self.gate), ("up", self.up)):
                    out[f"Y_sum_{name}"] = torch.empty((T, p.d_out), dtype=torch.float32, device=dev)
                    if want_experts:
                        out[f"Y_experts_{name}"] = torch.empty((T, p.top_k, p.d_out), dtype=torch.float32, device=dev)
                    if want_z:
                        out[f"Z_{name}"] = torch.empty((T, p.rank), dtype=torch.float32, device=dev)
            self._run(x, topk_ids, gate_w, T, out, self._ws.get(T), status, stream, next_layer)
        return out

    def _run(self, x, topk_ids, gate_w, T: int, out: dict, ws, status, stream, next_layer=None):
        ios = self._proj_ios(out)
        if next_layer is None:
            B.layer_forward(ios[0], ios[1], x, topk_ids, gate_w, T, ws, ws.numel(), status, stream)
        else:
            B.layer_forward_chained(ios[0], ios[1], x, topk_ids, gate_w, T, ws, ws.numel(), next_layer.gate.phi_t,
                                    next_layer.up.phi_t, status, stream)


class Q4Down:
    """Down matrices [E][d_model][d_ff] held in 4 bits, a scale per `group` (32, 64 or
    128) columns of a row."""

    def __init__(self, blob: torch.Tensor, shape: tuple, group: int):
        assert blob.dtype == torch.uint8 and blob.numel() >= B.q4_bytes(*shape, group) > 0
        self.blob, self.shape, self.group = blob, tuple(shape), group

    @classmethod
    def pack(cls, w_down: torch.Tensor, group: int = 64, status: torch.Tensor | None = None, stream=None) -> "Q4Down":
        """Quantise w_down [E][d_model][d_ff] (float32, float16 or bfloat16, on the GPU)."""
        n = B.q4_bytes(*w_down.shape, group)
        with _on(stream, w_down):
            blob = torch.empty(n, dtype=torch.uint8, device=w_down.device)
            B.q4_pack(w_down.contiguous(), group, blob, status, stream)
        return cls(blob, w_down.shape, group)

    def unpack(self, stream=None) -> torch.Tensor:
        """The stored values, [E][d_model][d_ff] f32."""
        with _on(stream, self.blob):
            w = torch.empty(self.shape, dtype=torch.float32, device=self.blob.device)
            B.q4_unpack(self.blob, self.group, w, stream)
        return w


class SpectralMoEFFN:
    """A routed expert FFN: the gate and up projections in shared-spectral form
    (SpectralMoELayer), then SiLU(gate) * up and a down projection per expert, summed
    over each token's slots with its gate weights -- one bitsmoe_ffn_forward call with
    dense fp16 down matrices, the layer call and bitsmoe_ffn_down_q4 with 4-bit ones.

    w_down [E][d_model][d_ff] fp16 on the GPU, or a Q4Down of that shape; d_model = the
    layer's d_in and d_ff = the gate/up d_out.  Calls for one token must not overlap on the
    GPU (see SpectralMoELayer)."""

    def __init__(self, layer: SpectralMoELayer, w_down: "torch.Tensor | Q4Down"):
        g = layer.gate
        assert layer.up.d_out == g.d_out
        assert tuple(w_down.shape) == (g.n_experts, g.d_in, g.d_out)
        self.layer = layer
        self.q4 = w_down if isinstance(w_down, Q4Down) else None
        if self.q4 is None:
            assert w_down.dtype == torch.float16
            self.w_down = w_down.contiguous()
        self.dims = B.ffn_dims(g.d_in, g.d_out, g.n_experts, g.top_k)
        if self.q4 is None:
            self._ws = _Workspaces(lambda T: B.ffn_workspace_bytes(g.plan, layer.up.plan, T), g.blob.device, True)
        else:
            self._q4_bytes = functools.lru_cache(64)(
                lambda T: B.ffn_down_q4_workspace_bytes(self.dims, self.q4.group, T))
            # the layer's is free again where the down step starts; one token's is the layer's own, and stays apart
            self._ws = _Workspaces(
                lambda T: max(self._q4_bytes(T), 0 if T == 1 else B.layer_workspace_bytes(g.plan, layer.up.plan, T)),
                g.blob.device, False)

    def workspace(self, T: int) -> torch.Tensor:
        """A workspace for a call of T tokens: with fp16 down matrices the layer's, then
        the down step's, one token's kept as SpectralMoELayer.workspace has it; with 4-bit
        ones enough for either step, which keeps nothing between calls."""
        return self._ws.get(T)

    def launches(self, T: int) -> int:
        """Kernels one forward launches for T tokens (the layer's, then the down step's)."""
        if self.q4 is not None:
            return (B.layer_launches(self.layer.gate.plan, self.layer.up.plan, T)
                    + B.ffn_down_q4_launches(self.dims, self.q4.group, T))
        return B.ffn_launches(self.layer.gate.plan, self.layer.up.plan, T)

    def gate_up_buffers(self, T: int, device) -> dict:
        """Output buffers of the gate and up projections (routed sums and per-slot outputs)."""
        out = {}
        for name, p in (("gate", self.layer.gate), ("up", self.layer.up)):
            out[f"Y_sum_{name}"] = torch.empty((T, p.d_out), dtype=torch.float32, device=device)
            out[f"Y_experts_{name}"] = torch.empty((T, p.top_k, p.d_out), dtype=torch.float32, device=device)
        return out

    def forward(self, x: torch.Tensor, topk_ids: torch.Tensor, gate_w: torch.Tensor, out: torch.Tensor | None = None,
                gate_up: dict | None = None, status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """x [T][d_in] fp16, topk_ids [T][top_k] int32, gate_w [T][top_k] f32 -> out [T][d_model] f32.
        gate_up: the gate/up output buffers (gate_up_buffers) to reuse between calls."""
        T = x.shape[0]
        with _on(stream, x):
            if out is None:
                out = torch.empty((T, self.dims.d_model), dtype=torch.float32, device=x.device)
            if gate_up is None:
                gate_up = self.gate_up_buffers(T, x.device)
            if self.q4 is not None:
                n = self._q4_bytes(T)
                ws = self._ws.get(T) if T != 1 or n else None
                self.layer._run(x, topk_ids, gate_w, T, gate_up, self.layer._ws.get(1) if T == 1 else ws, status, stream)
                B.ffn_down_q4(self.dims, self.q4.blob, self.q4.group, gate_up["Y_experts_gate"], gate_up["Y_experts_up"],
                              topk_ids, gate_w, T, out, ws, n, status, stream)
            else:
                ws = self._ws.get(T)
                ios = self.layer._proj_ios(gate_up)
                B.ffn_forward(ios[0], ios[1], self.w_down, x, topk_ids, gate_w, T, out, ws, ws.numel(), status, stream)
        return out


class Routing:
    """The routing of T tokens: topk_ids [T][top_k] int32 and gate_w [T][top_k] f32, and
    the (token, slot) pairs grouped by expert: offsets [E + 1] and order [T * top_k] int32."""

    def __init__(self, topk_ids, gate_w, offsets, order):
        self.topk_ids, self.gate_w, self.offsets, self.order = topk_ids, gate_w, offsets, order


def route(logits: torch.Tensor, top_k: int, scoring: str = "softmax", renormalise: bool = True, scale: float = 1.0,
          status: torch.Tensor | None = None, stream=None) -> Routing:
    """Top-k routing of router logits [T][E] (f32, f16 or bf16, on the GPU)."""
    T, E = logits.shape
    i32 = {"dtype": torch.int32, "device": logits.device}
    with _on(stream, logits):
        r = Routing(torch.empty((T, top_k), **i32), torch.empty((T, top_k), dtype=torch.float32, device=logits.device),
                    torch.empty(E + 1, **i32), torch.empty(T * top_k, **i32))
        n = B.topk_route_workspace_bytes(T, E, top_k)
        ws = torch.empty(n, dtype=torch.uint8, device=logits.device) if n else None
        B.topk_route(logits, r.topk_ids, r.gate_w, r.offsets, r.order, scoring=scoring, renormalise=renormalise,
                     scale=scale, workspace=ws, status=status, stream=stream)
    return r


class DenseMoEFFN:
    """The routed FFN of experts with dense matrices (before the decomposition, or in a
    layer left without it): w_gate, w_up [E][d_ff][d_model] and w_down [E][d_model][d_ff],
    fp16 or bf16 on the GPU.  Grouped products: made for many tokens as for few."""

    def __init__(self, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, top_k: int):
        E, d_ff, d_model = w_gate.shape
        assert w_up.shape == w_gate.shape and tuple(w_down.shape) == (E, d_model, d_ff)
        assert w_gate.dtype == w_up.dtype == w_down.dtype and w_gate.dtype in (torch.float16, torch.bfloat16)
        self.w_gate, self.w_up, self.w_down = w_gate.contiguous(), w_up.contiguous(), w_down.contiguous()
        self.dims = B.ffn_dims(d_model, d_ff, E, top_k)

    def forward(self, x: torch.Tensor, routing: Routing, out: torch.Tensor | None = None,
                status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """x [T][d_model] in the matrices' type -> out [T][d_model] f32."""
        T = x.shape[0]
        with _on(stream, x):
            if out is None:
                out = torch.empty((T, self.dims.d_model), dtype=torch.float32, device=x.device)
            ws = torch.empty(B.dense_ffn_workspace_bytes(self.dims, T), dtype=torch.uint8, device=x.device)
            B.dense_ffn_forward(self.dims, self.w_gate, self.w_up, self.w_down, x, routing.topk_ids, routing.gate_w,
                                routing.offsets, routing.order, out, ws, status, stream)
        return out


class MoEBlock:
    """A pre-norm MoE block around an expert FFN:

        x = rmsnorm(h) w_norm,  logits = w_router x,  y = FFN(x, top-k routing of the logits),
        h <- h + alpha * gate * (y, or rmsnorm(y) w_post with w_post given)

    The last step is taken by the next block's forward, fused with that block's norm, or by
    finish.  w_post and alpha belong to the block that made y: the next block is told which
    one that is (made_by).  w_norm, w_post [d_model] f32, w_router [E][d_model] fp16; ffn a
    SpectralMoEFFN or an fp16 DenseMoEFFN; gate, of that y, f32 [T or 1][d_model or 1], None
    without a y.  eps is that of the norms in this block's calls.  A token with fewer than
    top_k open experts (logits of -inf) leaves its other slots out; over a SpectralMoEFFN
    status then holds ST_BADEXPERT, over a DenseMoEFFN it does not."""

    def __init__(self, ffn: "SpectralMoEFFN | DenseMoEFFN", w_norm: torch.Tensor, w_router: torch.Tensor,
                 w_post: torch.Tensor | None = None, alpha: float = 1.0, eps: float = 1e-6, scoring: str = "softmax",
                 renormalise: bool = True, scale: float = 1.0):
        d = ffn.dims
        assert w_router.dtype == torch.float16 and tuple(w_router.shape) == (d.n_experts, d.d_model)
        assert not isinstance(ffn, DenseMoEFFN) or ffn.w_gate.dtype == torch.float16
        self.ffn, self.w_norm, self.w_router, self.w_post = ffn, w_norm, w_router.contiguous(), w_post
        self.alpha, self.eps, self.scoring, self.renormalise, self.scale = alpha, eps, scoring, renormalise, scale

    def _post_of(self, made_by) -> tuple:
        """(w_post, alpha) of the output that a block, or such a pair, stands for."""
        if isinstance(made_by, MoEBlock):
            return made_by.w_post, made_by.alpha
        if made_by is not None:
            w_post, alpha = made_by
            return w_post, alpha
        if self.w_post is not None or self.alpha != 1.0:
            warnings.warn("MoEBlock.forward: y without made_by is added with this block's own w_post and alpha",
                          stacklevel=3)
        return self.w_post, self.alpha

    def forward(self, h: torch.Tensor, y: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                status: torch.Tensor | None = None, stream=None,
                made_by: "MoEBlock | tuple | None" = None) -> torch.Tensor:
        """h [T][d_model] (the residual stream, f32, f16 or bf16), y: the output of the block
        before, added to h in place first.  made_by: the MoEBlock that made y, or the pair
        (w_post or None, alpha) of another kind of block; left out, y is taken as of a block
        with this one's w_post and alpha.  Returns this block's output, f32."""
        T, d = h.shape
        E = self.ffn.dims.n_experts
        w_post, alpha = (None, 1.0) if y is None else self._post_of(made_by)
        with _on(stream, h):
            x = torch.empty((T, d), dtype=torch.float16, device=h.device)
            B.norm_residual(h, y, self.w_norm, x, w_post=w_post, gate=gate, alpha=alpha, eps=self.eps, stream=stream)
            logits = torch.empty((T, E), dtype=torch.float32, device=h.device)
            B.shared_proj(self.w_router, x, logits, T, d, E, stream)
            r = route(logits, self.ffn.dims.top_k, self.scoring, self.renormalise, self.scale, status, stream)
            if isinstance(self.ffn, DenseMoEFFN):
                return self.ffn.forward(x, r, status=status, stream=stream)
            return self.ffn.forward(x, r.topk_ids, r.gate_w, status=status, stream=stream)

    def finish(self, h: torch.Tensor, y: torch.Tensor, gate: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Adds y, this block's own output and the last of a stack, to h in place."""
        B.norm_residual(h, y, w_post=self.w_post, gate=gate, alpha=self.alpha, eps=self.eps, stream=stream)
        return h
