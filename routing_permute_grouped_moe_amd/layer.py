"""The MoE expert layer as a sequence of C-ABI calls on one GPU.

This module only allocates device buffers (through torch) and calls the
library entry points in order; every step of the layer runs in the HIP
kernels of ``libmoe.so``.

Forward:  router logits -> route -> permute -> grouped GEMM (+ shared expert)
          -> unpermute/combine.
Backward: combine bwd -> grouped GEMM dX and dW (one call, paired launches)
          -> route bwd -> router bwd -> permute bwd (which also adds the
          shared expert's and the router's input gradients).

The forward runs on one stream: with the grouped GEMM's workspace, the
routed and the shared expert's gate/up and down products are one persistent
launch, which leaves no idle CUs for a second stream to use (a persistent
GEMM holds every CU it gets, and a GEMM workgroup fills its CU's registers).
With ``overlap`` the backward runs the route and router backward on a second
stream of the same priority, beside the grouped GEMM's dX and dW; that
measured within noise of one stream, so it is off by default.  Results are
bitwise identical either way.

With ``shape.capacity`` = C the layer is the drop-and-pad variant: every
expert owns C rows, pairs past an expert's first C (in token order) are
dropped, unfilled rows are zero, and the grouped GEMM runs on the padded
groups.

With ``balance`` (a :class:`BalanceLoss`) the forward computes the router's losses
after the routing and the backward takes their gradient into dlogits, in one pass
with the gates'.  Without it the layer makes the calls it always made.

Experts outside ``[g0, g0+G)`` are remote: their rows are moved by the
permute and the combine, their expert outputs and input gradients are zero
(the buffers are cleared once at allocation and never written), and they get
no weight gradients.
"""
from __future__ import annotations

from dataclasses import dataclass, field
from typing import NamedTuple, Optional

import torch

from . import abi


@dataclass
class LayerShape:
    T: int
    H: int
    I: int
    E: int
    k: int
    dtype: torch.dtype          # torch.bfloat16 or torch.float32
    g0: int = 0
    G: Optional[int] = None     # experts run by the grouped GEMM (None = all E)
    shared: bool = False
    router: bool = True         # False: logits are an input
    capacity: Optional[int] = None   # drop-and-pad: rows per expert (None = dropless)

    @property
    def groups(self) -> int:
        return self.E - self.g0 if self.G is None else self.G

    @property
    def R(self) -> int:
        """Rows of the permuted buffers."""
        return self.T * self.k if self.capacity is None else self.E * self.capacity


class MoeLayer:
    """Device buffers of one layer plus the forward/backward call sequences."""

    def __init__(self, shape: LayerShape, device="cuda", overlap: bool = False,
                 recompute: bool = False, balance: "Optional[BalanceLoss]" = None):
        s = self.s = shape
        self.overlap = overlap
        # auxiliary losses of the router, over packed sequences ``seq`` and the
        # tokens to ``keep`` (set by the caller; None: one sequence, all tokens)
        self.balance = balance
        self.seq = self.keep = self.losses = None
        self._counted = (None, None, None)   # losses, and the seq and keep they were taken over
        # recompute: no permuted copy of x (the grouped GEMMs gather token
        # rows through src_token) and act is recomputed from h13 for dW
        self.recompute = recompute
        dev = self.device = torch.device(device)
        dt, f32, i32 = s.dtype, torch.float32, torch.int32
        self.dt = abi.MOE_BF16 if dt == torch.bfloat16 else abi.MOE_F32
        T, H, I, E, k, R, G = s.T, s.H, s.I, s.E, s.k, s.R, s.groups
        e = lambda *shp, d=dt: torch.empty(shp, dtype=d, device=dev)
        z = lambda *shp, d=dt: torch.zeros(shp, dtype=d, device=dev)
        # parameters / inputs (filled by the caller)
        self.x = e(T, H)
        self.wg = e(H, E, d=f32) if s.router else None
        self.bias = None
        self.logits = e(T, E, d=f32)
        self.w13 = e(G, 2 * I, H)
        self.w2 = e(G, H, I)
        self.ws13 = e(2 * I, H) if s.shared else None
        self.ws2 = e(H, I) if s.shared else None
        self.dy = e(T, H)
        # forward state
        self.idx = e(T, k, d=i32)
        self.gate = e(T, k, d=f32)
        self.xp = None if recompute else e(R, H)
        self.counts = e(E, d=i32)
        self.offsets = e(E + 1, d=i32)
        self.row_id_map = e(T, k, d=i32)
        # load statistics; an EP group is the window of experts one device runs
        self.epg = s.groups if E % s.groups == 0 else E
        self.load = e(E, d=f32)
        self.cv = e(2, d=f32)
        self.group_counts = e(E // self.epg, d=i32)
        self.src_token = e(R, d=i32)
        self.ws_bytes = abi.moe_permute_workspace_bytes(T, E, k)
        self.ws = torch.empty(max(self.ws_bytes, 16), dtype=torch.uint8, device=dev)
        self.rws_bytes = abi.moe_router_workspace_bytes(T, H, E, self.dt) if s.router else 0
        self.rws = torch.empty(max(self.rws_bytes, 256), dtype=torch.uint8, device=dev)
        self._wg_split = False
        # tile scheduler counters of the grouped GEMM (zero-filled once; every
        # call leaves them zero); set_gemm_dynamic(False) selects the static order
        self.gws_bytes = abi.moe_gmm_workspace_bytes()
        self.gws = torch.zeros(self.gws_bytes, dtype=torch.uint8, device=dev)
        self.aux = torch.cuda.Stream(device=dev) if overlap else None
        self._ev = [torch.cuda.Event() for _ in range(2)] if overlap else None
        self.h13 = e(R, 2 * I)
        self.act = e(R, I)
        self.yp = z(R, H)            # remote rows stay zero
        self.y = e(T, H)
        if s.shared:
            self.sh_h13 = e(T, 2 * I)
            self.sh_act = e(T, I)
            self.ys = e(T, H)
        # backward state
        self.dyp = e(R, H)
        self.dgate = e(T, k, d=f32)
        self.dh13 = e(R, 2 * I)
        self.dxp = z(R, H)           # remote rows stay zero
        self.dw13 = e(G, 2 * I, H)
        self.dw2 = e(G, H, I)
        self.dlogits = e(T, E, d=f32)
        self.dx = e(T, H)
        if s.router:
            self.dx_router = e(T, H)
            self.dwg = e(H, E, d=f32)
            self.dbias = e(E, d=f32)
        if s.shared:
            self.sh_dh13 = e(T, 2 * I)
            self.sh_dx = e(T, H)
            self.dws13 = e(2 * I, H)
            self.dws2 = e(H, I)

    # ------------------------------------------------------------------ helpers
    def set_gemm_dynamic(self, on: bool = True):
        """Grouped GEMM tiles from per-XCD counters (True) or a fixed share (False)."""
        if on:
            self.gws_bytes = abi.moe_gmm_workspace_bytes()
            self.gws = torch.zeros(self.gws_bytes, dtype=torch.uint8, device=self.device)
        else:
            self.gws_bytes, self.gws = 0, None

    def shared_desc(self):
        if not self.s.shared:
            return None
        return abi.shared_expert(
            T=self.s.T, x=self.x, w13=self.ws13, w2=self.ws2, h13=self.sh_h13, act=self.sh_act,
            y=self.ys, dy=self.dy, dh13=self.sh_dh13, dx=self.sh_dx, dw13=self.dws13,
            dw2=self.dws2)

    # ------------------------------------------------------------------ steps
    def router_fwd(self, stream=None):
        s = self.s
        abi.moe_router_logits(self.x, self.dt, self.wg, self.bias, s.T, s.H, s.E, self.logits,
                              self.rws, self.rws_bytes, stream)
        self._wg_split = True    # the router workspace now holds wg's split

    def route(self, stream=None):
        s = self.s
        abi.moe_route(self.logits, s.T, s.E, s.k, self.idx, self.gate, stream)

    def balance_loss(self, stream=None):
        """``losses`` (a :class:`Balance`): read its ``loss`` after the forward; the
        backward takes the gradient of ``loss[2]`` into dlogits, over the ``seq`` and
        ``keep`` of this call: a caller may have set other tensors by then, for the next
        batch, but leaves the contents of these."""
        seq, keep = self.seq, self.keep
        self.losses = self.balance.forward(self.logits, self.idx, seq=seq, keep=keep,
                                           stream=stream)
        self._counted = (self.losses, seq, keep)

    def permute(self, stream=None):
        s = self.s
        if s.capacity is not None:
            abi.moe_permute_capacity(self.x, self.dt, self.idx, s.T, s.H, s.E, s.k, s.capacity,
                                     self.xp, self.counts, self.offsets, self.row_id_map,
                                     self.src_token, self.ws, self.ws_bytes, stream)
            return
        abi.moe_permute(self.x, self.dt, self.idx, s.T, s.H, s.E, s.k, self.xp, self.counts,
                        self.offsets, self.row_id_map, self.src_token, self.ws, self.ws_bytes,
                        stream)

    def load_stats(self, stream=None):
        abi.moe_load_stats(self.counts, self.s.E, self.epg, self.load, self.cv, self.group_counts,
                           stream)

    def saved_bytes(self) -> int:
        """Bytes of activations kept from the forward for the backward (beyond
        the layer input, the weights and the routing maps)."""
        b = self.x.element_size()
        s = self.s
        n = s.R * 2 * s.I + (s.T * 2 * s.I if s.shared else 0)        # h13
        if not self.recompute:
            n += s.R * s.H + s.R * s.I + (s.T * s.I if s.shared else 0)  # xp, act
        return n * b

    def _gmm_sel(self):
        """(G, shared descriptor, workspace) of the grouped-GEMM calls."""
        return self.s.groups, self.shared_desc(), self.gws

    def gmm_fwd(self, stream=None):
        s = self.s
        G, sh, ws = self._gmm_sel()
        if self.recompute:
            abi.moe_grouped_gemm_fwd_gather(self.x, self.src_token, s.T, self.offsets, s.g0, G,
                                            s.R, self.dt, s.H, s.I, self.w13, self.w2, self.h13,
                                            self.act, self.yp, sh, ws, self.gws_bytes, stream)
            return
        abi.moe_grouped_gemm_fwd(self.xp, self.offsets, s.g0, G, s.R, self.dt, s.H, s.I,
                                 self.w13, self.w2, self.h13, self.act, self.yp, sh, ws,
                                 self.gws_bytes, stream)

    def combine(self, stream=None):
        s = self.s
        abi.moe_unpermute_combine(self.yp, self.row_id_map, self.gate,
                                  self.ys if s.shared else None, self.dt, s.T, s.H, s.k, s.R,
                                  self.y, stream)

    def combine_bwd(self, stream=None):
        s = self.s
        abi.moe_unpermute_combine_bwd(self.dy, self.yp, self.row_id_map, self.gate, self.dt, s.T,
                                      s.H, s.k, s.R, self.dyp, self.dgate, stream)
        if s.capacity is not None:   # padded rows of dyp: exact zeros through dX and dW
            abi.moe_clear_empty_rows(self.src_token, s.R, self.dt, s.H, self.dyp, stream)

    def gmm_bwd_dx(self, stream=None):
        s = self.s
        G, sh, ws = self._gmm_sel()
        abi.moe_grouped_gemm_bwd_dx(self.dyp, self.offsets, s.g0, G, s.R, self.dt, s.H, s.I,
                                    self.w13, self.w2, self.h13, self.dh13, self.dxp, sh, ws,
                                    self.gws_bytes, stream)

    def gmm_bwd_dw(self, stream=None):
        s = self.s
        G, sh, ws = self._gmm_sel()
        if self.recompute:
            abi.moe_grouped_gemm_bwd_dw_recompute(self.x, self.src_token, s.T, self.h13, self.act,
                                                  self.dyp, self.dh13, self.offsets, s.g0, G,
                                                  s.R, self.dt, s.H, s.I, self.dw13, self.dw2,
                                                  sh, ws, self.gws_bytes, stream)
            return
        abi.moe_grouped_gemm_bwd_dw(self.xp, self.act, self.dyp, self.dh13, self.offsets, s.g0,
                                    G, s.R, self.dt, s.H, s.I, self.dw13, self.dw2, sh, ws,
                                    self.gws_bytes, stream)

    def gmm_bwd(self, stream=None):
        """dX and dW in one call (paired launches); the recompute variant
        keeps its two calls (dW recomputes act and gathers x)."""
        if self.recompute:
            self.gmm_bwd_dx(stream)
            self.gmm_bwd_dw(stream)
            return
        s = self.s
        G, sh, ws = self._gmm_sel()
        abi.moe_grouped_gemm_bwd(self.xp, self.act, self.dyp, self.offsets, s.g0, G, s.R, self.dt,
                                 s.H, s.I, self.w13, self.w2, self.h13, self.dh13, self.dxp,
                                 self.dw13, self.dw2, sh, ws, self.gws_bytes, stream)

    def route_bwd(self, stream=None):
        s = self.s
        if self.balance is not None:      # the gates' and the losses' gradient in one pass
            if self.losses is None:
                raise RuntimeError("the backward of the router's losses before their forward")
            of, seq, keep = self._counted
            if of is not self.losses:     # (the caller's own)
                seq, keep = self.seq, self.keep
            self.balance.backward(self.logits, self.idx, self.losses.counts, self.losses.tokens,
                                  seq=seq, keep=keep, dgate=self.dgate, out=self.dlogits,
                                  stream=stream)
            return
        abi.moe_route_bwd(self.logits, self.idx, self.dgate, s.T, s.E, s.k, self.dlogits, stream)

    def router_bwd(self, stream=None):
        """Reuses the split of wg that router_fwd left in the router
        workspace (the step order: wg does not change between the two)."""
        s = self.s
        flags = abi.MOE_ROUTER_WG_SPLIT if self._wg_split else 0
        abi.moe_router_logits_bwd(self.dlogits, self.x, self.dt, self.wg, s.T, s.H, s.E,
                                  self.dx_router, self.dwg, self.dbias, self.rws, self.rws_bytes,
                                  stream, flags=flags)

    def permute_bwd(self, stream=None):
        s = self.s
        abi.moe_permute_bwd(self.dxp, self.row_id_map, self.dt, s.T, s.H, s.k, s.R,
                            self.sh_dx if s.shared else None,
                            self.dx_router if s.router else None, self.dx, stream)

    # ------------------------------------------------------------------ passes
    def _streams(self, stream):
        main = torch.cuda.current_stream(self.device) if stream is None else stream
        return main, self.aux

    def forward(self, stream=None):
        s = self.s
        if s.router:
            self.router_fwd(stream)
        self.route(stream)
        if self.balance is not None:
            self.balance_loss(stream)
        self.permute(stream)
        self.load_stats(stream)
        self.gmm_fwd(stream)
        self.combine(stream)

    def backward(self, stream=None):
        s = self.s
        if self.overlap and s.router:
            main, aux = self._streams(stream)
            ev_c, ev_aux = self._ev[0], self._ev[1]
            self.combine_bwd(main)
            ev_c.record(main)
            aux.wait_event(ev_c)
            self.route_bwd(aux)                         # needs dgate
            self.router_bwd(aux)
            ev_aux.record(aux)
            self.gmm_bwd(main)
            main.wait_event(ev_aux)
            self.permute_bwd(main)
            return
        self.combine_bwd(stream)
        self.gmm_bwd(stream)
        self.route_bwd(stream)
        if s.router:
            self.router_bwd(stream)
        self.permute_bwd(stream)

    def step(self, stream=None):
        self.forward(stream)
        self.backward(stream)

    def grads(self):
        """The gradients of the layer's parameters, in their buffers."""
        g = [self.dw13, self.dw2]
        if self.s.shared:
            g += [self.dws13, self.dws2]
        if self.s.router:
            g += [self.dwg] if self.bias is None else [self.dwg, self.dbias]
        return g

    def clip_grads(self, max_norm: float, stream=None):
        """Clips the layer's gradients by their norm together, in place; returns the
        norm (:class:`GradClip` takes the gradients of several layers, and one that is
        kept saves the 8 us of making it here)."""
        return GradClip(self.grads()).clip(max_norm, stream=stream)


# ---------------------------------------------------------------------- checked calls
def _check(name, t, dtype, device, *shape, beside="the weights are"):
    """A tensor the kernels can read as it lies: dense, of this shape, type and device
    (that of ``beside``)."""
    if (t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, not {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, {beside} on {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    raise ValueError(f"{name} is not contiguous")


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(device, stream, call, *inputs):
    """call(raw stream) with the device of a call's tensors current, and the
    given stream too (None: the device's current one; a raw handle as well as a
    torch stream, as the layer's own calls take both), so that outputs and workspaces
    allocated inside belong to it; the inputs and weights, which may not, are kept
    from reuse until the stream has passed."""
    if stream is None:
        if torch.cuda.current_device() == device.index:
            return call(_raw_stream(device.index))
        with torch.cuda.device(device):
            return call(_raw_stream(device.index))
    if isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, device=device) if stream else
                  torch.cuda.default_stream(device))
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    with torch.cuda.stream(stream):   # (makes the stream's device current too)
        for x in inputs:
            if x is not None:
                x.record_stream(stream)
        return call(stream.cuda_stream)


def _device(t, what="weights are"):
    if not t.is_cuda:
        raise ValueError(f"{what} on {t.device}, not on a GPU")
    return t.device


class Decoded(NamedTuple):
    """One pass of :class:`MoeDecode`."""
    y: torch.Tensor        # [T, H]
    idx: torch.Tensor      # [T, k] int32, chosen experts
    gate: torch.Tensor     # [T, k] fp32
    logits: torch.Tensor   # [T, E] fp32


class MoeDecode:
    """The expert layer for a few tokens (serving), on parameters that stay
    where they are: those of a ``MoeLayer``, or of a loaded model.

    ``shape.T`` is the most tokens of a call (at most 128); ``shape.router``
    says whether the logits come from ``wg`` (and ``bias``) or with each call;
    ``shape.g0`` / ``shape.G`` is the window of experts that w13 and w2 hold."""

    def __init__(self, shape: LayerShape, w13, w2, wg=None, bias=None, ws13=None, ws2=None):
        s = self.s = shape
        if s.capacity is not None:
            raise ValueError("the few-token layer drops no pairs: capacity must be None")
        if s.router != (wg is not None):
            raise ValueError("wg comes with shape.router, and only with it")
        if bias is not None and wg is None:
            raise ValueError("bias comes with wg, and only with it")
        if s.shared != (ws13 is not None) or s.shared != (ws2 is not None):
            raise ValueError("ws13 and ws2 come with shape.shared, and only with it")
        dev = self.device = _device(w13)
        f32 = torch.float32
        self.dt = abi.dtype_code(w13)
        _check("w13", w13, s.dtype, dev, s.groups, 2 * s.I, s.H)
        _check("w2", w2, s.dtype, dev, s.groups, s.H, s.I)
        if wg is not None:
            _check("wg", wg, f32, dev, s.H, s.E)
        if bias is not None:
            _check("bias", bias, f32, dev, s.E)
        if ws13 is not None:
            _check("ws13", ws13, s.dtype, dev, 2 * s.I, s.H)
            _check("ws2", ws2, s.dtype, dev, s.H, s.I)
        self.w13, self.w2, self.wg, self.bias, self.ws13, self.ws2 = w13, w2, wg, bias, ws13, ws2
        self._ws_bytes = {}

    @classmethod
    def of_layer(cls, layer: "MoeLayer", max_tokens: int = 128) -> "MoeDecode":
        """On the parameters of a training layer."""
        from dataclasses import replace
        return cls(replace(layer.s, T=max_tokens, capacity=None), layer.w13, layer.w2,
                   wg=layer.wg, bias=layer.bias, ws13=layer.ws13, ws2=layer.ws2)

    def forward(self, x, residual=None, logits=None, out=None, stream=None) -> Decoded:
        """``x`` [T, H] -> :class:`Decoded`.  ``out``: y's buffer (the
        residual's will do; allocated if None).  Everything is enqueued on
        ``stream`` (None: the current one)."""
        s, dev = self.s, self.device
        T = x.shape[0]
        if T > s.T:
            raise ValueError(f"{T} tokens in a layer built for at most {s.T}")
        _check("x", x, s.dtype, dev, T, s.H)
        if residual is not None:
            _check("residual", residual, s.dtype, dev, T, s.H)
        if (logits is None) != s.router:
            raise ValueError("logits come with the call if, and only if, there is no router")
        if logits is not None:
            _check("logits", logits, torch.float32, dev, T, s.E)
        if out is not None:
            _check("out", out, s.dtype, dev, T, s.H)

        def call(st):
            n = self._ws_bytes.get(T)
            if n is None:
                n = abi.moe_decode_workspace_bytes(T, s.H, s.I, s.E, s.k, self.dt)
                self._ws_bytes[T] = n
            y = torch.empty_like(x) if out is None else out
            lg = x.new_empty((T, s.E), dtype=torch.float32) if logits is None else logits
            idx = x.new_empty((T, s.k), dtype=torch.int32)
            gate = x.new_empty((T, s.k), dtype=torch.float32)
            # a workspace per call, from the stream's own pool: calls on several
            # streams, or captured into several graphs, never share one
            ws = x.new_empty(n, dtype=torch.uint8)
            abi.moe_decode(x, self.dt, self.wg, self.bias, T, s.H, s.I, s.E, s.k, s.g0, s.groups,
                           self.w13, self.w2, self.ws13, self.ws2, residual, lg, idx, gate, y, ws,
                           n, st)
            return Decoded(y, idx, gate, lg)
        return _on(dev, stream, call, x, residual, logits, out, self.w13, self.w2, self.wg,
                   self.bias, self.ws13, self.ws2)


ACTS = {"none": abi.MOE_ACT_NONE, "relu": abi.MOE_ACT_RELU, "silu": abi.MOE_ACT_SILU,
        "gelu": abi.MOE_ACT_GELU, "gelu_tanh": abi.MOE_ACT_GELU_TANH}


class Linear:
    """``y = act(x W^T + bias) + residual`` on a weight W [N, K], and its
    gradients; ``bias`` is [N] fp32."""

    def __init__(self, w, bias=None, act: str = "none"):
        self.device = _device(w)
        if w.dim() != 2:
            raise ValueError(f"w has {w.dim()} dimensions, not 2")
        self.N, self.K = w.shape
        self.dt, self.dtype = abi.dtype_code(w), w.dtype
        _check("w", w, w.dtype, self.device, self.N, self.K)
        if bias is not None:
            _check("bias", bias, torch.float32, self.device, self.N)
        if act not in ACTS:
            raise ValueError(f"act {act!r} is none of {', '.join(ACTS)}")
        self.w, self.bias, self.act = w, bias, ACTS[act]
        self._ws_bytes = {}

    def forward(self, x, residual=None, save_z=False, out=None, stream=None):
        """``x`` [M, K] -> y [M, N], or (y, z) with ``save_z``.  ``out``: y's
        buffer (the residual's will do)."""
        M, dev = x.shape[0], self.device
        _check("x", x, self.dtype, dev, M, self.K)
        if residual is not None:
            _check("residual", residual, self.dtype, dev, M, self.N)
        if out is not None:
            _check("out", out, self.dtype, dev, M, self.N)

        def call(st):
            n = self._ws_bytes.get(M)
            if n is None:
                n = self._ws_bytes[M] = abi.moe_linear_workspace_bytes(M, self.N, self.K, self.dt)
            y = x.new_empty((M, self.N)) if out is None else out
            z = x.new_empty((M, self.N)) if save_z else None
            ws = x.new_empty(n, dtype=torch.uint8) if n else None
            abi.moe_linear(x, self.dt, M, self.N, self.K, self.w, self.bias, self.act, residual,
                           z, y, ws, n, st)
            return (y, z) if save_z else y
        return _on(dev, stream, call, x, residual, out, self.w, self.bias)

    def backward(self, dy, x, z=None, bias_grad=None, stream=None, x_grad=True, w_grad=True):
        """(dx, dw, db) of ``dy`` [M, N], the forward's ``x`` and the ``z`` it
        kept (None without an activation).  Each is computed, or None, as
        ``x_grad`` (a first layer needs none), ``w_grad`` (frozen weights) and
        ``bias_grad`` (by default: whether there is a bias) say.  The residual's
        gradient is dy."""
        M, dev = dy.shape[0], self.device
        _check("dy", dy, self.dtype, dev, M, self.N)
        _check("x", x, self.dtype, dev, M, self.K)
        if (z is None) != (self.act == abi.MOE_ACT_NONE):
            raise ValueError("z comes with an activation, and only with it")
        if z is not None:
            _check("z", z, self.dtype, dev, M, self.N)
        if bias_grad is None:
            bias_grad = self.bias is not None

        def call(st):
            dx = torch.empty_like(x) if x_grad else None
            dw = torch.empty_like(self.w) if w_grad else None
            db = x.new_empty(self.N, dtype=torch.float32) if bias_grad else None
            n = abi.moe_linear_bwd_workspace_bytes(M, self.N, self.K, self.dt, self.act)
            ws = x.new_empty(n, dtype=torch.uint8)
            abi.moe_linear_bwd(dy, z, x, self.w, self.dt, M, self.N, self.K, self.act, dx, dw, db,
                               ws, n, st)
            return dx, dw, db
        return _on(dev, stream, call, dy, x, z, self.w)


class Balance(NamedTuple):
    """The losses of :class:`BalanceLoss` and what its backward needs."""
    loss: torch.Tensor             # [3] fp32: balance, z, and their weighted sum
    counts: torch.Tensor           # [S, E] int32, choices of each expert
    tokens: torch.Tensor           # [S + 1] int32, tokens that count of each sequence, and of all
    prob: torch.Tensor             # [S, E] fp32, mean probabilities (a statistic)


class BalanceLoss:
    """``weight`` times the balance loss of a routing step and ``z_weight`` times
    its z loss (defined at ``moe_balance_loss`` in ``include/moe.h``), with
    per-expert counts, and their gradient together with the gates'.

    ``seq`` [S + 1] int32 are the ends of packed sequences (None: all tokens are
    one), ``keep`` [T] uint8 or bool says which tokens count (None: all)."""

    def __init__(self, weight: float = 0.01, z_weight: float = 0.0):
        self.weight, self.z_weight = float(weight), float(z_weight)
        self._ws_bytes = {}

    @staticmethod
    def _inputs(logits, idx, seq, keep):
        dev = _device(logits, "logits are")
        if logits.dim() != 2:
            raise ValueError(f"logits have {logits.dim()} dimensions, not 2")
        T, E = logits.shape
        of = {"beside": "logits are"}
        _check("logits", logits, torch.float32, dev, T, E)
        if idx.dim() != 2:
            raise ValueError(f"idx has {idx.dim()} dimensions, not 2")
        k = idx.shape[1]
        _check("idx", idx, torch.int32, dev, T, k, **of)
        S = 1
        if seq is not None:
            if seq.dim() != 1 or seq.shape[0] < 2:
                raise ValueError(f"seq has shape {tuple(seq.shape)}, not one of S + 1 >= 2 ends")
            S = seq.shape[0] - 1
            _check("seq", seq, torch.int32, dev, S + 1, **of)
        if keep is not None:
            _check("keep", keep, torch.bool if keep.dtype == torch.bool else torch.uint8, dev, T,
                   **of)
        return dev, T, E, k, S

    def forward(self, logits, idx, seq=None, keep=None, stream=None) -> Balance:
        """``logits`` [T, E] and the chosen ``idx`` [T, k] -> :class:`Balance`."""
        dev, T, E, k, S = self._inputs(logits, idx, seq, keep)

        def call(st):
            n = self._ws_bytes.get((T, E, k, S))
            if n is None:
                n = abi.moe_balance_loss_workspace_bytes(T, E, k, S)
                self._ws_bytes[T, E, k, S] = n
            loss, prob = logits.new_empty(3), logits.new_empty((S, E))
            counts, tokens = idx.new_empty((S, E)), idx.new_empty(S + 1)
            # a workspace per call, from the stream's own pool: calls on several
            # streams, or captured into several graphs, never share one
            ws = logits.new_empty(n, dtype=torch.uint8) if n else None
            abi.moe_balance_loss(logits, idx, keep, seq, T, E, k, S, self.weight, self.z_weight,
                                 loss, counts, tokens, prob, ws, n, st)
            return Balance(loss, counts, tokens, prob)
        return _on(dev, stream, call, logits, idx, seq, keep)

    def backward(self, logits, idx, counts, tokens, seq=None, keep=None, dgate=None, dloss=None,
                 out=None, stream=None):
        """dlogits [T, E] (into ``out``, if given) of ``dloss`` (one fp32 value;
        None: 1) times the weighted sum of the losses and, with ``dgate`` [T, k],
        of the gates too.  ``counts`` and ``tokens`` are the forward's."""
        dev, T, E, k, S = self._inputs(logits, idx, seq, keep)
        f32, of = torch.float32, {"beside": "logits are"}
        _check("counts", counts, torch.int32, dev, S, E, **of)
        _check("tokens", tokens, torch.int32, dev, S + 1, **of)
        if dgate is not None:
            _check("dgate", dgate, f32, dev, T, k, **of)
        if dloss is not None:
            if dloss.numel() != 1:
                raise ValueError(f"dloss has {dloss.numel()} values, not 1")
            _check("dloss", dloss, f32, dev, *dloss.shape, **of)
        if out is not None:
            _check("out", out, f32, dev, T, E, **of)

        def call(st):
            dlogits = torch.empty_like(logits) if out is None else out
            abi.moe_balance_loss_bwd(logits, idx, dgate, keep, seq, counts, tokens, T, E, k, S,
                                     self.weight, self.z_weight, dloss, dlogits, st)
            return dlogits
        return _on(dev, stream, call, logits, idx, counts, tokens, seq, keep, dgate, dloss, out)


NORMS = {"layer": abi.MOE_NORM_LAYER, "rms": abi.MOE_NORM_RMS}


class Normed(NamedTuple):
    """One pass of :class:`Norm`."""
    y: torch.Tensor                # [M, H]
    h: torch.Tensor                # [M, H], x + residual (x itself without a residual)
    mean: Optional[torch.Tensor]   # [M] fp32, with ``save`` and of a layer norm
    rstd: Optional[torch.Tensor]   # [M] fp32, with ``save``


class Norm:
    """Layer norm (``kind="layer"``) or RMS norm (``"rms"``) of rows, with an
    optional residual sum in front, and its gradients; ``w`` and ``bias`` are
    [H] fp32."""

    def __init__(self, w, bias=None, kind: str = "layer", eps: float = 1e-5):
        self.device = _device(w)
        if w.dim() != 1:
            raise ValueError(f"w has {w.dim()} dimensions, not 1")
        self.H = w.shape[0]
        _check("w", w, torch.float32, self.device, self.H)
        if bias is not None:
            _check("bias", bias, torch.float32, self.device, self.H)
        if kind not in NORMS:
            raise ValueError(f"kind {kind!r} is none of {', '.join(NORMS)}")
        if not 0.0 < eps < float("inf"):
            raise ValueError(f"eps {eps} is not positive and finite")
        self.w, self.bias, self.kind, self.eps = w, bias, NORMS[kind], float(eps)
        self._ws_bytes = {}

    def _rows(self, x):
        if x.dim() != 2:
            raise ValueError(f"x has {x.dim()} dimensions, not 2")
        dt = abi.dtype_code(x)
        _check("x", x, x.dtype, self.device, x.shape[0], self.H)
        return dt, x.shape[0]

    def forward(self, x, residual=None, save=False, out=None, h_out=None, stream=None) -> Normed:
        """``x`` [M, H] -> :class:`Normed`; ``save``: with the statistics that the
        backward needs.  ``out``: y's buffer; ``h_out``: that of x + residual (the
        residual's will do, or x's)."""
        dt, M = self._rows(x)
        H, dev = self.H, self.device
        for name, t in (("residual", residual), ("out", out), ("h_out", h_out)):
            if t is not None:
                _check(name, t, x.dtype, dev, M, H)
        if h_out is not None and residual is None:
            raise ValueError("h_out comes with a residual, and only with it")

        def call(st):
            y = torch.empty_like(x) if out is None else out
            h = None if residual is None else torch.empty_like(x) if h_out is None else h_out
            rstd = self.w.new_empty(M) if save else None
            mean = self.w.new_empty(M) if save and self.kind == abi.MOE_NORM_LAYER else None
            abi.moe_norm(x, residual, dt, M, H, self.kind, self.eps, self.w, self.bias, h, y, mean,
                         rstd, st)
            return Normed(y, x if h is None else h, mean, rstd)
        return _on(dev, stream, call, x, residual, out, h_out, self.w, self.bias)

    def backward(self, dy, h, rstd, mean=None, dh=None, x_grad=True, w_grad=True, bias_grad=None,
                 out=None, stream=None):
        """(dx, dw, db) of ``dy`` [M, H], the forward's ``h``, ``rstd`` and ``mean``
        (None for RMS); ``dh``: the gradient that reaches h besides, added to dx,
        which is that of x and of the residual.  Each is computed, or None, as
        ``x_grad``, ``w_grad`` and ``bias_grad`` (by default: whether there is a
        bias) say.  ``out``: dx's buffer (dh's will do)."""
        dt, M = self._rows(h)
        H, dev, f32 = self.H, self.device, torch.float32
        for name, t in (("dy", dy), ("dh", dh), ("out", out)):
            if t is not None:
                _check(name, t, h.dtype, dev, M, H)
        if rstd is None:
            raise ValueError("no rstd: it comes from a forward with save")
        _check("rstd", rstd, f32, dev, M)
        if (mean is None) != (self.kind == abi.MOE_NORM_RMS):
            raise ValueError("mean comes with a layer norm, and only with it")
        if mean is not None:
            _check("mean", mean, f32, dev, M)
        if bias_grad is None:
            bias_grad = self.bias is not None

        def call(st):
            dx = None if not x_grad else torch.empty_like(h) if out is None else out
            dw = torch.empty_like(self.w) if w_grad else None
            db = torch.empty_like(self.w) if bias_grad else None
            n = 0
            if w_grad or bias_grad:
                n = self._ws_bytes.get((M, dt))
                if n is None:
                    n = self._ws_bytes[M, dt] = abi.moe_norm_bwd_workspace_bytes(M, H, dt)
            ws = h.new_empty(n, dtype=torch.uint8) if n else None
            abi.moe_norm_bwd(dy, h, dh, dt, M, H, self.kind, self.w, mean, rstd, dx, dw, db, ws, n,
                             st)
            return dx, dw, db
        return _on(dev, stream, call, dy, h, rstd, mean, dh, out, self.w)


GRAD_NORMS = {"l2": abi.MOE_GRAD_L2, "max": abi.MOE_GRAD_MAX}


class GradClip:
    """The norm of ``grads`` together (``kind``: ``"l2"``, the root of the sum of
    all squares, or ``"max"``, the largest magnitude) and clipping by it.

    ``grads`` are dense tensors of any shapes, fp32 or bf16, on one GPU; ``outs``:
    where the clipped ones go, of the same sizes and of the same type or fp32
    (None: in place).  The tensors stay the caller's and keep their sizes and
    types; each call takes their present contents, and their addresses as they are
    then.  Making one looks at every tensor (about 8 us for four, 1.1 ms for 700):
    where gradients keep their buffers, keep it from step to step."""

    def __init__(self, grads, outs=None, kind: str = "l2"):
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        if not self.grads:
            raise ValueError("no gradients")
        if len(self.outs) != len(self.grads):
            raise ValueError(f"{len(self.outs)} outs for {len(self.grads)} gradients")
        if kind not in GRAD_NORMS:
            raise ValueError(f"kind {kind!r} is none of {', '.join(GRAD_NORMS)}")
        self.kind = GRAD_NORMS[kind]
        self.device = _device(self.grads[0], "gradients are")
        self._tensors = self.grads if outs is None else self.grads + self.outs
        of = {"beside": "the first gradient is"}
        for i, (g, o) in enumerate(zip(self.grads, self.outs)):
            abi.dtype_code(g)
            _check(f"gradient {i}", g, g.dtype, self.device, *g.shape, **of)
            if o is not g:
                _check(f"out {i}", o, o.dtype if o.dtype == torch.float32 else g.dtype, self.device,
                       *g.shape, **of)
        self._lay_out()

    def _lay_out(self):
        self._at = list(map(torch.Tensor.data_ptr, self._tensors))
        self._arr = abi.grads(self.grads, self.outs)
        self._ws_bytes = abi.moe_grad_norm_workspace_bytes(self._arr, len(self.grads))

    def _array(self):
        if list(map(torch.Tensor.data_ptr, self._tensors)) != self._at:   # (storage was replaced)
            self.__init__(self.grads, None if self.outs is self.grads else self.outs,
                          {v: k for k, v in GRAD_NORMS.items()}[self.kind])
        return self._arr

    def norm(self, each=False, total=False, stream=None):
        """The norm (fp32, no dimensions), with ``each`` also those of the
        gradients one by one [n], with ``total`` also the sum of all squares in
        64 bits (the maximum): what ranks that hold parts of a model reduce."""
        arr, dev, n = self._array(), self.device, len(self.grads)

        def call(st):
            norm = torch.empty((), dtype=torch.float32, device=dev)
            norms = torch.empty(n, dtype=torch.float32, device=dev) if each else None
            whole = torch.empty((), dtype=torch.float64, device=dev) if total else None
            ws = torch.empty(self._ws_bytes, dtype=torch.uint8, device=dev)
            abi.moe_grad_norm(arr, n, self.kind, norm, norms, whole, ws, self._ws_bytes, st)
            more = tuple(t for t in (norms, whole) if t is not None)
            return (norm, *more) if more else norm
        return _on(dev, stream, call, *self.grads)

    def clip(self, max_norm: float, norm=None, stream=None):
        """Scales the gradients by min(1, max_norm / (norm + 1e-6)), not at all with an
        infinite ``max_norm``; returns the norm.  ``norm``: one fp32 value to take
        instead of the gradients' own."""
        arr, dev, n = self._array(), self.device, len(self.grads)
        if norm is not None:
            if norm.numel() != 1:
                raise ValueError(f"norm has {norm.numel()} values, not 1")
            _check("norm", norm, torch.float32, dev, *norm.shape, beside="the gradients are")

        def call(st):
            if norm is not None:
                abi.moe_grad_clip(arr, n, norm, max_norm, st)
                return norm
            own = torch.empty((), dtype=torch.float32, device=dev)
            ws = torch.empty(self._ws_bytes, dtype=torch.uint8, device=dev)
            abi.moe_grad_norm_clip(arr, n, self.kind, max_norm, own, None, ws, self._ws_bytes, st)
            return own
        return _on(dev, stream, call, norm, *self._tensors)
