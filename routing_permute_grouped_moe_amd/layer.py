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
                 recompute: bool = False):
        s = self.s = shape
        self.overlap = overlap
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


# ---------------------------------------------------------------------- checked calls
def _check(name, t, dtype, device, *shape):
    """A tensor the kernels can read as it lies: dense, of this shape, type and device."""
    if (t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, not {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the weights are on {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    raise ValueError(f"{name} is not contiguous")


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(device, stream, call, *inputs):
    """call(raw stream) with the device of a call's tensors current, and the
    given stream too (None: the device's current one), so that outputs and
    workspaces allocated inside belong to it; the inputs and weights, which may
    not, are kept from reuse until the stream has passed."""
    if stream is None:
        if torch.cuda.current_device() == device.index:
            return call(_raw_stream(device.index))
        with torch.cuda.device(device):
            return call(_raw_stream(device.index))
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the weights are on {device}")
    with torch.cuda.stream(stream):   # (makes the stream's device current too)
        for x in inputs:
            if x is not None:
                x.record_stream(stream)
        return call(stream.cuda_stream)


def _device(t):
    if not t.is_cuda:
        raise ValueError(f"weights are on {t.device}, not on a GPU")
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
