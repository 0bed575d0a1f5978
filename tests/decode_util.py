"""The few-token layer and the fused linear product in 64 bits, with a bound
on what their fp32 arithmetic may be off, derived term by term:

* a sum of n fp32 products: at most (n + 2) u of the sum of their magnitudes,
  u = 2^-24, whatever the order;
* the activations: their exp and reciprocal are a few ulp off, and the
  argument of the exp is rounded, so at most ACT (1 + |z|) of the value;
* a value kept as two bf16 (each off by at most half its step, 2^-8): 2^-16;
* storage: half a step, ``torch.finfo(t).eps / 2`` of the value.
"""
from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -24
ACT = 16 * U


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().double().cpu()


def ref_logits(x, wg, bias):
    """Exact logits (64 bits) of device tensors."""
    full = f64(x) @ f64(wg)
    return full if bias is None else full + f64(bias)


def ref_route(logits, k):
    """idx by (logit descending, index ascending) and softmax gates, of fp32
    logits; a row without a finite logit has gates of zero."""
    rows = logits.tolist()
    idx = torch.tensor([sorted(range(len(r)), key=lambda e: (-r[e], e))[:k] for r in rows],
                       dtype=torch.int64).reshape(len(rows), k)
    lg = logits.double()
    m = lg.amax(dim=1, keepdim=True)
    p = torch.exp(lg - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    s = p.sum(dim=1, keepdim=True)
    gate = torch.where(s > 0, p / s, torch.zeros_like(p)).gather(1, idx)
    # the exponent's argument and value, the sum over a lane's experts and the wave
    spread = torch.where(torch.isfinite(m - lg), m - lg, torch.zeros_like(lg)).gather(1, idx)
    return idx, gate, gate * U * (spread + 40)


def ref_ffn(x, w13, w2, planes):
    """(value, bound) of one expert on rows x, all in 64 bits; planes: the
    activations are kept as two bf16 (else in fp32)."""
    H, I = w13.shape[1], w2.shape[1]
    h = x @ w13.T
    dh = (H + 2) * U * (x.abs() @ w13.abs().T)
    g, u, dg, du = h[:, :I], h[:, I:], dh[:, :I], dh[:, I:]
    s = g * torch.sigmoid(g)
    a = s * u
    # |silu'| <= 1.1
    da = 1.1 * dg * (u.abs() + du) + s.abs() * du + ACT * (1 + g.abs()) * a.abs()
    da = da + (2.0 ** -16 if planes else U) * (a.abs() + da)
    y = a @ w2.T
    n = 2 * I if planes else I
    return y, da @ w2.abs().T + (n + 2) * U * ((a.abs() + da) @ w2.abs().T)


def ref_decode(x, idx, gate, dgate, g0, G, w13, w2, ws13, ws2, residual, dtype):
    """(y, bound) of the layer from its choices, on device tensors."""
    planes = dtype == torch.bfloat16
    xx = f64(x)
    y = torch.zeros_like(xx)
    b = torch.zeros_like(xx)
    mag = torch.zeros_like(xx)
    for e in sorted(set(idx.flatten().tolist())):
        if not g0 <= e < g0 + G:
            continue
        t, j = torch.nonzero(idx == e, as_tuple=True)
        v, dv = ref_ffn(xx[t], f64(w13[e - g0]), f64(w2[e - g0]), planes)
        gt, dg = gate[t, j, None], dgate[t, j, None]
        y[t] += gt * v
        b[t] += (gt + dg) * dv + dg * v.abs()
        mag[t] += gt * v.abs()
    terms = idx.shape[1]
    if ws13 is not None:
        v, dv = ref_ffn(xx, f64(ws13), f64(ws2), planes)
        y, b, mag, terms = y + v, b + dv, mag + v.abs(), terms + 1
    if residual is not None:
        y, mag, terms = y + f64(residual), mag + f64(residual).abs(), terms + 1
    b = b + (terms + 2) * U * (mag + b)
    return y, b + half_step(dtype) * (y.abs() + b)


def ref_act(z, act):
    """(value, slope, slope of the slope's bound) of an activation at z, 64 bits."""
    if act == "relu":
        return torch.where(z > 0, z, 0 * z), (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        c = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        a, q = math.sqrt(2 / math.pi), 0.044715
        t = torch.tanh(a * (z + q * z ** 3))
        return z / 2 * (1 + t), (1 + t) / 2 + z / 2 * (1 - t * t) * a * (1 + 3 * q * z * z)
    return z, torch.ones_like(z)


def ref_linear(x, w, bias, act, residual, dtype):
    """((y, bound), (z, bound)) of the fused product, on device tensors."""
    xx, ww = f64(x), f64(w)
    z = xx @ ww.T
    mag = xx.abs() @ ww.abs().T
    if bias is not None:
        z, mag = z + f64(bias), mag + f64(bias).abs()
    dz = (x.shape[1] + 3) * U * mag
    v = ref_act(z, act)[0]
    # every activation's slope is below 1.13; the tanh form's argument is a
    # cubic, so its exp's argument grows as z^3 until the value saturates
    dv = 1.13 * dz + ACT * (1 + z.abs() + (z.abs().clamp(max=6) ** 3 if act == "gelu_tanh" else 0)) \
        * (v.abs() + dz) * (act not in ("none", "relu"))
    y = v
    if residual is not None:
        y = v + f64(residual)
        dv = dv + U * (y.abs() + dv)
    h = half_step(dtype)
    return (y, dv + h * (y.abs() + dv)), (z, dz + h * (z.abs() + dz))


def ref_linear_bwd(dy, z, x, w, act, dtype):
    """((dx, bound), (dw, bound), (db, bound)) of the gradients."""
    d = f64(dy)
    M, N = d.shape
    K = x.shape[1]
    if act == "none":
        dz, e32 = d, torch.zeros_like(d)
    else:
        zz = f64(z)
        slope = ref_act(zz, act)[1]
        dz = d * slope
        # the slopes are sums of terms of at most about 1 + |z| each
        e32 = d.abs() * ACT * (1 + zz.abs().clamp(max=40)) ** 2 * (act != "relu") + U * dz.abs()
    r = half_step(dtype) if act != "none" else 0.0
    ed = e32 + r * (dz.abs() + e32)
    xx, ww = f64(x), f64(w)
    h = half_step(dtype)

    def product(a, ea, b, n):
        v = a @ b
        e = ea @ b.abs() + (n + 2) * U * ((a.abs() + ea) @ b.abs())
        return v, e + h * (v.abs() + e)

    db = dz.sum(dim=0)
    eb = e32.sum(dim=0) + (M + 2) * U * (dz.abs() + e32).sum(dim=0) + U * db.abs()
    return product(dz, ed, ww, N), product(dz.T, ed.T, xx, M), (db, eb)


def assert_within(name, got, ref):
    """Every element within its own bound."""
    v, b = ref
    g = f64(got)
    assert g.shape == v.shape, (name, g.shape, v.shape)
    over = (g - v).abs() - b
    bad = ~(over <= 0)
    if bad.any():
        at = np.unravel_index(int(torch.argmax(torch.nan_to_num(over, nan=math.inf))), v.shape)
        raise AssertionError(f"{name}: {int(bad.sum())} of {v.numel()} values out of bounds, the "
                             f"worst at {at}: {g[at].item()} for {v[at].item()} +- {b[at].item()}")
