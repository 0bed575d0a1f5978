"""The row norms, the router's losses and gradient clipping in 64 bits, with a
bound on what their fp32 arithmetic may be off, derived term by term (u = 2^-24):

* an fp32 sum whose longest chain has D additions: D u of the sum of magnitudes.
  A lane adds at most 1/64 of a row (or 8 values of a shorter one) before lanes
  and waves are joined, so D = H / 64 + 24 over a row;
* an exp is off by its argument's rounding (u times the argument) and 2 u; a
  reciprocal, a root or a log by 2 u;
* storage: half a step, ``torch.finfo(t).eps / 2`` of the value.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
EPS = {"layer": 1e-5, "rms": 1e-6}


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().double()


def assert_within(name, got, ref):
    want, bound = ref
    got = f64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    off = (got - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        at = tuple(int(i) for i in torch.nonzero(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} values out of bound, first at "
                             f"{at}: {got[at].item()} for {want[at].item()}, bound {bound[at].item()}")


# ---------------------------------------------------------------- norm

def ref_norm(h, w, b, kind, dtype):
    """{name: (value, bound)} of the norm of the stored rows h."""
    h, w = f64(h), f64(w)[None]
    H = h.shape[1]
    D = H / 64 + 24
    mean = h.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(h[:, :1])
    d = h - mean
    var = (d * d).mean(1, keepdim=True)
    if kind == "layer":
        # a first mean off by e; where it is beyond twice the deviations (5: or near), their
        # mean from it is added to it
        e = (D + 2) * U * h.abs().mean(1, keepdim=True)
        ad = d.abs().mean(1, keepdim=True)
        far = mean * mean > 5 * var
        dm = torch.where(far, 1.01 * U * mean.abs() + (D + 4) * U * (ad + e), e)
        dv = (D + 8) * U * (var + e * e) + torch.where(
            far, 2 * e * (D + 4) * U * (ad + e) + 1.01 * dm * dm, 2 * ad * e + e * e)
    else:
        dm, dv = 0.0 * mean, (D + 5) * U * var
    rstd = 1 / torch.sqrt(var + EPS[kind])
    rel = 0.5 * dv / (var + EPS[kind]) + 5 * U
    rel = rel + rel * rel * 2                       # (the root's second order)
    y = d * rstd * w
    by = y.abs() * (rel + 5 * U) + (rstd * w).abs() * (1 + rel) * (dm + U * d.abs())
    if b is not None:
        y = y + f64(b)[None]
        by = by + U * y.abs()
    by = by + half_step(dtype) * (y.abs() + by) * 1.01
    return {"y": (y, by), "mean": (mean[:, 0], dm[:, 0] + 0 * mean[:, 0]),
            "rstd": (rstd[:, 0], (rel * rstd)[:, 0])}


def ref_norm_bwd(dy, h, w, mean, rstd, dh, kind, dtype):
    """(dx, dw, db), each (value, bound), with the statistics that the call is given."""
    dy, h, w, rstd = f64(dy), f64(h), f64(w)[None], f64(rstd)[:, None]
    M, H = h.shape
    D, Dm = H / 64 + 24, M / 64 + 64
    q = (h - (f64(mean)[:, None] if kind == "layer" else 0.0)) * rstd
    dq = 2.01 * U * q.abs()
    g = dy * w
    s2 = (g * q).mean(1, keepdim=True)
    d2 = (D + 6) * U * (g * q).abs().mean(1, keepdim=True)
    s1 = g.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(s2)
    d1 = (D + 3) * U * g.abs().mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(s2)
    dx = rstd * (g - s1 - q * s2)
    mag = g.abs() + s1.abs() + (q * s2).abs()
    bx = rstd * (5 * U * mag + d1 + (q.abs() + dq) * d2 + dq * s2.abs())
    if dh is not None:
        dx = dx + f64(dh)
        bx = bx + U * dx.abs()
    bx = bx + half_step(dtype) * (dx.abs() + bx) * 1.01
    dw, db = (dy * q).sum(0), dy.sum(0)
    bw = (Dm + 5) * U * (dy * q).abs().sum(0)
    bb = (Dm + 1) * U * dy.abs().sum(0)
    return (dx, bx), (dw, bw), (db, bb)


# ---------------------------------------------------------------- losses of the router

def ref_rows(z, arg=1.0):
    """(p, lse, rel. bound of p, bound of lse, whether a logit is not -inf) of fp32 logits.

    ``arg``: roundings of the exp's argument: 1, the difference to the maximum; 2.4
    where it is taken as exp2 of the difference times log2 e, for the product is
    rounded too and the constant off by 0.4 u.  A log is off by 3 u: log2's own, and
    the product's, and the constant's."""
    z = f64(z)
    live = (z != -float("inf")).any(1)
    zz = torch.where(live[:, None], z, torch.zeros_like(z))
    m = zz.amax(1, keepdim=True)
    spread = torch.where(zz > -float("inf"), m - zz, torch.zeros_like(zz))
    p = torch.softmax(zz, 1)
    D = z.shape[1] / 64 + 12
    drift = ((arg * spread + 3) * p).sum(1, keepdim=True) + D
    rel = (arg * spread + 6 + drift) * U
    lse = torch.logsumexp(zz, 1)
    dl = drift[:, 0] * U + 3 * U * (lse - m[:, 0]).abs() + U * lse.abs() + U
    return p * live[:, None], lse * live, rel, dl, live


def ref_members(T, seq, keep, live, S):
    """[S, T] bool: the tokens of each sequence that count."""
    t = torch.arange(T, device=live.device)
    used = live if keep is None else live & (keep != 0)
    if seq is None:
        return used[None]
    return (t >= seq[:-1, None]) & (t < seq[1:, None]) & used


def ref_balance(z, idx, seq, keep, weight, z_weight):
    """{name: (value, bound)} of the forward; counts and tokens are exact."""
    T, E = z.shape
    k = idx.shape[1]
    S = 1 if seq is None else seq.shape[0] - 1
    p, lse, rel, dl, live = ref_rows(z, 2.4)
    of = ref_members(T, seq, keep, live, S).double()
    n = of.sum(1)
    N = max(1.0, n.sum().item())
    hot = torch.zeros_like(p)
    for j in range(k):
        hot.scatter_add_(1, idx[:, j:j + 1].long(), torch.ones_like(hot[:, :1]))
    counts = of @ hot
    some = n.clamp(min=1)[:, None]
    P = (of @ p) / some
    # a wave adds at most 256 tokens before the waves of a block are joined; then 64 bits
    dP = (of @ (p * rel)) / some + 270 * U * P + 1e-37
    frac = counts * E / (k * some)
    lb = (n[:, None] * frac * P).sum() / N
    db = (n[:, None] * frac * dP).sum() / N + U * lb
    used = of.sum(0)
    lz = (used * lse * lse).sum() / N
    dz = (used * (2 * lse.abs() + dl) * dl).sum() / N + U * lz
    tot = weight * lb + z_weight * lz
    dt = abs(weight) * db + abs(z_weight) * dz + 3 * U * (abs(weight) * lb + abs(z_weight) * lz)
    return {"loss": (torch.stack([lb, lz, tot]), torch.stack([db, dz, dt])),
            "counts": counts, "tokens": torch.cat([n, n.sum()[None]]), "prob": (P, dP)}


def ref_balance_bwd(z, idx, seq, keep, weight, z_weight, dloss, dgate):
    T, E = z.shape
    k = idx.shape[1]
    S = 1 if seq is None else seq.shape[0] - 1
    p, lse, rel, dl, live = ref_rows(z)
    of = ref_members(T, seq, keep, live, S).double()
    n = of.sum(1)
    N = max(1.0, n.sum().item())
    hot = torch.zeros_like(p)
    for j in range(k):
        hot.scatter_add_(1, idx[:, j:j + 1].long(), torch.ones_like(hot[:, :1]))
    frac = (of @ hot) * E / (k * n.clamp(min=1)[:, None])
    g = (of.t() @ frac) * (weight * dloss / N)
    dg = 9 * U * g.abs()
    if dgate is not None:
        for j in range(k):
            g = g.scatter_add(1, idx[:, j:j + 1].long(), f64(dgate[:, j:j + 1]))
        dg = dg + 2 * U * g.abs()
    add = (of.sum(0) * lse * (2 * z_weight * dloss / N))[:, None]
    dadd = (of.sum(0) * (dl + 6 * U * lse.abs()) * abs(2 * z_weight * dloss / N))[:, None]
    acc = (p * g).sum(1, keepdim=True)
    dacc = (p * (g.abs() * (rel + (E / 64 + 12) * U) + dg)).sum(1, keepdim=True)
    out = p * (g - acc + add)
    bound = (out.abs() * (rel + 3 * U)
             + p * (1 + rel) * (dg + dacc + dadd + 4 * U * (g.abs() + acc.abs() + add.abs())) + 1e-37)
    return out, bound


# ---------------------------------------------------------------- clipping

def ref_norms(grads, kind):
    """(norm, norms) in 64 bits, without overflow of a square."""
    flat = [f64(g).flatten() for g in grads]
    if kind == "max":
        each = [g.abs().max() if g.numel() else torch.zeros((), dtype=torch.float64, device=g.device)
                for g in flat]
        return torch.stack(each).max(), torch.stack(each)
    each = torch.stack([(g * g).sum() for g in flat])
    return each.sum().sqrt(), each.sqrt()


def ref_clip(g, norm, max_norm, dtype):
    """(value, bound) of a clipped gradient of fp32 norm ``norm``: the sum, the
    quotient, the product and its storage are each rounded once."""
    c = min(1.0, max_norm / (float(norm) + 1e-6))
    v = f64(g) * c
    return v, v.abs() * (4 * U + half_step(dtype)) + 2.0 ** -133
