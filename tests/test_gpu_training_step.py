"""A training step around the expert layer: norm with the residual in front, the
layer with its router's losses, the backward of both, and clipping of all
gradients, against 64-bit autograd of the same formulas (GPU only)."""
import pytest
import torch

import synth
from gpu_util import have_gpu, make_layer, rel_err, host
from training_util import assert_within, ref_balance_bwd

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

F32 = torch.float32
A, B = 0.3, 0.02


class Step:
    """x, residual -> h = x + residual, y = layer(norm(h)) and, from dy and the
    gradient dh of the residual stream, every gradient, clipped."""

    def __init__(self, name="tiny", overlap=False, limit=0.5):
        from routing_permute_grouped_moe_amd.layer import BalanceLoss, Norm
        cfg = self.cfg = synth.get_config(name)
        self.L = make_layer(cfg, synth.make_inputs(cfg), overlap=overlap)
        self.L.balance = BalanceLoss(A, B)
        T, H, E = cfg.T, cfg.H, cfg.E
        gen = torch.Generator(device="cuda").manual_seed(12)
        n = lambda *s, std=1.0, d=F32: torch.empty(s, dtype=d, device="cuda").normal_(0, std, generator=gen)
        dt = self.L.x.dtype
        self.x, self.res, self.dh = n(T, H, d=dt), n(T, H, d=dt), n(T, H, d=dt)
        self.norm = Norm(1 + n(H, std=0.2), bias=n(H, std=0.2))
        cuts = sorted(torch.randint(0, T, (3,), generator=gen, device="cuda").tolist())
        self.L.seq = torch.tensor([0, *cuts, T - 5], dtype=torch.int32, device="cuda")
        self.L.keep = (torch.rand(T, generator=gen, device="cuda") < 0.9).to(torch.uint8)
        self.dw, self.db = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
        self.limit = limit

    def run(self):
        from routing_permute_grouped_moe_amd.layer import GradClip
        L = self.L
        r = self.norm.forward(self.x, residual=self.res, save=True, out=L.x)
        L.forward()
        L.backward()
        dx, dw, db = self.norm.backward(L.dx, r.h, r.rstd, mean=r.mean, dh=self.dh)
        grads = [dw, db] + L.grads()
        total = GradClip(grads).clip(self.limit)
        return [r.h, L.y, L.losses.loss, L.losses.counts, dx, total] + grads


def test_against_autograd():
    s = Step()
    cfg, L = s.cfg, s.L
    out = s.run()
    h, y, loss, counts, dx, total = out[:6]
    d = lambda t: t.detach().double().cpu()
    leaf = lambda t: d(t).requires_grad_()
    x, w, b = leaf(s.x), leaf(s.norm.w), leaf(s.norm.bias)
    wg, w13, w2 = leaf(L.wg), leaf(L.w13), leaf(L.w2)
    params = [w, b, w13, w2, wg]
    hh = x + d(s.res)
    v = hh - hh.mean(1, keepdim=True)
    n = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-5) * w + b
    z = n @ wg
    if L.bias is not None:
        bias = leaf(L.bias)
        params.append(bias)
        z = z + bias
    idx = L.idx.long().cpu()          # (the choice is the layer's: tests of its own hold it)
    p = torch.softmax(z, 1)
    gate = p.gather(1, idx)
    yy = torch.zeros_like(hh)
    I = cfg.I
    for e in range(cfg.E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        a = n[t] @ w13[e].T
        a = torch.nn.functional.silu(a[:, :I]) * a[:, I:]
        yy = yy.index_add(0, t, gate[t, j, None] * (a @ w2[e].T))
    seq, keep = L.seq.cpu().tolist(), L.keep.cpu()
    bal, zl, N = 0.0, 0.0, 0
    for lo, hi in zip(seq, seq[1:]):
        rows = torch.nonzero(keep[lo:hi]).flatten() + lo
        if not len(rows):
            continue
        c = torch.bincount(idx[rows].flatten(), minlength=cfg.E)
        bal = bal + len(rows) * (c * cfg.E / (cfg.k * len(rows)) * p[rows].mean(0)).sum()
        zl = zl + (torch.logsumexp(z[rows], 1) ** 2).sum()
        N += len(rows)
    want_loss = torch.stack([bal / N, zl / N, A * bal / N + B * zl / N])
    ((yy * d(L.dy)).sum() + want_loss[2] + (hh * d(s.dh)).sum()).backward()
    tol = 1e-5                        # of the largest value, as the layer's fp32 outputs have it
    assert rel_err(host(h), hh.detach().numpy()) < tol
    assert rel_err(host(y), yy.detach().numpy()) < tol
    assert rel_err(host(loss), want_loss.detach().numpy()) < tol
    assert rel_err(host(dx), x.grad.numpy()) < tol
    grads = [t.grad for t in params]
    norm = torch.sqrt(sum((g * g).sum() for g in grads)).item()
    assert abs(total.item() - norm) <= tol * norm and norm > s.limit
    got = out[6:]
    assert len(got) == len(grads)
    for g, q in zip(got, grads):
        assert rel_err(host(g), q.numpy() * (s.limit / (norm + 1e-6))) < 2 * tol


@pytest.mark.parametrize("overlap", [False, True])
def test_step_replays_from_a_graph(overlap):
    s = Step("small", overlap)
    want = [t.clone() for t in s.run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = s.run()
    junk = torch.randn(1 << 18, device="cuda")
    for _ in range(3):
        for t in outs:
            t.fill_(-3)
        junk.mul_(1.01).sum().item()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), i


def test_the_layer_without_losses_is_as_it_was():
    """Weights of zero: every output and gradient has the layer's own bits."""
    from routing_permute_grouped_moe_amd.layer import BalanceLoss
    cfg = synth.get_config("tiny")
    inp = synth.make_inputs(cfg)
    one, two = make_layer(cfg, inp), make_layer(cfg, inp)
    two.balance = BalanceLoss(0.0, 0.0)
    one.step()
    two.step()
    for a, b in zip([one.y, one.dx, one.dlogits] + one.grads(), [two.y, two.dx, two.dlogits] + two.grads()):
        assert torch.equal(a, b)
    assert torch.equal(two.losses.counts[0], two.counts)


def test_the_layers_own_clipping():
    cfg = synth.get_config("tiny")
    L = make_layer(cfg, synth.make_inputs(cfg))
    L.step()
    before = [g.double().clone() for g in L.grads()]
    norm = L.clip_grads(0.25)
    want = torch.sqrt(sum((g * g).sum() for g in before))
    assert abs(norm.double() - want) <= 2.0 ** -23 * want
    for g, b in zip(L.grads(), before):
        assert torch.allclose(g.double(), b * (0.25 / (norm.double() + 1e-6)), rtol=2.0 ** -21, atol=1e-30)


def test_backward_before_forward_is_refused():
    from routing_permute_grouped_moe_amd.layer import BalanceLoss
    cfg = synth.get_config("tiny")
    L = make_layer(cfg, synth.make_inputs(cfg))
    L.balance = BalanceLoss()
    with pytest.raises(RuntimeError, match="before their forward"):
        L.route_bwd()


@pytest.mark.parametrize("how", ["recompute", "capacity", "overlap", "given logits"])
def test_layer_variants_with_losses(how):
    """The layer's dlogits are its gates' gradient and the losses' in one, whatever the
    experts do."""
    from routing_permute_grouped_moe_amd.layer import BalanceLoss
    cfg = synth.get_config("stress" if how == "given logits" else "small")
    kw = {"recompute": dict(recompute=True), "overlap": dict(overlap=True),
          "capacity": dict(capacity=300)}.get(how, {})
    L = make_layer(cfg, synth.make_inputs(cfg), **kw)
    L.balance = BalanceLoss(0.5, 0.01)
    L.step()
    torch.cuda.synchronize()
    one = L.balance.backward(L.logits, L.idx, L.losses.counts, L.losses.tokens, dgate=L.dgate)
    assert torch.equal(one, L.dlogits)
    assert_within("dlogits", L.dlogits, ref_balance_bwd(L.logits, L.idx, None, None, 0.5, 0.01, 1.0,
                                                        L.dgate))
    assert torch.equal(L.losses.counts[0], L.counts)


@pytest.mark.parametrize("null", [False, True])
def test_layer_on_a_raw_stream(null):
    """The layer's calls take a stream's handle; with losses and clipping they do too."""
    from routing_permute_grouped_moe_amd.layer import BalanceLoss
    cfg = synth.get_config("tiny")
    inp = synth.make_inputs(cfg)
    one, two = make_layer(cfg, inp), make_layer(cfg, inp)
    one.balance = two.balance = BalanceLoss(0.5, 0.01)
    side = torch.cuda.Stream()
    handle = 0 if null else side.cuda_stream
    torch.cuda.synchronize()
    one.step()
    a = one.clip_grads(0.25)
    two.step(handle)
    b = two.clip_grads(0.25, stream=handle)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    for u, v in zip([one.y, one.dlogits, one.losses.loss] + one.grads(),
                    [two.y, two.dlogits, two.losses.loss] + two.grads()):
        assert torch.equal(u, v)


@pytest.mark.parametrize("later", ["seq of as many", "seq of more", "keep", "both gone"])
@pytest.mark.parametrize("overlap", [False, True])
def test_the_backward_is_of_the_batch_that_the_forward_took(later, overlap):
    """seq and keep set for the next batch before this one's backward."""
    one, two = Step("small", overlap), Step("small", overlap)
    for s in (one, two):
        s.L.x.copy_(s.x)
        s.L.forward()
    one.L.backward()
    T, L = two.cfg.T, two.L
    if later == "seq of as many":
        L.seq = torch.tensor([0, 3, 9, 20, T], dtype=torch.int32, device="cuda")
    elif later == "seq of more":
        L.seq = torch.tensor([0, 1, 2, 3, 4, 5, T], dtype=torch.int32, device="cuda")
    elif later == "keep":
        L.keep = torch.zeros(T, dtype=torch.bool, device="cuda")
    else:
        L.seq = L.keep = None
    L.backward()
    torch.cuda.synchronize()
    assert torch.equal(one.L.losses.loss, L.losses.loss)
    for a, b in zip([one.L.dlogits, one.L.dx] + one.L.grads(), [L.dlogits, L.dx] + L.grads()):
        assert torch.equal(a, b)
    # the next forward takes what is set
    L.forward()
    want = L.balance.forward(L.logits, L.idx, seq=L.seq, keep=L.keep)
    assert torch.equal(want.counts, L.losses.counts) and torch.equal(want.loss, L.losses.loss)


def test_losses_that_the_caller_sets():
    """Losses of the caller's own, in place of the forward's: over what is set with them."""
    s = Step()
    L = s.L
    L.x.copy_(s.x)
    L.forward()
    L.seq = torch.tensor([0, 11, s.cfg.T], dtype=torch.int32, device="cuda")
    L.keep = None
    L.losses = L.balance.forward(L.logits, L.idx, seq=L.seq)
    L.backward()
    want = L.balance.backward(L.logits, L.idx, L.losses.counts, L.losses.tokens, seq=L.seq, dgate=L.dgate)
    assert torch.equal(want, L.dlogits)
