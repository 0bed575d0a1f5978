"""The router's balance and z losses, per-expert counts and the gradient against
64 bits (GPU only)."""
import pytest
import torch

from gpu_util import have_gpu
from training_util import assert_within, f64, ref_balance, ref_balance_bwd

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

F32, I32 = torch.float32, torch.int32
INF = float("inf")


def inputs(T, E, k, S=1, keep=False, dead=0, seed=0, tail=True):
    gen = torch.Generator(device="cuda").manual_seed(5000 + seed + T + E)
    n = lambda *s, std=1.0: torch.empty(s, device="cuda").normal_(0, std, generator=gen)
    z = n(T, E, std=1.8) + n(E, std=0.6)
    if dead:
        off = torch.randperm(E, generator=gen, device="cuda")[:dead]
        z[:, off] = -INF
    idx = torch.topk(z, k, dim=1).indices.int() if T else torch.empty(0, k, dtype=I32, device="cuda")
    seq = None
    if S > 1:
        end = T - (T // 7 if tail else 0)
        cuts = torch.randint(0, end + 1, (S - 1,), generator=gen, device="cuda").sort().values
        seq = torch.cat([torch.zeros_like(cuts[:1]), cuts, torch.full_like(cuts[:1], end)]).int()
    kp = (torch.rand(T, generator=gen, device="cuda") < 0.8).to(torch.uint8) if keep else None
    return z, idx, seq, kp, n


def loss_op(weight=0.02, z_weight=0.003):
    from routing_permute_grouped_moe_amd.layer import BalanceLoss
    return BalanceLoss(weight, z_weight)


CASES = [
    # T, E, k, S, keep, dead
    (1, 1, 1, 1, False, 0), (1, 8, 2, 1, False, 0), (3, 2, 2, 1, True, 0), (1, 1024, 1, 1, False, 0),
    (5, 7, 3, 2, False, 0), (64, 64, 6, 1, False, 3), (63, 65, 6, 5, True, 0),
    (256, 8, 2, 1, False, 0), (257, 128, 8, 3, False, 10), (777, 256, 8, 13, True, 0),
    (1000, 100, 10, 40, True, 7), (2049, 300, 4, 1, True, 0), (513, 512, 16, 2, False, 0),
    (130, 1024, 1024, 2, False, 0), (200, 1000, 70, 7, True, 20), (8192, 256, 8, 13, True, 0),
    (4097, 64, 6, 1500, False, 0), (65521, 256, 8, 1, False, 5), (30000, 8, 2, 9, True, 0),
    (10, 16, 2, 300, False, 0),
]


@pytest.mark.parametrize("T,E,k,S,keep,dead", CASES)
def test_forward_and_backward(T, E, k, S, keep, dead):
    print(f"\n[balance] T={T} E={E} k={k} S={S} keep={keep} dead={dead}", flush=True)
    z, idx, seq, kp, n = inputs(T, E, k, S, keep, dead)
    op = loss_op()
    r = op.forward(z, idx, seq=seq, keep=kp)
    want = ref_balance(z, idx, seq, kp, 0.02, 0.003)
    assert torch.equal(f64(r.counts), want["counts"])
    assert torch.equal(f64(r.tokens), want["tokens"])
    assert_within("prob", r.prob, want["prob"])
    assert_within("loss", r.loss, want["loss"])
    dgate, dloss = n(T, k, std=0.01), torch.tensor([1.7], device="cuda")
    for dg, dl in ((None, None), (dgate, dloss), (dgate, None), (None, dloss)):
        got = op.backward(z, idx, r.counts, r.tokens, seq=seq, keep=kp, dgate=dg, dloss=dl)
        assert_within("dlogits", got, ref_balance_bwd(z, idx, seq, kp, 0.02, 0.003,
                                                      1.0 if dl is None else f64(dl).item(), dg))


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (777, 256, 8), (130, 1000, 12), (64, 60, 60), (99, 5, 1)])
def test_without_losses_it_is_the_gates_backward(T, E, k):
    """Weights of zero: the bits of moe_route_bwd; and the losses' part is added to it."""
    from routing_permute_grouped_moe_amd import abi
    z, idx, _, _, n = inputs(T, E, k)
    dgate = n(T, k)
    want = torch.empty_like(z)
    abi.moe_route_bwd(z, idx, dgate, T, E, k, want)
    op = loss_op(0.0, 0.0)
    r = op.forward(z, idx)
    got = op.backward(z, idx, r.counts, r.tokens, dgate=dgate)
    assert torch.equal(got, want)


def test_counts_are_the_permutes():
    from routing_permute_grouped_moe_amd import abi
    T, E, k, H = 777, 256, 8, 64
    z, idx, _, _, _ = inputs(T, E, k)
    r = loss_op().forward(z, idx)
    i = lambda *s: torch.empty(s, dtype=I32, device="cuda")
    counts, ws = i(E), torch.empty(abi.moe_permute_workspace_bytes(T, E, k), dtype=torch.uint8,
                                   device="cuda")
    abi.moe_permute(None, abi.MOE_F32, idx, T, H, E, k, None, counts, i(E + 1), i(T, k), i(T * k), ws,
                    ws.numel())
    assert torch.equal(r.counts[0], counts) and r.tokens.tolist() == [T, T]


def test_gradient_against_differences():
    """The derivative of the weighted losses along random directions of the logits
    by central differences in 64 bits; the counts are constants."""
    T, E, k, S = 300, 24, 3, 6
    z, idx, seq, kp, _ = inputs(T, E, k, S, keep=True)
    a, b = 0.4, 0.02
    op = loss_op(a, b)
    r = op.forward(z, idx, seq=seq, keep=kp)
    got = f64(op.backward(z, idx, r.counts, r.tokens, seq=seq, keep=kp))
    n = f64(r.tokens)
    t = torch.arange(T, device="cuda")
    of = ((t >= seq[:-1, None]) & (t < seq[1:, None]) & (kp != 0)).double()
    frac = f64(r.counts) * E / (k * n[:S, None].clamp(min=1))

    def phi(Z):
        p = torch.softmax(Z, 1)
        lse = torch.logsumexp(Z, 1)
        return (a * ((of @ p) * frac).sum() + b * (of.sum(0) * lse * lse).sum()) / n[S]

    bound = ref_balance_bwd(z, idx, seq, kp, a, b, 1.0, None)[1]
    for seed in range(3):
        v = torch.randn(T, E, dtype=torch.float64, device="cuda",
                        generator=torch.Generator(device="cuda").manual_seed(seed))
        eps = 1e-5
        num = (phi(f64(z) + eps * v) - phi(f64(z) - eps * v)) / (2 * eps)
        have = (got * v).sum()
        slack = (bound * v.abs()).sum() + 1e-7 * (got * v).abs().sum() + 1e-9
        assert abs(num - have) <= slack, (num.item(), have.item(), slack.item())


def test_nothing_counts():
    """No tokens, none kept, logits of -inf alone: zeros and no gradient."""
    op = loss_op()
    for T, keep, off in ((0, None, False), (50, 0, False), (50, None, True)):
        z, idx, _, _, _ = inputs(T, 16, 2)
        if off:
            z.fill_(-INF)
        kp = None if keep is None else torch.zeros(T, dtype=torch.bool, device="cuda")
        r = op.forward(z, idx, keep=kp)
        assert (r.loss == 0).all() and (r.counts == 0).all() and (r.prob == 0).all()
        assert r.tokens.tolist() == [0, 0]
        d = op.backward(z, idx, r.counts, r.tokens, keep=kp)
        assert d.shape == z.shape and (d == 0).all()


def test_masked_rows_infinities_and_nan():
    """A token of -inf alone is left out; the type's lowest value is a number; a NaN
    or +inf in a token that counts gives NaN losses, in one that does not nothing."""
    op = loss_op()
    z, idx, _, _, n = inputs(200, 32, 4)
    low = torch.finfo(F32).min
    z[3] = -INF
    z[4, 5:] = -INF
    z[5] = low
    z[6, 1:] = low
    keep = torch.ones(200, dtype=torch.uint8, device="cuda")
    dgate = n(200, 4)
    r = op.forward(z, idx)
    # (the square of the lowest value's lse is beyond fp32)
    assert r.tokens.tolist() == [199, 199] and torch.isfinite(r.loss[0]) and torch.isinf(r.loss[1])
    d = op.backward(z, idx, r.counts, r.tokens, dgate=dgate)
    assert torch.isfinite(d).all() and (d[3] == 0).all() and (d[4, 5:] == 0).all()
    some = [i for i in range(200) if i not in (5, 6)]
    z2, i2 = z[some].contiguous(), idx[some].contiguous()
    r = op.forward(z2, i2)
    want = ref_balance(z2, i2, None, None, 0.02, 0.003)
    assert_within("loss", r.loss, want["loss"])
    assert_within("prob", r.prob, want["prob"])
    for bad in (float("nan"), INF):
        zz = z2.clone()
        zz[7, 2] = bad
        r = op.forward(zz, i2)
        assert torch.isnan(r.loss).all() and r.tokens.tolist() == [197, 197]
        kp = keep[:198].clone()
        kp[7] = 0
        r = op.forward(zz, i2, keep=kp)
        assert torch.isfinite(r.loss).all() and r.tokens.tolist() == [196, 196]
        d = op.backward(zz, i2, r.counts, r.tokens, keep=kp)
        rest = [i for i in range(198) if i != 7]
        assert torch.isfinite(d[rest]).all()
    zz = z2.clone()
    zz[7] = float("nan")
    assert torch.isnan(op.forward(zz, i2).loss).all()


def test_wrong_data_stays_inside():
    """Sequence ends out of order or range, and experts out of range: some numbers,
    and nothing written but the outputs."""
    T, E, k = 500, 40, 4
    z, idx, _, _, n = inputs(T, E, k)
    idx = idx.clone()
    idx[::3, 1] = 1 << 30
    idx[1::3, 2] = -5
    op = loss_op()
    for ends in ([0, 400, 100, 700, 500], [-5, 3, 2, 1 << 30, 9], [500, 400, 300, 200, 0]):
        seq = torch.tensor(ends, dtype=I32, device="cuda")
        r = op.forward(z, idx, seq=seq)
        d = op.backward(z, idx, r.counts, r.tokens, seq=seq, dgate=n(T, k))
        torch.cuda.synchronize()
        assert d.shape == z.shape
    r = op.forward(z, idx)
    assert r.counts.sum().item() == int(((idx >= 0) & (idx < E)).sum())


def test_on_views_off_sixteen_bytes():
    """Logits of odd rows, from a row on: aligned to a value alone."""
    T, E, k = 333, 37, 3
    z, idx, seq, kp, n = inputs(T + 1, E, k, 4, True)
    r = loss_op().forward(z[1:].clone(), idx[1:].clone(), seq=seq, keep=kp[1:].clone())
    got = loss_op().forward(z[1:], idx[1:], seq=seq, keep=kp[1:])
    for a, b in zip(r, got):
        assert torch.equal(a, b)
    dg = n(T + 1, k)
    a = loss_op().backward(z[1:].clone(), idx[1:].clone(), r.counts, r.tokens, seq=seq,
                           keep=kp[1:].clone(), dgate=dg[1:].clone())
    out = torch.full((T + 2, E), 7.0, device="cuda")
    loss_op().backward(z[1:], idx[1:], r.counts, r.tokens, seq=seq, keep=kp[1:], dgate=dg[1:],
                       out=out[1:T + 1])
    assert torch.equal(out[1:T + 1], a) and (out[0] == 7).all() and (out[T + 1] == 7).all()


def test_streams_and_inputs_dropped_behind_another():
    z, idx, seq, kp, n = inputs(3000, 256, 8, 9, True)
    dg = n(3000, 8)
    op = loss_op()
    want = op.forward(z, idx, seq=seq, keep=kp)
    back = op.backward(z, idx, want.counts, want.tokens, seq=seq, keep=kp, dgate=dg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    z1, i1, s1, k1, d1 = (t.clone() for t in (z, idx, seq, kp, dg))
    torch.cuda.current_stream().synchronize()
    got = op.forward(z1, i1, seq=s1, keep=k1, stream=side)
    d = op.backward(z1, i1, got.counts, got.tokens, seq=s1, keep=k1, dgate=d1, stream=side)
    del z1, i1, s1, k1, d1
    junk = [torch.full_like(t, 1) for t in (z, idx, seq, kp, dg) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(d, back)
    assert len(junk) == 20


@pytest.mark.parametrize("T,S", [(300, 1), (5000, 20)])
def test_replays_from_a_graph(T, S):
    z, idx, seq, kp, n = inputs(T, 64, 6, S, True)
    dg = n(T, 6)
    op = loss_op()

    def step():
        r = op.forward(z, idx, seq=seq, keep=kp)
        return tuple(r) + (op.backward(z, idx, r.counts, r.tokens, seq=seq, keep=kp, dgate=dg),)

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    junk = torch.randn(1 << 18, device="cuda")
    for _ in range(4):
        for t in outs:
            t.fill_(-7)
        junk.mul_(1.01).sum().item()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        for a, b in zip(step(), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,E", [(67_000_001, 16), (16_777_213, 64), (1_048_575, 1024)])
def test_tensors_of_almost_four_gib(T, E):
    """Byte offsets up to 2^32: all logits alike but those of the last tokens."""
    k, last = 1, 777
    z = torch.zeros(T, E, device="cuda")
    zl, il, _, _, _ = inputs(last, E, k)
    z[-last:] = zl
    idx = torch.zeros(T, k, dtype=I32, device="cuda")
    idx[-last:] = il
    keep = torch.zeros(T, dtype=torch.uint8, device="cuda")
    keep[-last:] = 1
    keep[0] = 1
    op = loss_op()
    r = op.forward(z, idx, keep=keep)
    some = torch.cat([z[:1], z[-last:]]), torch.cat([idx[:1], idx[-last:]])
    want = ref_balance(*some, None, None, 0.02, 0.003)
    assert torch.equal(f64(r.counts), want["counts"]) and r.tokens.tolist() == [last + 1] * 2
    assert_within("prob", r.prob, want["prob"])
    assert_within("loss", r.loss, want["loss"])
    out = torch.full_like(z, 7.0)
    op.backward(z, idx, r.counts, r.tokens, keep=keep, out=out)
    ref, bound = ref_balance_bwd(*some, None, None, 0.02, 0.003, 1.0, None)
    assert_within("dlogits", torch.cat([out[:1], out[-last:]]), (ref, bound))
    assert out[1:100].abs().max() == 0 and out[T // 2].abs().max() == 0


def test_two_at_once_and_again():
    """Calls on two streams side by side, over and over: the same bits."""
    z, idx, seq, kp, n = inputs(20000, 256, 8, 30, True)
    z2, idx2, _, _, _ = inputs(300, 1024, 4)
    op = loss_op()
    want, want2 = op.forward(z, idx, seq=seq, keep=kp), op.forward(z2, idx2)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (a, b):
        s.wait_stream(torch.cuda.current_stream())
    got = [(op.forward(z, idx, seq=seq, keep=kp, stream=a), op.forward(z2, idx2, stream=b))
           for _ in range(8)]
    torch.cuda.synchronize()
    for x, y in got:
        assert all(torch.equal(p, q) for p, q in zip(x, want))
        assert all(torch.equal(p, q) for p, q in zip(y, want2))


def test_many_sequences_of_few_experts():
    """More sequences than tokens, tokens of several sequences in a wave, an end at
    every token, padding behind."""
    T, E, k = 1000, 12, 3
    z, idx, _, kp, n = inputs(T, E, k, keep=True)
    op, dg = loss_op(), n(T, k)
    for ends in (torch.arange(0, T - 50), torch.arange(0, 3 * T, 2).clamp(max=T - 1),
                 torch.tensor([0] * 3000 + [T]), torch.tensor([0, 5] + [5] * 700 + [T - 1])):
        seq = ends.int().cuda()
        r = op.forward(z, idx, seq=seq, keep=kp)
        want = ref_balance(z, idx, seq, kp, 0.02, 0.003)
        assert torch.equal(f64(r.counts), want["counts"])
        assert torch.equal(f64(r.tokens), want["tokens"])
        assert_within("loss", r.loss, want["loss"])
        assert_within("prob", r.prob, want["prob"])
        got = op.backward(z, idx, r.counts, r.tokens, seq=seq, keep=kp, dgate=dg)
        assert_within("dlogits", got, ref_balance_bwd(z, idx, seq, kp, 0.02, 0.003, 1.0, dg))


@pytest.mark.parametrize("E", [9, 30, 64, 100, 256, 500, 1000])
def test_tokens_that_do_not_count_have_no_gradient_whatever_they_hold(E):
    """NaN or infinities in a token that is not kept, or lies in no sequence: zeros in its
    row, and in its neighbours' their own bits; with a gates' gradient there the row is
    the gates' (NaN), without it zeros."""
    T, k = 90, 4
    z, idx, _, _, n = inputs(T, E, k)
    keep = torch.ones(T, dtype=torch.uint8, device="cuda")
    out = [0, 7, 8, 21, 42, 43]
    keep[out] = 0
    seq = torch.tensor([5, 40, 40, T - 6], dtype=I32, device="cuda")
    away = sorted(set(out + [0, 1, 2, 3, 4] + list(range(T - 6, T))))
    stay = [t for t in range(T) if t not in away]
    dgate = n(T, k, std=0.1)
    dgate[away] = 0.0
    dgate[7, 1] = -0.0
    op = loss_op()
    r = op.forward(z, idx, seq=seq, keep=keep)
    want = [op.backward(z, idx, r.counts, r.tokens, seq=seq, keep=keep, dgate=dg)
            for dg in (None, dgate)]
    for bad in (float("nan"), INF, -INF):
        zz = z.clone()
        zz[away, 2] = bad
        zz[8] = bad
        q = op.forward(zz, idx, seq=seq, keep=keep)
        assert all(torch.equal(a, b) for a, b in zip(q, r))
        for dg, w in zip((None, dgate), want):
            d = op.backward(zz, idx, r.counts, r.tokens, seq=seq, keep=keep, dgate=dg)
            assert (d[away] == 0).all() and torch.equal(d[stay], w[stay])
    assert all((w[away] == 0).all() for w in want)
    # a gradient of the gates reaches such a token all the same
    dg = dgate.clone()
    dg[21, 3] = 0.25
    d = op.backward(z, idx, r.counts, r.tokens, seq=seq, keep=keep, dgate=dg)
    assert (d[21] != 0).any() and torch.equal(d[stay], want[1][stay])
    zz = z.clone()
    zz[21, 2] = float("nan")
    d = op.backward(zz, idx, r.counts, r.tokens, seq=seq, keep=keep, dgate=dg)
    assert torch.isnan(d[21]).all()
    rest = [t for t in range(T) if t != 21]
    assert torch.isfinite(d[rest]).all()


def test_a_padded_batch_does_not_poison_the_routers_weights():
    """NaN logits in the padding: dWg and dbias of the router are those without it."""
    from routing_permute_grouped_moe_amd import abi
    T, H, E, k = 512, 128, 64, 4
    z, idx, _, _, n = inputs(T, E, k)
    x, wg = n(T, H), n(H, E, std=0.1)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[400:] = False
    op = loss_op()
    got = []
    for bad in (False, True):
        zz = z.clone()
        if bad:
            zz[400:] = float("nan")
        r = op.forward(zz, idx, keep=keep)
        d = op.backward(zz, idx, r.counts, r.tokens, keep=keep)
        nb = abi.moe_router_workspace_bytes(T, H, E, abi.MOE_F32)
        ws = torch.empty(max(nb, 256), dtype=torch.uint8, device="cuda")
        dx, dwg, db = torch.empty_like(x), torch.empty_like(wg), torch.empty(E, device="cuda")
        abi.moe_router_logits_bwd(d, x, abi.MOE_F32, wg, T, H, E, dx, dwg, db, ws, nb)
        got.append((dx, dwg, db))
    for a, b in zip(*got):
        assert torch.isfinite(b).all() and torch.equal(a, b)


@pytest.mark.parametrize("T,E,rows", [(1 << 26, 3, [[0.3, -0.4, 0.05]]), ((1 << 26) - 65, 2, [[0.1, 0.4]]),
                                      (1 << 21, 500, None), (9_000_001, 48, None)])
def test_long_sums_of_like_probabilities(T, E, rows):
    """Every token counts and all are alike, so that every addition of a sum rounds the
    same way.  The bound's 270 u of the mean hold whatever T: a lane adds at most 240 in
    fp32, 2 additions join the lanes of a wave and 15 the waves of a block, whose sum is
    exact in fp32 then; the blocks are added in 64 bits and rounded once."""
    k = 2
    row = torch.linspace(-0.3, 0.4, E)[None] if rows is None else torch.tensor(rows)
    row = row.cuda()
    z = row.expand(T, E).contiguous()
    idx = torch.tensor([[0, 1]], dtype=I32, device="cuda").expand(T, k).contiguous()
    r = loss_op().forward(z, idx)
    want = ref_balance(row, idx[:1], None, None, 0.02, 0.003)   # (means: of one token as of T)
    assert torch.equal(f64(r.counts), want["counts"] * T) and r.tokens.tolist() == [T, T]
    assert_within("prob", r.prob, want["prob"])
    assert_within("loss", r.loss, want["loss"])
    # and in two sequences, the shorter ended inside a block
    ends = [0, 1_000_003, T]
    r = loss_op().forward(z, idx, seq=torch.tensor(ends, dtype=I32, device="cuda"))
    p, bound = want["prob"]
    assert_within("prob", r.prob, (p.expand(2, E), bound.expand(2, E)))
    assert r.counts[:, 0].tolist() == [ends[1], T - ends[1]] and (r.counts[:, 2:] == 0).all()


def guarded(n, dtype, fill):
    """n values between guards of 4 KB, and a check that the guards are as they were."""
    g = 4096 // torch.empty((), dtype=dtype).element_size()
    whole = torch.full((n + 2 * g,), fill, dtype=dtype, device="cuda")

    def untouched():
        return bool((whole[:g] == fill).all()) and bool((whole[g + n:] == fill).all())
    return whole[g:g + n], untouched


@pytest.mark.parametrize("T,E,k", [(500, 40, 4), (90, 12, 3), (3000, 300, 5), (700, 1024, 2)])
@pytest.mark.parametrize("S", [4, 90])
def test_writes_are_the_outputs_and_the_planned_workspace(T, E, k, S):
    """Through the C calls, with guards around every output and a workspace of exactly the
    planned bytes: sequence ends in order, out of order and out of range, experts out of
    range."""
    from routing_permute_grouped_moe_amd import abi
    z, idx, _, kp, n = inputs(T, E, k, keep=True)
    idx = idx.clone()
    idx[::3, 1] = 1 << 30
    idx[1::3, 0] = -5
    dgate = n(T, k)
    gen = torch.Generator().manual_seed(S)
    fine = torch.randint(0, T + 1, (S + 1,), generator=gen).sort().values
    some = torch.randint(-T, 2 * T, (S + 1,), generator=gen)
    far = some.clone()
    far[::2] = torch.tensor([-(1 << 31), (1 << 31) - 1])[torch.arange(far[::2].numel()) % 2]
    for ends in (fine, fine.flip(0), some, far):
        seq = ends.to(I32).cuda()
        nb = abi.moe_balance_loss_workspace_bytes(T, E, k, S)
        outs = {"loss": guarded(3, F32, 7.0), "counts": guarded(S * E, I32, -9),
                "tokens": guarded(S + 1, I32, -9), "prob": guarded(S * E, F32, 7.0),
                "ws": guarded(nb, torch.uint8, 201), "dlogits": guarded(T * E, F32, 7.0)}
        at = {name: t for name, (t, _) in outs.items()}
        abi.moe_balance_loss(z, idx, kp, seq, T, E, k, S, 0.02, 0.003, at["loss"], at["counts"],
                             at["tokens"], at["prob"], at["ws"] if nb else None, nb)
        abi.moe_balance_loss_bwd(z, idx, dgate, kp, seq, at["counts"], at["tokens"], T, E, k, S, 0.02,
                                 0.003, None, at["dlogits"])
        torch.cuda.synchronize()
        for name, (_, untouched) in outs.items():
            assert untouched(), name
        assert at["dlogits"].shape[0] == T * E and not (at["dlogits"] == 7.0).all()
