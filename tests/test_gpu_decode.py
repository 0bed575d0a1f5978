"""The few-token layer against its definition in 64 bits (GPU only)."""
import pytest
import torch

from decode_util import (U, assert_within, ref_decode, ref_linear, ref_logits, ref_route)
from decode_util import f64
from gpu_util import have_gpu

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32


def make(T, H, I, E, k, g0=0, G=None, dt=BF, shared=False, router=True, bias=True, seed=0):
    from routing_permute_grouped_moe_amd.layer import LayerShape, MoeDecode
    gen = torch.Generator(device="cuda").manual_seed(1000 + seed)
    shape = LayerShape(T=T, H=H, I=I, E=E, k=k, dtype=dt, g0=g0, G=G, shared=shared,
                       router=router)
    n = lambda *s, std=1.0, d=dt: torch.empty(s, dtype=d, device="cuda").normal_(0, std,
                                                                                generator=gen)
    G = shape.groups
    p = {"w13": n(G, 2 * I, H, std=H ** -0.5), "w2": n(G, H, I, std=I ** -0.5)}
    if router:
        p["wg"] = n(H, E, std=1.5 * H ** -0.5, d=F32)
        if bias:
            p["bias"] = n(E, std=0.5, d=F32)
    if shared:
        p["ws13"], p["ws2"] = n(2 * I, H, std=H ** -0.5), n(H, I, std=I ** -0.5)
    return MoeDecode(shape, **p), n


def check(op, x, r, residual=None, logits=None):
    """Every output of one pass: logits, choices, gates and y."""
    s = op.s
    if s.router:
        full = ref_logits(x, op.wg, op.bias)
        # one rounding to fp32 of a sum that is exact to far below it
        assert_within("logits", r.logits, (full, 1.001 * U * full.abs() + 1e-12))
        lg = full.float()
        same = lg == r.logits.cpu()
        assert same.float().mean() > 0.999      # (a sum within 1e-12 of a rounding border)
        lg = r.logits.cpu()
    else:
        assert torch.equal(r.logits, logits)
        lg = logits.cpu()
    idx, gate, dgate = ref_route(lg, s.k)
    assert torch.equal(r.idx.cpu().long(), idx)
    assert_within("gate", r.gate, (gate, dgate))
    assert_within("y", r.y, ref_decode(x, idx, gate, dgate, s.g0, s.groups, op.w13, op.w2, op.ws13,
                                       op.ws2, residual, s.dtype))


CASES = [
    # T, H, I, E, k, extra
    (1, 64, 64, 1, 1, {}),
    (1, 128, 64, 8, 2, {"dt": F32}),
    (1, 2048, 1408, 64, 6, {"residual": True}),
    (2, 192, 320, 5, 5, {"shared": True}),
    (5, 128, 64, 8, 2, {"dt": F32, "shared": True, "residual": True}),
    (7, 64, 192, 100, 3, {"bias": False}),
    (15, 320, 64, 300, 8, {"g0": 17, "G": 101}),
    (16, 1024, 512, 16, 4, {"residual": True, "shared": True}),
    (17, 448, 128, 3, 2, {}),
    (17, 448, 128, 3, 2, {"dt": F32}),
    (33, 256, 256, 6, 1, {"shared": True}),
    (64, 512, 64, 9, 3, {"g0": 2, "G": 4, "residual": True}),
    (65, 128, 128, 4, 4, {}),
    (128, 256, 192, 12, 6, {"shared": True, "residual": True}),
    (128, 192, 64, 33, 16, {}),                       # the most pairs
    (8, 128, 64, 300, 256, {}),                       # as many of few tokens
    (100, 64, 64, 40, 2, {"dt": F32, "g0": 39, "G": 1}),
    (2, 64, 64, 1024, 1024, {}),                      # every expert chosen
    (9, 128, 64, 1000, 7, {"g0": 0, "G": 1}),
    (3, 128, 64, 8, 2, {"G": 0, "shared": True}),     # no routed expert on this device
    (3, 128, 64, 8, 2, {"G": 0, "residual": True}),
]


@pytest.mark.parametrize("T,H,I,E,k,extra", CASES)
def test_layer(T, H, I, E, k, extra):
    extra = dict(extra)
    print(f"\n[decode] T={T} H={H} I={I} E={E} k={k} {extra}", flush=True)
    with_res = extra.pop("residual", False)
    op, n = make(T, H, I, E, k, **extra, seed=T + H)
    x = n(T, H)
    res = n(T, H) if with_res else None
    r = op.forward(x, residual=res)
    torch.cuda.synchronize()
    check(op, x, r, residual=res)


@pytest.mark.parametrize("T,E,k,g0,G,shared", [
    (8, 20, 8, 0, 20, False),      # 64 pairs, as many as lanes
    (13, 5, 5, 0, 5, True),        # 65: one more
    (16, 9, 4, 0, 9, True), (16, 9, 4, 3, 5, False), (12, 4, 4, 3, 1, True),
    (9, 1000, 7, 990, 10, False), (6, 64, 1, 0, 64, True), (16, 1, 1, 0, 1, False),
])
def test_few_pairs(T, E, k, g0, G, shared):
    """Calls of about 64 pairs, whose experts' rows are found in another way."""
    op, n = make(T, 192, 128, E, k, g0=g0, G=G, shared=shared, router=False, seed=E)
    x, lg = n(T, 192), n(T, E, d=F32)
    r = op.forward(x, logits=lg)
    torch.cuda.synchronize()
    check(op, x, r, logits=lg)


def test_inputs_dropped_behind_another_stream():
    """Inputs that the caller drops while the call still waits on its stream are
    not handed out again before it has read them."""
    op, n = make(4, 1024, 512, 16, 4)
    x, res = n(4, 1024), n(4, 1024)
    want = op.forward(x, residual=res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    x1, res1 = x.clone(), res.clone()
    torch.cuda.current_stream().synchronize()
    got = op.forward(x1, residual=res1, stream=side)
    del x1, res1
    junk = [torch.full_like(x, float("nan")) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and len(junk) == 8


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T", [1, 18, 70, 128])
def test_masked_and_hot_experts(T, dt):
    """Logits from elsewhere: experts masked by -inf, a token with every expert
    masked, one expert that every token takes, ties."""
    E, k, H, I = 11, 3, 128, 64
    op, n = make(T, H, I, E, k, dt=dt, router=False, g0=1, G=9, seed=T)
    lg = torch.round(n(T, E, d=F32) * 2) / 2               # many ties
    lg[:, 4] = 9.0                                         # the hot expert
    lg[:, 6:9] = -float("inf")
    lg[0, 1] = -0.0
    lg[0, 2] = 0.0
    lg[T // 2] = -float("inf")                             # nothing left (T = 1: of the only token)
    x = n(T, H)
    r = op.forward(x, logits=lg)
    torch.cuda.synchronize()
    assert (r.gate[T // 2] == 0).all() and (r.y[T // 2] == 0).all()
    check(op, x, r, logits=lg)


def test_token_with_no_expert_here():
    """Every choice outside the window: y is the residual, bit for bit."""
    op, n = make(6, 192, 64, 8, 2, g0=6, G=2, router=False)
    lg = torch.zeros(6, 8, device="cuda")
    lg[:, 1], lg[:, 3] = 3.0, 2.0
    x, res = n(6, 192), n(6, 192)
    r = op.forward(x, residual=res, logits=lg)
    assert torch.equal(r.y, res)


@pytest.mark.parametrize("T", [1, 40])
def test_in_place_on_the_residual_and_nothing_behind(T):
    op, n = make(T, 256, 128, 16, 4, shared=True)
    x = n(T, 256)
    buf = n(T + 3, 256)
    keep = buf.clone()
    r0 = op.forward(x, residual=keep[:T])
    r1 = op.forward(x, residual=buf[:T], out=buf[:T])
    assert r1.y.data_ptr() == buf.data_ptr()
    assert torch.equal(r0.y, buf[:T]) and torch.equal(buf[T:], keep[T:])


def test_same_bits_on_every_run():
    op, n = make(23, 640, 448, 24, 5, shared=True)
    x = n(23, 640)
    first = op.forward(x)
    for _ in range(5):
        r = op.forward(x)
        assert all(torch.equal(a, b) for a, b in zip(first, r))


def test_two_streams_at_once():
    """Calls of one layer on two streams, nothing between them: each has its own workspace."""
    op, n = make(64, 1024, 512, 32, 4, shared=True)
    xs = [n(64, 1024) for _ in range(2)]
    want = [op.forward(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for i, st in enumerate(streams):
            got[i].append(op.forward(xs[i], stream=st))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(want[i], r))


def test_two_captured_graphs():
    """Two graphs of one layer, replayed in turn and side by side, with eager
    work between."""
    op, n = make(5, 512, 256, 16, 4, shared=True)
    xs = [n(5, 512) for _ in range(2)]
    want = [op.forward(x) for x in xs]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            op.forward(x)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            outs.append(op.forward(x))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    junk = torch.randn(1 << 18, device="cuda")
    for rep in range(6):
        for o in outs:
            o.y.zero_()
            o.idx.fill_(-1)
        junk.mul_(1.01).sum().item()
        torch.cuda.synchronize()
        for st, g in zip(streams, graphs):
            if rep % 2:
                with torch.cuda.stream(st):
                    g.replay()
            else:
                g.replay()
        torch.cuda.synchronize()
        eager = op.forward(xs[0])
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w)), rep
        assert torch.equal(eager.y, want[0].y)


def test_fewer_tokens_than_built_for_and_none():
    op, n = make(16, 128, 64, 8, 2)
    for T in (16, 3, 0, 1):
        x = n(T, 128)
        r = op.forward(x)
        torch.cuda.synchronize()
        assert r.y.shape == (T, 128) and r.idx.shape == (T, 2)
        if T:
            check(op, x, r)


def test_of_a_training_layer():
    """On a MoeLayer's parameters: the choices and gates are its own, y agrees
    to the roundings the training path makes on the way (h13, act, yp)."""
    import synth
    from gpu_util import make_layer
    from routing_permute_grouped_moe_amd.layer import MoeDecode
    cfg = synth.get_config("small", T=48, H=512, I=256, E=16, k=4)
    L = make_layer(cfg, synth.make_inputs(cfg))
    L.forward()
    r = MoeDecode.of_layer(L).forward(L.x)
    torch.cuda.synchronize()
    assert torch.equal(r.idx, L.idx)
    # the training path rounds h13, act, yp and y to bf16: four half steps, each
    # spread over the sum by at most its magnitude
    mag = r.y.float().abs().amax()
    assert (r.y.float() - L.y.float()).abs().amax() <= 2e-2 * mag


def test_block_of_a_decoder():
    """A block's tail as it runs: attention output through the projection onto
    the residual stream, the expert layer onto it, then a dense feed-forward --
    every step from the values the step before left."""
    from routing_permute_grouped_moe_amd.layer import Linear
    T, H = 6, 512
    op, n = make(T, H, 256, 16, 4, shared=True)
    proj = Linear(n(H, H, std=H ** -0.5), bias=n(H, std=0.5, d=F32))
    up = Linear(n(4 * H, H, std=H ** -0.5), bias=n(4 * H, std=0.5, d=F32), act="gelu_tanh")
    down = Linear(n(H, 4 * H, std=(4 * H) ** -0.5))
    attn, stream = n(T, H), n(T, H)
    h0 = proj.forward(attn, residual=stream)
    assert_within("proj", h0, ref_linear(attn, proj.w, proj.bias, "none", stream, BF)[0])
    r = op.forward(h0, residual=h0)
    check(op, h0, r, residual=h0)
    f = up.forward(r.y)
    assert_within("up", f, ref_linear(r.y, up.w, up.bias, "gelu_tanh", None, BF)[0])
    keep = r.y.clone()
    y = down.forward(f, residual=r.y, out=r.y)
    assert_within("down", y, ref_linear(f, down.w, None, "none", keep, BF)[0])


def nan_of_either_sign(n):
    return torch.tensor([0x7fc00000, -0x400000], dtype=torch.int32).view(F32).repeat(n)[:n].cuda()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T", [1, 6, 40])
def test_nan_logits_are_no_mask(T, dt):
    """A row of NaN, or of NaN and -inf, is not a row whose experts are masked:
    its gates are NaN, as moe_route gives them, and so is its y; the other rows
    do not see it."""
    from routing_permute_grouped_moe_amd import abi
    E, k, H, I = 70, 3, 128, 64
    op, n = make(T, H, I, E, k, dt=dt, router=False, shared=True, seed=T)
    lg = n(T, E, d=F32)
    rows = [T // 2] if T < 6 else [1, 2, 4]
    for i, r in enumerate(rows):
        if i == 0:
            lg[r] = nan_of_either_sign(E)
        elif i == 1:
            lg[r] = -float("inf")
            lg[r, 66] = float("nan")
        else:
            lg[r, 7] = float("nan")                # among finite ones
    x, res = n(T, H, d=dt), n(T, H, d=dt)
    r = op.forward(x, residual=res, logits=lg)
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    gate = torch.empty(T, k, dtype=F32, device="cuda")
    abi.moe_route(lg, T, E, k, idx, gate)
    assert torch.equal(r.idx, idx) and torch.equal(torch.isnan(r.gate), torch.isnan(gate))
    bad = torch.zeros(T, dtype=torch.bool)
    bad[rows] = True
    assert torch.isnan(r.gate[bad]).all() and torch.isnan(r.y[bad]).all()
    if T > 1:
        alone = op.forward(x[~bad].contiguous(), residual=res[~bad].contiguous(),
                           logits=lg[~bad].contiguous())
        assert_within("gate", r.gate[~bad], ref_route(lg[~bad].cpu(), k)[1:])
        assert torch.equal(r.y[~bad], alone.y) and torch.isfinite(alone.y).all()


@pytest.mark.parametrize("T", [2, 30])
def test_nan_in_the_router_reaches_y(T):
    """A NaN in a row of Wg makes every logit NaN, one in x a token's: no finite y."""
    op, n = make(T, 128, 64, 9, 2, seed=3)
    x, res = n(T, 128), n(T, 128)
    wg = op.wg.clone()
    x[0, 5] = float("nan")
    r = op.forward(x, residual=res)
    assert torch.isnan(r.y[0]).all() and torch.isfinite(r.y[1:]).all()
    op.wg[77] = float("nan")
    r = op.forward(x, residual=res)
    assert torch.isnan(r.logits).all() and torch.isnan(r.gate).all() and torch.isnan(r.y).all()
    op.wg.copy_(wg)


@pytest.fixture
def no_patience():
    """Every wait within a call that finds its work missing is given up."""
    from routing_permute_grouped_moe_amd import abi
    abi.moe_decode_wait_limit(0)
    yield
    abi.moe_decode_wait_limit(1000000)


def nan_or_right(op, x, wanted, calls, **kw):
    """Calls whose every value is NaN or the right one; how many held a NaN."""
    held = 0
    for _ in range(calls):
        r = op.forward(x, **kw)
        torch.cuda.synchronize()
        nan = torch.isnan(r.y)
        assert torch.equal(torch.where(nan, wanted.y, r.y), wanted.y)
        assert torch.equal(r.idx, wanted.idx) and torch.equal(r.gate, wanted.gate)
        held += bool(nan.any())
    return held


@pytest.mark.parametrize("T,H,I,E,k,shared", [(1, 2048, 1408, 64, 6, False),
                                              (8, 512, 256, 16, 4, True),
                                              (3, 256, 512, 8, 8, False)])
def test_a_wait_given_up_is_nan_for_few_tokens(T, H, I, E, k, shared, no_patience):
    """The wait between the products, given up at once: what is not right is NaN,
    and the next call, with patience, is right again."""
    from routing_permute_grouped_moe_amd import abi
    op, n = make(T, H, I, E, k, shared=shared)
    x, res = n(T, H), n(T, H)
    abi.moe_decode_wait_limit(1000000)
    want = op.forward(x, residual=res)
    check(op, x, want, residual=res)
    abi.moe_decode_wait_limit(0)
    assert nan_or_right(op, x, want, 20, residual=res) > 0
    abi.moe_decode_wait_limit(1000000)
    r = op.forward(x, residual=res)
    assert all(torch.equal(a, b) for a, b in zip(want, r))


@pytest.mark.parametrize("T,H,I,E,k,shared", [(9, 512, 256, 16, 4, False), (40, 512, 256, 16, 4, True),
                                              (128, 256, 128, 24, 6, False),
                                              (8, 128, 64, 300, 256, False)])
def test_a_wait_given_up_is_nan_throughout(T, H, I, E, k, shared, no_patience):
    """Calls whose tokens are routed in units of their own: a workgroup that gives
    up waiting for them leaves units undone, and no value of y is taken for right."""
    from routing_permute_grouped_moe_amd import abi
    op, n = make(T, H, I, E, k, shared=shared)
    x, res = n(T, H), n(T, H)
    abi.moe_decode_wait_limit(1000000)
    want = op.forward(x, residual=res)
    check(op, x, want, residual=res)
    abi.moe_decode_wait_limit(0)
    assert nan_or_right(op, x, want, 20, residual=res) > 0
    abi.moe_decode_wait_limit(1000000)
    r = op.forward(x, residual=res)
    assert all(torch.equal(a, b) for a, b in zip(want, r))


@pytest.mark.parametrize("T", [1, 12, 20])
def test_activations_beyond_bf16(T):
    """An activation that overflows fp32 is an infinity in y (not NaN); one that is
    finite but above the largest bf16 counts as it is."""
    H = I = 64
    op, n = make(T, H, I, 2, 1, router=False, seed=T)
    lg = torch.zeros(T, 2, device="cuda")
    lg[:, 0] = 1.0
    x = torch.zeros(T, H, dtype=BF, device="cuda")
    x[:, :2] = 1.0
    for t in (op.w13, op.w2):
        t.zero_()
    # gate 1.99997 x 2^63 (the sum of two bf16), up 2^64
    op.w13[0, :2, 0] = 1.9921875 * 2.0 ** 63
    op.w13[0, :2, 1] = 1.9921875 * 2.0 ** 55
    op.w13[0, I, 0], op.w13[0, I + 1, 0] = 2.0 ** 64, -(2.0 ** 64)
    op.w2[0, 0, 0] = op.w2[0, 1, 1] = 2.0 ** -10
    y = f64(op.forward(x, logits=lg).y)
    s = torch.softmax(f64(lg), dim=1)[:, 0] * (1.9921875 + 1.9921875 / 256) * 2.0 ** 117
    # (within bf16's half step, and the 16 bits of the activation)
    assert ((y[:, 0] - s).abs() <= 1.01 * 2.0 ** -8 * s).all(), y[0, :2]
    assert ((y[:, 1] + s).abs() <= 1.01 * 2.0 ** -8 * s).all(), y[0, :2]
    # up 2^66: infinities, all of them, against weights without a zero
    op.w13[0, :I, :2] = op.w13[0, :1, :2].clone()
    op.w13[0, I:, 0] = 2.0 ** 66
    op.w2[0, 2], op.w2[0, 3] = 2.0 ** -10, -(2.0 ** -10)
    y = op.forward(x, logits=lg).y
    assert (y[:, 2] == float("inf")).all() and (y[:, 3] == -float("inf")).all(), y[0, :4]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T", [1, 8, 40])
def test_a_masked_expert_adds_nothing_whatever_it_holds(T, dt):
    """Experts masked by -inf that fill a token's last slots (fewer are left than
    k), or all slots of a token without any: their weights, or the token's own x,
    may hold infinities and NaN."""
    E, k, H, I = 5, 4, 128, 64
    op, n = make(T, H, I, E, k, dt=dt, router=False, seed=T)
    lg = n(T, E, d=F32)
    lg[:, 2:4] = -float("inf")
    x, res = n(T, H, d=dt), n(T, H, d=dt)
    want = op.forward(x, residual=res, logits=lg)
    assert torch.isfinite(want.y).all()
    op.w13[2] = float("nan")
    op.w2[3] = float("inf")
    r = op.forward(x, residual=res, logits=lg)
    assert all(torch.equal(a, b) for a, b in zip(want, r))
    lg[0] = -float("inf")
    x[0] = float("nan")
    r = op.forward(x, residual=res, logits=lg)
    assert torch.equal(r.y[0], res[0]) and torch.equal(r.y[1:], want.y[1:])


def test_weights_dropped_behind_another_stream():
    """Weights that the caller drops, layer and all, while the call still waits on
    its stream are not handed out again before it has read them."""
    from routing_permute_grouped_moe_amd.layer import MoeDecode
    op, n = make(4, 1024, 512, 16, 4, shared=True)
    x = n(4, 1024)
    want = op.forward(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    names = ("w13", "w2", "wg", "bias", "ws13", "ws2")
    other = MoeDecode(op.s, **{m: getattr(op, m).clone() for m in names})
    torch.cuda.current_stream().synchronize()
    got = other.forward(x, stream=side)
    del other
    junk = [torch.full_like(getattr(op, m), float("nan")) for m in names for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and len(junk) == 18


@pytest.mark.parametrize("T", [9, 40, 128])
@pytest.mark.parametrize("shared", [False, True])
def test_no_expert_on_this_device(T, shared):
    """More tokens than every workgroup routes itself, and an empty window."""
    op, n = make(T, 128, 64, 8, 2, G=0, shared=shared, seed=T)
    x, res = n(T, 128), n(T, 128)
    r = op.forward(x, residual=res)
    check(op, x, r, residual=res)
    assert shared or torch.equal(r.y, res)
