"""The norm of many gradients and clipping by it against 64 bits (GPU only)."""
import pytest
import torch

from gpu_util import have_gpu
from training_util import U, assert_within, f64, ref_clip, ref_norms

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def grads_of(sizes, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(6000 + seed)
    return [torch.empty(n, dtype=BF if i % 3 else F32, device="cuda").normal_(
        0, 0.1 * (1 + i % 5), generator=gen) for i, n in enumerate(sizes)]


def clipper(*a, **kw):
    from routing_permute_grouped_moe_amd.layer import GradClip
    return GradClip(*a, **kw)


SETS = [[1], [0, 5], [0, 0], [7, 8, 9], [255, 256, 257, 2047, 2048, 2049], [16383, 16384, 16385, 0, 1],
        [100003, 3, 70000], [(i * 37) % 90 for i in range(1000)], [17] * 176, [17] * 177,
        [0] * 176 + [5], [5] + [0] * 400, [(i * 7919) % 50000 + 1 for i in range(300)],
        [30_000_001, 12, 1 << 22], [1_000_000 + 977 * i for i in range(130)], [3] * 20000]


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("i", range(len(SETS)))
def test_norm_and_clip(i, kind):
    print(f"\n[clip] set {i}: {len(SETS[i])} gradients, {kind}", flush=True)
    grads = grads_of(SETS[i], i)
    norm, norms, total = clipper(grads, kind=kind).norm(each=True, total=True)
    want, each = ref_norms(grads, kind)
    assert_within("norm", norm, (want, 1.01 * U * want))
    assert_within("norms", norms, (each, 1.01 * U * each))
    whole = want * want if kind == "l2" else want
    assert_within("total", total, (whole, 1e-12 * whole))
    before = [g.clone() for g in grads]
    outs = [torch.full_like(g, NAN, dtype=F32 if j % 2 else g.dtype) for j, g in enumerate(grads)]
    limit = 0.37 * float(want) + 1e-3
    got = clipper(grads, outs=outs, kind=kind).clip(limit)
    assert torch.equal(got, norm) and all(torch.equal(a, b) for a, b in zip(grads, before))
    for g, o in zip(grads, outs):
        assert_within("out", o, ref_clip(g, got, limit, o.dtype))
    # in place: the bits of the outs of the same type
    assert torch.equal(clipper(grads, kind=kind).clip(limit), norm)
    for g, o in zip(grads, outs):
        if o.dtype == g.dtype:
            assert torch.equal(g, o)


def test_short_of_the_limit_nothing_changes():
    grads = grads_of([5000, 1, 333, 70001])
    before = [g.clone() for g in grads]
    norm = clipper(grads).clip(1e6)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    outs = [torch.empty_like(g) for g in grads]
    wide = [torch.empty_like(g, dtype=F32) for g in grads]
    assert torch.equal(clipper(grads, outs=outs).clip(1e6), norm)
    assert torch.equal(clipper(grads, outs=wide).clip(INF), norm)
    assert all(torch.equal(a, b) for a, b in zip(outs, before))
    assert all(torch.equal(a, b.float()) for a, b in zip(wide, before))


def test_a_norm_that_is_given():
    """What ranks have reduced; zero limits; the same clipper again."""
    grads = grads_of([5000, 1, 333])
    outs = [torch.empty_like(g) for g in grads]
    op = clipper(grads, outs=outs)
    given = torch.tensor(40.0, device="cuda")
    assert op.clip(2.5, norm=given) is given
    for g, o in zip(grads, outs):
        assert_within("out", o, ref_clip(g, given, 2.5, o.dtype))
    op.clip(0.0, norm=given)
    assert all((o == 0).all() for o in outs)
    grads[0].mul_(3.0)                       # new contents, the same handle
    norm = op.clip(2.5)
    want, _ = ref_norms(grads, "l2")
    assert_within("norm", norm, (want, 1.01 * U * want))


def test_views_into_a_flat_buffer():
    """Gradients aligned to their elements alone, side by side: what lies between
    and behind them stays."""
    for dt, other in ((BF, BF), (F32, F32), (BF, F32)):
        flat = torch.empty(200000, dtype=dt, device="cuda").normal_()
        out = torch.full((200000,), 7.0, dtype=other, device="cuda")
        cuts = [(1, 2), (3, 40), (45, 2100), (2101, 2102), (2103, 60000), (60001, 199999)]
        grads, outs = [flat[a:b] for a, b in cuts], [out[a:b] for a, b in cuts]
        norm = clipper(grads, outs=outs).clip(3.0)
        want, _ = ref_norms(grads, "l2")
        assert_within("norm", norm, (want, 1.01 * U * want))
        for g, o in zip(grads, outs):
            assert_within("out", o, ref_clip(g, norm, 3.0, other))
        between = torch.ones(200000, dtype=torch.bool, device="cuda")
        for a, b in cuts:
            between[a:b] = False
        assert (out[between] == 7).all()
        keep = flat.clone()
        clipper(grads).clip(3.0)             # in place
        assert torch.equal(flat[between], keep[between])
        if dt == other:
            assert torch.equal(flat[~between], out[~between])
        # outs off their gradients by one element
        shifted = torch.full((200003,), 7.0, dtype=other, device="cuda")
        outs = [shifted[a + 2:b + 2] for a, b in cuts]
        flat.copy_(keep)
        clipper(grads, outs=outs).clip(3.0)
        assert torch.equal(shifted[2:200002], out)
        assert (shifted[:2] == 7).all()


def test_extremes():
    """Squares beyond fp32's range, denormals, infinities, NaN."""
    big = [torch.tensor([3e38, -2e38], device="cuda"), torch.tensor([1e30], device="cuda").to(BF)]
    norm, norms = clipper(big).norm(each=True)
    want, each = ref_norms(big, "l2")
    assert torch.isinf(norm) and torch.isinf(norms[0])    # sqrt(13) 1e38 is beyond fp32 itself
    assert_within("norms", norms[1], (each[1], 1.01 * U * each[1]))
    one = [torch.tensor([2e38, 1e38], device="cuda")]
    want, _ = ref_norms(one, "l2")
    assert_within("norm", clipper(one).norm(), (want, 1.01 * U * want))
    tiny = [torch.full((1000,), 1e-30, device="cuda"), torch.full((10,), 1e-41, device="cuda")]
    norm, norms = clipper(tiny).norm(each=True)
    want, each = ref_norms(tiny, "l2")
    assert_within("norms", norms, (each, 1.01 * U * each + 2.0 ** -149))
    for kind in ("l2", "max"):
        g = grads_of([5000, 700])
        g[1][13] = -INF
        assert torch.isinf(clipper(g, kind=kind).norm())
        outs = [torch.empty_like(t) for t in g]
        clipper(g, outs=outs, kind=kind).clip(1.0)         # c = 0
        assert (outs[0] == 0).all() and torch.isnan(outs[1][13]) and outs[1].nan_to_num().abs().sum() == 0
        g[0][4999] = NAN
        norm, norms = clipper(g, kind=kind).norm(each=True)
        assert torch.isnan(norm) and torch.isnan(norms[0]) and torch.isinf(norms[1])
        clipper(g, outs=outs, kind=kind).clip(1.0)
        assert all(torch.isnan(o).all() for o in outs)


def test_more_than_two_to_the_31_elements():
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=BF, device="cuda")
    g[:1024] = 1.0
    g[-777:] = 2.0
    small = torch.full((3,), 0.5, device="cuda")
    norm, norms = clipper([g, small]).norm(each=True)
    want = torch.tensor([1024 + 4.0 * 777, 0.75], dtype=torch.float64, device="cuda")
    assert_within("norms", norms, (want.sqrt(), 1.01 * U * want.sqrt()))
    clipper([g, small]).clip(float(norm) / 2)
    assert (g[-777:] == 1.0).all() and (g[:1024] == 0.5).all() and g[1024:4096].abs().max() == 0


def test_shapes_and_storage_that_is_replaced():
    a, b = torch.randn(4, 6, 5, device="cuda"), torch.randn(7, 3, device="cuda").to(BF)
    op = clipper([a, b])
    want, _ = ref_norms([a, b], "l2")
    assert_within("norm", op.norm(), (want, 1.01 * U * want))
    a.data = torch.randn(4, 6, 5, device="cuda") * 9
    want, _ = ref_norms([a, b], "l2")
    assert_within("norm", op.norm(), (want, 1.01 * U * want))


def test_refusals_of_the_handle():
    a, b = torch.randn(8, 8, device="cuda"), torch.randn(8, device="cuda")
    from routing_permute_grouped_moe_amd import abi
    with pytest.raises(ValueError, match="no gradients"):
        clipper([])
    with pytest.raises(ValueError, match="contiguous"):
        clipper([a.t(), b])
    with pytest.raises(TypeError):
        clipper([a.half()])
    with pytest.raises(ValueError, match="on cpu"):
        clipper([a, b.cpu()])
    with pytest.raises(TypeError):
        clipper([a], outs=[a.to(BF)])
    with pytest.raises(ValueError, match="1 outs for 2"):
        clipper([a, b], outs=[a])
    with pytest.raises(ValueError, match="kind"):
        clipper([a], kind="l1")
    for grads, outs in (([a, a], None), ([a, a[2:5]], None), ([a[1], b], [b, a[0]]), ([b], [a.flatten()[0:8]])):
        keep = a.clone(), b.clone()
        op = clipper(grads, outs=outs)
        if grads[0] is b:
            op.clip(0.1)            # an out of its own: fine
        else:
            with pytest.raises(abi.MoeError, match="also another's"):
                op.clip(0.1)
            assert torch.equal(a, keep[0]) and torch.equal(b, keep[1])
    with pytest.raises(abi.MoeError, match="max_norm"):
        clipper([a]).clip(-1.0)


def test_streams_and_gradients_dropped_behind_another():
    grads = grads_of([500000, 7, 90001])
    want, outs = clipper(grads).norm(), [torch.empty_like(g) for g in grads]
    clipper(grads, outs=outs).clip(1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    mine, to = [g.clone() for g in grads], [torch.empty_like(g) for g in grads]
    torch.cuda.current_stream().synchronize()
    op = clipper(mine, outs=to)
    norm = op.clip(1.0, stream=side)
    del mine, op
    junk = [torch.full_like(g, NAN) for g in grads for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(outs, to))
    assert len(junk) == 12


def test_replays_from_a_graph():
    grads = grads_of([(i * 7919) % 30000 + 1 for i in range(200)])
    outs = [torch.empty_like(g) for g in grads]
    op = clipper(grads, outs=outs)

    def step():
        norm, norms = op.norm(each=True)
        return [norm, norms, op.clip(2.0)] + outs

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    junk = torch.randn(1 << 18, device="cuda")
    for _ in range(4):
        for t in got:
            t.fill_(NAN)
        junk.mul_(1.01).sum().item()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for a, b in zip(step(), want):
            assert torch.equal(a, b)


def test_two_at_once_and_again():
    """Calls on two streams side by side, over and over: the same bits."""
    one, two = grads_of([400000, 3, 77777]), grads_of([(i * 131) % 3000 for i in range(500)], 1)
    a, b = clipper(one), clipper(two)
    want, want2 = a.norm(each=True, total=True), b.norm(each=True, total=True)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for st in (s, t):
        st.wait_stream(torch.cuda.current_stream())
    got = [(a.norm(each=True, total=True, stream=s), b.norm(each=True, total=True, stream=t))
           for _ in range(8)]
    torch.cuda.synchronize()
    for x, y in got:
        assert all(torch.equal(p, q) for p, q in zip(x, want))
        assert all(torch.equal(p, q) for p, q in zip(y, want2))


def test_parts_of_a_model_reduce_to_the_whole():
    """Squares of two halves added, as ranks do, give the norm of all; each half is
    clipped by it."""
    grads = grads_of([5000, 70001, 12, 333])
    want, _ = ref_norms(grads, "l2")
    halves = clipper(grads[:2]), clipper(grads[2:])
    total = sum(h.norm(total=True)[1] for h in halves)
    norm = total.sqrt().float()
    assert_within("norm", norm, (want, 1.01 * U * want))
    before = [g.clone() for g in grads]
    for h in halves:
        h.clip(1.5, norm=norm)
    for g, b in zip(grads, before):
        assert_within("out", g, ref_clip(b, norm, 1.5, g.dtype))


@pytest.mark.parametrize("sizes", [[1], [0, 0, 3], [0], [2048] * 128, [2049] * 129, [8000] * 128,
                                   [1048576], [1048577], [300000, 7, 0, 600000, 100000], [70000] * 20])
@pytest.mark.parametrize("kind", ["l2", "max"])
def test_in_one_call_or_two(sizes, kind):
    """On either side of where the norm's last launch goes into the scaling: the bits of
    the norm by itself and of scaling by it."""
    grads = grads_of(sizes)
    one, two = [torch.empty_like(g) for g in grads], [torch.empty_like(g) for g in grads]
    norm = clipper(grads, kind=kind).norm()
    got = clipper(grads, outs=one, kind=kind).clip(0.05)
    clipper(grads, outs=two, kind=kind).clip(0.05, norm=norm)
    assert torch.equal(got, norm)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    from routing_permute_grouped_moe_amd import abi
    a = abi.grads(grads, one)
    nb = abi.moe_grad_norm_workspace_bytes(a, len(grads))
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    n1, each = torch.empty(1, device="cuda"), torch.empty(len(grads), device="cuda")
    abi.moe_grad_norm_clip(a, len(grads), abi.MOE_GRAD_MAX if kind == "max" else abi.MOE_GRAD_L2, 0.05, n1,
                           each, ws, nb)
    assert torch.equal(each, clipper(grads, kind=kind).norm(each=True)[1]) and n1.item() == norm.item()


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("sizes", [[5000, 700], [300000, 900001], [100] * 150])
def test_no_limit_scales_nothing_even_an_infinite_norm(sizes, kind):
    """In one call, in two, by a norm that is given, in place and not; a NaN norm is NaN."""
    grads = grads_of(sizes)
    grads[1][13] = -INF
    before = [g.clone() for g in grads]
    outs = [torch.empty_like(g, dtype=F32) for g in grads]
    given = torch.tensor(INF, device="cuda")
    for norm in (None, given):
        assert torch.isinf(clipper(grads, outs=outs, kind=kind).clip(INF, norm=norm))
        assert all(torch.equal(o, b.float()) for o, b in zip(outs, before))
        assert torch.isinf(clipper(grads, kind=kind).clip(INF, norm=norm))
        assert all(torch.equal(g, b) for g, b in zip(grads, before))
    # finite gradients whose norm is beyond fp32
    big = [torch.full((9,), 3e38, device="cuda")]
    if kind == "l2":
        assert torch.isinf(clipper(big).clip(INF)) and (big[0] == 3e38).all()
    # a finite limit still gives c = 0, a NaN norm NaN
    clipper(grads, outs=outs, kind=kind).clip(1e30, norm=given)
    assert (outs[0] == 0).all()
    clipper(grads, outs=outs, kind=kind).clip(INF, norm=torch.tensor(NAN, device="cuda"))
    assert all(torch.isnan(o).all() for o in outs)
    grads[0][7] = NAN
    assert torch.isnan(clipper(grads, outs=outs, kind=kind).clip(INF))
    assert all(torch.isnan(o).all() for o in outs)
