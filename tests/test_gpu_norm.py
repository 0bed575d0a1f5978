"""Layer norm and RMS norm of rows and their gradients against 64 bits (GPU only)."""
import pytest
import torch

from gpu_util import have_gpu
from training_util import EPS, U, assert_within, f64, half_step, ref_norm, ref_norm_bwd

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32


def normal(seed):
    gen = torch.Generator(device="cuda").manual_seed(4000 + seed)
    return lambda *s, std=1.0, mean=0.0, d=BF: torch.empty(s, dtype=d, device="cuda").normal_(
        mean, std, generator=gen)


def make(H, kind, bias, n):
    from routing_permute_grouped_moe_amd.layer import Norm
    return Norm(n(H, std=0.3, mean=1.0, d=F32), bias=n(H, std=0.2, d=F32) if bias else None,
                kind=kind, eps=EPS[kind])


SHAPES = [(1, 8), (3, 8), (1, 7680), (2, 16), (5, 24), (130, 32), (9, 40), (64, 64), (7, 72),
          (4099, 64), (33, 120), (17, 128), (70001, 128), (258, 192), (33, 256), (20, 264), (65, 512),
          (64, 520), (100, 1000), (31, 1024), (12, 1032), (129, 2048), (6, 2056), (1031, 2048),
          (31, 4096), (7, 4104), (257, 7680), (8, 8192), (9, 8200), (3, 12288), (2, 12296),
          (5, 16384), (600, 16384), (1, 16384)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_forward(i, dt):
    M, H = SHAPES[i]
    for kind in ("layer", "rms"):
        residual, bias = (i + (kind == "rms")) % 2 == 0, i % 3 != 0
        print(f"\n[norm] M={M} H={H} {kind} {dt} residual={residual} bias={bias}", flush=True)
        n = normal(M + H)
        op = make(H, kind, bias, n)
        x = n(M, H, std=0.7, mean=0.4, d=dt)
        res = n(M, H, std=2.0, d=dt) if residual else None
        r = op.forward(x, residual=res, save=True)
        if residual:
            full = f64(x) + f64(res)
            assert_within("h", r.h, (full, (half_step(dt) + 1.01 * U) * full.abs()))
        else:
            assert r.h is x
        want = ref_norm(r.h, op.w, op.bias, kind, dt)
        assert_within("y", r.y, want["y"])
        assert_within("rstd", r.rstd, want["rstd"])
        if kind == "layer":
            assert_within("mean", r.mean, want["mean"])
        else:
            assert r.mean is None
        # without the statistics: the same bits
        assert torch.equal(op.forward(x, residual=res).y, r.y)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_backward(i, dt):
    M, H = SHAPES[i]
    for kind in ("layer", "rms"):
        more = (i + (kind == "rms")) % 2 == 0
        print(f"\n[norm bwd] M={M} H={H} {kind} {dt} dh={more}", flush=True)
        n = normal(M + H + 1)
        op = make(H, kind, True, n)
        h, dy = n(M, H, std=1.3, mean=-0.2, d=dt), n(M, H, d=dt)
        dh = n(M, H, d=dt) if more else None
        r = op.forward(h, save=True)
        dx, dw, db = op.backward(dy, h, r.rstd, mean=r.mean, dh=dh)
        rx, rw, rb = ref_norm_bwd(dy, h, op.w, r.mean, r.rstd, dh, kind, dt)
        assert_within("dx", dx, rx)
        assert_within("dw", dw, rw)
        assert_within("db", db, rb)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("M,H", [(37, 72), (5, 2056)])
def test_gradients_against_differences(M, H, kind):
    """The derivative of <y, dy> + <h, dh> along random directions of x, w and the
    bias by central differences of the 64-bit forward."""
    n = normal(77)
    op = make(H, kind, True, n)
    x, res, dy, dh = (n(M, H, d=F32) for _ in range(4))
    r = op.forward(x, residual=res, save=True)
    grads = op.backward(dy, r.h, r.rstd, mean=r.mean, dh=dh)
    X, W, B = f64(r.h), f64(op.w), f64(op.bias)

    def phi(X, W, B):
        m = X.mean(1, keepdim=True) if kind == "layer" else 0.0
        q = (X - m) / torch.sqrt(((X - m) ** 2).mean(1, keepdim=True) + EPS[kind])
        return ((q * W + B) * f64(dy)).sum() + (X * f64(dh)).sum()

    bounds = ref_norm_bwd(dy, r.h, op.w, r.mean if kind == "layer" else None, r.rstd, dh, kind, F32)
    eps = 1e-5
    for at, grad in enumerate(grads):
        v = torch.randn((X, W, B)[at].shape, dtype=torch.float64, device="cuda",
                        generator=torch.Generator(device="cuda").manual_seed(at))
        args = lambda s: [p + s * v if i == at else p for i, p in enumerate((X, W, B))]
        num = (phi(*args(eps)) - phi(*args(-eps))) / (2 * eps)
        got = (f64(grad) * v).sum()
        # the statistics given are off by a few u of themselves; differences by eps^2
        slack = (bounds[at][1] * v.abs()).sum() + 1e-5 * (f64(grad) * v).abs().sum() + 1e-6
        assert abs(num - got) <= slack, (at, num.item(), got.item(), slack.item())


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,H", [(1, 7680), (3, 64), (300, 512), (70, 5120), (4, 16384)])
def test_buffers_of_the_inputs_and_nothing_behind(M, H, dt):
    """h over the residual or x, dx over dh: the same bits, rows behind the last
    as they were."""
    n = normal(3)
    op = make(H, "layer", True, n)
    x, res, dy = n(M, H, d=dt), n(M + 3, H, d=dt), n(M, H, d=dt)
    keep = res.clone()
    want = op.forward(x, residual=keep[:M], save=True)
    y = torch.full((M + 3, H), 7.0, dtype=dt, device="cuda")
    got = op.forward(x, residual=res[:M], h_out=res[:M], out=y[:M])
    assert torch.equal(got.h, want.h) and torch.equal(res[:M], want.h)
    assert torch.equal(res[M:], keep[M:])
    assert torch.equal(y[:M], want.y) and (y[M:] == 7).all()
    x2 = x.clone()
    got = op.forward(x2, residual=keep[:M], h_out=x2)
    assert torch.equal(x2, want.h) and torch.equal(got.y, want.y)
    dx, dw, db = op.backward(dy, want.h, want.rstd, mean=want.mean, dh=keep[:M])
    buf = keep.clone()
    dx2, dw2, db2 = op.backward(dy, want.h, want.rstd, mean=want.mean, dh=buf[:M], out=buf[:M])
    assert torch.equal(buf[:M], dx) and torch.equal(buf[M:], keep[M:])
    assert torch.equal(dw, dw2) and torch.equal(db, db2)


@pytest.mark.parametrize("M,H,dt", [(300, 256, BF), (700, 2048, F32), (40, 7680, BF), (2, 8, F32)])
def test_only_the_gradients_asked_for(M, H, dt):
    n = normal(5)
    op = make(H, "layer", True, n)
    h, dy = n(M, H, d=dt), n(M, H, d=dt)
    r = op.forward(h, save=True)
    want = op.backward(dy, h, r.rstd, mean=r.mean)
    for asked in range(8):
        on = [bool(asked >> i & 1) for i in range(3)]
        got = op.backward(dy, h, r.rstd, mean=r.mean, x_grad=on[0], w_grad=on[1], bias_grad=on[2])
        for i in range(3):
            assert torch.equal(got[i], want[i]) if on[i] else got[i] is None, (on, i)


def test_no_rows():
    n = normal(6)
    op = make(64, "layer", True, n)
    x = n(0, 64)
    r = op.forward(x, residual=x, save=True)
    assert r.y.shape == (0, 64) and r.rstd.shape == (0,)
    dx, dw, db = op.backward(x, x, r.rstd, mean=r.mean)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("M,H", [(40, 128), (9, 2048), (5, 8192)])
def test_equal_values_nan_and_infinities(M, H):
    """A row of one value has y = bias; a NaN or an infinity makes its own row NaN
    and, of the gradients, its row of dx and all of dw."""
    n = normal(8)
    for dt in (BF, F32):
        op = make(H, "layer", True, n)
        x = n(M, H, d=dt)
        x[1] = 1.5
        x[2, 3], x[3, H - 1] = float("nan"), float("inf")
        r = op.forward(x, save=True)
        assert torch.equal(r.y[1], op.bias.to(dt)) and torch.isfinite(r.rstd[1])
        bad = [2, 3]
        good = [i for i in range(M) if i not in bad]
        assert torch.isnan(r.y[bad]).all() and torch.isfinite(r.y[good]).all()
        dx, dw, _ = op.backward(n(M, H, d=dt), x, r.rstd, mean=r.mean)
        assert torch.isnan(dx[bad]).all() and torch.isfinite(dx[good]).all()
        assert torch.isnan(dw).all()


def test_rows_past_two_to_the_31_bytes():
    """2^31 - 2 million elements of bf16, just below the limit: the last rows."""
    n = normal(9)
    M, H = 262143, 8184
    op = make(H, "rms", False, n)
    x = torch.empty(M, H, dtype=BF, device="cuda").fill_(1.0)
    x[-5:] = n(5, H)
    r = op.forward(x, save=True)
    want = ref_norm(x[-5:], op.w, None, "rms", BF)
    assert_within("y", r.y[-5:], want["y"])
    assert torch.equal(r.y[0], r.y[M - 6])
    dx, dw, _ = op.backward(r.y, x, r.rstd, w_grad=False)
    rx, _, _ = ref_norm_bwd(r.y[-5:], x[-5:], op.w, None, r.rstd[-5:], None, "rms", BF)
    assert_within("dx", dx[-5:], rx)
    assert dw is None


def test_streams_and_inputs_dropped_behind_another():
    n = normal(10)
    M, H = 500, 1024
    op = make(H, "layer", True, n)
    x, res, dy = n(M, H), n(M, H), n(M, H)
    want = op.forward(x, residual=res, save=True)
    grads = op.backward(dy, want.h, want.rstd, mean=want.mean, dh=res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    x1, res1, dy1 = x.clone(), res.clone(), dy.clone()
    torch.cuda.current_stream().synchronize()
    got = op.forward(x1, residual=res1, save=True, stream=side)
    back = op.backward(dy1, got.h, got.rstd, mean=got.mean, dh=res1, stream=side)
    del x1, res1, dy1
    junk = [torch.full_like(x, float("nan")) for _ in range(9)]
    torch.cuda.synchronize()
    assert torch.equal(got.y, want.y) and torch.equal(got.h, want.h)
    assert all(torch.equal(a, b) for a, b in zip(grads, back)) and len(junk) == 9


@pytest.mark.parametrize("M,H,dt", [(520, 320, BF), (70, 7680, BF), (1, 2048, F32)])
def test_replays_from_a_graph(M, H, dt):
    n = normal(11)
    op = make(H, "layer", True, n)
    x, res, dy = n(M, H, d=dt), n(M, H, d=dt), n(M, H, d=dt)

    def step():
        r = op.forward(x, residual=res, save=True)
        return tuple(r) + op.backward(dy, r.h, r.rstd, mean=r.mean, dh=dy)

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
            t.fill_(float("nan"))
        junk.mul_(1.01).sum().item()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        for a, b in zip(step(), want):
            assert torch.equal(a, b)


def test_two_at_once_and_again():
    """Calls on two streams side by side, over and over: the same bits."""
    n = normal(12)
    one, two = make(7680, "layer", True, n), make(128, "rms", False, n)
    x, dy = n(600, 7680), n(600, 7680)
    x2, dy2 = n(30011, 128, d=F32), n(30011, 128, d=F32)

    def step(op, x, dy, stream=None):
        r = op.forward(x, residual=dy, save=True, stream=stream)
        grads = op.backward(dy, r.h, r.rstd, mean=r.mean, bias_grad=True, stream=stream)
        return [t for t in (*r, *grads) if t is not None]

    want, want2 = step(one, x, dy), step(two, x2, dy2)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (a, b):
        s.wait_stream(torch.cuda.current_stream())
    got = [(step(one, x, dy, a), step(two, x2, dy2, b)) for _ in range(6)]
    torch.cuda.synchronize()
    for p, q in got:
        assert all(torch.equal(u, v) for u, v in zip(p, want))
        assert all(torch.equal(u, v) for u, v in zip(q, want2))


@pytest.mark.parametrize("dt", [BF, F32])
def test_either_side_of_the_streaming_policy(dt):
    """Rows of just under and just over 256 MB, read and written: the same bits for
    the rows that both have."""
    n = normal(13)
    H = 2048
    M = (64 << 20) // (H * (2 if dt == BF else 4))          # four tensors of 64 MB
    op = make(H, "layer", True, n)
    x, res, dy = (n(M + 1, H, d=dt) for _ in range(3))
    out = []
    for m in (M, M + 1):
        r = op.forward(x[:m], residual=res[:m], save=True)
        dx, _, _ = op.backward(dy[:m], r.h, r.rstd, mean=r.mean, dh=res[:m])
        out.append([t[:M] for t in (r.y, r.h, r.mean, r.rstd, dx)])
    assert all(torch.equal(a, b) for a, b in zip(*out))


@pytest.mark.parametrize("M,H", [(50, 64), (40, 1000), (33, 2056), (9, 7680), (5, 16384)])
@pytest.mark.parametrize("offset", [1.5, 1000.0, -3e4])
def test_rows_far_from_zero(M, H, offset):
    """Deviations far smaller than the mean, or none at all: the mean is corrected by
    the deviations from it."""
    n = normal(14)
    for dt in (F32, BF):
        op = make(H, "layer", True, n)
        x = n(M, H, std=abs(offset) * (1e-4 if dt == F32 else 0.02), mean=offset, d=dt)
        x[1] = offset
        x[2, 1:] = offset
        r = op.forward(x, save=True)
        want = ref_norm(x, op.w, op.bias, "layer", dt)
        for name in ("mean", "rstd", "y"):
            assert_within(name, getattr(r, name), want[name])
        assert torch.equal(r.y[1], op.bias.to(dt)) and r.mean[1] == x[1, 0].float()


def test_backward_without_statistics_is_refused():
    n = normal(15)
    op = make(64, "layer", False, n)
    x = n(3, 64)
    r = op.forward(x)
    assert r.mean is None and r.rstd is None
    with pytest.raises(ValueError, match="a forward with save"):
        op.backward(x, r.h, r.rstd, mean=r.mean)


@pytest.mark.parametrize("M,H", [((1 << 27) - 70, 8), ((1 << 23) - 3, 128), (100_003, 8192)])
def test_long_sums_of_like_rows(M, H):
    """All rows alike, so that every addition of dw and db rounds the same way.  At most 240
    rows are added in fp32 by a thread, then 3 lanes' worth and 7 waves' (8 rows side by side
    in a wave, 8 waves), the rest in 64 bits, rounded once: 251 u; dy / 2 is exact."""
    n = normal(16)
    op = make(H, "rms", True, n)
    row = torch.tensor([0.1, 0.3, -0.7, 1.1, 1 / 3, 0.9, -0.123, 0.6], device="cuda").repeat(H // 8)
    dy = row.expand(M, H).contiguous()
    h = torch.full((M, H), 0.5, device="cuda")
    rstd = torch.ones(M, device="cuda")
    _, dw, db = op.backward(dy, h, rstd, x_grad=False)
    for name, got, each in (("db", db, f64(row)), ("dw", dw, 0.5 * f64(row))):
        assert_within(name, got, (M * each, 251 * U * M * each.abs()))
