"""What the row norms, the router's losses and gradient clipping refuse, and that
they do so on the host, before any GPU work (CPU)."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "routing_permute_grouped_moe_amd", "libmoe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")

# aligned addresses far apart that are never dereferenced on these paths
A, B, C, D, E, F, G, H, W = (0x10000000 * i for i in range(1, 10))


@pytest.fixture(scope="module")
def abi():
    from routing_permute_grouped_moe_amd import abi as a
    return a


def refused(abi, name, args, status, text):
    st = getattr(abi._lib, name)(*args.values())
    assert st == getattr(abi, "MOE_ERR_" + status), (st, abi.moe_last_error())
    assert text in abi.moe_last_error(), abi.moe_last_error()


NORM = dict(x=A, residual=None, dt=1, M=4, H=128, kind=0, eps=1e-5, w=B, bias=None, h=None, y=C,
            mean=D, rstd=E, stream=None)


@pytest.mark.parametrize("change,status,text", [
    ({"dt": 2}, "INVALID_ARG", "dtype"),
    ({"M": -1}, "INVALID_ARG", "M = -1"),
    ({"H": 0}, "UNSUPPORTED", "H = 0"),
    ({"H": 4}, "UNSUPPORTED", "H = 4"),
    ({"H": 100}, "UNSUPPORTED", "H = 100"),
    ({"H": 16392}, "UNSUPPORTED", "H = 16392"),
    ({"M": 1 << 20, "H": 2048}, "UNSUPPORTED", "above the limit"),
    ({"kind": 2}, "INVALID_ARG", "kind 2"),
    ({"eps": 0.0}, "INVALID_ARG", "eps"),
    ({"eps": -1.0}, "INVALID_ARG", "eps"),
    ({"eps": float("nan")}, "INVALID_ARG", "eps"),
    ({"eps": float("inf")}, "INVALID_ARG", "eps"),
    ({"x": None}, "INVALID_ARG", "x is NULL"),
    ({"x": A + 2}, "INVALID_ARG", "x is not"),
    ({"w": None}, "INVALID_ARG", "w is NULL"),
    ({"bias": B + 4}, "INVALID_ARG", "bias"),
    ({"residual": F + 8}, "INVALID_ARG", "residual"),
    ({"h": F}, "INVALID_ARG", "without a residual"),
    ({"y": None}, "INVALID_ARG", "y is NULL"),
    ({"rstd": E + 2}, "INVALID_ARG", "rstd"),
    ({"y": A}, "INVALID_ARG", "y overlaps x"),
    ({"y": A + 1008}, "INVALID_ARG", "y overlaps x"),
    ({"residual": F, "y": F}, "INVALID_ARG", "y overlaps residual"),
    ({"y": B}, "INVALID_ARG", "y overlaps w"),
    ({"bias": C + 512}, "INVALID_ARG", "y overlaps bias"),
    ({"residual": F, "h": C}, "INVALID_ARG", "y overlaps h"),
    ({"residual": F, "h": F + 256}, "INVALID_ARG", "h overlaps residual"),
    ({"residual": F, "h": A - 256}, "INVALID_ARG", "h overlaps x"),
    ({"mean": C + 16}, "INVALID_ARG", "mean overlaps y"),
    ({"rstd": D + 12}, "INVALID_ARG", "rstd overlaps mean"),
])
def test_norm_refuses(abi, change, status, text):
    refused(abi, "moe_norm", {**NORM, **change}, status, text)


NORM_BWD = dict(dy=A, h=B, dh=None, dt=1, M=4, H=128, kind=0, w=C, mean=D, rstd=E, dx=F, dw=G, db=H,
                ws=W, ws_bytes=1 << 26, stream=None)


@pytest.mark.parametrize("change,status,text", [
    ({"M": -3}, "INVALID_ARG", "M = -3"),
    ({"H": 12}, "UNSUPPORTED", "H = 12"),
    ({"kind": -1}, "INVALID_ARG", "kind"),
    ({"dy": None}, "INVALID_ARG", "dy is NULL"),
    ({"h": None}, "INVALID_ARG", "h is NULL"),
    ({"w": None}, "INVALID_ARG", "w is NULL"),
    ({"mean": None}, "INVALID_ARG", "mean is NULL"),
    ({"rstd": None}, "INVALID_ARG", "rstd is NULL"),
    ({"dh": 3}, "INVALID_ARG", "dh is not"),
    ({"dx": F + 4}, "INVALID_ARG", "dx is not"),
    ({"ws": None}, "INVALID_ARG", "ws is NULL"),
    ({"ws": W + 16}, "INVALID_ARG", "ws is not 256"),
    ({"ws_bytes": 100}, "WORKSPACE", "workspace 100"),
    ({"dx": A}, "INVALID_ARG", "dx overlaps dy"),
    ({"dx": B + 512}, "INVALID_ARG", "dx overlaps h"),
    ({"dh": F + 16}, "INVALID_ARG", "dx overlaps dh"),
    ({"dw": F + 512}, "INVALID_ARG", "dw overlaps dx"),
    ({"db": G + 256}, "INVALID_ARG", "db overlaps dw"),
    ({"db": C}, "INVALID_ARG", "db overlaps w"),
    ({"ws": F}, "INVALID_ARG", "ws overlaps dx"),
    ({"dh": W}, "INVALID_ARG", "ws overlaps dh"),
])
def test_norm_bwd_refuses(abi, change, status, text):
    refused(abi, "moe_norm_bwd", {**NORM_BWD, **change}, status, text)


def test_norm_of_nothing_is_a_noop(abi):
    none = dict.fromkeys(("x", "w", "y", "mean", "rstd"))
    assert abi._lib.moe_norm(*{**NORM, **none, "M": 0}.values()) == abi.MOE_OK
    none = dict.fromkeys(("dx", "dw", "db", "ws"))
    assert abi._lib.moe_norm_bwd(*{**NORM_BWD, **none, "M": 0}.values()) == abi.MOE_OK


def test_norm_workspace(abi):
    for M in (0, 1, 7, 300, 5000, 100000):
        for H_ in (8, 72, 1024, 7680, 16384):
            n = abi.moe_norm_bwd_workspace_bytes(M, H_, 1)
            assert n % 256 == 0 and n <= 2048 * 2 * H_ * 4 + 256
    assert abi.moe_norm_bwd_workspace_bytes(4, 12, 1) == 0
    n = abi.moe_norm_bwd_workspace_bytes(4000, 128, 1)
    refused(abi, "moe_norm_bwd", {**NORM_BWD, "M": 4000, "ws_bytes": n - 1}, "WORKSPACE", "needed")


BALANCE = dict(logits=A, idx=B, keep=None, seq=None, T=3000, E=8, k=2, S=1, w=0.1, wz=0.1, loss=C,
               counts=D, tokens=E, prob=F, ws=W, ws_bytes=1 << 26, stream=None)


@pytest.mark.parametrize("change,status,text", [
    ({"T": -1}, "INVALID_ARG", "T = -1"),
    ({"E": 0}, "UNSUPPORTED", "E = 0"),
    ({"E": 1025}, "UNSUPPORTED", "E = 1025"),
    ({"k": 9}, "UNSUPPORTED", "k = 9"),
    ({"k": 0}, "UNSUPPORTED", "k = 0"),
    ({"S": 0}, "INVALID_ARG", "S = 0"),
    ({"S": 65536, "seq": G}, "UNSUPPORTED", "S = 65536"),
    ({"S": 2}, "INVALID_ARG", "without seq"),
    ({"T": 1 << 28}, "UNSUPPORTED", "logits has"),
    ({"logits": None}, "INVALID_ARG", "logits is NULL"),
    ({"logits": A + 2}, "INVALID_ARG", "logits is not"),
    ({"idx": None}, "INVALID_ARG", "idx is NULL"),
    ({"seq": G + 1}, "INVALID_ARG", "seq is not"),
    ({"loss": None}, "INVALID_ARG", "loss is NULL"),
    ({"counts": None}, "INVALID_ARG", "counts is NULL"),
    ({"tokens": None}, "INVALID_ARG", "tokens is NULL"),
    ({"prob": F + 2}, "INVALID_ARG", "prob is not"),
    ({"ws": None}, "INVALID_ARG", "ws is NULL"),
    ({"ws_bytes": 16}, "WORKSPACE", "workspace 16"),
    ({"loss": A + 95992}, "INVALID_ARG", "loss needs a buffer of its own, it overlaps logits"),
    ({"counts": B}, "INVALID_ARG", "counts needs a buffer of its own, it overlaps idx"),
    ({"tokens": D + 28}, "INVALID_ARG", "tokens needs a buffer of its own, it overlaps counts"),
    ({"keep": F + 16}, "INVALID_ARG", "prob needs a buffer of its own, it overlaps keep"),
    ({"ws": F}, "INVALID_ARG", "ws needs a buffer of its own, it overlaps prob"),
])
def test_balance_refuses(abi, change, status, text):
    refused(abi, "moe_balance_loss", {**BALANCE, **change}, status, text)


BALANCE_BWD = dict(logits=A, idx=B, dgate=C, keep=None, seq=None, counts=D, tokens=E, T=100, E=8, k=2,
                   S=1, w=0.1, wz=0.1, dloss=None, dlogits=F, stream=None)


@pytest.mark.parametrize("change,status,text", [
    ({"T": -1}, "INVALID_ARG", "T = -1"),
    ({"k": 9}, "UNSUPPORTED", "k = 9"),
    ({"S": 3}, "INVALID_ARG", "without seq"),
    ({"T": 1 << 27, "E": 7}, "UNSUPPORTED", "T = 134217728"),
    ({"logits": None}, "INVALID_ARG", "logits is NULL"),
    ({"idx": None}, "INVALID_ARG", "idx is NULL"),
    ({"dgate": C + 1}, "INVALID_ARG", "dgate is not"),
    ({"counts": None}, "INVALID_ARG", "counts is NULL"),
    ({"tokens": None}, "INVALID_ARG", "tokens is NULL"),
    ({"dloss": G + 2}, "INVALID_ARG", "dloss is not"),
    ({"dlogits": None}, "INVALID_ARG", "dlogits is NULL"),
    ({"dlogits": A}, "INVALID_ARG", "it overlaps logits"),
    ({"dlogits": C - 64}, "INVALID_ARG", "it overlaps dgate"),
    ({"dlogits": D}, "INVALID_ARG", "it overlaps counts"),
    ({"dloss": F + 64}, "INVALID_ARG", "it overlaps dloss"),
])
def test_balance_bwd_refuses(abi, change, status, text):
    refused(abi, "moe_balance_loss_bwd", {**BALANCE_BWD, **change}, status, text)


def test_balance_sizes(abi):
    """Workspaces of every size are planned without a trip; T == 0 has a backward
    that does nothing."""
    for T in (0, 1, 2, 511, 512, 8192, 100000, (1 << 30) - 1):
        for S in (1, 2, 700, 65535):
            n = abi.moe_balance_loss_workspace_bytes(T, 1, 1, S)
            assert n % 256 == 0 and (n > 0 or T <= 512)
    assert abi.moe_balance_loss_workspace_bytes(4, 8, 9, 1) == 0
    none = dict.fromkeys(("logits", "idx", "dgate", "counts", "tokens", "dlogits"))
    assert abi._lib.moe_balance_loss_bwd(*{**BALANCE_BWD, **none, "T": 0}.values()) == abi.MOE_OK


def arr(abi, *rows):
    a = (abi.Grad * max(1, len(rows)))()
    for x, (g, out, n, dt, odt) in zip(a, rows):
        x.g, x.out, x.n, x.dt, x.out_dt = g, out, n, dt, odt
    return a


@pytest.mark.parametrize("rows,change,status,text", [
    ([(A, A, 5, 0, 0)], {"count": -1}, "INVALID_ARG", "count = -1"),
    ([(A, A, 5, 0, 0)], {"count": (1 << 20) + 1}, "UNSUPPORTED", "gradients"),
    ([(A, A, 5, 0, 0)], {"grads": None}, "INVALID_ARG", "grads is NULL"),
    ([(A, A, -5, 0, 0)], {}, "INVALID_ARG", "-5 elements"),
    ([(A, A, 5, 3, 0)], {}, "INVALID_ARG", "dtype 3"),
    ([(None, A, 5, 0, 0)], {}, "INVALID_ARG", "a gradient is NULL"),
    ([(A + 2, A, 5, 0, 0)], {}, "INVALID_ARG", "a gradient is not 4-byte"),
    ([(A + 1, A, 5, 1, 1)], {}, "INVALID_ARG", "a gradient is not 2-byte"),
])
def test_grad_calls_refuse(abi, rows, change, status, text):
    a = {"grads": arr(abi, *rows), "count": len(rows), **change}
    refused(abi, "moe_grad_norm", dict(a, kind=0, norm=B, norms=None, total=None, ws=W,
                                       ws_bytes=1 << 26, stream=None), status, text)
    refused(abi, "moe_grad_clip", dict(a, norm=B, max_norm=1.0, stream=None), status, text)


GN = dict(kind=0, norm=B, norms=C, total=D, ws=W, ws_bytes=1 << 26, stream=None)


@pytest.mark.parametrize("change,status,text", [
    ({"kind": 2}, "INVALID_ARG", "kind 2"),
    ({"norm": None}, "INVALID_ARG", "norm is NULL"),
    ({"norms": C + 2}, "INVALID_ARG", "norms is not"),
    ({"total": D + 4}, "INVALID_ARG", "total is not"),
    ({"ws": None}, "INVALID_ARG", "ws is NULL"),
    ({"ws": W + 128}, "INVALID_ARG", "ws is not 256"),
    ({"ws_bytes": 8}, "WORKSPACE", "workspace 8"),
    ({"norm": A + 16}, "INVALID_ARG", "norm needs a buffer of its own, it overlaps a gradient"),
    ({"norms": B - 4}, "INVALID_ARG", "norms needs a buffer of its own, it overlaps norm"),
    ({"ws": A - 256}, "INVALID_ARG", "ws needs a buffer of its own, it overlaps a gradient"),
])
def test_grad_norm_refuses(abi, change, status, text):
    a = arr(abi, (A, A, 5, 0, 0), (E, E, 0, 0, 0), (F, F, 1000, 1, 1))
    refused(abi, "moe_grad_norm", {**dict(grads=a, count=3), **GN, **change}, status, text)


@pytest.mark.parametrize("rows,max_norm,norm,text", [
    ([(A, None, 5, 0, 0)], 1.0, B, "an out is NULL"),
    ([(A, A + 1, 5, 1, 1)], 1.0, B, "an out is not 2-byte"),
    ([(A, C, 5, 0, 1)], 1.0, B, "neither its gradient's nor MOE_F32"),
    ([(A, A, 5, 1, 0)], 1.0, B, "of another type"),
    ([(A, A, 5, 0, 0)], -1.0, B, "max_norm"),
    ([(A, A, 5, 0, 0)], float("nan"), B, "max_norm"),
    ([(A, A, 5, 0, 0)], 1.0, None, "norm is NULL"),
    ([(A, A, 5, 0, 0)], 1.0, A + 16, "overlaps norm"),
    ([(A, A, 5, 0, 0), (A, A, 5, 0, 0)], 1.0, B, "also another's"),
    ([(A, A, 5, 0, 0), (A + 16, A + 16, 9, 0, 0)], 1.0, B, "also another's"),
    ([(A, C, 5, 0, 0), (D, C + 16, 9, 0, 0)], 1.0, B, "also another's"),
    ([(A, C, 5, 0, 0), (C + 8, D, 1, 0, 0)], 1.0, B, "also another's"),
    ([(A, A + 4, 5, 0, 0)], 1.0, B, "also another's"),
    ([(A, C, 500, 1, 0), (C + 1996, D, 1, 0, 0)], 1.0, B, "also another's"),
])
def test_grad_clip_refuses(abi, rows, max_norm, norm, text):
    args = dict(grads=arr(abi, *rows), count=len(rows), norm=norm, max_norm=max_norm, stream=None)
    refused(abi, "moe_grad_clip", args, "INVALID_ARG", text)


@pytest.mark.parametrize("rows,change,status,text", [
    ([(A, A, 5, 0, 0)], {"kind": 3}, "INVALID_ARG", "kind 3"),
    ([(A, A, 5, 0, 0)], {"max_norm": -0.5}, "INVALID_ARG", "max_norm"),
    ([(A, A, 5, 0, 0)], {"norm": None}, "INVALID_ARG", "norm is NULL"),
    ([(A, A, 5, 0, 0)], {"ws_bytes": 64}, "WORKSPACE", "workspace 64"),
    ([(A, None, 5, 0, 0)], {}, "INVALID_ARG", "an out is NULL"),
    ([(A, C, 5, 0, 1)], {}, "INVALID_ARG", "neither its gradient's nor MOE_F32"),
    ([(A, A, 5, 0, 0), (A + 8, A + 8, 5, 0, 0)], {}, "INVALID_ARG", "also another's"),
    ([(A, B + 4, 5, 0, 0)], {"norms": B + 16}, "INVALID_ARG", "overlaps norms"),
    ([(A, B, 5, 0, 0)], {}, "INVALID_ARG", "out 0 overlaps norm"),
    ([(A, W + 16, 5, 0, 0)], {}, "INVALID_ARG", "out 0 overlaps ws"),
    ([(A, A, 5, 0, 0)], {"norm": A}, "INVALID_ARG", "norm needs a buffer of its own"),
])
def test_grad_norm_clip_refuses(abi, rows, change, status, text):
    args = {**dict(grads=arr(abi, *rows), count=len(rows), kind=0, max_norm=1.0, norm=B, norms=None,
                   ws=W, ws_bytes=1 << 26, stream=None), **change}
    refused(abi, "moe_grad_norm_clip", args, status, text)


def test_clip_of_nothing_is_a_noop(abi):
    args = dict(grads=None, count=0, norm=B, max_norm=1.0, stream=None)
    assert abi._lib.moe_grad_clip(*args.values()) == abi.MOE_OK
    a = arr(abi, (None, None, 0, 0, 0), (None, None, 0, 1, 1))
    assert abi._lib.moe_grad_clip(*{**args, "grads": a, "count": 2}.values()) == abi.MOE_OK


def test_grad_workspace(abi):
    assert abi.moe_grad_norm_workspace_bytes(None, 0) % 256 == 0
    for n in (0, 1, 16384, 16385, 1 << 28, 1 << 35):
        a = arr(abi, (A, A, n, 0, 0), (B, B, 7, 1, 1))
        got = abi.moe_grad_norm_workspace_bytes(a, 2)
        assert got % 256 == 0 and 256 <= got <= (1 << 20)
    assert abi.moe_grad_norm_workspace_bytes(arr(abi, (A, A, -1, 0, 0)), 1) == 0
    assert ctypes.sizeof(abi.Grad) == 32


def test_classes_want_tensors_on_a_gpu(abi):
    from routing_permute_grouped_moe_amd.layer import BalanceLoss, GradClip, Norm
    w = torch.ones(64)
    with pytest.raises(ValueError, match="not on a GPU"):
        Norm(w)
    with pytest.raises(ValueError, match="logits are on cpu, not on a GPU"):
        BalanceLoss().forward(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="gradients are on cpu, not on a GPU"):
        GradClip([w])


@pytest.mark.parametrize("T", [1 << 27, (1 << 27) + 5, 1 << 28, (1 << 30) - 1])
def test_balance_forward_and_backward_refuse_the_same_tokens(abi, T):
    """What a forward takes its backward takes: neither takes 2^27 tokens."""
    text = f"T = {T}, above the limit"
    change = {"T": T, "E": 1, "k": 1, "ws_bytes": 1 << 40}
    far = dict(logits=A, idx=A + (1 << 34), loss=A + (2 << 34), counts=A + (3 << 34),
               tokens=A + (4 << 34), prob=A + (5 << 34), ws=A + (6 << 34))
    refused(abi, "moe_balance_loss", {**BALANCE, **change, **far}, "UNSUPPORTED", text)
    far = dict(logits=A, idx=A + (1 << 34), dgate=A + (2 << 34), counts=A + (3 << 34),
               tokens=A + (4 << 34), dlogits=A + (5 << 34))
    change = {n: change[n] for n in ("T", "E", "k")}
    refused(abi, "moe_balance_loss_bwd", {**BALANCE_BWD, **change, **far}, "UNSUPPORTED", text)
