"""What the few-token layer and the fused linear product refuse, and that they
do so on the host, before any GPU work (CPU)."""
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "routing_permute_grouped_moe_amd", "libmoe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")

P = 0x10000           # an aligned address that is never dereferenced on these paths
ODD = 0x10002


@pytest.fixture(scope="module")
def abi():
    from routing_permute_grouped_moe_amd import abi as a
    return a


DECODE = dict(x=P, dt=1, wg=P, bias=None, T=4, H=128, I=64, E=8, k=2, g0=0, G=8, w13=P, w2=P,
              ws13=None, ws2=None, residual=None, logits=P, idx=P, gate=P, y=2 * P, ws=P,
              ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,status,text", [
    ({"T": -1}, "INVALID_ARG", "T = -1"),
    ({"T": 129}, "UNSUPPORTED", "T = 129"),
    ({"T": 128, "E": 64, "G": 64, "k": 33}, "UNSUPPORTED", "pairs"),
    ({"dt": 5}, "INVALID_ARG", "dtype"),
    ({"H": 100}, "UNSUPPORTED", "H = 100"),
    ({"I": 96}, "UNSUPPORTED", "I = 96"),
    ({"I": 0}, "UNSUPPORTED", "I = 0"),
    ({"E": 0}, "UNSUPPORTED", "E = 0"),
    ({"E": 1025}, "UNSUPPORTED", "E = 1025"),
    ({"k": 0}, "UNSUPPORTED", "k = 0"),
    ({"k": 9}, "UNSUPPORTED", "k = 9"),
    ({"g0": -1}, "INVALID_ARG", "g0"),
    ({"G": -1}, "INVALID_ARG", "G"),
    ({"g0": 1}, "INVALID_ARG", "window"),
    ({"H": 1 << 15, "I": 1 << 14}, "UNSUPPORTED", "2 GiB"),
    ({"ws13": P}, "INVALID_ARG", "together"),
    ({"ws2": P}, "INVALID_ARG", "together"),
    ({"wg": None, "bias": P}, "INVALID_ARG", "bias without wg"),
    ({"x": None}, "INVALID_ARG", "x is NULL"),
    ({"x": ODD}, "INVALID_ARG", "x is not"),
    ({"w13": None}, "INVALID_ARG", "w13"),
    ({"w2": ODD}, "INVALID_ARG", "w2"),
    ({"residual": ODD}, "INVALID_ARG", "residual"),
    ({"logits": None}, "INVALID_ARG", "logits"),
    ({"idx": None}, "INVALID_ARG", "idx"),
    ({"gate": None}, "INVALID_ARG", "gate"),
    ({"y": None}, "INVALID_ARG", "y is NULL"),
    ({"y": P}, "INVALID_ARG", "x's buffer"),
    ({"ws": None}, "INVALID_ARG", "ws"),
    ({"ws": 0x10010}, "INVALID_ARG", "ws is not 256"),
    ({"ws_bytes": 1000}, "WORKSPACE", "workspace 1000"),
])
def test_decode_refuses(abi, change, status, text):
    args = {**DECODE, **change}
    st = abi._lib.moe_decode(*args.values())
    assert st == getattr(abi, "MOE_ERR_" + status), abi.moe_last_error()
    assert text in abi.moe_last_error()


def test_decode_without_tokens_is_a_noop(abi):
    args = {**DECODE, **dict.fromkeys(("x", "w13", "w2", "logits", "idx", "gate", "y", "ws")),
            "T": 0, "ws_bytes": 0}
    assert abi._lib.moe_decode(*args.values()) == abi.MOE_OK


def test_decode_workspace(abi):
    n = abi.moe_decode_workspace_bytes(4, 128, 64, 8, 2, abi.MOE_BF16)
    # the activations of 12 rows in two bf16 and their outputs in fp32 at the least
    assert n >= 12 * 64 * 4 + 12 * 128 * 4 and n % 256 == 0
    assert abi.moe_decode_workspace_bytes(200, 128, 64, 8, 2, abi.MOE_BF16) == 0
    args = {**DECODE, "ws_bytes": n - 1}
    assert abi._lib.moe_decode(*args.values()) == abi.MOE_ERR_WORKSPACE


LINEAR = dict(x=P, dt=1, M=4, N=128, K=64, w=P, bias=None, act=0, residual=None, z=None, y=2 * P,
              ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("change,status,text", [
    ({"M": -2}, "INVALID_ARG", "M"),
    ({"N": 100}, "UNSUPPORTED", "N = 100"),
    ({"N": 0}, "UNSUPPORTED", "N = 0"),
    ({"K": 72}, "UNSUPPORTED", "K = 72"),
    ({"dt": -1}, "INVALID_ARG", "dtype"),
    ({"act": 5}, "INVALID_ARG", "act 5"),
    ({"act": -1}, "INVALID_ARG", "act -1"),
    ({"M": 1 << 17, "K": 1 << 14}, "UNSUPPORTED", "x has"),
    ({"M": 1 << 15, "K": 1 << 15}, "UNSUPPORTED", "2 GiB"),
    ({"x": None}, "INVALID_ARG", "x is NULL"),
    ({"w": ODD}, "INVALID_ARG", "w is not"),
    ({"bias": 0x10004}, "INVALID_ARG", "bias"),
    ({"residual": ODD}, "INVALID_ARG", "residual"),
    ({"z": ODD}, "INVALID_ARG", "z is not"),
    ({"y": None}, "INVALID_ARG", "y is NULL"),
    ({"y": P}, "INVALID_ARG", "buffers of their own"),
    ({"z": 2 * P}, "INVALID_ARG", "buffers of their own"),
    ({"w": 2 * P}, "INVALID_ARG", "buffers of their own"),
    ({"z": 3 * P, "residual": 3 * P}, "INVALID_ARG", "buffers of their own"),
    ({"M": 100, "K": 4096}, "INVALID_ARG", "ws is NULL"),
    ({"M": 100, "K": 4096, "ws": P, "ws_bytes": 256}, "WORKSPACE", "workspace 256"),
])
def test_linear_refuses(abi, change, status, text):
    args = {**LINEAR, **change}
    st = abi._lib.moe_linear(*args.values())
    assert st == getattr(abi, "MOE_ERR_" + status), abi.moe_last_error()
    assert text in abi.moe_last_error()


BWD = dict(dy=P, z=P, x=P, w=P, dt=1, M=4, N=128, K=64, act=2, dx=2 * P, dw=3 * P, db=4 * P, ws=P,
           ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,status,text", [
    ({"M": -1}, "INVALID_ARG", "M"),
    ({"N": 65}, "UNSUPPORTED", "N = 65"),
    ({"K": 63}, "UNSUPPORTED", "K = 63"),
    ({"act": 9}, "INVALID_ARG", "act 9"),
    ({"dy": None}, "INVALID_ARG", "dy"),
    ({"z": None}, "INVALID_ARG", "z is NULL"),
    ({"x": None}, "INVALID_ARG", "x is NULL"),
    ({"w": None}, "INVALID_ARG", "w is NULL"),
    ({"dx": ODD}, "INVALID_ARG", "dx"),
    ({"dw": ODD}, "INVALID_ARG", "dw"),
    ({"db": ODD}, "INVALID_ARG", "db"),
    ({"dx": P}, "INVALID_ARG", "buffer of its own"),
    ({"dw": P}, "INVALID_ARG", "dw needs a buffer of its own"),
    ({"db": P}, "INVALID_ARG", "db needs a buffer of its own"),
    ({"dw": 2 * P}, "INVALID_ARG", "dw needs a buffer of its own"),
    ({"ws": None}, "INVALID_ARG", "ws"),
    ({"ws_bytes": 64}, "WORKSPACE", "workspace 64"),
    ({"M": 1 << 15, "K": 1 << 15}, "UNSUPPORTED", "2 GiB"),
])
def test_linear_bwd_refuses(abi, change, status, text):
    args = {**BWD, **change}
    st = abi._lib.moe_linear_bwd(*args.values())
    assert st == getattr(abi, "MOE_ERR_" + status), abi.moe_last_error()
    assert text in abi.moe_last_error()


def test_nothing_asked_for_is_a_noop(abi):
    args = {**LINEAR, "M": 0, "x": None, "w": None, "y": None}
    assert abi._lib.moe_linear(*args.values()) == abi.MOE_OK
    args = {**BWD, "dx": None, "dw": None, "db": None}
    assert abi._lib.moe_linear_bwd(*args.values()) == abi.MOE_OK


@pytest.mark.parametrize("dt", [0, 1])
def test_workspace_sizes_of_every_shape(abi, dt):
    """No shape, empty ones included, trips the host's planning; sizes grow
    from what the pieces need."""
    es = 2 if dt else 4
    for M in (0, 1, 63, 64, 65, 100, 1000, 5000, 100000):
        for N in (64, 192, 2048):
            for K in (64, 1088):
                assert abi.moe_linear_workspace_bytes(M, N, K, dt) % 256 == 0
                for act in (0, 2):
                    n = abi.moe_linear_bwd_workspace_bytes(M, N, K, dt, act)
                    assert n > 0 and n % 256 == 0
                    assert n >= (M * N * es if act else 0)
    assert abi.moe_linear_workspace_bytes(4, 100, 64, dt) == 0


def test_layers_want_weights_on_a_gpu(abi):
    from routing_permute_grouped_moe_amd.layer import LayerShape, Linear, MoeDecode
    w = torch.zeros(64, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="not on a GPU"):
        Linear(w)
    s = LayerShape(T=4, H=64, I=64, E=2, k=1, dtype=torch.bfloat16, router=False)
    with pytest.raises(ValueError, match="not on a GPU"):
        MoeDecode(s, torch.zeros(2, 128, 64), torch.zeros(2, 64, 64))
    with pytest.raises(ValueError, match="wg comes"):
        MoeDecode(s, w, w, wg=w)
    s2 = LayerShape(T=4, H=64, I=64, E=2, k=1, dtype=torch.bfloat16, router=False, capacity=3)
    with pytest.raises(ValueError, match="capacity"):
        MoeDecode(s2, w, w)


def test_tensors_are_checked(abi):
    from routing_permute_grouped_moe_amd.layer import _check
    t = torch.zeros(4, 8)
    cpu = torch.device("cpu")
    _check("t", t, torch.float32, cpu, 4, 8)
    with pytest.raises(TypeError, match="t is torch.float32"):
        _check("t", t, torch.bfloat16, cpu, 4, 8)
    with pytest.raises(ValueError, match="shape"):
        _check("t", t, torch.float32, cpu, 4, 9)
    with pytest.raises(ValueError, match="contiguous"):
        _check("t", torch.zeros(8, 4).t(), torch.float32, cpu, 4, 8)
    with pytest.raises(ValueError, match="the weights are on"):
        _check("t", t, torch.float32, torch.device("cuda", 0), 4, 8)


# ranges that do not meet; y may be residual's very buffer and nothing else
APART = dict(DECODE, w13=0x1000000, w2=0x2000000, wg=0x3000000, logits=0x40000, idx=0x50000,
             gate=0x60000, ws=0x10000000, residual=0x70000, y=0x80000)


@pytest.mark.parametrize("change,text", [
    ({"y": P + 16}, "y overlaps x"),                        # x is 4 x 128 bf16: 1024 bytes
    ({"y": P - 1008}, "y overlaps x"),
    ({"y": 0x70000 + 256}, "y overlaps residual"),          # the residual's, shifted by a row
    ({"y": 0x70000 - 256}, "y overlaps residual"),
    ({"y": 0x1000000 + 4096}, "y overlaps w13"),
    ({"y": 0x2000000 + 8 * 128 * 64 * 2 - 16}, "y overlaps w2"),
    ({"y": 0x3000000}, "y overlaps wg"),
    ({"logits": P}, "logits overlaps x"),
    ({"idx": 0x40000 + 64}, "idx overlaps logits"),
    ({"gate": 0x50000 + 16}, "gate overlaps idx"),
    ({"gate": 0x80000}, "gate overlaps y"),
    ({"ws": 0x80000 - 0x10000}, "ws overlaps"),
    ({"wg": None, "bias": None, "logits": 0x80000}, "logits overlaps y"),
    ({"ws13": 0x4000000, "ws2": 0x5000000, "y": 0x4000000 + 128}, "y overlaps ws13"),
])
def test_decode_refuses_outputs_over_operands(abi, change, text):
    st = abi._lib.moe_decode(*{**APART, **change}.values())
    assert st == abi.MOE_ERR_INVALID_ARG and text in abi.moe_last_error(), abi.moe_last_error()


@pytest.mark.parametrize("change,text", [
    ({"y": P + 16}, "y overlaps x"),
    ({"y": P - 512}, "y overlaps x"),                       # y is 4 x 128 bf16
    ({"w": 0x400000, "y": 0x400000 + 128 * 64 * 2 - 16}, "y overlaps w"),
    ({"residual": 2 * P + 256}, "y overlaps residual"),
    ({"residual": 2 * P - 256}, "y overlaps residual"),
    ({"bias": 2 * P + 64}, "y overlaps bias"),
    ({"z": 2 * P + 1008}, "y overlaps z"),
    ({"z": P + 16}, "z overlaps x"),
    ({"z": 3 * P, "residual": 3 * P - 16}, "z overlaps residual"),
    ({"z": 3 * P, "bias": 3 * P}, "z overlaps bias"),
    ({"M": 100, "K": 4096, "x": 0x1000000, "w": 0x2000000, "ws": 0x1000100, "ws_bytes": 1 << 30},
     "ws overlaps x"),
    ({"M": 100, "K": 4096, "x": 0x1000000, "w": 0x2000000, "ws": 2 * P - 256, "ws_bytes": 1 << 30},
     "y overlaps ws"),
])
def test_linear_refuses_outputs_over_operands(abi, change, text):
    st = abi._lib.moe_linear(*{**LINEAR, **change}.values())
    assert st == abi.MOE_ERR_INVALID_ARG and text in abi.moe_last_error(), abi.moe_last_error()


@pytest.mark.parametrize("change,text", [
    ({"db": 2 * P}, "db needs a buffer of its own, it overlaps dx"),
    ({"db": 3 * P}, "db needs a buffer of its own, it overlaps dw"),
    ({"db": 3 * P + 128 * 64 * 2 - 16}, "db needs a buffer of its own, it overlaps dw"),
    ({"dx": 3 * P + 64}, "dw needs a buffer of its own, it overlaps dx"),
    ({"dx": P + 128}, "overlaps dy"),
    ({"dw": P - 128 * 64 * 2 + 16}, "dw needs a buffer of its own"),
    ({"ws": 2 * P}, "ws overlaps dx"),
    ({"ws": P}, "ws overlaps dy"),
])
def test_linear_bwd_refuses_outputs_over_operands(abi, change, text):
    st = abi._lib.moe_linear_bwd(*{**BWD, "ws": 0x1000000, **change}.values())
    assert st == abi.MOE_ERR_INVALID_ARG and text in abi.moe_last_error(), abi.moe_last_error()


def test_a_bias_without_a_router_is_refused_when_the_layer_is_made(abi):
    from routing_permute_grouped_moe_amd.layer import LayerShape, MoeDecode
    s = LayerShape(T=4, H=64, I=64, E=2, k=1, dtype=torch.bfloat16, router=False)
    w = torch.zeros(2, 128, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="bias comes with wg"):
        MoeDecode(s, w, w, bias=torch.zeros(2))


def test_y_over_a_residual_that_is_x(abi):
    """y may be the residual's buffer, but not x's, also where x is the residual."""
    st = abi._lib.moe_decode(*{**APART, "residual": P, "y": P}.values())
    assert st == abi.MOE_ERR_INVALID_ARG and "y overlaps x" in abi.moe_last_error()
    st = abi._lib.moe_linear(*{**LINEAR, "N": 64, "residual": P, "y": P}.values())
    assert st == abi.MOE_ERR_INVALID_ARG and "y overlaps x" in abi.moe_last_error()


def test_given_logits_are_an_input(abi):
    """Inputs may share memory: given logits with x (the refusal is of gate, here)."""
    st = abi._lib.moe_decode(*{**APART, "wg": None, "logits": P, "gate": 0x50000}.values())
    assert st == abi.MOE_ERR_INVALID_ARG and "gate overlaps idx" in abi.moe_last_error()
