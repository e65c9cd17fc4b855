"""Argument checks of the norm, the weights' quantisation and the products on
FP8 rows, on the host: every call here fails a check, or returns, before
anything touches a GPU, so the pointers are never dereferenced."""

import ctypes
import math
import types

import pytest
import torch

from test_binding_devices_host import Tensor

FAKE, MIS = 0x10000, 0x10002
BF, F, I, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def moe():
    import combine_route_topk_amd
    return combine_route_topk_amd


def test_norm_validation(moe):
    def call(x=FAKE, r=FAKE, w=FAKE, T=4, H=64, eps=1e-6, flags=0, total=FAKE, y=FAKE, y8=FAKE):
        return moe.lib.moe_rms_norm(x, r, w, T, H, eps, flags, total, y, y8, None)

    bad, un = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    assert call(T=0, x=None, r=None, w=None, total=None, y=None, y8=None) == moe.MOE_OK
    assert call(T=-1) == bad and call(T=2 ** 31) == un
    assert call(H=0) == un and call(H=12) == un and call(H=65544) == un
    assert call(H=40) == un                       # FP8 rows need whole blocks of 32
    assert call(eps=-1.0) == bad and call(eps=math.nan) == bad and call(eps=math.inf) == bad
    assert call(flags=4) == bad and call(flags=8) == bad
    assert call(x=None) == bad and call(w=None) == bad and call(y=None, y8=None) == bad
    assert call(r=None) == bad and call(total=None) == bad  # together or not at all
    for name in ("x", "r", "w", "total", "y", "y8"):
        assert call(**{name: FAKE + 8}) == bad


def test_norm_backward_validation(moe):
    ws = moe.moe_rms_norm_backward_workspace_size(4, 64)

    def call(gy=FAKE, t=FAKE, w=FAKE, T=4, H=64, eps=1e-6, flags=0, gt=None, gx=FAKE, gw=FAKE, wsp=FAKE, n=ws):
        return moe.lib.moe_rms_norm_backward(gy, t, w, T, H, eps, flags, gt, gx, gw, wsp, n, None)

    bad, un = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    assert call(T=0, gy=None, t=None, w=None, gx=None, gw=None, wsp=None, n=0) == moe.MOE_OK
    assert call(T=-1) == bad and call(T=2 ** 31) == un and call(H=12) == un and call(H=65544) == un
    assert call(eps=-1.0) == bad and call(eps=math.nan) == bad and call(flags=8) == bad
    assert call(gy=None) == bad and call(t=None) == bad and call(w=None) == bad and call(gx=None, gw=None) == bad
    for name in ("gy", "t", "w", "gt", "gx"):
        assert call(**{name: FAKE + 8}) == bad
    assert call(gw=MIS) == bad
    assert call(wsp=None) == moe.MOE_ERR_WORKSPACE and call(n=ws - 1) == moe.MOE_ERR_WORKSPACE
    assert call(wsp=FAKE + 8) == moe.MOE_ERR_WORKSPACE
    n = ctypes.c_size_t(7)
    size = moe.lib.moe_rms_norm_backward_workspace_size
    assert size(4, 64, None) == bad and size(-1, 64, ctypes.byref(n)) == bad and size(4, 12, ctypes.byref(n)) == un
    assert n.value == 7 and moe.moe_rms_norm_backward_workspace_size(0, 64) == 0


def test_weights_validation(moe):
    def call(W=FAKE, n=2, O=64, H=64, flags=0, c=FAKE, s=FAKE, ct=FAKE, st=FAKE):
        return moe.lib.moe_fp8_quantize_weights(W, n, O, H, flags, c, s, ct, st, None)

    bad, un = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    assert call(n=0, W=None, c=None, s=None, ct=None, st=None) == moe.MOE_OK
    assert call(n=-1) == bad and call(n=1025) == un and call(flags=2) == bad
    for name in ("O", "H"):
        assert call(**{name: 0}) == un and call(**{name: -32}) == un and call(**{name: 48}) == un
    assert call(O=131104) == un and call(H=65568) == un
    assert call(W=None) == bad and call(c=None) == bad and call(s=None) == bad
    assert call(ct=None) == bad and call(st=None) == bad    # both or neither
    for name in ("W", "c", "ct"):
        assert call(**{name: FAKE + 8}) == bad
    assert call(s=MIS) == bad and call(st=MIS) == bad


@pytest.mark.parametrize("which", ["product", "dgrad"])
def test_product_validation(moe, which):
    def call(a=FAKE, off=FAKE, El=4, rows=100, H=64, O=128, W=FAKE, s=FAKE, pre=FAKE, act=2, flags=1, y=FAKE, y8=FAKE,
             bias=None, res=None):
        if which == "product":
            return moe.lib.moe_expert_product_fp8(a, off, El, rows, H, O, W, s, bias, res, act, flags, pre, y, y8, None)
        return moe.lib.moe_expert_product_fp8_dgrad(a, off, El, rows, O, H, W, s, pre, act, flags, y, y8, None)

    bad, un = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    assert call(rows=0, a=None, off=None, W=None, s=None, y=None, y8=None) == moe.MOE_OK
    assert call(El=0) == bad and call(El=1025) == un and call(rows=-1) == bad and call(rows=2 ** 31) == un
    for name in ("H", "O"):
        assert call(**{name: 0}) == un and call(**{name: 40}) == un and call(**{name: 65568}) == un
    assert call(act=-1) == bad and call(act=5) == bad and call(flags=2) == bad
    for name in ("a", "W", "y", "y8"):
        assert call(**{name: FAKE + 8}) == bad
    assert call(a=None) == bad and call(W=None) == bad and call(s=None) == bad and call(y=None, y8=None) == bad
    assert call(off=None) == bad and call(off=MIS) == bad and call(s=MIS) == bad and call(pre=FAKE + 8) == bad
    if which == "product":
        assert call(bias=FAKE + 8) == bad and call(res=FAKE + 8) == bad
    else:
        assert call(pre=None) == bad and call(pre=None, flags=0) == bad and call(pre=None, act=0) == bad
        assert call(H=32800, pre=FAKE, y8=FAKE) == un       # 2 H values in an FP8 row


@pytest.fixture
def stand_ins(moe, monkeypatch):
    """The binding on stand-ins for GPU tensors; the library must not be reached."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(moe, "_stream", lambda s: 0)

    def never(*a):
        raise AssertionError("the library was called")

    names = ("moe_rms_norm", "moe_rms_norm_backward", "moe_fp8_quantize_weights", "moe_expert_product_fp8",
             "moe_expert_product_fp8_dgrad")
    real = moe.lib
    monkeypatch.setattr(moe, "lib", types.SimpleNamespace(
        moe_fp8_row_bytes=real.moe_fp8_row_bytes, moe_status_string=real.moe_status_string,
        moe_rms_norm_backward_workspace_size=real.moe_rms_norm_backward_workspace_size, **{n: never for n in names}))
    return moe


def calls(moe, **kw):
    """Each call on tensors of GPU 0, with outputs given; keyword arguments replace some."""
    x, w, r8, off = Tensor((4, 32), BF), Tensor((32,), BF), Tensor((4, 160), U8), Tensor((3,), I)
    W, s, z = Tensor((2, 32, 32), U8), Tensor((2, 1, 1), F), Tensor((4, 32), BF)

    def norm(**o):
        return moe.moe_rms_norm(**dict(dict(x=x, weight=w, residual=x, total=x, y=x, y8=r8), **o))

    def back(**o):
        return moe.moe_rms_norm_backward(**dict(dict(grad_y=x, total=x, weight=w, grad_total=x, grad_x=x,
                                                     grad_weight=Tensor((32,), F), workspace=Tensor((4096,), U8)), **o))

    def weights(**o):
        return moe.moe_fp8_quantize_weights(**dict(dict(W=Tensor((2, 32, 32), F), codes=W, scale=s, codes_t=W, scale_t=s), **o))

    def product(**o):
        return moe.moe_expert_product_fp8(**dict(dict(x=r8, expert_offsets=off, W=W, W_scale=s, residual=z, pre=z, y=z,
                                                      y8=r8), **o))

    def dgrad(**o):
        return moe.moe_expert_product_fp8_dgrad(**dict(dict(grad_y=r8, expert_offsets=off, W_t=W, W_t_scale=s, pre=z,
                                                            act="silu", grad_x=z, grad_x8=r8), **o))

    return dict(norm=norm, back=back, weights=weights, product=product, dgrad=dgrad)


def test_stand_ins_reach_the_library(stand_ins):
    for call in calls(stand_ins).values():
        with pytest.raises(AssertionError, match="the library was called"):
            call()


@pytest.mark.parametrize("name", ["norm", "back", "weights", "product", "dgrad"])
def test_stream_of_another_device(stand_ins, monkeypatch, name):
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0x20000

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: pytest.fail("the other device was made current"))
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        calls(stand_ins)[name](stream=Stream())


BAD = {
    "norm": dict(weight=((32,), BF), residual=((4, 32), BF), total=((4, 32), BF), y=((4, 32), BF), y8=((4, 160), U8)),
    "back": dict(grad_y=((4, 32), BF), weight=((32,), BF), grad_total=((4, 32), BF), grad_x=((4, 32), BF),
                 grad_weight=((32,), F), workspace=((4096,), U8)),
    "weights": dict(codes=((2, 32, 32), U8), scale=((2, 1, 1), F), codes_t=((2, 32, 32), U8), scale_t=((2, 1, 1), F)),
    "product": dict(expert_offsets=((3,), I), W_scale=((2, 1, 1), F), residual=((4, 32), BF), pre=((4, 32), BF),
                    y=((4, 32), BF), y8=((4, 160), U8)),
    "dgrad": dict(expert_offsets=((3,), I), W_t_scale=((2, 1, 1), F), pre=((4, 32), BF), grad_x=((4, 32), BF),
                  grad_x8=((4, 160), U8)),
}


@pytest.mark.parametrize("name,arg", [(n, a) for n, d in BAD.items() for a in d])
def test_argument_of_another_device_shape_or_type(stand_ins, name, arg):
    shape, dt = BAD[name][arg]
    call = calls(stand_ins)[name]
    with pytest.raises(ValueError, match="cuda:1"):
        call(**{arg: Tensor(shape, dt, 1)})
    with pytest.raises(TypeError):
        call(**{arg: Tensor(shape, torch.float64)})
    if arg != "workspace":
        with pytest.raises(ValueError):
            call(**{arg: Tensor((*shape[:-1], shape[-1] + 1), dt)})


def test_binding_refusals(stand_ins):
    moe, c = stand_ins, calls(stand_ins)
    with pytest.raises(ValueError):
        c["norm"](x=torch.zeros(4, 32))                       # not on a GPU
    with pytest.raises(ValueError):
        c["norm"](residual=None)                              # total without residual
    with pytest.raises(TypeError):
        c["norm"](residual=Tensor((4, 32), F))                # another type than x
    with pytest.raises(moe.MoeError):
        moe.moe_rms_norm(Tensor((4, 40), BF), Tensor((40,), BF), y=Tensor((4, 40), BF), y8=Tensor((4, 200), U8))
    with pytest.raises(ValueError):
        c["back"](grad_weight=None, accumulate=True)
    for name, arg in (("product", "x"), ("dgrad", "grad_y")):
        with pytest.raises(ValueError):
            c[name](**{arg: Tensor((4, 32), U8)})             # codes without their scales
    with pytest.raises(ValueError):
        c["product"](W=Tensor((2, 33, 32), U8), gated=True)
    with pytest.raises(ValueError):
        c["product"](act="tanh")
