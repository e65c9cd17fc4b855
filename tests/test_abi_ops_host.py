"""Argument checks of the scored router, the combine's gradient and the
experts' products, on the host: every call here fails a check, or returns,
before anything touches a GPU, so the pointers are never dereferenced."""

import ctypes
import math

import pytest

FAKE, MIS = 0x10000, 0x10002


@pytest.fixture(scope="module")
def moe():
    import combine_route_topk_amd
    return combine_route_topk_amd


def test_route_scored_validation(moe):
    def call(lg=FAKE, b=None, T=4, E=64, k=2, G=1, M=1, scale=1.0, flags=1, idx=FAKE, w=FAKE):
        return moe.lib.moe_route_scored(lg, b, T, E, k, G, M, scale, flags, idx, w, None)

    bad, un = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    assert call(T=0, lg=None, idx=None, w=None) == moe.MOE_OK
    assert call(T=-1) == bad
    assert call(k=0) == un and call(k=33) == un and call(E=1025) == un and call(E=4, k=5) == un
    assert call(T=2 ** 30, k=2) == un
    assert call(G=0) == bad and call(G=3) == bad and call(G=4, M=5) == bad and call(G=4, M=0) == bad
    assert call(G=32, M=1, k=3) == bad                  # more experts than the groups hold
    assert call(E=1024, G=128, M=64) == un
    assert call(flags=16) == bad and call(flags=1 << 31) == bad
    assert call(scale=math.inf) == bad and call(scale=-math.inf) == bad and call(scale=math.nan) == bad
    assert call(lg=None) == bad and call(idx=None) == bad and call(w=None) == bad
    assert call(lg=MIS) == bad and call(b=MIS) == bad and call(idx=MIS) == bad and call(w=MIS) == bad
    assert call(lg=FAKE + 1, flags=8) == bad


def test_route_scored_backward_validation(moe):
    def call(lg=FAKE, idx=FAKE, g=FAKE, T=4, E=64, k=2, scale=1.0, flags=1, out=FAKE):
        return moe.lib.moe_route_scored_backward(lg, idx, g, T, E, k, scale, flags, out, None)

    bad = moe.MOE_ERR_INVALID_ARG
    assert call(T=0, lg=None, idx=None, g=None, out=None) == moe.MOE_OK
    assert call(T=-1) == bad and call(flags=4) == bad and call(flags=16) == bad and call(scale=math.nan) == bad
    assert call(k=65, E=64) == moe.MOE_ERR_UNSUPPORTED
    for name in ("lg", "idx", "g", "out"):
        assert call(**{name: None}) == bad and call(**{name: MIS}) == bad
    assert call(out=FAKE + 1, flags=8) == bad


def test_combine_backward_validation(moe):
    def call(go=FAKE, y=FAKE, rows=8, pos=FAKE, w=FAKE, T=4, H=64, k=2, flags=0, gy=FAKE, gw=FAKE):
        return moe.lib.moe_combine_backward(go, y, rows, pos, w, T, H, k, flags, gy, gw, None)

    bad, un = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    assert call(T=0, go=None, y=None, pos=None, w=None, gy=None, gw=None) == moe.MOE_OK
    assert call(T=-1) == bad and call(rows=-1) == bad and call(flags=2) == bad
    assert call(H=12) == un and call(H=65544) == un and call(k=0) == un and call(rows=2 ** 31) == un
    assert call(go=None) == bad and call(pos=None) == bad
    assert call(gy=None, gw=None) == bad
    assert call(y=None) == bad and call(w=None) == bad
    assert call(go=FAKE + 8) == bad and call(y=FAKE + 8) == bad and call(gy=FAKE + 8) == bad
    assert call(pos=MIS) == bad and call(w=MIS) == bad and call(gw=MIS) == bad
    assert call(rows=0, gw=None, y=None, w=None) == moe.MOE_OK  # no row to write, no weight asked for
    assert call(rows=0, gw=None, gy=None) == bad


@pytest.mark.parametrize("which", ["product", "dgrad"])
def test_product_validation(moe, which):
    def call(a=FAKE, off=FAKE, El=4, rows=100, H=64, O=128, W=FAKE, pre=FAKE, act=2, flags=1, out=FAKE, bias=None,
             res=None):
        if which == "product":
            return moe.lib.moe_expert_product(a, off, El, rows, H, O, W, bias, res, act, flags, pre, out, None)
        return moe.lib.moe_expert_product_dgrad(a, off, El, rows, O, H, W, pre, act, flags, out, None)

    bad, un = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    assert call(rows=0, a=None, off=None, W=None, out=None) == moe.MOE_OK
    assert call(El=0) == bad and call(El=1025) == un
    assert call(rows=-1) == bad and call(rows=2 ** 31) == un
    for name in ("H", "O"):
        assert call(**{name: 0}) == un and call(**{name: 12}) == un and call(**{name: 65544}) == un
    assert call(act=-1) == bad and call(act=5) == bad and call(flags=2) == bad
    for name in ("a", "W", "out"):
        assert call(**{name: None}) == bad and call(**{name: FAKE + 8}) == bad
    assert call(off=None) == bad and call(off=MIS) == bad and call(pre=FAKE + 8) == bad
    if which == "product":
        assert call(bias=FAKE + 8) == bad and call(res=FAKE + 8) == bad
    else:
        assert call(pre=None) == bad and call(pre=None, flags=0) == bad and call(pre=None, act=0) == bad


def test_wgrad_validation(moe):
    ws = moe.moe_expert_product_wgrad_workspace_size(4, 100, 128, 64)

    def call(gy=FAKE, x=FAKE, off=FAKE, El=4, rows=100, O=128, H=64, flags=1, gW=FAKE, gb=None, w=FAKE, wb=ws):
        return moe.lib.moe_expert_product_wgrad(gy, x, off, El, rows, O, H, flags, gW, gb, w, wb, None)

    bad, un = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    assert call(El=0) == bad and call(El=1025) == un and call(rows=-1) == bad and call(rows=2 ** 31) == un
    assert call(H=12) == un and call(O=0) == un
    assert call(flags=2) == bad and call(flags=4) == bad        # accumulation into bf16; unknown
    assert call(gy=None) == bad and call(x=None) == bad and call(off=None) == bad and call(gW=None) == bad
    assert call(gy=FAKE + 8) == bad and call(x=FAKE + 8) == bad and call(gW=FAKE + 8) == bad
    assert call(off=MIS) == bad and call(gb=MIS) == bad
    n = ctypes.c_size_t(7)
    size = moe.lib.moe_expert_product_wgrad_workspace_size
    assert size(4, 100, 128, 64, None) == bad and size(0, 100, 128, 64, ctypes.byref(n)) == bad
    assert size(4, 100, 12, 64, ctypes.byref(n)) == un and n.value == 7


def test_binding_refusals(moe):
    """Wrong shapes and host tensors end in a Python error, before the library is called."""
    import torch
    bf, z = torch.bfloat16, torch.zeros
    with pytest.raises(ValueError):
        moe.moe_route_scored(z(4, 8), None, 2)
    with pytest.raises(ValueError):
        moe.moe_route_scored(z(4, 8), None, 2, scores="tanh")
    with pytest.raises(ValueError):
        moe.moe_route_scored_backward(z(4, 8), z(4, 2, dtype=torch.int32), z(4, 2))
    with pytest.raises(ValueError):
        moe.moe_combine_backward(z(4, 8), None, z(4, 2, dtype=torch.int32), z(4, 2))
    off = z(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        moe.moe_expert_product(z(4, 8, dtype=bf), off, z(2, 8, 8, dtype=bf))
    with pytest.raises(ValueError):
        moe.moe_expert_product_dgrad(z(4, 8, dtype=bf), off, z(2, 8, 8, dtype=bf))
    with pytest.raises(ValueError):
        moe.moe_expert_product_wgrad(z(4, 8, dtype=bf), z(4, 8, dtype=bf), off)
