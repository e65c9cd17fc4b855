"""The workspace of the norm's gradient: partial sums of the weight's gradient
only where that is wanted, and the statistics of rows wider than 16384. Host
checks fail, or reach a stand-in, before anything touches a GPU."""

import pytest
import torch

from test_abi_layer8_host import FAKE, calls, moe, stand_ins  # noqa: F401  (fixtures)
from test_binding_devices_host import Tensor

BF, F = torch.bfloat16, torch.float32
DEV = "cuda:0"


@pytest.mark.parametrize("T,H", [(4, 16392), (7, 65536), (1000, 20000)])
def test_wide_rows_need_their_statistics(moe, T, H):
    def call(wsp, n, gw=None):
        return moe.lib.moe_rms_norm_backward(FAKE, FAKE, FAKE, T, H, 1e-6, 0, None, FAKE, gw, wsp, n, None)

    bad = moe.MOE_ERR_WORKSPACE
    assert call(None, 0) == bad and call(FAKE, 8 * T - 1) == bad and call(FAKE + 8, 8 * T) == bad
    assert call(FAKE, moe.moe_rms_norm_backward_workspace_size(T, H) - 1, FAKE) == bad


@pytest.mark.parametrize("T,H,need", [(5, 2048, 0), (5, 16384, 0), (0, 64, 0), (5, 16392, 40), (1000, 65536, 8000)])
def test_binding_makes_no_workspace_that_nothing_reads(stand_ins, monkeypatch, T, H, need):
    made, given = [], []
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: made.append(n) or Tensor((n,), dtype))
    stand_ins.lib.moe_rms_norm_backward = lambda *a: given.append(a) or 0
    x = Tensor((T, H), BF)
    grad_x, grad_weight = stand_ins.moe_rms_norm_backward(x, x, Tensor((H,), BF), grad_x=x, need_weight=False)
    assert grad_x is x and grad_weight is None
    assert made == ([need] if need else [])
    workspace, size = given[0][-3:-1]
    assert size == need and (workspace is not None) == (need > 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("T,H", [(1, 64), (9, 2048), (1030, 7168), (40, 16384), (7, 16392), (300, 40000)])
def test_input_gradient_alone(moe, T, H, dt):
    """Without the weight's gradient: the same bits, in a workspace of the statistics alone or in none."""
    print("[case] input gradient alone", T, H, dt, flush=True)
    g = torch.Generator(device=DEV).manual_seed(T + H)

    def randn(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device=DEV).to(dtype)

    gy, t, w, gt = randn(T, H, dtype=BF), randn(T, H), randn(H), randn(T, H)
    want, _ = moe.moe_rms_norm_backward(gy, t, w, 1e-5, gt)
    got, none = moe.moe_rms_norm_backward(gy, t, w, 1e-5, gt, need_weight=False)
    need = 8 * T if H > 16384 else 0
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(want)
    flags = (moe.MOE_NORM_FP32 | moe.MOE_NORM_WEIGHT_FP32) if dt == F else 0
    rc = moe.lib.moe_rms_norm_backward(gy.data_ptr(), t.data_ptr(), w.data_ptr(), T, H, 1e-5, flags, gt.data_ptr(),
                                       out.data_ptr(), None, ws.data_ptr() if need else None, need,
                                       torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == moe.MOE_OK and none is None
    assert torch.equal(got, want) and torch.equal(out, want)
    assert (ws[need:] == 0x5A).all()
