"""The norm on more rows than one launch has blocks of 1024 threads: 2^22 such
blocks are 2^32 threads, one more than a launch takes."""

import pytest
import torch

from test_gpu_norm import BF, DEV, EPS, moe, say  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [((1 << 20) + 5, 4128), ((1 << 22) + 5, 4128)])
def test_wide_rows_past_one_grid(moe, T, H):
    say("norm, wide rows past one grid", T, H)
    g = torch.Generator(device=DEV).manual_seed(0)
    x = torch.empty(T, H, dtype=BF, device=DEV)
    for a in range(0, T, 1 << 19):
        x[a:a + (1 << 19)] = torch.randn(min(1 << 19, T - a), 1, generator=g, device=DEV)
    x[:, 5] += 1
    w = torch.randn(H, generator=g, device=DEV).to(BF)
    _, y, y8 = moe.moe_rms_norm(x, w, eps=EPS, fp8=True, need_y=False)
    assert y is None
    for a in (0, (1 << 20) - 65, T - 70):
        rows = slice(a, a + 70)
        alone = moe.moe_rms_norm(x[rows].contiguous(), w, eps=EPS, fp8=True, need_y=False)[2]
        torch.cuda.synchronize()
        assert torch.equal(y8[rows], alone)
