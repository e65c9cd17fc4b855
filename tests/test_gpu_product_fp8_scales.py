"""Scales of the 8-bit weights: NaN and infinite ones reach exactly the columns
of their block, in exactly their expert's rows, and a gated product's gate and
up columns each meet their own. Sizes for each of the kernels: few rows, tiles
of 64 rows, of 128, and of 256 with a last round of slices.
"""

import numpy as np
import pytest
import torch

import fp8_reference as f8
from test_gpu_product import assert_rows, canary, dn, offsets
from test_gpu_product_fp8 import empty8, gpu, moe, rows8, say, weights8  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu
H = 384  # three blocks along K


def run(moe, x, off, W, s, n, O, **kw):
    y, y8 = canary(n, O), empty8(n, O)
    z = canary(n, W.shape[1]) if kw.get("gated") else None
    moe.moe_expert_product_fp8(gpu(x), gpu(off), gpu(W), gpu(s), y=y, y8=y8, pre=z, **kw)
    torch.cuda.synchronize()
    return y, y8, z


@pytest.mark.parametrize("counts,O", [([3, 4], 320), ([300, 20], 320), ([4000, 300], 1184), ([16000, 300], 1184)])
@pytest.mark.parametrize("first,second", [(np.nan, np.inf), (-np.inf, np.nan)])
def test_bad_scale_reaches_its_block_only(moe, counts, O, first, second):
    """Different blocks in the two experts: a result is not finite exactly where its own block's scale is not."""
    rng = np.random.default_rng(11)
    off = offsets(counts)
    n = int(off[-1])
    say("bad scales", counts, O, first, second)
    x, _ = rows8(rng, n, H)
    W, s, _ = weights8(rng, 2, O, H)
    s[0, 1, 1], s[1, 2, 2] = first, second
    y, y8, _ = run(moe, x, off, W, s, n, O)
    bad = np.zeros((n, O), bool)
    bad[:off[1], 128:256] = True
    bad[off[1]:, 256:384] = True
    got = dn(y.cpu())
    assert (np.isfinite(got) == ~bad).all()
    assert (np.isnan(f8.decode_rows(y8.cpu().numpy(), O)) == bad).all()
    # what is finite is what it is without the bad ones
    t = np.where(np.isfinite(s), s, np.float32(1))
    clean = dn(run(moe, x, off, W, t, n, O)[0].cpu())
    assert (got[~bad] == clean[~bad]).all()


GATED = [([3, 4], 288), ([300, 20], 288), ([4000, 300], 672), ([16000, 300], 672)]


@pytest.mark.parametrize("counts,O", GATED)
@pytest.mark.parametrize("kind", ["none", "silu"])
def test_bad_scale_of_a_gated_product(moe, counts, O, kind):
    """One block in which the gate columns end and the up columns begin, and one of up columns alone."""
    rng = np.random.default_rng(12)
    off = offsets(counts)
    n, both, last = int(off[-1]), O // 128, (2 * O - 1) // 128
    say("bad scales, gated", counts, O, kind)
    x, _ = rows8(rng, n, H)
    W, s, _ = weights8(rng, 2, 2 * O, H)
    s[0, both, 1], s[1, last, 0] = np.inf, np.nan
    y, y8, z = run(moe, x, off, W, s, n, O, act=kind, gated=True)
    pre = np.zeros((n, 2 * O), bool)
    pre[:off[1], both * 128:(both + 1) * 128] = True
    pre[off[1]:, last * 128:] = True
    bad = pre[:, :O] | pre[:, O:]
    assert (np.isfinite(dn(z.cpu())) == ~pre).all()
    assert (np.isfinite(dn(y.cpu())) == ~bad).all()
    assert (np.isnan(f8.decode_rows(y8.cpu().numpy(), O)) == bad).all()


@pytest.mark.parametrize("counts,O", GATED)
def test_gated_scales_of_every_size(moe, counts, O):
    """Negative, huge, tiny, subnormal and zero scales that differ between a column's gate and its up block. Bars as in
    test_gpu_product_fp8, and for a scale below 2^-126, which may count as 2^-127, that times the terms' sizes: e of
    gate and f of up put |up| e + |gate| f + e f on their product."""
    rng = np.random.default_rng(13)
    off = offsets(counts)
    n, both = int(off[-1]), O // 128
    say("gated scales", counts, O)
    x, xv = rows8(rng, n, H)
    W, s, _ = weights8(rng, 2, 2 * O, H)
    s[0, 0] = [-0.75, 2.0 ** -140, 1.5 * 2.0 ** 60]
    s[0, both + 1] = [1.25 * 2.0 ** -60, 0.0, 2.0 ** -126]
    s[1, 0] = [2.0 ** -70, -1.75 * 2.0 ** -70, 2.0 ** -140]
    s[1, both] = [-1.5 * 2.0 ** 40, 0.5, 2.0 ** -130]
    y, y8, z = run(moe, x, off, W, s, n, O, gated=True)
    wy, wz, ez, ey = f8.product(xv, f8.rows_largest(x, H), off, f8.decode_weights(W, s),
                                f8.weights_largest(W, np.abs(s)), gated=True)
    codes = np.abs(f8.e4m3(W)).max(2)
    for l in range(2):
        b, e = off[l], off[l + 1]
        lost = 2.0 ** -126 * np.abs(xv[b:e]).sum(1)[:, None] * codes[l]
        ez[b:e] += lost
        size = np.abs(wz[b:e]) + ez[b:e]
        ey[b:e] += size[:, O:] * lost[:, :O] + size[:, :O] * lost[:, O:]
    assert_rows(z, wz, ez, n, "pre")
    assert_rows(y, wy, ey, n, "y")
    f8.assert_rows8(y8, wy, ey, n, "y8")
