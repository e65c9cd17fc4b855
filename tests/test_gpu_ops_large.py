"""The combine's gradient and the experts' products where element offsets pass 2^31 and byte offsets 2^32.

Inputs are mostly one repeated value, so that a row read from a wrapped offset
differs: the rows checked, at the buffers' end, hold values of their own. The
bars are those of the small tests.
"""

import numpy as np
import pytest
import torch

import ops_reference as ref
from test_gpu_product import assert_rows, bf16, canary

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import combine_route_topk_amd
    return combine_route_topk_amd


def test_products(moe):
    """2^31 elements of x in two experts; the second has the last 300 rows, then one of 40 within few."""
    H, O = 4096, 40
    rows = 2 ** 31 // H + 700
    rng = np.random.default_rng(0)
    x = torch.full((rows, H), 0.5, dtype=torch.bfloat16, device=DEV)
    tail = bf16(rng, 300, H)
    x[-300:] = tail.to(DEV)
    W = bf16(rng, 2, O, H, scale=H ** -0.5)
    for mine in (300, 40):
        off = torch.tensor([rows - mine, rows - mine, rows], dtype=torch.int32, device=DEV)
        print("[case]", rows, H, O, mine, flush=True)
        y = canary(rows, O)
        moe.moe_expert_product(x, off, W.to(DEV), act="silu", y=y)
        wy, _, _, ey = ref.product(tail[-mine:].double().numpy(), [0, 0, mine], W.double().numpy(), None, None, "silu")
        assert_rows(y[-mine:], wy, ey, mine, "y")
        assert (y[:-mine].view(torch.int16) == 0x5A5A).all()
        # x in the gradient's place: W [2, H, O']
        W2 = bf16(rng, 2, H, O, scale=H ** -0.5)
        g = canary(rows, O)
        moe.moe_expert_product_dgrad(x, off, W2.to(DEV), grad_x=g)
        wg, eg = ref.dgrad(tail[-mine:].double().numpy(), [0, 0, mine], W2.double().numpy())
        assert_rows(g[-mine:], wg, eg, mine, "grad_x")
        gy = torch.full((rows, O), 0.25, dtype=torch.bfloat16, device=DEV)
        gt = bf16(rng, mine, O)
        gy[-mine:] = gt.to(DEV)
        gW, gb = torch.empty(2, O, H, device=DEV), torch.empty(2, O, device=DEV)
        moe.moe_expert_product_wgrad(gy, x, off, gW, gb)
        vW, vb, eW, eb = ref.wgrad(gt.double().numpy(), tail[-mine:].double().numpy(), [0, 0, mine], 2)
        assert (np.abs(gW.cpu().double().numpy() - vW) <= eW + 2.0 ** -126).all()
        assert (np.abs(gb.cpu().double().numpy() - vb) <= eb + 2.0 ** -126).all()


def test_many_rows(moe):
    """A first expert with more than 2^31 elements of its own: its sums over all rows, and its last rows."""
    H, O = 2048, 16
    rows = 2 ** 31 // H + 321
    rng = np.random.default_rng(1)
    x = torch.full((rows, H), 0.5, dtype=torch.bfloat16, device=DEV)
    gy = torch.zeros(rows, O, dtype=torch.bfloat16, device=DEV)
    tail, gt = bf16(rng, 200, H), bf16(rng, 200, O)
    x[-200:], gy[-200:] = tail.to(DEV), gt.to(DEV)
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    W = bf16(rng, 1, O, H, scale=H ** -0.5)
    print("[case]", rows, H, O, flush=True)
    y = moe.moe_expert_product(x, off, W.to(DEV))
    wy, _, _, ey = ref.product(tail.double().numpy(), [0, 200], W.double().numpy())
    assert_rows(y[-200:], wy, ey, 200, "y")
    gW = moe.moe_expert_product_wgrad(gy, x, off, torch.empty(1, O, H, device=DEV))
    # zeros ahead of the last 200 rows add nothing to the sum, nor to its error
    vW, _, eW, _ = ref.wgrad(gt.double().numpy(), tail.double().numpy(), [0, 200], 1)
    assert (np.abs(gW.cpu().double().numpy() - vW) <= eW + 2.0 ** -126).all()


def test_combine(moe):
    """2^31 elements of y, the replicas' rows at its end."""
    H, T, k = 8192, 40, 3
    rows = 2 ** 31 // H + 200
    rng = np.random.default_rng(2)
    y = torch.full((rows, H), 0.5, dtype=torch.bfloat16, device=DEV)
    tail = bf16(rng, 150, H)
    y[-150:] = tail.to(DEV)
    at = rng.permutation(150)[:T * k].reshape(T, k)
    pos = torch.from_numpy((rows - 150 + at).astype(np.int32)).to(DEV)
    g, w = bf16(rng, T, H), torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32))
    gy = canary(rows, H)
    print("[case]", rows, H, T, k, flush=True)
    gy, gw = moe.moe_combine_backward(g.to(DEV), y, pos, w.to(DEV), gy)
    want_y, want_w = ref.combine_backward(g.double().numpy(), tail.double().numpy(), at, w.double().numpy())
    left = np.isnan(want_y).any(1)
    got = gy[-150:].cpu()
    assert (gy[:-150].view(torch.int16) == 0x5A5A).all() and (got[left].view(torch.int16) == 0x5A5A).all()
    d = np.abs(got.double().numpy() - want_y)[~left]
    assert (d <= np.abs(want_y[~left]) * (2.0 ** -8 + 2.0 ** -20) + 2.0 ** -134).all()
    mag = (np.abs(tail.double().numpy()[at]) * np.abs(g.double().numpy())[:, None, :]).sum(2)
    assert (np.abs(gw.cpu().double().numpy() - want_w) <= 2 * H * 2.0 ** -24 * mag).all()
