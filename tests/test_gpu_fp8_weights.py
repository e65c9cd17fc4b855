"""Weights in 8 bits with a scale for each block of 128 x 128 on the GPU,
against the definition's float32 operations bit for bit."""

import numpy as np
import pytest
import torch

import fp8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import combine_route_topk_amd
    return combine_route_topk_amd


def check(moe, W, what):
    print("[case]", what, tuple(W.shape), W.dtype, flush=True)
    n, O, H = W.shape
    u8 = dict(dtype=torch.uint8, device=DEV)
    codes, codes_t = torch.full((n, O, H), 0x5A, **u8), torch.full((n, H, O), 0x5A, **u8)
    c, s, ct, st = moe.moe_fp8_quantize_weights(W.to(DEV), codes=codes, codes_t=codes_t)
    c2, s2, none, none2 = moe.moe_fp8_quantize_weights(W.to(DEV))
    torch.cuda.synchronize()
    assert none is None and none2 is None and c2.dtype == torch.float8_e4m3fn
    assert torch.equal(c2.view(torch.uint8), c) and torch.equal(s2, s)
    assert torch.equal(ct, c.transpose(1, 2)) and torch.equal(st, s.transpose(1, 2))
    for l in range(n):
        wc, ws = ref.quantize(W[l].float().numpy())
        assert (s[l].cpu().numpy() == ws).all(), "scales"
        got, v = c[l].cpu().numpy(), ref.e4m3(wc)
        nan = np.isnan(v)  # either sign of NaN
        assert (np.isnan(ref.e4m3(got)) == nan).all() and (got[~nan] == wc[~nan]).all(), "codes"


@pytest.mark.parametrize("n,O,H", [(1, 32, 32), (2, 128, 128), (3, 160, 96), (1, 256, 1056), (2, 288, 2048), (5, 96, 7168),
                                   (2, 4096, 160), (1024, 32, 32), (1, 32, 65536), (1, 131072, 32)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_sizes(moe, n, O, H, dt):
    rng = np.random.default_rng(O + H)
    W = rng.standard_normal((n, O, H)) * np.exp2(rng.integers(-20, 20, (n, (O + 31) // 32, 1, 1)).repeat(32, 2).reshape(n, -1, 1)[:, :O])
    check(moe, torch.from_numpy(W.astype(np.float32)).to(dt), "sizes")


def test_special_values(moe):
    W = torch.randn(1, 384, 256, generator=torch.Generator().manual_seed(0))
    W[0, :128, :128] = 0                # a block of zeros
    W[0, :128, 128:] *= 2.0 ** -126     # subnormal scales, held at the least normal
    W[0, 128:256, :128] = 2.0 ** -149
    W[0, 130, 140] = float("nan")       # the rest of its block as without it
    W[0, 256:, :128] *= 2.0 ** 125      # near the largest
    check(moe, W, "special values")


def test_infinite_weight(moe):
    """An infinity makes its block's scale infinite, and its own code NaN."""
    W = torch.ones(1, 128, 256)
    W[0, 3, 7] = float("inf")
    c, s, _, _ = moe.moe_fp8_quantize_weights(W.to(DEV))
    torch.cuda.synchronize()
    assert torch.isinf(s[0, 0, 0]) and s[0, 0, 1] == np.float32(1) / np.float32(448)
    f = c.float().cpu()
    assert torch.isnan(f[0, 3, 7]) and (f[0, :, 128:] == 448).all()


def test_past_32_bits(moe):
    """Elements past 2^31: the last matrices against the same ones alone."""
    n, O, H = 80, 4096, 7168
    print("[case] large", n, O, H, flush=True)
    g = torch.Generator(device=DEV).manual_seed(0)
    W = torch.empty(n, O, H, dtype=torch.bfloat16, device=DEV)
    for l in range(n):
        W[l] = torch.randn(O, H, generator=g, device=DEV)
    big = moe.moe_fp8_quantize_weights(W, transpose=True)
    one = moe.moe_fp8_quantize_weights(W[n - 2:].contiguous(), transpose=True)
    torch.cuda.synchronize()
    for a, b in zip(big, one):
        assert torch.equal(a[n - 2:].view(torch.uint8), b.view(torch.uint8))
