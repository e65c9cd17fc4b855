"""The experts' products on FP8 rows and their input gradient on the GPU
against float64.

The rows and weights decode to exact float64 values. Bars: the matrix unit's
error and that of a float32 computation, which tests/fp8_reference.py derives,
passed through the activation, plus half a step of the output's type (bf16
2^-8; FP8 rows as fp8_reference.assert_rows8 says). Rows of no expert stay as
they were. Every test prints its case before touching the GPU.
"""

import numpy as np
import pytest
import torch

import fp8_reference as f8
import ops_reference as ref
from test_gpu_product import COUNTS, assert_rows, bf16, canary, dn, offsets, up

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import combine_route_topk_amd
    return combine_route_topk_amd


def say(*a):
    print("[case]", *a, flush=True)


def rows8(rng, n, K, spread=4):
    """(bytes, values) of FP8 rows whose blocks of 32 differ in size."""
    v = rng.standard_normal((n, K // 32, 32)) * np.exp2(rng.integers(-spread, spread + 1, (n, K // 32, 1)))
    r = f8.encode_rows(v.reshape(n, K).astype(np.float32))
    return r, f8.decode_rows(r, K)


def weights8(rng, El, O, K):
    """(codes, scales, values) of weights whose blocks differ in size."""
    c = f8.to_e4m3(np.clip(rng.standard_normal((El, O, K)) * 105, -448, 448))
    s = np.exp(rng.standard_normal((El, (O + 127) // 128, (K + 127) // 128))).astype(np.float32) * np.float32(K ** -0.5 / 105)
    return c, s, f8.decode_weights(c, s)


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def empty8(n, width):
    return torch.full((n, f8.row_bytes(width)), 0x5A, dtype=torch.uint8, device=DEV)


def run_product(moe, counts, H, O, kind="none", gated=False, bias=False, residual=False, pre=False, out="both", pad=0,
                in_place=False):
    rng = np.random.default_rng(H + O)
    off = offsets(counts)
    used, El = int(off[-1]), len(counts)
    rows, wide = used + pad, 2 * O if gated else O
    say(counts, H, O, kind, gated, bias, residual, pre, out, pad)
    x, xv = rows8(rng, rows, H)
    W, s, Wv = weights8(rng, El, wide, H)
    b = bf16(rng, El, wide) if bias else None
    r = bf16(rng, rows, O) if residual else None
    y, y8 = canary(rows, O) if out != "fp8" else None, empty8(rows, O) if out != "bf16" else None
    z = canary(rows, wide) if pre else None
    if in_place:
        y[:used] = r[:used].to(DEV)
    a, c = moe.moe_expert_product_fp8(gpu(x), gpu(off), gpu(W).view(torch.float8_e4m3fn), gpu(s), bias=up(b),
                                      residual=y if in_place else up(r), act=kind, gated=gated, need_y=y is not None,
                                      y=y, y8=y8, pre=z)
    torch.cuda.synchronize()
    assert (a is None) == (y is None) and (c is None) == (y8 is None)
    wy, wz, ez, ey = f8.product(xv, f8.rows_largest(x, H), off, Wv, f8.weights_largest(W, s), dn(b), dn(r), kind, gated)
    if y is not None:
        assert_rows(y, wy, ey, used, "y")
    if y8 is not None:
        f8.assert_rows8(y8, wy, ey, used, "y8")
    if pre:
        assert_rows(z, wz, ez, used, "pre")


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("H,O", [(32, 32), (64, 64), (96, 160), (128, 128), (160, 288), (256, 256), (1056, 96), (640, 544)])
def test_product_sizes(moe, counts, H, O):
    run_product(moe, counts, H, O, pad=2)
    run_product(moe, counts, H, O, "silu", True, pre=True, pad=1)


@pytest.mark.parametrize("counts", [[3, 0, 9, 1], [70, 0, 300]])
@pytest.mark.parametrize("kind", ref.ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_product_epilogues(moe, counts, kind, gated):
    for bias, residual, pre, out in ((True, True, True, "both"), (True, False, False, "fp8"), (False, True, False, "bf16"),
                                     (False, False, True, "fp8")):
        run_product(moe, counts, 192, 160, kind, gated, bias, residual, pre, out, pad=3)


@pytest.mark.parametrize("counts", [[2, 1], [400]])
def test_product_residual_in_place(moe, counts):
    run_product(moe, counts, 128, 288, "gelu", False, True, True, True, pad=4, in_place=True)


@pytest.mark.parametrize("counts", [[1, 0, 1, 1, 0, 0, 1, 1], [9, 31, 0, 24], [260, 30]])
def test_product_long_rows(moe, counts):
    """Long K, over several slabs of scale bytes: a skipped or doubled step shows."""
    run_product(moe, counts, 7168, 256, "silu", True, pad=1)
    run_product(moe, counts, 8224, 160)


@pytest.mark.parametrize("counts", [[5, 0, 2], [300, 20]])
def test_product_wide_outputs(moe, counts):
    """Several slabs of scale bytes in the output, and an up half that starts inside a block of 128."""
    run_product(moe, counts, 96, 4160, "relu", True, out="fp8", pad=1)
    run_product(moe, counts, 64, 8224, pad=1)


def run_dgrad(moe, counts, O, H, kind="none", gated=False, pre=False, out="both", pad=0, in_place=False):
    rng = np.random.default_rng(H + O)
    off = offsets(counts)
    used, El = int(off[-1]), len(counts)
    rows, wide = used + pad, 2 * H if gated else H
    say("dgrad", counts, O, H, kind, gated, pre, out, pad)
    gy, gv = rows8(rng, rows, O)
    Wt, s, Wv = weights8(rng, El, H, O)
    z = bf16(rng, rows, wide, scale=2.0) if pre else None
    gx, gx8 = canary(rows, wide) if out != "fp8" else None, empty8(rows, wide) if out != "bf16" else None
    if in_place:
        gx[:used] = z[:used].to(DEV)
    moe.moe_expert_product_fp8_dgrad(gpu(gy), gpu(off), gpu(Wt), gpu(s), gx if in_place else up(z), kind, gated,
                                     need_x=gx is not None, grad_x=gx, grad_x8=gx8)
    torch.cuda.synchronize()
    want, err = f8.dgrad(gv, f8.rows_largest(gy, O), off, Wv, f8.weights_largest(Wt, s), dn(z), kind, gated)
    if gx is not None:
        assert_rows(gx, want, err, used, "grad_x")
    if gx8 is not None:
        f8.assert_rows8(gx8, want, err, used, "grad_x8")


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("O,H", [(32, 32), (96, 160), (128, 256), (288, 128), (1056, 96), (640, 544)])
def test_dgrad_sizes(moe, counts, O, H):
    run_dgrad(moe, counts, O, H, pad=2)
    run_dgrad(moe, counts, O, H, "silu", True, True, pad=1)


@pytest.mark.parametrize("counts", [[3, 0, 9, 1], [70, 0, 300]])
@pytest.mark.parametrize("kind", ref.ACTS)
def test_dgrad_activations(moe, counts, kind):
    for gated, out in ((False, "both"), (True, "fp8"), (True, "bf16"), (False, "fp8")):
        run_dgrad(moe, counts, 192, 160, kind, gated, True, out, pad=3)


def test_dgrad_in_place_and_wide(moe):
    run_dgrad(moe, [300, 5], 128, 288, "gelu", True, True, "both", 2, in_place=True)
    run_dgrad(moe, [40, 0, 270], 64, 4160, "silu", True, True, "fp8", 1)
    run_dgrad(moe, [9, 260], 8224, 96)


# Rows and columns enough that tiles of 64 rows, or of 128, are more than blocks run at once.
MANY = [[4200], [1300, 0, 2900, 1], [257] * 16, [255, 1, 64, 0, 192, 3690], [31, 4000, 65, 129]]


@pytest.mark.parametrize("counts", MANY)
@pytest.mark.parametrize("H", [32, 96, 128, 224, 256, 544, 1056])
def test_product_many_rows(moe, counts, H):
    run_product(moe, counts, H, 1184, pad=2)
    run_product(moe, counts, H, 640, "silu", True, pre=True, pad=1)


@pytest.mark.parametrize("kind", ref.ACTS)
def test_product_many_rows_epilogues(moe, kind):
    for gated, O in ((False, 1184), (True, 608)):
        for bias, residual, pre, out in ((True, True, True, "both"), (False, True, False, "bf16"), (False, False, True, "fp8")):
            run_product(moe, MANY[1], 192, O, kind, gated, bias, residual, pre, out, pad=3)
    run_product(moe, MANY[3], 128, 1312, kind, False, True, True, True, pad=4, in_place=True)


@pytest.mark.parametrize("counts", MANY)
@pytest.mark.parametrize("O", [32, 160, 384, 1056])
def test_dgrad_many_rows(moe, counts, O):
    run_dgrad(moe, counts, O, 1184, pad=2)
    run_dgrad(moe, counts, O, 1184, "silu", True, True, pad=1)


@pytest.mark.parametrize("kind", ref.ACTS)
def test_dgrad_many_rows_activations(moe, kind):
    for gated, out in ((False, "both"), (True, "fp8"), (True, "bf16"), (False, "fp8")):
        run_dgrad(moe, MANY[1], 192, 1184, kind, gated, True, out, pad=3)
    run_dgrad(moe, MANY[3], 128, 1312, kind, True, True, "both", 2, in_place=True)


# Whole tiles of 256 rows, over 256 of them, and a last round that is cut into slices or is not.
WHOLE = [[16400], [5200, 0, 11300, 1], [257] * 64, [20000, 255, 1]]


@pytest.mark.parametrize("counts", WHOLE)
@pytest.mark.parametrize("H", [32, 128, 224, 352, 544])
def test_product_whole_tiles(moe, counts, H):
    if H % 128:
        run_product(moe, counts, H, 1184, pad=2)
    else:
        run_product(moe, counts, H, 640, "silu", True, pre=True, pad=1)


@pytest.mark.parametrize("kind", ref.ACTS)
def test_product_whole_tiles_epilogues(moe, kind):
    run_product(moe, WHOLE[1], 160, 608, kind, True, True, True, True, "both", pad=3)
    run_product(moe, WHOLE[3], 96, 1312, kind, False, True, True, True, "bf16", pad=4, in_place=True)


@pytest.mark.parametrize("counts", WHOLE[:3])
@pytest.mark.parametrize("O", [32, 288, 384])
def test_dgrad_whole_tiles(moe, counts, O):
    run_dgrad(moe, counts, O, 1184, pad=2)


@pytest.mark.parametrize("kind", ref.ACTS)
def test_dgrad_whole_tiles_activations(moe, kind):
    run_dgrad(moe, WHOLE[1], 160, 1184, kind, True, True, "both", pad=3)
    run_dgrad(moe, WHOLE[3], 96, 1312, kind, False, True, "both", 2, in_place=True)


def test_offsets_out_of_range(moe):
    """Offsets past the buffer are clamped, and where they decrease nothing is computed."""
    rng = np.random.default_rng(5)
    for rows, O in ((40, 64), (600, 512), (4200, 1184), (16400, 1184)):
        x, xv = rows8(rng, rows, 128)
        W, s, Wv = weights8(rng, 3, O, 128)
        for off, used in (([-5, 10, 20, rows + 1000], rows), ([0, 30, 20, 25], 0)):
            say("offsets", off)
            off = np.array(off, np.int32)
            y, y8 = canary(rows, O), empty8(rows, O)
            moe.moe_expert_product_fp8(gpu(x), gpu(off), gpu(W), gpu(s), y=y, y8=y8)
            torch.cuda.synchronize()
            wy, _, _, ey = f8.product(xv, f8.rows_largest(x, 128), np.clip(off, 0, rows) if used else np.zeros(4, np.int32), Wv,
                                      f8.weights_largest(W, s))
            assert_rows(y, wy, ey, used, "y")
            f8.assert_rows8(y8, wy, ey, used, "y8")


@pytest.mark.parametrize("counts,O", [([3, 4], 96), ([300, 20], 96), ([4000, 300], 1184), ([16000, 300], 1184)])
def test_nan_and_infinities(moe, counts, O):
    """A NaN code or scale reaches its own row's results, or its own column's, and no others; codes and scales past K,
    in the padding, and of other rows do not. An infinite result becomes a NaN code, and bf16's infinity."""
    rng = np.random.default_rng(6)
    H = 160  # K ends inside a step of 128, scale bytes inside a word
    off = offsets(counts)
    n = int(off[-1])
    say("NaN", counts)
    x, xv = rows8(rng, n, H)
    W, s, Wv = weights8(rng, 2, O, H)
    x[1, 70] = 0x7F              # a code of row 1
    x[2, H + 4] = 0xFF           # the last scale of row 2
    x[:, H + H // 32:] = 0xFF    # padding, which the rows' readers must not multiply
    W[1, 5, 159] = 0xFF          # the last code of a column of expert 1
    bias = torch.zeros(2, O, dtype=torch.bfloat16)
    bias[0, 40] = float("inf")
    y, y8 = canary(n, O), empty8(n, O)
    moe.moe_expert_product_fp8(gpu(x), gpu(off), gpu(W), gpu(s), bias=up(bias), y=y, y8=y8)
    torch.cuda.synchronize()
    got, d = dn(y.cpu()), f8.decode_rows(y8.cpu().numpy(), O)
    bad = np.zeros((n, O), bool)
    bad[1:3] = True
    bad[off[1]:, 5] = True
    assert (np.isnan(got) == bad).all()
    inf = np.zeros((n, O), bool)
    inf[:off[1], 40] = True
    assert (np.isinf(got) == (inf & ~bad)).all()
    assert (np.isnan(d) == (bad | inf)).all()


@pytest.mark.parametrize("counts,O", [([3, 4], 96), ([300, 20], 96), ([4000, 300], 1184), ([16000, 300], 1184)])
def test_scales_of_every_size(moe, counts, O):
    """Negative, huge, least normal, subnormal and zero scales of the weights on each kernel; NaN and infinite ones reach
    the columns of their block, in their expert's rows, and nothing else."""
    rng = np.random.default_rng(7)
    H = 384
    off = offsets(counts)
    n = int(off[-1])
    say("scales", counts, O)
    x, xv = rows8(rng, n, H)
    W, s, _ = weights8(rng, 2, O, H)
    s[0, 0] = [-0.75, 2.0 ** -140, 1.5 * 2.0 ** 90]
    s[1, 0] = [0.0, 2.0 ** -126, -1.25 * 2.0 ** -100]
    for bad in (False, True):
        if bad:
            s[0, 0, 1], s[1, 0, 2] = np.nan, np.inf
        y, y8 = canary(n, O), empty8(n, O)
        moe.moe_expert_product_fp8(gpu(x), gpu(off), gpu(W), gpu(s), y=y, y8=y8)
        torch.cuda.synchronize()
        if bad:
            got, d = dn(y.cpu()), f8.decode_rows(y8.cpu().numpy(), O)
            assert not np.isfinite(got[:, :128]).any() and np.isnan(d[:, :128]).all()
            assert np.isfinite(got[:, 128:]).all() and np.isfinite(d[:, 128:]).all()
            continue
        wy, _, _, ey = f8.product(xv, f8.rows_largest(x, H), off, f8.decode_weights(W, s), f8.weights_largest(W, np.abs(s)))
        # a scale below 2^-126 may count as 2^-127
        codes = np.abs(f8.e4m3(W)).max(2)
        for l in range(2):
            b, e = off[l], off[l + 1]
            ey[b:e] += 2.0 ** -126 * np.abs(xv[b:e]).sum(1)[:, None] * codes[l]
        assert_rows(y, wy, ey, n, "y")
        f8.assert_rows8(y8, wy, ey, n, "y8")


@pytest.mark.parametrize("rows", [2, 300, 9000, 40000])
def test_weights_past_32_bits(moe, rows):
    """Weights past 2^31 bytes, on each kernel: the last expert's first and last 150 rows against float64."""
    El, O, H = 40, 2048, 7168
    say("large", El, O, H, rows)
    g = torch.Generator(device=DEV).manual_seed(0)
    W = torch.randint(0, 0x70, (El, 2 * O, H), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.rand(El, 2 * O // 128, H // 128, generator=g, device=DEV) * 1e-3
    x, xv = rows8(np.random.default_rng(1), rows, H)
    off = torch.zeros(El + 1, dtype=torch.int32, device=DEV)
    off[El] = rows
    y, y8 = moe.moe_expert_product_fp8(gpu(x), off, W, s, act="silu", gated=True, fp8=True)
    torch.cuda.synchronize()
    W, s = W[El - 1:].cpu().numpy(), s[El - 1:].cpu().numpy()
    some = np.unique(np.r_[:min(rows, 150), max(rows - 150, 0):rows])
    x, xv, y, y8 = x[some], xv[some], y.cpu()[some], y8.cpu()[some]
    wy, _, _, ey = f8.product(xv, f8.rows_largest(x, H), np.array([0, len(some)]), f8.decode_weights(W, s),
                              f8.weights_largest(W, s), kind="silu", gated=True)
    assert_rows(y, wy, ey, len(some), "y")
    f8.assert_rows8(y8, wy, ey, len(some), "y8")


def test_rows_past_32_bits(moe):
    """Rows past 2^31 bytes, in and out: the last ones against the same rows alone."""
    n, H, O = 320000, 7168, 7168
    say("rows", n, H, O)
    x = torch.full((n, moe.moe_fp8_row_bytes(H)), 0x38, dtype=torch.uint8, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(0)
    x[:, :H] = torch.randint(0, 0x40, (n, 1), generator=g, device=DEV, dtype=torch.uint8) + 8
    x[:, H:] = 127
    W = torch.randint(0, 0x60, (1, O, H), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.full((1, O // 128, H // 128), 1e-3, device=DEV)
    off = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    y, y8 = moe.moe_expert_product_fp8(x, off, W, s, fp8=True)
    k = 9000  # enough for the same kernel
    z, z8 = moe.moe_expert_product_fp8(x[n - k:].contiguous(), torch.tensor([0, k], dtype=torch.int32, device=DEV), W, s,
                                       fp8=True)
    torch.cuda.synchronize()
    assert torch.equal(y[n - k:], z) and torch.equal(y8[n - k:], z8)


@pytest.mark.parametrize("counts,H,O", [([3, 0, 2, 9], 512, 256), ([200, 0, 313, 41], 1024, 512), ([2000, 0, 2300, 41], 1184, 640),
                                          ([9000, 0, 7300, 41], 1184, 1184)])
def test_captured_and_replayed(moe, counts, H, O):
    """A layer's two products captured on a stream of their own, replayed on new rows and new offsets."""
    rng = np.random.default_rng(2)
    El, n = len(counts), sum(counts) + 3
    say("captured", counts, H, O)
    x, off = gpu(rows8(rng, n, H)[0]), gpu(offsets(counts))
    W1, s1, _ = weights8(rng, El, 2 * O, H)
    W2, s2, _ = weights8(rng, El, H, O)
    W1, s1, W2, s2 = gpu(W1), gpu(s1), gpu(W2), gpu(s2)
    h8, y = empty8(n, O), canary(n, H)

    def step():
        moe.moe_expert_product_fp8(x, off, W1, s1, act="silu", gated=True, need_y=False, y8=h8)
        moe.moe_expert_product_fp8(h8, off, W2, s2, y=y)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    torch.cuda.synchronize()
    for i in range(4):
        x.copy_(gpu(rows8(rng, n, H)[0]))
        off.copy_(gpu(offsets(rng.permutation(counts))))
        h8.fill_(0x5A), y.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        a, b = h8.clone(), y.clone()
        h8.fill_(0x5A), y.fill_(7)
        step()
        torch.cuda.synchronize()
        assert torch.equal(a, h8) and torch.equal(b, y), i
