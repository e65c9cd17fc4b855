"""The experts' products and their gradients on the GPU against float64.

Bars: the error bounds of a float32 computation that tests/ops_reference.py
derives next to each form, plus half a bf16 step (2^-8 of the value, itself
within that bound) where the output is bf16. Rows of no expert stay as they
were, bit for bit. Every test prints the case before touching the GPU.
"""

import numpy as np
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CANARY = 0x5A5A


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import combine_route_topk_amd
    return combine_route_topk_amd


def say(*a):
    print("[case]", *a, flush=True)


def bf16(rng, *shape, scale=1.0):
    """A bf16 CPU tensor of scaled normals."""
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).bfloat16()


def canary(*shape):
    return torch.full(shape, CANARY, dtype=torch.int16, device=DEV).view(torch.bfloat16)


def dn(t):
    return None if t is None else t.double().numpy()


def up(t):
    return None if t is None else t.to(DEV)


def offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def assert_rows(got, want, err, used, what):
    """bf16 rows within the bound and half a step; unused rows untouched."""
    got = got.cpu()
    assert (got[used:].view(torch.int16).numpy() == CANARY).all(), f"{what}: rows behind the last expert's changed"
    g, v, e = got[:used].double().numpy(), want[:used], err[:used]
    d = np.abs(g - v) - (e + 2.0 ** -8 * (np.abs(v) + e) + 2.0 ** -134)
    assert (d <= 0).all(), f"{what}: {int((d > 0).sum())} of {d.size} past the bound, worst by {d.max()}"


def run_product(moe, counts, H, O, kind="none", gated=False, bias=False, residual=False, pre=False, pad=0, seed=0,
                in_place=False):
    rng = np.random.default_rng(seed + H + O)
    off = offsets(counts)
    used, El = int(off[-1]), len(counts)
    rows, wide = used + pad, 2 * O if gated else O
    x, W = bf16(rng, rows, H), bf16(rng, El, wide, H, scale=H ** -0.5)
    b = bf16(rng, El, wide) if bias else None
    r = bf16(rng, rows, O) if residual else None
    say(counts, H, O, kind, gated, bias, residual, pre, pad)
    y = canary(rows, O)
    if in_place:
        y[:used] = r[:used].to(DEV)
    z = canary(rows, wide) if pre else None
    moe.moe_expert_product(up(x), torch.from_numpy(off).to(DEV), up(W), bias=up(b),
                           residual=y if in_place else up(r), act=kind, gated=gated, y=y, pre=z)
    torch.cuda.synchronize()
    wy, wz, ez, ey = ref.product(dn(x), off, dn(W), dn(b), dn(r), kind, gated)
    assert_rows(y, wy, ey, used, "y")
    if pre:
        assert_rows(z, wz, ez, used, "pre")


COUNTS = [[1], [0, 3, 0], [5, 0, 17], [16, 32, 48, 1], [33, 64, 65], [100, 0, 140, 7], [255, 257], [300], [129, 127]]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("H,O", [(8, 8), (64, 64), (72, 40), (200, 136), (256, 264), (1000, 48), (512, 520)])
def test_product_sizes(moe, counts, H, O):
    run_product(moe, counts, H, O, pad=2)
    run_product(moe, counts, H, O, "silu", True, pre=True, pad=1)


@pytest.mark.parametrize("counts", [[3, 0, 9, 1], [70, 0, 300]])
@pytest.mark.parametrize("kind", ref.ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_product_epilogues(moe, counts, kind, gated):
    for bias, residual, pre in ((True, True, True), (True, False, False), (False, True, False), (False, False, True)):
        run_product(moe, counts, 192, 152, kind, gated, bias, residual, pre, pad=3)


@pytest.mark.parametrize("counts", [[2, 1], [400]])
def test_product_residual_in_place(moe, counts):
    run_product(moe, counts, 128, 264, "gelu", False, True, True, True, pad=4, in_place=True)


@pytest.mark.parametrize("counts", [[1, 0, 1, 1, 0, 0, 1, 1], [9, 31, 0, 24], [260, 30]])
def test_product_long_rows(moe, counts):
    """The widest inner sizes of the workloads; K is long, so a skipped or doubled step shows."""
    run_product(moe, counts, 7168, 256, "silu", True)
    run_product(moe, counts, 2048, 1032, "none", False, True, True)


def test_product_many_experts(moe):
    rng = np.random.default_rng(0)
    run_product(moe, rng.integers(0, 3, 1024).tolist(), 64, 72, "relu", False, True)
    run_product(moe, rng.integers(0, 40, 200).tolist(), 72, 64, "silu", True)


def test_product_long_batch(moe):
    """More tiles than blocks: every block takes several, and rows stay with their expert."""
    rng = np.random.default_rng(1)
    run_product(moe, (rng.integers(0, 9000, 5)).tolist(), 96, 160, "gelu_tanh", False, True, pad=100)
    run_product(moe, [0, 20000, 1], 64, 520, "silu", True, pre=True)


def test_product_no_rows(moe):
    """Offsets that give no expert a row write nothing; an empty buffer is no error."""
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    W = torch.ones(3, 64, 64, dtype=torch.bfloat16, device=DEV)
    for rows in (1, 40, 3000):
        y = canary(rows, 64)
        moe.moe_expert_product(torch.ones(rows, 64, dtype=torch.bfloat16, device=DEV), off, W, y=y)
        g = canary(rows, 64)
        moe.moe_expert_product_dgrad(y, off, W, grad_x=g)
        assert (y.view(torch.int16) == CANARY).all() and (g.view(torch.int16) == CANARY).all()
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    assert moe.moe_expert_product(e, off, W).shape == (0, 64)
    assert moe.moe_expert_product_dgrad(e, off, W).shape == (0, 64)
    gW, gb = torch.full((3, 64, 64), 2.0, device=DEV), torch.full((3, 64), 2.0, device=DEV)
    moe.moe_expert_product_wgrad(e, e, off, gW, gb, accumulate=True)
    assert (gW == 2).all() and (gb == 2).all()
    moe.moe_expert_product_wgrad(e, e, off, gW, gb)
    assert (gW == 0).all() and (gb == 0).all()


def test_product_rows_do_not_mix(moe):
    """NaN and infinities in one expert's rows, and behind the last row, reach no other row or expert."""
    rng = np.random.default_rng(4)
    for counts, pad in (([20, 6, 30], 5), ([200, 60, 300], 70)):
        off = offsets(counts)
        rows = int(off[-1]) + pad
        x, W = bf16(rng, rows, 136), bf16(rng, 3, 72, 136, scale=0.1)
        clean = moe.moe_expert_product(up(x), torch.from_numpy(off).to(DEV), up(W), y=canary(rows, 72))
        dirty = x.clone()
        a = int(off[1])
        dirty[a:int(off[2])], dirty[int(off[3]):], dirty[3] = float("nan"), float("nan"), float("inf")
        y = moe.moe_expert_product(up(dirty), torch.from_numpy(off).to(DEV), up(W), y=canary(rows, 72))
        same = [i for i in range(rows) if i != 3 and not int(off[1]) <= i < int(off[2])]
        say(counts, "nan")
        assert torch.equal(y.view(torch.int16)[same], clean.view(torch.int16)[same])
        gW = moe.moe_expert_product_wgrad(up(dirty), up(dirty), torch.from_numpy(off).to(DEV))
        cW = moe.moe_expert_product_wgrad(up(x), up(x), torch.from_numpy(off).to(DEV))
        assert torch.equal(gW[2], cW[2]) and torch.isnan(gW[1]).all()


def test_product_broken_offsets(moe):
    """Offsets outside the buffer or decreasing are clamped: nothing outside the buffers is touched."""
    x = torch.ones(40, 64, dtype=torch.bfloat16, device=DEV)
    W = torch.ones(3, 64, 64, dtype=torch.bfloat16, device=DEV)
    for off in ([0, 10, 30, 99], [-5, 10, 20, 40], [20, 10, 40, 40], [2 ** 31 - 1, 0, 0, 0]):
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        buf = canary(60, 64)
        say(off)
        moe.moe_expert_product(x, o, W, y=buf[10:50])
        moe.moe_expert_product_wgrad(x, x, o)
        torch.cuda.synchronize()
        assert (buf[:10].view(torch.int16) == CANARY).all() and (buf[50:].view(torch.int16) == CANARY).all()
    assert (buf[10:50].view(torch.int16) == CANARY).all()


def run_dgrad(moe, counts, O, H, kind="none", gated=False, pre=False, pad=0, in_place=False):
    rng = np.random.default_rng(O + H)
    off = offsets(counts)
    used, El = int(off[-1]), len(counts)
    rows, wide = used + pad, 2 * H if gated else H
    gy, W = bf16(rng, rows, O), bf16(rng, El, O, H, scale=O ** -0.5)
    z = bf16(rng, rows, wide, scale=2.0) if pre else None
    say(counts, O, H, kind, gated, pre, pad)
    out = canary(rows, wide)
    if in_place:
        out[:used] = z[:used].to(DEV)
    moe.moe_expert_product_dgrad(up(gy), torch.from_numpy(off).to(DEV), up(W), pre=out if in_place else up(z),
                                 act=kind, gated=gated, grad_x=out)
    torch.cuda.synchronize()
    want, err = ref.dgrad(dn(gy), off, dn(W), dn(z), kind, gated)
    assert_rows(out, want, err, used, "grad_x")


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("O,H", [(8, 8), (64, 64), (40, 72), (136, 200), (264, 256), (48, 1000), (520, 512)])
def test_dgrad_sizes(moe, counts, O, H):
    run_dgrad(moe, counts, O, H, pad=2)
    run_dgrad(moe, counts, O, H, "silu", True, True, pad=1)


@pytest.mark.parametrize("kind", ref.ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_dgrad_activations(moe, kind, gated):
    run_dgrad(moe, [70, 0, 300, 3], 192, 152, kind, gated, True, pad=3)
    run_dgrad(moe, [7, 90], 104, 264, kind, gated, True, in_place=True, pad=2)


def test_dgrad_long(moe):
    run_dgrad(moe, [9, 260], 7168, 264, "silu", True, True)
    run_dgrad(moe, [0, 20000, 1], 64, 520, "silu", True, True)
    rng = np.random.default_rng(0)
    run_dgrad(moe, rng.integers(0, 3, 1024).tolist(), 64, 72)


def run_wgrad(moe, counts, O, H, bias=False, fp32=False, accumulate=False, pad=0):
    rng = np.random.default_rng(O + H)
    off = offsets(counts)
    El, rows = len(counts), int(off[-1]) + pad
    gy, x = bf16(rng, rows, O), bf16(rng, rows, H)
    say(counts, O, H, bias, fp32, accumulate, pad)
    had_W = torch.from_numpy(rng.standard_normal((El, O, H)).astype(np.float32))
    had_b = torch.from_numpy(rng.standard_normal((El, O)).astype(np.float32))
    gW = had_W.to(DEV) if fp32 else torch.full((El, O, H), 7.0, dtype=torch.bfloat16, device=DEV)
    gb = had_b.to(DEV) if bias else None
    moe.moe_expert_product_wgrad(up(gy), up(x), torch.from_numpy(off).to(DEV), gW, gb, accumulate)
    torch.cuda.synchronize()
    wW, wb, eW, eb = ref.wgrad(dn(gy), dn(x), off, El)
    if accumulate:
        wW, wb = wW + had_W.double().numpy(), wb + had_b.double().numpy()
        eW, eb = eW + 2.0 ** -23 * (np.abs(wW) + 1), eb + 2.0 ** -23 * (np.abs(wb) + 1)
    got = gW.cpu().double().numpy()
    tol = eW + 2.0 ** -126 + (0 if fp32 else 2.0 ** -8 * (np.abs(wW) + eW))
    assert (np.abs(got - wW) <= tol).all(), (np.abs(got - wW) - tol).max()
    if bias:
        assert (np.abs(gb.cpu().double().numpy() - wb) <= eb + 2.0 ** -126).all()


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("O,H", [(8, 8), (64, 64), (40, 72), (136, 200), (264, 256), (48, 1000), (520, 512)])
def test_wgrad_sizes(moe, counts, O, H):
    run_wgrad(moe, counts, O, H, pad=2)
    run_wgrad(moe, counts, O, H, True, True, True, pad=1)


@pytest.mark.parametrize("counts", [[5000], [0, 3000, 1, 0], [40, 2, 700, 9, 0, 1300]])
def test_wgrad_long(moe, counts):
    """Long sums: few tiles, so their rows are split over blocks and joined."""
    for O, H in ((64, 64), (256, 512), (520, 264)):
        run_wgrad(moe, counts, O, H, True, True)
        run_wgrad(moe, counts, O, H, True, False)
        run_wgrad(moe, counts, O, H, True, True, True)


def test_wgrad_many_experts(moe):
    rng = np.random.default_rng(0)
    run_wgrad(moe, rng.integers(0, 5, 1024).tolist(), 64, 72, True)


def test_repeats_bit_for_bit(moe):
    """Two runs of each call give the same bits."""
    rng = np.random.default_rng(6)
    counts = [700, 0, 33, 2000]
    off = torch.from_numpy(offsets(counts)).to(DEV)
    x, W = up(bf16(rng, 2733, 256)), up(bf16(rng, 4, 512, 256, scale=0.06))
    say("repeat")
    y = [moe.moe_expert_product(x, off, W, act="silu", gated=True) for _ in range(2)]
    gy = up(bf16(rng, 2733, 512))
    d = [moe.moe_expert_product_dgrad(gy, off, W) for _ in range(2)]
    g = [moe.moe_expert_product_wgrad(gy, x, off, torch.empty(4, 512, 256, device=DEV)) for _ in range(2)]
    for a, b in (y, d, g):
        assert torch.equal(a, b)


def test_stream_and_graph(moe):
    """Another stream, and one graph of all three replayed with eager work between."""
    rng = np.random.default_rng(7)
    for counts in ([3, 0, 20], [300, 0, 900]):
        off = torch.from_numpy(offsets(counts)).to(DEV)
        rows = sum(counts)
        x, W, gy = up(bf16(rng, rows, 192)), up(bf16(rng, 3, 136, 192, scale=0.1)), up(bf16(rng, rows, 136))
        ws = torch.empty(max(16, moe.moe_expert_product_wgrad_workspace_size(3, rows, 136, 192)), dtype=torch.uint8,
                         device=DEV)
        y, gx = torch.empty(rows, 136, dtype=torch.bfloat16, device=DEV), torch.empty_like(x)
        gW, gb = torch.empty(3, 136, 192, device=DEV), torch.empty(3, 136, device=DEV)

        def step(stream=None):
            moe.moe_expert_product(x, off, W, act="silu", y=y, stream=stream)
            moe.moe_expert_product_dgrad(gy, off, W, grad_x=gx, stream=stream)
            moe.moe_expert_product_wgrad(gy, x, off, gW, gb, workspace=ws, stream=stream)

        say(counts)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        step(side)
        side.synchronize()
        want = [t.clone() for t in (y, gx, gW, gb)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for i in range(4):
            for t in (y, gx, gW, gb):
                t.fill_(3.0)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, (y, gx, gW, gb)))
            x.copy_(torch.randn(rows, 192, generator=torch.Generator().manual_seed(i)).bfloat16())
            step()
            torch.cuda.synchronize()
            want = [t.clone() for t in (y, gx, gW, gb)]


def test_workspace_belongs_to_the_launch_s_stream(moe):
    """The current stream is held up with a write to memory that it has already given back: a workspace or an
    output for another stream's launch may not be that memory."""
    rng = np.random.default_rng(8)
    rows, O, H = 6000, 256, 512
    gy, x, off = bf16(rng, rows, O), bf16(rng, rows, H), torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    n = moe.moe_expert_product_wgrad_workspace_size(1, rows, O, H)
    assert n > 0
    g, v = up(gy), up(x)
    want = moe.moe_expert_product_wgrad(g, v, off)
    torch.cuda.synchronize()
    say("workspace", n)
    for side in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        blocks = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(3)]
        torch.cuda._sleep(20_000_000)
        for b in blocks:
            b.fill_(255)
        del b, blocks
        got = moe.moe_expert_product_wgrad(g, v, off, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
