"""The RMS norm and its gradient on the GPU against float64.

Bars: the bounds of a float32 computation that tests/fp8_reference.py derives,
plus half a step of the output's type (2^-8 bf16, 2^-24 float32); FP8 rows as
assert_rows8 says. The sum with the residual is compared bit for bit. Every
test prints its case before touching the GPU.
"""

import numpy as np
import pytest
import torch

import fp8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import combine_route_topk_amd
    return combine_route_topk_amd


def say(*a):
    print("[case]", *a, flush=True)


def rand(rng, *shape, dtype=BF):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)


def dn(t):
    return t.detach().cpu().double().numpy()


def near(got, want, err, what, ok=None):
    half = 2.0 ** -8 if got.dtype == BF else 2.0 ** -24
    d = np.abs(dn(got) - want) - (err + half * (np.abs(want) + err) + 2.0 ** -134)
    assert (d <= 0).all(), f"{what}: {int((d > 0).sum())} of {d.size} past the bound, worst by {d.max()}"


def rows8(T, H, moe):
    return torch.full((T, moe.moe_fp8_row_bytes(H)), 0x5A, dtype=torch.uint8, device=DEV)


def run_norm(moe, T, H, dt=BF, wdt=BF, residual=True, fp8=True, need_y=True, seed=0):
    rng = np.random.default_rng(seed + T + H)
    say("norm", T, H, dt, wdt, residual, fp8, need_y)
    x = (rand(rng, T, H, dtype=F) * torch.from_numpy(np.exp2(rng.integers(-8, 8, (T, 1))).astype(np.float32))).to(dt)
    w, r = rand(rng, H, dtype=wdt), rand(rng, T, H, dtype=dt) if residual else None
    y8 = rows8(T + 1, H, moe) if fp8 else None
    total, y, q = moe.moe_rms_norm(x.to(DEV), w.to(DEV), None if r is None else r.to(DEV), EPS, need_y=need_y,
                                   y8=y8[:T] if fp8 else None)
    torch.cuda.synchronize()
    t = (x.float() + r.float()).to(dt) if residual else x
    assert torch.equal(total.cpu(), t)
    v, e = ref.norm(dn(t), dn(w), np.float64(np.float32(EPS)))
    if need_y:
        near(y, v, e, "y")
    else:
        assert y is None
    if fp8:
        ref.assert_rows8(y8, v, e, T, "y8")
    else:
        assert q is None


WIDTHS = [32, 64, 480, 512, 544, 1024, 1056, 2048, 2080, 4096, 4128, 7168, 8192, 8224, 16384, 16416, 32768, 32800, 65536]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dt", [BF, F])
def test_norm_widths(moe, H, dt):
    for T in (1, 3, 5):
        run_norm(moe, T, H, dt)
    run_norm(moe, 6, H, dt, F, residual=False, need_y=False)


@pytest.mark.parametrize("H", [8, 24, 520, 1000, 3000, 8200, 20008, 65528])
@pytest.mark.parametrize("dt,wdt", [(BF, BF), (F, F), (BF, F), (F, BF)])
def test_norm_odd_widths(moe, H, dt, wdt):
    run_norm(moe, 7, H, dt, wdt, fp8=False)
    run_norm(moe, 2, H, dt, wdt, residual=False, fp8=False)


@pytest.mark.parametrize("T,H", [(128, 7168), (4099, 2048), (1023, 4096), (30000, 64)])
def test_norm_many_rows(moe, T, H):
    run_norm(moe, T, H)


def test_norm_past_one_grid(moe):
    """More rows than one launch has blocks: four rows a block of 64 columns."""
    T, H = (1 << 24) + 5, 64
    say("norm", T, H)
    g = torch.Generator(device=DEV).manual_seed(0)
    x = torch.randn(T, H, generator=g, device=DEV).to(BF)
    w = torch.ones(H, dtype=BF, device=DEV)
    _, y, y8 = moe.moe_rms_norm(x, w, eps=EPS, fp8=True)
    tail = slice(T - 70, T)
    _, y2, z8 = moe.moe_rms_norm(x[tail].contiguous(), w, eps=EPS, fp8=True)
    torch.cuda.synchronize()
    assert torch.equal(y[tail], y2) and torch.equal(y8[tail], z8)


@pytest.mark.parametrize("which", ["x", "residual"])
@pytest.mark.parametrize("dt", [BF, F])
def test_norm_total_in_place(moe, which, dt):
    rng = np.random.default_rng(1)
    for H in (96, 2048, 7168):
        say("in place", which, dt, H)
        x, r, w = rand(rng, 5, H, dtype=dt).to(DEV), rand(rng, 5, H, dtype=dt).to(DEV), rand(rng, H).to(DEV)
        t, y, y8 = moe.moe_rms_norm(x, w, r, EPS, fp8=True)
        a, b = x.clone(), r.clone()
        t2, y2, z8 = moe.moe_rms_norm(a, w, b, EPS, fp8=True, total=a if which == "x" else b)
        torch.cuda.synchronize()
        assert t2.data_ptr() == (a if which == "x" else b).data_ptr()
        assert torch.equal(t, t2) and torch.equal(y, y2) and torch.equal(y8, z8)


def test_norm_special_values(moe):
    """A NaN or an infinity takes its own row and no other; zeros give zeros; a row of tiny values is what eps leaves."""
    for H in (64, 2048, 7168):
        say("special values", H)
        x = torch.ones(6, H)
        x[1, 5], x[2, H - 1], x[3], x[4] = float("nan"), float("inf"), 0.0, 2.0 ** -100
        w = torch.full((H,), 2.0)
        _, y, y8 = moe.moe_rms_norm(x.to(DEV, BF), w.to(DEV, BF), eps=1.0, fp8=True)
        torch.cuda.synchronize()
        y, q = y.float().cpu(), y8.cpu().numpy()
        assert torch.isnan(y[1]).all() and torch.isnan(y[2, H - 1]) and (y[2, :H - 1] == 0).all()
        d = ref.decode_rows(q, H)
        assert np.isnan(d[1]).all() and np.isnan(d[2, H - 1]) and (d[2, :H - 32] == 0).all()
        assert (y[3] == 0).all() and (d[3] == 0).all() and (q[3, H:] == 0).all()
        assert (y[4] == 2.0 ** -99).all() and (d[4] == 2.0 ** -99).all()
        for i in (0, 5):
            assert (np.abs(d[i] - np.sqrt(2.0)) < 2.0 ** -4 * 1.5).all() and (y[i] == y[0, 0]).all()


def run_backward(moe, T, H, dt=BF, wdt=BF, stream=True, seed=0, wide=1.0):
    rng = np.random.default_rng(seed + T + H)
    say("backward", T, H, dt, wdt, stream)
    t, gy = (rand(rng, T, H, dtype=F) * wide).to(dt), rand(rng, T, H)
    w, gt = rand(rng, H, dtype=wdt), rand(rng, T, H, dtype=dt) if stream else None
    ws = torch.full((moe.moe_rms_norm_backward_workspace_size(T, H),), 0xFF, dtype=torch.uint8, device=DEV)
    gx, gw = moe.moe_rms_norm_backward(gy.to(DEV), t.to(DEV), w.to(DEV), EPS, None if gt is None else gt.to(DEV),
                                       workspace=ws)
    torch.cuda.synchronize()
    wx, ww, ex, ew = ref.norm_backward(dn(gy), dn(t), dn(w), np.float64(np.float32(EPS)), None if gt is None else dn(gt))
    near(gx, wx, ex, "grad_x")
    near(gw, ww, ew, "grad_weight")


@pytest.mark.parametrize("H", [8, 512, 1000, 1024, 2048, 2056, 4096, 7168, 8200, 16384, 16392, 40000, 65536])
@pytest.mark.parametrize("dt,wdt", [(BF, BF), (F, F), (BF, F), (F, BF)])
def test_backward_widths(moe, H, dt, wdt):
    for T in (1, 3, 9):
        run_backward(moe, T, H, dt, wdt, stream=T != 3, wide=0.01 if T == 9 else 1.0)


@pytest.mark.parametrize("T,H", [(128, 7168), (5000, 2048), (4097, 64), (1500, 4096), (1100, 16400)])
def test_backward_many_rows(moe, T, H):
    run_backward(moe, T, H)


def test_backward_parts_and_accumulation(moe):
    rng = np.random.default_rng(4)
    for T, H in ((0, 64), (5, 64), (40, 7168), (3, 20000)):
        say("parts", T, H)
        t, gy, w = rand(rng, T, H).to(DEV), rand(rng, T, H).to(DEV), rand(rng, H).to(DEV)
        gt = rand(rng, T, H).to(DEV)
        gx, gw = moe.moe_rms_norm_backward(gy, t, w, EPS, gt)
        a, none = moe.moe_rms_norm_backward(gy, t, w, EPS, gt, need_weight=False)
        assert none is None and torch.equal(a, gx)
        none, b = moe.moe_rms_norm_backward(gy, t, w, EPS, gt, need_x=False)
        assert none is None and torch.equal(b, gw)
        c = gt.clone()
        d, _ = moe.moe_rms_norm_backward(gy, t, w, EPS, c, grad_x=c)
        assert torch.equal(d, gx)
        acc = torch.full((H,), 3.0, device=DEV)
        moe.moe_rms_norm_backward(gy, t, w, EPS, grad_weight=acc, accumulate=True)
        torch.cuda.synchronize()
        assert torch.equal(acc, 3.0 + gw)
        if T == 0:
            assert (gw == 0).all()


def test_norm_captured_and_replayed(moe):
    """Forward and backward in one graph, on a stream of their own, replayed on new inputs."""
    rng = np.random.default_rng(8)
    T, H = 300, 2048
    say("captured", T, H)
    x, r, w, gy = (rand(rng, *s).to(DEV) for s in ((T, H), (T, H), (H,), (T, H)))
    out = [torch.empty_like(x), torch.empty_like(x), rows8(T, H, moe), torch.empty_like(x), torch.empty(H, device=DEV)]
    ws = torch.empty(moe.moe_rms_norm_backward_workspace_size(T, H), dtype=torch.uint8, device=DEV)

    def step():
        moe.moe_rms_norm(x, w, r, EPS, total=out[0], y=out[1], y8=out[2])
        moe.moe_rms_norm_backward(gy, out[0], w, EPS, grad_x=out[3], grad_weight=out[4], workspace=ws)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    torch.cuda.synchronize()
    for i in range(4):
        x.copy_(rand(rng, T, H))
        for o in out:
            o.fill_(7)
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, out)), i


def test_norm_on_a_given_stream(moe):
    rng = np.random.default_rng(9)
    x, w, gy = rand(rng, 64, 4096).to(DEV), rand(rng, 4096).to(DEV), rand(rng, 64, 4096).to(DEV)
    want = [*moe.moe_rms_norm(x, w, eps=EPS, fp8=True)[1:], *moe.moe_rms_norm_backward(gy, x, w, EPS)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for given in (s, s.cuda_stream):
        got = [*moe.moe_rms_norm(x, w, eps=EPS, fp8=True, stream=given)[1:],
               *moe.moe_rms_norm_backward(gy, x, w, EPS, stream=given)]
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
