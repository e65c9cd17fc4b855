"""The combine's gradient on the GPU against float64.

Bars: grad_y within half a bf16 step (2^-8 of the value) of the product, which
float32 rounds once more (2^-24), or half the smallest bf16 step near zero;
grad_w, a sum of H exact products, within 2 H 2^-24 of the sum of their
magnitudes. Rows that no replica points at, and rows past a smaller y_rows,
stay as they were, bit for bit.
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


def make(T, H, k, spare, drop, dtype, seed):
    rng = np.random.default_rng(seed)
    rows = T * k + spare
    pos = rng.permutation(rows)[:T * k].astype(np.int32)
    pos[rng.random(T * k) < drop] = -1
    bf = lambda a: torch.from_numpy(a.astype(np.float32)).bfloat16()  # noqa: E731
    g = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(dtype)
    return g, bf(rng.standard_normal((rows, H))), pos.reshape(T, k), rng.standard_normal((T, k)).astype(np.float32)


def check(moe, g, y, pos, w, **kw):
    rows, H = y.shape
    gy = torch.full((rows, H), CANARY, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    gy, gw = moe.moe_combine_backward(g.to(DEV), y.to(DEV), torch.from_numpy(pos).to(DEV),
                                      torch.from_numpy(w).to(DEV), grad_y=gy, **kw)
    gd, yd = g.double().numpy(), y.double().numpy()
    want_y, want_w = ref.combine_backward(gd, yd, pos, w.astype(np.float64))
    left = np.isnan(want_y)
    got = gy.cpu()
    assert (got.view(torch.int16).numpy()[left] == CANARY).all()
    err = np.abs(got.double().numpy() - want_y)[~left]
    v = np.abs(want_y[~left])
    assert (err <= v * (2.0 ** -8 + 2.0 ** -20) + 2.0 ** -134).all()
    mag = np.zeros(pos.shape)
    for t, j in zip(*np.nonzero((pos >= 0) & (pos < rows))):
        mag[t, j] = np.abs(gd[t]) @ np.abs(yd[pos[t, j]])
    assert (np.abs(gw.cpu().double().numpy() - want_w) <= 2 * H * 2.0 ** -24 * mag).all()
    return gy, gw


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,k,spare,drop", [(1, 8, 1, 0, 0), (7, 64, 2, 3, 0.3), (130, 512, 10, 0, 0.1),
                                              (33, 1000, 3, 5, 0), (65, 2048, 10, 0, 0), (17, 2056, 8, 2, 0.5),
                                              (9, 4096, 2, 0, 0.2), (20, 7168, 8, 1, 0), (5, 20480, 4, 0, 0),
                                              (11, 256, 32, 0, 0.1), (6, 136, 17, 9, 1.0), (2, 65536, 2, 0, 0)])
def test_gradients(moe, T, H, k, spare, drop, dtype):
    print("[case]", T, H, k, spare, drop, dtype, flush=True)
    check(moe, *make(T, H, k, spare, drop, dtype, T + H + k))


def test_one_of_them(moe):
    """grad_y alone and grad_w alone equal the ones computed together, bit for bit."""
    g, y, pos, w = make(50, 1024, 6, 4, 0.2, torch.bfloat16, 3)
    gy, gw = check(moe, g, y, pos, w)
    d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    only_w = moe.moe_combine_backward(g.to(DEV), y.to(DEV), d(pos), None, need_y=False)
    assert only_w[0] is None and torch.equal(only_w[1], gw)
    buf = torch.full_like(gy.view(torch.int16), CANARY).view(torch.bfloat16)
    only_y = moe.moe_combine_backward(g.to(DEV), None, d(pos), d(w), grad_y=buf, need_w=False)
    assert only_y[1] is None and torch.equal(only_y[0].view(torch.int16), gy.view(torch.int16))


def test_positions_out_of_range(moe):
    """Positions past y_rows count as dropped; no row at all gives zero weights' gradients."""
    g, y, pos, w = make(40, 256, 4, 0, 0, torch.bfloat16, 5)
    check(moe, g, y[:100].contiguous(), pos, w)
    d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    gy, gw = moe.moe_combine_backward(g.to(DEV), y[:0].to(DEV), d(pos), d(w))
    assert gy.shape == (0, 256) and (gw == 0).all()


def test_is_the_combine_s_adjoint(moe):
    """<grad_out, combine(y, w)> = <grad_y, y> = <grad_w, w>: against the library's own forward pass. Float
    output: each inner product is off by the roundings of its terms, 2^-8 of |grad_y y| for the first pair."""
    g, y, pos, w = make(64, 512, 4, 0, 0.2, torch.float32, 8)
    d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    out = moe.moe_combine_reduce(y.to(DEV), d(pos), d(w), out_fp32=True).double().cpu()
    gy, gw = moe.moe_combine_backward(g.to(DEV), y.to(DEV), d(pos), d(w), grad_y=torch.zeros_like(y, device=DEV))
    lhs = float((g.double() * out).sum())
    terms = gy.double().cpu() * y.double()
    wterms = gw.double().cpu() * torch.from_numpy(w).double()
    size = float(terms.abs().sum())
    assert abs(float(wterms.sum()) - lhs) <= 1e-5 * size
    assert abs(float(terms.sum()) - lhs) <= 2.0 ** -8 * size


def test_stream_and_graph(moe):
    g, y, pos, w = (t if isinstance(t, torch.Tensor) else torch.from_numpy(t) for t in
                    make(30, 2048, 5, 0, 0.1, torch.bfloat16, 9))
    g, y, pos, w = g.to(DEV), y.to(DEV), pos.to(DEV), w.to(DEV)
    gy, gw = torch.zeros_like(y), torch.empty(30, 5, device=DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    moe.moe_combine_backward(g, y, pos, w, gy, gw, stream=side)
    side.synchronize()
    want = gy.clone(), gw.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_combine_backward(g, y, pos, w, gy, gw)
    for i in range(4):
        gw.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gy, want[0]) and torch.equal(gw, want[1])
        g.copy_(torch.randn(30, 2048, generator=torch.Generator().manual_seed(i)).bfloat16())
        want = tuple(t.clone() for t in moe.moe_combine_backward(g, y, pos, w, gy.clone(), gw.clone()))
        gw.zero_()
