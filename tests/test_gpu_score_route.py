"""Scored routing and its gradient on the GPU against float64.

Bars, with u = 2^-24 (half a step of float32):
  * ids: equal. Inputs are random, or tie exactly, so no two different scores
    lie within 64-bit resolution of each other.
  * weights: an exponential is off by its argument's rounding, |x| u, and 2
    steps; a sum over n terms by n u at most; the quotients, products and
    the scale by a few u. For logits of at most A in magnitude:
    |w - v| <= v (E + 4 A + 24) u (softmax over all E; k in the place of E
    when normalised, E covers it), plus the smallest normal number.
  * logit gradients: each is a product of such factors and a difference
    g_j - sum, off by the same share of sum |g w| + |g_j|; bf16 adds half a
    step, 2^-8 of the value.
Every test prints the case it runs before touching the GPU.
"""

import numpy as np
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import combine_route_topk_amd
    return combine_route_topk_amd


def say(*a):
    print("[case]", *a, flush=True)


def make(T, E, dtype, seed, bias="uniform", width=0.1):
    rng = np.random.default_rng(seed)
    l = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(dtype)
    b = None
    if bias == "uniform":
        b = (rng.uniform(-width, width, E)).astype(np.float32)
    elif bias == "zeros":
        b = np.zeros(E, np.float32)
    return l, b


def check(moe, l, b, k, G=1, M=1, kind="softmax", normalize=True, top2=False, scale=1.0, weights=True):
    idx, w = moe.moe_route_scored(l.to(DEV), None if b is None else torch.from_numpy(b).to(DEV), k, G, M, kind,
                                  normalize, top2, scale)
    x = l.double().numpy()
    want, v = ref.route(x, b, k, G, M, kind, normalize, top2, scale)
    got = idx.cpu().numpy()
    bad = np.flatnonzero((got != want).any(1))
    assert not len(bad), f"{len(bad)} rows' ids differ; row {bad[0]}: {got[bad[0]]} against {want[bad[0]]}"
    if weights:
        live = x[np.isfinite(x)]
        A = np.abs(live).max() if live.size else 0.0
        err = np.abs(w.cpu().double().numpy() - v)
        assert (err <= np.abs(v) * (x.shape[1] + 4 * A + 24) * U + 2.0 ** -126).all(), err.max()
    return idx, w


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 3, 2), (33, 16, 4), (257, 60, 6), (130, 64, 8), (67, 96, 32),
                                   (300, 128, 8), (129, 255, 7), (260, 256, 8), (97, 384, 8), (130, 510, 10),
                                   (301, 512, 10), (40, 770, 12), (31, 1000, 32), (65, 1024, 9)])
def test_route(moe, T, E, k, kind, dtype):
    for bias, normalize, scale in (("uniform", True, 1.0), (None, False, 2.5), ("zeros", True, -0.5)):
        say(T, E, k, kind, dtype, bias, normalize, scale)
        l, b = make(T, E, dtype, 7 * E + k, bias, 0.1 if kind == "sigmoid" else 0.5 / E)
        check(moe, l, b, k, kind=kind, normalize=normalize, scale=scale)


@pytest.mark.parametrize("top2", [True, False])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,G,M", [(65, 16, 4, 4, 2), (130, 64, 6, 8, 3), (9, 64, 1, 64, 1), (70, 64, 8, 64, 8),
                                       (129, 256, 8, 8, 4), (66, 384, 8, 16, 4), (33, 512, 10, 32, 7),
                                       (35, 120, 5, 5, 2), (64, 1024, 32, 64, 2), (50, 512, 3, 2, 1),
                                       (21, 1000, 4, 8, 1)])
def test_route_groups(moe, T, E, k, G, M, kind, top2):
    for dtype, bias in ((torch.float32, "uniform"), (torch.bfloat16, None), (torch.bfloat16, "uniform")):
        say(T, E, k, G, M, kind, top2, dtype, bias)
        l, b = make(T, E, dtype, E + G, bias, 0.1 if kind == "sigmoid" else 0.5 / E)
        check(moe, l, b, k, G, M, kind, True, top2, 2.5)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,M", [(64, 8, 1, 1), (256, 8, 8, 4), (512, 10, 1, 1), (96, 5, 6, 2), (1024, 16, 32, 4)])
def test_close_scores(moe, E, k, G, M, kind):
    """Biases that bring the experts' scores within float32 rounding of each other, but not of 64 bits: score
    plus bias is a common value plus a multiple of 2^-34, in an order of their own."""
    rng = np.random.default_rng(E + k)
    T = 40
    for spread in (2.0 ** -34, 2.0 ** -27, 2.0 ** -22):
        # one row of logits for all tokens, so that one bias serves them; each token permutes nothing but its own few
        l = rng.standard_normal((1, E)).astype(np.float32).repeat(T, 0)
        p = ref.scores(l[:1], kind)[0]
        b = (0.75 - p + spread * rng.permutation(E)).astype(np.float32)
        # float32 biases round by up to 2^-25: what they leave is the order to find
        l[1:, :4] += rng.standard_normal((T - 1, 4)).astype(np.float32) * 1e-6
        say(E, k, G, M, kind, spread)
        s = np.sort(ref.scores(l, kind) + b, 1)
        assert np.diff(s, axis=1).min() > 2.0 ** -50  # distinct to 64 bits
        check(moe, torch.from_numpy(l), b, k, G, M, kind, True, G > 1)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,M", [(64, 8, 4), (256, 8, 3), (96, 6, 2), (24, 4, 2)])
def test_group_sums_that_cancel(moe, E, G, M, kind):
    """Groups ranked by two scores that nearly cancel (biases of +-40): the sums lie closer than the terms'
    float32 rounding, 2^-19."""
    rng = np.random.default_rng(E)
    l = rng.standard_normal((1, E)).astype(np.float32)
    p, size = ref.scores(l, kind)[0], E // G
    b = np.full(E, -100.0, np.float32)
    first, second = np.arange(G) * size, np.arange(G) * size + 1
    b[second] = -40.0
    b[first] = (40.75 - p[first] - p[second]).astype(np.float32)
    l = l.repeat(50, 0)
    l[1:, first] += rng.standard_normal((49, G)).astype(np.float32) * 1e-5
    say(E, G, M, kind)
    check(moe, torch.from_numpy(l), b, 2, G, M, kind, True, True)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,M", [(64, 1, 1), (256, 8, 4), (510, 1, 1), (768, 16, 3)])
def test_ties(moe, E, G, M, kind):
    """Few distinct logits and equal biases: exact ties go to the lower id and the lower group."""
    rng = np.random.default_rng(E)
    for levels in (1, 2, 5):
        l = torch.from_numpy(rng.integers(0, levels, (60, E)).astype(np.float32))
        for b in (None, np.zeros(E, np.float32), np.full(E, 0.25, np.float32)):
            say(E, G, M, kind, levels, None if b is None else b[0])
            check(moe, l, b, 8, G, M, kind, True, G > 1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,M", [(16, 4, 1, 1), (64, 8, 8, 4), (256, 8, 8, 4), (384, 6, 1, 1), (1000, 8, 10, 3)])
def test_masked(moe, E, k, G, M, kind, dtype):
    """-inf masks most experts, all experts, or all but one; large biases do not bring them back."""
    rng = np.random.default_rng(5)
    l, b = make(48, E, dtype, 3, "uniform", 0.1)
    b[rng.permutation(E)[:E // 3]] = 50.0
    l[:, :] = torch.where(torch.from_numpy(rng.random((48, E)) < 0.9), torch.tensor(-torch.inf, dtype=dtype), l)
    l[0], l[1, 1:], l[2, :-1] = -torch.inf, -torch.inf, -torch.inf
    say(E, k, G, M, kind, dtype)
    for normalize in (True, False):
        for top2 in (False, G > 1):
            idx, w = check(moe, l, b, k, G, M, kind, normalize, top2)
            assert (w[0] == 0).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_extreme_logits(moe, kind):
    """Logits that saturate: the type's lowest value in place of a mask, +-90, and rows of them only."""
    l = torch.zeros(6, 64)
    l[0, 5:] = torch.finfo(torch.float32).min
    l[1] = torch.linspace(-90, 90, 64)
    l[2] = torch.linspace(-100, -80, 64)
    l[3] = torch.linspace(60, 80, 64)
    l[4, ::2] = -700.0
    l[5] = torch.linspace(-3, 3, 64)
    say(kind)
    idx, w = check(moe, l[[0, 4, 5]], None, 4, kind=kind)
    idx, w = check(moe, l[[1, 2]], None, 4, kind=kind)
    w = moe.moe_route_scored(l[3:4].to(DEV), None, 4, scores=kind)[1]
    assert torch.isfinite(w).all() and abs(float(w.sum()) - 1) < 1e-5


@pytest.mark.parametrize("E,k,G,M", [(64, 8, 8, 4), (512, 10, 16, 4), (96, 6, 6, 2)])
def test_saturated_groups(moe, E, k, G, M):
    """Logits whose sigmoids are all 1: groups tie, experts go by their logits; then one infinite logit, whose
    score of exactly 1 is above a saturated one by less than float32 shows."""
    rng = np.random.default_rng(E)
    l = np.stack([rng.permutation(np.linspace(40, 80, E)) for _ in range(20)]).astype(np.float32)
    say(E, k, G, M)
    check(moe, torch.from_numpy(l), None, k, G, M, "sigmoid", True, True)
    x = np.full((3, E), -5.0, np.float32)
    x[0, 3], x[1, 3], x[2, 1] = 25.0, 25.0, np.inf
    x[0, 7], x[1, 1], x[2, 3] = np.inf, np.inf, 30.0
    idx = moe.moe_route_scored(torch.from_numpy(x).to(DEV), torch.zeros(E, device=DEV), 2, scores="sigmoid")[0]
    assert idx[:, 0].tolist() == [7, 1, 1] and idx[:, 1].tolist() == [3, 3, 3]


def test_nan_and_infinite(moe):
    """NaN ranks last under sigmoid; under softmax ids stay distinct and in range."""
    l = torch.randn(20, 64, generator=torch.Generator().manual_seed(1))
    l[3, 10], l[4, :], l[5, 7] = float("nan"), float("nan"), float("inf")
    say("nan")
    x = l.double().numpy()
    idx = moe.moe_route_scored(l.to(DEV), None, 8, scores="sigmoid")[0].cpu().numpy()
    assert (idx[:3] == ref.route(x[:3], None, 8, kind="sigmoid")[0]).all()
    assert 10 not in idx[3] and idx[4].tolist() == list(range(8)) and idx[5, 0] == 7
    for G, M, top2 in ((1, 1, False), (8, 2, True)):
        for b in (None, torch.linspace(-1, 1, 64).to(DEV)):
            idx = moe.moe_route_scored(l.to(DEV), b, 8, G, M, group_top2=top2)[0].cpu().numpy()
            assert all(len(set(r)) == 8 and min(r) >= 0 and max(r) < 64 for r in idx.tolist())


def test_unaligned_rows(moe):
    """Logits, bias and outputs at element alignment only."""
    for dtype in (torch.float32, torch.bfloat16):
        l, b = make(37, 256, dtype, 9)
        buf = torch.empty(37 * 256 + 1, dtype=dtype, device=DEV)
        v = buf[1:].view(37, 256)
        v.copy_(l)
        bb = torch.empty(257, device=DEV)
        bb[1:].copy_(torch.from_numpy(b))
        say(dtype)
        i0, w0 = check(moe, l, b, 8, kind="sigmoid")
        i1, w1 = moe.moe_route_scored(v, bb[1:], 8, scores="sigmoid")
        assert torch.equal(i0, i1)
        assert ((w0 - w1).abs() <= w0.abs() * 300 * U).all()
        g = torch.randn(37, 8, device=DEV)
        out = torch.empty_like(buf)[1:].view(37, 256)
        a = moe.moe_route_scored_backward(v, i0, g, "softmax", False, grad_logits=out)
        c = moe.moe_route_scored_backward(l.to(DEV), i0, g, "softmax", False)
        assert torch.allclose(a.float(), c.float(), rtol=2.0 ** -7, atol=1e-9)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 5), (65, 60, 4), (130, 64, 32), (77, 256, 8), (33, 383, 7),
                                   (129, 512, 10), (5, 1000, 3), (19, 1024, 16)])
def test_backward(moe, T, E, k, normalize, kind, dtype):
    say(T, E, k, normalize, kind, dtype)
    l, _ = make(T, E, dtype, E + 1)
    if E > 8 and T > 2:
        l[1, 2:] = -torch.inf          # masked: their gradient is 0
        l[2] = -torch.inf
    rng = np.random.default_rng(k)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    g = rng.standard_normal((T, k)).astype(np.float32)
    got = moe.moe_route_scored_backward(l.to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(g).to(DEV), kind,
                                        normalize, 2.5)
    assert got.dtype == dtype
    x = l.double().numpy()
    want = ref.route_backward(x, idx, g, kind, normalize, 2.5)
    # magnitudes of the terms: |g| in the place of g, sums in the place of differences
    size = 2.5 * (np.abs(g).max(1, keepdims=True) * 2) * np.ones((T, E))
    p = ref.scores(x, kind)
    if normalize:
        q = np.take_along_axis(p, idx.astype(np.int64), 1)
        s = q.sum(1, keepdims=True)
        p = np.divide(p, s, out=np.zeros_like(p), where=s > 0)
        p = np.minimum(p, 1.0)
    live = x[np.isfinite(x)]
    A = np.abs(live).max() if live.size else 0.0
    tol = size * p * (E + 8 * A + 48) * U + 2.0 ** -126
    if dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    err = np.abs(got.cpu().double().numpy() - want)
    assert (err <= tol).all(), (err - tol).max()
    chosen = np.zeros((T, E), bool)
    np.put_along_axis(chosen, idx.astype(np.int64), True, 1)
    if kind == "sigmoid" or normalize:
        assert (got.cpu().numpy() if dtype == torch.float32 else got.cpu().float().numpy())[~chosen].any() == False  # noqa: E712


def test_backward_ids_out_of_range(moe):
    """Ids outside [0, E) are left out of the sums."""
    l, _ = make(9, 64, torch.float32, 2)
    rng = np.random.default_rng(4)
    idx = np.stack([rng.permutation(64)[:6] for _ in range(9)]).astype(np.int32)
    idx[2, 1], idx[3, 0], idx[4, :] = -1, 64, 2 ** 31 - 1
    g = rng.standard_normal((9, 6)).astype(np.float32)
    for kind in ("softmax", "sigmoid"):
        for normalize in (True, False):
            say(kind, normalize)
            got = moe.moe_route_scored_backward(l.to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(g).to(DEV),
                                                kind, normalize)
            want = ref.route_backward(l.double().numpy(), idx, g, kind, normalize)
            assert np.abs(got.cpu().double().numpy() - want).max() < 1e-5 * np.abs(g).max()


def test_stream_and_graph(moe):
    """On another stream, and captured once and replayed on new logits."""
    l, b = make(64, 256, torch.float32, 21)
    ld, bd = l.to(DEV), torch.from_numpy(b).to(DEV)
    idx = torch.empty(64, 8, dtype=torch.int32, device=DEV)
    w, g = torch.empty(64, 8, device=DEV), torch.randn(64, 8, device=DEV)
    gl = torch.empty(64, 256, device=DEV)

    def step(stream=None):
        moe.moe_route_scored(ld, bd, 8, 8, 4, "sigmoid", group_top2=True, topk_idx=idx, topk_w=w, stream=stream)
        moe.moe_route_scored_backward(ld, idx, g, "sigmoid", grad_logits=gl, stream=stream)

    say("stream")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    first = idx.clone(), w.clone(), gl.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, (idx, w, gl)))
        ld.copy_(torch.randn(64, 256, generator=torch.Generator().manual_seed(i)))
        step()
        torch.cuda.synchronize()
        first = idx.clone(), w.clone(), gl.clone()
        idx.zero_(), w.zero_(), gl.fill_(7.0)
