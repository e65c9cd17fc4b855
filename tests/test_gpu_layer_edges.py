"""Edges of the layer's operators on the GPU against float64: scores that
cancel against their biases, logits of very large magnitude, NaN in saved
pre-activations, no kept row at all, weights past 2^31 elements.

Bars: ids equal; weights and gradients as derived beside each check, with
u = 2^-24, half a step of float32. Every test prints the case it runs before
touching the GPU.
"""

import numpy as np
import pytest
import torch

import ops_reference as ref
from test_gpu_product import assert_rows, bf16, canary, dn, up

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
LOWEST = {t: torch.finfo(t).min for t in (torch.float32, torch.bfloat16)}


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import combine_route_topk_amd
    return combine_route_topk_amd


def say(*a):
    print("[case]", *a, flush=True)


def same_ids(moe, l, b, k, G, M, kind, top2):
    """Ids equal to float64's, whose scores differ by more than 64 bits' rounding."""
    x = l.double().numpy()
    got = moe.moe_route_scored(l.to(DEV), torch.from_numpy(b).to(DEV), k, G, M, kind, True, top2)[0].cpu().numpy()
    want = ref.route(x, b, k, G, M, kind, True, top2)[0]
    bad = np.flatnonzero((got != want).any(1))
    assert not len(bad), f"{len(bad)} of {len(x)} rows differ; row {bad[0]}: {got[bad[0]]} against {want[bad[0]]}"


def rivals(E, k, kind, low, start, decoy, size):
    """Rows in which one expert's score cancels against its bias.

    Experts in front of it hold `low` logits, so that their scores are their
    biases with next to no error: k - 1 well above, then one at 0.001, with
    `decoy` another 7e-10 below it. The last expert of the group has a score
    of about 0.9 and a bias that leaves about 0.001 again, with the error of
    the 0.9. Its logit passes from row to row through consecutive float32
    values, which moves its exact score through 0.001 in steps of about 2e-8.
    Under softmax an expert far below by its bias shares the row with it.
    """
    l = np.full((64, E), low, np.float32)
    b = (-2.0 - 0.125 * (np.arange(E) // size)).astype(np.float32)  # later groups far apart, so that they are certain
    b[:k - 1] = 1.0 + 0.125 * np.arange(k - 1)
    s0 = np.float32(0.001)
    b[k - 1] = s0
    if decoy:
        b[k] = s0 - np.float32(7e-10)
    last = size - 1
    steps = np.arange(-32, 32).astype(np.int32) + np.float32(start).view(np.int32)
    l[:, last] = steps.view(np.float32)
    if kind == "softmax":
        l[:, last - 1], b[last - 1] = 0.0, -10.0
    p = ref.scores(l[32:33], kind)[0, last]
    b[last] = np.float32(float(s0) - p)
    return l, b


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,M", [(8, 1, 1, 1), (16, 3, 1, 1), (64, 8, 1, 1), (96, 2, 1, 1), (130, 4, 1, 1),
                                     (255, 3, 1, 1), (512, 10, 1, 1), (1000, 5, 1, 1), (64, 2, 8, 2), (510, 3, 5, 2)])
def test_score_that_cancels_behind_the_last_place(moe, E, k, G, M, kind):
    """The rival of the last place is not the one next to it in float32: two experts with hardly any error hold
    places k and k + 1, and the third, with an error far larger than the distance between those, is behind them."""
    for start in (1.3, 2.078628, 2.7):
        l, b = rivals(E, k, kind, -40.0, start, True, E // G)
        say(E, k, G, M, kind, start)
        s = np.sort(ref.scores(l, kind)[:, :E // G] + b[:E // G], 1)[:, -k - 2:]
        assert np.diff(s, axis=1).min() > 2.0 ** -48
        same_ids(moe, torch.from_numpy(l), b, k, G, M, kind, G > 1)


def large_rows(E, dtype):
    """Rows of large logits: one value throughout, two values, and values that differ by a few units."""
    v = [-1e10, -1e12, -1e30, LOWEST[dtype], 1e10, 1e12, 1e30, torch.finfo(dtype).max]
    l = torch.tensor(v).repeat(3, 1).t().reshape(-1, 1).repeat(1, E)
    l[1::3, :E // 2] = LOWEST[dtype]        # the other half, or all where that is the value
    l[2::3, E // 3:] = -torch.inf
    n = np.random.default_rng(E).integers(0, 8, (4, E))
    near = torch.from_numpy(n * 2.0 ** -4 + np.array([[2.0 ** 20], [-2.0 ** 20], [2.0 ** 19], [-2.0 ** 18]])).float()
    if dtype == torch.bfloat16:             # steps of 2 at 2^8
        near = torch.from_numpy(n * 2.0 + np.array([[2.0 ** 8], [-2.0 ** 9], [2.0 ** 8], [-2.0 ** 9]])).float()
    l = torch.cat([l, near]).to(dtype)
    assert torch.equal(l[-4:].float(), near)
    return l


def spread(x):
    """Largest |l - max of the row| among scores that do not vanish (exp(-110) is below half of float32's smallest)."""
    with np.errstate(invalid="ignore"):  # a row of -inf only
        d = x.max(1, keepdims=True) - x
    return np.where(d < 110, d, 0).max()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k,G,M", [(8, 2, 1, 1), (60, 4, 1, 1), (64, 8, 8, 4), (255, 7, 1, 1), (256, 8, 8, 4),
                                     (512, 10, 1, 1), (1000, 8, 10, 3)])
def test_softmax_of_large_logits(moe, E, k, G, M, dtype):
    """A softmax depends on differences of logits only, whatever their magnitude: 1 / E for a row of one value.

    Bar: an exponential is off by its argument's roundings, at most 2.5 A u for differences up to A, and 2 steps;
    the sum by that, E u and the additions; so |w - v| <= v (E + 8 A + 24) u."""
    l = large_rows(E, dtype)
    x = l.double().numpy()
    b = ((np.random.default_rng(E).permutation(E) - E / 2) * (0.5 / E / E)).astype(np.float32)
    for bias in (b, None):
        for normalize in (False, True):
            for top2 in ((False, True) if G > 1 else (False,)):
                say(E, k, G, M, dtype, bias is not None, normalize, top2)
                idx, w = moe.moe_route_scored(l.to(DEV), None if bias is None else torch.from_numpy(bias).to(DEV), k,
                                              G, M, "softmax", normalize, top2, 2.5)
                want, v = ref.route(x, bias, k, G, M, "softmax", normalize, top2, 2.5)
                bad = np.flatnonzero((idx.cpu().numpy() != want).any(1))
                assert not len(bad), f"rows {bad}: {idx[bad[0]].tolist()} against {want[bad[0]]}"
                err = np.abs(w.cpu().double().numpy() - v)
                assert (err <= np.abs(v) * (E + 8 * spread(x) + 24) * U + 2.0 ** -126).all(), err.max()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(8, 2), (60, 4), (256, 8), (383, 7), (512, 10), (1000, 5)])
def test_softmax_gradient_of_large_logits(moe, E, k, dtype):
    """The plain softmax's gradient on the same rows. Bar: a score off by (E + 8 A + 24) u of itself, in a product
    with a difference of gradients whose terms are at most max |g| each; bf16 adds half a step."""
    l = large_rows(E, dtype)
    x, rng = l.double().numpy(), np.random.default_rng(k)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(len(x))]).astype(np.int32)
    g = rng.standard_normal((len(x), k)).astype(np.float32)
    say(E, k, dtype)
    got = moe.moe_route_scored_backward(l.to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(g).to(DEV),
                                        "softmax", False, 2.5).cpu().double().numpy()
    want = ref.route_backward(x, idx, g, "softmax", False, 2.5)
    tol = 2.5 * 2 * np.abs(g).max(1, keepdims=True) * ref.scores(x, "softmax") * (E + 8 * spread(x) + 48) * U + 2.0 ** -126
    if dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) - tol).max()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(8, 2), (64, 4), (130, 1), (512, 6)])
def test_lowest_logit_beside_a_close_score(moe, E, k, kind, dtype):
    """An expert whose finite logit stands for a mask scores its bias exactly; another lies within float32's
    rounding of it, at the last place and inside the order."""
    for extra in (0, 1):  # the pair at places k and k + 1, or k - 1 and k
        if k + extra > E - 3:
            continue
        for i in range(12):
            l, b = rivals(E, k, kind, LOWEST[dtype], 1.3 + 0.125 * i, False, E)
            l = torch.from_numpy(l[32:33]).to(dtype)
            last = E - 1
            p = ref.scores(l.double().numpy(), kind)[0, last]
            b[last] = np.float32(0.001 - p)
            # what that bias leaves is a multiple of its own rounding, about 2^-25: set the other expert right beside
            exact = p + float(b[last])
            for d in (-2e-9, 2e-9):
                b[k - 1] = np.float32(exact + d)
                say(E, k, kind, dtype, extra, i, d)
                same_ids(moe, l, b, k + extra, 1, 1, kind, False)


@pytest.mark.parametrize("kind", ref.ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_nan_in_the_saved_pre_activations(moe, kind, gated):
    """A NaN in pre gives NaN in each gradient that depends on it, and changes nothing else."""
    rng = np.random.default_rng(11)
    off = torch.tensor([0, 70, 70, 300], dtype=torch.int32, device=DEV)
    H, wide = 152, 304 if gated else 152
    gy, W, z = bf16(rng, 300, 64), bf16(rng, 3, 64, H, scale=0.125), bf16(rng, 300, wide)
    at = np.zeros((300, wide), bool)
    at[rng.integers(0, 300, 50), rng.integers(0, wide, 50)] = True
    dirty = z.clone()
    dirty[torch.from_numpy(at)] = float("nan")
    say(kind, gated)
    clean, got = (moe.moe_expert_product_dgrad(up(gy), off, up(W), up(p), kind, gated).cpu() for p in (z, dirty))
    if not gated:
        want = at if kind != "none" else np.zeros_like(at)
    else:  # d u act'(g) depends on u, and on g but for the identity; d act(g) on g
        g, u = at[:, :H], at[:, H:]
        want = np.concatenate([u | g if kind != "none" else u, g], 1)
    assert (np.isnan(got.float().numpy()) == want).all()
    keep = torch.from_numpy(~want)
    assert torch.equal(got.view(torch.int16)[keep], clean.view(torch.int16)[keep])


def test_combine_gradient_without_rows(moe):
    """No replica was kept: an empty grad_y, alone or with the weights' gradients, which are 0."""
    g = torch.randn(6, 64, device=DEV).bfloat16()
    pos, w = torch.full((6, 2), -1, dtype=torch.int32, device=DEV), torch.ones(6, 2, device=DEV)
    y = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    for kw in (dict(y=y), dict(y=None, y_rows=0), dict(y=None, grad_y=torch.empty_like(y))):
        say(sorted(kw))
        gy, gw = moe.moe_combine_backward(g, pos=pos, topk_w=w, need_w=False, **kw)
        assert gy.shape == (0, 64) and gy.dtype == torch.bfloat16 and gw is None
    gy, gw = moe.moe_combine_backward(g, y, pos, w)
    assert gy.shape == (0, 64) and (gw == 0).all()
    gy, gw = moe.moe_combine_backward(g, y, pos, None, need_y=False)
    assert gy is None and (gw == 0).all()


def test_weights_past_32_bit_offsets(moe):
    """33 experts of 2^26 weights each; the last, behind 2^31 elements, holds values of its own and has all rows.
    Few rows take the kernel that reads W straight into fragments (at most 16 rows for each of the 33 experts on
    average, 2048 columns of x), more take the tiles; the input gradient reads W along its other axis."""
    El, O, H = 33, 32768, 2048
    rng = np.random.default_rng(12)
    W = torch.full((El, O, H), 0.5, dtype=torch.bfloat16, device=DEV)
    last = bf16(rng, 1, O, H, scale=H ** -0.5)
    W[-1] = last[0].to(DEV)
    V = dn(last)
    for rows in (20, 600):
        off = torch.zeros(El + 1, dtype=torch.int32, device=DEV)
        off[-1] = rows
        x, gy = bf16(rng, rows, H), bf16(rng, rows, O, scale=0.125)
        say(El, O, H, rows)
        for gated in (False, True):
            y = canary(rows, O // 2 if gated else O)
            moe.moe_expert_product(up(x), off, W, act="silu", gated=gated, y=y)
            wy, _, _, ey = ref.product(dn(x[:20]), [0, 20], V, None, None, "silu", gated)
            assert_rows(y[:20], wy, ey, 20, "y")
        g = canary(rows, H)
        moe.moe_expert_product_dgrad(up(gy), off, W, grad_x=g)
        assert_rows(g[:20], *ref.dgrad(dn(gy[:20]), [0, 20], V), 20, "grad_x")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,M", [(513, 10, 1, 1), (640, 32, 1, 1), (768, 8, 16, 3), (1000, 6, 8, 4), (1024, 9, 64, 5)])
def test_more_than_512_experts(moe, E, k, G, M, kind, dtype):
    """Wide rows have a kernel of their own: with and without a bias, masked rows, saturated logits in order. The
    weights' bar is that of test_softmax_of_large_logits, with A the largest |logit| for a sigmoid."""
    rng = np.random.default_rng(E + k)
    l = torch.from_numpy(rng.standard_normal((300, E)).astype(np.float32)).to(dtype)
    l[200:250] = torch.where(torch.from_numpy(rng.random((50, E)) < 0.97), torch.tensor(-torch.inf, dtype=dtype), l[200:250])
    l[250] = -torch.inf
    l[251:260] = torch.from_numpy(np.stack([rng.permutation(E) * 0.125 + 30 for _ in range(9)])).to(dtype)
    x = l.double().numpy()
    A = spread(x[:251]) if kind == "softmax" else np.abs(x[np.isfinite(x)]).max()
    b = (rng.permutation(E) * (0.2 / E / E)).astype(np.float32)
    for bias in (b, None):
        for normalize in (True, False):
            for top2 in ((False, True) if G > 1 else (False,)):
                say(E, k, G, M, kind, dtype, bias is not None, normalize, top2)
                rows = 260 if bias is None and not top2 else 251  # saturated scores are ordered by their logits
                idx, w = moe.moe_route_scored(l[:rows].to(DEV), None if bias is None else torch.from_numpy(bias).to(DEV),
                                              k, G, M, kind, normalize, top2, 2.5)
                want, v = ref.route(x[:rows], bias, k, G, M, kind, normalize, top2, 2.5)
                bad = np.flatnonzero((idx.cpu().numpy() != want).any(1))
                assert not len(bad), f"rows {bad}: {idx[bad[0]].tolist()} against {want[bad[0]]}"
                B = max(A, spread(x[251:])) if kind == "softmax" and rows == 260 else A
                err = np.abs(w.cpu().double().numpy() - v)
                assert (err <= np.abs(v) * (E + 8 * B + 24) * U + 2.0 ** -126).all(), err.max()


@pytest.mark.parametrize("rows", [3, 300])
def test_products_of_the_widest_rows(moe, rows):
    """H and O at their limit of 65536, one at a time, on both kernels of the product and in the gradients."""
    rng = np.random.default_rng(rows)
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    for H, O in ((65536, 16), (16, 65536)):
        x, gy = bf16(rng, rows, H), bf16(rng, rows, O)
        for gated in (False, True):
            W = bf16(rng, 1, 2 * O if gated else O, H, scale=H ** -0.5)
            say(rows, H, O, gated)
            y, z = canary(rows, O), canary(rows, 2 * O if gated else O)
            moe.moe_expert_product(up(x), off, up(W), act="silu", gated=gated, y=y, pre=z)
            wy, wz, ez, ey = ref.product(dn(x), [0, rows], dn(W), None, None, "silu", gated)
            assert_rows(y, wy, ey, rows, "y"), assert_rows(z, wz, ez, rows, "pre")
        V, p = bf16(rng, 1, O, H, scale=O ** -0.5), bf16(rng, rows, 2 * H)
        g = canary(rows, 2 * H)
        moe.moe_expert_product_dgrad(up(gy), off, up(V), up(p), "silu", True, g)
        assert_rows(g, *ref.dgrad(dn(gy), [0, rows], dn(V), dn(p), "silu", True), rows, "grad_x")
        gW, gb = torch.empty(1, O, H, device=DEV), torch.empty(1, O, device=DEV)
        moe.moe_expert_product_wgrad(up(gy), up(x), off, gW, gb)
        vW, vb, eW, eb = ref.wgrad(dn(gy), dn(x), [0, rows], 1)
        assert (np.abs(gW.cpu().double().numpy() - vW) <= eW + 2.0 ** -126).all()
        assert (np.abs(gb.cpu().double().numpy() - vb) <= eb + 2.0 ** -126).all()


@pytest.mark.parametrize("T,E,k", [(2 ** 22 + 3, 516, 4), (2 ** 24 + 9, 130, 2)])
def test_route_of_very_many_tokens(moe, T, E, k):
    """More than 2^31 logits, and more tokens than one launch takes: rows repeat, so their results do, bit for bit."""
    R = 1000
    base = torch.randn(R, E, generator=torch.Generator().manual_seed(E)).bfloat16().to(DEV)
    b = (torch.rand(E, generator=torch.Generator().manual_seed(k)) * 0.1).to(DEV)
    at = torch.arange(T, device=DEV) % R
    say(T, E, k)
    few = moe.moe_route_scored(base, b, k, scores="sigmoid")
    l = base[at]
    idx, w = moe.moe_route_scored(l, b, k, scores="sigmoid")
    assert torch.equal(idx, few[0][at]) and torch.equal(w, few[1][at])
    g = torch.randn(R, k, generator=torch.Generator().manual_seed(1)).to(DEV)
    want = moe.moe_route_scored_backward(base, few[0], g, "softmax", False)
    got = moe.moe_route_scored_backward(l, idx, g[at], "softmax", False)
    for t in range(0, T, 2 ** 20):  # in parts, so that no second copy of all of it is held
        assert torch.equal(got[t:t + 2 ** 20], want[at[t:t + 2 ** 20]])


def test_combine_gradient_of_very_many_tokens(moe):
    """More tokens than one launch takes, of one replica each."""
    T, H = 2 ** 24 + 5, 8
    gen = torch.Generator(device=DEV).manual_seed(0)
    g = torch.randn(T, H, generator=gen, device=DEV).bfloat16()
    y = torch.randn(T, H, generator=gen, device=DEV).bfloat16()
    w = torch.randn(T, 1, generator=gen, device=DEV)
    pos = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=DEV)[:, None]
    say(T, H)
    gy, gw = moe.moe_combine_backward(g, y, pos, w)
    # one product, rounded to float32 and to bf16; a sum of 8 exact products
    want = (w.double() * g.double()).flip(0)
    assert ((gy.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -20) + 2.0 ** -134).all()
    terms = g.double() * y.double().flip(0)
    assert ((gw[:, 0].double() - terms.sum(1)).abs() <= 16 * U * terms.abs().sum(1)).all()


def test_random_close_scores(moe):
    """Rows whose scores cancel against their biases to a common value within 1e-12 to 1e-4, deep, saturated and
    masked logits among them: ids equal wherever 64 bits tell the scores apart."""
    rng, rows = np.random.default_rng(17), 0
    for i in range(600):
        G = int(rng.choice([1, 1, 1, 2, 4, 8]))
        size = int(rng.integers(max(2, 8 // G), 600 // G + 1))
        E, M = G * size, int(rng.integers(1, G + 1))
        k = int(rng.integers(1, min(12, M * size) + 1))
        kind, top2 = ("softmax", "sigmoid")[int(rng.integers(2))], G > 1 and bool(rng.integers(2))
        x, at = rng.standard_normal(E) * rng.choice([0.3, 1, 4]), rng.random(E)
        pool = int(rng.integers(5))
        x = np.where((pool in (1, 2)) & (at < 0.4), -40 + rng.standard_normal(E), x)
        x = np.where((pool in (2, 3)) & (at > 0.7), LOWEST[torch.float32], x)
        x = np.where((pool == 4) & (at < 0.5), rng.uniform(5, 25, E), x).astype(np.float32)
        l, j = x[None].repeat(32, 0), rng.integers(0, E, (32, 3))
        near = (np.take_along_axis(l, j, 1).view(np.int32) + rng.integers(-40, 40, (32, 3))).astype(np.int32).view(np.float32)
        np.put_along_axis(l, j, np.where(np.isfinite(near), near, np.take_along_axis(l, j, 1)), 1)
        target, scale = rng.choice([0.0, 0.001, 0.75, 40.0, -3.0]), 10.0 ** rng.uniform(-12, -4)
        b = (target - ref.scores(x[None], kind)[0] + scale * rng.permutation(E)).astype(np.float32)
        b[rng.random(E) < rng.choice([0, 0.5, 0.9])] = -5 - target
        s = ref.scores(l, kind) + b.astype(np.float64)
        sure = np.full(32, np.inf)  # the smallest distance that decides
        if M < G:
            by = -np.sort(-s.reshape(32, G, size), 2)
            group = by[:, :, :2].sum(2) if top2 else by[:, :, 0]
            order = np.argsort(-group, 1, kind="stable")
            sure = np.take_along_axis(group, order[:, M - 1:M + 1], 1)
            sure = sure[:, 0] - sure[:, 1]
            left = np.ones((32, G), bool)
            np.put_along_axis(left, order[:, :M], False, 1)
            s = np.where(left.repeat(size, 1), -np.inf, s)
        want = np.argsort(-s, 1, kind="stable")
        v = np.take_along_axis(s, want[:, :k + 1], 1)
        if v.shape[1] > 1:
            sure = np.minimum(sure, (v[:, :-1] - v[:, 1:]).min(1))
        sure = sure > 2.0 ** -46 * max(1, abs(target))
        say(i, E, k, G, M, kind, top2, pool, target, scale)
        got = moe.moe_route_scored(torch.from_numpy(l).to(DEV), torch.from_numpy(b).to(DEV), k, G, M, kind, True, top2)[0]
        bad = np.flatnonzero((got.cpu().numpy() != want[:, :k]).any(1) & sure)
        assert not len(bad), f"{len(bad)} rows; row {bad[0]}: {got[bad[0]].tolist()} against {want[bad[0], :k]}"
        rows += int(sure.sum())
    assert rows > 10000  # 19200, less those too close even for 64 bits


def test_sigmoid_weights_keep_their_ratios_far_below_range(moe):
    """Normalised sigmoid weights of scores that vanish in float32 are the exact ones: exp(l) up to a factor."""
    d = torch.arange(8) * 0.5
    l = torch.stack([-200 - d, -1e4 - d, torch.full((8,), -1e10), torch.full((8,), LOWEST[torch.float32])]).float()
    say("ratios")
    idx, w = moe.moe_route_scored(l.to(DEV), None, 4, scores="sigmoid")
    want = np.exp(-0.5 * np.arange(4))
    want = np.stack([want / want.sum()] * 2 + [np.full(4, 0.25)] * 2)
    assert idx.tolist() == [[0, 1, 2, 3]] * 4
    assert (np.abs(w.cpu().double().numpy() - want) <= want * (8 + 8 * 1.5 + 24) * U).all()


@pytest.mark.parametrize("E", [8, 600])
def test_nan_logits_and_biases(moe, E):
    """A NaN logit or bias ranks its expert last under sigmoid, below masked ones; under softmax a NaN or infinite
    logit leaves ids distinct and in range."""
    rng = np.random.default_rng(E)
    l = rng.standard_normal((12, E)).astype(np.float32)
    l[1, ::2], l[2], l[3, 1:], l[4, 3] = np.nan, np.nan, -np.inf, np.inf
    l[5, : E - 2], l[5, E - 2:] = np.nan, -np.inf
    b = (rng.permutation(E) * (0.2 / E / E)).astype(np.float32)
    for bias in (None, b, np.where(np.arange(E) % 3 == 0, np.nan, b).astype(np.float32)):
        for G, M, top2 in ((1, 1, False), (4, 3, True), (4, 2, False)):
            k = 3
            say(E, bias is not None and np.isnan(bias).any(), G, M, top2)
            B = None if bias is None else torch.from_numpy(bias).to(DEV)
            idx = moe.moe_route_scored(torch.from_numpy(l).to(DEV), B, k, G, M, "sigmoid", True, top2)[0].cpu().numpy()
            if G == 1:  # a group's sum with a NaN in it has no order of its own
                assert (idx == ref.route(l.astype(np.float64), bias, k, G, M, "sigmoid", True, top2)[0]).all()
            soft = moe.moe_route_scored(torch.from_numpy(l).to(DEV), B, k, G, M, "softmax", True, top2)[0].cpu().numpy()
            for ids in (idx, soft):
                assert all(len(set(r)) == k and min(r) >= 0 and max(r) < E for r in ids.tolist())
