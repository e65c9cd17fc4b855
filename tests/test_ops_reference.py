"""The float64 references of the router's, combine's and products' gradients,
against central differences of their forward forms (CPU only).

A central difference with step h of a smooth f in float64 is off by at most
h^2 |f'''| / 6 + 2^-52 |f| / h; with h = 1e-5, values and third derivatives of
at most 1e3 here, both terms stay below 1e-6.
"""

import numpy as np
import pytest

import ops_reference as ref

STEP, TOL = 1e-5, 1e-6


def differences(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        v = x[i]
        x[i] = v + STEP
        hi = f(x)
        x[i] = v - STEP
        lo = f(x)
        x[i] = v
        g[i] = (hi - lo) / (2 * STEP)
    return g


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_gradient(kind, normalize):
    rng = np.random.default_rng(1)
    l = rng.standard_normal((3, 12))
    idx, w = ref.route(l, rng.standard_normal(12) * 0.1, 4, kind=kind, normalize=normalize, scale=2.5)
    assert np.allclose(w, ref.weights(l, idx, kind, normalize, 2.5), rtol=1e-12, atol=0)
    g = rng.standard_normal((3, 4))
    got = ref.route_backward(l, idx, g, kind, normalize, 2.5)
    want = differences(lambda v: (ref.weights(v, idx, kind, normalize, 2.5) * g).sum(), l)
    assert np.abs(got - want).max() < TOL


@pytest.mark.parametrize("kind", ref.ACTS)
def test_activation_gradient(kind):
    z = np.linspace(-6, 6, 41) + 0.013  # no point at ReLU's corner
    want = differences(lambda v: ref.act(v, kind).sum(), z.copy())
    assert np.abs(ref.act_grad(z, kind) - want).max() < TOL
    assert np.abs(ref.act_grad(np.linspace(-8, 8, 100001), kind)).max() <= ref.LIPSCHITZ[kind]


@pytest.mark.parametrize("kind,gated", [("none", False), ("silu", True), ("gelu", True), ("gelu_tanh", False)])
def test_layer_gradients(kind, gated):
    """Two products in a row: the second's input gradient through the first's activation, and every weight's."""
    rng = np.random.default_rng(2)
    off, H, I = [0, 2, 2, 5], 6, 4
    x, r = rng.standard_normal((5, H)), rng.standard_normal((5, H))
    W1 = rng.standard_normal((3, 2 * I if gated else I, H))
    b1 = rng.standard_normal(W1.shape[:2])
    W2 = rng.standard_normal((3, H, I))
    g = rng.standard_normal((5, H))

    def forward(x, W1, b1, W2):
        h, z, _, _ = ref.product(x, off, W1, b1, None, kind, gated)
        return h, z, ref.product(h, off, W2, None, r)[0]

    h, z, _ = forward(x, W1, b1, W2)
    dz, _ = ref.dgrad(g, off, W2, z, kind, gated)
    dx, _ = ref.dgrad(dz, off, W1)
    dW1, db1, _, _ = ref.wgrad(dz, x, off, 3)
    dW2, _, _, _ = ref.wgrad(g, h, off, 3)
    for got, f, at in ((dx, lambda v: (forward(v, W1, b1, W2)[2] * g).sum(), x),
                       (dW1, lambda v: (forward(x, v, b1, W2)[2] * g).sum(), W1),
                       (db1, lambda v: (forward(x, W1, v, W2)[2] * g).sum(), b1),
                       (dW2, lambda v: (forward(x, W1, b1, v)[2] * g).sum(), W2)):
        assert np.abs(got - differences(f, at.copy())).max() < TOL


def test_combine_gradient():
    rng = np.random.default_rng(3)
    pos = np.array([[2, 0], [-1, 3], [1, -1]])
    w, y, g = rng.standard_normal((3, 2)), rng.standard_normal((5, 4)), rng.standard_normal((3, 4))

    def forward(w, y):
        return sum((w[t, j] * y[pos[t, j]] * g[t]).sum() for t in range(3) for j in range(2) if pos[t, j] >= 0)

    gy, gw = ref.combine_backward(g, y, pos, w)
    assert np.isnan(gy[4]).all()
    assert np.abs(gw - differences(lambda v: forward(v, y), w.copy())).max() < TOL
    assert np.abs(np.nan_to_num(gy) - differences(lambda v: forward(w, v), y.copy())).max() < TOL


def test_route_masks():
    """A masked expert is taken last, whatever its bias, and weighs nothing."""
    l = np.full((2, 4), -np.inf)
    l[0, 2] = -3.0
    idx, w = ref.route(l, np.array([9.0, 0, 0, 0]), 2, kind="sigmoid")
    assert idx.tolist() == [[2, 0], [0, 1]] and w.tolist() == [[1.0, 0.0], [0.0, 0.0]]
