"""The float64 forms behind the 8-bit layer's tests, on the CPU: the norm's
gradient against differences, FP8 rows against the C oracle, weights in 8 bits
against their definition."""

import numpy as np
import pytest

import fp8_reference as ref


@pytest.mark.parametrize("T,H", [(1, 1), (3, 8), (5, 40)])
def test_norm_gradient_by_differences(T, H):
    rng = np.random.default_rng(T + H)
    t, w, gy, gt = (rng.standard_normal(s) for s in ((T, H), H, (T, H), (T, H)))
    eps, d = 1e-2, 1e-6
    gx, gw, _, _ = ref.norm_backward(gy, t, w, eps, gt)

    def loss(t, w):
        return (ref.norm(t, w, eps)[0] * gy).sum() + (t * gt).sum()

    for i in np.ndindex(T, H):
        e = np.zeros((T, H))
        e[i] = d
        assert abs((loss(t + e, w) - loss(t - e, w)) / (2 * d) - gx[i]) < 1e-7
    for h in range(H):
        e = np.zeros(H)
        e[h] = d
        assert abs((loss(t, w + e) - loss(t, w - e)) / (2 * d) - gw[h]) < 1e-7


def test_rows_are_the_payloads(orc):
    """The oracle's FP8 rows of bf16 values, from an identity map."""
    rng = np.random.default_rng(3)
    H = 4128  # two slabs
    v = (rng.standard_normal((6, H)) * np.exp2(rng.integers(-30, 30, (6, 1)))).astype(np.float32)
    bits = (v.view(np.uint32) >> 16).astype(np.uint16)
    v = (bits.astype(np.uint32) << 16).view(np.float32)
    v[2, 32:96] = 0
    bits[2, 32:96] = 0
    rows = orc.dispatch_permute_fp8(bits, np.arange(6, dtype=np.int32).reshape(6, 1), 6)
    got = ref.encode_rows(v)
    assert (np.asarray(rows).reshape(6, -1) == got).all()
    assert ref.row_bytes(H) == got.shape[1]


def test_exponent():
    a = np.array([0.0, 448.0, np.nextafter(448.0, 500), 449.0, 896.0, 1.75 * 2.0 ** -119, 2.0 ** -149])
    assert ref.exponent(a).tolist() == [-127, 0, 1, 1, 1, -127, -127]


def test_weights():
    rng = np.random.default_rng(0)
    W = rng.standard_normal((160, 288)).astype(np.float32)
    W[128:, 256:] = 0
    codes, scale = ref.quantize(W)
    assert scale.shape == (2, 3) and scale[1, 2] == 1
    v = ref.decode_weights(codes[None], scale[None])[0]
    for i, j, r, c in ref.blocks(W):
        top = np.abs(W[r, c]).max()
        # half a step of E4M3, and the roundings of the scale and of the product
        assert (np.abs(v[r, c] - W[r, c]) <= np.maximum((2.0 ** -4 + 2.0 ** -21) * np.abs(W[r, c]), top / 448 * 2.0 ** -10)).all()
        assert top == 0 or np.abs(ref.e4m3(codes[r, c])).max() == 448
