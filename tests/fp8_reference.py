"""Plain numpy float64 forms of the norm, its gradient, FP8 rows and weights in
8 bits, with bounds on the errors of a float32 computation, for their tests."""

import numpy as np
import torch

from ops_reference import LIPSCHITZ, LOST, act, act_grad, act_grad_error, act_share, experts

U = 2.0 ** -24  # half a step of float32, relative


# ---------------------------------------------------------------- E4M3 and FP8 rows

def e4m3(codes):
    """Values of E4M3 bytes."""
    c = torch.from_numpy(np.ascontiguousarray(codes, np.uint8))
    return c.view(torch.float8_e4m3fn).double().numpy()


def to_e4m3(v):
    """Bytes of the E4M3 values nearest to float32 v, |v| < 464; NaN and infinities give the NaN code."""
    t = torch.from_numpy(np.ascontiguousarray(v, np.float32))
    return t.to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def row_bytes(H):
    return H + 128 * ((H + 4095) // 4096)


def exponent(a):
    """Smallest integer e >= -127 with a <= 448 * 2^e."""
    a = np.asarray(a, np.float64)
    m, x = np.frexp(a)  # 448 = 0.875 * 2^9
    e = np.where(m > 0.875, x - 8, x - 9)
    return np.maximum(np.where(a == 0, -127, e), -127)


def encode_rows(v):
    """FP8 rows (bytes) of float32 values."""
    n, H = v.shape
    b = np.asarray(v, np.float32).reshape(n, H // 32, 32)
    e = exponent(np.abs(b).max(2))
    out = np.zeros((n, row_bytes(H)), np.uint8)
    out[:, :H] = to_e4m3(np.ldexp(b, -e[:, :, None])).reshape(n, H)
    out[:, H:H + H // 32] = e + 127
    return out


def decode_rows(rows, H):
    n = rows.shape[0]
    p = np.exp2(rows[:, H:H + H // 32].astype(np.float64) - 127)
    return (e4m3(rows[:, :H]).reshape(n, H // 32, 32) * p[:, :, None]).reshape(n, H)


def assert_rows8(got, want, err, used, what, canary=0x5A):
    """FP8 rows of values that are `want` to within `err`: each scale the one that some maximum within the error
    asks for, each value off by no more than half a step of E4M3 (2^-4 of the value, 2^-10 of the scale where codes are
    subnormal), zero padding, rows from `used` on untouched."""
    g = got.cpu().numpy()
    H = want.shape[1]
    assert (g[used:] == canary).all(), f"{what}: rows behind the last expert's changed"
    g, v, e = g[:used], want[:used], err[:used] + 2.0 ** -150
    if not used:
        return
    assert (g[:, H + H // 32:] == 0).all(), f"{what}: padding"
    x = g[:, H:H + H // 32].astype(np.int64) - 127
    nb = (used, H // 32, 32)
    lo = np.maximum(np.abs(v) - e, 0).reshape(nb).max(2)
    hi = (np.abs(v) + e).reshape(nb).max(2)
    ok = (x >= exponent(lo)) & (x <= exponent(hi))
    assert ok.all(), f"{what}: {int((~ok).sum())} of {ok.size} scales, first {x[~ok][:4]} for {lo[~ok][:4]}"
    step = np.repeat(np.exp2(x - 10.0), 32, axis=1)
    d = np.abs(decode_rows(g, H) - v) - (e + np.maximum(2.0 ** -4 * (np.abs(v) + e), step))
    assert (d <= 0).all(), f"{what}: {int((d > 0).sum())} of {d.size} past the bound, worst by {d.max()}"


# ---------------------------------------------------------------- weights in 8 bits

def blocks(a):
    """Each block's (row, column) slices of a matrix, 128 x 128."""
    for i in range(0, a.shape[0], 128):
        for j in range(0, a.shape[1], 128):
            yield i // 128, j // 128, slice(i, i + 128), slice(j, j + 128)


def quantize(W):
    """(codes, scale) of a float32 matrix, as the definition's float32 operations give them."""
    W = np.asarray(W, np.float32)
    codes = np.empty(W.shape, np.uint8)
    scale = np.empty(((W.shape[0] + 127) // 128, (W.shape[1] + 127) // 128), np.float32)
    for i, j, r, c in blocks(W):
        b = W[r, c]
        top = np.float32(np.nanmax(np.abs(b))) if not np.isnan(b).all() else np.float32(0)
        s = np.float32(1) if top == 0 else max(top / np.float32(448), np.float32(2.0 ** -126))
        with np.errstate(invalid="ignore"):
            codes[r, c] = to_e4m3(b * (np.float32(1) / s))
        scale[i, j] = s
    return codes, scale


def decode_weights(codes, scale):
    """float64 values of [n, O, H] codes."""
    n, O, H = codes.shape
    s = np.repeat(np.repeat(scale.astype(np.float64), 128, 1), 128, 2)[:, :O, :H]
    return e4m3(codes) * s


# ---------------------------------------------------------------- the norm

def norm(t, w, eps):
    """(v, bound of its float32 error). A term of the sum of squares passes through at most 64 additions of its lane,
    6 of the wave and 16 of the row's waves, a rounding each; all are positive, so the sum is off by 86 U of itself and
    its root by 43 U. The quotient, eps, the root and the two products add a rounding or two each."""
    r = 1 / np.sqrt((t * t).mean(1, keepdims=True) + eps)
    v = t * r * w
    return v, 64 * U * np.abs(v)


def norm_backward(gy, t, w, eps, gt=None):
    """(grad_x, grad_weight, bounds). As above with up to 128 additions of a lane, 6 of a wave and 16 of a row's waves:
    150 roundings in the mean of g t, of the sum of its terms' sizes, 75 U in r; and T additions, in whatever order,
    of terms off by 80 U each for the weight."""
    r = 1 / np.sqrt((t * t).mean(1, keepdims=True) + eps)
    g = gy * w
    m, size = (g * t).mean(1, keepdims=True), np.abs(g * t).mean(1, keepdims=True)
    dx = r * (g - t * r * r * m)
    ex = U * (100 * np.abs(r * g) + 420 * np.abs(t) * r ** 3 * size)
    if gt is not None:
        dx = dx + gt
        ex = ex + 2 * U * np.abs(dx)
    terms = gy * t * r
    return dx, terms.sum(0), ex, (t.shape[0] + 90) * U * np.abs(terms).sum(0)


# ---------------------------------------------------------------- products of FP8 rows and 8-bit weights

# The matrix unit's sums. It adds the products of eight neighbouring k after aligning them to the largest exponent
# among them, and keeps their bits down to 2^-13 of that power of two (measured on gfx950 with one large and several
# small products: 2^3 beside 2^16 is added, 2^2 is dropped). So up to seven products of each eight lose less than 2^-13
# of it each, in all less than 2^-10 of the largest product; a code below E4M3's normal range (2^-6) may count with
# that range's exponent. The sixteen sums of eight are then added to far more than 24 bits, and rounded once.

def largest_of_eight(v, least):
    """The largest |v| of each eight of a row, at least `least` (the smallest normal value there)."""
    return np.maximum(np.abs(v), least).reshape(*v.shape[:-1], -1, 8).max(-1)


def rows_largest(rows, H):
    p = np.exp2(rows[:, H:H + H // 32].astype(np.float64) - 127)
    return largest_of_eight(decode_rows(rows, H), np.repeat(p, 32, 1) * 2.0 ** -6)


def weights_largest(codes, scale):
    n, O, H = codes.shape
    s = np.repeat(np.repeat(scale.astype(np.float64), 128, 1), 128, 2)[:, :O, :H]
    return largest_of_eight(decode_weights(codes, scale), s * 2.0 ** -6)


def _sums(x, xg, off, W, Wg):
    """Per expert with rows: (l, first row, end, products, error): the matrix unit's error above, and 2 K 2^-24 of the
    terms' sizes, which holds the roundings of each 128 values' sum, of its product with the weights' scale and of the
    sum of those."""
    for l, b, e in experts(off, x.shape[0]):
        if e > b:
            err = 2.0 ** -10 * (xg[b:e] @ Wg[l].T) + 2 * max(x.shape[1], 32) * U * (np.abs(x[b:e]) @ np.abs(W[l]).T)
            yield l, b, e, x[b:e] @ W[l].T, err


def product(x, xg, off, W, Wg, bias=None, residual=None, kind="none", gated=False):
    """(y, pre, ez, ey) as ops_reference.product, on decoded rows and weights [E_l, O, K]."""
    rows, wide = x.shape[0], W.shape[1]
    O = wide // 2 if gated else wide
    y, z = np.full((rows, O), np.nan), np.full((rows, wide), np.nan)
    ez, ey = np.zeros((rows, wide)), np.zeros((rows, O))
    for l, b, e, v, err in _sums(x, xg, off, W, Wg):
        if bias is not None:
            v = v + bias[l]
            err = err + U * (np.abs(v) + np.abs(bias[l]))
        z[b:e], ez[b:e] = v, err
        a = act(v[:, :O], kind)
        ea = LIPSCHITZ[kind] * err[:, :O] + act_share(v[:, :O], kind) * np.abs(a) + LOST * np.abs(v[:, :O])
        if gated:
            u, eu = v[:, O:], err[:, O:]
            ea = ea * (np.abs(u) + eu) + np.abs(a) * eu
            a = a * u
        ea = ea + 2 * U * np.abs(a)
        if residual is not None:
            a = a + residual[b:e]
            ea = ea + 2 * U * (np.abs(a) + np.abs(residual[b:e]))
        y[b:e], ey[b:e] = a, ea
    return y, z, ez, ey


def dgrad(gy, gg, off, Wt, Wg, pre=None, kind="none", gated=False):
    """(grad_x, error bound) as ops_reference.dgrad, with transposed weights [E_l, H, O]."""
    rows, H = gy.shape[0], Wt.shape[1]
    out, eo = (np.full((rows, 2 * H if gated else H), np.nan) for _ in range(2))
    for l, b, e, d, err in _sums(gy, gg, off, Wt, Wg):
        if pre is None:
            out[b:e], eo[b:e] = d, err
            continue
        g = pre[b:e, :H]
        f, df = act(g, kind), act_grad(g, kind)
        ed = err * np.abs(df) + (np.abs(d) + err) * act_grad_error(g, kind) + 2 * U * np.abs(d * df)
        if not gated:
            out[b:e], eo[b:e] = d * df, ed
            continue
        u = pre[b:e, H:]
        out[b:e, :H], eo[b:e, :H] = d * u * df, ed * np.abs(u) + 2 * U * np.abs(d * u * df)
        out[b:e, H:] = d * f
        eo[b:e, H:] = err * np.abs(f) + ((np.abs(d) + err) * act_share(g, kind) + 2 * U * np.abs(d)) * np.abs(f) \
            + (np.abs(d) + err) * LOST * np.abs(g)
    return out, eo
