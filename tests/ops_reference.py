"""Plain numpy float64 forms of the scored router, the combine's gradient and
the experts' products with their gradients, for the tests of those calls."""

import math

import numpy as np

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")

# largest slope of each activation (GELU's 1.13 at sqrt(2), SiLU's 1.10)
LIPSCHITZ = {"none": 1.0, "relu": 1.0, "silu": 1.11, "gelu": 1.13, "gelu_tanh": 1.14}


def sigmoid(z):
    z = np.asarray(z, np.float64)
    with np.errstate(over="ignore"):
        return np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))


def scores(logits, kind):
    """p of every logit; -inf gives 0."""
    l = np.asarray(logits, np.float64)
    if kind == "sigmoid":
        return sigmoid(l)
    m = l.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(l == -np.inf, 0.0, np.exp(l - np.where(np.isfinite(m), m, 0.0)))
    total = e.sum(1, keepdims=True)
    return np.divide(e, total, out=np.zeros_like(e), where=total > 0)


def descending(s):
    """Positions of a row's scores from best to worst, ties to the lower, NaN last."""
    return sorted(range(len(s)), key=lambda e: (math.isnan(s[e]), -s[e] if not math.isnan(s[e]) else 0.0, e))


def route(logits, bias, k, n_groups=1, topk_groups=1, kind="softmax", normalize=True, top2=False, scale=1.0):
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    p = scores(l, kind)
    s = np.where(l == -np.inf, -np.inf, p + (0.0 if bias is None else np.asarray(bias, np.float64)))
    # both scores rise strictly with the logit, but not in 64 bits (sigmoid(40) and sigmoid(41) are both 1 there):
    # without a bias the logit's order is the exact one
    by = l if bias is None else s
    size = E // n_groups
    idx = np.empty((T, k), np.int32)
    for t in range(T):
        live = range(E)
        if topk_groups < n_groups:
            g = []
            for q in range(n_groups):
                part = (s if top2 and size > 1 else by)[t, q * size:(q + 1) * size]
                best = [part[i] for i in descending(part)]
                g.append(best[0] + best[1] if top2 and size > 1 else best[0])
            chosen = set(descending(g)[:topk_groups])
            live = [e for e in range(E) if e // size in chosen]
        order = descending([by[t, e] for e in live])
        idx[t] = [live[i] for i in order[:k]]
    w = np.take_along_axis(p, idx.astype(np.int64), 1)
    if normalize:
        if kind == "softmax":  # the same ratio, without the underflow of far smaller scores
            ls = np.take_along_axis(l, idx.astype(np.int64), 1)
            w = scores(ls, "softmax")
        else:
            total = w.sum(1, keepdims=True)
            w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return idx, w * scale


def weights(l, idx, kind, normalize, scale):
    """The weights as a function of the logits, ids held fixed."""
    p = scores(l, kind)
    w = np.take_along_axis(p, idx.astype(np.int64), 1)
    if normalize:
        w = w / w.sum(1, keepdims=True)
    return scale * w


def route_backward(logits, idx, grad_w, kind="softmax", normalize=True, scale=1.0):
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    out = np.zeros((T, E))
    p = scores(l, kind)
    for t in range(T):
        ok = (idx[t] >= 0) & (idx[t] < E)
        ids, g = idx[t][ok], np.asarray(grad_w[t], np.float64)[ok]
        q = p[t, ids]
        if normalize:
            if kind == "softmax":
                w = scores(l[t:t + 1, ids], "softmax")[0] if len(ids) else q
            else:
                w = q / q.sum() if q.sum() > 0 else np.zeros_like(q)
            d = scale * w * (g - (g * w).sum())
            out[t, ids] = d * (1 - q) if kind == "sigmoid" else d
        elif kind == "sigmoid":
            out[t, ids] = scale * g * q * (1 - q)
        else:
            dense = np.zeros(E)
            dense[ids] = g
            out[t] = scale * p[t] * (dense - (g * q).sum())
    return out


def combine_backward(grad_out, y, pos, w):
    """(grad_y rows by position, grad_w): rows nothing points at are NaN."""
    T, k = pos.shape
    gy = np.full(y.shape, np.nan)
    gw = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            q = pos[t, j]
            if 0 <= q < y.shape[0]:
                gy[q] = w[t, j] * grad_out[t]
                gw[t, j] = grad_out[t] @ y[q]
    return gy, gw


_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act(z, kind):
    if kind == "relu":
        return np.where(z > 0, z, 0.0)
    if kind == "silu":
        return z * sigmoid(z)
    if kind == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2))
    if kind == "gelu_tanh":  # (1 + tanh u) / 2 = sigmoid(2 u), which does not cancel
        return z * sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def act_grad(z, kind):
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "silu":
        p = sigmoid(z)
        return p * (1 + z * (1 - p))
    if kind == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2)) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        p = sigmoid(2 * c * (z + 0.044715 * z ** 3))
        return p + 2 * z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)
    return np.ones_like(z)


# A distribution factor p = 1 / (1 + exp(A)) below 2^-128 comes out as 0, since exp(A) passes float32's range, and
# one below 2^-126 may lose bits: up to this is missing from p, times what multiplies p.
LOST = 2.0 ** -126


def act_share(z, kind):
    """Relative error of the activation's distribution factor in float32.

    The factor is exp(-A) near its tail, A = |z| for SiLU, 2 u for GELU's tanh
    form and z^2 / 2 for its erfc: a relative rounding of the argument, at most
    four steps 2^-24 of it (twice that of z under the square), moves the
    factor by 4 A 2^-24 of itself. 32 steps more cover the exponential or
    erfc, the quotient and the products around it.
    """
    if kind in ("none", "relu"):
        return 4 * 2.0 ** -24 * np.ones_like(z)
    A = np.abs(z) if kind == "silu" else z * z if kind == "gelu" else np.abs(1.6 * (z + 0.044715 * z ** 3))
    return (32 + 4 * A) * 2.0 ** -24


def act_grad_error(z, kind):
    """Error of the activation's derivative in float32: the share above of each of its two terms, and where
    the second holds 1 - p, two steps of p there."""
    share = act_share(z, kind)
    if kind in ("none", "relu"):
        return share
    if kind == "gelu":
        return share * (0.5 * _erfc(-z / math.sqrt(2)) + np.abs(z) * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)) \
            + LOST * (1 + np.abs(z))
    slope = np.abs(z) if kind == "silu" else 1.6 * np.abs(z) * (1 + 3 * 0.044715 * z * z)
    p = sigmoid(z if kind == "silu" else 1.6 * (z + 0.044715 * z ** 3))
    return share * (p + slope * p * (1 - p)) + slope * p * 2.0 ** -23 + LOST * (1 + slope)


def experts(off, max_rows):
    """(expert, begin, end) as the offsets say, clamped into the buffer."""
    for l in range(len(off) - 1):
        b = min(max(int(off[l]), 0), max_rows)
        yield l, b, min(max(int(off[l + 1]), b), max_rows)


def product(x, off, W, bias=None, residual=None, kind="none", gated=False):
    """(y, pre, ez, ey): values, and bounds on the errors of a float32 computation of z and y.

    A sum of H exact products in any order is off by at most H 2^-24 times the
    sum of their magnitudes to first order, so 2 H 2^-24 covers it; the bias
    adds one rounding. That error passes through the activation times its
    slope; act_share covers the activation's own evaluation, and the product
    and sum after it are a rounding each.
    """
    rows, H = x.shape
    wide = W.shape[1]
    O = wide // 2 if gated else wide
    y, z = np.full((rows, O), np.nan), np.full((rows, wide), np.nan)
    ez, ey = np.zeros((rows, wide)), np.zeros((rows, O))
    for l, b, e in experts(off, rows):
        if e == b:
            continue
        v = x[b:e] @ W[l].T
        err = 2 * H * 2.0 ** -24 * (np.abs(x[b:e]) @ np.abs(W[l]).T)
        if bias is not None:
            v = v + bias[l]
            err = err + 2.0 ** -24 * (np.abs(v) + np.abs(bias[l]))
        z[b:e], ez[b:e] = v, err
        a = act(v[:, :O], kind)
        ea = LIPSCHITZ[kind] * err[:, :O] + act_share(v[:, :O], kind) * np.abs(a) + LOST * np.abs(v[:, :O])
        if gated:
            u, eu = v[:, O:], err[:, O:]
            ea = ea * (np.abs(u) + eu) + np.abs(a) * eu
            a = a * u
        ea = ea + 2.0 ** -23 * np.abs(a)
        if residual is not None:
            a = a + residual[b:e]
            ea = ea + 2.0 ** -23 * (np.abs(a) + np.abs(residual[b:e]))
        y[b:e], ey[b:e] = a, ea
    return y, z, ez, ey


def dgrad(gy, off, W, pre=None, kind="none", gated=False):
    """(grad_x, error bound of a float32 computation), as product()."""
    rows, O = gy.shape
    H = W.shape[2]
    wide = 2 * H if gated else H
    out, eo = np.full((rows, wide), np.nan), np.zeros((rows, wide))
    for l, b, e in experts(off, rows):
        if e == b:
            continue
        d = gy[b:e] @ W[l]
        err = 2 * O * 2.0 ** -24 * (np.abs(gy[b:e]) @ np.abs(W[l]))
        if pre is None:
            out[b:e], eo[b:e] = d, err
            continue
        g = pre[b:e, :H]
        f, df = act(g, kind), act_grad(g, kind)
        ed = err * np.abs(df) + (np.abs(d) + err) * act_grad_error(g, kind) + 2.0 ** -23 * np.abs(d * df)
        if not gated:
            out[b:e], eo[b:e] = d * df, ed
            continue
        u = pre[b:e, H:]
        out[b:e, :H], eo[b:e, :H] = d * u * df, ed * np.abs(u) + 2.0 ** -23 * np.abs(d * u * df)
        out[b:e, H:] = d * f
        eo[b:e, H:] = err * np.abs(f) + ((np.abs(d) + err) * act_share(g, kind) + 2.0 ** -23 * np.abs(d)) * np.abs(f) \
            + (np.abs(d) + err) * LOST * np.abs(g)
    return out, eo


def wgrad(gy, x, off, El):
    """(grad_W, grad_bias, bounds of each): sums over n rows are off by at most 2 n 2^-24 of their magnitudes."""
    O, H = gy.shape[1], x.shape[1]
    gW, gb = np.zeros((El, O, H)), np.zeros((El, O))
    eW, eb = np.zeros((El, O, H)), np.zeros((El, O))
    for l, b, e in experts(off, gy.shape[0]):
        gW[l], gb[l] = gy[b:e].T @ x[b:e], gy[b:e].sum(0)
        c = 2 * (e - b) * 2.0 ** -24
        eW[l], eb[l] = c * (np.abs(gy[b:e]).T @ np.abs(x[b:e])), c * np.abs(gy[b:e]).sum(0)
    return gW, gb, eW, eb
