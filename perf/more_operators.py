"""Measured calls of the layer in 8 bits: the norm before the router, the
weights' quantisation by blocks of 128 x 128, the experts' products on FP8 rows
and their input gradient.

Each case is one call as a training step or a serving step makes it. `run`
computes it with elementary torch operations in 32 bits or, with `own`, through
this framework's entry points. Batch shapes are those of the synthetic
workloads (decode, prefill with a capacity, ragged dropless, fine-grained);
the experts' inner widths are generic. FP8 rows are the dispatch payload's:
E4M3 codes, then one power-of-two scale byte per 32 values in whole 128-byte
lines. What is held in 8 bits is returned as the values it stands for: codes
as E4M3 numbers, scale bytes as powers of two.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step: the norm before the router, residual added, rows for the router and for the dispatch
        dict(name="norm_decode", op="norm", T=128, H=7168, residual=True, y=True, fp8=True, dtype="bfloat16"),
        # a long prefill of the fine-grained layer
        dict(name="norm_prefill", op="norm", T=32768, H=2048, residual=True, y=True, fp8=True, dtype="bfloat16"),
        # training: back through that norm, the residual stream's own gradient joined
        dict(name="norm_grad_fine", op="norm_grad", T=32768, H=2048, stream=True, dtype="bfloat16"),
        # training with a float32 residual stream, an odd batch of wide rows
        dict(name="norm_grad_wide", op="norm_grad", T=4099, H=7168, stream=True, dtype="float32"),
        # a training step's weights again in 8 bits: a rank's 8 fine-grained experts, and transposed for the gradient
        dict(name="weights_fine", op="weights", El=8, O=1536, H=2048, transpose=True, dtype="bfloat16"),
        # loading a wide layer for serving: gate and up weights of 32 experts
        dict(name="weights_wide", op="weights", El=32, O=4096, H=7168, transpose=False, dtype="bfloat16"),
        # one token's gate and up products on the rank that holds its eight experts among 32
        dict(name="product8_token", op="product", rows=8, El=32, H=7168, O=2048, act="silu", gated=True, bias=False,
             residual=False, pre=False, out="fp8", skew=0.0, pad=0),
        # a decoding step: 128 tokens from each of 8 ranks, about 32 rows for an expert
        dict(name="product8_decode", op="product", rows=1024, El=32, H=7168, O=2048, act="silu", gated=True, bias=False,
             residual=False, pre=False, out="fp8", skew=0.3, pad=0),
        # training, fine-grained: gate and up products of a rank's 8 experts, pre-activations kept, the activated rows
        # in 8 bits for the next product and in bf16 for the weights' gradient
        dict(name="product8_fine", op="product", rows=327680, El=8, H=2048, O=768, act="silu", gated=True, bias=False,
             residual=False, pre=True, out="both", skew=0.3, pad=0),
        # the always-on expert's product back to the model's width with bias and residual; an odd batch
        dict(name="product8_shared", op="product", rows=4093, El=1, H=2048, O=7168, act="none", gated=False, bias=True,
             residual=True, pre=False, out="bf16", skew=0.0, pad=3),
        # training: back through the second product and the gated activation, for the first product's gradients
        dict(name="dgrad8_prefill", op="dgrad", rows=32768, El=8, O=4096, H=2048, act="silu", gated=True, pre=True,
             out="both", skew=0.5, pad=0),
        # training, a ragged batch: back through the first product of 6 wide experts to the model's width
        dict(name="dgrad8_ragged", op="dgrad", rows=4093, El=6, O=4096, H=7168, act="none", gated=False, pre=False,
             out="bf16", skew=0.5, pad=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "norm_grad", "weights", "product", "product", "product", "dgrad", "dgrad"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    if op in ("norm", "norm_grad"):
        fp8 = op == "norm" and rng.random() < 0.6
        H = (32 if fp8 else 8) * _log(rng, 8, 224 if fp8 else 896)
        c = dict(op=op, T=_log(rng, 1, min(32768, 32768 * 2048 // H)), H=H, dtype=dtype)
        if op == "norm":
            c |= dict(residual=rng.random() < 0.7, y=not fp8 or rng.random() < 0.5, fp8=fp8)
        else:
            c |= dict(stream=rng.random() < 0.6)
        return c
    El = _log(rng, 1, 64)
    H, O = 32 * _log(rng, 8, 224), 32 * _log(rng, 8, 128)
    if op == "weights":
        most = max(1, 32 * 4096 * 7168 // 2 // (O * H))
        return dict(op=op, El=min(El, most), O=O, H=H, transpose=rng.random() < 0.5, dtype=dtype)
    flops = 2 * 327680 * 2048 * 1536
    most = max(1, min(65536, flops // 2 // (2 * H * O * 2)))
    c = dict(op=op, rows=_log(rng, 1, most), El=El, H=H, O=O, skew=rng.choice([0.0, 0.3, 0.8]), pad=rng.choice([0, 0, 5]),
             out=rng.choice(["bf16", "fp8", "both"]))
    acts = ["none", "relu", "silu", "gelu", "gelu_tanh"]
    if op == "product":
        c |= dict(act=rng.choice(acts), gated=rng.random() < 0.5, bias=rng.random() < 0.4, residual=rng.random() < 0.3,
                  pre=rng.random() < 0.4)
    else:
        pre = rng.random() < 0.7
        c |= dict(act=rng.choice(acts) if pre else "none", gated=pre and rng.random() < 0.6, pre=pre)
    return c


# ---------------------------------------------------------------- inputs

def _counts(case, seed):
    """Rows of each expert: distinct experts while there is at most one row for each, else a skewed draw."""
    g = np.random.default_rng([seed, 12])
    rows, El = case["rows"], case["El"]
    if rows <= El:
        c = np.zeros(El, np.int64)
        c[g.permutation(El)[:rows]] = 1
        return c
    p = np.exp(case["skew"] * g.standard_normal(El))
    return g.multinomial(rows, p / p.sum())


def _row_bytes(H):
    return H + 128 * ((H + 4095) // 4096)


def _blocks(n):
    return (n + 127) // 128


def _views(rows, H):
    """The codes and the scales of FP8 rows, as the values they stand for."""
    return rows[:, :H].view(E4M3), rows[:, H:H + H // 32].view(E8M0)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    def bytes8(n, width):
        return torch.zeros(n, _row_bytes(width), dtype=torch.uint8, device=DEV)

    def rows8(n, width):  # rows of normals of different sizes, as the dispatch sends them
        r = bytes8(n, width)
        for a in range(0, n, 65536):
            b = min(n, a + 65536)
            v = randn(b - a, width) * torch.exp(randn(b - a, 1))
            codes, exps = _encode_rows(v)
            r[a:b, :width] = codes.view(torch.uint8)
            r[a:b, width:width + width // 32] = exps
        return r

    def weights8(El, O, H):  # codes that fill their range as a block's do, and scales that differ by block
        W = torch.empty(El, O, H, dtype=torch.uint8, device=DEV)
        for l in range(El):
            W[l] = (randn(O, H, scale=105.0)).clamp_(-448, 448).to(E4M3).view(torch.uint8)
        return W.view(E4M3), torch.exp(randn(El, _blocks(O), _blocks(H), scale=0.3)) * (H ** -0.5 / 105)

    s = dict(case)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        T, H, dt = case["T"], case["H"], getattr(torch, case["dtype"])
        s["w"] = (1 + randn(H, scale=0.2)).to(torch.bfloat16)
        s["x"] = (randn(T, H) * torch.exp(randn(T, 1, scale=0.5))).to(dt)
        if op == "norm":
            s["r"] = randn(T, H, dtype=dt) if case["residual"] else None
            s["total"] = torch.empty(T, H, dtype=dt, device=DEV) if case["residual"] else None
            s["y"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV) if case["y"] else None
            s["y8"] = bytes8(T, H) if case["fp8"] else None
            s["y8_views"] = _views(s["y8"], H) if case["fp8"] else ()
        else:
            s["grad_y"] = randn(T, H, dtype=torch.bfloat16)
            s["grad_total"] = randn(T, H, dtype=dt) if case["stream"] else None
            s["grad_x"] = torch.empty(T, H, dtype=dt, device=DEV)
            s["grad_w"] = torch.empty(H, device=DEV)
        return s
    El, H, O = case["El"], case["H"], case["O"]
    if op == "weights":
        s["W"] = torch.empty(El, O, H, dtype=getattr(torch, case["dtype"]), device=DEV)
        for l in range(El):
            s["W"][l] = randn(O, H, scale=H ** -0.5)
        s["codes"] = torch.empty(El, O, H, dtype=E4M3, device=DEV)
        s["scale"] = torch.empty(El, _blocks(O), _blocks(H), device=DEV)
        s["codes_t"] = torch.empty(El, H, O, dtype=E4M3, device=DEV) if case["transpose"] else None
        s["scale_t"] = torch.empty(El, _blocks(H), _blocks(O), device=DEV) if case["transpose"] else None
        return s
    counts = _counts(case, seed)
    n = case["rows"] + case["pad"]
    s["offsets"] = torch.tensor([0, *np.cumsum(counts).tolist()], dtype=torch.int32, device=DEV)
    s["n"], s["most"] = n, int(counts.max())
    # K columns in, N columns out before a gate, and what a row of the output holds
    K, N = (H, O) if op == "product" else (O, H)
    wide = 2 * N if case["gated"] else N
    width = N if op == "product" else wide
    s["K"], s["N"], s["width"] = K, N, width
    s["x"] = rows8(n, K)
    s["W"], s["ws"] = weights8(El, wide if op == "product" else N, K)
    s["y"] = torch.zeros(n + 1, width, dtype=torch.bfloat16, device=DEV) if case["out"] != "fp8" else None
    s["y8"] = bytes8(n + 1, width) if case["out"] != "bf16" else None
    s["y8_views"] = _views(s["y8"][:n], width) if case["out"] != "bf16" else ()
    if op == "product":
        s["b"] = randn(El, wide, dtype=torch.bfloat16) if case["bias"] else None
        s["r"] = randn(n, N, dtype=torch.bfloat16) if case["residual"] else None
        s["z"] = torch.zeros(n + 1, wide, dtype=torch.bfloat16, device=DEV) if case["pre"] else None
    else:
        s["z"] = randn(n, wide, dtype=torch.bfloat16) if case["pre"] else None
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_norm(s):
    import combine_route_topk_amd as moe
    moe.moe_rms_norm(s["x"], s["w"], residual=s["r"], eps=EPS, total=s["total"], y=s["y"], y8=s["y8"],
                     need_y=s["y"] is not None)
    return s["total"], s["y"], *s["y8_views"]


def _own_norm_grad(s):
    import combine_route_topk_amd as moe
    return moe.moe_rms_norm_backward(s["grad_y"], s["x"], s["w"], eps=EPS, grad_total=s["grad_total"],
                                     grad_x=s["grad_x"], grad_weight=s["grad_w"])


def _own_weights(s):
    import combine_route_topk_amd as moe
    return moe.moe_fp8_quantize_weights(s["W"], codes=s["codes"], scale=s["scale"], codes_t=s["codes_t"],
                                        scale_t=s["scale_t"])


def _own_product(s):
    import combine_route_topk_amd as moe
    n = s["n"]
    y, y8, z = (None if s[k] is None else s[k][:n] for k in ("y", "y8", "z"))
    moe.moe_expert_product_fp8(s["x"], s["offsets"], s["W"], s["ws"], bias=s["b"], residual=s["r"], act=s["act"],
                               gated=s["gated"], y=y, y8=y8, pre=z, need_y=y is not None)
    return y, z, *s["y8_views"]


def _own_dgrad(s):
    import combine_route_topk_amd as moe
    n = s["n"]
    y, y8 = (None if s[k] is None else s[k][:n] for k in ("y", "y8"))
    moe.moe_expert_product_fp8_dgrad(s["x"], s["offsets"], s["W"], s["ws"], pre=s["z"], act=s["act"],
                                     gated=s["gated"], grad_x=y, grad_x8=y8, need_x=y is not None)
    return y, *s["y8_views"]


_own = dict(norm=_own_norm, norm_grad=_own_norm_grad, weights=_own_weights, product=_own_product, dgrad=_own_dgrad)


def _encode_rows(v):
    """Codes and scale bytes of float32 rows: the least power of two that keeps 32 values within E4M3's range."""
    n, H = v.shape
    b = v.view(n, H // 32, 32)
    m, e = torch.frexp(b.abs().amax(2))  # amax = m 2^e, 1/2 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-127)
    e = torch.where(m == 0, -127, e)
    codes = torch.ldexp(b, -e[:, :, None]).to(E4M3)
    return codes.view(n, H), (e + 127).to(torch.uint8)


def _decode_rows(rows, H):
    n = rows.shape[0]
    c, p = _views(rows, H)
    return (c.float().view(n, H // 32, 32) * p.float()[:, :, None]).view(n, H)


def _decode_weights(W, scale):
    El, O, H = W.shape
    by_block = scale[:, :, None, :, None].expand(-1, -1, 128, -1, 128).reshape(El, scale.shape[1] * 128, -1)
    return W.float() * by_block[:, :O, :H]


def _plain_norm(s):
    t = s["x"]
    if s["r"] is not None:
        t = (s["x"].float() + s["r"].float()).to(s["x"].dtype)
    h = t.float()
    v = h / torch.sqrt((h * h).sum(1, keepdim=True) / s["H"] + EPS) * s["w"].float()
    out = [t if s["r"] is not None else None, v.to(torch.bfloat16) if s["y"] is not None else None]
    if s["fp8"]:
        codes, exps = _encode_rows(v)
        out += [codes, exps.view(E8M0)]
    return tuple(out)


def _plain_norm_grad(s):
    h, g = s["x"].float(), s["grad_y"].float()
    r = 1 / torch.sqrt((h * h).sum(1, keepdim=True) / s["H"] + EPS)
    n = h * r
    a = g * s["w"].float()
    d = r * (a - n * ((a * n).sum(1, keepdim=True) / s["H"]))
    if s["grad_total"] is not None:
        d = d + s["grad_total"].float()
    return d.to(s["x"].dtype), (g * n).sum(0)


def _plain_weights(s):
    W = s["W"].float()
    El, O, H = W.shape
    full = torch.zeros(El, _blocks(O) * 128, _blocks(H) * 128, device=W.device)
    full[:, :O, :H] = W
    full = full.view(El, _blocks(O), 128, _blocks(H), 128)
    top = full.abs().amax((2, 4))
    scale = torch.where(top > 0, top / 448, 1.0)
    codes = (full / scale[:, :, None, :, None]).to(E4M3).view(El, _blocks(O) * 128, _blocks(H) * 128)
    codes = codes.view(torch.uint8)[:, :O, :H].contiguous()
    if not s["transpose"]:
        return codes.view(E4M3), scale, None, None
    return (codes.view(E4M3), scale, codes.transpose(1, 2).contiguous().view(E4M3),
            scale.transpose(1, 2).contiguous())


def _slots(s):
    """Each expert's rows as one padded batch: row of slot m of expert l, and whether it is one."""
    first, last = s["offsets"][:-1].long(), s["offsets"][1:].long()
    at = first[:, None] + torch.arange(s["most"], device=first.device)
    real = at < last[:, None]
    return torch.where(real, at, 0), real


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _sums(s):
    """The products in float32, slot by slot, and where the slots' rows lie (padding: the spare row)."""
    at, real = _slots(s)
    z = torch.bmm(_decode_rows(s["x"], s["K"])[at] * real[:, :, None], _decode_weights(s["W"], s["ws"]).transpose(1, 2))
    return z, at, torch.where(real, at, s["n"])


def _put(s, v, to):
    """Writes the results' rows as bf16 and as FP8 rows, and returns both."""
    n, width = s["n"], s["width"]
    if s["y"] is not None:
        s["y"][to] = v.to(torch.bfloat16)
    if s["y8"] is not None:
        codes, exps = _encode_rows(v.view(-1, width))
        s["y8"][to.view(-1), :width] = codes.view(torch.uint8)
        s["y8"][to.view(-1), width:width + width // 32] = exps
    return None if s["y"] is None else s["y"][:n]


def _plain_product(s):
    z, at, to = _sums(s)
    if s["b"] is not None:
        z = z + s["b"].float()[:, None, :]
    O = s["O"]
    v = _act(z[..., :O], s["act"]) * z[..., O:] if s["gated"] else _act(z, s["act"])
    if s["r"] is not None:
        v = v + s["r"][at].float()
    if s["z"] is not None:
        s["z"][to] = z.to(torch.bfloat16)
    return _put(s, v, to), None if s["z"] is None else s["z"][:s["n"]], *s["y8_views"]


def _plain_dgrad(s):
    d, at, to = _sums(s)
    if s["z"] is not None:
        z = s["z"][at].float()
        if s["gated"]:
            a, u = z[..., :s["N"]], z[..., s["N"]:]
            d = torch.cat([d * u * _act_grad(a, s["act"]), d * _act(a, s["act"])], dim=2)
        else:
            d = d * _act_grad(z, s["act"])
    return _put(s, d, to), *s["y8_views"]


_plain = dict(norm=_plain_norm, norm_grad=_plain_norm_grad, weights=_plain_weights, product=_plain_product,
              dgrad=_plain_dgrad)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        T, H = case["T"], case["H"]
        size = 4 if case["dtype"] == "float32" else 2
        if op == "norm":
            row = size * H * (3 if case["residual"] else 1) + (2 * H if case["y"] else 0)
            return {"bytes": T * (row + (H + H // 32 if case["fp8"] else 0)) + 2 * H, "flops": 5 * T * H}
        return {"bytes": T * H * (2 + size * (3 if case["stream"] else 2)) + 6 * H, "flops": 10 * T * H}
    El, H, O = case["El"], case["H"], case["O"]
    if op == "weights":
        size = (4 if case["dtype"] == "float32" else 2) + (2 if case["transpose"] else 1)
        return {"bytes": El * (O * H * size + 4 * _blocks(O) * _blocks(H) * (2 if case["transpose"] else 1)),
                "flops": 3 * El * O * H}
    rows = case["rows"]
    hit = rows if rows <= El else El * (1 - (1 - 1 / El) ** rows)  # experts that have rows
    K, N = (H, O) if op == "product" else (O, H)
    wide = 2 * N if case["gated"] else N
    made, width = (wide, N) if op == "product" else (N, wide)
    row = K + K // 32 + (2 * width if case["out"] != "fp8" else 0) + (width + width // 32 if case["out"] != "bf16" else 0)
    row += 2 * wide if case["pre"] else 0
    each = made * K + 4 * _blocks(made) * _blocks(K)
    if op == "product":
        row += 2 * N if case["residual"] else 0
        each += 2 * wide if case["bias"] else 0
    return {"bytes": int(rows * row + hit * each), "flops": 2 * rows * K * made}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    with torch.no_grad():
        return _exact[case["op"]](prepare(case, seed))


def _exact_rows(v):
    """What FP8 rows stand for, before the codes' rounding: values over their scales, and the scales."""
    by = v.reshape(v.shape[0], -1, 32)
    top = by.abs().amax(2)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 448))
    e = torch.where(top > 448 * 2 ** e, e + 1, torch.where(top <= 224 * 2 ** e, e - 1, e))
    p = 2 ** torch.where(top > 0, e.clamp(min=-127), -127.0)
    return (by / p[:, :, None]).reshape(v.shape), p


def _exact_norm(s):
    x, out = s["x"].double(), []
    if s["r"] is not None:
        x = x + s["r"].double()
    out.append(x if s["r"] is not None else None)
    t = x.float().to(s["x"].dtype).double()  # the norm is of the sum as it is stored
    v = t * (t.pow(2).mean(1, keepdim=True) + EPS).pow(-0.5) * s["w"].double()
    out.append(v if s["y"] is not None else None)
    if s["fp8"]:
        out += list(_exact_rows(v))
    return tuple(out)


def _exact_norm_grad(s):
    # the Jacobian of t -> t (mean t^2 + eps)^(-1/2), applied to the gradient
    t, g = s["x"].double(), s["grad_y"].double()
    m = t.pow(2).mean(1, keepdim=True) + EPS
    a = g * s["w"].double()
    d = a * m.pow(-0.5) - t * m.pow(-1.5) * (a * t).mean(1, keepdim=True)
    if s["grad_total"] is not None:
        d = d + s["grad_total"].double()
    return d, (g * t * m.pow(-0.5)).sum(0)


def _exact_weights(s):
    El, O, H = s["W"].shape
    codes = torch.empty(El, O, H, dtype=torch.float64, device=DEV)
    scale = torch.empty(El, _blocks(O), _blocks(H), dtype=torch.float64, device=DEV)
    for o in range(_blocks(O)):
        for h in range(_blocks(H)):
            b = s["W"][:, o * 128:(o + 1) * 128, h * 128:(h + 1) * 128].double()
            top = b.abs().amax((1, 2))
            scale[:, o, h] = torch.where(top > 0, top / 448, 1.0)
            codes[:, o * 128:(o + 1) * 128, h * 128:(h + 1) * 128] = b / scale[:, o, h, None, None]
    if not s["transpose"]:
        return codes, scale, None, None
    return codes, scale, codes.transpose(1, 2).contiguous(), scale.transpose(1, 2).contiguous()


def _exact_act(z, act):
    """(act(z), act'(z)) in 64 bits."""
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        p = torch.sigmoid(2 * u)
        return z * p, p + 2 * z * p * (1 - p) * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)
    return z, torch.ones_like(z)


def _exact_sums(s):
    """Of every expert with rows: its number, its rows, and their products in 64 bits."""
    K, off = s["K"], s["offsets"].tolist()
    for l, (a, b) in enumerate(zip(off, off[1:])):
        if b > a:
            x = s["x"][a:b, :K].view(E4M3).double()
            x = x * torch.exp2(s["x"][a:b, K:K + K // 32].double() - 127).repeat_interleave(32, 1)
            W = s["W"][l].double()
            W = W * s["ws"][l].double().repeat_interleave(128, 0)[:W.shape[0]].repeat_interleave(128, 1)[:, :K]
            yield l, a, b, x @ W.t()


def _exact_out(s, v):
    """The outputs that the case asks for, of the rows that experts have: zeros elsewhere, as the buffers hold."""
    n, off = s["n"], int(s["offsets"][-1])
    p, q = _exact_rows(v) if s["y8"] is not None else (None, None)
    if p is not None:
        p[off:], q[off:] = 0, 2.0 ** -127
    return (v if s["y"] is not None else None), () if p is None else (p, q)


def _exact_product(s):
    n, O = s["n"], s["O"]
    v = torch.zeros(n, O, dtype=torch.float64, device=DEV)
    z = None if s["z"] is None else torch.zeros(n, s["z"].shape[1], dtype=torch.float64, device=DEV)
    for l, a, b, t in _exact_sums(s):
        if s["b"] is not None:
            t = t + s["b"][l].double()
        if z is not None:
            z[a:b] = t
        v[a:b] = _exact_act(t[:, :O], s["act"])[0] * (t[:, O:] if s["gated"] else 1.0)
        if s["r"] is not None:
            v[a:b] += s["r"][a:b].double()
    y, p = _exact_out(s, v)
    return y, z, *p


def _exact_dgrad(s):
    v = torch.zeros(s["n"], s["width"], dtype=torch.float64, device=DEV)
    for l, a, b, d in _exact_sums(s):
        if s["z"] is not None:
            z = s["z"][a:b].double()
            f, df = _exact_act(z[:, :s["N"]], s["act"])
            d = torch.cat([d * z[:, s["N"]:] * df, d * f], 1) if s["gated"] else d * df
        v[a:b] = d
    y, p = _exact_out(s, v)
    return y, *p


_exact = dict(norm=_exact_norm, norm_grad=_exact_norm_grad, weights=_exact_weights, product=_exact_product,
              dgrad=_exact_dgrad)
