"""Measured calls of the scored router, the experts' products and their gradients.

Each case is one call as a training step or a serving step makes it. `run`
computes it with elementary torch operations in 32 bits (64 for the router's
selection, where two experts' scores can lie closer than 32 bits resolve), or,
with `own`, through this framework's entry points. Batch shapes are those of
the synthetic workloads (decode, prefill with a capacity, ragged dropless,
fine-grained); the experts' inner widths are generic.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step's router: sigmoid scores, balance bias, groups ranked by their two best
        dict(name="route_decode", op="route", T=128, E=256, k=8, G=8, M=4, scores="sigmoid", normalize=True,
             top2=True, scale=2.5, bias=True, dtype="float32"),
        # a long prefill over many small experts: softmax scores with a bias, bf16 logits from the router's product
        dict(name="route_prefill", op="route", T=32768, E=512, k=10, G=1, M=1, scores="softmax", normalize=True,
             top2=False, scale=1.0, bias=True, dtype="bfloat16"),
        # training: the plain softmax's gradient touches every logit
        dict(name="route_grad", op="route_grad", T=32768, E=512, k=10, scores="softmax", normalize=False,
             scale=1.0, dtype="float32"),
        # training: the combine's gradient over the fine-grained batch, one expert row per replica
        dict(name="combine_grad_fine", op="combine_grad", T=32768, H=2048, k=10, drop=0.0, dtype="bfloat16"),
        # the same with a capacity's drops, two wide rows per token and float gradients; an odd batch
        dict(name="combine_grad_capacity", op="combine_grad", T=4099, H=4096, k=2, drop=0.08, dtype="float32"),
        # one token's gate and up products on the rank that holds its eight experts among 32
        dict(name="product_token", op="product", rows=8, El=32, H=7168, O=2048, act="silu", gated=True, bias=False,
             residual=False, pre=False, skew=0.0, pad=0),
        # a decoding step: 128 tokens from each of 8 ranks, about 32 rows for an expert
        dict(name="product_decode", op="product", rows=1024, El=32, H=7168, O=2048, act="silu", gated=True, bias=False,
             residual=False, pre=False, skew=0.3, pad=0),
        # training, fine-grained: gate and up products of a rank's 8 experts, pre-activations kept
        dict(name="product_fine", op="product", rows=327680, El=8, H=2048, O=768, act="silu", gated=True, bias=False,
             residual=False, pre=True, skew=0.3, pad=0),
        # the always-on expert's product back to the model's width with bias and residual; an odd batch
        dict(name="product_shared", op="product", rows=4093, El=1, H=2048, O=7168, act="none", gated=False, bias=True,
             residual=True, pre=False, skew=0.0, pad=3),
        # training: back through the second product and the gated activation
        dict(name="dgrad_prefill", op="dgrad", rows=32768, El=8, O=4096, H=2048, act="silu", gated=True, pre=True,
             skew=0.5, pad=0),
        # training: weight gradients of the fine-grained experts' first product
        dict(name="wgrad_fine", op="wgrad", rows=327680, El=8, O=1536, H=2048, bias=False, dtype="bfloat16", skew=0.3),
        # training, a ragged batch: few rows for each of 6 wide experts, float gradients and the bias's
        dict(name="wgrad_ragged", op="wgrad", rows=4093, El=6, O=1536, H=7168, bias=True, dtype="float32", skew=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "combine_grad", "product", "product", "dgrad", "wgrad"])
    if op in ("route", "route_grad"):
        G = rng.choice([1, 1, 4, 8, 16])
        E = G * rng.randint(max(2, 16 // G), 512 // G)
        M = rng.randint(max(1, G // 4), G)
        k = min(rng.randint(1, 12), M * (E // G))
        c = dict(op=op, T=_log(rng, 1, 32768), E=E, k=k, scores=rng.choice(["softmax", "sigmoid"]),
                 normalize=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["float32", "bfloat16"]))
        if op == "route":
            c |= dict(G=G, M=M, top2=G > 1 and rng.random() < 0.5, bias=rng.random() < 0.8)
        return c
    if op == "combine_grad":
        H = 8 * _log(rng, 32, 1024)
        k = rng.randint(1, 10)
        most = 32768 * 2048 * 10 // (H * k)
        return dict(op=op, T=_log(rng, 1, min(32768, most)), H=H, k=k, drop=rng.choice([0.0, 0.0, 0.1]),
                    dtype=rng.choice(["bfloat16", "float32"]))
    El = _log(rng, 1, 64)
    H, O = 8 * _log(rng, 32, 896), 8 * _log(rng, 32, 512)
    flops = 2 * 327680 * 2048 * 1536
    most = max(1, min(65536, flops // 2 // (2 * H * O * 2)))
    rows = _log(rng, 1, most)
    c = dict(op=op, rows=rows, El=El, H=H, O=O, skew=rng.choice([0.0, 0.3, 0.8]))
    acts = ["none", "relu", "silu", "gelu", "gelu_tanh"]
    if op == "product":
        gated = rng.random() < 0.5
        c |= dict(act=rng.choice(acts), gated=gated, bias=rng.random() < 0.4, residual=rng.random() < 0.3,
                  pre=rng.random() < 0.4, pad=rng.choice([0, 0, 5]))
    elif op == "dgrad":
        pre = rng.random() < 0.7
        c |= dict(act=rng.choice(acts) if pre else "none", gated=pre and rng.random() < 0.6, pre=pre,
                  pad=rng.choice([0, 0, 5]))
    else:
        c |= dict(bias=rng.random() < 0.5, dtype=rng.choice(["bfloat16", "float32"]))
    return c


# ---------------------------------------------------------------- inputs

def _counts(case, seed):
    """Rows of each expert: distinct experts while there is at most one row for each, else a skewed draw."""
    g = np.random.default_rng([seed, 11])
    rows, El = case["rows"], case["El"]
    if rows <= El:
        c = np.zeros(El, np.int64)
        c[g.permutation(El)[:rows]] = 1
        return c
    p = np.exp(case["skew"] * g.standard_normal(El))
    return g.multinomial(rows, p / p.sum())


def _kept(case):
    """Replicas that a capacity leaves."""
    return max(1, int(case["T"] * case["k"] * (1 - case["drop"])))


def _dtype(case):
    return getattr(torch, case["dtype"])


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)

    def weights(El, O, H):  # layer by layer, so that no float copy of all of them is held
        W = torch.empty(El, O, H, dtype=torch.bfloat16, device=DEV)
        for l in range(El):
            W[l] = randn(O, H, scale=H ** -0.5)
        return W

    s = dict(case)
    op = case["op"]
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = randn(T, E).to(_dtype(case))
        if op == "route":
            width = 0.1 if case["scores"] == "sigmoid" else 0.2 / E
            s["b"] = (torch.rand(E, generator=g, device=DEV) * 2 - 1) * width if case["bias"] else None
            s["idx"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
            s["w"] = torch.empty(T, k, device=DEV)
        else:
            s["idx"] = s["logits"].float().topk(k, dim=1).indices.int()
            s["grad_w"] = randn(T, k)
            s["grad_logits"] = torch.empty_like(s["logits"])
        return s
    if op == "combine_grad":
        T, H, k = case["T"], case["H"], case["k"]
        N = _kept(case)
        pos = torch.randperm(T * k, generator=g, device=DEV).int()  # a row for each replica, none for the dropped
        pos[pos >= N] = -1
        s["N"], s["pos"] = N, pos.view(T, k)
        s["topk_w"] = torch.softmax(randn(T, k), 1)
        s["y"] = randn(N, H, dtype=torch.bfloat16)
        s["grad_out"] = randn(T, H).to(_dtype(case))
        s["grad_y"] = torch.zeros(N + 1, H, dtype=torch.bfloat16, device=DEV)
        s["grad_w"] = torch.empty(T, k, device=DEV)
        return s
    counts = _counts(case, seed)
    El, H, O, rows = case["El"], case["H"], case["O"], case["rows"]
    max_rows = rows + case.get("pad", 0)
    s["offsets"] = torch.tensor([0, *np.cumsum(counts).tolist()], dtype=torch.int32, device=DEV)
    s["max_rows"], s["most"] = max_rows, int(counts.max())
    if op == "product":
        wide = 2 * O if case["gated"] else O
        s["x"] = randn(max_rows, H, dtype=torch.bfloat16)
        s["W"] = weights(El, wide, H)
        s["b"] = randn(El, wide, dtype=torch.bfloat16) if case["bias"] else None
        s["r"] = randn(max_rows, O, dtype=torch.bfloat16) if case["residual"] else None
        s["y"] = torch.zeros(max_rows + 1, O, dtype=torch.bfloat16, device=DEV)
        s["z"] = torch.zeros(max_rows + 1, wide, dtype=torch.bfloat16, device=DEV) if case["pre"] else None
    elif op == "dgrad":
        wide = 2 * H if case["gated"] else H
        s["grad_y"] = randn(max_rows, O, dtype=torch.bfloat16)
        s["W"] = weights(El, O, H)
        s["z"] = randn(max_rows, wide, dtype=torch.bfloat16) if case["pre"] else None
        s["grad_x"] = torch.zeros(max_rows + 1, wide, dtype=torch.bfloat16, device=DEV)
    else:
        s["grad_y"] = randn(rows, O, dtype=torch.bfloat16)
        s["x"] = randn(rows, H, dtype=torch.bfloat16)
        s["grad_W"] = torch.empty(El, O, H, dtype=_dtype(case), device=DEV)
        s["grad_b"] = torch.empty(El, O, device=DEV) if case["bias"] else None
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_route(s):
    import combine_route_topk_amd as moe
    return moe.moe_route_scored(s["logits"], s["b"], s["k"], n_groups=s["G"], topk_groups=s["M"], scores=s["scores"],
                                normalize=s["normalize"], group_top2=s["top2"], scale=s["scale"],
                                topk_idx=s["idx"], topk_w=s["w"])


def _own_route_grad(s):
    import combine_route_topk_amd as moe
    return moe.moe_route_scored_backward(s["logits"], s["idx"], s["grad_w"], scores=s["scores"],
                                         normalize=s["normalize"], scale=s["scale"], grad_logits=s["grad_logits"])


def _own_combine_grad(s):
    import combine_route_topk_amd as moe
    return moe.moe_combine_backward(s["grad_out"], s["y"], s["pos"], s["topk_w"], grad_y=s["grad_y"][:s["N"]],
                                    grad_w=s["grad_w"])


def _own_product(s):
    import combine_route_topk_amd as moe
    n = s["max_rows"]
    z = s["z"][:n] if s["z"] is not None else None
    y = moe.moe_expert_product(s["x"], s["offsets"], s["W"], bias=s["b"], residual=s["r"], act=s["act"],
                               gated=s["gated"], y=s["y"][:n], pre=z)
    return (y,) if z is None else (y, z)


def _own_dgrad(s):
    import combine_route_topk_amd as moe
    return moe.moe_expert_product_dgrad(s["grad_y"], s["offsets"], s["W"], pre=s["z"], act=s["act"], gated=s["gated"],
                                        grad_x=s["grad_x"][:s["max_rows"]])


def _own_wgrad(s):
    import combine_route_topk_amd as moe
    moe.moe_expert_product_wgrad(s["grad_y"], s["x"], s["offsets"], grad_W=s["grad_W"], grad_bias=s["grad_b"])
    return (s["grad_W"],) if s["grad_b"] is None else (s["grad_W"], s["grad_b"])


_own = dict(route=_own_route, route_grad=_own_route_grad, combine_grad=_own_combine_grad, product=_own_product,
            dgrad=_own_dgrad, wgrad=_own_wgrad)


def _plain_route(s):
    l = s["logits"].double()
    T, E = l.shape
    p = 1 / (1 + torch.exp(-l))
    if s["scores"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    sel = p if s["b"] is None else p + s["b"].double()
    if s["M"] < s["G"]:
        by = sel.view(T, s["G"], E // s["G"]).sort(dim=2, descending=True).values
        score = by[:, :, :2].sum(2) if s["top2"] else by[:, :, 0]
        best = score.sort(dim=1, descending=True, stable=True).indices[:, :s["M"]]
        keep = torch.zeros(T, s["G"], dtype=torch.bool, device=l.device).scatter_(1, best, True)
        sel = torch.where(keep[:, :, None].expand(T, s["G"], E // s["G"]).reshape(T, E), sel, -math.inf)
    idx = sel.sort(dim=1, descending=True, stable=True).indices[:, :s["k"]]
    w = p.gather(1, idx)
    if s["normalize"]:
        w = w / w.sum(1, keepdim=True)
    return idx.int(), (w * s["scale"]).float()


def _plain_route_grad(s):
    l, idx, g, c = s["logits"].float(), s["idx"].long(), s["grad_w"], s["scale"]
    if s["scores"] == "sigmoid":
        p = 1 / (1 + torch.exp(-l.gather(1, idx)))
        if s["normalize"]:
            w = p / p.sum(1, keepdim=True)
            d = c * w * (1 - p) * (g - (g * w).sum(1, keepdim=True))
        else:
            d = c * g * p * (1 - p)
        return torch.zeros_like(l).scatter_(1, idx, d).to(s["logits"].dtype)
    if s["normalize"]:
        ls = l.gather(1, idx)
        w = torch.exp(ls - ls.amax(1, keepdim=True))
        w = w / w.sum(1, keepdim=True)
        d = c * w * (g - (g * w).sum(1, keepdim=True))
        return torch.zeros_like(l).scatter_(1, idx, d).to(s["logits"].dtype)
    p = torch.exp(l - l.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    dense = torch.zeros_like(l).scatter_(1, idx, c * g)
    return (p * (dense - (dense * p).sum(1, keepdim=True))).to(s["logits"].dtype)


def _plain_combine_grad(s):
    pos, d = s["pos"].long(), s["grad_out"].float()
    T, k = pos.shape
    kept = pos >= 0
    at = torch.where(kept, pos, 0)
    grad_w = torch.where(kept, (s["y"][at.view(-1)].float().view(T, k, -1) * d[:, None, :]).sum(2), 0.0)
    rows = (s["topk_w"][:, :, None] * d[:, None, :]).to(torch.bfloat16)
    s["grad_y"][torch.where(kept, pos, s["N"]).view(-1)] = rows.view(T * k, -1)  # dropped ones to the spare row
    return s["grad_y"][:s["N"]], grad_w


def _slots(s):
    """Each expert's rows as one padded batch: row of slot m of expert l, and whether it is one."""
    first, last = s["offsets"][:-1].long(), s["offsets"][1:].long()
    at = first[:, None] + torch.arange(s["most"], device=first.device)
    real = at < last[:, None]
    return torch.where(real, at, 0), real


def _padded(rows, at, real):
    return rows[at].float() * real[:, :, None]


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


def _plain_product(s):
    at, real = _slots(s)
    z = torch.bmm(_padded(s["x"], at, real), s["W"].float().transpose(1, 2))
    if s["b"] is not None:
        z = z + s["b"].float()[:, None, :]
    O = s["O"]
    v = _act(z[..., :O], s["act"]) * z[..., O:] if s["gated"] else _act(z, s["act"])
    if s["r"] is not None:
        v = v + s["r"][at].float()
    n = s["max_rows"]
    to = torch.where(real, at, n)  # padding goes to the spare row
    s["y"][to] = v.to(torch.bfloat16)
    if s["z"] is None:
        return (s["y"][:n],)
    s["z"][to] = z.to(torch.bfloat16)
    return s["y"][:n], s["z"][:n]


def _plain_dgrad(s):
    at, real = _slots(s)
    d = torch.bmm(_padded(s["grad_y"], at, real), s["W"].float())
    if s["z"] is not None:
        z = s["z"][at].float()
        H = s["H"]
        if s["gated"]:
            a, u = z[..., :H], z[..., H:]
            d = torch.cat([d * u * _act_grad(a, s["act"]), d * _act(a, s["act"])], dim=2)
        else:
            d = d * _act_grad(z, s["act"])
    n = s["max_rows"]
    s["grad_x"][torch.where(real, at, n)] = d.to(torch.bfloat16)
    return s["grad_x"][:n]


def _plain_wgrad(s):
    at, real = _slots(s)
    d = _padded(s["grad_y"], at, real)
    grad_W = torch.bmm(d.transpose(1, 2).contiguous(), _padded(s["x"], at, real)).to(s["grad_W"].dtype)
    return (grad_W,) if s["grad_b"] is None else (grad_W, d.sum(1))


_plain = dict(route=_plain_route, route_grad=_plain_route_grad, combine_grad=_plain_combine_grad,
              product=_plain_product, dgrad=_plain_dgrad, wgrad=_plain_wgrad)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "float32" else 2
        if op == "route":
            return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": 6 * T * E}
        dense = case["scores"] == "softmax" and not case["normalize"]
        return {"bytes": T * E * size + 8 * T * k + (T * E if dense else T * k) * size,
                "flops": (6 * T * E if dense else 8 * T * k)}
    if op == "combine_grad":
        T, H, k = case["T"], case["H"], case["k"]
        N = _kept(case)
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": T * H * size + 4 * N * H + 12 * T * k, "flops": 3 * N * H}
    rows, El, H, O = case["rows"], case["El"], case["H"], case["O"]
    hit = rows if rows <= El else El * (1 - (1 - 1 / El) ** rows)  # experts that have rows
    if op == "product":
        wide = 2 * O if case["gated"] else O
        return {"bytes": int(2 * (rows * H + hit * wide * H + rows * O * (2 if case["residual"] else 1)
                                  + (rows * wide if case["pre"] else 0) + (hit * wide if case["bias"] else 0))),
                "flops": 2 * rows * H * wide}
    if op == "dgrad":
        wide = 2 * H if case["gated"] else H
        return {"bytes": int(2 * (rows * O + hit * O * H + rows * wide * (2 if case["pre"] else 1))),
                "flops": 2 * rows * H * O}
    return {"bytes": 2 * rows * (O + H) + El * O * H * (4 if case["dtype"] == "float32" else 2)
            + (4 * El * O if case["bias"] else 0), "flops": 2 * rows * H * O}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    with torch.no_grad():
        return _exact[case["op"]](prepare(case, seed))


def _exact_route(s):
    l = s["logits"].double().cpu().numpy()
    T, E = l.shape
    p = 1.0 / (1.0 + np.exp(-l)) if s["scores"] == "sigmoid" else np.exp(l - np.log(np.exp(l).sum(1, keepdims=True)))
    sel = p + (0.0 if s["b"] is None else s["b"].double().cpu().numpy())
    if s["M"] < s["G"]:
        part = np.partition(sel.reshape(T, s["G"], -1), -2, axis=2) if E // s["G"] > 1 else sel.reshape(T, s["G"], 1)
        score = part[:, :, -1] + part[:, :, -2] if s["top2"] and E // s["G"] > 1 else part[:, :, -1]
        rank = np.argsort(np.argsort(-score, axis=1, kind="stable"), axis=1, kind="stable")
        sel = np.where(np.repeat(rank < s["M"], E // s["G"], axis=1), sel, -np.inf)
    idx = np.argsort(-sel, axis=1, kind="stable")[:, :s["k"]]
    w = np.take_along_axis(p, idx, axis=1)
    if s["normalize"]:
        w /= w.sum(1, keepdims=True)
    return idx.astype(np.int32), w * s["scale"]


def _exact_route_grad(s):
    # the Jacobian of the weights, applied to their gradients
    l, idx, g = s["logits"].double(), s["idx"].long(), s["grad_w"].double() * s["scale"]
    p = torch.sigmoid(l) if s["scores"] == "sigmoid" else torch.softmax(l, 1)
    q = p.gather(1, idx)
    if s["normalize"]:
        total = q.sum(1, keepdim=True)
        g = g / total - (g * q).sum(1, keepdim=True) / total ** 2
    gp = torch.zeros_like(p)
    gp.scatter_(1, idx, g)
    if s["scores"] == "sigmoid":
        return gp * p * (1 - p)
    return p * gp - p * (p * gp).sum(1, keepdim=True)


def _exact_combine_grad(s):
    pos = s["pos"].long()
    T, k = pos.shape
    gy = torch.zeros(s["N"], s["H"], dtype=torch.float64, device=DEV)
    gw = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    d = s["grad_out"].double()
    for j in range(k):
        t = torch.nonzero(pos[:, j] >= 0).view(-1)
        at = pos[t, j]
        gy[at] = s["topk_w"][t, j].double()[:, None] * d[t]
        gw[t, j] = (s["y"][at].double() * d[t]).sum(1)
    return gy, gw


def _experts(s):
    o = s["offsets"].tolist()
    return [(l, o[l], o[l + 1]) for l in range(len(o) - 1) if o[l + 1] > o[l]]


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


def _exact_product(s):
    y = torch.zeros(s["max_rows"], s["O"], dtype=torch.float64, device=DEV)
    z = None if s["z"] is None else torch.zeros(s["max_rows"], s["z"].shape[1], dtype=torch.float64, device=DEV)
    for l, a, b in _experts(s):
        v = s["x"][a:b].double() @ s["W"][l].double().t()
        if s["b"] is not None:
            v += s["b"][l].double()
        if z is not None:
            z[a:b] = v
        y[a:b] = _exact_act(v[:, :s["O"]], s["act"])[0] * (v[:, s["O"]:] if s["gated"] else 1.0)
        if s["r"] is not None:
            y[a:b] += s["r"][a:b].double()
    return (y,) if z is None else (y, z)


def _exact_dgrad(s):
    out = torch.zeros(s["max_rows"], s["grad_x"].shape[1], dtype=torch.float64, device=DEV)
    H = s["H"]
    for l, a, b in _experts(s):
        d = s["grad_y"][a:b].double() @ s["W"][l].double()
        if s["z"] is not None:
            z = s["z"][a:b].double()
            f, df = _exact_act(z[:, :H], s["act"])
            d = torch.cat([d * z[:, H:] * df, d * f], 1) if s["gated"] else d * df
        out[a:b] = d
    return out


def _exact_wgrad(s):
    out = torch.zeros(s["El"], s["O"], s["H"], dtype=torch.float64, device=DEV)
    db = torch.zeros(s["El"], s["O"], dtype=torch.float64, device=DEV)
    for l, a, b in _experts(s):
        d = s["grad_y"][a:b].double()
        out[l] = d.t() @ s["x"][a:b].double()
        db[l] = d.sum(0)
    return (out,) if s["grad_b"] is None else (out, db)


_exact = dict(route=_exact_route, route_grad=_exact_route_grad, combine_grad=_exact_combine_grad,
              product=_exact_product, dgrad=_exact_dgrad, wgrad=_exact_wgrad)
