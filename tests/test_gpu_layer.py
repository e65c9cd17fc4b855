"""One mixture-of-experts layer forward and backward on the GPU, every step
through the library: scored routing, layout, permute, gated experts' products,
a shared expert, combine; then the combine's gradient, the products' gradients,
the permute's (the combine with weights 1) and the router's. Each step is
compared with float64 on the very tensors that went into it, so no step's
rounding is charged to the next.
"""

import numpy as np
import pytest
import torch

import ops_reference as ref
from test_gpu_product import assert_rows, bf16, dn, up

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("T,H,I,E,k,G,M,kind", [(96, 128, 72, 16, 4, 4, 2, "sigmoid"), (1, 256, 64, 32, 8, 1, 1, "softmax"),
                                                (700, 192, 136, 8, 2, 1, 1, "softmax")])
def test_layer(T, H, I, E, k, G, M, kind):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import combine_route_topk_amd as moe
    rng = np.random.default_rng(T)
    print("[case]", T, H, I, E, k, G, M, kind, flush=True)
    x, logits = up(bf16(rng, T, H)), torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
    bias = torch.from_numpy(rng.uniform(-0.05, 0.05, E).astype(np.float32)).to(DEV)
    W1, b1 = up(bf16(rng, E, 2 * I, H, scale=H ** -0.5)), up(bf16(rng, E, 2 * I))
    W2 = up(bf16(rng, E, H, I, scale=I ** -0.5))
    S1, S2 = up(bf16(rng, 1, I, H, scale=H ** -0.5)), up(bf16(rng, 1, H, I, scale=I ** -0.5))
    grad = up(bf16(rng, T, H))

    # forward
    idx, w = moe.moe_route_scored(logits, bias, k, G, M, kind, True, G > 1, 2.0)
    L = moe.moe_dispatch_layout(idx, E, 1)
    off, pos = L["expert_offsets"], L["pos"]
    send = moe.moe_dispatch_permute(x, pos, E)
    z = torch.empty(T * k, 2 * I, dtype=torch.bfloat16, device=DEV)
    h = moe.moe_expert_product(send, off, W1, b1, act="silu", gated=True, pre=z)
    y = moe.moe_expert_product(h, off, W2)
    one = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    sz = torch.empty(T, I, dtype=torch.bfloat16, device=DEV)
    sh = moe.moe_expert_product(x, one, S1, act="gelu", pre=sz)
    shared = moe.moe_expert_product(sh, one, S2, residual=x)
    out = moe.moe_combine_reduce(y, pos, w, shared)
    # backward
    gy, gw = moe.moe_combine_backward(grad, y, pos, w)
    gz = moe.moe_expert_product_dgrad(gy, off, W2, z, "silu", True)
    gW2 = moe.moe_expert_product_wgrad(gy, h, off, torch.empty(E, H, I, device=DEV))
    gb1 = torch.empty(E, 2 * I, device=DEV)
    gW1 = moe.moe_expert_product_wgrad(gz, send, off, torch.empty(E, 2 * I, H, device=DEV), gb1)
    gsend = moe.moe_expert_product_dgrad(gz, off, W1)
    gsz = moe.moe_expert_product_dgrad(grad, one, S2, sz, "gelu")
    gshared = moe.moe_expert_product_dgrad(gsz, one, S1)
    gx = moe.moe_combine_reduce(gsend, pos, torch.ones(T, k, device=DEV), gshared, grad)
    gl = moe.moe_route_scored_backward(logits, idx, gw, kind, True, 2.0)
    torch.cuda.synchronize()

    c = {n: dn(t.cpu()) for n, t in dict(x=x, W1=W1, b1=b1, W2=W2, S1=S1, S2=S2, send=send, z=z, h=h, y=y, sz=sz, sh=sh,
                                         grad=grad, gy=gy, gz=gz, gsend=gsend, gsz=gsz, w=w, shared=shared,
                                         gshared=gshared).items()}
    o, p = off.cpu().numpy(), pos.cpu().numpy()
    n, so = T * k, np.array([0, T])
    i64, w64 = ref.route(logits.double().cpu().numpy(), bias.double().cpu().numpy(), k, G, M, kind, True, G > 1, 2.0)
    assert (idx.cpu().numpy() == i64).all() and np.abs(c["w"] - w64).max() < 2 * (E + 64) * 2.0 ** -24
    assert int(o[-1]) == n and sorted(p.ravel().tolist()) == list(range(n))
    wy, wz, ez, ey = ref.product(c["send"], o, c["W1"], c["b1"], None, "silu", True)
    assert_rows(h, wy, ey, n, "h"), assert_rows(z, wz, ez, n, "z")
    wy, _, _, ey = ref.product(c["h"], o, c["W2"])
    assert_rows(y, wy, ey, n, "y")
    wy, _, _, ey = ref.product(c["x"], so, c["S1"], None, None, "gelu")
    assert_rows(sh, wy, ey, T, "sh")
    wy, _, _, ey = ref.product(c["sh"], so, c["S2"], None, c["x"])
    assert_rows(shared, wy, ey, T, "shared")
    acc = (c["w"][:, :, None] * c["y"][p]).sum(1) + c["shared"]
    mag = (np.abs(c["w"])[:, :, None] * np.abs(c["y"][p])).sum(1) + np.abs(c["shared"])
    assert_rows(out, acc, (k + 4) * 2.0 ** -24 * mag, T, "out")
    wgy, wgw = ref.combine_backward(c["grad"], c["y"], p, c["w"])
    assert_rows(gy, wgy, 2.0 ** -23 * np.abs(wgy), n, "gy")
    assert (np.abs(gw.cpu().double().numpy() - wgw)
            <= 2 * H * 2.0 ** -24 * (np.abs(c["y"][p]) * np.abs(c["grad"])[:, None, :]).sum(2)).all()
    assert_rows(gz, *ref.dgrad(c["gy"], o, c["W2"], c["z"], "silu", True), n, "gz")
    assert_rows(gsend, *ref.dgrad(c["gz"], o, c["W1"]), n, "gsend")
    assert_rows(gsz, *ref.dgrad(c["grad"], so, c["S2"], c["sz"], "gelu"), T, "gsz")
    for got, gb, a, b in ((gW2, None, "gy", "h"), (gW1, gb1, "gz", "send")):
        vW, vb, eW, eb = ref.wgrad(c[a], c[b], o, E)
        assert (np.abs(got.cpu().double().numpy() - vW) <= eW + 2.0 ** -126).all()
        assert gb is None or (np.abs(gb.cpu().double().numpy() - vb) <= eb + 2.0 ** -126).all()
    acc = c["gsend"][p].sum(1) + c["gshared"] + c["grad"]
    mag = np.abs(c["gsend"][p]).sum(1) + np.abs(c["gshared"]) + np.abs(c["grad"])
    assert_rows(gx, acc, (k + 4) * 2.0 ** -24 * mag, T, "gx")
    gwd = gw.double().cpu().numpy()
    want = ref.route_backward(logits.double().cpu().numpy(), i64, gwd, kind, True, 2.0)
    assert np.abs(gl.cpu().double().numpy() - want).max() <= 4 * (E + 64) * 2.0 ** -24 * np.abs(gwd).max()
