"""One mixture-of-experts block with FP8 rows and weights in 8 bits, forward
and backward on the GPU, every step through the library: norm of the residual
stream, routing, layout, the norm's FP8 rows permuted, both experts' products
on FP8 rows, the combine onto the stream; then the combine's gradient, both
input gradients on FP8 rows, the weights' gradients, the permute's and the
norm's. Each step is compared with float64 on the very tensors that went into
it, so no step's rounding is charged to the next. Then the forward of a few
tokens, captured and replayed on other inputs, against the same calls made
eagerly.
"""

import numpy as np
import pytest
import torch

import fp8_reference as f8
import ops_reference as ref
from test_gpu_product import assert_rows, bf16, dn, up

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import combine_route_topk_amd
    return combine_route_topk_amd


def values(t):
    return dn(t.cpu())


def permute8(moe, y8, pos, E):
    """The permute moves whole rows, whatever they hold."""
    return moe.moe_dispatch_permute(y8.view(torch.bfloat16), pos, E).view(torch.uint8)


def rows8(moe, x):
    """bf16 rows as FP8 rows, in their order."""
    n = x.shape[0]
    return moe.moe_dispatch_permute_fp8(x, torch.arange(n, dtype=torch.int32, device=DEV)[:, None], 1, send_rows=n)


def weights(moe, W):
    c, s, ct, st = moe.moe_fp8_quantize_weights(W, transpose=True)
    codes = c.view(torch.uint8).cpu().numpy()
    v, g = f8.decode_weights(codes, s.cpu().numpy()), f8.weights_largest(codes, s.cpu().numpy())
    codes_t = ct.view(torch.uint8).cpu().numpy()
    vt, gt = f8.decode_weights(codes_t, st.cpu().numpy()), f8.weights_largest(codes_t, st.cpu().numpy())
    assert (vt == v.transpose(0, 2, 1)).all()
    return c, s, ct, st, v, g, vt, gt


def near32(got, want, err, what):
    """float32 results."""
    d = np.abs(values(got) - want) - (err + f8.U * (np.abs(want) + err) + 2.0 ** -126)
    assert (d <= 0).all(), f"{what}: worst by {d.max()}"


# the products' kernels for few rows (twice), for some tens of an expert's, for whole tiles
@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 64, 16, 4), (37, 128, 96, 8, 2), (300, 256, 160, 8, 4), (3000, 512, 288, 4, 4)])
def test_block(moe, T, H, I, E, k):
    rng = np.random.default_rng(T)
    print("[case]", T, H, I, E, k, flush=True)
    x, attn, nw, grad = up(bf16(rng, T, H)), up(bf16(rng, T, H)), up(bf16(rng, H)), up(bf16(rng, T, H))
    W1, W2 = up(bf16(rng, E, 2 * I, H, scale=H ** -0.5)), up(bf16(rng, E, H, I, scale=I ** -0.5))
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
    c1, s1, c1t, s1t, v1, g1, v1t, g1t = weights(moe, W1)
    c2, s2, c2t, s2t, v2, g2, v2t, g2t = weights(moe, W2)
    n = T * k

    # forward
    total, y, y8 = moe.moe_rms_norm(attn, nw, x, EPS, fp8=True)
    idx, w = moe.moe_route_scored(logits, None, k, 1, 1, "softmax", True, False, 1.0)
    L = moe.moe_dispatch_layout(idx, E, 1)
    off, pos = L["expert_offsets"], L["pos"]
    send8 = permute8(moe, y8, pos, E)
    z = torch.empty(n, 2 * I, dtype=torch.bfloat16, device=DEV)
    h, h8 = moe.moe_expert_product_fp8(send8, off, c1, s1, act="silu", gated=True, fp8=True, pre=z)
    o, _ = moe.moe_expert_product_fp8(h8, off, c2, s2)
    out = moe.moe_combine_reduce(o, pos, w, residual=total)
    # backward
    gy, gw = moe.moe_combine_backward(grad, o, pos, w)
    gy8 = rows8(moe, gy)
    gz, gz8 = moe.moe_expert_product_fp8_dgrad(gy8, off, c2t, s2t, z, "silu", True, fp8=True)
    gsend, _ = moe.moe_expert_product_fp8_dgrad(gz8, off, c1t, s1t)
    send = moe.moe_dispatch_permute(y, pos, E)
    gW2 = moe.moe_expert_product_wgrad(gy, h, off, torch.empty(E, H, I, device=DEV))
    gW1 = moe.moe_expert_product_wgrad(gz, send, off, torch.empty(E, 2 * I, H, device=DEV))
    gn = moe.moe_combine_reduce(gsend, pos, torch.ones(T, k, device=DEV))
    gx, gnw = moe.moe_rms_norm_backward(gn, total, nw, EPS, grad_total=grad)
    torch.cuda.synchronize()

    f = off.cpu().numpy()
    p = pos.cpu().numpy()
    assert int(f[-1]) == n and sorted(p.ravel().tolist()) == list(range(n))
    assert torch.equal(total, (x.float() + attn.float()).bfloat16())
    eps = np.float64(np.float32(EPS))
    v, e = f8.norm(values(total), values(nw), eps)
    assert_rows(y, v, e, T, "y")
    f8.assert_rows8(y8, v, e, T, "y8")
    a = send8.cpu().numpy()
    assert (a[p] == y8.cpu().numpy()[:, None]).all()
    wy, wz, ez, ey = f8.product(f8.decode_rows(a, H), f8.rows_largest(a, H), f, v1, g1, None, None, "silu", True)
    assert_rows(z, wz, ez, n, "z"), assert_rows(h, wy, ey, n, "h"), f8.assert_rows8(h8, wy, ey, n, "h8")
    a = h8.cpu().numpy()
    wy, _, _, ey = f8.product(f8.decode_rows(a, I), f8.rows_largest(a, I), f, v2, g2)
    assert_rows(o, wy, ey, n, "o")
    cw, co, cg = values(w), values(o)[p], values(grad)
    mag = (np.abs(cw)[:, :, None] * np.abs(co)).sum(1) + np.abs(values(total))
    assert_rows(out, (cw[:, :, None] * co).sum(1) + values(total), (k + 4) * f8.U * mag, T, "out")
    wgy, wgw = ref.combine_backward(cg, values(o), p, cw)
    assert_rows(gy, wgy, 2 * f8.U * np.abs(wgy), n, "gy")
    near32(gw, wgw, 2 * H * f8.U * (np.abs(co) * np.abs(cg)[:, None]).sum(2), "gw")
    a = gy8.cpu().numpy()
    wg, eg = f8.dgrad(f8.decode_rows(a, H), f8.rows_largest(a, H), f, v2t, g2t, values(z), "silu", True)
    assert_rows(gz, wg, eg, n, "gz"), f8.assert_rows8(gz8, wg, eg, n, "gz8")
    a = gz8.cpu().numpy()
    wg, eg = f8.dgrad(f8.decode_rows(a, 2 * I), f8.rows_largest(a, 2 * I), f, v1t, g1t)
    assert_rows(gsend, wg, eg, n, "gsend")
    for got, a, b in ((gW2, gy, h), (gW1, gz, send)):
        vW, _, eW, _ = ref.wgrad(values(a), values(b), f, E)
        assert (np.abs(values(got) - vW) <= eW + 2.0 ** -126).all()
    cs = values(gsend)[p]
    assert_rows(gn, cs.sum(1), (k + 4) * f8.U * np.abs(cs).sum(1), T, "gn")
    wx, ww, ex, ew = f8.norm_backward(values(gn), values(total), values(nw), eps, cg)
    assert_rows(gx, wx, ex, T, "gx"), near32(gnw, ww, ew, "gnw")


@pytest.mark.parametrize("T", [1, 24])
def test_block_captured(moe, T):
    """Replays on inputs written after the capture give the eager calls' bits, and two
    graphs of the same block with buffers of their own replay on two streams at once."""
    H, I, E, k = 512, 256, 8, 4
    rng = np.random.default_rng(T)
    print("[case] captured", T, flush=True)
    nw = up(bf16(rng, H))
    c1, s1, _, _ = moe.moe_fp8_quantize_weights(up(bf16(rng, E, 2 * I, H, scale=H ** -0.5)))
    c2, s2, _, _ = moe.moe_fp8_quantize_weights(up(bf16(rng, E, H, I, scale=I ** -0.5)))

    def block(x, attn, logits):
        total, _, y8 = moe.moe_rms_norm(attn, nw, x, EPS, fp8=True, need_y=False)
        idx, w = moe.moe_route_scored(logits, None, k, 1, 1, "softmax", True, False, 1.0)
        L = moe.moe_dispatch_layout(idx, E, 1)
        off, pos = L["expert_offsets"], L["pos"]
        send8 = permute8(moe, y8, pos, E)
        _, h8 = moe.moe_expert_product_fp8(send8, off, c1, s1, act="silu", gated=True, fp8=True, need_y=False)
        o, _ = moe.moe_expert_product_fp8(h8, off, c2, s2)
        return moe.moe_combine_reduce(o, pos, w, residual=total)

    def fresh():
        logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
        return up(bf16(rng, T, H)), up(bf16(rng, T, H)), logits

    graphs = []
    for _ in range(2):
        inputs = fresh()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            block(*inputs)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            out = block(*inputs)
        graphs.append((g, stream, inputs, out))
    for _ in range(4):
        want = []
        for _, _, inputs, _ in graphs:
            new = fresh()
            for a, b in zip(inputs, new):
                a.copy_(b)
            want.append(block(*new))
        torch.cuda.synchronize()
        for g, stream, _, _ in graphs:
            with torch.cuda.stream(stream):
                g.replay()
        torch.cuda.synchronize()
        for (_, _, _, out), y in zip(graphs, want):
            assert torch.equal(out.view(torch.int16), y.view(torch.int16))
