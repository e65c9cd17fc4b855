"""The layer's calls refuse a stream or a workspace of another GPU, before
anything is launched. Stand-ins take the place of GPU tensors and streams, and
of the library, which must not be reached."""

import types

import pytest
import torch


@pytest.fixture
def moe(monkeypatch):
    import combine_route_topk_amd as moe
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    def never(*a):
        raise AssertionError("the library was called")

    names = [n for n in moe.EXPORTS if n.startswith("moe_expert_product") or "scored" in n or n == "moe_combine_backward"]
    fakes = {n: never for n in names if not n.endswith("_size")}
    real = moe.lib
    monkeypatch.setattr(moe, "lib", types.SimpleNamespace(
        moe_expert_product_wgrad_workspace_size=real.moe_expert_product_wgrad_workspace_size,
        moe_status_string=real.moe_status_string, **fakes))
    return moe


class Tensor:
    """What the binding looks at in a contiguous GPU tensor."""

    is_cuda = True

    def __init__(self, shape, dtype, device=0):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", device)

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000

    def numel(self):
        return self.shape.numel()


BF, F, I = torch.bfloat16, torch.float32, torch.int32


def calls(moe, **kw):
    """Each of the layer's calls on tensors of GPU 0, with outputs given."""
    l, idx, w = Tensor((4, 8), F), Tensor((4, 2), I), Tensor((4, 2), F)
    x, y, off = Tensor((4, 8), BF), Tensor((4, 16), BF), Tensor((3,), I)
    W, V = Tensor((2, 16, 8), BF), Tensor((2, 16, 8), F)
    yield lambda: moe.moe_route_scored(l, None, 2, topk_idx=idx, topk_w=w, **kw)
    yield lambda: moe.moe_route_scored_backward(l, idx, w, grad_logits=Tensor((4, 8), F), **kw)
    yield lambda: moe.moe_combine_backward(x, x, idx, w, Tensor((4, 8), BF), w, **kw)
    yield lambda: moe.moe_expert_product(x, off, W, y=y, **kw)
    yield lambda: moe.moe_expert_product_dgrad(y, off, W, grad_x=x, **kw)
    yield lambda: moe.moe_expert_product_wgrad(y, x, off, V, **kw)


def test_stand_ins_reach_the_library(moe, monkeypatch):
    """Without a fault in the arguments every call gets as far as the library."""
    monkeypatch.setattr(moe, "_stream", lambda s: 0)
    for call in calls(moe):
        with pytest.raises(AssertionError, match="the library was called"):
            call()


def test_stream_of_another_device(moe, monkeypatch):
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0x20000

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: pytest.fail("the other device was made current"))
    for call in calls(moe, stream=Stream()):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call()


def test_workspace_of_another_device(moe, monkeypatch):
    monkeypatch.setattr(moe, "_stream", lambda s: 0)
    y, x, off, V = Tensor((4, 16), BF), Tensor((4, 8), BF), Tensor((3,), I), Tensor((2, 16, 8), F)
    with pytest.raises(ValueError, match="workspace is on cuda:1"):
        moe.moe_expert_product_wgrad(y, x, off, V, workspace=Tensor((4096,), torch.uint8, 1))
    with pytest.raises(AssertionError, match="the library was called"):
        moe.moe_expert_product_wgrad(y, x, off, V, workspace=Tensor((4096,), torch.uint8))
