"""A function behind the layer that gives no gradient of its input: the layer's
leaves get zeros, and what reaches them on other paths, as from the 16-bit layer."""
import pytest
import torch

F = pytest.importorskip("dora_fine_tuning_amd.torch_ops")


class Drop(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x):
        return x.clone()

    @staticmethod
    def backward(ctx, dy):
        return None


def check(device, dtype):
    for kw in (dict(), dict(q8_checkpoint=True), dict(q8_weight=True), dict(q8_weight=True, detach_norm=False)):
        layer = F.DoRALinear(200, 152, 8, dtype=dtype, device=device, **kw)
        x = torch.randn(5, 200, device=device).to(dtype).requires_grad_()
        (Drop.apply(layer(x)).sum() + x.sum()).backward()
        assert torch.equal(x.grad, torch.ones_like(x)), kw
        for p in (layer.lora_A, layer.lora_B, layer.magnitude):
            assert torch.equal(p.grad, torch.zeros_like(p)), kw


def test_undefined_gradient_eager():
    check("cpu", torch.float32)
    check("cpu", torch.bfloat16)


@pytest.mark.gpu
def test_undefined_gradient():
    check("cuda:0", torch.bfloat16)
    check("cuda:0", torch.float16)
