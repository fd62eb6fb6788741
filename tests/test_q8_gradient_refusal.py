"""The packed operators refuse a gradient wherever one could be lost: in traced
graphs, under functorch and in forward mode, as in an eager call.  Where no
gradient is asked for, the same calls run and give the eager result."""
import pytest
import torch
import torch.autograd.forward_ad as fwad

from test_q8_cpu import packed_operator_calls

F = pytest.importorskip("dora_fine_tuning_amd.torch_ops")
MATCH = "no gradient of its own"


def calls(dtype=torch.float32, device="cpu"):
    """(operator, arguments, positions of the floating arguments a user could differentiate)."""
    for op, args, where in packed_operator_calls(device, dtype):
        yield op, args, [i for i in where if args[i].dtype != torch.float8_e4m3fn]


def total(out):
    out = out if isinstance(out, tuple) else (out,)
    return sum(t.float().nan_to_num().sum() for t in out)


@pytest.mark.parametrize("backend", ["eager", "aot_eager", "inductor"])
def test_refused_when_compiled(backend):
    for op, args, where in calls():
        for i in where:
            torch._dynamo.reset()

            def f(x):
                return total(op(*args[:i], x, *args[i + 1:])) + x.sum()

            with pytest.raises(RuntimeError, match=MATCH):
                torch.compile(f, backend=backend, fullgraph=True)(args[i].detach().requires_grad_())


def test_compiled_without_a_gradient():
    x, W = torch.randn(5, 200), torch.randn(140, 200)
    wq, we = F.q8_pack_weight(W)

    def product(x):
        return F.q8_linear(*F.q8_pack(x), wq, we, 140, torch.float32)

    def detached(x):
        return product(x.detach()).sum() + x.sum()

    def no_grad(x):
        with torch.no_grad():
            y = product(x)
        return y.sum() + x.sum()

    for f in (detached, no_grad):
        for backend in ("aot_eager", "inductor"):
            torch._dynamo.reset()
            v = x.clone().requires_grad_()
            g, = torch.autograd.grad(torch.compile(f, backend=backend, fullgraph=True)(v), v)
            assert torch.equal(g, torch.ones_like(x))
    torch._dynamo.reset()
    assert torch.equal(torch.compile(product, backend="aot_eager", fullgraph=True)(x), product(x))


def test_refused_when_traced_for_autograd():
    from torch._functorch.aot_autograd import aot_function

    for op, args, where in calls():
        for i in where:
            f = lambda x: total(op(*args[:i], x, *args[i + 1:])) + x.sum()
            with pytest.raises(RuntimeError, match=MATCH):
                aot_function(f, lambda m, _: m)(args[i].detach().requires_grad_())


def test_refused_under_functorch_and_in_forward_mode():
    for op, args, where in calls():
        for i in where:
            f = lambda x: total(op(*args[:i], x, *args[i + 1:])) + x.sum()
            x = args[i]
            with pytest.raises(RuntimeError, match=MATCH):
                torch.func.grad(f)(x)
            with pytest.raises(RuntimeError, match=MATCH):
                torch.func.jvp(f, (x,), (x,))
            with fwad.dual_level(), torch.no_grad(), pytest.raises(RuntimeError, match=MATCH):
                f(fwad.make_dual(x, x))
            # the argument stands still: the other term's gradient is the whole one
            assert torch.equal(torch.func.grad(lambda v: f(x) + v.sum())(x), torch.ones_like(x))
            assert torch.equal(torch.func.grad(lambda v: f(v.detach()) + v.sum())(x), torch.ones_like(x))


def test_modes_without_gradients():
    for op, args, where in calls():
        ref = total(op(*args))
        for i in where:
            with_grad = [a.detach().requires_grad_() if j == i else a for j, a in enumerate(args)]
            for mode in (torch.no_grad, torch.inference_mode):
                with mode():
                    assert torch.equal(total(op(*with_grad)), ref)


@pytest.mark.gpu
def test_refused_on_the_gpu():
    for op, args, where in calls(torch.bfloat16, "cuda:0"):
        for i in where:
            torch._dynamo.reset()
            f = lambda x: total(op(*args[:i], x, *args[i + 1:])) + x.sum()
            with pytest.raises(RuntimeError, match=MATCH):
                torch.compile(f, backend="aot_eager", fullgraph=True)(args[i].detach().requires_grad_())
            with pytest.raises(RuntimeError, match=MATCH):
                torch.func.grad(f)(args[i])
            with torch.inference_mode():
                assert torch.equal(f(args[i]), f(args[i]))
