"""gated is not recorded by autograd: inputs that require gradients are refused while it
records, instead of a result that has silently lost them."""
import pytest

from helpers import say
from test_gpu_dense_products import halves

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import torch
    assert torch.cuda.is_available(), "GPU test without a GPU"
    from trellis_coded_weight_amd import api as a
    return a


@pytest.mark.parametrize("which", [0, 1, 2])
def test_gated_refuses_what_autograd_records(api, which):
    import torch
    t = torch.bfloat16
    args = [halves(4, 64, t, 1), halves(24, 64, t, 2, 0.1), halves(24, 64, t, 3, 0.1)]
    say("gated with inputs that require gradients")
    want = api.gated(*args)
    leaves = list(args)
    leaves[which] = args[which].clone().requires_grad_()
    with pytest.raises(ValueError, match="gated_vjp"):
        api.gated(*leaves)
    with pytest.raises(ValueError, match="gated_vjp"):
        api.gated(*leaves, save=True)
    with torch.no_grad():
        assert torch.equal(api.gated(*leaves), want)
    leaves[which] = leaves[which].detach()
    assert torch.equal(api.gated(*leaves), want)


def test_gated_inside_an_autograd_function(api):
    """The way to have both: forward and backward of a torch.autograd.Function, where nothing is
    recorded."""
    import torch
    t = torch.bfloat16

    class Gated(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, wg, wu):
            h, gate, up = api.gated(x, wg, wu, save=True)
            ctx.save_for_backward(x, wg, wu, gate, up)
            return h

        @staticmethod
        def backward(ctx, gh):
            return api.gated_vjp(*ctx.saved_tensors, gh.contiguous())

    args = [halves(5, 64, t, 1), halves(24, 64, t, 2, 0.1), halves(24, 64, t, 3, 0.1)]
    say("gated inside an autograd function")
    leaves = [a.clone().requires_grad_() for a in args]
    h = Gated.apply(*leaves)
    gh = halves(5, 24, t, 4)
    h.backward(gh)
    _, gate, up = api.gated(*args, save=True)
    torch.cuda.synchronize()
    for leaf, g in zip(leaves, api.gated_vjp(*args, gate, up, gh)):
        assert torch.equal(leaf.grad, g)
