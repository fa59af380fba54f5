"""Inputs that require gradients while autograd records: the model operators, which it does not
see, refuse each of them, and take them without recording."""
import pytest

import test_gpu_blocks
import test_gpu_distill
from test_gpu_layer_norm import normal

pytestmark = pytest.mark.gpu


def calls():
    """(function, its arguments, keyword arguments)"""
    import torch
    from trellis_coded_weight_amd import api
    x, gy, w, b = normal(6, 64, seed=1), normal(6, 64, seed=2), normal(64, seed=3), normal(64, seed=4)
    _, mean, rstd = api.layer_norm(x, w, b, save=True)
    z, index, t, gl = test_gpu_distill.inputs(6, 500, 8, "float32")
    lz = torch.logsumexp(t, 1)
    _, stats = api.distill_topk(z, index, t, save=True)
    return [(api.quantize_blocks, (x,), {}), (api.quantize_blocks, (x,), dict(block_rows=128)),
            (api.matmul_fp8, test_gpu_blocks.operands(5, 40, 200), {}), (api.layer_norm, (x, w, b), {}),
            (api.layer_norm_vjp, (x, w, mean, rstd, gy), {}),
            (api.distill_topk, (z, index, t), dict(teacher_log_z=lz, grad_loss=gl)),
            (api.distill_topk_vjp, (z, index, t, stats, gl), {})]


@pytest.mark.parametrize("i", range(7))
def test_inputs_that_require_gradients(i):
    import torch
    f, args, kw = calls()[i]
    plain = f(*args, **kw)
    names = list(range(len(args))) + [k for k, v in kw.items() if isinstance(v, torch.Tensor)]
    for n in names:
        v = args[n] if isinstance(n, int) else kw[n]
        if v.dtype not in (torch.float32, torch.float8_e4m3fn):
            continue
        v = v.detach().requires_grad_()
        a = tuple(v if j == n else u for j, u in enumerate(args))
        k = {j: v if j == n else u for j, u in kw.items()}
        with pytest.raises(ValueError, match="does not record gradients"):
            f(*a, **k)
            pytest.fail("%s took %s" % (f.__name__, n), pytrace=False)
        with torch.no_grad():
            out = f(*a, **k)
        for p, q in zip(plain if isinstance(plain, tuple) else (plain,), out if isinstance(out, tuple) else (out,)):
            assert p.dtype == q.dtype and torch.equal(p.float(), q.float())
    torch.cuda.synchronize()
