"""Layer norm with a bias and no weight: its gradient comes in the bias's own type."""
import pytest

import model_ref as ref
from helpers import say
from test_gpu_layer_norm import check_forward, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,C", [(3, 100), (300, 1500), (2000, 264), (4, 20000)])
@pytest.mark.parametrize("btype", ["float32", None])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_bias_alone(R, C, dtype, btype):
    import torch
    from trellis_coded_weight_amd import api
    x, gy, b = normal(R, C, seed=1, dtype=dtype), normal(R, C, seed=2, dtype=dtype), normal(C, seed=3, dtype=btype or dtype)
    say("layer_norm bias alone %dx%d %s %s" % (R, C, dtype, btype))
    mean, rstd = check_forward(api, x, None, b)
    got = api.layer_norm_vjp(x, None, mean, rstd, gy, weight_dtype=b.dtype)
    plain = api.layer_norm_vjp(x, None, mean, rstd, gy)
    torch.cuda.synchronize()
    one = torch.ones(C, dtype=torch.float64, device="cuda")
    for g, (want, e), t in zip(got, ref.layer_norm_vjp(x, one, mean, rstd, gy, b.dtype), (x.dtype, b.dtype, b.dtype)):
        assert g.dtype == t
        ref.within(g, want, e, "gradient")
    for g, p in zip(got, plain):
        assert p.dtype == x.dtype and torch.equal(g.to(x.dtype), p)


def test_refusals():
    import torch
    from trellis_coded_weight_amd import api
    from trellis_coded_weight_amd._native import QtcqError
    x, w = normal(4, 64, dtype="bfloat16"), normal(64)
    _, mean, rstd = api.layer_norm(x, w, save=True)
    z, index, t = normal(4, 64), torch.zeros(4, 2, dtype=torch.int64, device="cuda"), normal(4, 2)
    _, stats = api.distill_topk(z, index, t, save=True)
    for f in (lambda: api.layer_norm_vjp(x, w, mean, rstd, x, weight_dtype=torch.bfloat16),
              lambda: api.layer_norm_vjp(x, None, mean, rstd, x, weight_dtype=torch.float16),
              lambda: api.layer_norm_vjp(x, None, mean, rstd, x, weight_dtype=torch.int8),
              lambda: api.layer_norm(x, 1.0), lambda: api.layer_norm(x, None, 0.0), lambda: api.layer_norm(x, w, 0.0),
              lambda: api.layer_norm_vjp(x, 1.0, mean, rstd, x),
              lambda: api.distill_topk_vjp(z, index, t, stats.t().contiguous().t(), normal(4))):
        with pytest.raises((ValueError, QtcqError)):
            f()
    torch.cuda.synchronize()
