"""The weights' gradients of few rows are added by twos behind the rows of a thread (128 threads
for the rows of a column), not one after the other: equal values show it."""
import pytest

from dense_ref import U
from helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("C", [1, 40, 333, 2731, 8192])
@pytest.mark.parametrize("R", [1, 2, 128, 256, 384, 512])
def test_equal_rows(R, C):
    """Every row gives v of 24 bits to each sum.  Sums of two equal values are exact, and of 384
    rows a thread adds three, with one rounding: 2 v + v.  Of 512 it adds four: v on the rounded
    3 v is 4 v again, as 4 v lies nearest, or on the even side of a tie."""
    import torch
    from trellis_coded_weight_amd import api
    g = torch.Generator(device="cuda")
    g.manual_seed(R + C)
    v = torch.rand(C, generator=g, device="cuda") + 0.5
    one = torch.ones(R, C, device="cuda")
    say("layer_norm_vjp equal rows %dx%d" % (R, C))
    _, gw, gb = api.layer_norm_vjp(one, None, torch.zeros(R, device="cuda"), torch.ones(R, device="cuda"), one * v)
    torch.cuda.synchronize()
    want = v.double() * R
    for got in (gw, gb):
        assert bool(((got.double() - want).abs() <= (U * want if R == 384 else 0.0 * want)).all()), (R, C)
