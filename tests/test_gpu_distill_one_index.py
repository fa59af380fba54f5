"""Distillation whose entries all name one vocabulary index: its gradient takes off the sum of
their p, a sum of up to 1024 values."""
import pytest

from dense_ref import U
from helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [600, 9001, 70000])
@pytest.mark.parametrize("k", [700, 777, 900, 1000, 1023])
def test_sum_of_many_entries(k, V):
    """Equal entries, each p = 1 / k, and q of the index below e^-100: the gradient there is the
    sum of p, 1.  The logarithm of k and its difference from 0 are each off by U ln k at most, 2^x
    by 2 U, the sum's rounding and the scale's product by U each."""
    import math

    import torch
    from trellis_coded_weight_amd import api
    z = torch.zeros(3, V, device="cuda")
    z[:, 5] = -1e4
    index = torch.full((3, k), 5, device="cuda")
    t = torch.full((3, k), 2.5, device="cuda")
    say("distill one index k=%d V=%d" % (k, V))
    loss, grad = api.distill_topk(z, index, t, grad_loss=torch.ones(3, device="cuda"))
    torch.cuda.synchronize()
    assert float((grad[:, 5].double() + 1).abs().max()) <= (2 * math.log(k) + 2 + 2) * U * 1.01
