"""Distillation with the teacher's log-normaliser given: far logits and low temperatures.  The
entries' p in the gradient is exp2 of a difference of what is left of the teacher's logit and of
the normaliser once the row's largest logit is off both, each rounded to binary32."""
import pytest

import test_gpu_distill
from dense_ref import U
from helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [600, 9001, 70000])
@pytest.mark.parametrize("far,tau", [(25.0, 0.5), (300.0, 0.5), (-4000.0, 1.0), (30000.0, 4.0)])
def test_entries_far_from_zero(V, far, tau):
    """Logits of the model so low at the entries that their gradient is the entry's p alone, which
    is held to 64 bits.  In x = (t - max t) log2 e / T the difference, the constant and the product
    are each rounded (T, a power of two, costs nothing), tls = log_z log2 e - max t log2 e / T once,
    their difference once more, each by at most U of itself, and 2^x is within one unit, 2 U.  ln 2
    times an error of the exponent is one of p, relative.  Scale and product cost 2 U."""
    import torch
    from trellis_coded_weight_amd import api
    z, index, t, gl = test_gpu_distill.inputs(6, V, 24, "float32", seed=3)
    index = torch.arange(24, device="cuda").repeat(6, 1) * 11
    index[2, 5:] = -1
    z.scatter_(1, index.clamp(min=0), -1e4)
    t = (t + far).float()
    T = t.double() / tau
    there = index >= 0
    lz = (torch.logsumexp(T.masked_fill(~there, -torch.inf), 1) + 0.25).float()
    say("distill given sum far=%g tau=%g V=%d" % (far, tau, V))
    loss, grad = api.distill_topk(z, index, t, temperature=tau, teacher_log_z=lz, grad_loss=gl)
    saved, stats = api.distill_topk(z, index, t, temperature=tau, teacher_log_z=lz, save=True)
    late = api.distill_topk_vjp(z, index, t, stats, gl, temperature=tau)
    torch.cuda.synchronize()
    assert torch.equal(saved, loss) and torch.equal(late, grad)
    top = T.masked_fill(~there, -torch.inf).amax(1, keepdim=True)
    x, n = (T - top).abs(), (lz.double()[:, None] - top).abs()
    p = torch.exp(T - lz.double()[:, None])
    want = -(gl.double() / tau)[:, None] * p
    bound = want.abs() * (3 * x + n + (x + n) + 8) * U * 1.01
    got = grad.double().gather(1, index.clamp(min=0))
    off = ((got - want).abs() > bound) & there
    assert not bool(off.any()), (off.nonzero()[:4].tolist(), float((got - want).abs().div(want.abs())[there].max()))


def test_rows_sum_to_zero():
    """q is 1 at one element, which no entry names, so a token's gradient sums to scale (mass -
    sum p), 0 but for roundings: with x as above p is off by (4 x + 2 n + 4) U, and the mean of x
    over 16 entries is at most ln 16; the mass and its product with the scale are 3 U."""
    import torch
    from trellis_coded_weight_amd import api
    z, _, t, gl = test_gpu_distill.inputs(5, 9001, 16, "float32", seed=4)
    z.fill_(-1e4)
    z[:, 0] = 0
    index = 1 + torch.arange(16, device="cuda").repeat(5, 1) * 11
    t = t + 300
    lz = (torch.logsumexp(t.double() / 0.5, 1) + 0.25).float()
    say("distill given sum: rows sum to zero")
    _, grad = api.distill_topk(z, index, t, temperature=0.5, teacher_log_z=lz, grad_loss=torch.ones_like(gl))
    torch.cuda.synchronize()
    assert float(grad.double().sum(1).abs().max()) <= (4 * 2.78 + 2 * 0.26 + 4 + 3) * 2 * U


@pytest.mark.parametrize("V", [600, 70000])
def test_teachers_that_are_not_finite(V):
    """A teacher's logit of -infinity has no share, whatever the normaliser; a row of them, or of
    padding, has none at all; an infinite or NaN one reaches its own row alone."""
    import torch
    from trellis_coded_weight_amd import api
    z, index, t, gl = test_gpu_distill.inputs(8, V, 10, "float32")
    index = torch.arange(10, device="cuda").repeat(8, 1) * 7
    lz = torch.logsumexp(t, 1) + 0.25
    t[0, 3:], t[1], index[2] = -float("inf"), -float("inf"), -1
    lz[2] = float("nan")
    clean, grad0 = api.distill_topk(z, index, t, teacher_log_z=lz, grad_loss=gl)
    t[4, 2], t[5, 1] = float("inf"), float("nan")
    say("distill given sum, teachers not finite V=%d" % V)
    loss, grad = api.distill_topk(z, index, t, teacher_log_z=lz, grad_loss=gl)
    torch.cuda.synchronize()
    for r in (1, 2):
        assert float(loss[r]) == 0 and not bool(grad[r].any()), r
    for r in (4, 5):
        assert not bool(torch.isfinite(loss[r])), r
    for r in (0, 1, 2, 3, 6, 7):
        assert bool(torch.isfinite(loss[r])) and torch.equal(loss[r], clean[r]) and torch.equal(grad[r], grad0[r]), r
