"""relu's gradients against central differences of the loss, for all three inputs: gates of 0,
where the loss has a kink, get no upstream gradient, so every direction may be compared."""
import pytest

import dense_ref as ref
from helpers import say
from test_gpu_dense_products import gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_relu_gradients_against_differences(seed):
    """Inputs whose projections are exact in 16 bits.  Along a direction v the loss is a sum of
    grad_h (gate + t dgate) (up + t dup) over the gates that are on: quadratic in t as long as
    none of them changes sign, so its central difference is its slope.  A nonzero gate is an
    eighth at least, and t (2^-13) times the direction's change of it, some tens, stays below.
    Left are the gradients' own bounds along the direction and the rounding of two losses in 64
    bits, 2^-50 of their terms over the step."""
    import torch
    from trellis_coded_weight_amd import api
    t = torch.bfloat16
    M, F, K = 5, 24, 8
    g = gen(seed)
    x = torch.randint(-1, 2, (M, K), generator=g, device="cuda").to(t)
    wg, wu = (torch.randint(-4, 5, (F, K), generator=g, device="cuda").div(8).to(t) for _ in range(2))
    gh = torch.randint(-4, 5, (M, F), generator=g, device="cuda").div(4).to(t)
    say("relu gradients against differences, seed %d" % seed)
    _, gate, up = api.gated(x, wg, wu, activation="relu", save=True)
    assert torch.equal(gate.double(), x.double() @ wg.double().t())
    gh[gate == 0] = 0
    assert int((gh != 0).sum()) > M * F // 2
    grads = api.gated_vjp(x, wg, wu, gate, up, gh, activation="relu")
    torch.cuda.synchronize()
    bounds = ref.gated_vjp(x, wg, wu, gate, up, gh, "relu")
    base = [x.double(), wg.double(), wu.double()]
    step = 2.0 ** -13

    def loss(X, G, W):
        terms = gh.double() * (X @ G.t()).clamp(min=0) * (X @ W.t())
        return terms.sum(), terms.abs().sum()

    for i, name in enumerate(("grad_x", "grad_w_gate", "grad_w_up")):
        v = torch.randn(base[i].shape, generator=g, device="cuda", dtype=torch.float64)
        change = v @ base[1].t() if i == 0 else base[0] @ v.t()
        assert float(change.abs().max()) * step < 1 / 8
        hi, lo = list(base), list(base)
        hi[i], lo[i] = base[i] + step * v, base[i] - step * v
        (a, size), (b, _) = loss(*hi), loss(*lo)
        want, got = float((a - b) / (2 * step)), float((grads[i].double() * v).sum())
        tol = float((bounds[i][1] * v.abs()).sum()) + 2.0 ** -50 * float(size) / step
        assert tol < 0.05 * float((grads[i].double() * v).abs().sum()), (name, tol)    # it says something
        assert abs(got - want) <= tol, (name, got, want, tol)
