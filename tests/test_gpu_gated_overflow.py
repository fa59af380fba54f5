"""fp16 projections past the type's range: the forward pass works on their binary32 values and
saves infinities, and the gradients take the activations' limits there."""
import pytest

import dense_ref as ref
from helpers import say
from test_gpu_dense_products import ACTS
from test_gpu_gated_slopes import bounds

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import torch
    assert torch.cuda.is_available(), "GPU test without a GPU"
    from trellis_coded_weight_amd import api as a
    return a


def inputs16(M, F, K, gates):
    """Tokens around 100, gate weights that make the first gates the given values, and small up
    weights, so that h = act(gate) up stays in fp16's range."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    x = (100 + torch.randint(-3, 4, (M, K), generator=g, device="cuda")).half()
    wg = (torch.randn(F, K, generator=g, device="cuda") * 0.01).half()
    wu = (torch.randn(F, K, generator=g, device="cuda") * 1e-4).half()
    for i, v in enumerate(gates):
        wg[i] = v / 100 / K
    gh = torch.randn(M, F, generator=g, device="cuda").half()
    return x, wg, wu, gh


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,F,K", [(2, 6, 8), (140, 70, 64), (300, 90, 65)])
def test_gates_past_the_type(api, M, F, K, act):
    import torch
    inf = float("inf")
    x, wg, wu, gh = inputs16(M, F, K, [80000.0, -80000.0])
    say("gated fp16 gates past 65504, %s %dx%dx%d" % (act, M, F, K))
    h, gate, up = api.gated(x, wg, wu, activation=act, save=True)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(h).all()) and bool((gate[:, 0] == inf).all()) and bool((gate[:, 1] == -inf).all())
    # the true gates are so far out that act' is its limit: 1 and 0, act(-80000) is 0
    true = gate.double().clamp(-80000, 80000)
    gx, gwg, gwu = api.gated_vjp(x, wg, wu, gate, up, gh, activation=act)
    torch.cuda.synchronize()
    _, (w1, e1), (w2, e2) = bounds(x, wg, wu, true, up, gh, act)
    ref.within(gwg, w1, e1, "grad_w_gate")
    if act == "sigmoid":
        ref.within(gwu, w2, e2, "grad_w_up")
    else:
        # d_up = grad_h act(gate) is infinite for the gate saved as +inf, and nothing else is
        ref.within(gwu[1:], w2[1:], e2[1:], "grad_w_up")
        assert not bool(torch.isfinite(gwu[0]).any())
    # without the column of +inf everything is finite
    part = [t[:, 1:] for t in (gate, up, gh)]
    gx, gwg, gwu = api.gated_vjp(x, wg[1:], wu[1:], *part, activation=act)
    torch.cuda.synchronize()
    want = bounds(x, wg[1:], wu[1:], true[:, 1:], up[:, 1:], gh[:, 1:], act)
    for name, got, (w, e) in zip(("grad_x", "grad_w_gate", "grad_w_up"), (gx, gwg, gwu), want):
        ref.within(got, w, e, name)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_slopes_at_infinite_gates(api, act, dtype):
    """One token and ones: the limits themselves, in both types; NaN stays NaN."""
    import torch
    t = getattr(torch, dtype)
    inf = float("inf")
    gate = torch.tensor([[inf, -inf, 0.5, float("nan")]], dtype=t, device="cuda")
    one = torch.ones((1, 8), dtype=t, device="cuda")
    w = torch.ones((4, 8), dtype=t, device="cuda")
    say("slopes at infinite gates %s %s" % (act, dtype))
    _, gg, gu = api.gated_vjp(one, w, w, gate, one[:, :4].contiguous(), one[:, :4].contiguous(), activation=act)
    torch.cuda.synchronize()
    top = 1.0 if act == "sigmoid" else inf
    assert gg[0].tolist() == [0.0 if act == "sigmoid" else 1.0] * 8 and gg[1].tolist() == [0.0] * 8
    assert gu[0].tolist() == [top] * 8 and gu[1].tolist() == [0.0] * 8
    assert bool(torch.isfinite(gg[2]).all()) and bool(torch.isnan(gg[3]).all()) and bool(torch.isnan(gu[3]).all())


@pytest.mark.parametrize("round_slopes", [False, True])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_zero_factors_beside_infinite_projections(api, act, dtype, round_slopes):
    """Masked tokens (grad_h 0) and closed gates (act' 0) whose saved projections are infinite
    add nothing: the weight gradients are those of the other tokens, bit for bit."""
    import torch
    t = getattr(torch, dtype)
    inf = float("inf")
    M, F, K = 9, 72, 40
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def draw(r, c):
        return torch.randn(r, c, generator=g, device="cuda").to(t)

    x, wg, wu, gate, up, gh = draw(M, K), draw(F, K), draw(F, K), draw(M, F), draw(M, F), draw(M, F)
    gh[2] = 0                                              # a masked token
    gate[4] = -1000                                        # a token whose gates are all closed
    say("zero factors beside infinite projections %s %s" % (act, dtype))
    kw = dict(activation=act, round_slopes=round_slopes)
    clean = api.gated_vjp(x, wg, wu, gate, up, gh, **kw)
    gate[2, ::2], gate[2, 1::2], up[2, ::3], up[2, 1::3] = inf, -inf, inf, -inf
    up[4, ::2], up[4, 1::2] = -inf, inf
    got = api.gated_vjp(x, wg, wu, gate, up, gh, **kw)
    torch.cuda.synchronize()
    for a, b in zip(got, clean):
        assert bool(torch.isfinite(b).all()) and torch.equal(a, b)
    # NaN is not taken away, and neither is an infinite upstream gradient
    up[4, 5] = float("nan")
    gh[2, 7] = inf
    gx, gwg, gwu = api.gated_vjp(x, wg, wu, gate, up, gh, **kw)
    torch.cuda.synchronize()
    assert bool(torch.isnan(gx[4]).all()) and bool(torch.isnan(gwg[5]).all())
    assert not bool(torch.isfinite(gwg[7]).any()) and not bool(torch.isfinite(gx[2]).any())
