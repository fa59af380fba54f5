"""The activations and their slopes over gates far from 0, where one side of them is tiny: each
value on its own, held to a bound relative to the terms of its formula."""
import math

import pytest

import dense_ref as ref
from helpers import say
from test_gpu_dense_products import ACTS, dtype_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import torch
    assert torch.cuda.is_available(), "GPU test without a GPU"
    from trellis_coded_weight_amd import api as a
    return a


def terms(g, name):
    """act(g), act'(g) and the sum of the magnitudes of act's terms, in 64 bits without
    cancellation."""
    import torch
    if name == "relu":
        return g.clamp(min=0), (g > 0).double(), (g > 0).double()
    if name == "gelu":
        c = 0.5 * torch.special.erfc(-g / math.sqrt(2))
        p = g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        return g * c, c + p, c + p.abs()
    if name == "gelu_tanh":
        k = math.sqrt(8 / math.pi)
        z = k * (g + 0.044715 * g ** 3)
        s = torch.sigmoid(z)
        p = g * s * torch.sigmoid(-z) * k * (1 + 3 * 0.044715 * g * g)
        return g * s, s + p, s + p.abs()
    s, t = torch.sigmoid(g), torch.sigmoid(-g)
    if name == "sigmoid":
        return s, s * t, s * t
    return g * s, s + g * s * t, s + (g * s * t).abs()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_slopes_of_large_gates(api, act, dtype):
    """One token and inputs of 1: grad_w_gate is act'(gate) and grad_w_up is act(gate), rounded
    once from binary32.  An exponential's argument is rounded to a few U times its size: up to
    88 here (gelu's g^2 / 2, and the tanh form's z, end where the result leaves binary32's
    normal range, the half step's absolute part), so 256 U of the terms; the parts the slopes
    are held in lose 2^-15 (bf16) or 2^-21 and 2^-25 absolute (fp16)."""
    import torch
    t = dtype_of(dtype)
    gate = torch.cat([torch.linspace(-30, 30, 961, device="cuda"),
                      torch.tensor([-1e4, -300.0, -89.0, -60.0, 60.0, 89.0, 300.0, 1e4], device="cuda")]).to(t)[None]
    F, K = gate.shape[1], 8
    one = torch.ones((1, F), dtype=t, device="cuda")
    w = torch.ones((F, K), dtype=t, device="cuda")
    say("slopes of large gates %s %s" % (act, dtype))
    _, gg, gu = api.gated_vjp(one[:, :K].contiguous(), w, w, gate, one, one, activation=act)
    torch.cuda.synchronize()
    a, d, size = terms(gate[0].double(), act)
    rel, tiny = (2.0 ** -15, 0.0) if t == torch.bfloat16 else (2.0 ** -21, 2.0 ** -25)
    for name, got, want, mag in (("act'", gg, d, size), ("act", gu, a, a.abs())):
        e = (256 * ref.U * mag + rel * want.abs() + tiny)
        e = e + ref.half_step(t, want.abs() + e)
        ref.within(got, want[:, None].expand(F, K), e[:, None].expand(F, K), name)
