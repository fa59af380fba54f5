"""The gradients of the two projections, d_gate = grad_h up act'(gate) and d_up = grad_h
act(gate), which the gradients' products take as sums of two values of the operands' type
each: held to bounds far below one rounding of them, with the infinities of the other
factors, at the largest magnitudes, and rounded once where the caller asks for that."""
import pytest

import dense_ref as ref
from helpers import say
from test_gpu_dense_products import dtype_of, vjp_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import torch
    assert torch.cuda.is_available(), "GPU test without a GPU"
    from trellis_coded_weight_amd import api as a
    return a


def bounds(x, wg, wu, gate, up, gh, name):
    """[(gradient, bound)] for x, wg, wu.  A slope's binary32 arithmetic is within 256 U of its
    terms (dense_ref); its two parts lose at most half a step of the second, which is itself at
    most a step of the first: 2^-7 2^-8 of it in bf16, 2^-10 2^-11 and half the smallest
    subnormal in fp16.  Their signs are the slope's, so the terms' magnitudes add up to its
    own; the sums have two terms a slope."""
    import torch
    X, G, W, H = x.double(), wg.double(), wu.double(), gh.double()
    a, d = ref.act(gate.double(), name)
    dg, du = H * up.double() * d, H * a
    rel, tiny = (2.0 ** -15, 0.0) if x.dtype == torch.bfloat16 else (2.0 ** -21, 2.0 ** -25)
    eg = 256 * ref.U * H.abs() * up.double().abs() * 1.13 + rel * dg.abs() + tiny
    eu = 256 * ref.U * du.abs() + rel * du.abs() + tiny
    M, F = gate.shape
    r = dg @ G + du @ W
    mag = dg.abs() @ G.abs() + du.abs() @ W.abs()
    e = eg @ G.abs() + eu @ W.abs() + 2 * (4 * F + 8) * ref.U * mag * 1.01
    out = [(r, e + ref.half_step(x.dtype, r.abs() + e))]
    for s, es in ((dg, eg), (du, eu)):
        r = s.t() @ X
        e = es.t() @ X.abs() + 2 * (2 * M + 8) * ref.U * (s.abs().t() @ X.abs()) * 1.01
        out.append((r, e + ref.half_step(x.dtype, r.abs() + e)))
    return out


# few terms a sum, where the bound is tightest; then several steps and shares of k, odd rows,
# every tile height of grad_x, alone and beside the weight gradients in one launch
SIZES = [(1, 1, 1), (9, 8, 500), (8, 300, 24), (5, 16, 1000), (16, 12, 264), (33, 72, 520), (140, 264, 136),
         (129, 257, 65), (120, 1000, 512), (300, 700, 328), (64, 4096, 256), (4100, 96, 2056)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("M,F,K", SIZES)
def test_slopes_in_two_parts(api, M, F, K, dtype):
    import torch
    args = vjp_inputs(M, F, K, dtype_of(dtype), 1)
    say("gated_vjp, slopes in two parts, %dx%dx%d %s" % (M, F, K, dtype))
    got = api.gated_vjp(*args)
    torch.cuda.synchronize()
    for name, g, (want, e) in zip(("grad_x", "grad_w_gate", "grad_w_up"), got, bounds(*args, "silu")):
        ref.within(g, want, e, name)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "relu", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_slopes_of_each_activation(api, act, dtype):
    import torch
    args = vjp_inputs(12, 24, 264, dtype_of(dtype), 3)
    say("gated_vjp, slopes in two parts, %s %s" % (act, dtype))
    got = api.gated_vjp(*args, activation=act)
    torch.cuda.synchronize()
    for name, g, (want, e) in zip(("grad_x", "grad_w_gate", "grad_w_up"), got, bounds(*args, act)):
        ref.within(g, want, e, name)


def powers(M, F, K, t):
    """Operands whose slopes under relu are powers of two, values of every type: d_gate = grad_h
    up, d_up = grad_h, none of them 0."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def draw(r, c):
        sign = 1 - 2 * torch.randint(0, 2, (r, c), generator=g, device="cuda")
        return (sign * 2.0 ** torch.randint(-3, 4, (r, c), generator=g, device="cuda")).to(t)

    return draw(M, K), draw(F, K), draw(F, K), torch.ones((M, F), dtype=t, device="cuda"), draw(M, F), draw(M, F)


@pytest.mark.parametrize("round_slopes", [False, True])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("M,F,K", [(3, 5, 8), (140, 90, 72), (300, 70, 130)])
def test_infinite_factors(api, M, F, K, dtype, round_slopes):
    """An infinite weight gives its column of grad_x the slopes' infinities, an infinite
    activation its column of the weight gradients; the rest keeps its bits."""
    import torch
    x, wg, wu, gate, up, gh = powers(M, F, K, dtype_of(dtype))
    say("gated_vjp infinite factors %dx%dx%d %s" % (M, F, K, dtype))
    kw = dict(activation="relu", round_slopes=round_slopes)
    clean = api.gated_vjp(x, wg, wu, gate, up, gh, **kw)
    wg[F - 1, 3], x[M - 1, 2] = float("inf"), float("-inf")
    gx, gwg, gwu = api.gated_vjp(x, wg, wu, gate, up, gh, **kw)
    torch.cuda.synchronize()
    inf = float("inf")
    assert torch.equal(gx[:, 3].float(), inf * (gh * up)[:, F - 1].float().sign())
    assert torch.equal(gwg[:, 2].float(), -inf * (gh * up)[M - 1].float().sign())
    assert torch.equal(gwu[:, 2].float(), -inf * gh[M - 1].float().sign())
    for a, b, col in ((gx, clean[0], 3), (gwg, clean[1], 2), (gwu, clean[2], 2)):
        keep = [i for i in range(K) if i != col]
        assert torch.equal(a[:, keep], b[:, keep])


@pytest.mark.parametrize("M,F,K", [(1, 1, 8), (130, 40, 64)])
def test_slopes_past_the_type(api, M, F, K):
    """fp16 slopes of 100000 stay finite in two parts (65504 is fp16's largest value) and give
    their gradients; rounded they are infinite."""
    import torch
    t = torch.float16

    def full(r, c, v):
        return torch.full((r, c), v, dtype=t, device="cuda")

    args = (full(M, K, 2.0 ** -9), full(F, K, 2.0 ** -9), full(F, K, 2.0 ** -9), full(M, F, 1.0), full(M, F, 100.0),
            full(M, F, 1000.0))
    say("gated_vjp slopes past fp16 %dx%dx%d" % (M, F, K))
    got = api.gated_vjp(*args, activation="relu")
    rounded = api.gated_vjp(*args, activation="relu", round_slopes=True)
    torch.cuda.synchronize()
    for name, g, (want, e) in zip(("grad_x", "grad_w_gate", "grad_w_up"), got, bounds(*args, "relu")):
        ref.within(g, want, e, name)
    assert bool(torch.isinf(rounded[0]).all()) and bool(torch.isinf(rounded[1]).all())
    assert torch.equal(rounded[2], got[2])


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("M,F,K", [(1, 1, 1), (9, 8, 500), (140, 264, 136), (129, 257, 65), (64, 4096, 256),
                                   (4100, 96, 2056)])
def test_rounded_slopes(api, M, F, K, dtype):
    """One rounding of each slope on request, in the same workspace, either half alone too, and
    captured in a graph."""
    import torch
    from test_gpu_graphs import capture
    args = vjp_inputs(M, F, K, dtype_of(dtype), 1)
    ws = api.gated_vjp_workspace(M, F, K)
    ws.fill_(0xFF)
    say("gated_vjp rounded slopes %dx%dx%d %s" % (M, F, K, dtype))
    got = api.gated_vjp(*args, round_slopes=True, workspace=ws)
    gx, _, _ = api.gated_vjp(*args, round_slopes=True, want_w=False)
    _, gg, gu = api.gated_vjp(*args, round_slopes=True, want_x=False)
    graph, out = capture(lambda: api.gated_vjp(*args, round_slopes=True))
    graph.replay()
    torch.cuda.synchronize()
    for name, g, (want, e) in zip(("grad_x", "grad_w_gate", "grad_w_up"), got, ref.gated_vjp(*args, "silu")):
        ref.within(g, want, e, name)
    for a, b, c in zip(got, (gx, gg, gu), out):
        assert torch.equal(a, b) and torch.equal(a, c)
