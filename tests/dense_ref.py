"""Plain 64-bit forms of the dense operators and the error bounds their tests hold the
kernels to.  U is the unit roundoff of binary32; a sum of n terms in binary32, in any
order and with each addition inside a matrix instruction allowed one unit in the last
place, is within 2 (n + 8) U sum |terms| of the exact sum to first order; a result rounded
once to type t is off by at most eps(t) / 2 relative (and 2^-25 absolute in fp16, half its
smallest subnormal).  Elementary functions: the activations and their slopes take an exp or
erfc of a rounded argument, a few units each times the argument (below 40 for the
inputs used here), 256 U of the value altogether."""
import math

import torch

U = 2.0 ** -24


def half_step(dtype, v):
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -126
    return torch.finfo(dtype).eps / 2 * v.abs() * (1 + 2.0 ** -7) + tiny


def act(g, name):
    """act(g) and act'(g) in 64 bits."""
    if name == "relu":
        return g.clamp(min=0), (g > 0).double()
    if name == "gelu":
        c = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        a, b = math.sqrt(2 / math.pi), 0.044715
        t = torch.tanh(a * (g + b * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * a * (1 + 3 * b * g * g)
    s = torch.sigmoid(g)
    if name == "sigmoid":
        return s, s * (1 - s)
    return g * s, s * (1 + g * (1 - s))


def gated(x, wg, wu, name):
    """(h, its bound, gate, up, their bounds) for operands of a 16-bit type."""
    X, G, W = x.double(), wg.double(), wu.double()
    n = X.shape[1]
    g, u = X @ G.t(), X @ W.t()
    eg, eu = (2 * (n + 8) * U * (X.abs() @ A.abs().t()) for A in (G, W))
    a, _ = act(g, name)
    h = a * u
    # |act'| <= 1.13 for every activation
    e = 1.13 * eg * (u.abs() + eu) + a.abs() * eu + 256 * U * h.abs()
    return h, e + half_step(x.dtype, h.abs() + e), g, u, eg + half_step(x.dtype, g), eu + half_step(x.dtype, u)


def gated_vjp(x, wg, wu, gate, up, gh, name):
    """[(gradient, bound)] for x, wg, wu, from the saved gate and up as they are."""
    X, G, W, H = x.double(), wg.double(), wu.double(), gh.double()
    a, d = act(gate.double(), name)
    dg, du = H * up.double() * d, H * a
    slope = H.abs() * up.double().abs() * 1.13
    # slopes in binary32 (the derivative of an activation has terms of up to its argument's
    # size that cancel: 256 U of 1.13), then rounded to the operands' type
    eg = 256 * U * slope + half_step(x.dtype, dg)
    eu = 256 * U * du.abs() + half_step(x.dtype, du)
    M, F = gate.shape
    out = []
    r = dg @ G + du @ W
    mag = dg.abs() @ G.abs() + du.abs() @ W.abs()
    e = eg @ G.abs() + eu @ W.abs() + 2 * (2 * F + 8) * U * mag * 1.01
    out.append((r, e + half_step(x.dtype, r.abs() + e)))
    for s, es in ((dg, eg), (du, eu)):
        r = s.t() @ X
        e = es.t() @ X.abs() + 2 * (M + 8) * U * (s.abs().t() @ X.abs()) * 1.01
        out.append((r, e + half_step(x.dtype, r.abs() + e)))
    return out


def quantize(v):
    """Rows of the 64-bit matrix v (finite) as (q int8, scale float32), by definition."""
    scale = (v.abs().amax(1) / 127).float() if v.shape[1] else torch.zeros(v.shape[0], device=v.device)
    s = scale.double()[:, None]
    q = torch.where(s > 0, v / torch.where(s > 0, s, 1.0), 0.0)
    return torch.round(q).clamp(-127, 127).to(torch.int8), scale


def within(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    if bool(bad.any()):
        i = bad.nonzero()[0].tolist()
        raise AssertionError("%s: %d of %d off, first at %s: %r, not %r within %.3g" % (
            what, int(bad.sum()), bad.numel(), i, float(got[tuple(i)]), float(want[tuple(i)]),
            float(bound[tuple(i)])))
