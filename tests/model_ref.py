"""Plain 64-bit forms of the model operators and the error bounds their tests hold the
kernels to.  U is the unit roundoff of binary32.  A thread adds at most 64 + n / 256 of a
row's n values in order, then 6 levels of lanes and at most 16 waves: depth(n) additions on
the way of any value, so a row's sum is within depth(n) U sum |terms| to first order (the
bounds below are a per cent wider).  A sum over rows is within (rows + 40) U sum |terms|.  The
matrix instruction's additions may each be off by one unit in the last place.  A result
rounded once to type t is off by at most half a step of t (dense_ref.half_step)."""
import torch

from dense_ref import U, half_step, within  # noqa: F401

E4M3 = [(-1.0 if b >> 7 else 1.0) * (float("nan") if b & 127 == 127 else (b & 7) * 2.0 ** -9 if b & 120 == 0
                                     else (8 + (b & 7)) * 2.0 ** ((b >> 3 & 15) - 10)) for b in range(256)]


def depth(n):
    return 96 + n / 256


def e4m3(q):
    """The values of a float8_e4m3fn tensor in 64 bits, from its bits."""
    return torch.tensor(E4M3, dtype=torch.float64, device=q.device)[q.contiguous().view(torch.uint8).long()]


def spread(scale, rows, cols, block_rows):
    """Block scales for each element, in 64 bits."""
    return scale.double().repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def quantize_blocks(x, block_rows):
    """(the bits of q, scale) by definition, for any x; bits of NaN blocks are 0."""
    R, C = x.shape
    v = x.double()
    down, wide = -(-R // block_rows), -(-C // 128)
    pad = torch.zeros(down * block_rows, wide * 128, dtype=torch.float64, device=x.device)
    pad[:R, :C] = v.abs()
    top = pad.reshape(down, block_rows, wide, 128).amax((1, 3))      # NaN where there is one
    finite = torch.isfinite(top)
    scale = torch.where(finite, top / 448, float("nan")).float()
    s = spread(scale, R, C, block_rows)
    a = torch.where(s > 0, v.abs() / s, 0.0).clamp(max=448.0)
    points = torch.tensor(E4M3[:127], dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(points, a.contiguous()).clamp(1, 126)
    down_by, up_by = a - points[hi - 1], points[hi] - a
    bits = torch.where((up_by < down_by) | ((up_by == down_by) & (hi % 2 == 0)), hi, hi - 1)
    # the sign stays, of a value rounded to zero too; a block of scale 0 or NaN is all +0
    return torch.where((s > 0) & torch.signbit(v), bits + 128, bits).to(torch.uint8), scale


def group_sums(a, w, sa, sw):
    """What the 8-bit matrix instruction may lose, in 64 bits: it sums 8 neighbours of k at a
    time, each product cut off at 2^-13 of the group's largest power of two (which is at most
    the largest product), 7 of them, and keeps 12 bits of the group's sum: 2^-12 of it."""
    K = a.shape[1]
    pad = -K % 8
    A, W = (torch.nn.functional.pad(e4m3(t).nan_to_num(0), (0, pad)).reshape(t.shape[0], -1, 8) for t in (a, w))
    blocks = torch.arange(A.shape[1], device=a.device) // 16
    ca, cw = sa.double()[:, blocks], sw.double().repeat_interleave(128, 0)[:w.shape[0]][:, blocks]
    cut = 7 * 2.0 ** -13 * (ca * A.abs().amax(2)) @ (cw * W.abs().amax(2)).t()
    kept = torch.zeros_like(cut)
    for g in range(A.shape[1]):
        kept += (ca[:, g:g + 1] * cw[:, g] * (A[:, g] @ W[:, g].t())).abs()
    return cut + 2.0 ** -12 * (kept + cut)


def matmul_fp8(a, sa, w, sw, dtype):
    """(y, its bound); 16-bit results may come from the 8-bit matrix instruction."""
    K, N = a.shape[1], w.shape[0]
    A, W = e4m3(a) * spread(sa, a.shape[0], K, 1), e4m3(w) * spread(sw, N, K, 128)
    y, mag = A @ W.t(), A.abs() @ W.abs().t()
    e = (2 * 136 + -(-K // 128) + 40) * U * mag * 1.01 + 2.0 ** -126 * K
    if dtype != torch.float32:
        e = e + group_sums(a, w, sa, sw)
    return y, e + half_step(dtype, y.abs() + e)


def layer_norm(x, w, b, eps):
    """(y, bound, mean, bound, rstd, bound) for weights in 64 bits."""
    v, n = x.double(), x.shape[1]
    D = depth(n)
    mean = v.mean(1)
    em = D * U * v.abs().mean(1) + 2 * U * mean.abs()
    d = v - mean[:, None]
    var = d.square().mean(1)
    rstd = 1 / torch.sqrt(var + eps)
    # the sum of squares about a mean that is off by em is too large by n em^2
    er = 0.5 * ((D + 4) * U * var + em * em) / (var + eps) + 6 * U
    xh = d * rstd[:, None]
    ex = (em[:, None] + 2 * U * d.abs()) * rstd[:, None] + xh.abs() * er[:, None]
    y = xh * w + b
    e = 1.01 * (ex * w.abs() + 3 * U * ((xh * w).abs() + b.abs()))
    return y, e + half_step(x.dtype, y.abs() + e), mean, 1.01 * em, rstd, 1.01 * rstd * er


def layer_norm_vjp(x, w, mean, rstd, gy, wdtype):
    """[(gradient, bound)] for x, weight and bias, from the mean and rstd as they are."""
    v, g, n, R = x.double(), gy.double(), x.shape[1], x.shape[0]
    D = depth(n)
    rs = rstd.double()[:, None]
    xh = (v - mean.double()[:, None]) * rs
    gw = g * w
    m1, m2 = gw.mean(1, keepdim=True), (gw * xh).mean(1, keepdim=True)
    dx = rs * (gw - m1 - xh * m2)
    e1 = (D + 3) * U * gw.abs().mean(1, keepdim=True)
    e2 = (D + 6) * U * (gw * xh).abs().mean(1, keepdim=True)
    e = 1.01 * rs * (4 * U * gw.abs() + e1 + xh.abs() * e2 + 8 * U * ((xh * m2).abs() + m1.abs()))
    out = [(dx, e + half_step(x.dtype, dx.abs() + e))]
    for t in (g * xh, g):
        r = t.sum(0)
        e = 1.01 * (R + 44) * U * t.abs().sum(0)
        out.append((r, e + half_step(wdtype, r.abs() + e)))
    return out


def distill(z, index, t, tau, log_z=None, grad_loss=None, dtype=None):
    """(loss, its bound, [gradient, its bound]) for finite teachers; z and t in 64 bits."""
    V = z.shape[1]
    z, t = z.double() / tau, t.double() / tau
    there = (index >= 0) & (index < V)
    at = torch.where(there, index, 0).long()
    empty = ~there.any(1, keepdim=True)
    m = z.amax(1, keepdim=True)
    a = torch.where(empty, 0.0, z - torch.where(torch.isfinite(m), m, 0.0))
    e = torch.exp(a)
    s = e.sum(1, keepdim=True)
    log_q = a - torch.log(s)
    masked = torch.where(there, t, -torch.inf)
    total = torch.logsumexp(masked, 1, keepdim=True) if log_z is None else log_z.double()[:, None]
    lp = torch.where(there, t - total, -torch.inf)
    p = torch.where(torch.isneginf(lp), 0.0, torch.exp(lp))
    mass = p.sum(1, keepdim=True)
    picked = log_q.gather(1, at)
    loss = torch.where(p > 0, p * (lp - picked), 0.0).sum(1)
    # the sum of exponentials: each term's argument and exponential, the additions, and the
    # running sum's factors when the maximum rises, whose logs add up to the range of z
    far = torch.where(torch.isfinite(a), a, 0.0).abs().clamp(max=104.0)
    es = U * (depth(V) + 16 + 8 * far.amax(1)) if V else 0.0
    # log p and log q are sums in binary64 of products and of two logarithms of sums, each within
    # 2 U; p is an exp2 of what is behind the point (8 U) of a logarithm that is off by so much
    terms = torch.where(p > 0, p * (lp - picked), 0.0).abs().sum(1)
    bound = 1.01 * (mass[:, 0] * (es + 8 * U) + 16 * U * terms + 4 * U * loss.abs()) + 2.0 ** -120
    if grad_loss is None:
        return loss, bound
    scale = (grad_loss.double() / tau)[:, None]
    q = torch.exp(log_q) * (mass > 0)
    grad = mass * q
    eq = grad * (es[:, None] + U * (24 + 8 * far + 4 * torch.log(s).abs()))
    ep = p * U * (24 + 8 * lp.clamp(min=-104.0).abs() + 8 * total.clamp(-1e4, 1e4).abs())
    back, over = torch.zeros_like(z), torch.zeros_like(z)
    back.scatter_add_(1, at, torch.where(there, p, 0.0))
    over.scatter_add_(1, at, torch.where(there, ep, 0.0))
    eg = 1.01 * scale.abs() * (eq + over + 8 * U * (grad + back)) + 2.0 ** -120
    grad = torch.where(mass > 0, scale * (grad - back), 0.0)
    return loss, bound, grad, eg + half_step(dtype, grad.abs() + eg)
