"""Layer norm and its gradients against 64 bits, at the sizes, strides, types and values where
row shapes, tails and sums over rows can go wrong."""
import pytest

import model_ref as ref
from helpers import say

pytestmark = pytest.mark.gpu

TYPES = ["float32", "bfloat16", "float16"]
EPS = 1e-5
SIZES = [(1, 1), (3, 2), (1, 8), (5, 63), (4, 64), (7, 65), (2, 511), (9, 513), (33, 1000), (6, 1024), (3, 2049),
         (5, 2731), (2, 4099), (3, 8192), (4, 8200), (2, 16384), (2, 16400), (1, 40001), (2, 70000), (1031, 40), (2500, 300),
         (700, 2048), (600, 5000), (768, 2730), (769, 1000), (800, 2048), (801, 4100), (770, 8192)]


@pytest.fixture(scope="module")
def api():
    import torch
    assert torch.cuda.is_available(), "GPU test without a GPU"
    from trellis_coded_weight_amd import api as a
    return a


def normal(*shape, seed=0, dtype="float32", scale=1.0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(getattr(torch, dtype))


def inputs(R, C, dtype, wtype):
    x = normal(R, C, seed=1, dtype=dtype, scale=2.0)
    x += normal(R, 1, seed=2, dtype=dtype)                     # rows with a mean
    return x, normal(C, seed=3, dtype=wtype) * 0.2 + 1, normal(C, seed=4, dtype=wtype)


def check_forward(api, x, w, b, eps=EPS):
    import torch
    y, mean, rstd = api.layer_norm(x, w, b, eps=eps, save=True)
    only = api.layer_norm(x, w, b, eps=eps)
    torch.cuda.synchronize()
    C = x.shape[1]
    W = torch.ones(C, dtype=torch.float64, device="cuda") if w is None else w.double()
    B = torch.zeros(C, dtype=torch.float64, device="cuda") if b is None else b.double()
    want, e, m, em, r, er = ref.layer_norm(x, W, B, eps)
    ref.within(mean, m, em, "mean")
    ref.within(rstd, r, er, "rstd")
    ref.within(y, want, e, "y")
    assert y.dtype == x.dtype and torch.equal(y, only)
    return mean, rstd


def check_vjp(api, x, w, mean, rstd, gy):
    import torch
    got = api.layer_norm_vjp(x, w, mean, rstd, gy)
    only_x = api.layer_norm_vjp(x, w, mean, rstd, gy, want_w=False)
    only_w = api.layer_norm_vjp(x, w, mean, rstd, gy, want_x=False)
    torch.cuda.synchronize()
    W = torch.ones(x.shape[1], dtype=torch.float64, device="cuda") if w is None else w.double()
    wt = x.dtype if w is None else w.dtype
    for g, (want, e), name in zip(got, ref.layer_norm_vjp(x, W, mean, rstd, gy, wt), ("grad_x", "grad_weight", "grad_bias")):
        ref.within(g, want, e, name)
    assert got[0].dtype == x.dtype and got[1].dtype == wt and got[2].dtype == wt
    assert torch.equal(only_x[0], got[0]) and only_x[1] is None and only_x[2] is None
    assert torch.equal(only_w[1], got[1]) and torch.equal(only_w[2], got[2]) and only_w[0] is None
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,C", SIZES)
def test_layer_norm(api, R, C, dtype):
    for wtype in {dtype, "float32"}:
        x, w, b = inputs(R, C, dtype, wtype)
        say("layer_norm %dx%d %s %s" % (R, C, dtype, wtype))
        mean, rstd = check_forward(api, x, w, b)
        check_vjp(api, x, w, mean, rstd, normal(R, C, seed=5, dtype=dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,C", [(3, 100), (300, 1500)])
def test_layer_norm_without_weight_or_bias(api, R, C, dtype):
    x, w, b = inputs(R, C, dtype, dtype)
    say("layer_norm without weights %dx%d %s" % (R, C, dtype))
    check_forward(api, x, w, None)
    check_forward(api, x, None, b)
    mean, rstd = check_forward(api, x, None, None)
    check_vjp(api, x, None, mean, rstd, normal(R, C, seed=5, dtype=dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_layer_norm_strided(api, dtype):
    """Slices of wider rows, aligned and not; what lies beside the slice is not read, and rows
    of a wider buffer keep what lies beside them."""
    import torch
    from trellis_coded_weight_amd import _native as nat
    for off, C in ((0, 96), (8, 264), (1, 97), (3, 1025), (16, 1800)):
        x0, w, b = inputs(6, C, dtype, dtype)
        g0 = normal(6, C, seed=9, dtype=dtype)

        def wide(v):
            t = torch.full((6, 2000), float("nan"), dtype=v.dtype, device="cuda")
            t[:, off:off + C] = v
            return t[:, off:off + C]
        x, gy = wide(x0), wide(g0)
        say("layer_norm strided off=%d C=%d %s" % (off, C, dtype))
        mean, rstd = check_forward(api, x, w, b)
        check_vjp(api, x, w, mean, rstd, gy)
        y = api.layer_norm(x0, w, b)
        size, st = x0.element_size(), torch.cuda.current_stream().cuda_stream
        out = torch.full((6, 2000), 7.0, dtype=x0.dtype, device="cuda")
        nat.qtcq_layer_norm(x0.data_ptr(), api.DTYPES[x0.dtype], 6, C, C, w.data_ptr(), b.data_ptr(), api.DTYPES[x0.dtype],
                            EPS, out.data_ptr() + off * size, 2000, None, None, st)
        gout = torch.full((6, 2000), 7.0, dtype=x0.dtype, device="cuda")
        nat.qtcq_layer_norm_vjp(x0.data_ptr(), api.DTYPES[x0.dtype], 6, C, C, w.data_ptr(), api.DTYPES[x0.dtype],
                                mean.data_ptr(), rstd.data_ptr(), g0.data_ptr(), C, gout.data_ptr() + off * size, 2000,
                                None, None, None, 0, st)
        torch.cuda.synchronize()
        gx = api.layer_norm_vjp(x0, w, mean, rstd, g0, want_w=False)[0]
        for o, v in ((out, y), (gout, gx)):
            assert torch.equal(o[:, off:off + C], v)
            assert bool((o[:, :off] == 7).all()) and bool((o[:, off + C:] == 7).all())


@pytest.mark.parametrize("C", [64, 1000, 5000])
def test_layer_norm_far_mean(api, C):
    """Rows whose mean is far larger than their spread, and rows of one value (variance 0)."""
    import torch
    x = normal(9, C, seed=1) * 0.01 + 1000
    x[4:] = normal(5, 1, seed=2)
    w, b = normal(C, seed=3), normal(C, seed=4)
    say("layer_norm far mean C=%d" % C)
    check_forward(api, x, w, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("C", [40, 3001, 20000])
def test_layer_norm_non_finite(api, C, dtype):
    """An infinity or NaN reaches its own row, and of the weights' gradients every column by
    way of the row's statistics; other rows keep their bits."""
    import torch
    R = 7
    x, w, b = inputs(R, C, dtype, "float32")
    gy = normal(R, C, seed=5, dtype=dtype)
    y0, mean0, rstd0 = api.layer_norm(x, w, b, save=True)
    gx0 = api.layer_norm_vjp(x, w, mean0, rstd0, gy)[0]
    x[2, C // 2], x[5, C - 1] = float("inf"), float("nan")
    say("layer_norm non-finite C=%d %s" % (C, dtype))
    y, mean, rstd = api.layer_norm(x, w, b, save=True)
    gx, gw, gb = api.layer_norm_vjp(x, w, mean, rstd, gy)
    torch.cuda.synchronize()
    for r in (2, 5):
        assert bool(torch.isnan(y[r]).all()) and bool(torch.isnan(gx[r]).all())
    keep = [r for r in range(R) if r not in (2, 5)]
    assert torch.equal(y[keep], y0[keep]) and torch.equal(gx[keep], gx0[keep])
    assert bool(torch.isnan(gw).all()) and bool(torch.isfinite(gb).all())


def test_layer_norm_empty(api):
    import torch
    for R, C in ((0, 5), (4, 0), (0, 0), (0, 9000), (0, 20000)):
        x, w = torch.empty(R, C, device="cuda"), torch.empty(C, device="cuda")
        y, mean, rstd = api.layer_norm(x, w, w, save=True)
        gx, gw, gb = api.layer_norm_vjp(x, w, mean, rstd, x)
        torch.cuda.synchronize()
        assert y.shape == (R, C) and gx.shape == (R, C) and gw.shape == (C,)
        assert not bool(gw.any()) and not bool(gb.any())


def test_layer_norm_gradient_against_differences(api):
    """Central differences of the 64-bit function of the definition: the error of a difference
    with step h is of order h^2 (third derivatives below 10 here), and the gradient's own."""
    import torch
    R, C, h = 3, 24, 1e-4
    x, w, b = inputs(R, C, "float32", "float32")
    gy = normal(R, C, seed=5)
    _, mean, rstd = api.layer_norm(x, w, b, save=True)
    got = api.layer_norm_vjp(x, w, mean, rstd, gy)

    def total(x, w, b):
        d = x - x.mean(1, keepdim=True)
        return float((gy.double() * (d / torch.sqrt(d.square().mean(1, keepdim=True) + EPS) * w + b)).sum())
    args = [x.double(), w.double(), b.double()]
    say("layer_norm gradients against differences")
    for i, g in enumerate(got):
        flat = args[i].view(-1)
        for j in range(0, flat.numel(), 7):
            keep = float(flat[j])
            flat[j] = keep + h
            up = total(*args)
            flat[j] = keep - h
            down = total(*args)
            flat[j] = keep
            want = (up - down) / (2 * h)
            assert abs(float(g.view(-1)[j]) - want) <= 1e-5 * (1 + abs(want)), (i, j)
