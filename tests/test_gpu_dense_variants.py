"""Every variant of the dense products' kernels (dense_variants.py) against 64-bit forms, with
operands that make most of them exact: small integers, whose sums binary32 holds whatever
their order, so that results are equal to the exact ones rounded once."""
import pytest

from dense_variants import ACTS, DTYPES, GATED, HALVES, INT8, VJP
from helpers import say
from test_gpu_dense_products import check_gated, check_int8, dtype_of, gen, halves, ints, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import torch
    assert torch.cuda.is_available(), "GPU test without a GPU"
    from trellis_coded_weight_amd import api as a
    yield a
    torch.cuda.empty_cache()


def small(r, c, t, seed, top, one_in=1):
    """Integers up to `top` in magnitude, all but one in `one_in` of them 0."""
    import torch
    g = gen(seed)
    v = torch.randint(-top, top + 1, (r, c), generator=g, device="cuda", dtype=torch.int32)
    if one_in > 1:
        v *= torch.randint(0, one_in, (r, c), generator=g, device="cuda", dtype=torch.int32) == 0
    return v.to(t)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", INT8)
def test_matmul_int8(api, M, N, K, dtype):
    say("matmul_int8 variants %dx%dx%d %s" % (M, N, K, dtype))
    check_int8(api, ints(M, K, 1), scales(M, 2), ints(N, K, 3), scales(N, 4), dtype_of(dtype))


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M,F,K", GATED)
def test_gated_exact(api, M, F, K, dtype):
    """relu and integers: sums, and their products, of at most 2^24."""
    import torch
    t = dtype_of(dtype)
    x, wg, wu = small(M, K, t, 1, 2), small(F, K, t, 2, 2), small(F, K, t, 3, 2)
    say("gated variants %dx%dx%d %s" % (M, F, K, dtype))
    h, gate, up = api.gated(x, wg, wu, activation="relu", save=True)
    only = api.gated(x, wg, wu, activation="relu")
    torch.cuda.synchronize()
    g, u = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    want = g.clamp(min=0) * u
    assert float(want.abs().max()) < 1 << 24 and 4 * K < 1 << 24
    assert torch.equal(gate, g.to(t)) and torch.equal(up, u.to(t))
    assert torch.equal(h, want.to(t)) and torch.equal(only, h)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M,F,K", [s for s in GATED if s[2] < 2000])
def test_gated_activations(api, M, F, K, dtype, act):
    t = dtype_of(dtype)
    say("gated variants %s %dx%dx%d %s" % (act, M, F, K, dtype))
    check_gated(api, halves(M, K, t, 1), halves(F, K, t, 2, K ** -0.5), halves(F, K, t, 3, K ** -0.5), act)


@pytest.mark.parametrize("round_slopes", [False, True])
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M,F,K", VJP)
def test_gated_vjp_exact(api, M, F, K, dtype, round_slopes):
    """relu, gates of 1 and -1 and integers: the slopes are integers of at most 4.  The two
    parts that such a slope is held in are multiples of 2^-8 (bf16) or 2^-11 (fp16) of its
    sign, so sums whose terms' magnitudes stay below 2^13 are exact; few nonzero slopes see
    to that."""
    import torch
    t = dtype_of(dtype)
    few = max(1, max(M, F) // 512)
    x, wg, wu = small(M, K, t, 1, 2), small(F, K, t, 2, 2), small(F, K, t, 3, 2)
    gate = small(M, F, t, 4, 1) * 2 + 1                       # -1, 1 and 3
    gate.clamp_(max=1)
    up, gh = small(M, F, t, 5, 2), small(M, F, t, 6, 2, few)
    say("gated_vjp variants %dx%dx%d %s" % (M, F, K, dtype))
    gx, gwg, gwu = api.gated_vjp(x, wg, wu, gate, up, gh, activation="relu", round_slopes=round_slopes)
    torch.cuda.synchronize()
    on = (gate > 0).double()
    dg, du = gh.double() * up.double() * on, gh.double() * on
    X, G, U = x.double(), wg.double(), wu.double()
    assert float((dg.abs() @ G.abs() + du.abs() @ U.abs()).max()) < 1 << 13
    assert float((dg.abs().t() @ X.abs()).max()) < 1 << 13
    assert torch.equal(gx, (dg @ G + du @ U).to(t))
    assert torch.equal(gwg, (dg.t() @ X).to(t)) and torch.equal(gwu, (du.t() @ X).to(t))
