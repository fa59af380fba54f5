"""Distillation from top logits against 64 bits: losses, gradients in the same call and alone,
padding, masks, repeated indices, and the sizes where a row is split."""
import pytest

import model_ref as ref
from helpers import say

pytestmark = pytest.mark.gpu

TYPES = ["float32", "bfloat16", "float16"]
# rows, vocabulary, entries: a row in one piece and in several, odd rows and lengths
SIZES = [(1, 1, 1), (3, 7, 2), (2, 64, 64), (5, 1000, 8), (4, 4099, 20), (1, 8192, 1), (2, 8193, 100), (3, 50021, 64),
         (7, 32000, 256), (1, 131072, 1024), (1000, 300, 5), (600, 9001, 17), (2, 20, 0), (40, 20001, 3)]


@pytest.fixture(scope="module")
def api():
    import torch
    assert torch.cuda.is_available(), "GPU test without a GPU"
    from trellis_coded_weight_amd import api as a
    return a


def inputs(R, V, k, dtype, ttype="float32", seed=0, wide=0):
    """wide > 0: logits in rows so much longer, with NaN beside the slice."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 7 * V + R)
    z = (torch.randn(R, V, generator=g, device="cuda") * 3).to(getattr(torch, dtype))
    if wide:
        t = torch.full((R, V + wide), float("nan"), dtype=z.dtype, device="cuda")
        t[:, wide // 2:wide // 2 + V] = z
        z = t[:, wide // 2:wide // 2 + V]
    index = torch.rand(R, V, generator=g, device="cuda").argsort(1)[:, :k]
    if k > V:
        index = torch.randint(0, V, (R, k), generator=g, device="cuda")
    index = torch.where(torch.rand(index.shape, generator=g, device="cuda") < 0.15, -1, index)
    if R > 2:
        index[1] = -1                                            # a token without entries
    t = (torch.randn(index.shape, generator=g, device="cuda") * 2 + 5).to(getattr(torch, ttype))
    gl = torch.rand(R, generator=g, device="cuda") + 0.5
    if R > 3:
        gl[3] = 0
    return z, index, t, gl


def check(api, z, index, t, gl, tau, log_z=None):
    import torch
    loss, grad = api.distill_topk(z, index, t, temperature=tau, teacher_log_z=log_z, grad_loss=gl)
    only = api.distill_topk(z, index, t, temperature=tau, teacher_log_z=log_z)
    saved, stats = api.distill_topk(z, index, t, temperature=tau, teacher_log_z=log_z, save=True)
    late = api.distill_topk_vjp(z, index, t, stats, gl, temperature=tau)
    torch.cuda.synchronize()
    want, e, g, eg = ref.distill(z, index, t, tau, log_z, gl, z.dtype)
    ref.within(loss, want, e, "loss")
    ref.within(grad, g, eg, "grad")
    assert loss.dtype == torch.float32 and grad.dtype == z.dtype and grad.shape == z.shape
    assert torch.equal(only, loss) and torch.equal(saved, loss) and torch.equal(late, grad)
    return loss, grad


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,V,k", SIZES)
def test_distill(api, R, V, k, dtype):
    say("distill %dx%d k=%d %s" % (R, V, k, dtype))
    z, index, t, gl = inputs(R, V, k, dtype)
    check(api, z, index, t, gl, 1.0)


@pytest.mark.parametrize("tau", [0.25, 1.0, 4.0])
@pytest.mark.parametrize("ttype", TYPES)
def test_distill_types_and_temperatures(api, ttype, tau):
    say("distill teacher %s tau=%g" % (ttype, tau))
    z, index, t, gl = inputs(6, 5000, 30, "bfloat16", ttype)
    a = check(api, z, index, t, gl, tau)
    b = check(api, z, index.int(), t, gl, tau)
    assert (a[0] == b[0]).all() and (a[1] == b[1]).all()


@pytest.mark.parametrize("R", [3, 700])
@pytest.mark.parametrize("wide", [1, 6, 16])
@pytest.mark.parametrize("dtype", TYPES)
def test_distill_strided(api, dtype, wide, R):
    """Slices of longer rows of logits, of indices and of the teacher's."""
    import torch
    say("distill strided +%d %s R=%d" % (wide, dtype, R))
    z, index, t, gl = inputs(R, 9000, 20, dtype, wide=wide)
    big = torch.full((R, 33), 5, device="cuda")
    big[:, 7:27] = index
    tb = torch.full((R, 29), float("nan"), device="cuda")
    tb[:, 4:24] = t
    check(api, z, big[:, 7:27], tb[:, 4:24], gl, 1.0)


@pytest.mark.parametrize("V", [3000, 40000, 70000])
def test_distill_given_sum(api, V):
    """The teacher's probabilities over its whole vocabulary: their sum here is below 1."""
    import torch
    z, index, t, gl = inputs(5, V, 16, "float32")
    lz = torch.logsumexp(t / 2.0, 1) + 0.3
    say("distill given sum V=%d" % V)
    loss, grad = check(api, z, index, t, gl, 2.0, lz)
    # the gradient of a token sums to 0: sum p times the sum of q, less sum p
    assert float(grad.double().sum(1).abs().max()) < 1e-5


@pytest.mark.parametrize("V", [500, 30000, 70000])
def test_distill_repeated_indices(api, V):
    import torch
    z, index, t, gl = inputs(5, V, 40, "float32")
    index[:, 1::2] = index[:, ::2]                               # each twice
    index[0] = index[0, 0]                                       # all the same
    index[2] = V - 1
    say("distill repeated indices V=%d" % V)
    check(api, z, index, t, gl, 1.0)


@pytest.mark.parametrize("V", [700, 30000, 70000])
def test_distill_indices_out_of_range(api, V):
    """Any index outside the vocabulary is padding, whatever its teacher's value."""
    import torch
    z, index, t, gl = inputs(6, V, 12, "bfloat16")
    index[:, 3], index[:, 5], index[:, 7], index[4] = V, -2 ** 40, 2 ** 40, 2 ** 32
    a = check(api, z, index, t, gl, 1.0)
    bad = t.clone()
    bad[(index < 0) | (index >= V)] = float("nan")
    say("distill indices out of range V=%d" % V)
    loss, grad = api.distill_topk(z, index, bad, grad_loss=gl)
    torch.cuda.synchronize()
    assert torch.equal(loss, a[0]) and torch.equal(grad, a[1])
    assert float(loss[4]) == 0 and not bool(grad[4].any())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [600, 40000, 70000])
def test_distill_masked_vocabulary(api, V, dtype):
    """Logits of -infinity or of the type's lowest value at most of the vocabulary; rows of
    them alone; teachers of -infinity."""
    import torch
    z, index, t, gl = inputs(8, V, 10, dtype)
    index = torch.arange(10, device="cuda").repeat(8, 1) * 3
    lowest = torch.finfo(z.dtype).min
    z[0, 40:] = -float("inf")
    z[1, 40:] = lowest
    z[2, :40] = lowest
    z[3] = lowest                                               # uniform
    t[4, 2:] = -float("inf")
    t[5] = -float("inf")                                        # nothing has a share
    say("distill masked vocabulary V=%d %s" % (V, dtype))
    loss, grad = api.distill_topk(z, index, t, grad_loss=gl)
    torch.cuda.synchronize()
    want, e, g, eg = ref.distill(z[[0, 1, 3, 4, 6, 7]], index[:6], t[[0, 1, 3, 4, 6, 7]], 1.0, None, gl[[0, 1, 3, 4, 6, 7]],
                                 z.dtype)
    rows = [0, 1, 3, 4, 6, 7]
    ref.within(loss[rows], want, e, "loss")
    ref.within(grad[rows], g, eg, "grad")
    assert not bool(grad[0, 40:].any())
    assert float(loss[2]) > 1e4                                 # the teacher's entries have no share of q
    assert float(loss[5]) == 0 and not bool(grad[5].any())
    # an entry with a share at a masked one: infinite; without a share: nothing
    z[6, 3] = -float("inf")
    z[7, 6] = -float("inf")
    t[7, 2] = -float("inf")
    loss2 = api.distill_topk(z, index, t)
    torch.cuda.synchronize()
    assert float(loss2[6]) == float("inf") and bool(torch.isfinite(loss2[7]))


@pytest.mark.parametrize("V", [600, 40000, 70000])
def test_distill_non_finite_rows(api, V):
    """NaN or +infinity in a row's logits or teacher's values reach that token alone, and a
    token without entries is 0 even then."""
    import torch
    z, index, t, gl = inputs(9, V, 10, "float32")
    index = torch.arange(10, device="cuda").repeat(9, 1) * 7
    loss0, grad0 = api.distill_topk(z, index, t, grad_loss=gl)
    z[1, V - 1], z[2, 5], z[3], t[4, 3], t[5, 0] = float("nan"), float("inf"), -float("inf"), float("nan"), float("inf")
    z[6], index[6] = float("nan"), -1
    say("distill non-finite rows V=%d" % V)
    loss, grad = api.distill_topk(z, index, t, grad_loss=gl)
    torch.cuda.synchronize()
    for r in (1, 2, 3, 4, 5):
        assert bool(torch.isnan(loss[r])), r
    for r in (1, 4, 5):
        assert bool(torch.isnan(grad[r]).all()), r
    assert float(loss[6]) == 0 and not bool(grad[6].any())
    for r in (0, 7, 8):
        assert torch.equal(loss[r], loss0[r]) and torch.equal(grad[r], grad0[r])


def test_distill_large_logits(api):
    """Logits of thousands: the maximum is taken off first."""
    z, index, t, gl = inputs(5, 9000, 12, "float32")
    z = z * 1000 - 5000
    t = t * 500
    say("distill large logits")
    check(api, z, index, t, gl, 1.0)


def test_distill_empty(api):
    import torch
    for R, V, k in ((0, 5, 2), (3, 0, 2), (3, 9, 0)):
        z = torch.randn(R, V, device="cuda")
        loss, grad = api.distill_topk(z, torch.zeros(R, k, dtype=torch.int64, device="cuda"),
                                      torch.zeros(R, k, device="cuda"), grad_loss=torch.ones(R, device="cuda"))
        torch.cuda.synchronize()
        assert loss.shape == (R,) and grad.shape == (R, V) and not bool(loss.any()) and not bool(grad.any())


@pytest.mark.parametrize("tau", [0.7, 2.0])
def test_distill_gradient_against_differences(api, tau):
    """Central differences of the 64-bit loss of the definition (error of order h^2)."""
    import torch
    z, index, t, gl = inputs(3, 50, 6, "float32")
    index[0, 3] = index[0, 2]
    _, grad = api.distill_topk(z, index, t, temperature=tau, grad_loss=gl)
    torch.cuda.synchronize()
    Z, h = z.double(), 1e-4
    say("distill gradients against differences")
    for r in range(3):
        for v in list(range(0, 50, 9)) + [int(i) for i in index[r] if i >= 0]:
            keep = float(Z[r, v])
            Z[r, v] = keep + h
            up = ref.distill(Z, index, t, tau)[0][r]
            Z[r, v] = keep - h
            down = ref.distill(Z, index, t, tau)[0][r]
            Z[r, v] = keep
            want = float(gl[r]) * float(up - down) / (2 * h)
            assert abs(float(grad[r, v]) - want) <= 1e-6 + 1e-5 * abs(want), (r, v)
