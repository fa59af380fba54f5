"""The model operators on matrices whose element and byte offsets pass 32 bits: rows and columns
at both ends and in between against the 64-bit forms."""
import pytest

import model_ref as ref
import test_gpu_blocks
from helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import torch
    assert torch.cuda.is_available(), "GPU test without a GPU"
    from trellis_coded_weight_amd import api as a
    yield a
    torch.cuda.empty_cache()


def filled(R, C, dtype, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty((R, C), dtype=getattr(torch, dtype), device="cuda").normal_(generator=g)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_blocks_past_32_bits(api, block_rows):
    import torch
    R, C = 131080, 32785
    x = filled(R, C, "bfloat16", 1)
    assert x.numel() > 1 << 32
    say("quantize_blocks %dx%d /%d" % (R, C, block_rows))
    q, s = api.quantize_blocks(x, block_rows=block_rows)
    torch.cuda.synchronize()
    for lo in (0, 65408, R // 128 * 128 - 128, R // 128 * 128):
        hi = min(lo + 128, R)
        bits, v = ref.quantize_blocks(x[lo:hi], block_rows)
        assert torch.equal(q[lo:hi].view(torch.uint8), bits), lo
        assert torch.equal(s[lo // block_rows:-(-hi // block_rows)], v), lo


def bytes_of(R, C, seed):
    """e4m3 codes of every value but NaN and the largest exponents."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    v = torch.empty((R, C), dtype=torch.uint8, device="cuda")
    v.random_(0, 0x70, generator=g)
    v[:, ::2] |= 0x80
    return v.view(torch.float8_e4m3fn)


@pytest.mark.parametrize("M,K", [(2, 32768), (100, 32768), (100, 32765)])
def test_matmul_fp8_weights_past_4_gb(api, M, K):
    import torch
    N = (1 << 17) + 48
    a, sa = test_gpu_blocks.codes(M, K, 1), test_gpu_blocks.scales(M, 256, 2)
    w, sw = bytes_of(N, K, 3), test_gpu_blocks.scales(-(-N // 128), 256, 4)
    assert w.numel() > 1 << 32
    say("matmul_fp8 %dx%dx%d" % (M, N, K))
    y = api.matmul_fp8(a, sa, w, sw, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    for lo, hi in ((0, 128), (65536, 65664), (N - 48, N)):
        want, e = ref.matmul_fp8(a, sa, w[lo:hi], sw[lo // 128:-(-hi // 128)], torch.bfloat16)
        ref.within(y[:, lo:hi], want, e, "columns from %d" % lo)


def test_matmul_fp8_activations_past_4_gb(api):
    import torch
    M, N, K = (1 << 17) + 48, 40, 32784
    a, sa = bytes_of(M, K, 1), test_gpu_blocks.scales(M, 257, 2)
    w, sw = test_gpu_blocks.codes(N, K, 3), test_gpu_blocks.scales(1, 257, 4)
    say("matmul_fp8 %dx%dx%d" % (M, N, K))
    y = api.matmul_fp8(a, sa, w, sw)
    torch.cuda.synchronize()
    for lo in (0, 65536, M - 64):
        want, e = ref.matmul_fp8(a[lo:lo + 64], sa[lo:lo + 64], w, sw, torch.float32)
        ref.within(y[lo:lo + 64], want, e, "rows from %d" % lo)


def test_matmul_fp8_result_past_32_bits(api):
    import torch
    M, N, K = 70000, 32776, 144
    a, sa, w, sw = test_gpu_blocks.operands(M, N, K)
    say("matmul_fp8 %dx%dx%d" % (M, N, K))
    y = api.matmul_fp8(a, sa, w, sw, dtype=torch.float16)
    torch.cuda.synchronize()
    assert y.numel() > 1 << 31
    for lo in (0, 65500, M - 40):
        want, e = ref.matmul_fp8(a[lo:lo + 40], sa[lo:lo + 40], w, sw, torch.float16)
        ref.within(y[lo:lo + 40], want, e, "rows from %d" % lo)


def test_layer_norm_past_32_bits(api):
    import torch
    R, C = 140000, 16385
    x, gy = filled(R, C, "bfloat16", 1), filled(R, C, "bfloat16", 2)
    w, b = test_gpu_blocks.normal(1, C, 3)[0], test_gpu_blocks.normal(1, C, 4)[0]
    assert x.numel() > 1 << 31
    say("layer_norm %dx%d" % (R, C))
    y, mean, rstd = api.layer_norm(x, w, b, save=True)
    gx, gw, gb = api.layer_norm_vjp(x, w, mean, rstd, gy)
    torch.cuda.synchronize()
    for lo in (0, 65530, 131070, R - 20):
        at = slice(lo, lo + 20)
        want, e, m, em, r, er = ref.layer_norm(x[at], w.double(), b.double(), 1e-5)
        ref.within(mean[at], m, em, "mean")
        ref.within(rstd[at], r, er, "rstd")
        ref.within(y[at], want, e, "y")
        want, e = ref.layer_norm_vjp(x[at], w.double(), mean[at], rstd[at], gy[at], torch.float32)[0]
        ref.within(gx[at], want, e, "grad_x")
    # the weights' gradients of some columns: sums over all rows
    at = torch.tensor([0, 1, 8191, 16384], device="cuda")
    xh = (x[:, at].double() - mean.double()[:, None]) * rstd.double()[:, None]
    for got, t in ((gw, xh * gy[:, at].double()), (gb, gy[:, at].double())):
        v = t.sum(0)
        ref.within(got[at], v, 1.01 * (R + 44) * 2.0 ** -24 * t.abs().sum(0), "weights' gradients")


@pytest.mark.parametrize("R,V", [(20000, 128008), (100, 1 << 24)])
def test_distill_past_32_bits(api, R, V):
    import torch
    k = 16 if R > 1000 else 3
    z = filled(R, V, "bfloat16" if R > 1000 else "float16", 1)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    index = torch.randint(0, V, (R, k), generator=g, device="cuda")
    index[:, 0] = V - 1
    t = torch.randn(R, k, generator=g, device="cuda")
    gl = torch.rand(R, generator=g, device="cuda") + 0.5
    step = 64 if R > 1000 else 2
    say("distill %dx%d" % (R, V))
    loss, grad = api.distill_topk(z, index, t, grad_loss=gl)
    torch.cuda.synchronize()
    assert z.numel() > 1 << 30
    for lo in (0, R // 2, R - step):
        at = slice(lo, lo + step)
        want, e, gr, eg = ref.distill(z[at], index[at], t[at], 1.0, None, gl[at], z.dtype)
        ref.within(loss[at], want, e, "loss")
        ref.within(grad[at], gr, eg, "grad")
