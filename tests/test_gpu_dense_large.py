"""The dense operators on matrices whose element and byte offsets pass 32 bits: rows and
columns at both ends against the same operator on a slice (where it is exact) or against
the 64-bit forms."""
import pytest

import dense_ref as ref
from helpers import say
from test_gpu_dense_products import gen, halves, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import torch
    assert torch.cuda.is_available(), "GPU test without a GPU"
    from trellis_coded_weight_amd import api as a
    yield a
    torch.cuda.empty_cache()


@pytest.mark.parametrize("K", [32768, 32765])
@pytest.mark.parametrize("M", [3, 100])
def test_matmul_int8_weights_past_4_gb(api, M, K):
    import torch
    N = (1 << 17) + 48
    a = torch.randint(-128, 128, (M, K), generator=gen(1), device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=gen(2), device="cuda", dtype=torch.int8)
    sa, sw = scales(M, 3), scales(N, 4)
    assert w.numel() > 1 << 32
    say("matmul_int8 %dx%dx%d" % (M, N, K))
    y = api.matmul_int8(a, sa, w, sw)
    torch.cuda.synchronize()
    for lo, hi in ((0, 70), (65500, 65600), (N - 70, N)):
        part = (a.double() @ w[lo:hi].double().t()).float() * sa[:, None] * sw[lo:hi]
        assert torch.equal(y[:, lo:hi], part), (lo, hi)


def test_matmul_int8_result_past_32_bits(api):
    import torch
    M, N, K = 70000, 32776, 64
    a = torch.randint(-128, 128, (M, K), generator=gen(1), device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=gen(2), device="cuda", dtype=torch.int8)
    sa, sw = scales(M, 3), scales(N, 4)
    say("matmul_int8 %dx%dx%d" % (M, N, K))
    y = api.matmul_int8(a, sa, w, sw, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert y.numel() > 1 << 31
    for lo, hi in ((0, 40), (65500, 65540), (M - 40, M)):
        part = ((a[lo:hi].double() @ w.double().t()).float() * sa[lo:hi, None] * sw).to(torch.bfloat16)
        assert torch.equal(y[lo:hi], part), (lo, hi)


def test_quantize_rows_past_32_bits(api):
    import torch
    R, C = 65539, 33001
    x = torch.empty((R, C), dtype=torch.bfloat16, device="cuda").normal_(generator=gen(1))
    assert x.numel() > 1 << 31
    say("quantize %dx%d" % (R, C))
    q, s = api.quantize_rows(x)
    torch.cuda.synchronize()
    for lo, hi in ((0, 5), (65000, 65005), (R - 5, R)):
        qr, sr = ref.quantize(x[lo:hi].double())
        assert torch.equal(q[lo:hi], qr) and torch.equal(s[lo:hi], sr), (lo, hi)


def test_decode_matrix_past_32_bits(api):
    import torch
    M, N = 65536 + 16, 32768 + 16
    n = (M // 16) * (N // 16)
    bits = torch.randint(-2 ** 31, 2 ** 31, (n, 17), generator=gen(3), device="cuda", dtype=torch.int64).to(torch.int32)
    say("decode_matrix %dx%d" % (M, N))
    q, s = api.decode_matrix(bits, M, N, code="3inst")
    torch.cuda.synchronize()
    assert q.numel() > 1 << 31
    per = N // 16
    for band in (0, M // 32, M // 16 - 1):
        v = api.decode(bits[band * per:(band + 1) * per].contiguous(), 256, code="3inst")[0]
        v = v.reshape(1, per, 16, 16).permute(0, 2, 1, 3).reshape(16, N)
        qr, sr = ref.quantize(v.double())
        assert torch.equal(q[16 * band:16 * band + 16], qr) and torch.equal(s[16 * band:16 * band + 16], sr), band


def test_gated_and_gradients_past_32_bits(api):
    import torch
    t = torch.bfloat16
    M, F, K = 40000, 54000, 40
    x, wg, wu = halves(M, K, t, 1), halves(F, K, t, 2, 0.2), halves(F, K, t, 3, 0.2)
    say("gated %dx%dx%d" % (M, F, K))
    h, gate, up = api.gated(x, wg, wu, save=True)
    assert h.numel() > 1 << 31
    gh = torch.empty_like(h).normal_(generator=gen(4)).mul_(0.1)
    say("gated_vjp %dx%dx%d" % (M, F, K))
    gx, gwg, gwu = api.gated_vjp(x, wg, wu, gate, up, gh)
    torch.cuda.synchronize()
    for lo, hi in ((0, 20), (M - 20, M)):
        want, e, g, u, eg, eu = ref.gated(x[lo:hi], wg, wu, "silu")
        ref.within(h[lo:hi], want, e, "h")
        ref.within(gate[lo:hi], g, eg, "gate")
        ref.within(up[lo:hi], u, eu, "up")
        r, e = ref.gated_vjp(x[lo:hi], wg, wu, gate[lo:hi], up[lo:hi], gh[lo:hi], "silu")[0]
        ref.within(gx[lo:hi], r, e, "grad_x")
    for lo, hi in ((0, 20), (F - 20, F)):
        r = ref.gated_vjp(x, wg[lo:hi], wu[lo:hi], gate[:, lo:hi], up[:, lo:hi], gh[:, lo:hi], "silu")
        ref.within(gwg[lo:hi], *r[1], "grad_w_gate")
        ref.within(gwu[lo:hi], *r[2], "grad_w_up")
