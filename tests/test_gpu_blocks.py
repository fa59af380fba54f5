"""e4m3 with block scales: the quantization against its definition (equality), and the product
against 64 bits, at the sizes, strides and values where tiles and tails can go wrong."""
import pytest

import model_ref as ref
from helpers import say

pytestmark = pytest.mark.gpu

TYPES = ["float32", "bfloat16", "float16"]


@pytest.fixture(scope="module")
def api():
    import torch
    assert torch.cuda.is_available(), "GPU test without a GPU"
    from trellis_coded_weight_amd import api as a
    return a


def normal(R, C, seed, dtype="float32"):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(R, C, generator=g, device="cuda").to(getattr(torch, dtype))


def check(api, x, block_rows):
    import torch
    q, s = api.quantize_blocks(x, block_rows=block_rows)
    torch.cuda.synchronize()
    bits, sr = ref.quantize_blocks(x, block_rows)
    assert q.dtype == torch.float8_e4m3fn and q.shape == x.shape and s.shape == sr.shape
    assert torch.equal(torch.isnan(s), torch.isnan(sr)) and torch.equal(s.nan_to_num(-1), sr.nan_to_num(-1))
    got = q.view(torch.uint8)
    assert torch.equal(got, bits), (x.shape, (got != bits).nonzero()[:4].tolist())
    return q, s


SIZES = [(1, 1), (1, 16), (3, 7), (2, 127), (5, 128), (9, 129), (8, 511), (7, 513), (130, 100), (127, 257), (128, 384),
         (129, 1000), (300, 2049), (1, 14336), (2, 28679)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("R,C", SIZES)
def test_quantize_blocks(api, R, C, block_rows, dtype):
    say("quantize_blocks %dx%d /%d %s" % (R, C, block_rows, dtype))
    check(api, normal(R, C, R + C, dtype), block_rows)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_strided_rows(api, block_rows, dtype):
    """Slices of wider rows, aligned and not; what lies beside the slice is not read."""
    for off, C in ((0, 96), (8, 264), (1, 97), (3, 1025), (16, 1024)):
        wide = normal(140, 2000, off, dtype)
        x = wide[:, off:off + C]
        keep = x.clone()
        wide.fill_(float("nan"))
        wide[:, off:off + C] = keep
        say("quantize_blocks strided off=%d C=%d %s" % (off, C, dtype))
        check(api, x, block_rows)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_written_where_asked(api, block_rows):
    """Rows of a wider buffer and scales of any strides; what lies beside them stays."""
    import torch
    from trellis_coded_weight_amd import _native as nat
    R, C = 133, 300
    x = normal(R, C, 3)
    bits, s = ref.quantize_blocks(x, block_rows)
    down, wide = s.shape
    for row, col in ((wide + 2, 1), (1, down + 3), (2 * wide, 2)):
        q = torch.full((R, 400), 99, dtype=torch.uint8, device="cuda")
        scale = torch.full((4000,), -5.0, device="cuda")
        say("quantize_blocks strides %d %d" % (row, col))
        nat.qtcq_quantize_blocks(x.data_ptr(), nat.QTCQ_F32, R, C, C, block_rows, q.data_ptr() + 5, 400,
                                 scale.data_ptr() + 12, row, col, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(q[:, 5:5 + C], bits) and bool((q[:, :5] == 99).all()) and bool((q[:, 5 + C:] == 99).all())
        assert torch.equal(scale[3:].as_strided((down, wide), (row, col)), s)
        scale[3:].as_strided((down, wide), (row, col)).fill_(-5.0)
        assert bool((scale == -5.0).all())


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_halves_and_small_values(api, block_rows):
    """Points half way between e4m3 values, their neighbours, and magnitudes down to the
    smallest subnormals."""
    import torch
    points = torch.tensor(ref.E4M3[:127], dtype=torch.float64, device="cuda")
    half = (points[1:] + points[:-1]) / 2
    values = torch.cat([points, half, -half])
    rows = []
    for top, e in ((448.0, 0), (448.0, -60), (448.0, 100), (448.0, -135), (448.0, -141), (300.0, 0), (7.0, -20)):
        # scale exactly 2^e for 448; else the points times a scale that is no power of two
        s = (torch.tensor(top * 2.0 ** e, dtype=torch.float64) / 448).float().double().item()
        v = (values * s).float()
        rows += [v, torch.nextafter(v, v * 0), torch.nextafter(v, v * 4)]
    x = torch.stack(rows)
    x = torch.where(x.abs() > 0, x, torch.zeros_like(x))
    n = x.shape[1]
    # every block holds its row's largest value, so that all have the scale meant
    wide = torch.zeros(x.shape[0], 4 * 128, device="cuda")
    for b in range(4):
        part = x[:, b * 100:min(n, (b + 1) * 100)]
        wide[:, b * 128:b * 128 + part.shape[1]] = part
        wide[:, b * 128 + 127] = x.abs().amax(1)
    say("quantize_blocks halves and small values")
    if block_rows == 1:
        check(api, wide, 1)
    else:
        for r in range(0, wide.shape[0], 3):
            check(api, wide[r:r + 3], 128)


def test_quantize_every_pair_of_short_numbers(api):
    """Each 8-bit number by each as its block's largest, over 20 powers of two: many quotients
    by 448ths of them lie half way."""
    import torch
    m = torch.arange(128, 256, device="cuda", dtype=torch.float32)
    blocks = []
    for e in range(20):
        v = m.expand(128, 128) * 2.0 ** -e
        v = torch.where(v <= m[:, None], v, v / 2)
        for half in (v[:, :64], v[:, 64:]):
            blocks.append(torch.cat([half, -half[:, 1:], m[:, None]], 1))
    x = torch.cat(blocks, 1)
    say("quantize_blocks every pair of short numbers")
    for scale in (1.0, 2.0 ** -80, 2.0 ** 100):
        check(api, (x * scale).bfloat16(), 1)
        check(api, x * scale, 1)
    for r in range(0, 128, 9):
        check(api, (x[r] * 2.0 ** -20).bfloat16().view(40, 128).repeat(4, 1)[:128], 128)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_zero_and_non_finite_blocks(api, block_rows, dtype):
    import torch
    x = normal(300, 600, 5, dtype)
    x[130:140] = 0
    x[0, 5] = float("inf")
    x[7, 300] = float("-inf")
    x[270, 599] = float("nan")
    x[140:260, 128:256] = 0
    x[200, 400] = torch.finfo(x.dtype).max
    if dtype == "float32":
        x[150, 512:] = 1e-44                                  # the scale underflows
    say("quantize_blocks zero and non-finite %s" % dtype)
    check(api, x, block_rows)


def test_quantize_empty(api):
    import torch
    for shape in ((0, 300), (3, 0), (0, 0)):
        for br in (1, 128):
            q, s = api.quantize_blocks(torch.empty(shape, device="cuda"), block_rows=br)
            assert q.shape == shape and s.shape == ((shape[0] if br == 1 else -(-shape[0] // 128)), -(-shape[1] // 128))


# ---- the product -------------------------------------------------------------------------------

def codes(r, c, seed, wide=0):
    """e4m3 values of every magnitude; wide > 0: in rows so much longer, NaN beside the slice."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    v = (torch.randn(r, c, generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    if not wide:
        return v
    t = torch.full((r, c + wide), 0x7F, dtype=torch.uint8, device="cuda")
    t[:, wide // 2:wide // 2 + c] = v.view(torch.uint8)
    return t.view(torch.float8_e4m3fn)[:, wide // 2:wide // 2 + c]


def scales(r, c, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.rand(r, c, generator=g, device="cuda") * 0.01 + 1e-3


def operands(M, N, K, wide=0):
    kb = -(-K // 128)
    return codes(M, K, 1, wide), scales(M, kb, 2), codes(N, K, 3, wide), scales(-(-N // 128), kb, 4)


def check_product(api, a, sa, w, sw, dtype):
    import torch
    t = getattr(torch, dtype)
    y = api.matmul_fp8(a, sa, w, sw, dtype=t)
    torch.cuda.synchronize()
    want, bound = ref.matmul_fp8(a, sa, w, sw, t)
    assert y.dtype == t and y.shape == want.shape
    ref.within(y, want, bound, "matmul_fp8 %s %s" % (list(a.shape), list(w.shape)))
    return y


PRODUCTS = [(1, 1, 1), (1, 16, 128), (1, 33, 129), (2, 256, 512), (5, 100, 24), (8, 1000, 1024), (16, 130, 4096),
            (17, 64, 136), (31, 513, 520), (33, 520, 1000), (64, 128, 256), (65, 127, 255), (96, 704, 320),
            (128, 256, 64), (129, 257, 65), (200, 48, 2056), (256, 512, 768), (300, 1032, 328), (512, 256, 1024),
            (1, 5000, 16), (4, 24, 14336), (100, 264, 4104), (150, 130, 5001), (70, 2000, 72), (257, 1000, 2048),
            (1000, 1500, 640), (48, 4096, 1280), (48, 300, 9000)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_matmul_fp8(api, M, N, K, dtype):
    say("matmul_fp8 %dx%dx%d %s" % (M, N, K, dtype))
    check_product(api, *operands(M, N, K), dtype)


@pytest.mark.parametrize("wide", [6, 16, 64])
@pytest.mark.parametrize("M,N,K", [(1, 70, 100), (40, 200, 333), (130, 300, 512), (7, 64, 64), (600, 300, 272)])
def test_matmul_fp8_strided(api, M, N, K, wide):
    """Slices of longer rows, with NaN beside them."""
    say("matmul_fp8 strided %dx%dx%d +%d" % (M, N, K, wide))
    check_product(api, *operands(M, N, K, wide), "float32")


@pytest.mark.parametrize("M", [3, 40, 300])
def test_matmul_fp8_scale_strides(api, M):
    """Scales stored row by row, column by column, in a wider buffer, and broadcast."""
    import torch
    N, K = 300, 700
    a, sa, w, sw = operands(M, N, K)
    say("matmul_fp8 scale strides M=%d" % M)
    y = check_product(api, a, sa, w, sw, "float32")
    wide = torch.full((M, 40), float("nan"), device="cuda")
    wide[:, 4:16:2] = sa
    for s, t in ((sa.t().contiguous().t(), sw.t().contiguous().t()), (wide[:, 4:16:2], sw)):
        assert torch.equal(api.matmul_fp8(a, s, w, t), y)
    one = torch.full((1, 1), 0.01, device="cuda")
    check_product(api, a, one.expand(M, 6), w, one.expand(3, 6), "float32")


def test_matmul_fp8_every_value(api):
    """All 256 codes in each operand: NaN codes reach the results that they take part in and
    no others."""
    import torch
    for M in (256, 16):
        a = torch.zeros(M, 128, dtype=torch.uint8, device="cuda")
        w = torch.zeros(256, 128, dtype=torch.uint8, device="cuda")
        a[:, 0] = torch.arange(M, device="cuda") * (256 // M)
        w[:, 0] = torch.arange(256, device="cuda")
        a, w = a.view(torch.float8_e4m3fn), w.view(torch.float8_e4m3fn)
        say("matmul_fp8 every value M=%d" % M)
        y = api.matmul_fp8(a, torch.ones(M, 1, device="cuda"), w, torch.ones(2, 1, device="cuda"))
        torch.cuda.synchronize()
        want = ref.e4m3(a)[:, :1] * ref.e4m3(w)[:, 0]
        assert torch.equal(torch.isnan(y), torch.isnan(want))
        assert torch.equal(y.nan_to_num(0), want.nan_to_num(0).float())


@pytest.mark.parametrize("M,N,K", [(3, 140, 384), (20, 140, 384), (150, 300, 384), (300, 520, 1024), (60, 300, 8192)])
def test_matmul_fp8_non_finite_scales(api, M, N, K):
    """A NaN token scale reaches that token's row, an infinite weight scale its 128 columns;
    scales of 0 (blocks of zeros) give zeros."""
    import torch
    a, sa, w, sw = operands(M, N, K)
    clean = api.matmul_fp8(a, sa, w, sw)
    sa[1, 2], sw[1, 0] = float("nan"), float("inf")
    say("matmul_fp8 non-finite scales %dx%dx%d" % (M, N, K))
    y = api.matmul_fp8(a, sa, w, sw)
    torch.cuda.synchronize()
    assert bool(torch.isnan(y[1]).all())
    keep = [i for i in range(M) if i != 1]
    inside = y[keep][:, 128:256]
    assert not bool(torch.isfinite(inside).any())
    assert torch.equal(y[keep][:, :128], clean[keep][:, :128]) and torch.equal(y[keep][:, 256:], clean[keep][:, 256:])
    sa.zero_()
    sw[1, 0] = 1
    y = api.matmul_fp8(a, sa, w, sw)
    torch.cuda.synchronize()
    assert not bool(y.any())


def test_matmul_fp8_empty(api):
    import torch
    f8 = torch.float8_e4m3fn
    for M, N, K in ((0, 5, 128), (5, 0, 128), (500, 0, 300), (4, 300, 0), (300, 300, 0), (0, 0, 0)):
        y = api.matmul_fp8(torch.empty(M, K, device="cuda").to(f8), torch.empty(M, -(-K // 128), device="cuda"),
                           torch.empty(N, K, device="cuda").to(f8), torch.empty(-(-N // 128), -(-K // 128), device="cuda"))
        torch.cuda.synchronize()
        assert y.shape == (M, N) and not bool(y.any())


@pytest.mark.parametrize("M", [1, 77, 600])
def test_quantized_product_is_near_the_full_one(api, M):
    """Quantized activations and weights: each value is within half a step of e4m3 of itself
    (2^-4 relative, or 2^-10 of its block's scale, whose 448th is the step's unit), so the
    product is within the sum of what these make."""
    import torch
    x, w = normal(M, 1000, 1, "bfloat16"), normal(400, 1000, 2, "bfloat16")
    x[:, ::97] *= 8
    q, s = api.quantize_blocks(x)
    wq, ws = api.quantize_blocks(w, block_rows=128)
    say("quantized product M=%d" % M)
    y = check_product(api, q, s, wq, ws, "float32")
    X, W = x.double(), w.double()
    ex = torch.maximum(X.abs() * 2.0 ** -4, ref.spread(s, M, 1000, 1) * 2.0 ** -10)
    ew = torch.maximum(W.abs() * 2.0 ** -4, ref.spread(ws, 400, 1000, 128) * 2.0 ** -10)
    bound = ex @ W.abs().t() + X.abs() @ ew.t() + ex @ ew.t() + 1e-4 * (X.abs() @ W.abs().t())
    ref.within(y, X @ W.t(), bound, "quantized product")
