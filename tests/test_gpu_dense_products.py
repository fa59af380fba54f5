"""The 8-bit product, the gated projections and their gradients against 64-bit forms, at
the sizes, strides, types and values where tiles, tails and epilogues can go wrong."""
import pytest

from trellis_coded_weight_amd import inputs

import dense_ref as ref
from helpers import dev, say

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu", "gelu_tanh", "relu", "sigmoid"]
# rows that are whole 16-byte chunks and rows that are not, tiles with every kind of edge,
# a single row, column or term, batches on both sides of each choice of kernel
SIZES = [(1, 1, 1), (1, 16, 64), (1, 33, 129), (2, 256, 512), (5, 100, 24), (8, 1000, 1024), (16, 130, 4096),
         (17, 64, 136), (31, 513, 520), (33, 520, 1000), (64, 128, 256), (65, 127, 255), (96, 704, 320),
         (128, 256, 64), (129, 257, 65), (200, 48, 2056), (256, 512, 768), (300, 1032, 328), (512, 256, 1024),
         (1, 5000, 16), (4, 24, 14336), (100, 264, 4104), (150, 130, 5001), (70, 2000, 72)]


@pytest.fixture(scope="module")
def api():
    import torch
    assert torch.cuda.is_available(), "GPU test without a GPU"
    from trellis_coded_weight_amd import api as a
    return a


def gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(r, c, seed, wide=False):
    """8-bit integers; wide: in a buffer of longer rows, surrounded by other values."""
    import torch
    t = torch.randint(-128, 128, (r, c + 37), generator=gen(seed), device="cuda", dtype=torch.int8)
    return t[:, 5:5 + c] if wide else t[:, :c].contiguous()


def scales(n, seed):
    import torch
    return torch.rand(n, generator=gen(seed), device="cuda") * 0.02 + 1e-3


def halves(r, c, dtype, seed, scale=1.0, wide=0):
    """wide > 0: in a buffer of rows `wide` longer, NaN beside the slice."""
    import torch
    v = (torch.randn(r, c, generator=gen(seed), device="cuda") * scale).to(dtype)
    if not wide:
        return v
    t = torch.full((r, c + wide), float("nan"), dtype=dtype, device="cuda")
    t[:, wide // 2:wide // 2 + c] = v
    return t[:, wide // 2:wide // 2 + c]


def dtype_of(name):
    import torch
    return getattr(torch, name)


# ---- 8-bit product -----------------------------------------------------------------------------

def check_int8(api, a, sa, w, sw, dtype):
    import torch
    y = api.matmul_int8(a, sa, w, sw, dtype=dtype)
    torch.cuda.synchronize()
    # the sum is exact; its conversion and two products round to binary32, in this order
    want = ((a.double() @ w.double().t()).float() * sa[:, None] * sw).to(dtype)
    assert y.dtype == dtype and torch.equal(y, want), (a.shape, w.shape)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul_int8(api, M, N, K, dtype):
    say("matmul_int8 %dx%dx%d %s" % (M, N, K, dtype))
    check_int8(api, ints(M, K, 1), scales(M, 2), ints(N, K, 3), scales(N, 4), dtype_of(dtype))


@pytest.mark.parametrize("M,N,K", [(1, 70, 100), (40, 200, 333), (130, 300, 512), (7, 64, 64), (600, 300, 200)])
def test_matmul_int8_strided(api, M, N, K):
    say("matmul_int8 strided %dx%dx%d" % (M, N, K))
    check_int8(api, ints(M, K, 1, True), scales(M, 2), ints(N, K, 3, True), scales(N, 4), dtype_of("float32"))


@pytest.mark.parametrize("M", [1, 40, 300])
def test_matmul_int8_largest_sums(api, M):
    """Every product -128 * -128 at the longest sum: just below 2^31."""
    import torch
    K, N = 131071, 48
    a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    say("matmul_int8 largest sums M=%d" % M)
    y = api.matmul_int8(a, torch.ones(M, device="cuda"), w, torch.ones(N, device="cuda"))
    torch.cuda.synchronize()
    assert bool((y == float(K * 16384)).all())


def test_matmul_int8_row_does_not_depend_on_the_batch(api):
    import torch
    M, N, K = 700, 260, 1024
    a, sa, w, sw = ints(M, K, 1), scales(M, 2), ints(N, K, 3), scales(N, 4)
    say("matmul_int8 batches")
    y = api.matmul_int8(a, sa, w, sw)
    for lo, hi in ((0, 1), (5, 21), (100, 164), (200, 460)):
        assert torch.equal(api.matmul_int8(a[lo:hi], sa[lo:hi], w, sw), y[lo:hi])


@pytest.mark.parametrize("M,N,K", [(3, 40, 128), (150, 140, 128)])
def test_matmul_int8_non_finite_scales(api, M, N, K):
    """A NaN token scale reaches that token's row, an infinite channel scale that column."""
    import torch
    a, sa, w, sw = ints(M, K, 1), scales(M, 2), ints(N, K, 3), scales(N, 4)
    a[0] = 0                                                     # 0 * inf is NaN
    clean = api.matmul_int8(a, sa, w, sw)
    sa[1], sw[5] = float("nan"), float("inf")
    say("matmul_int8 non-finite scales")
    y = api.matmul_int8(a, sa, w, sw)
    torch.cuda.synchronize()
    want = (a.double() @ w.double().t()).float() * sa[:, None] * sw
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[0, 5]))
    keep = [i for i in range(M) if i != 1]
    cols = [j for j in range(N) if j != 5]
    assert torch.equal(y[keep][:, cols], clean[keep][:, cols])


# ---- gated projections -------------------------------------------------------------------------

def check_gated(api, x, wg, wu, act):
    import torch
    h, gate, up = api.gated(x, wg, wu, activation=act, save=True)
    only = api.gated(x, wg, wu, activation=act)
    torch.cuda.synchronize()
    want, e, g, u, eg, eu = ref.gated(x, wg, wu, act)
    ref.within(gate, g, eg, "gate")
    ref.within(up, u, eu, "up")
    ref.within(h, want, e, "h")
    assert torch.equal(h, only)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("M,F,K", SIZES)
def test_gated(api, M, F, K, dtype):
    t = dtype_of(dtype)
    say("gated %dx%dx%d %s" % (M, F, K, dtype))
    check_gated(api, halves(M, K, t, 1), halves(F, K, t, 2, K ** -0.5), halves(F, K, t, 3, K ** -0.5), "silu")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 24, 150, 300])
def test_gated_activations(api, M, act):
    t = dtype_of("float16")
    F, K = 264, 72
    say("gated %s M=%d" % (act, M))
    check_gated(api, halves(M, K, t, 1), halves(F, K, t, 2, 0.2), halves(F, K, t, 3, 0.2), act)


@pytest.mark.parametrize("wide", [6, 16, 64])
@pytest.mark.parametrize("M,F,K", [(1, 70, 200), (20, 90, 128), (140, 130, 136), (300, 300, 264)])
def test_gated_strided(api, M, F, K, wide):
    """Slices of wider rows with NaN beside them."""
    t = dtype_of("bfloat16")
    say("gated strided %dx%dx%d wide=%d" % (M, F, K, wide))
    check_gated(api, halves(M, K, t, 1, wide=wide), halves(F, K, t, 2, K ** -0.5, wide),
                halves(F, K, t, 3, K ** -0.5, wide), "gelu")


@pytest.mark.parametrize("M,F,K", [(1, 96, 64), (1, 90, 63), (50, 90, 128), (300, 260, 64)])
def test_gated_halves_of_one_matrix(api, M, F, K):
    t = dtype_of("bfloat16")
    w = halves(2 * F, K, t, 2, K ** -0.5)
    say("gated halves of one matrix %dx%dx%d" % (M, F, K))
    check_gated(api, halves(M, K, t, 1), w[:F], w[F:], "silu")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [2, 140, 300])
def test_gated_large_and_non_finite(api, M, act):
    """Saturated gates of either sign give the formula's finite values; infinities and NaN
    stay in their own row and column."""
    import torch
    t = dtype_of("bfloat16")
    F, K = 132, 64
    x, wg, wu = halves(M, K, t, 1), halves(F, K, t, 2, 20.0), halves(F, K, t, 3, 0.1)
    say("gated large %s M=%d" % (act, M))
    h = api.gated(x, wg, wu, activation=act)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(h).all())
    want, e, g, *_ = ref.gated(x, wg, wu, act)
    sure = g.abs() > 60                                  # saturated: act(g) is g or 0 (1 or 0)
    ref.within(h[sure].reshape(1, -1), want[sure].reshape(1, -1), e[sure].reshape(1, -1), "saturated")
    clean = h.clone()
    x[1, 3] = float("nan")
    wg[7, 2] = float("inf")
    h = api.gated(x, wg, wu, activation=act)
    torch.cuda.synchronize()
    assert bool(torch.isnan(h[1]).all())
    rows = [i for i in range(M) if i != 1]
    cols = [j for j in range(F) if j != 7]
    assert torch.equal(h[rows][:, cols], clean[rows][:, cols])


@pytest.mark.parametrize("M,F,K", [(3, 50, 70), (200, 200, 96), (300, 300, 64)])
def test_results_stay_inside_their_rows(M, F, K):
    """Row strides above the row length: what lies between rows, before the first and after
    the last is left as it was."""
    import torch
    from trellis_coded_weight_amd import _native as nat
    t = torch.bfloat16
    st = torch.cuda.current_stream().cuda_stream
    x, wg, wu = halves(M, K, t, 1), halves(F, K, t, 2, 0.1), halves(F, K, t, 3, 0.1)
    from trellis_coded_weight_amd import api
    h, gate, up = api.gated(x, wg, wu, save=True)
    gh = halves(M, F, t, 4)
    gx, gwg, gwu = api.gated_vjp(x, wg, wu, gate, up, gh)

    def buf(r, c):
        return torch.full((r + 2, c + 9), 77.0, dtype=t, device="cuda")

    def same(b, want):
        r, c = want.shape
        assert torch.equal(b[1:1 + r, 3:3 + c], want)
        b[1:1 + r, 3:3 + c] = 77.0
        assert bool((b == 77.0).all())

    def at(b):
        return b.data_ptr() + 2 * (b.shape[1] + 3)

    bh, bg, bu = buf(M, F), buf(M, F), buf(M, F)
    wf, w8 = api.gated_workspace(M, F, K), api.matmul_int8_workspace(M, F, K)
    say("gated inside rows %dx%dx%d" % (M, F, K))
    nat.qtcq_gated_forward(x.data_ptr(), K, wg.data_ptr(), wu.data_ptr(), K, nat.QTCQ_BF16, M, F, K,
                           nat.QTCQ_ACT_SILU, at(bh), F + 9, at(bg), at(bu), F + 9, wf.data_ptr(), wf.numel(), st)
    bx, bwg, bwu = buf(M, K), buf(F, K), buf(F, K)
    ws = api.gated_vjp_workspace(M, F, K)
    nat.qtcq_gated_vjp(x.data_ptr(), K, wg.data_ptr(), wu.data_ptr(), K, at(bg), at(bu), F + 9, gh.data_ptr(), F,
                       nat.QTCQ_BF16, M, F, K, nat.QTCQ_ACT_SILU, at(bx), K + 9, at(bwg), at(bwu), K + 9,
                       ws.data_ptr(), ws.numel(), st)
    a, w = ints(M, K, 5), ints(F, K, 6)
    sa, sw = scales(M, 7), scales(F, 8)
    by = buf(M, F)
    nat.qtcq_matmul_int8(a.data_ptr(), K, sa.data_ptr(), w.data_ptr(), K, sw.data_ptr(), M, F, K, nat.QTCQ_BF16,
                         at(by), F + 9, w8.data_ptr(), w8.numel(), st)
    torch.cuda.synchronize()
    for b, want in ((bh, h), (bg, gate), (bu, up), (bx, gx), (bwg, gwg), (bwu, gwu),
                    (by, api.matmul_int8(a, sa, w, sw, dtype=t))):
        same(b, want)


# ---- gradients ---------------------------------------------------------------------------------

def vjp_inputs(M, F, K, t, seed, wide=0):
    return (halves(M, K, t, seed, wide=wide), halves(F, K, t, seed + 1, K ** -0.5, wide),
            halves(F, K, t, seed + 2, K ** -0.5, wide), halves(M, F, t, seed + 3, wide=wide),
            halves(M, F, t, seed + 4, wide=wide), halves(M, F, t, seed + 5, 0.5, wide))


def check_vjp(api, args, act):
    import torch
    got = api.gated_vjp(*args, activation=act)
    torch.cuda.synchronize()
    for name, g, (want, e) in zip(("grad_x", "grad_w_gate", "grad_w_up"), got, ref.gated_vjp(*args, act)):
        ref.within(g, want, e, name)
    return got


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("M,F,K", SIZES)
def test_gated_vjp(api, M, F, K, dtype):
    say("gated_vjp %dx%dx%d %s" % (M, F, K, dtype))
    check_vjp(api, vjp_inputs(M, F, K, dtype_of(dtype), 1), "silu")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,F,K", [(3, 72, 40), (140, 264, 136), (264, 300, 520)])
def test_gated_vjp_activations(api, M, F, K, act):
    say("gated_vjp %s %dx%dx%d" % (act, M, F, K))
    check_vjp(api, vjp_inputs(M, F, K, dtype_of("float16"), 7), act)


@pytest.mark.parametrize("wide", [6, 16])
@pytest.mark.parametrize("M,F,K", [(1, 70, 200), (140, 130, 136), (300, 272, 264)])
def test_gated_vjp_strided(api, M, F, K, wide):
    say("gated_vjp strided %dx%dx%d wide=%d" % (M, F, K, wide))
    check_vjp(api, vjp_inputs(M, F, K, dtype_of("bfloat16"), 3, wide), "gelu_tanh")


@pytest.mark.parametrize("M,F,K", [(9, 80, 48), (300, 264, 256)])
def test_gated_vjp_parts(api, M, F, K):
    """Either half alone gives the same bits."""
    import torch
    args = vjp_inputs(M, F, K, dtype_of("bfloat16"), 11)
    say("gated_vjp parts %dx%dx%d" % (M, F, K))
    gx, gg, gu = api.gated_vjp(*args)
    x1, n1, n2 = api.gated_vjp(*args, want_w=False)
    n3, g1, u1 = api.gated_vjp(*args, want_x=False)
    torch.cuda.synchronize()
    assert n1 is None and n2 is None and n3 is None
    assert torch.equal(gx, x1) and torch.equal(gg, g1) and torch.equal(gu, u1)


@pytest.mark.parametrize("act", ACTS)
def test_gated_vjp_against_differences(api, act):
    """Inputs whose projections are exact in 16 bits (few, small multiples of powers of two):
    the gradients' products with a direction are the loss's central differences in 64 bits.
    Bound: the gradients' own bounds along the direction, and the differences' truncation,
    (step^2 / 6) times a third derivative that stays below 100 sum |.| here, and rounding."""
    import torch
    t = torch.bfloat16
    M, F, K = 5, 24, 8
    g = gen(5)
    x = torch.randint(-1, 2, (M, K), generator=g, device="cuda").to(t)
    wg, wu = (torch.randint(-4, 5, (F, K), generator=g, device="cuda").div(8).to(t) for _ in range(2))
    gh = torch.randint(-4, 5, (M, F), generator=g, device="cuda").div(4).to(t)
    say("gated_vjp differences %s" % act)
    h, gate, up = api.gated(x, wg, wu, activation=act, save=True)
    assert torch.equal(gate.double(), x.double() @ wg.double().t())
    assert torch.equal(up.double(), x.double() @ wu.double().t())
    grads = check_vjp(api, (x, wg, wu, gate, up, gh), act)
    bounds = ref.gated_vjp(x, wg, wu, gate, up, gh, act)

    def loss(X, G, W):
        return (gh.double() * ref.act(X @ G.t(), act)[0] * (X @ W.t())).sum()

    base = [x.double(), wg.double(), wu.double()]
    step = 2.0 ** -13
    for i in range(3):
        v = torch.randn(base[i].shape, generator=g, device="cuda", dtype=torch.float64)
        if act == "relu" and i < 2:
            # a gate of 0 has a kink: leave out directions that cross it
            d = v @ base[1].t() if i == 0 else base[0] @ v.t()
            if bool(((gate.double() == 0) & (d != 0) & (gh != 0) & (up != 0)).any()):
                continue
        hi, lo = list(base), list(base)
        hi[i], lo[i] = base[i] + step * v, base[i] - step * v
        want = float((loss(*hi) - loss(*lo)) / (2 * step))
        got = float((grads[i].double() * v).sum())
        size = float((gh.abs().sum()) * (1 + v.abs().max()) ** 3)
        tol = float((bounds[i][1] * v.abs()).sum()) + 100 * step * step * size
        assert abs(got - want) <= tol, (act, i, got, want, tol)


def test_gated_empty(api):
    import torch
    t = torch.bfloat16

    def e(r, c):
        return torch.zeros((r, c), dtype=t, device="cuda")

    assert api.gated(e(0, 8), e(4, 8), e(4, 8)).shape == (0, 4)
    assert api.gated(e(3, 8), e(0, 8), e(0, 8)).shape == (3, 0)
    h = api.gated(e(3, 0), e(4, 0), e(4, 0), activation="sigmoid")
    torch.cuda.synchronize()
    assert h.shape == (3, 4) and not bool(h.any())
    gx, gg, gu = api.gated_vjp(e(0, 8), e(4, 8), e(4, 8), e(0, 4), e(0, 4), e(0, 4))
    torch.cuda.synchronize()
    assert gx.shape == (0, 8) and not bool(gg.any()) and not bool(gu.any())
    gx, gg, gu = api.gated_vjp(e(3, 8), e(0, 8), e(0, 8), e(3, 0), e(3, 0), e(3, 0))
    torch.cuda.synchronize()
    assert not bool(gx.any()) and gg.shape == (0, 8)
    y = api.matmul_int8(torch.zeros((3, 0), dtype=torch.int8, device="cuda"), torch.ones(3, device="cuda"),
                        torch.zeros((5, 0), dtype=torch.int8, device="cuda"), torch.ones(5, device="cuda"))
    torch.cuda.synchronize()
    assert y.shape == (3, 5) and not bool(y.any())


# ---- together ----------------------------------------------------------------------------------

def test_coded_weights_through_the_8_bit_product(api):
    """Encode a matrix, decode it to 8-bit rows, quantize activations and multiply: within
    the quantization's own error of the decode -> product kernel.  |x - q s| <= s / 2 for both
    operands, so the product is off by at most sum |x| sw/2 + |w| sx/2 + sx sw/4 (plus the
    binary32 roundings of either side, below 100 U sum |x w| here)."""
    import torch
    M, N, L = 96, 160, 12
    bits, _, _ = api.tailbiting_encode(dev(inputs.targets((M // 16) * (N // 16), 256, 5)), L=L)
    x = dev(inputs.targets(6, N, 6))
    say("coded weights through the 8-bit product")
    y0 = api.decode_matvec(bits, M, N, x, L=L, tailbiting=True)
    w, sw = api.decode_matrix(bits, M, N, L=L, tailbiting=True)
    a, sa = api.quantize_rows(x)
    y = api.matmul_int8(a, sa, w, sw)
    w32 = api.decode_matrix(bits, M, N, L=L, tailbiting=True, dtype=torch.float32)
    torch.cuda.synchronize()
    X, W = x.double().abs(), w32.double().abs()
    e = (X.sum(1)[:, None] * sw.double() / 2 + W.sum(1) * sa.double()[:, None] / 2
         + N * sa.double()[:, None] * sw.double() / 4 + 100 * ref.U * (X @ W.t()))
    ref.within(y, y0.double(), e, "8-bit product")


def test_soft_codewords_through_the_gated_projections(api):
    """A training step of soft-coded weights: soft codewords to 16-bit rows, the gated
    projections, their gradients, and the weight gradient back through the soft codeword.
    The last step is checked by its own test; here the chain's gradient is the product of
    the parts' and reaches every target."""
    import torch
    F, K, M, L = 32, 48, 12, 8
    t = torch.bfloat16
    n = (F // 16) * (K // 16)
    say("soft codewords through the gated projections")
    seq = [dev(inputs.targets(n, 256, s)) for s in (1, 2)]
    soft = [api.bcjr_soft(s, 0.5, L=L)[0] for s in seq]

    def to_rows(v):
        return v.reshape(F // 16, K // 16, 16, 16).permute(0, 2, 1, 3).reshape(F, K)

    wg, wu = ((to_rows(s) / K ** 0.5).to(t).contiguous() for s in soft)
    x, gh = halves(M, K, t, 3), halves(M, F, t, 4)
    h, gate, up = api.gated(x, wg, wu, save=True)
    gx, gwg, gwu = check_vjp(api, (x, wg, wu, gate, up, gh), "silu")
    for s, gw in zip(seq, (gwg, gwu)):
        g = (gw.float() / K ** 0.5).reshape(F // 16, 16, K // 16, 16).permute(0, 2, 1, 3).reshape(n, 256).contiguous()
        gs, _, _ = api.bcjr_vjp(s, 0.5, g, L=L)
        torch.cuda.synchronize()
        assert bool(torch.isfinite(gs).all()) and bool((gs.abs().amax(1) > 0).all())


def chain(api, x, bits_g, bits_u, gh, M, F, K):
    """8-bit and 16-bit paths of one feed-forward in a row."""
    import torch
    wg = api.decode_matrix(bits_g, F, K, dtype=torch.bfloat16)
    wu = api.decode_matrix(bits_u, F, K, dtype=torch.bfloat16)
    h, gate, up = api.gated(x, wg, wu, save=True)
    grads = api.gated_vjp(x, wg, wu, gate, up, gh)
    q, s = api.quantize_rows(x)
    w8, s8 = api.decode_matrix(bits_g, F, K)
    return (h, gate, up) + tuple(grads) + (q, s, w8, s8, api.matmul_int8(q, s, w8, s8))


def coded(n, seed):
    import torch
    return torch.randint(-2 ** 31, 2 ** 31, (n, 17), generator=gen(seed), device="cuda", dtype=torch.int64).to(torch.int32)


@pytest.mark.parametrize("M,F,K", [(1, 96, 64), (40, 128, 512), (300, 256, 320)])
def test_dense_chain_in_a_graph(api, M, F, K):
    """Captured once, replayed on new inputs with eager work between, the same bits as the
    eager calls each time."""
    import torch
    from test_gpu_graphs import capture
    n = (F // 16) * (K // 16)
    t = torch.bfloat16
    x, gh, bg, bu = halves(M, K, t, 1), halves(M, F, t, 2), coded(n, 3), coded(n, 4)
    say("dense chain in a graph %dx%dx%d" % (M, F, K))
    graph, out = capture(lambda: chain(api, x, bg, bu, gh, M, F, K))
    for rep in range(3):
        x.copy_(halves(M, K, t, 10 + rep))
        gh.copy_(halves(M, F, t, 20 + rep))
        bg.copy_(coded(n, 30 + rep))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, chain(api, x, bg, bu, gh, M, F, K)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M,F,K", [(2, 70, 333), (90, 130, 2999), (300, 75, 1001)])
def test_odd_rows_in_a_graph(api, M, F, K):
    """Rows that are copied into the workspace first, and shares of k, captured and replayed."""
    import torch
    from test_gpu_graphs import capture
    t = torch.float16
    args = list(vjp_inputs(M, F, K, t, 1))
    a, w = ints(M, K, 8), ints(F, K, 9)
    sa, sw = scales(M, 10), scales(F, 11)

    def step():
        return (api.matmul_int8(a, sa, w, sw), api.gated(*args[:3])) + api.gated_vjp(*args)

    say("odd rows in a graph %dx%dx%d" % (M, F, K))
    graph, out = capture(step)
    for rep in range(3):
        for x, y in zip(args, vjp_inputs(M, F, K, t, 20 + rep)):
            x.copy_(y)
        a.copy_(ints(M, K, 30 + rep))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, step()):
            assert torch.equal(x, y)


@pytest.mark.parametrize("M,F,K", [(100, 64, 4096), (100, 70, 4099)])
def test_given_workspaces(api, M, F, K):
    """A workspace of the caller's gives the same bits and serves one call after another; one
    that is too small, or not on 16 bytes, is refused."""
    import torch
    t = torch.bfloat16
    args = vjp_inputs(M, F, K, t, 1)
    a, w = ints(M, K, 8), ints(F, K, 9)
    sa, sw = scales(M, 10), scales(F, 11)
    w8, wg, wv = api.matmul_int8_workspace(M, F, K), api.gated_workspace(M, F, K), api.gated_vjp_workspace(M, F, K)
    one = torch.empty(max(x.numel() for x in (w8, wg, wv)) + 16, dtype=torch.uint8, device="cuda")
    say("given workspaces %dx%dx%d" % (M, F, K))
    want = (api.matmul_int8(a, sa, w, sw), api.gated(*args[:3])) + api.gated_vjp(*args)
    for ws in ((w8, wg, wv), (one[:-16],) * 3):
        for x in ws:
            x.fill_(0xFF)                                        # what is in it does not matter
        got = (api.matmul_int8(a, sa, w, sw, workspace=ws[0]), api.gated(*args[:3], workspace=ws[1])) + \
            api.gated_vjp(*args, workspace=ws[2])
        torch.cuda.synchronize()
        for x, y in zip(want, got):
            assert torch.equal(x, y)
    for bad in (one[:64], one[8:]):
        for call in (lambda: api.matmul_int8(a, sa, w, sw, workspace=bad), lambda: api.gated(*args[:3], workspace=bad),
                     lambda: api.gated_vjp(*args, workspace=bad)):
            with pytest.raises(RuntimeError, match="workspace"):
                call()


@pytest.mark.parametrize("stride", [1 << 21, (1 << 21) + 8])
def test_rows_far_apart(api, stride):
    """Rows 4 MB apart, the most that is read where it is, and a little more, which is copied."""
    import torch
    t = torch.bfloat16
    M, F, K = 130, 260, 72

    def apart(v, ld):
        o = torch.empty_strided(v.shape, (ld, 1), dtype=v.dtype, device="cuda")
        o.copy_(v)
        return o

    say("rows far apart, stride %d" % stride)
    x, wg, wu, gate, up, gh = vjp_inputs(M, F, K, t, 1)
    far = (apart(x, stride), apart(wg, stride), apart(wu, stride))
    assert torch.equal(api.gated(*far), api.gated(x, wg, wu))
    for a, b in zip(api.gated_vjp(*far, gate, up, gh), api.gated_vjp(x, wg, wu, gate, up, gh)):
        assert torch.equal(a, b)
    a, w = ints(M, 64, 8), ints(F, 64, 9)
    sa, sw = scales(M, 10), scales(F, 11)
    y = api.matmul_int8(apart(a, 2 * stride), sa, apart(w, 2 * stride), sw)
    torch.cuda.synchronize()
    assert torch.equal(y, api.matmul_int8(a, sa, w, sw))


def test_dense_chains_on_two_streams(api):
    """Two chains at once on streams of their own, each with its own workspace."""
    import torch
    t = torch.bfloat16
    M, F, K = 130, 256, 512
    n = (F // 16) * (K // 16)
    sets = [(halves(M, K, t, s), coded(n, s + 1), coded(n, s + 2), halves(M, F, t, s + 3)) for s in (1, 11)]
    say("dense chains on two streams")
    want = [chain(api, x, bg, bu, gh, M, F, K) for x, bg, bu, gh in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(3):
        got = []
        for st, (x, bg, bu, gh) in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(chain(api, x, bg, bu, gh, M, F, K))
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            for a, b in zip(w, g):
                assert torch.equal(a, b)


def test_wrappers_refuse(api):
    """Shapes, types and layouts the kernels do not take raise before any launch."""
    import torch
    bf, dv = torch.bfloat16, "cuda"
    x, w = torch.zeros((4, 32), dtype=bf, device=dv), torch.zeros((8, 32), dtype=bf, device=dv)
    p = torch.zeros((4, 8), dtype=bf, device=dv)
    i8, one = torch.zeros((4, 32), dtype=torch.int8, device=dv), torch.ones(4, device=dv)
    for call in (
            lambda: api.quantize_rows(torch.zeros((4, 4), dtype=torch.float64, device=dv)),
            lambda: api.quantize_rows(torch.zeros(4, device=dv)),
            lambda: api.quantize_rows(torch.zeros((4, 4))),
            lambda: api.quantize_rows(x.t()),
            lambda: api.quantize_rows(torch.zeros((1, 8), device=dv).expand(4, 8)),
            lambda: api.decode_matrix(torch.zeros((3, 17), dtype=torch.int32, device=dv), 32, 32),
            lambda: api.decode_matrix(torch.zeros((4, 17), dtype=torch.int32, device=dv), 24, 32),
            lambda: api.decode_matrix(torch.zeros((4, 17), dtype=torch.int32, device=dv), 32, 32, dtype=torch.float64),
            lambda: api.matmul_int8(i8, one, i8[:, :16], one),
            lambda: api.matmul_int8(i8.float(), one, i8, one),
            lambda: api.matmul_int8(i8, one[:3], i8, one),
            lambda: api.matmul_int8(i8, one.double(), i8, one),
            lambda: api.matmul_int8(i8, one, i8, one, dtype=torch.int32),
            lambda: api.gated(x.float(), w.float(), w.float()),
            lambda: api.gated(x, w.half(), w.half()),
            lambda: api.gated(x, w[:, :16], w[:, :16]),
            lambda: api.gated(x, w, w[:4]),
            lambda: api.gated(x, w, w, activation="tanh"),
            lambda: api.gated(x, w, torch.zeros((8, 40), dtype=bf, device=dv)[:, :32]),
            lambda: api.gated_vjp(x, w, w, p, p[:, :4], p),
            lambda: api.gated_vjp(x, w, w, p, p, p.float()),
            lambda: api.gated_vjp(x, w, w, p[:3], p[:3], p[:3]),
            lambda: api.gated_vjp(x, w, w, p, p, p, workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(RuntimeError, match="workspace"):
        api.gated_vjp(x, w, w, p, p, p, workspace=torch.empty(16, dtype=torch.uint8, device=dv))
    torch.cuda.synchronize()
