"""Row quantization and the decode of streams to rows, against their definitions in 64
bits.  The int8 values and the scales are functions of the row alone, so every check is
for equality."""
import numpy as np
import pytest

import oracle
from trellis_coded_weight_amd import inputs

from dense_ref import quantize
from helpers import dev, say

pytestmark = pytest.mark.gpu

TYPES = ["float32", "bfloat16", "float16"]


@pytest.fixture(scope="module")
def api():
    import torch
    assert torch.cuda.is_available(), "GPU test without a GPU"
    from trellis_coded_weight_amd import api as a
    return a


def rows(R, C, dtype, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(R, C, generator=g, device="cuda").to(getattr(torch, dtype))


def check(api, x):
    import torch
    q, s = api.quantize_rows(x)
    torch.cuda.synchronize()
    qr, sr = quantize(x.double())
    assert q.shape == x.shape and q.dtype == torch.int8
    assert torch.equal(s, sr)
    assert torch.equal(q, qr)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,C", [(1, 1), (1, 8), (3, 7), (5, 64), (7, 255), (2, 513), (9, 1000), (4, 2049), (1, 4096),
                                 (3, 8193), (2, 14336), (2, 28679), (1, 70000), (1031, 40)])
def test_quantize_rows(api, dtype, R, C):
    say("quantize %dx%d %s" % (R, C, dtype))
    check(api, rows(R, C, dtype, R + C))


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_strided_rows(api, dtype):
    """Slices of wider rows, aligned and not; what lies beside the slice is not read."""
    import torch
    for off, C in ((0, 96), (8, 104), (1, 97), (3, 1025), (16, 1024)):
        wide = rows(6, 2000, dtype, off)
        x = wide[:, off:off + C]
        keep = x.clone()
        wide.fill_(float("nan"))
        wide[:, off:off + C] = keep
        say("quantize strided off=%d C=%d %s" % (off, C, dtype))
        check(api, x)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_half_steps_and_small_rows(api, dtype):
    """Exact halves go to the even integer; magnitudes down to the smallest subnormal."""
    import torch
    t = getattr(torch, dtype)
    # scale exactly 2^e: values at odd multiples of half a step
    steps = torch.arange(-127, 128, device="cuda").double()
    halves = torch.cat([steps, steps[:-1] + 0.5])
    tests = []
    for e in (0, -3, 4):
        tests.append((halves * 2.0 ** e).to(t)[None])
    if dtype == "float32":
        for e in (-148, -140, -126, -110, -101, -100, -99, 120):
            tests.append((halves * 2.0 ** e).to(t)[None])
        # neighbours of the half steps of a scale that is no power of two
        s = torch.tensor(3.0 / 127.0, device="cuda")
        near = (halves[255:] * s.double()).float()
        near = torch.cat([near, torch.nextafter(near, near * 0), torch.nextafter(near, near * 4),
                          torch.tensor([3.0], device="cuda")])
        tests.append(near[None])
    else:
        lowest = 2.0 ** -24 if dtype == "float16" else 2.0 ** -133
        tests.append((halves * lowest).to(t)[None])
    for x in tests:
        say("quantize halves %s max %g" % (dtype, float(x.double().abs().max())))
        check(api, x)
        check(api, x.repeat(5, 5))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("C", [5, 64, 3001])
def test_quantize_zero_and_non_finite_rows(api, dtype, C):
    import torch
    x = rows(6, C, dtype, C)
    x[1] = 0
    x[2, C // 2] = float("inf")
    x[3, C - 1] = float("-inf")
    x[4, 0] = float("nan")
    say("quantize zero and non-finite rows %s C=%d" % (dtype, C))
    q, s = api.quantize_rows(x)
    torch.cuda.synchronize()
    for r in (0, 5):
        qr, sr = quantize(x[r:r + 1].double())
        assert torch.equal(q[r:r + 1], qr) and torch.equal(s[r:r + 1], sr)
    assert float(s[1]) == 0 and not bool(q[1].any())
    for r in (2, 3, 4):
        assert bool(torch.isnan(s[r])) and not bool(q[r].any())


def test_quantize_empty(api):
    import torch
    q, s = api.quantize_rows(torch.empty((0, 16), device="cuda"))
    assert q.shape == (0, 16) and s.shape == (0,)
    q, s = api.quantize_rows(torch.empty((3, 0), device="cuda"))
    torch.cuda.synchronize()
    assert q.shape == (3, 0) and s.tolist() == [0, 0, 0]


# ---- streams to rows ---------------------------------------------------------------------------

CODES = {"1mad": "1mad", "3inst": "3inst", "xor": None}


def streams(api, M, N, L, tb, seed):
    import torch
    W = api.tailbiting_words(L, 2, 256) if tb else api.bitstream_words(L, 2, 256)
    g = np.random.default_rng(seed)
    words = g.integers(0, 2 ** 32, ((M // 16) * (N // 16), W), dtype=np.uint64).astype(np.uint32)
    return torch.from_numpy(words.view(np.int32)).cuda()


def code_arg(code, L):
    return ("xor", inputs.xor_masks(L)) if code == "xor" else code


def as_matrix(recon, M, N):
    return recon.reshape(M // 16, N // 16, 16, 16).permute(0, 2, 1, 3).reshape(M, N)


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("code", ["1mad", "3inst", "xor"])
@pytest.mark.parametrize("L", [6, 8, 10, 12, 14, 16])
def test_decode_matrix(api, L, code, tb):
    """Every trellis size and code: the decoded tiles (checked bit for bit against the
    oracle elsewhere) as rows, in each type."""
    import torch
    c = code_arg(code, L)
    for M, N in ((16, 16), (48, 4096 + 16), (32, 80)):
        bits = streams(api, M, N, L, tb, L + M)
        dec = api.tailbiting_decode if tb else api.decode
        ref = as_matrix(dec(bits, 256, L=L, code=c)[0], M, N)
        say("decode_matrix L=%d %s tb=%s %dx%d" % (L, code, tb, M, N))
        for t in (torch.float32, torch.bfloat16, torch.float16):
            w = api.decode_matrix(bits, M, N, L=L, code=c, tailbiting=tb, dtype=t)
            torch.cuda.synchronize()
            assert torch.equal(w, ref.to(t))
        q, s = api.decode_matrix(bits, M, N, L=L, code=c, tailbiting=tb)
        torch.cuda.synchronize()
        qr, sr = quantize(ref.double())
        assert torch.equal(s, sr)
        assert torch.equal(q, qr)


def test_decode_matrix_against_oracle(api):
    """One matrix of encoded weights against the oracle's decode."""
    import torch
    M, N, L = 64, 96, 16
    s = inputs.targets((M // 16) * (N // 16), 256, 7)
    say("decode_matrix against the oracle")
    bits, _, _ = api.encode(dev(s), L=L)
    w = api.decode_matrix(bits, M, N, L=L, dtype=torch.float32)
    q, sc = api.decode_matrix(bits, M, N, L=L)
    torch.cuda.synchronize()
    _, rec = oracle.decode(bits.cpu().numpy().view(np.uint32), 256, oracle.code_table("1mad", L), L, 2)
    ref = oracle.tiles_to_matrix(rec, M, N)
    assert np.array_equal(w.cpu().numpy(), ref)
    qr, sr = quantize(torch.from_numpy(ref).double())
    assert torch.equal(q.cpu(), qr) and torch.equal(sc.cpu(), sr)


def test_decode_matrix_row_stride_and_zero_rows(api):
    """Rows of a wider buffer, which keeps what lies beside them; XOR palette rows of zeros
    (masks of zero leave palette 0 and the branch as the entry, whose entry 2 is 0) have
    scale 0."""
    import torch
    from trellis_coded_weight_amd import _native as nat
    M, N = 32, 48
    bits = streams(api, M, N, 16, True, 3)
    q, s = api.decode_matrix(bits, M, N, tailbiting=True)
    wide = torch.full((M, 112), 99, dtype=torch.int8, device="cuda")
    s2 = torch.empty(M, device="cuda")
    say("decode_matrix row stride")
    nat.qtcq_decode_matrix(bits.data_ptr(), M, N, 16, 2, nat.QTCQ_CODE_1MAD, True, nat.QTCQ_I8,
                           wide.data_ptr() + 32, 112, s2.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(wide[:, 32:32 + N], q) and torch.equal(s, s2)
    assert bool((wide[:, :32] == 99).all()) and bool((wide[:, 32 + N:] == 99).all())
    # every 2-bit branch 2: words of 0b1010...
    bits.fill_(-0x55555556)
    q, s = api.decode_matrix(bits, M, N, code=("xor", (0, 0, 0, 0)), tailbiting=True)
    torch.cuda.synchronize()
    assert not bool(q.any()) and not bool(s.any())


def test_decode_matrix_empty(api):
    import torch
    none = torch.empty((0, 17), dtype=torch.int32, device="cuda")
    q, s = api.decode_matrix(none, 0, 32)
    assert q.shape == (0, 32) and s.shape == (0,)
    q, s = api.decode_matrix(none, 32, 0)
    torch.cuda.synchronize()
    assert q.shape == (32, 0) and not bool(s.any())
