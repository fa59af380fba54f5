"""Grids of the model operators' launches, from the smallest sizes to the largest accepted: every
launch has blocks and stays below 2^32 threads, the most a launch holds; and every kernel that
is built is launched by the sizes that the GPU tests run.  No GPU needed."""
import os
import re

import pytest

import model_launches
import model_variants
import test_gpu_blocks
import test_gpu_distill
import test_gpu_layer_norm

F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    if not os.path.exists(model_launches.HIPCC):
        pytest.skip("hipcc not installed")
    return model_launches.build(str(tmp_path_factory.mktemp("launches")))


def every_size():
    dims = [1, 2, 63, 127, 129, 768, 769, 1000, 8192, 28672, 131071, (1 << 20) + 3, 1 << 24]
    calls = []
    for m in dims:
        for n in dims:
            calls += ["blocks %d %d %d %d" % (t, m, n, r) for t in (F32, F16) for r in (1, 128)]
            calls += ["norm %d %d %d %d" % (t, w, m, n) for t, w in ((F32, F32), (BF16, F32), (F16, F16))]
            calls += ["norm_vjp %d 0 %d %d %d" % (t, m, n, o) for t in (F32, BF16) for o in (1, 2, 3)]
            calls += ["distill %d %d %d %d %d" % (t, m, n, k, g) for t in (F32, F16) for k in (0, 1024) for g in (0, 1)]
            calls += ["distill_vjp %d %d %d %d" % (t, m, n, 64) for t in (F32, F16)]
            calls += ["fp8 %d %d %d %d %d" % (t, m, n, k, al) for t in (F32, BF16) for k in dims
                      for al in range(2 - (k % 16 != 0))]
    return calls


def test_every_grid_fits_a_launch(recorder):
    calls = every_size()
    accepted = 0
    for call, (status, launches) in zip(calls, model_launches.record(recorder, calls)):
        if status != 0:
            assert status == 2 and not launches, call
            continue
        accepted += 1
        assert launches, call
        for name, x, y, block in launches:
            x, y, block = int(x), int(y), int(block)
            assert 0 < x and 0 < y < 1 << 16 and x * y * block < 1 << 32, (call, name, x, y, block)
    assert accepted > len(calls) // 4


def test_plans_are_whole(recorder):
    """Over sizes from 0 to the limits: a tile the kernels have, shares that cover every block of
    k and are none of them empty, scratch that holds the shares' sums and the copies."""
    dims = [0, 1, 2, 16, 17, 64, 65, 129, 1000, 4096, 28672, 131071, (1 << 20) + 3, 1 << 22]
    calls = ["plan %d %d %d %d %d" % (m, n, k, o, d) for m in dims for n in dims for k in dims
             for o in (0, 1) for d in (0, 1) if -(-m // 128) * -(-n // 64) <= 1 << 22]
    for call, (_, [words]) in zip(calls, model_launches.record(recorder, calls)):
        m, n, k, whole, precise = map(int, call.split()[1:])
        skinny, fp, qg, shares, steps, pitch, part, a, w = map(int, words)
        if skinny:
            assert (m <= 64 or n == 0) and part == a == w == 0, call
            continue
        assert (fp, qg) in ((2, 2), (2, 4), (4, 2), (4, 4)) + (() if precise else ((8, 4),)), call
        blocks = -(-k // 128)
        assert shares >= 1 and steps >= 1 and shares * steps >= blocks, call
        assert shares == 1 or (shares - 1) * steps < blocks, call
        assert pitch % 4 == 0 and pitch >= n and part % 256 == a % 256 == w % 256 == 0, call
        assert part == 0 if shares == 1 else part >= shares * m * pitch * 4, call
        assert a >= m * (-(-k // 16) * 16) and w >= n * (-(-k // 16) * 16), call


def test_sizes_that_reach_every_kernel(recorder):
    families = ("quantize_row_blocks", "quantize_square_blocks", "fp8_", "layer_norm", "norm_column_sums",
                "join_norm_sums", "distill_", "pad_rows")
    built = {w[0] for w in model_launches.record(recorder, ["kernels"])[0][1] if any(f in w[0] for f in families)}
    assert len(built) > 150
    calls = model_variants.calls(test_gpu_blocks.SIZES, test_gpu_blocks.PRODUCTS, test_gpu_layer_norm.SIZES,
                                 test_gpu_distill.SIZES)
    reached, tiles = set(), set()
    for call, (status, launches) in zip(calls, model_launches.record(recorder, calls)):
        assert status == 0 and launches, call
        names = [w[0] for w in launches]
        reached |= set(names)
        joined, padded = any("join_shares" in n for n in names), any("pad_rows" in n for n in names)
        for n in names:
            m = re.search(r"fp8_block_product.*Li(\d)ELi(\d)E", n)
            if m:
                tiles.add((m[1] + "x" + m[2], joined, padded))
    assert not built - reached, sorted(built - reached)
    # each tile with whole sums and with shares of k
    assert len({t[:2] for t in tiles}) == 2 * 5 and len(tiles) >= 4 * 5 - 1, sorted(tiles)


def test_measured_choices(recorder):
    """Sizes measured with both kernels: few rows or tiles, one launch or two, whole rows or
    segments."""
    choices = {
        "fp8_skinny_product": ["fp8 1 8 28672 8192 1", "fp8 1 12 8192 8192 1", "fp8 1 24 4096 8192 1", "fp8 1 64 4096 4096 1",
                               "fp8 1 4 8192 8193 0", "fp8 1 40 4096 2047 0"],
        "fp8_block_product": ["fp8 1 16 28672 8192 1", "fp8 1 16 8192 8192 1", "fp8 1 64 1024 8192 1", "fp8 1 48 14336 1024 1",
                              "fp8 1 8 8192 8193 0", "fp8 1 64 2000 2047 0"],
        "layer_norm_grad_few": ["norm_vjp 0 0 333 2731 3", "norm_vjp 1 0 512 8192 3", "norm_vjp 1 0 768 4096 3",
                                "norm_vjp 1 0 1024 2048 3", "norm_vjp 1 0 1536 1000 3"],
        "join_norm_sums": ["norm_vjp 1 0 2048 1000 3", "norm_vjp 0 0 1024 4096 3", "norm_vjp 0 0 768 8192 3"],
        "distill_train": ["distill 1 64 50000 64 1", "distill 1 256 128000 64 1"],
        "distill_partial": ["distill 1 16 128000 64 1", "distill 1 64 128000 64 1", "distill 1 1 131072 64 1"],
    }
    for kernel, calls in choices.items():
        for call, (status, launches) in zip(calls, model_launches.record(recorder, calls)):
            assert status == 0 and any(kernel in w[0] for w in launches), (kernel, call, launches)


def test_host_layer_under_sanitizers(tmp_path):
    """The same calls, and refused ones, with the host code under AddressSanitizer and
    UndefinedBehaviorSanitizer."""
    if not os.path.exists(model_launches.HIPCC):
        pytest.skip("hipcc not installed")
    flags = ["-g", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=undefined"]
    exe = model_launches.build(str(tmp_path), flags)
    big = [0, 1, 127, (1 << 24) - 1, 1 << 24, (1 << 24) + 1, 2 ** 31 - 1]
    calls = every_size()
    for m in big + [2 ** 62]:
        for n in big:
            calls += ["blocks 1 %d %d %d" % (m, n, r) for r in (1, 2, 128)]
            calls += ["norm %d 0 %d %d" % (t, m, n) for t in (0, 1, 7)] + ["norm_vjp 2 2 %d %d 3" % (m, n)]
            calls += ["distill 0 %d %d %d 1" % (m, n, k) for k in (0, 1024, 1025)] + ["distill_vjp 1 %d %d 3" % (m, n)]
            calls += ["fp8 1 %d %d %d 1" % (min(m, 2 ** 31 - 1), n, k) for k in (0, 1 << 22, (1 << 22) + 16)]
    assert {s for s, _ in model_launches.record(exe, calls)} == {0, 2}
