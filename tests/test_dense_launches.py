"""Grids of the dense operators' launches, from the smallest sizes to the largest accepted:
every launch has blocks and stays below 2^32 threads, the most a launch holds, and rows that
need more go in several.  No GPU needed."""
import os
import re

import pytest

import dense_launches
import dense_variants

F32, BF16, F16, I8 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    if not os.path.exists(dense_launches.HIPCC):
        pytest.skip("hipcc not installed")
    return dense_launches.build(str(tmp_path_factory.mktemp("launches")))


@pytest.mark.parametrize("dtype,size", [(F32, 4), (BF16, 2), (F16, 2)])
def test_quantize_rows_in_launches(recorder, dtype, size):
    """Each launch takes the rows after those of the one before, all of them together."""
    calls = ["quantize %d %d %d" % (dtype, rows, cols) for rows in (1, 5, 4096, (1 << 23) + 1, (1 << 24) - 1, 1 << 24)
             for cols in (0, 1, 64, 1025, 2049, 8192, 8193, 70000)]
    for call, (status, launches) in zip(calls, dense_launches.record(recorder, calls)):
        rows, cols = map(int, call.split()[2:])
        assert status == 0 and launches, call
        done = 0
        for _, grid, block, n, x, q, scale in launches:
            grid, block, n = int(grid), int(block), int(n)
            assert 0 < grid and grid * block < 1 << 32, (call, grid, block)
            assert int(x) == (1 << 40) + done * cols * size and int(q) == (2 << 40) + done * cols, call
            assert int(scale) == (3 << 40) + 4 * done, call
            done += n
        assert done == rows, call


def test_every_grid_fits_a_launch(recorder):
    dims = [1, 2, 16, 63, 65, 129, 1000, 4096, 28672, 131071, (1 << 20) + 3, 1 << 21, 1 << 24]
    calls = ["decode %d %d %d %d" % (t, m // 16 * 16, n // 16 * 16, t & 1) for t in (F32, BF16, F16, I8)
             for m in dims for n in dims if m >= 16 and n >= 16]
    for al in (0, 1):
        for m in dims:
            for n in dims:
                for k in dims:
                    calls.append("int8 %d %d %d %d %d" % (BF16, m, n, k, al))
                    calls.append("gated %d %d %d %d %d %d" % (F16, m, n, k, al, 0))
                    calls.append("vjp %d %d %d %d %d %d" % (BF16, m, n, k, al, 0))
    accepted = 0
    for call, (status, launches) in zip(calls, dense_launches.record(recorder, calls)):
        if status != 0:
            assert not launches, call
            continue
        accepted += 1
        assert launches, call
        for words in launches:
            grid, block = int(words[1]), int(words[2])
            assert 0 < grid and grid * block < 1 << 32, (call, words)
    assert accepted > len(calls) // 4


def test_sizes_that_reach_every_product_kernel(recorder):
    """The lists of dense_variants.py launch every kernel that the products are built as."""
    families = ("skinny_product", "block_product", "join_shares", "pad_rows", "gated_slopes", "gradient_products")
    built = {w[0] for w in dense_launches.record(recorder, ["kernels"])[0][1] if any(f in w[0] for f in families)}
    assert len(built) > 150
    reached, shares = set(), set()
    for call, (status, launches) in zip(dense_variants.calls(), dense_launches.record(recorder, dense_variants.calls())):
        assert status == 0 and launches, call
        names = [w[0] for w in launches]
        reached |= set(names)
        joined = any("join_shares" in n for n in names)
        for n in names:
            # the operator and the tile height, 32 times the last template argument
            m = re.search(r"block_product.*Li([012])ELi\dELi([248])E|gradient_products.*Li([248])E", n)
            if m:
                shares.add((m[1] or "2", m[2] or m[3], joined))
    assert not built - reached, sorted(built - reached)
    # each height of each operator's tiles on whole sums and on shares
    assert len(shares) == 3 * 3 * 2, sorted(shares)


def test_few_rows_go_where_they_are_faster(recorder):
    """Sizes measured with both kernels: the kernel for few rows or the block kernel."""
    few = ["int8 1 1 8192 28672 1", "gated 1 8 14336 4096 1 0", "gated 1 32 4096 4096 1 0", "int8 1 1 28672 8193 0",
           "gated 1 16 4096 4097 0 0"]
    block = ["int8 1 16 8192 28672 1", "int8 1 16 28672 8192 1", "gated 1 24 14336 4096 1 0",
             "gated 1 64 4096 4096 1 0", "int8 1 8 28672 8193 0", "gated 1 32 4096 4097 0 0"]
    for calls, kernel in ((few, "skinny_product"), (block, "block_product")):
        for call, (status, launches) in zip(calls, dense_launches.record(recorder, calls)):
            assert status == 0 and any(kernel in w[0] for w in launches), call
