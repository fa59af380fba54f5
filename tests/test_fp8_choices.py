"""The e4m3 product of 9 to 32 rows by many columns of short k: sizes measured in the kernel for few
rows and in tiles, on the host without a GPU (the launch recorder)."""
import os

import pytest

import model_launches

FEW = {1: [(8, 28672, 2048), (9, 8192, 2560), (32, 12288, 2048), (32, 16384, 1536), (16, 20480, 2048), (9, 14336, 1024)],
       0: [(9, 28672, 2048), (16, 24576, 2048), (16, 28672, 1536), (32, 16384, 1536)]}
TILES = {1: [(9, 24576, 2048), (32, 24576, 1024), (9, 28672, 2048), (16, 28672, 1536), (32, 26392, 512)],
         0: [(24, 24576, 1024), (32, 24576, 1024), (32, 28672, 512)]}


def test_measured_choices(tmp_path):
    if not os.path.exists(model_launches.HIPCC):
        pytest.skip("hipcc not installed")
    recorder = model_launches.build(str(tmp_path))
    for kernel, sizes in (("fp8_skinny_product", FEW), ("fp8_block_product", TILES)):
        calls = ["fp8 %d %d %d %d 1" % (t, *s) for t in sizes for s in sizes[t]]
        for call, (status, launches) in zip(calls, model_launches.record(recorder, calls)):
            assert status == 0 and any(kernel in w[0] for w in launches), (kernel, call, launches)
