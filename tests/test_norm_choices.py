"""Layer norm's gradients in one launch or two: sizes measured with both, in 16 bits and in
float32, on the host without a GPU (the launch recorder); and the workspace that any type of them
gets along with."""
import os

import pytest

import model_launches
from trellis_coded_weight_amd import _native as nat

ONE = {1: [(512, 8192), (768, 4096), (1024, 3000), (1280, 2048), (1536, 1000), (1536, 2048)],
       0: [(333, 2731), (400, 8192), (768, 4096), (1024, 2048), (1536, 1024)]}
TWO = {1: [(1400, 2200), (2048, 1000), (1000, 8192), (1024, 4096)],
       0: [(640, 4900), (900, 3400), (1024, 2560), (1280, 1600), (1400, 1500), (1536, 1300), (1536, 2048)]}


def test_measured_choices(tmp_path):
    if not os.path.exists(model_launches.HIPCC):
        pytest.skip("hipcc not installed")
    recorder = model_launches.build(str(tmp_path))
    for kernel, sizes in (("layer_norm_grad_few", ONE), ("join_norm_sums", TWO)):
        calls = ["norm_vjp %d 0 %d %d 3" % (t, *s) for t in sizes for s in sizes[t]]
        for call, (status, launches) in zip(calls, model_launches.record(recorder, calls)):
            assert status == 0 and any(kernel in w[0] for w in launches), (kernel, call, launches)


def test_queried_workspace_holds_both_types():
    """One launch needs none, so the query is at least what the type with two launches needs: for
    up to 256 workgroups two sums a column."""
    for sizes in (TWO[0], TWO[1]):
        for R, C in sizes:
            assert nat.qtcq_layer_norm_vjp_workspace_bytes(R, C) >= min(R, 256) * 2 * C * 4, (R, C)
