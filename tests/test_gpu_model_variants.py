"""Every variant of the model operators' kernels (model_variants.py) against 64 bits."""
import pytest

import test_gpu_blocks
import test_gpu_distill
import test_gpu_layer_norm
from helpers import say
from model_variants import DISTILL, FP8, NORM

pytestmark = pytest.mark.gpu

TYPES = ["float32", "bfloat16", "float16"]


@pytest.fixture(scope="module")
def api():
    import torch
    assert torch.cuda.is_available(), "GPU test without a GPU"
    from trellis_coded_weight_amd import api as a
    yield a
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", FP8)
def test_matmul_fp8(api, M, N, K, dtype):
    say("matmul_fp8 variants %dx%dx%d %s" % (M, N, K, dtype))
    test_gpu_blocks.check_product(api, *test_gpu_blocks.operands(M, N, K), dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,C", NORM)
def test_layer_norm(api, R, C, dtype):
    for wtype in {dtype, "float32"}:
        x, w, b = test_gpu_layer_norm.inputs(R, C, dtype, wtype)
        say("layer_norm variants %dx%d %s %s" % (R, C, dtype, wtype))
        mean, rstd = test_gpu_layer_norm.check_forward(api, x, w, b)
        test_gpu_layer_norm.check_vjp(api, x, w, mean, rstd, test_gpu_layer_norm.normal(R, C, seed=5, dtype=dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,V,k", DISTILL)
def test_distill(api, R, V, k, dtype):
    say("distill variants %dx%d k=%d %s" % (R, V, k, dtype))
    z, index, t, gl = test_gpu_distill.inputs(R, V, k, dtype)
    test_gpu_distill.check(api, z, index, t, gl, 1.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("wide", [1, 6, 16])
def test_distill_segments_strided(api, wide, dtype):
    say("distill segments strided +%d %s" % (wide, dtype))
    z, index, t, gl = test_gpu_distill.inputs(4, 70003, 20, dtype, wide=wide)
    test_gpu_distill.check(api, z, index, t, gl, 0.5)
