"""The e4m3 product on both sides of the rule for few rows by many columns, against 64 bits."""
import pytest

import test_gpu_blocks
from helpers import say
from test_fp8_choices import FEW, TILES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("M,N,K", sorted({s for d in (FEW, TILES) for t in d.values() for s in t if s[1] > 20000 and s[2] <= 1536}))
def test_matmul_fp8(M, N, K, dtype):
    from trellis_coded_weight_amd import api
    say("matmul_fp8 choices %dx%dx%d %s" % (M, N, K, dtype))
    test_gpu_blocks.check_product(api, *test_gpu_blocks.operands(M, N, K), dtype)
