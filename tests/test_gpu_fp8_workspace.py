"""The e4m3 product with the workspace that its documentation prescribes, whatever the operands'
layout: sizes at which rows of whole chunks take shares of k and others none."""
import pytest

import test_gpu_blocks
from helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [0, 6, 16])
@pytest.mark.parametrize("M,N,K", [(40, 512, 8192), (33, 1024, 8192), (48, 16, 14336), (33, 8208, 1536), (70, 264, 4112)])
def test_workspace_as_documented(M, N, K, wide):
    import torch
    from trellis_coded_weight_amd import api
    o = test_gpu_blocks.operands(M, N, K, wide)
    say("matmul_fp8 workspace %dx%dx%d +%d" % (M, N, K, wide))
    for dtype in (torch.float32, torch.bfloat16):
        y = api.matmul_fp8(*o, dtype=dtype, workspace=api.matmul_fp8_workspace(M, N, K))
        assert torch.equal(y, api.matmul_fp8(*o, dtype=dtype))
    torch.cuda.synchronize()
