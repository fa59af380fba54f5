"""Layer norm's gradients at sizes where 16 bits take one launch and float32 two: the first needs no
workspace, the second is refused without one, and both hold to 64 bits."""
import pytest

import test_gpu_layer_norm as ln
from helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("R,C", [(600, 5200), (640, 4900), (900, 3400), (1024, 2560), (1280, 1600), (1536, 2048), (1400, 2200),
                                 (768, 4096), (1024, 2048), (1536, 1024)])
def test_layer_norm(R, C, dtype):
    from trellis_coded_weight_amd import api
    x, w, b = ln.inputs(R, C, dtype, "float32")
    say("layer_norm choices %dx%d %s" % (R, C, dtype))
    mean, rstd = ln.check_forward(api, x, w, b)
    ln.check_vjp(api, x, w, mean, rstd, ln.normal(R, C, seed=5, dtype=dtype))


def test_workspace_where_one_launch_needs_none():
    import torch
    from trellis_coded_weight_amd import _native as nat
    from trellis_coded_weight_amd import api
    R, C = 1280, 1600
    say("layer_norm_vjp without a workspace %dx%d" % (R, C))
    for dtype in (torch.bfloat16, torch.float32):
        x, w = torch.randn(R, C, device="cuda").to(dtype), torch.randn(C, device="cuda")
        _, mean, rstd = api.layer_norm(x, w, save=True)
        gw, gb = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")

        def call():
            nat.qtcq_layer_norm_vjp(x.data_ptr(), api.DTYPES[dtype], R, C, C, w.data_ptr(), nat.QTCQ_F32, mean.data_ptr(),
                                    rstd.data_ptr(), x.data_ptr(), C, None, C, gw.data_ptr(), gb.data_ptr(), None, 0,
                                    torch.cuda.current_stream().cuda_stream)
        if dtype == torch.float32:
            with pytest.raises(nat.QtcqError):
                call()
        else:
            call()
            want = api.layer_norm_vjp(x, w, mean, rstd, x)
            torch.cuda.synchronize()
            assert torch.equal(gw, want[1]) and torch.equal(gb, want[2])
