"""The row quantization at its largest row count with a workgroup a row, which takes more than
one launch."""
import pytest

import dense_ref as ref
from helpers import say
from test_gpu_dense_products import gen

pytestmark = pytest.mark.gpu


def test_quantize_most_rows():
    import torch
    from trellis_coded_weight_amd import api
    R, C = 1 << 24, 2049
    if torch.cuda.mem_get_info()[0] < R * C * 3 + (8 << 30):
        pytest.skip("needs 111 GB of device memory")
    x = torch.empty((R, C), dtype=torch.bfloat16, device="cuda")
    g = gen(1)
    for lo in range(0, R, 1 << 20):
        x[lo:lo + (1 << 20)].normal_(generator=g)
    say("quantize %dx%d" % (R, C))
    q, s = api.quantize_rows(x)
    torch.cuda.synchronize()
    for lo in (0, (1 << 23) - 4, (1 << 23), R - 8):
        qr, sr = ref.quantize(x[lo:lo + 8].double())
        assert torch.equal(q[lo:lo + 8], qr) and torch.equal(s[lo:lo + 8], sr), lo
    del x, q
    torch.cuda.empty_cache()
