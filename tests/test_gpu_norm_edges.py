"""The residual norm at the ends of the fp32 range: single rounding of y and codes, and what is reported."""
import numpy as np
import pytest
import torch

from oracle import mx as omx
from tests.test_gpu_norm import check, clean_status, definition, gsg, rows  # noqa: F401  (fixtures, comparison)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


def check_nearest(gsg, x, w, eps, fmts=(4, 8)):
    """y the nearest bf16 number to the 64-bit value (of normal size; ties do not occur here), codes exact."""
    y = definition(x, w, None, eps)[1]
    for fmt in fmts:
        n = gsg.add_rmsnorm_mx(x.to(DEV), w.to(DEV), eps=eps, fmt=fmt)
        got = n.y.cpu()
        best = (got.double() - y).abs()
        for s in (1, -1):
            other = torch.nextafter(got, torch.tensor(s * INF, dtype=BF)).double()
            assert (best <= (other - y).abs()).all()
        codes, sc = omx.quantize(y.numpy(), fmt)
        np.testing.assert_array_equal(n.act.codes.cpu().numpy(), omx.pack_nibbles(codes) if fmt == 4 else codes)
        np.testing.assert_array_equal(n.act.scales.cpu().numpy(), omx.quad_scales(sc).reshape(-1))



@pytest.mark.parametrize("dtype", [F32, BF])
def test_weights_past_the_middle_of_the_range(gsg, dtype):
    """h * w may leave the fp32 range where y does not."""
    K = 512
    g = torch.Generator().manual_seed(31)
    unit = (0.5 + torch.rand(K, generator=g)).to(dtype)
    x = rows(5, K, 32, outliers=False)
    x[2, 8:] = 0.0
    for up, wp in ((40, 88), (59, 70), (50, 100), (-40, -100), (-55, -60), (0, 119), (0, -95), (0, 60)):
        check_nearest(gsg, (x.double() * 2.0 ** up).to(BF), (unit.double() * 2.0 ** wp).to(dtype), 0.0)
