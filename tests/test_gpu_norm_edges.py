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


@pytest.mark.parametrize("power", [0, -30, -51, -62, -70, -90, -100])
def test_values_next_to_a_border(gsg, power):
    """A row of ones with eps 2^-30 has y = w (1 - 2^-31): weights on the borders between bf16 numbers and between
    codes give values just inside them, which fp32 rounds onto the border."""
    K = 512
    borders = torch.cat([1 + (2 * torch.arange(128) + 1) * 2.0 ** -8,      # midpoints of bf16 numbers
                         1 + (2 * torch.arange(8) + 1) * 2.0 ** -4,        # of E4M3 numbers
                         torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])]).float()
    w = borders.repeat(4)[:K] * torch.where(torch.arange(K) % 3 == 0, -1.0, 1.0)
    x = torch.ones(3, K, dtype=BF)
    x[1] = -1.0
    check_nearest(gsg, x, w * 2.0 ** power, 2.0 ** -30)


def test_every_output_reports_what_is_not_finite(gsg):
    """Rows without a norm, weights and products that are not finite, with and without codes, with y or h alone."""
    K = 256
    x = rows(4, K, 1).to(DEV)
    w = torch.ones(K, device=DEV)

    def status(x, w, eps=1e-6, **kw):
        gsg.add_rmsnorm_mx(x, w, eps=eps, **kw)
        return gsg.get_device_status()
    outputs = (dict(fmt=None), dict(fmt=8), dict(fmt=4, want_y=False))
    for kw in outputs:
        assert status(x, w, **kw) == 0
        assert status(torch.zeros_like(x), w, eps=0.0, **kw) == -5          # a row of zeros has no norm
        assert status(torch.zeros_like(x), w, **kw) == 0
        for v in (float("nan"), INF):
            y, u = x.clone(), w.clone()
            y[2, 3] = v
            u[7] = v
            assert status(y, w, **kw) == -5
            assert status(x, u, **kw) == -5
        big = torch.zeros(1, K, dtype=BF, device=DEV)
        big[0, 0] = 1.0                                                     # h / rms = 16
        assert status(big, w * 2.0 ** 123, **kw) == 0
        assert status(big, w * 2.0 ** 126, **kw) == -5                      # y past the fp32 range
    r = x.float().clone()
    r[1, 1] = INF
    assert status(x, w, residual=r, fmt=None, want_y=False) == -5           # the residual stream alone
    bad = w.clone()
    bad[0] = INF                                                            # (the weight has no part in it)
    assert status(x, bad, residual=x.float(), fmt=None, want_y=False) == 0
