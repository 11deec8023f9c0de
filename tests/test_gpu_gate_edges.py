"""The router on rows and biases at the ends of the fp32 range, against the oracle in 64 bits."""
import pytest
import torch

from tests.test_gpu_gate import check, clean_status, gsg, randn  # noqa: F401  (fixtures and the comparison)

pytestmark = pytest.mark.gpu
INF = float("inf")
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("E,k,n_group", [(1, 1, 1), (8, 2, 2), (31, 4, 1), (96, 8, 8), (160, 8, 8), (385, 8, 5), (520, 8, 4),
                                         (64, 4, 4)])
def test_rows_of_the_lowest_number(gsg, E, k, n_group, dtype):
    """Softmax scores are over the E logits, also where each of them is the type's lowest number."""
    low = torch.finfo(dtype).min
    x = randn(7, E, 21, dtype)
    x[0] = low
    x[1, ::2] = low
    x[2] = low
    x[2, E // 2] = 0.5
    x[3] = -INF
    x[3, 1::2] = low
    x[4] = low
    x[4, :1] = torch.finfo(dtype).max
    x[5] = low
    bias = randn(1, E, 22)[0] * 0.05
    for b in (None, bias):
        for renorm in (False, True):
            check(gsg, x, k, False, b, renorm=renorm)
            check(gsg, x, k, True, b, renorm=renorm)
            if n_group > 1:
                for top in (1, 2):
                    check(gsg, x, k, False, b, n_group, max(1, n_group // 2), top, renorm=renorm)
