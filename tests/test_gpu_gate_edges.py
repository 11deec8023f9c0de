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


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("size", [1e3, 1e5, 1e6, 1e9])
def test_groups_whose_two_best_cancel(gsg, sigmoid, size):
    """Biases of both signs: the sum of a group's two best choices is small, its terms and their errors are not."""
    E, n_group = 64, 8
    bias = torch.tensor([size, -size] + [-2 * size] * 6).repeat(n_group)
    x = randn(200, E, 23)
    for dtype in (F32, BF):
        check(gsg, x.to(dtype), 4, sigmoid, bias, n_group, 3, 2)
    check(gsg, x, 8, sigmoid, bias * (1 + 2.0 ** -20 * randn(1, E, 24)[0]), n_group, 4, 2, renorm=False)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_group_sums_past_the_fp32_range(gsg, sigmoid):
    """Sums of two choices that fp32 does not hold are still ordered, and above a group that has nothing."""
    low, E = torch.finfo(F32).min, 24
    levels = torch.tensor([low, -2.5e38, -INF, 3.0e38, 3.2e38, 0.0])
    for seed in range(6):
        order = torch.randperm(6, generator=torch.Generator().manual_seed(seed))
        bias = levels[order].repeat_interleave(4)
        for topk_group in range(1, 6):
            check(gsg, randn(9, E, 25), 3, sigmoid, bias, 6, topk_group, 2, renorm=seed % 2 == 0)
    for bias in (torch.tensor([low, -2.5e38, -3e38]), torch.tensor([-INF, low, -2.5e38])):   # no sum in the range
        for topk_group in (1, 2):
            check(gsg, randn(9, 12, 26), 3, sigmoid, bias.repeat_interleave(4), 3, topk_group, 2, renorm=False)
