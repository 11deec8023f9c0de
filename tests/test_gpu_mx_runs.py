"""The microscaled product where its wide pair tiles are irregular: against the oracle, and run after run."""
import numpy as np
import pytest
import torch

from oracle import gemm as ogemm
from oracle import mx as omx
from tests import gsg_testlib as tl
from tests.test_gpu_mx import clean_status, gsg, pack, weights  # noqa: F401  (fixtures, inputs)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def layout(counts, K, seed):
    """Offsets of experts with these rows, and normal rows."""
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x = torch.randn(int(off[-1]), K, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
    return off, x


@pytest.mark.parametrize("fmt", [4, 8])
@pytest.mark.parametrize("N", [512, 640])
def test_experts_of_a_few_rows_between_long_ones(gsg, N, fmt):
    """Tiles of at most eight rows, all of them in the pair's first CTA: several in a row, first, last and alone."""
    K = 1280
    for counts in ([3, 900, 1, 8, 2, 7, 5, 830, 4, 1, 1000, 6], [900, 850, 1], [1, 2, 3, 4, 5, 6, 7, 8, 1500, 1500]):
        E = len(counts)
        codes, sc = weights(E, N, K, 3)
        off, x = layout(counts, K, 4)
        a = gsg.quantize_act_mx(x.to(DEV), fmt)
        y = gsg.grouped_mx_gemm(a, pack(gsg, codes, sc), torch.from_numpy(off).to(DEV), out_dtype=torch.float32)
        A = omx.dequantize(*omx.quantize(x.double().numpy(), fmt), fmt)
        for e in range(E):
            rows = np.arange(off[e], off[e + 1])
            rows = rows if len(rows) < 20 else rows[:: len(rows) // 7]
            yr, b = ogemm.gemm_rows(A[rows], omx.dequantize(codes[e], sc[e], 4), 1.0)
            tl.assert_gemm_close(y[torch.from_numpy(rows).to(DEV)], yr, b, f"expert {e}")
