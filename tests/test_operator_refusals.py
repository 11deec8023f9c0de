"""Calls of the router, the residual norm and the microscaled experts that are refused on the host (no GPU needed)."""
import ctypes

import pytest
import torch

import grouped_sparse_gemm_b200 as gsg

BF = torch.bfloat16


def test_norm_refuses_outputs_that_it_would_not_write():
    """A buffer for h without a residual, one for codes without a format."""
    x, w = torch.zeros(4, 256, dtype=BF), torch.zeros(256)
    act = gsg.MxActivations(torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(128, dtype=torch.uint8), 4, 256, 8)
    with pytest.raises(ValueError, match="out_h"):
        gsg.add_rmsnorm_mx(x, w, out_h=torch.zeros(4, 256, dtype=BF))
    with pytest.raises(ValueError, match="out_act"):
        gsg.add_rmsnorm_mx(x, w, fmt=None, out_act=act)
