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


def test_sizes_past_31_bits_are_refused():
    """The library takes 32-bit sizes: a longer batch or a larger option is refused, not cut to its low bits."""
    meta = dict(device="meta")
    with pytest.raises(ValueError, match="31 bits"):
        gsg.moe_gate(torch.empty((1 << 32) + 3, 1, dtype=BF, **meta), 1)
    for kw in (dict(top_k=(1 << 32) + 2), dict(top_k=2, n_group=(1 << 32) + 1), dict(top_k=2, topk_group=(1 << 32) + 1),
               dict(top_k=2, group_top=(1 << 32) + 1)):
        with pytest.raises(ValueError, match="31 bits"):
            gsg.moe_gate(torch.empty(4, 8, **meta), **kw)
    with pytest.raises(ValueError, match="31 bits"):
        gsg.add_rmsnorm_mx(torch.empty((1 << 32) + 3, 8, dtype=BF, **meta), torch.empty(8, **meta), fmt=None)
    with pytest.raises(ValueError, match="31 bits"):
        gsg.quantize_act_mx(torch.empty(2, 256, dtype=BF, **meta), 8, top_k=(1 << 32) + 1)
