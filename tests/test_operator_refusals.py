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


INVALID = -1
P, ODD4, ODD2 = ctypes.c_void_p(256), ctypes.c_void_p(258), ctypes.c_void_p(257)   # aligned, not to 4, not to 2


@pytest.fixture(scope="module")
def L():
    from grouped_sparse_gemm_b200 import _build
    _build.build()
    return gsg.load_library()


@pytest.mark.parametrize("name,dtype,bad", [("logits", 1, ODD4), ("logits", 0, ODD2), ("bias", 1, ODD4), ("ids", 1, ODD4),
                                            ("gates", 1, ODD4)])
def test_gate_refuses_misaligned_pointers(L, name, dtype, bad):
    """A kernel's access to one would fault; the types of the C interface do not rule it out (void *)."""
    p = dict(logits=P, bias=P, ids=P, gates=P)
    p[name] = bad
    assert L.gsg_moe_gate(p["logits"], dtype, p["bias"], 4, 8, 2, 0, 1, 1, 1, 1, 1.0, p["ids"], p["gates"], None) == INVALID


def test_quantizer_and_product_refuse_misaligned_indices(L):
    assert L.gsg_quantize_act_mx(P, 4, 256, 8, ODD4, 2, P, P, None, 0, None) == INVALID
    assert L.gsg_grouped_mx_gemm(P, P, 8, P, ODD4, 4, 128, 256, 8, -1, P, 0, None) == INVALID
