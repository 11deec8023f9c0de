"""Host side of the router, the residual norm and the microscaled experts: sizes, and refusals that return
before any CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch

import grouped_sparse_gemm_b200 as gsg

P = ctypes.c_void_p(128)   # a non-NULL, aligned placeholder that none of these checks dereferences
ODD = ctypes.c_void_p(136)
OK, INVALID, SHAPE, WORKSPACE = 0, -1, -2, -7


@pytest.fixture(scope="module")
def L():
    from grouped_sparse_gemm_b200 import _build
    _build.build()
    return gsg.load_library()


def test_sizes(L):
    assert L.gsg_mx_packed_bytes(3, 256, 512) * 8 == 4.25 * 3 * 256 * 512
    assert L.gsg_mx_act_codes_bytes(10, 256, gsg.MXFP4) == 1280
    assert L.gsg_mx_act_codes_bytes(10, 256, gsg.MXFP8) == 2560
    assert L.gsg_mx_act_scales_bytes(10, 256) == 2 * 10 * 16
    assert L.gsg_workspace_size(gsg.OP_QUANTIZE_MX, 0, 0, 2048, 512, 8) == 0
    assert L.gsg_workspace_size(gsg.OP_QUANTIZE_MX, 0, 0, 8192, 2048, 8) == 16384 * 64 * 4   # R*K = 2^27


@pytest.mark.parametrize("want,args", [
    # logits, dtype, bias, T, E, k, scoring, n_group, topk_group, group_top, renorm, scale, ids, gates
    (OK, (P, 1, None, 0, 8, 2, 0, 1, 1, 1, 1, 1.0, None, None)),        # no tokens
    (INVALID, (P, 1, None, -1, 8, 2, 0, 1, 1, 1, 1, 1.0, P, P)),
    (INVALID, (P, 2, None, 4, 8, 2, 0, 1, 1, 1, 1, 1.0, P, P)),         # type
    (INVALID, (P, 1, None, 4, 8, 2, 2, 1, 1, 1, 1, 1.0, P, P)),         # scoring
    (INVALID, (P, 1, None, 4, 8, 0, 0, 1, 1, 1, 1, 1.0, P, P)),         # k
    (INVALID, (P, 1, None, 4, 8, 9, 0, 1, 1, 1, 1, 1.0, P, P)),         # k above E
    (SHAPE, (P, 1, None, 4, 64, 33, 0, 1, 1, 1, 1, 1.0, P, P)),
    (SHAPE, (P, 1, None, 4, 1025, 2, 0, 1, 1, 1, 1, 1.0, P, P)),
    (INVALID, (P, 1, None, 4, 0, 1, 0, 1, 1, 1, 1, 1.0, P, P)),
    (INVALID, (P, 1, None, 4, 10, 2, 0, 4, 1, 1, 1, 1.0, P, P)),        # E not in whole groups
    (INVALID, (P, 1, None, 4, 8, 2, 0, 4, 5, 1, 1, 1.0, P, P)),         # more groups kept than there are
    (INVALID, (P, 1, None, 4, 8, 2, 0, 4, 0, 1, 1, 1.0, P, P)),
    (INVALID, (P, 1, None, 4, 8, 5, 0, 4, 2, 1, 1, 1.0, P, P)),         # k above the kept groups' experts
    (INVALID, (P, 1, None, 4, 8, 2, 0, 8, 4, 2, 1, 1.0, P, P)),         # two of a one-expert group
    (INVALID, (P, 1, None, 4, 8, 2, 0, 4, 2, 3, 1, 1.0, P, P)),
    (SHAPE, (P, 1, None, 4, 66, 2, 0, 33, 2, 2, 1, 1.0, P, P)),         # 33 groups
    (INVALID, (None, 1, None, 4, 8, 2, 0, 1, 1, 1, 1, 1.0, P, P)),
    (INVALID, (P, 1, None, 4, 8, 2, 0, 1, 1, 1, 1, 1.0, P, None)),
])
def test_gate_checks(L, want, args):
    assert L.gsg_moe_gate(*args, None) == want


@pytest.mark.parametrize("want,args", [
    # x, residual, r_dtype, weight, w_dtype, T, K, eps, h, y, fmt, codes, scales
    (OK, (P, None, 0, P, 0, 0, 256, 1e-6, None, P, 8, P, P)),
    (INVALID, (P, None, 0, P, 0, -1, 256, 1e-6, None, P, 8, P, P)),
    (SHAPE, (P, None, 0, P, 0, 4, 12, 1e-6, None, P, 0, None, None)),
    (SHAPE, (P, None, 0, P, 0, 4, 264, 1e-6, None, P, 8, P, P)),        # codes need whole 256
    (SHAPE, (P, None, 0, P, 0, 4, 33024, 1e-6, None, P, 8, P, P)),
    (INVALID, (P, None, 0, P, 0, 4, 256, -1.0, None, P, 8, P, P)),
    (INVALID, (P, None, 0, P, 0, 4, 256, float("nan"), None, P, 8, P, P)),
    (INVALID, (P, None, 0, P, 0, 4, 256, 1e-6, None, P, 6, P, P)),
    (INVALID, (P, P, 0, P, 0, 4, 256, 1e-6, None, P, 8, P, P)),         # a residual without h
    (INVALID, (P, None, 0, P, 0, 4, 256, 1e-6, None, None, 0, None, None)),   # nothing asked for
    (INVALID, (P, None, 0, P, 0, 4, 256, 1e-6, None, P, 8, None, P)),
    (INVALID, (P, None, 3, P, 0, 4, 256, 1e-6, None, P, 8, P, P)),
    (INVALID, (ODD, None, 0, P, 0, 4, 256, 1e-6, None, P, 8, P, P)),    # alignment
    (INVALID, (P, None, 0, None, 0, 4, 256, 1e-6, None, P, 8, P, P)),
])
def test_norm_checks(L, want, args):
    assert L.gsg_add_rmsnorm_mx(*args, None) == want


@pytest.mark.parametrize("want,args", [
    # X, T, K, fmt, inv_perm, k, codes, scales, workspace, bytes
    (OK, (None, 0, 256, 8, None, 1, None, None, None, 0)),
    (INVALID, (P, 4, 256, 5, None, 1, P, P, None, 0)),
    (INVALID, (P, 4, 256, 8, None, 2, P, P, None, 0)),                  # top-k without a routing
    (INVALID, (P, 4, 256, 8, P, 0, P, P, None, 0)),
    (SHAPE, (P, 4, 128, 8, P, 2, P, P, None, 0)),
    (SHAPE, (P, 1 << 28, 256, 8, P, 8, P, P, None, 0)),
    (INVALID, (P, 4, 256, 8, P, 2, None, P, None, 0)),
    (INVALID, (P, 4, 256, 8, P, 2, ODD, P, None, 0)),
    (WORKSPACE, (P, 2048, 8192, 8, P, 8, P, P, None, 0)),
    (WORKSPACE, (P, 2048, 8192, 8, P, 8, P, P, P, 100)),
])
def test_quantize_checks(L, want, args):
    assert L.gsg_quantize_act_mx(*args, None) == want


@pytest.mark.parametrize("want,args", [
    # codes, scales, fmt, packed, offsets, E, N, K, R, hint, Y, dtype
    (OK, (None, None, 8, P, P, 4, 128, 256, 0, -1, None, 0)),
    (INVALID, (P, P, 5, P, P, 4, 128, 256, 8, -1, P, 0)),
    (INVALID, (P, P, 8, P, P, 4, 128, 256, -1, -1, P, 0)),
    (INVALID, (P, P, 8, P, P, 4, 128, 256, 8, -1, P, 2)),
    (SHAPE, (P, P, 8, P, P, 4, 100, 256, 8, -1, P, 0)),
    (SHAPE, (P, P, 8, P, P, 4, 128, 128, 8, -1, P, 0)),
    (SHAPE, (P, P, 8, P, P, 2000, 128, 256, 8, -1, P, 0)),
    (SHAPE, (P, P, 8, P, P, 1024, 65536, 16384, 8, -1, P, 0)),          # packed rows past 32 bits
    (INVALID, (P, P, 8, None, P, 4, 128, 256, 8, -1, P, 0)),
    (INVALID, (P, P, 8, P, None, 4, 128, 256, 8, -1, P, 0)),
    (INVALID, (P, P, 8, P, P, 4, 128, 256, 8, -1, None, 0)),
    (INVALID, (P, P, 8, ODD, P, 4, 128, 256, 8, -1, P, 0)),
])
def test_gemm_checks(L, want, args):
    assert L.gsg_grouped_mx_gemm(*args, None) == want


def test_pack_checks(L):
    assert L.gsg_pack_mxfp4(None, 1, 1, 128, 256, P, None) == INVALID
    assert L.gsg_pack_mxfp4(P, 4, 1, 128, 256, P, None) == INVALID
    assert L.gsg_pack_mxfp4(P, 1, 1, 130, 256, P, None) == SHAPE
    assert L.gsg_pack_mxfp4(P, 1, 1, 128, 256, ODD, None) == INVALID
    assert L.gsg_pack_mxfp4_codes(P, None, 1, 128, 256, P, None) == INVALID
    assert L.gsg_pack_mxfp4_codes(P, P, 1, 128, 200, P, None) == SHAPE
    assert L.gsg_pack_mxfp4_codes(ODD, P, 1, 128, 256, P, None) == INVALID


def test_group_of_an_expert_by_multiplication():
    """The router divides an expert's index by the group size with one multiplication and a shift."""
    for size in range(1, 1025):
        magic = ((1 << 20) + size - 1) // size
        assert all((e * magic) >> 20 == e // size for e in range(0, 1024))


def test_binding_refuses_wrong_shapes_and_types():
    bf = torch.bfloat16
    with pytest.raises(ValueError):
        gsg.moe_gate(torch.zeros(4, 8, dtype=torch.float16), 2)
    with pytest.raises(ValueError):
        gsg.moe_gate(torch.zeros(4, 8), 2, scoring="tanh")
    with pytest.raises(ValueError):
        gsg.moe_gate(torch.zeros(4, 8), 2, bias=torch.zeros(7))
    with pytest.raises(ValueError):
        gsg.add_rmsnorm_mx(torch.zeros(4, 256), torch.zeros(256))
    with pytest.raises(ValueError):
        gsg.add_rmsnorm_mx(torch.zeros(4, 256, dtype=bf), torch.zeros(128))
    with pytest.raises(ValueError):
        gsg.pack_mxfp4(torch.zeros(128, 256))
    with pytest.raises(ValueError):
        gsg.pack_mxfp4_codes(torch.zeros(1, 128, 128, dtype=torch.uint8), torch.zeros(1, 128, 4, dtype=torch.uint8))
    with pytest.raises(ValueError):
        gsg.quantize_act_mx(torch.zeros(4, 256))
    act = gsg.MxActivations(torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(128, dtype=torch.uint8), 4, 256, 8)
    w = gsg.PackedMxWeights(torch.zeros(2 * 17408, dtype=torch.uint8), 2, 128, 256)
    with pytest.raises(ValueError):
        gsg.grouped_mx_gemm(act, gsg.PackedMxWeights(w.packed, 1, 128, 512), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        gsg.grouped_mx_gemm(act, w, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        gsg.grouped_mx_gemm(act, w, torch.zeros(3, dtype=torch.int32), out_dtype=torch.float16)
    e = gsg.PackedMxWeights(torch.arange(2 * 17408) % 251, 2, 128, 256).expert(1)
    assert e.E == 1 and e.packed.numel() == 17408 and e.packed[0] == 17408 % 251


@pytest.mark.skipif(torch.cuda.is_available(), reason="for machines without a device")
def test_binding_refuses_cpu_tensors():
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        gsg.quantize_act_mx(torch.zeros(4, 256, dtype=torch.bfloat16))


def test_packed_mx_storage(tmp_path):
    w = gsg.PackedMxWeights((torch.arange(2 * 3 * 17408) % 253).to(torch.uint8), 2, 128, 768)
    p = str(tmp_path / "w.npz")
    gsg.save_packed(w, p)
    r = gsg.load_packed(p)
    assert isinstance(r, gsg.PackedMxWeights) and (r.E, r.N, r.K) == (2, 128, 768) and torch.equal(r.packed, w.packed)
    gsg.save_packed(gsg.PackedMxWeights(w.packed[:-1], 2, 128, 768), p)
    with pytest.raises(ValueError):
        gsg.load_packed(p)


def test_product_refuses_buffers_of_another_size():
    off = torch.zeros(2, dtype=torch.int32)
    codes, scales = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(128, dtype=torch.uint8)
    w = gsg.PackedMxWeights(torch.zeros(17408, dtype=torch.uint8), 1, 128, 256)
    for act, ww in ((gsg.MxActivations(codes, scales, 5, 256, 8), w), (gsg.MxActivations(codes, scales, 4, 256, 4), w),
                    (gsg.MxActivations(codes, scales[:64], 4, 256, 8), w),
                    (gsg.MxActivations(codes, scales, 4, 256, 8), gsg.PackedMxWeights(w.packed[:100], 1, 128, 256))):
        with pytest.raises(ValueError):
            gsg.grouped_mx_gemm(act, ww, off)
