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


@pytest.mark.parametrize("fmt,N,mean", [(8, 768, 130), (4, 768, 130), (8, 768, 40)])
def test_runs_are_bit_identical(gsg, fmt, N, mean):
    """The same product some thousand times over: scales that arrive late, or that are overwritten while they are
    still read, show in one launch of many."""
    E, K = 64, 2304
    g = torch.Generator(device=DEV).manual_seed(5)
    counts = (-mean * torch.log(torch.rand(E, generator=g, device=DEV).clamp(min=1e-3))).int()
    off = torch.cat([counts.new_zeros(1), counts.cumsum(0).int()]).int()
    R = int(off[-1])
    codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    sc = torch.randint(120, 130, (E, N, K // 32), dtype=torch.uint8, device=DEV, generator=g)
    w = gsg.pack_mxfp4_codes(codes, sc)
    x = (torch.randn(R, K, generator=g, device=DEV) * torch.exp2(torch.randint(-3, 4, (R, K // 32), generator=g, device=DEV)
                                                                 .float()).repeat_interleave(32, 1)).to(torch.bfloat16)
    a = gsg.quantize_act_mx(x, fmt)
    want = gsg.grouped_mx_gemm(a, w, off)
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    y = torch.empty_like(want)
    for _ in range(6000):
        gsg.grouped_mx_gemm(a, w, off, out=y)
        differ += (y.view(torch.int16) != want.view(torch.int16)).any()
    assert int(differ) == 0


@pytest.mark.parametrize("fmt", [4, 8])
def test_other_shapes_padded_with_zeros(gsg, fmt):
    """Widths that are no multiple of 256 and 128: zero codes, zero columns of X, dropped columns of Y."""
    E, N, K, Np, Kp = 3, 200, 352, 256, 512
    codes, sc = weights(E, N, K, 8)
    off, x = layout([40, 0, 77], K, 9)
    pc, ps, px = np.zeros((E, Np, Kp), np.uint8), np.zeros((E, Np, Kp // 32), np.uint8), torch.zeros(117, Kp, dtype=x.dtype)
    pc[:, :N, :K], ps[:, :N, :K // 32], px[:, :K] = codes, sc, x
    ps[:, N:], ps[:, :, K // 32:] = 254, 200     # (any scale)
    a = gsg.quantize_act_mx(px.to(DEV), fmt)
    y = gsg.grouped_mx_gemm(a, pack(gsg, pc, ps), torch.from_numpy(off).to(DEV), out_dtype=torch.float32)[:, :N]
    A = omx.dequantize(*omx.quantize(x.double().numpy(), fmt), fmt)
    for e in (0, 2):
        yr, b = ogemm.gemm_rows(A[off[e]:off[e + 1]], omx.dequantize(codes[e], sc[e], 4), 1.0)
        tl.assert_gemm_close(y[off[e]:off[e + 1]], yr, b, f"expert {e}")
