"""The oracle of the microscaled formats and of the router, pinned to definitions and brute force (CPU)."""
import numpy as np
import pytest
import torch

from oracle import gate as ogate
from oracle import mx as omx


def test_e4m3_table_is_torchs():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(omx.E4M3_MAGNITUDES, t)
    assert torch.tensor([127], dtype=torch.uint8).view(torch.float8_e4m3fn).isnan().all()


@pytest.mark.parametrize("bits", [4, 8])
def test_encode_is_nearest_ties_even_saturating(bits):
    g = omx.grid(bits)
    mid = (g[1:] + g[:-1]) / 2
    v = np.concatenate([g, mid, mid * (1 + 2.0 ** -30), mid * (1 - 2.0 ** -30), [g[-1] * 3]])
    c = omx.encode(v, bits)
    for x, code in zip(v, c):
        d = np.abs(g - min(x, g[-1]))
        best = np.flatnonzero(d == d.min())
        assert code == (best[0] if len(best) == 1 else [b for b in best if b % 2 == 0][0])
    np.testing.assert_array_equal(omx.encode(-v, bits), c | (1 << (bits - 1)))
    np.testing.assert_array_equal(omx.decode(c, bits), np.minimum(g, g[-1])[c])


@pytest.mark.parametrize("bits", [4, 8])
def test_quantize_scale_rule(bits):
    v = np.zeros((6, 32))
    v[1, 3] = -1.0
    v[2, 0], v[2, 1] = 6.0, 1e-3
    v[3, 5] = 2.0 ** -140          # clamps at 2^-127: too small for the format, codes 0
    v[4, 9] = 3.0e38
    v[5] = np.linspace(-1.999, 1.999, 32)
    codes, sc = omx.quantize(v, bits)
    emax = omx.EMAX[bits]
    assert sc[0, 0] == 0 and (codes[0] == 0).all()
    assert sc[1, 0] == 127 - emax and omx.dequantize(codes, sc, bits)[1, 3] == -1.0
    assert sc[2, 0] == 127 + 2 - emax
    assert sc[3, 0] == 0
    assert sc[4, 0] == 127 + 127 - emax
    back = omx.dequantize(codes, sc, bits)
    # half a step of the largest binade, or the saturation of what lies between the largest code and
    # 2^(emax+1): 8 - 6 = 1 step of 2 (E2M1), 512 - 448 = 2 steps of 32 (E4M3)
    most = 2.0 ** (sc.astype(float) - 127) * (8 - 6 if bits == 4 else 512 - 448)
    assert (np.abs(back - v)[[0, 1, 2, 5]] <= most[[0, 1, 2, 5]]).all()


def test_packed_weights_positions():
    N, K = 128, 512
    codes = (np.arange(N * K).reshape(N, K) * 7 % 16).astype(np.uint8)
    scales = (np.arange(N * K // 32).reshape(N, K // 32) % 251).astype(np.uint8)
    p = omx.packed_weights(codes, scales)
    assert p.size == N * K * 17 // 32
    assert p[5 * 128 + 3] == codes[5, 6] | (codes[5, 7] << 4)
    assert p[17408 + 9 * 128] == codes[9, 256] | (codes[9, 257] << 4)
    assert p[17408 + 16384 + 512 + 16 * (70 % 32) + 4 * (70 // 32) + 2] == scales[70, 8 + 4 + 2]


def test_quad_scales_positions():
    s = (np.arange(40 * 8).reshape(40, 8) % 200 + 1).astype(np.uint8)
    q = omx.quad_scales(s)
    assert q.shape == (2, 40, 4, 4)
    assert (q[1, 3, 1] == s[35, 4:8]).all() and (q[0, 39, 0] == s[39, :4]).all()
    assert (q[0, 8, 1] == 0).all() and (q[:, :, 2:] == 0).all()      # rows 40 and up do not exist


@pytest.mark.parametrize("sigmoid", [False, True])
def test_gate_plain_is_torch_topk(sigmoid):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(40, 24, generator=g, dtype=torch.float64)
    ids, w = ogate.gate(x.numpy(), 5, sigmoid, renorm=False, scale=2.0)
    p = torch.sigmoid(x) if sigmoid else torch.softmax(x, -1)
    tv, ti = torch.topk(p, 5, dim=-1)
    np.testing.assert_array_equal(ids, ti.numpy())
    np.testing.assert_allclose(w, 2 * tv.numpy(), rtol=1e-14)
    _, wr = ogate.gate(x.numpy(), 5, sigmoid)
    np.testing.assert_allclose(wr, (tv / tv.sum(-1, keepdim=True)).numpy(), rtol=1e-13)


def test_gate_groups_bias_ties_and_masks():
    x = np.zeros((1, 8))
    ids, w = ogate.gate(x, 3, True)
    assert ids.tolist() == [[0, 1, 2]] and np.allclose(w, 1 / 3)
    bias = np.array([0, 0, 0, 0, 0, 0, .3, .3])
    assert ogate.gate(x, 2, True, bias)[0].tolist() == [[6, 7]]
    # groups of two, scored by their best expert or by both
    x = np.array([[5.0, -9, 3, 3, 2, 2, -9, -9]])
    assert ogate.gate(x, 2, True, np.zeros(8), n_group=4, topk_group=1, group_top=1)[0].tolist() == [[0, 1]]
    assert ogate.gate(x, 2, True, np.zeros(8), n_group=4, topk_group=1, group_top=2)[0].tolist() == [[2, 3]]
    x[0, 2:4] = -np.inf
    ids, w = ogate.gate(x, 3, False)
    assert ids.tolist() == [[0, 4, 5]] and np.isclose(w.sum(), 1)
    ids, w = ogate.gate(np.full((1, 4), -np.inf), 2, True)
    assert ids.tolist() == [[0, 1]] and (w == 0).all()
