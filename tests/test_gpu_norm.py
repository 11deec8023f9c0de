"""Residual addition + RMS norm + microscaled output against the definition in 64 bits: h and the codes bit
for bit, y rounded once."""
import numpy as np
import pytest
import torch

from oracle import mx as omx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def gsg():
    import grouped_sparse_gemm_b200 as g
    g.load_library()
    return g


@pytest.fixture(autouse=True)
def clean_status(gsg):
    gsg.get_device_status()
    yield
    assert gsg.get_device_status() == 0


def rows(T, K, seed, dtype=BF, outliers=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g)
    if outliers:
        x[:, torch.randperm(K, generator=g)[: max(1, K // 64)]] *= 30
    return x.to(dtype)


def definition(x, w, r, eps):
    h = x.double()
    if r is not None:
        h = (x.float() + r.float()).to(r.dtype).double()   # (one fp32 addition, then h's own rounding)
    y = h * w.double() / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h, y


def check(gsg, x, w, r=None, eps=1e-6, fmt=8, want_y=True, scales_of=None):
    n = gsg.add_rmsnorm_mx(x.to(DEV), w.to(DEV), residual=None if r is None else r.to(DEV), eps=eps, fmt=fmt,
                           want_y=want_y)
    h, y = definition(x, w, r, eps)
    if r is None:
        assert n.h is None
    else:
        assert n.h.dtype == r.dtype and torch.equal(n.h.cpu().double(), h)
    if want_y:
        got = n.y.double().cpu()
        # one rounding to bf16 (2^-8 relative) of a value good to 2^-40; subnormals: half their step
        assert ((got - y).abs() <= y.abs() * (2.0 ** -8 * (1 + 2.0 ** -30)) + 2.0 ** -134).all()
        exact = (y.abs() > 1e-30)                         # nearest: no other bf16 number is closer
        up, dn = (torch.nextafter(n.y.cpu(), torch.tensor(s * float("inf"), dtype=BF)).double() for s in (1, -1))
        best = torch.minimum((up - y).abs(), (dn - y).abs())
        assert ((got - y).abs() <= best + y.abs() * 2.0 ** -40)[exact].all()
    else:
        assert n.y is None
    if fmt is None:
        assert n.act is None
        return n
    codes, sc = omx.quantize(y.numpy(), fmt)
    got = n.act.codes.cpu().numpy()
    np.testing.assert_array_equal(got, omx.pack_nibbles(codes) if fmt == 4 else codes)
    np.testing.assert_array_equal(n.act.scales.cpu().numpy(), omx.quad_scales(sc).reshape(-1))
    return n


@pytest.mark.parametrize("residual", [None, BF, F32])
@pytest.mark.parametrize("fmt", [4, 8, None])
@pytest.mark.parametrize("T,K", [(1, 256), (3, 512), (33, 2048), (130, 768), (5, 4096), (97, 4352), (2, 7168), (4, 8192),
                                 (3, 12288), (2, 16384), (2, 16640), (1, 32768)])
def test_norm(gsg, T, K, residual, fmt):
    w = (1 + 0.1 * rows(1, K, 1, F32, False)[0]).to(F32 if K % 512 else BF)
    r = None if residual is None else rows(T, K, 3, F32).to(residual) * 2
    check(gsg, rows(T, K, 2), w, r, fmt=fmt, want_y=fmt is None or T % 2 == 1)


@pytest.mark.parametrize("K", [8, 24, 264, 1000])
def test_norm_without_codes_any_multiple_of_eight(gsg, K):
    check(gsg, rows(9, K, 2), rows(1, K, 1, F32)[0], rows(9, K, 3), fmt=None)


def test_norm_extremes(gsg):
    K = 512
    w = torch.ones(K)
    x = torch.zeros(6, K, dtype=BF)
    x[1, 7] = 1.0                       # one value
    x[2] = 3e38                         # the squares pass the fp32 range
    x[3] = 1e-30                        # and fall below it
    x[4, ::2], x[4, 1::2] = 1e30, 1e-30
    x[5] = -2.0 ** -133                 # subnormal
    check(gsg, x, w, eps=1e-6)
    check(gsg, x[1:], w, eps=0.0)
    check(gsg, x[:2], w, rows(2, K, 5, F32) * 1e-20, eps=1e-12)
    check(gsg, rows(3, K, 6), -w * 1e-3, eps=1e-5, fmt=4)


def test_norm_flags_non_finite(gsg):
    x = rows(4, 256, 1).to(DEV)
    w = torch.ones(256, device=DEV)
    gsg.add_rmsnorm_mx(torch.zeros_like(x), w, eps=0.0)     # a row of zeros has no norm
    assert gsg.get_device_status() == -5
    for v in (float("nan"), float("inf")):
        y = x.clone()
        y[2, 3] = v
        n = gsg.add_rmsnorm_mx(y, w)
        assert gsg.get_device_status() == -5
        m = gsg.add_rmsnorm_mx(x, w)                        # the other rows are not touched by it
        for t in (0, 1, 3):
            assert torch.equal(n.y[t], m.y[t]) and torch.equal(n.act.codes[t], m.act.codes[t])


def test_norm_zero_rows_and_empty(gsg):
    check(gsg, torch.zeros(3, 256, dtype=BF), torch.ones(256))
    n = gsg.add_rmsnorm_mx(torch.zeros(0, 256, dtype=BF, device=DEV), torch.ones(256, device=DEV))
    assert n.y.shape == (0, 256) and n.act.R == 0


def test_norm_in_place_streams_graphs_and_refusals(gsg):
    x, r = rows(40, 1024, 1).to(DEV), rows(40, 1024, 2).to(DEV)
    w = torch.ones(1024, dtype=BF, device=DEV)
    want = gsg.add_rmsnorm_mx(x, w, residual=r)
    for dt in (BF, F32):                                    # the residual stream updated in place
        rr = r.to(dt, copy=True)
        a = gsg.add_rmsnorm_mx(x, w, residual=rr.clone(), fmt=4)
        b = gsg.add_rmsnorm_mx(x, w, residual=rr, out_h=rr, fmt=4)
        assert b.h is rr and torch.equal(a.h, rr) and torch.equal(a.act.codes, b.act.codes)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = gsg.add_rmsnorm_mx(x, w, residual=r, stream=s)
    s.synchronize()
    assert torch.equal(got.act.codes, want.act.codes) and torch.equal(got.act.scales, want.act.scales)
    xi, ri = torch.zeros_like(x), torch.zeros_like(r)
    out = gsg.add_rmsnorm_mx(xi, w, residual=ri)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gsg.add_rmsnorm_mx(xi, w, residual=ri, out_act=out.act, out_y=out.y, out_h=out.h)
    xi.copy_(x)
    ri.copy_(r)
    g.replay()
    torch.cuda.synchronize()
    for a, b in ((out.h, want.h), (out.y, want.y), (out.act.codes, want.act.codes), (out.act.scales, want.act.scales)):
        assert torch.equal(a, b)
    del g
    for bad in (lambda: gsg.add_rmsnorm_mx(x.t(), w), lambda: gsg.add_rmsnorm_mx(x, w[:512]),
                lambda: gsg.add_rmsnorm_mx(x, w, residual=r[:10]),
                lambda: gsg.add_rmsnorm_mx(x, w, out_y=torch.empty(40, 1024, device=DEV)),
                lambda: gsg.add_rmsnorm_mx(x, w, fmt=6)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gsg.GsgError):                       # 8-byte aligned rows
        gsg.add_rmsnorm_mx(torch.empty(40 * 1024 + 4, dtype=BF, device=DEV)[4:].view(40, 1024), w)


def test_norm_many_rows(gsg):
    """More rows than blocks at a time; the last rows of the scale layout."""
    x = rows(5000, 256, 1)
    n = gsg.add_rmsnorm_mx(x.to(DEV), torch.ones(256, device=DEV), fmt=8)
    codes, sc = omx.quantize(definition(x, torch.ones(256), None, 1e-6)[1].numpy(), 8)
    np.testing.assert_array_equal(n.act.codes.cpu().numpy(), codes)
    np.testing.assert_array_equal(n.act.scales.cpu().numpy(), omx.quad_scales(sc).reshape(-1))


def test_norm_long(gsg):
    """Offsets past 2^32 bytes in every input and output."""
    T, K = 270000, 16384
    x = rows(1000, K, 1).to(DEV)
    w = torch.ones(K, device=DEV)
    n = gsg.add_rmsnorm_mx(x.repeat(270, 1), w, residual=x.repeat(270, 1))
    m = gsg.add_rmsnorm_mx(x, w, residual=x)
    for t0 in (0, 131000, 262000, 269000):
        for a, b in ((n.h, m.h), (n.y, m.y), (n.act.codes, m.act.codes)):
            assert torch.equal(a[t0:t0 + 1000], b)
    long, short = n.act.scales.view(K // 128, T, 4, 4), m.act.scales.view(K // 128, 1000, 4, 4)
    assert torch.equal(long[:, -1000:], short) and torch.equal(long[:, 262000:263000, 0], short[:, :, 0])
