"""The microscaled experts against the oracle: packers and quantizer bit for bit, the grouped product on
every tile shape within the GEMM's stated tolerance, and what a serving loop does around them."""
import numpy as np
import pytest
import torch

from grouped_sparse_gemm_b200 import inputs
from oracle import gemm as ogemm
from oracle import mx as omx
from oracle import unpermute as ounperm
from tests import gsg_testlib as tl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


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


def weights(E, N, K, seed=0):
    """Checkpoint-style MXFP4 codes [E, N, K] and scales [E, N, K/32] (numpy), of normal weights."""
    g = np.random.default_rng(seed)
    out = [omx.quantize(g.standard_normal((N, K)) * 0.05, 4) for _ in range(E)]
    return np.stack([c for c, _ in out]), np.stack([s for _, s in out])


def pack(gsg, codes, scales):
    return gsg.pack_mxfp4_codes(torch.from_numpy(omx.pack_nibbles(codes)).to(DEV), torch.from_numpy(scales).to(DEV))


def oracle_rows(x, bits, src):
    codes, sc = omx.quantize(x.astype(np.float64), bits)
    return codes[src], sc[src]


# ------------------------------------------------------------------ packers
@pytest.mark.parametrize("E,N,K,dtype", [(1, 128, 256, torch.float32), (2, 256, 768, torch.bfloat16),
                                         (3, 128, 1280, torch.float32)])
def test_pack_bit_exact(gsg, E, N, K, dtype):
    g = torch.Generator().manual_seed(E)
    W = torch.randn(E, N, K, generator=g) * torch.exp(3 * torch.randn(E, N, 1, generator=g))
    W[0, 3, :64] = 0.0
    W[0, 4, :32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4)     # every E2M1 midpoint
    W[0, 5, 32:64] *= 2.0 ** -120
    W = W.to(dtype)
    p = gsg.pack_mxfp4(W.to(DEV))
    want = [omx.packed_weights(*omx.quantize(W[e].double().numpy(), 4)) for e in range(E)]
    np.testing.assert_array_equal(p.packed.cpu().numpy(), np.concatenate(want))


def test_pack_codes_keeps_the_bytes(gsg):
    codes, sc = weights(2, 256, 512, 4)
    p = pack(gsg, codes, sc)
    want = np.concatenate([omx.packed_weights(codes[e], sc[e]) for e in range(2)])
    np.testing.assert_array_equal(p.packed.cpu().numpy(), want)
    np.testing.assert_array_equal(p.expert(1).packed.cpu().numpy(), want[want.size // 2:])


def test_pack_flags(gsg):
    W = torch.zeros(1, 128, 256, device=DEV)
    W[0, 1, 2] = float("inf")
    gsg.pack_mxfp4(W)
    assert gsg.get_device_status() == -5
    gsg.pack_mxfp4_codes(torch.zeros(1, 128, 128, dtype=torch.uint8, device=DEV),
                         torch.full((1, 128, 8), 255, dtype=torch.uint8, device=DEV))
    assert gsg.get_device_status() == -5


# ------------------------------------------------------------------ quantizer
@pytest.mark.parametrize("fmt", [4, 8])
@pytest.mark.parametrize("T,k,E,K", [(1, 1, 4, 256), (33, 2, 4, 512), (64, 8, 128, 768), (130, 8, 16, 2048),
                                     (7, 40, 64, 256), (1, 8, 8, 7168)])
def test_quantize_bit_exact(gsg, T, k, E, K, fmt):
    cfg = inputs.custom_config("mx", E=E, K=K, N=128, T=T, top_k=k)
    X = inputs.activations(cfg)
    X[0, :32] = 0.0
    X[T // 2, 32:64] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4)
    X[T - 1, 64:96] = torch.linspace(-500, 500, 32)
    off, ps, ip = tl.route_np(inputs.routing(cfg), E)
    a = gsg.quantize_act_mx(X.to(DEV), fmt, inv_perm=torch.from_numpy(ip).to(DEV), top_k=k)
    codes, sc = oracle_rows(X.double().numpy(), fmt, ps // k)
    np.testing.assert_array_equal(a.codes.cpu().numpy(), omx.pack_nibbles(codes) if fmt == 4 else codes)
    np.testing.assert_array_equal(a.scales.cpu().numpy(), omx.quad_scales(sc).reshape(-1))


@pytest.mark.parametrize("fmt", [4, 8])
def test_quantize_two_phase_scales(gsg, fmt):
    T, k, K = 2049, 8, 8192       # R * K just past 2^27
    cfg = inputs.custom_config("mx2", E=64, K=K, N=128, T=T, top_k=k)
    X = inputs.activations(cfg)
    off, ps, ip = tl.route_np(inputs.routing(cfg), 64)
    a = gsg.quantize_act_mx(X.to(DEV), fmt, inv_perm=torch.from_numpy(ip).to(DEV), top_k=k)
    codes, sc = omx.quantize(X.double().numpy(), fmt)
    codes = omx.pack_nibbles(codes) if fmt == 4 else codes
    np.testing.assert_array_equal(a.codes.cpu().numpy(), codes[ps // k])
    s = torch.from_numpy(sc)[torch.from_numpy((ps // k).astype(np.int64))].view(T * k, K // 128, 4)
    got = a.scales.cpu().view(K // 128, T * k, 4, 4)
    for c in range(4):
        n = T * k - 32 * c
        assert torch.equal(got[:, :n, c], s[32 * c:].transpose(0, 1)) and (got[:, n:, c] == 0).all()


def test_quantize_flags_and_skips(gsg):
    X = torch.randn(4, 256, device=DEV).to(torch.bfloat16)
    ip = torch.tensor([0, 1, -1, 3, 4, 99, 6, 7], dtype=torch.int32, device=DEV)
    out = gsg.MxActivations(torch.full((8, 256), 77, dtype=torch.uint8, device=DEV),
                            torch.zeros(2 * 8 * 16, dtype=torch.uint8, device=DEV), 8, 256, 8)
    gsg.quantize_act_mx(X, 8, inv_perm=ip, top_k=2, out=out)
    assert gsg.get_device_status() == -4
    assert (out.codes[2] == 77).all() and (out.codes[5] == 77).all() and (out.codes[0] != 77).any()
    X[1, 5] = float("nan")
    gsg.quantize_act_mx(X, 4)
    assert gsg.get_device_status() == -5


# ------------------------------------------------------------------ product
def check_product(gsg, rows, N, K, fmt, hint, seed=0, out_dtype=torch.bfloat16, sample=None):
    E, R = len(rows), sum(rows)
    codes, sc = weights(E, N, K, seed)
    w = pack(gsg, codes, sc)
    X = np.random.default_rng(seed + 1).standard_normal((R, K)).astype(np.float32)
    X = torch.from_numpy(X).to(torch.bfloat16)
    off = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    a = gsg.quantize_act_mx(X.to(DEV), fmt)
    y = gsg.grouped_mx_gemm(a, w, torch.from_numpy(off).to(DEV), max_rows_per_expert=hint, out_dtype=out_dtype)
    q, s = omx.quantize(X.double().numpy(), fmt)
    A = omx.dequantize(q, s, fmt)
    for e in range(E):
        r = np.arange(off[e], off[e + 1])
        if sample and r.size > sample:    # the ends of the tiles and some rows between
            r = np.unique(np.r_[r[:3], r[-3:], r[::max(1, r.size // sample)], r[127:130], r[191:194], r[63:66]])
        if r.size:
            yr, b = ogemm.gemm_rows(A[r], omx.dequantize(codes[e], sc[e], 4), 1.0)
            tl.assert_gemm_close(y[torch.from_numpy(r).to(DEV)], yr, b, f"expert {e} of {rows}, N {N} K {K} fmt {fmt}")
    return a, w, torch.from_numpy(off).to(DEV), y


@pytest.mark.parametrize("fmt", [4, 8])
@pytest.mark.parametrize("rows,N,K,hint", [
    ([1], 128, 256, 1), ([16, 0, 5], 128, 512, 16), ([3] * 9, 640, 256, 3),      # 16-token tiles
    ([17, 32, 0, 1], 384, 768, 32),                                              # 32
    ([33, 64, 2], 256, 1280, 64), ([65, 200, 1, 0, 66], 128, 512, -1),           # 64, also over several tiles
    ([200] * 8, 4096, 1024, 200), ([128, 100, 7, 0, 129] * 4, 2048, 512, -1),    # 128-token wide pairs
    ([150, 180, 190, 0, 192, 193, 170, 160] * 4, 1536, 1792, 193),               # 192-token wide pairs
    ([400, 260, 31] * 6, 1152, 2048, -1),                                        # N not in whole 512
    ([1023], 4096, 512, 1023), ([700] * 3, 1920, 256, -1),
])
def test_product(gsg, rows, N, K, hint, fmt):
    check_product(gsg, rows, N, K, fmt, hint, sample=24)


@pytest.mark.parametrize("fmt", [4, 8])
@pytest.mark.parametrize("rows,N,K,hint", [([9, 0, 16], 256, 512, 16), ([70, 300, 100] * 8, 1664, 512, -1)])
def test_product_fp32_output_and_determinism(gsg, rows, N, K, hint, fmt):
    a, w, off, y = check_product(gsg, rows, N, K, fmt, hint, 5, torch.float32, sample=24)
    y2 = gsg.grouped_mx_gemm(a, w, off, max_rows_per_expert=hint, out_dtype=torch.float32)
    assert torch.equal(y, y2)
    yb = gsg.grouped_mx_gemm(a, w, off, max_rows_per_expert=hint)
    assert torch.equal(yb, y.to(torch.bfloat16))


@pytest.mark.parametrize("fmt", [4, 8])
def test_product_extreme_scales(gsg, fmt):
    """Scale bytes over their whole range (products that neither overflow nor vanish in fp32), zero rows,
    and the largest codes."""
    N, K, R = 128, 256, 20
    g = np.random.default_rng(7)
    codes = g.integers(0, 16, (1, N, K)).astype(np.uint8)
    sc = g.integers(0, 255, (1, N, K // 32)).astype(np.uint8)
    x = np.zeros((R, K))
    for r in range(R):       # row r: one block, scaled so that its products with one weight row are near 1
        b = r % (K // 32)
        x[r, 32 * b:32 * b + 32] = g.standard_normal(32) * 2.0 ** np.clip(127 - int(sc[0, r, b]), -100, 100)
    X = torch.from_numpy(x).to(torch.bfloat16)
    a = gsg.quantize_act_mx(X.to(DEV), fmt)
    y = gsg.grouped_mx_gemm(a, pack(gsg, codes, sc), torch.tensor([0, R], dtype=torch.int32, device=DEV), R,
                            out_dtype=torch.float32).double().cpu().numpy()
    q, s = omx.quantize(X.double().numpy(), fmt)
    yr, b = ogemm.gemm_rows(omx.dequantize(q, s, fmt), omx.dequantize(codes[0], sc[0], 4), 1.0)
    ok = b < 1e37            # (sums past the fp32 range are infinities)
    assert ok[np.arange(R), np.arange(R)].all()
    # the product's stated bound, without its absolute part (results below 2^-126 may be flushed)
    assert (np.abs(y - yr)[ok] <= ogemm.REL_TOL * b[ok] + 2.0 ** -126).all()


def test_product_leaves_other_rows(gsg):
    codes, sc = weights(2, 640, 256)
    w = pack(gsg, codes, sc)
    for R, n, hint in ((40, (7, 9), 16), (600, (200, 190), -1)):
        a = gsg.quantize_act_mx(torch.randn(R, 256, device=DEV).to(torch.bfloat16), 8)
        off = torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device=DEV)
        for dt in (torch.bfloat16, torch.float32):
            y = torch.full((R, 640), 3.0, dtype=dt, device=DEV)
            gsg.grouped_mx_gemm(a, w, off, hint, out=y)
            assert (y[sum(n):] == 3.0).all() and not (y[:sum(n)] == 3.0).all(dim=1).any()


@pytest.mark.parametrize("offs", [[0, 50, 20, 64], [0, -5, 40, 64], [0, 10, 900, 64]])
def test_product_corrupt_offsets(gsg, offs):
    codes, sc = weights(3, 512, 256)
    a = gsg.quantize_act_mx(torch.randn(64, 256, device=DEV).to(torch.bfloat16), 4)
    gsg.grouped_mx_gemm(a, pack(gsg, codes, sc), torch.tensor(offs, dtype=torch.int32, device=DEV))
    assert gsg.get_device_status() == -4


@pytest.mark.parametrize("fmt", [4, 8])
@pytest.mark.parametrize("rows,N,hint", [([9, 16], 128, 16), ([200] * 8, 2048, -1), ([180] * 32, 1536, 180)])
def test_product_timeout_then_clean(gsg, rows, N, hint, fmt):
    """A bounded wait made to run out: status, a clean return, and a correct next launch."""
    a, w, off, y = check_product(gsg, rows, N, 512, fmt, hint, 3, sample=8)
    L = gsg.lib()
    L.gsg_test_set_gemm_stall_ns(2_000_000)
    try:
        gsg.grouped_mx_gemm(a, w, off, hint)
        assert gsg.get_device_status() == -6
    finally:
        L.gsg_test_set_gemm_stall_ns(0)
    assert torch.equal(gsg.grouped_mx_gemm(a, w, off, hint), y)


@pytest.mark.parametrize("cap", [0, 1])
def test_product_tiles_decoded_without_table(gsg, cap):
    for rows, N, hint in (([9, 16, 3] * 20, 2048, 16), ([180, 100, 300] * 10, 2176, -1)):
        a, w, off, y = check_product(gsg, rows, N, 512, 8, hint, 3, sample=4)
        gsg.lib().gsg_test_set_gemm_table_cap(cap)
        try:
            assert torch.equal(gsg.grouped_mx_gemm(a, w, off, hint), y)
        finally:
            gsg.lib().gsg_test_set_gemm_table_cap(-1)


def test_product_long_output(gsg):
    """Output offsets past 2^32 bytes."""
    R, N, K = 270000, 8192, 256
    codes, sc = weights(1, N, K)
    w = pack(gsg, codes, sc)
    X = torch.randn(R, K, device=DEV).to(torch.bfloat16)
    a = gsg.quantize_act_mx(X, 4)
    y = gsg.grouped_mx_gemm(a, w, torch.tensor([0, R], dtype=torch.int32, device=DEV))
    r = torch.tensor([0, 131071, 262143, 262144, R - 129, R - 1], device=DEV)
    q, s = omx.quantize(X[r].double().cpu().numpy(), 4)
    yr, b = ogemm.gemm_rows(omx.dequantize(q, s, 4), omx.dequantize(codes[0], sc[0], 4), 1.0)
    tl.assert_gemm_close(y[r], yr, b, "long output")


@pytest.mark.parametrize("fmt", [4, 8])
def test_product_hint_below_the_truth(gsg, fmt):
    """The hint sets the tile, never the result: experts with more rows than it says."""
    check_product(gsg, [40, 0, 130, 3], 384, 512, fmt, 4, sample=24)
    check_product(gsg, [300] * 3 + [2] * 60, 1024, 256, fmt, 30, sample=8)
    check_product(gsg, [2] * 40, 4096, 256, fmt, 1)          # (runs of tiles by bytes)


@pytest.mark.parametrize("fmt", [4, 8])
@pytest.mark.parametrize("n,hint", [(3, 16), (150, -1)])
def test_product_many_experts(gsg, fmt, n, hint):
    """E = 1024: the expert tables take shared memory from the ring."""
    E, N, K = 1024, 128, 256
    codes, sc = weights(4, N, K)
    i = np.arange(E) % 4
    w = pack(gsg, codes[i], sc[i])
    X = torch.randn(E * n, K, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    off = torch.arange(E + 1, dtype=torch.int32, device=DEV) * n
    y = gsg.grouped_mx_gemm(gsg.quantize_act_mx(X.to(DEV), fmt), w, off, hint)
    for e in (0, 1, 511, 1023):
        q, s = omx.quantize(X[e * n:(e + 1) * n].double().numpy(), fmt)
        yr, b = ogemm.gemm_rows(omx.dequantize(q, s, fmt), omx.dequantize(codes[e % 4], sc[e % 4], 4), 1.0)
        tl.assert_gemm_close(y[e * n:(e + 1) * n], yr, b, f"expert {e}")


@pytest.mark.parametrize("fmt", [4, 8])
@pytest.mark.parametrize("hint", [3, 1])
def test_product_runs_of_tiles(gsg, fmt, hint):
    """Enough tiles per CTA for the schedule by bytes; with a hint below the truth too (20-row experts)."""
    E, N, K = 128, 4864, 256
    codes, sc = weights(2, N, K)
    i = np.arange(E) % 2
    w = pack(gsg, codes[i], sc[i])
    rows = np.full(E, 3) if hint == 3 else np.where(np.arange(E) % 9 == 4, 20, 1)
    off = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    X = torch.randn(int(off[-1]), K, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    y = gsg.grouped_mx_gemm(gsg.quantize_act_mx(X.to(DEV), fmt), w, torch.from_numpy(off).to(DEV), hint)
    q, s = omx.quantize(X.double().numpy(), fmt)
    A = omx.dequantize(q, s, fmt)
    W = [omx.dequantize(codes[e], sc[e], 4) for e in range(2)]
    for e in range(E):
        yr, b = ogemm.gemm_rows(A[off[e]:off[e + 1]], W[e % 2], 1.0)
        tl.assert_gemm_close(y[off[e]:off[e + 1]], yr, b, f"expert {e}")


@pytest.mark.parametrize("fmt", [4, 8])
def test_quantize_long(gsg, fmt):
    """Offsets past 2^32 bytes (and the two-launch scales of rows in token order)."""
    T, K = 270000, 16384
    x = torch.randn(1000, K, device=DEV).to(torch.bfloat16)
    X = x.repeat(270, 1)
    a = gsg.quantize_act_mx(X, fmt)
    codes, sc = omx.quantize(x.double().cpu().numpy(), fmt)
    codes = torch.from_numpy(omx.pack_nibbles(codes) if fmt == 4 else codes).to(DEV)
    for t0 in (0, 130000, 262000, 269000):
        assert torch.equal(a.codes[t0:t0 + 1000], codes)
    quad = a.scales.view(K // 128, T, 4, 4)
    words = torch.from_numpy(sc).to(DEV).view(1000, K // 128, 4).transpose(0, 1)
    assert torch.equal(quad[:, 269000:, 0], words) and torch.equal(quad[:, 262000:262968, 1], words[:, 32:])
    assert (quad[:, -32:, 1] == 0).all() and (quad[:, -96:, 3] == 0).all()


# ------------------------------------------------------------------ as a program uses them
def test_streams_graphs_and_own_outputs(gsg):
    rows, N, K = [40, 0, 70, 90], 512, 512
    a, w, off, y = check_product(gsg, rows, N, K, 8, -1, 2, sample=8)
    R = sum(rows)
    X1, X2 = (torch.randn(R, K, device=DEV).to(torch.bfloat16) for _ in range(2))
    want = []
    for x in (X1, X2):
        want.append(gsg.grouped_mx_gemm(gsg.quantize_act_mx(x, 8), w, off))
    # another stream, given and current
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a1 = gsg.quantize_act_mx(X1, 8, stream=s)
    with torch.cuda.stream(s):
        y1 = gsg.grouped_mx_gemm(a1, w, off)
    s.synchronize()
    assert torch.equal(y1, want[0])
    # captured once, replayed on new inputs, into the caller's buffers
    x = X1.clone()
    act = gsg.quantize_act_mx(x, 8)
    out = torch.empty_like(y1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gsg.quantize_act_mx(x, 8, out=act)
        gsg.grouped_mx_gemm(act, w, off, out=out)
    for x_, w_ in ((X2, want[1]), (X1, want[0])):
        x.copy_(x_)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w_)
    del g
    # two streams at once (no workspace is shared)
    s2 = torch.cuda.Stream()
    s2.wait_stream(torch.cuda.current_stream())
    s.wait_stream(torch.cuda.current_stream())
    ys = [gsg.grouped_mx_gemm(gsg.quantize_act_mx(x, 8, stream=t), w, off, stream=t) for x, t in ((X1, s), (X2, s2))]
    torch.cuda.synchronize()
    assert torch.equal(ys[0], want[0]) and torch.equal(ys[1], want[1])


def test_refuses_wrong_outputs(gsg):
    X = torch.randn(4, 256, device=DEV).to(torch.bfloat16)
    a = gsg.quantize_act_mx(X, 8)
    w = pack(gsg, *weights(1, 128, 256))
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        gsg.grouped_mx_gemm(a, w, off, out=torch.empty(4, 256, device=DEV))
    with pytest.raises(ValueError):
        gsg.quantize_act_mx(X, 4, out=a)
    with pytest.raises(ValueError):
        gsg.quantize_act_mx(X.t(), 8)
    with pytest.raises(ValueError):
        gsg.quantize_act_mx(X, 8, inv_perm=torch.zeros(7, dtype=torch.int32, device=DEV), top_k=2)
    with pytest.raises(ValueError):
        gsg.quantize_act_mx(X, 6)
    with pytest.raises(gsg.GsgError):
        gsg.quantize_act_mx(torch.zeros(4, 128, dtype=torch.bfloat16, device=DEV), 8)


def test_routed_layer(gsg):
    """A layer as it is served: residual norm -> router -> routing -> MXFP8 rows -> up-projection (gate | up)
    -> SwiGLU -> MXFP8 -> down-projection -> scatter; every stage against the oracle on the stage's inputs."""
    from oracle import gate as ogate
    E, H, I, T, k = 16, 512, 256, 70, 4
    g = torch.Generator().manual_seed(11)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    res = torch.randn(T, H, generator=g).to(torch.bfloat16)
    nw = (1 + 0.1 * torch.randn(H, generator=g)).to(torch.bfloat16)
    router = torch.randn(E, H, generator=g) / H ** 0.5
    bias = 0.05 * torch.randn(E, generator=g)
    up, down = weights(E, 2 * I, H, 1), weights(E, H, I, 2)
    wu, wd = pack(gsg, *up), pack(gsg, *down)

    n = gsg.add_rmsnorm_mx(x.to(DEV), nw.to(DEV), residual=res.to(DEV))
    logits = n.y.float() @ router.to(DEV).T
    ids, gates = gsg.moe_gate(logits, k, "sigmoid", bias=bias.to(DEV), n_group=4, topk_group=2, group_top=2, scale=2.5)
    oi, og = ogate.gate(logits.double().cpu().numpy(), k, True, bias.double().numpy(), 4, 2, 2, True, 2.5)
    np.testing.assert_array_equal(ids.cpu().numpy(), oi)
    np.testing.assert_allclose(gates.double().cpu().numpy(), og, rtol=2.0 ** -18)
    r = gsg.moe_route_permute(ids, E)
    off, ps, ip = tl.route_np(ids, E)
    np.testing.assert_array_equal(r.offsets.cpu().numpy(), off)

    a = gsg.quantize_act_mx(n.y, 8, r.inv_perm, k)
    h = gsg.grouped_mx_gemm(a, wu, r.offsets)
    act = (torch.nn.functional.silu(h[:, :I].float()) * h[:, I:].float()).to(torch.bfloat16)
    a2 = gsg.quantize_act_mx(act, 8)
    y = gsg.grouped_mx_gemm(a2, wd, r.offsets)
    out = gsg.unpermute_scale(y, r.inv_perm, gates, k)

    def product(act_rows, w, got):
        q, s = omx.quantize(act_rows.double().cpu().numpy(), 8)
        A = omx.dequantize(q, s, 8)
        for e in range(E):
            if off[e] < off[e + 1]:
                yr, b = ogemm.gemm_rows(A[off[e]:off[e + 1]], omx.dequantize(w[0][e], w[1][e], 4), 1.0)
                tl.assert_gemm_close(got[off[e]:off[e + 1]], yr, b, f"expert {e}")
    product(n.y[torch.from_numpy(ps.astype(np.int64) // k).to(DEV)], up, h)
    product(act, down, y)
    want = ounperm.unpermute_scale(y.cpu().view(torch.uint16).numpy(), ip, gates.cpu().numpy(), k)
    np.testing.assert_array_equal(out.cpu().view(torch.uint16).numpy(), want)
    # a shared expert takes the norm's 8-bit rows directly, as a plain linear layer
    ws = weights(1, 640, H, 9)
    ys = gsg.grouped_mx_gemm(n.act, pack(gsg, *ws), torch.tensor([0, T], dtype=torch.int32, device=DEV))
    codes = n.act.codes.cpu().numpy()
    sc = n.act.scales.cpu().numpy().reshape(H // 128, T, 4, 4)[:, :, 0].transpose(1, 0, 2).reshape(T, -1)
    yr, b = ogemm.gemm_rows(omx.dequantize(codes, sc, 8), omx.dequantize(ws[0][0], ws[1][0], 4), 1.0)
    tl.assert_gemm_close(ys, yr, b, "shared expert")
