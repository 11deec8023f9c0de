"""The router against the oracle in 64 bits: ids equal, gates within the error of their fp32 arithmetic."""
import numpy as np
import pytest
import torch

from oracle import gate as ogate

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LOWEST = float(torch.finfo(torch.float32).min)
INF = float("inf")


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


def rel_tol(x, softmax_sum):
    """Relative error of a gate, in units of 2^-23 (1 ulp at most): the exponentials of a numerator and of the
    sum, each 2 ulp and half an ulp of its argument (at most the spread of the finite logits, which enters as
    an absolute error); sum, quotient, product half an ulp each, k <= 32 terms added over 5 levels; with a softmax
    denominator, its fast exponentials ((2 + 1.16 d) e^-d <= 2.2 ulp of the sum) and at most 37 additions."""
    f = x[np.isfinite(x) & (np.abs(x) < 1e30)]
    spread = float(f.max() - f.min()) if f.size else 0.0
    return 2.0 ** -23 * (10 + min(spread, 700.0) + (22 if softmax_sum else 0))


def check(gsg, x, k, sigmoid, bias=None, n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0, stream=None):
    """x fp32 or bf16 tensor on the CPU."""
    kw = dict(n_group=n_group, topk_group=topk_group, group_top=group_top, renormalize=renorm, scale=scale)
    ids, gates = gsg.moe_gate(x.to(DEV), k, "sigmoid" if sigmoid else "softmax",
                              bias=None if bias is None else bias.to(DEV), **kw)
    assert ids.shape == gates.shape == (x.shape[0], k) and ids.dtype == torch.int32
    xd = x.double().numpy()
    oi, og = ogate.gate(xd, k, sigmoid, None if bias is None else bias.double().numpy(), n_group, topk_group,
                        group_top, renorm, scale)
    np.testing.assert_array_equal(ids.cpu().numpy(), oi)
    # (gates below the fp32 range's normal numbers may be flushed)
    np.testing.assert_allclose(gates.double().cpu().numpy(), og, rtol=rel_tol(xd, not sigmoid and not renorm),
                               atol=2.0 ** -126 * max(abs(scale), 1.0))
    return ids, gates


def randn(T, E, seed=0, dtype=torch.float32, spread=1.0):
    return (torch.randn(T, E, generator=torch.Generator().manual_seed(seed)) * spread).to(dtype)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,k,dtype", [(1, 1, 1, torch.float32), (3, 2, 2, torch.bfloat16), (65, 8, 2, torch.float32),
                                         (33, 31, 5, torch.float32), (5, 32, 32, torch.bfloat16),
                                         (130, 33, 8, torch.float32), (257, 64, 6, torch.bfloat16),
                                         (70, 100, 10, torch.float32), (200, 128, 8, torch.bfloat16),
                                         (64, 160, 6, torch.float32), (100, 256, 8, torch.float32),
                                         (50, 384, 8, torch.float32), (20, 385, 16, torch.bfloat16),
                                         (30, 512, 12, torch.float32), (9, 1000, 24, torch.float32),
                                         (4, 1024, 32, torch.float32)])
def test_plain(gsg, T, E, k, dtype, with_bias, sigmoid):
    bias = randn(1, E, 5)[0] * 0.05 if with_bias else None
    check(gsg, randn(T, E, E + k, dtype), k, sigmoid, bias, renorm=(T % 2 == 0), scale=1.0 if k < 8 else 2.5)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,n_group,topk_group,group_top,k", [(256, 8, 4, 2, 8), (256, 8, 4, 1, 8), (64, 4, 1, 2, 4),
                                                              (160, 8, 3, 1, 6), (512, 16, 7, 2, 16), (96, 32, 5, 2, 7),
                                                              (384, 2, 1, 2, 8), (72, 3, 2, 2, 5), (36, 18, 9, 1, 9),
                                                              (1024, 32, 8, 2, 32), (8, 8, 3, 1, 3)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_groups(gsg, E, n_group, topk_group, group_top, k, sigmoid, with_bias):
    bias = randn(1, E, 6)[0] * 0.05 if with_bias else None
    for dtype in (torch.float32, torch.bfloat16):    # (bf16 logits tie often)
        check(gsg, randn(61, E, 7, dtype), k, sigmoid, bias, n_group, topk_group, group_top, scale=2.5)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
def test_ties_and_masks(gsg, sigmoid, with_bias):
    E, k = 96, 8
    x = randn(14, E, 8)
    x[0] = 0.0                                 # all alike
    x[1] = 3.25
    x[2, ::2] = x[2, 0]                        # half alike
    x[3] = -INF                                # nothing available
    x[4, 3:] = -INF                            # fewer than k available
    x[5, :90] = -INF
    x[6] = LOWEST                              # masked by the type's lowest value
    x[6, 50] = 1.0
    x[7, ::3] = LOWEST
    x[8] = 0.0
    x[8, 40] = -0.0
    x[9] *= 1e4                                # saturated scores
    x[10] = torch.linspace(-80, 80, E)
    x[11] *= 1e-30
    x[12, 1:] = LOWEST
    x[13] = torch.linspace(88, 90, E)
    bias = None
    if with_bias:
        bias = randn(1, E, 9)[0] * 0.05
        bias[10:20] = -INF                     # experts taken out of service
        bias[30:40] = bias[30]
    for renorm in (True, False):
        check(gsg, x, k, sigmoid, bias, renorm=renorm)
        check(gsg, x, k, sigmoid, bias, 8, 3, 2, renorm=renorm)
        check(gsg, x, k, sigmoid, bias, 8, 3, 1, renorm=renorm)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,k,n_group", [(64, 6, 1), (256, 8, 8), (48, 20, 1), (320, 16, 1)])
def test_close_choices_are_settled_in_64_bits(gsg, sigmoid, E, k, n_group):
    """Scores that fp32 cannot tell apart: logits one unit apart, and biases that undo differences of the scores
    to within fractions of an fp32 unit."""
    g = torch.Generator().manual_seed(12)
    base = torch.randn(24, 1, generator=g)
    x = base.repeat(1, E)
    u = x.view(torch.int32) + torch.randint(-2, 3, x.shape, generator=g, dtype=torch.int32)
    x = u.view(torch.float32)                  # many near ties in a row: the general path
    x[8:16, k + 4:] -= 4.0                     # some near ties: the candidates' path
    x[16:] = torch.randn(8, E, generator=g)
    x[16:, 1::2] = x[16:, 0::2]                # equal logits under different biases
    bias = torch.zeros(E)
    bias[1::2] = torch.randint(-3, 4, (E // 2,), generator=g) * 2.0 ** -26
    check(gsg, x, k, sigmoid, bias, n_group, max(1, n_group // 2), 2 if n_group > 1 else 1)
    p = (torch.sigmoid(x[20].double()) if sigmoid else torch.softmax(x[20].double(), 0))
    check(gsg, x[20:21].repeat(3, 1), k, sigmoid, (0.7 - p).float(), n_group, max(1, n_group // 2))


def test_large_bias_and_scale(gsg):
    E = 40
    b = randn(1, E, 3)[0]
    for s in (1e3, 1e8, 1e30):
        check(gsg, randn(9, E, 2), 4, True, b * s, scale=-3.0)
        check(gsg, randn(9, E, 2), 4, False, b * s, renorm=False)


def test_non_finite_is_reported(gsg):
    x = randn(5, 64, 1).to(DEV)
    for bad in (float("nan"), INF):
        y = x.clone()
        y[2, 7] = bad
        ids, gates = gsg.moe_gate(y, 4, "sigmoid")
        assert gsg.get_device_status() == -5
        y[2, 7] = -INF                          # the expert counts as unavailable; nothing else changes
        i2, g2 = gsg.moe_gate(y, 4, "sigmoid")
        assert torch.equal(ids, i2) and torch.equal(gates, g2)
        b = torch.zeros(64, device=DEV)
        b[3] = bad
        ids, _ = gsg.moe_gate(x, 4, "softmax", bias=b)
        assert gsg.get_device_status() == -5 and not (ids == 3).any()


def test_empty_strides_streams_graphs_outputs(gsg):
    x = randn(300, 128, 4).to(DEV)
    ids, gates = gsg.moe_gate(x[:0], 8)
    assert ids.shape == (0, 8) and gates.shape == (0, 8)
    with pytest.raises(ValueError):
        gsg.moe_gate(x.t(), 8)
    with pytest.raises(ValueError):
        gsg.moe_gate(x[:, :64], 8)
    with pytest.raises(ValueError):
        gsg.moe_gate(x, 8, out_ids=torch.empty(300, 8, dtype=torch.int64, device=DEV))
    with pytest.raises(gsg.GsgError):
        gsg.moe_gate(x, 33)
    want = gsg.moe_gate(x, 8)
    odd = torch.empty(300 * 128 + 1, device=DEV)[1:].view(300, 128).copy_(x)      # 4-byte alignment
    for got in (gsg.moe_gate(odd, 8), gsg.moe_gate(x, 8, stream=torch.cuda.default_stream())):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = gsg.moe_gate(x, 8)
    s.synchronize()
    assert torch.equal(a[0], want[0])
    xi = torch.zeros_like(x)
    oi, og = torch.empty_like(want[0]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gsg.moe_gate(xi, 8, out_ids=oi, out_gates=og)
    xi.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(oi, want[0]) and torch.equal(og, want[1])
    del g


def test_many_tokens(gsg):
    """More tokens than resident warps, over every kernel width; checked on a sample."""
    for E, k in ((24, 3), (60, 4), (128, 8), (256, 8), (384, 8), (500, 8), (1024, 9)):
        x = randn(40000, E, E)
        b = randn(1, E, 1)[0] * 0.02
        ids, gates = gsg.moe_gate(x.to(DEV), k, "sigmoid", bias=b.to(DEV))
        p = torch.sigmoid(x.double())
        order = torch.sort(p + b.double(), dim=1, descending=True, stable=True)[1][:, :k]
        assert torch.equal(ids.cpu().long(), order)
        w = p.gather(1, order)
        torch.testing.assert_close(gates.cpu().double(), w / w.sum(1, keepdim=True), rtol=2.0 ** -23 * 20, atol=0)


def test_long_batch(gsg):
    """Offsets past 2^32 bytes in the logits."""
    x = randn(1000, 256, 3).to(DEV)
    ids, gates = gsg.moe_gate(x.repeat(5000, 1), 4, "sigmoid")
    i1, g1 = gsg.moe_gate(x, 4, "sigmoid")
    assert torch.equal(ids.view(5000, 1000, 4), i1.expand(5000, -1, -1))
    assert torch.equal(gates.view(5000, 1000, 4), g1.expand(5000, -1, -1))
