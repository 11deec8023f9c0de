"""Layers run back to back on one set of buffers, eagerly and as a captured graph: every kernel sees what the kernels
before it have written, however many of them are on the device at once."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


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


def mx_layer(gsg, E, N, K, T, k, fmt):
    """f(inputs, buffers or None) -> buffers by name: norm -> router -> routing -> rows -> product -> scatter."""
    g = torch.Generator(device=DEV).manual_seed(6)
    w = gsg.pack_mxfp4(torch.randn(E, N, K, generator=g, device=DEV) * 0.05)
    nw = 1 + 0.1 * torch.randn(K, generator=g, device=DEV)
    inputs = [(torch.randn(T, K, generator=g, device=DEV).to(BF), torch.randn(T, E, generator=g, device=DEV))
              for _ in range(2)]

    def run(x, o):
        n = gsg.add_rmsnorm_mx(x[0], nw, residual=x[0], out_y=o.get("y"), out_act=o.get("act"), out_h=o.get("h"))
        ids, gates = gsg.moe_gate(x[1], k, "sigmoid", out_ids=o.get("ids"), out_gates=o.get("gates"))
        r = gsg.moe_route_permute(ids, E, out=o.get("r"), workspace=o.get("ws"))
        a = gsg.quantize_act_mx(n.y, fmt, r.inv_perm, k, out=o.get("a"))
        Y = gsg.grouped_mx_gemm(a, w, r.offsets, out=o.get("Y"))
        out = gsg.unpermute_scale(Y, r.inv_perm, gates, k, out=o.get("out"))
        return dict(y=n.y, act=n.act, h=n.h, ids=ids, gates=gates, r=r, a=a, Y=Y, out=out,
                    ws=torch.empty(1 << 20, dtype=torch.uint8, device=DEV))
    return run, inputs


def nvfp4_layer(gsg, E, N, K, T, k, separate):
    """Routing and quantizer (in one call or two) -> product -> scatter on the sparse weights."""
    g = torch.Generator(device=DEV).manual_seed(7)
    w = gsg.pack_sparse_nvfp4(torch.randn(E, N, K, generator=g, device=DEV) * 0.05)
    inputs = [(torch.randn(T, K, generator=g, device=DEV).to(BF),
               torch.rand(T, E, generator=g, device=DEV).topk(k, dim=1)[1].to(torch.int32),
               torch.rand(T, k, generator=g, device=DEV)) for _ in range(2)]

    def run(x, o):
        if separate:
            r = gsg.moe_route_permute(x[1], E, out=o.get("r"), workspace=o.get("ws"))
            a = gsg.quantize_act_nvfp4(x[0], 32, r.inv_perm, k, out=o.get("a"), workspace=o.get("ws"))
        else:
            r, a = gsg.moe_dispatch_nvfp4(x[1], x[0], E, out_route=o.get("r"), out_act=o.get("a"), workspace=o.get("ws"))
        Y = gsg.grouped_sparse_gemm(a, w, r.offsets, out=o.get("Y"))
        out = gsg.unpermute_scale(Y, r.inv_perm, x[2], k, out=o.get("out"))
        return dict(r=r, a=a, Y=Y, out=out, ws=torch.empty(1 << 20, dtype=torch.uint8, device=DEV))
    return run, inputs


def fused_layer(gsg, E, K, I, T, k):
    """Routing and quantizer -> up-projection with SwiGLU -> down-projection with the combine."""
    g = torch.Generator(device=DEV).manual_seed(9)
    up = gsg.pack_sparse_nvfp4(torch.randn(E, 2 * I, K, generator=g, device=DEV) * 0.05)
    down = gsg.pack_sparse_nvfp4(torch.randn(E, K, I, generator=g, device=DEV) * 0.05)
    h_scale = torch.full((1,), 0.002, device=DEV)
    comb = gsg.combine_workspace(E, K, I, T, k, DEV)
    inputs = [(torch.randn(T, K, generator=g, device=DEV).to(BF),
               torch.rand(T, E, generator=g, device=DEV).topk(k, dim=1)[1].to(torch.int32),
               torch.rand(T, k, generator=g, device=DEV)) for _ in range(2)]

    def run(x, o):
        r, a = gsg.moe_dispatch_nvfp4(x[1], x[0], E, out_route=o.get("r"), out_act=o.get("a"), workspace=o.get("ws"))
        h = gsg.grouped_sparse_gemm_swiglu(a, up, r.offsets, h_scale, out=o.get("h"))
        out = gsg.grouped_sparse_gemm_combine(h, down, r, x[2], comb, out=o.get("out"))
        return dict(r=r, a=a, h=h, out=out, ws=torch.empty(1 << 20, dtype=torch.uint8, device=DEV))
    return run, inputs


LAYERS = [("fused", (8, 512, 256, 16, 2)), ("fused", (64, 1024, 512, 64, 8)), ("fused", (16, 1024, 512, 700, 4)),
          ("mx", (64, 1024, 2048, 64, 8, 8)), ("mx", (8, 1024, 1024, 16, 2, 4)), ("mx", (8, 256, 512, 1, 2, 8)),
          ("mx", (1, 1024, 2048, 300, 1, 8)), ("mx", (128, 768, 1024, 512, 8, 4)),
          ("nvfp4", (64, 1024, 2048, 64, 8, False)), ("nvfp4", (8, 1024, 1024, 16, 2, False)),
          ("nvfp4", (8, 1024, 1024, 16, 2, True)), ("nvfp4", (128, 768, 1024, 512, 8, True))]


@pytest.mark.parametrize("kind,sizes", LAYERS)
def test_layers_in_a_row_on_the_same_buffers(gsg, kind, sizes):
    run, inputs = {"mx": mx_layer, "nvfp4": nvfp4_layer, "fused": fused_layer}[kind](gsg, *sizes)
    want = [run(x, {})["out"].clone() for x in inputs]      # each on buffers of its own
    o = run(inputs[0], {})
    torch.cuda.synchronize()
    outs = [torch.empty_like(want[0]) for _ in inputs]
    order = (0, 1, 1, 0, 1, 0, 0, 1)
    differ = torch.zeros((), dtype=torch.int64, device=DEV)

    def some():
        for i in order:
            run(inputs[i], dict(o, out=outs[i]))

    def check(step):
        for t in outs:
            t.zero_()
        step()
        for t, v in zip(outs, want):
            differ.add_((t.view(torch.int16) != v.view(torch.int16)).any())
    for _ in range(100):
        check(some)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        some()
    for _ in range(300):
        check(graph.replay)
    torch.cuda.synchronize()
    assert int(differ) == 0
    del graph


@pytest.mark.parametrize("T", [1, 16, 200])
def test_weights_and_bias_changed_between_replays(gsg, T):
    """The norm's weight and the router's bias are rewritten in place, by the framework's own copies, between
    replays of a graph that reads them in every kernel."""
    E, K, k = 64, 1024, 4
    g = torch.Generator(device=DEV).manual_seed(8)
    x = torch.randn(T, K, generator=g, device=DEV).to(BF)
    logits = torch.randn(T, E, generator=g, device=DEV)
    sets = [(1 + 0.1 * torch.randn(K, generator=g, device=DEV), 0.3 * torch.randn(E, generator=g, device=DEV))
            for _ in range(3)]
    want = [(gsg.add_rmsnorm_mx(x, w), gsg.moe_gate(logits, k, "sigmoid", bias=b)) for w, b in sets]
    w, b = sets[0][0].clone(), sets[0][1].clone()
    outs = []
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(6):
            outs.append((gsg.add_rmsnorm_mx(x, w), gsg.moe_gate(logits, k, "sigmoid", bias=b)))
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for i in range(300):
        w.copy_(sets[i % 3][0])
        b.copy_(sets[i % 3][1])
        graph.replay()
        n, (ids, gates) = want[i % 3]
        for m, (jds, hates) in (outs[0], outs[-1]):
            differ.add_((m.act.codes != n.act.codes).any())
            differ.add_((m.y.view(torch.int16) != n.y.view(torch.int16)).any())
            differ.add_((jds != ids).any())
            differ.add_((hates != gates).any())
    torch.cuda.synchronize()
    assert int(differ) == 0
    del graph
