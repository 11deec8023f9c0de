"""Calls on a stream of the caller's: their buffers belong to that stream, whatever the current one does meanwhile."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
PAUSE = 100_000_000   # clock cycles, some 50 ms: longer than the host needs for what follows it


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


def tensors(o):
    """The tensors of a call's result."""
    if isinstance(o, torch.Tensor):
        return [o]
    if isinstance(o, (tuple, list)):
        return [t for v in o for t in tensors(v)]
    return tensors(list(vars(o).values())) if hasattr(o, "__dict__") else []


def same(a, b):
    a, b = tensors(a), tensors(b)
    assert len(a) == len(b) > 0
    for s, t in zip(a, b):
        assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))


def calls(gsg):
    """name -> f(stream): every call that allocates outputs, on small inputs made once."""
    g = torch.Generator().manual_seed(41)
    E, N, K, T, k = 4, 256, 512, 96, 2
    X = torch.randn(T, K, generator=g).to(BF).to(DEV)
    W = (torch.randn(E, N, K, generator=g) * 0.05).to(DEV)
    logits = torch.randn(T, E, generator=g).to(DEV)
    ids, gates = gsg.moe_gate(logits, k)
    r = gsg.moe_route_permute(ids, E)
    act = gsg.quantize_act_nvfp4(X, 32, r.inv_perm, k)
    act16 = gsg.quantize_act_nvfp4(X, 16, r.inv_perm, k)
    mx = gsg.quantize_act_mx(X, 8, r.inv_perm, k)
    ws, wd, wm = gsg.pack_sparse_nvfp4(W), gsg.pack_dense_nvfp4(W), gsg.pack_mxfp4(W)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8).to(DEV)
    scales = torch.full((E, N, K // 32), 120, dtype=torch.uint8, device=DEV)
    h_scale = torch.full((1,), 0.01, device=DEV)
    comb = gsg.combine_workspace(E, N, K, T, k, DEV)
    Y = gsg.grouped_sparse_gemm(act, ws, r.offsets)
    torch.cuda.synchronize()
    w1 = torch.ones(K, device=DEV)
    return {
        "pack_sparse_nvfp4": lambda s: gsg.pack_sparse_nvfp4(W, stream=s),
        "pack_dense_nvfp4": lambda s: gsg.pack_dense_nvfp4(W, stream=s),
        "moe_route_permute": lambda s: gsg.moe_route_permute(ids, E, stream=s),
        "quantize_act_nvfp4": lambda s: gsg.quantize_act_nvfp4(X, 16, r.inv_perm, k, stream=s),
        "moe_dispatch_nvfp4": lambda s: gsg.moe_dispatch_nvfp4(ids, X, E, 16, stream=s),
        "grouped_sparse_gemm": lambda s: gsg.grouped_sparse_gemm(act, ws, r.offsets, stream=s),
        "grouped_sparse_gemm_swiglu": lambda s: gsg.grouped_sparse_gemm_swiglu(act, ws, r.offsets, h_scale, stream=s).codes,
        "grouped_sparse_gemm_combine": lambda s: gsg.grouped_sparse_gemm_combine(act, ws, r, gates, comb, stream=s),
        "grouped_dense_gemm": lambda s: gsg.grouped_dense_gemm(act16, wd, r.offsets, stream=s),
        "grouped_dense_gemm_native": lambda s: gsg.grouped_dense_gemm_native(act16, wd, r.offsets, stream=s),
        "unpermute_scale": lambda s: gsg.unpermute_scale(Y, r.inv_perm, gates, k, stream=s),
        "moe_gate": lambda s: gsg.moe_gate(logits, k, stream=s),
        "add_rmsnorm_mx": lambda s: gsg.add_rmsnorm_mx(X, w1, residual=X, stream=s),
        "pack_mxfp4": lambda s: gsg.pack_mxfp4(W, stream=s),
        "pack_mxfp4_codes": lambda s: gsg.pack_mxfp4_codes(codes, scales, stream=s),
        "quantize_act_mx": lambda s: gsg.quantize_act_mx(X, 4, r.inv_perm, k, stream=s),
        "grouped_mx_gemm": lambda s: gsg.grouped_mx_gemm(mx, wm, r.offsets, stream=s),
    }


NAMES = ["pack_sparse_nvfp4", "pack_dense_nvfp4", "moe_route_permute", "quantize_act_nvfp4", "moe_dispatch_nvfp4",
         "grouped_sparse_gemm", "grouped_sparse_gemm_swiglu", "grouped_sparse_gemm_combine", "grouped_dense_gemm",
         "grouped_dense_gemm_native", "unpermute_scale", "moe_gate", "add_rmsnorm_mx", "pack_mxfp4", "pack_mxfp4_codes",
         "quantize_act_mx", "grouped_mx_gemm"]


@pytest.fixture(scope="module")
def table(gsg):
    return calls(gsg)


def test_every_call_is_here(table):
    assert sorted(table) == sorted(NAMES)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_not_what_the_current_stream_still_writes(table, name):
    """Memory that the current stream has been given back but still has work queued on."""
    call, s = table[name], torch.cuda.Stream()
    want = call(None)
    torch.cuda.synchronize()
    junk = [torch.empty_like(t) for _ in range(3) for t in tensors(want)]
    torch.cuda._sleep(PAUSE)
    for t in junk:
        t.view(torch.uint8).fill_(7)
    del t, junk
    got = call(s)
    torch.cuda.synchronize()
    same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_read_on_the_current_stream_stay(table, name):
    """An output dropped while the current stream still reads it is not the next call's on its own stream."""
    call, s, now = table[name], torch.cuda.Stream(), torch.cuda.current_stream()
    want = call(None)
    torch.cuda.synchronize()
    got = call(s)
    now.wait_stream(s)
    torch.cuda._sleep(PAUSE)
    copies = [t.clone() for t in tensors(got)]
    del got
    with torch.cuda.stream(s):
        junk = [torch.empty_like(t) for _ in range(3) for t in copies]
        for t in junk:
            t.view(torch.uint8).fill_(9)
    torch.cuda.synchronize()
    same(copies, want)


@pytest.mark.parametrize("which", ["quantize_act_mx", "quantize_act_nvfp4", "moe_dispatch_nvfp4", "pack_sparse_nvfp4"])
def test_workspace_is_not_given_away_while_it_is_used(gsg, which):
    """The library's own workspace, on a stream that has yet to run the call (sizes whose scale words take two
    launches)."""
    g = torch.Generator().manual_seed(42)
    T, k, K, E = 2049, 8, 8192, 16
    X = torch.randn(T, K, generator=g).to(BF).to(DEV)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).to(DEV)
    W = torch.randn(2, 128, 1024, generator=g).to(DEV)
    r = gsg.moe_route_permute(ids, E)
    op, args = {"quantize_act_mx": (gsg.OP_QUANTIZE_MX, (0, 0, K, T, k)), "quantize_act_nvfp4": (gsg.OP_QUANTIZE, (0, 0, K, T, k)),
                "moe_dispatch_nvfp4": (gsg.OP_DISPATCH, (E, 0, K, T, k)),
                "pack_sparse_nvfp4": (gsg.OP_PACK_SPARSE, (2, 128, 1024, 0, 1))}[which]
    size = gsg.workspace_size(op, *args)
    assert size > 0
    call = {"quantize_act_mx": lambda out, s: gsg.quantize_act_mx(X, 8, r.inv_perm, k, out=out, stream=s),
            "quantize_act_nvfp4": lambda out, s: gsg.quantize_act_nvfp4(X, 32, r.inv_perm, k, out=out, stream=s),
            "moe_dispatch_nvfp4": lambda out, s: gsg.moe_dispatch_nvfp4(ids, X, E, out_route=out and out[0],
                                                                        out_act=out and out[1], stream=s),
            "pack_sparse_nvfp4": lambda out, s: gsg.pack_sparse_nvfp4(W, out=out, stream=s)}[which]
    want, out = call(None, None), call(None, None)
    torch.cuda.synchronize()
    for t in tensors(out):
        t.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(PAUSE)
    call(out, s)
    mine = [torch.full((size,), 0xA5, dtype=torch.uint8, device=DEV) for _ in range(16)]
    torch.cuda.synchronize()
    assert all(bool((t == 0xA5).all()) for t in mine)
    same(out, want)


def test_two_streams_at_once_past_the_workspace_size(gsg):
    g = torch.Generator().manual_seed(43)
    T, k, K, E = 2049, 4, 8192, 16
    Xs = [torch.randn(T, K, generator=g).to(BF).to(DEV) for _ in range(2)]
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).to(DEV)
    r = gsg.moe_route_permute(ids, E)
    want = [gsg.quantize_act_mx(x, 4, r.inv_perm, k) for x in Xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [gsg.quantize_act_mx(x, 4, r.inv_perm, k, stream=s) for x, s in zip(Xs, streams)]
        torch.cuda.synchronize()
        same(got, want)


def test_captured_on_a_forked_stream_and_replayed_two_at_once(gsg):
    """Calls on a stream of their own inside a capture; two such graphs, each with the library's workspace, at once."""
    g = torch.Generator().manual_seed(44)
    T, k, K, E = 2049, 4, 8192, 16
    Xs = [torch.randn(T, K, generator=g).to(BF).to(DEV) for _ in range(2)]
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).to(DEV)
    r = gsg.moe_route_permute(ids, E)
    want = [gsg.quantize_act_mx(x, 8, r.inv_perm, k) for x in Xs]
    graphs, outs = [], []
    for x in Xs:
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            side.wait_stream(torch.cuda.current_stream())
            outs.append(gsg.quantize_act_mx(x, 8, r.inv_perm, k, stream=side))
            torch.cuda.current_stream().wait_stream(side)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for o in outs:
            for t in tensors(o):
                t.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        same(outs, want)
    del graphs, graph
