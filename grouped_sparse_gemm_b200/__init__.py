"""grouped_sparse_gemm_b200 -- grouped paired-4:8 NVFP4 expert GEMM for routed MoE on B200.

Thin Python binding over the C ABI of ``libgsg.so`` (declared in ``include/gsg.h``).  The
functions keep the ABI's names without the ``gsg_`` prefix and only marshal arguments: torch
provides device memory and the current stream, every step runs in the library's CUDA kernels.
A call given a `stream` runs there: its outputs and workspaces come from that stream's memory, and the caller
keeps its inputs until it has run and lets other streams wait for it.
There is no CPU fallback: if the library is missing or no GPU is present the calls raise.

Beside that path: the router (moe_gate), the residual RMS norm with microscaled output (add_rmsnorm_mx) and
the same grouped product on OCP microscaled weights (pack_mxfp4, pack_mxfp4_codes -> quantize_act_mx ->
grouped_mx_gemm).

The path (after "Hardware-Native Joint Sparse-Quantization for Trillion-Scale Mixture-of-Experts",
paperlayer.ai summary, §3.4 and §D.1): pack_sparse_nvfp4 (offline weights) ->
moe_route_permute -> quantize_act_nvfp4 -> grouped_sparse_gemm -> unpermute_scale
(moe_dispatch_nvfp4 = the routing and quantizer calls in one).  save_packed / load_packed keep
packed weights in a file: the packed format is the storage format.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

from . import _build

__all__ = [
    "GsgError", "lib", "load_library", "library_path",
    "PackedSparseWeights", "PackedDenseWeights", "Routing", "QuantizedActivations",
    "pack_sparse_nvfp4", "pack_dense_nvfp4", "moe_route_permute", "moe_route_permute_noalloc",
    "quantize_act_nvfp4", "moe_dispatch_nvfp4",
    "grouped_sparse_gemm", "grouped_sparse_gemm_swiglu", "grouped_sparse_gemm_combine", "combine_workspace",
    "grouped_dense_gemm", "grouped_dense_gemm_native", "unpermute_scale", "OP_COMBINE", "OP_DISPATCH",
    "get_device_status",
    "PackedMxWeights", "MxActivations", "pack_mxfp4", "pack_mxfp4_codes", "quantize_act_mx", "grouped_mx_gemm",
    "OP_QUANTIZE_MX", "MXFP4", "MXFP8", "moe_gate", "NormOutput", "add_rmsnorm_mx",
    "save_packed", "load_packed",
    "act_scales_bytes", "workspace_size", "OP_PACK_SPARSE", "OP_PACK_DENSE", "OP_ROUTE",
    "OP_QUANTIZE", "OP_GEMM", "EXPORTED_SYMBOLS",
]

OP_PACK_SPARSE, OP_PACK_DENSE, OP_ROUTE, OP_QUANTIZE, OP_GEMM, OP_COMBINE, OP_DISPATCH = 1, 2, 3, 4, 5, 6, 7
OP_QUANTIZE_MX = 8
OUT_BF16, OUT_F32 = 0, 1
MXFP4, MXFP8 = 4, 8
ACT_SCALE_PAD_ROWS = 256

EXPORTED_SYMBOLS = [
    "gsg_sparse_packed_bytes", "gsg_dense_packed_bytes", "gsg_act_codes_bytes", "gsg_act_scales_bytes",
    "gsg_workspace_size",
    "gsg_pack_sparse_nvfp4", "gsg_pack_dense_nvfp4", "gsg_moe_route_permute",
    "gsg_quantize_act_nvfp4", "gsg_grouped_sparse_gemm", "gsg_grouped_dense_gemm",
    "gsg_unpermute_scale", "gsg_get_device_status", "gsg_status_string", "gsg_version",
    "gsg_moe_route_permute_noalloc", "gsg_grouped_sparse_gemm_swiglu", "gsg_grouped_sparse_gemm_combine",
    "gsg_moe_dispatch_nvfp4", "gsg_test_set_gemm_stall_ns", "gsg_grouped_dense_gemm_native",
    "gsg_test_set_gemm_table_cap",
    "gsg_mx_packed_bytes", "gsg_mx_act_codes_bytes", "gsg_mx_act_scales_bytes", "gsg_pack_mxfp4",
    "gsg_pack_mxfp4_codes", "gsg_quantize_act_mx", "gsg_grouped_mx_gemm", "gsg_moe_gate", "gsg_add_rmsnorm_mx",
]

_STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported shape", -3: "CUDA error",
           -4: "bad routing", -5: "non-finite input", -6: "device timeout", -7: "workspace"}


class GsgError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {_STATUS.get(status, status)} ({status})")
        self.status = status


_lib: Optional[ctypes.CDLL] = None


def library_path() -> str:
    return _build.LIB


def load_library(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load libgsg.so (optionally compiling it first).  Raises when it is not there."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        if not build_if_missing:
            raise RuntimeError(f"libgsg.so is not built ({path}); run grouped_sparse_gemm_b200._build.build()")
        _build.build()
    L = ctypes.CDLL(path)
    vp, i, sz, fp = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
    sig = {
        "gsg_sparse_packed_bytes": (sz, [i, i, i]),
        "gsg_dense_packed_bytes": (sz, [i, i, i]),
        "gsg_act_codes_bytes": (sz, [i, i]),
        "gsg_act_scales_bytes": (sz, [i, i, i]),
        "gsg_workspace_size": (sz, [i, i, i, i, i, i]),
        "gsg_pack_sparse_nvfp4": (i, [vp, i, i, i, vp, fp, vp, sz, vp]),
        "gsg_pack_dense_nvfp4": (i, [vp, i, i, i, vp, fp, vp, sz, vp]),
        "gsg_moe_route_permute": (i, [vp, i, i, i, vp, vp, vp, vp, sz, vp]),
        "gsg_quantize_act_nvfp4": (i, [vp, i, i, i, vp, i, vp, vp, vp, vp, vp, sz, vp]),
        "gsg_moe_dispatch_nvfp4": (i, [vp, vp, i, i, i, i, i, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "gsg_grouped_sparse_gemm": (i, [vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, i, vp]),
        "gsg_grouped_dense_gemm": (i, [vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, i, vp]),
        "gsg_grouped_dense_gemm_native": (i, [vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, i, vp]),
        "gsg_unpermute_scale": (i, [vp, vp, vp, i, i, i, vp, vp]),
        "gsg_get_device_status": (i, [vp]),
        "gsg_status_string": (ctypes.c_char_p, [i]),
        "gsg_version": (i, []),
        "gsg_moe_route_permute_noalloc": (i, [vp, i, i, i, vp, vp, vp, vp]),
        "gsg_grouped_sparse_gemm_swiglu": (i, [vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, vp, vp, vp]),
        "gsg_grouped_sparse_gemm_combine": (i, [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, vp, vp, sz, vp, vp]),
        "gsg_test_set_gemm_stall_ns": (None, [ctypes.c_ulonglong]),
        "gsg_test_set_gemm_table_cap": (None, [ctypes.c_int]),
        "gsg_mx_packed_bytes": (sz, [i, i, i]),
        "gsg_mx_act_codes_bytes": (sz, [i, i, i]),
        "gsg_mx_act_scales_bytes": (sz, [i, i]),
        "gsg_pack_mxfp4": (i, [vp, i, i, i, i, vp, vp]),
        "gsg_pack_mxfp4_codes": (i, [vp, vp, i, i, i, vp, vp]),
        "gsg_quantize_act_mx": (i, [vp, i, i, i, vp, i, vp, vp, vp, sz, vp]),
        "gsg_moe_gate": (i, [vp, i, vp, i, i, i, i, i, i, i, i, ctypes.c_float, vp, vp, vp]),
        "gsg_add_rmsnorm_mx": (i, [vp, vp, i, vp, i, i, i, ctypes.c_float, vp, vp, i, vp, vp, vp]),
        "gsg_grouped_mx_gemm": (i, [vp, vp, i, vp, vp, i, i, i, i, i, vp, i, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def lib() -> ctypes.CDLL:
    return load_library()


# ------------------------------------------------------------------ helpers
def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream: Optional[torch.cuda.Stream] = None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn: str, st: int):
    if st != 0:
        raise GsgError(fn, st)


def _tensors(o) -> list:
    """The tensors of a call's result (a tensor, a tuple, one of the classes below)."""
    if isinstance(o, torch.Tensor):
        return [o]
    return [t for v in (o if isinstance(o, tuple) else vars(o).values() if hasattr(o, "__dict__") else ())
            for t in _tensors(v)]


def _on_stream(fn, stream, *args):
    """fn(*args), a call of this module, with `stream` current.  What it allocates is that stream's memory: neither
    what the stream current until now has yet to write, nor given to it while the call still runs.  That stream
    may read the outputs (once it waits for `stream`), also if they are dropped before it has."""
    # (by the stream's numbers: torch.cuda.stream() and the Stream objects that it makes take 15 us)
    now = torch._C._cuda_getCurrentStream(torch.cuda.current_device())
    new = (stream.stream_id, stream.device_index, stream.device_type)
    if new == now:
        return fn(*args)
    _set_stream(new)
    try:
        out = fn(*args)
    finally:
        _set_stream(now)
    for o in out if isinstance(out, tuple) else (out,):
        if not any(o is a for a in args):   # (not the caller's own buffers)
            for t in _tensors(o):
                t.record_stream(torch.cuda.current_stream())
    return out


def _set_stream(s) -> None:
    torch._C._cuda_setStream(stream_id=s[0], device_index=s[1], device_type=s[2])


def _need_cuda(*ts: Optional[torch.Tensor]):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("grouped_sparse_gemm_b200 works on CUDA tensors only (no CPU fallback)")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def workspace_size(op: int, E: int = 0, N: int = 0, K: int = 0, T: int = 0, k: int = 1) -> int:
    return int(lib().gsg_workspace_size(op, E, N, K, T, k))


def act_scales_bytes(R: int, K: int, sf_block: int) -> int:
    return int(lib().gsg_act_scales_bytes(R, K, sf_block))


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ packed containers
SPARSE_CHUNK_BYTES = 11264     # one (expert, n-tile, 256-wide K chunk) block: values | metadata | scales
DENSE_CHUNK_BYTES = 18432


@dataclass
class PackedSparseWeights:
    packed: torch.Tensor   # uint8 [E*N*K*11/32], chunk blocks (see include/gsg.h)
    w_scale: torch.Tensor  # fp32 [E]
    E: int
    N: int
    K: int

    def nbytes(self) -> int:
        return self.packed.numel()

    def expert(self, e: int) -> "PackedSparseWeights":
        """View of expert e alone (E = 1)."""
        n = self.packed.numel() // self.E
        return PackedSparseWeights(self.packed[e * n:(e + 1) * n], self.w_scale[e:e + 1], 1, self.N, self.K)


@dataclass
class PackedDenseWeights:
    packed: torch.Tensor   # uint8 [E*N*K*9/16]
    w_scale: torch.Tensor  # fp32 [E]
    E: int
    N: int
    K: int

    def nbytes(self) -> int:
        return self.packed.numel()

    def expert(self, e: int) -> "PackedDenseWeights":
        n = self.packed.numel() // self.E
        return PackedDenseWeights(self.packed[e * n:(e + 1) * n], self.w_scale[e:e + 1], 1, self.N, self.K)


@dataclass
class Routing:
    offsets: torch.Tensor   # int32 [E+1]
    perm_src: torch.Tensor  # int32 [R]
    inv_perm: torch.Tensor  # int32 [R]
    T: int
    k: int
    E: int


@dataclass
class QuantizedActivations:
    codes: torch.Tensor     # uint8 [R, K/2]
    scales: torch.Tensor    # uint8, quad layout
    x_scale: torch.Tensor   # fp32 [1]
    R: int
    K: int
    sf_block: int


MX_CHUNK_BYTES = 17408         # one (expert, n-tile, 256-wide K chunk) block: codes | scales


@dataclass
class PackedMxWeights:
    packed: torch.Tensor   # uint8 [E*N*K*17/32], MXFP4 chunk blocks (see include/gsg.h)
    E: int
    N: int
    K: int

    def nbytes(self) -> int:
        return self.packed.numel()

    def expert(self, e: int) -> "PackedMxWeights":
        """View of expert e alone (E = 1)."""
        n = self.packed.numel() // self.E
        return PackedMxWeights(self.packed[e * n:(e + 1) * n], 1, self.N, self.K)


@dataclass
class MxActivations:
    codes: torch.Tensor     # uint8 [R, K/2] (MXFP4) or [R, K] (MXFP8, E4M3)
    scales: torch.Tensor    # uint8 [K/128 * R * 16], UE8M0, quad layout without padding rows
    R: int
    K: int
    fmt: int                # MXFP4 (4) or MXFP8 (8)


@dataclass
class NormOutput:
    act: Optional[MxActivations]   # microscaled rows (None when fmt is None)
    y: Optional[torch.Tensor]      # bf16 [T, K] (None when not wanted)
    h: Optional[torch.Tensor]      # [T, K], the residual stream after the addition (None without a residual)


# ------------------------------------------------------------------ storage
PACKED_FILE_VERSION = 1


def save_packed(w, path: str) -> None:
    """Packed weights (PackedSparseWeights, PackedDenseWeights or PackedMxWeights, any device) to an .npz
    file: the packed bytes exactly as the GEMM reads them, the per-expert FP32 tensor scales (the MXFP4
    weights have none), E, N, K and the format.  No re-encoding: load_packed gives back the same bytes."""
    import numpy as np
    fmt = "sparse" if isinstance(w, PackedSparseWeights) else "mxfp4" if isinstance(w, PackedMxWeights) else "dense"
    scale = {} if fmt == "mxfp4" else {"w_scale": w.w_scale.detach().cpu().numpy()}
    np.savez(path, version=PACKED_FILE_VERSION, format=fmt, E=w.E, N=w.N, K=w.K,
             packed=w.packed.detach().cpu().numpy(), **scale)


def load_packed(path: str, device=None):
    """Packed weights from a save_packed file, on `device` (default: CPU).  Checks the version,
    the format and that the byte count is the library's size for (E, N, K); raises ValueError
    otherwise."""
    import numpy as np
    with np.load(path, allow_pickle=False) as d:
        if int(d["version"]) != PACKED_FILE_VERSION:
            raise ValueError(f"{path}: packed-weights file version {int(d['version'])}, expected "
                             f"{PACKED_FILE_VERSION}")
        fmt = str(d["format"])
        E, N, K = int(d["E"]), int(d["N"]), int(d["K"])
        packed, w_scale = d["packed"], None if fmt == "mxfp4" else d["w_scale"]
    if fmt not in ("sparse", "dense", "mxfp4"):
        raise ValueError(f"{path}: unknown packed format {fmt!r}")
    # the shape rule of the packers (whole 128-row n-tiles, whole 256-wide K chunks, int range),
    # checked before the byte count so that a wrong N or K of the right size is still rejected
    int_max = 2 ** 31 - 1
    if not (1 <= E <= int_max and 128 <= N <= int_max and 256 <= K <= int_max and N % 128 == 0
            and K % 256 == 0):
        raise ValueError(f"{path}: E={E} N={N} K={K} is not a packed shape (E >= 1, N a multiple of 128, "
                         f"K a multiple of 256)")
    L = lib()
    need = {"sparse": L.gsg_sparse_packed_bytes, "dense": L.gsg_dense_packed_bytes,
            "mxfp4": L.gsg_mx_packed_bytes}[fmt](E, N, K)
    if packed.dtype != np.uint8 or packed.ndim != 1 or packed.size != need:
        raise ValueError(f"{path}: {packed.size} packed bytes, expected {need} for {fmt} E={E} N={N} K={K}")
    pk = torch.from_numpy(packed.copy()).to(device or "cpu")
    if fmt == "mxfp4":
        return PackedMxWeights(packed=pk, E=E, N=N, K=K)
    if w_scale.dtype != np.float32 or w_scale.shape != (E,):
        raise ValueError(f"{path}: tensor scales of shape {w_scale.shape} / {w_scale.dtype}, expected ({E},) float32")
    ws = torch.from_numpy(w_scale.copy()).to(device or "cpu")
    cls = PackedSparseWeights if fmt == "sparse" else PackedDenseWeights
    return cls(packed=pk, w_scale=ws, E=E, N=N, K=K)


# ------------------------------------------------------------------ entry points
def pack_sparse_nvfp4(W: torch.Tensor, out: Optional[PackedSparseWeights] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> PackedSparseWeights:
    """W fp32 [E, N, K] -> paired 4:8 NVFP4 packed weights (gsg_pack_sparse_nvfp4)."""
    if stream is not None:
        return _on_stream(pack_sparse_nvfp4, stream, W, out, workspace)
    _need_cuda(W)
    assert W.dtype == torch.float32 and W.dim() == 3
    E, N, K = W.shape
    L = lib()
    dev = W.device
    if out is None:
        out = PackedSparseWeights(
            packed=torch.empty(L.gsg_sparse_packed_bytes(E, N, K), dtype=torch.uint8, device=dev),
            w_scale=torch.empty(E, dtype=torch.float32, device=dev), E=E, N=N, K=K)
    need = workspace_size(OP_PACK_SPARSE, E, N, K)
    ws = workspace if workspace is not None else _workspace(need, dev)
    _check("gsg_pack_sparse_nvfp4", L.gsg_pack_sparse_nvfp4(
        _ptr(W), E, N, K, _ptr(out.packed), _ptr(out.w_scale), _ptr(ws), ws.numel(), _stream()))
    return out


def pack_dense_nvfp4(W: torch.Tensor, out: Optional[PackedDenseWeights] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> PackedDenseWeights:
    """W fp32 [E, N, K] -> dense NVFP4 (16-element blocks) for the control GEMM."""
    if stream is not None:
        return _on_stream(pack_dense_nvfp4, stream, W, out, workspace)
    _need_cuda(W)
    assert W.dtype == torch.float32 and W.dim() == 3
    E, N, K = W.shape
    L = lib()
    dev = W.device
    if out is None:
        out = PackedDenseWeights(
            packed=torch.empty(L.gsg_dense_packed_bytes(E, N, K), dtype=torch.uint8, device=dev),
            w_scale=torch.empty(E, dtype=torch.float32, device=dev), E=E, N=N, K=K)
    need = workspace_size(OP_PACK_DENSE, E, N, K)
    ws = workspace if workspace is not None else _workspace(need, dev)
    _check("gsg_pack_dense_nvfp4", L.gsg_pack_dense_nvfp4(
        _ptr(W), E, N, K, _ptr(out.packed), _ptr(out.w_scale), _ptr(ws), ws.numel(), _stream()))
    return out


def moe_route_permute(topk_ids: torch.Tensor, E: int, out: Optional[Routing] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> Routing:
    """topk ids int32 [T, k] -> expert offsets, perm_src, inv_perm (gsg_moe_route_permute)."""
    if stream is not None:
        return _on_stream(moe_route_permute, stream, topk_ids, E, out, workspace)
    _need_cuda(topk_ids)
    assert topk_ids.dtype == torch.int32 and topk_ids.dim() == 2
    T, k = topk_ids.shape
    dev = topk_ids.device
    if out is None:
        out = Routing(offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                      perm_src=torch.empty(max(T * k, 1), dtype=torch.int32, device=dev),
                      inv_perm=torch.empty(max(T * k, 1), dtype=torch.int32, device=dev), T=T, k=k, E=E)
    ws = workspace
    if ws is None:   # the size query only when the call has to allocate
        need = workspace_size(OP_ROUTE, E, 0, 0, T, k)
        ws = _workspace(need, dev) if need else None
    _check("gsg_moe_route_permute", lib().gsg_moe_route_permute(
        _ptr(topk_ids), T, k, E, _ptr(out.offsets), _ptr(out.perm_src), _ptr(out.inv_perm),
        _ptr(ws), 0 if ws is None else ws.numel(), _stream()))
    return out


def moe_route_permute_noalloc(topk_ids: torch.Tensor, E: int, out: Routing, stream=None) -> Routing:
    """gsg_moe_route_permute_noalloc: the same routing with the library's fixed scratch instead of
    a workspace, for callers that may not allocate device memory at this point (outputs in `out`
    are caller-allocated; nothing is allocated here)."""
    _need_cuda(topk_ids, out.offsets, out.perm_src, out.inv_perm)
    assert topk_ids.dtype == torch.int32 and topk_ids.dim() == 2
    T, k = topk_ids.shape
    _check("gsg_moe_route_permute_noalloc", lib().gsg_moe_route_permute_noalloc(
        _ptr(topk_ids), T, k, E, _ptr(out.offsets), _ptr(out.perm_src), _ptr(out.inv_perm), _stream(stream)))
    return out


def quantize_act_nvfp4(X: torch.Tensor, sf_block: int = 32, inv_perm: Optional[torch.Tensor] = None,
                       top_k: int = 1, x_scale_in: Optional[torch.Tensor] = None,
                       out: Optional[QuantizedActivations] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> QuantizedActivations:
    """X bf16 [T, K] -> NVFP4 codes/scales in routed row order (gsg_quantize_act_nvfp4)."""
    if stream is not None:
        return _on_stream(quantize_act_nvfp4, stream, X, sf_block, inv_perm, top_k, x_scale_in, out, workspace)
    _need_cuda(X, inv_perm, x_scale_in)
    assert X.dtype == torch.bfloat16 and X.dim() == 2
    T, K = X.shape
    R = T * top_k
    dev = X.device
    if out is None:
        out = QuantizedActivations(
            codes=torch.empty(max(R, 1), K // 2, dtype=torch.uint8, device=dev),
            scales=torch.empty(act_scales_bytes(R, K, sf_block), dtype=torch.uint8, device=dev),
            x_scale=torch.empty(1, dtype=torch.float32, device=dev), R=R, K=K, sf_block=sf_block)
    ws = workspace if workspace is not None else _workspace(workspace_size(OP_QUANTIZE, 0, 0, K, T, top_k), dev)
    _check("gsg_quantize_act_nvfp4", lib().gsg_quantize_act_nvfp4(
        _ptr(X), T, K, sf_block, _ptr(inv_perm), top_k, _ptr(x_scale_in), _ptr(out.codes),
        _ptr(out.scales), _ptr(out.x_scale), _ptr(ws), ws.numel(), _stream()))
    return out


def moe_dispatch_nvfp4(topk_ids: torch.Tensor, X: torch.Tensor, E: int, sf_block: int = 32,
                       x_scale_in: Optional[torch.Tensor] = None, out_route: Optional[Routing] = None,
                       out_act: Optional[QuantizedActivations] = None, workspace: Optional[torch.Tensor] = None,
                       stream=None):
    """moe_route_permute + quantize_act_nvfp4 in one call (gsg_moe_dispatch_nvfp4): the same
    outputs bit for bit, one launch fewer.  Returns (Routing, QuantizedActivations)."""
    if stream is not None:
        return _on_stream(moe_dispatch_nvfp4, stream, topk_ids, X, E, sf_block, x_scale_in, out_route, out_act,
                          workspace)
    _need_cuda(topk_ids, X, x_scale_in)
    assert topk_ids.dtype == torch.int32 and topk_ids.dim() == 2
    assert X.dtype == torch.bfloat16 and X.dim() == 2 and X.shape[0] == topk_ids.shape[0]
    T, k = topk_ids.shape
    K = X.shape[1]
    R = T * k
    dev = X.device
    if out_route is None:
        out_route = Routing(offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                            perm_src=torch.empty(max(R, 1), dtype=torch.int32, device=dev),
                            inv_perm=torch.empty(max(R, 1), dtype=torch.int32, device=dev), T=T, k=k, E=E)
    if out_act is None:
        out_act = QuantizedActivations(
            codes=torch.empty(max(R, 1), K // 2, dtype=torch.uint8, device=dev),
            scales=torch.empty(act_scales_bytes(R, K, sf_block), dtype=torch.uint8, device=dev),
            x_scale=torch.empty(1, dtype=torch.float32, device=dev), R=R, K=K, sf_block=sf_block)
    ws = workspace if workspace is not None else _workspace(workspace_size(OP_DISPATCH, E, 0, K, T, k), dev)
    _check("gsg_moe_dispatch_nvfp4", lib().gsg_moe_dispatch_nvfp4(
        _ptr(topk_ids), _ptr(X), T, k, E, K, sf_block, _ptr(x_scale_in), _ptr(out_route.offsets),
        _ptr(out_route.perm_src), _ptr(out_route.inv_perm), _ptr(out_act.codes), _ptr(out_act.scales),
        _ptr(out_act.x_scale), _ptr(ws), ws.numel(), _stream()))
    return out_route, out_act


def grouped_sparse_gemm(act: QuantizedActivations, w: PackedSparseWeights, offsets: torch.Tensor,
                        max_rows_per_expert: int = -1, out: Optional[torch.Tensor] = None,
                        out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """Y [R, N] = per-expert X_e . W_e^T on paired 4:8 NVFP4 weights (gsg_grouped_sparse_gemm)."""
    if stream is not None:
        return _on_stream(grouped_sparse_gemm, stream, act, w, offsets, max_rows_per_expert, out, out_dtype)
    assert act.sf_block == 32 and act.K == w.K
    _need_cuda(act.codes, act.scales, offsets)
    if out is None:
        out = torch.empty(max(act.R, 1), w.N, dtype=out_dtype, device=act.codes.device)
    ydt = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    _check("gsg_grouped_sparse_gemm", lib().gsg_grouped_sparse_gemm(
        _ptr(act.codes), _ptr(act.scales), _ptr(act.x_scale), _ptr(w.packed), _ptr(w.w_scale),
        _ptr(offsets), w.E, w.N, w.K, act.R, max_rows_per_expert, _ptr(out), ydt, _stream()))
    return out


def grouped_sparse_gemm_swiglu(act: QuantizedActivations, w: PackedSparseWeights, offsets: torch.Tensor,
                               h_scale: torch.Tensor, max_rows_per_expert: int = -1,
                               out: Optional[QuantizedActivations] = None, stream=None) -> QuantizedActivations:
    """Up-projection (fused gate|up weights [2I, K]) with SwiGLU and NVFP4 quantization of
    h = silu(gate) * up in the epilogue (gsg_grouped_sparse_gemm_swiglu): returns h's codes and
    scales, ready as the down-projection's activations (tensor scale h_scale, fp32 [1])."""
    if stream is not None:
        return _on_stream(grouped_sparse_gemm_swiglu, stream, act, w, offsets, h_scale, max_rows_per_expert, out)
    assert act.sf_block == 32 and act.K == w.K and w.N % 256 == 0
    _need_cuda(act.codes, act.scales, offsets, h_scale)
    I = w.N // 2
    dev = act.codes.device
    if out is None:
        out = QuantizedActivations(codes=torch.empty(max(act.R, 1), I // 2, dtype=torch.uint8, device=dev),
                                   scales=torch.empty(act_scales_bytes(act.R, I, 32), dtype=torch.uint8, device=dev),
                                   x_scale=h_scale, R=act.R, K=I, sf_block=32)
    _check("gsg_grouped_sparse_gemm_swiglu", lib().gsg_grouped_sparse_gemm_swiglu(
        _ptr(act.codes), _ptr(act.scales), _ptr(act.x_scale), _ptr(w.packed), _ptr(w.w_scale),
        _ptr(offsets), w.E, w.N, w.K, act.R, max_rows_per_expert, _ptr(h_scale), _ptr(out.codes),
        _ptr(out.scales), _stream()))
    return out


def combine_workspace(E: int, N: int, K: int, T: int, k: int, device) -> torch.Tensor:
    """A zeroed workspace for grouped_sparse_gemm_combine (reusable call after call)."""
    return torch.zeros(max(workspace_size(OP_COMBINE, E, N, K, T, k), 16), dtype=torch.uint8, device=device)


def grouped_sparse_gemm_combine(act: QuantizedActivations, w: PackedSparseWeights, routing: "Routing",
                                gates: torch.Tensor, workspace: torch.Tensor, max_rows_per_expert: int = -1,
                                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Down-projection with the gate-weighted combine fused into the epilogue
    (gsg_grouped_sparse_gemm_combine): out [T, N] bf16, bit for bit grouped_sparse_gemm followed by
    unpermute_scale.  workspace from combine_workspace (zero before the first call, left zero)."""
    if stream is not None:
        return _on_stream(grouped_sparse_gemm_combine, stream, act, w, routing, gates, workspace, max_rows_per_expert,
                          out)
    assert act.sf_block == 32 and act.K == w.K and act.R == routing.T * routing.k
    _need_cuda(act.codes, act.scales, routing.offsets, routing.perm_src, gates, workspace)
    T, k = routing.T, routing.k
    if out is None:
        out = torch.empty(max(T, 1), w.N, dtype=torch.bfloat16, device=act.codes.device)
    _check("gsg_grouped_sparse_gemm_combine", lib().gsg_grouped_sparse_gemm_combine(
        _ptr(act.codes), _ptr(act.scales), _ptr(act.x_scale), _ptr(w.packed), _ptr(w.w_scale),
        _ptr(routing.offsets), w.E, w.N, w.K, T, k, max_rows_per_expert, _ptr(routing.perm_src), _ptr(gates),
        _ptr(workspace), workspace.numel(), _ptr(out), _stream()))
    return out


def grouped_dense_gemm(act: QuantizedActivations, w: PackedDenseWeights, offsets: torch.Tensor,
                       max_rows_per_expert: int = -1, out: Optional[torch.Tensor] = None,
                       out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """Dense-NVFP4 control on the same skeleton (gsg_grouped_dense_gemm)."""
    if stream is not None:
        return _on_stream(grouped_dense_gemm, stream, act, w, offsets, max_rows_per_expert, out, out_dtype)
    assert act.sf_block == 16 and act.K == w.K
    _need_cuda(act.codes, act.scales, offsets)
    if out is None:
        out = torch.empty(max(act.R, 1), w.N, dtype=out_dtype, device=act.codes.device)
    ydt = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    _check("gsg_grouped_dense_gemm", lib().gsg_grouped_dense_gemm(
        _ptr(act.codes), _ptr(act.scales), _ptr(act.x_scale), _ptr(w.packed), _ptr(w.w_scale),
        _ptr(offsets), w.E, w.N, w.K, act.R, max_rows_per_expert, _ptr(out), ydt, _stream()))
    return out


def grouped_dense_gemm_native(act: QuantizedActivations, w: PackedDenseWeights, offsets: torch.Tensor,
                              max_rows_per_expert: int = -1, out: Optional[torch.Tensor] = None,
                              out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """The dense-NVFP4 control with the token rows as MMA operand A (the activation-stationary
    orientation, gsg_grouped_dense_gemm_native); the same result as grouped_dense_gemm."""
    if stream is not None:
        return _on_stream(grouped_dense_gemm_native, stream, act, w, offsets, max_rows_per_expert, out, out_dtype)
    assert act.sf_block == 16 and act.K == w.K
    _need_cuda(act.codes, act.scales, offsets)
    if out is None:
        out = torch.empty(max(act.R, 1), w.N, dtype=out_dtype, device=act.codes.device)
    ydt = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    _check("gsg_grouped_dense_gemm_native", lib().gsg_grouped_dense_gemm_native(
        _ptr(act.codes), _ptr(act.scales), _ptr(act.x_scale), _ptr(w.packed), _ptr(w.w_scale),
        _ptr(offsets), w.E, w.N, w.K, act.R, max_rows_per_expert, _ptr(out), ydt, _stream()))
    return out


# ------------------------------------------------------------------ router, norm, microscaled experts
def _args(*ts: Optional[torch.Tensor]) -> int:
    """The checks of the tensors of one call (CUDA, contiguous, on the current device, where the kernels
    run) and the current stream, to launch on."""
    dev = torch.cuda.current_device()
    for t in ts:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            if not t.is_cuda:
                raise ValueError("grouped_sparse_gemm_b200 works on CUDA tensors only (no CPU fallback)")
            if t.get_device() != dev:
                raise ValueError(f"tensor on cuda:{t.get_device()}, but the current device is cuda:{dev}")
            raise ValueError("tensors must be contiguous")
    # (the raw handle: building a Stream object takes 3 us, as long as the rest of a small call)
    return torch._C._cuda_getCurrentRawStream(dev)


def _new(rows: int, cols: int, dtype, device) -> torch.Tensor:
    """A new [rows, cols] (with its strides given, a third cheaper to allocate than torch.empty)."""
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _too_long(what: str) -> ValueError:
    return ValueError(f"{what}: the library's sizes have 31 bits")


def _check_out(t: torch.Tensor, shape, dtype, what: str) -> torch.Tensor:
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{what}: {tuple(t.shape)} {t.dtype}, expected {tuple(shape)} {dtype}")
    return t


def _ptr_of(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _mx_activations(out: Optional[MxActivations], R: int, K: int, fmt: int, like: torch.Tensor) -> MxActivations:
    if fmt != MXFP4 and fmt != MXFP8:
        raise ValueError(f"fmt {fmt!r}: MXFP4 (4) or MXFP8 (8)")
    if out is None:
        dev = like.device
        return MxActivations(_new(R, K * fmt // 8, torch.uint8, dev),
                             torch.empty_strided((K // 128 * R * 16,), (1,), dtype=torch.uint8, device=dev), R, K, fmt)
    if (out.R, out.K, out.fmt) != (R, K, fmt):
        raise ValueError(f"out: R={out.R} K={out.K} fmt={out.fmt}, expected R={R} K={K} fmt={fmt}")
    _check_out(out.codes, (R, K * fmt // 8), torch.uint8, "codes")
    _check_out(out.scales, (K // 128 * R * 16,), torch.uint8, "scales")
    return out


def _mx_weights(out: Optional[PackedMxWeights], E: int, N: int, K: int, like: torch.Tensor) -> PackedMxWeights:
    n = int(lib().gsg_mx_packed_bytes(E, N, K))
    if out is not None and (out.E, out.N, out.K) != (E, N, K):
        raise ValueError(f"out: E={out.E} N={out.N} K={out.K}, expected E={E} N={N} K={K}")
    if out is None:
        return PackedMxWeights(like.new_empty((n,), dtype=torch.uint8), E, N, K)
    _check_out(out.packed, (n,), torch.uint8, "packed")
    return out


_SCORES = {"softmax": 0, "sigmoid": 1}


def moe_gate(logits: torch.Tensor, top_k: int, scoring: str = "softmax", bias: Optional[torch.Tensor] = None,
             n_group: int = 1, topk_group: int = 1, group_top: int = 1, renormalize: bool = True, scale: float = 1.0,
             out_ids: Optional[torch.Tensor] = None, out_gates: Optional[torch.Tensor] = None, stream=None):
    """Router logits bf16 or fp32 [T, E] -> (topk ids int32 [T, top_k], gates fp32 [T, top_k]), as the routing
    calls and unpermute_scale take them (gsg_moe_gate)."""
    if stream is not None:
        return _on_stream(moe_gate, stream, logits, top_k, scoring, bias, n_group, topk_group, group_top, renormalize,
                          scale, out_ids, out_gates)
    if logits.dim() != 2 or logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"logits: fp32 or bf16 [T, E] wanted, got {logits.dtype} {tuple(logits.shape)}")
    if scoring not in _SCORES:
        raise ValueError(f"scoring {scoring!r}: 'softmax' or 'sigmoid'")
    T, E = logits.shape
    if (T | top_k | n_group | topk_group | group_top) >> 31:   # (ctypes would keep the low 32 bits)
        raise _too_long(f"{T} tokens, top_k {top_k}, groups {n_group}, {topk_group}, {group_top}")
    if bias is not None and (bias.dtype != torch.float32 or bias.numel() != E):
        raise ValueError(f"bias: fp32 of {E} entries wanted")
    s = _args(logits, bias, out_ids, out_gates)
    if out_ids is None:
        out_ids = _new(T, top_k, torch.int32, logits.device)
    else:
        _check_out(out_ids, (T, top_k), torch.int32, "out_ids")
    if out_gates is None:
        out_gates = _new(T, top_k, torch.float32, logits.device)
    else:
        _check_out(out_gates, (T, top_k), torch.float32, "out_gates")
    _check("gsg_moe_gate", lib().gsg_moe_gate(
        logits.data_ptr(), OUT_F32 if logits.dtype == torch.float32 else OUT_BF16, _ptr_of(bias), T, E, top_k,
        _SCORES[scoring], n_group, topk_group, group_top, 1 if renormalize else 0, scale, out_ids.data_ptr(),
        out_gates.data_ptr(), s))
    return out_ids, out_gates


def add_rmsnorm_mx(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
                   fmt: Optional[int] = MXFP8, want_y: bool = True, out_act: Optional[MxActivations] = None,
                   out_y: Optional[torch.Tensor] = None, out_h: Optional[torch.Tensor] = None,
                   stream=None) -> NormOutput:
    """h = x + residual, y = rmsnorm(h) * weight; y in bf16 (want_y) and in MXFP8 or MXFP4 (fmt, None: not)
    from one pass (gsg_add_rmsnorm_mx).  x bf16 [T, K], residual bf16 or fp32 (out_h may be the residual
    itself), weight bf16 or fp32 [K]."""
    if stream is not None:
        return _on_stream(add_rmsnorm_mx, stream, x, weight, residual, eps, fmt, want_y, out_act, out_y, out_h)
    if x.dim() != 2 or x.dtype != torch.bfloat16:
        raise ValueError(f"x: bf16 [T, K] wanted, got {x.dtype} {tuple(x.shape)}")
    T, K = x.shape
    if T >> 31:
        raise _too_long(f"{T} tokens")
    if weight.numel() != K or weight.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"weight: fp32 or bf16 of {K} entries wanted")
    if out_h is not None and residual is None:
        raise ValueError("out_h: without a residual there is no h to write")
    if out_act is not None and fmt is None:
        raise ValueError("out_act: without a fmt there are no codes to write")
    s = _args(x, weight, residual, out_y, out_h, None if out_act is None else out_act.codes,
              None if out_act is None else out_act.scales)
    h = y = act = None
    if residual is not None:
        if residual.shape != x.shape or residual.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"residual: fp32 or bf16 {tuple(x.shape)} wanted")
        h = torch.empty_like(residual) if out_h is None else _check_out(out_h, x.shape, residual.dtype, "out_h")
    if want_y or out_y is not None:
        y = torch.empty_like(x) if out_y is None else _check_out(out_y, x.shape, torch.bfloat16, "out_y")
    if fmt is not None:
        act = _mx_activations(out_act, T, K, fmt, x)
    _check("gsg_add_rmsnorm_mx", lib().gsg_add_rmsnorm_mx(
        x.data_ptr(), _ptr_of(residual), OUT_F32 if h is not None and h.dtype == torch.float32 else OUT_BF16,
        weight.data_ptr(), OUT_F32 if weight.dtype == torch.float32 else OUT_BF16, T, K, eps, _ptr_of(h), _ptr_of(y),
        0 if fmt is None else fmt, None if act is None else act.codes.data_ptr(),
        None if act is None else act.scales.data_ptr(), s))
    return NormOutput(act, y, h)


def pack_mxfp4(W: torch.Tensor, out: Optional[PackedMxWeights] = None, stream=None) -> PackedMxWeights:
    """W fp32 or bf16 [E, N, K] -> MXFP4 packed weights (gsg_pack_mxfp4)."""
    if stream is not None:
        return _on_stream(pack_mxfp4, stream, W, out)
    if W.dim() != 3 or W.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"W: fp32 or bf16 [E, N, K] wanted, got {W.dtype} {tuple(W.shape)}")
    E, N, K = W.shape
    s = _args(W, None if out is None else out.packed)
    out = _mx_weights(out, E, N, K, W)
    _check("gsg_pack_mxfp4", lib().gsg_pack_mxfp4(
        W.data_ptr(), OUT_F32 if W.dtype == torch.float32 else OUT_BF16, E, N, K, out.packed.data_ptr(), s))
    return out


def pack_mxfp4_codes(codes: torch.Tensor, scales: torch.Tensor, out: Optional[PackedMxWeights] = None,
                     stream=None) -> PackedMxWeights:
    """MXFP4 weights as checkpoints store them (codes uint8 [E, N, K/2], low nibble = even k; scale bytes
    uint8 [E, N, K/32]) -> packed weights, values unchanged (gsg_pack_mxfp4_codes)."""
    if stream is not None:
        return _on_stream(pack_mxfp4_codes, stream, codes, scales, out)
    if codes.dim() != 3 or codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise ValueError("codes uint8 [E, N, K/2] and scales uint8 [E, N, K/32] wanted")
    E, N, K = codes.shape[0], codes.shape[1], codes.shape[2] * 2
    if tuple(scales.shape) != (E, N, K // 32):
        raise ValueError(f"scales: {tuple(scales.shape)}, expected {(E, N, K // 32)}")
    s = _args(codes, scales, None if out is None else out.packed)
    out = _mx_weights(out, E, N, K, codes)
    _check("gsg_pack_mxfp4_codes", lib().gsg_pack_mxfp4_codes(
        codes.data_ptr(), scales.data_ptr(), E, N, K, out.packed.data_ptr(), s))
    return out


def quantize_act_mx(X: torch.Tensor, fmt: int = MXFP8, inv_perm: Optional[torch.Tensor] = None, top_k: int = 1,
                    out: Optional[MxActivations] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> MxActivations:
    """X bf16 [T, K] -> MXFP4 or MXFP8 codes and scales in routed row order (gsg_quantize_act_mx)."""
    if stream is not None:
        return _on_stream(quantize_act_mx, stream, X, fmt, inv_perm, top_k, out, workspace)
    if X.dim() != 2 or X.dtype != torch.bfloat16:
        raise ValueError(f"X: bf16 [T, K] wanted, got {X.dtype} {tuple(X.shape)}")
    T, K = X.shape
    if (T | top_k) >> 31:
        raise _too_long(f"{T} tokens, top_k {top_k}")
    if inv_perm is not None and (inv_perm.dtype != torch.int32 or inv_perm.numel() < T * top_k):
        raise ValueError(f"inv_perm: int32 of {T * top_k} entries wanted")
    s = _args(X, inv_perm, workspace, None if out is None else out.codes, None if out is None else out.scales)
    out = _mx_activations(out, T * top_k, K, fmt, X)
    L = lib()
    if workspace is None and T * top_k * K >= 1 << 26:   # (below that the call needs none)
        workspace = _workspace(L.gsg_workspace_size(OP_QUANTIZE_MX, 0, 0, K, T, top_k), X.device)
    _check("gsg_quantize_act_mx", L.gsg_quantize_act_mx(
        X.data_ptr(), T, K, fmt, _ptr_of(inv_perm), top_k, out.codes.data_ptr(), out.scales.data_ptr(),
        _ptr_of(workspace), 0 if workspace is None else workspace.numel(), s))
    return out


def grouped_mx_gemm(act: MxActivations, w: PackedMxWeights, offsets: torch.Tensor, max_rows_per_expert: int = -1,
                    out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                    stream=None) -> torch.Tensor:
    """Y [R, N] = per-expert X_e . W_e^T on MXFP4 weights, MXFP4 or MXFP8 activations
    (gsg_grouped_mx_gemm).  One expert with offsets [0, R] is a plain linear layer."""
    if stream is not None:
        return _on_stream(grouped_mx_gemm, stream, act, w, offsets, max_rows_per_expert, out, out_dtype)
    if act.K != w.K:
        raise ValueError(f"activations have K = {act.K}, weights K = {w.K}")
    if offsets.dtype != torch.int32 or offsets.numel() != w.E + 1:
        raise ValueError(f"offsets: int32 of {w.E + 1} entries wanted")
    if act.codes.numel() != act.R * act.K * act.fmt // 8 or act.scales.numel() != act.K // 8 * act.R:
        raise ValueError(f"activations: {act.codes.numel()} codes' and {act.scales.numel()} scales' bytes are not R = "
                         f"{act.R}, K = {act.K}, fmt = {act.fmt}")
    if w.packed.numel() != w.E * w.N * w.K // 32 * 17:
        raise ValueError(f"weights: {w.packed.numel()} bytes are not E = {w.E}, N = {w.N}, K = {w.K}")
    if out is not None:
        out_dtype = out.dtype
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"out: bf16 or fp32, got {out_dtype}")
    s = _args(act.codes, act.scales, w.packed, offsets, out)
    if out is None:
        out = _new(act.R, w.N, out_dtype, act.codes.device)
    else:
        _check_out(out, (act.R, w.N), out_dtype, "out")
    _check("gsg_grouped_mx_gemm", lib().gsg_grouped_mx_gemm(
        act.codes.data_ptr(), act.scales.data_ptr(), act.fmt, w.packed.data_ptr(), offsets.data_ptr(), w.E, w.N, w.K,
        act.R, max_rows_per_expert, out.data_ptr(), OUT_F32 if out_dtype == torch.float32 else OUT_BF16, s))
    return out


def unpermute_scale(Y: torch.Tensor, inv_perm: torch.Tensor, gates: torch.Tensor, top_k: int,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t] = bf16(sum_j gates[t, j] * Y[inv_perm[t*k + j]]) (gsg_unpermute_scale)."""
    if stream is not None:
        return _on_stream(unpermute_scale, stream, Y, inv_perm, gates, top_k, out)
    _need_cuda(Y, inv_perm, gates)
    assert Y.dtype == torch.bfloat16 and gates.dtype == torch.float32
    T = gates.shape[0]
    N = Y.shape[1]
    if out is None:
        out = torch.empty(T, N, dtype=torch.bfloat16, device=Y.device)
    _check("gsg_unpermute_scale", lib().gsg_unpermute_scale(
        _ptr(Y), _ptr(inv_perm), _ptr(gates), T, top_k, N, _ptr(out), _stream()))
    return out


def get_device_status(stream=None) -> int:
    """Synchronise the stream; return and clear the device status word (0 = ok)."""
    return int(lib().gsg_get_device_status(_stream(stream)))
