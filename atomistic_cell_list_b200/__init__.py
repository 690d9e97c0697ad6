"""Python binding of libe2f.so: a GPU cell-list neighbour build, the
on-the-fly equivariant attention of E2Former-V2 with its gradients, and the
operators around it (norm, 8-bit checkpoints, species embedding), written
for B200 (sm_100a).

This module only marshals arguments: every step of the computation runs in
the library's CUDA kernels. PyTorch supplies device memory and the current
stream. Functions carry the C entry points' names (see include/e2f.h); the
library must be built (``python -m atomistic_cell_list_b200.build``) and a
CUDA device must be present, otherwise the calls raise.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libe2f.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "e2f.h")

E2F_OK = 0
STATUS_NAMES = {0: "E2F_OK", 1: "E2F_ERR_INVALID_ARG", 2: "E2F_ERR_UNSUPPORTED", 3: "E2F_ERR_CAPACITY",
                4: "E2F_ERR_ALIGNMENT", 5: "E2F_ERR_TIMEOUT", 6: "E2F_ERR_CUDA", 7: "E2F_ERR_NONFINITE",
                8: "E2F_ERR_STALE"}
E2F_F32, E2F_BF16, E2F_MXI8 = 0, 1, 2


class E2FError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)} ({status_string(code)})")


class e2f_attn_cfg(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int), ("C", ctypes.c_int), ("H", ctypes.c_int), ("n_rbf", ctypes.c_int),
                ("cutoff", ctypes.c_float), ("feat_dtype", ctypes.c_int), ("m_max", ctypes.c_int)]


class e2f_sixj_cfg(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int), ("Lf", ctypes.c_int), ("C", ctypes.c_int), ("H", ctypes.c_int),
                ("n_rbf", ctypes.c_int), ("cutoff", ctypes.c_float)]


class e2f_norm_cfg(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int), ("C", ctypes.c_int), ("eps", ctypes.c_float), ("x_dtype", ctypes.c_int),
                ("y_dtype", ctypes.c_int)]


class e2f_embed_cfg(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int), ("C", ctypes.c_int), ("n_tokens", ctypes.c_int), ("scale", ctypes.c_float),
                ("table_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int)]


_lib = None
_vp, _i64, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t

_SIGS = {
    "e2f_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "e2f_neighbors_workspace_size": (_sz, [_i64, _vp, ctypes.c_float, ctypes.c_int32]),
    "e2f_build_neighbors": (ctypes.c_int, [_vp, _i64, _vp, ctypes.c_float, _vp, ctypes.c_int32, _vp, _vp, _i64,
                                           ctypes.POINTER(_i64), _vp, _sz, _vp]),
    "e2f_build_neighbors_rows": (ctypes.c_int, [_vp, _i64, _i64, _vp, ctypes.c_float, _vp, ctypes.c_int32, _vp, _vp,
                                                _i64, ctypes.POINTER(_i64), _vp, _sz, _vp]),
    "e2f_build_neighbors_noalloc": (ctypes.c_int, [_vp, _i64, _vp, ctypes.c_float, _vp, ctypes.c_int32, _vp, _vp,
                                                   _i64, ctypes.POINTER(_i64), _vp]),
    "e2f_attention_workspace_size": (_sz, [_i64, _i64, ctypes.POINTER(e2f_attn_cfg)]),
    "e2f_onfly_attention": (ctypes.c_int, [ctypes.POINTER(e2f_attn_cfg), _vp, _i64, _vp, _vp, _vp, _i64, _vp, _vp,
                                           _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "e2f_attention_status": (ctypes.c_int, [_vp, _sz, _vp]),
    "e2f_attention_cells_workspace_size": (_sz, [_i64, _vp, ctypes.POINTER(e2f_attn_cfg)]),
    "e2f_onfly_attention_cells": (ctypes.c_int, [ctypes.POINTER(e2f_attn_cfg), _vp, _i64, _vp, _vp, _vp, _vp, _vp,
                                                 _vp, _vp, _vp, _sz, _vp]),
    "e2f_attention_cells_skin_workspace_size": (_sz, [_i64, _vp, ctypes.POINTER(e2f_attn_cfg), ctypes.c_float]),
    "e2f_onfly_attention_cells_skin": (ctypes.c_int, [ctypes.POINTER(e2f_attn_cfg), _vp, _i64, _vp, ctypes.c_float,
                                                      ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "e2f_attention_backward_workspace_size": (_sz, [_i64, _i64, ctypes.POINTER(e2f_attn_cfg)]),
    "e2f_onfly_attention_backward": (ctypes.c_int, [ctypes.POINTER(e2f_attn_cfg), _vp, _i64, _vp, _vp, _vp, _i64,
                                                    _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                    _vp, _sz, _vp]),
    "e2f_edge_wigner_blocks": (ctypes.c_int, [_vp, _i64, ctypes.c_int, _vp, _vp, _vp]),
    "e2f_launch_count": (_i64, []),
    "e2f_attention_uses_tensor_cores": (ctypes.c_int, [ctypes.POINTER(e2f_attn_cfg)]),
    "e2f_attention_set_kernel_events": (None, [_vp, _vp]),
    "e2f_attention_set_debug": (None, [ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "e2f_attention_debug_timers": (ctypes.c_int, [_vp, _sz, _i64, ctypes.POINTER(e2f_attn_cfg),
                                                  ctypes.POINTER(_i64), ctypes.c_int, _vp]),
    "e2f_sixj_n_paths": (ctypes.c_int, [ctypes.c_int, ctypes.c_int]),
    "e2f_sixj_workspace_size": (_sz, [_i64, ctypes.POINTER(e2f_sixj_cfg)]),
    "e2f_sixj_attention": (ctypes.c_int, [ctypes.POINTER(e2f_sixj_cfg), _vp, _i64, _vp, ctypes.c_int32, _vp, _vp,
                                          _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "e2f_layer_norm": (ctypes.c_int, [ctypes.POINTER(e2f_norm_cfg), _i64] + [_vp] * 12),
    "e2f_layer_norm_backward_workspace_size": (_sz, [_i64, ctypes.POINTER(e2f_norm_cfg)]),
    "e2f_layer_norm_backward": (ctypes.c_int, [ctypes.POINTER(e2f_norm_cfg), _i64] + [_vp] * 11 + [_sz, _vp]),
    "e2f_checkpoint_store": (ctypes.c_int, [_vp, ctypes.c_int, _i64, ctypes.c_int, _vp, _vp, _vp]),
    "e2f_checkpoint_load": (ctypes.c_int, [_vp, _vp, _i64, ctypes.c_int, ctypes.c_int, _vp, _vp]),
    "e2f_embedding": (ctypes.c_int, [ctypes.POINTER(e2f_embed_cfg), _vp, _i64, _vp, _vp, _vp, _sz, _vp]),
    "e2f_embedding_backward_workspace_size": (_sz, [_i64, ctypes.POINTER(e2f_embed_cfg)]),
    "e2f_embedding_backward": (ctypes.c_int, [ctypes.POINTER(e2f_embed_cfg), _vp, _i64, _vp, _vp, _vp, _sz, _vp]),
}


def lib() -> ctypes.CDLL:
    """Load libe2f.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m atomistic_cell_list_b200.build`")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(h, name)
            f.restype, f.argtypes = res, args
        _lib = h
    return _lib


def header_symbols(path: str = HEADER) -> list[str]:
    """Names of the functions include/e2f.h declares."""
    src = open(path).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(e2f_[a-z0-9_]+)\s*\(", src)))


def status_string(code: int) -> str:
    return lib().e2f_status_string(int(code)).decode()


def e2f_status_string(code: int) -> str:
    return status_string(code)


def _check(code: int, where: str):
    if code != E2F_OK:
        raise E2FError(code, where)


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _box_arg(box):
    if box is None:
        return None, None
    arr = (ctypes.c_float * 3)(*[float(v) for v in box])
    return ctypes.cast(arr, ctypes.c_void_p), arr


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def e2f_neighbors_workspace_size(n_atoms: int, box, cutoff: float, n_graphs: int = 1) -> int:
    b, keep = _box_arg(box)
    return int(lib().e2f_neighbors_workspace_size(int(n_atoms), b, float(cutoff), int(n_graphs)))


def e2f_build_neighbors(pos: torch.Tensor, box, cutoff: float, graph_ptr: torch.Tensor | None = None,
                        col_capacity: int | None = None, stream=None, rows: int | None = None):
    """CSR neighbour list (row_ptr int32 [N+1], col int32 [E]) by the GPU cell list; with
    rows = n, only the rows of atoms 0 .. n-1 (e2f_build_neighbors_rows)."""
    _need_cuda(pos, graph_ptr)
    assert pos.dtype == torch.float32 and pos.dim() == 2 and pos.shape[1] == 3
    n = pos.shape[0]
    n_graphs = 1 if graph_ptr is None else graph_ptr.numel() - 1
    dev = pos.device
    ws_bytes = e2f_neighbors_workspace_size(n, box, cutoff, n_graphs)
    ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
    row_ptr = torch.empty(n + 1, dtype=torch.int32, device=dev)
    cap = int(col_capacity) if col_capacity is not None else max(1024, 128 * n)
    b, keep = _box_arg(box)
    for _ in range(2):
        col = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
        npairs = ctypes.c_int64(0)
        if rows is None:
            code = lib().e2f_build_neighbors(_ptr(pos), n, b, float(cutoff), _ptr(graph_ptr), n_graphs,
                                             _ptr(row_ptr), _ptr(col), cap, ctypes.byref(npairs), _ptr(ws),
                                             ws_bytes, _stream(stream))
        else:
            code = lib().e2f_build_neighbors_rows(_ptr(pos), n, int(rows), b, float(cutoff), _ptr(graph_ptr),
                                                  n_graphs, _ptr(row_ptr), _ptr(col), cap, ctypes.byref(npairs),
                                                  _ptr(ws), ws_bytes, _stream(stream))
        if code == 3:  # capacity: grow to the exact size and retry
            cap = int(npairs.value)
            continue
        _check(code, "e2f_build_neighbors")
        return row_ptr, col[: npairs.value]
    raise E2FError(3, "e2f_build_neighbors")


NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024


def e2f_build_neighbors_noalloc(pos: torch.Tensor, box, cutoff: float, graph_ptr: torch.Tensor | None = None,
                                row_ptr: torch.Tensor | None = None, col: torch.Tensor | None = None,
                                stream=None):
    """CSR neighbour list built in the library's static scratch (no workspace).

    row_ptr / col may be passed in (int32, [N+1] and [capacity]); the call
    then writes them and returns (row_ptr, col[:E]). With col=None a buffer
    of 128 N entries is made here, grown once on E2F_ERR_CAPACITY.
    """
    _need_cuda(pos, graph_ptr, row_ptr, col)
    assert pos.dtype == torch.float32 and pos.dim() == 2 and pos.shape[1] == 3
    n = pos.shape[0]
    n_graphs = 1 if graph_ptr is None else graph_ptr.numel() - 1
    if row_ptr is None:
        row_ptr = torch.empty(n + 1, dtype=torch.int32, device=pos.device)
    given = col is not None
    if col is None:
        col = torch.empty(max(1024, 128 * n), dtype=torch.int32, device=pos.device)
    b, keep = _box_arg(box)
    for _ in range(2):
        npairs = ctypes.c_int64(0)
        code = lib().e2f_build_neighbors_noalloc(_ptr(pos), n, b, float(cutoff), _ptr(graph_ptr), n_graphs,
                                                 _ptr(row_ptr), _ptr(col), col.numel(), ctypes.byref(npairs),
                                                 _stream(stream))
        if code == 3 and not given:
            col = torch.empty(int(npairs.value), dtype=torch.int32, device=pos.device)
            continue
        _check(code, "e2f_build_neighbors_noalloc")
        return row_ptr, col[: npairs.value]
    raise E2FError(3, "e2f_build_neighbors_noalloc")


def make_cfg(L: int, C: int, H: int, n_rbf: int, cutoff: float, dtype: str, m_max: int = -1) -> e2f_attn_cfg:
    """m_max: SO(2) truncation order (-1 = full layer; W_so2 then holds blocks m <= m_max only)."""
    return e2f_attn_cfg(L, C, H, n_rbf, float(cutoff), E2F_BF16 if dtype == "bf16" else E2F_F32, int(m_max))


def e2f_attention_workspace_size(n_atoms: int, n_pairs: int, cfg: e2f_attn_cfg) -> int:
    return int(lib().e2f_attention_workspace_size(int(n_atoms), int(n_pairs), ctypes.byref(cfg)))


def e2f_onfly_attention(cfg: e2f_attn_cfg, pos, box, row_ptr, col, x, W_q, W_k, W_rad, W_so2,
                        out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        stream=None, check: bool = True) -> torch.Tensor:
    """out[N, (L+1)^2, C] fp32 = on-the-fly equivariant attention (see include/e2f.h)."""
    _need_cuda(pos, row_ptr, col, x, W_q, W_k, W_rad, W_so2, out, workspace)
    n = pos.shape[0]
    K = (cfg.L + 1) ** 2
    if out is None:
        out = torch.empty((n, K, cfg.C), dtype=torch.float32, device=pos.device)
    ws_bytes = e2f_attention_workspace_size(n, col.numel(), cfg)
    if workspace is None or workspace.numel() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=pos.device)
    b, keep = _box_arg(box)
    s = _stream(stream)
    code = lib().e2f_onfly_attention(ctypes.byref(cfg), _ptr(pos), n, b, _ptr(row_ptr), _ptr(col), col.numel(),
                                     _ptr(x), _ptr(W_q), _ptr(W_k), _ptr(W_rad), _ptr(W_so2), _ptr(out),
                                     _ptr(workspace), workspace.numel(), s)
    _check(code, "e2f_onfly_attention")
    if check:
        _check(lib().e2f_attention_status(_ptr(workspace), workspace.numel(), s), "e2f_onfly_attention (device)")
    return out


def e2f_attention_cells_workspace_size(n_atoms: int, box, cfg: e2f_attn_cfg) -> int:
    b, keep = _box_arg(box)
    return int(lib().e2f_attention_cells_workspace_size(int(n_atoms), b, ctypes.byref(cfg)))


def e2f_onfly_attention_cells(cfg: e2f_attn_cfg, pos, box, x, W_q, W_k, W_rad, W_so2,
                              out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                              stream=None, check: bool = True) -> torch.Tensor:
    """The attention with the cell-list traversal fused in: no neighbour list (see include/e2f.h)."""
    _need_cuda(pos, x, W_q, W_k, W_rad, W_so2, out, workspace)
    n = pos.shape[0]
    if out is None:
        out = torch.empty((n, (cfg.L + 1) ** 2, cfg.C), dtype=torch.float32, device=pos.device)
    ws_bytes = e2f_attention_cells_workspace_size(n, box, cfg)
    if ws_bytes == 0:
        raise E2FError(2, "e2f_onfly_attention_cells")
    if workspace is None or workspace.numel() < ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=pos.device)
    b, keep = _box_arg(box)
    s = _stream(stream)
    code = lib().e2f_onfly_attention_cells(ctypes.byref(cfg), _ptr(pos), n, b, _ptr(x), _ptr(W_q), _ptr(W_k),
                                           _ptr(W_rad), _ptr(W_so2), _ptr(out), _ptr(workspace),
                                           workspace.numel(), s)
    _check(code, "e2f_onfly_attention_cells")
    if check:
        _check(lib().e2f_attention_status(_ptr(workspace), workspace.numel(), s),
               "e2f_onfly_attention_cells (device)")
    return out


def e2f_attention_cells_skin_workspace_size(n_atoms: int, box, cfg: e2f_attn_cfg, skin: float) -> int:
    b, keep = _box_arg(box)
    return int(lib().e2f_attention_cells_skin_workspace_size(int(n_atoms), b, ctypes.byref(cfg), float(skin)))


def e2f_onfly_attention_cells_skin(cfg: e2f_attn_cfg, pos, box, skin: float, rebuild: bool, x, W_q, W_k, W_rad,
                                   W_so2, workspace: torch.Tensor, out: torch.Tensor | None = None, stream=None,
                                   check: bool = True) -> torch.Tensor:
    """The fused attention with Verlet-skin reuse of the cell lists held in
    `workspace` (see include/e2f.h). With check, a stale reuse raises
    E2FError(E2F_ERR_STALE); the caller then calls again with rebuild=True."""
    _need_cuda(pos, x, W_q, W_k, W_rad, W_so2, out, workspace)
    n = pos.shape[0]
    if out is None:
        out = torch.empty((n, (cfg.L + 1) ** 2, cfg.C), dtype=torch.float32, device=pos.device)
    ws_bytes = e2f_attention_cells_skin_workspace_size(n, box, cfg, skin)
    if ws_bytes == 0:
        raise E2FError(2, "e2f_onfly_attention_cells_skin")
    if workspace.numel() < ws_bytes:
        raise E2FError(1, "e2f_onfly_attention_cells_skin: workspace too small")
    b, keep = _box_arg(box)
    s = _stream(stream)
    code = lib().e2f_onfly_attention_cells_skin(ctypes.byref(cfg), _ptr(pos), n, b, float(skin), int(bool(rebuild)),
                                                _ptr(x), _ptr(W_q), _ptr(W_k), _ptr(W_rad), _ptr(W_so2), _ptr(out),
                                                _ptr(workspace), workspace.numel(), s)
    _check(code, "e2f_onfly_attention_cells_skin")
    if check:
        _check(lib().e2f_attention_status(_ptr(workspace), workspace.numel(), s),
               "e2f_onfly_attention_cells_skin (device)")
    return out


def e2f_attention_backward_workspace_size(n_atoms: int, n_pairs: int, cfg: e2f_attn_cfg) -> int:
    return int(lib().e2f_attention_backward_workspace_size(int(n_atoms), int(n_pairs), ctypes.byref(cfg)))


def e2f_onfly_attention_backward(cfg: e2f_attn_cfg, pos, box, row_ptr, col, x, W_q, W_k, W_rad, W_so2, grad_out,
                                 want_weights: bool = True, workspace: torch.Tensor | None = None,
                                 out: dict | None = None, stream=None, check: bool = True) -> dict:
    """Gradients of sum(grad_out * layer(...)) (see include/e2f.h): a dict with
    pos, x, W_rad and, when want_weights, W_q, W_k, W_so2 (all fp32)."""
    _need_cuda(pos, row_ptr, col, x, W_q, W_k, W_rad, W_so2, grad_out, workspace)
    n = pos.shape[0]
    dev = pos.device
    f32 = torch.float32
    g = dict(out) if out is not None else {}
    g.setdefault("pos", torch.empty((n, 3), dtype=f32, device=dev))
    g.setdefault("x", torch.empty(x.shape, dtype=f32, device=dev))
    g.setdefault("W_rad", torch.empty(W_rad.shape, dtype=f32, device=dev))
    if want_weights:
        g.setdefault("W_q", torch.empty(W_q.shape, dtype=f32, device=dev))
        g.setdefault("W_k", torch.empty(W_k.shape, dtype=f32, device=dev))
        g.setdefault("W_so2", torch.empty(W_so2.shape, dtype=f32, device=dev))
    ws_bytes = e2f_attention_backward_workspace_size(n, col.numel(), cfg)
    if workspace is None or workspace.numel() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
    b, keep = _box_arg(box)
    code = lib().e2f_onfly_attention_backward(
        ctypes.byref(cfg), _ptr(pos), n, b, _ptr(row_ptr), _ptr(col), col.numel(), _ptr(x), _ptr(W_q), _ptr(W_k),
        _ptr(W_rad), _ptr(W_so2), _ptr(grad_out), _ptr(g["pos"]), _ptr(g["x"]), _ptr(g.get("W_q")),
        _ptr(g.get("W_k")), _ptr(g["W_rad"]), _ptr(g.get("W_so2")), _ptr(workspace), workspace.numel(),
        _stream(stream))
    _check(code, "e2f_onfly_attention_backward")
    if check:
        _check(lib().e2f_attention_status(_ptr(workspace), workspace.numel(), _stream(stream)),
               "e2f_onfly_attention_backward (device)")
    return g


def e2f_attention_status(workspace: torch.Tensor, stream=None) -> int:
    return int(lib().e2f_attention_status(_ptr(workspace), workspace.numel(), _stream(stream)))


def e2f_edge_wigner_blocks(r: torch.Tensor, L: int, with_frames: bool = False, stream=None):
    _need_cuda(r)
    n = r.shape[0]
    S = sum((2 * l + 1) ** 2 for l in range(L + 1))
    out = torch.empty((n, S), dtype=torch.float32, device=r.device)
    fr = torch.empty((n, 3, 3), dtype=torch.float32, device=r.device) if with_frames else None
    _check(lib().e2f_edge_wigner_blocks(_ptr(r), n, int(L), _ptr(out), _ptr(fr), _stream(stream)),
           "e2f_edge_wigner_blocks")
    return (out, fr) if with_frames else out


def e2f_attention_uses_tensor_cores(cfg: e2f_attn_cfg) -> bool:
    return bool(lib().e2f_attention_uses_tensor_cores(ctypes.byref(cfg)))


DEBUG_SLOTS = 32


def e2f_attention_debug_timers(workspace: torch.Tensor, n_atoms: int, cfg: e2f_attn_cfg, n_ctas: int = 160,
                               stream=None):
    """Per-CTA role cycle counters of the last tensor-core call (timers on: e2f_attention_set_debug)."""
    import numpy as np
    n = DEBUG_SLOTS * n_ctas
    buf = (_i64 * n)()
    _check(lib().e2f_attention_debug_timers(_ptr(workspace), workspace.numel(), int(n_atoms), ctypes.byref(cfg), buf,
                                            n, _stream(stream)), "e2f_attention_debug_timers")
    return np.frombuffer(buf, dtype=np.int64).reshape(n_ctas, DEBUG_SLOTS).copy()


def e2f_attention_set_kernel_events(start=None, stop=None):
    """Record torch.cuda.Event pair around the next calls' main kernel (None, None: off)."""
    a = None if start is None else ctypes.c_void_p(start.cuda_event)
    b = None if stop is None else ctypes.c_void_p(stop.cuda_event)
    lib().e2f_attention_set_kernel_events(a, b)


def e2f_attention_set_debug(max_ctas: int = 0, timers: bool = False, drop_arrive: bool = False):
    """Debug and test controls of the tensor-core kernel (process-wide; all off restores the default)."""
    lib().e2f_attention_set_debug(int(max_ctas), int(bool(timers)), int(bool(drop_arrive)))


def e2f_launch_count() -> int:
    return int(lib().e2f_launch_count())


def make_sixj_cfg(L: int, Lf: int, C: int, H: int, n_rbf: int, cutoff: float) -> e2f_sixj_cfg:
    return e2f_sixj_cfg(int(L), int(Lf), int(C), int(H), int(n_rbf), float(cutoff))


def e2f_sixj_n_paths(L: int, Lf: int) -> int:
    return int(lib().e2f_sixj_n_paths(int(L), int(Lf)))


def e2f_sixj_workspace_size(n_atoms: int, cfg: e2f_sixj_cfg) -> int:
    return int(lib().e2f_sixj_workspace_size(int(n_atoms), ctypes.byref(cfg)))


def e2f_sixj_attention(cfg: e2f_sixj_cfg, pos, row_ptr, col, x, W_q, W_k, W_rad, w_path,
                       graph_ptr: torch.Tensor | None = None, out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[N, (L+1)^2, C] fp32 = the Wigner-6j node-level convolution layer (see include/e2f.h)."""
    _need_cuda(pos, row_ptr, col, x, W_q, W_k, W_rad, w_path, graph_ptr, out, workspace)
    n = pos.shape[0]
    if out is None:
        out = torch.empty((n, (cfg.L + 1) ** 2, cfg.C), dtype=torch.float32, device=pos.device)
    ws_bytes = e2f_sixj_workspace_size(n, cfg)
    if ws_bytes == 0:
        raise E2FError(2, "e2f_sixj_workspace_size")
    if workspace is None or workspace.numel() < ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=pos.device)
    n_graphs = 0 if graph_ptr is None else graph_ptr.numel() - 1
    code = lib().e2f_sixj_attention(ctypes.byref(cfg), _ptr(pos), n, _ptr(graph_ptr), n_graphs, _ptr(row_ptr),
                                    _ptr(col), col.numel(), _ptr(x), _ptr(W_q), _ptr(W_k), _ptr(W_rad),
                                    _ptr(w_path), _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(code, "e2f_sixj_attention")
    return out


_DTYPES = {"f32": E2F_F32, "bf16": E2F_BF16, "mxi8": E2F_MXI8}
_TORCH = {E2F_F32: torch.float32, E2F_BF16: torch.bfloat16, E2F_MXI8: torch.int8}


def _operand(name: str, t: torch.Tensor, dtype: torch.dtype, shape, device=None) -> int:
    """Address of a tensor that must be contiguous, of this dtype and shape, and on the current CUDA device."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}")
    if device is None:
        if not t.is_cuda or t.get_device() != torch.cuda.current_device():
            raise ValueError(f"{name} must be on the current CUDA device")
    elif t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return t.data_ptr()


def _empty(shape, dtype: torch.dtype, like: torch.Tensor, stream) -> torch.Tensor:
    """New memory for a call on `stream` (None: the current one), from that stream's pool."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)  # half the time of torch.empty
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _on(stream) -> int:
    """Handle of the stream of a call (None: the current one); it must belong to the current device."""
    device = torch.cuda.current_device()
    if stream is None:  # the handle alone: current_stream() builds an object, 3 us
        return torch._C._cuda_getCurrentRawStream(device)
    if stream.device_index != device:
        raise ValueError("stream must belong to the current CUDA device")
    return int(stream.cuda_stream)


def _result(out: dict, name: str, dtype: torch.dtype, shape, like: torch.Tensor, stream) -> int:
    """Address of out[name], allocated here when the caller did not give it."""
    t = out.get(name)
    if t is None:
        t = out[name] = _empty(shape, dtype, like, stream)
        return t.data_ptr()
    return _operand(f"out[{name!r}]", t, dtype, shape, like.device)


def _scratch(workspace, n_bytes: int, like: torch.Tensor, stream) -> torch.Tensor:
    """The caller's workspace, or a new one when it is absent or too small."""
    if workspace is None or workspace.numel() < n_bytes:
        return _empty((max(n_bytes, 256),), torch.uint8, like, stream)
    if workspace.dtype is not torch.uint8 or workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {like.device}")
    return workspace


def make_norm_cfg(L: int, C: int, x_dtype: str = "f32", y_dtype: str = "bf16", eps: float = 1e-5) -> e2f_norm_cfg:
    """x_dtype: "f32", "bf16" or "mxi8" (x is an 8-bit checkpoint); y_dtype: "f32" or "bf16"."""
    return e2f_norm_cfg(int(L), int(C), float(eps), _DTYPES[x_dtype], _DTYPES[y_dtype])


def e2f_layer_norm(cfg: e2f_norm_cfg, x, weight, bias=None, residual=None, x_scales=None, checkpoint: bool = False,
                   stats: bool = True, out: dict | None = None, stream=None) -> dict:
    """Layer norm of x[N, (L+1)^2, C] (see include/e2f.h): a dict with y, with stats mean and rstd, with
    residual sum, and with checkpoint codes and scales of what was normalised. Tensors given in `out`
    under these names are written in place of new ones; out["sum"] may be x."""
    L, C = cfg.L, cfg.C
    K, n = (L + 1) ** 2, x.shape[0] if x.dim() else 0
    shape, dev = (n, K, C), x.device
    xt = _TORCH[cfg.x_dtype]
    px = _operand("x", x, xt, shape)
    pw = _operand("weight", weight, torch.float32, (L + 1, C), dev)
    pb = None if bias is None else _operand("bias", bias, torch.float32, (C,), dev)
    pr = ps = psum = pm = pi = pc = pcs = None
    nb = (C + 31) // 32
    res = {} if out is None else dict(out)
    if cfg.x_dtype == E2F_MXI8:
        if x_scales is None:
            raise ValueError("an mxi8 input needs x_scales")
        ps = _operand("x_scales", x_scales, torch.uint8, (n, K, nb), dev)
    if residual is not None:
        pr = _operand("residual", residual, torch.float32, shape, dev)
        psum = _result(res, "sum", xt, shape, x, stream)
    py = _result(res, "y", _TORCH[cfg.y_dtype], shape, x, stream)
    if stats:
        pm = _result(res, "mean", torch.float32, (n,), x, stream)
        pi = _result(res, "rstd", torch.float32, (n, L + 1), x, stream)
    if checkpoint:
        pc = _result(res, "codes", torch.int8, shape, x, stream)
        pcs = _result(res, "scales", torch.uint8, (n, K, nb), x, stream)
    _check(lib().e2f_layer_norm(ctypes.byref(cfg), n, px, ps, pr, pw, pb, psum, py, pm, pi, pc, pcs, _on(stream)),
           "e2f_layer_norm")
    return res


def e2f_layer_norm_backward_workspace_size(n_atoms: int, cfg: e2f_norm_cfg) -> int:
    return int(lib().e2f_layer_norm_backward_workspace_size(int(n_atoms), ctypes.byref(cfg)))


def e2f_layer_norm_backward(cfg: e2f_norm_cfg, x, weight, mean, rstd, grad_y, grad_skip=None, x_scales=None,
                            want_weights: bool = True, workspace: torch.Tensor | None = None,
                            out: dict | None = None, stream=None) -> dict:
    """Gradients of e2f_layer_norm (see include/e2f.h): a dict with x and, when want_weights, weight and bias
    (all fp32). out["x"] may be grad_skip or grad_y."""
    L, C = cfg.L, cfg.C
    K, n = (L + 1) ** 2, x.shape[0] if x.dim() else 0
    shape, dev, f32 = (n, K, C), x.device, torch.float32
    px = _operand("x", x, _TORCH[cfg.x_dtype], shape)
    ps = None
    if cfg.x_dtype == E2F_MXI8:
        if x_scales is None:
            raise ValueError("an mxi8 input needs x_scales")
        ps = _operand("x_scales", x_scales, torch.uint8, (n, K, (C + 31) // 32), dev)
    pw = _operand("weight", weight, f32, (L + 1, C), dev)
    pm = _operand("mean", mean, f32, (n,), dev)
    pi = _operand("rstd", rstd, f32, (n, L + 1), dev)
    pg = _operand("grad_y", grad_y, f32, shape, dev)
    pk = None if grad_skip is None else _operand("grad_skip", grad_skip, f32, shape, dev)
    g = {} if out is None else dict(out)
    pgx = _result(g, "x", f32, shape, x, stream)
    pgw = pgb = None
    if want_weights:
        pgw = _result(g, "weight", f32, (L + 1, C), x, stream)
        pgb = _result(g, "bias", f32, (C,), x, stream)
    workspace = _scratch(workspace, e2f_layer_norm_backward_workspace_size(n, cfg), x, stream)
    _check(lib().e2f_layer_norm_backward(ctypes.byref(cfg), n, px, ps, pw, pm, pi, pg, pk, pgx, pgw, pgb,
                                         workspace.data_ptr(), workspace.numel(), _on(stream)),
           "e2f_layer_norm_backward")
    return g


def e2f_checkpoint_store(x: torch.Tensor, out: dict | None = None, stream=None):
    """(codes int8 [..., C], scales uint8 [..., ceil(C/32)]): the 8-bit checkpoint of x[..., C], fp32 or bf16
    (see include/e2f.h). Tensors given in `out` as codes and scales are written in place of new ones."""
    if x.dim() < 1 or x.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("x must be an fp32 or bf16 tensor of at least one dimension")
    px, C = _operand("x", x, x.dtype, x.shape), x.shape[-1]
    res = {} if out is None else dict(out)
    pc = _result(res, "codes", torch.int8, x.shape, x, stream)
    ps = _result(res, "scales", torch.uint8, x.shape[:-1] + ((C + 31) // 32,), x, stream)
    _check(lib().e2f_checkpoint_store(px, E2F_F32 if x.dtype is torch.float32 else E2F_BF16,
                                      x.numel() // max(C, 1), C, pc, ps, _on(stream)), "e2f_checkpoint_store")
    return res["codes"], res["scales"]


def e2f_checkpoint_load(codes: torch.Tensor, scales: torch.Tensor, dtype: str = "f32",
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values (fp32 or bf16) that a checkpoint stands for (see include/e2f.h)."""
    if codes.dim() < 1 or dtype not in ("f32", "bf16"):
        raise ValueError("codes must have at least one dimension and dtype be f32 or bf16")
    pc, C = _operand("codes", codes, torch.int8, codes.shape), codes.shape[-1]
    ps = _operand("scales", scales, torch.uint8, codes.shape[:-1] + ((C + 31) // 32,), codes.device)
    res = {} if out is None else {"out": out}
    po = _result(res, "out", _TORCH[_DTYPES[dtype]], codes.shape, codes, stream)
    _check(lib().e2f_checkpoint_load(pc, ps, codes.numel() // max(C, 1), C, _DTYPES[dtype], po, _on(stream)),
           "e2f_checkpoint_load")
    return res["out"]


def make_embed_cfg(n_tokens: int, C: int, L: int = 0, scale: float = 1.0, table_dtype: str = "f32",
                   out_dtype: str = "f32") -> e2f_embed_cfg:
    return e2f_embed_cfg(int(L), int(C), int(n_tokens), float(scale), _DTYPES[table_dtype], _DTYPES[out_dtype])


def e2f_embedding(cfg: e2f_embed_cfg, tokens, table, out: torch.Tensor | None = None, stream=None,
                  check: bool = True) -> torch.Tensor:
    """out[N, (L+1)^2, C]: scaled table rows of int32 tokens as degree-0 features (see include/e2f.h). Negative
    tokens are padding. With check, a token beyond the table raises E2FError; this waits for the stream, so a
    call that is captured into a graph passes check=False."""
    n, dev = tokens.shape[0] if tokens.dim() else 0, tokens.device
    pt = _operand("tokens", tokens, torch.int32, (n,))
    pw = _operand("table", table, _TORCH[cfg.table_dtype], (cfg.n_tokens, cfg.C), dev)
    res = {} if out is None else {"out": out}
    po = _result(res, "out", _TORCH[cfg.out_dtype], (n, (cfg.L + 1) ** 2, cfg.C), tokens, stream)
    ws = _empty((256,), torch.uint8, tokens, stream) if check else None
    s = _on(stream)
    _check(lib().e2f_embedding(ctypes.byref(cfg), pt, n, pw, po, _ptr(ws), 256 if check else 0, s), "e2f_embedding")
    if check:
        _check(lib().e2f_attention_status(_ptr(ws), 256, s), "e2f_embedding (device)")
    return res["out"]


def e2f_embedding_backward_workspace_size(n_atoms: int, cfg: e2f_embed_cfg) -> int:
    return int(lib().e2f_embedding_backward_workspace_size(int(n_atoms), ctypes.byref(cfg)))


def e2f_embedding_backward(cfg: e2f_embed_cfg, tokens, grad_out, workspace: torch.Tensor | None = None,
                           out: torch.Tensor | None = None, stream=None, check: bool = True) -> torch.Tensor:
    """grad_table[n_tokens, C] fp32 of e2f_embedding from grad_out[N, (L+1)^2, C] fp32 (see include/e2f.h)."""
    n, dev = tokens.shape[0] if tokens.dim() else 0, tokens.device
    pt = _operand("tokens", tokens, torch.int32, (n,))
    pg = _operand("grad_out", grad_out, torch.float32, (n, (cfg.L + 1) ** 2, cfg.C), dev)
    res = {} if out is None else {"out": out}
    po = _result(res, "out", torch.float32, (cfg.n_tokens, cfg.C), tokens, stream)
    workspace = _scratch(workspace, e2f_embedding_backward_workspace_size(n, cfg), tokens, stream)
    s = _on(stream)
    _check(lib().e2f_embedding_backward(ctypes.byref(cfg), pt, n, pg, po, _ptr(workspace), workspace.numel(), s),
           "e2f_embedding_backward")
    if check:
        _check(lib().e2f_attention_status(_ptr(workspace), workspace.numel(), s), "e2f_embedding_backward (device)")
    return res["out"]


# short aliases
build_neighbors = e2f_build_neighbors
onfly_attention = e2f_onfly_attention
edge_wigner_blocks = e2f_edge_wigner_blocks
