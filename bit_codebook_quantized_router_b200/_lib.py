"""ctypes binding of libmoe_q4 (argument marshalling only: every step of the
layer runs in the library's CUDA kernels).  Torch provides device memory and
streams; tensors are passed as raw pointers."""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# MOE_Q4_LIB=debug selects the bounds-checking build (libmoe_q4_debug.so)
LIB_PATH = os.path.join(_HERE, "libmoe_q4_debug.so" if os.environ.get("MOE_Q4_LIB") == "debug" else "libmoe_q4.so")

OK, EINVAL, ECUDA, EWORKSPACE, ETIMEOUT, EDEVICE, ENOTSUP, EBOUNDS = range(8)
MAX_TABLES, MAX_EXPERTS, MAX_TOPK = 16, 512, 16


class MoeQ4Error(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: moe_q4 status {status} ({status_string(status)})")


class _SharedStruct(ctypes.Structure):
    _fields_ = [("I", ctypes.c_int), ("gate_up", ctypes.c_void_p), ("down", ctypes.c_void_p)]


class _LayerStruct(ctypes.Structure):
    _fields_ = [
        ("E", ctypes.c_int), ("H", ctypes.c_int), ("I", ctypes.c_int),
        ("gate_w", ctypes.c_void_p), ("gate_s", ctypes.c_void_p),
        ("up_w", ctypes.c_void_p), ("up_s", ctypes.c_void_p),
        ("down_w", ctypes.c_void_p), ("down_s", ctypes.c_void_p),
        ("tables", ctypes.c_void_p), ("n_tables", ctypes.c_int), ("table_id", ctypes.c_void_p),
    ]


class _MlpStruct(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int), ("I", ctypes.c_int), ("gate_up", ctypes.c_void_p),
                ("ld_gate_up", ctypes.c_longlong), ("gate_up_scale", ctypes.c_void_p), ("down", ctypes.c_void_p),
                ("ld_down", ctypes.c_longlong), ("down_scale", ctypes.c_void_p)]


_lib = None


def lib():
    """The loaded library.  Raises if it was not built: there is no fallback."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m bit_codebook_quantized_router_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, ci, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.moe_q4_abi_version.restype = ci
        L.moe_q4_status_string.argtypes = [ci]
        L.moe_q4_status_string.restype = ctypes.c_char_p
        L.moe_q4_pack.argtypes = [vp, ci, ci, ci, vp, ci, vp, vp, vp, vp, vp]
        L.moe_q4_dequant.argtypes = [vp, vp, vp, ci, vp, ci, ci, ci, vp, vp]
        L.moe_q4_forward_workspace.argtypes = [ctypes.POINTER(_LayerStruct), ci, ci]
        L.moe_q4_forward_workspace.restype = sz
        L.moe_q4_forward_host_workspace.argtypes = [ctypes.POINTER(_LayerStruct), ci, ci]
        L.moe_q4_forward_host_workspace.restype = sz
        L.moe_q4_forward.argtypes = [ctypes.POINTER(_LayerStruct), vp, vp, ci, ci, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_q4_forward_host.argtypes = [ctypes.POINTER(_LayerStruct), vp, vp, ci, ci, vp, vp, sz, vp]
        L.moe_q4_forward_status.argtypes = [vp, vp]
        L.moe_q4_read_status.argtypes = [vp, vp]
        L.moe_q4_route_workspace.argtypes = [ci, ci, ci]
        L.moe_q4_route_workspace.restype = sz
        L.moe_q4_route.argtypes = [vp, ci, ci, ci, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_q4_forward_stages.argtypes = [ctypes.POINTER(_LayerStruct), vp, vp, ci, ci, vp, vp, sz, vp,
                                            ctypes.POINTER(ctypes.c_void_p), ci]
        L.moe_q4_router_workspace.argtypes = [ci, ci, ci]
        L.moe_q4_router_workspace.restype = sz
        L.moe_q4_router.argtypes = [vp, vp, ci, ci, ci, vp, vp, sz, vp]
        L.moe_q4_forward_ex_workspace.argtypes = [ctypes.POINTER(_LayerStruct), ctypes.POINTER(_SharedStruct), ci, ci]
        L.moe_q4_forward_ex_workspace.restype = sz
        L.moe_q4_forward_ex.argtypes = [ctypes.POINTER(_LayerStruct), ctypes.POINTER(_SharedStruct), vp, vp, ci, ci,
                                        vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_q4_forward_ex.restype = ci
        L.moe_q4_forward_gated_workspace.argtypes = [ctypes.POINTER(_LayerStruct), ctypes.POINTER(_SharedStruct),
                                                     ci, ci]
        L.moe_q4_forward_gated_workspace.restype = sz
        L.moe_q4_forward_gated.argtypes = [ctypes.POINTER(_LayerStruct), ctypes.POINTER(_SharedStruct), vp, vp, ci,
                                           ci, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_q4_forward_gated.restype = ci
        L.moe_q4_combine.argtypes = [vp, vp, vp, ci, ci, ci, vp, vp, vp]
        L.moe_q4_combine.restype = ci
        L.moe_q4_selftest_wait.argtypes = [vp, ctypes.c_uint, vp]
        L.moe_q4_selftest_wait.restype = ci
        L.moe_q4_lloyd_workspace.argtypes = [vp]
        L.moe_q4_lloyd_workspace.restype = sz
        L.moe_q4_lloyd_hist.argtypes = [vp, ctypes.c_longlong, vp, ci, vp, sz, vp]
        L.moe_q4_lloyd_solve.argtypes = [vp, ci, ctypes.c_double, vp, vp, vp, sz, vp]
        L.moe_q4_forward_host_async.argtypes = L.moe_q4_forward_host.argtypes
        ll, mlp = ctypes.c_longlong, ctypes.POINTER(_MlpStruct)
        L.moe_q4_quant_rows.argtypes = [vp, ci, ll, ci, ci, vp, ll, vp, vp]
        L.moe_q4_add_norm.argtypes = [vp, ci, ll, vp, ci, ll, vp, ll, vp, ci, ctypes.c_float, ci, ci, vp, ll, vp, ll,
                                      vp, vp]
        L.moe_q4_linear_i8.argtypes = [vp, ll, vp, vp, ll, vp, vp, ci, ci, ci, vp, ci, ll, vp, vp]
        L.moe_q4_i8_status.argtypes = [vp]
        L.moe_q4_mlp_i8_workspace.argtypes = [mlp, ci]
        L.moe_q4_mlp_i8.argtypes = [mlp, vp, ll, vp, ci, vp, ci, ll, vp, vp, sz, vp]
        layer = ctypes.POINTER(_LayerStruct)
        L.moe_q4_forward_ex_i8_workspace.argtypes = [layer, mlp, ci, ci]
        L.moe_q4_forward_ex_i8.argtypes = [layer, mlp, vp, vp, ll, vp, vp, ci, ci, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_q4_forward_gated_i8_workspace.argtypes = [layer, mlp, ci, ci]
        L.moe_q4_forward_gated_i8.argtypes = [layer, mlp, vp, vp, vp, ll, vp, ci, ci, vp, vp, vp, vp, vp, vp, vp, sz,
                                              vp]
        for f in (L.moe_q4_mlp_i8_workspace, L.moe_q4_forward_ex_i8_workspace, L.moe_q4_forward_gated_i8_workspace):
            f.restype = sz
        for f in (L.moe_q4_quant_rows, L.moe_q4_add_norm, L.moe_q4_linear_i8, L.moe_q4_mlp_i8, L.moe_q4_i8_status,
                  L.moe_q4_forward_ex_i8, L.moe_q4_forward_gated_i8):
            f.restype = ci
        for f in (L.moe_q4_pack, L.moe_q4_dequant, L.moe_q4_forward, L.moe_q4_forward_host,
                  L.moe_q4_forward_host_async,
                  L.moe_q4_forward_status, L.moe_q4_read_status, L.moe_q4_route,
                  L.moe_q4_forward_stages, L.moe_q4_router, L.moe_q4_lloyd_hist, L.moe_q4_lloyd_solve):
            f.restype = ci
        if L.moe_q4_abi_version() != 1:
            raise ImportError("libmoe_q4 ABI version mismatch")
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_q4_status_string(int(status)).decode()


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _hold(stream, *tensors):
    """Memory this binding allocated for a call (contiguous copies, internal
    workspaces) is read by work enqueued on `stream`, which may run after the
    call returns: when that is not torch's current stream, tell the caching
    allocator, so the blocks are not handed out again before the work ran.
    (On the current stream, stream order already keeps reuse safe.)"""
    if stream is None:
        return
    for t in tensors:
        if t is not None and t.is_cuda:
            t.record_stream(stream)


def _check(rc, what):
    if rc != OK:
        raise MoeQ4Error(rc, what)


def _host_tables(tables, table_id, E):
    t = np.ascontiguousarray(np.asarray(tables, np.float32).reshape(-1, 8))
    tid = np.ascontiguousarray(np.asarray(table_id, np.uint8).reshape(-1))
    if tid.shape[0] != E:
        raise ValueError("table_id must hold one entry per expert")
    return t, tid


class Layer:
    """A packed layer resident on the device.

    gate_w/up_w: uint8 [E, I, H/2], gate_s/up_s: uint8 [E, I, H/32],
    down_w: uint8 [E, H, I/2], down_s: uint8 [E, H, I/32] (CUDA tensors);
    tables: fp32 [n, 8] magnitudes; table_id: uint8 [E] (host arrays)."""

    def __init__(self, gate_w, gate_s, up_w, up_s, down_w, down_s, tables, table_id):
        self.E, self.I, hh = gate_w.shape
        self.H = hh * 2
        self.gate_w, self.gate_s, self.up_w, self.up_s = gate_w, gate_s, up_w, up_s
        self.down_w, self.down_s = down_w, down_s
        self.tables, self.table_id = _host_tables(tables, table_id, self.E)
        for t in (gate_w, gate_s, up_w, up_s, down_w, down_s):
            if not (t.is_cuda and t.dtype == torch.uint8 and t.is_contiguous()):
                raise ValueError("packed tensors must be contiguous uint8 CUDA tensors")

    def struct(self) -> _LayerStruct:
        return _LayerStruct(self.E, self.H, self.I,
                            self.gate_w.data_ptr(), self.gate_s.data_ptr(),
                            self.up_w.data_ptr(), self.up_s.data_ptr(),
                            self.down_w.data_ptr(), self.down_s.data_ptr(),
                            self.tables.ctypes.data, self.tables.shape[0], self.table_id.ctypes.data)


def pack(w: torch.Tensor, tables, table_id, status: torch.Tensor | None = None, stream=None):
    """bf16 [E, N, K] CUDA tensor -> (codes uint8 [E, N, K/2], scales uint8 [E, N, K/32])."""
    if w.dim() != 3 or w.dtype != torch.bfloat16 or not w.is_cuda:
        raise ValueError("w must be a bf16 CUDA tensor [E, N, K]")
    w = w.contiguous()
    E, N, K = w.shape
    t, tid = _host_tables(tables, table_id, E)
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((E, N, K // 32), dtype=torch.uint8, device=w.device)
    own = status is None
    if own:
        status = torch.zeros(1, dtype=torch.int32, device=w.device)
    _check(lib().moe_q4_pack(_ptr(w), E, N, K, t.ctypes.data, t.shape[0], tid.ctypes.data,
                             _ptr(codes), _ptr(scales), _ptr(status), _stream(stream)), "moe_q4_pack")
    _hold(stream, w, status)
    if own:
        st = lib().moe_q4_read_status(_ptr(status), _stream(stream))
        _check(st, "moe_q4_pack (device)")
    return codes, scales


def dequant(codes: torch.Tensor, scales: torch.Tensor, tables, table_id, stream=None,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """uint8 codes [E, N, K/2] + scales [E, N, K/32] -> bf16 [E, N, K] (into `out` if given)."""
    E, N, Kh = codes.shape
    K = Kh * 2
    t, tid = _host_tables(tables, table_id, E)
    if out is None:
        out = torch.empty((E, N, K), dtype=torch.bfloat16, device=codes.device)
    elif out.shape != (E, N, K) or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 tensor [E, N, K]")
    codes, scales = codes.contiguous(), scales.contiguous()
    _check(lib().moe_q4_dequant(_ptr(codes), _ptr(scales), t.ctypes.data,
                                t.shape[0], tid.ctypes.data, E, N, K, _ptr(out), _stream(stream)),
           "moe_q4_dequant")
    _hold(stream, codes, scales)
    return out


def forward_workspace(layer: Layer, T: int, k: int) -> int:
    return int(lib().moe_q4_forward_workspace(ctypes.byref(layer.struct()), T, k))


def forward_host_workspace(layer: Layer, T: int, k: int) -> int:
    return int(lib().moe_q4_forward_host_workspace(ctypes.byref(layer.struct()), T, k))


def alloc_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    # torch's caching allocator returns 512-byte aligned blocks
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def forward(layer: Layer, x: torch.Tensor, logits: torch.Tensor, k: int, out=None, ws=None,
            topk_ids=None, topk_w=None, counts=None, out_f32=None, stream=None) -> torch.Tensor:
    """One MoE layer: x bf16 [T, H], logits fp32 [T, E] -> out bf16 [T, H]
    (and, when given, the fp32 combine result in out_f32 [T, H])."""
    T = x.shape[0]
    if out is None:
        out = torch.empty((T, layer.H), dtype=torch.bfloat16, device=x.device)
    own_ws = ws is None
    if own_ws:
        ws = alloc_workspace(forward_workspace(layer, T, k), x.device)
    st = layer.struct()
    _check(lib().moe_q4_forward(ctypes.byref(st), _ptr(x), _ptr(logits), T, k, _ptr(out),
                                _ptr(out_f32), _ptr(topk_ids), _ptr(topk_w), _ptr(counts), _ptr(ws), ws.numel(),
                                _stream(stream)), "moe_q4_forward")
    if own_ws:
        _hold(stream, ws)
    return out


class Shared:
    """A BF16 shared expert: gate_up bf16 [2I, H] (gate rows first), down
    bf16 [H, I] (CUDA tensors)."""

    def __init__(self, gate_up: torch.Tensor, down: torch.Tensor):
        if gate_up.dtype != torch.bfloat16 or down.dtype != torch.bfloat16 or not (gate_up.is_cuda and down.is_cuda):
            raise ValueError("shared expert weights must be bf16 CUDA tensors")
        if gate_up.dim() != 2 or down.dim() != 2 or gate_up.shape[0] % 2 or down.shape != (gate_up.shape[1],
                                                                                          gate_up.shape[0] // 2):
            raise ValueError("shared expert shapes: gate_up [2I, H], down [H, I]")
        self.gate_up, self.down = gate_up.contiguous(), down.contiguous()
        self.I = gate_up.shape[0] // 2

    def struct(self) -> _SharedStruct:
        return _SharedStruct(self.I, self.gate_up.data_ptr(), self.down.data_ptr())


def forward_ex_workspace(layer: Layer, shared, T: int, k: int) -> int:
    if isinstance(shared, MlpI8):
        return int(lib().moe_q4_forward_ex_i8_workspace(ctypes.byref(layer.struct()), shared.ref, T, k))
    sh = ctypes.byref(shared.struct()) if shared is not None else None
    return int(lib().moe_q4_forward_ex_workspace(ctypes.byref(layer.struct()), sh, T, k))


def forward_ex(layer: Layer, shared, x: torch.Tensor, logits: torch.Tensor, k: int, out=None, ws=None,
               topk_ids=None, topk_w=None, counts=None, out_f32=None, stream=None, xq=None,
               x_scale=None) -> torch.Tensor:
    """One MoE layer with a shared expert: a Shared (bf16), an MlpI8 (int8;
    xq and x_scale are x's int8 rows where the caller has them, as add_norm
    gives them, else the call makes them) or None."""
    T = x.shape[0]
    ldq = _shared_rows(layer, shared, x, xq, x_scale)
    if out is None:
        out = torch.empty((T, layer.H), dtype=torch.bfloat16, device=x.device)
    own_ws = ws is None
    if own_ws:
        ws = alloc_workspace(forward_ex_workspace(layer, shared, T, k), x.device)
    st = layer.struct()
    if isinstance(shared, MlpI8):
        _check(lib().moe_q4_forward_ex_i8(ctypes.byref(st), shared.ref, _ptr(x), _ptr(xq), ldq, _ptr(x_scale),
                                          _ptr(logits), T, k, _ptr(out), _ptr(out_f32), _ptr(topk_ids), _ptr(topk_w),
                                          _ptr(counts), _ptr(ws), ws.numel(), _stream(stream)),
               "moe_q4_forward_ex_i8")
        if own_ws:
            _hold(stream, ws)
        return out
    ss = shared.struct() if shared is not None else None
    _check(lib().moe_q4_forward_ex(ctypes.byref(st), ctypes.byref(ss) if ss is not None else None, _ptr(x),
                                   _ptr(logits), T, k, _ptr(out), _ptr(out_f32), _ptr(topk_ids), _ptr(topk_w),
                                   _ptr(counts), _ptr(ws), ws.numel(), _stream(stream)), "moe_q4_forward_ex")
    if own_ws:
        _hold(stream, ws)
    return out


def forward_gated_workspace(layer: Layer, shared, T: int, k: int) -> int:
    if isinstance(shared, MlpI8):
        return int(lib().moe_q4_forward_gated_i8_workspace(ctypes.byref(layer.struct()), shared.ref, T, k))
    sh = ctypes.byref(shared.struct()) if shared is not None else None
    return int(lib().moe_q4_forward_gated_workspace(ctypes.byref(layer.struct()), sh, T, k))


def forward_gated(layer: Layer, shared, router_w: torch.Tensor, x: torch.Tensor, k: int, out=None, ws=None,
                  logits=None, topk_ids=None, topk_w=None, counts=None, out_f32=None, stream=None, xq=None,
                  x_scale=None) -> torch.Tensor:
    """One MoE layer from the hidden states: the bf16 router gate router_w
    [E, H] computes the logits (into `logits` [T, E] fp32 when given), then
    the layer as forward_ex (shared, xq and x_scale as there)."""
    if router_w.dtype != torch.bfloat16 or tuple(router_w.shape) != (layer.E, layer.H):
        raise ValueError(f"router_w must be bf16 [{layer.E}, {layer.H}]")
    T = x.shape[0]
    ldq = _shared_rows(layer, shared, x, xq, x_scale)
    if out is None:
        out = torch.empty((T, layer.H), dtype=torch.bfloat16, device=x.device)
    own_ws = ws is None
    if own_ws:
        ws = alloc_workspace(forward_gated_workspace(layer, shared, T, k), x.device)
    st = layer.struct()
    if isinstance(shared, MlpI8):
        _check(lib().moe_q4_forward_gated_i8(ctypes.byref(st), shared.ref, _ptr(router_w), _ptr(x), _ptr(xq), ldq,
                                             _ptr(x_scale), T, k, _ptr(out), _ptr(out_f32), _ptr(logits),
                                             _ptr(topk_ids), _ptr(topk_w), _ptr(counts), _ptr(ws), ws.numel(),
                                             _stream(stream)), "moe_q4_forward_gated_i8")
        if own_ws:
            _hold(stream, ws)
        return out
    ss = shared.struct() if shared is not None else None
    _check(lib().moe_q4_forward_gated(ctypes.byref(st), ctypes.byref(ss) if ss is not None else None,
                                      _ptr(router_w), _ptr(x), T, k, _ptr(out), _ptr(out_f32), _ptr(logits),
                                      _ptr(topk_ids), _ptr(topk_w), _ptr(counts), _ptr(ws), ws.numel(),
                                      _stream(stream)), "moe_q4_forward_gated")
    if own_ws:
        _hold(stream, ws)
    return out


def forward_status(ws: torch.Tensor, stream=None) -> int:
    return int(lib().moe_q4_forward_status(_ptr(ws), _stream(stream)))


def forward_host(layer: Layer, x_host: torch.Tensor, logits_host: torch.Tensor, k: int,
                 out_host: torch.Tensor, ws: torch.Tensor, stream=None) -> int:
    """Host tensors in and out (pinned memory for asynchronous copies)."""
    T = x_host.shape[0]
    st = layer.struct()
    return int(lib().moe_q4_forward_host(ctypes.byref(st), _ptr(x_host), _ptr(logits_host), T, k,
                                         _ptr(out_host), _ptr(ws), ws.numel(), _stream(stream)))


def forward_host_async(layer: Layer, x_host: torch.Tensor, logits_host: torch.Tensor, k: int,
                       out_host: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """forward_host without the wait (pinned host tensors; read the device
    status later with forward_status on the same stream)."""
    T = x_host.shape[0]
    st = layer.struct()
    _check(lib().moe_q4_forward_host_async(ctypes.byref(st), _ptr(x_host), _ptr(logits_host), T, k,
                                           _ptr(out_host), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_q4_forward_host_async")


def route(logits: torch.Tensor, k: int, stream=None):
    """Routing + grouping alone: (ids, w, counts, offsets, row_token, inv)."""
    T, E = logits.shape
    dev = logits.device
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), dtype=torch.float32, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    row_token = torch.empty(T * k, dtype=torch.int32, device=dev)
    inv = torch.empty((T, k), dtype=torch.int32, device=dev)
    need = int(lib().moe_q4_route_workspace(E, T, k))
    if need == 0:
        raise MoeQ4Error(EINVAL, "moe_q4_route_workspace")
    ws = alloc_workspace(need, dev)
    logits = logits.contiguous()
    _check(lib().moe_q4_route(_ptr(logits), T, E, k, _ptr(ids), _ptr(w), _ptr(counts),
                              _ptr(offsets), _ptr(row_token), _ptr(inv), _ptr(ws), ws.numel(),
                              _stream(stream)), "moe_q4_route")
    _hold(stream, logits, ws)
    st = forward_status(ws, stream)
    return ids, w, counts, offsets, row_token, inv, st


def router_workspace(T: int, H: int, E: int) -> int:
    return int(lib().moe_q4_router_workspace(T, H, E))


def router(x: torch.Tensor, w: torch.Tensor, out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
           stream=None) -> torch.Tensor:
    """Router logits: bf16 hidden states x [T, H] and bf16 gate w [E, H] ->
    fp32 logits [T, E] (into `out` if given)."""
    if x.dtype != torch.bfloat16 or w.dtype != torch.bfloat16 or x.dim() != 2 or w.dim() != 2:
        raise ValueError("x [T, H] and w [E, H] must be bf16 matrices")
    T, H = x.shape
    E = w.shape[0]
    if out is None:
        out = torch.empty((T, E), dtype=torch.float32, device=x.device)
    need = router_workspace(T, H, E)
    own_ws = ws is None and need > 0
    if own_ws:
        ws = alloc_workspace(need, x.device)
    x, w = x.contiguous(), w.contiguous()
    _check(lib().moe_q4_router(_ptr(x), _ptr(w), T, H, E, _ptr(out), _ptr(ws),
                               0 if ws is None else ws.numel(), _stream(stream)), "moe_q4_router")
    _hold(stream, x, w, ws if own_ws else None)
    return out


def forward_stages(layer: Layer, x, logits, k: int, out, ws, events, stream=None) -> None:
    """moe_q4_forward with torch.cuda.Event records at the 8 kernel boundaries
    (the events must have been recorded once: torch creates them lazily)."""
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    st = layer.struct()
    _check(lib().moe_q4_forward_stages(ctypes.byref(st), _ptr(x), _ptr(logits), x.shape[0], k, _ptr(out),
                                       _ptr(ws), ws.numel(), _stream(stream), arr, len(events)),
           "moe_q4_forward_stages")


def lloyd_fit(weights, grid0, max_iter: int = 300, tol: float = 1e-12, stream=None):
    """Weighted Lloyd-Max fit of an 8-level grid over the pooled ratios of one
    or more bf16 CUDA tensors (each a whole number of 32-weight blocks along
    its last dimension).  Returns (grid fp32 CUDA [8], iters int32 CUDA [1],
    status)."""
    if isinstance(weights, torch.Tensor):
        weights = [weights]
    g0 = np.ascontiguousarray(np.asarray(grid0, np.float32).reshape(8))
    need = int(lib().moe_q4_lloyd_workspace(g0.ctypes.data))
    if need == 0:
        raise MoeQ4Error(EINVAL, "moe_q4_lloyd_workspace")
    dev = weights[0].device
    ws = alloc_workspace(need, dev)
    for i, w in enumerate(weights):
        if w.dtype != torch.bfloat16 or not w.is_cuda or w.numel() % 32:
            raise ValueError("weights must be bf16 CUDA tensors holding whole 32-weight blocks")
        w = w.contiguous()
        _check(lib().moe_q4_lloyd_hist(_ptr(w), w.numel() // 32, g0.ctypes.data, 1 if i == 0 else 0, _ptr(ws),
                                       ws.numel(), _stream(stream)), "moe_q4_lloyd_hist")
        _hold(stream, w)
    grid = torch.empty(8, dtype=torch.float32, device=dev)
    iters = torch.empty(1, dtype=torch.int32, device=dev)
    _check(lib().moe_q4_lloyd_solve(g0.ctypes.data, int(max_iter), float(tol), _ptr(grid), _ptr(iters), _ptr(ws),
                                    ws.numel(), _stream(stream)), "moe_q4_lloyd_solve")
    _hold(stream, ws)
    status = int(lib().moe_q4_read_status(_ptr(ws), _stream(stream)))
    return grid, iters, status


def combine(y: torch.Tensor, w: torch.Tensor, inv=None, out=None, out_f32=None, stream=None) -> torch.Tensor:
    """Weighted combine: y fp32 [T*k, H] (rows in (token, slot) order unless
    inv [T, k] places them), w fp32 [T, k] -> bf16 [T, H]."""
    T, k = w.shape
    H = y.shape[1]
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=y.device)
    y, w = y.contiguous(), w.contiguous()
    _check(lib().moe_q4_combine(_ptr(y), _ptr(w), _ptr(inv), T, k, H, _ptr(out), _ptr(out_f32), _stream(stream)),
           "moe_q4_combine")
    _hold(stream, y, w)
    return out


# ---- 8-bit integer rows, products and the int8 MLP -------------------------

_ROW_TYPE = {torch.bfloat16: 0, torch.float32: 1}
_INT8, _BF16, _FP32, _INT32 = (torch.int8,), (torch.bfloat16,), (torch.float32,), (torch.int32,)
# the current stream's handle without building a Stream object (a few us of a small call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _first(t, what, dtypes):
    """A call's first matrix: its device, shape and row stride."""
    dev = t.get_device()
    if dev < 0 or t.dtype not in dtypes or t.dim() != 2:
        raise ValueError(f"{what} must be a CUDA matrix of {' or '.join(str(d) for d in dtypes)}")
    n, k = t.shape
    ld, inner = t.stride()
    if inner != 1 and k > 1:
        raise ValueError(f"{what}: the elements of a row must be consecutive")
    return dev, n, k, ld if n > 1 else -(-k // 16) * 16


def _rows(t, what, dev, n, k, dtypes):
    """Check a [n, k] matrix of consecutive elements in each row; its row stride
    in elements (that of a single row is of no consequence)."""
    if t.shape == (n, k) and t.dtype in dtypes and t.get_device() == dev:
        ld, inner = t.stride()
        if inner == 1 or k <= 1:
            return ld if n > 1 else -(-k // 16) * 16
    raise ValueError(f"{what} must be a matrix [{n}, {k}] of {' or '.join(str(d) for d in dtypes)} with consecutive "
                     f"elements in a row, on cuda:{dev}; not {t.dtype} {list(t.shape)} with strides {t.stride()} on "
                     f"{t.device}")


def _vector(t, what, dev, n, dtypes=_FP32):
    if t.shape != (n,) or t.dtype not in dtypes or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous vector of {n} {' or '.join(str(d) for d in dtypes)} on "
                         f"cuda:{dev}; not {t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


def _call(what, dev, stream, fn, *args):
    """fn(*args, stream handle) with the tensors' device as the current one."""
    if stream is None:
        handle = _raw_stream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"the stream must be of the tensors' device, cuda:{dev}")
    else:
        handle = stream.cuda_stream
    if torch.cuda.current_device() == dev:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc != OK:
        raise MoeQ4Error(rc, what)


def _new(shape, dtype, like, stream):
    """A result's memory, allocated on the stream that the call runs on."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _codes(T, K, like, stream):
    """An int8 [T, K] whose rows start on 16 bytes, as the products read them."""
    if K % 16 == 0:
        return _new((T, K), torch.int8, like, stream)
    return _new((T, -(-K // 16) * 16), torch.int8, like, stream)[:, :K]


def quant_rows(x: torch.Tensor, q: torch.Tensor | None = None, scale: torch.Tensor | None = None, stream=None):
    """bf16 or fp32 rows x [T, K] -> (codes int8 [T, K], scales fp32 [T]): for
    each row scale = max|x| / 127 and the codes nearest to 127 x / max|x|, ties
    to even.  A new q has rows on 16-byte boundaries (linear_i8's operands)."""
    dev, T, K, ldx = _first(x, "x", _ROW_TYPE)
    if q is None:
        q = _codes(T, K, x, stream)
    if scale is None:
        scale = _new((T,), torch.float32, x, stream)
    _call("moe_q4_quant_rows", dev, stream, lib().moe_q4_quant_rows, x.data_ptr(), _ROW_TYPE[x.dtype], ldx, T, K,
          q.data_ptr(), _rows(q, "q", dev, T, K, _INT8), _vector(scale, "scale", dev, T))
    return q, scale


def add_norm(x: torch.Tensor, weight: torch.Tensor | None, eps: float = 1e-6, residual: torch.Tensor | None = None,
             residual_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
             q: torch.Tensor | None = None, scale: torch.Tensor | None = None, bf16: bool = True,
             quant: bool = True, stream=None):
    """Residual addition, root-mean-square norm and the norm's rows in bf16 and
    int8 in one pass: r = x + residual (the fp32 sum, rounded to the residual's
    type), then r * weight / sqrt(mean(r^2) + eps).  x and residual bf16 or fp32
    [T, H], weight bf16 or fp32 [H] or None (ones).  Returns (r or None without
    a residual, out bf16 [T, H] or None with bf16=False, codes int8 [T, H] and
    scales fp32 [T] or None with quant=False).  residual_out may be residual
    itself (in place), out may be a bf16 x."""
    dev, T, H, ldx = _first(x, "x", _ROW_TYPE)
    ldr = ldro = ldo = ldq = rt = wt = 0
    rp = rop = wp = op = qp = sp = None
    if residual is not None:
        dtype = residual.dtype
        ldr, rp = _rows(residual, "residual", dev, T, H, _ROW_TYPE), residual.data_ptr()
        if residual_out is None:
            residual_out = _new((T, H), dtype, x, stream)
        ldro, rop, rt = _rows(residual_out, "residual_out", dev, T, H, (dtype,)), residual_out.data_ptr(), _ROW_TYPE[dtype]
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if weight is not None:
        wp, wt = _vector(weight, "weight", dev, H, _ROW_TYPE), _ROW_TYPE[weight.dtype]
    if bf16 or out is not None:
        if out is None:
            out = _new((T, H), torch.bfloat16, x, stream)
        ldo, op = _rows(out, "out", dev, T, H, _BF16), out.data_ptr()
    if quant or q is not None or scale is not None:
        if q is None:
            q = _codes(T, H, x, stream)
        if scale is None:
            scale = _new((T,), torch.float32, x, stream)
        ldq, qp, sp = _rows(q, "q", dev, T, H, _INT8), q.data_ptr(), _vector(scale, "scale", dev, T)
    _call("moe_q4_add_norm", dev, stream, lib().moe_q4_add_norm, x.data_ptr(), _ROW_TYPE[x.dtype], ldx, rp, rt,
          ldr, rop, ldro, wp, wt, eps, T, H, op, ldo, qp, ldq, sp)
    return residual_out, out, q, scale


def linear_i8(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
              bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
              dtype: torch.dtype = torch.bfloat16, status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Int8 rows x [T, K] with scales x_scale [T] times int8 weights w [N, K]
    with scales w_scale [N], sums exact in int32: out [T, N] in bf16 or fp32
    (dtype, or out's), plus an fp32 bias [N].  The rows of x and w start on
    16-byte boundaries (quant_rows makes them so).  status: an int32 CUDA
    tensor [1] that receives the code of a device wait that gave up; without
    one i8_status() tells."""
    dev, T, K, ldx = _first(x, "x", _INT8)
    N = w.shape[0]
    if out is None:
        out = _new((T, N), dtype, x, stream)
    _call("moe_q4_linear_i8", dev, stream, lib().moe_q4_linear_i8, x.data_ptr(), ldx,
          _vector(x_scale, "x_scale", dev, T), w.data_ptr(), _rows(w, "w", dev, N, K, _INT8), _vector(w_scale, "w_scale", dev, N),
          None if bias is None else _vector(bias, "bias", dev, N), T, N, K, out.data_ptr(),
          _ROW_TYPE.get(out.dtype, -1), _rows(out, "out", dev, T, N, _ROW_TYPE),
          None if status is None else _vector(status, "status", dev, 1, _INT32))
    return out


def i8_status(device=None, stream=None) -> int:
    """Waits for the stream; the code of a device wait that gave up in a
    linear_i8 or mlp_i8 call without a status tensor on the device (0: none),
    which is cleared once it was returned."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return int(lib().moe_q4_i8_status(_stream(stream)))


class MlpI8:
    """A SwiGLU MLP with int8 weights: gate_up int8 [2I, H] (gate rows first)
    with scales [2I], down int8 [H, I] with scales [H], as quant_rows makes
    them of the bf16 matrices.  Also a layer's shared expert (forward_ex,
    forward_gated)."""

    def __init__(self, gate_up: torch.Tensor, gate_up_scale: torch.Tensor, down: torch.Tensor,
                 down_scale: torch.Tensor):
        dev, n, self.H, ldg = _first(gate_up, "gate_up", _INT8)
        if n % 2:
            raise ValueError("gate_up holds the gate's rows and as many rows of the up projection")
        self.I = n // 2
        ldd = _rows(down, "down", dev, self.H, self.I, _INT8)
        gp, dp = _vector(gate_up_scale, "gate_up_scale", dev, n), _vector(down_scale, "down_scale", dev, self.H)
        self.tensors = gate_up, gate_up_scale, down, down_scale
        self.struct = _MlpStruct(self.H, self.I, gate_up.data_ptr(), ldg, gp, down.data_ptr(), ldd, dp)
        self.ref = ctypes.byref(self.struct)


def mlp_i8_workspace(mlp: MlpI8, T: int) -> int:
    return int(lib().moe_q4_mlp_i8_workspace(mlp.ref, T))


def mlp_i8(mlp: MlpI8, x: torch.Tensor, x_scale: torch.Tensor, out: torch.Tensor | None = None,
           dtype: torch.dtype = torch.bfloat16, ws: torch.Tensor | None = None, status: torch.Tensor | None = None,
           stream=None) -> torch.Tensor:
    """The int8 SwiGLU MLP: int8 rows x [T, H] with scales x_scale [T] -> out
    [T, H] in bf16 or fp32 (dtype, or out's); status as for linear_i8."""
    dev, T, H, ldx = _first(x, "x", _INT8)
    if H != mlp.H:
        raise ValueError(f"x must have the MLP's {mlp.H} columns, not {H}")
    if out is None:
        out = _new((T, H), dtype, x, stream)
    if ws is None:
        ws = _new((max(mlp_i8_workspace(mlp, T), 256),), torch.uint8, x, stream)
    elif ws.get_device() != dev or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous uint8 on cuda:{dev} (alloc_workspace)")
    if mlp.tensors[0].get_device() != dev:
        raise ValueError(f"the MLP's weights must be on cuda:{dev}")
    _call("moe_q4_mlp_i8", dev, stream, lib().moe_q4_mlp_i8, mlp.ref, x.data_ptr(), ldx,
          _vector(x_scale, "x_scale", dev, T), T, out.data_ptr(),
          _ROW_TYPE.get(out.dtype, -1), _rows(out, "out", dev, T, H, _ROW_TYPE),
          None if status is None else _vector(status, "status", dev, 1, _INT32), ws.data_ptr(), ws.numel())
    return out


def _shared_rows(layer, shared, x, xq, x_scale):
    """Row stride of the int8 rows given to a forward beside x (0 for none); an
    int8 shared expert, those rows, the layer and x are on one device."""
    if (xq is None) != (x_scale is None):
        raise ValueError("xq and x_scale go together")
    if not isinstance(shared, MlpI8):
        if xq is not None:
            raise ValueError("xq and x_scale are read by an int8 shared expert (MlpI8)")
        return 0
    dev = x.get_device()
    for t, what in ((shared.tensors[0], "the MLP's weights"), (layer.gate_w, "the layer's weights")):
        if dev < 0 or t.get_device() != dev:
            raise ValueError(f"{what} (on {t.device}) and x (on {x.device}) must be on one CUDA device")
    if xq is None:
        return 0
    _vector(x_scale, "x_scale", dev, x.shape[0])
    return _rows(xq, "xq", dev, x.shape[0], layer.H, _INT8)
