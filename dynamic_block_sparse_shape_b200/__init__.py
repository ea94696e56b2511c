"""Python binding of libprism.so, the C ABI of the Prism block-sparse attention
hot path on B200 (see include/prism.h).

Argument marshalling only: every step runs in the CUDA library. PyTorch
provides device memory and streams. Importing this module does not need a GPU;
calling an entry point without the built library raises ``PrismError``.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

__all__ = [
    "PrismError", "Geometry", "ShapeParams", "lib", "library_path", "workspace_size", "Workspace", "zone_shapes",
    "block_pool", "block_select", "block_select_ex", "select_workspace_size", "topk_from_sparsity",
    "block_audio_bias", "mask_to_csr",
    "bsa_fwd", "bsa_bwd", "check_device_status", "STATUS", "OP", "DEFAULT_CDF_THRESHOLD",
    "RopeSpec", "rope", "rope_bwd", "gated_ffn_fwd", "gated_ffn_bwd", "GradList", "grad_norm", "scale_grads", "clip_grad_norm",
]

DEFAULT_CDF_THRESHOLD = 0.20

_HERE = os.path.dirname(os.path.abspath(__file__))
# PRISM_LIBRARY names another build of the library (a test variant) to load instead
_LIB_PATH = os.environ.get("PRISM_LIBRARY") or os.path.join(_HERE, "libprism.so")

STATUS = {
    0: "PRISM_OK", 1: "PRISM_ERR_ARG", 2: "PRISM_ERR_SHAPE", 3: "PRISM_ERR_DTYPE", 4: "PRISM_ERR_WORKSPACE",
    5: "PRISM_ERR_CAPACITY", 6: "PRISM_ERR_CUDA", 7: "PRISM_ERR_TIMEOUT", 8: "PRISM_ERR_DEVICE",
    9: "PRISM_ERR_UNSUPPORTED",
}
OP = {"zone_shapes": 0, "block_select": 1, "bsa_fwd": 2, "bsa_bwd": 3}
BF16, FP32 = 0, 1


class PrismError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        self.name = STATUS.get(status, str(status))
        msg = _lib.prism_status_string(status).decode() if _lib is not None else self.name
        super().__init__(f"{what}: {self.name} ({msg})")


class _Dim3(ctypes.Structure):
    _fields_ = [("t", ctypes.c_int32), ("h", ctypes.c_int32), ("w", ctypes.c_int32)]


class _Geometry(ctypes.Structure):
    _fields_ = [("grid", _Dim3), ("zone", _Dim3), ("cand", ctypes.POINTER(_Dim3)), ("n_cand", ctypes.c_int32)]


class _ShapeParams(ctypes.Structure):
    _fields_ = [("w_audio", ctypes.c_float), ("gamma", ctypes.c_float), ("gate_max", ctypes.c_float)]


class _RopeParams(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("scaling", ctypes.c_int32), ("n_axes", ctypes.c_int32),
                ("axis_dim", ctypes.c_int32 * 3), ("theta", ctypes.c_double), ("factor", ctypes.c_double),
                ("trained_len", ctypes.c_double), ("magnitude", ctypes.c_double), ("pos_scale", ctypes.c_double * 3),
                ("pos_offset", ctypes.c_double * 3)]


class _Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _FfnWeights(ctypes.Structure):
    _fields_ = [("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("gate_stride", ctypes.c_int64), ("up_stride", ctypes.c_int64), ("down_stride", ctypes.c_int64),
                ("d", ctypes.c_int32), ("f", ctypes.c_int32)]


class _SelectParams(ctypes.Structure):
    _fields_ = [("top_k", ctypes.c_int32), ("cdf_threshold", ctypes.c_float),
                ("head_top_k", ctypes.POINTER(ctypes.c_int32)), ("head_cdf_threshold", ctypes.POINTER(ctypes.c_float)),
                ("key_bias", ctypes.c_void_p)]


_P = ctypes.c_void_p
_I32, _I64, _F32, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_GEO = ctypes.POINTER(_Geometry)
_DIM3 = ctypes.POINTER(_Dim3)

_SIGNATURES = {
    "prism_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "prism_version": (_I32, []),
    "prism_geometry_counts": (ctypes.c_int, [_GEO, ctypes.POINTER(_I32), ctypes.POINTER(_I32)]),
    "prism_workspace_size": (ctypes.c_int, [ctypes.c_int, _GEO, _I32, _I32, _I32, _I32, ctypes.c_int, _I64,
                                            ctypes.POINTER(_SZ)]),
    "prism_check_device_status": (ctypes.c_int, [_P, _P]),
    "prism_clear_device_status": (ctypes.c_int, [_P, _P]),
    "prism_keep_device_status": (ctypes.c_int, [_P, _P]),
    "prism_check_kept_status": (ctypes.c_int, [_P, _P]),
    "prism_zone_shapes": (ctypes.c_int, [_GEO, _P, _I64, _I32, ctypes.c_int, _P, _I64, _I32, ctypes.c_int,
                                         ctypes.POINTER(_ShapeParams), _P, _P, _P, _SZ, _P]),
    "prism_zone_shapes_static": (ctypes.c_int, [_GEO, _P, _I64, _I32, ctypes.c_int, _P, _I64, _I32, ctypes.c_int,
                                                ctypes.POINTER(_ShapeParams), _P, _P, _P]),
    "prism_block_pool": (ctypes.c_int, [_GEO, _P, _P, _P, ctypes.c_int, _I32, _I32, _I64, _P, _P, _P, _SZ, _P]),
    "prism_block_select": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _F32, _I32, _F32, _P, _P, _P, _P, _I64,
                                          ctypes.POINTER(_I64), _P, _SZ, _P]),
    "prism_block_select_ex": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _F32, ctypes.POINTER(_SelectParams), _P, _P,
                                             _P, _P, _I64, ctypes.POINTER(_I64), _P, _SZ, _P]),
    "prism_topk_from_sparsity": (ctypes.c_int, [_F32, _I32, ctypes.POINTER(_I32)]),
    "prism_block_select_workspace_size": (ctypes.c_int, [_I32, _I32, _I32, ctypes.POINTER(_SZ)]),
    "prism_block_audio_bias": (ctypes.c_int, [_GEO, _P, _P, _I64, _I32, ctypes.c_int, _F32, _P, _P, _SZ, _P]),
    "prism_mask_to_csr": (ctypes.c_int, [_P, _P, _I32, _I32, _P, _I64, _P, _SZ, _P]),
    "prism_bsa_fwd": (ctypes.c_int, [_GEO, _P, _P, _P, _P, ctypes.c_int, _I32, _I32, _I64, _F32, _P, _P, _I64, _P,
                                     _P, _P, _P, _SZ, _P]),
    "prism_bsa_bwd": (ctypes.c_int, [_GEO, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int, _I32, _I32, _I64, _F32,
                                     _P, _P, _I64, _P, _P, _P, _P, _SZ, _P]),
    "prism_rope": (ctypes.c_int, [ctypes.POINTER(_RopeParams), _DIM3, _P, _I64, _P, _P, _I32, _I64, _I64, _P, _P, _I32,
                                  _I64, _I64, ctypes.c_int, _I32, _I32, _P]),
    "prism_gated_ffn_fwd": (ctypes.c_int, [ctypes.POINTER(_FfnWeights), _I64, _I32, ctypes.c_int, _P, _I64, _P, _I64, _P,
                                           _P, _P, _SZ, _P]),
    "prism_gated_ffn_bwd": (ctypes.c_int, [ctypes.POINTER(_FfnWeights), _I64, _I32, ctypes.c_int, _P, _I64, _P, _I64, _P,
                                           _P, _P, _I64, _P, _P, _P, _P, _SZ, _P]),
    "prism_gated_ffn_forms": (ctypes.c_int, [ctypes.POINTER(_FfnWeights), _I64, _I32, ctypes.POINTER(_I32)]),
    "prism_gated_ffn_workspace_size": (ctypes.c_int, [_I64, _I32, _I32, ctypes.POINTER(_SZ)]),
    "prism_grad_norm": (ctypes.c_int, [_P, _I64, _I32, _P, _P, _SZ, _P]),
    "prism_grad_norm_workspace_size": (ctypes.c_int, [_I64, ctypes.POINTER(_SZ)]),
    "prism_grad_scale": (ctypes.c_int, [_P, _I64, _P, _F32, _F32, _P]),
    "prism_grad_clip": (ctypes.c_int, [_P, _I64, _I32, _F32, _F32, _P, _P, _SZ, _P]),
}


def _load():
    if not os.path.exists(_LIB_PATH):
        return None
    lib = ctypes.CDLL(_LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = None  # loaded on first use, so that building the library needs no library


def lib():
    """The loaded ctypes library; raises if libprism.so was not built."""
    global _lib
    if _lib is None:
        _lib = _load()
    if _lib is None:
        raise PrismError(6, f"libprism.so not found at {_LIB_PATH}; run dynamic_block_sparse_shape_b200.build")
    return _lib


def library_path() -> str:
    return _LIB_PATH


def _check(status: int, what: str):
    if status != 0:
        raise PrismError(status, what)


@dataclass(frozen=True)
class Geometry:
    """Token grid (T, H, W), macro-zone extents and candidate block shapes."""
    grid: tuple
    zone: tuple
    cand: tuple

    def c(self):
        arr = (_Dim3 * len(self.cand))(*[_Dim3(*c) for c in self.cand])
        g = _Geometry(_Dim3(*self.grid), _Dim3(*self.zone), arr, len(self.cand))
        g._keep = arr  # keep the candidate array alive with the struct
        return g

    @property
    def n_tokens(self):
        return self.grid[0] * self.grid[1] * self.grid[2]

    def counts(self):
        nz, nb = _I32(), _I32()
        g = self.c()
        _check(lib().prism_geometry_counts(ctypes.byref(g), ctypes.byref(nz), ctypes.byref(nb)), "geometry")
        return nz.value, nb.value


@dataclass(frozen=True)
class ShapeParams:
    w_audio: float = 1.0
    gamma: float = 0.25
    gate_max: float = 4.0


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return FP32
    raise PrismError(3, f"dtype {t.dtype}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def workspace_size(op: str, geo: Geometry, heads=1, head_dim=128, feat_c=0, res_c=0, dtype=torch.bfloat16,
                   nnz=0) -> int:
    out = _SZ()
    g = geo.c()
    code = FP32 if dtype == torch.float32 else BF16
    _check(lib().prism_workspace_size(OP[op], ctypes.byref(g), heads, head_dim, feat_c, res_c, code, nnz,
                                      ctypes.byref(out)), f"workspace_size({op})")
    return out.value


class Workspace:
    """A caller-owned device scratch buffer (torch allocation, 256-byte aligned)
    that grows on demand. The library itself never allocates. It belongs to the
    stream that is current when it is made or grows; calls on other streams are
    noted, so its memory is not handed on before they are done. Calls that share
    a workspace must be ordered one behind the other. A buffer that a captured
    graph may hold stays allocated when a larger one takes its place."""

    def __init__(self, device="cuda", nbytes=1 << 20):
        self.device = torch.device(device)
        self.buf = None
        self.captured = False  # `buf` was used under a stream capture
        self.kept = []
        self.ensure(nbytes)

    def ensure(self, nbytes: int):
        """Makes room for `nbytes`, for work on the current stream."""
        nbytes = max(int(nbytes), 256)
        if self.device.type == "cuda" and self.device.index not in (None, torch._C._cuda_getDevice()):
            with torch.cuda.device(self.device):
                return self._ensure(nbytes)
        return self._ensure(nbytes)

    def _ensure(self, nbytes: int):
        if self.buf is None or self.nbytes < nbytes:
            if self.captured:
                self.kept.append(self.buf)
            self.buf = torch.empty(nbytes + 256, dtype=torch.uint8, device=self.device)
            self.start = (self.buf.data_ptr() + 255) // 256 * 256
            self.nbytes = nbytes
            self.captured = False
            self.device, self.index = self.buf.device, self.buf.get_device()
            # the status word; every call writes the rest before it reads it
            if self.index >= 0:
                self.home = _raw_stream(self.index)
                _check(lib().prism_clear_device_status(self.start, self.home), "workspace")
            else:
                at = self.start - self.buf.data_ptr()
                self.buf[at:at + 256].zero_()
        if self.index >= 0:
            if _raw_stream(self.index) != self.home:
                self.buf.record_stream(torch.cuda.current_stream(self.device))
            if torch.cuda.is_current_stream_capturing():
                self.captured = True
        return self

    @property
    def ptr(self):
        return ctypes.c_void_p(self.start)


_raw_stream = torch._C._cuda_getCurrentRawStream  # of a device's current stream


def _require(ok: bool, what: str, status: int = 1):
    if not ok:
        raise PrismError(status, what)


class _On:
    """The device and the stream of a call made current: those of its tensors (of the current device without any), and
    the stream given or that device's current one (`ptr`). What the call allocates then belongs to its stream; results
    are noted on the caller's stream as well (`made`), which goes on to read them."""
    __slots__ = ("guard", "caller", "ptr", "device", "passing")

    def __init__(self, tensors, stream, what):
        index = tensors[0].get_device() if tensors else torch.cuda.current_device()
        for t in tensors:
            if t.get_device() != index:
                _require(False, what + ": tensors on different devices")
        if index < 0:
            _require(False, what + ": tensors must be on a CUDA device")
        if stream is not None and stream.device_index != index:
            _require(False, what + ": a stream of another device")
        self.device = index
        self.guard = self.caller = self.passing = None
        self.ptr = _raw_stream(index)
        if stream is not None and stream.cuda_stream != self.ptr:
            self.caller = torch.cuda.current_stream(index)
            self.ptr = stream.cuda_stream
            self.guard = torch.cuda.stream(stream)
        elif index != torch._C._cuda_getDevice():
            self.guard = torch.cuda.device(index)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        try:
            if self.passing is not None and exc[0] is None:
                # the workspace goes, what its status word says stays
                _check(lib().prism_keep_device_status(self.passing.start, self.ptr), "device status")
        finally:
            if self.guard is not None:
                self.guard.__exit__(*exc)

    def made(self, *tensors):
        if self.caller is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.caller)

    def workspace(self, ws: Optional[Workspace], nbytes: int, what: str) -> Workspace:
        """The workspace given, or one for this call, with room for `nbytes`."""
        if ws is None:
            self.passing = Workspace(torch.device("cuda", self.device), nbytes)
            return self.passing
        if ws.index != self.device:
            _require(False, what + ": a workspace of another device", 4)
        return ws._ensure(nbytes)


def check_device_status(ws: Optional[Workspace] = None, stream=None):
    """Waits for the stream and raises what a kernel that used ``ws`` reported: a wait that ran out, a bad index. Without
    ``ws``: what the calls without a workspace on the current device did."""
    what = "device status"
    with _On([ws.buf] if ws is not None else [], stream, what) as on:
        if ws is not None:
            _check(lib().prism_check_device_status(ws.ptr, on.ptr), what)
        else:
            tmp = Workspace(torch.device("cuda", on.device), 256)
            _check(lib().prism_check_kept_status(tmp.ptr, on.ptr), what)


def zone_shapes(geo: Geometry, feat: Optional[torch.Tensor] = None, res: Optional[torch.Tensor] = None,
                params: Optional[ShapeParams] = None, ws: Optional[Workspace] = None, stream=None):
    """a1+a2: per-zone candidate index (int32 [n_zones]) and cost margin (fp32)."""
    what = "prism_zone_shapes"
    nz, _ = geo.counts()
    feat_c = feat.shape[1] if feat is not None else 0
    res_c = res.shape[1] if res is not None else 0
    fdt = feat.dtype if feat is not None else torch.bfloat16
    need = workspace_size("zone_shapes", geo, feat_c=feat_c, res_c=res_c, dtype=fdt)
    p = params or ShapeParams()
    cp = _ShapeParams(p.w_audio, p.gamma, p.gate_max)
    g = geo.c()
    if feat is not None:
        assert feat.stride(1) == 1
    if res is not None:
        assert res.stride(1) == 1
    tensors = [t for t in (feat, res) if t is not None] or ([ws.buf] if ws is not None else [])
    with _On(tensors, stream, what) as on:
        ws = on.workspace(ws, need, what)
        shape = torch.empty(nz, dtype=torch.int32, device=ws.device)
        margin = torch.empty(nz, dtype=torch.float32, device=ws.device)
        on.made(shape, margin)
        _check(lib().prism_zone_shapes(
            ctypes.byref(g), _ptr(feat), feat.stride(0) if feat is not None else 0, feat_c,
            _dtype_code(feat) if feat is not None else BF16, _ptr(res), res.stride(0) if res is not None else 0, res_c,
            _dtype_code(res) if res is not None else BF16, ctypes.byref(cp), _ptr(shape), _ptr(margin), ws.ptr,
            ws.nbytes, on.ptr), what)
    return shape, margin


def block_pool(geo: Geometry, zone_shape: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
               ws: Optional[Workspace] = None, stream=None):
    """a3: mean-pooled block features, fp32 [heads, n_blocks, head_dim] each."""
    _, nb = geo.counts()
    N, H, d = q.shape
    assert q.stride(2) == 1 and q.stride(1) == d and k.stride() == q.stride()
    what = "prism_block_pool"
    g = geo.c()
    with _On((zone_shape, q, k), stream, what) as on:
        ws = on.workspace(ws, 256, what)
        qp = torch.empty((H, nb, d), dtype=torch.float32, device=q.device)
        kp = torch.empty_like(qp)
        on.made(qp, kp)
        _check(lib().prism_block_pool(ctypes.byref(g), _ptr(zone_shape), _ptr(q), _ptr(k), _dtype_code(q), H, d,
                                      q.stride(0), _ptr(qp), _ptr(kp), ws.ptr, ws.nbytes, on.ptr), what)
    return qp, kp


def select_workspace_size(heads: int, n_blocks: int, head_dim: int) -> int:
    """Workspace bytes of block_select / block_select_ex for these pooled shapes."""
    b = _SZ()
    _check(lib().prism_block_select_workspace_size(int(heads), int(n_blocks), int(head_dim), ctypes.byref(b)),
           "prism_block_select_workspace_size")
    return int(b.value)


def _select(call, tensors, ws, csr, stream, what):
    """Outputs of a selection over the pooled tensors; `call` runs it."""
    H, nb, d = tensors[0].shape
    words = (nb + 31) // 32
    dev = tensors[0].device
    with _On(tensors, stream, what) as on:
        ws = on.workspace(ws, select_workspace_size(H, nb, d), what)
        mask = torch.empty((H, nb, words), dtype=torch.int32, device=dev)
        kept = torch.empty((H, nb), dtype=torch.int32, device=dev)
        row_ptr = torch.empty(H * nb + 1, dtype=torch.int32, device=dev)
        on.made(mask, kept, row_ptr)
        total = _I64()
        _check(call(ws, mask, kept, row_ptr, total, on.ptr), what)
        out = {"mask": mask, "kept": kept, "row_ptr": row_ptr, "total": int(total.value), "col_idx": None}
        if csr:
            col = torch.empty(max(1, total.value), dtype=torch.int32, device=dev)
            on.made(col)
            mask_to_csr(mask, row_ptr, nb, col, ws=ws)
            out["col_idx"] = col[:total.value]
    return out


def block_select(qp: torch.Tensor, kp: torch.Tensor, scale: float, top_k: int,
                 cdf_threshold: float = DEFAULT_CDF_THRESHOLD, ws: Optional[Workspace] = None, csr: bool = True,
                 stream=None):
    """a4+a5: hybrid top-k + CDF selection. Returns dict with mask (int32 view of
    the uint32 words [H, nb, ceil(nb/32)]), kept [H, nb], row_ptr [H*nb+1],
    col_idx [total] and total (int)."""
    H, nb, d = qp.shape

    def call(ws, mask, kept, row_ptr, total, ptr):
        return lib().prism_block_select(_ptr(qp), _ptr(kp), H, nb, d, float(scale), int(top_k), float(cdf_threshold),
                                        _ptr(mask), _ptr(kept), _ptr(row_ptr), None, 0, ctypes.byref(total), ws.ptr,
                                        ws.nbytes, ptr)

    return _select(call, (qp, kp), ws, csr, stream, "prism_block_select")


def block_select_ex(qp: torch.Tensor, kp: torch.Tensor, scale: float, top_k,
                    cdf_threshold=DEFAULT_CDF_THRESHOLD, key_bias: Optional[torch.Tensor] = None,
                    ws: Optional[Workspace] = None, csr: bool = True, stream=None):
    """a4+a5 with per-head settings: ``top_k`` and ``cdf_threshold`` are scalars
    or sequences of one value per head; ``key_bias`` is None or a device fp32
    [n_blocks] added to every head's logit of each key block (for example from
    ``block_audio_bias``). Returns the same dict as ``block_select``."""
    H, nb, d = qp.shape
    cp = _SelectParams()
    keep, tensors = [], [qp, kp]
    if isinstance(top_k, (int,)) or (torch.is_tensor(top_k) and top_k.dim() == 0):
        cp.top_k = int(top_k)
    else:
        arr = (ctypes.c_int32 * H)(*[int(x) for x in top_k])
        keep.append(arr)
        cp.top_k = int(arr[0]) if H else 1
        cp.head_top_k = ctypes.cast(arr, ctypes.POINTER(ctypes.c_int32))
    if isinstance(cdf_threshold, (int, float)) or (torch.is_tensor(cdf_threshold) and cdf_threshold.dim() == 0):
        cp.cdf_threshold = float(cdf_threshold)
    else:
        arr = (ctypes.c_float * H)(*[float(x) for x in cdf_threshold])
        keep.append(arr)
        cp.cdf_threshold = float(arr[0]) if H else 0.0
        cp.head_cdf_threshold = ctypes.cast(arr, ctypes.POINTER(ctypes.c_float))
    if key_bias is not None:
        assert key_bias.dtype == torch.float32 and key_bias.numel() == nb and key_bias.is_contiguous()
        cp.key_bias = key_bias.data_ptr()
        tensors.append(key_bias)

    def call(ws, mask, kept, row_ptr, total, ptr):
        return lib().prism_block_select_ex(_ptr(qp), _ptr(kp), H, nb, d, float(scale), ctypes.byref(cp), _ptr(mask),
                                           _ptr(kept), _ptr(row_ptr), None, 0, ctypes.byref(total), ws.ptr, ws.nbytes,
                                           ptr)

    return _select(call, tensors, ws, csr, stream, "prism_block_select_ex")


def topk_from_sparsity(sparsity: float, n_blocks: int) -> int:
    """Top-k floor for a top-k sparsity ratio: n_blocks - floor(sparsity * n_blocks), at least 1."""
    k = _I32()
    _check(lib().prism_topk_from_sparsity(float(sparsity), int(n_blocks), ctypes.byref(k)), "prism_topk_from_sparsity")
    return int(k.value)


def block_audio_bias(geo: Geometry, zone_shape: torch.Tensor, res: torch.Tensor, beta: float,
                     ws: Optional[Workspace] = None, stream=None) -> torch.Tensor:
    """Audio-norm bias of every key block, device fp32 [n_blocks]:
    beta * (block mean of ||res[n]||) / (grid mean of ||res[n]||)."""
    _, nb = geo.counts()
    assert res.dim() == 2 and res.stride(1) == 1
    what = "prism_block_audio_bias"
    g = geo.c()
    with _On((zone_shape, res), stream, what) as on:
        ws = on.workspace(ws, 256, what)
        out = torch.empty(nb, dtype=torch.float32, device=res.device)
        on.made(out)
        _check(lib().prism_block_audio_bias(ctypes.byref(g), _ptr(zone_shape), _ptr(res), res.stride(0), res.shape[1],
                                            _dtype_code(res), float(beta), _ptr(out), ws.ptr, ws.nbytes, on.ptr), what)
    return out


def mask_to_csr(mask: torch.Tensor, row_ptr: torch.Tensor, n_blocks: int, col_idx: torch.Tensor,
                ws: Optional[Workspace] = None, stream=None):
    """Expands selection bitmask rows into ascending CSR column lists."""
    rows = row_ptr.numel() - 1
    what = "prism_mask_to_csr"
    with _On((mask, row_ptr, col_idx), stream, what) as on:
        ws = on.workspace(ws, 256, what)
        _check(lib().prism_mask_to_csr(_ptr(mask), _ptr(row_ptr), rows, n_blocks, _ptr(col_idx), col_idx.numel(),
                                       ws.ptr, ws.nbytes, on.ptr), what)
    return col_idx


def bsa_fwd(geo: Geometry, zone_shape, q, k, v, scale, row_ptr, col_idx, ws: Optional[Workspace] = None,
            out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None,
            o_lo: Optional[torch.Tensor] = None, nnz: Optional[int] = None):
    """a6: block-sparse attention forward. Returns (O like q, LSE fp32 [H, N]).

    o_lo (optional, bf16 like a bf16 q): receives the rounding residual of O,
    to be passed to bsa_bwd so that D = dO . O is formed from O to ~16 bits.
    nnz (optional): the selection's total kept pairs; it chooses the kernels'
    plan (rows short on average: no block images), not the result."""
    N, H, d = q.shape
    assert q.stride(2) == 1 and q.stride(1) == d and k.stride() == q.stride() and v.stride() == q.stride()
    need = workspace_size("bsa_fwd", geo, heads=H, head_dim=d, dtype=q.dtype)
    what = "prism_bsa_fwd"
    if o_lo is not None:
        assert o_lo.dtype == torch.bfloat16 and o_lo.stride() == q.stride()
    g = geo.c()
    given = [t for t in (out, lse, o_lo) if t is not None]
    with _On([zone_shape, q, k, v, row_ptr, col_idx, *given], stream, what) as on:
        ws = on.workspace(ws, need, what)
        o, lse_t = out, lse
        if out is None:
            o = torch.empty_like(q)
            on.made(o)
        assert o.stride() == q.stride()
        if lse is None:
            lse_t = torch.empty((H, N), dtype=torch.float32, device=q.device)
            on.made(lse_t)
        _check(lib().prism_bsa_fwd(ctypes.byref(g), _ptr(zone_shape), _ptr(q), _ptr(k), _ptr(v), _dtype_code(q), H, d,
                                   q.stride(0), float(scale), _ptr(row_ptr), _ptr(col_idx),
                                   -1 if nnz is None else int(nnz), _ptr(o), _ptr(lse_t),
                                   _ptr(o_lo), ws.ptr, ws.nbytes, on.ptr), what)
    return o, lse_t


def bsa_bwd(geo: Geometry, zone_shape, q, k, v, o, lse, do, scale, row_ptr, col_idx, nnz: int,
            ws: Optional[Workspace] = None, grads: Optional[Sequence[torch.Tensor]] = None, stream=None,
            o_lo: Optional[torch.Tensor] = None):
    """a7: block-sparse attention backward. Returns (dQ, dK, dV) like q.

    o_lo: the forward's rounding residual of O (bsa_fwd's o_lo), or None."""
    N, H, d = q.shape
    for t in (k, v, o, do):
        assert t.stride() == q.stride()
    need = workspace_size("bsa_bwd", geo, heads=H, head_dim=d, dtype=q.dtype, nnz=nnz)
    what = "prism_bsa_bwd"
    g = geo.c()
    if o_lo is not None:
        assert o_lo.dtype == torch.bfloat16 and o_lo.stride() == q.stride()
    given = [t for t in (o_lo, *(grads or ())) if t is not None]
    with _On([zone_shape, q, k, v, o, lse, do, row_ptr, col_idx, *given], stream, what) as on:
        ws = on.workspace(ws, need, what)
        if grads is None:
            dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
            on.made(dq, dk, dv)
        else:
            dq, dk, dv = grads
        _check(lib().prism_bsa_bwd(ctypes.byref(g), _ptr(zone_shape), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(o_lo),
                                   _ptr(lse), _ptr(do), _dtype_code(q), H, d, q.stride(0), float(scale), _ptr(row_ptr),
                                   _ptr(col_idx), int(nnz), _ptr(dq), _ptr(dk), _ptr(dv), ws.ptr, ws.nbytes, on.ptr),
               what)
    return dq, dk, dv


# ------------------------------------------------- around the attention
_ROPE_LAYOUT = {"interleaved": 0, "half": 1}
_ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


class RopeSpec:
    """The rotation of ``rope``: how many channels of a head each axis rotates and by which angles.

    axis_dims: rotated channels per axis, (t, h, w) of the token grid or one entry for a single position; the channels
        behind their sum stay as they are. In the Prism models' video towers a 128-wide head has (44, 42, 42).
    layout: "interleaved" (pair i is channels 2i, 2i + 1) or "half" (i, i + rot_dim / 2).
    theta: pair j of an axis of n channels turns by theta ** (-2 j / n) per position.
    scaling, factor, trained_len: "none"; "linear" (frequencies / factor); "ntk" (theta * factor ** (n / (n - 2)));
        "yarn" (pairs that turn over 32 times in trained_len positions kept, those below once / factor, a ramp between).
    magnitude: multiplies the rotated channels; None is 1, or 0.1 ln(factor) + 1 with "yarn" and a factor above 1.
    pos_scale, pos_offset: per axis, the position p counts as pos_offset + p * pos_scale (for example video frames on
        the time axis of the audio tokens).
    """

    def __init__(self, axis_dims, layout="interleaved", theta=10000.0, scaling="none", factor=1.0, trained_len=4096.0,
                 magnitude=None, pos_scale=None, pos_offset=None):
        dims = tuple(int(x) for x in axis_dims)
        _require(len(dims) in (1, 3), "RopeSpec: axis_dims has one or three entries")
        _require(layout in _ROPE_LAYOUT, f"RopeSpec: layout {layout!r}")
        _require(scaling in _ROPE_SCALING, f"RopeSpec: scaling {scaling!r}")
        if magnitude is None:
            _require(scaling != "yarn" or factor > 0, "RopeSpec: factor must be positive")
            magnitude = 0.1 * math.log(max(factor, 1.0)) + 1.0 if scaling == "yarn" else 1.0
        scale = tuple(pos_scale) if pos_scale is not None else (1.0,) * len(dims)
        offset = tuple(pos_offset) if pos_offset is not None else (0.0,) * len(dims)
        _require(len(scale) == len(dims) and len(offset) == len(dims), "RopeSpec: one pos_scale and pos_offset per axis")
        self.axis_dims, self.layout, self.magnitude = dims, layout, float(magnitude)
        pad = (0,) * (3 - len(dims))
        self._c = _RopeParams(_ROPE_LAYOUT[layout], _ROPE_SCALING[scaling], len(dims),
                              (ctypes.c_int32 * 3)(*dims, *pad), float(theta), float(factor), float(trained_len),
                              float(magnitude), (ctypes.c_double * 3)(*scale, *pad), (ctypes.c_double * 3)(*offset, *pad))
        self._ref = ctypes.byref(self._c)


def _token_stride(t: torch.Tensor, what: str) -> int:
    """Elements between tokens of a [N, heads, d] tensor with contiguous heads and channels."""
    if t.dim() != 3:
        _require(False, what + ": [tokens, heads, head_dim] expected")
    n, h, d = t.shape
    sn, sh, sd = t.stride()
    if (sd != 1 and d != 1) or (sh != d and h != 1):
        _require(False, what + ": heads and channels must be contiguous")
    return sn if n > 1 else max(sn, h * d)


def _like(o, t, what):
    if o.shape != t.shape or o.dtype != t.dtype or o.device != t.device:
        _require(False, what + ": an output is not like its input")


def _rope(q, k, spec, grid, positions, out, stream, transposed, what):
    sq = _token_stride(q, what)
    n, hq, d = q.shape
    code = _dtype_code(q)
    tensors = [q]
    hk, sk, sok, ok, kp, okp = 0, 0, 0, None, None, None
    if k is not None:
        sk = _token_stride(k, what)
        nk, hk, dk = k.shape
        if nk != n or dk != d:
            _require(False, what + ": q and k differ in tokens or head_dim")
        if k.dtype != q.dtype:
            _require(False, what + ": q and k differ in type", 3)
        tensors.append(k)
        kp = k.data_ptr()
    pp = None
    if positions is not None:
        if positions.dtype != torch.int32:
            _require(False, what + ": positions must be int32", 3)
        axes = len(spec.axis_dims)
        if positions.numel() != n * axes or (axes > 1 and positions.shape != (n, axes)) or not positions.is_contiguous():
            _require(False, what + ": positions must be contiguous [tokens, axes]")
        tensors.append(positions)
        pp = positions.data_ptr()
    with _On(tensors, stream, what) as on:
        if out is None:
            oq = torch.empty_like(q) if q.is_contiguous() else q.new_empty(n, hq, d)
            soq = hq * d
            if k is not None:
                ok = torch.empty_like(k) if k.is_contiguous() else k.new_empty(n, hk, d)
                sok = hk * d
            on.made(oq, ok)
        else:
            oq, ok = out if k is not None else ((out, None) if torch.is_tensor(out) else (out[0], None))
            _like(oq, q, what)
            soq = _token_stride(oq, what)
            if k is not None:
                _like(ok, k, what)
                sok = _token_stride(ok, what)
        if k is not None:
            okp = ok.data_ptr()
        g = None if grid is None else ctypes.byref(_Dim3(*(int(x) for x in grid)))
        _check(lib().prism_rope(spec._ref, g, pp, n, q.data_ptr(), oq.data_ptr(), hq, sq, soq, kp, okp, hk, sk, sok,
                                code, d, transposed, on.ptr), what)
    return oq, ok


def rope(q: torch.Tensor, k: Optional[torch.Tensor], spec: RopeSpec, grid=None,
         positions: Optional[torch.Tensor] = None, out=None, stream=None):
    """Rotary positions of Q [N, heads, d] and K [N, heads_k, d] (or None): returns the rotated (q, k).

    grid: the (T, H, W) token grid in raster order, for a three-axis spec; positions: int32 [N, axes] instead of it
    (one axis: N values of any shape).
    With neither, a one-axis spec takes the token's index. out: the pair of tensors to write, (q, k) for in place."""
    return _rope(q, k, spec, grid, positions, out, stream, 0, "prism_rope")


def rope_bwd(dq: torch.Tensor, dk: Optional[torch.Tensor], spec: RopeSpec, grid=None,
             positions: Optional[torch.Tensor] = None, out=None, stream=None):
    """The gradient of ``rope``: dQ and dK of the rotated tensors (from ``bsa_bwd``) to those of the unrotated ones."""
    return _rope(dq, dk, spec, grid, positions, out, stream, 1, "prism_rope (transposed)")


_ACT = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}


def _row_stride(t: torch.Tensor, rows, cols, what: str, name: str) -> int:
    """Elements between the rows of a [rows, cols] matrix with contiguous rows."""
    if t.is_contiguous() and t.shape == (rows, cols) and cols % 8 == 0:
        return cols
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        _require(False, f"{what}: {name} must be [{rows}, {cols}]")
    s0, s1 = t.stride()
    if s1 != 1 and cols != 1:
        _require(False, f"{what}: the rows of {name} must be contiguous")
    return s0 if rows > 1 else max(s0, -(-cols // 8) * 8)


def _ffn_weights(w_gate, w_up, w_down, what):
    if w_gate.dim() != 2:
        _require(False, what + ": w_gate must be [f, d]")
    f, d = w_gate.shape
    return _FfnWeights(w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
                       _row_stride(w_gate, f, d, what, "w_gate"), _row_stride(w_up, f, d, what, "w_up"),
                       _row_stride(w_down, d, f, what, "w_down"), d, f), d, f


@functools.lru_cache(maxsize=256)
def _ffn_workspace_bytes(m, f, backward):
    b = _SZ()
    _check(lib().prism_gated_ffn_workspace_size(m, f, backward, ctypes.byref(b)), "prism_gated_ffn_workspace_size")
    return b.value


def _new_like(t: torch.Tensor, rows: int, cols: int) -> torch.Tensor:
    """A contiguous [rows, cols] matrix of t's type; t has that shape."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(rows, cols)


def _same_type(tensors, what):
    kind = tensors[0].dtype
    for t in tensors:
        if t.dtype != kind:
            _require(False, what + ": tensors of different types", 3)
    return _dtype_code(tensors[0])


def gated_ffn_fwd(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, act: str = "silu",
                  save: bool = True, out: Optional[torch.Tensor] = None, ws: Optional[Workspace] = None, stream=None):
    """Gated feed-forward block y = (act(x Wg^T) * (x Wu^T)) Wd^T of x [m, d], weights Wg, Wu [f, d], Wd [d, f] (bf16).

    act: "silu", "gelu", "gelu_tanh" or "relu". Returns (y, gate, up): with ``save`` the projections [m, f] that
    ``gated_ffn_bwd`` needs, else None. out: where y goes."""
    what = "prism_gated_ffn_fwd"
    if act not in _ACT:
        _require(False, f"{what}: act {act!r}")
    every = (x, w_gate, w_up, w_down) if out is None else (x, w_gate, w_up, w_down, out)
    code = _same_type(every, what)
    w, d, f = _ffn_weights(w_gate, w_up, w_down, what)
    m = x.shape[0] if x.dim() else 0
    sx = _row_stride(x, m, d, what, "x")
    with _On(every, stream, what) as on:
        ws = on.workspace(ws, _ffn_workspace_bytes(m, f, 0), what)
        y, gate, up, gp, upp = out, None, None, None, None
        if out is None:
            y = _new_like(x, m, d)
            sy = d
        else:
            sy = _row_stride(y, m, d, what, "out")
        if save:
            gate = x.new_empty(m, f)
            up = x.new_empty(m, f)
            gp, upp = gate.data_ptr(), up.data_ptr()
        on.made(None if out is not None else y, gate, up)
        _check(lib().prism_gated_ffn_fwd(ctypes.byref(w), m, _ACT[act], code, x.data_ptr(), sx, y.data_ptr(), sy, gp, upp,
                                         ws.start, ws.nbytes, on.ptr), what)
    return y, gate, up


def gated_ffn_bwd(dy: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
                  gate: torch.Tensor, up: torch.Tensor, act: str = "silu", need_dx: bool = True, need_dw: bool = True,
                  ws: Optional[Workspace] = None, stream=None):
    """Gradient of ``gated_ffn_fwd`` at its saved projections: (dx, dw_gate, dw_up, dw_down); without ``need_dx`` or
    ``need_dw`` None in their places."""
    what = "prism_gated_ffn_bwd"
    if act not in _ACT:
        _require(False, f"{what}: act {act!r}")
    every = (dy, x, w_gate, w_up, w_down, gate, up)
    code = _same_type(every, what)
    w, d, f = _ffn_weights(w_gate, w_up, w_down, what)
    m = x.shape[0] if x.dim() else 0
    sx, sdy = _row_stride(x, m, d, what, "x"), _row_stride(dy, m, d, what, "dy")
    for t in (gate, up):
        if t.shape != (m, f) or not t.is_contiguous():
            _require(False, what + ": gate and up must be contiguous [m, f]")
    with _On(every, stream, what) as on:
        ws = on.workspace(ws, _ffn_workspace_bytes(m, f, 1), what)
        dx = dwg = dwu = dwd = xp = gp = upp = dp = None
        if need_dx:
            dx = _new_like(x, m, d)
            xp = dx.data_ptr()
        if need_dw:
            dwg, dwu, dwd = _new_like(w_gate, f, d), _new_like(w_up, f, d), _new_like(w_down, d, f)
            gp, upp, dp = dwg.data_ptr(), dwu.data_ptr(), dwd.data_ptr()
        on.made(dx, dwg, dwu, dwd)
        _check(lib().prism_gated_ffn_bwd(ctypes.byref(w), m, _ACT[act], code, dy.data_ptr(), sdy, x.data_ptr(), sx,
                                         gate.data_ptr(), up.data_ptr(), xp, d, gp, upp, dp, ws.start, ws.nbytes, on.ptr), what)
    return dx, dwg, dwu, dwd


_NORM = {2: 0, 2.0: 0, "l2": 0, math.inf: 1, "inf": 1}


def _dense(t: torch.Tensor) -> bool:
    """Whether the values fill one run of memory, in any order of the dimensions."""
    if t.is_contiguous():
        return True
    run = 1
    for stride, size in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n != 1):
        if stride != run:
            return False
        run *= size
    return True


class GradList:
    """A list of gradients (and where their scaled values go) for ``grad_norm``, ``scale_grads`` and
    ``clip_grad_norm``, laid out once: a program whose gradients stay in place keeps it from step to step. It holds
    the tensors, so their memory stays theirs. grads: dense bf16 / fp32 tensors of one device, any mix, in any order of
    their dimensions; out: None (in place) or one tensor for each, of its shape, strides and type."""

    def __init__(self, grads: Sequence[torch.Tensor], out: Optional[Sequence[torch.Tensor]] = None):
        self.grads = list(grads)
        self.out = None if out is None else list(out)
        n = len(self.grads)
        _require(self.out is None or len(self.out) == n, "GradList: as many outputs as gradients")
        self.device = self.grads[0].device if n else None
        self._c = (_Tensor * max(n, 1))()
        for i, t in enumerate(self.grads):
            _require(_dense(t), "GradList: gradients must be dense")
            _require(t.device == self.device, "GradList: gradients on different devices")
            o = None
            if self.out is not None:
                o = self.out[i]
                _require(o.shape == t.shape and o.dtype == t.dtype and o.device == self.device and
                         (o.stride() == t.stride() or (o.is_contiguous() and t.is_contiguous())),
                         "GradList: an output is not like its gradient")
                o = o.data_ptr()
            self._c[i] = (t.data_ptr(), o, t.numel(), _dtype_code(t), 0)
        b = _SZ()
        _check(lib().prism_grad_norm_workspace_size(n, ctypes.byref(b)), "prism_grad_norm_workspace_size")
        self.n, self.workspace_bytes = n, int(b.value)


def _grad_list(grads, out=None) -> GradList:
    if isinstance(grads, GradList):
        _require(out is None, "the GradList has its outputs already")
        return grads
    return GradList(grads, out)


def _norm_call(grads, ws, device, stream, what, call):
    """The norm that `call` (workspace, norm, stream) writes."""
    tensors = grads.grads[:1] or [torch.empty(0, device=device)]
    with _On(tensors, stream, what) as on:
        ws = on.workspace(ws, grads.workspace_bytes, what)
        norm = tensors[0].new_empty((), dtype=torch.float32)
        on.made(norm)
        _check(call(ws, norm.data_ptr(), on.ptr), what)
    return norm


def grad_norm(grads, ord=2, ws: Optional[Workspace] = None, device="cuda", stream=None) -> torch.Tensor:
    """Global norm (2 or inf) over a list of gradients or a ``GradList``, a device fp32 scalar. ``device`` is read for
    an empty list only."""
    grads = _grad_list(grads)
    _require(ord in _NORM, f"prism_grad_norm: ord {ord!r}")
    return _norm_call(grads, ws, device, stream, "prism_grad_norm", lambda ws, norm, ptr: lib().prism_grad_norm(
        grads._c, grads.n, _NORM[ord], norm, ws.start, ws.nbytes, ptr))


def scale_grads(grads, norm: torch.Tensor, max_norm: float, out=None, eps: float = 1e-6, stream=None):
    """Multiplies every gradient by min(1, max_norm / (norm + eps)), ``norm`` a device fp32 scalar (for example the
    root of the sum of ``grad_norm`` squared over the ranks of a sharded layer). In place, or into ``out``."""
    grads = _grad_list(grads, out)
    _require(norm.dtype == torch.float32 and norm.numel() == 1, "prism_grad_scale: norm must be one fp32 value", 3)
    with _On(grads.grads[:1] + [norm], stream, "prism_grad_scale") as on:
        _check(lib().prism_grad_scale(grads._c, grads.n, _ptr(norm), float(max_norm), float(eps), on.ptr),
               "prism_grad_scale")


def clip_grad_norm(grads, max_norm: float, ord=2, out=None, eps: float = 1e-6, ws: Optional[Workspace] = None,
                   device="cuda", stream=None) -> torch.Tensor:
    """``grad_norm`` and ``scale_grads`` of a list of gradients or a ``GradList``: returns the norm before clipping."""
    grads = _grad_list(grads, out)
    if ord not in _NORM:
        _require(False, f"prism_grad_clip: ord {ord!r}")
    return _norm_call(grads, ws, device, stream, "prism_grad_clip", lambda ws, norm, ptr: lib().prism_grad_clip(
        grads._c, grads.n, _NORM[ord], float(max_norm), float(eps), norm, ws.start, ws.nbytes, ptr))


def default_scale(head_dim: int) -> float:
    return 1.0 / math.sqrt(head_dim)
