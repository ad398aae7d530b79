"""Thin ctypes binding of libqlora (include/qlora.h), same names as the C ABI.

Argument marshalling only: every step of the computation runs in the HIP
library. PyTorch provides device memory (outputs and workspaces are
allocated here with torch) and the stream (torch's current stream).
If libqlora.so is missing, every call raises: there is no fallback.
"""

from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass
from typing import Optional, Tuple

HERE = os.path.dirname(os.path.abspath(__file__))
# Always the in-tree build next to this file (python -m
# quantized_frozen_weight_amd.build_lib); no other copy is ever loaded.
LIB_PATH = os.path.join(HERE, "libqlora.so")

QLORA_OK, QLORA_EINVAL, QLORA_EUNSUPPORTED, QLORA_EWORKSPACE, QLORA_ERANGE, QLORA_EHIP = range(6)
QLORA_F32, QLORA_BF16 = 0, 1
QLORA_W8, QLORA_W4G128, QLORA_W8O = 0, 1, 2

_ACT = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}      # qlora_act
_CFMT = {"c8row": 0, "c8g32": 1}                                         # qlora_cfmt
CKPT_GROUP = 32          # columns per scale of a "c8g32" checkpoint

_FMT = {"w8": QLORA_W8, "w4g128": QLORA_W4G128, "w8o": QLORA_W8O}


class QloraError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {qlora_status_str(status)} ({status})")


class qlora_linear(ctypes.Structure):
    _fields_ = [
        ("K", ctypes.c_int32),
        ("N", ctypes.c_int32),
        ("r", ctypes.c_int32),
        ("alpha", ctypes.c_float),
        ("fmt", ctypes.c_int32),
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("A", ctypes.c_void_p),
        ("B", ctypes.c_void_p),
        ("heads", ctypes.c_int32),
    ]


_lib = None

EXPORTS = (
    "qlora_status_str", "qlora_weight_bytes", "qlora_quantize",
    "qlora_fwd_workspace", "qlora_fwd", "qlora_bwd_workspace", "qlora_bwd",
    "qlora_quantize_rows", "qlora_fwd_acc", "qlora_fwd_timed", "qlora_bwd_timed",
    "qlora_merge", "qlora_bwd_partial", "qlora_bwd_finish", "qlora_fwd_a8w4",
    "qlora_quantize_heads", "qlora_outlier_layout", "qlora_bwd_finish_batch",
    "qlora_bwd_partials_bytes", "qlora_bwd_main_kernel", "qlora_bwd_noalloc",
    "qlora_ckpt_bytes", "qlora_ckpt_write", "qlora_ckpt_read", "qlora_fwd_epi",
    "qlora_fwd_ckpt", "qlora_bwd_epi", "qlora_bwd_epi_partial", "qlora_bwd_epi_workspace",
    "qlora_act_bwd_workspace", "qlora_act_bwd",
)
QLORA_NOALLOC_SCRATCH_BYTES = 16 << 20
# include/qlora_probe.h: measurement probes (not part of the layer)
PROBE_EXPORTS = ("qlora_probe_mfma", "qlora_probe_copy", "qlora_probe_read", "qlora_probe_empty")
QLORA_PROBE_BF16, QLORA_PROBE_I8 = 0, 1


class qlora_finish_item(ctypes.Structure):
    _fields_ = [
        ("L", ctypes.c_void_p),
        ("M", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("dA", ctypes.c_void_p),
        ("dB", ctypes.c_void_p),
        ("ws", ctypes.c_void_p),
        ("ws_bytes", ctypes.c_size_t),
    ]


class qlora_epilogue(ctypes.Structure):
    _fields_ = [
        ("act", ctypes.c_int32),
        ("bias", ctypes.c_void_p),
        ("residual", ctypes.c_void_p),
        ("z", ctypes.c_void_p),
        ("z_codes", ctypes.c_void_p),
        ("z_scales", ctypes.c_void_p),
        ("x_codes", ctypes.c_void_p),
        ("x_scales", ctypes.c_void_p),
    ]


class qlora_grad_epilogue(ctypes.Structure):
    _fields_ = [
        ("act", ctypes.c_int32),
        ("z", ctypes.c_void_p),
        ("z_codes", ctypes.c_void_p),
        ("z_scales", ctypes.c_void_p),
        ("add", ctypes.c_void_p),
    ]


def lib() -> ctypes.CDLL:
    """Load libqlora.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with "
            "`python -m quantized_frozen_weight_amd.build_lib`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    psz = ctypes.POINTER(ctypes.c_size_t)
    plin = ctypes.POINTER(qlora_linear)
    L.qlora_status_str.argtypes = [i]
    L.qlora_status_str.restype = ctypes.c_char_p
    L.qlora_weight_bytes.argtypes = [i, i, i, psz, psz]
    L.qlora_quantize.argtypes = [vp, i, i, i, vp, vp, vp]
    L.qlora_fwd_workspace.argtypes = [plin, i, i, psz]
    L.qlora_fwd.argtypes = [plin, i, i, vp, vp, vp, vp, sz, vp]
    L.qlora_bwd_workspace.argtypes = [plin, i, i, psz]
    L.qlora_bwd.argtypes = [plin, i, i, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.qlora_quantize_rows.argtypes = [vp, i, i, i, vp, vp, vp]
    L.qlora_fwd_acc.argtypes = [plin, i, i, vp, vp, vp, sz, vp]
    L.qlora_fwd_timed.argtypes = [plin, i, i, vp, vp, vp, vp, sz, vp, i, vp, vp]
    L.qlora_bwd_timed.argtypes = [plin, i, i, vp, vp, vp, vp, vp, vp, vp, sz, vp, i, vp, vp]
    L.qlora_merge.argtypes = [plin, vp, vp, vp]
    L.qlora_bwd_partial.argtypes = [plin, i, i, vp, vp, vp, vp, vp, sz, vp]
    L.qlora_bwd_finish.argtypes = [plin, i, i, vp, vp, vp, sz, vp]
    L.qlora_bwd_finish_batch.argtypes = [ctypes.POINTER(qlora_finish_item), i, vp]
    L.qlora_bwd_partials_bytes.argtypes = [plin, i, i, psz]
    L.qlora_fwd_a8w4.argtypes = [plin, i, i, vp, vp, vp, vp, sz, vp]
    L.qlora_quantize_heads.argtypes = [vp, i, i, i, i, vp, vp, vp]
    L.qlora_outlier_layout.argtypes = [i, i, psz, psz, psz, ctypes.POINTER(ctypes.c_int32)]
    L.qlora_bwd_main_kernel.argtypes = [plin, i, i]
    L.qlora_bwd_noalloc.argtypes = [plin, i, i, vp, vp, vp, vp, vp, vp, vp]
    L.qlora_ckpt_bytes.argtypes = [i, i, i, psz, psz]
    L.qlora_ckpt_write.argtypes = [vp, i, i, i, i, vp, vp, vp]
    L.qlora_ckpt_read.argtypes = [vp, vp, i, i, i, i, vp, vp]
    pepi, pge = ctypes.POINTER(qlora_epilogue), ctypes.POINTER(qlora_grad_epilogue)
    L.qlora_fwd_epi.argtypes = [plin, i, i, vp, pepi, vp, vp, vp, sz, vp]
    L.qlora_fwd_ckpt.argtypes = [plin, i, i, vp, vp, vp, pepi, vp, vp, sz, vp]
    L.qlora_bwd_epi.argtypes = [plin, i, i, vp, vp, vp, vp, vp, pge, vp, vp, vp, vp, sz, vp]
    L.qlora_bwd_epi_partial.argtypes = [plin, i, i, vp, vp, vp, vp, vp, pge, vp, vp, sz, vp]
    L.qlora_bwd_epi_workspace.argtypes = [plin, i, i, psz]
    L.qlora_act_bwd_workspace.argtypes = [i, i, psz]
    L.qlora_act_bwd.argtypes = [i, i, i, i, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    for name in EXPORTS[1:]:
        getattr(L, name).restype = ctypes.c_int
    L.qlora_bwd_main_kernel.restype = ctypes.c_char_p
    L.qlora_probe_mfma.argtypes = [i, i, i, vp, vp, ctypes.POINTER(ctypes.c_double)]
    L.qlora_probe_copy.argtypes = [vp, vp, sz, i, vp]
    L.qlora_probe_read.argtypes = [vp, sz, i, vp, vp]
    L.qlora_probe_empty.argtypes = [i, i, vp]
    for name in PROBE_EXPORTS:
        getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def loaded_path() -> str:
    """Path of the libqlora.so this process has mapped (from
    /proc/self/maps), after lib() has loaded it; '' if none is mapped."""
    lib()
    with open("/proc/self/maps") as f:
        for line in f:
            if line.rstrip().endswith("/libqlora.so"):
                return line.split()[-1]
    return ""


def qlora_bwd_main_kernel(layer: "QLinear", M: int, dtype: int) -> str:
    """Name of the kernel qlora_bwd_timed times for this layer (static)."""
    s = layer.cstruct()
    name = lib().qlora_bwd_main_kernel(ctypes.byref(s), M, dtype)
    if name is None:
        raise QloraError(QLORA_EINVAL, "qlora_bwd_main_kernel")
    return name.decode()


def _check(status: int, what: str) -> None:
    if status != QLORA_OK:
        raise QloraError(status, what)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream() -> int:
    """The current device's current stream."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:            # the handle without a Stream object around it
        return raw(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return QLORA_F32
    if t.dtype == torch.bfloat16:
        return QLORA_BF16
    raise TypeError(f"unsupported activation dtype {t.dtype}")


def qlora_status_str(status: int) -> str:
    return lib().qlora_status_str(int(status)).decode()


def qlora_weight_bytes(K: int, N: int, fmt: str = "w8") -> Tuple[int, int]:
    cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().qlora_weight_bytes(K, N, _FMT[fmt], ctypes.byref(cb), ctypes.byref(sb)),
           "qlora_weight_bytes")
    return cb.value, sb.value


@dataclass
class QLinear:
    """A frozen quantized weight plus its adapter (device tensors)."""
    K: int
    N: int
    r: int
    alpha: float
    fmt: str
    codes: object     # int8 [N, K]  or uint8 [N, K/2]
    scales: object    # float32 [N], float16 [N, K/128], or the w8o side buffer (uint8)
    A: object         # float32 [K, r]
    B: object         # float32 [r, N], or [heads, r, N / heads]
    heads: int = 1

    def cstruct(self) -> qlora_linear:
        return qlora_linear(self.K, self.N, self.r, float(self.alpha), _FMT[self.fmt],
                            _ptr(self.codes), _ptr(self.scales), _ptr(self.A),
                            _ptr(self.B), int(self.heads))


def _b_shape(layer: QLinear):
    """Shape of B and dB: [r, N], or [heads, r, N / heads]."""
    if layer.heads > 1:
        return (layer.heads, layer.r, layer.N // layer.heads)
    return (layer.r, layer.N)


def qlora_quantize(W, fmt: str = "w8"):
    """W float32 [K, N], or per head [heads, K, hd] (N = heads * hd), on the
    GPU -> (codes, scales) in the library's layout."""
    import torch
    if W.dim() == 3:
        heads, K, hd = W.shape
        N = heads * hd
    else:
        heads, (K, N) = 1, W.shape
    cb, sb = qlora_weight_bytes(K, N, fmt)
    if fmt == "w8":
        codes = torch.empty((N, K), dtype=torch.int8, device=W.device)
        scales = torch.empty((N,), dtype=torch.float32, device=W.device)
    elif fmt == "w8o":
        codes = torch.empty((N, K), dtype=torch.int8, device=W.device)
        scales = torch.empty((sb,), dtype=torch.uint8, device=W.device)
    else:
        codes = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device)
        scales = torch.empty((N, K // 128), dtype=torch.float16, device=W.device)
    assert codes.numel() * codes.element_size() == cb
    assert scales.numel() * scales.element_size() == sb
    W = W.contiguous()
    _check(lib().qlora_quantize_heads(_ptr(W), heads, K, N, _FMT[fmt], _ptr(codes),
                                      _ptr(scales), _stream()), "qlora_quantize_heads")
    return codes, scales


def qlora_outlier_layout(K: int, N: int) -> Tuple[int, int, int, int]:
    """(rowptr, col, val) byte offsets of a w8o side buffer's outlier list,
    and its capacity."""
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    cap = ctypes.c_int32()
    _check(lib().qlora_outlier_layout(K, N, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c),
                                      ctypes.byref(cap)), "qlora_outlier_layout")
    return a.value, b.value, c.value, cap.value


def qlora_outliers(side, K: int, N: int):
    """Read a w8o side buffer back (device -> host): (header dict with lo, hi,
    scale, nnz; rowptr int32 [K + 1]; col int32 [nnz]; val float16 [nnz])."""
    import numpy as np
    ro, co, vo, _ = qlora_outlier_layout(K, N)
    raw = side.cpu().numpy()
    hdr = raw[:16].view(np.float32)
    nnz = int(raw[12:16].view(np.int32)[0])
    head = dict(lo=hdr[0], hi=hdr[1], scale=hdr[2], nnz=nnz)
    rowptr = raw[ro:ro + 4 * (K + 1)].view(np.int32).copy()
    col = raw[co:co + 4 * nnz].view(np.int32).copy()
    val = raw[vo:vo + 2 * nnz].view(np.float16).copy()
    return head, rowptr, col, val


def qlora_merge(layer: QLinear):
    """The adapter merged into the layer's int8 weight, re-quantized: new
    (codes int8 [N, K], scales float32 [N]) on the layer's device."""
    import torch
    codes = torch.empty((layer.N, layer.K), dtype=torch.int8, device=layer.codes.device)
    scales = torch.empty((layer.N,), dtype=torch.float32, device=layer.codes.device)
    s = layer.cstruct()
    _check(lib().qlora_merge(ctypes.byref(s), _ptr(codes), _ptr(scales), _stream()),
           "qlora_merge")
    return codes, scales


def qlora_fwd_workspace(layer: QLinear, M: int, dtype: int) -> int:
    n = ctypes.c_size_t()
    s = layer.cstruct()
    _check(lib().qlora_fwd_workspace(ctypes.byref(s), M, dtype, ctypes.byref(n)),
           "qlora_fwd_workspace")
    return n.value


def qlora_bwd_workspace(layer: QLinear, M: int, dtype: int) -> int:
    n = ctypes.c_size_t()
    s = layer.cstruct()
    _check(lib().qlora_bwd_workspace(ctypes.byref(s), M, dtype, ctypes.byref(n)),
           "qlora_bwd_workspace")
    return n.value


def _workspace(nbytes: int, device, ws=None):
    import torch
    if ws is not None:
        return ws
    return torch.empty((max(nbytes, 256),), dtype=torch.uint8, device=device)


def qlora_fwd(layer: QLinear, x, save_t: bool = True, y=None, t=None, ws=None):
    """y = x deq(W) + s (x A) B. Returns (y, t) (t is None if not saved)."""
    import torch
    M = x.shape[0]
    dt = _dtype_code(x)
    if y is None:
        y = torch.empty((M, layer.N), dtype=x.dtype, device=x.device)
    if save_t and t is None:
        t = torch.empty((M, layer.r), dtype=torch.float32, device=x.device)
    nbytes = qlora_fwd_workspace(layer, M, dt)
    ws = _workspace(nbytes, x.device, ws)
    s = layer.cstruct()
    _check(lib().qlora_fwd(ctypes.byref(s), M, dt, _ptr(x), _ptr(y),
                           _ptr(t) if save_t else None, _ptr(ws),
                           ws.numel() * ws.element_size(), _stream()), "qlora_fwd")
    return y, (t if save_t else None)


def qlora_fwd_a8w4(layer: QLinear, x, save_t: bool = True, y=None, t=None, ws=None):
    """Integer forward of a 4-bit layer with int8 activations: (y, t or None)."""
    import torch
    M = x.shape[0]
    dt = _dtype_code(x)
    if y is None:
        y = torch.empty((M, layer.N), dtype=x.dtype, device=x.device)
    if save_t and t is None:
        t = torch.empty((M, layer.r), dtype=torch.float32, device=x.device)
    ws = _workspace(qlora_fwd_workspace(layer, M, dt), x.device, ws)
    s = layer.cstruct()
    _check(lib().qlora_fwd_a8w4(ctypes.byref(s), M, dt, _ptr(x), _ptr(y),
                                _ptr(t) if save_t else None, _ptr(ws),
                                ws.numel() * ws.element_size(), _stream()),
           "qlora_fwd_a8w4")
    return y, (t if save_t else None)


def qlora_bwd(layer: QLinear, x, dy, t=None, need_dx: bool = True, dx=None,
              dA=None, dB=None, ws=None):
    """Returns (dx or None, dA [K, r], dB [r, N])."""
    import torch
    M = x.shape[0]
    dt = _dtype_code(x)
    if need_dx and dx is None:
        dx = torch.empty((M, layer.K), dtype=x.dtype, device=x.device)
    if dA is None:
        dA = torch.empty((layer.K, layer.r), dtype=torch.float32, device=x.device)
    if dB is None:
        dB = torch.empty(_b_shape(layer), dtype=torch.float32, device=x.device)
    nbytes = qlora_bwd_workspace(layer, M, dt)
    ws = _workspace(nbytes, x.device, ws)
    s = layer.cstruct()
    _check(lib().qlora_bwd(ctypes.byref(s), M, dt, _ptr(x), _ptr(dy), _ptr(t),
                           _ptr(dx) if need_dx else None, _ptr(dA), _ptr(dB),
                           _ptr(ws), ws.numel() * ws.element_size(), _stream()),
           "qlora_bwd")
    return (dx if need_dx else None), dA, dB


def qlora_bwd_partial(layer: QLinear, x, dy, t=None, need_dx: bool = True, dx=None,
                      ws=None, stream=None):
    """First half of qlora_bwd: dx (or None) and the adapter-gradient partial
    sums, which stay in the returned workspace for qlora_bwd_finish."""
    import torch
    M = x.shape[0]
    dt = _dtype_code(x)
    if need_dx and dx is None:
        dx = torch.empty((M, layer.K), dtype=x.dtype, device=x.device)
    ws = _workspace(qlora_bwd_workspace(layer, M, dt), x.device, ws)
    s = layer.cstruct()
    _check(lib().qlora_bwd_partial(ctypes.byref(s), M, dt, _ptr(x), _ptr(dy), _ptr(t),
                                   _ptr(dx) if need_dx else None, _ptr(ws),
                                   ws.numel() * ws.element_size(),
                                   _stream() if stream is None else stream.cuda_stream),
           "qlora_bwd_partial")
    return (dx if need_dx else None), ws


def qlora_bwd_partials_bytes(layer: QLinear, M: int, dtype: int) -> int:
    """Leading bytes of a backward workspace that outlive qlora_bwd_partial."""
    n = ctypes.c_size_t()
    s = layer.cstruct()
    _check(lib().qlora_bwd_partials_bytes(ctypes.byref(s), M, dtype, ctypes.byref(n)),
           "qlora_bwd_partials_bytes")
    return n.value


def qlora_bwd_finish_batch(items, stream=None):
    """qlora_bwd_finish for several layers in one launch (per 32 layers).
    items: (layer, M, dtype, ws) or (layer, M, dtype, ws, dA, dB) tuples, each
    ws holding that layer's qlora_bwd_partial results. The items' partial
    sums (the first qlora_bwd_partials_bytes of each ws) must not overlap;
    the scratch past them may (packed workspaces).
    Returns the list of (dA, dB)."""
    import torch
    arr = (qlora_finish_item * len(items))()
    keep, out = [], []
    for n, it in enumerate(items):
        layer, M, dtype, ws = it[:4]
        dA = it[4] if len(it) > 4 else None
        dB = it[5] if len(it) > 5 else None
        if dA is None:
            dA = torch.empty((layer.K, layer.r), dtype=torch.float32, device=ws.device)
        if dB is None:
            dB = torch.empty(_b_shape(layer), dtype=torch.float32, device=ws.device)
        s = layer.cstruct()
        keep.append(s)
        arr[n] = qlora_finish_item(ctypes.cast(ctypes.pointer(s), ctypes.c_void_p), M,
                                   QLORA_F32 if dtype == torch.float32 else QLORA_BF16,
                                   _ptr(dA), _ptr(dB), _ptr(ws), ws.numel() * ws.element_size())
        out.append((dA, dB))
    _check(lib().qlora_bwd_finish_batch(arr, len(items),
                                        _stream() if stream is None else stream.cuda_stream),
           "qlora_bwd_finish_batch")
    return out


def qlora_bwd_finish(layer: QLinear, M: int, dtype, ws, dA=None, dB=None, stream=None):
    """Second half of qlora_bwd: dA [K, r] and dB [r, N] from the partial sums
    that qlora_bwd_partial left in ws. dtype: the activations' torch dtype."""
    import torch
    dt = QLORA_F32 if dtype == torch.float32 else QLORA_BF16
    if dA is None:
        dA = torch.empty((layer.K, layer.r), dtype=torch.float32, device=ws.device)
    if dB is None:
        dB = torch.empty(_b_shape(layer), dtype=torch.float32, device=ws.device)
    s = layer.cstruct()
    _check(lib().qlora_bwd_finish(ctypes.byref(s), M, dt, _ptr(dA), _ptr(dB), _ptr(ws),
                                  ws.numel() * ws.element_size(),
                                  _stream() if stream is None else stream.cuda_stream),
           "qlora_bwd_finish")
    return dA, dB


def qlora_quantize_rows(x):
    """Test hook: (xq int8 [M, K], sx float32 [M]) from the forward's quantizer."""
    import torch
    M, K = x.shape
    xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    sx = torch.empty((M,), dtype=torch.float32, device=x.device)
    _check(lib().qlora_quantize_rows(_ptr(x), M, K, _dtype_code(x), _ptr(xq), _ptr(sx),
                                     _stream()), "qlora_quantize_rows")
    return xq, sx


def qlora_fwd_acc(layer: QLinear, x):
    """Test hook: exact int32 product of the quantized rows and codes [M, N]."""
    import torch
    M = x.shape[0]
    dt = _dtype_code(x)
    acc = torch.empty((M, layer.N), dtype=torch.int32, device=x.device)
    ws = _workspace(qlora_fwd_workspace(layer, M, dt), x.device)
    s = layer.cstruct()
    _check(lib().qlora_fwd_acc(ctypes.byref(s), M, dt, _ptr(x), _ptr(acc), _ptr(ws),
                               ws.numel() * ws.element_size(), _stream()),
           "qlora_fwd_acc")
    return acc


# ---------------------------------------------------------------------------
# The layer with its epilogue, and 8-bit activation checkpoints. These calls
# run on the device their tensors are on (that device's current stream) and
# raise ValueError / TypeError for tensors the C ABI could not check.
# ---------------------------------------------------------------------------
@dataclass
class Checkpoint:
    """An activation [M, C] in 8 bits: codes int8 [M, C] and its scales,
    float32 [M] ("c8row") or uint8 [M, ceil(C / 32)] ("c8g32")."""
    codes: object
    scales: object
    fmt: str

    @property
    def shape(self):
        return self.codes.shape


class _here:
    """Context that changes nothing: the device is the current one."""
    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_HERE = _here()


def _on(device):
    """Context in which `device` is the current one."""
    import torch
    if device.index == torch.cuda.current_device():
        return _HERE
    return torch.cuda.device(device)


def _tensor(t, what: str, shape, dtype, device):
    """t, checked to be a dense tensor of this shape, type and device."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t
    if t.dtype != dtype:
        raise TypeError(f"{what}: {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    raise ValueError(f"{what}: not contiguous")


def _rows(x, what: str, columns=None):
    """(M, C, dtype code) of a dense [M, C] activation on a GPU."""
    shape = x.shape
    if len(shape) != 2 or not x.is_cuda or not x.is_contiguous():
        raise ValueError(f"{what}: a contiguous 2-D GPU tensor is needed")
    if columns is not None and shape[1] != columns:
        raise ValueError(f"{what}: {shape[1]} columns, expected {columns}")
    return shape[0], shape[1], _dtype_code(x)


def _ckpt(c, what: str, fmt: str, shape, device) -> Checkpoint:
    import torch
    if c.fmt != fmt:
        raise ValueError(f"{what}: form {c.fmt!r}, expected {fmt!r}")
    if fmt not in _CFMT:
        raise ValueError(f"{what}: unknown checkpoint form {fmt!r}")
    _tensor(c.codes, f"{what}.codes", shape, torch.int8, device)
    if fmt == "c8row":
        _tensor(c.scales, f"{what}.scales", (shape[0],), torch.float32, device)
    else:
        _tensor(c.scales, f"{what}.scales", (shape[0], -(-shape[1] // CKPT_GROUP)), torch.uint8, device)
    return c


def _new_ckpt(M: int, C: int, fmt: str, like) -> Checkpoint:
    """A checkpoint's tensors on the device of `like`."""
    import torch
    if fmt not in _CFMT:
        raise ValueError(f"unknown checkpoint form {fmt!r}")
    codes = like.new_empty((M, C), dtype=torch.int8)
    if fmt == "c8row":
        scales = like.new_empty((M,), dtype=torch.float32)
    else:
        scales = like.new_empty((M, -(-C // CKPT_GROUP)), dtype=torch.uint8)
    return Checkpoint(codes, scales, fmt)


@functools.lru_cache(maxsize=4096)
def _weight_form(K: int, N: int, fmt: str):
    """Shape and dtype of a layer's codes, then of its scales."""
    import torch
    if fmt == "w8":
        return (N, K), torch.int8, (N,), torch.float32
    if fmt == "w4g128":
        return (N, K // 2), torch.uint8, (N, K // 128), torch.float16
    if fmt == "w8o":
        return (N, K), torch.int8, (qlora_weight_bytes(K, N, fmt)[1],), torch.uint8
    raise ValueError(f"unknown weight form {fmt!r}")


def _layer_on(layer: QLinear, device) -> qlora_linear:
    """The layer's C struct, its four tensors checked."""
    import torch
    c, s, A, B = layer.codes, layer.scales, layer.A, layer.B
    cshape, ctype, sshape, stype = _weight_form(layer.K, layer.N, layer.fmt)
    f32 = torch.float32
    if (c.dtype is ctype and s.dtype is stype and A.dtype is f32 and B.dtype is f32
            and c.device == device and s.device == device and A.device == device and B.device == device
            and c.shape == cshape and s.shape == sshape and A.shape == (layer.K, layer.r)
            and B.shape == _b_shape(layer) and c.is_contiguous() and s.is_contiguous()
            and A.is_contiguous() and B.is_contiguous()):
        return layer.cstruct()
    _tensor(c, "layer codes", cshape, ctype, device)
    _tensor(s, "layer scales", sshape, stype, device)
    _tensor(A, "layer A", (layer.K, layer.r), f32, device)
    _tensor(B, "layer B", _b_shape(layer), f32, device)
    raise AssertionError("unreachable: one of the checks above fails")


def _unused(t, what: str, flag: str) -> None:
    if t is not None:
        raise ValueError(f"{what}: given, but {flag} does not ask for it")


def _act(act: str) -> int:
    if act not in _ACT:
        raise ValueError(f"unknown activation {act!r}")
    return _ACT[act]


@functools.lru_cache(maxsize=4096)
def _sizes(query: str, K: int, N: int, r: int, fmt: int, heads: int, M: int, dtype: int) -> int:
    """A workspace query's answer for these sizes (host arithmetic alone; the
    pointers only have to pass its checks)."""
    n = ctypes.c_size_t()
    s = qlora_linear(K, N, r, 1.0, fmt, 256, 256, 256, 256, heads)
    _check(getattr(lib(), query)(ctypes.byref(s), M, dtype, ctypes.byref(n)), query)
    return n.value


@functools.lru_cache(maxsize=4096)
def _act_bwd_bytes(M: int, N: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().qlora_act_bwd_workspace(M, N, ctypes.byref(n)), "qlora_act_bwd_workspace")
    return n.value


def _scratch(query: str, layer: QLinear, cs: qlora_linear, M: int, dtype: int, device, ws):
    """The caller's workspace, or a new one of the queried size (bytes, as the
    codes are)."""
    if ws is not None:
        if ws.device != device or not ws.is_contiguous():
            raise ValueError(f"ws: a contiguous tensor on {device} is needed")
        return ws
    n = _sizes(query, cs.K, cs.N, cs.r, cs.fmt, cs.heads, M, dtype)
    return layer.codes.new_empty((max(n, 256),))


def qlora_ckpt_write(x, fmt: str = "c8row", out: Optional[Checkpoint] = None) -> Checkpoint:
    """x [M, C] as an 8-bit checkpoint of form fmt."""
    M, C, dt = _rows(x, "x")
    c = _new_ckpt(M, C, fmt, x) if out is None else _ckpt(out, "out", fmt, (M, C), x.device)
    with _on(x.device):
        _check(lib().qlora_ckpt_write(_ptr(x), M, C, dt, _CFMT[fmt], _ptr(c.codes), _ptr(c.scales),
                                      _stream()), "qlora_ckpt_write")
    return c


def qlora_ckpt_read(ckpt: Checkpoint, dtype, out=None):
    """The values of a checkpoint in dtype (torch.float32 or torch.bfloat16)."""
    import torch
    M, C = ckpt.codes.shape
    dev = ckpt.codes.device
    _ckpt(ckpt, "ckpt", ckpt.fmt, (M, C), dev)
    if not ckpt.codes.is_cuda:
        raise ValueError("ckpt: GPU tensors are needed")
    x = torch.empty((M, C), dtype=dtype, device=dev) if out is None else _tensor(out, "out", (M, C), dtype, dev)
    with _on(dev):
        _check(lib().qlora_ckpt_read(_ptr(ckpt.codes), _ptr(ckpt.scales), M, C, _CFMT[ckpt.fmt],
                                     _dtype_code(x), _ptr(x), _stream()), "qlora_ckpt_read")
    return x


def _epilogue(layer, M, dtype, device, act, bias, residual, save_z, z, xc):
    """(C struct, z) of a forward epilogue."""
    import torch
    e = qlora_epilogue(act=_act(act))
    if bias is not None:
        e.bias = _ptr(_tensor(bias, "bias", (layer.N,), torch.float32, device))
    if residual is not None:
        e.residual = _ptr(_tensor(residual, "residual", (M, layer.N), dtype, device))
    if save_z == "full":
        z = torch.empty((M, layer.N), dtype=dtype, device=device) if z is None else \
            _tensor(z, "z", (M, layer.N), dtype, device)
        e.z = _ptr(z)
    elif save_z == "c8g32":
        z = _new_ckpt(M, layer.N, "c8g32", layer.A) if z is None else \
            _ckpt(z, "z", "c8g32", (M, layer.N), device)
        e.z_codes, e.z_scales = _ptr(z.codes), _ptr(z.scales)
    elif save_z is not None:
        raise ValueError(f"save_z: {save_z!r} is neither None, 'full' nor 'c8g32'")
    else:
        _unused(z, "z", "save_z")
    if xc is not None:
        e.x_codes, e.x_scales = _ptr(xc.codes), _ptr(xc.scales)
    return e, z


def qlora_fwd_epi(layer: QLinear, x, act: str = "none", bias=None, residual=None, save_t: bool = True,
                  save_z: Optional[str] = None, save_x: bool = False, y=None, t=None, z=None,
                  xc: Optional[Checkpoint] = None, ws=None):
    """y = act(x deq(W) + s (x A) B + bias) + residual. Returns (y, t, z, xc):
    t = x A (None unless save_t), z the pre-activation (save_z "full": in x's
    dtype, "c8g32": a Checkpoint, None: not saved) and xc x's row checkpoint
    (None unless save_x). y may be the residual tensor itself."""
    import torch
    M, _, dt = _rows(x, "x", layer.K)
    dev = x.device
    cs = _layer_on(layer, dev)
    y = x.new_empty((M, layer.N)) if y is None else \
        _tensor(y, "y", (M, layer.N), x.dtype, dev)
    if save_t:
        t = layer.A.new_empty((M, layer.r)) if t is None else \
            _tensor(t, "t", (M, layer.r), torch.float32, dev)
    else:
        _unused(t, "t", "save_t")
    if save_x:
        xc = _new_ckpt(M, layer.K, "c8row", x) if xc is None else _ckpt(xc, "xc", "c8row", (M, layer.K), dev)
    else:
        _unused(xc, "xc", "save_x")
    e, z = _epilogue(layer, M, x.dtype, dev, act, bias, residual, save_z, z, xc)
    ws = _scratch("qlora_fwd_workspace", layer, cs, M, dt, dev, ws)
    with _on(dev):
        _check(lib().qlora_fwd_epi(ctypes.byref(cs), M, dt, _ptr(x), ctypes.byref(e), _ptr(y),
                                   _ptr(t), _ptr(ws), ws.nbytes, _stream()), "qlora_fwd_epi")
    return y, t, z, xc


def qlora_fwd_ckpt(layer: QLinear, xc: Checkpoint, t, dtype, act: str = "none", bias=None, residual=None,
                   save_z: Optional[str] = None, y=None, z=None, ws=None):
    """qlora_fwd_epi's y (and z) again from x's row checkpoint and t; dtype is
    the activations' torch dtype. Returns (y, z)."""
    import torch
    M, dev = xc.codes.shape[0], xc.codes.device
    _ckpt(xc, "xc", "c8row", (M, layer.K), dev)
    if not xc.codes.is_cuda:
        raise ValueError("xc: GPU tensors are needed")
    _tensor(t, "t", (M, layer.r), torch.float32, dev)
    cs = _layer_on(layer, dev)
    y = torch.empty((M, layer.N), dtype=dtype, device=dev) if y is None else \
        _tensor(y, "y", (M, layer.N), dtype, dev)
    dt = _dtype_code(y)
    e, z = _epilogue(layer, M, dtype, dev, act, bias, residual, save_z, z, None)
    ws = _scratch("qlora_fwd_workspace", layer, cs, M, dt, dev, ws)
    with _on(dev):
        _check(lib().qlora_fwd_ckpt(ctypes.byref(cs), M, dt, _ptr(xc.codes), _ptr(xc.scales), _ptr(t),
                                    ctypes.byref(e), _ptr(y), _ptr(ws), ws.nbytes,
                                    _stream()), "qlora_fwd_ckpt")
    return y, z


def _bwd_epi_args(layer, x, dy, t, act, z, add, need_dx, dx):
    """The checked arguments that qlora_bwd_epi and its first half share."""
    import torch
    M, _, dt = _rows(dy, "dy", layer.N)
    dev, shape = dy.device, (M, layer.K)
    cs = _layer_on(layer, dev)
    xp = xcodes = xscales = None
    if isinstance(x, Checkpoint):
        _ckpt(x, "x", "c8row", shape, dev)
        if t is None:
            raise ValueError("t: needed with a checkpoint")
        xcodes, xscales = _ptr(x.codes), _ptr(x.scales)
    else:
        xp = _ptr(_tensor(x, "x", shape, dy.dtype, dev))
    if t is not None:
        _tensor(t, "t", (M, layer.r), torch.float32, dev)
    g = qlora_grad_epilogue(act=_act(act))
    if isinstance(z, Checkpoint):
        _ckpt(z, "z", "c8g32", shape, dev)
        g.z_codes, g.z_scales = _ptr(z.codes), _ptr(z.scales)
    elif z is not None:
        g.z = _ptr(_tensor(z, "z", shape, dy.dtype, dev))
    if add is not None:
        g.add = _ptr(_tensor(add, "add", shape, dy.dtype, dev))
    if need_dx:
        dx = dy.new_empty(shape) if dx is None else \
            _tensor(dx, "dx", shape, dy.dtype, dev)
    else:
        if act != "none" or z is not None or add is not None:
            raise ValueError("need_dx: act, z and add apply to dx")
        _unused(dx, "dx", "need_dx")
    gp = ctypes.byref(g) if need_dx else None
    return cs, M, dt, dev, (xp, xcodes, xscales, _ptr(dy), _ptr(t), gp, _ptr(dx)), dx, g


def qlora_bwd_epi(layer: QLinear, x, dy, t=None, act: str = "none", z=None, add=None, need_dx: bool = True,
                  dx=None, dA=None, dB=None, ws=None):
    """qlora_bwd with x a tensor or its row Checkpoint (t then required), and
    dx = (dy deq(W)^T + s u A^T) act'(z) + add, z a tensor or a "c8g32"
    Checkpoint. dx may be the add tensor itself. Returns (dx or None, dA, dB)."""
    import torch
    cs, M, dt, dev, args, dx, _keep = _bwd_epi_args(layer, x, dy, t, act, z, add, need_dx, dx)
    dA = layer.A.new_empty((layer.K, layer.r)) if dA is None else \
        _tensor(dA, "dA", (layer.K, layer.r), torch.float32, dev)
    dB = layer.B.new_empty(_b_shape(layer)) if dB is None else \
        _tensor(dB, "dB", _b_shape(layer), torch.float32, dev)
    ws = _scratch("qlora_bwd_epi_workspace", layer, cs, M, dt, dev, ws)
    with _on(dev):
        _check(lib().qlora_bwd_epi(ctypes.byref(cs), M, dt, *args, _ptr(dA), _ptr(dB), _ptr(ws),
                                   ws.nbytes, _stream()), "qlora_bwd_epi")
    return dx, dA, dB


def qlora_bwd_epi_partial(layer: QLinear, x, dy, t=None, act: str = "none", z=None, add=None,
                          need_dx: bool = True, dx=None, ws=None):
    """First half of qlora_bwd_epi: (dx or None, workspace), the adapter
    gradients left to qlora_bwd_finish or qlora_bwd_finish_batch."""
    cs, M, dt, dev, args, dx, _keep = _bwd_epi_args(layer, x, dy, t, act, z, add, need_dx, dx)
    ws = _scratch("qlora_bwd_epi_workspace", layer, cs, M, dt, dev, ws)
    with _on(dev):
        _check(lib().qlora_bwd_epi_partial(ctypes.byref(cs), M, dt, *args, _ptr(ws),
                                           ws.nbytes, _stream()),
               "qlora_bwd_epi_partial")
    return dx, ws


def qlora_act_bwd(act: str, dy, z=None, need_dz: bool = True, need_dbias: bool = True, dz=None, dbias=None,
                  ws=None):
    """dz = dy act'(z) and dbias = its float32 column sums, z a tensor or a
    "c8g32" Checkpoint. dz may be dy itself. Returns (dz or None, dbias or
    None); act "none" takes no z."""
    import torch
    M, N, dt = _rows(dy, "dy")
    dev = dy.device
    zp = zc = zs = None
    if isinstance(z, Checkpoint):
        _ckpt(z, "z", "c8g32", (M, N), dev)
        zc, zs = _ptr(z.codes), _ptr(z.scales)
    elif z is not None:
        zp = _ptr(_tensor(z, "z", (M, N), dy.dtype, dev))
    if need_dz:
        dz = torch.empty_like(dy) if dz is None else _tensor(dz, "dz", (M, N), dy.dtype, dev)
    else:
        _unused(dz, "dz", "need_dz")
    if need_dbias:
        dbias = torch.empty((N,), dtype=torch.float32, device=dev) if dbias is None else \
            _tensor(dbias, "dbias", (N,), torch.float32, dev)
        if ws is None:
            need = _act_bwd_bytes(M, N)
            ws = torch.empty((need,), dtype=torch.uint8, device=dev) if need else None
        elif ws.device != dev or not ws.is_contiguous():
            raise ValueError(f"ws: a contiguous tensor on {dev} is needed")
    else:
        _unused(dbias, "dbias", "need_dbias")
        ws = None
    with _on(dev):
        _check(lib().qlora_act_bwd(_act(act), M, N, dt, _ptr(dy), zp, zc, zs, _ptr(dz), _ptr(dbias),
                                   _ptr(ws), 0 if ws is None else ws.nbytes,
                                   _stream()), "qlora_act_bwd")
    return dz, dbias
