"""ctypes binding of libfa.so: argument marshalling only.

Names and argument order follow ``include/fa.h``.  Tensors must be CUDA bf16
(inputs/outputs) or fp32 (lse, D) and contiguous; the functions allocate the
outputs with PyTorch when they are not given.  Calls are asynchronous on the
current PyTorch stream of the tensors' device unless ``stream`` is given.  All
tensors of one call must live on one GPU; that GPU is made current for the
call (the library launches on the current device).
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = os.path.join(_HERE, "_build", "libfa.so")
_lock = threading.Lock()
_lib = None

FA_OK = 0
STATUS_NAMES = {
    0: "FA_OK", -1: "FA_ERR_NULL", -2: "FA_ERR_SHAPE", -3: "FA_ERR_HEADDIM", -4: "FA_ERR_ALIGN",
    -5: "FA_ERR_ARCH", -6: "FA_ERR_WORKSPACE", -7: "FA_ERR_CUDA", -8: "FA_ERR_DEVICE_TIMEOUT",
}


class _CacheStruct(ctypes.Structure):
    """fa_cache of include/fa.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("B", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("cap", ctypes.c_int), ("d", ctypes.c_int), ("format", ctypes.c_int)]


# fa_heads of include/fa.h, as the bytes that a call passes the address of (a third of what
# a ctypes structure costs; the small calls are as long as their Python).
_pack_heads = struct.Struct("Pqqqi4x").pack


class _RotationStruct(ctypes.Structure):
    """fa_rotation of include/fa.h."""
    _fields_ = [("turns", ctypes.c_void_p), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("amplitude", ctypes.c_float)]


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} "
                         f"({fa_status_string(status)})")


def library_path() -> str:
    return _LIB


def library():
    """Load libfa.so (raises if it has not been built: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB):
            raise ImportError(f"libfa.so not built ({_LIB}); run exact_io_aware_16_gb300/build.py")
        lib = ctypes.CDLL(_LIB)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.fa_forward.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        lib.fa_forward.restype = i
        lib.fa_backward_workspace_size.argtypes = [i, i, i, i]
        lib.fa_backward_workspace_size.restype = sz
        lib.fa_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, sz,
                                    vp]
        lib.fa_backward.restype = i
        ll = ctypes.c_longlong
        lib.fa_forward_blocksparse.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, ll, vp]
        lib.fa_forward_blocksparse.restype = i
        lib.fa_backward_blocksparse.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f,
                                                i, vp, ll, vp, sz, vp]
        lib.fa_backward_blocksparse.restype = i
        u64, u32 = ctypes.c_ulonglong, ctypes.c_uint
        lib.fa_forward_dropout.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, f, u64, u32, vp,
                                           ll, vp]
        lib.fa_forward_dropout.restype = i
        lib.fa_backward_dropout.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i,
                                            f, u64, u32, vp, ll, vp, sz, vp]
        lib.fa_backward_dropout.restype = i
        lib.fa_forward_fp8.argtypes = [vp, vp, vp, f, f, f, vp, vp, i, i, i, i, f, i, vp]
        lib.fa_forward_fp8.restype = i
        lib.fa_host_plan_create.argtypes = [i, i, i, i, f, i, ctypes.POINTER(vp)]
        lib.fa_host_plan_create.restype = i
        lib.fa_host_step.argtypes = [vp] * 10
        lib.fa_host_step.restype = i
        lib.fa_host_wait.argtypes = [vp]
        lib.fa_host_wait.restype = i
        lib.fa_host_plan_destroy.argtypes = [vp]
        lib.fa_host_plan_destroy.restype = i
        lib.fa_decode_workspace_size.argtypes = [i, i, i, i, i]
        lib.fa_decode_workspace_size.restype = sz
        lib.fa_decode.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, sz, vp]
        lib.fa_decode.restype = i
        pc = ctypes.POINTER(_CacheStruct)
        lib.fa_cache_write.argtypes = [pc, vp, vp, vp, vp, i, vp]
        lib.fa_cache_write.restype = i
        lib.fa_cache_read.argtypes = [pc, vp, vp, vp, vp, i, vp]
        lib.fa_cache_read.restype = i
        lib.fa_cache_commit.argtypes = [pc, vp, vp, vp, vp, i, vp]
        lib.fa_cache_commit.restype = i
        lib.fa_decode_tree_workspace_size.argtypes = [pc, i, i]
        lib.fa_decode_tree_workspace_size.restype = sz
        lib.fa_decode_tree.argtypes = [pc, vp, vp, vp, ll, vp, vp, i, i, f, vp, sz, vp]
        lib.fa_decode_tree.restype = i
        ph, pr, dbl = vp, ctypes.POINTER(_RotationStruct), ctypes.c_double
        for fn in (lib.fa_forward_packed_workspace_size, lib.fa_backward_packed_workspace_size):
            fn.argtypes = [i] * 6
            fn.restype = sz
        lib.fa_forward_packed.argtypes = [ph] * 4 + [vp] * 3 + [i] * 4 + [f, i, vp, sz, vp]
        lib.fa_forward_packed.restype = i
        lib.fa_backward_packed.argtypes = [ph] * 5 + [vp] + [ph] * 3 + [vp] * 2 + [i] * 4 + \
            [f, i, vp, sz, vp]
        lib.fa_backward_packed.restype = i
        lib.fa_rotary_table.argtypes = [vp, i, dbl, i, dbl, dbl, dbl, dbl]
        lib.fa_rotary_table.restype = i
        for fn in (lib.fa_rotary, lib.fa_rotary_backward):
            fn.argtypes = [pr] + [ph] * 4 + [vp, i, i, i, vp]
            fn.restype = i
        lib.fa_norm_rotary.argtypes = [pr] + [ph] * 4 + [vp] * 3 + [i, f, i, i, i, vp]
        lib.fa_norm_rotary.restype = i
        lib.fa_norm_rotary_backward.argtypes = [pr] + [ph] * 6 + [vp] * 5 + [i, f, i, i, i, vp, sz, vp]
        lib.fa_norm_rotary_backward.restype = i
        lib.fa_backward_preprocess.argtypes = [vp, vp, vp, i, i, i, i, vp]
        lib.fa_backward_preprocess.restype = i
        lib.fa_backward_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i,
                                             vp]
        lib.fa_backward_noalloc.restype = i
        lib.fa_backward_dkdv.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        lib.fa_backward_dkdv.restype = i
        lib.fa_backward_dq.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        lib.fa_selftest_wait_timeout.argtypes = [vp]
        lib.fa_selftest_wait_timeout.restype = i
        lib.fa_backward_dq.restype = i
        lib.fa_get_device_error.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
        lib.fa_get_device_error.restype = i
        lib.fa_status_string.argtypes = [i]
        lib.fa_status_string.restype = ctypes.c_char_p
        lib.fa_forward_tile_count.argtypes = [i, i]
        lib.fa_forward_tile_count.restype = ctypes.c_longlong
        _lib = lib
        return lib


def fa_status_string(status: int) -> str:
    return library().fa_status_string(int(status)).decode()


def _stream_handle(stream, device) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _on_device(t) -> bool:
    return bool(t.is_cuda)


def _device_index(t) -> int:
    return t.get_device()


def _one_device(*named):
    """The device index shared by every (tensor, name) given (None entries
    skipped): a tensor on another GPU would be read or written through an
    address the launching GPU may not map."""
    dev = _device_index(named[0][0])
    for t, nm in named[1:]:
        if t is not None and _device_index(t) != dev:
            raise ValueError(f"{nm} is on device {_device_index(t)}, the call's other tensors "
                             f"on device {dev}")
    return dev


def _device_guard(dev: int):
    """Makes device `dev` current for a library call when it is not already."""
    if dev < 0 or dev == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def _check(t, name, dtype, shape=None):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not _on_device(t):
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _check_grads(dq, dk, dv, shape):
    for t, nm in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        _check(t, nm, torch.bfloat16, shape)


def _check_workspace(ws):
    if not isinstance(ws, torch.Tensor) or not _on_device(ws) or not ws.is_contiguous() \
            or ws.dtype != torch.uint8:
        raise TypeError("workspace must be a contiguous uint8 CUDA tensor")


def fa_forward_tile_count(N: int, causal: bool) -> int:
    return int(library().fa_forward_tile_count(int(N), int(bool(causal))))


def fa_forward(q, k, v, causal: bool = False, scale: float | None = None, o=None, lse=None,
               stream=None):
    """O = softmax(scale q k^T) v and the per-row lse; q, k, v bf16 [B,H,N,d]."""
    B, H, N, d = q.shape
    for t, nm in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, nm, torch.bfloat16, (B, H, N, d))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check(o, "o", torch.bfloat16, (B, H, N, d))
    _check(lse, "lse", torch.float32, (B, H, N))
    dev = _one_device((q, "q"), (k, "k"), (v, "v"), (o, "o"), (lse, "lse"))
    with _device_guard(dev):
        st = library().fa_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                                  float(scale), int(bool(causal)),
                                  ctypes.c_void_p(_stream_handle(stream, q.device)))
    if st != FA_OK:
        raise FaError(st, "fa_forward")
    return o, lse


def _mask_args(mask, B, H, N):
    """(pointer, head stride) of a uint8 CUDA block mask [nt,nt] or [B*H,nt,nt]."""
    nt = -(-N // 128)
    if mask.dtype != torch.uint8 or not _on_device(mask) or not mask.is_contiguous():
        raise TypeError("block mask must be a contiguous uint8 CUDA tensor")
    if tuple(mask.shape) == (nt, nt):
        return ctypes.c_void_p(mask.data_ptr()), 0
    if tuple(mask.shape) == (B * H, nt, nt):
        return ctypes.c_void_p(mask.data_ptr()), nt * nt
    raise ValueError(f"block mask must be [{nt},{nt}] or [{B * H},{nt},{nt}]")


def fa_forward_blocksparse(q, k, v, block_mask, causal: bool = False, scale: float | None = None,
                           o=None, lse=None, stream=None):
    """fa_forward restricted to the 128x128 tiles a uint8 block mask keeps."""
    B, H, N, d = q.shape
    for t, nm in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, nm, torch.bfloat16, (B, H, N, d))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(o, "o", torch.bfloat16, (B, H, N, d))
    _check(lse, "lse", torch.float32, (B, H, N))
    mp, ms = _mask_args(block_mask, B, H, N)
    dev = _one_device((q, "q"), (k, "k"), (v, "v"), (o, "o"), (lse, "lse"),
                      (block_mask, "block_mask"))
    with _device_guard(dev):
        st = library().fa_forward_blocksparse(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H,
                                              N, d, float(scale), int(bool(causal)), mp, ms,
                                              ctypes.c_void_p(_stream_handle(stream, q.device)))
    if st != FA_OK:
        raise FaError(st, "fa_forward_blocksparse")
    return o, lse


def fa_backward_blocksparse(q, k, v, o, dO, lse, block_mask, causal: bool = False,
                            scale: float | None = None, dq=None, dk=None, dv=None,
                            workspace=None, stream=None):
    """fa_backward restricted to the 128x128 tiles a uint8 block mask keeps."""
    B, H, N, d = q.shape
    for t, nm in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dO, "dO")):
        _check(t, nm, torch.bfloat16, (B, H, N, d))
    _check(lse, "lse", torch.float32, (B, H, N))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check_grads(dq, dk, dv, (B, H, N, d))
    need = fa_backward_workspace_size(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check_workspace(workspace)
    mp, ms = _mask_args(block_mask, B, H, N)
    dev = _one_device((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dO, "dO"), (lse, "lse"),
                      (dq, "dq"), (dk, "dk"), (dv, "dv"), (workspace, "workspace"),
                      (block_mask, "block_mask"))
    with _device_guard(dev):
        st = library().fa_backward_blocksparse(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO),
                                               _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), B, H, N,
                                               d, float(scale), int(bool(causal)), mp, ms,
                                               _ptr(workspace), workspace.numel(),
                                               ctypes.c_void_p(_stream_handle(stream, q.device)))
    if st != FA_OK:
        raise FaError(st, "fa_backward_blocksparse")
    return dq, dk, dv


def fa_forward_dropout(q, k, v, p_drop: float, seed: int, offset: int = 0,
                       causal: bool = False, scale: float | None = None, block_mask=None,
                       o=None, lse=None, stream=None):
    """O = (softmax(scale q k^T) o Z / (1 - p_drop)) v and the lse of the
    undropped softmax; Z is replayed from Philox4x32-10 at (seed, offset).
    block_mask: None (dense) or a uint8 CUDA block mask as for
    fa_forward_blocksparse."""
    B, H, N, d = q.shape
    for t, nm in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, nm, torch.bfloat16, (B, H, N, d))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(o, "o", torch.bfloat16, (B, H, N, d))
    _check(lse, "lse", torch.float32, (B, H, N))
    mp, ms = (None, 0) if block_mask is None else _mask_args(block_mask, B, H, N)
    dev = _one_device((q, "q"), (k, "k"), (v, "v"), (o, "o"), (lse, "lse"),
                      (block_mask, "block_mask"))
    with _device_guard(dev):
        st = library().fa_forward_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N,
                                          d, float(scale), int(bool(causal)), float(p_drop),
                                          int(seed) & (2**64 - 1), int(offset) & 0xFFFFFFFF, mp,
                                          ms, ctypes.c_void_p(_stream_handle(stream, q.device)))
    if st != FA_OK:
        raise FaError(st, "fa_forward_dropout")
    return o, lse


def fa_backward_dropout(q, k, v, o, dO, lse, p_drop: float, seed: int, offset: int = 0,
                        causal: bool = False, scale: float | None = None, block_mask=None,
                        dq=None, dk=None, dv=None, workspace=None, stream=None):
    """(dq, dk, dv) of fa_forward_dropout with the same p_drop, seed, offset."""
    B, H, N, d = q.shape
    for t, nm in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dO, "dO")):
        _check(t, nm, torch.bfloat16, (B, H, N, d))
    _check(lse, "lse", torch.float32, (B, H, N))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check_grads(dq, dk, dv, (B, H, N, d))
    need = fa_backward_workspace_size(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check_workspace(workspace)
    mp, ms = (None, 0) if block_mask is None else _mask_args(block_mask, B, H, N)
    dev = _one_device((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dO, "dO"), (lse, "lse"),
                      (dq, "dq"), (dk, "dk"), (dv, "dv"), (workspace, "workspace"),
                      (block_mask, "block_mask"))
    with _device_guard(dev):
        st = library().fa_backward_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO),
                                           _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d,
                                           float(scale), int(bool(causal)), float(p_drop),
                                           int(seed) & (2**64 - 1), int(offset) & 0xFFFFFFFF, mp,
                                           ms, _ptr(workspace), workspace.numel(),
                                           ctypes.c_void_p(_stream_handle(stream, q.device)))
    if st != FA_OK:
        raise FaError(st, "fa_backward_dropout")
    return dq, dk, dv


def fa_forward_fp8(q8, k8, vt8, q_descale: float, k_descale: float, v_descale: float,
                   causal: bool = False, scale: float | None = None, o=None, lse=None,
                   stream=None):
    """O and lse of the attention of the dequantised e4m3 inputs.

    q8, k8: torch.float8_e4m3fn (or uint8 holding e4m3) [B,H,N,d]; vt8: V
    transposed per head, [B,H,d,N]; the descales map stored values to real
    ones.  d = 128, N a multiple of 16.
    """
    B, H, N, d = q8.shape
    for t, nm, shp in ((q8, "q8", (B, H, N, d)), (k8, "k8", (B, H, N, d)),
                       (vt8, "vt8", (B, H, d, N))):
        if t.element_size() != 1 or not _on_device(t) or not t.is_contiguous():
            raise TypeError(f"{nm} must be a contiguous one-byte (e4m3) CUDA tensor")
        if tuple(t.shape) != shp:
            raise ValueError(f"{nm} has shape {tuple(t.shape)}, expected {shp}")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q8.device) if o is None else o
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q8.device) if lse is None else lse
    _check(o, "o", torch.bfloat16, (B, H, N, d))
    _check(lse, "lse", torch.float32, (B, H, N))
    dev = _one_device((q8, "q8"), (k8, "k8"), (vt8, "vt8"), (o, "o"), (lse, "lse"))
    with _device_guard(dev):
        st = library().fa_forward_fp8(_ptr(q8), _ptr(k8), _ptr(vt8), float(q_descale),
                                      float(k_descale), float(v_descale), _ptr(o), _ptr(lse), B,
                                      H, N, d, float(scale), int(bool(causal)),
                                      ctypes.c_void_p(_stream_handle(stream, q8.device)))
    if st != FA_OK:
        raise FaError(st, "fa_forward_fp8")
    return o, lse


class HostPlan:
    """Training steps on HOST tensors through the library's host runtime
    (fa_host_plan_create / fa_host_step / fa_host_wait).

    step() enqueues one fa_forward + fa_backward whose inputs q, k, v, dO and
    outputs o, lse, dq, dk, dv are CPU tensors (bf16 [B,H,N,d], lse fp32
    [B,H,N]; pin them for the copies to overlap the kernels) and returns at
    once; the tensors must stay untouched until wait().
    """

    def __init__(self, B: int, H: int, N: int, d: int, causal: bool = False,
                 scale: float | None = None, device=None):
        self.shape = (B, H, N, d)
        scale = 1.0 / math.sqrt(d) if scale is None else scale
        dev = torch.device("cuda") if device is None else torch.device(device)
        lib = library()
        h = ctypes.c_void_p()
        with torch.cuda.device(dev):
            st = lib.fa_host_plan_create(B, H, N, d, float(scale), int(bool(causal)),
                                         ctypes.byref(h))
        if st != FA_OK:
            raise FaError(st, "fa_host_plan_create")
        self._h = h
        self._keep = []

    def step(self, q, k, v, dO, o, lse, dq, dk, dv):
        B, H, N, d = self.shape
        for t, nm in ((q, "q"), (k, "k"), (v, "v"), (dO, "dO"), (o, "o"), (dq, "dq"),
                      (dk, "dk"), (dv, "dv")):
            if t.device.type != "cpu" or t.dtype != torch.bfloat16 or not t.is_contiguous() \
                    or tuple(t.shape) != (B, H, N, d):
                raise TypeError(f"{nm} must be a contiguous bf16 CPU tensor of shape "
                                f"{(B, H, N, d)}")
        if lse.device.type != "cpu" or lse.dtype != torch.float32 or not lse.is_contiguous() \
                or tuple(lse.shape) != (B, H, N):
            raise TypeError(f"lse must be a contiguous fp32 CPU tensor of shape {(B, H, N)}")
        ts = (q, k, v, dO, o, lse, dq, dk, dv)
        st = library().fa_host_step(self._h, *(ctypes.c_void_p(t.data_ptr()) for t in ts))
        if st != FA_OK:
            raise FaError(st, "fa_host_step")
        self._keep.append(ts)  # the buffers stay referenced until wait()

    def wait(self):
        st = library().fa_host_wait(self._h)
        self._keep.clear()
        if st != FA_OK:
            raise FaError(st, "fa_host_wait")

    def close(self):
        if getattr(self, "_h", None):
            st = library().fa_host_plan_destroy(self._h)
            self._h = None
            self._keep.clear()
            if st != FA_OK:
                raise FaError(st, "fa_host_plan_destroy")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def fa_decode_workspace_size(B: int, H: int, Nq: int, Nk: int, d: int) -> int:
    return int(library().fa_decode_workspace_size(B, H, Nq, Nk, d))


def fa_decode(q, k, v, causal: bool = False, scale: float | None = None, o=None, lse=None,
              workspace=None, stream=None):
    """Nq (<= 16) query rows q [B,H,Nq,d] against a key/value cache k, v [B,H,Nk,d]."""
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    _check(q, "q", torch.bfloat16)
    _check(k, "k", torch.bfloat16, (B, H, Nk, d))
    _check(v, "v", torch.bfloat16, (B, H, Nk, d))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(o, "o", torch.bfloat16, (B, H, Nq, d))
    _check(lse, "lse", torch.float32, (B, H, Nq))
    need = fa_decode_workspace_size(B, H, Nq, Nk, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check_workspace(workspace)
    dev = _one_device((q, "q"), (k, "k"), (v, "v"), (o, "o"), (lse, "lse"),
                      (workspace, "workspace"))
    with _device_guard(dev):
        st = library().fa_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Nq, Nk, d,
                                 float(scale), int(bool(causal)), _ptr(workspace),
                                 workspace.numel(),
                                 ctypes.c_void_p(_stream_handle(stream, q.device)))
    if st != FA_OK:
        raise FaError(st, "fa_decode")
    return o, lse


class KvCache:
    """A key/value cache on one GPU: B sequences of up to `capacity` tokens for
    Hkv key heads of d elements, in bf16 or quantised to e4m3 (one power-of-two
    scale a row) as rows are written.

    k, v: [B, Hkv, capacity, d], torch.bfloat16 or torch.float8_e4m3fn (codes);
    k_scale, v_scale: torch.uint8 [B, Hkv, capacity] (exponent + 127), None for
    bf16; lens: torch.int32 [B], the committed tokens of each sequence, which
    the calls below use where they are given no other lengths.  The tensors may
    be written in place; the object keeps these very tensors for its life.
    """

    def __init__(self, B: int, Hkv: int, capacity: int, d: int, format: str = "e4m3",
                 device=None):
        if format not in ("e4m3", "bf16"):
            raise ValueError(f"format must be 'e4m3' or 'bf16', got {format!r}")
        dev = torch.device("cuda") if device is None else torch.device(device)
        dt = torch.float8_e4m3fn if format == "e4m3" else torch.bfloat16
        shape = (int(B), int(Hkv), int(capacity), int(d))
        scales = [None, None] if format == "bf16" else \
            [torch.zeros(shape[:3], dtype=torch.uint8, device=dev) for _ in range(2)]
        self._hold(torch.zeros(shape, dtype=dt, device=dev),
                   torch.zeros(shape, dtype=dt, device=dev), *scales, None)

    @classmethod
    def from_tensors(cls, k, v, k_scale=None, v_scale=None, lens=None):
        """A cache over tensors that the caller already holds."""
        self = cls.__new__(cls)
        self._hold(k, v, k_scale, v_scale, lens)
        return self

    def _hold(self, k, v, k_scale, v_scale, lens):
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise TypeError(f"k must be torch.bfloat16 or torch.float8_e4m3fn, got {k.dtype}")
        e4m3 = k.dtype == torch.float8_e4m3fn
        if k.dim() != 4:
            raise ValueError(f"k has shape {tuple(k.shape)}, expected [B, Hkv, capacity, d]")
        B, Hkv, cap, d = k.shape
        _check(k, "k", k.dtype)
        _check(v, "v", k.dtype, k.shape)
        if e4m3:
            if k_scale is None or v_scale is None:
                raise ValueError("an e4m3 cache needs k_scale and v_scale")
            _check(k_scale, "k_scale", torch.uint8, (B, Hkv, cap))
            _check(v_scale, "v_scale", torch.uint8, (B, Hkv, cap))
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a bf16 cache has no scales")
        if lens is None:
            lens = torch.zeros(B, dtype=torch.int32, device=k.device)
        _check(lens, "lens", torch.int32, (B,))
        self._dev = _one_device((k, "k"), (v, "v"), (k_scale, "k_scale"), (v_scale, "v_scale"),
                                (lens, "lens"))
        self._t = (k, v, k_scale, v_scale, lens)
        self._shape = (B, Hkv, cap, d)
        self._struct = _CacheStruct(
            k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if e4m3 else None,
            v_scale.data_ptr() if e4m3 else None, B, Hkv, cap, d, int(e4m3))
        self._ref = ctypes.byref(self._struct)
        self._sizes = {}  # workspace bytes by (Hq, T)

    k = property(lambda self: self._t[0])
    v = property(lambda self: self._t[1])
    k_scale = property(lambda self: self._t[2])
    v_scale = property(lambda self: self._t[3])
    lens = property(lambda self: self._t[4])
    shape = property(lambda self: self._shape)
    format = property(lambda self: "e4m3" if self._struct.format else "bf16")


def _check_on(cache, t, name, dtype, shape):
    """_check, and the cache's GPU.  The calls on a cache take a few microseconds on
    the GPU, so what is as it should be passes on one line."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() \
            and _device_index(t) == cache._dev and _on_device(t):
        return
    _check(t, name, dtype, shape)
    if _device_index(t) != cache._dev:
        raise ValueError(f"{name} is on device {_device_index(t)}, the cache on device "
                         f"{cache._dev}")


def _check_ints(cache, t, name, shape):
    if t is not None:
        _check_on(cache, t, name, torch.int32, shape)


def _alloc_on(cache, stream):
    """Tensors that a call allocates for itself belong to the stream that it runs on:
    the memory they get, and give back, is in no other stream's use."""
    if stream is None or cache._dev < 0:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=cache._dev)
    return torch.cuda.stream(stream)


def _cache_call(cache, fn, stream, *args):
    """fn(cache, *args, stream) with the cache's device current."""
    dev = cache._dev
    if stream is None and dev >= 0:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    else:
        stream = _stream_handle(stream, cache._t[0].device)
    if dev < 0 or dev == torch.cuda.current_device():
        st = fn(cache._ref, *args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(cache._ref, *args, stream)
    if st != FA_OK:
        raise FaError(st, fn.__name__)


def fa_cache_write(cache: KvCache, k, v, lens=None, counts=None, stream=None):
    """Write rows k, v (bf16 [B,Hkv,N,d]) to positions lens[b] + i of the cache
    (lens: cache.lens unless given; it is not advanced), quantised if the
    cache is; counts (int32 [B], optional): rows i >= counts[b] are not
    written.  Positions outside the cache are not written."""
    B, Hkv, cap, d = cache._shape
    if k.dim() != 4:
        raise ValueError(f"k has shape {tuple(k.shape)}, expected [B, Hkv, N, d]")
    N = k.shape[2]
    lens = cache._t[4] if lens is None else lens
    _check_on(cache, k, "k", torch.bfloat16, (B, Hkv, N, d))
    _check_on(cache, v, "v", torch.bfloat16, (B, Hkv, N, d))
    _check_ints(cache, lens, "lens", (B,))
    _check_ints(cache, counts, "counts", (B,))
    _cache_call(cache, library().fa_cache_write, stream, k.data_ptr(), v.data_ptr(),
                lens.data_ptr(), None if counts is None else counts.data_ptr(), N)


def fa_cache_read(cache: KvCache, N: int, first=None, counts=None, k=None, v=None, stream=None):
    """(k, v), bf16 [B,Hkv,N,d]: positions first[b] + i (first: 0 unless given)
    for i < counts[b] (cache.lens unless given), zero for the other i < N and
    for positions outside the cache."""
    B, Hkv, cap, d = cache._shape
    shape = (B, Hkv, int(N), d)
    dev = cache._t[0].device
    if k is None or v is None:
        with _alloc_on(cache, stream):
            k = torch.empty(shape, dtype=torch.bfloat16, device=dev) if k is None else k
            v = torch.empty(shape, dtype=torch.bfloat16, device=dev) if v is None else v
    counts = cache._t[4] if counts is None else counts
    _check_on(cache, k, "k", torch.bfloat16, shape)
    _check_on(cache, v, "v", torch.bfloat16, shape)
    _check_ints(cache, first, "first", (B,))
    _check_ints(cache, counts, "counts", (B,))
    _cache_call(cache, library().fa_cache_read, stream, k.data_ptr(), v.data_ptr(),
                None if first is None else first.data_ptr(), counts.data_ptr(), int(N))
    return k, v


def fa_cache_commit(cache: KvCache, path, n_accept, lens=None, new_lens=None, stream=None):
    """Move the rows of drafts path[b, 0 .. n_accept[b]) (int32 [B,T], int32 [B])
    to positions lens[b] + i and return new_lens = lens + n_accept.  lens and
    new_lens: cache.lens, advanced in place, unless given (new_lens: lens
    itself if only lens is given)."""
    B = cache._shape[0]
    if path.dim() != 2:
        raise ValueError(f"path has shape {tuple(path.shape)}, expected [B, T]")
    T = path.shape[1]
    lens = cache._t[4] if lens is None else lens
    new_lens = lens if new_lens is None else new_lens
    _check_on(cache, path, "path", torch.int32, (B, T))
    _check_ints(cache, n_accept, "n_accept", (B,))
    _check_ints(cache, lens, "lens", (B,))
    _check_ints(cache, new_lens, "new_lens", (B,))
    _cache_call(cache, library().fa_cache_commit, stream, lens.data_ptr(), path.data_ptr(),
                n_accept.data_ptr(), new_lens.data_ptr(), T)
    return new_lens


def tree_mask(parents):
    """The mask row of each draft (torch.int64 [T] on the CPU; bit j: draft j is
    seen) of the tree in which draft t's parent is draft parents[t] < t, or
    none for -1: a draft sees itself and its ancestors."""
    if not 1 <= len(parents) <= 64:
        raise ValueError(f"a tree has 1 .. 64 drafts, got {len(parents)}")
    rows = []
    for t, p in enumerate(int(p) for p in parents):
        if not -1 <= p < t:
            raise ValueError(f"parents[{t}] must be -1 or an earlier draft, got {p}")
        rows.append((rows[p] if p >= 0 else 0) | 1 << t)
    return torch.tensor([r - (1 << 64) if r >> 63 else r for r in rows], dtype=torch.int64)


def fa_decode_tree_workspace_size(cache: KvCache, Hq: int, T: int) -> int:
    """Bytes of workspace of fa_decode_tree (0 for an invalid shape)."""
    size = cache._sizes.get((Hq, T))
    if size is None:
        size = int(library().fa_decode_tree_workspace_size(cache._ref, Hq, T))
        cache._sizes[(Hq, T)] = size
    return size


def fa_decode_tree(cache: KvCache, q, mask=None, lens=None, scale: float | None = None, o=None,
                   lse=None, workspace=None, stream=None):
    """Attention of T (<= 64) drafted tokens q (bf16 [B,Hq,T,d], Hq a multiple of
    the cache's Hkv) over the cache: (o, lse).

    Draft j lies at position lens[b] + j (lens: cache.lens unless given; write
    the drafts there first).  Each draft sees the lens[b] committed tokens and
    the drafts of its mask row: mask is torch.int64 [B,T], or [T] for one tree
    shared by the batch, bit j for draft j; None: the drafts j <= t.  A draft
    that sees nothing has o = 0 and lse = -inf.  Calls that may overlap on the
    GPU need workspaces of their own (a new one is allocated by default)."""
    B, Hkv, cap, d = cache._shape
    if q.dim() != 4:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [B, Hq, T, d]")
    _, Hq, T, _ = q.shape
    shape = (B, Hq, T, d)
    _check_on(cache, q, "q", torch.bfloat16, shape)
    lens = cache._t[4] if lens is None else lens
    _check_ints(cache, lens, "lens", (B,))
    stride = 0
    if mask is not None:
        stride = T if mask.dim() == 2 else 0
        _check_on(cache, mask, "mask", torch.int64, (B, T) if stride else (T,))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    for t, name, dtype, shp in ((o, "o", torch.bfloat16, shape),
                                (lse, "lse", torch.float32, shape[:3])):
        if t is not None:
            _check_on(cache, t, name, dtype, shp)
    if workspace is not None:
        _check_workspace(workspace)
        if _device_index(workspace) != cache._dev:
            raise ValueError(f"workspace is on device {_device_index(workspace)}, the cache on "
                             f"device {cache._dev}")
    if o is None or lse is None or workspace is None:
        with _alloc_on(cache, stream):
            o = torch.empty_like(q) if o is None else o
            lse = torch.empty(shape[:3], dtype=torch.float32, device=q.device) \
                if lse is None else lse
            if workspace is None:
                need = fa_decode_tree_workspace_size(cache, Hq, T)
                workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _cache_call(cache, library().fa_decode_tree, stream, q.data_ptr(), lens.data_ptr(),
                None if mask is None else mask.data_ptr(), stride, o.data_ptr(), lse.data_ptr(),
                Hq, T, float(scale), workspace.data_ptr(), workspace.numel())
    return o, lse


def _alloc(dev, stream):
    """_alloc_on for a device index."""
    if stream is None or dev < 0:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    return torch.cuda.stream(stream)


def _call(dev, fn, stream, *args):
    """fn(*args, stream) with device `dev` current."""
    if dev >= 0:
        if stream is None:
            stream = torch._C._cuda_getCurrentRawStream(dev)
        elif hasattr(stream, "cuda_stream"):
            stream = stream.cuda_stream
        if dev != torch._C._cuda_getDevice():
            with torch.cuda.device(dev):
                st = fn(*args, stream)
        else:
            st = fn(*args, stream)
    else:
        st = fn(*args, _stream_handle(stream, dev))
    if st != FA_OK:
        raise FaError(st, fn.__name__)


def _heads(t, name, dev, shape):
    """fa_heads of a bf16 tensor of rows on device `dev`: [tokens, heads, d] or
    [B, heads, N, d] in any strides, as long as each row is contiguous."""
    s = t.stride()
    if not (t.dtype is torch.bfloat16 and t.shape == shape and _device_index(t) == dev
            and s[-1] == 1 and _on_device(t)):
        _bad_heads(t, name, dev, shape)
    if len(s) == 3:
        return _pack_heads(t.data_ptr(), 0, s[0], s[1], shape[1])
    return _pack_heads(t.data_ptr(), s[0], s[2], s[1], shape[1])


def _bad_heads(t, name, dev, shape):
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if not _on_device(t):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if _device_index(t) != dev:
        raise ValueError(f"{name} is on device {_device_index(t)}, the call's other tensors on "
                         f"device {dev}")
    raise ValueError(f"the rows of {name} must be contiguous (strides {t.stride()})")


def _vector(t, name, dev, dtype, shape):
    """Address of a small contiguous tensor, checked."""
    if not (t.dtype is dtype and t.shape == shape and _device_index(t) == dev
            and t.is_contiguous() and _on_device(t)):
        _check(t, name, dtype, shape)
        raise ValueError(f"{name} is on device {_device_index(t)}, the call's other tensors on "
                         f"device {dev}")
    return t.data_ptr()


def _outputs(dev, device, stream, *wanted):
    """The tensors of (tensor or None, shape, dtype), made where they were not given, by
    the stream that the call runs on."""
    if stream is not None and dev >= 0:
        with _alloc(dev, stream):
            return _outputs(dev, device, None, *wanted)
    return [torch.empty(shape, dtype=dtype, device=device) if t is None else t
            for t, shape, dtype in wanted]


def _packed_shapes(q, k, v, cu_q, cu_k):
    """(total_q, total_k, Hq, Hkv, d, B) of a packed call."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError(f"q and k have shapes {tuple(q.shape)} and {tuple(k.shape)}, expected "
                         "[tokens, heads, d]")
    if cu_q.dim() != 1 or cu_q.shape[0] < 2:
        raise ValueError(f"cu_q has shape {tuple(cu_q.shape)}, expected [B + 1]")
    tq, Hq, d = q.shape
    tk, Hkv, _ = k.shape
    if cu_k is None and tk != tq:
        raise ValueError(f"q has {tq} tokens and k {tk}: cu_k is needed")
    return tq, tk, Hq, Hkv, d, cu_q.shape[0] - 1


def _packed_workspace(workspace, need, dev, stream, device):
    if workspace is None:
        need = max(need, 256)
        if stream is None:
            return torch.empty(need, dtype=torch.uint8, device=device)
        with _alloc(dev, stream):
            return torch.empty(need, dtype=torch.uint8, device=device)
    _check_workspace(workspace)
    if _device_index(workspace) != dev:
        raise ValueError(f"workspace is on device {_device_index(workspace)}, the call's other "
                         f"tensors on device {dev}")
    return workspace


def fa_forward_packed_workspace_size(B: int, total_q: int, total_k: int, Hq: int, Hkv: int,
                                     d: int) -> int:
    """Bytes of workspace of fa_forward_packed (0 for an invalid shape)."""
    return int(library().fa_forward_packed_workspace_size(B, total_q, total_k, Hq, Hkv, d))


def fa_backward_packed_workspace_size(B: int, total_q: int, total_k: int, Hq: int, Hkv: int,
                                      d: int) -> int:
    """Bytes of workspace of fa_backward_packed (0 for an invalid shape)."""
    return int(library().fa_backward_packed_workspace_size(B, total_q, total_k, Hq, Hkv, d))


def fa_forward_packed(q, k, v, cu_q, cu_k=None, causal: bool = False, scale: float | None = None,
                      o=None, lse=None, workspace=None, stream=None):
    """Attention over packed sequences: (o, lse).

    q: bf16 [total_q, Hq, d]; k, v: bf16 [total_k, Hkv, d], Hq a multiple of Hkv;
    rows contiguous, other strides any multiple of 8 (parts of one projection's
    output are taken as they lie).  cu_q: int32 [B + 1] on the GPU, the first token
    of each sequence and the end of the last; cu_k: the same for the keys (None:
    cu_q).  causal: query i of n sees the keys j <= i + m - n of its m.  o: as q,
    lse: fp32 [Hq, total_q].  A query that sees no key has o = 0 and lse = -inf;
    tokens in no sequence are left as they were.  Calls that may overlap on
    the GPU need workspaces of their own (a new one is allocated by default)."""
    tq, tk, Hq, Hkv, d, B = _packed_shapes(q, k, v, cu_q, cu_k)
    dev = _device_index(q)
    device = q.device
    hq = _heads(q, "q", dev, (tq, Hq, d))
    hk = _heads(k, "k", dev, (tk, Hkv, d))
    hv = _heads(v, "v", dev, (tk, Hkv, d))
    pq = _vector(cu_q, "cu_q", dev, torch.int32, (B + 1,))
    pk = None if cu_k is None else _vector(cu_k, "cu_k", dev, torch.int32, (B + 1,))
    o, lse = _outputs(dev, device, stream, (o, (tq, Hq, d), torch.bfloat16),
                      (lse, (Hq, tq), torch.float32))
    ho = _heads(o, "o", dev, (tq, Hq, d))
    pl = _vector(lse, "lse", dev, torch.float32, (Hq, tq))
    lib = library()
    workspace = _packed_workspace(
        workspace, lib.fa_forward_packed_workspace_size(B, tq, tk, Hq, Hkv, d), dev, stream, device)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    _call(dev, lib.fa_forward_packed, stream, hq, hk, hv, ho, pl, pq, pk, B, tq, tk, d, scale,
          bool(causal), workspace.data_ptr(), workspace.numel())
    return o, lse


def fa_backward_packed(q, k, v, o, dO, lse, cu_q, cu_k=None, causal: bool = False,
                       scale: float | None = None, dq=None, dk=None, dv=None, workspace=None,
                       stream=None):
    """(dq, dk, dv) of fa_forward_packed from the gradient dO of o; dk and dv are sums
    over the query heads of each key head's group.  Shapes, strides and lengths as
    there.  Keys that no query sees get zeros; tokens in no sequence are left as
    they were."""
    tq, tk, Hq, Hkv, d, B = _packed_shapes(q, k, v, cu_q, cu_k)
    dev = _device_index(q)
    device = q.device
    qs, ks = (tq, Hq, d), (tk, Hkv, d)
    hq, hk, hv = _heads(q, "q", dev, qs), _heads(k, "k", dev, ks), _heads(v, "v", dev, ks)
    ho, hg = _heads(o, "o", dev, qs), _heads(dO, "dO", dev, qs)
    pl = _vector(lse, "lse", dev, torch.float32, (Hq, tq))
    pq = _vector(cu_q, "cu_q", dev, torch.int32, (B + 1,))
    pk = None if cu_k is None else _vector(cu_k, "cu_k", dev, torch.int32, (B + 1,))
    bf16 = torch.bfloat16
    dq, dk, dv = _outputs(dev, device, stream, (dq, qs, bf16), (dk, ks, bf16), (dv, ks, bf16))
    hdq, hdk, hdv = _heads(dq, "dq", dev, qs), _heads(dk, "dk", dev, ks), _heads(dv, "dv", dev, ks)
    lib = library()
    workspace = _packed_workspace(
        workspace, lib.fa_backward_packed_workspace_size(B, tq, tk, Hq, Hkv, d), dev, stream, device)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    _call(dev, lib.fa_backward_packed, stream, hq, hk, hv, ho, hg, pl, hdq, hdk, hdv, pq, pk, B,
          tq, tk, d, scale, bool(causal), workspace.data_ptr(), workspace.numel())
    return dq, dk, dv


class Rotary:
    """The rotation of heads of d elements by their tokens' positions: the first
    `rot` elements (all unless given; a multiple of 16) turn in pairs, (i, i + rot / 2)
    or, interleaved, (2i, 2i + 1), pair i by base^(-2i / rot) radians a position.

    scaling, for contexts longer than those trained on: None; "linear" (all
    angles divided by factor); "base" (the base raised so that the slowest pair is
    divided by factor); "turns" or "index" (pairs that turn more than `high` times
    within the `original` context stay, those below `low` are divided by factor,
    between them a blend, linear in the turns or in the pair's index).  amplitude
    multiplies the rotated elements.  turns: the table, torch.int64 [rot / 2] on
    the GPU (unsigned 64-bit fractions of a turn), which the object keeps: keep the
    object until the calls that use it have run."""

    _SCALING = {None: 0, "linear": 1, "base": 2, "turns": 3, "index": 4}

    def __init__(self, d: int, rot: int | None = None, base: float = 10000.0,
                 interleaved: bool = False, scaling: str | None = None, factor: float = 1.0,
                 original: float = 0.0, low: float = 1.0, high: float = 32.0,
                 amplitude: float = 1.0, device=None):
        rot = d if rot is None else int(rot)
        if scaling not in self._SCALING:
            raise ValueError(f"scaling must be one of {list(self._SCALING)}, got {scaling!r}")
        if not 16 <= rot <= d or rot % 16:
            raise ValueError(f"rot must be a multiple of 16 up to d = {d}, got {rot}")
        table = (ctypes.c_ulonglong * (rot // 2))()
        st = library().fa_rotary_table(table, rot, float(base), self._SCALING[scaling],
                                       float(factor), float(original), float(low), float(high))
        if st != FA_OK:
            raise FaError(st, "fa_rotary_table")
        dev = torch.device("cuda") if device is None else torch.device(device)
        self._hold(d, torch.tensor([x - (1 << 64) if x >> 63 else x for x in table],
                                   dtype=torch.int64).to(dev), interleaved, amplitude)

    @classmethod
    def from_table(cls, d: int, turns, interleaved: bool = False, amplitude: float = 1.0):
        """The rotation by a table of the caller's: torch.int64 [rot / 2] on the GPU, the
        turns of each pair a position times 2^64, modulo 2^64."""
        self = cls.__new__(cls)
        if turns.dim() != 1:
            raise ValueError(f"turns has shape {tuple(turns.shape)}, expected [rot / 2]")
        _check(turns, "turns", torch.int64)
        self._hold(d, turns, interleaved, amplitude)
        return self

    def _hold(self, d, turns, interleaved, amplitude):
        self.d, self.turns, self.rot = int(d), turns, 2 * turns.shape[0]
        self.interleaved, self.amplitude = bool(interleaved), float(amplitude)
        self._dev = _device_index(turns)
        self._struct = _RotationStruct(turns.data_ptr(), self.rot, int(self.interleaved),
                                       self.amplitude)
        self._ref = ctypes.byref(self._struct)


def _rotary_shapes(rotary, q, k, positions):
    """(B, N, shape of k or None, pointer of the positions) of a call on q and k."""
    if q.dim() not in (3, 4):
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [tokens, heads, d] or "
                         "[B, heads, N, d]")
    if q.shape[-1] != rotary.d:
        raise ValueError(f"q has rows of {q.shape[-1]} elements, the rotation of {rotary.d}")
    B, N = (1, q.shape[0]) if q.dim() == 3 else (q.shape[0], q.shape[2])
    ks = None
    if k is not None:
        if k.dim() != q.dim():
            raise ValueError(f"k has shape {tuple(k.shape)}, q {tuple(q.shape)}")
        ks = (N, k.shape[1], rotary.d) if q.dim() == 3 else (B, k.shape[1], N, rotary.d)
    pos = None
    if positions is not None:
        pos = _vector(positions, "positions", rotary._dev, torch.int32,
                      (N,) if q.dim() == 3 else (B, N))
    return B, N, ks, pos


def _rotary_outputs(rotary, stream, q, k, q_out, k_out):
    """(q_out, k_out), made as the inputs without gaps where not given (k None: None)."""
    bf16, device = torch.bfloat16, q.device
    if stream is None:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=bf16, device=device)
        if k is None:
            return q_out, None
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=bf16, device=device)
        return q_out, k_out
    with _alloc(rotary._dev, stream):
        return _rotary_outputs(rotary, None, q, k, q_out, k_out)


def _rotate(fn, rotary, q, k, positions, names, q_out, k_out, stream):
    B, N, ks, pos = _rotary_shapes(rotary, q, k, positions)
    q_out, k_out = _rotary_outputs(rotary, stream, q, k, q_out, k_out)
    dev, qs = rotary._dev, q.shape
    hk = ho = None
    if k is not None:
        hk, ho = _heads(k, names[1], dev, ks), _heads(k_out, names[3], dev, ks)
    _call(dev, fn, stream, rotary._ref, _heads(q, names[0], dev, qs), hk,
          _heads(q_out, names[2], dev, qs), ho, pos, B, N, rotary.d)
    return q_out, k_out


def fa_rotary(rotary: Rotary, q, k=None, positions=None, q_out=None, k_out=None, stream=None):
    """(q, k) rotated by their tokens' positions (k None: q alone).

    q, k: bf16 [tokens, heads, d] with positions int32 [tokens], or [B, heads, N, d]
    with positions int32 [B, N]; None: each token's place, from 0.  Rows
    contiguous, other strides any multiple of 8.  q_out may be q, and k_out k."""
    return _rotate(library().fa_rotary, rotary, q, k, positions, ("q", "k", "q_out", "k_out"),
                   q_out, k_out, stream)


def fa_rotary_backward(rotary: Rotary, dq, dk=None, positions=None, dq_in=None, dk_in=None,
                       stream=None):
    """The gradients of fa_rotary's inputs from those of its results; arguments as
    there (dq_in may be dq, and dk_in dk)."""
    return _rotate(library().fa_rotary_backward, rotary, dq, dk, positions,
                   ("dq", "dk", "dq_in", "dk_in"), dq_in, dk_in, stream)


def _weights(rotary, k, q_weight, k_weight):
    """(pointers, 1 for bf16) of a norm's weights."""
    dtype = q_weight.dtype
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"q_weight must be torch.float32 or torch.bfloat16, got {dtype}")
    if k is not None and k_weight is None:
        raise ValueError("k needs k_weight")
    return (_vector(q_weight, "q_weight", rotary._dev, dtype, (rotary.d,)),
            None if k is None else _vector(k_weight, "k_weight", rotary._dev, dtype, (rotary.d,)),
            int(dtype is torch.bfloat16))


def fa_norm_rotary(rotary: Rotary, q, k, positions, q_weight, k_weight=None, eps: float = 1e-6,
                   q_out=None, k_out=None, stream=None):
    """(q, k) with each head divided by its root mean square (eps added to the mean
    square), times q_weight or k_weight ([d], both fp32 or both bf16), and rotated.
    Otherwise as fa_rotary."""
    B, N, ks, pos = _rotary_shapes(rotary, q, k, positions)
    wq, wk, wfmt = _weights(rotary, k, q_weight, k_weight)
    q_out, k_out = _rotary_outputs(rotary, stream, q, k, q_out, k_out)
    dev, qs = rotary._dev, q.shape
    hk = ho = None
    if k is not None:
        hk, ho = _heads(k, "k", dev, ks), _heads(k_out, "k_out", dev, ks)
    _call(dev, library().fa_norm_rotary, stream, rotary._ref, _heads(q, "q", dev, qs), hk,
          _heads(q_out, "q_out", dev, qs), ho, pos, wq, wk, wfmt, eps, B, N, rotary.d)
    return q_out, k_out


FA_NORM_WORKSPACE = 1048576


def fa_norm_rotary_backward(rotary: Rotary, dq, dk, q, k, positions, q_weight, k_weight=None,
                            eps: float = 1e-6, dq_in=None, dk_in=None, dq_weight=None,
                            dk_weight=None, workspace=None, stream=None):
    """(dq_in, dk_in, dq_weight, dk_weight) of fa_norm_rotary from the gradients dq, dk of
    its results and its inputs q, k.  The weights' gradients are fp32 [d].  dq_in may be
    dq, and dk_in dk.  Calls that may overlap need workspaces of their own
    (FA_NORM_WORKSPACE bytes; a new one is allocated by default)."""
    B, N, ks, pos = _rotary_shapes(rotary, q, k, positions)
    if k is not None and dk is None:
        raise ValueError("k needs dk")
    wq, wk, wfmt = _weights(rotary, k, q_weight, k_weight)
    dq_in, dk_in = _rotary_outputs(rotary, stream, q, k, dq_in, dk_in)
    dev, qs, wd, f32 = rotary._dev, q.shape, (rotary.d,), torch.float32
    if dq_weight is None or (k is not None and dk_weight is None):
        new = _outputs(dev, q.device, stream, (None, (2, *wd), f32))[0]
        dq_weight = new[0] if dq_weight is None else dq_weight
        dk_weight = new[1] if dk_weight is None else dk_weight
    pwq = _vector(dq_weight, "dq_weight", dev, f32, wd)
    workspace = _packed_workspace(workspace, FA_NORM_WORKSPACE, dev, stream, q.device)
    hk = hg = ho = pwk = None
    if k is None:
        dk_weight = None
    else:
        pwk = _vector(dk_weight, "dk_weight", dev, f32, wd)
        hk, hg = _heads(k, "k", dev, ks), _heads(dk, "dk", dev, ks)
        ho = _heads(dk_in, "dk_in", dev, ks)
    _call(dev, library().fa_norm_rotary_backward, stream, rotary._ref,
          _heads(dq, "dq", dev, qs), hg, _heads(q, "q", dev, qs), hk,
          _heads(dq_in, "dq_in", dev, qs), ho, pwq, pwk, pos, wq, wk, wfmt, eps, B, N, rotary.d,
          workspace.data_ptr(), workspace.numel())
    return dq_in, dk_in, dq_weight, dk_weight


def fa_backward_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(library().fa_backward_workspace_size(B, H, N, d))


def fa_backward_preprocess(o, dO, D=None, stream=None):
    B, H, N, d = o.shape
    _check(o, "o", torch.bfloat16)
    _check(dO, "dO", torch.bfloat16, (B, H, N, d))
    if D is None:
        D = torch.empty((B, H, N), dtype=torch.float32, device=o.device)
    _check(D, "D", torch.float32, (B, H, N))
    dev = _one_device((o, "o"), (dO, "dO"), (D, "D"))
    with _device_guard(dev):
        st = library().fa_backward_preprocess(_ptr(o), _ptr(dO), _ptr(D), B, H, N, d,
                                              ctypes.c_void_p(_stream_handle(stream, o.device)))
    if st != FA_OK:
        raise FaError(st, "fa_backward_preprocess")
    return D


def fa_backward(q, k, v, o, dO, lse, causal: bool = False, scale: float | None = None,
                dq=None, dk=None, dv=None, workspace=None, stream=None):
    """(dq, dk, dv) of the attention; workspace is a uint8 CUDA tensor or None."""
    B, H, N, d = q.shape
    for t, nm in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dO, "dO")):
        _check(t, nm, torch.bfloat16, (B, H, N, d))
    _check(lse, "lse", torch.float32, (B, H, N))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check_grads(dq, dk, dv, (B, H, N, d))
    need = fa_backward_workspace_size(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check_workspace(workspace)
    dev = _one_device((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dO, "dO"), (lse, "lse"),
                      (dq, "dq"), (dk, "dk"), (dv, "dv"), (workspace, "workspace"))
    with _device_guard(dev):
        st = library().fa_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse),
                                   _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, float(scale),
                                   int(bool(causal)), _ptr(workspace), workspace.numel(),
                                   ctypes.c_void_p(_stream_handle(stream, q.device)))
    if st != FA_OK:
        raise FaError(st, "fa_backward")
    return dq, dk, dv


def fa_backward_noalloc(q, k, v, o, dO, lse, causal: bool = False, scale: float | None = None,
                        dq=None, dk=None, dv=None, stream=None):
    """fa_backward for callers that cannot allocate: the library's built-in
    8 MiB workspace replaces the caller's (B*H*N <= 2,097,152)."""
    B, H, N, d = q.shape
    for t, nm in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dO, "dO")):
        _check(t, nm, torch.bfloat16, (B, H, N, d))
    _check(lse, "lse", torch.float32, (B, H, N))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check_grads(dq, dk, dv, (B, H, N, d))
    dev = _one_device((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dO, "dO"), (lse, "lse"),
                      (dq, "dq"), (dk, "dk"), (dv, "dv"))
    with _device_guard(dev):
        st = library().fa_backward_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO),
                                           _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d,
                                           float(scale), int(bool(causal)),
                                           ctypes.c_void_p(_stream_handle(stream, q.device)))
    if st != FA_OK:
        raise FaError(st, "fa_backward_noalloc")
    return dq, dk, dv


def fa_backward_dkdv(q, k, v, dO, lse, D, causal: bool = False, scale: float | None = None,
                     dk=None, dv=None, stream=None):
    """dk, dv from the D pre-pass output D (fp32 [B,H,N])."""
    B, H, N, d = q.shape
    for t, nm in ((q, "q"), (k, "k"), (v, "v"), (dO, "dO")):
        _check(t, nm, torch.bfloat16, (B, H, N, d))
    _check(lse, "lse", torch.float32, (B, H, N))
    _check(D, "D", torch.float32, (B, H, N))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check(dk, "dk", torch.bfloat16, (B, H, N, d))
    _check(dv, "dv", torch.bfloat16, (B, H, N, d))
    dev = _one_device((q, "q"), (k, "k"), (v, "v"), (dO, "dO"), (lse, "lse"), (D, "D"),
                      (dk, "dk"), (dv, "dv"))
    with _device_guard(dev):
        st = library().fa_backward_dkdv(_ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(lse), _ptr(D),
                                        _ptr(dk), _ptr(dv), B, H, N, d, float(scale),
                                        int(bool(causal)),
                                        ctypes.c_void_p(_stream_handle(stream, q.device)))
    if st != FA_OK:
        raise FaError(st, "fa_backward_dkdv")
    return dk, dv


def fa_backward_dq(q, k, v, dO, lse, D, causal: bool = False, scale: float | None = None,
                   dq=None, stream=None):
    """dq from the D pre-pass output D (fp32 [B,H,N])."""
    B, H, N, d = q.shape
    for t, nm in ((q, "q"), (k, "k"), (v, "v"), (dO, "dO")):
        _check(t, nm, torch.bfloat16, (B, H, N, d))
    _check(lse, "lse", torch.float32, (B, H, N))
    _check(D, "D", torch.float32, (B, H, N))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq = torch.empty_like(q) if dq is None else dq
    _check(dq, "dq", torch.bfloat16, (B, H, N, d))
    dev = _one_device((q, "q"), (k, "k"), (v, "v"), (dO, "dO"), (lse, "lse"), (D, "D"),
                      (dq, "dq"))
    with _device_guard(dev):
        st = library().fa_backward_dq(_ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(lse), _ptr(D),
                                      _ptr(dq), B, H, N, d, float(scale), int(bool(causal)),
                                      ctypes.c_void_p(_stream_handle(stream, q.device)))
    if st != FA_OK:
        raise FaError(st, "fa_backward_dq")
    return dq


def fa_selftest_wait_timeout(stream=None):
    """Launch the library's failure-reporting self-test: a wait that can never
    complete gives up after its limit; fa_get_device_error then reports it."""
    dev = torch.cuda.current_device()
    st = library().fa_selftest_wait_timeout(ctypes.c_void_p(_stream_handle(stream, dev)))
    if st != FA_OK:
        raise FaError(st, "fa_selftest_wait_timeout")


def fa_get_device_error(stream=None):
    """(status, raw detail word); synchronises the stream."""
    detail = ctypes.c_uint32(0)
    dev = torch.cuda.current_device()
    st = library().fa_get_device_error(ctypes.c_void_p(_stream_handle(stream, dev)),
                                       ctypes.byref(detail))
    return st, int(detail.value)
