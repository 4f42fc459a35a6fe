"""Python binding of libwal (include/wal.h): argument marshalling only.

Every step of a product runs in the HIP kernels of ``libwal.so``; this module
converts numpy arrays and torch tensors to pointers and sizes, passes torch's
current HIP stream, and raises ``WalError`` on a negative status.  torch is
used for device memory and streams only.  If the library is missing the
import fails: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libwal.so")

WAL_TRIT_2BIT, WAL_TRIT_BASE3 = 0, 1
WAL_SCALE_FP16, WAL_SCALE_FP24 = 0, 1
WAL_X_F32, WAL_X_BF16 = 0, 1
WAL_X_ROT_H128 = 16   # x_dtype flag: the product rotates x by the normalised H128 first
WAL_GEMM_AUTO, WAL_GEMM_VALU, WAL_GEMM_MFMA = 0, 1, 2
WAL_PHASE_LOWRANK, WAL_PHASE_STREAM, WAL_PHASE_ALL = 1, 2, 3
WAL_MAX_PATHS = 4
WAL_MAX_BATCH = 32
WAL_MAX_PREFILL_BATCH = 16384
WAL_SYNC_BYTES = 4352
WAL_MAX_ROW_BLOCKS = 4096
WAL_WS_ZERO_BYTES = WAL_SYNC_BYTES + 4 * WAL_MAX_ROW_BLOCKS
WAL_SYNC_FALLBACK_WORD = 0
WAL_ROPE_HALF, WAL_ROPE_INTERLEAVED = 0, 1
WAL_ROPE_PLAIN, WAL_ROPE_LINEAR, WAL_ROPE_NTK, WAL_ROPE_PARTS = 0, 1, 2, 3
WAL_KV_BF16, WAL_KV_INT8 = 0, 1
WAL_ATTN_WS_ZERO_BYTES = 65536

STATUS = {0: "WAL_OK", -1: "WAL_ERR_ARG", -2: "WAL_ERR_SHAPE", -3: "WAL_ERR_CODE",
          -4: "WAL_ERR_INEXACT", -5: "WAL_ERR_BUFFER", -6: "WAL_ERR_ALIGN", -7: "WAL_ERR_FORMAT",
          -8: "WAL_ERR_DEVICE", -9: "WAL_ERR_UNSUPPORTED"}


class WalError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


class wal_desc(ctypes.Structure):
    _fields_ = [("out", ctypes.c_uint32), ("in_", ctypes.c_uint32), ("k", ctypes.c_uint32),
                ("n_paths", ctypes.c_uint32), ("rank", ctypes.c_uint32),
                ("trit_fmt", ctypes.c_uint32), ("scale_fmt", ctypes.c_uint32)]


class wal_info(ctypes.Structure):
    _fields_ = [("d", wal_desc), ("row_stride", ctypes.c_uint32), ("groups", ctypes.c_uint32),
                ("total_bytes", ctypes.c_uint64), ("off_codes", ctypes.c_uint64),
                ("off_sites", ctypes.c_uint64), ("off_alpha", ctypes.c_uint64),
                ("off_beta", ctypes.c_uint64), ("off_V", ctypes.c_uint64 * 4),
                ("off_U", ctypes.c_uint64 * 4), ("off_s", ctypes.c_uint64 * 4),
                ("algorithmic_bytes", ctypes.c_uint64)]


WAL_MAX_CLASSES = 16


class wal_grouped_info(ctypes.Structure):
    _fields_ = [("n", ctypes.c_uint32), ("n_classes", ctypes.c_uint32), ("n_segs", ctypes.c_uint32),
                ("n_zjobs", ctypes.c_uint32), ("x_dtype", ctypes.c_uint32), ("zjob_terms", ctypes.c_uint32),
                ("rows_per_batch", ctypes.c_uint32), ("grid", ctypes.c_uint32),
                ("plan_bytes", ctypes.c_uint64), ("algorithmic_bytes", ctypes.c_uint64),
                ("off_descs", ctypes.c_uint64), ("off_zjobs", ctypes.c_uint64),
                ("class_id", ctypes.c_uint32 * WAL_MAX_CLASSES), ("class_grid", ctypes.c_uint32 * WAL_MAX_CLASSES),
                ("class_blockseg", ctypes.c_uint64 * WAL_MAX_CLASSES),
                ("class_segs", ctypes.c_uint64 * WAL_MAX_CLASSES), ("sync_dev", ctypes.c_void_p)]


class wal_rope_desc(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_uint32), ("scaling", ctypes.c_uint32), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("trained_len", ctypes.c_double), ("turns_low", ctypes.c_double),
                ("turns_high", ctypes.c_double)]


class wal_rotary(ctypes.Structure):
    _fields_ = [("turns_dev", ctypes.c_void_p), ("pos_dev", ctypes.c_void_p), ("rot_dim", ctypes.c_uint32),
                ("layout", ctypes.c_uint32), ("magnitude", ctypes.c_float)]


class wal_norms(ctypes.Structure):
    _fields_ = [("q_weight_dev", ctypes.c_void_p), ("k_weight_dev", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("eps", ctypes.c_float)]


class wal_kv_desc(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_uint32), ("page_size", ctypes.c_uint32), ("kv_heads", ctypes.c_uint32),
                ("head_dim", ctypes.c_uint32), ("fmt", ctypes.c_uint32)]


class wal_delta_desc(ctypes.Structure):
    _fields_ = [("key_heads", ctypes.c_uint32), ("value_heads", ctypes.c_uint32), ("key_dim", ctypes.c_uint32),
                ("value_dim", ctypes.c_uint32), ("norm_eps", ctypes.c_float), ("scale", ctypes.c_float)]


class wal_kv_info(ctypes.Structure):
    _fields_ = [("d", wal_kv_desc), ("total_bytes", ctypes.c_uint64), ("off_k", ctypes.c_uint64),
                ("off_v", ctypes.c_uint64), ("off_ks", ctypes.c_uint64), ("off_vs", ctypes.c_uint64)]


if not os.path.exists(LIB_PATH):
    raise ImportError(f"libwal.so is not built ({LIB_PATH}); run python ternary_hybrid_bit_amd/build.py")
_lib = ctypes.CDLL(LIB_PATH)

_P = ctypes.c_void_p
_I = ctypes.c_int
_U32 = ctypes.c_uint32
_SZ = ctypes.c_size_t
_F = ctypes.c_float
_sig = {
    "wal_status_str": (ctypes.c_char_p, [_I]),
    "wal_packed_size": (_I, [ctypes.POINTER(wal_desc), ctypes.POINTER(wal_info)]),
    "wal_pack": (_I, [ctypes.POINTER(wal_desc), _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ,
                      ctypes.POINTER(wal_info)]),
    "wal_inspect": (_I, [_P, _SZ, ctypes.POINTER(wal_info)]),
    "wal_verify": (_I, [_P, _SZ]),
    "wal_unpack": (_I, [_P, _SZ, _P, _P, _P, _P, _P, _P, _P, _P]),
    "wal_workspace_size": (_I, [ctypes.POINTER(wal_info), _U32, ctypes.POINTER(_SZ)]),
    "wal_gemv": (_I, [ctypes.POINTER(wal_info), _P, _P, _I, _P, _P, _SZ, _P]),
    "wal_gemv_noalloc": (_I, [ctypes.POINTER(wal_info), _P, _P, _I, _P, _P]),
    "wal_gemm_small": (_I, [ctypes.POINTER(wal_info), _P, _P, _I, _U32, _U32, _P, _U32, _I, _P, _SZ, _P]),
    "wal_prefill_workspace_size": (_I, [ctypes.POINTER(wal_info), _U32, ctypes.POINTER(_SZ)]),
    "wal_gemm_prefill": (_I, [ctypes.POINTER(wal_info), _P, _P, _I, _U32, _U32, _P, _U32, _P, _SZ, _P]),
    "wal_grouped_plan_size": (_I, [_U32, _P, _U32, _I, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ)]),
    "wal_grouped_plan": (_I, [_U32, _P, _P, _P, _I, _P, _P, _SZ, _U32, _P, _SZ,
                              ctypes.POINTER(wal_grouped_info)]),
    "wal_gemv_grouped": (_I, [ctypes.POINTER(wal_grouped_info), _P, _P]),
    "wal_gemv_grouped_phases": (_I, [ctypes.POINTER(wal_grouped_info), _P, _I, _P]),
    "wal_rotate_h128": (_I, [_P, _I, _U32, _U32, _U32, _P, _I, _U32, _P]),
    "wal_int4_size": (_I, [_U32, _U32, ctypes.POINTER(_SZ)]),
    "wal_int4_pack": (_I, [_U32, _U32, _P, _P, _P, _SZ]),
    "wal_int4_unpack": (_I, [_U32, _U32, _P, _SZ, _P, _P]),
    "wal_int4_gemv": (_I, [_P, _U32, _U32, _P, _I, _P, _P]),
    "wal_int3_size": (_I, [_U32, _U32, ctypes.POINTER(_SZ)]),
    "wal_int3_pack": (_I, [_U32, _U32, _P, _P, _P, _SZ]),
    "wal_int3_unpack": (_I, [_U32, _U32, _P, _SZ, _P, _P]),
    "wal_embed_rows": (_I, [_P, _I, _U32, _U32, _P, _U32, _P, _I, _U32, _P]),
    "wal_embed_rows_mixed": (_I, [_P, _U32, _P, _U32, _U32, _P, _U32, _P, _U32, _P, _I, _U32, _P]),
    "wal_int5_size": (_I, [_U32, _U32, ctypes.POINTER(_SZ)]),
    "wal_int5_pack": (_I, [_U32, _U32, _P, _P, _P, _SZ]),
    "wal_int5_unpack": (_I, [_U32, _U32, _P, _SZ, _P, _P]),
    "wal_int5_gemv": (_I, [_P, _U32, _U32, _P, _I, _P, _P]),
    "wal_gemv_grouped_seq": (_I, [_U32, _P, _P, _P]),
    "wal_graph_create": (_I, [_U32, _P, _P, ctypes.POINTER(_P)]),
    "wal_graph_launch": (_I, [_P, _P]),
    "wal_graph_destroy": (_I, [_P]),
    "wal_rope_freqs": (_I, [ctypes.POINTER(wal_rope_desc), _P, ctypes.POINTER(_F)]),
    "wal_rope": (_I, [_P, _I, _U32, _U32, _U32, _U32, ctypes.POINTER(wal_rotary), _P, _I, _U32, _P]),
    "wal_kv_size": (_I, [ctypes.POINTER(wal_kv_desc), ctypes.POINTER(wal_kv_info)]),
    "wal_kv_write": (_I, [ctypes.POINTER(wal_kv_desc), _P, _P, _U32, _P, _U32, _P, _U32, _I,
                          ctypes.POINTER(wal_rotary), _P, _U32, _U32, _P, _U32, _P]),
    "wal_kv_write_normed": (_I, [ctypes.POINTER(wal_kv_desc), _P, _P, _U32, _P, _U32, _P, _U32, _I,
                                 ctypes.POINTER(wal_norms), ctypes.POINTER(wal_rotary), _P, _U32, _U32, _P, _U32, _P]),
    "wal_head_norm": (_I, [_P, _I, _U32, _U32, _U32, _U32, _P, _I, _F, ctypes.POINTER(wal_rotary), _P, _I, _U32, _P,
                           _I, _U32, _P]),
    "wal_kv_read": (_I, [ctypes.POINTER(wal_kv_desc), _P, _P, _U32, _P, _U32, _P, _U32, _I, _P]),
    "wal_attn_paged_workspace_size": (_I, [ctypes.POINTER(wal_kv_desc), _U32, _U32, _U32, _U32, _U32,
                                           ctypes.POINTER(_SZ)]),
    "wal_attn_paged": (_I, [ctypes.POINTER(wal_kv_desc), _P, _P, _U32, _P, _P, _U32, _U32, _U32, _U32, _P, _U32, _U32,
                            _F, _P, _U32, _P, _SZ, _P]),
    "wal_conv": (_I, [_P, _I, _U32, _U32, _U32, _P, _I, _U32, _P, _I, _P, _U32, _P, _P, _U32, _P, _I, _U32, _P]),
    "wal_delta_workspace_size": (_I, [ctypes.POINTER(wal_delta_desc), _U32, _U32, _U32, ctypes.POINTER(_SZ)]),
    "wal_delta": (_I, [ctypes.POINTER(wal_delta_desc), _P, _U32, _P, _U32, _P, _U32, _P, _U32, _P, _U32, _P, _P, _P,
                       _U32, _U32, _U32, _P, _P, _U32, _P, _U32, _P, _SZ, _P]),
    "wal_attn_prompt": (_I, [_P, _U32, _P, _U32, _P, _U32, _P, _U32, _U32, _U32, _U32, _U32, _U32, _F, _I, _P, _U32,
                             _P]),
}
for _name, (_res, _args) in _sig.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def _check(st: int, where: str):
    if st != 0:
        raise WalError(st, where)


def _ptr(a) -> Optional[int]:
    if a is None:
        return None
    if isinstance(a, np.ndarray):
        return a.ctypes.data
    return a.data_ptr()  # torch tensor


def _c(a, dtype):
    return None if a is None else np.ascontiguousarray(a, dtype=dtype)


_raw_stream = None


def _stream(stream=None) -> Optional[int]:
    """The given stream, or torch's current one on its current device."""
    global _raw_stream
    if stream is not None:
        return int(stream)
    if _raw_stream is None:
        import torch
        of, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
        if of is None or device is None:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
        else:   # the same number without building a Stream object, which costs as much as a launch
            _raw_stream = lambda: of(device())  # noqa: E731
    return _raw_stream()


# ---------------------------------------------------------------------------
# Checks of device arguments.  The C ABI takes bare pointers and cannot see a
# buffer's size, dtype or device, so the binding checks them before any call:
# a wrong dtype or a short buffer would otherwise become out-of-bounds device
# reads or writes.  Type, dtype, shape and size are checked before the device,
# so every check can be exercised on CPU tensors.

def _torch():
    import torch
    return torch


def _dev(t, name: str, dtypes, min_numel: int = 0):
    """t must be a torch tensor of one of ``dtypes`` (torch dtypes), with at
    least ``min_numel`` elements and unit stride along its last axis."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor on the GPU, not {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}; expected one of {[str(d) for d in dtypes]}")
    if t.numel() < min_numel:
        raise ValueError(f"{name} holds {t.numel()} elements; at least {min_numel} are needed")
    if t.dim() > 0 and t.numel() > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride along its last axis")
    if t.dim() > 2:
        raise ValueError(f"{name} must be 1-D or 2-D")
    return t


def _dev_bytes(t, name: str, min_bytes: int):
    """A byte buffer (any dtype) of at least min_bytes bytes, contiguous."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor on the GPU, not {type(t).__name__}")
    nb = t.numel() * t.element_size()
    if nb < min_bytes:
        raise ValueError(f"{name} holds {nb} bytes; at least {min_bytes} are needed")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _gpu(**tensors):
    """Every named tensor (None skipped) must live on a GPU; checked after
    all other checks of a call."""
    for name, t in tensors.items():
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name} must be on the GPU (device {t.device})")


def _xdtype(t) -> int:
    torch = _torch()
    return WAL_X_BF16 if t.dtype == torch.bfloat16 else WAL_X_F32


def _act(t, name: str, n: int):
    """An activation vector: bf16 or fp32, at least n elements."""
    torch = _torch()
    return _dev(t, name, (torch.bfloat16, torch.float32), n)


def _rows(t, name: str, dtypes, cols: int, rows: Optional[int] = None):
    """A 2-D [rows][ld] device matrix with ld >= cols (unit column stride)."""
    _dev(t, name, dtypes)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D [rows][ld]")
    if t.shape[1] < cols:
        raise ValueError(f"{name} has {t.shape[1]} columns; at least {cols} are needed")
    if rows is not None and t.shape[0] < rows:
        raise ValueError(f"{name} has {t.shape[0]} rows; at least {rows} are needed")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} rows overlap (stride {t.stride(0)} < {t.shape[1]})")
    return t


def _ws_bytes(ws, name: str = "ws") -> int:
    """Byte size of a workspace tensor (0 for None); the library checks it
    against what the product needs."""
    if ws is None:
        return 0
    _dev_bytes(ws, name, 0)
    return ws.numel() * ws.element_size()


def sync_fallbacks(ws) -> int:
    """The fallback count of a workspace's synchronisation words: the
    workgroups of earlier calls whose bounded wait for the low-rank terms
    gave up and which computed the terms themselves.  Synchronises the
    device."""
    words = ws.view(-1).view(_torch().uint8)[:WAL_SYNC_BYTES].view(_torch().int32)
    return int(words[WAL_SYNC_FALLBACK_WORD].item())


def clear_sync_fallbacks(ws):
    """Clears that count (on the current stream)."""
    words = ws.view(-1).view(_torch().uint8)[:WAL_SYNC_BYTES].view(_torch().int32)
    words[WAL_SYNC_FALLBACK_WORD] = 0


def wal_status_str(status: int) -> str:
    return _lib.wal_status_str(status).decode()


def make_desc(out, inp, k=8, n_paths=0, rank=0, trit_fmt=WAL_TRIT_2BIT, scale_fmt=WAL_SCALE_FP16) -> wal_desc:
    return wal_desc(out, inp, k, n_paths, rank if n_paths else 0, trit_fmt, scale_fmt)


def wal_packed_size(desc: wal_desc) -> wal_info:
    info = wal_info()
    _check(_lib.wal_packed_size(ctypes.byref(desc), ctypes.byref(info)), "wal_packed_size")
    return info


def wal_pack(desc: wal_desc, T, site_pos=None, site_sign=None, alpha=None, beta=None,
             U=None, V=None, s=None):
    """Pack logical arrays (numpy) into a new uint8 blob; returns (blob, info)."""
    info = wal_packed_size(desc)
    dst = np.zeros(info.total_bytes, dtype=np.uint8)
    arrays = [_c(T, np.int8), _c(site_pos, np.uint8), _c(site_sign, np.int8), _c(alpha, np.float32),
              _c(beta, np.float32), _c(U, np.int8), _c(V, np.int8), _c(s, np.float32)]
    out = wal_info()
    st = _lib.wal_pack(ctypes.byref(desc), *[_ptr(a) for a in arrays], dst.ctypes.data, dst.size,
                       ctypes.byref(out))
    _check(st, "wal_pack")
    return dst, out


def pack_matrix(m) -> tuple:
    """Pack a ``synth.Matrix``-like object (fields T, site_pos, ...)."""
    desc = make_desc(m.out, m.inp, m.k, m.U.shape[0], m.U.shape[2] if m.U.shape[0] else 0,
                     m.trit_fmt, m.scale_fmt)
    k = m.k
    return wal_pack(desc, m.T, m.site_pos if k else None, m.site_sign if k else None, m.alpha,
                    m.beta if k else None, m.U if m.U.shape[0] else None,
                    m.V if m.U.shape[0] else None, m.s if m.U.shape[0] else None)


def wal_inspect(blob) -> wal_info:
    b = np.ascontiguousarray(blob, dtype=np.uint8) if not isinstance(blob, np.ndarray) else blob
    info = wal_info()
    _check(_lib.wal_inspect(b.ctypes.data, b.size, ctypes.byref(info)), "wal_inspect")
    return info


def wal_verify(blob) -> int:
    b = np.frombuffer(blob, dtype=np.uint8) if isinstance(blob, (bytes, bytearray)) else blob
    return _lib.wal_verify(b.ctypes.data, b.size)


def wal_unpack(blob) -> dict:
    b = np.frombuffer(blob, dtype=np.uint8) if isinstance(blob, (bytes, bytearray)) else blob
    info = wal_inspect(b)
    d = info.d
    G = d.in_ // 128
    P, r = d.n_paths, d.rank
    o = {"T": np.zeros((d.out, d.in_), np.int8), "site_pos": np.zeros((d.out, G, d.k), np.uint8),
         "site_sign": np.zeros((d.out, G, d.k), np.int8), "alpha": np.zeros((d.out, G), np.float32),
         "beta": np.zeros((d.out, G), np.float32) if d.k else None,
         "U": np.zeros((P, d.out, r), np.int8), "V": np.zeros((P, d.in_, r), np.int8),
         "s": np.zeros((P, r), np.float32)}
    st = _lib.wal_unpack(b.ctypes.data, b.size, *[_ptr(o[k]) if o[k] is not None and o[k].size else None
                                                   for k in ("T", "site_pos", "site_sign", "alpha", "beta",
                                                             "U", "V", "s")])
    _check(st, "wal_unpack")
    return o


def wal_workspace_size(info: wal_info, batch: int = 1) -> int:
    n = _SZ()
    _check(_lib.wal_workspace_size(ctypes.byref(info), batch, ctypes.byref(n)), "wal_workspace_size")
    return n.value


def wal_prefill_workspace_size(info: wal_info, batch: int) -> int:
    n = _SZ()
    _check(_lib.wal_prefill_workspace_size(ctypes.byref(info), batch, ctypes.byref(n)), "wal_prefill_workspace_size")
    return n.value


def wal_gemv(info: wal_info, W, x, y, ws=None, stream=None, rotate=False):
    """y = W(x) on the GPU; W, x, y (and ws, see wal_workspace_size) are device
    tensors; y is fp32 [out].  rotate: the blob is stored rotated, and the
    launch rotates x by the normalised H128 first (WAL_X_ROT_H128)."""
    torch = _torch()
    _dev_bytes(W, "W", int(info.total_bytes))
    _act(x, "x", int(info.d.in_))
    _dev(y, "y", (torch.float32,), int(info.d.out))
    xdt = _xdtype(x) | (WAL_X_ROT_H128 if rotate else 0)
    wsb = _ws_bytes(ws)
    _gpu(W=W, x=x, y=y, ws=ws)
    st = _lib.wal_gemv(ctypes.byref(info), _ptr(W), _ptr(x), xdt, _ptr(y), _ptr(ws), wsb, _stream(stream))
    _check(st, "wal_gemv")
    return y


def wal_gemv_noalloc(info: wal_info, W, x, y, stream=None, rotate=False):
    """y = W(x) as wal_gemv, with the library's per-device scratch as the
    workspace (nothing is allocated; overlapping calls on one GPU race)."""
    torch = _torch()
    _dev_bytes(W, "W", int(info.total_bytes))
    _act(x, "x", int(info.d.in_))
    _dev(y, "y", (torch.float32,), int(info.d.out))
    _gpu(W=W, x=x, y=y)
    xdt = _xdtype(x) | (WAL_X_ROT_H128 if rotate else 0)
    st = _lib.wal_gemv_noalloc(ctypes.byref(info), _ptr(W), _ptr(x), xdt, _ptr(y), _stream(stream))
    _check(st, "wal_gemv_noalloc")
    return y


def wal_gemm_small(info: wal_info, W, X, Y, mode=WAL_GEMM_AUTO, ws=None, stream=None):
    """Y = X W^T on the GPU; X [batch][ldx], Y [batch][ldy] device tensors."""
    torch = _torch()
    _dev_bytes(W, "W", int(info.total_bytes))
    _rows(X, "X", (torch.bfloat16, torch.float32), int(info.d.in_))
    _rows(Y, "Y", (torch.float32,), int(info.d.out), X.shape[0])
    xdt = _xdtype(X)
    if not 1 <= X.shape[0] <= WAL_MAX_BATCH:
        raise ValueError(f"batch {X.shape[0]} outside 1..{WAL_MAX_BATCH}")
    wsb = _ws_bytes(ws)
    _gpu(W=W, X=X, Y=Y, ws=ws)
    st = _lib.wal_gemm_small(ctypes.byref(info), _ptr(W), _ptr(X), xdt, X.shape[0], X.stride(0), _ptr(Y),
                             Y.stride(0), mode, _ptr(ws), wsb, _stream(stream))
    _check(st, "wal_gemm_small")
    return Y


def wal_gemm_prefill(info: wal_info, W, X, Y, ws=None, stream=None):
    """Y = X W^T for a prefill-size batch; X [batch][ldx] bf16, Y [batch][ldy]
    fp32 device tensors, ws of wal_prefill_workspace_size bytes (or None when 0)."""
    torch = _torch()
    _dev_bytes(W, "W", int(info.total_bytes))
    _rows(X, "X", (torch.bfloat16, torch.float32), int(info.d.in_))
    _rows(Y, "Y", (torch.float32,), int(info.d.out), X.shape[0])
    xdt = _xdtype(X)
    if not 1 <= X.shape[0] <= WAL_MAX_PREFILL_BATCH:
        raise ValueError(f"batch {X.shape[0]} outside 1..{WAL_MAX_PREFILL_BATCH}")
    wsb = _ws_bytes(ws)
    _gpu(W=W, X=X, Y=Y, ws=ws)
    st = _lib.wal_gemm_prefill(ctypes.byref(info), _ptr(W), _ptr(X), xdt, X.shape[0], X.stride(0), _ptr(Y),
                               Y.stride(0), _ptr(ws), wsb, _stream(stream))
    _check(st, "wal_gemm_prefill")
    return Y


def wal_grouped_plan_size(infos: Sequence[wal_info], grid: int = 0, x_dtype: int = WAL_X_BF16):
    """(plan_bytes, ws_bytes) of a grouped plan; grid 0 = what the current GPU holds at once."""
    arr = (wal_info * len(infos))(*infos)
    pb, wb = _SZ(), _SZ()
    _check(_lib.wal_grouped_plan_size(len(infos), arr, grid, x_dtype, ctypes.byref(pb), ctypes.byref(wb)),
           "wal_grouped_plan_size")
    return pb.value, wb.value


def wal_grouped_plan(infos: Sequence[wal_info], Ws, xs, ys, ws, x_dtype: int, grid: int = 0):
    """Build a grouped plan; returns (plan bytes as numpy uint8, wal_grouped_info).
    x_dtype may carry WAL_X_ROT_H128 (every matrix of the plan rotated)."""
    torch = _torch()
    n = len(infos)
    if not (len(Ws) == len(xs) == len(ys) == n):
        raise ValueError("infos, Ws, xs and ys must have the same length")
    xt = torch.bfloat16 if (x_dtype & ~WAL_X_ROT_H128) == WAL_X_BF16 else torch.float32
    for i, (f, w, x, y) in enumerate(zip(infos, Ws, xs, ys)):
        _dev_bytes(w, f"Ws[{i}]", int(f.total_bytes))
        _dev(x, f"xs[{i}]", (xt,), int(f.d.in_))
        _dev(y, f"ys[{i}]", (torch.float32,), int(f.d.out))
    arr = (wal_info * n)(*infos)
    pb, _ = wal_grouped_plan_size(infos, grid, x_dtype)
    plan = np.zeros(pb, dtype=np.uint8)
    Wp = (ctypes.c_void_p * n)(*[_ptr(w) for w in Ws])
    xp = (ctypes.c_void_p * n)(*[_ptr(x) for x in xs])
    yp = (ctypes.c_void_p * n)(*[_ptr(y) for y in ys])
    g = wal_grouped_info()
    wsb = _ws_bytes(ws)
    for i, (w, x, y) in enumerate(zip(Ws, xs, ys)):
        _gpu(**{f"Ws[{i}]": w, f"xs[{i}]": x, f"ys[{i}]": y})
    _gpu(ws=ws)
    st = _lib.wal_grouped_plan(n, arr, Wp, xp, x_dtype, yp, _ptr(ws), wsb, grid, plan.ctypes.data, plan.size,
                               ctypes.byref(g))
    _check(st, "wal_grouped_plan")
    return plan, g


def _plan(ginfo: wal_grouped_info, plan_dev, name="plan_dev"):
    _dev_bytes(plan_dev, name, int(ginfo.plan_bytes))
    _gpu(**{name: plan_dev})
    return plan_dev


def wal_gemv_grouped(ginfo: wal_grouped_info, plan_dev, stream=None):
    _plan(ginfo, plan_dev)
    _check(_lib.wal_gemv_grouped(ctypes.byref(ginfo), _ptr(plan_dev), _stream(stream)), "wal_gemv_grouped")


def wal_gemv_grouped_phases(ginfo: wal_grouped_info, plan_dev, phases: int, stream=None):
    _plan(ginfo, plan_dev)
    _check(_lib.wal_gemv_grouped_phases(ctypes.byref(ginfo), _ptr(plan_dev), phases, _stream(stream)),
           "wal_gemv_grouped_phases")


def exported_symbols() -> list:
    return list(_sig)


def _chain_args(chain):
    """chain: [(wal_grouped_info, plan device tensor)] -> ctypes arrays."""
    n = len(chain)
    for i, (g, p) in enumerate(chain):
        _plan(g, p, f"chain[{i}] plan")
    infos = (wal_grouped_info * n)(*[g for g, _ in chain])
    plans = (ctypes.c_void_p * n)(*[_ptr(p) for _, p in chain])
    return n, infos, plans


def wal_gemv_grouped_seq(chain, stream=None):
    """Launch the grouped products of ``chain`` in order on the stream."""
    n, infos, plans = _chain_args(chain)
    _check(_lib.wal_gemv_grouped_seq(n, infos, plans, _stream(stream)), "wal_gemv_grouped_seq")


class WalGraph:
    """A chain of grouped products captured in a HIP graph (wal_graph_create);
    launch() replays it on a stream; the buffers the plans name must outlive it."""

    def __init__(self, chain):
        n, infos, plans = _chain_args(chain)
        h = ctypes.c_void_p()
        _check(_lib.wal_graph_create(n, infos, plans, ctypes.byref(h)), "wal_graph_create")
        self._h = h

    def launch(self, stream=None):
        _check(_lib.wal_graph_launch(self._h, _stream(stream)), "wal_graph_launch")

    def close(self):
        if self._h:
            _check(_lib.wal_graph_destroy(self._h), "wal_graph_destroy")
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001
            pass


def wal_rotate_h128(X, out, stream=None):
    """out = X rotated by the normalised Hadamard-128 along its last axis (1-D
    or 2-D device tensors, bf16 or fp32; out may be X itself)."""
    torch = _torch()
    acts = (torch.bfloat16, torch.float32)
    _dev(X, "X", acts)
    _dev(out, "out", acts)
    X2 = X if X.dim() == 2 else X.view(1, -1)
    O2 = out if out.dim() == 2 else out.view(1, -1)
    _rows(O2, "out", acts, X2.shape[1], X2.shape[0])
    _gpu(X=X, out=out)
    dt = _xdtype
    st = _lib.wal_rotate_h128(_ptr(X2), dt(X), X2.shape[0], X2.shape[1], X2.stride(0), _ptr(O2), dt(out),
                              O2.stride(0), _stream(stream))
    _check(st, "wal_rotate_h128")
    return out


def wal_int4_size(V: int, inp: int) -> int:
    n = _SZ()
    _check(_lib.wal_int4_size(V, inp, ctypes.byref(n)), "wal_int4_size")
    return n.value


def wal_int4_pack(q, s) -> np.ndarray:
    """INT4/g128 codes q [V][in] in [-8, 7] and scales s [V][in/128] -> packed bytes (host)."""
    q = np.ascontiguousarray(q, dtype=np.int8)
    s = np.ascontiguousarray(s, dtype=np.float32)
    V, inp = q.shape
    out = np.zeros(wal_int4_size(V, inp), dtype=np.uint8)
    _check(_lib.wal_int4_pack(V, inp, q.ctypes.data, s.ctypes.data, out.ctypes.data, out.size), "wal_int4_pack")
    return out


def wal_int4_unpack(blob: np.ndarray, V: int, inp: int):
    q = np.zeros((V, inp), dtype=np.int8)
    s = np.zeros((V, inp // 128), dtype=np.float32)
    _check(_lib.wal_int4_unpack(V, inp, blob.ctypes.data, blob.size, q.ctypes.data, s.ctypes.data), "wal_int4_unpack")
    return q, s


def wal_int4_gemv(W, V: int, inp: int, x, y, stream=None):
    """y = W x for an INT4/g128 matrix W (device bytes), x [in] bf16, y [V] fp32."""
    torch = _torch()
    _dev_bytes(W, "W", wal_int4_size(V, inp))
    _act(x, "x", inp)
    _dev(y, "y", (torch.float32,), V)
    xdt = _xdtype(x)
    _gpu(W=W, x=x, y=y)
    _check(_lib.wal_int4_gemv(_ptr(W), V, inp, _ptr(x), xdt, _ptr(y), _stream(stream)), "wal_int4_gemv")
    return y


def wal_int3_size(V: int, inp: int) -> int:
    n = _SZ()
    _check(_lib.wal_int3_size(V, inp, ctypes.byref(n)), "wal_int3_size")
    return n.value


def wal_int3_pack(q, s) -> np.ndarray:
    """INT3/g128 codes q [V][in] in [-4, 3] and scales s [V][in/128] -> packed bytes (host)."""
    q = np.ascontiguousarray(q, dtype=np.int8)
    s = np.ascontiguousarray(s, dtype=np.float32)
    V, inp = q.shape
    out = np.zeros(wal_int3_size(V, inp), dtype=np.uint8)
    _check(_lib.wal_int3_pack(V, inp, q.ctypes.data, s.ctypes.data, out.ctypes.data, out.size), "wal_int3_pack")
    return out


def wal_int3_unpack(blob: np.ndarray, V: int, inp: int):
    q = np.zeros((V, inp), dtype=np.int8)
    s = np.zeros((V, inp // 128), dtype=np.float32)
    _check(_lib.wal_int3_unpack(V, inp, blob.ctypes.data, blob.size, q.ctypes.data, s.ctypes.data), "wal_int3_unpack")
    return q, s


def wal_int5_size(V: int, inp: int) -> int:
    n = _SZ()
    _check(_lib.wal_int5_size(V, inp, ctypes.byref(n)), "wal_int5_size")
    return n.value


def wal_int5_pack(q, s) -> np.ndarray:
    """INT5/g128 codes q [V][in] in [-16, 15] and scales s [V][in/128] -> packed bytes (host)."""
    q = np.ascontiguousarray(q, dtype=np.int8)
    s = np.ascontiguousarray(s, dtype=np.float32)
    V, inp = q.shape
    out = np.zeros(wal_int5_size(V, inp), dtype=np.uint8)
    _check(_lib.wal_int5_pack(V, inp, q.ctypes.data, s.ctypes.data, out.ctypes.data, out.size), "wal_int5_pack")
    return out


def wal_int5_unpack(blob: np.ndarray, V: int, inp: int):
    q = np.zeros((V, inp), dtype=np.int8)
    s = np.zeros((V, inp // 128), dtype=np.float32)
    _check(_lib.wal_int5_unpack(V, inp, blob.ctypes.data, blob.size, q.ctypes.data, s.ctypes.data), "wal_int5_unpack")
    return q, s


def wal_int5_gemv(W, V: int, inp: int, x, y, stream=None):
    """y = W x for an INT5/g128 matrix W (device bytes), x [in] bf16, y [V] fp32."""
    torch = _torch()
    _dev_bytes(W, "W", wal_int5_size(V, inp))
    _act(x, "x", inp)
    _dev(y, "y", (torch.float32,), V)
    xdt = _xdtype(x)
    _gpu(W=W, x=x, y=y)
    _check(_lib.wal_int5_gemv(_ptr(W), V, inp, _ptr(x), xdt, _ptr(y), _stream(stream)), "wal_int5_gemv")
    return y


def wal_embed_rows(W, bits: int, V: int, inp: int, ids, out, stream=None):
    """out[i] = row ids[i] of an INT3 (bits 3) or INT4 (bits 4) matrix W (device
    bytes); ids int32 [n] and out [n][ldo] (fp32 or bf16) device tensors."""
    torch = _torch()
    if bits not in (3, 4):
        raise ValueError("bits must be 3 or 4")
    _dev_bytes(W, "W", wal_int3_size(V, inp) if bits == 3 else wal_int4_size(V, inp))
    _dev(ids, "ids", (torch.int32,))
    _rows(out, "out", (torch.float32, torch.bfloat16), inp, ids.numel())
    odt = _xdtype(out)
    _gpu(W=W, ids=ids, out=out)
    _check(_lib.wal_embed_rows(_ptr(W), bits, V, inp, _ptr(ids), ids.numel(), _ptr(out), odt, out.stride(0),
                               _stream(stream)), "wal_embed_rows")
    return out


def wal_embed_rows_mixed(W3, V3: int, W4, V4: int, inp: int, row_map, ids, out, stream=None):
    """out[i] = vocabulary row ids[i] of a mixed table: row_map[v] >= 0 names
    a row of the INT3 table W3, a negative entry m row -1 - m of the INT4
    table W4 (device bytes); row_map and ids int32, out [n][ldo] device."""
    torch = _torch()
    _dev_bytes(W3, "W3", wal_int3_size(V3, inp) if V3 else 0)
    _dev_bytes(W4, "W4", wal_int4_size(V4, inp) if V4 else 0)
    _dev(row_map, "row_map", (torch.int32,))
    _dev(ids, "ids", (torch.int32,))
    _rows(out, "out", (torch.float32, torch.bfloat16), inp, ids.numel())
    odt = _xdtype(out)
    _gpu(W3=W3, W4=W4, row_map=row_map, ids=ids, out=out)
    _check(_lib.wal_embed_rows_mixed(_ptr(W3), V3, _ptr(W4), V4, inp, _ptr(row_map), row_map.numel(), _ptr(ids),
                                     ids.numel(), _ptr(out), odt, out.stride(0), _stream(stream)),
           "wal_embed_rows_mixed")
    return out



# ---------------------------------------------------------------------------
# Attention: rotary positions, the paged key/value cache, attention over the
# cache and over packed prompts.

def make_rope_desc(rot_dim: int, base: float = 10000.0, scaling: int = WAL_ROPE_PLAIN, factor: float = 1.0,
                   trained_len: float = 0.0, turns_low: float = 1.0, turns_high: float = 32.0) -> wal_rope_desc:
    return wal_rope_desc(rot_dim, scaling, base, factor, trained_len, turns_low, turns_high)


def wal_rope_freqs(desc: wal_rope_desc):
    """(turns, magnitude): the frequency table as int64 numpy [rot_dim / 2] (2^-64
    turns a position; copy it to the GPU) and the factor on rotated values."""
    turns = np.zeros(max(int(desc.rot_dim) // 2, 1), dtype=np.int64)
    m = ctypes.c_float()
    _check(_lib.wal_rope_freqs(ctypes.byref(desc), turns.ctypes.data, ctypes.byref(m)), "wal_rope_freqs")
    return turns, m.value


# These calls run once per layer and token, a few microseconds on the GPU each, so
# their checks are written out flat: one pass over each tensor's attributes.
class _Types:
    """torch's types, looked up once."""

    def __init__(self):
        import torch
        self.tensor, self.bf16, self.i32, self.i64 = torch.Tensor, torch.bfloat16, torch.int32, torch.int64
        self.f32, self.only_f32 = torch.float32, (torch.float32,)
        self.acts, self.only_bf16 = (torch.bfloat16, torch.float32), (torch.bfloat16,)
        self.only_i32 = (torch.int32,)


_types_made = None


def _types() -> _Types:
    global _types_made
    if _types_made is None:
        _types_made = _Types()
    return _types_made


_U32_MAX = 0xFFFFFFFF   # ctypes would pass the low 32 bits of anything larger


def _mat(T, t, name: str, dtypes, cols: int, rows: int = 0):
    """A 2-D device matrix of one of the dtypes with at least so many columns
    and rows, unit stride along its rows, rows apart: (rows, columns, row pitch)."""
    if not isinstance(t, T.tensor):
        raise TypeError(f"{name} must be a torch tensor on the GPU, not {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}; expected one of {[str(d) for d in dtypes]}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D [rows][ld]")
    n, c = shape
    if c < cols:
        raise ValueError(f"{name} has {c} columns; at least {cols} are needed")
    if n < rows:
        raise ValueError(f"{name} has {n} rows; at least {rows} are needed")
    ld, step = t.stride()
    if step != 1 and c > 1 and n:   # (one without rows may have any: numpy's have 0)
        raise ValueError(f"{name} must have unit stride along its last axis")
    if n <= 1:
        ld = (c + 7) & ~7   # the pitch of an only row means nothing: one of whole 16 bytes
    elif ld < c:
        raise ValueError(f"{name} rows overlap (stride {ld} < {c})")
    if (n | ld) > _U32_MAX:
        raise ValueError(f"{name} has {n} rows, {ld} elements apart: more than 32 bits hold")
    return n, c, ld


def _vec(T, t, name: str, dtype, n: int) -> int:
    """A contiguous 1-D device vector of at least n elements: its length."""
    if not isinstance(t, T.tensor):
        raise TypeError(f"{name} must be a torch tensor on the GPU, not {type(t).__name__}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}; expected {dtype}")
    shape = t.shape
    if len(shape) != 1:
        raise ValueError(f"{name} must be 1-D")
    if shape[0] < n:
        raise ValueError(f"{name} holds {shape[0]} elements; at least {n} are needed")
    if shape[0] > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must have unit stride along its last axis")
    if shape[0] > _U32_MAX:
        raise ValueError(f"{name} holds {shape[0]} elements: more than 32 bits hold")
    return shape[0]


def _whole_heads(cols: int, name: str, head_dim: int) -> int:
    if head_dim < 1 or cols % head_dim or not cols:
        raise ValueError(f"{name} has {cols} columns, not a multiple of head_dim {head_dim}")
    return cols // head_dim


def _rotary(T, pos, turns, n: int, layout: int, magnitude: float) -> wal_rotary:
    _vec(T, pos, "pos", T.i32, n)
    pairs = _vec(T, turns, "turns", T.i64, 1)
    return wal_rotary(turns.data_ptr(), pos.data_ptr(), 2 * pairs, layout, magnitude)


def wal_rope(X, out, pos, turns, head_dim: int, layout=WAL_ROPE_HALF, magnitude: float = 1.0, stream=None):
    """out = X [n][heads * head_dim] with every head rotated at its row's
    position; pos int32 [n], turns int64 [rot_dim / 2] (wal_rope_freqs); bf16
    or fp32 device tensors, out may be X itself."""
    T = _types()
    n, cols, ldx = _mat(T, X, "X", T.acts, head_dim)
    heads = _whole_heads(cols, "X", head_dim)
    _, _, ldo = _mat(T, out, "out", T.acts, cols, n)
    r = _rotary(T, pos, turns, n, layout, magnitude)
    if not (X.is_cuda and out.is_cuda and pos.is_cuda and turns.is_cuda):
        _gpu(X=X, out=out, pos=pos, turns=turns)
    if n:   # an empty tensor has no address: nothing to do
        st = _lib.wal_rope(X.data_ptr(), X.dtype is T.bf16, n, heads, head_dim, ldx, r, out.data_ptr(),
                           out.dtype is T.bf16, ldo, _stream(stream))
        if st:
            _check(st, "wal_rope")
    return out


def _norm_weight(T, t, name: str, head_dim: int):
    """A norm's weight: as many fp32 or bf16 values as a head has, one after another."""
    if not isinstance(t, T.tensor):
        raise TypeError(f"{name} must be a torch tensor on the GPU, not {type(t).__name__}")
    if t.dtype not in T.acts:
        raise TypeError(f"{name} has dtype {t.dtype}; expected one of {[str(d) for d in T.acts]}")
    if t.shape != (head_dim,) or (head_dim > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be 1-D, {head_dim} elements with unit stride (shape {tuple(t.shape)})")


def wal_head_norm(X, out, weight, head_dim: int, eps: float = 1e-6, pos=None, turns=None, layout=WAL_ROPE_HALF,
                  magnitude: float = 1.0, gate=None, stream=None):
    """out = X [n][heads * head_dim] with every head over the root of its mean square, times weight [head_dim];
    then rotated as by wal_rope when pos and turns are given, or times silu(gate), gate [n][heads * head_dim].
    bf16 or fp32 device tensors, out may be X itself."""
    T = _types()
    n, cols, ldx = _mat(T, X, "X", T.acts, head_dim)
    heads = _whole_heads(cols, "X", head_dim)
    _, _, ldo = _mat(T, out, "out", T.acts, cols, n)
    _norm_weight(T, weight, "weight", head_dim)
    if (pos is None) != (turns is None):
        raise ValueError("pos and turns go together")
    if pos is not None and gate is not None:
        raise ValueError("a rotation and a gate do not go together")
    r = None if pos is None else _rotary(T, pos, turns, n, layout, magnitude)
    g, gdt, ldg = None, 0, 0
    if gate is not None:
        _, _, ldg = _mat(T, gate, "gate", T.acts, cols, n)
        g, gdt = gate.data_ptr(), gate.dtype is T.bf16
    if not (X.is_cuda and out.is_cuda and weight.is_cuda and (r is None or (pos.is_cuda and turns.is_cuda))
            and (gate is None or gate.is_cuda)):
        _gpu(X=X, out=out, weight=weight, pos=pos, turns=turns, gate=gate)
    if n:
        st = _lib.wal_head_norm(X.data_ptr(), X.dtype is T.bf16, n, heads, head_dim, ldx, weight.data_ptr(),
                                weight.dtype is T.bf16, eps, r, g, gdt, ldg, out.data_ptr(), out.dtype is T.bf16, ldo,
                                _stream(stream))
        if st:
            _check(st, "wal_head_norm")
    return out


def make_kv_desc(n_pages: int, page_size: int, kv_heads: int, head_dim: int, fmt: int = WAL_KV_BF16) -> wal_kv_desc:
    return wal_kv_desc(n_pages, page_size, kv_heads, head_dim, fmt)


def wal_kv_size(desc: wal_kv_desc) -> wal_kv_info:
    """Plane offsets and total_bytes of a cache (allocate that many device bytes, contents arbitrary)."""
    info = wal_kv_info()
    _check(_lib.wal_kv_size(ctypes.byref(desc), ctypes.byref(info)), "wal_kv_size")
    return info


def _kv_cache(T, desc: wal_kv_desc, cache):
    """The cache's buffer, as large as its descriptor says (whose other
    limits the library checks): the width of a token's keys."""
    width = desc.kv_heads * desc.head_dim
    tokens = desc.n_pages * desc.page_size
    int8 = desc.fmt == WAL_KV_INT8
    need = 2 * (-(-(tokens * width * (1 if int8 else 2)) // 256) * 256)
    if int8:
        need += 2 * (-(-(tokens * desc.kv_heads * 4) // 256) * 256)
    if not isinstance(cache, T.tensor):
        raise TypeError(f"cache must be a torch tensor on the GPU, not {type(cache).__name__}")
    if cache.numel() * cache.element_size() < need:
        raise ValueError(f"cache holds {cache.numel() * cache.element_size()} bytes; at least {need} are needed")
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    return width


def wal_kv_write(desc: wal_kv_desc, cache, slots, K, V, pos=None, turns=None, layout=WAL_ROPE_HALF,
                 magnitude: float = 1.0, Q=None, Q_out=None, stream=None, q_norm=None, k_norm=None,
                 eps: float = 1e-6):
    """Writes K, V [n][kv_heads * head_dim] (bf16 or fp32) to the cache's slots
    [n] (int32).  With pos and turns the keys are rotated first, and Q, when
    given, is rotated into Q_out (bf16).  k_norm, q_norm [head_dim] (one type, fp32 or bf16): the heads of K and of
    Q are normed before that, as by wal_head_norm with such a weight and eps."""
    T = _types()
    width = _kv_cache(T, desc, cache)
    n, _, ldk = _mat(T, K, "K", T.acts, width)
    same = (K.dtype,)
    _, _, ldv = _mat(T, V, "V", same, width, n)
    _vec(T, slots, "slots", T.i32, n)
    if (pos is None) != (turns is None):
        raise ValueError("pos and turns go together")
    if (Q is None) != (Q_out is None) or (Q is not None and pos is None):
        raise ValueError("Q needs Q_out, pos and turns")
    r = None if pos is None else _rotary(T, pos, turns, n, layout, magnitude)
    q_heads = ldq = ldqo = 0
    q = q_out = None
    if Q is not None:
        _, cols, ldq = _mat(T, Q, "Q", same, desc.head_dim, n)
        q_heads = _whole_heads(cols, "Q", desc.head_dim)
        _, _, ldqo = _mat(T, Q_out, "Q_out", T.only_bf16, cols, n)
        q, q_out = Q.data_ptr(), Q_out.data_ptr()
    norms = None
    if k_norm is not None or q_norm is not None:
        for t, name in ((k_norm, "k_norm"), (q_norm, "q_norm")):
            if t is not None:
                _norm_weight(T, t, name, desc.head_dim)
        if q_norm is not None and Q is None:
            raise ValueError("q_norm needs Q")
        if k_norm is not None and q_norm is not None and k_norm.dtype is not q_norm.dtype:
            raise TypeError(f"k_norm has dtype {k_norm.dtype}, q_norm {q_norm.dtype}: they must be the same")
        first = k_norm if k_norm is not None else q_norm
        norms = wal_norms(None if q_norm is None else q_norm.data_ptr(), None if k_norm is None else k_norm.data_ptr(),
                          first.dtype is T.bf16, eps)
        if not (first.is_cuda and (q_norm is None or q_norm.is_cuda)):
            _gpu(k_norm=k_norm, q_norm=q_norm)
    if not (cache.is_cuda and slots.is_cuda and K.is_cuda and V.is_cuda and (r is None or (pos.is_cuda and turns.is_cuda))
            and (Q is None or (Q.is_cuda and Q_out.is_cuda))):
        _gpu(cache=cache, slots=slots, K=K, V=V, pos=pos, turns=turns, Q=Q, Q_out=Q_out)
    if n and norms is not None:
        st = _lib.wal_kv_write_normed(desc, cache.data_ptr(), slots.data_ptr(), n, K.data_ptr(), ldk, V.data_ptr(), ldv,
                                      K.dtype is T.bf16, norms, r, q, q_heads, ldq, q_out, ldqo, _stream(stream))
        if st:
            _check(st, "wal_kv_write_normed")
    elif n:
        st = _lib.wal_kv_write(desc, cache.data_ptr(), slots.data_ptr(), n, K.data_ptr(), ldk, V.data_ptr(), ldv,
                               K.dtype is T.bf16, r, q, q_heads, ldq, q_out, ldqo, _stream(stream))
        if st:
            _check(st, "wal_kv_write")


def wal_kv_read(desc: wal_kv_desc, cache, slots, K=None, V=None, stream=None):
    """Reads the cache's slots [n] into K, V [n][kv_heads * head_dim] (bf16 or
    fp32; either may be None); returns (K, V)."""
    T = _types()
    width = _kv_cache(T, desc, cache)
    if K is None and V is None:
        raise ValueError("K or V must be given")
    n = _vec(T, slots, "slots", T.i32, 0)
    first = K if K is not None else V
    ldk = ldv = 0
    if K is not None:
        _, _, ldk = _mat(T, K, "K", T.acts, width, n)
    if V is not None:
        _, _, ldv = _mat(T, V, "V", T.acts if K is None else (first.dtype,), width, n)
    if not (cache.is_cuda and slots.is_cuda and first.is_cuda and (V is None or V.is_cuda)):
        _gpu(cache=cache, slots=slots, K=K, V=V)
    if n:
        st = _lib.wal_kv_read(desc, cache.data_ptr(), slots.data_ptr(), n, None if K is None else K.data_ptr(), ldk,
                              None if V is None else V.data_ptr(), ldv, first.dtype is T.bf16, _stream(stream))
        if st:
            _check(st, "wal_kv_read")
    return K, V


def wal_attn_paged_workspace_size(desc: wal_kv_desc, q_heads: int, n_seqs: int, n: int, max_new: int,
                                  max_len: int) -> int:
    if max(q_heads, n_seqs, n, max_new, max_len) > _U32_MAX:
        raise ValueError(f"q_heads {q_heads}, n_seqs {n_seqs}, n {n}, max_new {max_new}, max_len {max_len}: more than 32 bits hold")
    b = _SZ()
    _check(_lib.wal_attn_paged_workspace_size(ctypes.byref(desc), q_heads, n_seqs, n, max_new, max_len,
                                              ctypes.byref(b)), "wal_attn_paged_workspace_size")
    return b.value


def wal_attn_paged(desc: wal_kv_desc, cache, tables, lens, starts, Q, out, ws=None, scale: Optional[float] = None,
                   max_new: Optional[int] = None, max_len: int = 0, stream=None):
    """out = attention of Q's rows over the paged cache: tables int32
    [n_seqs][pages], lens int32 [n_seqs], starts int32 [n_seqs + 1], Q and out
    bf16 [n][q_heads * head_dim], ws of wal_attn_paged_workspace_size bytes, the
    first WAL_ATTN_WS_ZERO_BYTES of them zero before its first call (torch.zeros).
    scale: 1 / sqrt(head_dim) unless given; max_new and max_len bound the
    sequences' new tokens and lengths: rows and tokens past them are not computed.
    max_new left out: 1 if there are no more rows than sequences (a token each),
    else as many as Q has rows; max_len 0: what the tables hold."""
    T = _types()
    _kv_cache(T, desc, cache)
    dim = desc.head_dim
    n_seqs, pages, ldt = _mat(T, tables, "tables", T.only_i32, 1)
    _vec(T, lens, "lens", T.i32, n_seqs)
    _vec(T, starts, "starts", T.i32, n_seqs + 1)
    n, cols, ldq = _mat(T, Q, "Q", T.only_bf16, dim)
    q_heads = _whole_heads(cols, "Q", dim)
    _, _, ldo = _mat(T, out, "out", T.only_bf16, cols, n)
    if n_seqs == 1:
        ldt = pages
    holds = pages * desc.page_size
    max_len = max_len or holds
    if max_new is None:
        max_new = 1 if n <= n_seqs else n
    if not 0 <= max_new <= _U32_MAX or not 0 <= max_len <= min(holds, _U32_MAX):
        raise ValueError(f"max_new {max_new}, max_len {max_len}: the tables hold {holds}")
    wsp, wsb = None, 0
    if ws is not None:
        wsb = _ws_bytes(ws)
        wsp = ws.data_ptr()
    if not (cache.is_cuda and tables.is_cuda and lens.is_cuda and starts.is_cuda and Q.is_cuda and out.is_cuda
            and (ws is None or ws.is_cuda)):
        _gpu(cache=cache, tables=tables, lens=lens, starts=starts, Q=Q, out=out, ws=ws)
    if n and n_seqs:
        st = _lib.wal_attn_paged(desc, cache.data_ptr(), tables.data_ptr(), ldt, lens.data_ptr(), starts.data_ptr(),
                                 n_seqs, n, max_new, max_len, Q.data_ptr(), q_heads, ldq,
                                 dim ** -0.5 if scale is None else scale, out.data_ptr(), ldo, wsp, wsb,
                                 _stream(stream))
        if st:
            _check(st, "wal_attn_paged")
    return out


def wal_attn_prompt(Q, K, V, starts, out, head_dim: int, max_len: int, scale: Optional[float] = None,
                    causal: bool = True, stream=None):
    """out = attention over packed prompts: Q, out bf16 [n][q_heads * head_dim],
    K, V bf16 [n][kv_heads * head_dim], starts int32 [n_seqs + 1]; max_len
    bounds the sequences' lengths; scale as for wal_attn_paged."""
    T = _types()
    n, cols, ldq = _mat(T, Q, "Q", T.only_bf16, head_dim)
    q_heads = _whole_heads(cols, "Q", head_dim)
    _, kv_cols, ldk = _mat(T, K, "K", T.only_bf16, head_dim, n)
    kv_heads = _whole_heads(kv_cols, "K", head_dim)
    _, _, ldv = _mat(T, V, "V", T.only_bf16, kv_cols, n)
    _, _, ldo = _mat(T, out, "out", T.only_bf16, cols, n)
    n_seqs = _vec(T, starts, "starts", T.i32, 1) - 1
    if not 0 <= max_len <= _U32_MAX:
        raise ValueError(f"max_len {max_len}")
    if not (Q.is_cuda and K.is_cuda and V.is_cuda and starts.is_cuda and out.is_cuda):
        _gpu(Q=Q, K=K, V=V, starts=starts, out=out)
    if n:
        st = _lib.wal_attn_prompt(Q.data_ptr(), ldq, K.data_ptr(), ldk, V.data_ptr(), ldv, starts.data_ptr(), n_seqs,
                                  n, max_len, q_heads, kv_heads, head_dim,
                                  head_dim ** -0.5 if scale is None else scale, 1 if causal else 0, out.data_ptr(),
                                  ldo, _stream(stream))
        if st:
            _check(st, "wal_attn_prompt")
    return out


# ---------------------------------------------------------------------------
# Blocks of the gated delta rule.

def _state(T, t, name: str, dtype, shape) -> int:
    """A contiguous device tensor [places][*shape] of what sequences carry between calls: its places."""
    if not isinstance(t, T.tensor):
        raise TypeError(f"{name} must be a torch tensor on the GPU, not {type(t).__name__}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}; expected {dtype}")
    if t.dim() != 1 + len(shape) or tuple(t.shape[1:]) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected [places, {', '.join(map(str, shape))}]")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.shape[0] > _U32_MAX:
        raise ValueError(f"{name} has {t.shape[0]} places: more than 32 bits hold")
    return t.shape[0]


def _gate_mat(T, t, name: str, cols: int, rows: int) -> int:
    """fp32 rows of any pitch: their pitch."""
    return max(_mat(T, t, name, T.only_f32, cols, rows)[2], cols)


def wal_conv(X, weight, starts, out, state=None, slots=None, bias=None, silu: bool = True, stream=None):
    """Causal convolution of each channel over rows packed by sequence: X [n][channels] (bf16 or fp32), weight
    [channels][taps] and bias [channels] (bf16 or fp32), starts int32 [n_seqs + 1], out [n][channels] (bf16 or fp32),
    through silu unless that is False.  state [places][taps - 1][channels] of X's type holds, in place slots[s]
    (int32 [n_seqs]), sequence s's rows before the call, and its last ones after it; None: no rows before."""
    T = _types()
    n, channels, ldx = _mat(T, X, "X", T.acts, 8)
    w_rows, taps, pitch = _mat(T, weight, "weight", T.acts, 1)
    if w_rows != channels:
        raise ValueError(f"weight has {w_rows} rows for {channels} channels")
    if not weight.is_contiguous():
        raise ValueError("weight must be contiguous")
    _, _, ldo = _mat(T, out, "out", T.acts, channels, n)
    n_seqs = _vec(T, starts, "starts", T.i32, 1) - 1
    if (state is None) != (slots is None):
        raise ValueError("state and slots go together")
    st_p = sl_p = bias_p = None
    n_slots = 0
    if state is not None:
        n_slots = _state(T, state, "state", X.dtype, (taps - 1, channels))
        _vec(T, slots, "slots", T.i32, n_seqs)
        if n_slots:
            st_p, sl_p = state.data_ptr(), slots.data_ptr()
    if bias is not None:
        _norm_weight(T, bias, "bias", channels)
        if bias.dtype is not weight.dtype:
            raise TypeError(f"bias has dtype {bias.dtype}, weight {weight.dtype}: they must be the same")
        bias_p = bias.data_ptr()
    if not (X.is_cuda and weight.is_cuda and starts.is_cuda and out.is_cuda and (state is None or (state.is_cuda and slots.is_cuda))
            and (bias is None or bias.is_cuda)):
        _gpu(X=X, weight=weight, starts=starts, out=out, state=state, slots=slots, bias=bias)
    if n and n_seqs:
        st = _lib.wal_conv(X.data_ptr(), X.dtype is T.bf16, n, channels, ldx, weight.data_ptr(), weight.dtype is T.bf16,
                           taps, bias_p, 1 if silu else 0, starts.data_ptr(), n_seqs, st_p, sl_p, n_slots,
                           out.data_ptr(), out.dtype is T.bf16, ldo, _stream(stream))
        if st:
            _check(st, "wal_conv")
    return out


def make_delta_desc(key_heads: int, value_heads: int, key_dim: int, value_dim: int, norm_eps: float = 1e-6,
                    scale: Optional[float] = None) -> wal_delta_desc:
    """scale: 1 / sqrt(key_dim) unless given; norm_eps 0: q and k are taken as they are."""
    return wal_delta_desc(key_heads, value_heads, key_dim, value_dim, norm_eps,
                          (key_dim ** -0.5 if key_dim > 0 else 0.0) if scale is None else scale)


def wal_delta_workspace_size(desc: wal_delta_desc, n_seqs: int, n: int, max_new: int) -> int:
    if not all(0 <= x <= _U32_MAX for x in (n_seqs, n, max_new)):
        raise ValueError(f"n_seqs {n_seqs}, n {n}, max_new {max_new}: more than 32 bits hold")
    b = _SZ()
    _check(_lib.wal_delta_workspace_size(ctypes.byref(desc), n_seqs, n, max_new, ctypes.byref(b)),
           "wal_delta_workspace_size")
    return b.value


def wal_delta(desc: wal_delta_desc, Q, K, V, A, B, starts, out, state=None, slots=None, ws=None, decay=None,
              shift=None, max_new: Optional[int] = None, stream=None):
    """The gated delta rule over rows packed by sequence: Q, K bf16 [n][key_heads * key_dim], V, out bf16
    [n][value_heads * value_dim], A, B fp32 [n][value_heads], starts int32 [n_seqs + 1].  With decay and shift (fp32
    [value_heads]) A and B are what the gates are made of, else the logarithm of the decay and the step themselves.
    state fp32 [places][value_heads][key_dim][value_dim] holds sequence s's state in place slots[s] (int32 [n_seqs]);
    None: every sequence begins with zeros and none is kept.  ws of wal_delta_workspace_size bytes.
    max_new bounds the sequences' rows (rows past it are not computed); left out: as many as Q has."""
    T = _types()
    kw, h, vw = desc.key_heads * desc.key_dim, desc.value_heads, desc.value_heads * desc.value_dim
    n, _, ldq = _mat(T, Q, "Q", T.only_bf16, kw)
    _, _, ldk = _mat(T, K, "K", T.only_bf16, kw, n)
    _, _, ldv = _mat(T, V, "V", T.only_bf16, vw, n)
    lda, ldb = _gate_mat(T, A, "A", h, n), _gate_mat(T, B, "B", h, n)
    _, _, ldo = _mat(T, out, "out", T.only_bf16, vw, n)
    n_seqs = _vec(T, starts, "starts", T.i32, 1) - 1
    if (state is None) != (slots is None):
        raise ValueError("state and slots go together")
    if (decay is None) != (shift is None):
        raise ValueError("decay and shift go together")
    st_p = sl_p = de_p = sh_p = wsp = None
    n_slots = wsb = 0
    if state is not None:
        n_slots = _state(T, state, "state", T.f32, (h, desc.key_dim, desc.value_dim))
        _vec(T, slots, "slots", T.i32, n_seqs)
        if n_slots:
            st_p, sl_p = state.data_ptr(), slots.data_ptr()
    if decay is not None:
        _vec(T, decay, "decay", T.f32, h)
        _vec(T, shift, "shift", T.f32, h)
        de_p, sh_p = decay.data_ptr(), shift.data_ptr()
    if max_new is None:
        max_new = n
    if not 0 <= max_new <= _U32_MAX:
        raise ValueError(f"max_new {max_new}")
    if ws is not None:
        wsb, wsp = _ws_bytes(ws), ws.data_ptr()
    if not (Q.is_cuda and K.is_cuda and V.is_cuda and A.is_cuda and B.is_cuda and starts.is_cuda and out.is_cuda
            and (state is None or (state.is_cuda and slots.is_cuda)) and (decay is None or (decay.is_cuda and shift.is_cuda))
            and (ws is None or ws.is_cuda)):
        _gpu(Q=Q, K=K, V=V, A=A, B=B, starts=starts, out=out, state=state, slots=slots, decay=decay, shift=shift, ws=ws)
    if n and n_seqs:
        st = _lib.wal_delta(desc, Q.data_ptr(), ldq, K.data_ptr(), ldk, V.data_ptr(), ldv, A.data_ptr(), lda,
                            B.data_ptr(), ldb, de_p, sh_p, starts.data_ptr(), n_seqs, n, max_new, st_p, sl_p, n_slots,
                            out.data_ptr(), ldo, wsp, wsb, _stream(stream))
        if st:
            _check(st, "wal_delta")
    return out
