"""ctypes binding of libstief.so: argument marshalling only.

Every function here takes torch tensors, checks dtype / device / contiguity /
shape agreement, and passes raw device pointers, sizes and the current CUDA
stream to the C entry point of the same name.  All arithmetic runs in the
library's CUDA kernels.  There is no fallback path: a missing or unloadable
library raises ``StiefError``.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.environ.get("STIEF_LIBRARY", os.path.join(_PKG, "libstief.so"))

STATUS = {
    0: "STIEF_OK",
    1: "STIEF_ERR_INVALID_ARG",
    2: "STIEF_ERR_ALIGNMENT",
    3: "STIEF_ERR_CAPACITY",
    4: "STIEF_ERR_WORKSPACE",
    5: "STIEF_ERR_CUDA",
    6: "STIEF_ERR_DEVICE_STATUS",
    7: "STIEF_ERR_UNSUPPORTED_DEVICE",
}
DEV_CAPACITY_OVERFLOW = 0x1
DEV_WAIT_TIMEOUT = 0x2
DEV_BAD_LENGTH = 0x4
DEV_TMEM_PAIR = 0x10


class StiefError(RuntimeError):
    """A libstief call returned a non-OK status (or the library is missing)."""

    def __init__(self, func: str, code: int):
        self.code = code
        super().__init__(f"{func}: {STATUS.get(code, code)}")


_lock = threading.Lock()
_lib = None

_u16p = ctypes.c_void_p
_i = ctypes.c_int


def library_path() -> str:
    return _LIB_PATH


def library() -> ctypes.CDLL:
    """Load libstief.so (once).  Raises StiefError if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise StiefError(f"libstief.so not found at {_LIB_PATH}; build it with "
                                 "python -m decode_attention_stief_b200.build", -1)
            lib = ctypes.CDLL(_LIB_PATH)
            vp = ctypes.c_void_p
            lib.stief_compress_append.restype = _i
            lib.stief_compress_append.argtypes = [vp] * 7 + [_i] * 7 + [vp, vp]
            lib.stief_decode_attention.restype = _i
            lib.stief_decode_attention.argtypes = ([vp] * 8 + [ctypes.c_size_t] + [_i] * 9
                                                   + [vp, vp])
            lib.stief_decode_workspace_bytes.restype = ctypes.c_size_t
            lib.stief_decode_workspace_bytes.argtypes = [_i] * 5
            lib.stief_decode_max_splits.restype = _i
            lib.stief_decode_max_splits.argtypes = [_i]
            lib.stief_decode_auto_splits.restype = _i
            lib.stief_decode_auto_splits.argtypes = [_i] * 5
            lib.stief_append_decode.restype = _i
            lib.stief_append_decode.argtypes = ([vp] * 10 + [ctypes.c_size_t] + [_i] * 9
                                                + [vp, vp])
            lib.stief_compress_append_paged.restype = _i
            lib.stief_compress_append_paged.argtypes = [vp] * 8 + [_i] * 9 + [vp, vp]
            lib.stief_decode_attention_paged.restype = _i
            lib.stief_decode_attention_paged.argtypes = ([vp] * 9 + [ctypes.c_size_t] + [_i] * 11
                                                         + [vp, vp])
            lib.stief_append_decode_paged.restype = _i
            lib.stief_append_decode_paged.argtypes = ([vp] * 11 + [ctypes.c_size_t] + [_i] * 11
                                                      + [vp, vp])
            lib.stief_compress_append_q8.restype = _i
            lib.stief_compress_append_q8.argtypes = [vp] * 9 + [_i] * 7 + [vp, vp]
            lib.stief_decode_attention_q8.restype = _i
            lib.stief_decode_attention_q8.argtypes = ([vp] * 10 + [ctypes.c_size_t] + [_i] * 9
                                                      + [vp, vp])
            lib.stief_append_decode_q8.restype = _i
            lib.stief_append_decode_q8.argtypes = ([vp] * 12 + [ctypes.c_size_t] + [_i] * 9
                                                   + [vp, vp])
            lib.stief_compress_append_q8_paged.restype = _i
            lib.stief_compress_append_q8_paged.argtypes = [vp] * 10 + [_i] * 9 + [vp, vp]
            lib.stief_decode_attention_q8_paged.restype = _i
            lib.stief_decode_attention_q8_paged.argtypes = ([vp] * 11 + [ctypes.c_size_t] + [_i] * 11
                                                            + [vp, vp])
            lib.stief_compress_append_q4.restype = _i
            lib.stief_compress_append_q4.argtypes = [vp] * 9 + [_i] * 7 + [vp, vp]
            lib.stief_decode_attention_q4.restype = _i
            lib.stief_decode_attention_q4.argtypes = ([vp] * 10 + [ctypes.c_size_t] + [_i] * 9
                                                      + [vp, vp])
            lib.stief_compress_append_joint_v.restype = _i
            lib.stief_compress_append_joint_v.argtypes = [vp] * 7 + [_i] * 7 + [vp, vp]
            lib.stief_decode_attention_joint_v.restype = _i
            lib.stief_decode_attention_joint_v.argtypes = ([vp] * 8 + [ctypes.c_size_t] + [_i] * 9
                                                           + [vp, vp])
            lib.stief_decode_latent_joint_v.restype = _i
            lib.stief_decode_latent_joint_v.argtypes = ([vp] * 6 + [ctypes.c_size_t] + [_i] * 9
                                                        + [vp, vp])
            lib.stief_decode_latent.restype = _i
            lib.stief_decode_latent.argtypes = ([vp] * 6 + [ctypes.c_size_t] + [_i] * 9
                                                + [vp, vp])
            lib.stief_decode_attention_noalloc.restype = _i
            lib.stief_decode_attention_noalloc.argtypes = [vp] * 7 + [_i] * 9 + [vp, vp]
            i64 = ctypes.c_longlong
            lib.stief_plan_workspace_bytes.restype = ctypes.c_size_t
            lib.stief_plan_workspace_bytes.argtypes = []
            lib.stief_plan_pages.restype = _i
            lib.stief_plan_pages.argtypes = [vp] * 11 + [ctypes.c_size_t] + [_i] * 5 + [vp, vp]
            lib.stief_append_shared_paged.restype = _i
            lib.stief_append_shared_paged.argtypes = ([vp] * 4 + [_i] * 3 + [i64, i64] + [_i] * 2
                                                      + [vp, vp])
            lib.stief_decode_shared_workspace_bytes.restype = ctypes.c_size_t
            lib.stief_decode_shared_workspace_bytes.argtypes = [_i] * 3
            lib.stief_decode_shared_paged.restype = _i
            lib.stief_decode_shared_paged.argtypes = ([vp] * 6 + [ctypes.c_size_t] + [_i] * 8
                                                      + [ctypes.c_float, vp, vp])
            lib.stief_expand_shared_paged.restype = _i
            lib.stief_expand_shared_paged.argtypes = [vp] * 8 + [_i] * 9 + [vp, vp]
            lib.stief_prefill_attention.restype = _i
            lib.stief_prefill_attention.argtypes = ([vp] * 7 + [_i] * 8
                                                    + [ctypes.c_float, vp, vp])
            lib.stief_read_device_status.restype = _i
            lib.stief_read_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), vp]
            lib.stief_status_string.restype = ctypes.c_char_p
            lib.stief_status_string.argtypes = [_i]
            _load_marshal(lib)
            _lib = lib
    return _lib


_marshal = None  # the extension of csrc/marshal.cpp, once the library is loaded


def _load_marshal(lib) -> None:
    """Loads the extension that makes the newer calls without their checks in Python, if it has
    been built, and gives it the library's addresses."""
    global _marshal
    try:
        from . import _marshal as m
    except ImportError:
        return
    m.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
             for n in ("stief_plan_pages", "stief_append_shared_paged", "stief_decode_shared_paged",
                       "stief_expand_shared_paged", "stief_prefill_attention")))
    _marshal = m


def _short_way(stream) -> bool:
    """Whether a call may go through the extension: it knows the current stream only, and
    prepare() wants the arguments, not the call."""
    return _marshal is not None and stream is None and getattr(_capture, "calls", None) is None


def _check(func: str, code: int) -> None:
    if code != 0:
        raise StiefError(func, code)



class Prepared:
    """A library call validated once (see prepare): calling it launches the same call again with
    the same device pointers, sizes and stream, at the C call's own host cost.  It keeps the
    argument tensors alive; their storage, shapes and contents-to-be are the caller's to keep
    as they were when it was prepared (in-place updates of their values are what it is for)."""

    __slots__ = ("name", "_fn", "_cargs", "_keep")

    def __init__(self, name, cargs, keep):
        self.name = name
        self._fn = getattr(library(), name)
        self._cargs = cargs
        self._keep = keep

    def __call__(self):
        code = self._fn(*self._cargs)
        if code != 0:
            raise StiefError(self.name, code)


_capture = threading.local()


def _invoke(name: str, cargs: tuple) -> None:
    """Calls the library entry point `name` with the marshalled arguments, or, while prepare()
    is capturing, records them instead."""
    if getattr(_capture, "calls", None) is not None:
        _capture.calls.append((name, cargs))
        return
    _check(name, getattr(library(), name)(*cargs))


def prepare(fn, *args, **kwargs) -> Prepared:
    """Validates and marshals the arguments of the binding function `fn` (e.g.
    stief_append_decode) exactly as calling it would, without launching anything, and returns
    a Prepared call: a serving loop that reuses the same buffers every step calls that object
    instead, skipping the per-call checks (the library still validates sizes on every call).
    The stream is the one given, or the current stream at preparation."""
    _capture.calls = []
    try:
        fn(*args, **kwargs)
        calls = _capture.calls
    finally:
        _capture.calls = None
    if len(calls) != 1:
        raise ValueError(f"{getattr(fn, '__name__', fn)} makes {len(calls)} library calls; prepare takes one")
    name, cargs = calls[0]
    return Prepared(name, cargs, (args, kwargs))

def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _opt_status(dev_status: Optional[torch.Tensor]) -> Optional[int]:
    if dev_status is None:
        return None
    if dev_status.dtype not in (torch.int32, torch.uint32) or dev_status.numel() < 1 or not dev_status.is_cuda:
        raise ValueError("dev_status must be a CUDA int32/uint32 tensor with at least one element")
    return dev_status.data_ptr()


def stief_status_string(code: int) -> str:
    return library().stief_status_string(int(code)).decode()


def stief_decode_max_splits(max_seq_len: int) -> int:
    return int(library().stief_decode_max_splits(int(max_seq_len)))


def stief_decode_auto_splits(B: int, Hq: int, Hkv: int, max_seq_len: int, num_sms: int) -> int:
    return int(library().stief_decode_auto_splits(B, Hq, Hkv, max_seq_len, num_sms))


def stief_decode_workspace_bytes(B: int, Hq: int, Hkv: int, rV: int, max_seq_len: int) -> int:
    return int(library().stief_decode_workspace_bytes(B, Hq, Hkv, rV, max_seq_len))


def workspace_for(B: int, Hq: int, Hkv: int, rV: int, max_seq_len: int,
                  device="cuda") -> torch.Tensor:
    """A zero-filled uint8 device tensor of stief_decode_workspace_bytes(...) bytes.

    Zero-filled once here; every completed decode call leaves its ticket counters at
    zero, so the tensor can be reused for any later call on the same stream.
    """
    n = stief_decode_workspace_bytes(B, Hq, Hkv, rV, max_seq_len)
    if n == 0:
        raise ValueError("invalid sizes for the decode workspace")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def stief_compress_append(k_new: torch.Tensor, v_new: torch.Tensor, P_K: torch.Tensor,
                          P_V: torch.Tensor, k_lat: torch.Tensor, v_lat: torch.Tensor,
                          seq_lens: torch.Tensor, dev_status: Optional[torch.Tensor] = None,
                          stream=None) -> None:
    """Project T new rows per (sequence, KV head) into the latent cache and advance seq_lens.

    k_new, v_new [B][Hkv][T][d] bf16; P_K [Hkv][d][rK], P_V [Hkv][d][rV] bf16;
    k_lat [B][Hkv][L_max][rK], v_lat [B][Hkv][L_max][rV] bf16; seq_lens [B] int32.
    """
    pk = _dev(k_new, "k_new", torch.bfloat16, 4)
    pv = _dev(v_new, "v_new", torch.bfloat16, 4)
    ppk = _dev(P_K, "P_K", torch.bfloat16, 3)
    ppv = _dev(P_V, "P_V", torch.bfloat16, 3)
    pkl = _dev(k_lat, "k_lat", torch.bfloat16, 4)
    pvl = _dev(v_lat, "v_lat", torch.bfloat16, 4)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    B, Hkv, T, d = k_new.shape
    rK, rV = P_K.shape[2], P_V.shape[2]
    L_max = k_lat.shape[2]
    if tuple(v_new.shape) != (B, Hkv, T, d) or tuple(P_K.shape) != (Hkv, d, rK) \
            or tuple(P_V.shape) != (Hkv, d, rV) or tuple(k_lat.shape) != (B, Hkv, L_max, rK) \
            or tuple(v_lat.shape) != (B, Hkv, L_max, rV) or seq_lens.shape[0] != B:
        raise ValueError("stief_compress_append: inconsistent shapes")
    _invoke("stief_compress_append", (pk, pv, ppk, ppv, pkl, pvl, psl, B, Hkv, T, d, rK,
                                           rV, L_max, _opt_status(dev_status),
                                           _stream_ptr(stream),))


def stief_decode_attention(q: torch.Tensor, P_K: torch.Tensor, P_V: torch.Tensor,
                           k_lat: torch.Tensor, v_lat: torch.Tensor, seq_lens: torch.Tensor,
                           out: torch.Tensor, workspace: torch.Tensor, max_seq_len: int,
                           num_splits: int = 0, dev_status: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """One decode step: out [B][Hq][d] = softmax(q K~^T / sqrt(d)) V~ over the latent cache.

    q [B][Hq][d] bf16; P_K [Hkv][d][rK], P_V [Hkv][d][rV] bf16;
    k_lat [B][Hkv][L_max][rK], v_lat [B][Hkv][L_max][rV] bf16; seq_lens [B] int32;
    out [B][Hq][d] bf16 (written); workspace: uint8 device tensor of at least
    stief_decode_workspace_bytes(...) bytes.
    """
    pq = _dev(q, "q", torch.bfloat16, 3)
    ppk = _dev(P_K, "P_K", torch.bfloat16, 3)
    ppv = _dev(P_V, "P_V", torch.bfloat16, 3)
    pkl = _dev(k_lat, "k_lat", torch.bfloat16, 4)
    pvl = _dev(v_lat, "v_lat", torch.bfloat16, 4)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    po = _dev(out, "out", torch.bfloat16, 3)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    B, Hq, d = q.shape
    Hkv, _, rK = P_K.shape
    rV = P_V.shape[2]
    L_max = k_lat.shape[2]
    if tuple(P_K.shape) != (Hkv, d, rK) or tuple(P_V.shape) != (Hkv, d, rV) \
            or tuple(k_lat.shape) != (B, Hkv, L_max, rK) \
            or tuple(v_lat.shape) != (B, Hkv, L_max, rV) or seq_lens.shape[0] != B \
            or tuple(out.shape) != (B, Hq, d):
        raise ValueError("stief_decode_attention: inconsistent shapes")
    ws_bytes = workspace.numel() * workspace.element_size()
    _invoke("stief_decode_attention", (pq, ppk, ppv, pkl, pvl, psl, po,
                                            workspace.data_ptr(), ws_bytes, B, Hq, Hkv, d, rK,
                                            rV, L_max, int(max_seq_len), int(num_splits),
                                            _opt_status(dev_status), _stream_ptr(stream),))
    return out


def stief_append_decode(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                        P_K: torch.Tensor, P_V: torch.Tensor, k_lat: torch.Tensor,
                        v_lat: torch.Tensor, seq_lens: torch.Tensor, out: torch.Tensor,
                        workspace: torch.Tensor, max_seq_len: int, num_splits: int = 0,
                        dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One whole decode step in one kernel: append the new token's compressed key and value
    rows (k_new P_K, v_new P_V at row seq_lens[b]), attend over the grown cache, and
    increment seq_lens.

    q [B][Hq][d] bf16; k_new, v_new [B][Hkv][d] (or [B][Hkv][1][d]) bf16; the other
    arguments as for stief_decode_attention; max_seq_len bounds the lengths after the append.
    """
    pq = _dev(q, "q", torch.bfloat16, 3)
    kn = k_new.reshape(k_new.shape[0], k_new.shape[1], -1) if k_new.dim() == 4 else k_new
    vn = v_new.reshape(v_new.shape[0], v_new.shape[1], -1) if v_new.dim() == 4 else v_new
    pkn = _dev(kn, "k_new", torch.bfloat16, 3)
    pvn = _dev(vn, "v_new", torch.bfloat16, 3)
    ppk = _dev(P_K, "P_K", torch.bfloat16, 3)
    ppv = _dev(P_V, "P_V", torch.bfloat16, 3)
    pkl = _dev(k_lat, "k_lat", torch.bfloat16, 4)
    pvl = _dev(v_lat, "v_lat", torch.bfloat16, 4)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    po = _dev(out, "out", torch.bfloat16, 3)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    B, Hq, d = q.shape
    Hkv, _, rK = P_K.shape
    rV = P_V.shape[2]
    L_max = k_lat.shape[2]
    if tuple(P_K.shape) != (Hkv, d, rK) or tuple(P_V.shape) != (Hkv, d, rV) \
            or tuple(kn.shape) != (B, Hkv, d) or tuple(vn.shape) != (B, Hkv, d) \
            or tuple(k_lat.shape) != (B, Hkv, L_max, rK) \
            or tuple(v_lat.shape) != (B, Hkv, L_max, rV) or seq_lens.shape[0] != B \
            or tuple(out.shape) != (B, Hq, d):
        raise ValueError("stief_append_decode: inconsistent shapes")
    ws_bytes = workspace.numel() * workspace.element_size()
    _invoke("stief_append_decode", (pq, pkn, pvn, ppk, ppv, pkl, pvl, psl, po,
                                         workspace.data_ptr(), ws_bytes, B, Hq, Hkv, d, rK, rV,
                                         L_max, int(max_seq_len), int(num_splits),
                                         _opt_status(dev_status), _stream_ptr(stream),))
    return out


def _pages(k_pages, v_pages, block_table, B):
    """Pointers and sizes of a paged cache: pools [num_pages][Hkv][page_size][r] bf16 and a
    block table [B][max_pages] int32."""
    pkp = _dev(k_pages, "k_pages", torch.bfloat16, 4)
    pvp = _dev(v_pages, "v_pages", torch.bfloat16, 4)
    pbt = _dev(block_table, "block_table", torch.int32, 2)
    num_pages, Hkv, page_size, rK = k_pages.shape
    rV = v_pages.shape[3]
    if tuple(v_pages.shape) != (num_pages, Hkv, page_size, rV) or block_table.shape[0] != B:
        raise ValueError("paged cache: inconsistent shapes")
    return pkp, pvp, pbt, num_pages, Hkv, page_size, rK, rV, block_table.shape[1]


def stief_compress_append_paged(k_new, v_new, P_K, P_V, k_pages, v_pages, block_table, seq_lens,
                                dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """stief_compress_append into a paged cache (pools [num_pages][Hkv][page_size][r], block
    table [B][max_pages])."""
    pk = _dev(k_new, "k_new", torch.bfloat16, 4)
    pv = _dev(v_new, "v_new", torch.bfloat16, 4)
    ppk = _dev(P_K, "P_K", torch.bfloat16, 3)
    ppv = _dev(P_V, "P_V", torch.bfloat16, 3)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    B, Hkv, T, d = k_new.shape
    pkp, pvp, pbt, num_pages, Hkv2, page_size, rK, rV, max_pages = _pages(k_pages, v_pages,
                                                                          block_table, B)
    if Hkv2 != Hkv or tuple(P_K.shape) != (Hkv, d, rK) or tuple(P_V.shape) != (Hkv, d, rV) \
            or tuple(v_new.shape) != (B, Hkv, T, d) or seq_lens.shape[0] != B:
        raise ValueError("stief_compress_append_paged: inconsistent shapes")
    _invoke("stief_compress_append_paged", (pk, pv, ppk, ppv, pkp, pvp, pbt, psl, B, Hkv, T,
                                                 d, rK, rV, num_pages, page_size, max_pages,
                                                 _opt_status(dev_status), _stream_ptr(stream),))


def stief_decode_attention_paged(q, P_K, P_V, k_pages, v_pages, block_table, seq_lens, out,
                                 workspace, max_seq_len: int, num_splits: int = 0,
                                 dev_status: Optional[torch.Tensor] = None, stream=None):
    """stief_decode_attention over a paged cache."""
    pq = _dev(q, "q", torch.bfloat16, 3)
    ppk = _dev(P_K, "P_K", torch.bfloat16, 3)
    ppv = _dev(P_V, "P_V", torch.bfloat16, 3)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    po = _dev(out, "out", torch.bfloat16, 3)
    B, Hq, d = q.shape
    pkp, pvp, pbt, num_pages, Hkv, page_size, rK, rV, max_pages = _pages(k_pages, v_pages,
                                                                         block_table, B)
    if tuple(P_K.shape) != (Hkv, d, rK) or tuple(P_V.shape) != (Hkv, d, rV) \
            or seq_lens.shape[0] != B or tuple(out.shape) != (B, Hq, d):
        raise ValueError("stief_decode_attention_paged: inconsistent shapes")
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    ws_bytes = workspace.numel() * workspace.element_size()
    _invoke("stief_decode_attention_paged", (pq, ppk, ppv, pkp, pvp, pbt, psl, po,
                                                  workspace.data_ptr(), ws_bytes, B, Hq, Hkv, d,
                                                  rK, rV, num_pages, page_size, max_pages,
                                                  int(max_seq_len), int(num_splits),
                                                  _opt_status(dev_status), _stream_ptr(stream),))
    return out


def stief_append_decode_paged(q, k_new, v_new, P_K, P_V, k_pages, v_pages, block_table, seq_lens,
                              out, workspace, max_seq_len: int, num_splits: int = 0,
                              dev_status: Optional[torch.Tensor] = None, stream=None):
    """stief_append_decode over a paged cache."""
    pq = _dev(q, "q", torch.bfloat16, 3)
    kn = k_new.reshape(k_new.shape[0], k_new.shape[1], -1) if k_new.dim() == 4 else k_new
    vn = v_new.reshape(v_new.shape[0], v_new.shape[1], -1) if v_new.dim() == 4 else v_new
    pkn = _dev(kn, "k_new", torch.bfloat16, 3)
    pvn = _dev(vn, "v_new", torch.bfloat16, 3)
    ppk = _dev(P_K, "P_K", torch.bfloat16, 3)
    ppv = _dev(P_V, "P_V", torch.bfloat16, 3)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    po = _dev(out, "out", torch.bfloat16, 3)
    B, Hq, d = q.shape
    pkp, pvp, pbt, num_pages, Hkv, page_size, rK, rV, max_pages = _pages(k_pages, v_pages,
                                                                         block_table, B)
    if tuple(kn.shape) != (B, Hkv, d) or tuple(vn.shape) != (B, Hkv, d) \
            or tuple(P_K.shape) != (Hkv, d, rK) or tuple(P_V.shape) != (Hkv, d, rV) \
            or seq_lens.shape[0] != B or tuple(out.shape) != (B, Hq, d):
        raise ValueError("stief_append_decode_paged: inconsistent shapes")
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    ws_bytes = workspace.numel() * workspace.element_size()
    _invoke("stief_append_decode_paged", (pq, pkn, pvn, ppk, ppv, pkp, pvp, pbt, psl, po,
                                               workspace.data_ptr(), ws_bytes, B, Hq, Hkv, d, rK,
                                               rV, num_pages, page_size, max_pages,
                                               int(max_seq_len), int(num_splits),
                                               _opt_status(dev_status), _stream_ptr(stream),))
    return out


def stief_compress_append_q8(k_new, v_new, P_K, P_V, k_q, v_q, k_s, v_s, seq_lens,
                             dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """stief_compress_append into an int8 cache: codes k_q [B][Hkv][L_max][rK] (int8) and row
    scales k_s [B][Hkv][L_max] (float32), likewise v_q, v_s; L_max a multiple of 64."""
    pk = _dev(k_new, "k_new", torch.bfloat16, 4)
    pv = _dev(v_new, "v_new", torch.bfloat16, 4)
    ppk = _dev(P_K, "P_K", torch.bfloat16, 3)
    ppv = _dev(P_V, "P_V", torch.bfloat16, 3)
    pkq = _dev(k_q, "k_q", torch.int8, 4)
    pvq = _dev(v_q, "v_q", torch.int8, 4)
    pks = _dev(k_s, "k_s", torch.float32, 3)
    pvs = _dev(v_s, "v_s", torch.float32, 3)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    B, Hkv, T, d = k_new.shape
    rK, rV = P_K.shape[2], P_V.shape[2]
    L_max = k_q.shape[2]
    if tuple(v_new.shape) != (B, Hkv, T, d) or tuple(P_K.shape) != (Hkv, d, rK) \
            or tuple(P_V.shape) != (Hkv, d, rV) or tuple(k_q.shape) != (B, Hkv, L_max, rK) \
            or tuple(v_q.shape) != (B, Hkv, L_max, rV) or tuple(k_s.shape) != (B, Hkv, L_max) \
            or tuple(v_s.shape) != (B, Hkv, L_max) or seq_lens.shape[0] != B:
        raise ValueError("stief_compress_append_q8: inconsistent shapes")
    _invoke("stief_compress_append_q8", (pk, pv, ppk, ppv, pkq, pvq, pks, pvs, psl, B, Hkv, T,
                                              d, rK, rV, L_max, _opt_status(dev_status),
                                              _stream_ptr(stream),))


def stief_decode_attention_q8(q, P_K, P_V, k_q, v_q, k_s, v_s, seq_lens, out, workspace,
                              max_seq_len: int, num_splits: int = 0,
                              dev_status: Optional[torch.Tensor] = None, stream=None):
    """stief_decode_attention over an int8 cache (codes and row scales as for
    stief_compress_append_q8)."""
    pq = _dev(q, "q", torch.bfloat16, 3)
    ppk = _dev(P_K, "P_K", torch.bfloat16, 3)
    ppv = _dev(P_V, "P_V", torch.bfloat16, 3)
    pkq = _dev(k_q, "k_q", torch.int8, 4)
    pvq = _dev(v_q, "v_q", torch.int8, 4)
    pks = _dev(k_s, "k_s", torch.float32, 3)
    pvs = _dev(v_s, "v_s", torch.float32, 3)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    po = _dev(out, "out", torch.bfloat16, 3)
    B, Hq, d = q.shape
    Hkv, _, rK = P_K.shape
    rV = P_V.shape[2]
    L_max = k_q.shape[2]
    if tuple(P_V.shape) != (Hkv, d, rV) or tuple(k_q.shape) != (B, Hkv, L_max, rK) \
            or tuple(v_q.shape) != (B, Hkv, L_max, rV) or tuple(k_s.shape) != (B, Hkv, L_max) \
            or tuple(v_s.shape) != (B, Hkv, L_max) or seq_lens.shape[0] != B \
            or tuple(out.shape) != (B, Hq, d):
        raise ValueError("stief_decode_attention_q8: inconsistent shapes")
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    ws_bytes = workspace.numel() * workspace.element_size()
    _invoke("stief_decode_attention_q8", (pq, ppk, ppv, pkq, pvq, pks, pvs, psl, po,
                                               workspace.data_ptr(), ws_bytes, B, Hq, Hkv, d, rK,
                                               rV, L_max, int(max_seq_len), int(num_splits),
                                               _opt_status(dev_status), _stream_ptr(stream),))
    return out


def stief_append_decode_q8(q, k_new, v_new, P_K, P_V, k_q, v_q, k_s, v_s, seq_lens, out,
                           workspace, max_seq_len: int, num_splits: int = 0,
                           dev_status: Optional[torch.Tensor] = None, stream=None):
    """stief_append_decode on an int8 cache: the new token's rows are quantised into k_q, v_q
    (codes) and k_s, v_s (row scales) at row seq_lens[b] as stief_compress_append_q8 stores
    them, the decode attends over the grown cache, and seq_lens is incremented.  k_new, v_new
    [B][Hkv][d] (or [B][Hkv][1][d]) bf16; the rest as for stief_decode_attention_q8."""
    pq = _dev(q, "q", torch.bfloat16, 3)
    kn = k_new.reshape(k_new.shape[0], k_new.shape[1], -1) if k_new.dim() == 4 else k_new
    vn = v_new.reshape(v_new.shape[0], v_new.shape[1], -1) if v_new.dim() == 4 else v_new
    pkn = _dev(kn, "k_new", torch.bfloat16, 3)
    pvn = _dev(vn, "v_new", torch.bfloat16, 3)
    ppk = _dev(P_K, "P_K", torch.bfloat16, 3)
    ppv = _dev(P_V, "P_V", torch.bfloat16, 3)
    pkq = _dev(k_q, "k_q", torch.int8, 4)
    pvq = _dev(v_q, "v_q", torch.int8, 4)
    pks = _dev(k_s, "k_s", torch.float32, 3)
    pvs = _dev(v_s, "v_s", torch.float32, 3)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    po = _dev(out, "out", torch.bfloat16, 3)
    B, Hq, d = q.shape
    Hkv, _, rK = P_K.shape
    rV = P_V.shape[2]
    L_max = k_q.shape[2]
    if tuple(P_V.shape) != (Hkv, d, rV) or tuple(kn.shape) != (B, Hkv, d) \
            or tuple(vn.shape) != (B, Hkv, d) or tuple(k_q.shape) != (B, Hkv, L_max, rK) \
            or tuple(v_q.shape) != (B, Hkv, L_max, rV) or tuple(k_s.shape) != (B, Hkv, L_max) \
            or tuple(v_s.shape) != (B, Hkv, L_max) or seq_lens.shape[0] != B \
            or tuple(out.shape) != (B, Hq, d):
        raise ValueError("stief_append_decode_q8: inconsistent shapes")
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    ws_bytes = workspace.numel() * workspace.element_size()
    _invoke("stief_append_decode_q8", (pq, pkn, pvn, ppk, ppv, pkq, pvq, pks, pvs, psl, po,
                                       workspace.data_ptr(), ws_bytes, B, Hq, Hkv, d, rK, rV,
                                       L_max, int(max_seq_len), int(num_splits),
                                       _opt_status(dev_status), _stream_ptr(stream),))
    return out


def stief_compress_append_q8_paged(k_new, v_new, P_K, P_V, k_pages, v_pages, k_s_pages,
                                   v_s_pages, block_table, seq_lens,
                                   dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """stief_compress_append into int8 page pools: codes k_pages [num_pages][Hkv][page_size][rK]
    (int8) and row scales k_s_pages [num_pages][Hkv][page_size] (float32), likewise the values;
    block_table [B][max_pages] int32."""
    pk = _dev(k_new, "k_new", torch.bfloat16, 4)
    pv = _dev(v_new, "v_new", torch.bfloat16, 4)
    ppk = _dev(P_K, "P_K", torch.bfloat16, 3)
    ppv = _dev(P_V, "P_V", torch.bfloat16, 3)
    pkq = _dev(k_pages, "k_pages", torch.int8, 4)
    pvq = _dev(v_pages, "v_pages", torch.int8, 4)
    pks = _dev(k_s_pages, "k_s_pages", torch.float32, 3)
    pvs = _dev(v_s_pages, "v_s_pages", torch.float32, 3)
    pbt = _dev(block_table, "block_table", torch.int32, 2)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    B, Hkv, T, d = k_new.shape
    rK, rV = P_K.shape[2], P_V.shape[2]
    num_pages, _, page_size, _ = k_pages.shape
    max_pages = block_table.shape[1]
    if tuple(v_new.shape) != (B, Hkv, T, d) or tuple(P_K.shape) != (Hkv, d, rK) \
            or tuple(P_V.shape) != (Hkv, d, rV) \
            or tuple(k_pages.shape) != (num_pages, Hkv, page_size, rK) \
            or tuple(v_pages.shape) != (num_pages, Hkv, page_size, rV) \
            or tuple(k_s_pages.shape) != (num_pages, Hkv, page_size) \
            or tuple(v_s_pages.shape) != (num_pages, Hkv, page_size) \
            or block_table.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("stief_compress_append_q8_paged: inconsistent shapes")
    _invoke("stief_compress_append_q8_paged", (pk, pv, ppk, ppv, pkq, pvq, pks, pvs, pbt, psl,
                                                    B, Hkv, T, d, rK, rV, num_pages, page_size,
                                                    max_pages, _opt_status(dev_status),
                                                    _stream_ptr(stream),))


def stief_decode_attention_q8_paged(q, P_K, P_V, k_pages, v_pages, k_s_pages, v_s_pages,
                                    block_table, seq_lens, out, workspace, max_seq_len: int,
                                    num_splits: int = 0,
                                    dev_status: Optional[torch.Tensor] = None, stream=None):
    """stief_decode_attention over int8 page pools (as for stief_compress_append_q8_paged)."""
    pq = _dev(q, "q", torch.bfloat16, 3)
    ppk = _dev(P_K, "P_K", torch.bfloat16, 3)
    ppv = _dev(P_V, "P_V", torch.bfloat16, 3)
    pkq = _dev(k_pages, "k_pages", torch.int8, 4)
    pvq = _dev(v_pages, "v_pages", torch.int8, 4)
    pks = _dev(k_s_pages, "k_s_pages", torch.float32, 3)
    pvs = _dev(v_s_pages, "v_s_pages", torch.float32, 3)
    pbt = _dev(block_table, "block_table", torch.int32, 2)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    po = _dev(out, "out", torch.bfloat16, 3)
    B, Hq, d = q.shape
    Hkv, _, rK = P_K.shape
    rV = P_V.shape[2]
    num_pages, _, page_size, _ = k_pages.shape
    max_pages = block_table.shape[1]
    if tuple(P_V.shape) != (Hkv, d, rV) or tuple(k_pages.shape) != (num_pages, Hkv, page_size, rK) \
            or tuple(v_pages.shape) != (num_pages, Hkv, page_size, rV) \
            or tuple(k_s_pages.shape) != (num_pages, Hkv, page_size) \
            or tuple(v_s_pages.shape) != (num_pages, Hkv, page_size) \
            or block_table.shape[0] != B or seq_lens.shape[0] != B or tuple(out.shape) != (B, Hq, d):
        raise ValueError("stief_decode_attention_q8_paged: inconsistent shapes")
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    ws_bytes = workspace.numel() * workspace.element_size()
    _invoke("stief_decode_attention_q8_paged", (pq, ppk, ppv, pkq, pvq, pks, pvs, pbt, psl, po,
                                                     workspace.data_ptr(), ws_bytes, B, Hq, Hkv, d,
                                                     rK, rV, num_pages, page_size, max_pages,
                                                     int(max_seq_len), int(num_splits),
                                                     _opt_status(dev_status), _stream_ptr(stream),))
    return out


def stief_compress_append_q4(k_new, v_new, P_K, P_V, k_q, v_q, k_s, v_s, seq_lens,
                             dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """stief_compress_append into a 4-bit cache: codes k_q [B][Hkv][L_max][rK / 2] (uint8, two
    per byte) and row scales k_s [B][Hkv][L_max] (float32), likewise v_q, v_s; ranks multiples
    of 32, L_max a multiple of 64."""
    pk = _dev(k_new, "k_new", torch.bfloat16, 4)
    pv = _dev(v_new, "v_new", torch.bfloat16, 4)
    ppk = _dev(P_K, "P_K", torch.bfloat16, 3)
    ppv = _dev(P_V, "P_V", torch.bfloat16, 3)
    pkq = _dev(k_q, "k_q", torch.uint8, 4)
    pvq = _dev(v_q, "v_q", torch.uint8, 4)
    pks = _dev(k_s, "k_s", torch.float32, 3)
    pvs = _dev(v_s, "v_s", torch.float32, 3)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    B, Hkv, T, d = k_new.shape
    rK, rV = P_K.shape[2], P_V.shape[2]
    L_max = k_q.shape[2]
    if tuple(v_new.shape) != (B, Hkv, T, d) or tuple(P_K.shape) != (Hkv, d, rK) \
            or tuple(P_V.shape) != (Hkv, d, rV) or tuple(k_q.shape) != (B, Hkv, L_max, rK // 2) \
            or tuple(v_q.shape) != (B, Hkv, L_max, rV // 2) or tuple(k_s.shape) != (B, Hkv, L_max) \
            or tuple(v_s.shape) != (B, Hkv, L_max) or seq_lens.shape[0] != B:
        raise ValueError("stief_compress_append_q4: inconsistent shapes")
    _invoke("stief_compress_append_q4", (pk, pv, ppk, ppv, pkq, pvq, pks, pvs, psl, B, Hkv, T,
                                              d, rK, rV, L_max, _opt_status(dev_status),
                                              _stream_ptr(stream),))


def stief_decode_attention_q4(q, P_K, P_V, k_q, v_q, k_s, v_s, seq_lens, out, workspace,
                              max_seq_len: int, num_splits: int = 0,
                              dev_status: Optional[torch.Tensor] = None, stream=None):
    """stief_decode_attention over a 4-bit cache (codes and row scales as for
    stief_compress_append_q4)."""
    pq = _dev(q, "q", torch.bfloat16, 3)
    ppk = _dev(P_K, "P_K", torch.bfloat16, 3)
    ppv = _dev(P_V, "P_V", torch.bfloat16, 3)
    pkq = _dev(k_q, "k_q", torch.uint8, 4)
    pvq = _dev(v_q, "v_q", torch.uint8, 4)
    pks = _dev(k_s, "k_s", torch.float32, 3)
    pvs = _dev(v_s, "v_s", torch.float32, 3)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    po = _dev(out, "out", torch.bfloat16, 3)
    B, Hq, d = q.shape
    Hkv, _, rK = P_K.shape
    rV = P_V.shape[2]
    L_max = k_q.shape[2]
    if tuple(P_V.shape) != (Hkv, d, rV) or tuple(k_q.shape) != (B, Hkv, L_max, rK // 2) \
            or tuple(v_q.shape) != (B, Hkv, L_max, rV // 2) or tuple(k_s.shape) != (B, Hkv, L_max) \
            or tuple(v_s.shape) != (B, Hkv, L_max) or seq_lens.shape[0] != B \
            or tuple(out.shape) != (B, Hq, d):
        raise ValueError("stief_decode_attention_q4: inconsistent shapes")
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    ws_bytes = workspace.numel() * workspace.element_size()
    _invoke("stief_decode_attention_q4", (pq, ppk, ppv, pkq, pvq, pks, pvs, psl, po,
                                               workspace.data_ptr(), ws_bytes, B, Hq, Hkv, d, rK,
                                               rV, L_max, int(max_seq_len), int(num_splits),
                                               _opt_status(dev_status), _stream_ptr(stream),))
    return out


def stief_decode_latent(q_lat: torch.Tensor, k_lat: torch.Tensor, v_lat: torch.Tensor,
                        seq_lens: torch.Tensor, out_lat: torch.Tensor, workspace: torch.Tensor,
                        max_seq_len: int, num_splits: int = 0, d: int = 128,
                        dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The decode step in the latent space (bases folded into the attention weights):
    out_lat [B][Hq][rV] = softmax(q_lat k_lat^T / sqrt(d)) v_lat.

    q_lat [B][Hq][rK] bf16; k_lat [B][Hkv][L_max][rK], v_lat [B][Hkv][L_max][rV] bf16;
    seq_lens [B] int32; out_lat [B][Hq][rV] bf16 (written); d the head dimension (score
    scale); workspace as for stief_decode_attention.
    """
    pq = _dev(q_lat, "q_lat", torch.bfloat16, 3)
    pkl = _dev(k_lat, "k_lat", torch.bfloat16, 4)
    pvl = _dev(v_lat, "v_lat", torch.bfloat16, 4)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    po = _dev(out_lat, "out_lat", torch.bfloat16, 3)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    B, Hq, rK = q_lat.shape
    Hkv, L_max = k_lat.shape[1], k_lat.shape[2]
    rV = v_lat.shape[3]
    if tuple(k_lat.shape) != (B, Hkv, L_max, rK) or tuple(v_lat.shape) != (B, Hkv, L_max, rV) \
            or seq_lens.shape[0] != B or tuple(out_lat.shape) != (B, Hq, rV):
        raise ValueError("stief_decode_latent: inconsistent shapes")
    ws_bytes = workspace.numel() * workspace.element_size()
    _invoke("stief_decode_latent", (pq, pkl, pvl, psl, po, workspace.data_ptr(), ws_bytes,
                                         B, Hq, Hkv, int(d), rK, rV, L_max, int(max_seq_len),
                                         int(num_splits), _opt_status(dev_status),
                                         _stream_ptr(stream),))
    return out_lat


def stief_decode_attention_noalloc(q: torch.Tensor, P_K: torch.Tensor, P_V: torch.Tensor,
                                   k_lat: torch.Tensor, v_lat: torch.Tensor,
                                   seq_lens: torch.Tensor, out: torch.Tensor, max_seq_len: int,
                                   num_splits: int = 0, dev_status: Optional[torch.Tensor] = None,
                                   stream=None) -> torch.Tensor:
    """stief_decode_attention for callers that cannot allocate: no workspace argument.

    The library keeps the split partial states in its own fixed 8 MiB device array
    (one per GPU); calls that overlap on the GPU race on it.  Raises StiefError
    (STIEF_ERR_WORKSPACE) when the sizes need more than that.
    """
    pq = _dev(q, "q", torch.bfloat16, 3)
    ppk = _dev(P_K, "P_K", torch.bfloat16, 3)
    ppv = _dev(P_V, "P_V", torch.bfloat16, 3)
    pkl = _dev(k_lat, "k_lat", torch.bfloat16, 4)
    pvl = _dev(v_lat, "v_lat", torch.bfloat16, 4)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    po = _dev(out, "out", torch.bfloat16, 3)
    B, Hq, d = q.shape
    Hkv, _, rK = P_K.shape
    rV = P_V.shape[2]
    L_max = k_lat.shape[2]
    if tuple(P_K.shape) != (Hkv, d, rK) or tuple(P_V.shape) != (Hkv, d, rV) \
            or tuple(k_lat.shape) != (B, Hkv, L_max, rK) \
            or tuple(v_lat.shape) != (B, Hkv, L_max, rV) or seq_lens.shape[0] != B \
            or tuple(out.shape) != (B, Hq, d):
        raise ValueError("stief_decode_attention_noalloc: inconsistent shapes")
    _invoke("stief_decode_attention_noalloc", (pq, ppk, ppv, pkl, pvl, psl, po, B, Hq, Hkv,
                                                    d, rK, rV, L_max, int(max_seq_len),
                                                    int(num_splits), _opt_status(dev_status),
                                                    _stream_ptr(stream),))
    return out


def stief_read_device_status(dev_status: torch.Tensor, stream=None) -> int:
    """Synchronise the stream and return the device status word (0 = no condition seen)."""
    v = ctypes.c_uint32(0)
    code = library().stief_read_device_status(_opt_status(dev_status), ctypes.byref(v),
                                              _stream_ptr(stream))
    if code not in (0, 6):
        raise StiefError("stief_read_device_status", code)
    return int(v.value)


def stief_decode_attention_joint_v(q: torch.Tensor, P_K: torch.Tensor, P_VJ: torch.Tensor,
                                   k_lat: torch.Tensor, v_joint: torch.Tensor,
                                   seq_lens: torch.Tensor, out: torch.Tensor,
                                   workspace: torch.Tensor, max_seq_len: int, num_splits: int = 0,
                                   dev_status: Optional[torch.Tensor] = None,
                                   stream=None) -> torch.Tensor:
    """stief_decode_attention with a joint value latent: P_VJ [Hkv*d][rV] bf16 over the
    concatenated KV-head values, v_joint [B][L_max][rV] bf16 (one row per token, shared by the
    KV heads); keys, q, out and the workspace as for stief_decode_attention."""
    pq = _dev(q, "q", torch.bfloat16, 3)
    ppk = _dev(P_K, "P_K", torch.bfloat16, 3)
    ppv = _dev(P_VJ, "P_VJ", torch.bfloat16, 2)
    pkl = _dev(k_lat, "k_lat", torch.bfloat16, 4)
    pvl = _dev(v_joint, "v_joint", torch.bfloat16, 3)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    po = _dev(out, "out", torch.bfloat16, 3)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    B, Hq, d = q.shape
    Hkv, _, rK = P_K.shape
    rV = P_VJ.shape[1]
    L_max = k_lat.shape[2]
    if tuple(P_K.shape) != (Hkv, d, rK) or tuple(P_VJ.shape) != (Hkv * d, rV) \
            or tuple(k_lat.shape) != (B, Hkv, L_max, rK) \
            or tuple(v_joint.shape) != (B, L_max, rV) or seq_lens.shape[0] != B \
            or tuple(out.shape) != (B, Hq, d):
        raise ValueError("stief_decode_attention_joint_v: inconsistent shapes")
    ws_bytes = workspace.numel() * workspace.element_size()
    _invoke("stief_decode_attention_joint_v", (pq, ppk, ppv, pkl, pvl, psl, po,
                                                    workspace.data_ptr(), ws_bytes, B, Hq, Hkv, d,
                                                    rK, rV, L_max, int(max_seq_len),
                                                    int(num_splits), _opt_status(dev_status),
                                                    _stream_ptr(stream),))
    return out


def stief_decode_latent_joint_v(q_lat: torch.Tensor, k_lat: torch.Tensor, v_joint: torch.Tensor,
                                seq_lens: torch.Tensor, out_lat: torch.Tensor,
                                workspace: torch.Tensor, max_seq_len: int, num_splits: int = 0,
                                d: int = 128, dev_status: Optional[torch.Tensor] = None,
                                stream=None) -> torch.Tensor:
    """stief_decode_latent with a joint value latent v_joint [B][L_max][rV] bf16 (one row per
    token, shared by the KV heads)."""
    pq = _dev(q_lat, "q_lat", torch.bfloat16, 3)
    pkl = _dev(k_lat, "k_lat", torch.bfloat16, 4)
    pvl = _dev(v_joint, "v_joint", torch.bfloat16, 3)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    po = _dev(out_lat, "out_lat", torch.bfloat16, 3)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    B, Hq, rK = q_lat.shape
    Hkv, L_max = k_lat.shape[1], k_lat.shape[2]
    rV = v_joint.shape[2]
    if tuple(k_lat.shape) != (B, Hkv, L_max, rK) or tuple(v_joint.shape) != (B, L_max, rV) \
            or seq_lens.shape[0] != B or tuple(out_lat.shape) != (B, Hq, rV):
        raise ValueError("stief_decode_latent_joint_v: inconsistent shapes")
    ws_bytes = workspace.numel() * workspace.element_size()
    _invoke("stief_decode_latent_joint_v", (pq, pkl, pvl, psl, po, workspace.data_ptr(),
                                                 ws_bytes, B, Hq, Hkv, int(d), rK, rV, L_max,
                                                 int(max_seq_len), int(num_splits),
                                                 _opt_status(dev_status), _stream_ptr(stream),))
    return out_lat


def stief_compress_append_joint_v(k_new: torch.Tensor, v_new: torch.Tensor, P_K: torch.Tensor,
                                  P_VJ: torch.Tensor, k_lat: torch.Tensor, v_joint: torch.Tensor,
                                  seq_lens: torch.Tensor, dev_status: Optional[torch.Tensor] = None,
                                  stream=None) -> None:
    """stief_compress_append with the values projected jointly over the KV heads: keys per head
    into k_lat [B][Hkv][L_max][rK], values through P_VJ [Hkv*d][rV] into v_joint [B][L_max][rV]
    (one row per token); k_new, v_new [B][Hkv][T][d] bf16; seq_lens [B] int32 advanced by T."""
    pk = _dev(k_new, "k_new", torch.bfloat16, 4)
    pv = _dev(v_new, "v_new", torch.bfloat16, 4)
    ppk = _dev(P_K, "P_K", torch.bfloat16, 3)
    ppv = _dev(P_VJ, "P_VJ", torch.bfloat16, 2)
    pkl = _dev(k_lat, "k_lat", torch.bfloat16, 4)
    pvl = _dev(v_joint, "v_joint", torch.bfloat16, 3)
    psl = _dev(seq_lens, "seq_lens", torch.int32, 1)
    B, Hkv, T, d = k_new.shape
    rK, rV = P_K.shape[2], P_VJ.shape[1]
    L_max = k_lat.shape[2]
    if tuple(v_new.shape) != (B, Hkv, T, d) or tuple(P_K.shape) != (Hkv, d, rK) \
            or tuple(P_VJ.shape) != (Hkv * d, rV) or tuple(k_lat.shape) != (B, Hkv, L_max, rK) \
            or tuple(v_joint.shape) != (B, L_max, rV) or seq_lens.shape[0] != B:
        raise ValueError("stief_compress_append_joint_v: inconsistent shapes")
    _invoke("stief_compress_append_joint_v", (pk, pv, ppk, ppv, pkl, pvl, psl, B, Hkv, T, d,
                                                   rK, rV, L_max, _opt_status(dev_status),
                                                   _stream_ptr(stream),))


def stief_plan_workspace_bytes() -> int:
    return int(library().stief_plan_workspace_bytes())


def plan_workspace(device="cuda") -> torch.Tensor:
    """A zero-filled uint8 device tensor for stief_plan_pages (every call leaves it zero)."""
    return torch.zeros(stief_plan_workspace_bytes(), dtype=torch.uint8, device=device)


# The calls below first try the extension (_marshal): it makes the call if every argument is as it
# should be, and returns None otherwise.  What follows in each function is the whole check, which
# says what is wrong, and the way for other streams, prepare(), and an extension that is not built.

def _here(t, name, dtype, ndim, dev):
    """Data pointer of a contiguous `ndim`-dimensional tensor of `dtype` on device `dev`, the
    current one: the library launches there."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == ndim and t.get_device() == dev \
            and t.is_contiguous():
        return t.data_ptr()
    _dev(t, name, dtype, ndim)
    raise ValueError(f"{name} must be on the current device (cuda:{dev}), got {t.device}")


def _current():
    """The current device's number; -2, which no tensor has, without a GPU."""
    return torch.cuda.current_device() if torch.cuda.is_available() else -2


def _int32(value, name):
    """The number as an int that the C call's 32 bits hold (ctypes would cut the rest off)."""
    value = int(value)
    if not -0x80000000 <= value <= 0x7fffffff:
        raise ValueError(f"{name} does not fit 32 bits: {value}")
    return value


def _sizes(func, *sizes):
    """The sizes of tensors, which 32 bits must hold too."""
    if max(sizes) > 0x7fffffff or min(sizes) < -0x80000000:
        raise ValueError(f"{func}: a size does not fit 32 bits: {sizes}")
    return sizes


def _status_here(dev_status, dev):
    """Pointer of the status word, which must be on device `dev`: its kernels write there."""
    ptr = _opt_status(dev_status)
    if ptr is not None and dev_status.get_device() != dev:
        raise ValueError(f"dev_status must be on the current device (cuda:{dev}), got {dev_status.device}")
    return ptr


def _ws(workspace, dev):
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    if workspace.get_device() != dev:
        raise ValueError(f"workspace must be on the current device (cuda:{dev}), got {workspace.device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(stream, dev):
    """The stream given, or device `dev`'s current one."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream_ptr(stream)


def stief_plan_pages(new_tokens, seq_lens, block_table, free_pages, free_count, slots, q_start,
                     kv_start, seq_lens_out, free_count_out, workspace, page_size: int,
                     dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Block-table entries and pool slots of a step's new tokens, on the GPU.

    new_tokens, seq_lens [B]; block_table [B][max_pages] (new entries written); free_pages
    [num_pages], a stack whose top is entry free_count[0] - 1; slots [max_tokens], q_start and
    kv_start [B + 1], seq_lens_out [B] (each written, or None); free_count_out [1].  All int32.
    seq_lens_out may be seq_lens and free_count_out may be free_count.
    """
    if _short_way(stream):
        code = _marshal.plan_pages(new_tokens, seq_lens, block_table, free_pages, free_count, slots, q_start,
                                   kv_start, seq_lens_out, free_count_out, workspace, page_size, dev_status)
        if code is not None:
            _check("stief_plan_pages", code)
            return
    page_size = _int32(page_size, "page_size")
    dev, i32 = _current(), torch.int32
    status = _status_here(dev_status, dev)
    pn, pl = _here(new_tokens, "new_tokens", i32, 1, dev), _here(seq_lens, "seq_lens", i32, 1, dev)
    pt, pf = _here(block_table, "block_table", i32, 2, dev), _here(free_pages, "free_pages", i32, 1, dev)
    pc, po = _here(free_count, "free_count", i32, 1, dev), _here(free_count_out, "free_count_out", i32, 1, dev)
    B, max_pages = block_table.shape
    ps = pq = pk = pso = None
    max_tokens, ok = 0, new_tokens.shape[0] == B == seq_lens.shape[0] and free_count.shape[0] == 1 == free_count_out.shape[0]
    if slots is not None:
        ps, max_tokens = _here(slots, "slots", i32, 1, dev), slots.shape[0]
        if max_tokens == 0:
            raise ValueError("stief_plan_pages: slots must not be empty (pass None)")
    if q_start is not None:
        pq, ok = _here(q_start, "q_start", i32, 1, dev), ok and q_start.shape[0] == B + 1
    if kv_start is not None:
        pk, ok = _here(kv_start, "kv_start", i32, 1, dev), ok and kv_start.shape[0] == B + 1
    if seq_lens_out is not None:
        pso, ok = _here(seq_lens_out, "seq_lens_out", i32, 1, dev), ok and seq_lens_out.shape[0] == B
    if not ok:
        raise ValueError("stief_plan_pages: inconsistent shapes")
    pw, nw = _ws(workspace, dev)
    _invoke("stief_plan_pages", (pn, pl, pt, pf, pc, ps, pq, pk, pso, po, pw, nw,
                                 *_sizes("stief_plan_pages", B, free_pages.shape[0], page_size, max_pages, max_tokens),
                                 status, _stream_on(stream, dev)))


def _rows(t, name, dev):
    """Pointer, shape and row stride of a 2-D bf16 tensor on device `dev` whose rows are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current device (cuda:{dev}), got {t.device}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions, got {tuple(t.shape)}")
    n, w = t.shape
    stride, step = t.stride()
    if w > 1 and step != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), n, w, stride if n > 1 else w


def stief_append_shared_paged(c_new, pe_new, slots, pages,
                              dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Write rows [c_new[i] | pe_new[i]] to the pool rows slots[i] (negative: skipped).

    c_new [N][r] and pe_new [N][dr] bf16 (pe_new None, or with dr = 0, for rows without a
    position part), rows contiguous, any row stride that is a multiple of 8; slots [N] int32;
    pages [num_pages][page_size][r + dr] bf16.
    """
    if _short_way(stream):
        code = _marshal.append_shared_paged(c_new, pe_new, slots, pages, dev_status)
        if code is not None:
            _check("stief_append_shared_paged", code)
            return
    dev = _current()
    status = _status_here(dev_status, dev)
    pc, N, r, sc = _rows(c_new, "c_new", dev)
    pp, n_pe, dr, sp = (None, N, 0, 0) if pe_new is None else _rows(pe_new, "pe_new", dev)
    psl = _here(slots, "slots", torch.int32, 1, dev)
    ppg = _here(pages, "pages", torch.bfloat16, 3, dev)
    num_pages, page_size, w = pages.shape
    if slots.shape[0] != N or w != r + dr or n_pe != N:
        raise ValueError("stief_append_shared_paged: inconsistent shapes")
    N, r, dr, num_pages, page_size = _sizes("stief_append_shared_paged", N, r, dr, num_pages, page_size)
    _invoke("stief_append_shared_paged", (pc, pp if dr else None, psl, ppg, N, r, dr, sc, sp, num_pages,
                                          page_size, status, _stream_on(stream, dev)))


def stief_decode_shared_workspace_bytes(B: int, Hq: int, r: int) -> int:
    return int(library().stief_decode_shared_workspace_bytes(B, Hq, r))


def shared_workspace_for(B: int, Hq: int, r: int, device="cuda") -> torch.Tensor:
    """A uint8 device tensor of stief_decode_shared_workspace_bytes(...) bytes."""
    n = stief_decode_shared_workspace_bytes(B, Hq, r)
    if n == 0:
        raise ValueError("invalid sizes for the shared decode workspace")
    return torch.empty(n, dtype=torch.uint8, device=device)


def stief_decode_shared_paged(q, pages, block_table, seq_lens, out, workspace, max_seq_len: int,
                              scale: float, dev_status: Optional[torch.Tensor] = None,
                              stream=None) -> torch.Tensor:
    """Absorbed attention of one query token a sequence over shared latent rows:
    out_h = sum_t softmax_t(scale * q_h . row_t) c_t.

    q [B][Hq][r + dr], pages [num_pages][page_size][r + dr], out [B][Hq][r] (written), bf16;
    block_table [B][max_pages], seq_lens [B] int32; workspace from shared_workspace_for.
    """
    if _short_way(stream):
        code = _marshal.decode_shared_paged(q, pages, block_table, seq_lens, out, workspace, max_seq_len, scale,
                                            dev_status)
        if code is not None:
            _check("stief_decode_shared_paged", code)
            return out
    max_seq_len = _int32(max_seq_len, "max_seq_len")
    dev, b16, i32 = _current(), torch.bfloat16, torch.int32
    status = _status_here(dev_status, dev)
    pq, ppg = _here(q, "q", b16, 3, dev), _here(pages, "pages", b16, 3, dev)
    pt, psl = _here(block_table, "block_table", i32, 2, dev), _here(seq_lens, "seq_lens", i32, 1, dev)
    po = _here(out, "out", b16, 3, dev)
    B, Hq, w = q.shape
    Bo, Ho, r = out.shape
    num_pages, page_size, wp = pages.shape
    Bt, max_pages = block_table.shape
    if wp != w or r > w or Ho != Hq or not Bo == Bt == B == seq_lens.shape[0]:
        raise ValueError("stief_decode_shared_paged: inconsistent shapes")
    pw, nw = _ws(workspace, dev)
    _invoke("stief_decode_shared_paged", (pq, ppg, pt, psl, po, pw, nw,
                                          *_sizes("stief_decode_shared_paged", B, Hq, r, w - r, num_pages, page_size,
                                                  max_pages), max_seq_len, float(scale),
                                          status, _stream_on(stream, dev)))
    return out


def stief_expand_shared_paged(pages, block_table, kv_start, W_K, W_V, k, v, k_pe=None,
                              dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Keys and values of every head from shared latent rows: sequence b's token t becomes row
    kv_start[b] + t of k and v, k_h = c_t . W_K[h]^T, v_h = c_t . W_V[h]^T.

    pages [num_pages][page_size][r + dr], W_K and W_V [H][d][r], k and v [N][H][d], k_pe [N][dr]
    (None, or with dr = 0, for rows without a position part) bf16; block_table [B][max_pages],
    kv_start [B + 1] int32.
    """
    if _short_way(stream):
        code = _marshal.expand_shared_paged(pages, block_table, kv_start, W_K, W_V, k, v, k_pe, dev_status)
        if code is not None:
            _check("stief_expand_shared_paged", code)
            return
    dev, b16, i32 = _current(), torch.bfloat16, torch.int32
    status = _status_here(dev_status, dev)
    ppg, pt = _here(pages, "pages", b16, 3, dev), _here(block_table, "block_table", i32, 2, dev)
    pst = _here(kv_start, "kv_start", i32, 1, dev)
    pwk, pwv = _here(W_K, "W_K", b16, 3, dev), _here(W_V, "W_V", b16, 3, dev)
    pk, pv = _here(k, "k", b16, 3, dev), _here(v, "v", b16, 3, dev)
    H, d, r = W_K.shape
    B, max_pages = block_table.shape
    num_pages, page_size, w = pages.shape
    N, dr = k.shape[0], w - r
    ppe = _here(k_pe, "k_pe", b16, 2, dev) if dr > 0 and k_pe is not None else None
    if dr < 0 or W_V.shape != W_K.shape or k.shape != (N, H, d) or v.shape != k.shape \
            or kv_start.shape[0] != B + 1 or (dr > 0 and (k_pe is None or k_pe.shape != (N, dr))):
        raise ValueError("stief_expand_shared_paged: inconsistent shapes")
    _invoke("stief_expand_shared_paged", (ppg, pt, pst, pwk, pwv, pk, pv, ppe,
                                          *_sizes("stief_expand_shared_paged", B, N, H, d, r, dr, num_pages,
                                                  page_size, max_pages), status, _stream_on(stream, dev)))


def stief_prefill_attention(q, k, v, q_start, kv_start, out, max_q_len: int, scale: float,
                            k_pe=None, dev_status: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """Causal attention of ragged prompts: query i of sequence b sees keys
    j <= i + n_k - n_q; out = softmax_j(scale * (q . k_j + q^R . k_pe_j)) v_j.

    q [Nq][Hq][d + dr], k and v [Nkv][Hkv][d], k_pe [Nkv][dr] (None when dr = 0), out
    [Nq][Hq][d] (written), bf16; q_start, kv_start [B + 1] int32.
    """
    if _short_way(stream):
        code = _marshal.prefill_attention(q, k, v, q_start, kv_start, out, max_q_len, scale, k_pe, dev_status)
        if code is not None:
            _check("stief_prefill_attention", code)
            return out
    max_q_len = _int32(max_q_len, "max_q_len")
    dev, b16, i32 = _current(), torch.bfloat16, torch.int32
    status = _status_here(dev_status, dev)
    pq, pk = _here(q, "q", b16, 3, dev), _here(k, "k", b16, 3, dev)
    pv, po = _here(v, "v", b16, 3, dev), _here(out, "out", b16, 3, dev)
    pqs, pks = _here(q_start, "q_start", i32, 1, dev), _here(kv_start, "kv_start", i32, 1, dev)
    Nq, Hq, dq = q.shape
    Nkv, Hkv, d = k.shape
    ppe, n_pe, dr = None, Nkv, 0
    if k_pe is not None:
        ppe = _here(k_pe, "k_pe", b16, 2, dev)
        n_pe, dr = k_pe.shape
    B = q_start.shape[0] - 1
    if v.shape != k.shape or dq != d + dr or out.shape != (Nq, Hq, d) or kv_start.shape[0] != B + 1 \
            or n_pe != Nkv:
        raise ValueError("stief_prefill_attention: inconsistent shapes")
    _invoke("stief_prefill_attention", (pq, pk, pv, ppe if dr else None, pqs, pks, po,
                                        *_sizes("stief_prefill_attention", B, Hq, Hkv, d, dr, Nq, Nkv), max_q_len,
                                        float(scale), status, _stream_on(stream, dev)))
    return out
