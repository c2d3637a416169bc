"""Binding of libarcserve.so (include/serve/): loading, error codes, structs.

The operators of a decode step before the sampler live in kv_cache.py, w4.py,
norm.py and edit.py; every step of them runs in the library's CUDA kernels.  There is no
fallback: if the library is not built, `load()` raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import sampler
from .workloads import DTYPE_BF16, DTYPE_F16, DTYPE_F32

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libarcserve.so")

P, I32, I64, SIZE = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class KvCache(ctypes.Structure):
    """arc_kv_cache, 64 bytes."""
    _fields_ = [("k", P), ("v", P), ("k_scale", P), ("v_scale", P), ("page_stride", I64), ("head_stride", I64),
                ("pages", I32), ("heads", I32), ("page_size", I32), ("head_dim", I32)]


class KvStep(ctypes.Structure):
    """arc_kv_step, 56 bytes."""
    _fields_ = [("page_table", P), ("table_stride", I64), ("positions", P), ("row_offsets", P), ("B", I64), ("T", I64),
                ("max_pages", I32), ("reserved", I32)]


class RopeArgs(ctypes.Structure):
    """arc_rope, 24 bytes."""
    _fields_ = [("turns", P), ("amplitude", ctypes.c_float), ("rot_dim", I32), ("layout", I32), ("reserved", I32)]


class KvRows(ctypes.Structure):
    """arc_kv_rows, 104 bytes."""
    _fields_ = [("q", P), ("k", P), ("v", P), ("q_out", P), ("q_token_stride", I64), ("q_head_stride", I64),
                ("k_token_stride", I64), ("k_head_stride", I64), ("v_token_stride", I64), ("v_head_stride", I64),
                ("out_token_stride", I64), ("out_head_stride", I64), ("q_heads", I32), ("dtype", I32)]


class KvQuery(ctypes.Structure):
    """arc_kv_query, 64 bytes."""
    _fields_ = [("q", P), ("out", P), ("q_token_stride", I64), ("q_head_stride", I64), ("out_token_stride", I64),
                ("out_head_stride", I64), ("q_heads", I32), ("dtype", I32), ("scale", ctypes.c_float), ("window", I32)]


class NormRows(ctypes.Structure):
    """arc_norm_rows, 136 bytes."""
    _fields_ = [("x", P), ("y", P), ("gate", P), ("post_weight", P), ("weight", P), ("h", P), ("n", P), ("x_stride", I64),
                ("y_stride", I64), ("gate_stride", I64), ("h_stride", I64), ("n_stride", I64), ("rows", I64), ("dim", I32),
                ("stream_dtype", I32), ("dtype", I32), ("weight_dtype", I32), ("activation", I32),
                ("alpha", ctypes.c_float), ("offset", ctypes.c_float), ("eps", ctypes.c_float)]


class LogitEdits(ctypes.Structure):
    """arc_logit_edits, 96 bytes."""
    _fields_ = [("params", P), ("hist_offsets", P), ("hist_ids", P), ("hist_len", I64), ("bias_offsets", P),
                ("bias_ids", P), ("bias", P), ("bias_len", I64), ("allowed", P), ("allowed_stride", I64),
                ("allowed_count", I64), ("allowed_rows", P)]


class W4Weight(ctypes.Structure):
    """arc_w4_weight, 48 bytes."""
    _fields_ = [("q", P), ("scales", P), ("zeros", P), ("row_bytes", I64), ("outs", I64), ("ins", I32), ("group", I32)]


# exported symbol -> (restype, argtypes)
SIGNATURES = {
    "arc_kv_append": (ctypes.c_int, [P, P, P, P, P, P]),
    "arc_kv_attend": (ctypes.c_int, [P, P, P, P, P, SIZE, P]),
    "arc_kv_attend_sinks": (ctypes.c_int, [P, P, P, I32, P, P, SIZE, P]),
    "arc_kv_attend_shared": (ctypes.c_int, [P, P, P, P, I32, P, P, SIZE, P]),
    "arc_kv_attend_shared_workspace_bytes": (SIZE, [P, I64, I32]),
    "arc_kv_attend_workspace_bytes": (SIZE, [P]),
    "arc_w4_matvec": (ctypes.c_int, [P, P, I64, I64, I32, P, I64, I32, P, SIZE, P]),
    "arc_w4_workspace_bytes": (SIZE, [P, I64]),
    "arc_norm_join": (ctypes.c_int, [P, P]),
    "arc_edit_logits": (ctypes.c_int, [P, I64, I64, I64, I32, P, I64, I32, P, P, P]),
    "arc_serve_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "arc_serve_abi_version": (ctypes.c_int, []),
}

_lib = None


def load():
    """Load libarcserve.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
                "(there is no CPU fallback)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


class ServeError(sampler.ArcError):
    """A call of libarcserve refused its arguments or could not launch."""

    def __init__(self, rc: int):
        RuntimeError.__init__(self, f"arc_serve error {rc}: {load().arc_serve_strerror(rc).decode()}")
        self.rc = rc


_CODES = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}


def dtype_code(t, f32: bool = False) -> int:
    """ARC_* code of a tensor's type: bfloat16 or float16 (or float32 where allowed)."""
    code = _CODES.get(t.dtype)
    if code is not None:
        return code
    if f32 and t.dtype == torch.float32:
        return DTYPE_F32
    raise TypeError(f"must be bfloat16 or float16{' or float32' if f32 else ''}, not {t.dtype}")


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def stream_of(stream, device: int) -> int:
    """The stream's handle; the device's current stream where None (torch.cuda.current_stream()
    builds a Stream object and resolves the device's name, 7 us of a 20 us call on the Arm host)."""
    if stream is not None:
        return int(stream.cuda_stream)
    return _raw_stream(device) if _raw_stream is not None else int(torch.cuda.current_stream(device).cuda_stream)


try:  # the allocation that compiled graphs of this torch make: 4 us a call less than torch.empty on the Arm host
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:
    _empty_strided_cuda = None


def foreign(stream, device: int) -> bool:
    """Whether a call is to run on a stream that is not the device's current one."""
    return stream is not None and int(stream.cuda_stream) != stream_of(None, device)


def on_stream(stream, device: int):
    """Context whose allocations are the stream's; any object that has the handle of one as cuda_stream will do."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream.cuda_stream), device=device)
    return torch.cuda.stream(stream)


def new_output(like, shape: tuple, strides: tuple, dtype, stream=None):
    """An uninitialised contiguous tensor on the device of `like`, for a call on `stream`.

    Memory is handed out in the order of the stream it is allocated on, so a call on another
    stream than the current one gets its output from that stream; the current one is recorded
    as a user too, since that is where the caller goes on.  On the current stream the short
    allocation is taken, which no dispatch mode of torch sees."""
    if foreign(stream, like.get_device()):
        with on_stream(stream, like.get_device()):
            out = like.new_empty(shape, dtype=dtype)
        out.record_stream(torch.cuda.current_stream(like.device))
        return out
    if _empty_strided_cuda is not None and like.is_cuda and torch._C._cuda_getDevice() == like.get_device():
        return _empty_strided_cuda(shape, strides, dtype)
    return like.new_empty(shape, dtype=dtype)


def new_workspace(like, nbytes: int, zeroed: bool, stream=None):
    """Memory for one call on `stream`: allocated (and filled) there, so that its fill comes before the
    call and its next user after it."""
    make = torch.zeros if zeroed else torch.empty
    if foreign(stream, like.get_device()):
        with on_stream(stream, like.get_device()):
            return make(nbytes, dtype=torch.uint8, device=like.device)
    if not zeroed:
        return new_output(like, (nbytes,), (1,), torch.uint8)
    return make(nbytes, dtype=torch.uint8, device=like.device)


def on_current_gpu(device: int) -> None:
    """Refuses host tensors (their device is -1) and those of a GPU that a launch would not go to."""
    want(device >= 0, "every tensor must be a CUDA tensor")
    want(torch._C._cuda_getDevice() == device, "every tensor must be on the current CUDA device")


def err_word_ptr(err_word, device: int):
    """Address of a 32-bit error word on the device, or None."""
    if err_word is None:
        return None
    if err_word.dtype != torch.int32 and err_word.dtype != torch.uint32:
        raise TypeError(f"err_word must be int32 or uint32, not {err_word.dtype}")
    want(err_word.numel() >= 1 and err_word.get_device() == device, "err_word must be a word on the tensors' device")
    return err_word.data_ptr()


def workspace_of(workspace, device: int):
    """(address, bytes) of a workspace on the device."""
    want(workspace.get_device() == device and workspace.is_contiguous(),
         "workspace must be contiguous, on the tensors' device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def want(ok: bool, text: str) -> None:
    if not ok:
        raise ValueError(text)


def finish(rc: int, check: bool) -> int:
    if check and rc != sampler.ARC_OK:
        raise ServeError(rc)
    return rc
