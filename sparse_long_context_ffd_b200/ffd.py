"""Thin ctypes binding of the C ABI in include/ffd.h (argument marshalling only).

Every step of the decode path runs in the CUDA library; this module only turns
torch tensors into pointers, picks the current CUDA stream and maps status
codes to exceptions.  There is no fallback: if the library is missing and
cannot be built, importing a function raises.
"""
from __future__ import annotations

import ctypes
import math
import threading
from typing import Optional

from . import build as _build

FFD_OK = 0
FFD_ERR_INVALID_ARG = 1
FFD_ERR_UNSUPPORTED = 2
FFD_ERR_WORKSPACE = 3
FFD_ERR_CUDA = 4
FFD_ERR_DEVICE_CHECK = 5
FFD_ERR_TIMEOUT = 6

FFD_DEVICE_FLAG_BAD_LENGTH = 0x1
FFD_DEVICE_FLAG_TIMEOUT = 0x2
FFD_DEVICE_FLAG_BOUNDS = 0x4  # debug build only (use_debug_library())
FFD_LAST_BLOCK = -1
FFD_MAX_SPLIT_BLOCKS = 512

# Every function the header declares; the library must export all of them.
EXPORTED = (
    "ffd_packed_bytes", "ffd_scale_bytes", "ffd_mask_words", "ffd_decode_workspace_bytes",
    "ffd_workspace_init", "ffd_quantize_keys", "ffd_decode", "ffd_check_device_status",
    "ffd_status_string", "ffd_abi_version", "ffd_decode_no_alloc", "ffd_decode_step",
    "ffd_decode_ex", "ffd_decode_partials", "ffd_partials_region", "ffd_merge_partials",
    "ffd_thumb_bytes", "ffd_residual_bytes", "ffd_quantize_keys_tr", "ffd_decode_tr",
    "ffd_decode_partials_tr", "ffd_decode_append", "ffd_decode_append_tr",
    "ffd_step_graph_create", "ffd_step_graph_run", "ffd_step_graph_destroy",
    "ffd_read_probe", "ffd_no_alloc_device_status",
    "ffd_rope_init", "ffd_rotate", "ffd_append_tokens", "ffd_read_cache", "ffd_decode_tree",
    "ffd_decode_tree_workspace_bytes", "ffd_decode_tree_workspace_init",
)

FFD_REFERENCE_RUNNING_MAX = 0
FFD_REFERENCE_SINK_LOCAL = 1        # running maximum started at the sink/local pseudo-max
FFD_REFERENCE_SINK_LOCAL_FIXED = 2  # the sink/local pseudo-max as a fixed threshold

FFD_ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
FFD_ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "by_parts": 3}
FFD_CACHE_BF16 = 0
FFD_CACHE_BYTE = 1
FFD_MAX_TREE_NODES = 64

# Size of the library's built-in scratch array used by ffd_decode_no_alloc.
FFD_NO_ALLOC_SCRATCH_BYTES = 16 << 20


class FFDError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


class DecodeOptions(ctypes.Structure):
    _fields_ = [("reference", ctypes.c_int32), ("requant_last", ctypes.c_int32),
                ("wait_limit_us", ctypes.c_int32)]


class Shape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("capacity", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("split_blocks", ctypes.c_int32)]

    def __repr__(self):
        return "Shape(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class _RopeOptions(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_length", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("amplitude", ctypes.c_double)]


class Rope(ctypes.Structure):
    """A rotary plan (ffd_rope): made once from a model's settings, given to
    rotate, append_tokens, StandInAttentionLayer and TreeStep.

    layout: "half" (channels i and i + rotary_dim / 2 are a pair) or
    "interleaved" (2i and 2i + 1); scaling: "none", "linear", "base" or
    "by_parts" (the header has the formulas); by_parts takes original_length,
    low and high."""
    _fields_ = [("turns", ctypes.c_uint64 * 64), ("amplitude", ctypes.c_float),
                ("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]

    def __init__(self, rotary_dim: int = 128, layout: str = "half", base: float = 10000.0,
                 scaling: str = "none", factor: float = 1.0, original_length: float = 0.0,
                 low: float = 0.0, high: float = 0.0, amplitude: float = 1.0):
        super().__init__()
        if layout not in FFD_ROPE_LAYOUTS or scaling not in FFD_ROPE_SCALINGS:
            raise ValueError("unknown rotary layout or scaling")
        opts = _RopeOptions(int(rotary_dim), FFD_ROPE_LAYOUTS[layout], FFD_ROPE_SCALINGS[scaling], 0,
                            float(base), float(factor), float(original_length), float(low),
                            float(high), float(amplitude))
        _check(load_library().ffd_rope_init(ctypes.byref(opts), ctypes.byref(self)),
               "ffd_rope_init")


class _Cache(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p)]


def make_shape(batch, num_q_heads, num_kv_heads, capacity, block_size, split_blocks,
               head_dim=128) -> Shape:
    return Shape(batch, num_q_heads, num_kv_heads, head_dim, capacity, block_size, split_blocks)


_lock = threading.Lock()
_lib = None


_use_debug = False


def use_debug_library() -> None:
    """Load the bounds-checking debug build (libffd_b200_debug.so: FFD_DEBUG,
    FFD_DEVICE_FLAG_BOUNDS) instead of the product library.  For tests; call
    it before the process's first library call."""
    global _use_debug
    with _lock:
        if _lib is not None and not _use_debug:
            raise RuntimeError("the product library is already loaded in this process")
        _use_debug = True


def _debug_requested() -> bool:
    return _use_debug


def library_path() -> str:
    """The library this process loads: libffd_b200.so, or after
    use_debug_library() the bounds-checking debug build."""
    return _build.DEBUG_LIB if _debug_requested() else _build.LIB


def load_library() -> ctypes.CDLL:
    """Load the library, building it with nvcc first if it is missing or stale."""
    global _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if _build.is_stale(path):
                _build.build(debug=_debug_requested())
            lib = ctypes.CDLL(path)
            sp = ctypes.POINTER(Shape)
            p, sz, st = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
            for name in ("ffd_packed_bytes", "ffd_scale_bytes", "ffd_mask_words",
                         "ffd_decode_workspace_bytes", "ffd_thumb_bytes", "ffd_residual_bytes"):
                getattr(lib, name).argtypes = [sp]
                getattr(lib, name).restype = sz
            lib.ffd_workspace_init.argtypes = [sp, p, sz, p]
            lib.ffd_workspace_init.restype = st
            lib.ffd_quantize_keys.argtypes = [sp, p, p, ctypes.c_int32, p, p, p]
            lib.ffd_quantize_keys.restype = st
            lib.ffd_quantize_keys_tr.argtypes = [sp, p, p, ctypes.c_int32, p, p, p, p]
            lib.ffd_quantize_keys_tr.restype = st
            lib.ffd_decode_tr.argtypes = [sp, ctypes.POINTER(DecodeOptions), p, p, p, p, p, p, p,
                                          ctypes.c_float, p, p, p, sz, p]
            lib.ffd_decode_tr.restype = st
            lib.ffd_decode_partials_tr.argtypes = [sp, ctypes.POINTER(DecodeOptions), p, p, p, p,
                                                   p, p, p, ctypes.c_float, p, sz, p]
            lib.ffd_decode_partials_tr.restype = st
            i32 = ctypes.c_int32
            lib.ffd_decode_append.argtypes = [sp, i32, p, p, p, p, p, p, p, p, ctypes.c_float, p,
                                              p, p, sz, p]
            lib.ffd_decode_append.restype = st
            lib.ffd_decode_append_tr.argtypes = [sp, i32, p, p, p, p, p, p, p, p, p,
                                                 ctypes.c_float, p, p, p, sz, p]
            lib.ffd_decode_append_tr.restype = st
            lib.ffd_step_graph_create.argtypes = [sp, i32, i32, ctypes.c_float, i32, p, p, p, p,
                                                  p, p, p, p, p, p, sz, p, sz,
                                                  ctypes.POINTER(ctypes.c_void_p)]
            lib.ffd_step_graph_create.restype = st
            lib.ffd_step_graph_run.argtypes = [p]
            lib.ffd_step_graph_run.restype = st
            lib.ffd_step_graph_destroy.argtypes = [p]
            lib.ffd_step_graph_destroy.restype = None
            lib.ffd_decode.argtypes = [sp, p, p, p, p, p, p, ctypes.c_float, p, p, p, sz, p]
            lib.ffd_decode.restype = st
            lib.ffd_decode_ex.argtypes = [sp, ctypes.POINTER(DecodeOptions), p, p, p, p, p, p,
                                          ctypes.c_float, p, p, p, sz, p]
            lib.ffd_decode_ex.restype = st
            lib.ffd_decode_partials.argtypes = [sp, ctypes.POINTER(DecodeOptions), p, p, p, p, p,
                                                p, ctypes.c_float, p, sz, p]
            lib.ffd_decode_partials.restype = st
            lib.ffd_partials_region.argtypes = [sp, ctypes.POINTER(sz), ctypes.POINTER(sz)]
            lib.ffd_partials_region.restype = st
            lib.ffd_merge_partials.argtypes = [sp, ctypes.c_int32, p, sz, p, p, p, p]
            lib.ffd_merge_partials.restype = st
            lib.ffd_decode_step.argtypes = [sp, p, p, p, p, p, p, ctypes.c_float, p, p, p, sz, p]
            lib.ffd_decode_step.restype = st
            lib.ffd_decode_no_alloc.argtypes = [sp, p, p, p, p, p, p, ctypes.c_float, p, p, p]
            lib.ffd_decode_no_alloc.restype = st
            lib.ffd_no_alloc_device_status.argtypes = [p, p]
            lib.ffd_no_alloc_device_status.restype = st
            lib.ffd_check_device_status.argtypes = [p, ctypes.POINTER(ctypes.c_uint32), p]
            lib.ffd_check_device_status.restype = st
            lib.ffd_rope_init.argtypes = [ctypes.POINTER(_RopeOptions), ctypes.POINTER(Rope)]
            rp, cp = ctypes.POINTER(Rope), ctypes.POINTER(_Cache)
            lib.ffd_rotate.argtypes = [rp, ctypes.c_int64, p, i32, i32, p, p, i32, p, p, p]
            lib.ffd_append_tokens.argtypes = [sp, cp, rp, i32, p, p, p, p, p, p, p, p]
            lib.ffd_read_cache.argtypes = [sp, cp, p, i32, i32, p, p, p]
            lib.ffd_decode_tree.argtypes = [sp, cp, i32, p, p, p, p, p, p, sz, p]
            lib.ffd_decode_tree_workspace_bytes.argtypes = [sp, i32]
            lib.ffd_decode_tree_workspace_bytes.restype = sz
            lib.ffd_decode_tree_workspace_init.argtypes = [sp, i32, p, sz, p]
            for name in ("ffd_rope_init", "ffd_rotate", "ffd_append_tokens", "ffd_read_cache",
                         "ffd_decode_tree", "ffd_decode_tree_workspace_init"):
                getattr(lib, name).restype = st
            lib.ffd_read_probe.argtypes = [p, sz, p, p]
            lib.ffd_read_probe.restype = st
            lib.ffd_status_string.argtypes = [st]
            lib.ffd_status_string.restype = ctypes.c_char_p
            lib.ffd_abi_version.argtypes = []
            lib.ffd_abi_version.restype = ctypes.c_int32
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load_library().ffd_status_string(int(status)).decode()


def abi_version() -> int:
    return int(load_library().ffd_abi_version())


def _check(status: int, what: str) -> None:
    if status != FFD_OK:
        raise FFDError(status, what)


def _ptr(t) -> Optional[int]:
    """Device pointer of a CUDA tensor (None passes a null pointer)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("FFD entry points take CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("FFD entry points take contiguous tensors")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def packed_bytes(shape: Shape) -> int:
    return int(load_library().ffd_packed_bytes(ctypes.byref(shape)))


def scale_bytes(shape: Shape) -> int:
    return int(load_library().ffd_scale_bytes(ctypes.byref(shape)))


def thumb_bytes(shape: Shape) -> int:
    return int(load_library().ffd_thumb_bytes(ctypes.byref(shape)))


def residual_bytes(shape: Shape) -> int:
    return int(load_library().ffd_residual_bytes(ctypes.byref(shape)))


def mask_words(shape: Shape) -> int:
    return int(load_library().ffd_mask_words(ctypes.byref(shape)))


def decode_workspace_bytes(shape: Shape) -> int:
    return int(load_library().ffd_decode_workspace_bytes(ctypes.byref(shape)))


def workspace_init(shape: Shape, workspace, stream=None) -> None:
    _check(load_library().ffd_workspace_init(ctypes.byref(shape), _ptr(workspace),
                                             workspace.numel() * workspace.element_size(),
                                             _stream(stream)), "ffd_workspace_init")


def quantize_keys(shape: Shape, k, lengths, block_begin: int, k_packed, k_scales,
                  stream=None) -> None:
    _check(load_library().ffd_quantize_keys(ctypes.byref(shape), _ptr(k), _ptr(lengths),
                                            int(block_begin), _ptr(k_packed), _ptr(k_scales),
                                            _stream(stream)), "ffd_quantize_keys")


def quantize_keys_tr(shape: Shape, k, lengths, block_begin: int, k_thumb, k_resid, k_scales,
                     stream=None) -> None:
    """2-bit thumbnails + 8-bit residuals (+ bf16 scales) of the keys."""
    _check(load_library().ffd_quantize_keys_tr(ctypes.byref(shape), _ptr(k), _ptr(lengths),
                                               int(block_begin), _ptr(k_thumb), _ptr(k_resid),
                                               _ptr(k_scales), _stream(stream)),
           "ffd_quantize_keys_tr")


def decode_tr(shape: Shape, q, k, v, k_thumb, k_resid, k_scales, lengths, delta: float, out,
              mask, workspace, reference: int = FFD_REFERENCE_RUNNING_MAX,
              requant_last: bool = False, stream=None, wait_limit_us: int = 0) -> None:
    """Decode step on the thumbnail + residual key format (k is read only when
    requant_last re-quantises the last block; it may be None otherwise)."""
    opts = DecodeOptions(int(reference), 1 if requant_last else 0, int(wait_limit_us))
    _check(load_library().ffd_decode_tr(ctypes.byref(shape), ctypes.byref(opts), _ptr(q), _ptr(k),
                                         _ptr(v), _ptr(k_thumb), _ptr(k_resid), _ptr(k_scales),
                                         _ptr(lengths), float(delta), _ptr(out), _ptr(mask),
                                         _ptr(workspace),
                                         workspace.numel() * workspace.element_size(),
                                         _stream(stream)), "ffd_decode_tr")


def decode_append(shape: Shape, q, k_new, v_new, k, v, k_packed, k_scales, lengths,
                  delta: float, out, mask, workspace,
                  reference: int = FFD_REFERENCE_RUNNING_MAX, stream=None) -> None:
    """One launch per step: write the new token's K/V rows (k_new, v_new
    [B,Hkv,D]) at position lengths-1, re-quantise the last block, decode."""
    _check(load_library().ffd_decode_append(ctypes.byref(shape), int(reference), _ptr(q),
                                             _ptr(k_new), _ptr(v_new), _ptr(k), _ptr(v),
                                             _ptr(k_packed), _ptr(k_scales), _ptr(lengths),
                                             float(delta), _ptr(out), _ptr(mask), _ptr(workspace),
                                             workspace.numel() * workspace.element_size(),
                                             _stream(stream)), "ffd_decode_append")


def decode_append_tr(shape: Shape, q, k_new, v_new, k, v, k_thumb, k_resid, k_scales, lengths,
                     delta: float, out, mask, workspace,
                     reference: int = FFD_REFERENCE_RUNNING_MAX, stream=None) -> None:
    """decode_append on the thumbnail + residual key format."""
    _check(load_library().ffd_decode_append_tr(ctypes.byref(shape), int(reference), _ptr(q),
                                                _ptr(k_new), _ptr(v_new), _ptr(k), _ptr(v),
                                                _ptr(k_thumb), _ptr(k_resid), _ptr(k_scales),
                                                _ptr(lengths), float(delta), _ptr(out), _ptr(mask),
                                                _ptr(workspace),
                                                workspace.numel() * workspace.element_size(),
                                                _stream(stream)), "ffd_decode_append_tr")


def decode_partials_tr(local_shape: Shape, q, k, v, k_thumb, k_resid, k_scales, local_lengths,
                       delta: float, workspace, requant_last: bool = False, stream=None) -> None:
    """Context shard on the thumbnail + residual format (see decode_partials)."""
    opts = DecodeOptions(FFD_REFERENCE_RUNNING_MAX, 1 if requant_last else 0)
    _check(load_library().ffd_decode_partials_tr(ctypes.byref(local_shape), ctypes.byref(opts),
                                                  _ptr(q), _ptr(k), _ptr(v), _ptr(k_thumb),
                                                  _ptr(k_resid), _ptr(k_scales),
                                                  _ptr(local_lengths), float(delta),
                                                  _ptr(workspace),
                                                  workspace.numel() * workspace.element_size(),
                                                  _stream(stream)), "ffd_decode_partials_tr")


def decode(shape: Shape, q, k, v, k_packed, k_scales, lengths, delta: float, out, mask,
           workspace, stream=None) -> None:
    _check(load_library().ffd_decode(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v),
                                      _ptr(k_packed), _ptr(k_scales), _ptr(lengths),
                                      float(delta), _ptr(out), _ptr(mask), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(),
                                      _stream(stream)), "ffd_decode")


def decode_step(shape: Shape, q, k, v, k_packed, k_scales, lengths, delta: float, out, mask,
                workspace, stream=None) -> None:
    """Re-quantise each sequence's last key block and decode, in one launch."""
    _check(load_library().ffd_decode_step(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v),
                                           _ptr(k_packed), _ptr(k_scales), _ptr(lengths),
                                           float(delta), _ptr(out), _ptr(mask), _ptr(workspace),
                                           workspace.numel() * workspace.element_size(),
                                           _stream(stream)), "ffd_decode_step")


def decode_ex(shape: Shape, q, k, v, k_packed, k_scales, lengths, delta: float, out, mask,
              workspace, reference: int = FFD_REFERENCE_RUNNING_MAX, requant_last: bool = False,
              stream=None, wait_limit_us: int = 0) -> None:
    """ffd_decode / ffd_decode_step with the reference-maximum mode and the
    kernel's wait limit (0: the default 2 s; see ffd_decode_options)."""
    opts = DecodeOptions(int(reference), 1 if requant_last else 0, int(wait_limit_us))
    _check(load_library().ffd_decode_ex(ctypes.byref(shape), ctypes.byref(opts), _ptr(q), _ptr(k),
                                         _ptr(v), _ptr(k_packed), _ptr(k_scales), _ptr(lengths),
                                         float(delta), _ptr(out), _ptr(mask), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(),
                                         _stream(stream)), "ffd_decode_ex")


def decode_partials(local_shape: Shape, q, k, v, k_packed, k_scales, local_lengths,
                    delta: float, workspace, requant_last: bool = False, stream=None) -> None:
    """Context shard: split partials and bits into the workspace, no merge."""
    opts = DecodeOptions(FFD_REFERENCE_RUNNING_MAX, 1 if requant_last else 0)
    _check(load_library().ffd_decode_partials(ctypes.byref(local_shape), ctypes.byref(opts),
                                               _ptr(q), _ptr(k), _ptr(v), _ptr(k_packed),
                                               _ptr(k_scales), _ptr(local_lengths), float(delta),
                                               _ptr(workspace),
                                               workspace.numel() * workspace.element_size(),
                                               _stream(stream)), "ffd_decode_partials")


def partials_region(local_shape: Shape):
    """(offset, bytes) of the workspace region the shards exchange."""
    off, nbytes = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(load_library().ffd_partials_region(ctypes.byref(local_shape), ctypes.byref(off),
                                               ctypes.byref(nbytes)), "ffd_partials_region")
    return int(off.value), int(nbytes.value)


def merge_partials(local_shape: Shape, num_shards: int, gathered, global_lengths, out, mask,
                   stream=None) -> None:
    """Merge the gathered shard regions into the output rows and global mask."""
    _check(load_library().ffd_merge_partials(ctypes.byref(local_shape), int(num_shards),
                                              _ptr(gathered),
                                              gathered.numel() * gathered.element_size(),
                                              _ptr(global_lengths), _ptr(out), _ptr(mask),
                                              _stream(stream)), "ffd_merge_partials")


def decode_no_alloc(shape: Shape, q, k, v, k_packed, k_scales, lengths, delta: float, out,
                    mask, stream=None) -> None:
    """ffd_decode without a workspace: for callers that cannot allocate device
    memory.  Uses the library's built-in 16 MiB scratch array; calls on one
    device must not overlap on the GPU.  The first call on a device should
    come before any stream capture.  Device-side flags: no_alloc_device_status."""
    _check(load_library().ffd_decode_no_alloc(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v),
                                              _ptr(k_packed), _ptr(k_scales), _ptr(lengths),
                                              float(delta), _ptr(out), _ptr(mask),
                                              _stream(stream)), "ffd_decode_no_alloc")


def no_alloc_device_status(stream=None) -> int:
    """Synchronise, read and clear the flags the last decode_no_alloc call on
    the current device left in the library's built-in array; returns
    FFD_DEVICE_FLAG_* bits."""
    flags = ctypes.c_uint32(0)
    st = load_library().ffd_no_alloc_device_status(ctypes.byref(flags), _stream(stream))
    if st not in (FFD_OK, FFD_ERR_DEVICE_CHECK, FFD_ERR_TIMEOUT):
        raise FFDError(st, "ffd_no_alloc_device_status")
    return int(flags.value)


def read_probe(buf, sink, stream=None) -> None:
    """ffd_read_probe: read the whole (16-byte aligned) device tensor `buf`
    once; `sink` is a device int32/uint32 tensor of at least one element."""
    _check(load_library().ffd_read_probe(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink),
                                         _stream(stream)), "ffd_read_probe")


def check_device_status(workspace, stream=None) -> int:
    """Synchronise, read and clear the device flags; returns FFD_DEVICE_FLAG_* bits."""
    flags = ctypes.c_uint32(0)
    st = load_library().ffd_check_device_status(_ptr(workspace), ctypes.byref(flags),
                                                _stream(stream))
    if st not in (FFD_OK, FFD_ERR_DEVICE_CHECK, FFD_ERR_TIMEOUT):
        raise FFDError(st, "ffd_check_device_status")
    return int(flags.value)


# ---- Several new tokens a sequence (rotary positions, cache writes, trees) ----
# These wrappers check dtypes, shapes and devices before they pass pointers on,
# and launch on the tensors' device: on its current stream unless one is given.


class _Entry:
    """What these wrappers ask torch and the library for on every call, looked
    up once: a call costs the host a few microseconds in all."""

    def __init__(self):
        import torch
        self.bf16, self.i32, self.i64 = torch.bfloat16, torch.int32, torch.int64
        self.device, self.raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        self.use_device = torch.cuda.device
        lib = load_library()
        self.rotate, self.append_tokens = lib.ffd_rotate, lib.ffd_append_tokens
        self.read_cache, self.decode_tree = lib.ffd_read_cache, lib.ffd_decode_tree


_the_entry: Optional[_Entry] = None


def _entry() -> _Entry:
    global _the_entry
    if _the_entry is None:
        _the_entry = _Entry()
    return _the_entry


def _tensor(t, dtype, shape, what: str, device: int) -> int:
    """Data pointer of a dense CUDA tensor of exactly this type, shape and device."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == device:
        return t.data_ptr()
    raise ValueError(f"{what}: want a contiguous {dtype} tensor of shape {tuple(shape)} on "
                     f"cuda:{device}, got {t.dtype} {tuple(t.shape)} on {t.device}"
                     f"{'' if t.is_contiguous() else ' (not contiguous)'}")


def _device_of(t) -> int:
    if not t.is_cuda:
        raise ValueError("FFD entry points take CUDA tensors")
    return t.get_device()


def _call(device: int, stream, what: str, fn, *args) -> None:
    """fn(*args, stream) with `device` current."""
    e = _entry()
    if stream is None:
        stream = e.raw_stream(device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if e.device() == device:
        status = fn(*args, stream)
    else:
        with e.use_device(device):
            status = fn(*args, stream)
    if status != FFD_OK:
        raise FFDError(status, what)


class KVCache:
    """A KV cache of one layer: bf16 k and v [B, Hkv, cap, 128], or
    float8_e4m3fn k and v with bf16 k_scales and v_scales [B, Hkv, cap] (one
    scale a row).  Wraps the caller's tensors; `KVCache.empty` makes new ones."""

    def __init__(self, k, v, k_scales=None, v_scales=None):
        import torch
        device = _device_of(k)
        if k.dim() != 4 or k.shape[-1] != 128 or k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError("k is bf16 or float8_e4m3fn [B, Hkv, cap, 128]")
        self.format = FFD_CACHE_BF16 if k.dtype == torch.bfloat16 else FFD_CACHE_BYTE
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.device, self.key = device, tuple(k.shape[:3])
        if (self.format == FFD_CACHE_BYTE) != (k_scales is not None) or (k_scales is None) != (v_scales is None):
            raise ValueError("an 8-bit cache has k_scales and v_scales, a bf16 cache has neither")
        s = torch.Size(self.key)
        self._c = _Cache(self.format, 0, _tensor(k, k.dtype, k.shape, "k", device),
                         _tensor(v, k.dtype, k.shape, "v", device),
                         None if k_scales is None else _tensor(k_scales, torch.bfloat16, s, "k_scales", device),
                         None if v_scales is None else _tensor(v_scales, torch.bfloat16, s, "v_scales", device))

    @classmethod
    def empty(cls, shape: Shape, format: int = FFD_CACHE_BF16, device="cuda"):
        """A cache without tokens, all zero: ffd_decode wants finite values past a
        sequence's length."""
        import torch
        key = (shape.batch, shape.num_kv_heads, shape.capacity)
        if format == FFD_CACHE_BF16:
            kv = [torch.zeros((*key, 128), dtype=torch.bfloat16, device=device) for _ in range(2)]
            return cls(*kv)
        if format != FFD_CACHE_BYTE:
            raise ValueError("unknown cache format")
        kv = [torch.zeros((*key, 128), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2)]
        return cls(*kv, *(torch.zeros(key, dtype=torch.bfloat16, device=device) for _ in range(2)))

    def _of(self, shape: Shape):
        if self.key != (shape.batch, shape.num_kv_heads, shape.capacity):
            raise ValueError(f"cache {self.key} does not fit {shape}")
        return self._c


def rotate(rope: Rope, positions, q, q_out, k=None, k_out=None, inverse: bool = False,
           stream=None) -> None:
    """ffd_rotate: rotary positions of bf16 q [tokens, Hq, 128] and, if given,
    k [tokens, Hkv, 128]; positions int32 [tokens].  An output may be its
    input."""
    e, dev, shape = _entry(), _device_of(q), q.shape
    if len(shape) != 3 or shape[2] != 128:
        raise ValueError("q is [tokens, heads, 128]")
    tokens = shape[0]
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    if k is None:
        heads, k_at, k_out_at = 0, None, None
    else:
        k_shape = k.shape
        if len(k_shape) != 3 or k_shape[0] != tokens or k_shape[2] != 128:
            raise ValueError("k is [tokens, heads, 128]")
        heads = k_shape[1]
        k_at, k_out_at = _tensor(k, e.bf16, k_shape, "k", dev), _tensor(k_out, e.bf16, k_shape, "k_out", dev)
    _call(dev, stream, "ffd_rotate", e.rotate, rope, tokens,
          _tensor(positions, e.i32, (tokens,), "positions", dev), 1 if inverse else 0, shape[1],
          _tensor(q, e.bf16, shape, "q", dev), _tensor(q_out, e.bf16, shape, "q_out", dev), heads, k_at, k_out_at)


def append_tokens(shape: Shape, cache: KVCache, k_new, v_new, lengths, rope: Optional[Rope] = None,
                  positions=None, new_lengths=None, q=None, q_out=None, stream=None) -> None:
    """ffd_append_tokens: rotate the new queries and keys (with `rope`) and
    write the new K/V rows into the cache.  k_new, v_new bf16 [B, n, Hkv, 128];
    q, q_out bf16 [B, n, Hq, 128] or neither; lengths int32 [B], the new tokens
    counted; new_lengths int32 [B] for fewer than n; positions int32 [B, n]
    (default: the slots).  For ffd.decode on the same cache, quantize_keys again from
    the first block that changed on."""
    e, dev = _entry(), cache.device
    if k_new.dim() != 4:
        raise ValueError("k_new is [B, n, Hkv, 128]")
    bf16, i32, B, n = e.bf16, e.i32, shape.batch, k_new.shape[1]
    kv = (B, n, shape.num_kv_heads, 128)
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    qs = (B, n, shape.num_q_heads, 128)
    _call(dev, stream, "ffd_append_tokens", e.append_tokens, shape, cache._of(shape), rope, n,
          None if q is None else _tensor(q, bf16, qs, "q", dev), _tensor(k_new, bf16, kv, "k_new", dev),
          _tensor(v_new, bf16, kv, "v_new", dev),
          None if positions is None else _tensor(positions, i32, (B, n), "positions", dev),
          _tensor(lengths, i32, (B,), "lengths", dev),
          None if new_lengths is None else _tensor(new_lengths, i32, (B,), "new_lengths", dev),
          None if q_out is None else _tensor(q_out, bf16, qs, "q_out", dev))


def read_cache(shape: Shape, cache: KVCache, lengths, token_begin: int, k_out=None, v_out=None,
               stream=None) -> None:
    """ffd_read_cache: tokens from token_begin on of an 8-bit cache back to
    bf16; k_out, v_out [B, Hkv, count, 128], either may be None."""
    if k_out is None and v_out is None:
        raise ValueError("nothing to read: k_out and v_out are None")
    e, dev = _entry(), cache.device
    what, out = ("k_out", k_out) if k_out is not None else ("v_out", v_out)
    if out.dim() != 4:
        raise ValueError(f"{what} is [B, Hkv, count, 128]")
    count = out.shape[2]
    want = (shape.batch, shape.num_kv_heads, count, 128)
    _call(dev, stream, "ffd_read_cache", e.read_cache, shape, cache._of(shape),
          _tensor(lengths, e.i32, (shape.batch,), "lengths", dev), int(token_begin), count,
          None if k_out is None else _tensor(k_out, e.bf16, want, "k_out", dev),
          None if v_out is None else _tensor(v_out, e.bf16, want, "v_out", dev))


def decode_tree_workspace_bytes(shape: Shape, num_nodes: int) -> int:
    return int(load_library().ffd_decode_tree_workspace_bytes(ctypes.byref(shape), int(num_nodes)))


def tree_workspace(shape: Shape, num_nodes: int, device="cuda"):
    """A cleared workspace for decode_tree with up to num_nodes nodes."""
    import torch
    nbytes = decode_tree_workspace_bytes(shape, num_nodes)
    if nbytes == 0:
        raise ValueError(f"decode_tree does not take {shape} with {num_nodes} nodes")
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _call(ws.get_device(), None, "ffd_decode_tree_workspace_init",
          load_library().ffd_decode_tree_workspace_init, ctypes.byref(shape), int(num_nodes),
          ws.data_ptr(), nbytes)
    return ws


def decode_tree(shape: Shape, cache: KVCache, q, lengths, out, workspace, tree_mask=None,
                tree_sizes=None, stream=None) -> None:
    """ffd_decode_tree: attention of n drafted tokens a sequence over the cache
    that holds them in its last rows.  q, out bf16 [B, n, Hq, 128]; lengths
    int32 [B], the tree counted; tree_mask int64 [B, n] (bit j of node i's
    word: i sees j; default a chain); tree_sizes int32 [B] for fewer than n
    nodes.  tree_from_parents makes masks from parent lists."""
    e, dev = _entry(), cache.device
    if q.dim() != 4:
        raise ValueError("q is [B, n, Hq, 128]")
    B, n = shape.batch, q.shape[1]
    qs = (B, n, shape.num_q_heads, 128)
    if workspace.dim() != 1 or workspace.element_size() != 1:
        raise ValueError("workspace: the bytes that tree_workspace gives")
    nbytes = workspace.numel()
    _call(dev, stream, "ffd_decode_tree", e.decode_tree, shape, cache._of(shape), n,
          _tensor(q, e.bf16, qs, "q", dev), _tensor(lengths, e.i32, (B,), "lengths", dev),
          None if tree_sizes is None else _tensor(tree_sizes, e.i32, (B,), "tree_sizes", dev),
          None if tree_mask is None else _tensor(tree_mask, e.i64, (B, n), "tree_mask", dev),
          _tensor(out, e.bf16, qs, "out", dev), _tensor(workspace, workspace.dtype, (nbytes,), "workspace", dev), nbytes)


def tree_from_parents(parents):
    """(mask, depth) of trees given as parent lists: parents[b][i] is node i's
    parent (an earlier node) or -1.  mask int64 [B, n]: each node sees its
    ancestors and itself; depth int32 [B, n]: 0 at the roots, to be added to
    the tree's first position.  Host tensors; shorter lists are padded with
    nodes that see nothing."""
    import torch
    n = max((len(p) for p in parents), default=0)
    if n > FFD_MAX_TREE_NODES:
        raise ValueError(f"a tree has at most {FFD_MAX_TREE_NODES} nodes")
    mask = torch.zeros((len(parents), n), dtype=torch.int64)
    depth = torch.zeros((len(parents), n), dtype=torch.int32)
    for b, tree in enumerate(parents):
        words, depths = [], []
        for i, parent in enumerate(tree):
            if not -1 <= parent < i:
                raise ValueError(f"node {i}: its parent is -1 or an earlier node, not {parent}")
            words.append((words[parent] if parent >= 0 else 0) | 1 << i)
            depths.append(depths[parent] + 1 if parent >= 0 else 0)
            mask[b, i] = words[i] - (1 << 64) if words[i] >> 63 else words[i]
            depth[b, i] = depths[i]
    return mask, depth


class DecodeBuffers:
    """Device buffers one decode step needs besides the caller's KV cache.

    Allocation is PyTorch's job (caching allocator); the library only
    receives pointers.
    """

    def __init__(self, shape: Shape, device="cuda"):
        import torch
        self.shape = shape
        B, Hq, Hkv = shape.batch, shape.num_q_heads, shape.num_kv_heads
        cap, T, D = shape.capacity, shape.block_size, shape.head_dim
        self.k_packed = torch.empty((B, Hkv, cap, D // 2), dtype=torch.uint8, device=device)
        self.k_scales = torch.empty((B, Hkv, cap // T, D), dtype=torch.bfloat16, device=device)
        self.out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=device)
        self.mask = torch.empty((B, Hkv, math.ceil(cap // T / 32)), dtype=torch.int32,
                                device=device)
        ws = decode_workspace_bytes(shape)
        self.workspace = torch.empty((max(ws, 256) + 15) // 16 * 16, dtype=torch.uint8,
                                     device=device)
        workspace_init(shape, self.workspace)


class ThumbResidBuffers(DecodeBuffers):
    """DecodeBuffers plus the thumbnail + residual key copy (k_packed unused)."""

    def __init__(self, shape: Shape, device="cuda"):
        import torch
        super().__init__(shape, device)
        B, Hkv, cap, D = shape.batch, shape.num_kv_heads, shape.capacity, shape.head_dim
        self.k_packed = None
        self.k_thumb = torch.empty((B, Hkv, cap, D // 4), dtype=torch.uint8, device=device)
        self.k_resid = torch.empty((B, Hkv, cap, D), dtype=torch.uint8, device=device)


class StepGraph:
    """Owner of a native decode-step graph (ffd_step_graph_*): one call runs
    H2D of the inputs, the fused append + decode and D2H of the results."""

    def __init__(self, shape: Shape, fmt: int, reference: int, delta: float, advance: bool,
                 host_in, dev_in, k, v, k_copy, k_resid, k_scales, lengths, dev_result,
                 host_result, mask_offset: int, workspace):
        self._lib = load_library()
        handle = ctypes.c_void_p(None)
        _check(self._lib.ffd_step_graph_create(
            ctypes.byref(shape), int(fmt), int(reference), float(delta), 1 if advance else 0,
            host_in.data_ptr(), _ptr(dev_in), _ptr(k), _ptr(v), _ptr(k_copy), _ptr(k_resid),
            _ptr(k_scales), _ptr(lengths), _ptr(dev_result), host_result.data_ptr(),
            int(mask_offset), _ptr(workspace), workspace.numel() * workspace.element_size(),
            ctypes.byref(handle)), "ffd_step_graph_create")
        self._handle = handle

    def run(self) -> None:
        _check(self._lib.ffd_step_graph_run(self._handle), "ffd_step_graph_run")

    def close(self) -> None:
        if self._handle is not None and self._handle.value:
            self._lib.ffd_step_graph_destroy(self._handle)
        self._handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # interpreter shutdown
            pass
