"""Python binding of libcb (C ABI in include/cb.h): argument marshalling only.

Every step of the attention path runs in the library's CUDA kernels; this
module only turns torch tensors into device pointers and sizes, passes the
caller's current CUDA stream, and raises ``CbError`` on a non-OK status. If
libcb.so has not been built, every call raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

from .build import LIB_PATH

CB_F32 = 0
CB_BF16 = 1
CB_FLAG_PORTABLE_ONLY = 0x1
CB_FLAG_TEST_WAIT_EXPIRY = 0x2  # tests of the failure path only (see include/cb.h)
CB_FLAG_SHARE_ALWAYS = 0x4  # paged_attention_shared: share also where it would not pay
CB_DEVERR_BLOCK_ID = 0x1
CB_DEVERR_SLOT = 0x2
CB_DEVERR_TIMEOUT = 0x4

STATUS = {0: "CB_OK", 1: "CB_ERR_INVALID_ARG", 2: "CB_ERR_METADATA", 3: "CB_ERR_UNSUPPORTED",
          4: "CB_ERR_WORKSPACE", 5: "CB_ERR_CUDA", 6: "CB_ERR_DEVICE_CHECK"}


class CbError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


_LIB = None

_i32 = ctypes.c_int32
_vp = ctypes.c_void_p
_SIGNATURES = {
    "cb_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "cb_last_error_message": (ctypes.c_char_p, []),
    "cb_last_cuda_error": (ctypes.c_int, []),
    "cb_abi_version": (ctypes.c_int, []),
    "cb_write_kv": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                   _vp, _vp]),
    "cb_copy_blocks": (ctypes.c_int, [_vp, _vp, _vp, _vp, ctypes.c_int64, ctypes.c_int64, _vp,
                                      _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp]),
    "cb_workspace_size": (ctypes.c_size_t, [_i32, _i32, _i32, _i32, _i32]),
    "cb_workspace_init": (ctypes.c_int, [_vp, ctypes.c_size_t, _vp]),
    "cb_paged_attention": (ctypes.c_int, [
        _vp, _vp, _vp, _vp,            # out, q, k_cache, v_cache
        _vp, _vp, _vp,                 # k_new, v_new, slot_mapping
        _vp, _vp, _vp, _i32,           # query_start_loc, seq_lens, block_table, stride
        _vp, _vp,                      # host mirrors
        _i32, _i32, _i32, _i32,        # R, T, num_blocks, block_size
        _i32, _i32, _i32,              # Hq, Hkv, D
        ctypes.c_float, _i32, _i32,    # scale, sliding_window, dtype
        ctypes.c_uint32, _vp, ctypes.c_size_t, _vp]),  # flags, workspace, bytes, stream
    "cb_paged_attention_ring": (ctypes.c_int, [
        _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32,  # ... stride, ring_blocks
        _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
        ctypes.c_float, _i32, _i32, ctypes.c_uint32, _vp, ctypes.c_size_t, _vp]),
    "cb_graph_cache_create": (ctypes.c_int, [_i32, _i32, ctypes.POINTER(ctypes.c_void_p)]),
    "cb_graph_cache_destroy": (None, [_vp]),
    "cb_graph_cache_stats": (ctypes.c_int, [_vp, ctypes.POINTER(ctypes.c_int64),
                                            ctypes.POINTER(ctypes.c_int64),
                                            ctypes.POINTER(ctypes.c_int64)]),
    "cb_paged_attention_graphed": (ctypes.c_int, [_vp] + [
        _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp,
        _i32, _i32, _i32, _i32, _i32, _i32, _i32, ctypes.c_float, _i32, _i32, ctypes.c_uint32,
        _vp, ctypes.c_size_t, _vp]),
    "cb_read_error_word": (ctypes.c_int, [_vp, _vp, _vp]),
    "cb_no_alloc_read_error_word": (ctypes.c_int, [_vp, _vp]),
    "cb_paged_attention_no_alloc": (ctypes.c_int, [
        _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp,
        _i32, _i32, _i32, _i32, _i32, _i32, _i32, ctypes.c_float, _i32, _i32, ctypes.c_uint32,
        _vp]),
    "cb_write_kv_q8": (ctypes.c_int, [_vp] * 7 + [_i32] * 6 + [_vp, _vp]),
    "cb_read_kv_q8": (ctypes.c_int, [_vp] * 7 + [_i32] * 6 + [_vp, _vp]),
    "cb_workspace_size_q8": (ctypes.c_size_t, [_i32] * 6 + [ctypes.c_int64]),
    "cb_paged_attention_q8": (ctypes.c_int, [_vp] * 12 + [_i32, _vp, _vp] + [_i32] * 7 + [
        ctypes.c_float, _i32, _i32, ctypes.c_uint32, _vp, ctypes.c_size_t, _vp]),
    "cb_workspace_size_shared": (ctypes.c_size_t, [_i32] * 5),
    "cb_paged_attention_shared": (ctypes.c_int, [_vp] * 10 + [_i32] + [_vp] * 5 + [_i32] * 8 + [
        ctypes.c_float, _i32, _i32, ctypes.c_uint32, _vp, ctypes.c_size_t, _vp]),
    "cb_launch_count": (ctypes.c_longlong, [ctypes.c_int]),
    "cb_num_kernels": (ctypes.c_int, []),
    "cb_kernel_name": (ctypes.c_char_p, [ctypes.c_int]),
    "cb_kernel_timing": (ctypes.c_int, [ctypes.c_int]),
    "cb_kernel_timing_collect": (ctypes.c_int, [_vp, _vp, ctypes.c_int]),
}


def lib_path() -> str:
    return os.environ.get("CB_LIB", LIB_PATH)


def lib() -> ctypes.CDLL:
    """The loaded libcb.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libcb.so not built at {path}: run paged_kv_attention_cb_gb300.build")
        handle = ctypes.CDLL(path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = handle
    return _LIB


def _check(status: int):
    if status != 0:
        msg = lib().cb_last_error_message().decode()
        raise CbError(status, msg)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch

        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t) -> int:
    import torch

    if t.dtype == torch.float32:
        return CB_F32
    if t.dtype == torch.bfloat16:
        return CB_BF16
    raise CbError(1, f"unsupported dtype {t.dtype}")


def _host_i32(a) -> np.ndarray:
    if hasattr(a, "detach"):
        a = a.detach().cpu().numpy()
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def write_kv(k_new, v_new, k_cache, v_cache, slot_mapping, error_word=None, stream=None):
    """Scatter k_new/v_new [T, Hkv, D] into the caches [NB, BS, Hkv, D] at slot_mapping [T]."""
    T, Hkv, D = k_new.shape
    NB, BS = k_cache.shape[0], k_cache.shape[1]
    _check(lib().cb_write_kv(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                             _ptr(slot_mapping), T, NB, BS, Hkv, D, _dtype_code(k_new),
                             _ptr(error_word), _stream(stream)))


def copy_blocks(k_src, v_src, k_dst, v_dst, src_ids, dst_ids, error_word=None, stream=None):
    """Block dst_ids[i] of k_dst/v_dst [NBd, BS, Hkv, D] = block src_ids[i] of k_src/v_src."""
    NBs, BS, Hkv, D = k_src.shape
    n = int(src_ids.numel())
    if int(dst_ids.numel()) != n or tuple(k_dst.shape[1:]) != (BS, Hkv, D):
        raise ValueError("copy_blocks: id counts or block shapes differ")
    _check(lib().cb_copy_blocks(_ptr(k_src), _ptr(v_src), _ptr(k_dst), _ptr(v_dst), NBs,
                                k_dst.shape[0], _ptr(src_ids), _ptr(dst_ids), n, BS, Hkv, D,
                                _dtype_code(k_src), _ptr(error_word), _stream(stream)))


def workspace_size(num_requests, num_tokens, num_q_heads, num_kv_heads, head_dim) -> int:
    return int(lib().cb_workspace_size(num_requests, num_tokens, num_q_heads, num_kv_heads,
                                       head_dim))


def workspace_init(workspace, stream=None):
    _check(lib().cb_workspace_init(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                   _stream(stream)))


def read_error_word(workspace, stream=None) -> int:
    """Synchronise, return and clear the device error word (0 = no error recorded)."""
    word = ctypes.c_int32(0)
    status = lib().cb_read_error_word(_ptr(workspace), ctypes.byref(word), _stream(stream))
    if status not in (0, 6):
        _check(status)
    return int(word.value)


def paged_attention(out, q, k_cache, v_cache, query_start_loc, seq_lens, block_table,
                    h_query_start_loc, h_seq_lens, workspace, *, scale=0.0, sliding_window=0,
                    k_new=None, v_new=None, slot_mapping=None, flags=0, stream=None,
                    ring_blocks=0):
    """One ragged paged-attention step (see cb_paged_attention in include/cb.h).

    out, q: [T, Hq, D]; caches [NB, BS, Hkv, D]; device metadata int32 (slot_mapping
    int64); h_query_start_loc / h_seq_lens: host copies of the same metadata.
    ring_blocks > 0: a sliding-window layer whose pages are recycled in a ring
    (cb_paged_attention_ring): logical block b at block_table[r, b % ring_blocks].
    """
    T, Hq, D = q.shape
    NB, BS, Hkv, _ = k_cache.shape
    R = int(seq_lens.shape[0])
    hq = _host_i32(h_query_start_loc)
    hs = _host_i32(h_seq_lens)
    if hq.shape[0] != R + 1 or hs.shape[0] != R:
        raise CbError(2, "host mirrors must have R+1 and R entries")
    stride = int(block_table.shape[1]) if block_table.dim() == 2 else 0
    head = (_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new),
            _ptr(slot_mapping), _ptr(query_start_loc), _ptr(seq_lens), _ptr(block_table), stride)
    tail = (hq.ctypes.data_as(ctypes.c_void_p), hs.ctypes.data_as(ctypes.c_void_p),
            R, T, NB, BS, Hq, Hkv, D, float(scale), int(sliding_window), _dtype_code(q),
            int(flags), _ptr(workspace), workspace.numel() * workspace.element_size(),
            _stream(stream))
    if ring_blocks:
        _check(lib().cb_paged_attention_ring(*head, int(ring_blocks), *tail))
    else:
        _check(lib().cb_paged_attention(*head, *tail))
    return out


class GraphCache:
    """CUDA graphs of the step, one per padded shape (cb_graph_cache in include/cb.h)."""

    def __init__(self, q_interval=64, kv_interval=0):
        h = ctypes.c_void_p()
        _check(lib().cb_graph_cache_create(int(q_interval), int(kv_interval), ctypes.byref(h)))
        self._h = h
        self.q_interval = int(q_interval)

    def close(self):
        if self._h:
            lib().cb_graph_cache_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def stats(self):
        g, c, r = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(lib().cb_graph_cache_stats(self._h, ctypes.byref(g), ctypes.byref(c),
                                          ctypes.byref(r)))
        return {"graphs": g.value, "captures": c.value, "replays": r.value}


def paged_attention_graphed(cache, out, q, k_cache, v_cache, query_start_loc, seq_lens,
                            block_table, h_query_start_loc, h_seq_lens, workspace, *, scale=0.0,
                            sliding_window=0, k_new=None, v_new=None, slot_mapping=None, flags=0,
                            stream=None):
    """paged_attention through a GraphCache: the buffers hold the padded shape (R and T
    multiples of the cache's q_interval; padding requests q_len 0 / seq_len 0, padding
    tokens past query_start_loc[R] with slot -1)."""
    T, Hq, D = q.shape
    NB, BS, Hkv, _ = k_cache.shape
    R = int(seq_lens.shape[0])
    hq = _host_i32(h_query_start_loc)
    hs = _host_i32(h_seq_lens)
    if hq.shape[0] != R + 1 or hs.shape[0] != R:
        raise CbError(2, "host mirrors must have R+1 and R entries")
    stride = int(block_table.shape[1]) if block_table.dim() == 2 else 0
    _check(lib().cb_paged_attention_graphed(
        cache._h, _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new),
        _ptr(slot_mapping), _ptr(query_start_loc), _ptr(seq_lens), _ptr(block_table), stride,
        hq.ctypes.data_as(ctypes.c_void_p), hs.ctypes.data_as(ctypes.c_void_p),
        R, T, NB, BS, Hq, Hkv, D, float(scale), int(sliding_window), _dtype_code(q), int(flags),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


class PreparedGraphStep:
    """paged_attention_graphed with the argument marshalling done once.

    For a serving loop over persistent buffers: the caller writes each step's inputs
    into the same device tensors and the same host-mirror arrays (numpy int32,
    updated in place), then calls the object; each call is one C call (a replay, or a
    capture for a new padded shape). The padded counts R and T are fixed by the
    tensors' shapes.
    """

    def __init__(self, cache, out, q, k_cache, v_cache, query_start_loc, seq_lens, block_table,
                 h_query_start_loc, h_seq_lens, workspace, *, scale=0.0, sliding_window=0,
                 k_new=None, v_new=None, slot_mapping=None, flags=0, stream=None):
        import numpy as np

        T, Hq, D = q.shape
        NB, BS, Hkv, _ = k_cache.shape
        R = int(seq_lens.shape[0])
        for h, n in ((h_query_start_loc, R + 1), (h_seq_lens, R)):
            if not (isinstance(h, np.ndarray) and h.dtype == np.int32 and h.flags.c_contiguous
                    and h.shape == (n,)):
                raise ValueError("host mirrors must be contiguous int32 numpy arrays of R+1 / R")
        self._keep = (cache, out, q, k_cache, v_cache, query_start_loc, seq_lens, block_table,
                      h_query_start_loc, h_seq_lens, workspace, k_new, v_new, slot_mapping)
        stride = int(block_table.shape[1]) if block_table.dim() == 2 else 0
        self._fn = lib().cb_paged_attention_graphed
        self._args = (
            cache._h, _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new),
            _ptr(slot_mapping), _ptr(query_start_loc), _ptr(seq_lens), _ptr(block_table), stride,
            h_query_start_loc.ctypes.data_as(ctypes.c_void_p),
            h_seq_lens.ctypes.data_as(ctypes.c_void_p), R, T, NB, BS, Hq, Hkv, D, float(scale),
            int(sliding_window), _dtype_code(q), int(flags), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream))

    def __call__(self):
        status = self._fn(*self._args)
        if status != 0:
            _check(status)


NO_ALLOC_SCRATCH_BYTES = 8 << 20


def paged_attention_no_alloc(out, q, k_cache, v_cache, query_start_loc, seq_lens, block_table,
                             h_query_start_loc, h_seq_lens, *, scale=0.0, sliding_window=0,
                             k_new=None, v_new=None, slot_mapping=None, flags=0, stream=None):
    """paged_attention without a workspace, for callers that may not allocate device memory
    at call time (see cb_paged_attention_no_alloc in include/cb.h)."""
    T, Hq, D = q.shape
    NB, BS, Hkv, _ = k_cache.shape
    R = int(seq_lens.shape[0])
    hq = _host_i32(h_query_start_loc)
    hs = _host_i32(h_seq_lens)
    if hq.shape[0] != R + 1 or hs.shape[0] != R:
        raise CbError(2, "host mirrors must have R+1 and R entries")
    stride = int(block_table.shape[1]) if block_table.dim() == 2 else 0
    _check(lib().cb_paged_attention_no_alloc(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new),
        _ptr(slot_mapping), _ptr(query_start_loc), _ptr(seq_lens), _ptr(block_table), stride,
        hq.ctypes.data_as(ctypes.c_void_p), hs.ctypes.data_as(ctypes.c_void_p),
        R, T, NB, BS, Hq, Hkv, D, float(scale), int(sliding_window), _dtype_code(q), int(flags),
        _stream(stream)))
    return out


def no_alloc_read_error_word(stream=None) -> int:
    """Synchronise, return and clear the error word of paged_attention_no_alloc on the
    current device (0 = no error recorded)."""
    word = ctypes.c_int32(0)
    status = lib().cb_no_alloc_read_error_word(ctypes.byref(word), _stream(stream))
    if status not in (0, 6):
        _check(status)
    return int(word.value)


# ------------------------------------------------- checked calls (8-bit cache, shared prefixes)
#
# These entry points check every tensor (type, shape, contiguity, device) before the call. The
# checks run on whole lists at once: a small decode step takes ~10 us on the GPU, and a Python
# statement per tensor and property took longer than that.


class _Torch:
    """torch's types and methods that the checks use, looked up on first use (the module itself
    imports without torch)."""

    def __init__(self):
        import torch

        self.e4m3 = (torch.float8_e4m3fn, torch.uint8)
        self.e8m0 = (torch.float8_e8m0fnu, torch.uint8)
        self.i32, self.i64 = torch.int32, torch.int64
        self.code = {torch.float32: CB_F32, torch.bfloat16: CB_BF16}
        self.device_of = torch.Tensor.get_device
        self.contiguous = torch.Tensor.is_contiguous
        self.ptr = torch.Tensor.data_ptr
        self.current_device = torch.cuda.current_device
        self.device = torch.cuda.device
        # the raw handle of the current stream; the public call wraps it in an object first
        self.stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda d: torch.cuda.current_stream(d).cuda_stream)


_TORCH = None
_NP_I32 = np.dtype(np.int32)
_addressof, _from_buffer = ctypes.addressof, ctypes.c_char.from_buffer


def _torch() -> _Torch:
    global _TORCH
    if _TORCH is None:
        _TORCH = _Torch()
    return _TORCH


def _pointers(tensors, shapes, dtypes, names):
    """The data pointers of contiguous tensors of these shapes and dtypes, all on one CUDA device,
    and its index. ``names``: a function that gives their names, for the error."""
    t = _torch()
    device = t.device_of(tensors[0])
    if (device >= 0 and tuple([x.shape for x in tensors]) == shapes
            and tuple([x.dtype for x in tensors]) == dtypes and all(map(t.contiguous, tensors))
            and set(map(t.device_of, tensors)) == {device}):
        return list(map(t.ptr, tensors)), device
    names = names()
    for x, name, shape, dtype in zip(tensors, names, shapes, dtypes):
        if x.dtype != dtype:
            raise CbError(1, f"{name}: dtype {x.dtype}, not {dtype}")
        if tuple(x.shape) != tuple(shape):
            raise CbError(1, f"{name}: shape {tuple(x.shape)}, not {tuple(shape)}")
        if not x.is_contiguous():
            raise CbError(1, f"{name} must be contiguous")
        if not x.is_cuda or x.device != tensors[0].device:
            raise CbError(1, f"{name} must be on the CUDA device of {names[0]}")
    raise CbError(1, "tensors must be on a CUDA device")


def _call(fn, device, stream, *args):
    """fn(*args, stream) with the tensors' device current: the library launches on it."""
    t = _torch()
    if stream is None:
        stream = t.stream(device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if device == t.current_device():
        status = fn(*args, stream)
    else:
        with t.device(device):
            status = fn(*args, stream)
    if status:
        _check(status)


def _mirror(a, n, name):
    """A host mirror as a contiguous int32 array of n entries, and its address (ndarray.ctypes takes
    a microsecond; the buffer protocol a third of it, for writable arrays)."""
    if type(a) is not np.ndarray or a.dtype != _NP_I32 or not a.flags.c_contiguous:
        a = _host_i32(a)
    if a.shape != (n,):
        raise CbError(2, f"{name}: {a.shape} entries, not {n}")
    if a.flags.writeable and n:
        return a, _addressof(_from_buffer(a))
    return a, a.ctypes.data


def _dims(t, n, name):
    if t.dim() != n:
        raise CbError(1, f"{name}: {t.dim()} dimensions, not {n}")
    return t.shape


def _float_type(t, name):
    code = _torch().code.get(t.dtype)
    if code is None:
        raise CbError(1, f"{name}: dtype {t.dtype}, not torch.float32 or torch.bfloat16")
    return code


# ---------------------------------------------------------------- 8-bit paged cache


_CACHE_NAMES = ("k_cache", "v_cache", "k_scale", "v_scale")


def _cache_q8(k_cache, v_cache, k_scale, v_scale):
    """(tensors, shapes, dtypes) of an 8-bit cache."""
    t = _torch()
    shape = _dims(k_cache, 4, "k_cache")
    value, scale = k_cache.dtype, k_scale.dtype
    if value not in t.e4m3:
        raise CbError(1, f"k_cache: dtype {value}, not {' or '.join(map(str, t.e4m3))}")
    if scale not in t.e8m0:
        raise CbError(1, f"k_scale: dtype {scale}, not {' or '.join(map(str, t.e8m0))}")
    rows = shape[:3]
    return ((k_cache, v_cache, k_scale, v_scale), (shape, shape, rows, rows),
            (value, value, scale, scale))


def _rows_q8(fn, rows, names, cache, slot_mapping, error_word, stream):
    t = _torch()
    a, b = rows
    code = _float_type(a, names[0])
    shape = T, Hkv, D = _dims(a, 3, names[0])
    tensors, shapes, dtypes = _cache_q8(*cache)
    NB, BS, H, Dc = shapes[0]
    if H != Hkv or Dc != D:
        raise CbError(1, f"k_cache: rows of {(H, Dc)}, not {(Hkv, D)}")
    kind = a.dtype
    tensors = (a, b, *tensors, slot_mapping)
    shapes = (shape, shape, *shapes, (T,))
    dtypes = (kind, kind, *dtypes, t.i64)
    if error_word is not None:
        tensors, shapes, dtypes = (*tensors, error_word), (*shapes, error_word.shape), (*dtypes, t.i32)
    p, device = _pointers(tensors, shapes, dtypes,
                          lambda: (*names, *_CACHE_NAMES, "slot_mapping", "error_word"))
    word = p[7] if error_word is not None else None
    if names[0] == "k_out":
        _call(fn, device, stream, p[2], p[3], p[4], p[5], p[6], p[0], p[1], T, NB, BS, Hkv, D,
              code, word)
    else:
        _call(fn, device, stream, p[0], p[1], p[2], p[3], p[4], p[5], p[6], T, NB, BS, Hkv, D,
              code, word)


def write_kv_q8(k_new, v_new, k_cache, v_cache, k_scale, v_scale, slot_mapping, error_word=None,
                stream=None):
    """Quantise k_new/v_new [T, Hkv, D] (bf16 or fp32) into the 8-bit caches [NB, BS, Hkv, D]
    (float8_e4m3fn) and their scales [NB, BS, Hkv] (float8_e8m0fnu) at slot_mapping [T].
    uint8 tensors are taken for either as well (see cb_write_kv_q8 in include/cb.h)."""
    _rows_q8(lib().cb_write_kv_q8, (k_new, v_new), ("k_new", "v_new"),
             (k_cache, v_cache, k_scale, v_scale), slot_mapping, error_word, stream)


def read_kv_q8(k_cache, v_cache, k_scale, v_scale, slot_mapping, k_out, v_out, error_word=None,
               stream=None):
    """k_out/v_out [T, Hkv, D] (bf16 or fp32) = the 8-bit caches' rows at slot_mapping [T]
    (rows of negative slots stay as they are; see cb_read_kv_q8 in include/cb.h)."""
    _rows_q8(lib().cb_read_kv_q8, (k_out, v_out), ("k_out", "v_out"),
             (k_cache, v_cache, k_scale, v_scale), slot_mapping, error_word, stream)


def workspace_size_q8(num_requests, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size,
                      chunk_kv_tokens=0) -> int:
    return int(lib().cb_workspace_size_q8(num_requests, num_tokens, num_q_heads, num_kv_heads,
                                          head_dim, block_size, chunk_kv_tokens))


def alloc_workspace_q8(num_requests, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size,
                       chunk_kv_tokens=0, device="cuda"):
    """Allocate (with torch) and zero a workspace of cb_workspace_size_q8 bytes."""
    import torch

    n = workspace_size_q8(num_requests, num_tokens, num_q_heads, num_kv_heads, head_dim,
                          block_size, chunk_kv_tokens)
    return torch.zeros((n + 15) // 16 * 16, dtype=torch.uint8, device=device)


_STEP_NAMES = ("q", "out", "query_start_loc", "seq_lens", "block_table", "workspace")
_NEW_NAMES = ("k_new", "v_new", "slot_mapping")


def _step(out, q, query_start_loc, seq_lens, block_table, workspace, cache, cache_names, k_new,
          v_new, slot_mapping):
    """Checks the tensors of a step over `cache` (tensors, shapes, dtypes; the first one the K
    cache). Returns the pointers -- q, out, query_start_loc, seq_lens, block_table, workspace,
    cache..., k_new, v_new, slot_mapping -- the device, and the sizes."""
    t = _torch()
    code = _float_type(q, "q")
    qs = T, Hq, D = _dims(q, 3, "q")
    (R,) = rs = _dims(seq_lens, 1, "seq_lens")
    stride = _dims(block_table, 2, "block_table")[1]
    ctensors, cshapes, cdtypes = cache
    NB, BS, Hkv, Dc = cshapes[0]
    if Dc != D:
        raise CbError(1, f"k_cache: head_dim {Dc}, not {D}")
    i32, kind = t.i32, q.dtype
    if k_new is not None:
        if v_new is None or slot_mapping is None:
            raise CbError(1, "k_new given without v_new or slot_mapping")
        rows = (T, Hkv, D)
        p, device = _pointers(
            (q, out, query_start_loc, seq_lens, block_table, workspace, *ctensors, k_new, v_new,
             slot_mapping),
            (qs, qs, (R + 1,), rs, (R, stride), workspace.shape, *cshapes, rows, rows, (T,)),
            (kind, kind, i32, i32, i32, workspace.dtype, *cdtypes, kind, kind, t.i64),
            lambda: (*_STEP_NAMES, *cache_names, *_NEW_NAMES))
    else:
        p, device = _pointers(
            (q, out, query_start_loc, seq_lens, block_table, workspace, *ctensors),
            (qs, qs, (R + 1,), rs, (R, stride), workspace.shape, *cshapes),
            (kind, kind, i32, i32, i32, workspace.dtype, *cdtypes),
            lambda: (*_STEP_NAMES, *cache_names))
        p += (None, None, None)
    return p, device, code, T, Hq, D, R, stride, NB, BS, Hkv


def paged_attention_q8(out, q, k_cache, v_cache, k_scale, v_scale, query_start_loc, seq_lens,
                       block_table, h_query_start_loc, h_seq_lens, workspace, *, scale=0.0,
                       sliding_window=0, k_new=None, v_new=None, slot_mapping=None, flags=0,
                       stream=None):
    """paged_attention over an 8-bit cache (see cb_paged_attention_q8 in include/cb.h).

    out, q: [T, Hq, D] bf16 or fp32; caches [NB, BS, Hkv, D] float8_e4m3fn and scales
    [NB, BS, Hkv] float8_e8m0fnu (or uint8); the step's k_new/v_new are quantised into their
    slots first. workspace: alloc_workspace_q8.
    """
    p, device, dtype, T, Hq, D, R, stride, NB, BS, Hkv = _step(
        out, q, query_start_loc, seq_lens, block_table, workspace,
        _cache_q8(k_cache, v_cache, k_scale, v_scale), _CACHE_NAMES, k_new, v_new, slot_mapping)
    hq, hq_at = _mirror(h_query_start_loc, R + 1, "h_query_start_loc")
    hs, hs_at = _mirror(h_seq_lens, R, "h_seq_lens")
    pq, pout, pqsl, pseq, pbt, pws, pk, pv, pks, pvs, pkn, pvn, psl = p
    _call(lib().cb_paged_attention_q8, device, stream, pout, pq, pk, pv, pks, pvs, pkn, pvn, psl,
          pqsl, pseq, pbt, stride, hq_at, hs_at, R, T, NB, BS, Hq, Hkv, D, scale, sliding_window,
          dtype, flags, pws, workspace.numel() * workspace.element_size())
    return out


# ---------------------------------------------------------------- shared prefixes


def workspace_size_shared(num_requests, num_tokens, num_q_heads, num_kv_heads, head_dim) -> int:
    return int(lib().cb_workspace_size_shared(num_requests, num_tokens, num_q_heads, num_kv_heads,
                                              head_dim))


def alloc_workspace_shared(num_requests, num_tokens, num_q_heads, num_kv_heads, head_dim,
                           device="cuda"):
    """Allocate (with torch) and zero a workspace of cb_workspace_size_shared bytes."""
    import torch

    n = workspace_size_shared(num_requests, num_tokens, num_q_heads, num_kv_heads, head_dim)
    return torch.zeros((n + 15) // 16 * 16, dtype=torch.uint8, device=device)


def paged_attention_shared(out, q, k_cache, v_cache, query_start_loc, seq_lens, block_table,
                           prefix_lens, h_query_start_loc, h_seq_lens, h_prefix_lens,
                           h_group_start, workspace, *, scale=0.0, sliding_window=0, k_new=None,
                           v_new=None, slot_mapping=None, flags=0, stream=None):
    """paged_attention for groups of requests that share a prompt prefix (see
    cb_paged_attention_shared in include/cb.h).

    prefix_lens [R] int32 on the device and h_prefix_lens on the host: positions each request
    shares with its group; h_group_start [n_groups + 1] on the host: group g is the requests
    h_group_start[g] .. h_group_start[g + 1] - 1. workspace: alloc_workspace_shared.
    """
    shape = _dims(k_cache, 4, "k_cache")
    cache = ((k_cache, v_cache, prefix_lens), (shape, shape, seq_lens.shape),
             (q.dtype, q.dtype, _torch().i32))
    p, device, dtype, T, Hq, D, R, stride, NB, BS, Hkv = _step(
        out, q, query_start_loc, seq_lens, block_table, workspace, cache,
        ("k_cache", "v_cache", "prefix_lens"), k_new, v_new, slot_mapping)
    groups = len(h_group_start) - 1
    if groups < 0:
        raise CbError(2, "h_group_start must have n_groups + 1 entries")
    hq, hq_at = _mirror(h_query_start_loc, R + 1, "h_query_start_loc")
    hs, hs_at = _mirror(h_seq_lens, R, "h_seq_lens")
    hp, hp_at = _mirror(h_prefix_lens, R, "h_prefix_lens")
    hg, hg_at = _mirror(h_group_start, groups + 1, "h_group_start")
    pq, pout, pqsl, pseq, pbt, pws, pk, pv, ppl, pkn, pvn, psl = p
    _call(lib().cb_paged_attention_shared, device, stream, pout, pq, pk, pv, pkn, pvn, psl, pqsl,
          pseq, pbt, stride, ppl, hq_at, hs_at, hp_at, hg_at, groups, R, T, NB, BS, Hq, Hkv, D,
          scale, sliding_window, dtype, flags, pws, workspace.numel() * workspace.element_size())
    return out


def launch_count(kernel: int = -1) -> int:
    """Kernels launched by libcb in this process (all kernels when kernel < 0)."""
    return int(lib().cb_launch_count(kernel))


def kernel_names():
    n = lib().cb_num_kernels()
    return [lib().cb_kernel_name(k).decode() for k in range(n)]


def kernel_timing(enable: bool):
    _check(lib().cb_kernel_timing(1 if enable else 0))


def kernel_timing_collect():
    """{kernel name: (total ms, launches)} since the previous collect (synchronises)."""
    n = lib().cb_num_kernels()
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_longlong * n)()
    _check(lib().cb_kernel_timing_collect(ms, cnt, n))
    names = kernel_names()
    return {names[k]: (float(ms[k]), int(cnt[k])) for k in range(n) if cnt[k]}


def alloc_workspace(num_requests, num_tokens, num_q_heads, num_kv_heads, head_dim, device="cuda"):
    """Allocate (with torch) and zero a workspace of cb_workspace_size bytes."""
    import torch

    n = workspace_size(num_requests, num_tokens, num_q_heads, num_kv_heads, head_dim)
    return torch.zeros((n + 15) // 16 * 16, dtype=torch.uint8, device=device)
