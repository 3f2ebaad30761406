"""B200-native split-KV decode attention (Flash-Decoding).

Python binding of libfd.so.  Every function here marshals arguments for the C
ABI declared in ``include/fd.h`` and calls it; all arithmetic runs in the
library's CUDA kernels.  There is no fallback: if libfd.so is missing or a
call fails, an exception is raised.

The functions named ``fd_*`` mirror the C entry points one to one and take
raw device pointers (ints) or torch tensors.  ``decode`` is a convenience
wrapper that allocates the outputs and workspace with torch and calls
``fd_decode`` on the current stream.
"""
from __future__ import annotations

import ctypes
import os
import sysconfig
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfd.so")
CALLS_PATH = os.path.join(_HERE, "_fdcall" + sysconfig.get_config_var("EXT_SUFFIX"))

FD_OK = 0
FD_ERR_INVALID_ARGUMENT = -1
FD_ERR_UNSUPPORTED = -2
FD_ERR_WORKSPACE = -3
FD_ERR_CUDA = -4
FD_ERR_DEVICE_TIMEOUT = -5

# Entry points declared in include/fd.h.
EXPORTS = ("fd_plan", "fd_plan_sm", "fd_plan_seqlens", "fd_plan_problem", "fd_split_chunk",
           "fd_effective_splits", "fd_workspace_bytes", "fd_decode",
           "fd_decode_partial", "fd_combine", "fd_combine_strided", "fd_quantize_keys",
           "fd_decode_sparse", "fd_append_int4", "fd_expand_int4", "fd_decode_int4",
           "fd_alloc_pages", "fd_release_pages",
           "fd_decode_static_workspace", "fd_check_device_error",
           "fd_selftest_device_timeout", "fd_status_string")

# Mirrors FD_STATIC_WORKSPACE_BYTES in include/fd.h (a CPU test compares the two).
FD_STATIC_WORKSPACE_BYTES = 8 << 20


class FdError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {fd_status_string(status)} ({status})" if what
                         else f"{fd_status_string(status)} ({status})")


FD_LAYOUT_HND = 0  # cache [.., Hkv, tokens, D]
FD_LAYOUT_NHD = 1  # cache [.., tokens, Hkv, D]
FD_KV_BF16 = 0       # bf16 cache
FD_KV_FP8_E4M3 = 1   # fp8 e4m3 cache, real value = scale * code
FD_KV_INT4 = 2       # 4-bit cache, value = s * (code - 8) + b per half row (the *_int4 calls)
FD_FP8_MMA_SYNC = 0     # fp8: codes converted to f16, mma.sync (default)
FD_FP8_MMA_TCGEN05 = 1  # fp8: tcgen05 kind::f8f6f4 on the codes in shared memory


class fd_problem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("D", ctypes.c_int32), ("max_len", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("kv_layout", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float), ("fp8_mma", ctypes.c_int32)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libfd.so (raises if it is not built: there is no fallback path)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing; build it with __graft_entry__.build()")
        lib = ctypes.CDLL(path)
        I, vp, sz, F = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
        lib.fd_plan.argtypes = [I] * 6
        lib.fd_plan.restype = I
        lib.fd_plan_sm.argtypes = [I] * 7
        lib.fd_plan_sm.restype = I
        lib.fd_plan_seqlens.argtypes = [I] * 7 + [vp]
        lib.fd_plan_seqlens.restype = I
        lib.fd_plan_problem.argtypes = [I, ctypes.POINTER(fd_problem), vp]
        lib.fd_plan_problem.restype = I
        lib.fd_split_chunk.argtypes = [I, I]
        lib.fd_split_chunk.restype = I
        lib.fd_effective_splits.argtypes = [I, I]
        lib.fd_effective_splits.restype = I
        lib.fd_workspace_bytes.argtypes = [I, I, I, I]
        lib.fd_workspace_bytes.restype = sz
        lib.fd_decode.argtypes = [ctypes.POINTER(fd_problem), vp, vp, vp, vp, vp, F, I, vp, vp,
                                  vp, sz, vp]
        lib.fd_decode.restype = I
        lib.fd_decode_partial.argtypes = [ctypes.POINTER(fd_problem), vp, vp, vp, vp, vp, F, I,
                                          vp, vp, vp, sz, vp]
        lib.fd_decode_partial.restype = I
        lib.fd_quantize_keys.argtypes = [ctypes.POINTER(fd_problem), vp, vp, vp, vp, vp]
        lib.fd_quantize_keys.restype = I
        lib.fd_decode_sparse.argtypes = [ctypes.POINTER(fd_problem), vp, vp, vp, vp, vp, vp, F,
                                         F, I, vp, vp, vp, vp, sz, vp]
        lib.fd_decode_sparse.restype = I
        lib.fd_combine.argtypes = [I, I, I, I, vp, vp, vp, vp, vp]
        lib.fd_combine.restype = I
        lib.fd_combine_strided.argtypes = [I, I, I, I, vp, sz, vp, sz, vp, vp, vp]
        lib.fd_combine_strided.restype = I
        P = ctypes.POINTER(fd_problem)
        lib.fd_append_int4.argtypes = [P, I, vp, ctypes.c_int64, vp, ctypes.c_int64, vp, vp, vp,
                                       vp, vp]
        lib.fd_append_int4.restype = I
        lib.fd_expand_int4.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.fd_expand_int4.restype = I
        lib.fd_decode_int4.argtypes = [P, vp, vp, vp, vp, vp, vp, F, I, vp, vp, vp, sz, vp]
        lib.fd_decode_int4.restype = I
        lib.fd_alloc_pages.argtypes = [I] * 5 + [vp] * 11
        lib.fd_alloc_pages.restype = I
        lib.fd_release_pages.argtypes = [I] * 4 + [vp] * 8
        lib.fd_release_pages.restype = I
        lib.fd_decode_static_workspace.argtypes = [ctypes.POINTER(fd_problem), vp, vp, vp, vp,
                                                   vp, F, I, vp, vp, vp]
        lib.fd_decode_static_workspace.restype = I
        lib.fd_selftest_device_timeout.argtypes = [ctypes.c_uint, vp]
        lib.fd_selftest_device_timeout.restype = I
        lib.fd_check_device_error.argtypes = [vp]
        lib.fd_check_device_error.restype = I
        lib.fd_status_string.argtypes = [I]
        lib.fd_status_string.restype = ctypes.c_char_p
        _lib = lib
    return _lib


_calls = None


class _CtypesCalls:
    """The calls of csrc/fdcall.c through ctypes."""

    def __init__(self, lib):
        self.lib = lib

    def append_int4(self, p, n, k, k_stride, v, v_stride, *rest):
        return self.lib.fd_append_int4(ctypes.byref(p), n, _ptr(k), k_stride, _ptr(v), v_stride,
                                       *map(_ptr, rest))

    def expand_int4(self, p, *rest):
        return self.lib.fd_expand_int4(ctypes.byref(p), *map(_ptr, rest))

    def decode_int4(self, p, q, k4, v4, params, seqlens, table, scale, splits, out, lse, workspace,
                    size, stream):
        return self.lib.fd_decode_int4(ctypes.byref(p), _ptr(q), _ptr(k4), _ptr(v4), _ptr(params),
                                       _ptr(seqlens), _ptr(table), scale, splits, _ptr(out),
                                       _ptr(lse), _ptr(workspace), max(size, 0), stream)

    def alloc_pages(self, *args):
        return self.lib.fd_alloc_pages(*args[:5], *map(_ptr, args[5:]))

    def release_pages(self, *args):
        return self.lib.fd_release_pages(*args[:4], *map(_ptr, args[4:]))


def _load_calls():
    """The calls whose time on the host counts (csrc/fdcall.c), on the library's
    functions; through ctypes where the module was not built."""
    global _calls
    if _calls is None:
        lib = load_library()
        if not os.path.exists(CALLS_PATH):
            _calls = _CtypesCalls(lib)
            return _calls
        from importlib import util
        spec = util.spec_from_file_location(__name__ + "._fdcall", CALLS_PATH)
        native = util.module_from_spec(spec)
        spec.loader.exec_module(native)
        native.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in
                      (lib.fd_append_int4, lib.fd_expand_int4, lib.fd_decode_int4,
                       lib.fd_alloc_pages, lib.fd_release_pages)))
        _calls = native
    return _calls


def _ptr(x) -> Optional[int]:
    """Device address of a torch tensor, an int address, or None."""
    if x is None or x.__class__ is int:
        return x or None
    return x.data_ptr() or None


_raw_stream = _device = None


def _forget_stream():
    global _raw_stream, _device
    _raw_stream = _device = None


# In a forked child torch has to say again whether CUDA may be used.
os.register_at_fork(after_in_child=_forget_stream)


def _stream(stream) -> Optional[int]:
    global _raw_stream, _device
    if stream is None:
        # The raw handle: building torch's Stream object takes 3.2 us, half of a
        # small call, and the checks of torch.cuda.current_device() are made once
        # in a process.
        if _raw_stream is None:
            import torch
            torch.cuda.current_device()
            _device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        return _raw_stream(_device()) or None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


# ---- one-to-one mirrors of the C entry points --------------------------------

def fd_status_string(status: int) -> str:
    return load_library().fd_status_string(int(status)).decode()


def fd_plan(B: int, Hq: int, Hkv: int, D: int, max_len: int, block_size: int = 0) -> int:
    return int(load_library().fd_plan(B, Hq, Hkv, D, max_len, block_size))


def fd_plan_sm(num_sms: int, B: int, Hq: int, Hkv: int, D: int, max_len: int,
               block_size: int = 0) -> int:
    return int(load_library().fd_plan_sm(num_sms, B, Hq, Hkv, D, max_len, block_size))


def fd_plan_seqlens(num_sms: int, B: int, Hq: int, Hkv: int, D: int, max_len: int,
                    block_size: int, seqlens) -> int:
    """Length-aware planner; `seqlens` is a host sequence of B ints (0 or a
    negative num_sms plans for the current device)."""
    import numpy as np
    sl = np.ascontiguousarray(np.asarray(seqlens, dtype=np.int32))
    return int(load_library().fd_plan_seqlens(num_sms, B, Hq, Hkv, D, max_len, block_size,
                                              sl.ctypes.data))


def fd_plan_problem(num_sms: int, prob: "fd_problem", seqlens=None) -> int:
    """Planner for a whole problem (element type included); `seqlens` is a
    host sequence of B ints or None (every sequence holds max_len)."""
    import numpy as np
    sl = None if seqlens is None else np.ascontiguousarray(np.asarray(seqlens, dtype=np.int32))
    return int(load_library().fd_plan_problem(num_sms, ctypes.byref(prob),
                                              None if sl is None else sl.ctypes.data))


def fd_split_chunk(max_len: int, num_splits: int) -> int:
    return int(load_library().fd_split_chunk(max_len, num_splits))


def fd_effective_splits(max_len: int, num_splits: int) -> int:
    return int(load_library().fd_effective_splits(max_len, num_splits))


def fd_workspace_bytes(B: int, Hq: int, D: int, num_splits: int) -> int:
    return int(load_library().fd_workspace_bytes(B, Hq, D, num_splits))


def fd_decode(problem: fd_problem, q, k_cache, v_cache, seqlens, block_table, scale: float,
              num_splits: int, out, lse, workspace, workspace_bytes: int, stream=None) -> int:
    """Call the C fd_decode; returns its status code.  Tensor arguments may be
    torch tensors, int device addresses or None; `stream` a torch stream, an
    int cudaStream_t or None (torch's current stream)."""
    f = _lib.fd_decode if _lib is not None else load_library().fd_decode
    return f(ctypes.byref(problem), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens),
             _ptr(block_table), scale, num_splits, _ptr(out), _ptr(lse), _ptr(workspace),
             workspace_bytes, _stream(stream))


def fd_decode_partial(problem: fd_problem, q, k_cache, v_cache, seqlens, block_table,
                      scale: float, num_splits: int, out_f32, lse, workspace,
                      workspace_bytes: int, stream=None) -> int:
    """Call the C fd_decode_partial: exact attention over this shard of the
    history as fp32 output and lse, for fd_combine.  Returns the status."""
    return int(load_library().fd_decode_partial(
        ctypes.byref(problem), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens),
        _ptr(block_table), scale, num_splits, _ptr(out_f32), _ptr(lse), _ptr(workspace),
        workspace_bytes, _stream(stream)))


def fd_quantize_keys(problem: fd_problem, k_cache, seqlens, k8, k8_scale, stream=None) -> int:
    """Call the C fd_quantize_keys: int8 key codes and per-64-token-block
    scales for fd_decode_sparse.  Returns the status."""
    return int(load_library().fd_quantize_keys(ctypes.byref(problem), _ptr(k_cache),
                                               _ptr(seqlens), _ptr(k8), _ptr(k8_scale),
                                               _stream(stream)))


def fd_decode_sparse(problem: fd_problem, q, k_cache, v_cache, k8, k8_scale, seqlens,
                     scale: float, delta: float, num_splits: int, out, lse, kept, workspace,
                     workspace_bytes: int, stream=None) -> int:
    """Call the C fd_decode_sparse: the low-bit scan and top-delta block
    selection, then exact attention over the kept blocks.  Returns the status."""
    return int(load_library().fd_decode_sparse(
        ctypes.byref(problem), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k8), _ptr(k8_scale),
        _ptr(seqlens), scale, delta, num_splits, _ptr(out), _ptr(lse), _ptr(kept),
        _ptr(workspace), workspace_bytes, _stream(stream)))


def fd_append_int4(problem: fd_problem, n_tokens: int, k_new, k_stride: int, v_new,
                   v_stride: int, slots, k4, v4, params, stream=None) -> int:
    """Call the C fd_append_int4: quantise new rows and write them at their
    slots.  Strides count elements from one token to the next.  Returns the
    status."""
    return (_calls or _load_calls()).append_int4(problem, n_tokens, k_new, k_stride, v_new,
                                                 v_stride, slots, k4, v4, params,
                                                 _stream(stream))


def fd_expand_int4(problem: fd_problem, k4, v4, params, seqlens, block_table, k_out, v_out,
                   stream=None) -> int:
    """Call the C fd_expand_int4: a 4-bit cache as a contiguous bf16 cache.
    Returns the status."""
    return (_calls or _load_calls()).expand_int4(problem, k4, v4, params, seqlens, block_table,
                                                 k_out, v_out, _stream(stream))


def fd_decode_int4(problem: fd_problem, q, k4, v4, params, seqlens, block_table, scale: float,
                   num_splits: int, out, lse, workspace, workspace_bytes: int,
                   stream=None) -> int:
    """Call the C fd_decode_int4: decode attention over a 4-bit cache.  Returns
    the status."""
    return (_calls or _load_calls()).decode_int4(problem, q, k4, v4, params, seqlens,
                                                 block_table, scale, num_splits, out, lse,
                                                 workspace, workspace_bytes, _stream(stream))


def fd_alloc_pages(B: int, block_size: int, max_blocks_per_seq: int, max_tokens: int,
                   num_pages: int, seqlens, new_lens, free_pages, free_count, block_table,
                   seqlens_out, cu_new, slots, positions, free_count_out, stream=None) -> int:
    """Call the C fd_alloc_pages: pages, slots and positions for the new tokens
    of a batch.  Returns the status."""
    return (_calls or _load_calls()).alloc_pages(B, block_size, max_blocks_per_seq, max_tokens,
                                                 num_pages, seqlens, new_lens, free_pages,
                                                 free_count, block_table, seqlens_out, cu_new,
                                                 slots, positions, free_count_out,
                                                 _stream(stream))


def fd_release_pages(B: int, block_size: int, max_blocks_per_seq: int, num_pages: int, seqlens,
                     done, block_table, free_pages, free_count, seqlens_out, free_count_out,
                     stream=None) -> int:
    """Call the C fd_release_pages: pages of finished requests back to the
    pool.  Returns the status."""
    return (_calls or _load_calls()).release_pages(B, block_size, max_blocks_per_seq, num_pages,
                                                   seqlens, done, block_table, free_pages,
                                                   free_count, seqlens_out, free_count_out,
                                                   _stream(stream))


def fd_combine(R: int, B: int, Hq: int, D: int, part_o, part_lse, out, lse, stream=None) -> int:
    """Call the C fd_combine: merge R partials [R, B, Hq, D] / [R, B, Hq].
    Returns the status."""
    return int(load_library().fd_combine(R, B, Hq, D, _ptr(part_o), _ptr(part_lse), _ptr(out),
                                         _ptr(lse), _stream(stream)))


def fd_combine_strided(R: int, B: int, Hq: int, D: int, part_o, o_stride: int, part_lse,
                       lse_stride: int, out, lse, stream=None) -> int:
    """Call the C fd_combine_strided: merge R partials placed at strides
    (counted in floats), e.g. R packed per-rank buffers gathered end to end.
    Returns the status."""
    return int(load_library().fd_combine_strided(R, B, Hq, D, _ptr(part_o), o_stride,
                                                 _ptr(part_lse), lse_stride, _ptr(out),
                                                 _ptr(lse), _stream(stream)))


def fd_decode_static_workspace(problem: fd_problem, q, k_cache, v_cache, seqlens, block_table,
                               scale: float, num_splits: int, out, lse, stream=None) -> int:
    """Call the C fd_decode_static_workspace: fd_decode for callers that cannot
    allocate device memory; its scratch is the library's static device array
    of FD_STATIC_WORKSPACE_BYTES.  Returns the status code.

    When q is a torch tensor, the tensors are checked as decode() checks them
    (dtype, shape, contiguity, device, and a contiguous cache's row count
    against problem.max_len) and against the problem's sizes, and a mismatch
    raises ValueError before anything is launched: the C ABI sees only
    addresses, and a strided or padded view would be read as dense memory."""
    if q is not None and q.__class__ is not int:
        if q.dim() == 3 and k_cache.dim() == 4:
            _check_problem_sizes(problem, q, k_cache)
        _check_decode_args(q, k_cache, v_cache, seqlens, block_table, problem.kv_layout,
                           problem.max_len if problem.block_size == 0 else None, out, lse, None)
    return int(load_library().fd_decode_static_workspace(
        ctypes.byref(problem), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens),
        _ptr(block_table), ctypes.c_float(scale), int(num_splits), _ptr(out), _ptr(lse),
        _stream(stream)))


def fd_check_device_error(stream=None) -> int:
    return int(load_library().fd_check_device_error(_stream(stream)))


def fd_selftest_device_timeout(limit_us: int, stream=None) -> int:
    return int(load_library().fd_selftest_device_timeout(int(limit_us), _stream(stream)))


# ---- convenience wrapper -----------------------------------------------------

def make_problem(B, Hq, Hkv, D, max_len, block_size=0, num_blocks=0, max_blocks_per_seq=0,
                 kv_layout=FD_LAYOUT_HND, kv_dtype=FD_KV_BF16, k_scale=1.0, v_scale=1.0,
                 fp8_mma=0):
    return fd_problem(B, Hq, Hkv, D, max_len, block_size, num_blocks, max_blocks_per_seq,
                      kv_layout, kv_dtype, k_scale, v_scale, fp8_mma)


def _check(t, name, dtypes, shape=None):
    """Checks a tensor argument of decode() before its address is passed on:
    the kernels read and write dense row-major buffers of the stated shapes."""
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")


def _check_decode_args(q, k_cache, v_cache, seqlens, block_table, kv_layout, max_len, out, lse,
                       workspace):
    """Shape, dtype, layout and device checks of decode(); raises ValueError.
    The device checks come last."""
    import torch
    cache_types = [torch.bfloat16, torch.uint8]
    if hasattr(torch, "float8_e4m3fn"):
        cache_types.append(torch.float8_e4m3fn)
    if q.dim() != 3:
        raise ValueError(f"q: expected [B, Hq, D], got shape {tuple(q.shape)}")
    B, Hq, D = q.shape
    _check(q, "q", [torch.bfloat16])
    if kv_layout not in (FD_LAYOUT_HND, FD_LAYOUT_NHD):
        raise ValueError(f"kv_layout: {kv_layout}, expected FD_LAYOUT_HND or FD_LAYOUT_NHD")
    if k_cache.dim() != 4:
        raise ValueError(f"k_cache: expected 4 dimensions, got shape {tuple(k_cache.shape)}")
    _check(k_cache, "k_cache", cache_types)
    _check(v_cache, "v_cache", [k_cache.dtype], k_cache.shape)
    if k_cache.shape[3] != D:
        raise ValueError(f"k_cache: head dim {k_cache.shape[3]}, q has {D}")
    if block_table is None:
        if k_cache.shape[0] != B:
            raise ValueError(f"k_cache: {k_cache.shape[0]} sequences, q has {B}")
        rows = k_cache.shape[2] if kv_layout == FD_LAYOUT_HND else k_cache.shape[1]
        if max_len is not None and max_len != rows:
            raise ValueError(f"max_len {max_len}: a contiguous cache holds {rows} rows per "
                             "sequence and KV head, and max_len must equal it")
    else:
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError(f"block_table: expected [B={B}, max_blocks], got "
                             f"{tuple(block_table.shape)}")
        _check(block_table, "block_table", [torch.int32])
    if seqlens is not None:
        _check(seqlens, "seqlens", [torch.int32], (B,))
    if out is not None:
        _check(out, "out", [torch.bfloat16], (B, Hq, D))
    if lse is not None:
        _check(lse, "lse", [torch.float32], (B, Hq))
    if workspace is not None:
        _check(workspace, "workspace", None)
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("seqlens", seqlens),
                    ("block_table", block_table), ("out", out), ("lse", lse),
                    ("workspace", workspace)):
        if t is not None and (not t.is_cuda or t.device != q.device):
            raise ValueError(f"{name} is on {t.device}; every tensor must be on q's CUDA device "
                             f"({q.device})")


def _check_problem_sizes(problem: fd_problem, q, k_cache):
    """The problem's B, Hq, D, Hkv (and page size) must describe the tensors."""
    B, Hq, D = q.shape
    if (problem.B, problem.Hq, problem.D) != (B, Hq, D):
        raise ValueError(f"problem (B, Hq, D) = {(problem.B, problem.Hq, problem.D)}, q has "
                         f"{(B, Hq, D)}")
    hnd = problem.kv_layout == FD_LAYOUT_HND
    Hkv = k_cache.shape[1] if hnd else k_cache.shape[2]
    if problem.Hkv != Hkv:
        raise ValueError(f"problem Hkv = {problem.Hkv}, the cache holds {Hkv} KV heads")
    if problem.block_size:
        bs = k_cache.shape[2] if hnd else k_cache.shape[1]
        if (problem.block_size, problem.num_blocks) != (bs, k_cache.shape[0]):
            raise ValueError(f"problem pages {(problem.num_blocks, problem.block_size)}, the "
                             f"cache holds {(k_cache.shape[0], bs)}")


def decode(q, k_cache, v_cache, seqlens=None, block_table=None, *, max_len: Optional[int] = None,
           kv_layout: int = FD_LAYOUT_HND, scale: Optional[float] = None,
           num_splits: Optional[int] = None, out=None, lse=None, workspace=None, stream=None,
           k_scale: float = 1.0, v_scale: float = 1.0, fp8_mma: int = FD_FP8_MMA_SYNC):
    """Decode attention on torch CUDA tensors.

    q [B, Hq, D] bf16.  Caches: bf16, or E4M3 codes (torch.uint8 or
    torch.float8_e4m3fn, D = 128) whose real values are k_scale * code and
    v_scale * code.  FD_LAYOUT_HND contiguous [B, Hkv, max_len, D] or paged
    [num_blocks, Hkv, block_size, D]; FD_LAYOUT_NHD contiguous
    [B, max_len, Hkv, D] or paged [num_blocks, block_size, Hkv, D].  Paged
    caches come with block_table [B, max_blocks] int32.  seqlens [B] int32
    or None.  Returns (out [B, Hq, D] bf16, lse [B, Hq] fp32).  num_splits
    defaults to fd_plan_problem's choice.  fp8_mma picks the tensor-core path
    of an fp8 cache (FD_FP8_MMA_SYNC or FD_FP8_MMA_TCGEN05).  Raises
    ValueError for tensors of the wrong dtype, shape or device, or not
    contiguous, before anything is launched, and FdError for a failing
    status."""
    import torch
    _check_decode_args(q, k_cache, v_cache, seqlens, block_table, kv_layout, max_len, out, lse,
                       workspace)
    B, Hq, D = q.shape
    block_size = 0
    fp8 = k_cache.element_size() == 1
    kv_dtype = FD_KV_FP8_E4M3 if fp8 else FD_KV_BF16
    if block_table is None:
        if kv_layout == FD_LAYOUT_HND:
            _, Hkv, L, _ = k_cache.shape
        else:
            _, L, Hkv, _ = k_cache.shape
        max_len = L if max_len is None else max_len
        prob = make_problem(B, Hq, Hkv, D, max_len, kv_layout=kv_layout, kv_dtype=kv_dtype,
                            k_scale=k_scale, v_scale=v_scale, fp8_mma=fp8_mma)
    else:
        if kv_layout == FD_LAYOUT_HND:
            nb, Hkv, bs, _ = k_cache.shape
        else:
            nb, bs, Hkv, _ = k_cache.shape
        block_size = bs
        mbps = block_table.shape[1]
        max_len = mbps * bs if max_len is None else max_len
        prob = make_problem(B, Hq, Hkv, D, max_len, bs, nb, mbps, kv_layout, kv_dtype, k_scale,
                            v_scale, fp8_mma)
    if scale is None:
        scale = 1.0 / (D ** 0.5)
    if num_splits is None:
        num_splits = fd_plan_problem(0, prob)
        if num_splits < 0:
            raise FdError(num_splits, "fd_plan_problem")
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    wbytes = fd_workspace_bytes(B, Hq, D, num_splits)
    if workspace is None and wbytes:
        workspace = torch.empty(wbytes // 4, dtype=torch.float32, device=q.device)
    have = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = fd_decode(prob, q, k_cache, v_cache, seqlens, block_table, scale, num_splits, out, lse,
                   workspace, have, stream)
    if st != FD_OK:
        raise FdError(st, "fd_decode")
    return out, lse


# ---- a KV cache held in 4 bits, and the pages of a paged cache -----------------

def _launch_stream(stream, device):
    """The torch stream to run on: the one given, or the device's current one."""
    import torch
    if stream is None:
        return torch.cuda.current_stream(device)
    if isinstance(stream, int):
        return torch.cuda.ExternalStream(stream, device=device)
    return stream


def _check_cuda(named):
    """Every tensor on one CUDA device (the first one's).  Comes last."""
    first = next(t for _, t in named if t is not None)
    for name, t in named:
        if t is not None and (not t.is_cuda or t.device != first.device):
            raise ValueError(f"{name} is on {t.device}; every tensor must be on one CUDA device "
                             f"({first.device})")
    return first.device


def _check_int4_cache(k4, v4, params, kv_layout):
    """(planes, Hkv, rows, D) of a 4-bit cache; raises ValueError."""
    import torch
    if kv_layout not in (FD_LAYOUT_HND, FD_LAYOUT_NHD):
        raise ValueError(f"kv_layout: {kv_layout}, expected FD_LAYOUT_HND or FD_LAYOUT_NHD")
    if k4.dim() != 4:
        raise ValueError(f"k4: expected 4 dimensions, got shape {tuple(k4.shape)}")
    _check(k4, "k4", [torch.uint8])
    _check(v4, "v4", [torch.uint8], k4.shape)
    _check(params, "params", [torch.bfloat16], tuple(k4.shape[:3]) + (8,))
    planes, a, b, half = k4.shape
    return (planes, a, b, 2 * half) if kv_layout == FD_LAYOUT_HND else (planes, b, a, 2 * half)


def _int4_problem(shape, B, Hq, block_table, max_len, kv_layout):
    planes, Hkv, rows, D = shape
    if block_table is None:
        if planes != B:
            raise ValueError(f"k4: {planes} sequences, expected {B}")
        if max_len is not None and max_len != rows:
            raise ValueError(f"max_len {max_len}: a contiguous cache holds {rows} rows per "
                             "sequence and KV head, and max_len must equal it")
        return make_problem(B, Hq, Hkv, D, rows, kv_layout=kv_layout, kv_dtype=FD_KV_INT4)
    _check_table(block_table, B)
    blocks = block_table.shape[1]
    return make_problem(B, Hq, Hkv, D, blocks * rows if max_len is None else max_len, rows, planes,
                        blocks, kv_layout, FD_KV_INT4)


def _check_table(block_table, B):
    import torch
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError(f"block_table: expected [B={B}, max_blocks], got "
                         f"{tuple(block_table.shape)}")
    _check(block_table, "block_table", [torch.int32])


def _raise(status, what):
    if status != FD_OK:
        raise FdError(status, what)


def append_int4(k_new, v_new, slots, k4, v4, params, *, kv_layout: int = FD_LAYOUT_HND,
                stream=None):
    """Quantise K and V rows and write them into a 4-bit cache, in place.

    k_new, v_new [T, Hkv, D] bf16: the last two dimensions dense, tokens at any
    stride that is a multiple of 8 (slices of a fused projection's output).
    slots [T] int64: page * block_size + row in a paged cache [num_blocks, ...],
    b * max_len + t in a contiguous one; a token with a negative slot, or one
    outside the cache, is skipped.  k4, v4 uint8 and params bf16 as in
    include/fd.h.  Raises ValueError for tensors that do not fit and FdError
    for a failing status."""
    import torch
    shape = planes, Hkv, rows, D = _check_int4_cache(k4, v4, params, kv_layout)
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name}: dtype {t.dtype}, expected {torch.bfloat16}")
        if t.dim() != 3 or tuple(t.shape[1:]) != (Hkv, D):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [T, {Hkv}, {D}]")
        if t.shape[0] and (t.stride(2) != 1 or (Hkv > 1 and t.stride(1) != D)):
            raise ValueError(f"{name}: the heads of a token must be dense")
    T = k_new.shape[0]
    if v_new.shape[0] != T:
        raise ValueError(f"v_new: {v_new.shape[0]} tokens, k_new has {T}")
    _check(slots, "slots", [torch.int64], (T,))
    strides = [t.stride(0) if T > 1 else Hkv * D for t in (k_new, v_new)]
    for name, s in zip(("k_new", "v_new"), strides):
        if s < Hkv * D or s % 8:
            raise ValueError(f"{name}: token stride {s}, expected a multiple of 8 of at least "
                             f"{Hkv * D}")
    device = _check_cuda((("k4", k4), ("v4", v4), ("params", params), ("k_new", k_new),
                          ("v_new", v_new), ("slots", slots)))
    # The place of a slot depends on the rows of a plane alone; as pages the
    # planes may be more than a batch's 65,535.
    if rows in (8, 16, 32, 64, 128, 256):
        prob = make_problem(1, Hkv, Hkv, D, rows, rows, planes, 1, kv_layout, FD_KV_INT4)
    else:
        prob = make_problem(planes, Hkv, Hkv, D, rows, kv_layout=kv_layout, kv_dtype=FD_KV_INT4)
    if T:
        with torch.cuda.device(device):
            _raise(fd_append_int4(prob, T, k_new, strides[0], v_new, strides[1], slots, k4, v4,
                                  params, _launch_stream(stream, device)), "fd_append_int4")


def expand_int4(k4, v4, params, seqlens=None, block_table=None, *, max_len: Optional[int] = None,
                kv_layout: int = FD_LAYOUT_HND, k_out=None, v_out=None, stream=None):
    """A 4-bit cache as a contiguous bf16 cache (k, v), [B, Hkv, max_len, D] or
    (FD_LAYOUT_NHD) [B, max_len, Hkv, D].

    Rows at or past a sequence's length are left as they were in k_out and
    v_out, and are zeros when these are allocated here.  Arguments as
    decode_int4's."""
    import torch
    shape = _check_int4_cache(k4, v4, params, kv_layout)
    B = shape[0] if block_table is None else block_table.shape[0]
    prob = _int4_problem(shape, B, shape[1], block_table, max_len, kv_layout)
    hnd = kv_layout == FD_LAYOUT_HND
    want = (B, prob.Hkv, prob.max_len, prob.D) if hnd else (B, prob.max_len, prob.Hkv, prob.D)
    if seqlens is not None:
        _check(seqlens, "seqlens", [torch.int32], (B,))
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is not None:
            _check(t, name, [torch.bfloat16], want)
    device = _check_cuda((("k4", k4), ("v4", v4), ("params", params), ("seqlens", seqlens),
                          ("block_table", block_table), ("k_out", k_out), ("v_out", v_out)))
    s = _launch_stream(stream, device)
    with torch.cuda.device(device), torch.cuda.stream(s):
        k_out = torch.zeros(want, dtype=torch.bfloat16, device=device) if k_out is None else k_out
        v_out = torch.zeros(want, dtype=torch.bfloat16, device=device) if v_out is None else v_out
        if prob.max_len:
            _raise(fd_expand_int4(prob, k4, v4, params, seqlens, block_table, k_out, v_out, s),
                   "fd_expand_int4")
    return k_out, v_out


def decode_int4(q, k4, v4, params, seqlens=None, block_table=None, *,
                max_len: Optional[int] = None, kv_layout: int = FD_LAYOUT_HND,
                scale: Optional[float] = None, num_splits: Optional[int] = None, out=None,
                lse=None, workspace=None, stream=None):
    """Decode attention over a 4-bit cache on torch CUDA tensors.

    q [B, Hq, D] bf16.  k4, v4 uint8 [.., D / 2] and params bf16 [.., 8] in the
    orders of decode()'s caches (include/fd.h has the format; append_int4 fills
    it).  Paged caches come with block_table [B, max_blocks] int32.  seqlens
    [B] int32 or None.  Returns (out [B, Hq, D] bf16, lse [B, Hq] fp32).
    num_splits (1: one cluster per row; above, the batch is dealt to the SMs) defaults
    to fd_plan_problem's choice for sequences of max_len tokens: with a block table of
    many more places than the sequences hold, pass fd_plan_problem's for their lengths,
    or 1 for few short ones.  Raises ValueError for tensors of the wrong dtype,
    shape or device, or not contiguous, before anything is launched, and FdError for
    a failing status."""
    import torch
    if q.dim() != 3:
        raise ValueError(f"q: expected [B, Hq, D], got shape {tuple(q.shape)}")
    B, Hq, D = q.shape
    _check(q, "q", [torch.bfloat16])
    shape = _check_int4_cache(k4, v4, params, kv_layout)
    if shape[3] != D:
        raise ValueError(f"k4: head dim {shape[3]}, q has {D}")
    prob = _int4_problem(shape, B, Hq, block_table, max_len, kv_layout)
    if seqlens is not None:
        _check(seqlens, "seqlens", [torch.int32], (B,))
    if out is not None:
        _check(out, "out", [torch.bfloat16], (B, Hq, D))
    if lse is not None:
        _check(lse, "lse", [torch.float32], (B, Hq))
    if workspace is not None:
        _check(workspace, "workspace", None)
    device = _check_cuda((("q", q), ("k4", k4), ("v4", v4), ("params", params),
                          ("seqlens", seqlens), ("block_table", block_table), ("out", out),
                          ("lse", lse), ("workspace", workspace)))
    scale = 1.0 / (D ** 0.5) if scale is None else scale
    s = _launch_stream(stream, device)
    # Temporaries belong to the stream that the kernels run on.
    with torch.cuda.device(device), torch.cuda.stream(s):
        if num_splits is None:
            num_splits = fd_plan_problem(0, prob)
            if num_splits < 0:
                raise FdError(num_splits, "fd_plan_problem")
        if out is None:
            out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=device)
        if lse is None:
            lse = torch.empty((B, Hq), dtype=torch.float32, device=device)
        need = fd_workspace_bytes(B, Hq, D, num_splits)
        if workspace is None and need:
            workspace = torch.empty(need // 4, dtype=torch.float32, device=device)
        have = workspace.numel() * workspace.element_size() if workspace is not None else 0
        _raise(fd_decode_int4(prob, q, k4, v4, params, seqlens, block_table, scale, num_splits,
                              out, lse, workspace, have, s), "fd_decode_int4")
    return out, lse


def _check_pool(seqlens, block_table, free_pages, free_count, seqlens_out, free_count_out):
    import torch
    if seqlens.dim() != 1:
        raise ValueError(f"seqlens: expected [B], got shape {tuple(seqlens.shape)}")
    B = seqlens.shape[0]
    _check(seqlens, "seqlens", [torch.int32])
    _check_table(block_table, B)
    if free_pages.dim() != 1:
        raise ValueError(f"free_pages: expected [num_pages], got shape {tuple(free_pages.shape)}")
    _check(free_pages, "free_pages", [torch.int32])
    _check(free_count, "free_count", [torch.int32], (1,))
    if seqlens_out is not None:
        _check(seqlens_out, "seqlens_out", [torch.int32], (B,))
    if free_count_out is not None:
        _check(free_count_out, "free_count_out", [torch.int32], (1,))
    return B


def alloc_pages(seqlens, new_lens, block_table, free_pages, free_count, *, block_size: int,
                max_tokens: int, seqlens_out=None, free_count_out=None, cu_new=None, slots=None,
                positions=None, stream=None):
    """Pages and slots for the new tokens of a batch, on the device.

    seqlens, new_lens [B] int32; block_table [B, max_blocks] int32, whose new
    entries are written in place; free_pages [num_pages] int32 with the free
    ones in its first free_count[0] places.  max_tokens is the capacity of
    slots and positions (a host number of at least the new tokens, so that the
    call can be captured).  seqlens_out and free_count_out default to new
    tensors; pass seqlens and free_count to update these in place.  Returns
    (slots [max_tokens] int64, positions [max_tokens] int32, cu_new [B + 1]
    int32, seqlens_out, free_count_out); see fd_alloc_pages in include/fd.h."""
    import torch
    B = _check_pool(seqlens, block_table, free_pages, free_count, seqlens_out, free_count_out)
    _check(new_lens, "new_lens", [torch.int32], (B,))
    if max_tokens < 0:
        raise ValueError(f"max_tokens: {max_tokens}, expected >= 0")
    for name, t, dtype, n in (("cu_new", cu_new, torch.int32, B + 1),
                              ("slots", slots, torch.int64, max_tokens),
                              ("positions", positions, torch.int32, max_tokens)):
        if t is not None:
            _check(t, name, [dtype], (n,))
    device = _check_cuda((("seqlens", seqlens), ("new_lens", new_lens),
                          ("block_table", block_table), ("free_pages", free_pages),
                          ("free_count", free_count), ("seqlens_out", seqlens_out),
                          ("free_count_out", free_count_out), ("cu_new", cu_new),
                          ("slots", slots), ("positions", positions)))
    s = _launch_stream(stream, device)
    with torch.cuda.device(device), torch.cuda.stream(s):
        new = dict(device=device)
        seqlens_out = torch.empty(B, dtype=torch.int32, **new) if seqlens_out is None else seqlens_out
        free_count_out = (torch.empty(1, dtype=torch.int32, **new) if free_count_out is None
                          else free_count_out)
        cu_new = torch.empty(B + 1, dtype=torch.int32, **new) if cu_new is None else cu_new
        slots = torch.empty(max_tokens, dtype=torch.int64, **new) if slots is None else slots
        positions = (torch.empty(max_tokens, dtype=torch.int32, **new) if positions is None
                     else positions)
        _raise(fd_alloc_pages(B, block_size, block_table.shape[1], max_tokens,
                              free_pages.shape[0], seqlens, new_lens, free_pages, free_count,
                              block_table, seqlens_out, cu_new, slots, positions, free_count_out,
                              s), "fd_alloc_pages")
    return slots, positions, cu_new, seqlens_out, free_count_out


def release_pages(seqlens, done, block_table, free_pages, free_count, *, block_size: int,
                  seqlens_out=None, free_count_out=None, stream=None):
    """Gives the pages of finished requests (done [B] uint8 or bool, not 0) back
    to free_pages, in place.  Returns (seqlens_out, free_count_out), new tensors
    unless given; pass seqlens and free_count to update these in place."""
    import torch
    B = _check_pool(seqlens, block_table, free_pages, free_count, seqlens_out, free_count_out)
    _check(done, "done", [torch.uint8, torch.bool], (B,))
    device = _check_cuda((("seqlens", seqlens), ("done", done), ("block_table", block_table),
                          ("free_pages", free_pages), ("free_count", free_count),
                          ("seqlens_out", seqlens_out), ("free_count_out", free_count_out)))
    s = _launch_stream(stream, device)
    with torch.cuda.device(device), torch.cuda.stream(s):
        seqlens_out = (torch.empty(B, dtype=torch.int32, device=device) if seqlens_out is None
                       else seqlens_out)
        free_count_out = (torch.empty(1, dtype=torch.int32, device=device)
                          if free_count_out is None else free_count_out)
        _raise(fd_release_pages(B, block_size, block_table.shape[1], free_pages.shape[0], seqlens,
                                done, block_table, free_pages, free_count, seqlens_out,
                                free_count_out, s), "fd_release_pages")
    return seqlens_out, free_count_out
