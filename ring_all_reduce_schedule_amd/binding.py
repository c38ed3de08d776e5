"""Thin ctypes binding of libra.so: the C ABI of include/ra.h under the same names.

Only argument marshalling happens here: torch tensors are turned into device
pointers, element counts, dtype codes and the current HIP stream, and nonzero
status codes are raised as ``RaError``.  Every step of the all-reduce runs in the
library's HIP kernels.  If libra.so has not been built, the first call raises:
there is no fallback path.
"""

import array
import ctypes
import os
import re

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libra.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "ra.h")

RA_OK, RA_ERR_INVALID_ARG, RA_ERR_UNSUPPORTED, RA_ERR_ALIAS = 0, 1, 2, 3
RA_ERR_MISALIGNED, RA_ERR_HIP, RA_ERR_TIMEOUT = 4, 5, 6
RA_INT32, RA_FLOAT32, RA_BFLOAT16, RA_FLOAT16, RA_FLOAT64, RA_INT64 = 0, 1, 2, 3, 4, 5
RA_FLOAT8_E4M3 = 6
RA_SUM, RA_MAX, RA_AVG = 0, 1, 2
RA_MAX_RANKS = 64
RA_FLAG_FORCE_TIMEOUT = 1
RA_FLAG_WIDE_ACCUM = 2
RA_FLAG_STRESS = 4
RA_FLAG_RENEW_COUNTERS = 8
RA_FLAG_PHASES = 16
RA_FLAG_NO_PHASES = 32
OPS = {"sum": RA_SUM, "max": RA_MAX, "avg": RA_AVG}

ALGOS = {"default": -1, "ring_step": 0, "ring_pipelined": 1, "ring_bidir": 2,
         "fused": 3, "tree": 4, "ring_channels": 5, "auto": 6, "hier": 7,
         "hier_fused": 8, "ring_pipelined_flags": 9}
ALGO_NAMES = {v: k for k, v in ALGOS.items()}
DTYPE_NAMES = {"int32": RA_INT32, "float32": RA_FLOAT32, "bfloat16": RA_BFLOAT16,
               "float16": RA_FLOAT16, "float64": RA_FLOAT64, "int64": RA_INT64}


class RaError(RuntimeError):
    """A libra.so call returned a nonzero status."""

    def __init__(self, code, name, message):
        super().__init__(f"{name}: {message}")
        self.code, self.name, self.message = code, name, message


class ra_options(ctypes.Structure):
    _fields_ = [("slice_elems", ctypes.c_int64),
                ("timeout_us", ctypes.c_int64),
                ("grid", ctypes.c_int32),
                ("flags", ctypes.c_uint32),
                ("step_ts", ctypes.c_void_p),
                ("channels", ctypes.c_int32),
                ("group", ctypes.c_int32),
                ("link_alpha_us", ctypes.c_double),
                ("link_GBps", ctypes.c_double)]


_lib = None
_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_f32 = ctypes.c_float

_SIGNATURES = {
    "ra_chunk_bounds": (_int, [_i64, _int, ctypes.POINTER(ctypes.c_int64)]),
    "ra_reduce_scatter": (_int, [ctypes.POINTER(_vp), _int, _i64, _int, _int, _vp]),
    "ra_all_gather": (_int, [ctypes.POINTER(_vp), _int, _i64, _int, _vp]),
    "ra_allreduce": (_int, [ctypes.POINTER(_vp), _int, _i64, _int, _int, _vp]),
    "ra_allreduce_ex": (_int, [ctypes.POINTER(_vp), _int, _i64, _int, _int, _int,
                               ctypes.POINTER(ra_options), _vp]),
    "ra_allreduce_noalloc": (_int, [ctypes.POINTER(_vp), _int, _i64, _int, _int, _int,
                                    ctypes.POINTER(ra_options), _vp]),
    "ra_reduce_scatter_ex": (_int, [ctypes.POINTER(_vp), _int, _i64, _int, _int, _int,
                                    ctypes.POINTER(ra_options), _vp]),
    "ra_all_gather_ex": (_int, [ctypes.POINTER(_vp), _int, _i64, _int, _int,
                                ctypes.POINTER(ra_options), _vp]),
    "ra_stream_status": (_int, [_vp]),
    "ra_select_algo": (_int, [_int, _i64, _int, ctypes.POINTER(ra_options),
                              ctypes.POINTER(_int)]),
    "ra_status_string": (ctypes.c_char_p, [_int]),
    "ra_last_error": (ctypes.c_char_p, []),
    "ra_wallclock_hz": (_int, [ctypes.POINTER(ctypes.c_int64)]),
    "ra_stream_copy": (_int, [_vp, _vp, _i64, _vp]),
    "ra_stream_copy_resident": (_int, [_vp, _vp, _i64, _int, _vp]),
    "ra_allreduce_rmsnorm": (_int, [_vp, _int, _i64, _i64, _int, _vp, _vp, _int, _vp, _f32, _vp,
                                    _int, _int, _vp, _int, _vp, _vp]),
    "ra_allreduce_rmsnorm_backward": (_int, [_vp, _int, _i64, _i64, _int, _vp, _int, _vp, _vp, _vp,
                                             _vp, _vp, _int, _vp, _vp, _i64, _vp]),
    "ra_allreduce_rmsnorm_backward_workspace": (_int, [_i64, _i64, ctypes.POINTER(_i64)]),
    "ra_cross_entropy": (_int, [_vp, _int, _i64, _i64, _i64, _int, _vp, _int, _vp, _vp, _vp, _vp,
                                _f32, _vp, _i64, _vp]),
    "ra_cross_entropy_workspace": (_int, [_i64, _i64, _int, ctypes.POINTER(_i64)]),
    "ra_cross_entropy_backward": (_int, [_vp, _int, _i64, _i64, _i64, _int, _vp, _int, _vp, _vp,
                                         _vp, _f32, _vp]),
    "ra_token_logprobs": (_int, [_vp, _int, _i64, _i64, _i64, _int, _f32, _vp, _int, _vp, _vp, _vp,
                                 _int, _vp, _vp, _vp, _i64, _vp]),
    "ra_token_logprobs_workspace": (_int, [_i64, _i64, _int, _int, ctypes.POINTER(_i64)]),
    "ra_token_logprobs_backward": (_int, [_vp, _int, _i64, _i64, _i64, _int, _f32, _vp, _int, _vp,
                                          _vp, _vp, _vp, _vp, _vp]),
    "ra_grad_norm": (_int, [_vp, _vp, _vp, _i64, _f32, _vp, _vp, _i64, _vp]),
    "ra_grad_norm_workspace": (_int, [_i64, ctypes.POINTER(_i64)]),
    "ra_grad_clip": (_int, [_vp, _vp, _vp, _i64, _i64, _f32, _f32, _vp, _vp, _vp, _vp, _i64, _vp]),
    "ra_allreduce_clip": (_int, [_vp, _int, _i64, _int, _int, _f32, _f32, _vp, _int, _vp, _vp, _i64,
                                 _vp]),
    "ra_allreduce_clip_workspace": (_int, [_i64, ctypes.POINTER(_i64)]),
    "ra_embedding": (_int, [_vp, _int, _i64, _i64, _int, _vp, _int, _i64, _f32, _vp, _int, _vp]),
    "ra_embedding_backward": (_int, [_vp, _i64, _i64, _int, _vp, _int, _f32, _vp, _int, _i64, _int,
                                     _int, _vp, _i64, _vp]),
    "ra_embedding_backward_workspace": (_int, [_i64, _i64, _i64, ctypes.POINTER(_i64)]),
}


def lib():
    """The loaded libra.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} not found: build it with "
                "`python -m ring_all_reduce_schedule_amd.build` (there is no fallback)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype, fn.argtypes = res, args
        _lib = handle
    return _lib


def header_symbols():
    """Function names declared in include/ra.h."""
    with open(HEADER_PATH) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:int|const char\*)\s+(ra_\w+)\s*\(", text, re.M)))


def ra_status_string(code):
    return lib().ra_status_string(int(code)).decode()


def ra_last_error():
    return lib().ra_last_error().decode()


def _check(code):
    if code != RA_OK:
        raise RaError(code, ra_status_string(code), ra_last_error())
    return code


# ---------------------------------------------------------------- marshalling

_torch_module = None
_codes = {}
_get_device = _is_contiguous = _data_ptr = _numel = None    # torch.Tensor's


def _torch():
    global _torch_module, _get_device, _is_contiguous, _data_ptr, _numel
    if _torch_module is None:
        import torch
        _codes.update({torch.int32: RA_INT32, torch.float32: RA_FLOAT32,
                       torch.bfloat16: RA_BFLOAT16, torch.float16: RA_FLOAT16,
                       torch.float64: RA_FLOAT64, torch.int64: RA_INT64})
        _get_device, _is_contiguous = torch.Tensor.get_device, torch.Tensor.is_contiguous
        _data_ptr, _numel = torch.Tensor.data_ptr, torch.Tensor.numel
        _torch_module = torch
    return _torch_module


def dtype_code(t):
    code = _codes.get(t.dtype)
    if code is None:
        _torch()
        code = _codes.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} "
                        "(int32, int64, float16, bfloat16, float32, float64)")
    return code


def _stream_handle(stream, device):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _buffer_code(t):
    """dtype_code, or that of 8-bit outputs."""
    if t.dtype is _torch().float8_e4m3fn:
        return RA_FLOAT8_E4M3
    return dtype_code(t)


def _marshal_list(tensors, code_of=dtype_code):
    """(pointer array, p, n, dtype code, device) for a sequence of rank tensors,
    checked: same dtype, length and device, contiguous, on a GPU.  The pointer
    array is a ctypes view of an array.array, which is several times cheaper to
    build than a ctypes array from a list."""
    if len(tensors) == 0:
        raise ValueError("need at least one rank buffer")
    t0 = tensors[0]
    if not t0.is_cuda:
        raise ValueError("rank buffers must be device tensors")
    dt, n, dev = t0.dtype, t0.numel(), t0.get_device()
    for t in tensors:
        if t.dtype is not dt or t.numel() != n or t.get_device() != dev:
            raise ValueError("rank buffers must share dtype, length and device")
        if not t.is_contiguous():
            raise ValueError("rank buffers must be contiguous")
    code = code_of(t0)
    table = array.array("Q", [t.data_ptr() for t in tensors])
    ptrs = (ctypes.c_void_p * len(tensors)).from_buffer(table)
    return ptrs, len(tensors), n, code, t0.device


class RankBuffers:
    """p rank tensors checked and marshalled once, for repeated calls.

    Every entry point accepts one in place of a list of tensors that all have the same
    length (the row operators save its checks for the buffers they fold, and check their
    other lists anew; their 8-bit outputs may be one, which the other calls refuse).  A
    list is checked and turned into a pointer table on every call, which costs about
    0.8 us of host time per rank (about 50 us at p = 64, more than a fused
    all-reduce of 1 MiB per rank takes on the GPU); this object does it once.
    It holds references to the tensors, so their memory stays allocated while it
    lives.  The tensors must not be resized or re-pointed (``resize_``,
    ``set_``) meanwhile: the table holds the addresses they had when it was made,
    and a call raises if the first rank's address or length has changed."""

    __slots__ = ("tensors", "ptrs", "p", "n", "dtype", "device", "shapes", "_first")

    def __init__(self, tensors):
        self.tensors = tuple(tensors)
        marshalled = _marshal_list(self.tensors, _buffer_code)
        self.ptrs, self.p, self.n, self.dtype, self.device = marshalled
        self.shapes = tuple({t.shape for t in self.tensors})
        self._first = (self.tensors[0].data_ptr(), self.n)

    def __len__(self):
        return self.p


def _marshal(tensors):
    """(pointer array, p, n, dtype code, device) for a list of rank tensors or a
    RankBuffers."""
    if isinstance(tensors, RankBuffers):
        t0 = tensors.tensors[0]
        if (t0.data_ptr(), t0.numel()) != tensors._first:
            raise ValueError("a rank tensor of this RankBuffers was resized or re-pointed")
        return tensors.ptrs, tensors.p, tensors.n, tensors.dtype, tensors.device
    return _marshal_list(tensors)


def _options(slice_elems=0, timeout_us=0, grid=0, flags=0, step_ts=None, channels=0,
             link_alpha_us=0.0, link_GBps=0.0, wide=False, group=0):
    o = ra_options()
    o.slice_elems = int(slice_elems)
    o.timeout_us = int(timeout_us)
    o.grid = int(grid)
    o.flags = int(flags) | (RA_FLAG_WIDE_ACCUM if wide else 0)
    o.step_ts = None if step_ts is None else int(step_ts.data_ptr())
    o.channels = int(channels)
    o.group = int(group)
    o.link_alpha_us = float(link_alpha_us)
    o.link_GBps = float(link_GBps)
    return o


def _algo(algo):
    return ALGOS[algo] if isinstance(algo, str) else int(algo)


def _op(op):
    if isinstance(op, str):
        return OPS.get(op, -1)
    return int(op)


# ---------------------------------------------------------------- entry points

def ra_chunk_bounds(n, p):
    """List of p + 1 chunk starts (host only)."""
    starts = (ctypes.c_int64 * (max(p, 0) + 1))()
    _check(lib().ra_chunk_bounds(int(n), int(p), starts))
    return list(starts)


def ra_allreduce(tensors, op="sum", stream=None):
    ptrs, p, n, dt, dev = _marshal(tensors)
    return _check(lib().ra_allreduce(ptrs, p, n, dt, _op(op), _stream_handle(stream, dev)))


def ra_allreduce_ex(tensors, algo="default", op="sum", stream=None, **opts):
    ptrs, p, n, dt, dev = _marshal(tensors)
    o = _options(**opts)
    return _check(lib().ra_allreduce_ex(ptrs, p, n, dt, _op(op), _algo(algo), ctypes.byref(o),
                                        _stream_handle(stream, dev)))


def ra_allreduce_noalloc(tensors, algo="default", op="sum", stream=None, **opts):
    ptrs, p, n, dt, dev = _marshal(tensors)
    o = _options(**opts)
    return _check(lib().ra_allreduce_noalloc(ptrs, p, n, dt, _op(op), _algo(algo), ctypes.byref(o),
                                             _stream_handle(stream, dev)))


def ra_reduce_scatter(tensors, op="sum", stream=None):
    ptrs, p, n, dt, dev = _marshal(tensors)
    return _check(lib().ra_reduce_scatter(ptrs, p, n, dt, _op(op), _stream_handle(stream, dev)))


def ra_reduce_scatter_ex(tensors, algo="default", op="sum", stream=None, **opts):
    ptrs, p, n, dt, dev = _marshal(tensors)
    o = _options(**opts)
    return _check(lib().ra_reduce_scatter_ex(ptrs, p, n, dt, _op(op), _algo(algo),
                                             ctypes.byref(o), _stream_handle(stream, dev)))


def ra_all_gather(tensors, stream=None):
    ptrs, p, n, dt, dev = _marshal(tensors)
    return _check(lib().ra_all_gather(ptrs, p, n, dt, _stream_handle(stream, dev)))


def ra_all_gather_ex(tensors, algo="default", stream=None, **opts):
    ptrs, p, n, dt, dev = _marshal(tensors)
    o = _options(**opts)
    return _check(lib().ra_all_gather_ex(ptrs, p, n, dt, _algo(algo), ctypes.byref(o),
                                         _stream_handle(stream, dev)))


def ra_select_algo(p, n, dtype, **opts):
    """Name of the algorithm RA_ALGO_AUTO would run (host only)."""
    code = DTYPE_NAMES[dtype] if isinstance(dtype, str) else int(dtype)
    o = _options(**opts)
    out = ctypes.c_int(-1)
    _check(lib().ra_select_algo(int(p), int(n), code, ctypes.byref(o), ctypes.byref(out)))
    return ALGO_NAMES[out.value]


def ra_stream_status(stream=None, device=None):
    torch = _torch()
    dev = device if device is not None else torch.cuda.current_device()
    return _check(lib().ra_stream_status(_stream_handle(stream, dev)))


def ra_wallclock_hz():
    hz = ctypes.c_int64()
    _check(lib().ra_wallclock_hz(ctypes.byref(hz)))
    return hz.value


def ra_stream_copy(dst, src, stream=None):
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() < nbytes:
        raise ValueError("dst smaller than src")
    return _check(lib().ra_stream_copy(ctypes.c_void_p(dst.data_ptr()),
                                       ctypes.c_void_p(src.data_ptr()), nbytes,
                                       _stream_handle(stream, src.device)))


def ra_stream_copy_resident(dst, src, grid=0, stream=None):
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() < nbytes:
        raise ValueError("dst smaller than src")
    return _check(lib().ra_stream_copy_resident(ctypes.c_void_p(dst.data_ptr()),
                                                ctypes.c_void_p(src.data_ptr()), nbytes,
                                                int(grid), _stream_handle(stream, src.device)))


# ---------------------------------------------------------------- row operators
# Arrays of rows are tensors [..., hidden] whose other dimensions together are the
# tokens, or flat ones, whose rows lie one behind the other; of values for each token
# only the number counts.  The calls write into the tensors they are given and return
# None; scratch memory is taken from torch's allocator on the call's stream, so that a
# captured graph owns its own.

def _refuse(what, t, numel, dtype, dev, hidden=None):
    if t.get_device() != dev:
        raise ValueError(f"{what} must be on the device of the other tensors")
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if t.numel() != numel:
        raise ValueError(f"{what} has {t.numel()} elements, expected {numel}")
    if hidden is not None and _other_rows(t.shape, hidden):
        raise ValueError(f"{what} of shape {tuple(t.shape)} are no rows of {hidden}")
    raise ValueError(f"{what} must be contiguous")


def _other_rows(shape, hidden):
    """Whether a tensor of this shape has rows, but not of `hidden` elements."""
    return len(shape) > 1 and shape[-1] != hidden


# Small calls take less time on the GPU than these checks do on the host, so the
# helpers below make one pass over their tensors and look up nothing twice.

def _table(what, tensors, numel, dtype, dev):
    """array.array of the tensors' addresses, each checked."""
    for t in tensors:
        if (t.dtype is not dtype or t.numel() != numel or t.get_device() != dev
                or not t.is_contiguous()):
            _refuse(what, t, numel, dtype, dev)
    return array.array("Q", [t.data_ptr() for t in tensors])


def _row_table(what, tensors, shape, numel, hidden, dtype, dev):
    """The same for arrays of rows; `shape` is one that is `numel` elements in such rows, and
    the tensors of a call mostly have it."""
    for t in tensors:
        if (t.dtype is not dtype or _get_device(t) != dev or not _is_contiguous(t)
                or t.shape != shape and (t.numel() != numel or _other_rows(t.shape, hidden))):
            _refuse(what, t, numel, dtype, dev, hidden)
    return array.array("Q", list(map(_data_ptr, tensors)))


def _cut_table(what, tensors, dim, other):
    """(table, total): the same for matrices that are the ranks' pieces of a length, cut along
    `dim` as ra_chunk_bounds cuts it; `other` is their other dimension."""
    t0 = tensors[0]
    dtype, dev = t0.dtype, t0.get_device()
    sizes = []
    for t in tensors:
        shape = t.shape
        if len(shape) != 2 or shape[1 - dim] != other:
            raise ValueError(f"{what} must be matrices with {other} in dimension {1 - dim}")
        if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
            _refuse(what, t, t.numel(), dtype, dev)
        sizes.append(shape[dim])
    total, p = sum(sizes), len(sizes)
    base, extra = divmod(total, p)
    if sizes != [base + 1] * extra + [base] * (p - extra):
        raise ValueError(f"{what}: {sizes} is not how ra_chunk_bounds cuts {total} over {p} ranks")
    return array.array("Q", [t.data_ptr() for t in tensors]), total


def _address(table):
    """Where a pointer table starts; the caller keeps the table while the call reads it."""
    return table.buffer_info()[0] if table else None


def _arg(what, t, numel, dtype, dev):
    """Address of one tensor (None: NULL), checked."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != numel or t.get_device() != dev or not t.is_contiguous():
        _refuse(what, t, numel, dtype, dev)
    return t.data_ptr()


def _row_arg(what, t, shape, numel, hidden, dtype, dev):
    """The same for an array of rows."""
    if t is None:
        return None
    if (t.dtype is not dtype or _get_device(t) != dev or not _is_contiguous(t)
            or t.shape != shape and (t.numel() != numel or _other_rows(t.shape, hidden))):
        _refuse(what, t, numel, dtype, dev, hidden)
    return _data_ptr(t)


def _list(tensors):
    """The tensors of a list or a RankBuffers."""
    return tensors.tensors if isinstance(tensors, RankBuffers) else tensors


def _first(what, tensors):
    if len(tensors) == 0:
        raise ValueError(f"need at least one tensor in {what}")
    t = tensors[0]
    if not t.is_cuda:
        raise ValueError(f"{what} must be device tensors")
    return t


def _run_on(dev, stream, function, args):
    """function(*args, stream handle) with the tensors' device current."""
    core = _torch_module._C
    handle = core._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if core._cuda_getDevice() == dev:
        return _check(function(*args, handle))
    with _torch_module.cuda.device(dev):
        return _check(function(*args, handle))


def _workspace(workspace, like, stream, size_call, *sizes):
    """(tensor to keep alive, address, bytes): the caller's tensor, or one allocated for the
    stream that the call runs on."""
    torch = _torch()
    if workspace is not None:
        if workspace.get_device() != like.get_device() or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous, on the device of the other tensors")
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    n = ctypes.c_int64()
    _check(size_call(*sizes, ctypes.byref(n)))
    if n.value == 0:
        return None, None, 0
    if stream is None:
        workspace = torch.empty(n.value, dtype=torch.uint8, device=like.device)
    else:
        with torch.cuda.stream(stream):
            workspace = torch.empty(n.value, dtype=torch.uint8, device=like.device)
    return workspace, workspace.data_ptr(), n.value


def ra_allreduce_rmsnorm_backward_workspace(tokens, hidden):
    """Bytes of workspace (host only)."""
    n = ctypes.c_int64()
    _check(lib().ra_allreduce_rmsnorm_backward_workspace(int(tokens), int(hidden), ctypes.byref(n)))
    return n.value


def ra_cross_entropy_workspace(tokens, vocab, p):
    """Bytes of workspace (host only)."""
    n = ctypes.c_int64()
    _check(lib().ra_cross_entropy_workspace(int(tokens), int(vocab), int(p), ctypes.byref(n)))
    return n.value


def ra_embedding_backward_workspace(tokens, vocab, hidden):
    """Bytes of workspace (host only)."""
    n = ctypes.c_int64()
    _check(lib().ra_embedding_backward_workspace(int(tokens), int(vocab), int(hidden),
                                                 ctypes.byref(n)))
    return n.value


def ra_token_logprobs_workspace(tokens, vocab, p, top):
    """Bytes of workspace (host only)."""
    n = ctypes.c_int64()
    _check(lib().ra_token_logprobs_workspace(int(tokens), int(vocab), int(p), int(top),
                                             ctypes.byref(n)))
    return n.value


def ra_grad_norm_workspace(n):
    """Bytes of workspace for n tensors (host only)."""
    size = ctypes.c_int64()
    _check(lib().ra_grad_norm_workspace(int(n), ctypes.byref(size)))
    return size.value


def ra_allreduce_clip_workspace(n):
    """Bytes of workspace for n elements (host only)."""
    size = ctypes.c_int64()
    _check(lib().ra_allreduce_clip_workspace(int(n), ctypes.byref(size)))
    return size.value


def _rows(bufs, weight):
    """(first tensor, its shape, pointer table, address, p, dtype code, tokens, hidden, device
    index)."""
    hidden = weight.numel()
    if isinstance(bufs, RankBuffers):
        at, p, n, code, _ = _marshal(bufs)
        b0, table = bufs.tensors[0], at
        shape, dev = b0.shape, b0.get_device()
        others = [s for s in bufs.shapes if _other_rows(s, hidden)]
        shape = others[0] if others else shape
    else:
        b0 = _first("rank buffers", bufs)
        code, shape, n, dev = dtype_code(b0), b0.shape, b0.numel(), b0.get_device()
        table = _row_table("rank buffers", bufs, shape, n, hidden, b0.dtype, dev)
        p, at = len(bufs), _address(table)
    if hidden == 0 or n % hidden or len(shape) > 1 and shape[-1] != hidden:
        raise ValueError(f"rank buffers of shape {tuple(shape)} are no rows of {hidden}")
    return b0, shape, table, at, p, code, n // hidden, hidden, dev


def ra_allreduce_rmsnorm(bufs, weight, eps, outs, residual=None, residual_out=None, scales=None,
                         group=0, rstd=None, stream=None):
    """outs = RMS norm of (residual + the sum of bufs) times weight; see include/ra.h.

    bufs, outs: lists of tensors.  outs of float8_e4m3fn take scales: as many float32
    tensors, one value a token or a group of columns."""
    b0, shape, table, at, p, code, tokens, hidden, dev = _rows(bufs, weight)
    torch = _torch_module
    n, dtype, f32, outs = tokens * hidden, b0.dtype, torch.float32, _list(outs)
    if len(outs) == 0:
        raise ValueError("need at least one tensor in outs")
    out_type = outs[0].dtype
    f8 = out_type is torch.float8_e4m3fn
    out_table = _row_table("outs", outs, shape, n, hidden, out_type, dev)
    res = residual if residual is not None else residual_out
    res_type = dtype if res is None else res.dtype
    scale_table, scales = None, _list(scales)
    if f8:
        if scales is None or len(scales) != len(outs):
            raise ValueError("8-bit outputs need as many scales")
        groups = -(-hidden // group) if group > 0 else 1
        scale_table = _table("scales", scales, tokens * groups, f32, dev)
    args = (at, p, tokens, hidden, code,
            _row_arg("residual", residual, shape, n, hidden, res_type, dev),
            _row_arg("residual_out", residual_out, shape, n, hidden, res_type, dev),
            code if res_type is dtype else dtype_code(res),
            _arg("weight", weight, hidden, dtype, dev), eps, _address(out_table), len(out_table),
            RA_FLOAT8_E4M3 if f8 else code if out_type is dtype else dtype_code(outs[0]),
            _address(scale_table), int(group),
            _arg("rstd", rstd, tokens, f32, dev))
    _run_on(dev, stream, lib().ra_allreduce_rmsnorm, args)


def ra_allreduce_rmsnorm_backward(dys, h, rstd, weight, dh, dh_in=None, dxs=(), dweight=None,
                                  workspace=None, stream=None):
    """Gradient of ra_allreduce_rmsnorm from the ranks' parts dys of the gradient of its
    output; see include/ra.h."""
    d0, shape, table, at, p, code, tokens, hidden, dev = _rows(dys, weight)
    n, dtype, h_type, f32, dxs = tokens * hidden, d0.dtype, h.dtype, _torch_module.float32, _list(dxs)
    dx_table = _row_table("dxs", dxs, shape, n, hidden, dtype, dev)
    keep, wp, wn = None, None, 0
    if dweight is not None:
        keep, wp, wn = _workspace(workspace, d0, stream,
                                  lib().ra_allreduce_rmsnorm_backward_workspace, tokens, hidden)
    args = (at, p, tokens, hidden, code, _row_arg("h", h, shape, n, hidden, h_type, dev),
            code if h_type is dtype else dtype_code(h), _arg("rstd", rstd, tokens, f32, dev),
            _arg("weight", weight, hidden, dtype, dev),
            _row_arg("dh_in", dh_in, shape, n, hidden, h_type, dev),
            _row_arg("dh", dh, shape, n, hidden, h_type, dev),
            _address(dx_table), len(dx_table), _arg("dweight", dweight, hidden, f32, dev), wp, wn)
    _run_on(dev, stream, lib().ra_allreduce_rmsnorm_backward, args)


def _index(what, t, tokens, dev):
    """(address, dtype code) of token numbers."""
    torch = _torch()
    dtype = t.dtype
    if dtype is not torch.int64 and dtype is not torch.int32:
        raise TypeError(f"{what} must be int32 or int64, not {dtype}")
    return _arg(what, t, tokens, dtype, dev), _codes[dtype]


def _xent_args(logits, targets, grads, what="targets"):
    """(first tensor, tables to keep, targets' arguments, tokens, vocab, device index)."""
    logits, grads = _list(logits), _list(grads)
    x0 = _first("logits", logits)
    dev = x0.get_device()
    tokens = x0.shape[0] if targets is None else targets.numel()
    table, vocab = _cut_table("logits", logits, 1, tokens)
    grad_table = None
    if grads is not None:
        if len(grads) != len(logits):
            raise ValueError("grads must be as many as the logits")
        g0 = _first("grads", grads)
        if g0.dtype is not x0.dtype or g0.get_device() != dev:
            _refuse("grads", g0, g0.numel(), x0.dtype, dev)
        grad_table, columns = _cut_table("grads", grads, 1, tokens)
        if columns != vocab:
            raise ValueError("grads must have the logits' shapes")
    goal = (None, RA_INT64) if targets is None else _index(what, targets, tokens, dev)
    return x0, (table, grad_table), goal, tokens, vocab, dev


def ra_cross_entropy(logits, targets, loss=None, lse=None, grads=None, dloss=None, grad_scale=1.0,
                     valid=None, workspace=None, stream=None):
    """Softmax cross entropy over a vocabulary cut over the ranks, with its gradient where
    grads are given (they may be the logits themselves); see include/ra.h.

    logits: a list of [tokens, columns of the rank] tensors."""
    f32 = _torch().float32
    x0, (table, grad_table), goal, tokens, vocab, dev = _xent_args(logits, targets, grads)
    keep, wp, wn = _workspace(workspace, x0, stream, lib().ra_cross_entropy_workspace,
                              tokens, vocab, len(table))
    args = (_address(table), len(table), tokens, vocab, vocab if valid is None else int(valid),
            dtype_code(x0), *goal, _arg("loss", loss, tokens, f32, dev),
            _arg("lse", lse, tokens, f32, dev), _address(grad_table),
            _arg("dloss", dloss, tokens, f32, dev), grad_scale, wp, wn)
    _run_on(dev, stream, lib().ra_cross_entropy, args)


def ra_cross_entropy_backward(logits, targets, lse, grads, dloss=None, grad_scale=1.0, valid=None,
                              stream=None):
    """The gradient of ra_cross_entropy from the logits and lse; see include/ra.h."""
    f32 = _torch().float32
    x0, (table, grad_table), goal, tokens, vocab, dev = _xent_args(logits, targets, grads)
    args = (_address(table), len(table), tokens, vocab, vocab if valid is None else int(valid),
            dtype_code(x0), *goal, _arg("lse", lse, tokens, f32, dev), _address(grad_table),
            _arg("dloss", dloss, tokens, f32, dev), grad_scale)
    _run_on(dev, stream, lib().ra_cross_entropy_backward, args)


def ra_token_logprobs(logits, ids=None, logprob=None, entropy=None, lse=None, top_ids=None,
                      top_logprobs=None, scale=1.0, valid=None, workspace=None, stream=None):
    """Log probabilities of given tokens, entropy and the best alternatives over a vocabulary
    cut over the ranks; see include/ra.h.

    logits: a list of [tokens, columns of the rank] tensors.  top_ids, top_logprobs:
    [tokens, k] tensors for the k best columns; top_ids of the type of ids (without ids:
    int32 or int64)."""
    torch = _torch()
    f32 = torch.float32
    x0, (table, _), (id_at, id_code), tokens, vocab, dev = _xent_args(logits, ids, None, "ids")
    top, id_type = 0, torch.int64 if ids is None else ids.dtype
    for t in (top_ids, top_logprobs):
        if t is None:
            continue
        if t.dim() != 2 or t.shape[0] != tokens or top and t.shape[1] != top:
            raise ValueError(f"top_ids and top_logprobs must be [{tokens}, k], with the same k")
        top = t.shape[1]
        if top == 0:
            raise ValueError("top_ids and top_logprobs must have a column")
    if top_ids is not None and ids is None:
        id_type = top_ids.dtype
        id_code = _index("top_ids", top_ids, tokens * top, dev)[1]
    keep, wp, wn = _workspace(workspace, x0, stream, lib().ra_token_logprobs_workspace,
                              tokens, vocab, len(table), top)
    args = (_address(table), len(table), tokens, vocab, vocab if valid is None else int(valid),
            dtype_code(x0), scale, id_at, id_code, _arg("logprob", logprob, tokens, f32, dev),
            _arg("entropy", entropy, tokens, f32, dev), _arg("lse", lse, tokens, f32, dev), top,
            _arg("top_ids", top_ids, tokens * top, id_type, dev),
            _arg("top_logprobs", top_logprobs, tokens * top, f32, dev), wp, wn)
    _run_on(dev, stream, lib().ra_token_logprobs, args)


def ra_token_logprobs_backward(logits, ids, lse, grads, dlogprob=None, entropy=None, dentropy=None,
                               scale=1.0, valid=None, stream=None):
    """The gradient of ra_token_logprobs' logprob and entropy, from the lse and entropy that it
    left; see include/ra.h.  grads may be the logits themselves."""
    f32 = _torch().float32
    x0, (table, grad_table), goal, tokens, vocab, dev = _xent_args(logits, ids, grads, "ids")
    args = (_address(table), len(table), tokens, vocab, vocab if valid is None else int(valid),
            dtype_code(x0), scale, *goal, _arg("lse", lse, tokens, f32, dev),
            _arg("entropy", entropy, tokens, f32, dev), _arg("dlogprob", dlogprob, tokens, f32, dev),
            _arg("dentropy", dentropy, tokens, f32, dev), _address(grad_table))
    _run_on(dev, stream, lib().ra_token_logprobs_backward, args)


def ra_embedding(tables, ids, outs, scale=1.0, stream=None):
    """outs = scale times the rows of a table cut over the ranks; see include/ra.h.

    tables: a list of [rows of the rank, hidden] tensors."""
    tables, outs = _list(tables), _list(outs)
    t0 = _first("tables", tables)
    hidden, dev, tokens = t0.shape[-1], t0.get_device(), ids.numel()
    table, vocab = _cut_table("tables", tables, 0, hidden)
    _first("outs", outs)
    code, dtype, shape = dtype_code(t0), t0.dtype, (*ids.shape, hidden)
    out_table = _row_table("outs", outs, shape, tokens * hidden, hidden, dtype, dev)
    args = (_address(table), len(table), vocab, hidden, code,
            *_index("ids", ids, tokens, dev), tokens, scale, _address(out_table), len(out_table))
    _run_on(dev, stream, lib().ra_embedding, args)


def ra_embedding_backward(dy, ids, dtables, scale=1.0, accumulate=False, workspace=None, stream=None):
    """dtables = (or with accumulate +=) scale times the sums of dy's rows by token; see
    include/ra.h."""
    dtables = _list(dtables)
    t0 = _first("dtables", dtables)
    hidden, dev, tokens = t0.shape[-1], t0.get_device(), ids.numel()
    table, vocab = _cut_table("dtables", dtables, 0, hidden)
    keep, wp, wn = _workspace(workspace, t0, stream, lib().ra_embedding_backward_workspace,
                              tokens, vocab, hidden)
    args = (_row_arg("dy", dy, (*ids.shape, hidden), tokens * hidden, hidden, dy.dtype, dev),
            tokens, hidden, dtype_code(dy), *_index("ids", ids, tokens, dev), scale,
            _address(table), len(table), vocab, dtype_code(t0), 1 if accumulate else 0, wp, wn)
    _run_on(dev, stream, lib().ra_embedding_backward, args)


# ---------------------------------------------------------------- gradients

class TensorList:
    """Tensors of any sizes and types, checked and marshalled once, for repeated calls of
    ra_grad_norm and ra_grad_clip, which accept one in place of a list of tensors or a
    RankBuffers.  It holds references to the tensors, which must not be resized or re-pointed
    (``resize_``, ``set_``, ``.data =``) meanwhile: the table holds the addresses they had when it
    was made, and a call raises if any tensor's address or length has changed.  Looking at them
    costs about 0.09 us of host time a tensor, checking and marshalling a list 0.3: the norm of 75
    tensors takes 17 us of it a call with this and 33 with a list.  (A loop whose gradients are
    new tensors in every step has to make a new TensorList, or to pass the list.)"""

    __slots__ = ("tensors", "device", "_ptrs", "_counts", "_codes", "_addresses", "_lengths")

    def __init__(self, tensors):
        self.tensors = tuple(_list(tensors))
        _torch()
        dev = _get_device(self.tensors[0]) if self.tensors else -1
        for t in self.tensors:
            if not t.is_cuda or _get_device(t) != dev:
                raise ValueError("tensors must be on one device")
            if not _is_contiguous(t):
                raise ValueError("tensors must be contiguous")
        self.device = dev
        self._addresses, self._lengths = self._now()
        self._ptrs = array.array("Q", self._addresses)
        self._counts = array.array("q", self._lengths)
        self._codes = array.array("i", [dtype_code(t) for t in self.tensors])

    def _now(self):
        """(addresses, lengths) as the tensors have them."""
        return list(map(_data_ptr, self.tensors)), list(map(_numel, self.tensors))

    def __len__(self):
        return len(self.tensors)


def _marshalled(tensors):
    if not isinstance(tensors, TensorList):
        return TensorList(tensors)
    if tensors._now() != (tensors._addresses, tensors._lengths):
        raise ValueError("a tensor of this TensorList was resized or re-pointed")
    return tensors


def _tensor_list(tensors, norm):
    """(TensorList, address of norm, device index)."""
    t = _marshalled(tensors)
    if not norm.is_cuda:
        raise ValueError("norm must be a device tensor")
    dev = norm.get_device()
    if t.device not in (dev, -1):
        raise ValueError("tensors must be on the device of norm")
    return t, _arg("norm", norm, 1, _torch().float32, dev), dev


def ra_grad_norm(tensors, norm, scale=1.0, workspace=None, stream=None):
    """norm = scale times the 2-norm over all elements of a list of tensors (or a TensorList);
    see include/ra.h.  norm: one float32."""
    t, to, dev = _tensor_list(tensors, norm)
    keep, wp, wn = _workspace(workspace, norm, stream, lib().ra_grad_norm_workspace, len(t))
    args = (_address(t._ptrs), _address(t._counts), _address(t._codes), len(t), scale, to, wp, wn)
    _run_on(dev, stream, lib().ra_grad_norm, args)


def ra_grad_clip(tensors, max_norm, norm, outs=None, counted=None, scale=1.0, workspace=None,
                 stream=None):
    """Scales tensors (a list or a TensorList; in place, or into outs) so that their norm is at
    most max_norm; see include/ra.h.  norm, one float32, gets the norm before.  counted: how many
    of the tensors, from the first on, the norm is of (None: all)."""
    t, to, dev = _tensor_list(tensors, norm)
    n, o = len(t), None
    if outs is not None:
        o = _marshalled(outs)
        if o._counts != t._counts or o.device != t.device:
            raise ValueError("outs must be tensors of the same sizes, on the same device")
    keep, wp, wn = _workspace(workspace, norm, stream, lib().ra_grad_norm_workspace, n)
    args = (_address(t._ptrs), _address(t._counts), _address(t._codes), n,
            n if counted is None else int(counted), max_norm, scale,
            None if o is None else _address(o._ptrs), None if o is None else _address(o._codes), to, wp, wn)
    _run_on(dev, stream, lib().ra_grad_clip, args)


def ra_allreduce_clip(bufs, max_norm, norm, outs=None, op="avg", scale=1.0, workspace=None,
                      stream=None):
    """The ranks' buffers averaged (op "avg") or added ("sum"), scaled so that their norm is at
    most max_norm, into outs (None: in place); see include/ra.h, also for gradients in more buffers
    than one a rank.  norm, one float32, gets the norm before."""
    ptrs, p, n, code, _ = _marshal(bufs)
    b0 = _list(bufs)[0]
    dev = b0.get_device()
    table, n_out = ptrs, p
    if outs is not None:
        outs = _list(outs)
        _first("outs", outs)
        table, n_out = _table("outs", outs, n, b0.dtype, dev), len(outs)
    keep, wp, wn = _workspace(workspace, norm, stream, lib().ra_allreduce_clip_workspace, n)
    args = (ptrs, p, n, code, _op(op), max_norm, scale,
            ptrs if outs is None else _address(table), n_out,
            _arg("norm", norm, 1, _torch().float32, dev), wp, wn)
    _run_on(dev, stream, lib().ra_allreduce_clip, args)
