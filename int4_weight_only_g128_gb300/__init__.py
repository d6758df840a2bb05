"""Python binding of libw4g128, the int4-g128 weight-streaming GEMV for GB300.

Argument marshalling only: every function forwards to the C entry point of
the same name in ``include/*.h``; every step of the computation runs in the
library's CUDA kernels.  Tensors are passed as device pointers taken from
``torch.Tensor.data_ptr()`` (plain integers are accepted as raw pointers), and
the stream defaults to torch's current CUDA stream.  There is no CPU fallback:
if the library cannot be built or loaded, the first call raises.
"""
import ctypes
import os

__all__ = [
    "W4G128Error", "lib", "lib_debug", "exported_symbols",
    "w4g128_status_string", "w4g128_packed_bytes", "w4g128_pack", "w4g128_unpack", "w4g128_quantize",
    "w4g128_workspace_bytes", "w4g128_gemv", "w4g128_gemm_verify",
    "w4g128_decode_step_workspace_bytes", "w4g128_decode_step", "w4g128_verify_step", "w4g128_workspace_status",
    "w4g128_probe_read", "w4g128_probe_copy", "w4g128_probe_sink_bytes", "w4g128_gemv_noalloc",
    "w4g128_noalloc_status", "w4g128_selftest_wait", "w4g128_gemm_add_rmsnorm", "w4g128_decode_step_host",
    "w4g128_schedule", "DecodeStep",
    "w4g128_sample", "SampleArgs", "SampleStep", "MAX_SAMPLE_ROWS", "MAX_VOCAB",
    "w4g128_attend", "w4g128_attend_workspace_bytes", "AttendArgs", "AttendStep", "MAX_SEQUENCES", "ERR_CACHE",
    "w4g128_moe", "w4g128_moe_workspace_bytes", "MoEArgs", "MoEStep", "MAX_EXPERTS", "MAX_TOP_K",
    "MAX_M", "MAX_MATRICES", "SELFTEST_WS_BYTES", "SCHEDULE_FIELDS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_INCLUDE = os.path.join(os.path.dirname(_HERE), "include")
MAX_M = 16          # W4G128_MAX_M
MAX_MATRICES = 512  # W4G128_MAX_MATRICES
SELFTEST_WS_BYTES = 512  # W4G128_SELFTEST_WS_BYTES
SCHEDULE_FIELDS = 8  # W4G128_SCHEDULE_FIELDS
MAX_SAMPLE_ROWS = 4096  # W4G128_MAX_SAMPLE_ROWS
MAX_VOCAB = 524160      # W4G128_MAX_VOCAB
MAX_SEQUENCES = 1024    # W4G128_MAX_SEQUENCES
ERR_CACHE = 9           # W4G128_ERR_CACHE
MAX_EXPERTS = 512       # W4G128_MAX_EXPERTS
MAX_TOP_K = 16          # W4G128_MAX_TOP_K

_lib = None


class W4G128Error(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {status} ({w4g128_status_string(status)})")


class _Matrix(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("K", ctypes.c_int), ("N", ctypes.c_int)]


def exported_symbols(headers=None):
    """Names of every function the named public headers of include/ declare
    (by default all but those of w4g128_ops.h, the operators around the weight
    stream)."""
    if headers is None:
        headers = sorted(fn for fn in os.listdir(_INCLUDE) if fn.endswith(".h") and fn != "w4g128_ops.h")
    names = []
    for fn in headers:
        with open(os.path.join(_INCLUDE, fn)) as f:
            for line in f:
                line = line.strip()
                if line.startswith("W4G128_API") and "(" in line:
                    names.append(line.split("(")[0].split()[-1].lstrip("*"))
    return names


_lib_debug = None


def lib():
    """Load libw4g128.so (building it in-tree if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    from . import build as _build
    path = _build.LIB
    if not os.path.exists(path):
        _build.build()
    _lib = _declare(ctypes.CDLL(path))
    return _lib


def lib_debug():
    """Load libw4g128_debug.so, the range-checked build of the same sources
    (W4G128_DEBUG: every global access of the weight stream derived from the
    schedule is checked, a failure recorded as W4G128_ERR_INTERNAL in the status
    word); for tests.
    Call its functions directly (the wrappers below use lib())."""
    global _lib_debug
    if _lib_debug is not None:
        return _lib_debug
    from . import build as _build
    path = _build.LIB_DEBUG
    if not os.path.exists(path):
        _build.build(debug=True)
    _lib_debug = _declare(ctypes.CDLL(path))
    return _lib_debug


def _declare(L):
    """Argument and result types of every entry point."""
    p, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.w4g128_status_string.restype = ctypes.c_char_p
    L.w4g128_status_string.argtypes = [i]
    L.w4g128_packed_bytes.restype = sz
    L.w4g128_packed_bytes.argtypes = [i, i]
    L.w4g128_pack.restype = i
    L.w4g128_pack.argtypes = [p, p, p, i, i, p, p]
    L.w4g128_unpack.restype = i
    L.w4g128_unpack.argtypes = [p, i, i, p, p, p, p]
    L.w4g128_quantize.restype = i
    L.w4g128_quantize.argtypes = [p, i, i, i, p, p, p, p]
    L.w4g128_workspace_bytes.restype = sz
    L.w4g128_workspace_bytes.argtypes = [i, i, i]
    L.w4g128_gemv.restype = i
    L.w4g128_gemv.argtypes = [p, p, p, i, i, p, sz, p]
    L.w4g128_gemm_verify.restype = i
    L.w4g128_gemm_verify.argtypes = [p, p, p, i, i, i, p, sz, p]
    L.w4g128_decode_step_workspace_bytes.restype = sz
    L.w4g128_decode_step_workspace_bytes.argtypes = [ctypes.POINTER(_Matrix), i, i]
    L.w4g128_decode_step.restype = i
    L.w4g128_decode_step.argtypes = [ctypes.POINTER(_Matrix), i, i, p, sz, p]
    L.w4g128_workspace_status.restype = i
    L.w4g128_workspace_status.argtypes = [p, ctypes.POINTER(ctypes.c_int), p]
    L.w4g128_probe_read.restype = i
    L.w4g128_probe_read.argtypes = [p, sz, p, p]
    L.w4g128_probe_copy.restype = i
    L.w4g128_probe_copy.argtypes = [p, p, sz, p]
    L.w4g128_probe_sink_bytes.restype = sz
    L.w4g128_probe_sink_bytes.argtypes = []
    L.w4g128_decode_step_host.restype = i
    L.w4g128_decode_step_host.argtypes = [ctypes.POINTER(_Matrix), i, i, p, p, sz, p, p, sz, p, sz, p]
    L.w4g128_verify_step.restype = i
    L.w4g128_verify_step.argtypes = [ctypes.POINTER(_Matrix), i, i, p, sz, p]
    L.w4g128_gemv_noalloc.restype = i
    L.w4g128_gemv_noalloc.argtypes = [p, p, p, i, i, p]
    L.w4g128_noalloc_status.restype = i
    L.w4g128_noalloc_status.argtypes = [ctypes.POINTER(ctypes.c_int), p]
    L.w4g128_selftest_wait.restype = i
    L.w4g128_selftest_wait.argtypes = [p, sz, ctypes.c_ulonglong, i, p]
    L.w4g128_gemm_add_rmsnorm.restype = i
    L.w4g128_gemm_add_rmsnorm.argtypes = [p, p, p, p, ctypes.c_float, p, p, i, i, i, i, p, sz, p]
    L.w4g128_schedule.restype = i
    L.w4g128_schedule.argtypes = [ctypes.POINTER(_Matrix), i, i, ctypes.POINTER(ctypes.c_longlong), i]
    L.w4g128_sample.restype = i
    L.w4g128_sample.argtypes = [ctypes.POINTER(SampleArgs), p]
    L.w4g128_attend_workspace_bytes.restype = sz
    L.w4g128_attend_workspace_bytes.argtypes = [ctypes.POINTER(AttendArgs)]
    L.w4g128_attend.restype = i
    L.w4g128_attend.argtypes = [ctypes.POINTER(AttendArgs), p, sz, p]
    L.w4g128_moe_workspace_bytes.restype = sz
    L.w4g128_moe_workspace_bytes.argtypes = [ctypes.POINTER(MoEArgs)]
    L.w4g128_moe.restype = i
    L.w4g128_moe.argtypes = [ctypes.POINTER(MoEArgs), p, sz, p]
    return L


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _nbytes(t):
    return t.numel() * t.element_size()


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(fn, rc):
    if rc != 0:
        raise W4G128Error(fn, rc)


def w4g128_status_string(status):
    return lib().w4g128_status_string(int(status)).decode()


def w4g128_packed_bytes(K, N):
    return int(lib().w4g128_packed_bytes(K, N))


def w4g128_pack(codes, scales, mins, K, N, packed, stream=None):
    _check("w4g128_pack", lib().w4g128_pack(_ptr(codes), _ptr(scales), _ptr(mins), K, N, _ptr(packed),
                                            _stream(stream)))


def w4g128_unpack(packed, K, N, codes, scales, mins, stream=None):
    _check("w4g128_unpack", lib().w4g128_unpack(_ptr(packed), K, N, _ptr(codes), _ptr(scales), _ptr(mins),
                                                _stream(stream)))


def w4g128_quantize(w, K, N, search, codes, scales, mins, stream=None):
    """bf16 weights [K][N] -> canonical codes, scales, mins (search: 0 RTN, 1 range search)."""
    _check("w4g128_quantize", lib().w4g128_quantize(_ptr(w), K, N, int(search), _ptr(codes), _ptr(scales),
                                                    _ptr(mins), _stream(stream)))


def w4g128_workspace_bytes(M, K, N):
    return int(lib().w4g128_workspace_bytes(M, K, N))


def w4g128_gemv(packed, x, y, K, N, ws, ws_bytes=None, stream=None):
    wb = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check("w4g128_gemv", lib().w4g128_gemv(_ptr(packed), _ptr(x), _ptr(y), K, N, _ptr(ws), wb, _stream(stream)))


def w4g128_gemm_verify(packed, x, y, M, K, N, ws, ws_bytes=None, stream=None):
    wb = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check("w4g128_gemm_verify", lib().w4g128_gemm_verify(_ptr(packed), _ptr(x), _ptr(y), M, K, N, _ptr(ws), wb,
                                                          _stream(stream)))


def _matrices(mats):
    arr = (_Matrix * len(mats))()
    for i, (packed, x, y, K, N) in enumerate(mats):
        arr[i] = _Matrix(_ptr(packed), _ptr(x), _ptr(y), K, N)
    return arr


def w4g128_decode_step_workspace_bytes(mats, M):
    """mats: sequence of (packed, x, y, K, N)."""
    arr = _matrices(mats)
    return int(lib().w4g128_decode_step_workspace_bytes(arr, len(mats), M))


def w4g128_decode_step(mats, M, ws, ws_bytes=None, stream=None):
    """mats: sequence of (packed, x, y, K, N); one persistent launch for all."""
    arr = _matrices(mats)
    wb = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check("w4g128_decode_step", lib().w4g128_decode_step(arr, len(mats), M, _ptr(ws), wb, _stream(stream)))


def w4g128_verify_step(mats, M, ws, ws_bytes=None, stream=None):
    """decode_step with the verify (warp-MMA) arithmetic at every M, M = 1 included."""
    arr = _matrices(mats)
    wb = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check("w4g128_verify_step", lib().w4g128_verify_step(arr, len(mats), M, _ptr(ws), wb, _stream(stream)))


def w4g128_schedule(mats, M):
    """The schedule a decode_step of mats (sequence of (packed, x, y, K, N);
    only K, N and x are read, pointers may be None) takes at M rows: a dict
    of the W4G128_SCHEDULE_FIELDS values."""
    arr = _matrices(mats)
    out = (ctypes.c_longlong * SCHEDULE_FIELDS)()
    _check("w4g128_schedule", lib().w4g128_schedule(arr, len(mats), M, out, SCHEDULE_FIELDS))
    keys = ("local", "ctas", "cta_warps", "second_pass", "pair_quads", "ring_depth", "workspace_bytes", "items")
    return dict(zip(keys, (int(v) for v in out)))


def w4g128_gemm_add_rmsnorm(packed, x, residual, gamma, eps, h, out, M, K, N, verify, ws, ws_bytes=None,
                            stream=None):
    """h = residual + x W (bf16, one rounding), out = gamma h / rms(h) per row."""
    wb = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check("w4g128_gemm_add_rmsnorm",
           lib().w4g128_gemm_add_rmsnorm(_ptr(packed), _ptr(x), _ptr(residual), _ptr(gamma), float(eps), _ptr(h),
                                         _ptr(out), M, K, N, int(verify), _ptr(ws), wb, _stream(stream)))


def w4g128_workspace_status(ws, stream=None):
    out = ctypes.c_int(0)
    _check("w4g128_workspace_status", lib().w4g128_workspace_status(_ptr(ws), ctypes.byref(out), _stream(stream)))
    return out.value


def w4g128_probe_sink_bytes():
    return int(lib().w4g128_probe_sink_bytes())


def w4g128_probe_read(buf, nbytes, sink, stream=None):
    _check("w4g128_probe_read", lib().w4g128_probe_read(_ptr(buf), nbytes, _ptr(sink), _stream(stream)))


def w4g128_probe_copy(src, dst, nbytes, stream=None):
    _check("w4g128_probe_copy", lib().w4g128_probe_copy(_ptr(src), _ptr(dst), nbytes, _stream(stream)))


def w4g128_gemv_noalloc(packed, x, y, K, N, stream=None):
    """w4g128_gemv without a workspace argument: for callers that must not
    allocate device memory (see include/w4g128.h)."""
    _check("w4g128_gemv_noalloc", lib().w4g128_gemv_noalloc(_ptr(packed), _ptr(x), _ptr(y), K, N,
                                                            _stream(stream)))


def w4g128_noalloc_status(stream=None):
    """Status word the last w4g128_gemv_noalloc call on this device left."""
    out = ctypes.c_int(0)
    _check("w4g128_noalloc_status", lib().w4g128_noalloc_status(ctypes.byref(out), _stream(stream)))
    return out.value


def w4g128_selftest_wait(ws, limit_ns, set_flag, ws_bytes=None, stream=None):
    """Diagnostic: a bounded device wait on a flag of `ws` (see include/w4g128.h)."""
    wb = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check("w4g128_selftest_wait", lib().w4g128_selftest_wait(_ptr(ws), wb, int(limit_ns), int(set_flag),
                                                              _stream(stream)))


def w4g128_decode_step_host(mats, M, x_host, x_dev, x_bytes, y_host, y_dev, y_bytes, ws, ws_bytes=None,
                            stream=None):
    """decode_step with the activations copied from / to host buffers in the same call."""
    arr = _matrices(mats)
    wb = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check("w4g128_decode_step_host",
           lib().w4g128_decode_step_host(arr, len(mats), M, _ptr(x_host), _ptr(x_dev), x_bytes, _ptr(y_host),
                                         _ptr(y_dev), y_bytes, _ptr(ws), wb, _stream(stream)))


class DecodeStep:
    """A decode step whose arguments are marshalled once: the descriptor
    array and the pointers are fixed, so each call is one C call.

    mats: sequence of (packed, x, y, K, N); ws: the workspace.  ``run`` calls
    w4g128_decode_step, ``run_host`` w4g128_decode_step_host with the host
    and device buffers given here."""

    def __init__(self, mats, M, ws, stream=None, x_host=None, x_dev=None, y_host=None, y_dev=None):
        self._keep = (mats, ws, x_host, x_dev, y_host, y_dev)  # the buffers outlive the step
        self._arr = _matrices(mats)
        self._n = len(mats)
        self._M = M
        self._ws = _ptr(ws)
        self._wb = _nbytes(ws)
        self._stream = _stream(stream)
        self._xh, self._xd = _ptr(x_host), _ptr(x_dev)
        self._xb = 0 if x_host is None else _nbytes(x_host)
        self._yh, self._yd = _ptr(y_host), _ptr(y_dev)
        self._yb = 0 if y_host is None else _nbytes(y_host)
        self._fn = lib().w4g128_decode_step
        self._fn_host = lib().w4g128_decode_step_host

    def run(self):
        rc = self._fn(self._arr, self._n, self._M, self._ws, self._wb, self._stream)
        if rc != 0:
            raise W4G128Error("w4g128_decode_step", rc)

    def run_host(self):
        rc = self._fn_host(self._arr, self._n, self._M, self._xh, self._xd, self._xb, self._yh, self._yd, self._yb,
                           self._ws, self._wb, self._stream)
        if rc != 0:
            raise W4G128Error("w4g128_decode_step_host", rc)


class _Args(ctypes.Structure):
    """Argument struct of an operator of include/w4g128_ops.h, filled from
    keywords.  A tensor becomes its device pointer (the struct keeps the tensor
    alive); it has to be on a GPU, of the element size that the field holds,
    contiguous (where the struct has strides for it: in its last dimension), and
    reach at least as far as the sizes say, and all tensors on one
    (W4G128_ERR_INVALID_ARG).  Plain integers are raw pointers and are not
    checked."""

    _fn = ""
    _itemsize = {}  # tensor field: bytes of an element
    _strided = ()   # tensor fields that the struct has strides for
    _device = None  # the tensors' GPU

    def __init__(self, **fields):
        known = {f[0] for f in self._fields_}
        for name in fields:
            if name not in known:
                raise TypeError(f"{type(self).__name__} has no field {name!r}")
        super().__init__(**{k: (_ptr(v) if k in self._itemsize else v) for k, v in fields.items()})
        self._keep = {k: v for k, v in fields.items() if k in self._itemsize and hasattr(v, "data_ptr")}
        for name, t in self._keep.items():
            size = self._itemsize[name]
            if not t.is_cuda or (size and t.element_size() != size):
                raise W4G128Error(f"{self._fn} ({name})", 1)
            if self._device is None:
                self._device = t.device.index
            if t.device.index != self._device:
                raise W4G128Error(f"{self._fn} ({name})", 1)
            rows_whole = t.dim() == 0 or t.shape[-1] <= 1 or t.stride(-1) == 1
            if not (rows_whole if name in self._strided else t.is_contiguous()):
                raise W4G128Error(f"{self._fn} ({name})", 1)
            need = self._reach(name)
            # the last element that the tensor's own storage holds behind its first
            have = t.untyped_storage().nbytes() - t.storage_offset() * t.element_size()
            if need * max(size, 1) > have:
                raise W4G128Error(f"{self._fn} ({name})", 1)

    def _reach(self, name):
        """Elements (bytes where the field has no element size) that the call may touch from `name` on."""
        return 0


def _check_device(fn, args, ws=None):
    """The kernels run on the current device: the call's tensors and its workspace have to be there."""
    on = [] if args._device is None else [("arguments", args._device)]
    if hasattr(ws, "data_ptr"):
        on.append(("ws", ws.device.index if ws.is_cuda else None))
    if on:
        import torch
        current = torch.cuda.current_device()
        for what, device in on:
            if device != current:
                raise W4G128Error(f"{fn} ({what} on another device)", 1)


class _Step:
    """An operator call whose arguments are marshalled once, like DecodeStep:
    the struct, the workspace and the stream are fixed, `run` is one C call."""

    _entry = ""

    def __init__(self, args, ws=None, stream=None):
        _check_device(self._entry, args, ws)
        self._keep = (args, ws)  # the buffers outlive the step
        self._args = ctypes.byref(args)
        self._fn = getattr(lib(), self._entry)
        s = _stream(stream)
        self._rest = (s,) if ws is None else (_ptr(ws), _nbytes(ws), s)

    def run(self):
        rc = self._fn(self._args, *self._rest)
        if rc != 0:
            raise W4G128Error(self._entry, rc)


class SampleArgs(_Args):
    """w4g128_sample_args: logits bf16 (row r at r * row_stride), temperature,
    top_p, min_p, u float32 [rows], top_k int32 [rows] (each filter may be
    None), tokens int32 [rows], logprobs float32 [rows] or None."""

    _fn = "w4g128_sample"
    _fields_ = [("logits", ctypes.c_void_p), ("row_stride", ctypes.c_longlong), ("temperature", ctypes.c_void_p),
                ("top_k", ctypes.c_void_p), ("top_p", ctypes.c_void_p), ("min_p", ctypes.c_void_p),
                ("u", ctypes.c_void_p), ("tokens", ctypes.c_void_p), ("logprobs", ctypes.c_void_p),
                ("rows", ctypes.c_int), ("vocab", ctypes.c_int)]
    _itemsize = {"logits": 2, "temperature": 4, "top_k": 4, "top_p": 4, "min_p": 4, "u": 4, "tokens": 4,
                 "logprobs": 4}
    _strided = ("logits",)

    def _reach(self, name):
        return (self.rows - 1) * self.row_stride + self.vocab if name == "logits" else self.rows


def w4g128_sample(args, stream=None):
    """One token per row (see include/w4g128_ops.h); args: SampleArgs."""
    _check_device("w4g128_sample", args)
    _check("w4g128_sample", lib().w4g128_sample(ctypes.byref(args), _stream(stream)))


class SampleStep(_Step):
    """w4g128_sample with its arguments marshalled once: SampleStep(args).run()."""

    _entry = "w4g128_sample"


class AttendArgs(_Args):
    """w4g128_attend_args: bf16 q, k_new, v_new (or None), k_cache, v_cache,
    out and int32 page_table, row_offsets, lens; strides in elements."""

    _fn = "w4g128_attend"
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k_new", "v_new", "k_cache", "v_cache", "page_table",
                                               "row_offsets", "lens", "out")] + \
               [(n, ctypes.c_longlong) for n in ("q_row", "kv_row", "out_row", "page_stride", "slot_stride",
                                                 "head_stride", "table_row")] + \
               [(n, ctypes.c_int) for n in ("rows", "count", "q_heads", "kv_heads", "head_dim", "pages", "page_size",
                                            "max_len", "max_new", "window", "sinks")] + [("scale", ctypes.c_float)]
    _itemsize = {"q": 2, "k_new": 2, "v_new": 2, "k_cache": 2, "v_cache": 2, "page_table": 4, "row_offsets": 4,
                 "lens": 4, "out": 2}
    _strided = ("q", "k_new", "v_new", "k_cache", "v_cache", "page_table", "out")

    def _reach(self, name):
        if name in ("q", "out"):
            return (self.rows - 1) * (self.q_row if name == "q" else self.out_row) + self.q_heads * self.head_dim
        if name in ("k_new", "v_new"):
            return (self.rows - 1) * self.kv_row + self.kv_heads * self.head_dim
        if name in ("k_cache", "v_cache"):
            return (self.pages - 1) * self.page_stride + (self.page_size - 1) * self.slot_stride + \
                (self.kv_heads - 1) * self.head_stride + self.head_dim
        if name == "page_table":
            return (self.count - 1) * self.table_row + (self.max_len - 1) // max(self.page_size, 1) + 1
        return self.count + 1 if name == "row_offsets" else self.count


def w4g128_attend_workspace_bytes(args):
    return int(lib().w4g128_attend_workspace_bytes(ctypes.byref(args)))


def w4g128_attend(args, ws, ws_bytes=None, stream=None):
    """Attention of each sequence's new tokens over its pages (see include/w4g128_ops.h); args: AttendArgs."""
    wb = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check_device("w4g128_attend", args, ws)
    _check("w4g128_attend", lib().w4g128_attend(ctypes.byref(args), _ptr(ws), wb, _stream(stream)))


class AttendStep(_Step):
    """w4g128_attend with its arguments marshalled once: AttendStep(args, ws).run()."""

    _entry = "w4g128_attend"


class MoEArgs(_Args):
    """w4g128_moe_args: bf16 x, residual (or None), y [M][D] and router [E][D];
    gate_up and down: E packed matrices one after another."""

    _fn = "w4g128_moe"
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "residual", "y", "router", "gate_up", "down")] + \
               [(n, ctypes.c_int) for n in ("M", "D", "F", "E", "top_k", "renormalize")]
    _itemsize = {"x": 2, "residual": 2, "y": 2, "router": 2, "gate_up": 0, "down": 0}

    def _reach(self, name):
        if name == "gate_up":
            return self.E * self.D * self.F * 17 // 16
        if name == "down":
            return self.E * self.D * self.F * 17 // 32
        return self.D * (self.E if name == "router" else self.M)


def w4g128_moe_workspace_bytes(args):
    return int(lib().w4g128_moe_workspace_bytes(ctypes.byref(args)))


def w4g128_moe(args, ws, ws_bytes=None, stream=None):
    """The mixture-of-experts layer (see include/w4g128_ops.h); args: MoEArgs."""
    wb = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check_device("w4g128_moe", args, ws)
    _check("w4g128_moe", lib().w4g128_moe(ctypes.byref(args), _ptr(ws), wb, _stream(stream)))


class MoEStep(_Step):
    """w4g128_moe with its arguments marshalled once: MoEStep(args, ws).run()."""

    _entry = "w4g128_moe"
