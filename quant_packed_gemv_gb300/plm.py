"""Python binding of libplm: the C ABI of include/plm.h, same names.

Argument marshalling only.  Device buffers are torch tensors (or raw integer
device addresses); the stream is a torch.cuda.Stream, a raw cudaStream_t
integer, or None for torch's current stream.  Every computation runs in the
library's CUDA kernels; there is no host or library fallback, and loading
fails loudly when libplm.so is missing.
"""
import ctypes
import os
import struct

from . import build as _build

PLM_OK = 0
PLM_ERR_INVALID_ARG = 1
PLM_ERR_MISALIGNED = 2
PLM_ERR_UNSUPPORTED = 3
PLM_ERR_CUDA = 4

QK = 256
Q4K_BYTES = 144
Q5K_BYTES = 176
Q2K_BYTES = 84
Q3K_BYTES = 110
Q6K_BYTES = 210
Q8K_BYTES = 292
GEMV_MAX_M = 8
PLM_NOALLOC_WORKSPACE_BYTES = 32 << 20   # the fixed array of plm_gemm_q4K_noalloc


class PlmError(RuntimeError):
    def __init__(self, fn, status, lib):
        self.status = status
        msg = lib.plm_status_string(status).decode()
        if status == PLM_ERR_CUDA:
            msg += " (cudaError %d)" % lib.plm_last_cuda_error()
        super().__init__("%s: %s" % (fn, msg))


class _Problem(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("xq", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("k", ctypes.c_int64)]


class _SProblem(ctypes.Structure):
    _fields_ = [("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("xq", ctypes.c_void_p),
                ("h", ctypes.c_void_p), ("n", ctypes.c_int64), ("k", ctypes.c_int64)]


class _QProblem(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("k", ctypes.c_int64)]


class _RopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("factor", ctypes.c_double), ("trained", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double)]


class _RopeTensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("heads", ctypes.c_int64),
                ("x_token_stride", ctypes.c_int64), ("x_head_stride", ctypes.c_int64),
                ("y_token_stride", ctypes.c_int64), ("y_head_stride", ctypes.c_int64),
                ("page_tokens", ctypes.c_int64), ("page_stride", ctypes.c_int64), ("pages", ctypes.c_int64),
                ("x_type", ctypes.c_int32), ("y_type", ctypes.c_int32), ("rotate", ctypes.c_int32)]


class _KvState(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("page_bytes", ctypes.c_int64), ("pages", ctypes.c_int64),
                ("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("refs", ctypes.c_void_p),
                ("status", ctypes.c_void_p), ("max_seqs", ctypes.c_int64), ("max_pages", ctypes.c_int64),
                ("page_tokens", ctypes.c_int64)]


class _AttnProblem(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_void_p) for f in ("q", "o", "lse", "k", "v", "table", "lens", "seqs")] +
                [(f, ctypes.c_int64) for f in ("batch", "tokens", "heads", "kv_heads", "head_dim", "q_token_stride",
                                               "q_head_stride", "o_token_stride", "o_head_stride", "page_tokens",
                                               "pages", "page_stride", "kv_head_stride", "kv_token_stride",
                                               "table_stride", "rows", "prefix_len", "max_len")] +
                [("scale", ctypes.c_float), ("type", ctypes.c_int32), ("o_type", ctypes.c_int32)])


class _RmsnormProblem(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_void_p) for f in ("x", "residual", "weight", "sum", "xq", "y")] +
                [(f, ctypes.c_int64) for f in ("m", "k", "x_stride", "residual_stride", "sum_stride", "y_stride")] +
                [("eps", ctypes.c_float)] + [(f, ctypes.c_int32) for f in ("x_type", "r_type", "w_type", "y_type")])


class _Kv8Tensor(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_void_p) for f in ("rows", "codes", "exps", "slots")] +
                [(f, ctypes.c_int64) for f in ("heads", "row_token_stride", "row_head_stride", "page_tokens", "pages", "page_stride",
                                               "head_stride", "token_stride", "exp_page_stride", "exp_head_stride")] +
                [("type", ctypes.c_int32), ("rotate", ctypes.c_int32)])


class _AttnKv8Problem(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_void_p) for f in ("q", "o", "lse", "k", "v", "k_exps", "v_exps", "table", "lens", "seqs")] +
                [(f, ctypes.c_int64) for f in ("batch", "tokens", "heads", "kv_heads", "head_dim", "q_token_stride",
                                               "q_head_stride", "o_token_stride", "o_head_stride", "page_tokens",
                                               "pages", "page_stride", "kv_head_stride", "kv_token_stride",
                                               "exp_page_stride", "exp_head_stride", "table_stride", "rows",
                                               "prefix_len", "max_len")] +
                [("scale", ctypes.c_float), ("type", ctypes.c_int32), ("o_type", ctypes.c_int32)])


class _SampleProblem(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_void_p) for f in ("logits", "u", "temperature", "top_k", "top_p", "min_p", "tokens", "prob")] +
                [(f, ctypes.c_int64) for f in ("m", "n", "stride")] + [("type", ctypes.c_int32)])


_lib = None


def library_path():
    return _build.LIB


def load(build_if_missing=True):
    """Loads libplm.so (building it first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if build_if_missing and not _build.up_to_date():
        _build.build()
    if not os.path.exists(path):
        raise RuntimeError("libplm.so not found at %s; run quant_packed_gemv_gb300.build" % path)
    lib = ctypes.CDLL(path)
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    lib.plm_abi_version.argtypes = []
    lib.plm_abi_version.restype = ctypes.c_int
    lib.plm_set_overlap.argtypes = [ctypes.c_int]
    lib.plm_set_overlap.restype = ctypes.c_int
    lib.plm_status_string.argtypes = [ctypes.c_int]
    lib.plm_status_string.restype = ctypes.c_char_p
    lib.plm_last_cuda_error.argtypes = []
    lib.plm_last_cuda_error.restype = ctypes.c_int
    lib.plm_device_fault.argtypes = [ctypes.POINTER(ctypes.c_uint32), ctypes.c_int]
    lib.plm_device_fault.restype = ctypes.c_int
    lib.plm_probe_mma_rates.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)]
    lib.plm_probe_mma_rates.restype = ctypes.c_int
    lib.plm_probe_tcgen05_rate.argtypes = [ctypes.POINTER(ctypes.c_double)] * 3
    lib.plm_probe_tcgen05_rate.restype = ctypes.c_int
    lib.plm_selftest_bounded_wait.argtypes = [ctypes.c_uint32, ctypes.c_int, vp]
    lib.plm_selftest_bounded_wait.restype = ctypes.c_int
    for f in ("q4K", "q6K"):
        getattr(lib, "plm_%s_x16_size" % f).argtypes = [i64, i64]
        getattr(lib, "plm_%s_x16_size" % f).restype = ctypes.c_size_t
        getattr(lib, "plm_%s_to_x16" % f).argtypes = [vp, vp, i64, i64, vp]
        getattr(lib, "plm_%s_to_x16" % f).restype = ctypes.c_int
    lib.plm_quantize_q8K.argtypes = [vp, vp, i64, i64, vp]
    lib.plm_quantize_q8K.restype = ctypes.c_int
    lib.plm_gemm_workspace_size.argtypes = [ctypes.c_int, i64, i64]
    lib.plm_gemm_workspace_size.restype = ctypes.c_size_t
    lib.plm_gemm_workspace_size_split.argtypes = [ctypes.c_int, i64, i64, i64]
    lib.plm_gemm_workspace_size_split.restype = ctypes.c_size_t
    for name in ("plm_gemm_q2K_ws", "plm_gemm_q3K_ws", "plm_gemm_q4K_ws", "plm_gemm_q5K_ws", "plm_gemm_q6K_ws"):
        fn = getattr(lib, name)
        fn.argtypes = [vp, vp, vp, i64, i64, i64, vp, ctypes.c_size_t, vp]
        fn.restype = ctypes.c_int
    for name in ("plm_gemv_q2K_grouped", "plm_gemv_q3K_grouped", "plm_gemv_q4K_grouped", "plm_gemv_q5K_grouped",
                 "plm_gemv_q6K_grouped"):
        fn = getattr(lib, name)
        fn.argtypes = [ctypes.POINTER(_Problem), i64, i64, vp]
        fn.restype = ctypes.c_int
    lib.plm_gemv_q4K_swiglu.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
    lib.plm_gemv_q4K_swiglu.restype = ctypes.c_int
    lib.plm_gemv_q4K_swiglu_grouped.argtypes = [ctypes.POINTER(_SProblem), i64, i64, vp]
    lib.plm_gemv_q4K_swiglu_grouped.restype = ctypes.c_int
    lib.plm_gemm_q4K_swiglu.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
    lib.plm_gemm_q4K_swiglu.restype = ctypes.c_int
    lib.plm_gemm_q4K_swiglu_ws.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, ctypes.c_size_t, vp]
    lib.plm_gemm_q4K_swiglu_ws.restype = ctypes.c_int
    lib.plm_gemm_swiglu_workspace_size.argtypes = [i64, i64, i64]
    lib.plm_gemm_swiglu_workspace_size.restype = ctypes.c_size_t
    lib.plm_quantize_gemv_q4K_grouped.argtypes = [ctypes.POINTER(_QProblem), i64, i64, vp]
    lib.plm_quantize_gemv_q4K_grouped.restype = ctypes.c_int
    for name in ("plm_gemv_q4K", "plm_gemv_q6K", "plm_gemm_q4K", "plm_gemm_q6K", "plm_gemm_q4K_noalloc",
                 "plm_subdots_q4K", "plm_subdots_q6K", "plm_quantize_gemv_q4K",
                 "plm_gemv_q5K", "plm_gemm_q5K", "plm_subdots_q5K",
                 "plm_gemv_q2K", "plm_gemm_q2K", "plm_subdots_q2K", "plm_gemv_q3K", "plm_gemm_q3K", "plm_subdots_q3K",
                 "plm_gemv_q4K_x16", "plm_gemv_q6K_x16"):
        fn = getattr(lib, name)
        fn.argtypes = [vp, vp, vp, i64, i64, i64, vp]
        fn.restype = ctypes.c_int
    dbl, sz, i32, f32 = ctypes.c_double, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
    for name, res, args in (
            ("plm_rope_freqs", i32, [vp, i64, dbl, ctypes.POINTER(_RopeScaling), ctypes.POINTER(f32)]),
            ("plm_rope", i32, [vp, i64, vp, vp, i64, i64, i64, i32, f32, i32, vp]),
            ("plm_kv_workspace_size", sz, [i64, i64]),
            ("plm_kv_reserve", i32, [vp, vp, vp, i64, vp, i64, vp, sz, vp]),
            ("plm_kv_fork", i32, [vp, vp, vp, vp, i64, vp, sz, vp]),
            ("plm_kv_free", i32, [vp, vp, i64, vp]),
            ("plm_kv_compact", i32, [vp, vp, vp, sz, vp]),
            ("plm_kv_copy_pages", i32, [vp, vp, vp, i64, vp]),
            ("plm_call", i32, [i32, vp]),
            ("plm_attn_workspace_size", sz, [i64] * 7),
            ("plm_attn_shared_prefix", i32, [vp, vp, sz, vp]),
            ("plm_rmsnorm", i32, [vp, vp]),
            ("plm_kv8_write", i32, [vp, i64, vp, vp, i64, i64, i64, i32, f32, vp]),
            ("plm_kv8_read", i32, [vp, i64, i64, i64, vp]),
            ("plm_attn_kv8_workspace_size", sz, [i64] * 7),
            ("plm_attn_kv8", i32, [vp, vp, sz, vp]),
            ("plm_sample", i32, [vp, vp])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = res
    _lib = lib
    return lib


def _current_stream():
    """Address of torch's current stream (by the call that gives it without a Stream object, where torch has it)."""
    global _current_stream
    import torch
    get, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    if get is None or dev is None:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    else:
        torch.cuda.current_stream()   # initializes CUDA
        _current_stream = lambda: get(dev())  # noqa: E731
    return _current_stream()


def _addr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(s):
    if s is None:
        return _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(fn, status):
    if status != PLM_OK:
        raise PlmError(fn, status, _lib)


def plm_abi_version():
    return load().plm_abi_version()


PLM_OVERLAP_OFF, PLM_OVERLAP_LAUNCH, PLM_OVERLAP_PREFETCH = 0, 1, 2


def plm_set_overlap(mode):
    """Early-launch mode for later launches (PLM_OVERLAP_*); returns the previous mode."""
    lib = load()
    r = lib.plm_set_overlap(int(mode))
    if r < 0:
        raise PlmError("plm_set_overlap", -r, lib)
    return r


def plm_device_fault(clear=True):
    """Reads (and by default clears) the device fault word; synchronizes."""
    lib = load()
    code = ctypes.c_uint32(0)
    _check("plm_device_fault", lib.plm_device_fault(ctypes.byref(code), 1 if clear else 0))
    return code.value


def plm_selftest_bounded_wait(rounds, complete, stream=None):
    """Launches the bounded-wait self-test (see include/plm.h); asynchronous."""
    lib = load()
    _check("plm_selftest_bounded_wait", lib.plm_selftest_bounded_wait(int(rounds), 1 if complete else 0,
                                                                      _stream(stream)))


def plm_probe_mma_rates():
    """(mma.sync s8 TOPS, mma.sync f16 TFLOPS) measured on the current device; synchronizes."""
    lib = load()
    a, b = ctypes.c_double(0), ctypes.c_double(0)
    _check("plm_probe_mma_rates", lib.plm_probe_mma_rates(ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def plm_probe_tcgen05_rate():
    """(cycles per MMA, cycles per MMA with an mbarrier wait after each commit, TFLOPS on every
    SM) of the GEMM's tcgen05 MMA on the current device; synchronizes."""
    lib = load()
    a, b, c = ctypes.c_double(0), ctypes.c_double(0), ctypes.c_double(0)
    _check("plm_probe_tcgen05_rate", lib.plm_probe_tcgen05_rate(ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)))
    return a.value, b.value, c.value


def plm_quantize_q8K(x, xq, m, k, stream=None):
    lib = load()
    _check("plm_quantize_q8K", lib.plm_quantize_q8K(_addr(x), _addr(xq), m, k, _stream(stream)))


def _mm(name):
    def call(w, xq, y, m, n, k, stream=None):
        lib = load()
        _check(name, getattr(lib, name)(_addr(w), _addr(xq), _addr(y), m, n, k, _stream(stream)))
    call.__name__ = name
    call.__doc__ = "Binding of the C entry point %s(w, xq, out, m, n, k, stream)." % name
    return call


plm_gemv_q4K = _mm("plm_gemv_q4K")
plm_gemv_q6K = _mm("plm_gemv_q6K")
plm_gemv_q5K = _mm("plm_gemv_q5K")
plm_gemm_q5K = _mm("plm_gemm_q5K")
plm_subdots_q5K = _mm("plm_subdots_q5K")
plm_gemv_q2K = _mm("plm_gemv_q2K")
plm_gemm_q2K = _mm("plm_gemm_q2K")
plm_subdots_q2K = _mm("plm_subdots_q2K")
plm_gemv_q3K = _mm("plm_gemv_q3K")
plm_gemm_q3K = _mm("plm_gemm_q3K")
plm_subdots_q3K = _mm("plm_subdots_q3K")
plm_gemm_q4K = _mm("plm_gemm_q4K")
plm_gemm_q6K = _mm("plm_gemm_q6K")
# q4_K GEMM whose workspace is a fixed array inside the library: for callers
# that must not allocate device memory while running (see include/plm.h).
plm_gemm_q4K_noalloc = _mm("plm_gemm_q4K_noalloc")
plm_subdots_q4K = _mm("plm_subdots_q4K")
# fused q8_K producer: f32 activations x in place of xq
plm_quantize_gemv_q4K = _mm("plm_quantize_gemv_q4K")
plm_subdots_q6K = _mm("plm_subdots_q6K")


plm_gemv_q4K_x16 = _mm("plm_gemv_q4K_x16")
plm_gemv_q6K_x16 = _mm("plm_gemv_q6K_x16")


def plm_q4K_x16_size(n, k):
    """Bytes of the row-interleaved x16 form of an n x k q4_K matrix (0: invalid)."""
    return load().plm_q4K_x16_size(n, k)


def plm_q6K_x16_size(n, k):
    """Bytes of the row-interleaved x16 form of an n x k q6_K matrix (0: invalid)."""
    return load().plm_q6K_x16_size(n, k)


def plm_q4K_to_x16(w, w_x16, n, k, stream=None):
    """Repacks q4_K weights into the x16 layout (see include/plm.h)."""
    lib = load()
    _check("plm_q4K_to_x16", lib.plm_q4K_to_x16(_addr(w), _addr(w_x16), n, k, _stream(stream)))


def plm_q6K_to_x16(w, w_x16, n, k, stream=None):
    """Repacks q6_K weights into the x16 layout (see include/plm.h)."""
    lib = load()
    _check("plm_q6K_to_x16", lib.plm_q6K_to_x16(_addr(w), _addr(w_x16), n, k, _stream(stream)))


def _grouped(name):
    def call(problems, m, stream=None):
        """problems: sequence of (w, xq, y, n, k) with device tensors or addresses."""
        lib = load()
        arr = (_Problem * len(problems))()
        for j, (w, xq, y, n, k) in enumerate(problems):
            arr[j] = _Problem(_addr(w), _addr(xq), _addr(y), n, k)
        _check(name, getattr(lib, name)(arr, len(problems), m, _stream(stream)))
    call.__name__ = name
    call.__doc__ = "Binding of %s(problems, count, m, stream)." % name
    return call


plm_gemv_q4K_grouped = _grouped("plm_gemv_q4K_grouped")
plm_gemv_q6K_grouped = _grouped("plm_gemv_q6K_grouped")
plm_gemv_q5K_grouped = _grouped("plm_gemv_q5K_grouped")
plm_gemv_q2K_grouped = _grouped("plm_gemv_q2K_grouped")
plm_gemv_q3K_grouped = _grouped("plm_gemv_q3K_grouped")


def plm_gemv_q4K_swiglu(w_gate, w_up, xq, h, m, n, k, stream=None):
    """h = silu(W_gate . x) * (W_up . x) (see include/plm.h)."""
    lib = load()
    _check("plm_gemv_q4K_swiglu", lib.plm_gemv_q4K_swiglu(_addr(w_gate), _addr(w_up), _addr(xq), _addr(h), m, n, k,
                                                          _stream(stream)))


def plm_gemm_swiglu_workspace_size(m, n, k):
    """Workspace bytes of plm_gemm_q4K_swiglu_ws (0: none needed, or invalid arguments)."""
    return load().plm_gemm_swiglu_workspace_size(m, n, k)


def plm_gemm_q4K_swiglu(w_gate, w_up, xq, h, m, n, k, stream=None):
    """Prefill gate/up pair: h = silu(W_gate . x) * (W_up . x) (see include/plm.h)."""
    lib = load()
    _check("plm_gemm_q4K_swiglu", lib.plm_gemm_q4K_swiglu(_addr(w_gate), _addr(w_up), _addr(xq), _addr(h), m, n, k,
                                                          _stream(stream)))


def plm_gemm_q4K_swiglu_ws(w_gate, w_up, xq, h, m, n, k, workspace, workspace_bytes=None, stream=None):
    """plm_gemm_q4K_swiglu with a caller-owned workspace (plm_gemm_swiglu_workspace_size bytes)."""
    lib = load()
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("plm_gemm_q4K_swiglu_ws", lib.plm_gemm_q4K_swiglu_ws(_addr(w_gate), _addr(w_up), _addr(xq), _addr(h), m,
                                                                n, k, _addr(workspace), workspace_bytes,
                                                                _stream(stream)))


def plm_gemv_q4K_swiglu_grouped(problems, m, stream=None):
    """problems: sequence of (w_gate, w_up, xq, h, n, k) with device tensors or addresses."""
    lib = load()
    arr = (_SProblem * len(problems))()
    for j, (wg, wu, xq, h, n, k) in enumerate(problems):
        arr[j] = _SProblem(_addr(wg), _addr(wu), _addr(xq), _addr(h), n, k)
    _check("plm_gemv_q4K_swiglu_grouped", lib.plm_gemv_q4K_swiglu_grouped(arr, len(problems), m, _stream(stream)))


def plm_quantize_gemv_q4K_grouped(problems, m, stream=None):
    """problems: sequence of (w, x_f32, y, n, k) with device tensors or addresses."""
    lib = load()
    arr = (_QProblem * len(problems))()
    for j, (w, x, y, n, k) in enumerate(problems):
        arr[j] = _QProblem(_addr(w), _addr(x), _addr(y), n, k)
    _check("plm_quantize_gemv_q4K_grouped", lib.plm_quantize_gemv_q4K_grouped(arr, len(problems), m, _stream(stream)))


def plm_gemm_workspace_size(fmt, m, k):
    """fmt: 'q2K' .. 'q6K' or 2 .. 6."""
    f = {"q2K": 2, "q3K": 3, "q4K": 4, "q5K": 5, "q6K": 6}.get(fmt, fmt)
    return load().plm_gemm_workspace_size(f, m, k)


def plm_gemm_workspace_size_split(fmt, m, n, k):
    """Workspace bytes that let the GEMM split K (see include/plm.h)."""
    f = {"q2K": 2, "q3K": 3, "q4K": 4, "q5K": 5, "q6K": 6}.get(fmt, fmt)
    return load().plm_gemm_workspace_size_split(f, m, n, k)


def _gemm_ws(name):
    def call(w, xq, y, m, n, k, workspace, workspace_bytes=None, stream=None):
        lib = load()
        if workspace_bytes is None:
            workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check(name, getattr(lib, name)(_addr(w), _addr(xq), _addr(y), m, n, k, _addr(workspace),
                                        workspace_bytes, _stream(stream)))
    call.__name__ = name
    call.__doc__ = "Binding of %s(w, xq, y, m, n, k, workspace, bytes, stream)." % name
    return call


plm_gemm_q4K_ws = _gemm_ws("plm_gemm_q4K_ws")
plm_gemm_q6K_ws = _gemm_ws("plm_gemm_q6K_ws")
plm_gemm_q5K_ws = _gemm_ws("plm_gemm_q5K_ws")
plm_gemm_q2K_ws = _gemm_ws("plm_gemm_q2K_ws")
plm_gemm_q3K_ws = _gemm_ws("plm_gemm_q3K_ws")


def raw_status(name, *args):
    """Calls an entry point and returns its status code without raising
    (used by the argument-check tests)."""
    return getattr(load(), name)(*args)


# ---------------------------------------------------------------------------
# Rotary positions, cache pages, attention over a shared prefix.  Shapes and
# strides come from the torch tensors.
# ---------------------------------------------------------------------------
PLM_F32, PLM_F16, PLM_BF16 = 0, 1, 2
PLM_ROPE_HALF, PLM_ROPE_INTERLEAVED = 0, 1
PLM_KV_OUT_OF_PAGES, PLM_KV_BAD_ITEM = 1, 2
_LAYOUTS = {"half": PLM_ROPE_HALF, "interleaved": PLM_ROPE_INTERLEAVED}
_SCALINGS = {"none": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}


_types = {}    # torch type -> PLM_F32 .., filled on first use (torch is imported where it is needed)


def _type(t):
    code = _types.get(t.dtype)
    if code is None:
        if not _types:
            import torch
            _types.update({torch.float32: PLM_F32, torch.float16: PLM_F16, torch.bfloat16: PLM_BF16,
                           torch.int32: -32, torch.int64: -64})
            return _type(t)
        code = -1
    if code < 0:
        raise ValueError("expected float32, float16 or bfloat16, got %s" % t.dtype)
    return code


def _ints(t, bits, name, shape=None):
    """Address of a contiguous CUDA tensor of 32- or 64-bit integers (None stays None)."""
    if t is None:
        return None
    code = _types.get(t.dtype)
    if code is None and not _types:
        import torch
        _type(torch.empty(0))
        code = _types.get(t.dtype)
    if code != -bits:
        raise ValueError("%s: expected int%d, got %s" % (name, bits, t.dtype))
    if shape is not None and t.shape != shape:
        raise ValueError("%s: expected shape %s, got %s" % (name, shape, tuple(t.shape)))
    if not (t.is_cuda and t.is_contiguous()):
        return _addr(t)   # says why
    return t.data_ptr()


def _rows(t, name, dims):
    """Strides of a CUDA tensor whose last axis is dense."""
    st = t.stride()
    if len(st) != dims:
        raise ValueError("%s: expected %d dimensions, got %d" % (name, dims, len(st)))
    if not t.is_cuda:
        raise ValueError("%s: expected a CUDA tensor" % name)
    if st[-1] != 1 and t.shape[-1] > 1:
        raise ValueError("%s: the last dimension has to be dense" % name)
    return st


def plm_rope_freqs(rotary_dim, base, scaling="none", factor=1.0, trained=0.0, low=1.0, high=32.0, device=None):
    """(freqs, scale): an int64 tensor with the bits of plm_rope's uint64 frequencies (on `device`, the CPU if None)
    and the factor of cos and sin; scaling: "none", "linear", "base", "bands" or "ramp" (see include/plm.h)."""
    import torch
    lib = load()
    freqs = torch.empty(max(0, rotary_dim // 2), dtype=torch.int64)
    s = _RopeScaling(_SCALINGS[scaling], factor, trained, low, high)
    scale = ctypes.c_float(0)
    _check("plm_rope_freqs", lib.plm_rope_freqs(freqs.data_ptr() or None, rotary_dim, base, ctypes.byref(s),
                                                ctypes.byref(scale)))
    return (freqs if device is None else freqs.to(device)), scale.value


# These calls are packed: their structs and arguments go to plm_call as bytes,
# which costs a fifth of filling ctypes structures and converting arguments one by
# one.  A decode step makes them for a few microseconds of GPU time each.
_ROPE_TENSOR = struct.Struct("@11q3i4x")
_KV_STATE = struct.Struct("@10q")
_ATTN_PROBLEM = struct.Struct("@26qf2i4x")
_ROPE_CALL = struct.Struct("@7qd2q")
_RESERVE_CALL, _FORK_CALL, _FREE_CALL, _COMPACT_CALL, _COPY_CALL, _ATTN_CALL = (
    struct.Struct("@%dq" % n) for n in (8, 7, 3, 4, 4, 3))
_RMSNORM_PROBLEM = struct.Struct("@12qf4i4x")
_KV8_TENSOR = struct.Struct("@14q2i")
_ATTN_KV8_PROBLEM = struct.Struct("@30qf2i4x")
_SAMPLE_PROBLEM = struct.Struct("@11qi4x")
_ONE, _KV8_WRITE_CALL, _KV8_READ_CALL = struct.Struct("@q"), struct.Struct("@7qdq"), struct.Struct("@4q")
_ROPE, _RESERVE, _FORK, _FREE, _COMPACT, _COPY, _ATTN = range(7)
_RMSNORM, _KV8_WRITE, _KV8_READ, _ATTN_KV8, _SAMPLE = range(8, 13)
_NAMES = ("plm_rope", "plm_kv_reserve", "plm_kv_fork", "plm_kv_free", "plm_kv_compact", "plm_kv_copy_pages",
          "plm_attn_shared_prefix", "", "plm_rmsnorm", "plm_kv8_write", "plm_kv8_read", "plm_attn_kv8", "plm_sample")


def _call(entry, args):
    status = (_lib or load()).plm_call(entry, args)
    if status != PLM_OK:
        raise PlmError(_NAMES[entry], status, _lib)


def plm_rope_tensor(x, y, slots=None, rotate=True):
    """One tensor of a plm_rope call; it holds x, y and slots.  x [tokens][heads][head_dim]; y the same shape, or with
    slots (int64 [tokens]) the pages [pages][heads][page_tokens][head_dim] of a cache, as any strided view."""
    xs, shape, ys, xtype, ytype = x.stride(), x.shape, y.stride(), _types.get(x.dtype, -1), _types.get(y.dtype, -1)
    if len(xs) != 3 or xs[2] != 1 or len(ys) != (3 if slots is None else 4) or ys[-1] != 1 or xtype < 0 or ytype < 0 or not (
            x.is_cuda and y.is_cuda):   # an error, or a dimension of one: look closer
        _rows(x, "x", 3)
        _rows(y, "y", 3 if slots is None else 4)
        xtype, ytype = _type(x), _type(y)
    xt, xh, _ = xs
    tokens, heads, d = shape
    if slots is None:
        yt, yh, _ = ys
        if y.shape != shape:
            raise ValueError("y: expected shape %s, got %s" % (tuple(shape), tuple(y.shape)))
        at = page_tokens = page_stride = pages = 0
    else:
        page_stride, yh, yt, _ = ys
        pages, yheads, page_tokens, yd = y.shape
        if yheads != heads or yd != d:
            raise ValueError("y: expected pages [.][%d][.][%d], got %s" % (heads, d, tuple(y.shape)))
        at = _ints(slots, 64, "slots", (tokens,))
    return (_ROPE_TENSOR.pack(x.data_ptr(), y.data_ptr(), at, heads, xt, xh, yt, yh, page_tokens, page_stride, pages,
                              xtype, ytype, 1 if rotate else 0), tokens, d, (x, y, slots))


def plm_rope(tensors, positions, freqs, rotary_dim, layout="half", scale=1.0, inverse=False, stream=None):
    """Turns the heads of the tensors (plm_rope_tensor) by their positions (int32 [tokens]); see include/plm.h."""
    packed, tokens, d, _ = tensors[0] if tensors else (b"", positions.numel(), 0, None)
    if len(tensors) > 1:
        for t in tensors:
            if t[1] != tokens or t[2] != d:
                raise ValueError("the tensors differ in tokens or head size")
        packed = b"".join([t[0] for t in tensors])
    if freqs.numel() != rotary_dim // 2:
        raise ValueError("freqs: expected %d values, got %d" % (rotary_dim // 2, freqs.numel()))
    if tokens == 0 and tensors:
        return
    _call(_ROPE, _ROPE_CALL.pack(len(tensors), _ints(positions, 32, "positions", (tokens,)), _ints(freqs, 64, "freqs"),
                                 tokens, d, rotary_dim, _LAYOUTS.get(layout, layout), scale, 1 if inverse else 0,
                                 _stream(stream)) + packed)


def plm_kv_state(pool, table, lens, refs, page_tokens, status=None):
    """Page state over device tensors: pool [pages][...] of any type, table int32 [max_seqs][max_pages], lens int32
    [max_seqs], refs int32 [pages], status int32 [1] or None.  It holds the tensors."""
    pages, (seqs, width) = pool.shape[0], table.shape
    return (_KV_STATE.pack(_addr(pool), pool.nbytes // pages if pages else 0, pages, _ints(table, 32, "table"),
                           _ints(lens, 32, "lens", (seqs,)), _ints(refs, 32, "refs", (pages,)),
                           _ints(status, 32, "status") or 0, seqs, width, page_tokens), (pool, table, lens, refs, status))


def plm_kv_workspace_size(pages, n):
    """Workspace bytes of the page calls for n items (0: invalid arguments)."""
    return load().plm_kv_workspace_size(pages, n)


def _ws(workspace):
    """Address and size of a workspace tensor (None: 0, 0)."""
    return (0, 0) if workspace is None else (_addr(workspace), workspace.nbytes)


def plm_kv_reserve(kv, seqs, add, slots, workspace, stream=None):
    """Sequences seqs grow by add tokens (int32 [n]); slots int64 [n][most] or None gets the new tokens' slots."""
    n, most = seqs.numel(), 0
    if slots is not None:
        rows, most = slots.shape
        if rows != n:
            raise ValueError("slots: expected [%d][.], got %s" % (n, tuple(slots.shape)))
    ws, size = _ws(workspace)
    _call(_RESERVE, _RESERVE_CALL.pack(_ints(seqs, 32, "seqs"), _ints(add, 32, "add", (n,)), n, _ints(slots, 64, "slots") or 0,
                                       most, ws, size, _stream(stream)) + kv[0])


def plm_kv_fork(kv, parents, children, workspace, keep=None, stream=None):
    """Unused sequences children (int32 [n]) become copies of parents, of their first keep tokens if given."""
    n, (ws, size) = parents.numel(), _ws(workspace)
    _call(_FORK, _FORK_CALL.pack(_ints(parents, 32, "parents"), _ints(children, 32, "children", (n,)),
                                 _ints(keep, 32, "keep", (n,)) or 0, n, ws, size, _stream(stream)) + kv[0])


def plm_kv_free(kv, seqs, stream=None):
    """The sequences (int32 [n]) give their pages back."""
    _call(_FREE, _FREE_CALL.pack(_ints(seqs, 32, "seqs"), seqs.numel(), _stream(stream)) + kv[0])


def plm_kv_compact(kv, live, workspace, stream=None):
    """Packs the pages in use to the front of the pool; live (int32 [1] or None) gets their number."""
    ws, size = _ws(workspace)
    _call(_COMPACT, _COMPACT_CALL.pack(_ints(live, 32, "live") or 0, ws, size, _stream(stream)) + kv[0])


def plm_kv_copy_pages(kv, src, dst, stream=None):
    """Page dst[i] = page src[i] (int32 lists of the same length)."""
    n = src.numel()
    _call(_COPY, _COPY_CALL.pack(_ints(src, 32, "src"), _ints(dst, 32, "dst", (n,)), n, _stream(stream)) + kv[0])


def plm_attn_workspace_size(batch, tokens, heads, kv_heads, head_dim, prefix_len, max_len):
    """Workspace bytes of plm_attn_shared_prefix (0: none needed, or invalid arguments)."""
    return load().plm_attn_workspace_size(batch, tokens, heads, kv_heads, head_dim, prefix_len, max_len)


def plm_attn_shared_prefix(q, o, k, v, table, lens, tokens, prefix_len, max_len, scale, workspace, lse=None, seqs=None,
                           stream=None):
    """Attention of q [batch*tokens][heads][head_dim] over the pages k, v [pages][kv_heads][page_tokens][head_dim]
    (strided views of one shape and strides) into o; the batch's first prefix_len tokens are shared (see include/plm.h)."""
    qs, os_, ks, shape, kshape = q.stride(), o.stride(), k.stride(), q.shape, k.shape
    ktype, otype = _types.get(k.dtype, -1), _types.get(o.dtype, -1)
    if len(qs) != 3 or len(os_) != 3 or len(ks) != 4 or qs[2] != 1 or os_[2] != 1 or ks[3] != 1 or ktype < 0 or otype < 0 or not (
            q.is_cuda and o.is_cuda and k.is_cuda):   # an error, or a dimension of one: look closer
        _rows(q, "q", 3)
        _rows(o, "o", 3)
        _rows(k, "k", 4)
        ktype, otype = _type(k), _type(o)
    (qt, qh, _), (ot, oh, _), (kp, kh, kt, _) = qs, os_, ks
    if o.shape != shape:
        raise ValueError("o: expected shape %s, got %s" % (tuple(shape), tuple(o.shape)))
    if v.shape != kshape or v.stride() != ks or v.dtype != k.dtype or q.dtype != k.dtype or not v.is_cuda:
        raise ValueError("k and v have to agree in shape, strides and type, and q in type")
    n, heads, d = shape
    pages, kv_heads, page_tokens, kd = kshape
    if kd != d:
        raise ValueError("k: expected heads of %d, got %d" % (d, kd))
    if tokens < 1 or n % tokens:
        raise ValueError("q: %d rows are no multiple of %d tokens" % (n, tokens))
    rows, width = table.shape
    batch = n // tokens
    if seqs is None and batch > rows:
        raise ValueError("table: %d rows for a batch of %d" % (rows, batch))
    if lse is not None and (_type(lse) != PLM_F32 or lse.shape != (n, heads)):
        raise ValueError("lse: expected float32 %s" % ((n, heads),))
    if batch == 0:
        return
    ws, size = _ws(workspace)
    p = _ATTN_PROBLEM.pack(q.data_ptr(), o.data_ptr(), _addr(lse) or 0, k.data_ptr(), v.data_ptr(),
                           _ints(table, 32, "table"), _ints(lens, 32, "lens", (rows,)),
                           _ints(seqs, 32, "seqs", (batch,)) or 0, batch, tokens, heads, kv_heads, d, qt, qh, ot, oh,
                           page_tokens, pages, kp, kh, kt, width, rows, prefix_len, max_len, scale, ktype, otype)
    _call(_ATTN, _ATTN_CALL.pack(ws, size, _stream(stream)) + p)


# ---------------------------------------------------------------------------
# The residual sum and norm before a product, a cache in 8 bits and the
# attention over it, the next token.
# ---------------------------------------------------------------------------
def _matrix(t, name, shape=None):
    """Row stride and type of a CUDA tensor [m][k] with dense rows."""
    st = t.stride()
    if len(st) != 2 or st[1] != 1 or not t.is_cuda:
        _rows(t, name, 2)
    if shape is not None and t.shape != shape:
        raise ValueError("%s: expected shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return st[0], _types[t.dtype] if _types.get(t.dtype, -1) >= 0 else _type(t)


def plm_rmsnorm(x, weight, eps, residual=None, sum=None, xq=None, y=None, stream=None):
    """h = x + residual (into sum if given, of the residual's type; sum may be x or residual); h / sqrt(mean h^2 + eps) *
    weight into xq as q8_K blocks (contiguous bytes) and / or into y; x [m][k], weight [k] or None (see include/plm.h)."""
    shape = x.shape
    xs, xt = _matrix(x, "x")
    m, k = shape
    rs = rt = ss = ys = yt = wt = st = 0
    r = w = o = b = yo = 0
    if residual is not None:
        rs, rt = _matrix(residual, "residual", shape)
        r = residual.data_ptr()
    if sum is not None:
        ss, st = _matrix(sum, "sum", shape)
        if residual is None or st != rt:
            raise ValueError("sum: there is none without a residual, and it has the residual's type")
        o = sum.data_ptr()
    if weight is not None:
        if weight.shape != (k,):
            raise ValueError("weight: expected shape (%d,), got %s" % (k, tuple(weight.shape)))
        w, wt = _addr(weight), _type(weight)
    if xq is not None:
        if xq.nbytes != m * (k // QK) * Q8K_BYTES:
            raise ValueError("xq: expected %d bytes, got %d" % (m * (k // QK) * Q8K_BYTES, xq.nbytes))
        b = _addr(xq)
    if y is not None:
        ys, yt = _matrix(y, "y", shape)
        yo = y.data_ptr()
    if m == 0:
        return
    _call(_RMSNORM, _ONE.pack(_stream(stream)) + _RMSNORM_PROBLEM.pack(x.data_ptr(), r, w, o, b, yo, m, k, xs, rs, ss, ys, eps, xt, rt, wt, yt))


def plm_kv8_page_bytes(kv_heads, page_tokens, head_dim):
    """Bytes of a page of plm_kv8_views: keys and values, codes and exponents."""
    return 2 * kv_heads * page_tokens * (head_dim + head_dim // 32)


def plm_kv8_views(pool, kv_heads, page_tokens, head_dim):
    """(k, v, k_exps, v_exps) of a pool uint8 [pages][page bytes]: codes int8 [pages][kv_heads][page_tokens][head_dim],
    exponents uint8 [pages][kv_heads][page_tokens][head_dim / 32].  A page holds the keys' codes, the values' codes, then the
    exponents of both, so that the page calls (plm_kv_state over the same pool) move them together."""
    import torch
    n, size = kv_heads * page_tokens * head_dim, plm_kv8_page_bytes(kv_heads, page_tokens, head_dim)
    pages, width = pool.shape
    if head_dim % 32 or width < size or pool.dtype != torch.uint8 or (width > 1 and pool.stride(1) != 1):
        raise ValueError("pool: expected uint8 [.][%d or more], and heads of a multiple of 32" % size)
    blocks, pitch, at, codes = head_dim // 32, pool.stride(0), pool.storage_offset(), pool.view(torch.int8)
    shape, st = (pages, kv_heads, page_tokens, head_dim), (pitch, page_tokens * head_dim, head_dim, 1)
    eshape, est, e = (pages, kv_heads, page_tokens, blocks), (pitch, page_tokens * blocks, blocks, 1), at + 2 * n
    return (codes.as_strided(shape, st, at), codes.as_strided(shape, st, at + n), pool.as_strided(eshape, est, e),
            pool.as_strided(eshape, est, e + n // 32))


def _kv8_pages(codes, exps, name):
    """Strides of 8-bit pages: of the codes, and of the exponents."""
    import torch
    cs, es, shape, eshape = codes.stride(), exps.stride(), codes.shape, exps.shape
    if codes.dtype != torch.int8 or exps.dtype != torch.uint8:
        raise ValueError("%s: expected int8 codes and uint8 exponents" % name)
    if len(cs) != 4 or len(es) != 4 or cs[3] != 1 or es[3] != 1 or not (codes.is_cuda and exps.is_cuda):
        _rows(codes, name, 4)   # an error, or a dimension of one: look closer
        _rows(exps, name + " exponents", 4)
    blocks = shape[3] // 32
    if shape[3] % 32 or eshape[:3] != shape[:3] or eshape[3] != blocks or (es[2] != blocks and shape[2] > 1):
        raise ValueError("%s: expected exponents [pages][heads][page_tokens][head_dim / 32], a head's tokens dense" % name)
    return cs, es


def plm_kv8_tensor(rows, codes, exps, slots, rotate=True):
    """One tensor of a plm_kv8_write or plm_kv8_read call; it holds the tensors.  rows [tokens][heads][head_dim], codes and
    exps as plm_kv8_views gives them (any strided views), slots int64 [tokens]."""
    rt, rh, _ = _rows(rows, "rows", 3)
    (cp, ch, ct, _), (ep, eh, _, _) = _kv8_pages(codes, exps, "codes")
    tokens, heads, d = rows.shape
    pages, cheads, page_tokens, cd = codes.shape
    if cheads != heads or cd != d:
        raise ValueError("codes: expected pages [.][%d][.][%d], got %s" % (heads, d, tuple(codes.shape)))
    return (_KV8_TENSOR.pack(rows.data_ptr(), codes.data_ptr(), exps.data_ptr(), _ints(slots, 64, "slots", (tokens,)), heads, rt, rh,
                             page_tokens, pages, cp, ch, ct, ep, eh, _type(rows), 1 if rotate else 0),
            tokens, d, (rows, codes, exps, slots), rotate)


def _kv8_join(tensors):
    if not tensors:
        raise ValueError("no tensors")
    tokens, d = tensors[0][1:3]
    for t in tensors:
        if t[1] != tokens or t[2] != d:
            raise ValueError("the tensors differ in tokens or head size")
    return b"".join([t[0] for t in tensors]), tokens, d


def plm_kv8_write(tensors, positions=None, freqs=None, rotary_dim=0, layout="half", scale=1.0, stream=None):
    """Writes the tensors' rows (plm_kv8_tensor) to their slots in 8 bits, those with rotate turned by their positions
    (int32 [tokens]) first; see include/plm.h."""
    packed, tokens, d = _kv8_join(tensors)
    turned = False
    for t in tensors:
        turned = turned or t[4]
    if turned and (positions is None or freqs is None or freqs.numel() != rotary_dim // 2):
        raise ValueError("a tensor that rotates needs positions, and %d frequencies" % (rotary_dim // 2))
    if tokens == 0:
        return
    _call(_KV8_WRITE, _KV8_WRITE_CALL.pack(len(tensors), _ints(positions, 32, "positions", (tokens,)) or 0, _ints(freqs, 64, "freqs") or 0,
                                           tokens, d, rotary_dim, _LAYOUTS.get(layout, layout), scale, _stream(stream)) + packed)


def plm_kv8_read(tensors, stream=None):
    """Reads the tensors' slots (plm_kv8_tensor) into their rows; a slot out of range reads as zeros."""
    packed, tokens, d = _kv8_join(tensors)
    if tokens == 0:
        return
    _call(_KV8_READ, _KV8_READ_CALL.pack(len(tensors), tokens, d, _stream(stream)) + packed)


def plm_attn_kv8_workspace_size(batch, tokens, heads, kv_heads, head_dim, prefix_len, max_len):
    """Workspace bytes of plm_attn_kv8 (0: none needed, or invalid arguments)."""
    return load().plm_attn_kv8_workspace_size(batch, tokens, heads, kv_heads, head_dim, prefix_len, max_len)


def plm_attn_kv8(q, o, k, v, k_exps, v_exps, table, lens, tokens, prefix_len, max_len, scale, workspace, lse=None, seqs=None,
                 stream=None):
    """plm_attn_shared_prefix over 8-bit pages (plm_kv8_views, or strided views like them); see include/plm.h."""
    shape, kshape = q.shape, k.shape
    (qt, qh, _), (ot, oh, _) = _rows(q, "q", 3), _rows(o, "o", 3)
    cs, es = _kv8_pages(k, k_exps, "k")
    if o.shape != shape:
        raise ValueError("o: expected shape %s, got %s" % (tuple(shape), tuple(o.shape)))
    if (v.shape != kshape or v.stride() != cs or v.dtype != k.dtype or v_exps.shape != k_exps.shape or v_exps.stride() != es or
            v_exps.dtype != k_exps.dtype or not (v.is_cuda and v_exps.is_cuda)):
        raise ValueError("keys and values have to agree in shapes, strides and types")
    n, heads, d = shape
    pages, kv_heads, page_tokens, kd = kshape
    if kd != d:
        raise ValueError("k: expected heads of %d, got %d" % (d, kd))
    if tokens < 1 or n % tokens:
        raise ValueError("q: %d rows are no multiple of %d tokens" % (n, tokens))
    rows, width = table.shape
    batch = n // tokens
    if seqs is None and batch > rows:
        raise ValueError("table: %d rows for a batch of %d" % (rows, batch))
    if lse is not None and (_type(lse) != PLM_F32 or lse.shape != (n, heads)):
        raise ValueError("lse: expected float32 %s" % ((n, heads),))
    if batch == 0:
        return
    ws, size = _ws(workspace)
    p = _ATTN_KV8_PROBLEM.pack(q.data_ptr(), o.data_ptr(), _addr(lse) or 0, k.data_ptr(), v.data_ptr(), k_exps.data_ptr(),
                               v_exps.data_ptr(), _ints(table, 32, "table"), _ints(lens, 32, "lens", (rows,)),
                               _ints(seqs, 32, "seqs", (batch,)) or 0, batch, tokens, heads, kv_heads, d, qt, qh, ot, oh,
                               page_tokens, pages, cs[0], cs[1], cs[2], es[0], es[1], width, rows, prefix_len, max_len, scale,
                               _type(q), _type(o))
    _call(_ATTN_KV8, _ATTN_CALL.pack(ws, size, _stream(stream)) + p)


def _per_row(t, name, m):
    """Address of a float32 value a row on the device, or 0."""
    if t is None:
        return 0
    if t.shape != (m,) or _type(t) != PLM_F32:
        raise ValueError("%s: expected float32 (%d,), got %s %s" % (name, m, t.dtype, tuple(t.shape)))
    return _addr(t)


def plm_sample(logits, tokens, u=None, temperature=None, top_k=None, top_p=None, min_p=None, prob=None, stream=None):
    """tokens (int32 [m]) = the next token of each row of logits [m][n] by the row's random number u in 0 .. 1 (None:
    the largest logit) and what else is given, all [m] on the device, top_k int32, the others float32; prob gets the
    probability with which it was met (see include/plm.h)."""
    stride, code = _matrix(logits, "logits")
    m, n = logits.shape
    f = (_per_row(u, "u", m), _per_row(temperature, "temperature", m), _per_row(top_p, "top_p", m), _per_row(min_p, "min_p", m),
         _per_row(prob, "prob", m))
    k, out = _ints(top_k, 32, "top_k", (m,)) or 0, _ints(tokens, 32, "tokens", (m,))
    if m == 0:
        return
    _call(_SAMPLE, _ONE.pack(_stream(stream)) +
          _SAMPLE_PROBLEM.pack(logits.data_ptr(), f[0], f[1], k, f[2], f[3], out, f[4], m, n, stride, code))
