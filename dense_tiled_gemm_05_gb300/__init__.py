"""Python binding of the GB300 blocked-GEMM library (``include/gemm.h``).

The binding only marshals arguments: it reads shapes, strides, data pointers
and the current CUDA stream from torch tensors and calls the C ABI through
ctypes. Every step of the product runs in the library's own CUDA kernels; if
the compiled library is missing, importing the binding's entry points raises
instead of falling back to anything else.

    import dense_tiled_gemm_05_gb300 as g
    c = g.matmul(a, b)                       # a: M x K, b: K x N, CUDA tensors
    c = g.matmul(a32, b32, precision="tf32") # fp32 inputs on the tf32 tensor cores

Layouts follow the tensors' strides: a row-major view has stride (ld, 1), a
column-major view stride (1, ld) (e.g. ``b_storage.t()`` for a B stored as
[N, K]). The output is row-major.
"""
import ctypes
import importlib.util
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libgemm_gb300.so")
NATIVE_PATH = os.path.join(_PKG, "_lib", "gemm_gb300_torch.so")

# enums of include/gemm.h
F32, F16, BF16 = 0, 1, 2
PREC = {"default": 0, "tf32": 1, "exact": 2, "f16acc": 3}
ROW, COL = 0, 1
STATUS = {0: "GEMM_OK", 1: "GEMM_ERR_INVALID_ARG", 2: "GEMM_ERR_UNSUPPORTED",
          3: "GEMM_ERR_ALIGNMENT", 4: "GEMM_ERR_NO_MEMORY", 5: "GEMM_ERR_CUDA",
          6: "GEMM_ERR_TIMEOUT", 7: "GEMM_ERR_DEVICE"}
OPTIONS = {"wait_timeout_us": 0, "force_path": 1, "group_m": 2, "max_ctas": 3,
           "fault_stall_producer": 4, "force_staging": 5, "cta_pair": 6,
           "block_n": 7, "exact_chunk": 8, "stream_k": 9, "host_panel": 10, "acc_chunk": 11, "stage_k": 12,
           "tile_rows": 13, "tf32_transpose": 14}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid")  # gemm_activation_t
PATHS = {0: "none", 1: "zero_fill", 2: "tcgen05", 3: "fma", 4: "tcgen05_3xtf32",
         5: "tcgen05_f16acc"}
_DT = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_DT_NAMES = {"f32": F32, "f16": F16, "bf16": BF16}
_TORCH_OF = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}

# Every symbol include/gemm.h declares.
EXPORTS = ("gemm_create", "gemm_destroy", "gemm_run", "gemm_run_ex", "gemm_get_status",
           "gemm_strerror", "gemm_set_option", "gemm_get_launch_count", "gemm_plan",
           "gemm_version", "gemm_run_noalloc", "gemm_schedule_segments", "gemm_run_host",
           "gemm_run_strided", "gemm_plan_strided", "gemm_tune", "gemm_tune_clear",
           "gemm_softmax_rows", "gemm_set_kernel_events", "gemm_run_epilogue",
           "gemm_run_epilogue_backward", "gemm_run_gated", "gemm_run_gated_backward",
           "gemm_layer_norm", "gemm_layer_norm_backward")


class GemmError(RuntimeError):
    def __init__(self, code, what=""):
        self.code = code
        self.status = STATUS.get(code, str(code))
        super().__init__("%s%s (%s)" % (what + ": " if what else "", self.status, _strerror(code)))


class TuneResult(ctypes.Structure):
    _fields_ = [("cta_pair", ctypes.c_int32), ("block_n", ctypes.c_int32),
                ("stream_k", ctypes.c_int32), ("stage_k", ctypes.c_int32),
                ("group_m", ctypes.c_int32), ("tile_rows", ctypes.c_int32),
                ("candidates", ctypes.c_int32),
                ("best_us", ctypes.c_float), ("default_us", ctypes.c_float)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class Epilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("ld_residual", ctypes.c_int64), ("pre", ctypes.c_void_p),
                ("ld_pre", ctypes.c_int64), ("bias_dtype", ctypes.c_int32),
                ("activation", ctypes.c_int32)]


class StridedInfo(ctypes.Structure):
    _fields_ = [("a_gathered", ctypes.c_int32), ("b_gathered", ctypes.c_int32),
                ("c_mode", ctypes.c_int32), ("buffer_bytes", ctypes.c_int64)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class PlanInfo(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32),
                ("tile_k", ctypes.c_int32), ("grid_m", ctypes.c_int64), ("grid_n", ctypes.c_int64),
                ("k_iters", ctypes.c_int64), ("stages", ctypes.c_int32), ("stage_a", ctypes.c_int32),
                ("stage_b", ctypes.c_int32), ("a_mn_major", ctypes.c_int32),
                ("b_mn_major", ctypes.c_int32), ("tma_store", ctypes.c_int32),
                ("ctas", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
                ("cta_pair", ctypes.c_int32), ("split_tiles", ctypes.c_int32)]

    def as_dict(self):
        d = {name: getattr(self, name) for name, _ in self._fields_}
        d["path"] = PATHS.get(d["path"], d["path"])
        return d


_lib = None
_lib_lock = threading.Lock()


def lib():
    """The loaded C library; raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is None:
        with _lib_lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        "libgemm_gb300.so is not built; run "
                        "`python -c 'import __graft_entry__ as g; g.build()'` "
                        "(or python dense_tiled_gemm_05_gb300/build.py)")
                L = ctypes.CDLL(LIB_PATH)
                i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
                run_args = [vp, i64, i64, i64, vp, i64, vp, i64, vp, i64, i32, i32, i32]
                L.gemm_create.argtypes = [ctypes.POINTER(vp), i32]
                L.gemm_create.restype = i32
                L.gemm_destroy.argtypes = [vp]
                L.gemm_destroy.restype = None
                L.gemm_run.argtypes = run_args
                L.gemm_run.restype = i32
                L.gemm_run_ex.argtypes = run_args + [i32, i32, vp]
                L.gemm_run_ex.restype = i32
                L.gemm_run_host.argtypes = run_args + [i32, i32, vp]
                L.gemm_run_host.restype = i32
                strided = [vp, i64, i64, i64, vp, i64, i64, vp, i64, i64, vp, i64, i64, i32,
                           i32, i32]
                L.gemm_run_strided.argtypes = strided + [vp]
                L.gemm_run_strided.restype = i32
                L.gemm_plan_strided.argtypes = strided + [i32, ctypes.POINTER(PlanInfo),
                                                          ctypes.POINTER(StridedInfo)]
                L.gemm_plan_strided.restype = i32
                L.gemm_tune.argtypes = run_args + [i32, i32, vp, i32, ctypes.POINTER(TuneResult)]
                L.gemm_tune.restype = i32
                L.gemm_softmax_rows.argtypes = [vp, i64, i64, vp, i64, vp, i64, i32, i32, vp]
                L.gemm_softmax_rows.restype = i32
                L.gemm_run_epilogue.argtypes = run_args + [i32, i32, ctypes.POINTER(Epilogue), vp]
                L.gemm_run_epilogue.restype = i32
                L.gemm_run_epilogue_backward.argtypes = (
                    [vp] + [i64] * 3 + [vp, i64] * 6 + [vp] + [i32] * 7 + [vp])
                L.gemm_run_epilogue_backward.restype = i32
                L.gemm_run_gated.argtypes = [vp] + [i64] * 3 + [vp, i64] * 6 + [i32] * 4 + [vp]
                L.gemm_run_gated.restype = i32
                L.gemm_run_gated_backward.argtypes = (
                    [vp] + [i64] * 3 + [vp, i64] * 9 + [i32] * 4 + [vp])
                L.gemm_run_gated_backward.restype = i32
                L.gemm_layer_norm.argtypes = [vp, i64, i64, vp, i64, vp, vp, vp, i64, vp, vp,
                                              ctypes.c_float, i32, i32, i32, vp]
                L.gemm_layer_norm.restype = i32
                L.gemm_layer_norm_backward.argtypes = [vp, i64, i64, vp, i64, vp, i64, vp, vp, vp,
                                                       vp, i64, vp, vp, i32, i32, i32, vp]
                L.gemm_layer_norm_backward.restype = i32
                L.gemm_tune_clear.argtypes = [vp]
                L.gemm_tune_clear.restype = i32
                L.gemm_get_status.argtypes = [vp, vp]
                L.gemm_get_status.restype = i32
                L.gemm_strerror.argtypes = [i32]
                L.gemm_strerror.restype = ctypes.c_char_p
                L.gemm_set_option.argtypes = [vp, i32, i64]
                L.gemm_set_option.restype = i32
                L.gemm_get_launch_count.argtypes = [vp, ctypes.POINTER(ctypes.c_uint64)]
                L.gemm_get_launch_count.restype = i32
                L.gemm_set_kernel_events.argtypes = [vp, vp, vp]
                L.gemm_set_kernel_events.restype = i32
                L.gemm_plan.argtypes = run_args + [i32, i32, ctypes.c_int32,
                                                   ctypes.POINTER(PlanInfo)]
                L.gemm_plan.restype = i32
                L.gemm_run_noalloc.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, i32,
                                               i32, i32, i32, i32, vp, vp]
                L.gemm_run_noalloc.restype = i32
                L.gemm_schedule_segments.argtypes = [i32, i32, i32, i32, i32,
                                                     ctypes.POINTER(ctypes.c_int32), vp, i32]
                L.gemm_schedule_segments.restype = i32
                L.gemm_version.argtypes = []
                L.gemm_version.restype = ctypes.c_char_p
                _lib = L
    return _lib


def _strerror(code):
    try:
        return lib().gemm_strerror(code).decode()
    except RuntimeError:
        return "library not loaded"


def _check(code, what=""):
    if code != 0:
        raise GemmError(code, what)


def operand_layout(x):
    """(layout, ld) of a 2-D view: ROW for stride (ld, 1), COL for stride (1, ld)."""
    if x.dim() != 2:
        raise ValueError("operands must be 2-D")
    r, c = x.shape
    s0, s1 = x.stride()
    if s1 == 1 and (s0 >= max(c, 1) or r <= 1):
        return ROW, max(s0, c, 1)
    if s0 == 1 and (s1 >= max(r, 1) or c <= 1):
        return COL, max(s1, r, 1)
    raise ValueError("operand must be row- or column-major, got stride %s" % (x.stride(),))


_native_module = None


def native():
    """The compiled binding of the feed-forward operators, with the C functions it calls;
    raises if it has not been built."""
    global _native_module
    if _native_module is None:
        L = lib()
        if not os.path.exists(NATIVE_PATH):
            raise RuntimeError("gemm_gb300_torch.so is not built; run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        spec = importlib.util.spec_from_file_location("gemm_gb300_torch", NATIVE_PATH)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        m.init(*[ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in (
            "gemm_run_epilogue", "gemm_run_epilogue_backward", "gemm_run_gated",
            "gemm_run_gated_backward", "gemm_layer_norm", "gemm_layer_norm_backward")], _check)
        _native_module = m
    return _native_module


def _dtype_code(d):
    if isinstance(d, str):
        return _DT_NAMES[d]
    if d in _DT:
        return _DT[d]
    raise TypeError("unsupported dtype %s" % d)


class _Streams:
    """The stream of a call: the current one, or another that the caller names. On another, the
    call does what it would with that stream current -- its output comes from that stream's
    memory -- and the allocator learns of every tensor that two streams use."""

    def __init__(self, stream, device):
        self.call = self.current = torch.cuda.current_stream(device)
        if stream is not None and stream.cuda_stream != self.current.cuda_stream:
            self.call = (stream if isinstance(stream, torch.cuda.Stream)
                         else torch.cuda.ExternalStream(stream.cuda_stream, device))

    def empty(self, shape, dtype, device):
        if self.call is self.current:
            return torch.empty(shape, dtype=dtype, device=device)
        with torch.cuda.stream(self.call):
            return torch.empty(shape, dtype=dtype, device=device)

    def used(self, out, *operands):
        if self.call is not self.current:
            for t in (out,) + operands:
                t.record_stream(self.call)
            out.record_stream(self.current)


class Gemm:
    """A library handle bound to one CUDA device. A call's ``stream`` (default: the current one)
    runs it as if that stream were current; ordering it after the operands' work, and other
    work after it, is the caller's."""

    def __init__(self, device=None):
        if device is None:
            device = torch.cuda.current_device()
        self.device = int(device)
        h = ctypes.c_void_p()
        _check(lib().gemm_create(ctypes.byref(h), self.device), "gemm_create")
        self._h = h
        self._address = h.value

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().gemm_destroy(self._h)
            self._h = None
            self._address = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    def set_option(self, name, value):
        _check(lib().gemm_set_option(self._h, OPTIONS[name], int(value)), "gemm_set_option")

    def launch_count(self):
        n = ctypes.c_uint64()
        _check(lib().gemm_get_launch_count(self._h, ctypes.byref(n)))
        return n.value

    def set_kernel_events(self, start=None, end=None):
        """Record two torch.cuda.Event objects around the main GEMM kernel of every later
        product on this handle (after any staging copies); no arguments turn it off. The
        events must have been recorded once, so that their CUDA events exist."""
        if start is None or end is None:
            _check(lib().gemm_set_kernel_events(self._h, None, None), "gemm_set_kernel_events")
            self._kernel_events = None
            return
        self._kernel_events = (start, end)  # kept alive while the hook is set
        _check(lib().gemm_set_kernel_events(self._h, ctypes.c_void_p(start.cuda_event),
                                            ctypes.c_void_p(end.cuda_event)),
               "gemm_set_kernel_events")

    def status(self, stream=None):
        """Synchronise the stream and return the device status code (0 = OK), cleared."""
        s = torch.cuda.current_stream(self.device) if stream is None else stream
        return lib().gemm_get_status(self._h, ctypes.c_void_p(s.cuda_stream))

    def run_raw(self, M, N, K, A, lda, B, ldb, C, ldc, in_dtype, out_dtype, precision=0,
                a_layout=ROW, b_layout=COL, stream=0):
        """Direct C-ABI call with integer pointers; returns the status code."""
        return lib().gemm_run_ex(self._h, M, N, K, A, lda, B, ldb, C, ldc, in_dtype, out_dtype,
                                 precision, a_layout, b_layout, ctypes.c_void_p(stream))

    def matmul(self, a, b, out=None, out_dtype=None, precision="default", stream=None):
        """C = a @ b on the GPU; a is M x K, b is K x N, out M x N: any 2-D views (row- or
        column-major views go through gemm_run_ex, others through gemm_run_strided)."""
        if a.dtype != b.dtype:
            raise TypeError("a and b must share a dtype")
        if not (a.is_cuda and b.is_cuda):
            raise ValueError("operands must be CUDA tensors (see matmul_host for host buffers)")
        if a.dim() != 2 or b.dim() != 2:
            raise ValueError("operands must be 2-D")
        M, K = a.shape
        K2, N = b.shape
        if K != K2:
            raise ValueError("inner dimensions differ: %d vs %d" % (K, K2))
        in_dt = _dtype_code(a.dtype)
        streams = _Streams(stream, a.device)
        s = streams.call
        if out is None:
            od = _TORCH_OF[_dtype_code(out_dtype)] if out_dtype is not None else a.dtype
            out = streams.empty((M, N), od, a.device)
        if out.dim() != 2 or out.shape != (M, N):
            raise ValueError("out must be an M x N tensor")
        ptr = lambda t: ctypes.c_void_p(t.data_ptr())
        try:
            al, lda = operand_layout(a)
            bl, ldb = operand_layout(b)
            row_c = (N <= 1 or out.stride(1) == 1) and (M <= 1 or out.stride(0) >= N)
        except ValueError:
            row_c = False
        if row_c:
            ldc = max(out.stride(0) if M > 1 else N, N, 1)
            code = lib().gemm_run_ex(self._h, M, N, K, ptr(a), lda, ptr(b), ldb, ptr(out), ldc,
                                     in_dt, _dtype_code(out.dtype), PREC[precision], al, bl,
                                     ctypes.c_void_p(s.cuda_stream))
            _check(code, "gemm_run_ex")
        else:
            code = lib().gemm_run_strided(self._h, M, N, K, ptr(a), a.stride(0), a.stride(1),
                                          ptr(b), b.stride(0), b.stride(1), ptr(out),
                                          out.stride(0), out.stride(1), in_dt,
                                          _dtype_code(out.dtype), PREC[precision],
                                          ctypes.c_void_p(s.cuda_stream))
            _check(code, "gemm_run_strided")
        streams.used(out, a, b)
        return out

    def tune(self, a, b, out=None, out_dtype=None, precision="default", iters=5, stream=None):
        """Time the tile-shape configurations for this problem (row- or column-major CUDA
        views) and keep the fastest for its signature on this handle; returns the choice
        as a dict (see gemm_tune). C is written."""
        M, K = a.shape
        N = b.shape[1]
        streams = _Streams(stream, a.device)
        s = streams.call
        if out is None:
            od = _TORCH_OF[_dtype_code(out_dtype)] if out_dtype is not None else a.dtype
            out = streams.empty((M, N), od, a.device)
        al, lda = operand_layout(a)
        bl, ldb = operand_layout(b)
        r = TuneResult()
        code = lib().gemm_tune(self._h, M, N, K, ctypes.c_void_p(a.data_ptr()), lda,
                               ctypes.c_void_p(b.data_ptr()), ldb, ctypes.c_void_p(out.data_ptr()),
                               max(out.stride(0), N, 1), _dtype_code(a.dtype),
                               _dtype_code(out.dtype), PREC[precision], al, bl,
                               ctypes.c_void_p(s.cuda_stream), int(iters), ctypes.byref(r))
        _check(code, "gemm_tune")
        streams.used(out, a, b)
        return r.as_dict()

    def softmax_rows(self, x, out=None, out_dtype=None, stream=None):
        """Row softmax of a CUDA matrix with unit column stride (Lesson 4, homework 4):
        out[i] = exp(x[i] - max(x[i])) / sum(exp(x[i] - max(x[i]))). ``out=x`` runs in
        place."""
        if not x.is_cuda or x.dim() != 2:
            raise ValueError("x must be a 2-D CUDA tensor")
        M, N = x.shape
        if N > 1 and x.stride(1) != 1:
            raise ValueError("rows of x must be contiguous")
        streams = _Streams(stream, x.device)
        s = streams.call
        if out is None:
            od = _TORCH_OF[_dtype_code(out_dtype)] if out_dtype is not None else x.dtype
            out = streams.empty((M, N), od, x.device)
        if out.shape != (M, N) or (N > 1 and out.stride(1) != 1):
            raise ValueError("out must be an M x N tensor with contiguous rows")
        code = lib().gemm_softmax_rows(self._h, M, N, ctypes.c_void_p(x.data_ptr()),
                                       max(x.stride(0) if M > 1 else N, N, 1),
                                       ctypes.c_void_p(out.data_ptr()),
                                       max(out.stride(0) if M > 1 else N, N, 1),
                                       _dtype_code(x.dtype), _dtype_code(out.dtype),
                                       ctypes.c_void_p(s.cuda_stream))
        _check(code, "gemm_softmax_rows")
        streams.used(out, x)
        return out

    # ------------------------------------------------------- feed-forward operators
    #
    # Like matmul they record nothing for automatic differentiation: outputs require no
    # gradient, whatever the inputs do, and the backward methods are called by name.

    def matmul_epilogue(self, a, b, bias=None, activation=None, residual=None, out=None,
                        out_dtype=None, precision="default", save=False, stream=None):
        """act(a @ b + bias) + residual: a is M x K, b is K x N (row- or column-major views;
        a weight stored as [N, K] is passed as ``w.t()``), bias has N values, residual is
        M x N of the output's dtype (``out=residual`` updates it in place). activation: None,
        "relu", "gelu", "gelu_tanh", "silu" or "sigmoid". ``save=True`` returns (out, pre)
        with pre = a @ b + bias for :meth:`matmul_epilogue_backward` (which a program calls
        itself: no automatic differentiation, as in the other methods here)."""
        return (_native_module or native()).matmul_epilogue(
            self._address, a, b, bias, activation, residual, out, out_dtype, precision, save, stream)

    def matmul_epilogue_backward(self, grad, a, b, pre=None, activation=None,
                                 need=(True, True, True), bias_dtype=None, precision="default",
                                 stream=None):
        """Gradients of :meth:`matmul_epilogue` from grad (M x N, the output's dtype) and the
        saved pre (needed unless there is no activation): (da, db, dbias), each None where
        ``need`` says so; da and db in the layouts of a and b, dbias in ``bias_dtype``
        (default: a's). The residual's gradient is grad itself. For 16-bit operands the slopes
        are rounded to that type, with its range (f16: 65504), before the products."""
        return (_native_module or native()).matmul_epilogue_backward(
            self._address, grad, a, b, pre, activation, need, bias_dtype, precision, stream)

    def gated(self, x, w_gate, w_up, activation="silu", out=None, precision="default",
              save=False, stream=None):
        """act(x @ w_gate) * (x @ w_up), the gated half of a feed-forward block: x is M x K
        with contiguous rows, both weights K x F in one layout (stored as [F, K]: pass
        ``w.t()``). ``save=True`` returns (out, gate, up) with the two products for
        :meth:`gated_backward` (column ranges of one M x 2F buffer)."""
        return (_native_module or native()).gated(
            self._address, x, w_gate, w_up, activation, out, precision, save, stream)

    def gated_backward(self, grad, x, w_gate, w_up, gate, up, activation="silu",
                       need=(True, True, True), precision="default", stream=None):
        """Gradients of :meth:`gated` from grad (M x F) and the saved gate and up: (dx, dw_gate,
        dw_up), each None where ``need`` says so, the weights' in the weights' layout."""
        return (_native_module or native()).gated_backward(
            self._address, grad, x, w_gate, w_up, gate, up, activation, need, precision, stream)

    def layer_norm(self, x, weight=None, bias=None, eps=1e-5, out=None, out_dtype=None,
                   save=False, stream=None):
        """Layer norm of each row of a CUDA matrix with contiguous rows; weight and bias (None:
        1 and 0) share a dtype of their own. ``out=x`` runs in place. ``save=True`` returns
        (out, mean, rstd) with the rows' fp32 statistics for :meth:`layer_norm_backward`."""
        return (_native_module or native()).layer_norm(
            self._address, x, weight, bias, eps, out, out_dtype, save, stream)

    def layer_norm_backward(self, grad, x, weight, mean, rstd, need=(True, True, True),
                            param_dtype=None, stream=None):
        """Gradients of :meth:`layer_norm` from grad (the output's dtype), x, weight (or None)
        and the saved statistics: (dx, dweight, dbias), each None where ``need`` says so; the
        last two in ``param_dtype`` (default: weight's, or float32)."""
        return (_native_module or native()).layer_norm_backward(
            self._address, grad, x, weight, mean, rstd, need, param_dtype, stream)

    def tune_clear(self):
        _check(lib().gemm_tune_clear(self._h), "gemm_tune_clear")

    def matmul_host(self, a, b, out=None, out_dtype=None, precision="default", stream=None):
        """C = a @ b for HOST tensors through gemm_run_host: the library copies A and B to the
        GPU and C back, overlapping the copies of one row panel with the product of another.

        Pinned host tensors (``pin_memory=True``) give asynchronous copies; the call returns
        once the work is enqueued on the stream, so synchronise before reading ``out``.
        """
        if a.is_cuda or b.is_cuda:
            raise ValueError("matmul_host takes host tensors")
        if a.dtype != b.dtype:
            raise TypeError("a and b must share a dtype")
        M, K = a.shape
        K2, N = b.shape
        if K != K2:
            raise ValueError("inner dimensions differ: %d vs %d" % (K, K2))
        if out is None:
            od = _TORCH_OF[_dtype_code(out_dtype)] if out_dtype is not None else a.dtype
            out = torch.empty((M, N), dtype=od, pin_memory=True)
        if out.is_cuda or out.dim() != 2 or out.shape != (M, N) or (N > 1 and out.stride(1) != 1):
            raise ValueError("out must be a row-major M x N host tensor")
        al, lda = operand_layout(a)
        bl, ldb = operand_layout(b)
        s = torch.cuda.current_stream(self.device) if stream is None else stream
        code = lib().gemm_run_host(self._h, M, N, K, ctypes.c_void_p(a.data_ptr()), lda,
                                   ctypes.c_void_p(b.data_ptr()), ldb,
                                   ctypes.c_void_p(out.data_ptr()), max(out.stride(0), N, 1),
                                   _dtype_code(a.dtype), _dtype_code(out.dtype), PREC[precision],
                                   al, bl, ctypes.c_void_p(s.cuda_stream))
        _check(code, "gemm_run_host")
        return out

    def plan(self, a, b, out=None, out_dtype=None, precision="default", sm_count=None):
        """The planner's decision for these operands (host-only, nothing launched); by
        default for this handle's device's SM count."""
        if sm_count is None:
            sm_count = torch.cuda.get_device_properties(self.device).multi_processor_count
        return plan(a, b, out=out, out_dtype=out_dtype, precision=precision,
                    sm_count=sm_count, handle=self)


def plan_strided(a, b, out=None, out_dtype=None, precision="default", sm_count=148,
                 handle=None):
    """Host-only query of gemm_run_strided's decisions for these views (works without a
    GPU): (plan dict, strided-info dict)."""
    M, K = a.shape
    N = b.shape[1]
    od = _dtype_code(out_dtype) if out_dtype is not None else _dtype_code(a.dtype)
    if out is None:
        out = torch.empty((M, N), dtype=_TORCH_OF[od])
    info, sinfo = PlanInfo(), StridedInfo()
    h = handle.handle if handle is not None else None
    code = lib().gemm_plan_strided(h, M, N, K, ctypes.c_void_p(a.data_ptr()), a.stride(0),
                                   a.stride(1), ctypes.c_void_p(b.data_ptr()), b.stride(0),
                                   b.stride(1), ctypes.c_void_p(out.data_ptr()), out.stride(0),
                                   out.stride(1), _dtype_code(a.dtype), _dtype_code(out.dtype),
                                   PREC[precision], sm_count, ctypes.byref(info),
                                   ctypes.byref(sinfo))
    _check(code, "gemm_plan_strided")
    return info.as_dict(), sinfo.as_dict()


# Stand-in address of C for a plan made without an output tensor: 16-byte aligned and
# outside any process's address space, so the planner's check that C does not overlap A or
# B cannot be set off by where A and B happen to live.
_NO_C = 1 << 62


def plan(a, b, out=None, out_dtype=None, precision="default", sm_count=148, handle=None,
         a_ptr=None, b_ptr=None, c_ptr=None, ldc=None):
    """Host-only planner query (works without a GPU); returns a dict.

    Pointers default to the tensors' data pointers; pass integers to ask about
    alignments the tensors do not have.
    """
    M, K = a.shape
    N = b.shape[1]
    al, lda = operand_layout(a)
    bl, ldb = operand_layout(b)
    od = _dtype_code(out_dtype) if out_dtype is not None else (
        _dtype_code(out.dtype) if out is not None else _dtype_code(a.dtype))
    if ldc is None:
        ldc = max(out.stride(0), N, 1) if out is not None else max(N, 1)
    if c_ptr is None:
        c_ptr = out.data_ptr() if out is not None else _NO_C
    info = PlanInfo()
    code = lib().gemm_plan(handle.handle if handle is not None else None, M, N, K,
                           ctypes.c_void_p(a.data_ptr() if a_ptr is None else a_ptr), lda,
                           ctypes.c_void_p(b.data_ptr() if b_ptr is None else b_ptr), ldb,
                           ctypes.c_void_p(c_ptr), ldc, _dtype_code(a.dtype), od,
                           PREC[precision], al, bl, int(sm_count or 148), ctypes.byref(info))
    _check(code, "gemm_plan")
    return info.as_dict()


_handles = {}


def handle(device=None):
    """The per-device default handle (created on first use)."""
    dev = torch.cuda.current_device() if device is None else int(device)
    h = _handles.get(dev)
    if h is None:
        h = _handles[dev] = Gemm(dev)
    return h


def matmul(a, b, out=None, out_dtype=None, precision="default"):
    """C = a @ b with the default handle of a's device; see :meth:`Gemm.matmul`."""
    return handle(a.device.index).matmul(a, b, out=out, out_dtype=out_dtype, precision=precision)


def softmax_rows(x, out=None, out_dtype=None):
    """Row softmax with the default handle of x's device; see :meth:`Gemm.softmax_rows`."""
    return handle(x.device.index).softmax_rows(x, out=out, out_dtype=out_dtype)


def _handle_of(t):
    """The default handle of an operand's device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("operands must be tensors")
    if not t.is_cuda:
        raise ValueError("operands must be CUDA tensors")
    return handle(t.get_device())


def matmul_epilogue(a, b, **kw):
    """act(a @ b + bias) + residual; see :meth:`Gemm.matmul_epilogue`."""
    return _handle_of(a).matmul_epilogue(a, b, **kw)


def matmul_epilogue_backward(grad, a, b, **kw):
    """Gradients of :func:`matmul_epilogue`; see :meth:`Gemm.matmul_epilogue_backward`."""
    return _handle_of(a).matmul_epilogue_backward(grad, a, b, **kw)


def gated(x, w_gate, w_up, **kw):
    """act(x @ w_gate) * (x @ w_up); see :meth:`Gemm.gated`."""
    return _handle_of(x).gated(x, w_gate, w_up, **kw)


def gated_backward(grad, x, w_gate, w_up, gate, up, **kw):
    """Gradients of :func:`gated`; see :meth:`Gemm.gated_backward`."""
    return _handle_of(x).gated_backward(grad, x, w_gate, w_up, gate, up, **kw)


def layer_norm(x, weight=None, bias=None, **kw):
    """Layer norm of the rows of x; see :meth:`Gemm.layer_norm`."""
    return _handle_of(x).layer_norm(x, weight, bias, **kw)


def layer_norm_backward(grad, x, weight, mean, rstd, **kw):
    """Gradients of :func:`layer_norm`; see :meth:`Gemm.layer_norm_backward`."""
    return _handle_of(x).layer_norm_backward(grad, x, weight, mean, rstd, **kw)


def matmul_host(a, b, out=None, out_dtype=None, precision="default", device=None):
    """End-to-end product of host tensors with the default handle of ``device`` (default:
    the current device); see :meth:`Gemm.matmul_host`."""
    dev = torch.cuda.current_device() if device is None else int(device)
    return handle(dev).matmul_host(a, b, out=out, out_dtype=out_dtype, precision=precision)


class Segment(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_int32), ("kb_begin", ctypes.c_int32),
                ("kb_end", ctypes.c_int32), ("role", ctypes.c_int32),
                ("first_src", ctypes.c_int32), ("last_src", ctypes.c_int32)]


def schedule(tiles, k_blocks, slots, stream_k=True):
    """Host-only tile schedule: per worker, (whole tiles, [split pieces as tuples])."""
    out = []
    for s in range(slots):
        whole = ctypes.c_int32()
        n = lib().gemm_schedule_segments(tiles, k_blocks, slots, int(stream_k), s,
                                         ctypes.byref(whole), None, 0)
        if n < 0:
            raise ValueError("invalid schedule arguments")
        buf = (Segment * max(n, 1))()
        lib().gemm_schedule_segments(tiles, k_blocks, slots, int(stream_k), s,
                                     ctypes.byref(whole), buf, n)
        out.append((whole.value, [(x.tile, x.kb_begin, x.kb_end, x.role, x.first_src,
                                   x.last_src) for x in buf[:n]]))
    return out


def version():
    return lib().gemm_version().decode()
